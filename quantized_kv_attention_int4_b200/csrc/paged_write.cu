// New tokens into the paged cache, and cached tokens back as BF16 rows
// (include/flashloop_paged.h: fl_paged_append, fl_paged_read).
#include "paged.cuh"
#include "quant.cuh"

namespace fl {
namespace {

// ---- append -----------------------------------------------------------------------------
// A request whose blocks fill up is two items per such block and head, keys and values (half the
// registers of one item for both: 8 prompts of up to 4096 tokens, 16 heads, 71.7 -> 64.3 us with
// their read-back); the items of the first one also write the head's new tail rows: that block is
// the only one whose older rows lie in the tail, so the CTA has them in registers before it
// overwrites any.  A request that fills no block (most of a decode step) is one item per 16 heads,
// a copy of its rows.  Bound by instructions (19 a value) and the two barriers of a key item: those
// prompts' 105 MB in 35 us, 3.0 TB/s, 54.4 with the read-back.  Four CTAs an SM: 64.3 us with the
// read-back before the last steps, three 69.9, five 65.4, six 66.8, and a CTA per item 68.8.
// The division per word of eight codes with one near a half instead of per code: 63.7 for 58.6;
// each thread's own reciprocals of its channels' scales instead of one per channel: 58.6 for 55.6.
//
// 256 threads: thread t owns channels 8 (t % 16) .. + 7 of rows t / 16 + 16 i, i = 0..3
// (16-byte loads, 256-byte rows).  A value group (row, 64-channel half) is
// eight neighbouring threads: three steps of shuffles, after which each pair of threads has one
// of the four rows and computes its scale and zero for all eight.  A key group (channel) is 64 rows: four in the
// thread, two row sets in the warp, eight warps through shared memory.  Minima and maxima are
// taken on the BF16 values, exact.
constexpr int kAT = 256, kAppendCtas = 4;

struct alignas(16) AppendSmem {
  uint32_t mn[8][64], mx[8][64];  // per warp and channel pair
  uint32_t sz[kD];                // of each channel: scale and zero, -z, 1 / (15 s)
  float nz[kD], r15[kD];
  int red[kAT / 32];
  int ascend;  // entries in front of the first whose offsets descend
};

__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

__device__ __forceinline__ float rcp_approx(float s) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// One code by quant() of quant.cuh; one copy of the code, for the rare call below.
__device__ __noinline__ uint32_t quant_exact(uint16_t x, uint32_t sz) {
  const float2 f = unpack_sz(sz);
  return quant(__uint_as_float((uint32_t)x << 16), f.x, f.y);
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 a, b, c;\n"
      "mov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 a, a, b, c;\nmov.b64 {%0, %1}, a;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 a, b;\n"
      "mov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\n"
      "add.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float mul_sat(float a, float b) {
  float d;
  asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Eight codes, with the rounded division taken only near a half.  u = (x - z) r / 15, cut off to
// [0, 1], with r / 15 to 2^-22 and the product to 2^-24: 15 u is d / s to 4.8e-6 for codes up to 16
// (beyond, both clamp), and the rounded quotient is within 1e-6 of d / s, so away from a half by
// 1e-5 all of them round to the same code.  Not so rare: BF16 values and binary16 scales are
// coarse, and 7 of 10,000 normal values are exact halves.
// Cutting off is free in the product, and gives 0 for the NaN of an infinity, as quant() does.
// Rounding is an addition of 1.5 2^23, after which four codes add up to 16 bits exactly: no
// conversions, which issue at a quarter of the rate, and no shifts.  nz = -z of the channel
// pairs, r15 = r / 15; row: the values in memory, sz(e): scale and zero of value e.
template <class F>
__device__ __forceinline__ uint32_t quant_word(uint4 x, const float2* nz, const float2* r15, const uint16_t* row,
                                               F&& sz) {
  constexpr float kMagic = 12582912.f, kNear = 0.49999f;
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
  const float2 c15 = make_float2(15.f, 15.f), cm15 = make_float2(-15.f, -15.f), magic = make_float2(kMagic, kMagic),
               back = make_float2(-kMagic, -kMagic);
  float worst = 0.f;
  float2 code[4], up[4], off[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 d = add2(make_float2(bf16_lo(xs[e]), bf16_hi(xs[e])), nz[e]);
    const float2 u = make_float2(mul_sat(d.x, r15[e].x), mul_sat(d.y, r15[e].y));
    up[e] = fma2(u, c15, magic);
    code[e] = add2(up[e], back);
    off[e] = fma2(u, cm15, code[e]);
    worst = max_abs3(worst, off[e].x, off[e].y);
  }
  uint32_t half[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 c256 = make_float2(256.f, 256.f);
    const float2 two = fma2(code[2 * i + 1], c256, make_float2(up[2 * i].x, code[2 * i].y));
    half[i] = __float_as_uint(fmaf(two.y, 16.f, two.x));
  }
  uint32_t w = __byte_perm(half[0], half[1], 0x5410);
  if (worst >= kNear) {
    unsigned near = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      near |= (unsigned)(fabsf(off[e].x) >= kNear) << (2 * e) | (unsigned)(fabsf(off[e].y) >= kNear) << (2 * e + 1);
#pragma unroll 1
    for (; near; near &= near - 1) {
      const int e = __ffs(near) - 1;
      w = (w & ~(15u << (4 * e))) | quant_exact(row[e], sz(e)) << (4 * e);
    }
  }
  return w;
}

// 1 / (15 s) to 2^-22, and 0 for s = 0 (whose code is 0); binary16 scales are at least 2^-24.
__device__ __forceinline__ float rcp_scale(float s) { return s == 0.f ? 0.f : rcp_approx(s) * (1.f / 15.f); }

__global__ void __launch_bounds__(kAT, kAppendCtas) append_kernel(PagedAppendArgs a) {
  extern __shared__ int32_t prefix[];
  __shared__ AppendSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = a.p.kv_heads;
  const fl_paged_index& x = a.x;
  const bool tell = blockIdx.x == 0;
  if (tid == 0) sm.ascend = a.batch;
  grid_dep_launch();
  __syncthreads();
  grid_dep_wait();
  const int copies = (heads + 15) / 16;
  paged_scan<kAT>(a.batch, prefix, sm.red, [&](int b) {
    const int s = paged_slot(x, a.slots, b, tell);
    const int c = ld(a.start + b), r0 = ld(a.cu + b), r1 = ld(a.cu + b + 1);
    if (r1 < r0) {
      atomicMin(&sm.ascend, b);
      if (tell) paged_error(x, FL_DEV_COUNT, b);
      return 0;
    }
    if (s < 0 || c < 0 || r1 == r0) return 0;
    if (r0 < 0 || r1 > a.n_tokens) {
      if (tell) paged_error(x, FL_DEV_COUNT, b);
      return 0;
    }
    if ((int64_t)c + (r1 - r0) > (int64_t)x.max_pages * FL_PAGE) {
      if (tell) paged_error(x, FL_DEV_TOO_LONG, b);
      return 0;
    }
    const int fill = paged_full(c + r1 - r0) - paged_full(c);
    return fill ? 2 * fill * heads : copies;
  });
  // Offsets that ascend name each row once, so the items of the entries up to there are as few as
  // the host has checked; behind them sums of 32 bits may have wrapped.
  const int items = prefix[sm.ascend];
  const int chunk = tid & 15, r0 = tid >> 4;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int b = paged_find(prefix, sm.ascend, item), left = item - prefix[b];
    const int s = paged_slot(x, a.slots, b, false);
    const int c = ld(a.start + b), row0 = ld(a.cu + b), n = c + ld(a.cu + b + 1) - row0;
    const int full0 = paged_full(c), full1 = paged_full(n);
    if (full0 == full1) {
      const int h0 = 16 * left, hn = min(16, heads - h0);
      for (int y = tid; y < (n - c) * hn * 16; y += kAT) {
        const int at = y & 15, h = h0 + (y >> 4) % hn, r = (y >> 4) / hn;
        const int64_t from = (int64_t)(row0 + r) * a.token_stride + (int64_t)h * a.head_stride + 8 * at;
        const size_t to = (((size_t)s * heads + h) * FL_PAGE + (c - full0 * FL_PAGE) + r) * kD + 8 * at;
        *reinterpret_cast<uint4*>(a.p.tail_k + to) = *reinterpret_cast<const uint4*>(a.k + from);
        *reinterpret_cast<uint4*>(a.p.tail_v + to) = *reinterpret_cast<const uint4*>(a.v + from);
      }
      continue;
    }
    const bool values = left & 1;
    const int j = (left >> 1) / heads, h = (left >> 1) - j * heads, block = full0 + j;
    uint16_t* tail = (values ? a.p.tail_v : a.p.tail_k) + ((size_t)s * heads + h) * FL_PAGE * kD + 8 * chunk;
    const uint16_t* rows = (values ? a.v : a.k) + (int64_t)(row0 - c) * a.token_stride + (int64_t)h * a.head_stride + 8 * chunk;
    const int page = x.table[(int64_t)s * x.max_pages + block];
    const int64_t step = 16 * a.token_stride;
    const int t0 = block * FL_PAGE + r0;
    const uint16_t *old = tail + r0 * kD, *row_t0 = rows + t0 * a.token_stride;
    auto from = [&](int i) {
      return t0 + 16 * i < c ? old + 16 * i * kD : row_t0 + i * step;
    };
    uint4 x4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x4[i] = *reinterpret_cast<const uint4*>(from(i));
    const bool paged = page >= 0 && page < x.pages;
    if (!paged && !values && tid == 0) paged_error(x, FL_DEV_PAGE_RANGE, b);  // once a block and head
    uint8_t* rec = a.p.rec + ((size_t)(paged ? page : 0) * heads + h) * kRec;
    auto code_at = [&](int i) {
      return reinterpret_cast<uint32_t*>(rec + (r0 + 16 * i) * 128 + (values ? 64 : 0) + 4 * chunk);
    };
    if (paged && !values) {
      // keys: this thread's four rows, the warp's other row set, then the eight warps
      uint32_t mn[4], mx[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t p0 = (&x4[0].x)[e], p1 = (&x4[1].x)[e], p2 = (&x4[2].x)[e], p3 = (&x4[3].x)[e];
        mn[e] = bmin2(bmin2(p0, p1), bmin2(p2, p3));
        mx[e] = bmax2(bmax2(p0, p1), bmax2(p2, p3));
        mn[e] = bmin2(mn[e], __shfl_xor_sync(kFull, mn[e], 16));
        mx[e] = bmax2(mx[e], __shfl_xor_sync(kFull, mx[e], 16));
      }
      if (lane < 16) {
        *reinterpret_cast<uint4*>(&sm.mn[warp][4 * chunk]) = make_uint4(mn[0], mn[1], mn[2], mn[3]);
        *reinterpret_cast<uint4*>(&sm.mx[warp][4 * chunk]) = make_uint4(mx[0], mx[1], mx[2], mx[3]);
      }
      __syncthreads();
      if (tid < kD) {
        const int p = tid >> 1, sh = (tid & 1) * 16;
        uint32_t lo = sm.mn[0][p], hi = sm.mx[0][p];
#pragma unroll
        for (int q = 1; q < 8; ++q) {
          lo = bmin2(lo, sm.mn[q][p]);
          hi = bmax2(hi, sm.mx[q][p]);
        }
        __half hs, hz;
        group_sz(__uint_as_float((lo >> sh) << 16), __uint_as_float((hi >> sh) << 16), hs, hz);
        sm.sz[tid] = pack_sz(hs, hz);
        sm.nz[tid] = -__half2float(hz);
        sm.r15[tid] = rcp_scale(__half2float(hs));
        reinterpret_cast<uint32_t*>(rec + kRecKsz)[tid] = pack_sz(hs, hz);
      }
      __syncthreads();
      {
        float2 nz[4], r15[4];
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float4 z4 = *reinterpret_cast<const float4*>(&sm.nz[8 * chunk + 2 * e]);
          const float4 r4 = *reinterpret_cast<const float4*>(&sm.r15[8 * chunk + 2 * e]);
          nz[e] = make_float2(z4.x, z4.y), nz[e + 1] = make_float2(z4.z, z4.w);
          r15[e] = make_float2(r4.x, r4.y), r15[e + 1] = make_float2(r4.z, r4.w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *code_at(i) = quant_word(x4[i], nz, r15, from(i), [&](int e) { return sm.sz[8 * chunk + e]; });
      }
    } else if (paged) {
      // values: each step of the reduction halves the rows a thread still answers for
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = bmin2(bmin2(x4[i].x, x4[i].y), bmin2(x4[i].z, x4[i].w));
        hi[i] = bmax2(bmax2(x4[i].x, x4[i].y), bmax2(x4[i].z, x4[i].w));
      }
#pragma unroll
      for (int o = 4; o; o >>= 1) {
        const bool up = lane & o;
        const int rows = o == 4 ? 2 : 1;
#pragma unroll
        for (int i = 0; i < rows; ++i) {
          const int other = i + (o > 1 ? rows : 0);
          const uint32_t l = __shfl_xor_sync(kFull, up ? lo[i] : lo[other], o);
          const uint32_t h2 = __shfl_xor_sync(kFull, up ? hi[i] : hi[other], o);
          lo[i] = bmin2(up ? lo[other] : lo[i], l);
          hi[i] = bmax2(up ? hi[other] : hi[i], h2);
        }
      }
      uint32_t mine;
      {
        __half hs, hz;
        group_sz(fminf(bf16_lo(lo[0]), bf16_hi(lo[0])), fmaxf(bf16_lo(hi[0]), bf16_hi(hi[0])), hs, hz);
        mine = pack_sz(hs, hz);
        const int row = r0 + 16 * ((lane >> 1) & 3);
        if ((lane & 1) == 0) reinterpret_cast<uint32_t*>(rec + kRecVsz)[2 * row + (chunk >> 3)] = mine;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t both = __shfl_sync(kFull, mine, (lane & 24) + 2 * i);
        const float2 f = unpack_sz(both);
        const float rv = rcp_scale(f.x);
        const float2 z2 = make_float2(-f.y, -f.y), r2 = make_float2(rv, rv);
        const float2 nz[4] = {z2, z2, z2, z2}, r15[4] = {r2, r2, r2, r2};
        *code_at(i) = quant_word(x4[i], nz, r15, from(i), [&](int) { return both; });
      }
    }
    if (j == 0) {
      __syncthreads();  // every old tail row is in registers
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = full1 * FL_PAGE + r0 + 16 * i;
        if (t >= c && t < n)
          *reinterpret_cast<uint4*>(tail + (r0 + 16 * i) * kD) = *reinterpret_cast<const uint4*>(rows + t * a.token_stride);
      }
    }
  }
}

// ---- read -------------------------------------------------------------------------------
// One warp takes 8 consecutive rows of one head: lane l owns channels 8 (l % 16) .. + 7 of
// rows l / 16, l / 16 + 2, ....  Rows of one page in order, the usual case, are read all at once;
// otherwise one after the other, the key scales staying in registers while the page does not
// change.  Bound by memory at length (6 requests of up to 32768 tokens, 8 heads: 504 MB in 86 us,
// 5.9 TB/s), by one trip to it when short.  16 rows a warp, in two goes of loads: 13.6 us for
// 4096 tokens of 16 heads instead of 10.8.  Eight warps a CTA 93 us, four 90, 88 with nine of
// these an SM (56 registers; ten 91), 86 with nibbles taken by byte; packed arithmetic 87.
constexpr int kReadRows = 8, kReadWarps = 4, kReadCtas = 9;

__device__ __forceinline__ uint32_t bf2(float a, float b) {
  __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&r);
}
// Byte e of x, below 2^4, as an exact float: under the exponent of 2^23 it is 2^23 + x
template <int e>
__device__ __forceinline__ float low_byte(uint32_t x) {
  return __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7550 + e)) - 8388608.f;
}

__global__ void __launch_bounds__(kReadWarps * 32, kReadCtas) read_kernel(PagedReadArgs a) {
  const int lane = threadIdx.x & 31;
  const int heads = a.p.kv_heads;
  const int64_t job = (int64_t)blockIdx.x * kReadWarps + (threadIdx.x >> 5);
  const int64_t run = job / heads;
  const int h = (int)(job % heads), t0 = (int)(run * kReadRows);
  grid_dep_launch();
  grid_dep_wait();
  if (run * kReadRows >= a.n_tokens) return;
  const int cl = lane & 15, half = lane >> 4;
  const int mine = lane < kReadRows && t0 + lane < a.n_tokens ? ld(a.place + t0 + lane) : -1;
  const int page_end = a.x.pages, all_end = a.x.pages + a.x.slots;
  const int64_t out = (int64_t)t0 * a.token_stride + (int64_t)h * a.head_stride + 8 * cl;
  float2 ksz[8];
  auto key_scales = [&](const uint8_t* rec) {
    const uint4 s0 = ld_u4(rec + kRecKsz + 32 * cl), s1 = ld_u4(rec + kRecKsz + 32 * cl + 16);
    const uint32_t w[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) ksz[e] = unpack_sz(w[e]);
  };
  auto put = [&](int r, uint32_t kw, uint32_t vw, uint32_t vz) {
    const float2 vsz = unpack_sz(vz);
    uint4 ko, vo;
    const uint32_t k0 = kw & 0x0f0f0f0fu, k1 = kw >> 4 & 0x0f0f0f0fu, v0 = vw & 0x0f0f0f0fu, v1 = vw >> 4 & 0x0f0f0f0fu;
    ko.x = bf2(fmaf(low_byte<0>(k0), ksz[0].x, ksz[0].y), fmaf(low_byte<0>(k1), ksz[1].x, ksz[1].y));
    ko.y = bf2(fmaf(low_byte<1>(k0), ksz[2].x, ksz[2].y), fmaf(low_byte<1>(k1), ksz[3].x, ksz[3].y));
    ko.z = bf2(fmaf(low_byte<2>(k0), ksz[4].x, ksz[4].y), fmaf(low_byte<2>(k1), ksz[5].x, ksz[5].y));
    ko.w = bf2(fmaf(low_byte<3>(k0), ksz[6].x, ksz[6].y), fmaf(low_byte<3>(k1), ksz[7].x, ksz[7].y));
    vo.x = bf2(fmaf(low_byte<0>(v0), vsz.x, vsz.y), fmaf(low_byte<0>(v1), vsz.x, vsz.y));
    vo.y = bf2(fmaf(low_byte<1>(v0), vsz.x, vsz.y), fmaf(low_byte<1>(v1), vsz.x, vsz.y));
    vo.z = bf2(fmaf(low_byte<2>(v0), vsz.x, vsz.y), fmaf(low_byte<2>(v1), vsz.x, vsz.y));
    vo.w = bf2(fmaf(low_byte<3>(v0), vsz.x, vsz.y), fmaf(low_byte<3>(v1), vsz.x, vsz.y));
    __stcs(reinterpret_cast<uint4*>(a.k + out + r * a.token_stride), ko);
    __stcs(reinterpret_cast<uint4*>(a.v + out + r * a.token_stride), vo);
  };
  const int at0 = __shfl_sync(kFull, mine, 0), page0 = at0 >> 6;
  if (at0 >= 0 && page0 < page_end && (at0 & 63) <= FL_PAGE - kReadRows &&
      __all_sync(kFull, lane >= kReadRows || mine == at0 + lane)) {
    const uint8_t* rec = a.p.rec + ((size_t)page0 * heads + h) * kRec;
    const int row0 = (at0 & 63) + half;
    key_scales(rec);
    uint32_t kw[kReadRows / 2], vw[kReadRows / 2], vz[kReadRows / 2];
#pragma unroll
    for (int i = 0; i < kReadRows / 2; ++i) {
      const uint32_t* row = reinterpret_cast<const uint32_t*>(rec + (row0 + 2 * i) * 128);
      kw[i] = ld(row + cl);
      vw[i] = ld(row + 16 + cl);
      vz[i] = ld(reinterpret_cast<const uint32_t*>(rec + kRecVsz) + 2 * (row0 + 2 * i) + (cl >> 3));
    }
#pragma unroll
    for (int i = 0; i < kReadRows / 2; ++i) put(2 * i + half, kw[i], vw[i], vz[i]);
    return;
  }
  int cur = -1;
#pragma unroll 1
  for (int i = 0; i < kReadRows / 2; ++i) {
    const int r = 2 * i + half;
    const int at = __shfl_sync(kFull, mine, r);
    const int page = at >> 6, row = at & 63;
    if (at < 0 || page >= all_end) {
      if (h == 0 && cl == 0 && (at < -1 || page >= all_end)) paged_error(a.x, FL_DEV_PAGE_RANGE, t0 + r);
      continue;
    }
    if (page < page_end) {
      const uint8_t* rec = a.p.rec + ((size_t)page * heads + h) * kRec;
      const uint32_t* words = reinterpret_cast<const uint32_t*>(rec + row * 128);
      const uint32_t kw = ld(words + cl), vw = ld(words + 16 + cl);
      const uint32_t vz = ld(reinterpret_cast<const uint32_t*>(rec + kRecVsz) + 2 * row + (cl >> 3));
      if (page != cur) key_scales(rec);
      cur = page;
      put(r, kw, vw, vz);
    } else {
      const size_t off = (((size_t)(page - page_end) * heads + h) * FL_PAGE + row) * kD + 8 * cl;
      __stcs(reinterpret_cast<uint4*>(a.k + out + r * a.token_stride), ld_u4(a.p.tail_k + off));
      __stcs(reinterpret_cast<uint4*>(a.v + out + r * a.token_stride), ld_u4(a.p.tail_v + off));
    }
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
  if (a.batch == 0 || a.n_tokens == 0) return cudaSuccess;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // at most two items per entry, two more per 64 tokens
  const int64_t items = 2 * ((int64_t)a.batch + a.n_tokens / FL_PAGE) * a.p.kv_heads;
  const int grid = (int)(items < kAppendCtas * sms ? items : kAppendCtas * sms);
  return launch_pdl(append_kernel, dim3(grid), dim3(kAT), (size_t)(a.batch + 1) * 4, s, a);
}

cudaError_t launch_paged_read(const PagedReadArgs& a, cudaStream_t s) {
  if (a.n_tokens == 0) return cudaSuccess;
  const int64_t jobs = ((int64_t)a.n_tokens + kReadRows - 1) / kReadRows * a.p.kv_heads;
  const int64_t grid = (jobs + kReadWarps - 1) / kReadWarps;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(read_kernel, dim3((unsigned)grid), dim3(kReadWarps * 32), 0, s, a);
}

}  // namespace fl
