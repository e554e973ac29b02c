// Attention of one token per request over the paged cache (include/flashloop_paged.h:
// fl_paged_attn_decode), over every block or over selected ones.
//
// One CTA per (entry, key-value head, eight query heads); a warp takes one token at a time,
// lane l its channels 4l .. 4l + 3, with a running maximum and sum per query head; the warps'
// states are joined in shared memory at the end.
#include "paged.cuh"

namespace fl {
namespace {

constexpr int kAW = 8;

__global__ void __launch_bounds__(kAW * 32) paged_attn_kernel(PagedAttnArgs a) {
  __shared__ float s_o[kAW][8][kD];
  __shared__ float s_m[kAW][8], s_l[kAW][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunks = (a.group + 7) / 8, heads = a.p.kv_heads;
  const int b = blockIdx.y, h = blockIdx.x / chunks, g0 = blockIdx.x % chunks * 8;
  const int gn = min(8, a.group - g0);
  const fl_paged_index& x = a.x;
  const bool tell = blockIdx.x == 0 && threadIdx.x == 0;
  const int s = paged_slot(x, a.slots, b, tell);
  if (s < 0) return;
  const int n = paged_length(x, s, b, tell), full = paged_full(n);
  const int nb = a.sel ? a.keep : full;
  float q[8][4], acc[8][4], m[8], l[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
    const uint16_t* src = a.q + (int64_t)b * a.q_batch_stride + (int64_t)(h * a.group + g0 + (g < gn ? g : 0)) * a.q_head_stride;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      q[g][c] = __uint_as_float((uint32_t)src[4 * lane + c] << 16);
      acc[g][c] = 0.f;
    }
  }
  auto token = [&](const float* k, const float* v) {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      if (g < gn) {
        const float d = fmaf(q[g][0], k[0], fmaf(q[g][1], k[1], fmaf(q[g][2], k[2], q[g][3] * k[3])));
        const float sc = warp_sum(d) * kQScale;
        const float mn = fmaxf(m[g], sc), alpha = m[g] == -INFINITY ? 0.f : ex2(m[g] - mn), p = ex2(sc - mn);
        m[g] = mn;
        l[g] = fmaf(l[g], alpha, p);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[g][c] = fmaf(acc[g][c], alpha, p * v[c]);
      }
    }
  };
  for (int i = warp; i < nb * FL_PAGE; i += kAW) {
    int block = i >> 6;
    if (a.sel) {
      const int e = block;
      block = a.sel[((size_t)b * heads + h) * a.keep + e];
      if (block < 0 || block >= full) {
        if (block != -1 && lane == 0 && (i & 63) == 0) paged_error(x, FL_DEV_SEL_BLOCK, b);
        continue;
      }
    }
    const int page = x.table[(int64_t)s * x.max_pages + block], row = i & 63;
    if (page < 0 || page >= x.pages) {
      if (lane == 0 && row == 0) paged_error(x, FL_DEV_PAGE_RANGE, b);
      continue;
    }
    const uint8_t* rec = a.p.rec + ((size_t)page * heads + h) * kRec;
    const uint32_t kc = *reinterpret_cast<const uint16_t*>(rec + row * 128 + 2 * lane);
    const uint32_t vc = *reinterpret_cast<const uint16_t*>(rec + row * 128 + 64 + 2 * lane);
    const uint4 ks = ldg_u4(rec + kRecKsz + 16 * lane);
    const float2 vs = unpack_sz(ldg_u32(rec + kRecVsz + 8 * row + 4 * (lane >> 4)));
    float k[4], v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 f = unpack_sz((&ks.x)[c]);
      k[c] = fmaf((float)((kc >> (4 * c)) & 15u), f.x, f.y);
      v[c] = fmaf((float)((vc >> (4 * c)) & 15u), vs.x, vs.y);
    }
    token(k, v);
  }
  for (int row = warp; row < n - full * FL_PAGE; row += kAW) {
    const size_t off = (((size_t)s * heads + h) * FL_PAGE + row) * kD + 4 * lane;
    const uint2 kw = *reinterpret_cast<const uint2*>(a.p.tail_k + off), vw = *reinterpret_cast<const uint2*>(a.p.tail_v + off);
    const float k[4] = {bf16_lo(kw.x), bf16_hi(kw.x), bf16_lo(kw.y), bf16_hi(kw.y)};
    const float v[4] = {bf16_lo(vw.x), bf16_hi(vw.x), bf16_lo(vw.y), bf16_hi(vw.y)};
    token(k, v);
  }
#pragma unroll
  for (int g = 0; g < 8; ++g) {
#pragma unroll
    for (int c = 0; c < 4; ++c) s_o[warp][g][4 * lane + c] = acc[g][c];
    if (lane == 0) {
      s_m[warp][g] = m[g];
      s_l[warp][g] = l[g];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < gn * kD; i += kAW * 32) {
    const int g = i / kD, c = i % kD;
    float top = -INFINITY, sum = 0.f, o = 0.f;
    bool nan = false;
    for (int w = 0; w < kAW; ++w) {
      top = fmaxf(top, s_m[w][g]);
      nan |= s_l[w][g] != s_l[w][g];
    }
    for (int w = 0; w < kAW; ++w) {
      const float f = s_m[w][g] == -INFINITY && !nan ? 0.f : ex2(s_m[w][g] - top);
      sum = fmaf(f, s_l[w][g], sum);
      o = fmaf(f, s_o[w][g][c], o);
    }
    const int head = h * a.group + g0 + g;
    a.o[(int64_t)b * a.o_batch_stride + (int64_t)head * a.o_head_stride + c] = n > 0 ? o / sum : 0.f;
    if (c == 0 && a.lse) a.lse[(size_t)b * a.q_heads + head] = n > 0 ? top + log2f(sum) : -INFINITY;
  }
}

}  // namespace

uint64_t paged_attn_bytes(const fl_paged_pool&, int) { return 0; }

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s) {
  if (a.batch == 0) return cudaSuccess;
  paged_attn_kernel<<<dim3(a.p.kv_heads * ((a.group + 7) / 8), a.batch), kAW * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace fl
