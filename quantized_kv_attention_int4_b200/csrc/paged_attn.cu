// Attention of one token per request over the paged cache (include/flashloop_paged.h:
// fl_paged_attn_decode), over every block or over selected ones.
//
// Work.  A segment is one (entry, key-value head, up to 8 query heads of its group); its units
// are its blocks (one 9216-byte record each) and its tail in quarters of 16 BF16 rows (8192
// bytes), so a unit is about the same bytes whatever it is.  The units of all segments stand
// in one line; each CTA takes an equal stretch of it and each warp an equal part of that, so
// a batch of any mix of lengths keeps every SM equally busy and no length ever goes to the
// host.  A segment that lies inside a warp's part is finished by the warp; the states (max,
// sum, output) of one that several warps share are joined in shared memory, and of one that
// several CTAs share by the last of them to arrive, always in the same order.
//
// Inside a warp.  Lane 0 brings the next unit with one TMA copy (128-byte swizzle) into one
// of the warp's two or three stages while the warp computes on another: no warp waits for
// another before the end.  Matrix products are warp-wide m16n8k16 with tokens (keys) or channels
// (values) in the 16 rows and the query heads in the 8 columns: with 1 to 8 heads there is
// nothing for a 64-row tcgen05 tile, whose operands would also have to be widened to 16 bits
// in shared memory first.
//
//   q.k = sum_c (q_c s_c) (n_c - 8) + sum_c q_c (z_c + 8 s_c) for nibbles n.  A nibble under
//   the exponent of 1024 is the binary16 number 1024 + n (1024 + 16 n at bits 4..7), so one
//   logic and one packed fp16 operation turn two codes into two operands n - 8, exactly.  q_c
//   has 8 significant bits and s_c 11, so q_c s_c is two binary16 parts exactly: hi = fl(q s),
//   lo = fma(q, s, -hi); they fill columns 2j and 2j + 1 of query head j.  A power of two on q,
//   changed when a record's scales need it, keeps both in range.  The second sum is one more product
//   whose rows are all z, and then all 8.
//   o_c = sum_t (p_t s_t) (n_tc - 8) + sum_t p_t (z_t + 8 s_t) per 64-channel half.  p s goes
//   in two binary16 parts as well (2^-22 relative), the second sum in fp32.
//   The matrix unit's fp32 sums are cut off, not rounded: codes taken from the middle of
//   their range keep partial sums small (with 0..15, whose products and zero points cancel,
//   outputs over 8000 tokens were off by 1.7e-4), and a block's sums are added to the running
//   ones in ordinary fp32.
//   Weights are relative to a number that is raised only when p s would leave binary16's range,
//   and then by 8 (base 2) more than needed: the accumulators are hardly ever rescaled.
//   Tail rows are BF16: q.k exactly so, p in three BF16 parts (2^-24).
//
// Measured (device time; floor at the card's measured 6.56 TB/s): 16 requests of 32768, 8 x 4
// heads 131 us (607 MB, 4.6 TB/s; floor 93), 64 of up to 8191, 16 heads 42.6 us (137 MB; 21), one of
// 256 7.7 us.  Without the blocks' arithmetic, all else as it is, the first two take 100 and 39 us:
// the long call is bound by its instructions (1,240 a block and warp, 59 % of the issue slots over
// a launch), the mixed one by its copies and, as short ones are, by the trips to memory that wait for
// one another, lengths, table, record, join.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "paged.cuh"

namespace fl {
namespace {

constexpr int kMaxCtas = 160;
// Units a CTA should have.  With 1 x 32768, 16 heads, 52 blocks kept (the whole step): 4, 6, 8
// 23.0 us, 12 24.3, 24 28.3.
constexpr int kMinUnits = 8;
constexpr int kWarpScan = 128;     // entries up to which every warp scans the lengths by itself
constexpr int kPart = 132;         // floats of a head's state: o[128], max, sum, -, -
constexpr int kTailUnit = 16;      // tail rows of a unit
constexpr int kTailBytes = 2 * kTailUnit * kD * 2;

// Query heads of a segment: 4 kTiles.  Warps and stages: what registers (168 a thread for three
// warps of a quarter of an SM, 255 for two) and shared memory allow.
template <int kTiles>
struct Shape {
  static constexpr int kHeads = 4 * kTiles;
  static constexpr int kWarps = kTiles == 1 ? 12 : 8;
  static constexpr int kDepth = kTiles == 1 ? 2 : 3;  // stages of a warp
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = kWarps * kDepth * kRec;
  static constexpr int kSmem = 1024 + kStages;
};

// ---- instructions ---------------------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = a b
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_rows(void* dst, const CUtensorMap* map, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(0), "r"(row), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ uint4 lds128(unsigned addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(unsigned addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ __half2 h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t u2(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
// (a, b) rounded to a pair, a in the low half
__device__ __forceinline__ uint32_t pack_f16(float a, float b) { return u2(__floats2half2_rn(a, b)); }
__device__ __forceinline__ uint32_t pack_b16(float a, float b) {
  __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&r);
}
// x >= 0 in two binary16 parts, the first (its 11 leading bits, cut off) in the low half.  The
// second is rounded, 2^-22 of x at most; below 2^-14 both lose bits under 2^-24.
__device__ __forceinline__ uint32_t split_f16(float x) {
  const float hi = __uint_as_float(__float_as_uint(x) & 0xffffe000u);
  return pack_f16(hi, x - hi);
}

// ---- where a warp stands in the line of units --------------------------------------------
struct Cursor {
  int b, h, ch, u;  // entry, key-value head, which heads of its group, unit of the segment
  int units, np;    // units of a segment; the first np of them are blocks
  int n, slot;
};

// Where a segment stands: its stretch of the line, its entry and heads.
struct Segment {
  int begin, end, b, h, ch;
};

// kOne: a group's query heads make one segment (chunks = 1).
template <int kHeads, bool kSel, bool kOne>
struct Line {
  const PagedAttnArgs& a;

  __device__ __forceinline__ int chunks() const { return kOne ? 1 : (a.group + kHeads - 1) / kHeads; }

  __device__ __forceinline__ int blocks_of(int n) const {
    const int full = paged_full(n);
    return kSel ? min(full, a.keep) : full;
  }
  // Units of a segment of n tokens; one of no tokens has one unit, empty.
  __device__ __forceinline__ int units_of(int n) const {
    return n == 0 ? 1 : blocks_of(n) + (n - FL_PAGE * paged_full(n) + kTailUnit - 1) / kTailUnit;
  }
  __device__ __forceinline__ void place(Cursor& c, int n) const {
    c.n = n;
    c.np = blocks_of(n);
    c.units = units_of(n);
  }
  // The next unit; the entry behind the last one is a.batch.
  __device__ __forceinline__ void next(Cursor& c) const {
    if (++c.u < c.units) return;
    c.u = 0;
    if (!kOne) {
      if (++c.ch < chunks()) return;
      c.ch = 0;
    }
    if (++c.h < a.p.kv_heads) return;
    c.h = 0;
#pragma unroll 1
    while (++c.b < a.batch) {
      c.slot = paged_slot(a.x, a.slots, c.b, false);
      if (c.slot < 0) continue;
      place(c, paged_length(a.x, c.slot, c.b, false));
      return;
    }
  }
  // The first query head, and how many
  __device__ __forceinline__ int head(int h, int ch) const { return h * a.group + (kOne ? 0 : ch * kHeads); }
  __device__ __forceinline__ int live(int ch) const { return kOne ? a.group : min(kHeads, a.group - ch * kHeads); }
};

// Errors of a CTA, told at its end: the first one's code and entry, and how many.  In shared
// memory: they are rare, and registers are not.
struct Errors {
  int first, detail, count;

  __device__ __forceinline__ void add(int code, int b) {
    if (atomicAdd(&count, 1) == 0) {
      first = code;
      detail = b;
    }
  }
  __device__ __forceinline__ void tell(const fl_paged_index& x) const {
    if (count == 0 || !x.status) return;
    record_error(x.status, first, detail);
    if (count > 1) atomicAdd(&x.status[2], count - 1);
  }
};

// The state of a segment's query heads in one warp.  Lane (i = lane / 4, j = lane % 4): its
// accumulators' rows are channels, columns 2j, 2j + 1 the two parts of head j of each tile.
template <int kTiles>
struct State {
  float acc[8][kTiles][4];  // [2 q + f]: rows i: channel 32 q + 4 i + 2 f, rows i + 8: the next
  // weights are p = 2^(score - m), m one number for all lanes of a head; this lane's sums
  float m[kTiles], l[kTiles], z0[kTiles], z1[kTiles];

  // m, or 0 before the first score above -inf: those of -inf then weigh 0, not NaN
  __device__ __forceinline__ float base(int t) const { return m[t] == -INFINITY ? 0.f : m[t]; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[k][t][c] = 0.f;
      m[t] = -INFINITY;
      l[t] = z0[t] = z1[t] = 0.f;
    }
  }
  // Raise m so that no weight of a unit whose scores reach top[t] (this lane's, of its head)
  // passes 2^most; then the largest is 2^(most - 8), so that m rarely moves again.
  __device__ __forceinline__ void raise(const float (&top)[kTiles], float most) {
    bool over = false;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) over |= top[t] > m[t] + most;
    if (!__any_sync(kFull, over)) return;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      float x = top[t];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
      const float mn = fmaxf(m[t], x - (most - 8.f)), f = mn == m[t] ? 1.f : ex2(m[t] - mn);
      m[t] = mn;
      l[t] *= f;
      z0[t] *= f;
      z1[t] *= f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[k][t][c] *= f;
    }
  }
};

// (x & mask) | magic in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t magic) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(mask), "r"(magic));
  return y;
}
// Nibbles 0 and 4 of x (kOdd: 1 and 5) less 8, as a pair of binary16 numbers.
template <bool kOdd>
__device__ __forceinline__ uint32_t centred(uint32_t x) {
  if constexpr (kOdd)
    return u2(__hfma2(h2(and_or(x, 0x00f000f0u, 0x64006400u)), h2(0x2c002c00u), h2(0xd480d480u)));  // / 16 - 72
  else
    return u2(__hadd2(h2(and_or(x, 0x000f000fu, 0x64006400u)), h2(0xe408e408u)));  // - 1032
}

// The queries of a segment: lane (i, j) holds, for column i of each tile (head i / 2, part i
// % 2), channels 32 q + 8 j + {0, 4}, {1, 5}, {2, 6}, {3, 7} times a power of two: the largest in
// [2^shift, 2^(shift + 1)).
template <int kTiles>
struct Query {
  uint32_t w[kTiles][16];  // [4 q + pair]
  float scale[kTiles];     // of head j (not i / 2): scores in base 2 = scaled dot times this
  uint32_t part;           // all ones in the lanes of part 1
  int shift;
  uint4 raw[kTiles][4];    // as read

  // Start the loads; prepare() waits for them.
  __device__ __forceinline__ void fetch(const PagedAttnArgs& a, int b, int head0, int live) {
    const int lane = threadIdx.x & 31, i = lane >> 2, j = lane & 3;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int g = 4 * t + (i >> 1);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        raw[t][q] = g < live ? ld_u4(a.q + (int64_t)b * a.q_batch_stride + (int64_t)(head0 + g) * a.q_head_stride + 32 * q + 8 * j)
                             : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void prepare() {
    const int lane = threadIdx.x & 31, i = lane >> 2, j = lane & 3;
    part = i & 1 ? 0xffffffffu : 0u;
    shift = 5;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const uint4(&x)[4] = raw[t];
      uint32_t top = 0;  // largest magnitude's bits, in the high half
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t v = (&x[q].x)[c];
          top = max(top, max((v << 16) & 0x7fffffffu, v & 0x7fff0000u));
        }
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      // up = 2^(5 - floor(log2 top)), capped at 2^126; its reciprocal is exact
      const int up = top == 0 ? 0 : min(5 - ((int)(top >> 23) - 127), 126);
      const float f = pow2i(up), back = up > 120 ? pow2i(-60) * pow2i(60 - up) : pow2i(-up);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[8];
        v[0] = bf16_lo(x[q].x) * f, v[1] = bf16_hi(x[q].x) * f, v[2] = bf16_lo(x[q].y) * f, v[3] = bf16_hi(x[q].y) * f;
        v[4] = bf16_lo(x[q].z) * f, v[5] = bf16_hi(x[q].z) * f, v[6] = bf16_lo(x[q].w) * f, v[7] = bf16_hi(x[q].w) * f;
#pragma unroll
        for (int c = 0; c < 4; ++c) w[t][4 * q + c] = pack_f16(v[c], v[c + 4]);
      }
      scale[t] = __shfl_sync(kFull, back, 8 * j) * kQScale;
    }
  }
  // Fit the shift to a record whose largest scale has exponent field ek (below 2^(ek - 14)):
  // products q s stay below 2^15, and where they can above 2^3, far from binary16's last bit
  // 2^-24.  Rarely changes: records' scales are much alike.  Channels are held to 2^-25 of this
  // common range, so what is far below the head's largest is worth less: at 2^-17 of it against keys
  // 2^11 times the other channels' outputs are off by 1.2e-6, at 2^-20 and 2^14 by 1.2e-4.
  __device__ __forceinline__ void fit(int ek) {
    if (shift + ek <= 28 && (shift + ek >= 18 || shift == 14)) return;
    const int by = min(14, 25 - ek) - shift, a = by / 2, b = by - a;
    shift += by;
    const uint32_t fa = (uint32_t)(15 + a) * 0x04000400u, fb = (uint32_t)(15 + b) * 0x04000400u;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      scale[t] *= pow2i(-by);
#pragma unroll
      for (int k = 0; k < 16; ++k) w[t][k] = u2(__hmul2(__hmul2(h2(w[t][k]), h2(fa)), h2(fb)));
    }
  }
};

// One record in shared memory (swizzled rows of 128 bytes).
template <int kTiles>
__device__ __forceinline__ void block_unit(unsigned st, Query<kTiles>& qr, State<kTiles>& s) {
  const int lane = threadIdx.x & 31, i = lane >> 2, j = lane & 3;
  // largest key and value scales: 4 words a lane, scales in the low halves
  const uint4 kw = lds128(st + (68 + (lane >> 3)) * 128 + (((lane & 7) ^ (4 + (lane >> 3))) << 4));
  const uint4 vw = lds128(st + (64 + (lane >> 3)) * 128 + (((lane & 7) ^ (lane >> 3)) << 4));
  const uint32_t ktop = __reduce_max_sync(kFull, __vmaxu2(__vmaxu2(kw.x, kw.y), __vmaxu2(kw.z, kw.w)) << 16);
  const uint32_t vtop = __reduce_max_sync(kFull, __vmaxu2(__vmaxu2(vw.x, vw.y), __vmaxu2(vw.z, vw.w)) << 16);
  qr.fit((int)(ktop >> 26) & 31);
  constexpr uint32_t eight = 0x48004800u;

  // ---- scores: 64 tokens x 8 columns a tile, two chains of four products each
  float c[4][kTiles][4], zc[kTiles][4];
  // stages start at multiples of 1024 bytes and the swizzle changes address bits 4..6 alone, so
  // a chunk's place is one exclusive or away.  Row of token 8 (lane / 8) + lane % 8, its chunk 0:
  const unsigned code0 = st + (lane & 7) * 128 + (lane >> 3) * 1024 + ((lane & 7) << 4);
  const unsigned sz0 = st + 68 * 128 + (j << 5), vsz0 = st + 64 * 128 + ((i >> 1) << 4) + (i & 1) * 8;
#pragma unroll
  for (int hq = 0; hq < 2; ++hq) {
    float d[4][kTiles][4];
#pragma unroll
    for (int q = 2 * hq; q < 2 * hq + 2; ++q) {
      const uint4 w0 = lds128((sz0 ^ ((4 + q) << 4)) + q * 128), w1 = lds128((sz0 ^ ((5 ^ q) << 4)) + q * 128);
      uint32_t sp[4], zp[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sp[k] = __byte_perm((&w0.x)[k], (&w1.x)[k], 0x5410);
        zp[k] = __byte_perm((&w0.x)[k], (&w1.x)[k], 0x7632);
      }
      uint32_t bq[kTiles][4];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 qv = h2(qr.w[t][4 * q + k]), sv = h2(sp[k]);
          const uint32_t hi = u2(__hmul2(qv, sv)) & qr.part;  // part 0: fl(q s); part 1: q s - fl(q s)
          bq[t][k] = u2(__hfma2(qv, sv, __hneg2(h2(hi))));
        }
        // rows 0..7: q z + 8 hi (and, unused, q z + 8 lo); rows 8..15: 8 hi (unused) and 8 lo
        if (q == 0) mma_f16_first(zc[t], zp[0], 0u, zp[1], 0u, qr.w[t][4 * q], qr.w[t][4 * q + 1]);
        else mma_f16(zc[t], zp[0], 0u, zp[1], 0u, qr.w[t][4 * q], qr.w[t][4 * q + 1]);
        mma_f16(zc[t], eight, eight, eight, eight, bq[t][0], bq[t][1]);
        mma_f16(zc[t], zp[2], 0u, zp[3], 0u, qr.w[t][4 * q + 2], qr.w[t][4 * q + 3]);
        mma_f16(zc[t], eight, eight, eight, eight, bq[t][2], bq[t][3]);
      }
#pragma unroll
      for (int r2 = 0; r2 < 2; ++r2) {
        uint32_t k4[4];
        ldsm4(k4, (code0 ^ (q << 4)) + r2 * 4096);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t a0 = k4[2 * r], a1 = k4[2 * r + 1], b0 = a0 >> 8, b1 = a1 >> 8;
          const uint32_t e0 = centred<false>(a0), e1 = centred<false>(a1), o0 = centred<true>(a0), o1 = centred<true>(a1);
          const uint32_t e2 = centred<false>(b0), e3 = centred<false>(b1), o2 = centred<true>(b0), o3 = centred<true>(b1);
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            if (q == 2 * hq) mma_f16_first(d[2 * r2 + r][t], e0, e1, o0, o1, bq[t][0], bq[t][1]);
            else mma_f16(d[2 * r2 + r][t], e0, e1, o0, o1, bq[t][0], bq[t][1]);
            mma_f16(d[2 * r2 + r][t], e2, e3, o2, o3, bq[t][2], bq[t][3]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) c[r][t][k] = hq == 0 ? d[r][t][k] : c[r][t][k] + d[r][t][k];
  }
  // lane (i, j): tokens 16 r + i and 16 r + 8 + i of head j; a score is sum scale + off, scale >= 0
  float top[kTiles], off[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    off[t] = (zc[t][0] + zc[t][3]) * qr.scale[t];
    float mx = -INFINITY;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      c[r][t][0] += c[r][t][1];
      c[r][t][1] = c[r][t][2] + c[r][t][3];
      mx = fmaxf(mx, fmaxf(c[r][t][0], c[r][t][1]));
    }
    top[t] = fmaf(mx, qr.scale[t], off[t]);
  }
  // values' scales are below 2^(ev - 14): p s < 2^15
  s.raise(top, 29.f - (float)max((int)(vtop >> 26) & 31, 1));
#pragma unroll
  for (int t = 0; t < kTiles; ++t) off[t] -= s.base(t);
  uint32_t bv[kTiles][2][8];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint2 sz = lds64((vsz0 ^ ((r ^ (4 * k)) << 4)) + r * 128);  // of token 16 r + 8 k + i
      const float2 f0 = unpack_sz(sz.x), f1 = unpack_sz(sz.y);
      const float c0 = fmaf(8.f, f0.x, f0.y), c1 = fmaf(8.f, f1.x, f1.y);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const float p = ex2(fmaf(c[r][t][k], qr.scale[t], off[t]));
        s.l[t] += p;
        s.z0[t] = fmaf(p, c0, s.z0[t]);
        s.z1[t] = fmaf(p, c1, s.z1[t]);
        bv[t][0][2 * r + k] = transpose8(split_f16(p * f0.x));
        bv[t][1][2 * r + k] = transpose8(split_f16(p * f1.x));
      }
    }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float d[2][kTiles][4];
#pragma unroll
    for (int r2 = 0; r2 < 2; ++r2) {
      uint32_t v4[4];  // 32 channels of tokens 32 r2 + 0..7, 8..15, 16..23, 24..31
      ldsm4t(v4, (code0 ^ ((4 + q) << 4)) + r2 * 4096);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t a0 = v4[2 * r], a1 = v4[2 * r + 1], b0 = a0 >> 8, b1 = a1 >> 8;
        const uint32_t e0 = centred<false>(a0), e1 = centred<false>(a1), o0 = centred<true>(a0), o1 = centred<true>(a1);
        const uint32_t e2 = centred<false>(b0), e3 = centred<false>(b1), o2 = centred<true>(b0), o3 = centred<true>(b1);
        const int at = 4 * r2 + 2 * r;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (at == 0) {
            mma_f16_first(d[0][t], e0, o0, e1, o1, bv[t][q >> 1][at], bv[t][q >> 1][at + 1]);
            mma_f16_first(d[1][t], e2, o2, e3, o3, bv[t][q >> 1][at], bv[t][q >> 1][at + 1]);
          } else {
            mma_f16(d[0][t], e0, o0, e1, o1, bv[t][q >> 1][at], bv[t][q >> 1][at + 1]);
            mma_f16(d[1][t], e2, o2, e3, o3, bv[t][q >> 1][at], bv[t][q >> 1][at + 1]);
          }
        }
      }
    }
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) s.acc[2 * q + f][t][k] += d[f][t][k];
  }
}

// `live` tail rows (1..16) in shared memory: keys at st, values at st + 4096, row t in the
// 128-byte rows 2 t and 2 t + 1.  The queries come from the registers block_unit's products
// use, so channels go to the matrix unit in their order.
template <int kTiles>
__device__ __forceinline__ void tail_unit(unsigned st, int live, const Query<kTiles>& qr, State<kTiles>& s) {
  const int lane = threadIdx.x & 31, i = lane >> 2, j = lane & 3;
  float c[kTiles][4];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int k = 0; k < 4; ++k) c[t][k] = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    // channels 32 q + 8 j .. + 7 of tokens i and i + 8, as the pairs {0, 4}, {1, 5}, {2, 6}, {3, 7}
    uint32_t k4[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = 2 * (i + 8 * x) + (q >> 1);
      const uint4 v = lds128(st + row * 128 + (((4 * (q & 1) + j) ^ (row & 7)) << 4));
      k4[x][0] = __byte_perm(v.x, v.z, 0x5410);
      k4[x][1] = __byte_perm(v.x, v.z, 0x7632);
      k4[x][2] = __byte_perm(v.y, v.w, 0x5410);
      k4[x][3] = __byte_perm(v.y, v.w, 0x7632);
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      uint32_t b[4];  // the query in BF16, exact, in the columns of part 0
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(h2(qr.w[t][4 * q + k]));
        b[k] = pack_b16(f.x, f.y) & ~qr.part;
      }
      mma_bf16(c[t], k4[0][0], k4[1][0], k4[0][1], k4[1][1], b[0], b[1]);
      mma_bf16(c[t], k4[0][2], k4[1][2], k4[0][3], k4[1][3], b[2], b[3]);
    }
  }
  float top[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    c[t][0] = i < live ? c[t][0] * qr.scale[t] : -INFINITY;
    c[t][1] = i + 8 < live ? c[t][2] * qr.scale[t] : -INFINITY;
    top[t] = fmaxf(c[t][0], c[t][1]);
  }
  s.raise(top, 24.f);
  uint32_t bv[kTiles][2][2];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // rows behind the last: exactly 0, whatever their scores
      const float p = i + 8 * k < live ? ex2(c[t][k] - s.base(t)) : 0.f;
      s.l[t] += p;
      const float hi = __bfloat162float(__float2bfloat16_rn(p)), r1 = p - hi;  // parts of 8 bits
      const float mid = __bfloat162float(__float2bfloat16_rn(r1));
      // the first product has half of the high part in both columns: an infinite value meets no 0
      bv[t][0][k] = transpose8(pack_b16(0.5f * hi, 0.5f * hi));
      bv[t][1][k] = transpose8(pack_b16(mid, r1 - mid));
    }
  // rows behind the last may hold anything: their values are taken as 0
  const uint32_t m0 = (2 * j < live ? 0xffffu : 0u) | (2 * j + 1 < live ? 0xffff0000u : 0u);
  const uint32_t m1 = (2 * j + 8 < live ? 0xffffu : 0u) | (2 * j + 9 < live ? 0xffff0000u : 0u);
  // the high part of p, then the low ones, for which infinities and NaN are taken as 0
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t b[kTiles][2];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      b[t][0] = pass ? bv[t][1][0] : bv[t][0][0];
      b[t][1] = pass ? bv[t][1][1] : bv[t][0][1];
    }
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
    __nv_bfloat162 nan = zero;  // NaN once a value is not finite
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint2 v[4];  // channels 32 q + 4 i .. + 3 of tokens 2 j, 2 j + 1, 2 j + 8, 2 j + 9
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = 2 * j + (k & 1) + 8 * (k >> 1), row = 2 * t + (q >> 1);
        v[k] = lds64(st + 4096 + row * 128 + (((4 * (q & 1) + (i >> 1)) ^ (row & 7)) << 4) + 8 * (i & 1));
      }
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const uint32_t x0 = f ? v[0].y : v[0].x, x1 = f ? v[1].y : v[1].x, x2 = f ? v[2].y : v[2].x, x3 = f ? v[3].y : v[3].x;
        uint32_t av[4] = {__byte_perm(x0, x1, 0x5410) & m0, __byte_perm(x0, x1, 0x7632) & m0,
                          __byte_perm(x2, x3, 0x5410) & m1, __byte_perm(x2, x3, 0x7632) & m1};
#pragma unroll
        for (int e = 0; e < 4; ++e) nan = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&av[e]), zero, nan);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_bf16(d, av[0], av[1], av[2], av[3], b[t][0], b[t][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) s.acc[2 * q + f][t][e] += d[e];
        }
      }
    }
    if (pass == 0 && __any_sync(kFull, (*reinterpret_cast<uint32_t*>(&nan) & 0x7fff7fffu) != 0u)) {
      // rare: the values that are not finite give way to 0 in place
      __syncwarp();
#pragma unroll 1
      for (int w = lane; w < kTailBytes / 8; w += 32) {
        const unsigned at = st + 4096 + 4 * w;
        uint32_t x;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
        x &= ((x & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) | ((x & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
      }
      fence_proxy_async();  // before the next copy into this stage
      __syncwarp();
    }
  }
}

// 1 / l, and 0 where nothing was attended to (l = 0); log2 of the sum of 2^score
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : __frcp_rn(l); }
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.f ? -INFINITY : m + log2f(l); }

// States lie in shared memory, or in global memory where another SM may have written them: read
// by their generic address, past this SM's cache.
__device__ __forceinline__ float2 ld_part2(const float* p) {
  float2 v;
  asm volatile("ld.relaxed.gpu.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_part4(const float* p) {
  float4 v;
  asm volatile("ld.relaxed.gpu.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}

// Join n states of one head (the k-th at part(k)), 32 at a time: lane l weighs state l, then
// takes channels 4 l .. 4 l + 3 of each.
template <class F>
__device__ __forceinline__ void join(int n, F&& part, float4& o, float& m, float& l) {
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int k0 = 0; k0 < n; k0 += 32) {
    const float* p = part(min(k0 + lane, n - 1));
    float2 ml = ld_part2(p + kD);
    if (k0 + lane >= n) ml = make_float2(-INFINITY, 0.f);
    const float top = fmaxf(m, warp_max(fmaxf(ml.x, -INFINITY)));
    const float old = m == top ? 1.f : ex2(m - top);
    const float f = k0 + lane >= n ? 0.f : ml.x == top ? 1.f : ex2(ml.x - top);  // 1 also where no state has a maximum
    m = top;
    l = fmaf(l, old, warp_sum(f * ml.y));
    o.x *= old;
    o.y *= old;
    o.z *= old;
    o.w *= old;
    const int cnt = min(32, n - k0);
#pragma unroll 1
    for (int k = 0; k < cnt; k += 4) {  // (lanes from n on repeat the last state, with weight 0)
      float4 x[4];
#pragma unroll
      for (int y = 0; y < 4; ++y)
        x[y] = ld_part4(reinterpret_cast<const float*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(p), (k + y) & 31)) + 4 * lane);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float fk = __shfl_sync(kFull, f, (k + y) & 31);
        if (k + y < cnt) {
          o.x = fmaf(fk, x[y].x, o.x);
          o.y = fmaf(fk, x[y].y, o.y);
          o.z = fmaf(fk, x[y].z, o.z);
          o.w = fmaf(fk, x[y].w, o.w);
        }
      }
    }
  }
}

template <int kTiles, bool kSel, bool kOne>
__global__ void __launch_bounds__(Shape<kTiles>::kThreads, 1)
    paged_attn_kernel(const PagedAttnArgs a, const __grid_constant__ CUtensorMap map_rec,
                      const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using Sh = Shape<kTiles>;
  extern __shared__ uint8_t raw[];
  __shared__ alignas(8) uint64_t bars[Sh::kWarps][Sh::kDepth];
  __shared__ int red[Sh::kWarps];
  __shared__ Segment s_own[Sh::kWarps][2];  // segments whose first piece in this CTA a warp holds
  __shared__ int s_owned[Sh::kWarps];
  __shared__ Errors errors;
  __shared__ int s_begin[Sh::kWarps + 1];       // the warps' stretches
  __shared__ int s_total, s_ctas;
  __shared__ const float* s_first[Sh::kWarps];  // where the state of a warp's first piece is
  uint8_t* stages = raw + (1024 - (smem_addr(raw) & 1023)) % 1024;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = a.p.kv_heads;
  const Line<Sh::kHeads, kSel, kOne> line{a};

  if (lane == 0) {
    for (int d = 0; d < Sh::kDepth; ++d) mbar_init(&bars[warp][d], 1);
    fence_mbar_init();
    s_owned[warp] = 0;
    if (warp == 0) {
      errors.count = 0;
      prefetch_map(&map_rec);
      prefetch_map(&map_k);
      prefetch_map(&map_v);
    }
  }
  // (launched while its predecessor ends: nothing is read or written before this)
  grid_dep_launch();
  grid_dep_wait();
  __syncthreads();
  // the line of units, then this CTA's and this warp's stretch of it
  auto length_of = [&](int b, bool tell) {  // -1: padded
    const int s = a.slots ? ld(a.slots + b) : b;
    if (s < 0 || s >= a.x.slots) {
      if (s != -1 && tell) errors.add(FL_DEV_SLOT_RANGE, b);
      return -1;
    }
    const int n = a.x.length[s];
    if (n >= 0 && n <= a.x.max_pages * FL_PAGE) return n;
    if (tell) errors.add(FL_DEV_TOO_LONG, b);
    return 0;
  };
  const int per_entry = heads * line.chunks();  // segments of an entry
  int total = 0, most = 0, segments = 0;  // units, units of the longest segment
  int clo, chi, wlo, whi;
  // A small call takes fewer CTAs (a warp should have a unit).  One whose segments have all the
  // same length takes one CTA each where that costs a warp a unit more at most: none is cut
  // then, which saves the join between CTAs (1 x 256, 16 heads: 12.8 -> 8.5 us; 16 x 32768
  // with 52 blocks kept, 8 x 4 heads, the whole step: 62.6 -> 57 us).
  auto stretch = [&]() {
    int ctas = min((int)gridDim.x, max(total / kMinUnits, 1));
    if (segments > 0 && segments <= (int)gridDim.x && total == segments * most &&
        most <= total / (int)gridDim.x + Sh::kWarps)
      ctas = segments;
    clo = (int)((int64_t)total * blockIdx.x / ctas);
    chi = (int)blockIdx.x < ctas ? (int)((int64_t)total * (blockIdx.x + 1) / ctas) : clo;
    // (with fewer units than warps the last warps have none)
    const int n = chi - clo, q = n / Sh::kWarps, r = n % Sh::kWarps;
    auto begin = [&](int w) { return n >= Sh::kWarps ? clo + q * w + r * w / Sh::kWarps : min(clo + w, chi); };
    wlo = begin(warp);
    whi = begin(warp + 1);
    if (lane == 0) s_begin[warp] = wlo;
    if (lane == 0 && warp == Sh::kWarps - 1) {
      s_begin[Sh::kWarps] = whi;
      s_total = total;
      s_ctas = ctas;
    }
  };
  Cursor use{};
  int left = 0;  // units of the entry before this warp's first one
  if (a.batch <= kWarpScan) {
    // every warp goes through the lengths by itself: entry 32 y + l in lane l
    int n4[kWarpScan / 32], u4[kWarpScan / 32], p4[kWarpScan / 32];
#pragma unroll
    for (int y = 0; y < kWarpScan / 32; ++y) n4[y] = 32 * y + lane < a.batch ? length_of(32 * y + lane, blockIdx.x == 0 && warp == 0) : -1;
#pragma unroll
    for (int y = 0; y < kWarpScan / 32; ++y) {
      u4[y] = p4[y] = 0;
      if (32 * y >= a.batch) continue;
      const int u = n4[y] < 0 ? 0 : line.units_of(n4[y]);
      most = max(most, __reduce_max_sync(kFull, u));
      segments += per_entry * __popc(__ballot_sync(kFull, u > 0));
      u4[y] = u * per_entry;
      int sum = u4[y];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += v;
      }
      p4[y] = total + sum - u4[y];
      total += __shfl_sync(kFull, sum, 31);
    }
    stretch();
#pragma unroll
    for (int y = 0; y < kWarpScan / 32; ++y) {
      if (32 * y >= a.batch) continue;
      const unsigned in = __ballot_sync(kFull, wlo < whi && p4[y] <= wlo && wlo < p4[y] + u4[y]);
      if (in) {
        const int l = __ffs(in) - 1;
        use.b = 32 * y + l;
        use.n = __shfl_sync(kFull, n4[y], l);
        left = wlo - __shfl_sync(kFull, p4[y], l);
      }
    }
  } else {
    int32_t* prefix = reinterpret_cast<int32_t*>(stages);  // [batch + 1]
    int32_t* lengths = prefix + a.batch + 1;                // [batch]
    total = paged_scan<Sh::kThreads>(a.batch, prefix, red, [&](int b) {
      const int n = length_of(b, blockIdx.x == 0);
      lengths[b] = n;
      return n < 0 ? 0 : line.units_of(n) * per_entry;
    });
    stretch();
    if (wlo < whi) {
      use.b = paged_find(prefix, a.batch, wlo);
      use.n = lengths[use.b];
      left = wlo - prefix[use.b];
    }
    __syncthreads();  // the stages take over from the prefix sums
    fence_proxy_async();
  }
  if (clo == chi) {  // (CTA 0, which looks at the entries, has units or there are none)
    __syncthreads();
    if (threadIdx.x == 0) errors.tell(a.x);
    return;
  }
  if (wlo < whi) {
    use.slot = a.slots ? ld(a.slots + use.b) : use.b;
    line.place(use, use.n);
    const int seg = left / use.units;
    use.u = left - seg * use.units;
    use.h = kOne ? seg : seg / line.chunks();
    use.ch = seg - use.h * line.chunks();
  }

  // states of pieces: the last one of a warp in its own stages, one before it in the workspace
  auto smem_part = [&](int w) { return reinterpret_cast<float*>(stages + (size_t)w * Sh::kDepth * kRec); };
  auto global_part = [&](int w) {
    return static_cast<float*>(a.data) + (size_t)(blockIdx.x * Sh::kWarps + w) * Sh::kHeads * kPart;
  };

  if (wlo < whi) {
    Query<kTiles> qr;
    State<kTiles> s;
    Cursor load = use;
    int rows = -1, rows_at = 0, rows_end = 0;  // lane l: record row of unit rows_at + l of the segment
    uint8_t* const st0 = stages + (size_t)warp * Sh::kDepth * kRec;
    int issued = 0, in = 0;  // units issued, and the stage of the next one
    unsigned voids = 0;      // stages whose block could not be read
    const int count = whi - wlo;
    auto issue = [&]() {
      uint64_t* bar = &bars[warp][in];
      uint8_t* dst = st0 + in * kRec;
      voids &= ~(1u << in);
      if (load.u < load.np) {
        if (load.u >= rows_end) {
          rows_at = load.u;
          rows_end = min(load.u + 32, load.np);
          rows = -1;
          int block = load.u + lane;
          if (block < load.np) {
            if (kSel) block = ld(a.sel + ((size_t)load.b * heads + load.h) * a.keep + block);
            int error = 0;
            if (!kSel || (block >= 0 && block < paged_full(load.n))) {
              const int page = ld(a.x.table + (int64_t)load.slot * a.x.max_pages + block);
              if (page >= 0 && page < a.x.pages) rows = (page * heads + load.h) * (kRec / 128);
              else error = FL_DEV_PAGE_RANGE;
            } else if (block != -1) {
              error = FL_DEV_SEL_BLOCK;
            }
            if (error && load.ch == 0) errors.add(error, load.b);
          }
        }
        const int row = __shfl_sync(kFull, rows, load.u - rows_at);
        if (row < 0) {
          voids |= 1u << in;
          if (lane == 0) mbar_arrive(bar);
        } else if (lane == 0) {
          mbar_expect_tx(bar, kRec);
          tma_rows(dst, &map_rec, row, bar);
        }
      } else if (load.n == 0) {
        if (lane == 0) mbar_arrive(bar);
      } else if (lane == 0) {
        mbar_expect_tx(bar, kTailBytes);
        const int row = (load.slot * heads + load.h) * (2 * FL_PAGE) + 2 * kTailUnit * (load.u - load.np);
        tma_rows(dst, &map_k, row, bar);
        tma_rows(dst + kTailBytes / 2, &map_v, row, bar);
      }
      in = in + 1 == Sh::kDepth ? 0 : in + 1;
      ++issued;
      if (load.u + 1 == load.units) rows_end = 0;
      line.next(load);
    };
    int out = 0, phase = 0;  // the stage of the next unit to use, and its barrier's parity
    // One turn of the loop puts away the piece of the last turn while the queries of the next
    // one are on their way.  What a warp runs once or twice is paid for in instruction fetches:
    // it stands in one place where it can, and is not unrolled.
    int pos = wlo, k = 0, piece = 0;
    Segment seg{};
#pragma unroll 1
    for (;;) {
      const bool more = k < count;
      // (with two tiles the registers do not allow it)
      if (kTiles == 1 && more) qr.fetch(a, use.b, line.head(use.h, use.ch), line.live(use.ch));
      if (k > 0) {
        // this lane's channels of head j: 32 q + 4 i .. + 3
        const int i = lane >> 2, j = lane & 3;
        const int head0 = line.head(seg.h, seg.ch), live = line.live(seg.ch);
        const bool whole = piece == seg.end - seg.begin;
        float* const part = pos == whi ? smem_part(warp) : global_part(warp);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            s.l[t] += __shfl_xor_sync(kFull, s.l[t], o);
            s.z0[t] += __shfl_xor_sync(kFull, s.z0[t], o);
            s.z1[t] += __shfl_xor_sync(kFull, s.z1[t], o);
          }
          const int g = 4 * t + j;
          if (g >= live) continue;
          float* to = whole ? a.o + (int64_t)seg.b * a.o_batch_stride + (int64_t)(head0 + g) * a.o_head_stride : part + g * kPart;
          const float inv = whole ? inverse(s.l[t]) : 1.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float z = q < 2 ? s.z0[t] : s.z1[t];
            float4 v;
            v.x = (s.acc[2 * q][t][0] + s.acc[2 * q][t][1] + z) * inv;
            v.y = (s.acc[2 * q][t][2] + s.acc[2 * q][t][3] + z) * inv;
            v.z = (s.acc[2 * q + 1][t][0] + s.acc[2 * q + 1][t][1] + z) * inv;
            v.w = (s.acc[2 * q + 1][t][2] + s.acc[2 * q + 1][t][3] + z) * inv;
            *reinterpret_cast<float4*>(to + 32 * q + 4 * i) = v;
          }
          if (i == 0) {
            if (!whole) *reinterpret_cast<float2*>(to + kD) = make_float2(s.m[t], s.l[t]);
            else if (a.lse) a.lse[(size_t)seg.b * a.q_heads + head0 + g] = log_sum(s.m[t], s.l[t]);
          }
        }
        if (pos - piece == wlo && lane == 0) s_first[warp] = part;
        // the first piece of a segment in this CTA joins the others
        if (!whole && pos - piece == max(seg.begin, s_begin[0]) && lane == 0) s_own[warp][s_owned[warp]++] = seg;
      }
      if (!more) break;
      seg = Segment{pos - use.u, pos - use.u + use.units, use.b, use.h, use.ch};
      piece = min(use.units - use.u, whi - pos);
      s.clear();
      const int tail_rows = use.n - FL_PAGE * paged_full(use.n);
#pragma unroll 1
      while (issued < count && issued < k + Sh::kDepth) issue();  // (the first turn)
      if (kTiles > 1) qr.fetch(a, use.b, line.head(use.h, use.ch), line.live(use.ch));
      qr.prepare();
#pragma unroll 1
      for (int x = 0; x < piece; ++x, ++k) {
        if (!mbar_wait(&bars[warp][out], phase)) {
          if (lane == 0) errors.add(FL_DEV_TIMEOUT, use.b);
#pragma unroll 1
          for (int d = 1; d < issued - k; ++d) {  // copies still in flight
            out = out + 1 == Sh::kDepth ? 0 : out + 1;
            if (out == 0) phase ^= 1;
            mbar_wait(&bars[warp][out], phase);
          }
          k = count;
          break;
        }
        const unsigned st = smem_addr(st0) + out * kRec;
        const int tail = use.u + x - use.np;  // quarter of the tail, negative for a block
        if (tail >= 0) {
          if (use.n > 0) tail_unit<kTiles>(st, min(kTailUnit, tail_rows - kTailUnit * tail), qr, s);
        } else if (!((voids >> out) & 1u)) {
          block_unit<kTiles>(st, qr, s);
        }
        out = out + 1 == Sh::kDepth ? 0 : out + 1;
        if (out == 0) phase ^= 1;
        __syncwarp();
        if (issued < count) issue();
      }
      pos += piece;
      use.u += piece - 1;
      line.next(use);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) errors.tell(a.x);

  // head g of the segments that warp w holds is joined by warp w + g.  (The stretches are read
  // again: kept in registers over the loop above they would be spilled.)
  const int first = s_begin[0], last = s_begin[Sh::kWarps];
#pragma unroll 1
  for (int g = 0; g < min(Sh::kHeads, a.group); ++g) {
    const int w0 = warp >= g ? warp - g : warp - g + Sh::kWarps;
#pragma unroll 1
    for (int k = 0; k < s_owned[w0]; ++k) {
      const Segment seg = s_own[w0][k];
      if (g >= line.live(seg.ch)) continue;
      // warp w0 and the next ones hold its pieces: w0's is its last one unless the segment ended
      // inside its part, the others continue the segment with their first
      const float* const piece0 = s_begin[w0 + 1] > seg.end ? global_part(w0) : smem_part(w0);
      int n = 1, c0 = -1;
      while (s_begin[w0 + n] < min(seg.end, last)) ++n;
      // several CTAs may share the segment (c0 .. c1): the last one to arrive joins their states
      const bool inside = seg.begin >= first && seg.end <= last;
      float4 o;
      float m, l;
      auto cta_part = [&](int c) {
        return static_cast<float*>(a.data) + (((size_t)kMaxCtas * Sh::kWarps + 2 * c + (c == c0 ? 1 : 0)) * Sh::kHeads + g) * kPart;
      };
#pragma unroll 1
      for (;;) {
        join(n, [&](int x) -> const float* {
          if (c0 >= 0) return cta_part(c0 + x);
          return (x == 0 ? piece0 : s_first[w0 + x]) + g * kPart;
        }, o, m, l);
        if (inside || c0 >= 0) {
          const int head = line.head(seg.h, seg.ch) + g;
          const float inv = inverse(l);
          *reinterpret_cast<float4*>(a.o + (int64_t)seg.b * a.o_batch_stride + (int64_t)head * a.o_head_stride + 4 * lane) =
              make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
          if (lane == 0 && a.lse) a.lse[(size_t)seg.b * a.q_heads + head] = log_sum(m, l);
          break;
        }
        c0 = (int)(((uint64_t)(seg.begin + 1) * s_ctas - 1) / (unsigned)s_total);
        n = (int)(((uint64_t)seg.end * s_ctas - 1) / (unsigned)s_total) - c0 + 1;
        float* mine = cta_part(blockIdx.x);
        *(reinterpret_cast<float4*>(mine) + lane) = o;
        if (lane == 0) *reinterpret_cast<float2*>(mine + kD) = make_float2(m, l);
        __threadfence();
        __syncwarp();
        int32_t* ticket = a.tickets + c0 * 8 + g;
        int done = 0;
        if (lane == 0) done = atomicAdd(ticket, 1) == n - 1;
        if (!__shfl_sync(kFull, done, 0)) break;
        __threadfence();
        if (lane == 0) *ticket = 0;
      }
    }
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    return nullptr;
  }();
  return fn;
}

// `rows` rows of 128 bytes, copied `box` rows at a time with the 128-byte swizzle.
bool rows_map(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {128, rows};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t boxes[2] = {128, box};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::atomic<bool> g_attr_done[kMaxDevices];
std::mutex g_attr_mu;

template <int kTiles, bool kSel, bool kOne>
cudaError_t launch_as(const PagedAttnArgs& a, int ctas, cudaStream_t s) {
  using Sh = Shape<kTiles>;
  CUtensorMap rec, tk, tv;
  const uint64_t tail_rows = (uint64_t)a.x.slots * a.p.kv_heads * 2 * FL_PAGE;
  if (!rows_map(&rec, a.p.rec, (uint64_t)a.x.pages * a.p.kv_heads * (kRec / 128), kRec / 128) ||
      !rows_map(&tk, a.p.tail_k, tail_rows, 2 * kTailUnit) || !rows_map(&tv, a.p.tail_v, tail_rows, 2 * kTailUnit))
    return cudaErrorInvalidValue;
  return launch_pdl(paged_attn_kernel<kTiles, kSel, kOne>, dim3(ctas), dim3(Sh::kThreads), Sh::kSmem, s, a, rec, tk, tv);
}

template <int kTiles, bool kSel, bool kOne>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(paged_attn_kernel<kTiles, kSel, kOne>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Shape<kTiles>::kSmem);
}

// Up to 4 query heads a group make one tile of 8 columns.  More take two tiles, which halves
// the work on the codes, where there is much of it, and two segments of one tile where there is
// little (by what the call can hold: lengths are the device's): the larger code and its fewer
// warps start more slowly.  4 x 8 heads, 16 x 16384: two tiles 112 us, two segments 139; 64 x
// 8191 with 16 blocks kept: the step 33.3 and 31.2; 8 requests of up to 100: 13.1 and 8.2.
constexpr int kFewUnits = 8;  // a warp

template <bool kSel>
cudaError_t launch(const PagedAttnArgs& a, int ctas, cudaStream_t s) {
  if (a.group <= 4) return launch_as<1, kSel, true>(a, ctas, s);
  const int64_t units = (int64_t)a.batch * a.p.kv_heads * ((kSel && a.keep < a.x.max_pages ? a.keep : a.x.max_pages) + FL_PAGE / kTailUnit);
  if (units <= (int64_t)kFewUnits * Shape<1>::kWarps * ctas) return launch_as<1, kSel, false>(a, ctas, s);
  if (a.group <= 8) return launch_as<2, kSel, true>(a, ctas, s);
  return launch_as<2, kSel, false>(a, ctas, s);
}

}  // namespace

uint64_t paged_attn_bytes(const fl_paged_pool& p, int q_heads) {
  const uint64_t one = (Shape<1>::kWarps + 2) * Shape<1>::kHeads, two = (Shape<2>::kWarps + 2) * Shape<2>::kHeads;
  return (uint64_t)kMaxCtas * (q_heads / p.kv_heads <= 4 || one > two ? one : two) * kPart * sizeof(float);
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s) {
  if (a.batch == 0) return cudaSuccess;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const cudaError_t e = once_per_device(g_attr_done, g_attr_mu, [](int) {
    cudaError_t r = allow_smem<1, false, true>();
    if (r == cudaSuccess) r = allow_smem<1, true, true>();
    if (r == cudaSuccess) r = allow_smem<1, false, false>();
    if (r == cudaSuccess) r = allow_smem<1, true, false>();
    if (r == cudaSuccess) r = allow_smem<2, false, true>();
    if (r == cudaSuccess) r = allow_smem<2, true, true>();
    if (r == cudaSuccess) r = allow_smem<2, false, false>();
    if (r == cudaSuccess) r = allow_smem<2, true, false>();
    return r;
  });
  if (e != cudaSuccess) return e;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  return a.sel ? launch<true>(a, ctas, s) : launch<false>(a, ctas, s);
}

}  // namespace fl
