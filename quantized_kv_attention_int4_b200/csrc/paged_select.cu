// The blocks a request's new token attends to (include/flashloop_paged.h: fl_paged_select).
//
// score(block) = max over the group's queries of sum_c max(q_c lo_c, q_c hi_c), with lo = z
// and hi = z + 15 s of the record's key groups: the largest q.k any key of the block could
// have, from 512 of the record's 9216 bytes.  Two launches, the second one's start overlapped:
//   score_kernel  eight lanes a block, 16 channels each; every product is exact in fp64 (8
//                 significant bits times at most 45), so scores of equal blocks are equal
//                 and the order is the definition's but for differences of a few 1e-16.
//                 A binary16 number becomes an fp64 one by moving its bits (no conversion
//                 instruction, which the SM issues at a quarter of this rate): the exponent
//                 keeps its bias, which scales the number by 2^-1008, subnormals included;
//                 the queries carry 2^500 of that and the sum the rest.
//   topk_kernel   one CTA per (entry, head): radix select on the scores' 64-bit images
//                 from the highest bit in which they differ, the keys of up to 2048 blocks
//                 held in registers, then the chosen blocks in order.
#include "paged.cuh"

namespace fl {
namespace {

constexpr int kST = 256;   // threads of the score kernel: 32 blocks a round
constexpr int kRounds = 2;
constexpr int kChunk = 32 * kRounds;
constexpr int kTT = 256;   // threads of the top-k kernel
constexpr int kHeld = 8;   // keys a thread of it holds
constexpr int kDigit = 10;

__device__ __forceinline__ unsigned long long score_image(double v) {
  if (v != v) return 0ull;  // NaN ranks below everything
  const long long b = __double_as_longlong(v + 0.0);
  return (unsigned long long)(b < 0 ? ~b : b | (long long)0x8000000000000000ull);
}

// kG queries of a group at a time (a group's last ones are repeated to fill them).
template <int kG>
__global__ void __launch_bounds__(kST, 2) score_kernel(PagedAttnArgs a) {
  extern __shared__ int32_t prefix[];
  __shared__ int red[kST / 32];
  // high words of 2^500 q and of 2^500 15 max(q, 0): 8 and 12 significant bits, their low words are 0
  __shared__ alignas(16) int s_q[2][kG][kD];
  grid_dep_launch();
  const int tid = threadIdx.x, heads = a.p.kv_heads;
  const fl_paged_index& x = a.x;
  const bool tell = blockIdx.x == 0;
  const int total = paged_scan<kST>(a.batch, prefix, red, [&](int b) {
    const int s = paged_slot(x, a.slots, b, tell);
    if (s < 0) return 0;
    const int full = paged_full(paged_length(x, s, b, tell));
    return full > a.keep ? (full + kChunk - 1) / kChunk : 0;
  });
  const int sub = tid & 7, blk = tid >> 3;
  for (int64_t w = blockIdx.x; w < (int64_t)total * heads; w += gridDim.x) {
    const int item = (int)(w / heads), h = (int)(w % heads);
    const int b = paged_find(prefix, a.batch, item), c0 = (item - prefix[b]) * kChunk;
    const int s = paged_slot(x, a.slots, b, false);
    const int full = paged_full(paged_length(x, s, b, false));
    const uint8_t* rec[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int block = c0 + 32 * r + blk;
      const int page = block < full ? __ldg(x.table + (int64_t)s * x.max_pages + block) : -1;
      const bool ok = page >= 0 && page < x.pages;
      if (block < full && !ok && sub == 0) paged_error(x, FL_DEV_PAGE_RANGE, b);
      rec[r] = ok ? a.p.rec + ((size_t)page * heads + h) * kRec + kRecKsz : nullptr;
    }
    uint4 sz[kRounds][4];
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) sz[r][e] = rec[r] ? ldg_u4(rec[r] + 128 * e + 16 * sub) : make_uint4(0u, 0u, 0u, 0u);
    double best[kRounds];
    bool nan[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      best[r] = -INFINITY;
      // infinite or NaN scales and zeros (exponent 31) carry into the halves' top bits
      uint32_t over = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < 4; ++c) over |= ((&sz[r][e].x)[c] & 0x7fff7fffu) + 0x04000400u;
      nan[r] = rec[r] == nullptr || (over & 0x80008000u);  // such a block, or one that cannot be read, ranks last
    }
    for (int g0 = 0; g0 < a.group; g0 += kG) {
      __syncthreads();
#pragma unroll
      for (int i = tid; i < kG * kD; i += kST) {
        const int g = min(g0 + i / kD, a.group - 1);
        const uint16_t q = a.q[(int64_t)b * a.q_batch_stride + (int64_t)(h * a.group + g) * a.q_head_stride + i % kD];
        const double v = (double)__uint_as_float((uint32_t)q << 16) * 0x1p500;
        s_q[0][i / kD][i % kD] = __double2hiint(v);
        s_q[1][i / kD][i % kD] = __double2hiint(v > 0.0 ? 15.0 * v : 0.0);
      }
      __syncthreads();
      double sum[kRounds][kG];
#pragma unroll
      for (int r = 0; r < kRounds; ++r)
#pragma unroll
        for (int g = 0; g < kG; ++g) sum[r][g] = 0.0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // sum_c max(q lo, q hi) = sum_c q lo + 15 max(q, 0) s
        double lo[kRounds][4], sc[kRounds][4];
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v = (&sz[r][e].x)[c];
            asm volatile("" : "+r"(v));  // widened here each time: 128 registers if hoisted out of the loop
            sc[r][c] = __hiloint2double((int)((v & 0x7fffu) << 10), 0);
            lo[r][c] = __hiloint2double((int)(((v >> 6) & 0x01fffc00u) | (v & 0x80000000u)), 0);
          }
#pragma unroll
        for (int g = 0; g < kG; ++g) {
          const int4 qa = *reinterpret_cast<const int4*>(&s_q[0][g][32 * e + 4 * sub]);
          const int4 qb = *reinterpret_cast<const int4*>(&s_q[1][g][32 * e + 4 * sub]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const double q = __hiloint2double((&qa.x)[c], 0), p = __hiloint2double((&qb.x)[c], 0);
#pragma unroll
            for (int r = 0; r < kRounds; ++r) sum[r][g] = fma(p, sc[r][c], fma(q, lo[r][c], sum[r][g]));
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kRounds; ++r)
#pragma unroll
        for (int g = 0; g < kG; ++g) {
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) sum[r][g] += __shfl_xor_sync(kFull, sum[r][g], o);
          sum[r][g] *= 0x1p508;
          nan[r] |= sum[r][g] != sum[r][g];
          best[r] = fmax(best[r], sum[r][g]);
        }
    }
    unsigned long long* out = static_cast<unsigned long long*>(a.data) + ((size_t)b * heads + h) * x.max_pages;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int block = c0 + 32 * r + blk;
      const bool bad = __reduce_or_sync(kFull, nan[r] ? 1u << (threadIdx.x >> 3 & 3) : 0u) >> (threadIdx.x >> 3 & 3) & 1u;
      if (sub == 0 && block < full) out[block] = bad ? 0ull : score_image(best[r]);
    }
  }
}

// The k-th largest of n > k keys and the blocks to take; kSmall: n <= kHeld kTT, keys in
// registers.
template <bool kSmall>
__device__ __forceinline__ void topk(const unsigned long long* key, int n, int k, int32_t* sel) {
  __shared__ unsigned hist[1 << kDigit];
  __shared__ unsigned long long s_lo[kTT / 32], s_hi[kTT / 32];
  __shared__ int red[kTT / 32];
  __shared__ int s_digit, s_above, s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // thread t holds keys kHeld t .. + kHeld - 1, so that block order is thread order
  unsigned long long held[kHeld];
  unsigned long long lo = ~0ull, hi = 0ull;
  if constexpr (kSmall) {
#pragma unroll
    for (int y = 0; y < kHeld; ++y) {
      const int i = kHeld * tid + y;
      held[y] = i < n ? __ldcg(key + i) : 0ull;
      lo = i < n ? min(lo, held[y]) : lo;
      hi = max(hi, held[y]);
    }
  } else {
    for (int i = tid; i < n; i += kTT) {
      const unsigned long long u = __ldcg(key + i);
      lo = min(lo, u);
      hi = max(hi, u);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(kFull, lo, o));
    hi = max(hi, __shfl_xor_sync(kFull, hi, o));
  }
  if (lane == 0) {
    s_lo[warp] = lo;
    s_hi[warp] = hi;
  }
  for (int i = tid; i < 1 << kDigit; i += kTT) hist[i] = 0u;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTT / 32; ++w) {
    lo = min(lo, s_lo[w]);
    hi = max(hi, s_hi[w]);
  }
  // keys agree above bit `shift`; the wanted (k-th largest) key is found digit by digit until
  // every key that shares its known bits is taken
  int shift = lo == hi ? 0 : 64 - __clzll((long long)(lo ^ hi));
  unsigned long long known = shift == 64 ? 0ull : ~0ull << shift, prefix = hi & known;
  int krem = k;
  while (shift > 0) {
    const int wb = shift < kDigit ? shift : kDigit;
    shift -= wb;
    const int nb = 1 << wb;
    const unsigned dmask = (unsigned)nb - 1u;
    if constexpr (kSmall) {
#pragma unroll
      for (int y = 0; y < kHeld; ++y)
        if (kHeld * tid + y < n && (held[y] & known) == prefix) atomicAdd(&hist[(unsigned)(held[y] >> shift) & dmask], 1u);
    } else {
      for (int i = tid; i < n; i += kTT) {
        const unsigned long long u = __ldcg(key + i);
        if ((u & known) == prefix) atomicAdd(&hist[(unsigned)(u >> shift) & dmask], 1u);
      }
    }
    __syncthreads();
    constexpr int kPer = (1 << kDigit) / kTT;
    const int top = nb - kPer * tid;  // thread t owns bins top - 1 down to top - kPer
    int cb[kPer], sum = 0, total;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int bin = top - 1 - q;
      cb[q] = bin >= 0 ? (int)hist[bin] : 0;
      if (bin >= 0) hist[bin] = 0u;
      sum += cb[q];
    }
    int acc = paged_block_scan<kTT>(sum, red, total);
    if (acc < krem && acc + sum >= krem) {
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        if (acc < krem && acc + cb[q] >= krem) {
          s_digit = top - 1 - q;
          s_above = acc;
          s_count = cb[q];
        }
        acc += cb[q];
      }
    }
    __syncthreads();
    prefix |= (unsigned long long)s_digit << shift;
    known |= (unsigned long long)dmask << shift;
    krem -= s_above;
    if (s_count == krem) break;
    __syncthreads();
  }
  // every key above the wanted one, and the first krem equal to it, in block order
  int gt_run = 0, eq_run = 0;
  constexpr int kStep = kSmall ? kHeld * kTT : kTT, kMine = kSmall ? kHeld : 1;
  for (int i0 = 0; i0 < n; i0 += kStep) {
    unsigned gts = 0, eqs = 0;
#pragma unroll
    for (int y = 0; y < kMine; ++y) {
      const int i = i0 + kMine * tid + y;
      if (i < n) {
        const unsigned long long m = (kSmall ? held[y] : __ldcg(key + i)) & known;
        gts |= m > prefix ? 1u << y : 0u;
        eqs |= m == prefix ? 1u << y : 0u;
      }
    }
    int total;
    const int before = paged_block_scan<kTT>(__popc(gts) << 16 | __popc(eqs), red, total);
    int g = gt_run + (before >> 16), e = eq_run + (before & 0xffff);
#pragma unroll
    for (int y = 0; y < kMine; ++y) {
      if ((gts >> y) & 1u) sel[g++ + min(e, krem)] = i0 + kMine * tid + y;
      if ((eqs >> y) & 1u) {
        if (e < krem) sel[g + e] = i0 + kMine * tid + y;
        ++e;
      }
    }
    gt_run += total >> 16;
    eq_run += total & 0xffff;
  }
}

__global__ void __launch_bounds__(kTT) topk_kernel(PagedAttnArgs a) {
  const int h = blockIdx.x, b = blockIdx.y, heads = a.p.kv_heads, k = a.keep;
  const fl_paged_index& x = a.x;
  // (lengths and slots were there before the scores' launch)
  const int s = paged_slot(x, a.slots, b, false);
  const int n = s < 0 ? 0 : paged_full(paged_length(x, s, b, false));
  grid_dep_wait();
  if (s < 0) return;
  int32_t* sel = a.sel + ((size_t)b * heads + h) * k;
  if (n <= k) {
    for (int i = threadIdx.x; i < k; i += kTT) sel[i] = i < n ? i : -1;
    return;
  }
  const unsigned long long* key = static_cast<const unsigned long long*>(a.data) + ((size_t)b * heads + h) * x.max_pages;
  if (n <= kHeld * kTT) topk<true>(key, n, k, sel);
  else topk<false>(key, n, k, sel);
}

template <int kG>
cudaError_t launch_score(const PagedAttnArgs& a, int sms, cudaStream_t s) {
  const int64_t items = (int64_t)a.batch * ((a.x.max_pages + kChunk - 1) / kChunk) * a.p.kv_heads;
  const int grid = (int)(items < 4 * sms ? items : 4 * sms);
  score_kernel<kG><<<grid, kST, (size_t)(a.batch + 1) * 4, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

uint64_t paged_select_bytes(const fl_paged_index& x, const fl_paged_pool& p, int batch) {
  return (uint64_t)batch * p.kv_heads * x.max_pages * 8;
}

cudaError_t launch_paged_select(const PagedAttnArgs& a, cudaStream_t s) {
  if (a.batch == 0) return cudaSuccess;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const bool scored = a.keep < a.x.max_pages;  // otherwise every request keeps all it has
  if (scored) {
    const cudaError_t e = a.group == 1   ? launch_score<1>(a, sms, s)
                          : a.group == 2 ? launch_score<2>(a, sms, s)
                          : a.group <= 4 ? launch_score<4>(a, sms, s)
                                         : launch_score<8>(a, sms, s);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl_if(scored, topk_kernel, dim3(a.p.kv_heads, a.batch), dim3(kTT), 0, s, a);
}

}  // namespace fl
