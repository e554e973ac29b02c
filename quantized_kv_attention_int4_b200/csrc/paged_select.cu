// The blocks a request's new token attends to (include/flashloop_paged.h: fl_paged_select).
//
// score(block) = max over the group's queries of sum_c max(q_c lo_c, q_c hi_c), with lo = z
// and hi = z + 15 s of the record's key groups: the largest q.k any key of the block could
// have, from 512 of the record's 9216 bytes.  Two launches:
//   score_kernel  eight lanes a block, 16 channels each; every product is exact in fp64 (8
//                 significant bits times at most 45), so scores of equal blocks are equal
//                 and the order is the definition's but for differences of a few 1e-16;
//   topk_kernel   one CTA per (entry, head): radix select on the scores' 64-bit images
//                 from the highest bit in which they differ, then the chosen blocks in order.
#include "paged.cuh"

namespace fl {
namespace {

constexpr int kST = 256;       // threads of the score kernel
constexpr int kChunk = 128;    // blocks of one chunk: four rounds of 32
constexpr int kTT = 256;       // threads of the top-k kernel
constexpr int kDigit = 10;

__device__ __forceinline__ unsigned long long score_image(double v) {
  if (v != v) return 0ull;  // NaN ranks below everything
  const long long b = __double_as_longlong(v + 0.0);
  return (unsigned long long)(b < 0 ? ~b : b | (long long)0x8000000000000000ull);
}

// q+ and q- of one (entry, head) in fp64: sum_c max(q lo, q hi) = sum_c q+ hi + q- lo.
__global__ void __launch_bounds__(kST) score_kernel(PagedAttnArgs a) {
  extern __shared__ int32_t prefix[];
  __shared__ int red[kST / 32];
  __shared__ float s_q[8][kD];
  const int tid = threadIdx.x, lane = tid & 31, heads = a.p.kv_heads;
  const fl_paged_index& x = a.x;
  const bool tell = blockIdx.x == 0;
  const int total = paged_scan<kST>(a.batch, prefix, red, [&](int b) {
    const int s = paged_slot(x, a.slots, b, tell);
    if (s < 0) return 0;
    const int full = paged_full(paged_length(x, s, b, tell));
    return full > a.keep ? (full + kChunk - 1) / kChunk : 0;
  });
  const int sub = lane & 7, blk = tid >> 3;  // 32 blocks a round
  for (int64_t w = blockIdx.x; w < (int64_t)total * heads; w += gridDim.x) {
    const int item = (int)(w / heads), h = (int)(w % heads);
    const int b = paged_find(prefix, a.batch, item), c0 = (item - prefix[b]) * kChunk;
    const int s = paged_slot(x, a.slots, b, false);
    const int full = paged_full(paged_length(x, s, b, false));
    unsigned long long* out = static_cast<unsigned long long*>(a.data) + ((size_t)b * heads + h) * x.max_pages;
    double best[kChunk / 32];
#pragma unroll
    for (int r = 0; r < kChunk / 32; ++r) best[r] = -INFINITY;
    bool nan[kChunk / 32] = {};
    for (int g0 = 0; g0 < a.group; g0 += 8) {
      const int gn = min(8, a.group - g0);
      __syncthreads();
      for (int i = tid; i < gn * kD; i += kST) {
        const uint16_t* q = a.q + (int64_t)b * a.q_batch_stride + (int64_t)(h * a.group + g0 + i / kD) * a.q_head_stride;
        s_q[i / kD][i % kD] = __uint_as_float((uint32_t)q[i % kD] << 16);
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kChunk / 32; ++r) {
        const int block = c0 + 32 * r + blk;
        const int page = block < full ? x.table[(int64_t)s * x.max_pages + block] : -1;
        const bool ok = page >= 0 && page < x.pages;
        if (block < full && !ok && sub == 0 && g0 == 0) paged_error(x, FL_DEV_PAGE_RANGE, b);
        double sum[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) sum[g] = 0.0;
        if (ok) {
          const uint8_t* rec = a.p.rec + ((size_t)page * heads + h) * kRec + kRecKsz;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int ch = 32 * e + 4 * sub;
            const uint4 sz = ldg_u4(rec + 4 * ch);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float2 f = unpack_sz((&sz.x)[c]);
              const double lo = (double)f.y, hi = fma(15.0, (double)f.x, lo);
#pragma unroll
              for (int g = 0; g < 8; ++g) {
                if (g < gn) {
                  const float q = s_q[g][ch + c];
                  sum[g] = fma((double)q, q > 0.f ? hi : lo, sum[g]);
                }
              }
            }
          }
        }
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          if (g < gn) {
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) sum[g] += __shfl_xor_sync(kFull, sum[g], o);
            nan[r] |= sum[g] != sum[g];
            best[r] = fmax(best[r], sum[g]);
          }
        }
        if (!ok) nan[r] = true;
      }
    }
#pragma unroll
    for (int r = 0; r < kChunk / 32; ++r) {
      const int block = c0 + 32 * r + blk;
      if (sub == 0 && block < full) out[block] = nan[r] ? 0ull : score_image(best[r]);
    }
  }
}

__global__ void __launch_bounds__(kTT) topk_kernel(PagedAttnArgs a) {
  __shared__ unsigned hist[1 << kDigit];
  __shared__ unsigned long long s_lo[kTT / 32], s_hi[kTT / 32];
  __shared__ int red[kTT / 32];
  __shared__ int s_digit, s_above, s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y, heads = a.p.kv_heads, k = a.keep;
  const fl_paged_index& x = a.x;
  const int s = paged_slot(x, a.slots, b, false);
  if (s < 0) return;
  const int n = paged_full(paged_length(x, s, b, false));
  int32_t* sel = a.sel + ((size_t)b * heads + h) * k;
  if (n <= k) {
    for (int i = tid; i < k; i += kTT) sel[i] = i < n ? i : -1;
    return;
  }
  const unsigned long long* key = static_cast<const unsigned long long*>(a.data) + ((size_t)b * heads + h) * x.max_pages;
  unsigned long long lo = ~0ull, hi = 0ull;
  for (int i = tid; i < n; i += kTT) {
    const unsigned long long u = key[i];
    lo = min(lo, u);
    hi = max(hi, u);
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
    for (int i = tid; i < nb; i += kTT) hist[i] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += kTT) {
      const unsigned long long u = key[i];
      if ((u & known) == prefix) atomicAdd(&hist[(unsigned)(u >> shift) & dmask], 1u);
    }
    __syncthreads();
    constexpr int kPer = (1 << kDigit) / kTT;
    const int top = nb - kPer * tid;  // thread t owns bins top - 1 down to top - kPer
    int cb[kPer], sum = 0, total;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      cb[q] = top - 1 - q >= 0 ? (int)hist[top - 1 - q] : 0;
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
  for (int i0 = 0; i0 < n; i0 += kTT) {
    const int i = i0 + tid;
    const unsigned long long m = i < n ? key[i] & known : 0ull;
    const bool gt = i < n && m > prefix, eq = i < n && m == prefix;
    int total;
    const int before = paged_block_scan<kTT>((gt ? 1 << 16 : 0) | (eq ? 1 : 0), red, total);
    const int g = gt_run + (before >> 16), e = eq_run + (before & 0xffff);
    if (gt || (eq && e < krem)) sel[g + min(e, krem)] = i;
    gt_run += total >> 16;
    eq_run += total & 0xffff;
  }
}

}  // namespace

uint64_t paged_select_bytes(const fl_paged_index& x, const fl_paged_pool& p, int batch) {
  return (uint64_t)batch * p.kv_heads * x.max_pages * 8;
}

cudaError_t launch_paged_select(const PagedAttnArgs& a, cudaStream_t s) {
  if (a.batch == 0) return cudaSuccess;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  if (a.keep < a.x.max_pages) {  // otherwise every request keeps all it has
    const int64_t items = (int64_t)a.batch * ((a.x.max_pages + kChunk - 1) / kChunk) * a.p.kv_heads;
    const int grid = (int)(items < 4 * sms ? items : 4 * sms);
    score_kernel<<<grid, kST, (size_t)(a.batch + 1) * 4, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  topk_kernel<<<dim3(a.p.kv_heads, a.batch), kTT, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace fl
