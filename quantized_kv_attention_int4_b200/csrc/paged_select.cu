// The blocks a request's new token attends to (include/flashloop_paged.h: fl_paged_select).
//
// score(block) = max over the group's queries of sum_c max(q_c lo_c, q_c hi_c), with lo = z
// and hi = z + 15 s of the record's key groups: the largest q.k any key of the block could
// have, from 512 of the record's 9216 bytes.  Two launches, the second one's start overlapped:
//   score_kernel  sum_c max(q lo, q hi) = sum_c q lo + 15 max(q, 0) s as two fp64 matrix
//                 products, 8 blocks x 8 queries at a time.  Every product is exact (8 or 12
//                 significant bits times 11), so scores of equal blocks are equal and the
//                 order is the definition's but for differences of a few 1e-16.
//                 A binary16 number becomes an fp64 one by moving its bits (no conversion
//                 instruction, which the SM issues at a quarter of this rate): the exponent
//                 keeps its bias, which scales the number by 2^-1008, subnormals included;
//                 the queries carry 2^500 of that and the sum the rest.
//   topk          on the scores' 64-bit images, from the highest bit in which they differ:
//                 up to 256 blocks a warp per (entry, head) with every key in registers and
//                 one count a bit, until exactly k keys are left above; beyond, one CTA per
//                 (entry, head) and a radix select, ten bits a pass.
// Measured (a launch alone, cold caches): scores 23 us and top-k 7.2 for 16 requests of 32768, 8 x 4
// heads (34 MB in pieces of 512 bytes, 1.5 TB/s, the fp64 matrix unit 43 % busy: its instructions
// and the trips to memory bound it), 7.3 and 7.2 for one of 32768, 16 heads, 9.9 and 5.7 for 64 of
// up to 8191, 4 x 8 heads (latency).
#include "paged.cuh"

namespace fl {
namespace {

constexpr int kST = 256;   // threads of the score kernel: 8 blocks a warp
constexpr int kChunk = 64; // blocks it takes at a time
constexpr int kTT = 256;   // threads of the top-k kernel
constexpr int kDigit = 10;

__device__ __forceinline__ unsigned long long score_image(double v) {
  if (v != v) return 0ull;  // NaN ranks below everything
  const long long b = __double_as_longlong(v + 0.0);
  return (unsigned long long)(b < 0 ? ~b : b | (long long)0x8000000000000000ull);
}

// c += a b for 8 x 4 by 4 x 8: lane (i, j) holds a[i][j], b[j][i], c[i][2 j], c[i][2 j + 1].
__device__ __forceinline__ void mma_f64(double (&c)[2], double a, double b) {
  asm("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};" : "+d"(c[0]), "+d"(c[1]) : "d"(a), "d"(b));
}

// Eight queries of a group at a time (its last one is repeated to fill them).  A CTA takes an
// equal, consecutive share of the chunks of 64 blocks, so that it stages the queries of an
// (entry, head) once.  A record's words are replaced by the next chunk's as the products use them
// up, and the page numbers of the chunk after that are on their way: loads issued in one go kept
// the warps from computing until the memory system had taken them all.  Lane (i, j) reads channels 16 m + 4 j + t of
// block i, and these are the columns of product (m, t).
__global__ void __launch_bounds__(kST, 2) score_kernel(PagedAttnArgs a) {
  extern __shared__ int32_t prefix[];
  __shared__ int red[kST / 32];
  // per product pair (m, t / 2) and lane: 2^500 q, and 2^500 15 max(q, 0), of channels t, t + 1
  __shared__ double2 s_q[2][16][32];
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x, lane = tid & 31, i = lane >> 2, j = lane & 3, heads = a.p.kv_heads;
  const fl_paged_index& x = a.x;
  const bool tell = blockIdx.x == 0;
  const int total = paged_scan<kST>(a.batch, prefix, red, [&](int b) {
    const int s = paged_slot(x, a.slots, b, tell);
    if (s < 0) return 0;
    const int full = paged_full(paged_length(x, s, b, tell));
    return full > a.keep ? (full + kChunk - 1) / kChunk * heads : 0;
  });
  int w = (int)((int64_t)total * blockIdx.x / gridDim.x);
  const int end = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
  if (w >= end) return;

  struct At {
    int b, h, c, chunks, slot, full;  // entry, head, chunk of its blocks
  };
  auto enter = [&](At& p, int b) {
    p.b = b;
    p.slot = paged_slot(x, a.slots, b, false);
    p.full = paged_full(paged_length(x, p.slot, b, false));
    p.chunks = (p.full + kChunk - 1) / kChunk;
  };
  auto next = [&](At& p) {
    if (++p.c < p.chunks) return;
    p.c = 0;
    if (++p.h < heads) return;
    p.h = 0;
    int b = p.b + 1;
    while (b < a.batch && prefix[b + 1] == prefix[b]) ++b;
    if (b < a.batch) enter(p, b);
  };
  auto page_of = [&](const At& p) {
    const int block = p.c * kChunk + (tid >> 2);
    if (block >= p.full) return -1;
    const int page = ld(x.table + (int64_t)p.slot * x.max_pages + block);
    if (page >= 0 && page < x.pages) return page;
    if (j == 0) paged_error(x, FL_DEV_PAGE_RANGE, p.b);
    return -1;
  };
  auto scales = [&](const At& p, int page) { return a.p.rec + ((size_t)max(page, 0) * heads + p.h) * kRec + kRecKsz + 16 * j; };
  At cur, ahead;
  enter(cur, paged_find(prefix, a.batch, w));
  cur.h = (w - prefix[cur.b]) / cur.chunks;
  cur.c = (w - prefix[cur.b]) % cur.chunks;
  ahead = cur;
  int page = page_of(cur), page1 = -1;
  if (w + 1 < end) {
    next(ahead);  // ahead is the chunk behind the current one
    page1 = page_of(ahead);
  }
  uint4 sz[8];
#pragma unroll
  for (int m = 0; m < 8; ++m) sz[m] = ld_u4(scales(cur, page) + 64 * m);
  int staged_b = -1, staged_h = -1;
  for (; w < end; ++w) {
    At after = ahead;
    int page2 = -1;
    const uint8_t* rec1 = w + 1 < end ? scales(ahead, page1) : nullptr;
    if (w + 2 < end) {
      next(after);
      page2 = page_of(after);
    }
    // infinite or NaN scales and zeros (exponent 31) carry into the halves' top bits; such a
    // block, or one that cannot be read, ranks last
    uint32_t over = page < 0 ? 0x80008000u : 0u;
    bool nan = false;
    double best = -INFINITY;
    for (int g0 = 0; g0 < a.group; g0 += 8) {
      if (a.group > 8 || cur.b != staged_b || cur.h != staged_h) {
        __syncthreads();
        for (int y = tid; y < 1024; y += kST) {  // query y / 128, channel y % 128
          const int g = min(g0 + (y >> 7), a.group - 1), ch = y & 127;
          const uint16_t q = a.q[(int64_t)cur.b * a.q_batch_stride + (int64_t)(cur.h * a.group + g) * a.q_head_stride + ch];
          const double v = (double)__uint_as_float((uint32_t)q << 16) * 0x1p500;
          double* to = &s_q[0][ch >> 4 << 1 | (ch >> 1 & 1)][(y >> 7) << 2 | (ch >> 2 & 3)].x + (ch & 1);
          to[0] = v;
          to[2 * 16 * 32] = v > 0.0 ? 15.0 * v : 0.0;
        }
        staged_b = cur.b;
        staged_h = cur.h;
        __syncthreads();
      }
      double sum[4][2] = {};  // four chains of 16 products
#pragma unroll
      for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int t = 0; t < 4; t += 2) {
          const double2 q = s_q[0][2 * m + t / 2][lane], p = s_q[1][2 * m + t / 2][lane];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t v = (&sz[m].x)[t + y];
            asm volatile("" : "+r"(v));  // widened here each time: 128 registers more if hoisted out of the loop
            mma_f64(sum[2 * y], __hiloint2double((int)(((v >> 6) & 0x01fffc00u) | (v & 0x80000000u)), 0), y ? q.y : q.x);
            mma_f64(sum[2 * y + 1], __hiloint2double((int)((v & 0x7fffu) << 10), 0), y ? p.y : p.x);
            over |= (v & 0x7fff7fffu) + 0x04000400u;
          }
          if (t == 2 && rec1 && g0 + 8 >= a.group) sz[m] = ld_u4(rec1 + 64 * m);
        }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const double v = ((sum[0][y] + sum[1][y]) + (sum[2][y] + sum[3][y])) * 0x1p508;
        nan |= v != v;
        best = fmax(best, v);
      }
    }
    // the block's best over the four lanes of its queries
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) best = fmax(best, __shfl_xor_sync(kFull, best, o));
    const bool bad = (__ballot_sync(kFull, nan || (over & 0x80008000u)) >> (4 * i)) & 15u;
    const int block = cur.c * kChunk + (tid >> 2);
    if (j == 0 && block < cur.full)
      (static_cast<unsigned long long*>(a.data) + ((size_t)cur.b * heads + cur.h) * x.max_pages)[block] = bad ? 0ull : score_image(best);
    cur = ahead;
    ahead = after;
    page = page1;
    page1 = page2;
  }
}

constexpr int kWarpKeys = 8;

// A warp per (entry, head) with at most 32 kWarpKeys blocks: lane l holds keys 32 y + l.
__global__ void __launch_bounds__(128) topk_warp_kernel(PagedAttnArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, heads = a.p.kv_heads, k = a.keep;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (int64_t)a.batch * heads) return;
  const int b = (int)(row / heads);
  const fl_paged_index& x = a.x;
  const int s = paged_slot(x, a.slots, b, false);
  if (s < 0) return;
  const int n = paged_full(paged_length(x, s, b, false));
  int32_t* sel = a.sel + row * k;
  if (n <= k) {
    for (int i = lane; i < k; i += 32) sel[i] = i < n ? i : -1;
    return;
  }
  const unsigned long long* from = static_cast<const unsigned long long*>(a.data) + row * x.max_pages;
  unsigned long long key[kWarpKeys];
  unsigned long long lo = ~0ull, hi = 0ull;
#pragma unroll
  for (int y = 0; y < kWarpKeys; ++y) {
    const int i = 32 * y + lane;
    key[y] = i < n ? __ldcg(from + i) : 0ull;
  }
#pragma unroll
  for (int y = 0; y < kWarpKeys; ++y) {
    lo = 32 * y + lane < n ? min(lo, key[y]) : lo;
    hi = max(hi, key[y]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(kFull, lo, o));
    hi = max(hi, __shfl_xor_sync(kFull, hi, o));
  }
  // `floor`: the largest number so far that at least k keys reach (entries behind the last key
  // are 0, below every floor > lo); bit by bit
  int bit = lo == hi ? -1 : 63 - __clzll((long long)(lo ^ hi));
  unsigned long long floor = bit < 0 ? lo : bit == 63 ? 0ull : hi & (~0ull << (bit + 1));
  int reach = n;
  for (; bit >= 0 && reach != k; --bit) {
    const unsigned long long t = floor | 1ull << bit;
    int c = 0;
#pragma unroll
    for (int y = 0; y < kWarpKeys; ++y) c += key[y] >= t;
    c = __reduce_add_sync(kFull, c);
    if (c >= k) {
      floor = t;
      reach = c;
    }
  }
  // exactly k reach it; or, where keys are equal, the first of those
  int above = 0;
  if (reach != k) {
    int c = 0;
#pragma unroll
    for (int y = 0; y < kWarpKeys; ++y) c += key[y] > floor;
    above = __reduce_add_sync(kFull, c);
  }
  int equal = reach != k ? k - above : 0, at = 0;  // how many of the keys equal to it to take
#pragma unroll
  for (int y = 0; y < kWarpKeys; ++y) {
    if (32 * y >= n) break;
    const bool in = 32 * y + lane < n;
    bool take = in && (reach == k ? key[y] >= floor : key[y] > floor);
    if (reach != k) {
      const unsigned eq = __ballot_sync(kFull, in && key[y] == floor);
      take |= (eq >> lane & 1u) && __popc(eq & ((1u << lane) - 1u)) < equal;
      equal -= min(equal, __popc(eq));
    }
    const unsigned taken = __ballot_sync(kFull, take);
    if (take) sel[at + __popc(taken & ((1u << lane) - 1u))] = 32 * y + lane;
    at += __popc(taken);
  }
}

// A CTA per (entry, head): the k-th largest of n > k keys digit by digit.
__global__ void __launch_bounds__(kTT) topk_kernel(PagedAttnArgs a) {
  __shared__ unsigned hist[1 << kDigit];
  __shared__ unsigned long long s_lo[kTT / 32], s_hi[kTT / 32];
  __shared__ int red[kTT / 32];
  __shared__ int s_digit, s_above, s_count;
  const int h = blockIdx.x, b = blockIdx.y, heads = a.p.kv_heads, k = a.keep;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const fl_paged_index& x = a.x;
  grid_dep_launch();
  grid_dep_wait();
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
    const unsigned long long u = __ldcg(key + i);
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
    for (int i = tid; i < n; i += kTT) {
      const unsigned long long u = __ldcg(key + i);
      if ((u & known) == prefix) atomicAdd(&hist[(unsigned)(u >> shift) & dmask], 1u);
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
  for (int i0 = 0; i0 < n; i0 += kTT) {
    const int i = i0 + tid;
    const unsigned long long m = i < n ? __ldcg(key + i) & known : 0ull;
    const bool gt = i < n && m > prefix, eq = i < n && m == prefix;
    int total;
    const int before = paged_block_scan<kTT>((gt ? 1 << 16 : 0) | (eq ? 1 : 0), red, total);
    const int g = gt_run + (before >> 16), e = eq_run + (before & 0xffff);
    if (gt || (eq && e < krem)) sel[g + min(e, krem)] = i;
    gt_run += total >> 16;
    eq_run += total & 0xffff;
  }
}

std::atomic<bool> g_attr_done[kMaxDevices];
std::mutex g_attr_mu;

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
    // the queries and the offsets of the largest batches together pass what a launch has unasked
    const cudaError_t r = once_per_device(g_attr_done, g_attr_mu, [](int) {
      return cudaFuncSetAttribute(score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (FL_PAGED_MAX_BATCH + 1) * 4);
    });
    if (r != cudaSuccess) return r;
    const int64_t items = (int64_t)a.batch * ((a.x.max_pages + kChunk - 1) / kChunk) * a.p.kv_heads;
    const int grid = (int)(items < 2 * sms ? items : 2 * sms);
    const cudaError_t e = launch_pdl(score_kernel, dim3(grid), dim3(kST), (size_t)(a.batch + 1) * 4, s, a);
    if (e != cudaSuccess) return e;
  }
  // What a request can have decides, not what it has: lengths are the device's.  By kernel time:
  // up to 256 blocks a warp 5.7 us, the CTA 7.4; 511 blocks a warp (16 keys a lane) 7.9, the CTA 7.0.
  const int most = a.x.max_pages - 1;
  const unsigned grid = (unsigned)(((int64_t)a.batch * a.p.kv_heads + 3) / 4);
  if (most <= 32 * kWarpKeys || !scored) return launch_pdl(topk_warp_kernel, dim3(grid), dim3(128), 0, s, a);
  return launch_pdl(topk_kernel, dim3(a.p.kv_heads, a.batch), dim3(kTT), 0, s, a);
}

}  // namespace fl
