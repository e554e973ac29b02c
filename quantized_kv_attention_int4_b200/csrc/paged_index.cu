// Block tables, lengths, free pages and slot maps of the paged cache, from request lengths
// on the GPU (include/flashloop_paged.h): no length ever goes to the host.
//
// A request of c tokens owns ceil(c / 64) pages.  extend: need_i = ceil((c_i + n_i) / 64) -
// ceil(c_i / 64); with P_i the sum of need over the valid entries up to i, entry i is granted
// when need_i = 0 or P_i <= n_free, and its pages are free[n_free - 1 - (P_i - need_i) - j].
// The granted entries that need pages are a prefix of the valid ones that do, so the stack
// simply loses its top P.  One block does it: the work is a scan over at most 8192 entries
// and 8 bytes per page, and its time is the launch and four dependent trips to memory.
#include "paged.cuh"

namespace fl {
namespace {

constexpr int kT = 1024;

__global__ void index_init_kernel(fl_paged_index x) {
  const int64_t n = (int64_t)x.slots * x.max_pages, step = (int64_t)gridDim.x * blockDim.x;
  const int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t i = i0; i < n; i += step) x.table[i] = -1;
  for (int64_t i = i0; i < x.slots; i += step) x.length[i] = 0;
  for (int64_t i = i0; i < x.pages; i += step) x.free_pages[i] = x.pages - 1 - (int)i;
  if (i0 == 0) *x.n_free = x.pages;
  if (i0 < 3 && x.status) x.status[i0] = 0;
}

// One bit per slot (dynamic shared memory), set once the slot has been named.
struct Claims {
  uint32_t* bits;
  int32_t* slot;  // [kT] of this chunk

  __device__ void clear(int slots) {
    for (int i = threadIdx.x; i < (slots + 31) / 32; i += kT) bits[i] = 0u;
    __syncthreads();
  }
  // True for the entry that names its slot first (s < 0: no slot); all threads call it, one
  // chunk of kT entries after the other.
  __device__ bool first(int s) {
    const bool earlier = s >= 0 && ((bits[s >> 5] >> (s & 31)) & 1u);
    slot[threadIdx.x] = s;
    __syncthreads();
    bool twice = false;
    if (s >= 0) twice = (atomicOr(&bits[s >> 5], 1u << (s & 31)) >> (s & 31)) & 1u;
    bool mine = s >= 0 && !earlier;
    if (__syncthreads_or(twice && !earlier)) {
      // rare: some slot stands twice in this chunk, the first one counts
      for (int i = 0; i < (int)threadIdx.x && mine; ++i) mine = slot[i] != s;
      __syncthreads();
    }
    return mine;
  }
};

struct PageJobs {  // of one chunk: entry t moves pages [before[t], before[t] + count)
  int32_t before[kT + 1], slot[kT], block0[kT];
};

__global__ void __launch_bounds__(kT) extend_kernel(fl_paged_index x, int batch, const int32_t* slots,
                                                    const int32_t* n_new, int32_t* start, int32_t* cu) {
  extern __shared__ uint32_t s_bits[];
  __shared__ PageJobs jobs;
  __shared__ int32_t s_slot[kT];
  __shared__ int red[kT / 32];
  const int tid = threadIdx.x;
  Claims claims{s_bits, s_slot};
  claims.clear(x.slots);
  const int n_free = min(max(*x.n_free, 0), x.pages);
  int run_tokens = 0, run_pages = 0, taken = 0;
  for (int b0 = 0; b0 < batch; b0 += kT) {
    const int b = b0 + tid;
    int s = -1, n = 0, c = 0, need = 0;
    if (b < batch) {
      s = paged_slot(x, slots, b, true);
      n = __ldg(n_new + b);
    }
    const bool named = s >= 0;
    const bool mine = claims.first(s);
    if (named && !mine) paged_error(x, FL_DEV_SLOT_TWICE, b);
    if (!mine) s = -1;
    if (s >= 0 && n < 0) {
      paged_error(x, FL_DEV_COUNT, b);
      s = -1;
    }
    if (s >= 0) {
      c = x.length[s];
      if (c < 0 || (int64_t)c + n > (int64_t)x.max_pages * FL_PAGE) {
        paged_error(x, FL_DEV_TOO_LONG, b);
        s = -1;
      } else {
        need = ((c + n + FL_PAGE - 1) >> 6) - ((c + FL_PAGE - 1) >> 6);
      }
    }
    int total_tokens, total_pages;
    const int tok = run_tokens + paged_block_scan<kT>(max(n, 0), red, total_tokens);
    // at most FL_PAGED_MAX_BLOCKS pages an entry: 2^27 in all
    const int before = run_pages + paged_block_scan<kT>(need, red, total_pages);
    const bool granted = s >= 0 && (need == 0 || before + need <= n_free);
    if (s >= 0 && !granted) paged_error(x, FL_DEV_NO_PAGE, b);
    if (b < batch) {
      start[b] = granted ? c : -1;
      cu[b] = tok;
    }
    if (granted) x.length[s] = c + n;
    const int count = granted ? need : 0;
    int n_jobs;
    const int at = paged_block_scan<kT>(count, red, n_jobs);
    jobs.before[tid] = at;
    jobs.slot[tid] = s;
    jobs.block0[tid] = ((c + FL_PAGE - 1) >> 6) - at;
    if (tid == 0) jobs.before[kT] = n_jobs;
    __syncthreads();
    // the granted entries' pages are consecutive on the stack, from `taken` on
    for (int i = tid; i < n_jobs; i += kT) {
      const int t = paged_find(jobs.before, kT, i);
      x.table[(int64_t)jobs.slot[t] * x.max_pages + jobs.block0[t] + i] = x.free_pages[n_free - 1 - taken - i];
    }
    taken += n_jobs;
    run_tokens += total_tokens;
    run_pages += total_pages;
    __syncthreads();
  }
  if (tid == 0) {
    cu[batch] = run_tokens;
    *x.n_free = n_free - taken;
  }
}

__global__ void __launch_bounds__(kT) release_kernel(fl_paged_index x, int batch, const int32_t* slots) {
  extern __shared__ uint32_t s_bits[];
  __shared__ PageJobs jobs;
  __shared__ int32_t s_slot[kT];
  __shared__ int red[kT / 32];
  const int tid = threadIdx.x;
  Claims claims{s_bits, s_slot};
  claims.clear(x.slots);
  const int n_free = min(max(*x.n_free, 0), x.pages);
  int given = 0;
  for (int b0 = 0; b0 < batch; b0 += kT) {
    const int b = b0 + tid;
    int s = b < batch ? paged_slot(x, slots, b, true) : -1;
    const bool named = s >= 0;
    const bool mine = claims.first(s);
    if (named && !mine) paged_error(x, FL_DEV_SLOT_TWICE, b);
    int count = 0;
    if (mine) {
      count = (paged_length(x, s, b, true) + FL_PAGE - 1) >> 6;
      x.length[s] = 0;
    }
    int n_jobs;
    const int at = paged_block_scan<kT>(count, red, n_jobs);
    jobs.before[tid] = at;
    jobs.slot[tid] = s;
    jobs.block0[tid] = -at;
    if (tid == 0) jobs.before[kT] = n_jobs;
    __syncthreads();
    for (int i = tid; i < n_jobs; i += kT) {
      const int t = paged_find(jobs.before, kT, i);
      int32_t* e = x.table + (int64_t)jobs.slot[t] * x.max_pages + jobs.block0[t] + i;
      const int page = *e;
      *e = -1;
      if (page < 0 || page >= x.pages) paged_error(x, FL_DEV_PAGE_RANGE, b0 + t);
      // a stack that would grow beyond `pages` has been handed pages that are free already
      if (n_free + given + i < x.pages) x.free_pages[n_free + given + i] = page;
      else paged_error(x, FL_DEV_PAGE_RANGE, b0 + t);
    }
    given += n_jobs;
    __syncthreads();
  }
  if (tid == 0) *x.n_free = min(n_free + given, x.pages);
}

__global__ void __launch_bounds__(256) slot_map_kernel(fl_paged_index x, int batch, const int32_t* slots,
                                                       const int32_t* start, const int32_t* cu, int n_tokens,
                                                       int32_t* place, int32_t* pos) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= n_tokens || t < __ldg(cu) || t >= __ldg(cu + batch)) return;
  int lo = 0, hi = batch;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  const int s = paged_slot(x, slots, lo, t == __ldg(cu + lo));
  const int begin = __ldg(start + lo), first = __ldg(cu + lo);
  int at = -1, where = -1;
  if (s >= 0 && begin >= 0 && first >= 0 && begin <= INT32_MAX - (t - first)) {
    at = begin + (t - first);
    const int n = paged_length(x, s, lo, t == first), full = paged_full(n);
    if (at < n) {
      const int block = at >> 6;
      int page = block < full ? x.table[(int64_t)s * x.max_pages + block] : x.pages + s;
      if (page < 0 || (block < full && page >= x.pages)) {
        paged_error(x, FL_DEV_PAGE_RANGE, lo);
        page = -1;
      }
      where = page < 0 ? -1 : page * FL_PAGE + (at & 63);
    }
  }
  if (place) place[t] = where;
  if (pos) pos[t] = at;
}

}  // namespace

cudaError_t launch_paged_index_init(const fl_paged_index& x, cudaStream_t s) {
  index_init_kernel<<<296, 256, 0, s>>>(x);
  return cudaGetLastError();
}

cudaError_t launch_paged_extend(const fl_paged_index& x, int batch, const int32_t* slots, const int32_t* n_new,
                                int32_t* start, int32_t* cu, cudaStream_t s) {
  extend_kernel<<<1, kT, (size_t)(x.slots + 31) / 32 * 4, s>>>(x, batch, slots, n_new, start, cu);
  return cudaGetLastError();
}

cudaError_t launch_paged_release(const fl_paged_index& x, int batch, const int32_t* slots, cudaStream_t s) {
  release_kernel<<<1, kT, (size_t)(x.slots + 31) / 32 * 4, s>>>(x, batch, slots);
  return cudaGetLastError();
}

cudaError_t launch_paged_slot_map(const fl_paged_index& x, int batch, const int32_t* slots, const int32_t* start,
                                  const int32_t* cu, int n_tokens, int32_t* place, int32_t* pos, cudaStream_t s) {
  if (n_tokens == 0) return cudaSuccess;
  slot_map_kernel<<<(n_tokens + 255) / 256, 256, 0, s>>>(x, batch, slots, start, cu, n_tokens, place, pos);
  return cudaGetLastError();
}

}  // namespace fl
