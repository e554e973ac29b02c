// Block tables, lengths, free pages and slot maps of the paged cache, from request lengths
// on the GPU (include/flashloop_paged.h): no length ever goes to the host.
//
// A request of c tokens owns ceil(c / 64) pages.  extend: need_i = ceil((c_i + n_i) / 64) -
// ceil(c_i / 64); with P_i the sum of need over the valid entries up to i, entry i is granted
// when need_i = 0 or P_i <= n_free, and its pages are free[n_free - 1 - (P_i - need_i) - j].
// The granted entries that need pages are a prefix of the valid ones that do, so the stack
// simply loses its top P and every entry's place on it is P_i - need_i.  The work is a scan over
// at most 8192 entries and 8 bytes per page, and its time is the launch and four dependent trips
// to memory.  Up to 128 entries of not too many pages one block of 128 threads does it (whose
// barriers cost half of 1024 threads': 64 decode steps with their slot map 5.7 us on the device in
// a table of 256 columns, 6.7 by the cluster in one of 8192), else a cluster of eight blocks that share
// the moving of the pages out (512 requests of up to 8192 tokens leave and as many come, with their slot
// map: 15.4 us; when the size was chosen 14.4 in blocks of 512 threads, 16.4 of 1024, 19.4 of 256,
// and 25.4 in one block of 1024 threads).  The kernels here start while their
// predecessor ends (programmatic launch) and wait for it before they touch memory.
#include "paged.cuh"

namespace fl {
namespace {

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
template <int kT>
struct Claims {
  uint32_t* bits;
  int32_t* slot;  // [kT] of this chunk

  // Before the first chunk; the caller's next barrier comes before any use.
  __device__ void clear(int slots) {
    for (int i = threadIdx.x; i < (slots + 31) / 32; i += kT) bits[i] = 0u;
  }
  // True for the entry that names its slot first (s < 0: no slot); all threads call it, one
  // chunk of kT entries after the other.
  __device__ bool first(int s) {
    const uint32_t bit = s >= 0 ? 1u << (s & 31) : 0u;
    __syncthreads();
    const bool earlier = s >= 0 && (bits[s >> 5] & bit);
    slot[threadIdx.x] = s;
    __syncthreads();
    const bool twice = s >= 0 && (atomicOr(&bits[s >> 5], bit) & bit);
    bool mine = s >= 0 && !earlier;
    if (__syncthreads_or(twice && !earlier)) {
      // rare: some slot stands twice in this chunk, the first one counts
      for (int i = 0; i < (int)threadIdx.x && mine; ++i) mine = slot[i] != s;
    }
    return mine;
  }
};

// A chunk's tokens and pages are summed in one number, pages from this bit on: 512 entries of less
// than 2^31 tokens, refused ones among them, stay below it, and their 2^14 pages each in the rest.
constexpr int kPageBit = 40, kChunkMost = 512;
constexpr uint64_t kTokens = ((uint64_t)1 << kPageBit) - 1;

// Exclusive prefix sum of one such number per thread.
template <int kT>
__device__ __forceinline__ uint64_t scan_pair(uint64_t v, uint64_t* red, uint64_t& total) {
  static_assert(kT <= kChunkMost, "a chunk's tokens would reach its pages");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kT / 32; ++w) {
    const uint64_t r = red[w];
    before += w < warp ? r : 0;
    total += r;
  }
  __syncthreads();
  return before + x - v;
}

// One chunk's pages to move: entry t's are jobs [before[t], before[t + 1]), page j of them goes
// with block block0[t] + (job) of its slot.  Four jobs a thread are in flight at once.
template <int kT>
struct Jobs {
  int32_t before[kT + 1], slot[kT], block0[kT];

  // thread `first` of `kAll`
  template <int kAll, class F>
  __device__ void run(int first, F&& move) const {
    const int n = before[kT];
    for (int i0 = first; i0 < n; i0 += 4 * kAll) {
      int t[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) t[y] = i0 + y * kAll < n ? paged_find(before, kT, i0 + y * kAll) : -1;
      move(t, i0);
    }
  }
};

// A cluster's CTAs all take the same steps over the entries; each moves its share of the pages,
// and the first one alone writes what the others read (lengths, the count of free pages),
// once all have read it.
template <int kCtas>
__device__ __forceinline__ void cluster_arrive() {
  if constexpr (kCtas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
template <int kCtas>
__device__ __forceinline__ void cluster_wait() {
  if constexpr (kCtas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Whether any CTA of the cluster says so.  `flag`: 0 in every CTA since before a cluster barrier.
// Where none does, the usual case, nothing waits for the CTAs' stores (512 requests out and in:
// 16.0 us a call, 16.4 with an ordered arrival); where one does, their writes are ordered.
template <int kCtas>
__device__ __forceinline__ bool cluster_any(bool mine, int* flag) {
  if constexpr (kCtas == 1) return mine;
  if (mine && (int)threadIdx.x < kCtas) {
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_addr(flag)), "r"(threadIdx.x));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(1) : "memory");
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  cluster_wait<kCtas>();
  if (!*reinterpret_cast<volatile int*>(flag)) return false;
  cluster_arrive<kCtas>();
  cluster_wait<kCtas>();
  return true;
}

template <int kT, int kCtas>
__global__ void __launch_bounds__(kT) extend_kernel(fl_paged_index x, int batch, const int32_t* slots,
                                                    const int32_t* n_new, int32_t* start, int32_t* cu) {
  extern __shared__ uint32_t s_bits[];
  __shared__ int32_t s_slot[kT];
  __shared__ uint64_t red[kT / 32];
  __shared__ int s_taken;
  __shared__ Jobs<kT> jobs;
  constexpr int kAll = kT * kCtas;
  const int tid = threadIdx.x, rank = kCtas > 1 ? (int)blockIdx.x : 0;
  const bool tell = rank == 0;
  Claims<kT> claims{s_bits, s_slot};
  claims.clear(x.slots);
  if (tid == 0) s_taken = 0;
  grid_dep_launch();
  grid_dep_wait();
  const int n_free = min(max(*x.n_free, 0), x.pages);
  int64_t rows = 0;  // of the chunks before
  int base = 0;      // pages that they need (2^27 at most)
  for (int b0 = 0; b0 < batch; b0 += kT) {
    const int b = b0 + tid;
    int s = -1, n = 0, c = 0, need = 0;
    if (b < batch) {
      n = n_new[b];
      s = paged_slot(x, slots, b, tell);
      if (s >= 0) c = x.length[s];
    }
    __syncwarp();
    cluster_arrive<kCtas>();
    const bool named = s >= 0, mine = claims.first(s);
    if (named && !mine && tell) paged_error(x, FL_DEV_SLOT_TWICE, b);
    if (!mine) s = -1;
    if (s >= 0 && n < 0) {
      if (tell) paged_error(x, FL_DEV_COUNT, b);
      s = -1;
    }
    if (s >= 0) {
      if (c < 0 || (int64_t)c + n > (int64_t)x.max_pages * FL_PAGE) {
        if (tell) paged_error(x, FL_DEV_TOO_LONG, b);
        s = -1;
      } else {
        need = ((c + n + FL_PAGE - 1) >> 6) - ((c + FL_PAGE - 1) >> 6);
      }
    }
    uint64_t total;
    const uint64_t before = scan_pair<kT>((uint64_t)need << kPageBit | (uint32_t)max(n, 0), red, total);
    const int at = base + (int)(before >> kPageBit);
    const int64_t row0 = rows + (int64_t)(before & kTokens);
    // rows that offsets cannot name: this entry is refused, and so is all behind it that has rows
    // (so that the pages it would have needed hold up none that is granted)
    const bool counted = n <= 0 || row0 + n <= INT32_MAX;
    const bool granted = s >= 0 && counted && (need == 0 || at + need <= n_free);
    if (s >= 0 && !granted && tell) paged_error(x, counted ? FL_DEV_NO_PAGE : FL_DEV_COUNT, b);
    __syncwarp();
    cluster_wait<kCtas>();
    if (b < batch && tell) {
      start[b] = granted ? c : -1;
      cu[b] = (int)min(row0, (int64_t)INT32_MAX);
    }
    if (granted && tell) x.length[s] = c + n;
    const int count = granted ? need : 0;
    if (count > 0) atomicMax(&s_taken, at + count);
    const int block0 = (c + FL_PAGE - 1) >> 6;
    if (!__syncthreads_or(count > 1)) {
      // a decode step: a page a request at most
      if (count == 1 && (tid >> 5) % kCtas == rank) x.table[(int64_t)s * x.max_pages + block0] = x.free_pages[n_free - 1 - at];
    } else {
      // the granted entries' pages lie one behind the other on the stack, from `base` on
      const int taken = max(s_taken - base, 0);
      jobs.before[tid] = min(at - base, taken);
      jobs.slot[tid] = s;
      jobs.block0[tid] = block0 - (at - base);
      if (tid == 0) jobs.before[kT] = taken;
      __syncthreads();
      jobs.template run<kAll>(rank * kT + tid, [&](const int (&t)[4], int i0) {
        int page[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) page[y] = t[y] >= 0 ? x.free_pages[n_free - 1 - base - (i0 + y * kAll)] : 0;
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (t[y] >= 0) x.table[(int64_t)jobs.slot[t[y]] * x.max_pages + jobs.block0[t[y]] + i0 + y * kAll] = page[y];
      });
      __syncthreads();
    }
    rows += (int64_t)(total & kTokens);
    base += (int)(total >> kPageBit);
  }
  __syncthreads();
  if (tid == 0 && tell) {
    cu[batch] = (int)min(rows, (int64_t)INT32_MAX);
    *x.n_free = n_free - s_taken;
  }
}

template <int kT, int kCtas>
__global__ void __launch_bounds__(kT) release_kernel(fl_paged_index x, int batch, const int32_t* slots) {
  extern __shared__ uint32_t s_bits[];
  __shared__ int32_t s_slot[kT];
  __shared__ uint64_t red[kT / 32];
  __shared__ Jobs<kT> jobs;
  __shared__ int s_bad;  // a table entry was no page
  constexpr int kAll = kT * kCtas;
  const int tid = threadIdx.x, rank = kCtas > 1 ? (int)blockIdx.x : 0;
  const bool tell = rank == 0;
  Claims<kT> claims{s_bits, s_slot};
  claims.clear(x.slots);
  if (tid == 0) s_bad = 0;
  grid_dep_launch();
  grid_dep_wait();
  const int n_free = min(max(*x.n_free, 0), x.pages);
  uint64_t given = 0;  // 2^27 at most
  bool bad = false;
  for (int b0 = 0; b0 < batch; b0 += kT) {
    const int b = b0 + tid;
    const int s = b < batch ? paged_slot(x, slots, b, tell) : -1;
    int count = s >= 0 ? (paged_length(x, s, b, tell) + FL_PAGE - 1) >> 6 : 0;
    __syncwarp();
    cluster_arrive<kCtas>();
    const bool mine = claims.first(s);
    if (s >= 0 && !mine && tell) paged_error(x, FL_DEV_SLOT_TWICE, b);
    if (!mine) count = 0;
    uint64_t total;
    const int at = (int)scan_pair<kT>((uint64_t)count, red, total);
    cluster_wait<kCtas>();
    if (mine && tell) x.length[s] = 0;
    jobs.before[tid] = at;
    jobs.slot[tid] = s;
    jobs.block0[tid] = -at;
    if (tid == 0) jobs.before[kT] = (int)total;
    __syncthreads();
    const int64_t top = n_free + (int64_t)given;
    jobs.template run<kAll>(rank * kT + tid, [&](const int (&t)[4], int i0) {
      int page[4];
      int32_t* e[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if (t[y] < 0) continue;
        e[y] = x.table + (int64_t)jobs.slot[t[y]] * x.max_pages + jobs.block0[t[y]] + i0 + y * kAll;
        page[y] = *e[y];
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if (t[y] < 0) continue;
        const int64_t to = top + i0 + y * kAll;
        *e[y] = -1;
        // a stack that would grow beyond `pages` has been handed pages that are free already
        const bool none = page[y] < 0 || page[y] >= x.pages;
        if (none || to >= x.pages) paged_error(x, FL_DEV_PAGE_RANGE, b0 + t[y]);
        bad |= none;
        if (to < x.pages) x.free_pages[to] = page[y];
      }
    });
    __syncthreads();
    given += total;
  }
  bad = cluster_any<kCtas>(__syncthreads_or(bad), &s_bad);
  if (!tell) return;
  int n = (int)min((int64_t)n_free + (int64_t)given, (int64_t)x.pages);
  if (bad) {
    // rare: what is no page must not be granted to another request, so it leaves the stack's new part
    int kept = n_free;
    for (int i0 = n_free; i0 < n; i0 += kT) {
      const int i = i0 + tid, page = i < n ? __ldcg(x.free_pages + i) : -1;
      const bool good = page >= 0 && page < x.pages;
      uint64_t total;
      const int at = (int)scan_pair<kT>(good ? 1 : 0, red, total);  // (its barriers part reads and writes)
      if (good) x.free_pages[kept + at] = page;
      kept += (int)total;
    }
    n = kept;
  }
  if (tid == 0) *x.n_free = n;
}

// Four consecutive rows a thread; the offsets are searched in shared memory where they fit.
constexpr int kMapT = 256, kMapRows = 4, kMapHeld = 2048;

__global__ void __launch_bounds__(kMapT) slot_map_kernel(fl_paged_index x, int batch, const int32_t* slots,
                                                         const int32_t* start, const int32_t* cu, int n_tokens,
                                                         int32_t* place, int32_t* pos, int vec) {
  __shared__ int32_t s_cu[kMapHeld + 1];
  grid_dep_launch();
  grid_dep_wait();
  const bool held = batch <= kMapHeld;
  if (held) {
    for (int i = threadIdx.x; i <= batch; i += kMapT) s_cu[i] = cu[i];
    __syncthreads();
  }
  const int32_t* off = held ? s_cu : cu;
  const int t0 = (blockIdx.x * kMapT + threadIdx.x) * kMapRows;
  const int begin = off[0], end = min(off[batch], n_tokens);
  // (the last rows of 2^31 - 1: the thread's end is no number of 32 bits)
  if ((int64_t)t0 + kMapRows <= begin || t0 >= end) return;
  int at[kMapRows], where[kMapRows];
  int b = -1, first = 0, last = -1;  // rows [first, last) are entry b's
  int s = -1, from = -1, n = 0, full = 0;
#pragma unroll
  for (int y = 0; y < kMapRows; ++y) {
    const int t = t0 + y;
    at[y] = where[y] = -1;
    if (t < begin || t >= end) continue;
    if (t >= last || t < first) {
      int lo = 0, hi = batch;  // off[lo] <= t < off[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= t) lo = mid;
        else hi = mid;
      }
      b = lo;
      first = off[b];
      last = off[b + 1];
      s = paged_slot(x, slots, b, t == first);
      from = start[b];
      n = s >= 0 ? paged_length(x, s, b, t == first) : 0;
      full = paged_full(n);
    }
    if (s < 0 || from < 0 || from > INT32_MAX - (t - first)) continue;
    at[y] = from + (t - first);
    if (at[y] >= n) continue;
    const int block = at[y] >> 6;
    int page = x.pages + s;
    if (block < full) {
      page = x.table[(int64_t)s * x.max_pages + block];
      if (page < 0 || page >= x.pages) {
        paged_error(x, FL_DEV_PAGE_RANGE, b);
        continue;
      }
    }
    where[y] = page * FL_PAGE + (at[y] & 63);
  }
  if (vec && t0 >= begin && (int64_t)t0 + kMapRows <= end) {
    if (place) *reinterpret_cast<int4*>(place + t0) = make_int4(where[0], where[1], where[2], where[3]);
    if (pos) *reinterpret_cast<int4*>(pos + t0) = make_int4(at[0], at[1], at[2], at[3]);
    return;
  }
#pragma unroll
  for (int y = 0; y < kMapRows; ++y) {
    if (t0 + y < begin || t0 + y >= end) continue;
    if (place) place[t0 + y] = where[y];
    if (pos) pos[t0 + y] = at[y];
  }
}

// Threads of a CTA for few entries and for more, and CTAs of the cluster.
constexpr int kSmall = 128, kLarge = 512, kCluster = 8;
// Few entries take the cluster where they could have more pages than this.  It costs an extend
// and a release 1 us each (64 requests, one token: 3.9 us together, 5.9 as clusters) and saves
// 50 us for 128 x 8192 tokens (60.5, 10.0) and 390 for 128 x 32768 (412, 22.9).  An extend is
// called for every token, mostly without a page to move; a release once a request.
constexpr int kExtendPages = 16384, kReleasePages = 256;

// launch_pdl of one cluster of `ctas`
template <class... KArgs, class... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int ctas, int threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

}  // namespace

cudaError_t launch_paged_index_init(const fl_paged_index& x, cudaStream_t s) {
  index_init_kernel<<<296, 256, 0, s>>>(x);
  return cudaGetLastError();
}

cudaError_t launch_paged_extend(const fl_paged_index& x, int batch, const int32_t* slots, const int32_t* n_new,
                                int32_t* start, int32_t* cu, cudaStream_t s) {
  const size_t bits = (size_t)(x.slots + 31) / 32 * 4;
  if (batch <= kSmall && (int64_t)batch * x.max_pages <= kExtendPages)
    return launch_pdl(extend_kernel<kSmall, 1>, dim3(1), dim3(kSmall), bits, s, x, batch, slots, n_new, start, cu);
  return launch_cluster(extend_kernel<kLarge, kCluster>, kCluster, kLarge, bits, s, x, batch, slots, n_new, start, cu);
}

cudaError_t launch_paged_release(const fl_paged_index& x, int batch, const int32_t* slots, cudaStream_t s) {
  const size_t bits = (size_t)(x.slots + 31) / 32 * 4;
  if (batch <= kSmall && (int64_t)batch * x.max_pages <= kReleasePages)
    return launch_pdl(release_kernel<kSmall, 1>, dim3(1), dim3(kSmall), bits, s, x, batch, slots);
  return launch_cluster(release_kernel<kLarge, kCluster>, kCluster, kLarge, bits, s, x, batch, slots);
}

cudaError_t launch_paged_slot_map(const fl_paged_index& x, int batch, const int32_t* slots, const int32_t* start,
                                  const int32_t* cu, int n_tokens, int32_t* place, int32_t* pos, cudaStream_t s) {
  if (n_tokens == 0) return cudaSuccess;
  const int vec = (reinterpret_cast<uintptr_t>(place) | reinterpret_cast<uintptr_t>(pos)) % 16 == 0;
  const unsigned grid = (unsigned)(((int64_t)n_tokens + kMapT * kMapRows - 1) / (kMapT * kMapRows));
  return launch_pdl(slot_map_kernel, dim3(grid), dim3(kMapT), 0, s, x, batch, slots, start, cu, n_tokens, place, pos, vec);
}

}  // namespace fl
