// Shared pieces of the paged cache's kernels (include/flashloop_paged.h): argument structs,
// launchers, and the map from a flat work index to (batch entry, unit) over ragged lengths.
#pragma once

#include "flashloop_paged.h"
#include "kernels.h"

namespace fl {

struct PagedAppendArgs {
  fl_paged_index x;
  fl_paged_pool p;
  int batch, n_tokens;
  const int32_t *slots, *start, *cu;
  const uint16_t *k, *v;
  int64_t token_stride, head_stride;
};

struct PagedReadArgs {
  fl_paged_index x;
  fl_paged_pool p;
  int n_tokens;
  const int32_t* place;
  uint16_t *k, *v;
  int64_t token_stride, head_stride;
};

struct PagedAttnArgs {
  fl_paged_index x;
  fl_paged_pool p;
  int batch, q_heads, group, keep;
  const int32_t* slots;
  const uint16_t* q;
  int64_t q_batch_stride, q_head_stride;
  int32_t* sel;  // read by the attention, written by the selection
  float* o;
  int64_t o_batch_stride, o_head_stride;
  float* lse;
  int32_t* tickets;  // FL_PAGED_WS_HEAD bytes, zero between calls
  void* data;        // the workspace behind them
};

cudaError_t launch_paged_index_init(const fl_paged_index& x, cudaStream_t s);
cudaError_t launch_paged_extend(const fl_paged_index& x, int batch, const int32_t* slots, const int32_t* n_new,
                                int32_t* start, int32_t* cu, cudaStream_t s);
cudaError_t launch_paged_release(const fl_paged_index& x, int batch, const int32_t* slots, cudaStream_t s);
cudaError_t launch_paged_slot_map(const fl_paged_index& x, int batch, const int32_t* slots, const int32_t* start,
                                  const int32_t* cu, int n_tokens, int32_t* place, int32_t* pos, cudaStream_t s);
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s);
cudaError_t launch_paged_read(const PagedReadArgs& a, cudaStream_t s);
cudaError_t launch_paged_select(const PagedAttnArgs& a, cudaStream_t s);
cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s);
// Bytes of the workspace's data part that each needs.
uint64_t paged_select_bytes(const fl_paged_index& x, const fl_paged_pool& p, int batch);
uint64_t paged_attn_bytes(const fl_paged_pool& p, int q_heads);

// Plain loads.  These kernels start while their predecessor is still writing what they will read
// once they have waited for it (programmatic launch), so nothing they read may go through the
// read-only path, which wants data that no one writes while the kernel runs.
template <class T>
__device__ __forceinline__ T ld(const T* p) {
  return *p;
}
__device__ __forceinline__ uint4 ld_u4(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// Blocks of a request of n tokens that are records.
__host__ __device__ __forceinline__ int paged_full(int n) { return n > 0 ? (n - 1) >> 6 : 0; }

__device__ __forceinline__ void paged_error(const fl_paged_index& x, int code, int detail) {
  if (x.status) record_error(x.status, code, detail);
}

// The table row of batch entry b, or -1 for a padded entry or one out of range (recorded
// when `tell`).
__device__ __forceinline__ int paged_slot(const fl_paged_index& x, const int32_t* slots, int b, bool tell) {
  const int s = slots ? ld(slots + b) : b;
  if (s >= 0 && s < x.slots) return s;
  if (s != -1 && tell) paged_error(x, FL_DEV_SLOT_RANGE, b);
  return -1;
}

// A request's length, 0 where it is outside the table row's capacity (recorded when `tell`).
__device__ __forceinline__ int paged_length(const fl_paged_index& x, int slot, int b, bool tell) {
  const int n = x.length[slot];
  if (n >= 0 && n <= x.max_pages * FL_PAGE) return n;
  if (tell) paged_error(x, FL_DEV_TOO_LONG, b);
  return 0;
}

// Exclusive prefix sum of one value per thread of a block of kThreads threads; `red` holds
// kThreads / 32 words; `total` receives the sum.
template <int kThreads>
__device__ __forceinline__ int paged_block_scan(int v, int* red, int& total) {
  constexpr int kW = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    const int r = red[w];
    if (w < warp) before += r;
    sum += r;
  }
  total = sum;
  __syncthreads();
  return before + x - v;
}

// prefix[b] = units of the entries before b, prefix[batch] = their total (returned): every
// thread of the block takes part.
template <int kThreads, class F>
__device__ __forceinline__ int paged_scan(int batch, int32_t* prefix, int* red, F&& units) {
  int run = 0;
  for (int b0 = 0; b0 < batch; b0 += kThreads) {
    const int b = b0 + (int)threadIdx.x;
    const int u = b < batch ? units(b) : 0;
    int total;
    const int before = paged_block_scan<kThreads>(u, red, total);
    if (b < batch) prefix[b] = run + before;
    run += total;
  }
  if (threadIdx.x == 0) prefix[batch] = run;
  __syncthreads();
  return run;
}

// The entry that unit i (0 <= i < prefix[batch]) belongs to.
__device__ __forceinline__ int paged_find(const int32_t* prefix, int batch, int i) {
  int lo = 0, hi = batch;  // prefix[lo] <= i < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace fl
