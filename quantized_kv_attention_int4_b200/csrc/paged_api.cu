// Host side of include/flashloop_paged.h: argument validation and launches.  Nothing here
// allocates device memory or waits for the device.
#include "paged.cuh"

using namespace fl;

namespace {

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

fl_status check_index(const fl_paged_index* x) {
  if (!x || !x->table || !x->length || !x->free_pages || !x->n_free) return FL_ERR_INVALID;
  if (!aligned(x->table, 4) || !aligned(x->length, 4) || !aligned(x->free_pages, 4) || !aligned(x->n_free, 4) ||
      !aligned(x->status, 4))
    return FL_ERR_INVALID;
  if (x->slots < 1 || x->max_pages < 1 || x->pages < 1) return FL_ERR_INVALID;
  if (x->slots > FL_PAGED_MAX_SLOTS || x->max_pages > FL_PAGED_MAX_BLOCKS) return FL_ERR_UNSUPPORTED;
  // places are 32-bit
  if (((int64_t)x->pages + x->slots) * FL_PAGE > INT32_MAX) return FL_ERR_UNSUPPORTED;
  return FL_OK;
}

fl_status check_pool(const fl_paged_index* x, const fl_paged_pool* p) {
  const fl_status st = check_index(x);
  if (st != FL_OK) return st;
  if (!p || !p->rec || !p->tail_k || !p->tail_v) return FL_ERR_INVALID;
  if (p->head_dim != FL_HEAD_DIM || p->page_tokens != FL_PAGE) return FL_ERR_UNSUPPORTED;
  if (p->kv_heads < 1) return FL_ERR_INVALID;
  if (!aligned(p->rec, 16) || !aligned(p->tail_k, 16) || !aligned(p->tail_v, 16)) return FL_ERR_INVALID;
  // rows of 128 bytes are addressed with 32-bit coordinates
  if ((int64_t)x->pages * p->kv_heads * (FL_GROUP_RECORD / 128) > INT32_MAX ||
      (int64_t)x->slots * p->kv_heads * (2 * FL_PAGE) > INT32_MAX)
    return FL_ERR_UNSUPPORTED;
  return FL_OK;
}

fl_status check_batch(const fl_paged_index* x, int32_t batch, const int32_t* slots) {
  if (batch < 0 || !aligned(slots, 4)) return FL_ERR_INVALID;
  if (batch > FL_PAGED_MAX_BATCH) return FL_ERR_UNSUPPORTED;
  if (!slots && batch > x->slots) return FL_ERR_INVALID;
  return FL_OK;
}

// Strides in elements of `unit`-element rows: multiples of `unit`, none negative.
bool good_strides(int64_t a, int64_t b, int unit) { return a >= 0 && b >= 0 && a % unit == 0 && b % unit == 0; }

// Whether n0 x n1 rows of 128 elements at i s0 + j s1 lie apart from one another: outputs that
// overlap would be written by several warps at once.
bool rows_apart(int64_t n0, int64_t s0, int64_t n1, int64_t s1) {
  if (n0 == 1) return n1 == 1 || s1 >= FL_HEAD_DIM;
  if (n1 == 1) return s0 >= FL_HEAD_DIM;
  return (s1 >= FL_HEAD_DIM && s0 >= (n1 - 1) * s1 + FL_HEAD_DIM) || (s0 >= FL_HEAD_DIM && s1 >= (n0 - 1) * s0 + FL_HEAD_DIM);
}

uint64_t data_bytes(const fl_paged_index& x, const fl_paged_pool& p, int batch, int q_heads) {
  const uint64_t a = paged_select_bytes(x, p, batch), b = paged_attn_bytes(p, q_heads);
  return ((a > b ? a : b) + 255) / 256 * 256;
}

fl_status check_heads(const fl_paged_index* x, const fl_paged_pool* p, int32_t batch, int32_t q_heads) {
  if (q_heads < 1 || q_heads % p->kv_heads) return FL_ERR_INVALID;
  // work units of one call are counted in 32 bits: blocks and quarters of a tail, per entry,
  // key-value head and four query heads
  const int64_t chunks = (q_heads / p->kv_heads + 3) / 4;
  if ((int64_t)batch * p->kv_heads * chunks * ((int64_t)x->max_pages + 4) > INT32_MAX) return FL_ERR_UNSUPPORTED;
  return FL_OK;
}

fl_status attn_args(const fl_paged_index* x, const fl_paged_pool* p, int32_t batch, const int32_t* slots,
                    int32_t q_heads, const uint16_t* q, int64_t q_batch_stride, int64_t q_head_stride, void* ws,
                    size_t ws_bytes, PagedAttnArgs* a) {
  fl_status st = check_pool(x, p);
  if (st != FL_OK) return st;
  if ((st = check_batch(x, batch, slots)) != FL_OK) return st;
  if ((st = check_heads(x, p, batch, q_heads)) != FL_OK) return st;
  if (batch == 0) return FL_OK;
  if (!q || !aligned(q, 16) || !good_strides(q_batch_stride, q_head_stride, 8)) return FL_ERR_INVALID;
  if (!ws || !aligned(ws, 256) || ws_bytes < fl_paged_workspace_bytes(x, p, batch, q_heads)) return FL_ERR_WORKSPACE;
  *a = PagedAttnArgs{};
  a->x = *x;
  a->p = *p;
  a->batch = batch;
  a->slots = slots;
  a->q_heads = q_heads;
  a->group = q_heads / p->kv_heads;
  a->q = q;
  a->q_batch_stride = q_batch_stride;
  a->q_head_stride = q_head_stride;
  a->tickets = static_cast<int32_t*>(ws);
  a->data = static_cast<uint8_t*>(ws) + FL_PAGED_WS_HEAD;
  return FL_OK;
}

fl_status launched(cudaError_t e) { return e == cudaSuccess ? FL_OK : FL_ERR_CUDA; }

}  // namespace

extern "C" {

fl_status fl_paged_index_init(const fl_paged_index* index, void* stream) {
  const fl_status st = check_index(index);
  if (st != FL_OK) return st;
  return launched(launch_paged_index_init(*index, (cudaStream_t)stream));
}

fl_status fl_paged_extend(const fl_paged_index* index, int32_t batch, const int32_t* slots, const int32_t* n_new,
                          int32_t* start, int32_t* cu, void* stream) {
  fl_status st = check_index(index);
  if (st != FL_OK) return st;
  if ((st = check_batch(index, batch, slots)) != FL_OK) return st;
  if (!cu || !aligned(cu, 4) || (batch > 0 && (!n_new || !start)) || !aligned(n_new, 4) || !aligned(start, 4))
    return FL_ERR_INVALID;
  return launched(launch_paged_extend(*index, batch, slots, n_new, start, cu, (cudaStream_t)stream));
}

fl_status fl_paged_release(const fl_paged_index* index, int32_t batch, const int32_t* slots, void* stream) {
  fl_status st = check_index(index);
  if (st != FL_OK) return st;
  if ((st = check_batch(index, batch, slots)) != FL_OK) return st;
  if (batch == 0) return FL_OK;
  return launched(launch_paged_release(*index, batch, slots, (cudaStream_t)stream));
}

fl_status fl_paged_slot_map(const fl_paged_index* index, int32_t batch, const int32_t* slots, const int32_t* start,
                            const int32_t* cu, int32_t n_tokens, int32_t* place, int32_t* pos, void* stream) {
  fl_status st = check_index(index);
  if (st != FL_OK) return st;
  if ((st = check_batch(index, batch, slots)) != FL_OK) return st;
  if (n_tokens < 0 || !aligned(place, 4) || !aligned(pos, 4)) return FL_ERR_INVALID;
  if (batch == 0 || n_tokens == 0 || (!place && !pos)) return FL_OK;
  if (!start || !cu || !aligned(start, 4) || !aligned(cu, 4)) return FL_ERR_INVALID;
  return launched(launch_paged_slot_map(*index, batch, slots, start, cu, n_tokens, place, pos, (cudaStream_t)stream));
}

fl_status fl_paged_append(const fl_paged_index* index, const fl_paged_pool* pool, int32_t batch, const int32_t* slots,
                          const int32_t* start, const int32_t* cu, int32_t n_tokens, const uint16_t* k,
                          const uint16_t* v, int64_t token_stride, int64_t head_stride, void* stream) {
  fl_status st = check_pool(index, pool);
  if (st != FL_OK) return st;
  if ((st = check_batch(index, batch, slots)) != FL_OK) return st;
  if (n_tokens < 0) return FL_ERR_INVALID;
  if (batch == 0 || n_tokens == 0) return FL_OK;
  // work items are counted in 32 bits, with room for one more step of the grid
  if (2 * ((int64_t)batch + n_tokens / FL_PAGE) * pool->kv_heads > INT32_MAX - 65536) return FL_ERR_UNSUPPORTED;
  if (!start || !cu || !aligned(start, 4) || !aligned(cu, 4)) return FL_ERR_INVALID;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !good_strides(token_stride, head_stride, 8))
    return FL_ERR_INVALID;
  PagedAppendArgs a{*index, *pool, batch, n_tokens, slots, start, cu, k, v, token_stride, head_stride};
  return launched(launch_paged_append(a, (cudaStream_t)stream));
}

fl_status fl_paged_read(const fl_paged_index* index, const fl_paged_pool* pool, int32_t n_tokens,
                        const int32_t* place, uint16_t* k, uint16_t* v, int64_t token_stride, int64_t head_stride,
                        void* stream) {
  const fl_status st = check_pool(index, pool);
  if (st != FL_OK) return st;
  if (n_tokens < 0) return FL_ERR_INVALID;
  if (n_tokens == 0) return FL_OK;
  if (!place || !aligned(place, 4) || !k || !v || !aligned(k, 16) || !aligned(v, 16) ||
      !good_strides(token_stride, head_stride, 8))
    return FL_ERR_INVALID;
  if (!rows_apart(n_tokens, token_stride, pool->kv_heads, head_stride)) return FL_ERR_INVALID;
  PagedReadArgs a{*index, *pool, n_tokens, place, k, v, token_stride, head_stride};
  return launched(launch_paged_read(a, (cudaStream_t)stream));
}

size_t fl_paged_workspace_bytes(const fl_paged_index* index, const fl_paged_pool* pool, int32_t batch,
                                int32_t q_heads) {
  if (check_pool(index, pool) != FL_OK || batch < 0 || batch > FL_PAGED_MAX_BATCH) return 0;
  if (check_heads(index, pool, batch, q_heads) != FL_OK) return 0;
  return FL_PAGED_WS_HEAD + data_bytes(*index, *pool, batch, q_heads);
}

fl_status fl_paged_workspace_init(void* ws, size_t ws_bytes, void* stream) {
  if (!ws || !aligned(ws, 256) || ws_bytes < FL_PAGED_WS_HEAD) return FL_ERR_WORKSPACE;
  return launched(cudaMemsetAsync(ws, 0, FL_PAGED_WS_HEAD, (cudaStream_t)stream));
}

fl_status fl_paged_select(const fl_paged_index* index, const fl_paged_pool* pool, int32_t batch, const int32_t* slots,
                          int32_t q_heads, const uint16_t* q, int64_t q_batch_stride, int64_t q_head_stride,
                          int32_t keep, int32_t* sel, void* ws, size_t ws_bytes, void* stream) {
  PagedAttnArgs a;
  const fl_status st = attn_args(index, pool, batch, slots, q_heads, q, q_batch_stride, q_head_stride, ws, ws_bytes, &a);
  if (st != FL_OK) return st;
  if (keep < 1 || !aligned(sel, 4)) return FL_ERR_INVALID;
  if (keep > FL_PAGED_MAX_KEEP) return FL_ERR_UNSUPPORTED;
  if (batch == 0) return FL_OK;
  if (!sel) return FL_ERR_INVALID;
  a.keep = keep;
  a.sel = sel;
  return launched(launch_paged_select(a, (cudaStream_t)stream));
}

fl_status fl_paged_attn_decode(const fl_paged_index* index, const fl_paged_pool* pool, int32_t batch,
                               const int32_t* slots, int32_t q_heads, const uint16_t* q, int64_t q_batch_stride,
                               int64_t q_head_stride, const int32_t* sel, int32_t keep, float* o,
                               int64_t o_batch_stride, int64_t o_head_stride, float* lse, void* ws, size_t ws_bytes,
                               void* stream) {
  PagedAttnArgs a;
  const fl_status st = attn_args(index, pool, batch, slots, q_heads, q, q_batch_stride, q_head_stride, ws, ws_bytes, &a);
  if (st != FL_OK) return st;
  if (sel && (keep < 1 || !aligned(sel, 4))) return FL_ERR_INVALID;
  if (sel && keep > FL_PAGED_MAX_KEEP) return FL_ERR_UNSUPPORTED;
  if (batch == 0) return FL_OK;
  if (!o || !aligned(o, 16) || !good_strides(o_batch_stride, o_head_stride, 4) || !aligned(lse, 4))
    return FL_ERR_INVALID;
  if (!rows_apart(batch, o_batch_stride, q_heads, o_head_stride)) return FL_ERR_INVALID;
  a.sel = const_cast<int32_t*>(sel);
  a.keep = sel ? keep : 0;
  a.o = o;
  a.o_batch_stride = o_batch_stride;
  a.o_head_stride = o_head_stride;
  a.lse = lse;
  return launched(launch_paged_attn(a, (cudaStream_t)stream));
}

}  // extern "C"
