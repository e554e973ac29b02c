/*
 * flashloop_paged.h -- paged INT4 key-value cache of many requests (sm_100a), in the
 * library libflashloop_b200.so beside the single-sequence cache of flashloop.h.
 *
 * A request sits in one of `slots` rows of a block table.  Block j of a request is its
 * tokens 64j .. 64j+63; table[slot][j] is the page of a pool that holds the block, one
 * FL_GROUP_RECORD (9216 bytes, flashloop.h) per key-value head: 4-bit codes, keys grouped
 * per channel over the 64 tokens, values per (token, 64-channel half).  As in the
 * single-sequence cache the newest 1..64 tokens of a request stay in BF16: with n tokens,
 *     full(n) = n > 0 ? (n - 1) / 64 : 0
 * blocks are records and tokens 64 full(n) .. n - 1 are rows 0 .. of the slot's BF16 tail.
 * ceil(n / 64) pages belong to the request (the last one waits for the tail to fill).
 * One fl_paged_index (tables, lengths, free pages) serves any number of fl_paged_pools:
 * one pool per layer, or per (layer, loop) of a looped model whose every loop keeps its
 * full state in 4 bits (FL_CODEC_FULL_INT4's form).
 *
 * A serving step:
 *     fl_paged_extend    lengths += n_new, pages taken             (once a step)
 *     fl_paged_append    the new tokens' keys and values           (each pool)
 *     fl_paged_attn_decode, or fl_paged_select and then fl_paged_attn_decode with its
 *                        selection                                 (each pool)
 *     fl_paged_release   pages of finished requests given back
 * fl_paged_slot_map gives the place and position of tokens (for rotary positions, and for
 * fl_paged_read, which hands cached tokens back as BF16 rows, e.g. to
 * fl_prefill_attn_sparse).
 *
 * Conventions beyond those of flashloop.h (device pointers owned by the caller, calls only
 * enqueue, host validation before any launch, kernels never trap):
 *   - `slots` (device int32 [batch]) names the batch's requests in any order; NULL means
 *     rows 0 .. batch - 1.  -1 marks a padded entry: it is skipped and its output rows are
 *     left as they were.  Any other value outside [0, index.slots) is an error, and the
 *     entry is treated as padded.
 *   - Data errors are recorded in index.status (device int32[3]: first code, its detail, the
 *     number of errors; NULL: not recorded).
 *   - Calls that share an index, a pool or a workspace must be ordered (one stream, or
 *     events), also when they are replayed from CUDA graphs: two graphs that hold calls on
 *     one workspace must not run at the same time.
 *   - Offsets into pools are computed in 64 bits.
 *   - Every call is ordered behind the stream's earlier work as any launch is.  (The kernels are
 *     launched programmatically: their first instructions may run while the predecessor ends,
 *     and they wait for it before they touch memory.)
 */
#ifndef FLASHLOOP_PAGED_H
#define FLASHLOOP_PAGED_H

#include "flashloop.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FL_PAGE 64                    /* tokens of a block */
#define FL_PAGED_MAX_BATCH 8192       /* entries of one call */
#define FL_PAGED_MAX_SLOTS 131072     /* rows of a table */
#define FL_PAGED_MAX_BLOCKS 16384     /* blocks of one request (1,048,576 tokens) */
#define FL_PAGED_MAX_KEEP 16384       /* blocks one selection may keep */

/* Device error codes, beside those of flashloop.h (status[1] holds the batch entry). */
#define FL_DEV_SLOT_RANGE 16   /* a slot outside [-1, slots) */
#define FL_DEV_SLOT_TWICE 17   /* a slot named twice in a call that changes it: the first entry counts */
#define FL_DEV_NO_PAGE 18      /* not enough free pages: the request is left as it was */
#define FL_DEV_TOO_LONG 19     /* a length outside [0, 64 max_pages], or growth beyond it */
#define FL_DEV_COUNT 20        /* a negative token count, more than 2^31 - 1 rows, or offsets that do not ascend or pass n_tokens */
#define FL_DEV_PAGE_RANGE 21   /* a page, or a place of a slot map, outside the pool: skipped */
#define FL_DEV_SEL_BLOCK 22    /* a selected block that is no full block of its request: skipped */

typedef struct fl_paged_index {
  int32_t* table;       /* [slots][max_pages] page of each block; entries behind a request's blocks are unused */
  int32_t* length;      /* [slots] tokens of each request */
  int32_t* free_pages;  /* [pages] stack of free page ids, the next one at n_free - 1 */
  int32_t* n_free;      /* [1] */
  int32_t* status;      /* NULL or [3] */
  int32_t slots, max_pages, pages;
} fl_paged_index;

typedef struct fl_paged_pool {
  uint8_t* rec;         /* [pages][kv_heads][FL_GROUP_RECORD], 16-byte aligned */
  uint16_t* tail_k;     /* BF16 [slots][kv_heads][64][128], 16-byte aligned */
  uint16_t* tail_v;
  int32_t kv_heads;     /* >= 1 */
  int32_t head_dim;     /* must be 128 */
  int32_t page_tokens;  /* must be 64 */
} fl_paged_pool;

/* Empty index: length = 0, table = -1, free_pages = pages - 1 .. 0 (page 0 is taken first),
 * status cleared. */
fl_status fl_paged_index_init(const fl_paged_index* index, void* stream);

/* Give each request n_new[i] more tokens: for entries in batch order, request i of c tokens
 * takes ceil((c + n_new[i]) / 64) - ceil(c / 64) pages from the top of the free stack into
 * its table row, and its length becomes c + n_new[i].  start[i] receives c, or -1 for an
 * entry that is padded or refused (slot error, slot named before, negative n_new, more than
 * 64 max_pages tokens, or too few pages: an entry that needs pages is refused once the
 * pages needed by the valid entries up to it exceed the free ones; a refused request is left
 * as it was).  cu [batch + 1] receives the offsets of the entries' rows in the packed input:
 * cu[0] = 0, cu[i + 1] = cu[i] + max(n_new[i], 0), whether or not entry i is refused, but at
 * most 2^31 - 1: an entry with rows beyond that is refused too (FL_DEV_COUNT). */
fl_status fl_paged_extend(const fl_paged_index* index, int32_t batch, const int32_t* slots, const int32_t* n_new,
                          int32_t* start, int32_t* cu, void* stream);

/* Give every page of each request back (in batch order, block order: the last block's page
 * ends on top of the free stack) and empty the request: length 0, table row's used entries
 * -1.  A slot named twice is released once.  A used entry that is no page of the pool is told
 * (FL_DEV_PAGE_RANGE) and given to no one. */
fl_status fl_paged_release(const fl_paged_index* index, int32_t batch, const int32_t* slots, void* stream);

/* Place and position of tokens start[i] .. start[i] + (cu[i+1] - cu[i]) - 1 of each request,
 * in rows cu[i] ..: pos = the token's index, place = page * 64 + offset for a token of a full
 * block, or (pages + slot) * 64 + row for a row of the slot's tail; both -1 for rows of
 * padded entries and of entries with start < 0, and place -1 for a token at or beyond the
 * request's length.  Rows of [cu[batch], n_tokens) are left as they were.  Either output may
 * be NULL.  Places hold until the next append that fills the block. */
fl_status fl_paged_slot_map(const fl_paged_index* index, int32_t batch, const int32_t* slots, const int32_t* start,
                            const int32_t* cu, int32_t n_tokens, int32_t* place, int32_t* pos, void* stream);

/* Write the new tokens' keys and values into a pool, after fl_paged_extend (whose start and
 * cu these are): rows cu[i] .. cu[i+1] - 1 are tokens start[i] .. of request i.  Blocks that
 * are full now (fl_paged_extend's length) become records -- codes, scales and zeros are the
 * exact quantiser's of flashloop.h, the block's older rows taken from the tail -- and the
 * tokens behind them tail rows.  k, v: BF16, row t and head h at k + t token_stride + h
 * head_stride, 128 contiguous channels; strides multiples of 8, pointers 16-byte aligned;
 * k and v share strides.  n_tokens is the rows k and v hold; an entry whose rows pass it is
 * skipped (FL_DEV_COUNT), and so are the first entry with cu[i + 1] < cu[i], told for each such entry, and
 * all behind it.  A slot may be named once. */
fl_status fl_paged_append(const fl_paged_index* index, const fl_paged_pool* pool, int32_t batch, const int32_t* slots,
                          const int32_t* start, const int32_t* cu, int32_t n_tokens, const uint16_t* k,
                          const uint16_t* v, int64_t token_stride, int64_t head_stride, void* stream);

/* Cached tokens as BF16 rows: row t of k, v (same addressing and alignment as
 * fl_paged_append's, rows that do not overlap) receives the token at place[t]
 * (fl_paged_slot_map's): fma(code, s, z) rounded to BF16, or the tail's row.  Rows with place -1 are left as they were. */
fl_status fl_paged_read(const fl_paged_index* index, const fl_paged_pool* pool, int32_t n_tokens,
                        const int32_t* place, uint16_t* k, uint16_t* v, int64_t token_stride, int64_t head_stride,
                        void* stream);

/* Workspace of the two calls below for up to `batch` entries and q_heads query heads (0 for
 * arguments out of range).  fl_paged_workspace_init zeroes its first FL_PAGED_WS_HEAD bytes:
 * once before the first call, and again after FL_DEV_TIMEOUT. */
#define FL_PAGED_WS_HEAD 8192
size_t fl_paged_workspace_bytes(const fl_paged_index* index, const fl_paged_pool* pool, int32_t batch,
                                int32_t q_heads);
fl_status fl_paged_workspace_init(void* ws, size_t ws_bytes, void* stream);

/* Blocks to attend to: for each entry and key-value head h the `keep` full blocks of the
 * highest score (all of them when there are no more), ascending, into sel [batch][kv_heads]
 * [keep]; entries behind the last one are -1 (rows of padded entries are left as they were).
 * With lo_c = z_c and hi_c = z_c + 15 s_c from the record's key groups
 *     score(block) = max over the group's queries q of sum_c max(q_c lo_c, q_c hi_c),
 * the largest score any key of the block could have; summed in fp64, ties to the lower
 * block; blocks whose scales or zeros are not finite, or whose score is NaN, come last (an
 * infinite q makes it so wherever a channel's bounds differ in sign).  q as in fl_paged_attn_decode. */
fl_status fl_paged_select(const fl_paged_index* index, const fl_paged_pool* pool, int32_t batch, const int32_t* slots,
                          int32_t q_heads, const uint16_t* q, int64_t q_batch_stride, int64_t q_head_stride,
                          int32_t keep, int32_t* sel, void* ws, size_t ws_bytes, void* stream);

/* Attention of one token per request over its whole cache (sel == NULL), or over the blocks
 * sel[batch][kv_heads][keep] names (each once, -1 behind the last; fl_paged_select's) and
 * the tail:  o = softmax(q K^T / sqrt(128)) V, with K, V = fma(code, s, z) or the tail's
 * rows.  q: BF16, entry i and head h at q + i q_batch_stride + h q_head_stride (16-byte
 * aligned, strides multiples of 8); query heads g kv .. of a group share key-value head
 * h = head / (q_heads / kv_heads), q_heads a multiple of kv_heads.  o: fp32, strides
 * multiples of 4, 16-byte aligned, rows that do not overlap.  lse: NULL or fp32 [batch][q_heads], the base-2 logarithm
 * of the sum of 2^score with scores in base 2 (q.k log2(e) / sqrt(128)).  A token whose score is
 * -inf has no weight; a request of no tokens, or of such tokens alone, gives o = 0 and
 * lse = -inf; rows of padded entries are left as they were.  Sums in
 * fp32; results do not depend on what else is in the batch beyond fp32 rounding, and are the
 * same for the same call.  A head's q is held as binary16 numbers of one common power of two
 * (exactly, within 2^-16 of its largest channel): a channel below that is rounded, which shows
 * where its keys are 2^10 times the other channels' or more. */
fl_status fl_paged_attn_decode(const fl_paged_index* index, const fl_paged_pool* pool, int32_t batch,
                               const int32_t* slots, int32_t q_heads, const uint16_t* q, int64_t q_batch_stride,
                               int64_t q_head_stride, const int32_t* sel, int32_t keep, float* o,
                               int64_t o_batch_stride, int64_t o_head_stride, float* lse, void* ws, size_t ws_bytes,
                               void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FLASHLOOP_PAGED_H */
