/*
 * lime_kv.h — the paged 8-bit history cache of liblime.so.
 *
 * The key and value rows of a history item do not change once the event has
 * happened (the first LIME-XOR layer projects the item embedding alone), so a
 * serving program keeps them: lime_kv_reserve finds room for new rows,
 * lime_kv_append writes them, and lime_kv_attention lets a request's query
 * rows (its links, or its newest rows) attend over everything cached for it.
 * lime_kv_release gives blocks back.
 *
 * The cache.  A pool of n_blocks blocks of `block` rows, shared by all
 * requests; request u's row j lives in block table[u][j / block] at row
 * j % block, that is in slot  table[u][j / block] * block + j % block.
 *   k_cache, v_cache  device int8 [n_blocks, Hkv, block, dh]   codes
 *   scale             device fp32 [n_blocks, Hkv, 2]           (key, value)
 *   block_table       device int32 [B, max_blocks]
 * A code c of (block, head) stands for c * scale[block, head, key or value].
 * The caller owns all of it and needs to initialise none: a block's first row
 * (row 0) starts its scales anew.
 *
 * Conventions are those of lime.h: device pointers, 16-byte aligned tensors
 * (ids, lengths and offsets aligned to their own size), one workspace whose
 * sticky status word lime_get_status reads, asynchronous calls on `stream`,
 * jagged rows packed with int64 offsets[B + 1], negative return codes before
 * anything is launched.  Errors found on the device set LIME_FLAG_* bits and
 * leave every access in bounds.  All calls can be captured into a CUDA graph.
 */
#ifndef LIME_KV_H
#define LIME_KV_H

#include "lime.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Status bits beside those of lime.h.  LIME_FLAG_BAD_OFFSETS also reports a
 * length outside [0, max_blocks * block] (it is clamped). */
enum {
  LIME_FLAG_BAD_BLOCK = 8,  /* a block id, slot or free count outside the pool */
  LIME_FLAG_NO_BLOCKS = 16, /* a request's new rows found no room              */
  LIME_FLAG_NONFINITE = 32  /* an appended value was NaN or infinite           */
};

/* Sizes.  Supported: dh in {16, 32, 64, 128}; block in {16, 32, 64, 128};
 * 1 <= Hkv, Hq a multiple of Hkv, Hq <= 1024; 1 <= n_blocks, n_blocks * Hkv <
 * 2^31; max_blocks * block <= 2^30.  The cache may pass 2^32 bytes. */
typedef struct {
  int32_t Hq;         /* query heads                                           */
  int32_t Hkv;        /* key/value heads; query head h reads head h*Hkv/Hq     */
  int32_t dh;         /* head dim                                              */
  int32_t block;      /* rows of a block                                       */
  int32_t max_blocks; /* columns of the block table                            */
  int32_t dtype;      /* lime_dtype of appended rows, queries and outputs      */
  int64_t n_blocks;   /* blocks of the pool                                    */
} lime_kv_dims;

/* Bytes of device workspace for calls with up to B requests and total_q query
 * rows (256-byte aligned, prepared once by lime_kv_workspace_init); 0 for
 * unsupported dims.  The same for every total_q > 0: a workspace made for one
 * query row serves any number of them. */
size_t lime_kv_workspace_bytes(const lime_kv_dims* dims, int64_t B, int64_t total_q);

/* Clears the workspace's status word and the counters that the calls leave at
 * zero (asynchronous on stream).  Once before the first call, and again after
 * a call that set LIME_FLAG_TIMEOUT.  LIME_ERR_ARG for a workspace smaller
 * than any lime_kv_workspace_bytes. */
int lime_kv_workspace_init(void* workspace, size_t bytes, cudaStream_t stream);

/* Block table and slot map of new rows, built from the requests' lengths.
 *   lens          device int32 [B]      rows each request holds
 *   new_offsets   device int64 [B+1]    request u brings rows
 *                                       [new_offsets[u], new_offsets[u+1])
 *   total_new     new_offsets[B]
 *   block_table   in/out: entries of new blocks are written, others kept
 *   free_blocks   device int32 [free_cap]  stack of free block ids
 *   n_free        device int32 [1]      its height
 *   lens_out      device int32 [B]      lengths with the new rows
 *   n_free_out    device int32 [1]      the stack's height afterwards
 *   slot_map      device int64 [total_new]  slot of every new row
 * Request u needs ceil((lens + new) / block) - ceil(lens / block) blocks; they
 * are taken from the top of the stack in the order of the requests and of
 * their rows.  A request that does not get all it needs (the stack is too
 * short for it and the requests before it, or its rows pass max_blocks) gets
 * none: its slots are -1, its length stays, LIME_FLAG_NO_BLOCKS is set;
 * requests that need no new block are served all the same.  What a request
 * refused for want of blocks asked for counts for those behind it: none of them
 * that needs a block is served, even where enough for it are left.
 * Outputs may not overlap inputs or each other (LIME_ERR_ALIAS). */
int lime_kv_reserve(const lime_kv_dims* dims, int64_t B, const int32_t* lens,
                    const int64_t* new_offsets, int64_t total_new, int32_t* block_table,
                    const int32_t* free_blocks, int64_t free_cap, const int32_t* n_free,
                    int32_t* lens_out, int32_t* n_free_out, int64_t* slot_map, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream);

/* Shortens requests and gives their blocks back: request u keeps its first
 * min(keep[u], lens[u]) rows (a negative count, or keep == NULL: none).
 * Blocks that hold no kept row go onto the stack in the order of the requests
 * and of their rows, and their table entries become -1.  Arguments as in
 * lime_kv_reserve; free_blocks is written from n_free on, up to free_cap
 * (what would pass it is dropped and LIME_FLAG_BAD_BLOCK set).  An entry
 * outside the pool does not go onto the stack and sets LIME_FLAG_BAD_BLOCK. */
int lime_kv_release(const lime_kv_dims* dims, int64_t B, const int32_t* lens,
                    const int32_t* keep, int32_t* block_table, int32_t* free_blocks,
                    int64_t free_cap, const int32_t* n_free, int32_t* lens_out,
                    int32_t* n_free_out, void* workspace, size_t workspace_bytes,
                    cudaStream_t stream);

/* Quantises new rows into their slots.
 *   K, V      device [total_new, Hkv, dh] of dims->dtype; row t starts ldk
 *             (ldv) elements after row t - 1 (ld >= Hkv*dh, ld*size a multiple
 *             of 16 bytes), so both may be slices of one projection's output
 *   slot_map  device int64 [total_new]; -1: the row is skipped
 * Rows whose slots follow one another in a block form one group.  With a the
 * largest |value| of the group in head h, the scale becomes
 *   s' = max(s, fp32(a / 127)),  s = the block's scale, or 0 where the group
 *                                    starts at row 0;
 * when it grows, the rows before the group are requantised, c' = rint(c s / s').
 * New codes are rint(x / s') (exact quotient, ties to even; 0 where s' = 0).
 * Rows behind the group are left as they were.  A NaN is stored as 0, an
 * infinity as +-127; neither enters a, and LIME_FLAG_NONFINITE is set.
 * All new rows of a block have to stand together in the call, in slot order
 * (as lime_kv_reserve lists them); otherwise the codes and scales of that
 * block are unspecified.  A slot outside the pool is skipped and sets
 * LIME_FLAG_BAD_BLOCK. */
int lime_kv_append(const lime_kv_dims* dims, const void* K, int64_t ldk, const void* V,
                   int64_t ldv, int64_t total_new, const int64_t* slot_map, int8_t* k_cache,
                   int8_t* v_cache, float* scale, void* workspace, size_t workspace_bytes,
                   cudaStream_t stream);

/* Attention of query rows over the cached rows of their request:
 *   O[i, h] = sum_j softmax_j(sm_scale * Q[i, h] . k_j) v_j,
 * k_j, v_j the values that row j's codes of head h*Hkv/Hq stand for.
 *   Q            device [total_q, Hq, dh], row pitch ldq elements (ldq*size a
 *                multiple of 16 bytes)
 *   q_offsets    device int64 [B+1]; request u owns rows [q_offsets[u],
 *                q_offsets[u+1]); total_q = q_offsets[B]
 *   block_table, lens   as above; lens counts all cached rows
 *   causal       0: every query row sees all lens[u] rows.  1: the queries are
 *                the request's newest rows, already appended: query i of m sees
 *                the rows j <= lens[u] - m + i
 *   O            device [total_q, Hq, dh], contiguous
 *   lse          device fp32 [total_q, Hq] or NULL: log of the softmax's sum
 * |sm_scale| <= 2^100; scales are finite and not negative, and |sm_scale| times
 * a row's largest |q| times a key scale stays below 2^127.  A query that sees
 * no row gets a zero output and lse = -inf.  Scores, sums and outputs are fp32.
 * A query row enters the score product as fp16 terms, under a power of two that
 * brings its largest magnitude m to [2^14, 2^15): one term (bf16), which holds
 * elements from 2^-31 m on exactly, or two (fp32), off by up to 2^-22 of the
 * element.  Beside that an element is off by up to 2^-39 m, so a score by up to
 * |sm_scale| 2^-39 m sum_d |k_d|, even where the keys are 0 in m's own dim.
 * Probabilities enter the value product as one fp16 term (bf16 dtype) or two
 * (fp32), each times its block's value scale over the largest such scale among
 * the request's blocks (seen by the row or not), to 2^-39 of the row's largest
 * probability; one fp16 term loses bits from 2^-28 down.  What weighs less is
 * lost, so for each row an output is off by up to 2^-39 * 127 times the largest
 * value scale among the request's blocks.  Codes behind a request's last row
 * are never used.  A table entry outside the pool hides its rows and sets
 * LIME_FLAG_BAD_BLOCK. */
int lime_kv_attention(const lime_kv_dims* dims, int64_t B, const void* Q, int64_t ldq,
                      const int64_t* q_offsets, int64_t total_q, const int32_t* block_table,
                      const int32_t* lens, const int8_t* k_cache, const int8_t* v_cache,
                      const float* scale, float sm_scale, int32_t causal, void* O, float* lse,
                      void* workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* LIME_KV_H */
