/*
 * gqa_kv.h -- C ABI of the GB300 (sm_103a) steps that feed a paged KV cache:
 * block tables and slots from request lengths, the norm, rotation and cache
 * write of a step's new tokens, and what happens to a request's blocks later
 * (forks, accepted drafts, release). The cache is the one that
 * gqa_av_decode_paged (gqa_av.h) and gqa_prefix_attn_decode (gqa_prefix.h)
 * read: pools [num_blocks, block_size, Hkv, D], row c of sequence b in block
 * block_table[b][c / block_size]. A slot is a row of the flattened pool,
 * block * block_size + c % block_size. The source pages describe decode over
 * a cache that is already filled; these calls fill it.
 *
 * Execution: asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 * default stream), no host synchronisation, no workspace, no allocation, so
 * calls on different streams are independent and every call can be captured.
 * Errors: a status code from gqa_av.h; on error nothing is launched and
 * gqa_kv_last_error() holds a message for the calling thread.
 */
#ifndef GQA_KV_H
#define GQA_KV_H

#include <stdint.h>

#include "gqa_av.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Block tables, slots and positions of a step's new tokens. Request b holds
 * cached_lens[b] cached rows and brings new_lens[b] tokens; the batch's tokens
 * are packed request after request. With blocks(n) = ceil(n / block_size),
 *
 *     held[b]  = blocks(cached_lens[b]),
 *     need[b]  = blocks(cached_lens[b] + new_lens[b]) - held[b],
 *     token_start[b] = sum_{b' < b} new_lens[b'],     b = 0 .. B.
 *
 * Free blocks come off the end of free_list (free_count[0] entries) in request
 * order: with before[b] = sum_{b' < b} need[b'],
 *
 *     block_table[b][held[b] + i] = free_list[free_count[0] - 1 - before[b] - i],
 *                                   0 <= i < need[b].
 *
 * Request b is served when need[b] == 0 or before[b] + need[b] <= free_count[0].
 * A request whose blocks do not fit max_blocks, or whose tokens end past T, is
 * not served either, and its need counts as 0. For token t of request b, with
 * row = cached_lens[b] + t - token_start[b]:
 *
 *     slots[t]     = block_table[b][row / block_size] * block_size + row % block_size,
 *     positions[t] = row + (pos_base ? pos_base[b] : 0)
 *
 * (pos_base: rows of a shared prefix that come before the request's own).
 * slots[t] is -1 when the request is not served or the table entry lies
 * outside [0, num_blocks); tokens t >= token_start[B] are padding, with slot
 * -1 and position 0. seq_lens[b] = cached_lens[b] + new_lens[b] for served
 * requests and cached_lens[b] for others. free_left[0] = free_count[0] - the
 * served needs. Entries of block_table outside the new columns are kept. Where
 * cached_lens[b] ends inside a block, the request's next rows go into that block:
 * no other request may own it (gqa_kv_release says when one can, and what to do).
 *
 *     cached_lens, new_lens, pos_base  [B] int32 (pos_base may be NULL)
 *     free_list [n_free], free_count [1]  int32; free_count is clamped to [0, n_free]
 *     block_table [B, max_blocks] int32, updated in place
 *     seq_lens [B], token_start [B + 1], slots [T], positions [T], free_left [1] int32
 *
 * Negative lengths count as 0; token starts and lengths that pass 2^31 - 1 are
 * held there (such requests are not served). Limits: B <= 8192, num_blocks * block_size
 * < 2^31. T may be 0. No output (block_table among them) may overlap an input:
 * every CTA reads the inputs while others write.
 */
int gqa_kv_tables(const int32_t *cached_lens, const int32_t *new_lens, const int32_t *pos_base,
                  const int32_t *free_list, const int32_t *free_count, int32_t *block_table,
                  int32_t *seq_lens, int32_t *token_start, int32_t *slots, int32_t *positions,
                  int32_t *free_left, int B, int T, int max_blocks, int n_free, int block_size,
                  int num_blocks, void *stream);

/* Element type of q_out besides GQA_AV_BF16 and GQA_AV_FP16: float32, the
 * query type of gqa_attn_decode and gqa_qk_softmax_decode. */
#define GQA_KV_F32 2

/*
 * Norm, rotation and cache write of T tokens in one pass. For each query head
 * x = q[t, h, :] and each key head x = k[t, h, :] (bf16 or fp16),
 *
 *     y_d = x_d * rsqrt(mean_d x_d^2 + eps) * (weight_d + weight_offset)
 *           (skipped for q when q_weight is NULL, for k when k_weight is NULL),
 *     (y_a, y_b) -> (y_a cos(w) - y_b sin(w), y_b cos(w) + y_a sin(w)),
 *     w = positions[axis(i)][t] * inv_freq[i],   i < rot_dim / 2,
 *
 * for the pair i of elements (a, b) = (i, i + rot_dim / 2), or (2i, 2i + 1)
 * with interleaved != 0; elements from rot_dim on are not rotated. axis(i) is
 * the section that pair i falls in: sections (HOST memory, n_axes <= 4
 * entries that sum to rot_dim / 2) gives the pairs of each position axis in
 * order, for example time, height and width; NULL with n_axes = 1 means one
 * axis for all pairs. Queries go to q_out; rotated keys and the values (as
 * they are) go to row slots[t] of the pools, and nowhere when slots[t] is
 * outside [0, num_blocks * block_size) (padding: -1). A row that several tokens
 * name as their slot ends up with pieces of any of them.
 *
 *     q [T, Hq, D], k and v [T, Hkv, D]  kv_dtype; a token's heads are
 *         contiguous, tokens lie q_stride, k_stride, v_stride elements apart
 *         (views of one packed projection are fine)
 *     positions [n_axes, T], slots [T]   int32
 *     inv_freq [rot_dim / 2] float32     radians a position
 *     q_weight, k_weight [D]             kv_dtype, or NULL
 *     q_out [T, Hq, D]                   q_out_dtype: kv_dtype or GQA_KV_F32
 *     k_pool, v_pool [num_blocks, block_size, Hkv, D]  kv_dtype
 *
 * Numerics: fp32 throughout, one rounding at the end. The angle is reduced
 * modulo one turn exactly in 64-bit integers before it is rounded to fp32, so
 * far positions keep full accuracy: cos and sin are within 5e-7 of the exact
 * value for |inv_freq| <= 2 pi and positions below 2^27.
 *
 * Limits: D a multiple of 8, at most 256; rot_dim <= D, a multiple of 16
 * (interleaved: of 8), or 0 for no rotation (positions and inv_freq are then
 * unused); q, k, v, q_out, pools and weights 16-byte aligned; strides
 * multiples of 8; num_blocks * block_size < 2^31. T may be 0. Outputs must
 * not overlap inputs.
 */
int gqa_kv_norm_rope_append(const void *q, const void *k, const void *v, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, const int32_t *positions,
                            const int32_t *sections, int n_axes, const float *inv_freq,
                            const void *q_weight, const void *k_weight, float eps,
                            float weight_offset, int interleaved, const int32_t *slots,
                            void *q_out, int q_out_dtype, void *k_pool, void *v_pool, int T,
                            int Hq, int Hkv, int D, int rot_dim, int kv_dtype, int block_size,
                            int num_blocks, void *stream);

/*
 * The calls below handle blocks that requests share. shares[x] counts the
 * owners of block x beyond the first: 0 for a block that gqa_kv_tables handed
 * out, one more for every fork that shares it, one less for every owner that
 * releases it, and back to the free list when the last one does. `pools` is an
 * array in HOST memory of n_pools device pointers: the K and V pools of all
 * layers (their order does not matter), each [num_blocks, block_size,
 * row_bytes] bytes; a pool may not be named twice. Limits: n_pools <= 256,
 * row_bytes a multiple of 16 and at most 2^20, pools 16-byte aligned, B <= 8192,
 * max_blocks * block_size and num_blocks * block_size below 2^31.
 */

/*
 * Fork requests: fork f makes row child[f] of the block table a continuation of
 * row parent[f]. With L = seq_lens[parent[f]] (clamped to what a table row can
 * hold), the child gets the parent's L / block_size full blocks (shares += 1
 * each) and, where L ends inside a block, a block of its own with a copy of the
 * parent's L % block_size rows in every pool; seq_lens[child[f]] = L. The parent
 * keeps its partial block. Blocks for the copies come off the end of free_list
 * (free_count[0] entries) in the order of the forks that need one:
 *
 *     fork_block[f] = free_list[free_count[0] - 1 - (forks before f that need one)].
 *
 * fork_block[f] is -1 when no copy is needed, and -2 when the fork is not served
 * (its child's row, length and everything else are left as they are): a row
 * outside [0, B), a child that is a parent of any fork or that an earlier fork
 * names too, or no free block. free_left[0] = free_count[0] - the blocks taken.
 * Table entries and list entries outside [0, num_blocks) are handed on, but
 * nothing is counted or copied for them (a negative list entry is handed on as
 * 2^31 - 1). Entries of the child's row past its blocks are kept. Two served
 * forks must not get one block (a free list that names it twice).
 *
 *     parent, child [N] int32 (a parent may have several children)
 *     block_table [B, max_blocks], seq_lens [B], shares [num_blocks] int32, updated in place
 *     free_list [n_free], free_count [1] int32; free_count is clamped to [0, n_free]
 *     fork_block [N], free_left [1] int32
 *
 * N <= 8192 and may be 0. No output may overlap an input or another output.
 */
int gqa_kv_fork(void *const *pools, int n_pools, int64_t row_bytes, const int32_t *parent,
                const int32_t *child, int32_t *block_table, int32_t *seq_lens, int32_t *shares,
                const int32_t *free_list, const int32_t *free_count, int32_t *fork_block,
                int32_t *free_left, int N, int B, int max_blocks, int n_free, int block_size,
                int num_blocks, void *stream);

/*
 * Keep accepted drafts: request b holds cached_lens[b] rows and, behind them,
 * drafted rows up to seq_lens[b]. accepted[b][i], i < accepted_count[b], are the
 * accepted drafts' numbers, counted from cached_lens[b], in ascending order (a
 * path of a tree whose tokens are numbered parents first). In every pool
 *
 *     row cached_lens[b] + i = what row cached_lens[b] + accepted[b][i] held,   0 <= i < n_b,
 *     kept_lens[b] = cached_lens[b] + n_b,
 *
 * where n_b is the length of the longest leading part of the accepted numbers
 * that ascend strictly, are not negative and lie below seq_lens[b] (and within
 * W and the table's row). Rows from kept_lens[b] on are left as they are;
 * gqa_kv_release takes their blocks. A row whose table entry lies outside
 * [0, num_blocks) is neither read nor written. No two requests may share a block
 * that holds drafted rows: a fork copies partial blocks, so none do as long as no
 * row is cut inside a shared block and then extended (gqa_kv_release).
 *
 *     cached_lens, accepted_count, seq_lens [B], accepted [B, W], block_table [B, max_blocks] int32
 *     kept_lens [B] int32; must not overlap an input
 *
 * Negative cached_lens count as 0. W <= 2^20 and may be 0; n_pools >= 1.
 */
int gqa_kv_keep(void *const *pools, int n_pools, int64_t row_bytes, const int32_t *cached_lens,
                const int32_t *accepted, const int32_t *accepted_count, const int32_t *block_table,
                const int32_t *seq_lens, int32_t *kept_lens, int B, int W, int max_blocks,
                int block_size, int num_blocks, void *stream);

/*
 * Release blocks: row b of the block table is cut from old_lens[b] rows to
 * new_lens[b] (0: the request has ended). Its blocks of the columns from
 * blocks(new_lens[b]) to blocks(old_lens[b]) lose an owner, blocks(n) =
 * ceil(n / block_size). With k_x the number of such entries of the whole table
 * that name block x: if k_x <= shares[x], shares[x] -= k_x; else the last owner
 * is gone, shares[x] = 0 and x goes to the end of the free list. The blocks that
 * go there follow one another in the order of their first such entries, row
 * after row and column after column:
 *
 *     free_list[free_count[0] + i] = the i-th of them,   free_left[0] = free_count[0] + their number
 *
 * (those past n_free are dropped, and free_left is at most n_free). Entries outside
 * [0, num_blocks) are skipped. shares NULL: no block is shared, every entry goes
 * back, and no two entries may name one block. The block table itself is kept.
 *
 * A row that is cut keeps the block that new_lens[b] ends in. If that block has
 * other owners (a request that goes back behind its fork), the row can be read and
 * forked, but must not get new rows: gqa_kv_tables, gqa_kv_norm_rope_append and
 * gqa_kv_keep would write them over the other owners'. To go on from there, take
 * a copy of the row instead of a cut: gqa_kv_fork with parent[f] = b, an unused row as
 * child[f] and, in the seq_lens it is given, n for seq_lens[b], n being the rows to
 * keep. The child shares the full blocks and owns a copy of the last n % block_size
 * rows. Then release row b whole, from the length that it had.
 *
 *     block_table [B, max_blocks], old_lens, new_lens [B] int32 (new_lens is clamped to [0, old_lens])
 *     shares [num_blocks] int32 (not negative) and free_list [n_free] int32, updated in place
 *     free_count, free_left [1] int32; free_count is clamped to [0, n_free]
 *
 * B * max_blocks < 2^30. No output may overlap an input or another output.
 */
int gqa_kv_release(const int32_t *block_table, const int32_t *old_lens, const int32_t *new_lens,
                   int32_t *shares, int32_t *free_list, const int32_t *free_count,
                   int32_t *free_left, int B, int max_blocks, int n_free, int block_size,
                   int num_blocks, void *stream);

/* Message of the calling thread's last error of these calls ("" if none). */
const char *gqa_kv_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GQA_KV_H */
