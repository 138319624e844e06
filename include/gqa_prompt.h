/*
 * gqa_prompt.h -- C ABI of the GB300 (sm_103a) attention of several new tokens
 * a sequence over a paged KV cache: whole prompts or chunks of them (causal),
 * and trees of drafted tokens that are checked in one step. It is the step
 * after gqa_kv_norm_rope_append (gqa_kv.h), which writes the new tokens' rows.
 *
 * The batch's new tokens are packed sequence after sequence, as gqa_kv_tables
 * numbers them: token t = token_start[b] + i, 0 <= i < n_b = token_start[b + 1] -
 * token_start[b], is row r = cached_lens[b] + i of sequence b. With K_b and V_b
 * the rows that block_table[b] lists,
 *
 *     out[t, q_h, :] = sum_c softmax_c(scale * q[t, q_h, :] . K_b[c, kv_h, :]) * V_b[c, kv_h, :],
 *     kv_h = q_h / G,   G = Hq / Hkv,
 *
 * over the rows c < seq_lens[b] that the token sees:
 *
 *     gqa_prompt_attn   c <= r;
 *     gqa_tree_attn     c < cached_lens[b], and the drafted rows c = cached_lens[b] + j,
 *                       j < n_b, whose bit j is set in the token's mask (bit j % 32
 *                       of word j / 32; a token sees itself only if its own bit is
 *                       set; bits past the mask's words count as 0).
 *
 * A token that sees no row gives out = 0. Values of rows that a token does not
 * see do not reach it, NaN and infinities included.
 *
 *     q                  [T, Hq, D] kv_dtype; a token's heads are contiguous, tokens
 *                        lie q_stride elements apart
 *     out                [T, Hq, D] kv_dtype, contiguous; rows of tokens in no
 *                        sequence (padding behind the last) are left as they are
 *     k_pool, v_pool     [num_blocks, block_size, Hkv, D] kv_dtype
 *     token_start        [B + 1] int32; clamped to [0, T] and to their predecessors
 *     cached_lens        [B] int32, or NULL: 0 (whole prompts)
 *     tree_mask          [T, words] int32
 *     block_table        [B, max_blocks] int32
 *     seq_lens           [B] int32, or NULL: cached_lens[b] + n_b
 * (device memory). cached_lens and seq_lens are clamped to [0, max_blocks *
 * block_size]. Row c is in block table[c / block_size] at c % block_size; a
 * table entry outside [0, num_blocks) reads rows of zeros. Entries of blocks
 * past a length, and rows past a length inside a block, may hold anything. out
 * must not overlap an input (refused).
 *
 * Numerics: products on the tensor cores with fp32 accumulation; the running
 * maximum and sum of the softmax and the output sums are fp32; the weights
 * exp(s - m) are rounded once to kv_dtype before they multiply V (their fp32
 * values make the sum), out once at the end. Repeated calls with the same
 * shapes and lengths give bitwise-identical out.
 *
 * Limits: D 64, 128 or 256; G <= 128; block_size a multiple of 8; q, out and
 * the pools 16-byte aligned, q_stride a multiple of 8 and at least Hq * D;
 * B <= 8192, T <= 2^20, Hkv <= 2^10; num_blocks * block_size below 2^31 and at
 * most 2^26 rows in one table row; words <= 2^15. T may be 0.
 *
 * Execution: asynchronous on `stream`, one kernel; lengths are read on the
 * device, so a captured graph follows them. The call keeps workspaces of its
 * own as gqa_prefix_attn_decode does (gqa_prefix.h): one for each stream, and
 * one for each stream of a capture, which the calls of that capture share; they
 * are allocated with cudaMalloc when first needed or too small (the host then
 * waits for the calls under way on the stream; nothing else synchronises). Calls
 * on different streams, of any priority, and replays of different graphs may
 * overlap (the kernel never waits for a block that has not started); two
 * executable copies of one captured graph must not. A capture's workspace is
 * kept until gqa_prompt_release_graph_workspaces. Its size: slots of 128 * (D + 2)
 * floats (twice that for D below 256) for rows whose keys were cut, and 32 bytes an
 * item of 128 / G tokens. A stream's has 4 to 8 slots an SM whatever the call (41 to
 * 160 MB), a capture's no more than its calls can fill: for each KV head and item one
 * slot for every 512 rows (D = 256: 256) that a table row can hold. Errors: a
 * status code from gqa_av.h; on error nothing is launched and
 * gqa_prompt_last_error() holds a message.
 */
#ifndef GQA_PROMPT_H
#define GQA_PROMPT_H

#include <stdint.h>

#include "gqa_av.h"

#ifdef __cplusplus
extern "C" {
#endif

int gqa_prompt_attn(const void *q, int64_t q_stride, const void *k_pool, const void *v_pool,
                    const int32_t *token_start, const int32_t *cached_lens,
                    const int32_t *block_table, const int32_t *seq_lens, void *out, int B, int T,
                    int Hq, int Hkv, int D, int kv_dtype, int block_size, int num_blocks,
                    int max_blocks, float scale, void *stream);

int gqa_tree_attn(const void *q, int64_t q_stride, const void *k_pool, const void *v_pool,
                  const int32_t *token_start, const int32_t *cached_lens,
                  const int32_t *tree_mask, int words, const int32_t *block_table,
                  const int32_t *seq_lens, void *out, int B, int T, int Hq, int Hkv, int D,
                  int kv_dtype, int block_size, int num_blocks, int max_blocks, float scale,
                  void *stream);

/* Synchronise `stream`, then read the device's status word (set when a bounded
 * wait inside a kernel of either call runs out, in any call or graph replay on
 * the device): GQA_AV_OK or GQA_AV_ERR_DEVICE_TIMEOUT; with clear != 0 the word
 * is reset. */
int gqa_prompt_device_status(void *stream, int clear);

/* Free the workspaces of all captures. No graph that was captured before the
 * call may be launched after it. (cudaFree waits for launches under way.) */
int gqa_prompt_release_graph_workspaces(void);

/*
 * Self-test of that report: gqa_prompt_attn with bounded waits of wait_ns
 * (100 us to 2 s) instead of 2 s, and with every CTA leaving out its query loads
 * from number withhold_from on (nothing of them is ever issued). The waits for
 * them run out, the warps set the status word, wait for their own copies and
 * products in flight and leave; no GPU fault, trap or hang is caused. `out` is
 * left unspecified. Returns GQA_AV_OK once launched; gqa_prompt_device_status
 * then reports GQA_AV_ERR_DEVICE_TIMEOUT if a CTA had that many query loads.
 */
int gqa_prompt_selftest_wait_timeout(const void *q, int64_t q_stride, const void *k_pool,
                                     const void *v_pool, const int32_t *token_start,
                                     const int32_t *cached_lens, const int32_t *block_table,
                                     const int32_t *seq_lens, void *out, int B, int T, int Hq,
                                     int Hkv, int D, int kv_dtype, int block_size, int num_blocks,
                                     int max_blocks, float scale, long long wait_ns,
                                     int withhold_from, void *stream);

/*
 * Self-test of calls whose CTAs are not all placed at once (other kernels hold
 * SMs): gqa_prompt_attn with bounded waits of wait_ns (100 us to 2 s) and with the
 * CTAs from number late_from on starting late_ns (at most 2 s) after the others. No
 * CTA waits for one that has not started, so `out` is what gqa_prompt_attn gives
 * and no wait runs out, however late they are.
 */
int gqa_prompt_selftest_late_start(const void *q, int64_t q_stride, const void *k_pool,
                                   const void *v_pool, const int32_t *token_start,
                                   const int32_t *cached_lens, const int32_t *block_table,
                                   const int32_t *seq_lens, void *out, int B, int T, int Hq, int Hkv,
                                   int D, int kv_dtype, int block_size, int num_blocks,
                                   int max_blocks, float scale, long long wait_ns, int late_from,
                                   long long late_ns, void *stream);

/* Message of the calling thread's last error of these calls ("" if none). */
const char *gqa_prompt_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GQA_PROMPT_H */
