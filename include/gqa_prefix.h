/*
 * gqa_prefix.h -- C ABI of the GB300 (sm_103a) decode attention over a paged
 * KV cache for a batch whose sequences share prefixes: each shared prefix is
 * read and multiplied once for all sequences behind it.
 *
 * The sequences of the batch lie in groups: group p holds the sequences
 * group_start[p] <= b < group_start[p + 1], which share the prefix_lens[p]
 * rows that row p of prefix_table lists. Behind its group's prefix every
 * sequence has seq_lens[b] rows of its own, in the blocks of row b of
 * block_table. With K_b and V_b the prefix rows followed by the own rows,
 *
 *     out[b, q_h, :] = sum_c softmax_c(scale * q[b, q_h, :] . K_b[c, kv_h, :]) * V_b[c, kv_h, :],
 *     kv_h = q_h / G,   G = Hq / Hkv.
 *
 * A sequence in no group has no prefix; P = 0 means that none has, which is
 * plain decode attention over a paged cache. A sequence with no rows at all
 * gives out = 0.
 *
 *     q, out             [B, Hq, D]                          kv_dtype (bf16 or fp16)
 *     k_pool, v_pool     [num_blocks, block_size, Hkv, D]    kv_dtype
 *     prefix_table       [P, max_prefix_blocks] int32
 *     prefix_lens        [P] int32
 *     group_start        [P + 1] int32, not decreasing; NULL with P = 1: all
 *                        sequences share the one prefix
 *     block_table        [B, max_blocks] int32, or NULL with max_blocks = 0:
 *                        no sequence has rows of its own
 *     seq_lens           [B] int32, or NULL meaning max_blocks * block_size
 * (all contiguous device memory). Lengths are clamped to what their table row
 * can hold, group starts to [0, B] and to their predecessors. Row c is in
 * block table[c / block_size] at c % block_size; a table entry outside
 * [0, num_blocks) reads rows of zeros. Entries of blocks past a length, and
 * rows past a length inside a block, may hold anything.
 *
 * Numerics: products on the tensor cores with fp32 accumulation; the running
 * maximum and sum of the softmax and the output sums are fp32; the weights
 * exp(s - m) are rounded once to kv_dtype before they multiply V (their fp32
 * values make the sum), out once at the end. Repeated calls with the same
 * shapes and lengths give bitwise-identical out.
 *
 * Limits: D 64, 128 or 256; G <= 128; block_size a multiple of 8; q, out and
 * the pools 16-byte aligned; B <= 4096, Hkv <= 2^14, B * Hkv <= 2^20, P <= 32;
 * num_blocks * block_size below 2^31 and at most 2^26 rows in one table row.
 *
 * Execution: asynchronous on `stream`; the lengths and groups are read on the
 * device, so a captured graph follows them. The call keeps workspaces of its
 * own, allocated with cudaMalloc when they are first needed or too small (the
 * host then waits for the calls under way on the stream; nothing else
 * synchronises): one for each stream, and one for each stream of a capture,
 * which the calls of that capture share. So calls on different streams and
 * replays of different graphs may overlap, from one host thread or several. Two
 * executable copies of one captured graph share its workspace and must not
 * overlap. A stream's workspace outlives the stream, for the next one of the
 * same handle; a capture's is kept until gqa_prefix_release_graph_workspaces.
 * Its size: with R = 128 / G sequences a query tile, up to
 *     (ceil(B / R) + min(P, B)) * Hkv + 2 * SMs
 * slots of 128 * (D + 2) floats, twice that for D below 256, and (B * Hkv +
 * 4 * SMs) * G * (D + 2) floats for own rows (46 MB for 64 sequences, 32 + 8
 * heads of 128). Errors: a status code from gqa_av.h; on error nothing is
 * launched and gqa_prefix_last_error() holds a message.
 */
#ifndef GQA_PREFIX_H
#define GQA_PREFIX_H

#include <stddef.h>
#include <stdint.h>

#include "gqa_av.h"

#ifdef __cplusplus
extern "C" {
#endif

int gqa_prefix_attn_decode(const void *q, const void *k_pool, const void *v_pool,
                           const int32_t *prefix_table, const int32_t *prefix_lens,
                           const int32_t *group_start, const int32_t *block_table,
                           const int32_t *seq_lens, void *out, int B, int P, int Hq, int Hkv,
                           int D, int kv_dtype, int block_size, int num_blocks,
                           int max_prefix_blocks, int max_blocks, float scale, void *stream);

/* Synchronise `stream`, then read the device's status word (set when a bounded
 * wait inside a kernel runs out, in any call or graph replay on the device):
 * GQA_AV_OK or GQA_AV_ERR_DEVICE_TIMEOUT; with clear != 0 the word is reset. */
int gqa_prefix_device_status(void *stream, int clear);

/* Free the workspaces of all captures. No graph that was captured before the
 * call may be launched after it. (cudaFree waits for launches under way.) */
int gqa_prefix_release_graph_workspaces(void);

/*
 * Self-test of that report: the decode call with bounded waits of wait_ns
 * (100 us to 2 s) instead of 2 s, and with every CTA leaving out its query
 * loads from number withhold_from on (nothing of them is ever issued). The
 * waits for them run out, the warps set the status word, wait for their own
 * copies and products in flight and leave; no GPU fault, trap or hang is
 * caused. `out` is left unspecified. Returns GQA_AV_OK once launched;
 * gqa_prefix_device_status then reports GQA_AV_ERR_DEVICE_TIMEOUT if a CTA had
 * that many query loads (with withhold_from 0: if any sequence has rows).
 */
int gqa_prefix_selftest_wait_timeout(const void *q, const void *k_pool, const void *v_pool,
                                     const int32_t *prefix_table, const int32_t *prefix_lens,
                                     const int32_t *group_start, const int32_t *block_table,
                                     const int32_t *seq_lens, void *out, int B, int P, int Hq,
                                     int Hkv, int D, int kv_dtype, int block_size, int num_blocks,
                                     int max_prefix_blocks, int max_blocks, float scale,
                                     long long wait_ns, int withhold_from, void *stream);

/* Message of the calling thread's last error of these calls ("" if none). */
const char *gqa_prefix_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GQA_PREFIX_H */
