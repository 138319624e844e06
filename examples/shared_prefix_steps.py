"""Decode steps of a batch behind one shared prefix, on a paged KV cache.

    python examples/shared_prefix_steps.py

A prefix is written to the cache once. Then every step takes the new tokens'
projections through three calls: gqa_kv_tables gives each request its blocks
and slots, gqa_kv_norm_rope_append norms and rotates queries and keys and
writes keys and values to the slots, gqa_prefix_attn_decode attends to the
prefix (read once for the whole batch) and to each request's own rows. The
step is captured into a CUDA graph once and replayed: lengths, slots and
positions live on the device.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gqa_attention_weighted_gb300 as gq  # noqa: E402


def int32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


class PagedSteps:
    """The cache and the tables of a batch of B requests behind a shared prefix."""

    def __init__(self, B, Hq, Hkv, D, block, prefix_rows, max_rows, dtype=torch.bfloat16):
        self.B, self.Hq, self.Hkv, self.D, self.block = B, Hq, Hkv, D, block
        self.prefix_blocks = -(-prefix_rows // block)
        self.max_blocks = -(-max_rows // block)
        self.num_blocks = self.prefix_blocks + B * self.max_blocks
        shape = (self.num_blocks, block, Hkv, D)
        self.k_pool = torch.zeros(shape, dtype=dtype, device="cuda")
        self.v_pool = torch.zeros(shape, dtype=dtype, device="cuda")
        self.prefix_table = torch.arange(self.prefix_blocks, dtype=torch.int32, device="cuda")[None]
        self.prefix_lens = int32(1) + prefix_rows
        self.free_list = torch.arange(self.prefix_blocks, self.num_blocks, dtype=torch.int32,
                                      device="cuda")
        self.free_count = int32(1) + self.free_list.numel()
        self.free_left, self.block_table = int32(1), int32(B, self.max_blocks)
        self.cached, self.seq_lens = int32(B), int32(B)
        self.new, self.base = int32(B) + 1, int32(B) + prefix_rows
        self.token_start, self.slots, self.positions = int32(B + 1), int32(B), int32(B)
        self.inv_freq = (10000.0 ** (-torch.arange(D // 2, device="cuda") / (D // 2))).float()
        self.q_weight = torch.ones(D, dtype=dtype, device="cuda")
        self.k_weight = torch.ones(D, dtype=dtype, device="cuda")
        self.q = torch.empty((B, Hq, D), dtype=dtype, device="cuda")
        self.out = torch.empty_like(self.q)

    def append(self, qkv, positions, slots, q_out):
        q, k, v = (x.unflatten(1, (-1, self.D)) for x in
                   qkv.split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], dim=1))
        return gq.gqa_kv_norm_rope_append(q, k, v, positions, slots, self.inv_freq, q_out,
                                          self.k_pool, self.v_pool, q_weight=self.q_weight,
                                          k_weight=self.k_weight)

    def prefill_prefix(self, qkv):
        """Writes the shared prefix's rows: row c to slot c (the first blocks)."""
        rows = torch.arange(qkv.shape[0], dtype=torch.int32, device="cuda")
        return self.append(qkv, rows, rows, torch.empty((qkv.shape[0], self.Hq, self.D),
                                                        dtype=qkv.dtype, device="cuda"))

    def step(self, qkv):
        """One new token of every request: qkv [B, (Hq + 2 Hkv) D] -> out [B, Hq, D]."""
        gq.gqa_kv_tables(self.cached, self.new, self.free_list, self.free_count, self.block_table,
                         self.seq_lens, self.token_start, self.slots, self.positions,
                         self.free_left, block_size=self.block, num_blocks=self.num_blocks,
                         pos_base=self.base)
        self.append(qkv, self.positions, self.slots, self.q)
        gq.gqa_prefix_attn_decode(self.q, self.k_pool, self.v_pool, self.prefix_table,
                                  self.prefix_lens, None, self.block_table, self.seq_lens, self.out)
        # What this step leaves is what the next one starts from.
        self.cached.copy_(self.seq_lens)
        self.free_count.copy_(self.free_left)
        return self.out

    def reset(self):
        """Back to the prefix alone, all other blocks free."""
        self.cached.zero_()
        self.free_count.fill_(self.free_list.numel())


def main(steps=40, B=32, Hq=32, Hkv=8, D=128, block=16, prefix_rows=2000):
    g = torch.Generator(device="cuda").manual_seed(0)

    def draw(n):
        return torch.randn((n, (Hq + 2 * Hkv) * D), generator=g, device="cuda").bfloat16()

    batch = PagedSteps(B, Hq, Hkv, D, block, prefix_rows, max_rows=steps + 8)
    batch.prefill_prefix(draw(prefix_rows))
    qkv = draw(B)
    batch.step(qkv)                              # loads the kernels before capture
    batch.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        batch.step(qkv)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(steps):
        qkv.copy_(draw(B))
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    gq.gqa_prefix_device_status()
    lens = batch.seq_lens.tolist()
    print(f"{steps} steps of {B} requests behind {prefix_rows} shared rows: "
          f"{start.elapsed_time(end) / steps * 1e3:.0f} us a step, own rows {lens[0]}, "
          f"{batch.free_left.item()} blocks free")
    return lens


if __name__ == "__main__":
    main()
