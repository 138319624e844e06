"""From prompts to drafted tokens on a paged KV cache, and back to free blocks.

    python examples/draft_steps.py

Prompts of different lengths are written to the cache and attended to in one
call a layer (gqa_prompt_attn). Each is then forked into several samples that
share its full blocks (gqa_kv_fork). Every step drafts a tree of tokens a sample:
gqa_kv_tables gives them blocks and slots, gqa_kv_norm_rope_append writes their
keys and values, gqa_tree_attn attends to the cache and to each token's path,
gqa_kv_keep moves the accepted path together in all layers and gqa_kv_release
takes back the blocks that are left over. The step is captured into a CUDA graph
once and replayed: lengths, blocks and accepted paths live on the device. At the
end all blocks are back on the free list.
"""
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gqa_attention_weighted_gb300 as gq  # noqa: E402


def int32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def draft_tree(width, depth):
    """A root and `depth` levels of `width` tokens, each behind one of the level before: its
    depth, and the mask of what it sees (itself and its path), for each token."""
    depths, masks, parents = [0], [1], [-1]
    for level in range(1, depth + 1):
        first = 1 + (level - 2) * width
        for k in range(width):
            parent = 0 if level == 1 else first + k
            depths.append(level)
            parents.append(parent)
            masks.append(masks[parent] | 1 << len(masks))
    return depths, masks, parents


class Server:
    """The cache of `layers` layers and the tables of parents * (1 + copies) requests: request
    p * (1 + copies) is the p-th prompt, the ones behind it are its samples."""

    def __init__(self, parents, copies, layers, Hq, Hkv, D, block, max_rows, width=3, depth=3,
                 dtype=torch.bfloat16):
        self.B, self.step_rows = parents * (1 + copies), 1 + copies
        self.layers, self.Hq, self.Hkv, self.D, self.block = layers, Hq, Hkv, D, block
        B = self.B
        self.max_blocks = -(-max_rows // block)
        self.num_blocks = B * self.max_blocks
        shape = (self.num_blocks, block, Hkv, D)
        self.k = [torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(layers)]
        self.v = [torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(layers)]
        self.pools = gq.KvPools(self.k + self.v)
        self.block_table, self.shares = int32(B, self.max_blocks), int32(self.num_blocks)
        self.free_list = torch.arange(self.num_blocks, dtype=torch.int32, device="cuda")
        self.free_count, self.free_left = int32(1) + self.num_blocks, int32(1)
        self.cached, self.seq_lens, self.new = int32(B), int32(B), int32(B)
        self.token_start, self.kept = int32(B + 1), int32(B)
        self.inv_freq = (10000.0 ** (-torch.arange(D // 2, device="cuda") / (D // 2))).float()
        self.weight = torch.ones(D, dtype=dtype, device="cuda")
        depths, masks, self.parents = draft_tree(width, depth)
        self.drafts = len(depths)
        self.depths = ints(depths)
        self.mask = torch.tensor(masks, dtype=torch.int64).to(torch.int32).cuda()[:, None].repeat(B, 1)
        # What checking the drafts brings: the accepted tokens' numbers, parents first.
        self.accepted, self.count = int32(B, depth + 1), int32(B)

    def tables(self, T):
        slots, positions = int32(T), int32(T)
        gq.gqa_kv_tables(self.cached, self.new, self.free_list, self.free_count, self.block_table,
                         self.seq_lens, self.token_start, slots, positions, self.free_left,
                         block_size=self.block, num_blocks=self.num_blocks)
        return slots, positions

    def append(self, layer, qkv, slots, positions):
        q, k, v = (x.unflatten(1, (-1, self.D)) for x in
                   qkv.split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], dim=1))
        q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        return gq.gqa_kv_norm_rope_append(q, k, v, positions, slots, self.inv_freq, q_out,
                                          self.k[layer], self.v[layer], q_weight=self.weight,
                                          k_weight=self.weight)

    def prompts(self, lens, qkv):
        """Prompts of `lens` tokens, one a parent: qkv [layers, T, (Hq + 2 Hkv) D]. Returns the
        layers' queries and attention outputs."""
        new = [0] * self.B
        new[::self.step_rows] = lens
        self.new.copy_(ints(new))
        slots, positions = self.tables(qkv.shape[1])
        made = []
        for i in range(self.layers):
            q = self.append(i, qkv[i], slots, positions)
            made.append((q, gq.gqa_prompt_attn(q, self.k[i], self.v[i], self.token_start, self.cached,
                                               self.block_table, self.seq_lens, torch.empty_like(q))))
        self.cached.copy_(self.seq_lens)
        self.free_count.copy_(self.free_left)
        return made

    def fork(self):
        rows = range(self.B)
        child = [b for b in rows if b % self.step_rows]
        parent = [b - b % self.step_rows for b in child]
        served = int32(len(child))
        gq.gqa_kv_fork(self.pools, ints(parent), ints(child), self.block_table, self.cached,
                       self.shares, self.free_list, self.free_count, served, self.free_left)
        self.free_count.copy_(self.free_left)
        self.new.fill_(self.drafts)
        return served

    def step(self, qkv):
        """Drafts of every request: qkv [layers, B * drafts, (Hq + 2 Hkv) D]."""
        slots, _ = self.tables(self.B * self.drafts)
        positions = (self.cached[:, None] + self.depths).flatten()   # of a token: its depth
        made = []
        for i in range(self.layers):
            q = self.append(i, qkv[i], slots, positions)
            made.append((q, gq.gqa_tree_attn(q, self.k[i], self.v[i], self.token_start, self.cached,
                                             self.mask, self.block_table, self.seq_lens,
                                             torch.empty_like(q))))
        gq.gqa_kv_keep(self.pools, self.cached, self.accepted, self.count, self.block_table,
                       self.seq_lens, self.kept)
        gq.gqa_kv_release(self.block_table, self.seq_lens, self.kept, self.shares, self.free_list,
                          self.free_left, self.free_count, block_size=self.block)
        self.cached.copy_(self.kept)
        return made

    def accept(self, rng):
        """Random paths from the root on, as if the drafts had been checked."""
        paths = []
        for _ in range(self.B):
            path = [0]
            while rng.random() < 0.7:
                behind = [i for i, p in enumerate(self.parents) if p == path[-1]]
                if not behind:
                    break
                path.append(rng.choice(behind))
            paths.append(path)
        width = self.accepted.shape[1]
        self.accepted.copy_(ints([p + [0] * (width - len(p)) for p in paths]))
        self.count.copy_(ints([len(p) for p in paths]))
        return paths

    def end(self):
        gq.gqa_kv_release(self.block_table, self.cached, int32(self.B), self.shares, self.free_list,
                          self.free_count, self.free_left, block_size=self.block)
        self.free_count.copy_(self.free_left)
        return self.free_left.item()


def main(steps=20, parents=4, copies=3, layers=4, Hq=32, Hkv=8, D=128, block=16):
    g = torch.Generator(device="cuda").manual_seed(0)
    rng = random.Random(0)

    def draw(n):
        return torch.randn((layers, n, (Hq + 2 * Hkv) * D), generator=g, device="cuda").bfloat16()

    lens = [500 + 333 * p for p in range(parents)]
    server = Server(parents, copies, layers, Hq, Hkv, D, block, max_rows=max(lens) + 4 * steps + 64)
    server.prompts(lens, draw(sum(lens)))
    server.fork()
    qkv = draw(server.B * server.drafts)
    server.accept(rng)
    server.step(qkv)                             # loads the kernels before capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        server.step(qkv)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(steps):
        server.accept(rng)
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    gq.gqa_prompt_device_status()
    rows = server.cached.sum().item()
    free = server.end()
    print(f"{steps} steps of {server.B} samples of {parents} prompts, {server.drafts} drafts each, "
          f"{layers} layers: {start.elapsed_time(end) / steps * 1e3:.0f} us a step, {rows} rows at the "
          f"end, {free} of {server.num_blocks} blocks free after it")
    del graph
    gq.gqa_prompt_release_graph_workspaces()
    return free == server.num_blocks


if __name__ == "__main__":
    main()
