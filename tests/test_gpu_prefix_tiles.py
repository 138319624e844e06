"""gqa_prefix_attn_decode in units of several key tiles a stream: the ring of
stages wraps, sums run on over tiles, maxima move, streams end apart. Batches
and what they reach: prefix_tile_cases.py; reference: the definition in 64 bits.
"""
import numpy as np
import pytest
import torch

from helpers import TORCH_V
from prefix_tile_cases import CASES, reaches
from test_gpu_prefix import call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    yield pkg
    pkg.gqa_prefix_device_status()


def batch(name, vd, rng, spread=2.0, k_of=None):
    D, B, G, Hkv, plens, starts, lens, _ = CASES[name]
    return make(rng, B, G * Hkv, Hkv, D, 16, vd, plens, starts, lens, spread=spread, k_of=k_of)


def exact(x, scale):
    """out, the weighted sum of |V|, the keys a row over the sum of their weights (the largest
    counted 1), the longest row, and the largest sum of |q k| * scale, in 64 bits."""
    q, k, v = (x[n].cuda().double() for n in "qkv")
    B, Hq, D = q.shape
    bs, Hkv = k.shape[1:3]
    q = q.unflatten(1, (Hkv, -1))
    starts = x["starts"] or [0, B]
    out, size, top = torch.zeros_like(q), torch.zeros_like(q), 0.0
    thin, longest = torch.zeros_like(q[..., :1]), 0

    def rows(table, n):
        c = torch.arange(n)
        at = (torch.as_tensor(table)[c // bs] * bs + c % bs).cuda()
        return [t.flatten(0, 1)[at].transpose(0, 1) for t in (k, v)]       # [Hkv, n, D]

    shared = [rows(t, n) for t, n in zip(x["ptab"], x["plens"])] if x["plens"] else []
    for b in range(B):
        parts = [s for p, s in enumerate(shared) if starts[p] <= b < starts[p + 1]]
        parts.append(rows(x["tab"][b], x["lens"][b]))
        kb, vb = (torch.cat([p[i] for p in parts], 1) for i in range(2))
        if kb.shape[1] == 0:
            continue
        w = torch.softmax(scale * q[b] @ kb.mT, -1)
        out[b], size[b] = w @ vb, w @ vb.abs()
        thin[b], longest = kb.shape[1] * w.amax(-1, keepdim=True), max(longest, kb.shape[1])
        top = max(top, abs(scale) * (q[b].abs() @ kb.abs().mT).max().item())
    return out.flatten(1, 2), size.flatten(1, 2), thin.flatten(1, 2), longest, top


def compare(got, x, scale, score_error):
    """score_error: what a score may be off by, absolutely. A weight is off by that much, relatively,
    the common maximum by as much again, and by half a step of its type; fp16 weights carry 2^6,
    so those below the normal range are off by 2^-31 of the largest at most, each. The sums over
    keys run in fp32 (a tile's 8 steps of 16 keys, a tile after another, then the slots)."""
    ref, size, thin, n, top = exact(x, scale)
    eps = torch.finfo(x["q"].dtype).eps
    tol = eps / 2 * ref.abs() + (eps / 2 + 2 * score_error(top) + (n / 16 + 8) * 2.0 ** -23) * size
    if x["q"].dtype is torch.float16:
        tol = tol + thin * 2.0 ** -31 * x["v"].nan_to_num().abs().max().item() + 2.0 ** -25
    bad = ~((got.double() - ref).abs() <= tol * (1 + eps) + 1e-30)
    assert not bad.any(), (bad.nonzero()[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])


def test_reference_is_the_oracle():
    from oracle import gqa_prefix
    rng = np.random.default_rng(1)
    x = make(rng, 5, 6, 2, 64, 16, "bf16", [129, 40], [0, 2, 4], [7, 0, 40, 33, 1])
    out, size, _, _, _ = exact(x, 0.3)
    q, k, v = (x[n].double().numpy() for n in "qkv")
    ref = gqa_prefix.attention(q, k, v, x["ptab"], x["plens"], x["starts"], x["tab"], x["lens"], 0.3)
    assert np.allclose(out.cpu(), ref[0], atol=1e-12) and np.allclose(size.cpu(), ref[1], atol=1e-12)


@pytest.mark.parametrize("vd", ["bf16", "fp16"])
@pytest.mark.parametrize("name", CASES)
def test_several_key_tiles_a_stream(gq, name, vd):
    assert reaches(name, torch.cuda.get_device_properties(0).multi_processor_count)
    x = batch(name, vd, np.random.default_rng(len(name)))
    D = x["q"].shape[2]
    scale = D ** -0.5
    got = call(gq, x, scale)
    # A score: D / 16 steps of fp32 sums (2^-23 each, of sum |q k|), the scale and the exponent's
    # argument in fp32.
    compare(got, x, scale, lambda top: (D / 16 + 8) * 2.0 ** -23 * top)
    assert torch.equal(call(gq, x, scale), got)


@pytest.mark.parametrize("vd", ["bf16", "fp16"])
@pytest.mark.parametrize("name", CASES)
def test_maxima_that_move_at_every_tile(gq, name, vd):
    # Key c scores c / 10 for some rows, -c / 10 and c / 1000 for others: over a tile of 64 keys
    # the first grow by 2^9, past the growth that a maximum may lag behind by.
    rng = np.random.default_rng(3)
    D, _, G, Hkv = CASES[name][:4]

    def k_of(i, c):
        k = np.zeros((Hkv, D))
        k[:, 1] = c / 40.0
        return k

    x = batch(name, vd, rng, spread=0.0, k_of=k_of)
    heads = torch.arange(G * Hkv)
    x["q"][:, :, 1] = torch.tensor([16.0, -16.0, 0.15625])[heads % 3].to(TORCH_V[vd])
    got = call(gq, x, 0.25)
    # One product of a score is not zero and exact in fp32; the scale, the maximum and the
    # argument of the exponent round once each.
    compare(got, x, 0.25, lambda top: 4 * 2.0 ** -24 * top)


@pytest.mark.parametrize("name", ["single-d64", "single-d128", "single-d256", "own-d256"])
def test_small_fp16_weights_keep_their_bits(gq, name):
    # The first key of each tile outweighs the others by 2^20.4 and has a value of 0: the output is
    # made of weights that fp16, without the factor of 2^6, holds to 4 bits (12.13 steps of 2^-24).
    D, _, _, Hkv = CASES[name][:4]
    tile, high = 64 if D == 256 else 128, 14.140625

    def k_of(i, c):
        k = np.zeros((Hkv, D))
        k[:, 2] = high * (c % tile == 0)
        return k

    x = batch(name, "fp16", np.random.default_rng(4), spread=0.0, k_of=k_of)
    x["q"][:, :, 2] = 1.0
    x["v"] = torch.where(x["v"].isnan(), x["v"], 256.0 * (1.0 - x["k"][..., 2:3] / high))
    ref, size, thin, _, _ = exact(x, 1.0)
    # What is allowed is far below what 12 steps for 12.13 would make of it.
    rows = ref.abs().amax(-1) > 1e-3
    allowed = 2.0 ** -11 * (ref.abs() + size) + thin * 2.0 ** -23
    assert rows.any() and (allowed < 0.3 * 0.0107 * ref.abs())[rows].all()
    got = call(gq, x, 1.0)
    compare(got, x, 1.0, lambda top: 4 * 2.0 ** -24 * top)
