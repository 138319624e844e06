"""Batches whose sequences' own rows make an odd number of units, so that the
call's last one has a single stream: with one unit a CTA, and with several."""
import numpy as np
import pytest
import torch

from prefix_plan import OWN, plan
from test_gpu_prefix import i32, make
from test_gpu_prefix_tiles import compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    yield pkg
    pkg.gqa_prefix_device_status()


# B, Hq, Hkv, D, prefix lengths, own lengths
CASES = [
    (33, 25, 5, 64, [], [7] * 33),                                        # 165 own units
    (33, 25, 5, 128, [300], [7] * 33),
    (90, 15, 5, 64, [], [1 + 12 * i for i in range(90)]),                 # units of several sizes
    (200, 15, 5, 128, [], [(37 * i) % 296 for i in range(199)] + [9]),
    (200, 15, 5, 128, [2000], [(37 * i) % 296 for i in range(199)] + [140]),
    (300, 9, 3, 64, [], [(91 * i) % 700 for i in range(299)] + [1]),
]


@pytest.mark.parametrize("vd", ["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}-D{c[3]}-{i}" for i, c in enumerate(CASES)])
def test_last_unit_of_one_stream(gq, case, vd):
    B, Hq, Hkv, D, plens, lens = case
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    last = plan(B, Hq, Hkv, D, plens, None, lens, sms).units[-1]
    assert last.mode == OWN and last.tiles[1] == 0
    x = make(np.random.default_rng(B), B, Hq, Hkv, D, 16, vd, plens, None, lens)
    t = {n: x[n].cuda() for n in "qkv"}
    t.update({n: i32(x[n]) for n in ("ptab", "plens", "starts", "tab", "lens")})

    def call():
        out = torch.full_like(t["q"], float("nan"))
        return gq.gqa_prefix_attn_decode(t["q"], t["k"], t["v"], t["ptab"], t["plens"], t["starts"],
                                         t["tab"], t["lens"], out)

    first = call()
    gq.gqa_prefix_device_status()
    compare(first, x, D ** -0.5, lambda top: (D / 16 + 8) * 2.0 ** -23 * top)
    outs = [call() for _ in range(300)]            # the order of the warps varies
    gq.gqa_prefix_device_status()
    assert all(torch.equal(o, first) for o in outs)
