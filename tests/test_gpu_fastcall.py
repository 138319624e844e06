"""The calls for prompts, drafts and pages with tensors that do not fit: each is refused by
name, whichever side checks it, nothing runs, and the same call with what fits runs (CUDA GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

B, T, MB, Hq, H, D, N, NB = 2, 5, 4, 4, 2, 64, 2, 12
PROMPT = dict(q=(T, Hq, D), k_pool=(NB, 16, H, D), v_pool=(NB, 16, H, D), token_start=(B + 1,),
              cached_lens=(B,), block_table=(B, MB), seq_lens=(B,), out=(T, Hq, D))
CALLS = {
    "gqa_prompt_attn": PROMPT, "gqa_tree_attn": dict(PROMPT, tree_mask=(T, 1)),
    "gqa_kv_fork": dict(parent=(N,), child=(N,), block_table=(B, MB), seq_lens=(B,), shares=(NB,),
                        free_list=(5,), free_count=(1,), fork_block=(N,), free_left=(1,)),
    "gqa_kv_keep": dict(cached_lens=(B,), accepted=(B, 3), accepted_count=(B,), block_table=(B, MB),
                        seq_lens=(B,), kept_lens=(B,)),
    "gqa_kv_release": dict(block_table=(B, MB), old_lens=(B,), new_lens=(B,), shares=(NB,),
                           free_list=(5,), free_count=(1,), free_left=(1,))}
EACH = [(n, t) for n, c in CALLS.items() for t in c]


@pytest.fixture(scope="module")
def gq():
    from gqa_attention_weighted_gb300 import build
    build.build()
    import gqa_attention_weighted_gb300 as pkg
    return pkg


def arguments(name):
    args = {n: torch.zeros(shape, device="cuda", dtype=torch.bfloat16 if n in (
        "q", "out", "k_pool", "v_pool") else torch.int32) for n, shape in CALLS[name].items()}
    if name in ("gqa_kv_fork", "gqa_kv_keep"):
        args["pools"] = [torch.zeros((NB, 16, H, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    if name == "gqa_kv_release":
        args["block_size"] = 16
    return args


@pytest.mark.parametrize("name", CALLS)
def test_what_fits_runs(gq, name):
    args = arguments(name)
    getattr(gq, name)(**args)
    getattr(gq, name)(**args, stream=torch.cuda.current_stream())
    getattr(gq, name)(**args, stream=torch.cuda.current_stream().cuda_stream)
    if name in ("gqa_kv_fork", "gqa_kv_keep"):
        getattr(gq, name)(**dict(args, pools=gq.KvPools(args["pools"])))
    if name == "gqa_kv_release":
        getattr(gq, name)(**dict(args, shares=None), num_blocks=NB)
        getattr(gq, name)(**args, num_blocks=NB)
    torch.cuda.synchronize()
    gq.gqa_prompt_device_status()


@pytest.mark.parametrize("name,which", EACH)
def test_another_type_is_refused(gq, name, which):
    args = arguments(name)
    args[which] = args[which].to(torch.int64 if args[which].dtype == torch.int32 else torch.float32)
    with pytest.raises(ValueError, match=which if which not in ("k_pool", "v_pool") else "pool"):
        getattr(gq, name)(**args)


@pytest.mark.parametrize("name,which", EACH)
def test_a_tensor_of_the_host_is_refused(gq, name, which):
    args = arguments(name)
    args[which] = args[which].cpu()
    with pytest.raises(ValueError, match=which):
        getattr(gq, name)(**args)


@pytest.mark.parametrize("name,which", [e for e in EACH if e[1] not in ("free_count", "free_left")])
def test_a_tensor_with_gaps_is_refused(gq, name, which):
    args = arguments(name)
    t = args[which]
    gaps = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype, device="cuda")[..., ::2]
    args[which] = gaps
    with pytest.raises(ValueError, match="contiguous" if which == "q" else which):
        getattr(gq, name)(**args)


@pytest.mark.parametrize("name,which", EACH)
def test_another_shape_is_refused(gq, name, which):
    args = arguments(name)
    t = args[which]
    args[which] = torch.zeros((*t.shape, 1), dtype=t.dtype, device="cuda")
    with pytest.raises(ValueError):
        getattr(gq, name)(**args)
    if which not in ("block_table", "free_list", "accepted", "tree_mask") and which != "shares":
        args[which] = torch.zeros((*t.shape[:-1], t.shape[-1] + 1), dtype=t.dtype, device="cuda")
        with pytest.raises(ValueError):
            getattr(gq, name)(**args)


@pytest.mark.parametrize("name", CALLS)
def test_what_is_no_tensor_is_refused(gq, name):
    for which in CALLS[name]:
        for other in ([0, 0], 7) if which in ("cached_lens", "seq_lens", "shares") else (None, 7):
            if name == "gqa_prompt_attn" and which == "cached_lens" and other is None:
                continue
            with pytest.raises((ValueError, AttributeError, TypeError)):
                getattr(gq, name)(**dict(arguments(name), **{which: other}))


def test_the_library_s_refusals_come_through(gq):
    args = arguments("gqa_prompt_attn")
    args.update(k_pool=torch.zeros((NB, 12, H, D), dtype=torch.bfloat16, device="cuda"),
                v_pool=torch.zeros((NB, 12, H, D), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(gq.GqaAvError, match="block_size=12"):
        gq.gqa_prompt_attn(**args)
    with pytest.raises(gq.GqaAvError, match="block_size=12"):
        gq.gqa_tree_attn(**args, tree_mask=torch.zeros((T, 1), dtype=torch.int32, device="cuda"))
    with pytest.raises(gq.GqaAvError, match="finite"):
        gq.gqa_prompt_attn(**arguments("gqa_prompt_attn"), scale=float("nan"))
    args = arguments("gqa_kv_fork")
    with pytest.raises(gq.GqaAvError, match="overlaps"):
        gq.gqa_kv_fork(**dict(args, free_left=args["free_count"]))
    args = arguments("gqa_kv_keep")
    with pytest.raises(gq.GqaAvError, match="overlaps"):
        gq.gqa_kv_keep(**dict(args, kept_lens=args["seq_lens"]))
    with pytest.raises(gq.GqaAvError, match="two pools overlap"):
        gq.gqa_kv_keep(**dict(args, pools=[args["pools"][0]] * 2))
    args = arguments("gqa_kv_release")
    with pytest.raises(gq.GqaAvError, match="overlaps"):
        gq.gqa_kv_release(**dict(args, free_left=args["free_count"]))
    with pytest.raises(gq.GqaAvError, match="block_size=0"):
        gq.gqa_kv_release(**dict(args, block_size=0))


def test_views_with_offsets(gq):
    # Rows of larger tensors: addresses with an offset, 16 bytes apart where they have to be.
    big = torch.arange(40, dtype=torch.int32, device="cuda")
    kept = big[3:5]
    args = dict(arguments("gqa_kv_keep"), kept_lens=kept, cached_lens=torch.tensor([5, 9], dtype=torch.int32,
                                                                                   device="cuda"))
    gq.gqa_kv_keep(**args)
    assert big[2:6].tolist() == [2, 5, 9, 5]
