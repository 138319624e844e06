"""The bindings of the calls for prompts, drafts and pages refuse tensors that are not on the
current device before any library call (CPU only: tensors that say where they are)."""
import pytest
import torch

from test_binding_devices import native as binding, on  # noqa: F401  (binding: the fixture)

B, T, MB, H, D, N, bf = 2, 3, 4, 2, 64, 2, torch.bfloat16
PROMPT = dict(q=(T, H, D), k_pool=(4, 16, H, D), v_pool=(4, 16, H, D), token_start=(B + 1,),
              cached_lens=(B,), block_table=(B, MB), seq_lens=(B,), out=(T, H, D))
FORK = dict(parent=(N,), child=(N,), block_table=(B, MB), seq_lens=(B,), shares=(4,),
            free_list=(5,), free_count=(1,), fork_block=(N,), free_left=(1,))
KEEP = dict(cached_lens=(B,), accepted=(B, 3), accepted_count=(B,), block_table=(B, MB),
            seq_lens=(B,), kept_lens=(B,))
RELEASE = dict(block_table=(B, MB), old_lens=(B,), new_lens=(B,), shares=(4,), free_list=(5,),
               free_count=(1,), free_left=(1,))
CALLS = {"gqa_prompt_attn": PROMPT, "gqa_tree_attn": dict(PROMPT, tree_mask=(T, 1)),
         "gqa_kv_fork": FORK, "gqa_kv_keep": KEEP, "gqa_kv_release": RELEASE}


@pytest.fixture
def native(binding, monkeypatch):  # noqa: F811
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: 0)
    return binding


def arguments(name, elsewhere=None, pools=0):
    args = {n: on(1 if n == elsewhere else 0, *shape,
                  dtype=bf if n in ("q", "out", "k_pool", "v_pool") else torch.int32)
            for n, shape in CALLS[name].items()}
    if name in ("gqa_kv_fork", "gqa_kv_keep"):
        args["pools"] = [on(0, 4, 16, H, D, dtype=bf), on(pools, 4, 16, H, D, dtype=bf)]
    if name == "gqa_kv_release":
        args["block_size"] = 16
    return args


@pytest.mark.parametrize("name", CALLS)
def test_one_device_is_accepted(native, name):
    getattr(native, name)(**arguments(name))
    assert native.lib.calls == 1


@pytest.mark.parametrize("name,elsewhere", [(n, t) for n, c in CALLS.items() for t in c])
def test_a_tensor_on_another_device_is_refused(native, name, elsewhere):
    with pytest.raises(ValueError, match=f"{elsewhere} is on cuda:1"):
        getattr(native, name)(**arguments(name, elsewhere))
    assert native.lib.calls == 0


@pytest.mark.parametrize("name,wrong", [(n, t) for n, c in CALLS.items() for t in c])
def test_a_tensor_of_another_shape_is_refused(native, name, wrong):
    args = arguments(name)
    t = args[wrong]
    args[wrong] = on(0, *t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype)
    if wrong in ("block_table", "free_list", "accepted", "tree_mask", "shares"):
        args[wrong] = on(0, *t.shape, 1)     # their last length is free
    with pytest.raises(ValueError):
        getattr(native, name)(**args)
    assert native.lib.calls == 0


def test_pools_are_of_one_kind_and_device(native, monkeypatch):
    for name in ("gqa_kv_fork", "gqa_kv_keep"):
        with pytest.raises(ValueError, match=r"pools\[1\] is on cuda:1"):
            getattr(native, name)(**arguments(name, pools=1))
    with pytest.raises(ValueError, match=r"pools\[1\]"):
        native.KvPools([on(0, 4, 16, H, D, dtype=bf), on(0, 4, 16, H, D + 8, dtype=bf)])
    with pytest.raises(ValueError, match=r"pools\[1\]"):
        native.KvPools([on(0, 4, 16, H, D, dtype=bf), on(0, 4, 16, H, D, dtype=torch.float16)])
    handle = native.KvPools([on(0, 4, 16, H, D, dtype=bf)])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        native.gqa_kv_keep(**dict(arguments("gqa_kv_keep"), pools=handle))
    assert native.lib.calls == 0


def test_a_released_table_needs_shares_or_the_number_of_blocks(native):
    args = dict(arguments("gqa_kv_release"), shares=None)
    with pytest.raises(ValueError, match="num_blocks"):
        native.gqa_kv_release(**args)
    native.gqa_kv_release(**args, num_blocks=4)
    assert native.lib.calls == 1
