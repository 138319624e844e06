"""The bindings of the paged serving step refuse tensors that are not on the
current device before any library call (CPU only: tensors that say where they are)."""
import pytest
import torch


class Placed(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    is_cuda = property(lambda self: True)
    index = 0

    def get_device(self):
        return self.index


def on(index, *shape, dtype=torch.int32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Placed)
    t.index = index
    return t


B, T, MB, H, D, bf = 2, 3, 4, 2, 64, torch.bfloat16
TABLES = dict(cached_lens=(B,), new_lens=(B,), free_list=(5,), free_count=(1,),
              block_table=(B, MB), seq_lens=(B,), token_start=(B + 1,), slots=(T,),
              positions=(T,), free_left=(1,), pos_base=(B,))
ROPE = dict(q=(T, H, D), k=(T, H, D), v=(T, H, D), positions=(T,), slots=(T,), inv_freq=(D // 2,),
            q_out=(T, H, D), k_pool=(4, 16, H, D), v_pool=(4, 16, H, D), q_weight=(D,),
            k_weight=(D,))
PREFIX = dict(q=(B, H, D), k_pool=(4, 16, H, D), v_pool=(4, 16, H, D), prefix_table=(1, 3),
              prefix_lens=(1,), group_start=(2,), block_table=(B, MB), seq_lens=(B,),
              out=(B, H, D))
EXTRA = {"gqa_kv_tables": dict(block_size=16, num_blocks=4)}
CALLS = {"gqa_kv_tables": TABLES, "gqa_kv_norm_rope_append": ROPE,
         "gqa_prefix_attn_decode": PREFIX}


@pytest.fixture
def native(monkeypatch):
    from gqa_attention_weighted_gb300 import build
    build.build()
    from gqa_attention_weighted_gb300 import _native

    class Library:
        calls = 0

        def __getattr__(self, name):
            def call(*args):
                Library.calls += 1
                return 0
            return call

    monkeypatch.setattr(_native, "lib", Library())
    monkeypatch.setattr(_native, "_stream_handle", lambda stream: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return _native


def arguments(name, elsewhere=None):
    def kind(n):
        return (torch.float32 if n == "inv_freq" else bf if n in (
            "q", "k", "v", "out", "q_out", "k_pool", "v_pool", "q_weight", "k_weight")
            else torch.int32)
    return {n: on(1 if n == elsewhere else 0, *shape, dtype=kind(n))
            for n, shape in CALLS[name].items()} | EXTRA.get(name, {})


@pytest.mark.parametrize("name", CALLS)
def test_one_device_is_accepted(native, name):
    getattr(native, name)(**arguments(name))
    assert native.lib.calls == 1


@pytest.mark.parametrize("name,elsewhere", [(n, t) for n, c in CALLS.items() for t in c])
def test_a_tensor_on_another_device_is_refused(native, name, elsewhere):
    with pytest.raises(ValueError, match=f"{elsewhere} is on cuda:1"):
        getattr(native, name)(**arguments(name, elsewhere))
    assert native.lib.calls == 0


def test_a_prefix_table_needs_its_lengths(native):
    with pytest.raises(ValueError, match="prefix_lens"):
        native.gqa_prefix_attn_decode(**dict(arguments("gqa_prefix_attn_decode"), prefix_lens=None))
