"""The C++ side of the calls for prompts, drafts and pages may be missing or of another torch: the
library is built and every call works without it, and build() sees a changed torch (CPU only)."""
import os
import subprocess
import sys

import pytest

from gqa_attention_weighted_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WITHOUT = """
import sys, warnings
{spoil}
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import gqa_attention_weighted_gb300 as gq
    assert callable(gq.gqa_av_decode) and callable(gq.gqa_prompt_attn)
assert any("_fastcall" in str(w.message) for w in seen), seen
import torch
from gqa_attention_weighted_gb300 import _native
pool, i = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
for call, args in ((gq.gqa_prompt_attn, (q, pool, pool, i, None, i.view(1, 2), None, q)),
                   (gq.gqa_kv_keep, ([pool], i, i.view(2, 1), i, i.view(2, 1), i, i)),
                   (gq.gqa_kv_release, (i.view(2, 1), i, i, i, i, i[:1], i[1:], 16))):
    try:
        call(*args)
    except ValueError as e:
        assert "CUDA" in str(e) or "cuda" in str(e), e
    else:
        raise AssertionError(call)
print("fine")
"""
SPOILS = {"missing": "sys.modules['gqa_attention_weighted_gb300._fastcall'] = None",
          "another torch": "from gqa_attention_weighted_gb300 import build\n"
                           "build.torch_kind = lambda: 'another'"}


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("spoil", SPOILS)
def test_the_package_does_without(spoil):
    r = subprocess.run([sys.executable, "-c", WITHOUT.format(spoil=SPOILS[spoil])], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "fine\n", r.stderr


def test_another_torch_is_seen(monkeypatch):
    assert build.up_to_date() and build.fastcall_up_to_date()
    monkeypatch.setattr(build, "torch_kind", lambda: "another")
    assert not build.up_to_date() and not build.fastcall_up_to_date()
    done = []
    monkeypatch.setattr(build, "build_library", lambda verbose: done.append("library"))
    monkeypatch.setattr(build, "build_fastcall", lambda verbose: done.append("fastcall"))
    assert build.build() == build.LIBRARY and done == ["fastcall"]


def test_a_compiler_that_fails_leaves_the_library(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "FASTCALL", str(tmp_path / "_fastcall.so"))
    monkeypatch.setattr(build, "fastcall_command", lambda out: [sys.executable, "-c",
                                                                "raise SystemExit('no headers')"])
    with pytest.warns(UserWarning, match="no headers"):
        assert build.build() == build.LIBRARY
    assert os.path.exists(build.LIBRARY) and not os.path.exists(build.FASTCALL)


def test_no_memory_for_pools_is_an_error_and_not_the_end():
    # 2^26 addresses (one int, named 2^26 times) in a list of their own, where there is room for
    # no more than half of it.
    code = """
import resource
from gqa_attention_weighted_gb300 import _native
many = (1 << 20,) * (1 << 26)
size = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (size + (1 << 28), size + (1 << 28)))
try:
    _native._fast.pools(many, 0, 16, 1, 8)
except MemoryError:
    print("refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "refused\n", (r.returncode, r.stderr)


def test_a_library_without_torch(monkeypatch):
    # Who has no torch wants the library alone.
    def none():
        raise ImportError("no torch")

    done = []
    monkeypatch.setattr(build, "torch_kind", none)
    monkeypatch.setattr(build, "fastcall_command", lambda out: none())
    monkeypatch.setattr(build, "build_library", lambda verbose: done.append("library"))
    monkeypatch.setattr(build, "_newer", lambda path: path != build.LIBRARY)
    with pytest.warns(UserWarning, match="no torch"):
        assert build.build() == build.LIBRARY
    assert done == ["library"]
