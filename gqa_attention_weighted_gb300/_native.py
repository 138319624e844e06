"""ctypes binding of libgqa_av.so (include/gqa_*.h).

Argument marshalling only: every step of the reduction runs in the CUDA
library. Import fails loudly when the library has not been built; there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
import warnings
from typing import Optional

import torch

from . import build

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_PKG, "libgqa_av.so")

GQA_AV_OK = 0
GQA_AV_ERR_INVALID = 1
GQA_AV_ERR_UNSUPPORTED = 2
GQA_AV_ERR_CUDA = 3
GQA_AV_ERR_NOMEM = 4
GQA_AV_ERR_DEVICE_TIMEOUT = 5

GQA_AV_BF16 = 0
GQA_AV_FP16 = 1
MODE_AUTO, MODE_PER_HEAD, MODE_GQA = -1, 0, 1

_V_DTYPE = {torch.bfloat16: GQA_AV_BF16, torch.float16: GQA_AV_FP16}


class GqaAvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class Tuning(ctypes.Structure):
    _fields_ = [("nsplit", ctypes.c_int), ("dtile", ctypes.c_int),
                ("rows_per_stage", ctypes.c_int), ("stages", ctypes.c_int),
                ("early_stages", ctypes.c_int), ("engine", ctypes.c_int),
                ("split_mode", ctypes.c_int)]


class PlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "mode", "heads_per_cta", "head_chunk", "dtile", "rows_per_stage", "stages",
        "early_stages", "engine", "split_mode", "nsplit",
        "combine_ctas", "rows_per_split", "tiles", "ctas", "threads_per_cta", "smem_bytes",
        "ctas_per_sm")] + [
        ("workspace_bytes", ctypes.c_size_t)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIBRARY):
        raise ImportError(
            f"{LIBRARY} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIBRARY)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sizes = [I, I, I, I, I]
    lib.gqa_av_decode.argtypes = [P, P, P, P, *sizes, I, I, P]
    lib.gqa_av_decode_per_head.argtypes = [P, P, P, P, *sizes, I, P]
    lib.gqa_av_decode_tuned.argtypes = [P, P, P, P, *sizes, I, I, ctypes.POINTER(Tuning), P]
    lib.gqa_av_decode_noalloc.argtypes = [P, P, P, P, *sizes, I, I, P]
    lib.gqa_av_decode_paged.argtypes = [P, P, P, P, P, *sizes, I, I, I, I, I,
                                        ctypes.POINTER(Tuning), P]
    lib.gqa_av_plan.argtypes = [*sizes, I, I, ctypes.POINTER(Tuning), ctypes.POINTER(PlanInfo)]
    lib.gqa_av_selftest_wait_timeout.argtypes = [P, P, P, P, *sizes, I, ctypes.c_longlong, I, P]
    lib.gqa_av_workspace_bytes.argtypes = [*sizes, I, I]
    lib.gqa_av_workspace_bytes.restype = S
    lib.gqa_av_set_workspace.argtypes = [P, S]
    lib.gqa_av_device_status.argtypes = [P, I]
    lib.gqa_av_status_string.argtypes = [I]
    lib.gqa_av_status_string.restype = ctypes.c_char_p
    lib.gqa_av_last_error.argtypes = []
    lib.gqa_av_last_error.restype = ctypes.c_char_p
    lib.gqa_av_version.argtypes = []
    lib.gqa_qk_softmax_decode.argtypes = [P, P, P, P, *sizes, I, ctypes.c_float, I, P]
    lib.gqa_qk_softmax_decode_tuned.argtypes = [P, P, P, P, *sizes, I, ctypes.c_float, I, I, P]
    lib.gqa_qk_device_status.argtypes = [P, I]
    lib.gqa_qk_last_error.argtypes = []
    lib.gqa_qk_last_error.restype = ctypes.c_char_p
    lib.gqa_attn_decode.argtypes = [P, P, P, P, P, *sizes, I, ctypes.c_float, I, P]
    lib.gqa_attn_decode_tuned.argtypes = [P, P, P, P, P, *sizes, I, ctypes.c_float, I, I, I, I, I,
                                          P]
    lib.gqa_attn_plan.argtypes = [*sizes, I, I, I, I, I, I, I, ctypes.POINTER(ctypes.c_int), I]
    lib.gqa_attn_device_status.argtypes = [P, I]
    lib.gqa_attn_last_error.argtypes = []
    lib.gqa_attn_last_error.restype = ctypes.c_char_p
    L, F = ctypes.c_int64, ctypes.c_float
    lib.gqa_kv_tables.argtypes = [P] * 11 + [I] * 6 + [P]
    lib.gqa_kv_norm_rope_append.argtypes = [P, P, P, L, L, L, P, ctypes.POINTER(I), I, P, P, P, F,
                                            F, I, P, P, I, P, P, *[I] * 8, P]
    lib.gqa_kv_fork.argtypes = [P, I, L, *[P] * 9, *[I] * 6, P]
    lib.gqa_kv_keep.argtypes = [P, I, L, *[P] * 6, *[I] * 5, P]
    lib.gqa_kv_release.argtypes = [*[P] * 7, *[I] * 5, P]
    lib.gqa_kv_last_error.argtypes = []
    lib.gqa_kv_last_error.restype = ctypes.c_char_p
    lib.gqa_prefix_attn_decode.argtypes = [P] * 9 + [I] * 10 + [F, P]
    lib.gqa_prefix_device_status.argtypes = [P, I]
    lib.gqa_prefix_release_graph_workspaces.argtypes = []
    lib.gqa_prefix_selftest_wait_timeout.argtypes = [P] * 9 + [I] * 10 + [F, ctypes.c_longlong, I, P]
    lib.gqa_prefix_last_error.argtypes = []
    lib.gqa_prefix_last_error.restype = ctypes.c_char_p
    lib.gqa_prompt_attn.argtypes = [P, L, *[P] * 7, *[I] * 9, F, P]
    lib.gqa_tree_attn.argtypes = [P, L, *[P] * 5, I, *[P] * 3, *[I] * 9, F, P]
    lib.gqa_prompt_device_status.argtypes = [P, I]
    lib.gqa_prompt_release_graph_workspaces.argtypes = []
    lib.gqa_prompt_selftest_wait_timeout.argtypes = [P, L, *[P] * 7, *[I] * 9, F,
                                                     ctypes.c_longlong, I, P]
    lib.gqa_prompt_selftest_late_start.argtypes = [P, L, *[P] * 7, *[I] * 9, F, ctypes.c_longlong, I,
                                                   ctypes.c_longlong, P]
    lib.gqa_prompt_last_error.argtypes = []
    lib.gqa_prompt_last_error.restype = ctypes.c_char_p
    for f in ("gqa_kv_fork", "gqa_kv_keep", "gqa_kv_release",
              "gqa_prompt_attn", "gqa_tree_attn", "gqa_prompt_device_status",
              "gqa_prompt_release_graph_workspaces", "gqa_prompt_selftest_wait_timeout",
              "gqa_prompt_selftest_late_start"):
        getattr(lib, f).restype = I
    for f in ("gqa_kv_tables", "gqa_kv_norm_rope_append", "gqa_prefix_attn_decode",
              "gqa_prefix_device_status", "gqa_prefix_release_graph_workspaces",
              "gqa_prefix_selftest_wait_timeout"):
        getattr(lib, f).restype = I
    for f in ("gqa_attn_decode", "gqa_attn_decode_tuned", "gqa_attn_plan", "gqa_attn_device_status"):
        getattr(lib, f).restype = I
    for f in ("gqa_av_decode", "gqa_av_decode_per_head", "gqa_av_decode_tuned", "gqa_av_decode_paged",
              "gqa_av_decode_noalloc", "gqa_av_plan", "gqa_av_selftest_wait_timeout",
              "gqa_av_set_workspace", "gqa_av_device_status", "gqa_av_version",
              "gqa_qk_softmax_decode", "gqa_qk_softmax_decode_tuned", "gqa_qk_device_status"):
        getattr(lib, f).restype = I
    return lib


lib = _load()


class _NoFastcall:
    """In the place of _fastcall where it cannot be loaded: no call is taken there, so the checks
    below are made in Python (the kernels are the same, a call costs some microseconds more)."""

    def __getattr__(self, name):
        return lambda *args: None


def _load_fastcall():
    """The C++ side of the calls that check their tensors there."""
    try:
        if not build.fastcall_fits():
            raise ImportError("_fastcall is missing or was built against another torch")
        from . import _fastcall
    except ImportError as e:
        warnings.warn(f"the calls for prompts, drafts and pages check their tensors in Python: {e} "
                      "(python -c 'import __graft_entry__ as g; g.build()' builds _fastcall)")
        return _NoFastcall()
    _fastcall.bind(*[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in
                     ("gqa_prompt_attn", "gqa_tree_attn", "gqa_kv_fork", "gqa_kv_keep",
                      "gqa_kv_release")])
    return _fastcall


# Its calls return the library's status, or None where something is not as it should be: the
# checks below then say what.
_fast = _load_fastcall()


def _check(status: int) -> None:
    if status != GQA_AV_OK:
        name = lib.gqa_av_status_string(status).decode()
        msg = lib.gqa_av_last_error().decode()
        raise GqaAvError(status, f"{name}: {msg}")


# The current stream's handle without a Stream object around it (a few us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _shapes(attn: torch.Tensor, v_cache: torch.Tensor, seq_lens, out: torch.Tensor):
    if attn.dim() != 3 or v_cache.dim() != 4 or out.dim() != 3:
        raise ValueError("attn must be [B,Cmax,Hq], v_cache [B,Cmax,Hkv,D], out [B,Hq,D]")
    B, Cmax, Hq = attn.shape
    B2, C2, Hkv, D = v_cache.shape
    if (B2, C2) != (B, Cmax) or tuple(out.shape) != (B, Hq, D):
        raise ValueError(f"inconsistent shapes: attn {tuple(attn.shape)}, v "
                         f"{tuple(v_cache.shape)}, out {tuple(out.shape)}")
    for name, t in (("attn", attn), ("v_cache", v_cache), ("out", out)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if attn.dtype != torch.float32 or out.dtype != torch.float32:
        raise ValueError("attn and out must be float32")
    if v_cache.dtype not in _V_DTYPE:
        raise ValueError("v_cache must be bfloat16 or float16")
    if seq_lens is not None:
        if (not seq_lens.is_cuda or seq_lens.dtype != torch.int32 or seq_lens.numel() != B
                or not seq_lens.is_contiguous()):
            raise ValueError("seq_lens must be a contiguous CUDA int32 tensor of B elements")
    return B, Cmax, Hq, Hkv, D, _V_DTYPE[v_cache.dtype]


def _ptr(t):
    return None if t is None else t.data_ptr()


def gqa_av_decode(attn, v_cache, seq_lens, out, mode: int = MODE_AUTO, stream=None) -> torch.Tensor:
    """out[b,q,d] = sum_{c<L_b} attn[b,c,q] * v_cache[b,c,q//G,d]; writes and returns ``out``."""
    B, C, Hq, Hkv, D, vd = _shapes(attn, v_cache, seq_lens, out)
    _check(lib.gqa_av_decode(_ptr(attn), _ptr(v_cache), _ptr(seq_lens), _ptr(out),
                             B, C, Hq, Hkv, D, vd, int(mode), _stream_handle(stream)))
    return out


def gqa_av_decode_per_head(attn, v_cache, seq_lens, out, stream=None) -> torch.Tensor:
    B, C, Hq, Hkv, D, vd = _shapes(attn, v_cache, seq_lens, out)
    _check(lib.gqa_av_decode_per_head(_ptr(attn), _ptr(v_cache), _ptr(seq_lens), _ptr(out),
                                      B, C, Hq, Hkv, D, vd, _stream_handle(stream)))
    return out


def gqa_av_decode_noalloc(attn, v_cache, seq_lens, out, mode: int = MODE_AUTO,
                          stream=None) -> torch.Tensor:
    """gqa_av_decode for callers that may not allocate device memory: the
    library's fixed scratch array is used and no call allocates. The first call
    on a device looks up that array's address; make it before any capture."""
    B, C, Hq, Hkv, D, vd = _shapes(attn, v_cache, seq_lens, out)
    _check(lib.gqa_av_decode_noalloc(_ptr(attn), _ptr(v_cache), _ptr(seq_lens), _ptr(out),
                                     B, C, Hq, Hkv, D, vd, int(mode), _stream_handle(stream)))
    return out


def _tuning(t) -> Optional[Tuning]:
    if t is None:
        return None
    if isinstance(t, Tuning):
        return t
    return Tuning(int(t.get("nsplit", 0)), int(t.get("dtile", 0)),
                  int(t.get("rows_per_stage", 0)), int(t.get("stages", 0)),
                  int(t.get("early_stages", 0)), int(t.get("engine", 0)),
                  int(t.get("split_mode", 0)))


def gqa_av_decode_tuned(attn, v_cache, seq_lens, out, mode=MODE_AUTO, tuning=None,
                        stream=None) -> torch.Tensor:
    B, C, Hq, Hkv, D, vd = _shapes(attn, v_cache, seq_lens, out)
    t = _tuning(tuning)
    _check(lib.gqa_av_decode_tuned(_ptr(attn), _ptr(v_cache), _ptr(seq_lens), _ptr(out),
                                   B, C, Hq, Hkv, D, vd, int(mode),
                                   ctypes.byref(t) if t is not None else None,
                                   _stream_handle(stream)))
    return out


def gqa_av_decode_paged(attn, v_pool, block_table, seq_lens, out, mode=MODE_AUTO, tuning=None,
                        stream=None) -> torch.Tensor:
    """gqa_av_decode over a paged V cache: v_pool [num_blocks, block_size, Hkv, D],
    block_table [B, max_blocks] int32 (row c of sequence b in block
    block_table[b, c // block_size])."""
    if attn.dim() != 3 or v_pool.dim() != 4 or out.dim() != 3 or block_table.dim() != 2:
        raise ValueError("attn [B,Cmax,Hq], v_pool [blocks,block_size,Hkv,D], block_table "
                         "[B,max_blocks], out [B,Hq,D]")
    B, Cmax, Hq = attn.shape
    num_blocks, block_size, Hkv, D = v_pool.shape
    if tuple(out.shape) != (B, Hq, D) or block_table.shape[0] != B:
        raise ValueError("inconsistent shapes")
    for name, t in (("attn", attn), ("v_pool", v_pool), ("out", out), ("block_table", block_table)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if attn.dtype != torch.float32 or out.dtype != torch.float32:
        raise ValueError("attn and out must be float32")
    if v_pool.dtype not in _V_DTYPE or block_table.dtype != torch.int32:
        raise ValueError("v_pool must be bfloat16 or float16 and block_table int32")
    if seq_lens is not None and (not seq_lens.is_cuda or seq_lens.dtype != torch.int32
                                 or seq_lens.numel() != B or not seq_lens.is_contiguous()):
        raise ValueError("seq_lens must be a contiguous CUDA int32 tensor of B elements")
    t = _tuning(tuning)
    _check(lib.gqa_av_decode_paged(_ptr(attn), _ptr(v_pool), _ptr(block_table), _ptr(seq_lens),
                                   _ptr(out), B, Cmax, Hq, Hkv, D, _V_DTYPE[v_pool.dtype],
                                   block_size, num_blocks, block_table.shape[1], int(mode),
                                   ctypes.byref(t) if t is not None else None,
                                   _stream_handle(stream)))
    return out


def gqa_av_plan(B, Cmax, Hq, Hkv, D, v_dtype=GQA_AV_BF16, mode=MODE_AUTO, tuning=None) -> dict:
    info = PlanInfo()
    t = _tuning(tuning)
    _check(lib.gqa_av_plan(B, Cmax, Hq, Hkv, D, v_dtype, mode,
                           ctypes.byref(t) if t is not None else None, ctypes.byref(info)))
    return info.as_dict()


def gqa_av_workspace_bytes(B, Cmax, Hq, Hkv, D, v_dtype=GQA_AV_BF16, mode=MODE_AUTO) -> int:
    return int(lib.gqa_av_workspace_bytes(B, Cmax, Hq, Hkv, D, v_dtype, mode))


def gqa_av_set_workspace(buffer: Optional[torch.Tensor]) -> None:
    if buffer is None:
        _check(lib.gqa_av_set_workspace(None, 0))
    else:
        _check(lib.gqa_av_set_workspace(buffer.data_ptr(), buffer.numel() * buffer.element_size()))


def gqa_av_device_status(stream=None, clear: bool = True) -> None:
    _check(lib.gqa_av_device_status(_stream_handle(stream), 1 if clear else 0))


def gqa_av_status_string(status: int) -> str:
    return lib.gqa_av_status_string(status).decode()


def gqa_av_last_error() -> str:
    return lib.gqa_av_last_error().decode()


def v_dtype_code(dtype: torch.dtype) -> int:
    return _V_DTYPE[dtype]


# ------------------------------------------------------------ score step
def _check_qk(status: int) -> None:
    if status != GQA_AV_OK:
        name = lib.gqa_av_status_string(status).decode()
        raise GqaAvError(status, f"{name}: {lib.gqa_qk_last_error().decode()}")


def gqa_qk_softmax_decode(q, k_cache, seq_lens, attn, mode: int = MODE_AUTO, scale=None,
                          stream=None, engine: int = 0) -> torch.Tensor:
    """attn[b,c,q] = softmax over c < L_b of scale * q[b,q,:] . k_cache[b,c,q//G,:]
    (scale defaults to 1/sqrt(D)); rows c >= L_b of ``attn`` are left as they are."""
    if q.dim() != 3 or k_cache.dim() != 4 or attn.dim() != 3:
        raise ValueError("q must be [B,Hq,D], k_cache [B,Cmax,Hkv,D], attn [B,Cmax,Hq]")
    B, Hq, D = q.shape
    B2, Cmax, Hkv, D2 = k_cache.shape
    if (B2, D2) != (B, D) or tuple(attn.shape) != (B, Cmax, Hq):
        raise ValueError(f"inconsistent shapes: q {tuple(q.shape)}, k {tuple(k_cache.shape)}, "
                         f"attn {tuple(attn.shape)}")
    for name, t in (("q", q), ("k_cache", k_cache), ("attn", attn)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if q.dtype != torch.float32 or attn.dtype != torch.float32:
        raise ValueError("q and attn must be float32")
    if k_cache.dtype not in _V_DTYPE:
        raise ValueError("k_cache must be bfloat16 or float16")
    if seq_lens is not None and (not seq_lens.is_cuda or seq_lens.dtype != torch.int32
                                 or seq_lens.numel() != B or not seq_lens.is_contiguous()):
        raise ValueError("seq_lens must be a contiguous CUDA int32 tensor of B elements")
    sc = float(D) ** -0.5 if scale is None else float(scale)
    _check_qk(lib.gqa_qk_softmax_decode_tuned(_ptr(q), _ptr(k_cache), _ptr(seq_lens), _ptr(attn),
                                              B, Cmax, Hq, Hkv, D, _V_DTYPE[k_cache.dtype], sc,
                                              int(mode), int(engine), _stream_handle(stream)))
    return attn


def gqa_qk_device_status(stream=None, clear: bool = True) -> None:
    _check_qk(lib.gqa_qk_device_status(_stream_handle(stream), 1 if clear else 0))


# ------------------------------------------------------- fused attention
def _check_attn(status: int) -> None:
    if status != GQA_AV_OK:
        name = lib.gqa_av_status_string(status).decode()
        raise GqaAvError(status, f"{name}: {lib.gqa_attn_last_error().decode()}")


def gqa_attn_decode(q, k_cache, v_cache, seq_lens, out, mode: int = MODE_AUTO, scale=None,
                    stream=None, consumer_warps: int = 0, nsplit: int = 0,
                    split_mode: int = 0, column_blocks: int = 0) -> torch.Tensor:
    """out[b,q,:] = sum over c < L_b of softmax_c(scale * q[b,q,:] . k_cache[b,c,q//G,:])
    * v_cache[b,c,q//G,:] (scale defaults to 1/sqrt(D)); writes and returns ``out``."""
    if q.dim() != 3 or k_cache.dim() != 4 or v_cache.dim() != 4 or out.dim() != 3:
        raise ValueError("q [B,Hq,D], k_cache and v_cache [B,Cmax,Hkv,D], out [B,Hq,D]")
    B, Hq, D = q.shape
    B2, Cmax, Hkv, D2 = k_cache.shape
    if ((B2, D2) != (B, D) or tuple(v_cache.shape) != tuple(k_cache.shape)
            or tuple(out.shape) != (B, Hq, D)):
        raise ValueError(f"inconsistent shapes: q {tuple(q.shape)}, k {tuple(k_cache.shape)}, "
                         f"v {tuple(v_cache.shape)}, out {tuple(out.shape)}")
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("out", out)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if q.dtype != torch.float32 or out.dtype != torch.float32:
        raise ValueError("q and out must be float32")
    if k_cache.dtype not in _V_DTYPE or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must both be bfloat16 or both float16")
    if seq_lens is not None and (not seq_lens.is_cuda or seq_lens.dtype != torch.int32
                                 or seq_lens.numel() != B or not seq_lens.is_contiguous()):
        raise ValueError("seq_lens must be a contiguous CUDA int32 tensor of B elements")
    sc = float(D) ** -0.5 if scale is None else float(scale)
    _check_attn(lib.gqa_attn_decode_tuned(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
                                          _ptr(out), B, Cmax, Hq, Hkv, D, _V_DTYPE[k_cache.dtype],
                                          sc, int(mode), int(consumer_warps), int(nsplit),
                                          int(split_mode), int(column_blocks),
                                          _stream_handle(stream)))
    return out


def gqa_attn_plan(B, Cmax, Hq, Hkv, D, kv_dtype=GQA_AV_BF16, mode=MODE_AUTO, consumer_warps=0,
                  nsplit=0, split_mode=0, ragged=True, column_blocks=0) -> dict:
    info = (ctypes.c_int * 11)()
    _check_attn(lib.gqa_attn_plan(B, Cmax, Hq, Hkv, D, kv_dtype, mode, consumer_warps, nsplit,
                                  split_mode, column_blocks, 1 if ragged else 0, info, 11))
    keys = ("mode", "heads_per_cta", "consumer_warps", "stages", "rows_per_split", "nsplit",
            "tiles", "smem_bytes", "split_mode", "ctas", "column_blocks")
    return dict(zip(keys, list(info)))


def gqa_attn_device_status(stream=None, clear: bool = True) -> None:
    _check_attn(lib.gqa_attn_device_status(_stream_handle(stream), 1 if clear else 0))


# --------------------------------------------- block tables and cache write
GQA_KV_F32 = 2


def _check_kv(status: int) -> None:
    if status != GQA_AV_OK:
        name = lib.gqa_av_status_string(status).decode()
        raise GqaAvError(status, f"{name}: {lib.gqa_kv_last_error().decode()}")


def _device(name: str, t) -> int:
    """The device of a call's first tensor. It has to be the current one: the library's launches,
    workspaces and SM count are that device's."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor, not on {t.device}")
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return dev


def _refuse(name: str, t, dev: int, must: str) -> None:
    """Raises for a tensor that is not on ``dev`` or not what it ``must`` be."""
    at = t.get_device()
    if at >= 0 and at != dev:
        raise ValueError(f"{name} is on cuda:{at}, the current device is cuda:{dev}")
    raise ValueError(f"{name} must be {must}, not {t.dtype} {tuple(t.shape)} on {t.device}")


def _int32(name: str, t, shape, dev: int) -> None:
    """A contiguous int32 tensor of this shape on device ``dev``."""
    if (t.dtype is not torch.int32 or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(name, t, dev, f"a contiguous CUDA int32 tensor of shape {tuple(shape)}")


def _fast_stream(stream):
    """None, for the current stream, or a stream's handle."""
    return None if stream is None else _stream_handle(stream)


def _int32_at(name: str, t, shape, dev: int) -> int:
    """The address of such a tensor."""
    if (t.dtype is not torch.int32 or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(name, t, dev, f"a contiguous CUDA int32 tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _stream_on(stream, dev: int) -> Optional[int]:
    """The handle of ``stream``, or of the stream that is current on ``dev``."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream_handle(stream)


def _pools(k_pool: torch.Tensor, v_pool: torch.Tensor):
    shape, dtype = k_pool.shape, k_pool.dtype
    if len(shape) != 4 or v_pool.shape != shape:
        raise ValueError("k_pool and v_pool must both be [num_blocks, block_size, Hkv, D], not "
                         f"{tuple(shape)} and {tuple(v_pool.shape)}")
    if dtype not in _V_DTYPE or v_pool.dtype is not dtype:
        raise ValueError("k_pool and v_pool must both be bfloat16 or both float16")
    dev = _device("k_pool", k_pool)
    for name, t in (("k_pool", k_pool), ("v_pool", v_pool)):
        if t.get_device() != dev or not t.is_contiguous():
            _refuse(name, t, dev, "a contiguous CUDA tensor")
    return shape, dev


def gqa_kv_tables(cached_lens, new_lens, free_list, free_count, block_table, seq_lens, token_start,
                  slots, positions, free_left, block_size: int, num_blocks: int, pos_base=None,
                  stream=None) -> None:
    """Block-table entries, slots and positions of a step's new tokens: blocks come off the end
    of ``free_list[:free_count]`` in request order and ``block_table`` is updated in place;
    ``seq_lens``, ``token_start``, ``slots``, ``positions`` and ``free_left`` are written.
    Requests that find no blocks keep their length and get slots of -1. Where ``cached_lens[b]``
    ends inside a block, new rows go into it: it must be the request's own (gqa_kv_release)."""
    if block_table.dim() != 2 or free_list.dim() != 1 or slots.dim() != 1:
        raise ValueError("block_table must be [B, max_blocks], free_list and slots of one "
                         "dimension")
    B, max_blocks = block_table.shape
    T, n_free = slots.shape[0], free_list.shape[0]
    dev = _device("block_table", block_table)
    _int32("block_table", block_table, (B, max_blocks), dev)
    _int32("cached_lens", cached_lens, (B,), dev)
    _int32("new_lens", new_lens, (B,), dev)
    _int32("seq_lens", seq_lens, (B,), dev)
    if pos_base is not None:
        _int32("pos_base", pos_base, (B,), dev)
    _int32("free_list", free_list, (n_free,), dev)
    _int32("free_count", free_count, (1,), dev)
    _int32("free_left", free_left, (1,), dev)
    _int32("token_start", token_start, (B + 1,), dev)
    _int32("slots", slots, (T,), dev)
    _int32("positions", positions, (T,), dev)
    _check_kv(lib.gqa_kv_tables(_ptr(cached_lens), _ptr(new_lens), _ptr(pos_base), _ptr(free_list),
                                _ptr(free_count), _ptr(block_table), _ptr(seq_lens),
                                _ptr(token_start), _ptr(slots), _ptr(positions), _ptr(free_left),
                                B, T, max_blocks, n_free, int(block_size), int(num_blocks),
                                _stream_handle(stream)))


def gqa_kv_norm_rope_append(q, k, v, positions, slots, inv_freq, q_out, k_pool, v_pool,
                            q_weight=None, k_weight=None, eps: float = 1e-6,
                            weight_offset: float = 0.0, sections=None, interleaved: bool = False,
                            stream=None) -> torch.Tensor:
    """Per-head RMS norm of q [T,Hq,D] and k [T,Hkv,D] (where a weight is given), rotation by
    ``positions`` ([T], or [axes,T] with ``sections`` pairs an axis) times ``inv_freq``, queries to
    ``q_out`` (float32 or the input type), keys and values to rows ``slots`` of the pools. q, k and
    v may be views of one packed projection. Returns ``q_out``."""
    (num_blocks, block_size, Hkv, D), dev = _pools(k_pool, v_pool)
    dtype = k_pool.dtype
    if q.dim() != 3:
        raise ValueError("q must be [T,Hq,D], k and v [T,Hkv,D]")
    T, Hq = q.shape[:2]
    if (q.shape[2] != D or k.shape != (T, Hkv, D) or v.shape != (T, Hkv, D)
            or q_out.shape != (T, Hq, D)):
        raise ValueError(f"inconsistent shapes: q {tuple(q.shape)}, k {tuple(k.shape)}, v "
                         f"{tuple(v.shape)}, q_out {tuple(q_out.shape)}, pools "
                         f"{tuple(k_pool.shape)}")
    strides = []
    for name, t, heads in (("q", q, Hq), ("k", k, Hkv), ("v", v, Hkv)):
        if t.dtype is not dtype or t.get_device() != dev:
            _refuse(name, t, dev, "a CUDA tensor of the pools' type")
        st = t.stride()
        if T and (st[2] != 1 or (heads > 1 and st[1] != D)):
            raise ValueError(f"a token's heads must be contiguous in {name}")
        strides.append(st[0])
    q32 = q_out.dtype is torch.float32
    if (not (q32 or q_out.dtype is dtype) or q_out.get_device() != dev
            or not q_out.is_contiguous()):
        _refuse("q_out", q_out, dev, "a contiguous CUDA tensor, float32 or of the pools' type")
    _int32("slots", slots, (T,), dev)
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    _int32("positions", positions, (T,) if positions.dim() == 1 else (axes, T), dev)
    if (inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1
            or inv_freq.get_device() != dev or not inv_freq.is_contiguous()):
        _refuse("inv_freq", inv_freq, dev, "a contiguous CUDA float32 tensor of one dimension")
    if sections is not None and len(sections) != axes:
        raise ValueError(f"{len(sections)} sections for {axes} position axes")
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None and (t.dtype is not dtype or t.shape != (D,) or t.get_device() != dev
                              or not t.is_contiguous()):
            _refuse(name, t, dev, f"a contiguous CUDA tensor [{D}] of the pools' type")
    sec = None if sections is None else (ctypes.c_int * axes)(*[int(n) for n in sections])
    code = _V_DTYPE[dtype]
    _check_kv(lib.gqa_kv_norm_rope_append(
        _ptr(q), _ptr(k), _ptr(v), *strides, _ptr(positions), sec, axes, _ptr(inv_freq),
        _ptr(q_weight), _ptr(k_weight), float(eps), float(weight_offset), 1 if interleaved else 0,
        _ptr(slots), _ptr(q_out), GQA_KV_F32 if q32 else code, _ptr(k_pool), _ptr(v_pool), T, Hq,
        Hkv, D, 2 * inv_freq.shape[0], code, block_size, num_blocks, _stream_handle(stream)))
    return q_out


# ------------------------------------------------- forks, drafts, release
class KvPools:
    """The K and V pools of all layers (any order), each [num_blocks, block_size, ...] and all of one
    shape and type, as gqa_kv_fork and gqa_kv_keep take them. A server makes it once: it holds the
    tensors and what the library needs of them."""

    def __init__(self, pools):
        self.pools = pools = tuple(pools)
        if not pools or pools[0].dim() < 3:
            raise ValueError("pools must be tensors [num_blocks, block_size, ...], one at least")
        shape, dtype = pools[0].shape, pools[0].dtype
        self.device = _device("pools[0]", pools[0])
        for i, t in enumerate(pools):
            if (t.shape != shape or t.dtype is not dtype or t.get_device() != self.device
                    or not t.is_contiguous()):
                _refuse(f"pools[{i}]", t, self.device,
                        f"a contiguous CUDA {dtype} tensor of shape {tuple(shape)}")
        self.num_blocks, self.block_size = shape[:2]
        row = 1
        for n in shape[2:]:
            row *= n
        self.row_bytes = row * pools[0].element_size()
        at = tuple(t.data_ptr() for t in pools)
        self.array = (ctypes.c_void_p * len(pools))(*at)
        self.fast = _fast.pools(at, self.device, self.row_bytes, self.num_blocks, self.block_size)

    def args(self):
        if self.device != torch.cuda.current_device():
            raise ValueError(f"the pools are on cuda:{self.device}, the current device is "
                             f"cuda:{torch.cuda.current_device()}")
        return self.array, len(self.pools), self.row_bytes


def gqa_kv_fork(pools, parent, child, block_table, seq_lens, shares, free_list, free_count,
                fork_block, free_left, stream=None) -> None:
    """Row ``child[f]`` of ``block_table`` becomes a continuation of row ``parent[f]``: full blocks
    are shared (``shares`` += 1), a partial one is copied in all ``pools`` (a KvPools, or the
    tensors) into a block off the end of ``free_list[:free_count]``. ``seq_lens`` of the children,
    ``fork_block`` (the block of the copy, -1: none needed, -2: not served) and ``free_left`` are
    written."""
    if not isinstance(pools, KvPools):
        pools = KvPools(pools)
    rc = _fast.fork(pools.fast, parent, child, block_table, seq_lens, shares, free_list, free_count,
                    fork_block, free_left, _fast_stream(stream))
    if rc is not None:
        return _check_kv(rc)
    array, n_pools, row_bytes = pools.args()
    dev = pools.device
    if block_table.dim() != 2 or free_list.dim() != 1 or parent.dim() != 1:
        raise ValueError("block_table must be [B, max_blocks], free_list and parent of one dimension")
    B, max_blocks = block_table.shape
    N, n_free = parent.shape[0], free_list.shape[0]
    at = _int32_at
    _check_kv(lib.gqa_kv_fork(
        array, n_pools, row_bytes, at("parent", parent, (N,), dev), at("child", child, (N,), dev),
        at("block_table", block_table, (B, max_blocks), dev), at("seq_lens", seq_lens, (B,), dev),
        at("shares", shares, (pools.num_blocks,), dev), at("free_list", free_list, (n_free,), dev),
        at("free_count", free_count, (1,), dev), at("fork_block", fork_block, (N,), dev),
        at("free_left", free_left, (1,), dev), N, B, max_blocks, n_free, pools.block_size,
        pools.num_blocks, _stream_on(stream, dev)))


def gqa_kv_keep(pools, cached_lens, accepted, accepted_count, block_table, seq_lens, kept_lens,
                stream=None) -> torch.Tensor:
    """Moves the rows of accepted drafts together in all ``pools`` (a KvPools, or the tensors): row
    ``cached_lens[b] + i`` gets what row ``cached_lens[b] + accepted[b, i]`` held, for the leading
    numbers of ``accepted[b, :accepted_count[b]]`` that ascend and lie below ``seq_lens[b]``.
    Writes and returns ``kept_lens``: the cached rows and the kept ones. Blocks that hold drafted
    rows must be the request's own (gqa_kv_release)."""
    if not isinstance(pools, KvPools):
        pools = KvPools(pools)
    rc = _fast.keep(pools.fast, cached_lens, accepted, accepted_count, block_table, seq_lens,
                    kept_lens, _fast_stream(stream))
    if rc is not None:
        _check_kv(rc)
        return kept_lens
    array, n_pools, row_bytes = pools.args()
    dev = pools.device
    if block_table.dim() != 2 or accepted.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks], accepted [B, W]")
    B, max_blocks = block_table.shape
    W = accepted.shape[1]
    at = _int32_at
    _check_kv(lib.gqa_kv_keep(
        array, n_pools, row_bytes, at("cached_lens", cached_lens, (B,), dev),
        at("accepted", accepted, (B, W), dev), at("accepted_count", accepted_count, (B,), dev),
        at("block_table", block_table, (B, max_blocks), dev), at("seq_lens", seq_lens, (B,), dev),
        at("kept_lens", kept_lens, (B,), dev), B, W, max_blocks, pools.block_size,
        pools.num_blocks, _stream_on(stream, dev)))
    return kept_lens


def gqa_kv_release(block_table, old_lens, new_lens, shares, free_list, free_count, free_left,
                   block_size: int, num_blocks=None, stream=None) -> None:
    """Cuts row b of ``block_table`` from ``old_lens[b]`` rows to ``new_lens[b]`` (0: it has ended).
    Its blocks past the new end lose an owner (``shares`` -= 1); those whose last owner let go are
    appended to ``free_list[:free_count]``, and ``free_left`` gets the new count. ``shares`` [
    num_blocks] may be None where no block is shared; ``num_blocks`` is needed then.

    A row whose ``new_lens[b]`` ends inside a block that other rows own as well must not get new
    rows: they would overwrite the others'. To go back behind a fork and on from there, gqa_kv_fork
    row b into an unused row, with ``seq_lens[b]`` set to the rows to keep, and release row b
    whole."""
    rc = _fast.release(block_table, old_lens, new_lens, shares, free_list, free_count, free_left,
                       block_size, num_blocks, _fast_stream(stream))
    if rc is not None:
        return _check_kv(rc)
    if block_table.dim() != 2 or free_list.dim() != 1:
        raise ValueError("block_table must be [B, max_blocks], free_list of one dimension")
    if shares is None and num_blocks is None:
        raise ValueError("num_blocks is needed without shares")
    B, max_blocks = block_table.shape
    n_free = free_list.shape[0]
    num_blocks = int(shares.shape[0] if num_blocks is None else num_blocks)
    dev = _device("block_table", block_table)
    at = _int32_at
    _check_kv(lib.gqa_kv_release(
        at("block_table", block_table, (B, max_blocks), dev), at("old_lens", old_lens, (B,), dev),
        at("new_lens", new_lens, (B,), dev),
        None if shares is None else at("shares", shares, (num_blocks,), dev),
        at("free_list", free_list, (n_free,), dev), at("free_count", free_count, (1,), dev),
        at("free_left", free_left, (1,), dev), B, max_blocks, n_free, int(block_size), num_blocks,
        _stream_on(stream, dev)))


# ------------------------------------------- attention with shared prefixes
def _check_prefix(status: int) -> None:
    if status != GQA_AV_OK:
        name = lib.gqa_av_status_string(status).decode()
        raise GqaAvError(status, f"{name}: {lib.gqa_prefix_last_error().decode()}")


def gqa_prefix_attn_decode(q, k_pool, v_pool, prefix_table, prefix_lens, group_start, block_table,
                           seq_lens, out, scale=None, stream=None) -> torch.Tensor:
    """Decode attention over a paged cache: sequence b attends to the ``prefix_lens[p]`` rows of its
    group's ``prefix_table[p]`` (group p: ``group_start[p] <= b < group_start[p + 1]``; None: one
    group of all) and to its own ``seq_lens[b]`` rows of ``block_table[b]``. ``prefix_table`` None:
    no shared prefixes; ``block_table`` None: no own rows. q and out are [B,Hq,D] of the pools' type
    (scale defaults to 1/sqrt(D)); writes and returns ``out``. Calls on different streams and
    replays of different graphs may overlap: each stream, and each capture, has a workspace of its
    own."""
    (num_blocks, block_size, Hkv, D), dev = _pools(k_pool, v_pool)
    dtype = k_pool.dtype
    if q.dim() != 3 or q.shape[2] != D or out.shape != q.shape:
        raise ValueError(f"q and out must be [B,Hq,{D}], not {tuple(q.shape)} and "
                         f"{tuple(out.shape)}")
    B, Hq = q.shape[:2]
    for name, t in (("q", q), ("out", out)):
        if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            _refuse(name, t, dev, "a contiguous CUDA tensor of the pools' type")
    P = max_pblocks = max_blocks = 0
    if prefix_table is not None:
        if prefix_table.dim() != 2:
            raise ValueError("prefix_table must be [P, max_prefix_blocks]")
        if prefix_lens is None:
            raise ValueError("prefix_table needs prefix_lens")
        P, max_pblocks = prefix_table.shape
        _int32("prefix_table", prefix_table, (P, max_pblocks), dev)
        _int32("prefix_lens", prefix_lens, (P,), dev)
        if group_start is not None:
            _int32("group_start", group_start, (P + 1,), dev)
    if block_table is not None:
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B, max_blocks]")
        max_blocks = block_table.shape[1]
        _int32("block_table", block_table, (B, max_blocks), dev)
    if seq_lens is not None:
        _int32("seq_lens", seq_lens, (B,), dev)
    sc = float(D) ** -0.5 if scale is None else float(scale)
    _check_prefix(lib.gqa_prefix_attn_decode(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(prefix_table) if P else None,
        _ptr(prefix_lens) if P else None, _ptr(group_start) if P else None, _ptr(block_table),
        _ptr(seq_lens), _ptr(out), B, P, Hq, Hkv, D, _V_DTYPE[dtype], block_size, num_blocks,
        max_pblocks, max_blocks, sc, _stream_handle(stream)))
    return out


def gqa_prefix_device_status(stream=None, clear: bool = True) -> None:
    _check_prefix(lib.gqa_prefix_device_status(_stream_handle(stream), 1 if clear else 0))


def gqa_prefix_release_graph_workspaces() -> None:
    """Free what captured ``gqa_prefix_attn_decode`` calls hold. No graph that was captured before
    may be replayed afterwards."""
    _check_prefix(lib.gqa_prefix_release_graph_workspaces())


# -------------------------------- attention of prompts and of drafted tokens
def _check_prompt(status: int) -> None:
    if status != GQA_AV_OK:
        name = lib.gqa_av_status_string(status).decode()
        raise GqaAvError(status, f"{name}: {lib.gqa_prompt_last_error().decode()}")


def _packed_attn(q, k_pool, v_pool, token_start, cached_lens, block_table, seq_lens, out):
    """The checks of both calls; the arguments around the mask, and B, T, ... of the library's."""
    (num_blocks, block_size, Hkv, D), dev = _pools(k_pool, v_pool)
    dtype = k_pool.dtype
    if q.dim() != 3 or q.shape[2] != D or out.shape != q.shape:
        raise ValueError(f"q and out must be [T,Hq,{D}], not {tuple(q.shape)} and "
                         f"{tuple(out.shape)}")
    T, Hq = q.shape[:2]
    if q.dtype is not dtype or q.get_device() != dev:
        _refuse("q", q, dev, "a CUDA tensor of the pools' type")
    st = q.stride()
    if T and (st[2] != 1 or (Hq > 1 and st[1] != D)):
        raise ValueError("a token's heads must be contiguous in q")
    if out.dtype is not dtype or out.get_device() != dev or not out.is_contiguous():
        _refuse("out", out, dev, "a contiguous CUDA tensor of the pools' type")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    B, max_blocks = block_table.shape
    at = _int32_at
    return (dev, (q.data_ptr(), st[0], k_pool.data_ptr(), v_pool.data_ptr(),
                  at("token_start", token_start, (B + 1,), dev),
                  None if cached_lens is None else at("cached_lens", cached_lens, (B,), dev)),
            (at("block_table", block_table, (B, max_blocks), dev),
             None if seq_lens is None else at("seq_lens", seq_lens, (B,), dev),
             out.data_ptr(), B, T, Hq, Hkv, D, _V_DTYPE[dtype], block_size, num_blocks, max_blocks))


def gqa_prompt_attn(q, k_pool, v_pool, token_start, cached_lens, block_table, seq_lens, out,
                    scale=None, stream=None) -> torch.Tensor:
    """Causal attention of packed prompts, or chunks of them, over a paged cache that holds their
    rows: token ``token_start[b] + i`` is row ``cached_lens[b] + i`` of sequence b (None: 0) and
    attends to the rows up to itself that are below ``seq_lens[b]`` (None: all) of
    ``block_table[b]``. q is [T,Hq,D] of the pools' type, a view of a packed projection or not
    (scale defaults to 1/sqrt(D)); writes and returns ``out``, whose rows past the last sequence
    are left as they are. Calls on different streams and replays of different graphs may overlap."""
    rc = _fast.attend(q, k_pool, v_pool, token_start, cached_lens, None, block_table, seq_lens, out,
                      scale, _fast_stream(stream))
    if rc is not None:
        _check_prompt(rc)
        return out
    dev, before, after = _packed_attn(q, k_pool, v_pool, token_start, cached_lens, block_table,
                                      seq_lens, out)
    sc = float(q.shape[2]) ** -0.5 if scale is None else float(scale)
    _check_prompt(lib.gqa_prompt_attn(*before, *after, sc, _stream_on(stream, dev)))
    return out


def gqa_tree_attn(q, k_pool, v_pool, token_start, cached_lens, tree_mask, block_table, seq_lens,
                  out, scale=None, stream=None) -> torch.Tensor:
    """Attention of drafted tokens over a paged cache that holds their rows: token
    ``token_start[b] + i`` attends to the ``cached_lens[b]`` rows of ``block_table[b]`` and to the
    drafted rows behind them, row j where bit j % 32 of ``tree_mask[t, j // 32]`` is set (itself
    among them), all below ``seq_lens[b]`` (None: all). tree_mask is [T,words] int32; the rest as
    for gqa_prompt_attn."""
    if tree_mask is None:
        raise ValueError("gqa_tree_attn needs tree_mask")
    rc = _fast.attend(q, k_pool, v_pool, token_start, cached_lens, tree_mask, block_table, seq_lens,
                      out, scale, _fast_stream(stream))
    if rc is not None:
        _check_prompt(rc)
        return out
    if cached_lens is None:
        raise ValueError("gqa_tree_attn needs cached_lens")
    dev, before, after = _packed_attn(q, k_pool, v_pool, token_start, cached_lens, block_table,
                                      seq_lens, out)
    if tree_mask.dim() != 2:
        raise ValueError("tree_mask must be [T, words]")
    words = tree_mask.shape[1]
    mask = _int32_at("tree_mask", tree_mask, (q.shape[0], words), dev)
    sc = float(q.shape[2]) ** -0.5 if scale is None else float(scale)
    _check_prompt(lib.gqa_tree_attn(*before, mask, words, *after, sc,
                                    _stream_on(stream, dev)))
    return out


def gqa_prompt_device_status(stream=None, clear: bool = True) -> None:
    _check_prompt(lib.gqa_prompt_device_status(_stream_handle(stream), 1 if clear else 0))


def gqa_prompt_release_graph_workspaces() -> None:
    """Free what captured ``gqa_prompt_attn`` and ``gqa_tree_attn`` calls hold. No graph that was
    captured before may be replayed afterwards."""
    _check_prompt(lib.gqa_prompt_release_graph_workspaces())
