"""GB300-native bf16 forward attention.

The product is the C ABI in ``include/attn_fwd.h`` (library
``_lib/libattn_fwd.so``, built by ``build.py``). This module is the thin Python
binding: it checks tensors, marshals pointers and sizes, and calls the library on
the current torch stream; for the norm, rotation and paged-cache calls its compiled
part does so (``_lib/attn_binding-*.so``). Every step of the computation runs in the CUDA kernel;
there is no Python or CPU fallback - if the library is missing, calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os

from .build import LIB_DIR, binding_path, lib_path

LAYOUTS = {"bhsd": 0, "bshd": 1}
ROUNDINGS = {"rtne": 0, "rtna": 1, "rtz": 2}

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = -1
ATTN_ERR_UNSUPPORTED = -2
ATTN_ERR_MISALIGNED = -3
ATTN_ERR_ALIASING = -4
ATTN_ERR_NO_DEVICE = -5
ATTN_ERR_ARCH = -6
ATTN_ERR_LAUNCH = -7
ATTN_ERR_TIMEOUT = -8
ATTN_ERR_TOO_LARGE = -9
ATTN_ERR_SCRATCH = -10
ATTN_ERR_SEQLENS = -11
ATTN_ERR_DEBUG_CHECK = -12
ATTN_ERR_INDEX = -13
ATTN_FLAG_CAUSAL = 1
ATTN_FLAG_SPLIT_TAIL = 2
ATTN_FLAG_INTERLEAVED = 4

_libs: dict = {}


class AttnError(RuntimeError):
    """A nonzero status from the C library."""

    def __init__(self, status: int, msg: str):
        super().__init__(f"attn_fwd failed ({status}): {msg}")
        self.status = status


def load_library(debug: bool | None = None) -> ctypes.CDLL:
    """Load ``libattn_fwd.so``, or its debug flavour ``libattn_fwd_debug.so`` when
    ``debug`` (default: the environment variable ATTN_FWD_DEBUG=1). Raises if the
    library has not been built."""
    if debug is None:
        debug = os.environ.get("ATTN_FWD_DEBUG") == "1"
    if debug in _libs:
        return _libs[debug]
    path = lib_path(debug)
    if not os.path.exists(path):
        raise RuntimeError(
            f"CUDA library not built: {path} is missing. Run "
            f"`python -m bf16_forward_attention_gb300.build{' --debug' if debug else ''}` (needs nvcc).")
    lib = ctypes.CDLL(path)
    i64 = ctypes.c_int64
    lib.attn_fwd.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_int, i64, i64, i64, i64, i64,
                                                     ctypes.c_float, ctypes.c_int, ctypes.c_void_p]
    lib.attn_fwd.restype = ctypes.c_int
    lib.attn_status_str.argtypes = [ctypes.c_int]
    lib.attn_status_str.restype = ctypes.c_char_p
    lib.attn_fwd_last_error.argtypes = []
    lib.attn_fwd_last_error.restype = ctypes.c_int
    lib.attn_fwd_version.argtypes = []
    lib.attn_fwd_version.restype = ctypes.c_int
    lib.attn_fwd_timeout_selftest.argtypes = lib.attn_fwd.argtypes + [ctypes.c_uint64, ctypes.c_int]
    lib.attn_fwd_timeout_selftest.restype = ctypes.c_int
    lib.attn_fwd_splitkv.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_int, i64, i64, i64, i64, i64,
                                                             ctypes.c_float, ctypes.c_int,
                                                             ctypes.c_int, ctypes.c_void_p, i64,
                                                             ctypes.c_void_p]
    lib.attn_fwd_splitkv.restype = ctypes.c_int
    lib.attn_fwd_splitkv_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, ctypes.c_int]
    lib.attn_fwd_splitkv_workspace_bytes.restype = i64
    lib.attn_fwd_split_tail_items.argtypes = [i64, i64, i64, i64]
    lib.attn_fwd_split_tail_items.restype = ctypes.c_int
    lib.attn_fwd_splitkv_num_splits.argtypes = [i64, i64, i64, i64]
    lib.attn_fwd_splitkv_num_splits.restype = ctypes.c_int
    lib.attn_fwd_splitkv_noalloc.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_int, i64, i64, i64,
                                                                     i64, i64, ctypes.c_float,
                                                                     ctypes.c_int, ctypes.c_int,
                                                                     ctypes.c_void_p]
    lib.attn_fwd_splitkv_noalloc.restype = ctypes.c_int
    lib.attn_fwd_ex.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_int, i64, i64, i64, i64, i64, i64,
                                                        ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                                        ctypes.c_void_p]
    lib.attn_fwd_ex.restype = ctypes.c_int
    lib.attn_fwd_varlen.argtypes = ([ctypes.c_void_p] * 6 + [i64] * 7
                                    + [ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_void_p])
    lib.attn_fwd_varlen.restype = ctypes.c_int
    lib.attn_fwd_host_workspace_bytes.argtypes = [i64] * 6
    lib.attn_fwd_host_workspace_bytes.restype = i64
    lib.attn_fwd_host.argtypes = ([ctypes.c_void_p] * 4 + [ctypes.c_int] + [i64] * 6
                                  + [ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, i64,
                                     ctypes.c_void_p])
    lib.attn_fwd_host.restype = ctypes.c_int
    lib.attn_fwd_varlen_host_workspace_bytes.argtypes = [i64] * 6
    lib.attn_fwd_varlen_host_workspace_bytes.restype = i64
    lib.attn_fwd_varlen_host.argtypes = ([ctypes.c_void_p] * 6 + [i64] * 6
                                         + [ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                            ctypes.c_void_p, i64, ctypes.c_void_p])
    lib.attn_fwd_varlen_host.restype = ctypes.c_int
    lib.attn_fwd_debug_build.argtypes = []
    lib.attn_fwd_debug_build.restype = ctypes.c_int
    lib.attn_fwd_debug_selftest.argtypes = lib.attn_fwd.argtypes
    lib.attn_fwd_debug_selftest.restype = ctypes.c_int
    vp, ci, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.attn_fwd_lse.argtypes = [vp] * 5 + [ci] + [i64] * 6 + [cf, ci, ci, vp]
    lib.attn_fwd_lse.restype = ci
    lib.attn_fwd_varlen_lse.argtypes = [vp] * 7 + [i64] * 7 + [cf, ci, ci, vp]
    lib.attn_fwd_varlen_lse.restype = ci
    lib.attn_bwd.argtypes = [vp] * 9 + [ci] + [i64] * 6 + [cf, ci, ci, vp, i64, vp]
    lib.attn_bwd.restype = ci
    lib.attn_bwd_timeout_selftest.argtypes = lib.attn_bwd.argtypes + [ctypes.c_uint64, ci]
    lib.attn_bwd_timeout_selftest.restype = ci
    lib.attn_bwd_workspace_bytes.argtypes = [i64] * 6
    lib.attn_bwd_workspace_bytes.restype = i64
    lib.attn_bwd_varlen.argtypes = [vp] * 11 + [i64] * 8 + [cf, ci, ci, vp, i64, vp]
    lib.attn_bwd_varlen.restype = ci
    lib.attn_bwd_varlen_workspace_bytes.argtypes = [i64] * 8
    lib.attn_bwd_varlen_workspace_bytes.restype = i64
    lib.attn_fwd_prefix.argtypes = [vp] * 8 + [ci] + [i64] * 7 + [cf, ci, ci, vp, i64, vp]
    lib.attn_fwd_prefix.restype = ci
    lib.attn_fwd_prefix_workspace_bytes.argtypes = [i64] * 7
    lib.attn_fwd_prefix_workspace_bytes.restype = i64
    lib.attn_qk_norm_rope.argtypes = [vp] * 13 + [i64] * 7 + [cf, ci, ci, vp]
    lib.attn_qk_norm_rope.restype = ci
    lib.attn_qk_norm_rope_paged.argtypes = [vp] * 16 + [ci] + [i64] * 10 + [cf, ci, ci, vp]
    lib.attn_qk_norm_rope_paged.restype = ci
    lib.attn_qk_norm_rope_bwd.argtypes = [vp] * 19 + [i64] * 7 + [cf, ci, ci, vp, i64, vp]
    lib.attn_qk_norm_rope_bwd.restype = ci
    lib.attn_qk_norm_rope_bwd_workspace_bytes.argtypes = [i64] * 5
    lib.attn_qk_norm_rope_bwd_workspace_bytes.restype = i64
    lib.attn_fwd_paged.argtypes = [vp] * 8 + [ci] + [i64] * 9 + [cf, ci, ci, vp, i64, vp]
    lib.attn_fwd_paged.restype = ci
    lib.attn_fwd_paged_timeout_selftest.argtypes = lib.attn_fwd_paged.argtypes + [ctypes.c_uint64]
    lib.attn_fwd_paged_timeout_selftest.restype = ci
    lib.attn_fwd_paged_workspace_bytes.argtypes = [i64] * 7 + [ci]
    lib.attn_fwd_paged_workspace_bytes.restype = i64
    lib.attn_cache_evict.argtypes = [vp] * 7 + [ci] + [i64] * 9 + [vp, i64, vp]
    lib.attn_cache_evict.restype = ci
    lib.attn_cache_evict_workspace_bytes.argtypes = [i64] * 6
    lib.attn_cache_evict_workspace_bytes.restype = i64
    _libs[debug] = lib
    return lib


def status_str(status: int) -> str:
    return load_library().attn_status_str(int(status)).decode()


def attn_fwd_raw(q_ptr: int, k_ptr: int, v_ptr: int, out_ptr: int, layout: int, B: int, H: int,
                 Sq: int, Sk: int, d: int, scale: float, rounding_mode: int, stream: int) -> int:
    """Direct call of the C entry point ``attn_fwd``; returns its status code."""
    return load_library().attn_fwd(q_ptr, k_ptr, v_ptr, out_ptr, layout, B, H, Sq, Sk, d,
                                   ctypes.c_float(scale), rounding_mode, stream)


def attn_fwd_timeout_selftest_raw(q_ptr: int, k_ptr: int, v_ptr: int, out_ptr: int, layout: int,
                                  B: int, H: int, Sq: int, Sk: int, d: int, scale: float,
                                  rounding_mode: int, stream: int, timeout_ns: int,
                                  flags: int = 0) -> int:
    """Direct call of ``attn_fwd_timeout_selftest`` (a launch whose device-side
    wait must time out; see include/attn_fwd.h)."""
    return load_library().attn_fwd_timeout_selftest(q_ptr, k_ptr, v_ptr, out_ptr, layout, B, H, Sq,
                                                    Sk, d, ctypes.c_float(scale), rounding_mode,
                                                    stream, timeout_ns, flags)


def attn_fwd_splitkv_raw(q_ptr: int, k_ptr: int, v_ptr: int, out_ptr: int, layout: int, B: int,
                         H: int, Sq: int, Sk: int, d: int, scale: float, rounding_mode: int,
                         num_splits: int, workspace_ptr: int, workspace_bytes: int,
                         stream: int) -> int:
    """Direct call of the C entry point ``attn_fwd_splitkv``; returns its status."""
    return load_library().attn_fwd_splitkv(q_ptr, k_ptr, v_ptr, out_ptr, layout, B, H, Sq, Sk, d,
                                           ctypes.c_float(scale), rounding_mode, num_splits,
                                           workspace_ptr, workspace_bytes, stream)


def attn_fwd_splitkv_noalloc_raw(q_ptr: int, k_ptr: int, v_ptr: int, out_ptr: int, layout: int,
                                 B: int, H: int, Sq: int, Sk: int, d: int, scale: float,
                                 rounding_mode: int, num_splits: int, stream: int) -> int:
    """Direct call of ``attn_fwd_splitkv_noalloc``: split-KV whose workspace is the
    library's fixed device scratch array, for callers that cannot allocate device
    memory (see include/attn_fwd.h). Returns its status code."""
    return load_library().attn_fwd_splitkv_noalloc(q_ptr, k_ptr, v_ptr, out_ptr, layout, B, H, Sq,
                                                   Sk, d, ctypes.c_float(scale), rounding_mode,
                                                   num_splits, stream)


def splitkv_workspace_bytes(B: int, H: int, Sq: int, Sk: int, num_splits: int, d: int = 128) -> int:
    n = load_library().attn_fwd_splitkv_workspace_bytes(B, H, Sq, Sk, d, num_splits)
    if n < 0:
        raise AttnError(int(n), status_str(int(n)))
    return int(n)


def splitkv_num_splits(B: int, H: int, Sq: int, Sk: int) -> int:
    n = load_library().attn_fwd_splitkv_num_splits(B, H, Sq, Sk)
    if n < 0:
        raise AttnError(int(n), status_str(int(n)))
    return int(n)


def attn_fwd_splitkv(q, k, v, *, num_splits: int | None = None, layout: str = "bhsd",
                     scale: float | None = None, rounding: str = "rtne", out=None,
                     workspace=None):
    """attn_fwd with the key range split over several CTAs (see include/attn_fwd.h).

    ``workspace``: a CUDA tensor of at least ``splitkv_workspace_bytes(...)`` bytes;
    allocated here if not given (the C entry point itself never allocates).
    """
    import torch

    if layout not in LAYOUTS or rounding not in ROUNDINGS:
        raise ValueError("unknown layout or rounding mode")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D tensor")
    B, H, Sq, D = _dims(q, layout)
    Bk, Hk, Sk, Dk = _dims(k, layout)
    if (Bk, Hk, Dk) != (B, H, D) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("shape mismatch")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on one device")
    if num_splits is None:
        num_splits = splitkv_num_splits(B, H, Sq, Sk)
    need = splitkv_workspace_bytes(B, H, Sq, Sk, num_splits, D)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check_workspace(workspace, q.device)
    if out is None:
        out = torch.empty_like(q)
    _check_out(out, q)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on_device(q.device):
        stream = torch.cuda.current_stream(q.device).cuda_stream
        st = attn_fwd_splitkv_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                  LAYOUTS[layout], B, H, Sq, Sk, D, float(scale),
                                  ROUNDINGS[rounding], num_splits, workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), stream)
    if st != ATTN_OK:
        raise AttnError(st, status_str(st))
    return out


def split_tail_items(B: int, Hq: int, Sq: int, Sk: int) -> int:
    """Items of an ``attn_fwd_ex(..., split_tail=True)`` call of this size that run on
    pairs of CTAs on the current device (0: the flag changes nothing), or a negative
    status (see include/attn_fwd.h)."""
    return load_library().attn_fwd_split_tail_items(B, Hq, Sq, Sk)


def attn_fwd_ex_raw(q_ptr: int, k_ptr: int, v_ptr: int, out_ptr: int, layout: int, B: int, Hq: int,
                    Hkv: int, Sq: int, Sk: int, d: int, scale: float, rounding_mode: int,
                    flags: int, stream: int) -> int:
    """Direct call of ``attn_fwd_ex`` (grouped-query heads, causal flag)."""
    return load_library().attn_fwd_ex(q_ptr, k_ptr, v_ptr, out_ptr, layout, B, Hq, Hkv, Sq, Sk, d,
                                      ctypes.c_float(scale), rounding_mode, flags, stream)


def attn_fwd_ex(q, k, v, *, causal: bool = False, layout: str = "bhsd",
                scale: float | None = None, rounding: str = "rtne", out=None,
                split_tail: bool = False):
    """attn_fwd with grouped-query heads (k, v may have fewer heads than q, a divisor
    of q's) and an optional causal mask aligned at the bottom right.

    ``split_tail``: run the items of the last, partial wave on pairs of CTAs, each
    taking half of the key range (ATTN_FLAG_SPLIT_TAIL; no effect with the mask).
    Faster when that wave is short, but an item's bits then depend on the size
    of the call."""
    import torch

    if layout not in LAYOUTS or rounding not in ROUNDINGS:
        raise ValueError("unknown layout or rounding mode")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D tensor")
    B, Hq, Sq, D = _dims(q, layout)
    Bk, Hkv, Sk, Dk = _dims(k, layout)
    if (Bk, Dk) != (B, D) or tuple(v.shape) != tuple(k.shape) or Hq % Hkv:
        raise ValueError("shape mismatch")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on one device")
    if out is None:
        out = torch.empty_like(q)
    _check_out(out, q)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on_device(q.device):
        stream = torch.cuda.current_stream(q.device).cuda_stream
        st = attn_fwd_ex_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                             LAYOUTS[layout], B, Hq, Hkv, Sq, Sk, D, float(scale),
                             ROUNDINGS[rounding],
                             (ATTN_FLAG_CAUSAL if causal else 0)
                             | (ATTN_FLAG_SPLIT_TAIL if split_tail else 0), stream)
    if st != ATTN_OK:
        raise AttnError(st, status_str(st))
    return out


def attn_fwd_varlen_raw(q_ptr: int, k_ptr: int, v_ptr: int, out_ptr: int, cu_q_ptr: int,
                        cu_k_ptr: int, B: int, Hq: int, Hkv: int, total_q: int, total_k: int,
                        max_seqlen_q: int, d: int, scale: float, rounding_mode: int, flags: int,
                        stream: int) -> int:
    """Direct call of ``attn_fwd_varlen`` (packed variable-length batch)."""
    return load_library().attn_fwd_varlen(q_ptr, k_ptr, v_ptr, out_ptr, cu_q_ptr, cu_k_ptr, B, Hq,
                                          Hkv, total_q, total_k, max_seqlen_q, d,
                                          ctypes.c_float(scale), rounding_mode, flags, stream)


def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, *,
                    causal: bool = False, scale: float | None = None, rounding: str = "rtne",
                    out=None):
    """Attention over a packed batch of variable-length sequences.

    q: (total_q, Hq, 128), k and v: (total_k, Hkv, 128), bf16 CUDA tensors packed
    token after token; cu_seqlens_q / cu_seqlens_k: int32 CUDA tensors of B + 1
    offsets; max_seqlen_q: a bound on every sequence's query count. Invalid
    offsets are found on the device: check ``attn_fwd_last_error()`` after a sync.
    """
    import torch

    if rounding not in ROUNDINGS:
        raise ValueError("unknown rounding mode")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CUDA tensor")
        if t.dim() != 3 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous (tokens, heads, d) tensor")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda
                or t.dim() != 1 or not t.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous 1-D int32 CUDA tensor")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 2:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both have B + 1 >= 2 entries")
    total_q, Hq, D = q.shape
    total_k, Hkv, Dk = k.shape
    if Dk != D or tuple(v.shape) != tuple(k.shape) or Hq % Hkv:
        raise ValueError("shape mismatch")
    if not (q.device == k.device == v.device == cu_seqlens_q.device == cu_seqlens_k.device):
        raise ValueError("q, k, v and the offsets must be on one device")
    if out is None:
        out = torch.empty_like(q)
    _check_out(out, q)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on_device(q.device):
        stream = torch.cuda.current_stream(q.device).cuda_stream
        st = attn_fwd_varlen_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                 cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                                 cu_seqlens_q.numel() - 1, Hq, Hkv, total_q, total_k,
                                 int(max_seqlen_q), D, float(scale), ROUNDINGS[rounding],
                                 ATTN_FLAG_CAUSAL if causal else 0, stream)
    if st != ATTN_OK:
        raise AttnError(st, status_str(st))
    return out


def _check_bf16(named, dim: int, form: str):
    """Every (name, tensor) is a contiguous bf16 CUDA tensor of `dim` dimensions on
    one device."""
    import torch

    tensor, bf16 = torch.Tensor, torch.bfloat16
    first = None
    for name, t in named:
        if not isinstance(t, tensor) or t.dtype != bf16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CUDA tensor")
        if t.dim() != dim or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {form} tensor")
        index = t.get_device()
        if first is None:
            first = index
        elif index != first:
            raise ValueError(f"{name} must be on {named[0][0]}'s device")


def _check_offsets(named, device):
    import torch

    for name, t in named:
        if (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda
                or t.dim() != 1 or not t.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous 1-D int32 CUDA tensor")
        if t.device != device:
            raise ValueError("q, k, v and the offsets must be on one device")
    if named[0][1].numel() != named[1][1].numel() or named[0][1].numel() < 2:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both have B + 1 >= 2 entries")


def _lse_like(lse, shape, device):
    """lse as given (checked), or a new one."""
    import torch

    if lse is None:
        return torch.empty(shape, dtype=torch.float32, device=device)
    if (not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 or tuple(lse.shape) != shape
            or not lse.is_contiguous() or lse.device != device):
        raise ValueError(f"lse must be a contiguous fp32 tensor of shape {shape} on {device}")
    return lse


def _call(fn, *args):
    """A C entry point whose nonzero status is raised."""
    st = fn(*args)
    if st != ATTN_OK:
        raise AttnError(int(st), status_str(st))


@functools.lru_cache(maxsize=4096)
def _workspace_of(lib, entry: str, device: int, *sizes: int) -> int:
    """Bytes that a *_workspace_bytes entry point asks for at these sizes. They depend on the
    device's SM count beside the sizes, so they are looked up once."""
    n = getattr(lib, entry)(*sizes)
    if n < 0:
        raise AttnError(int(n), status_str(int(n)))
    return int(n)


def _stream_of(t) -> int:
    """The raw handle of the current stream of t's device. torch.cuda.current_stream wraps it in
    an object first (2.8 us of a small call's 35), so the call beneath it is taken, where this
    torch has it: it is not part of torch's public interface."""
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return raw(t.get_device())


def _here() -> int:
    """The current CUDA device, -1 without one."""
    import torch

    return torch.cuda.current_device() if torch.cuda.is_available() else -1


def attn_fwd_lse(q, k, v, *, causal: bool = False, layout: str = "bhsd",
                 scale: float | None = None, rounding: str = "rtne", out=None, lse=None):
    """attn_fwd_ex that also returns each query row's log-sum-exp: (out, lse), lse
    fp32 of shape (B, Hq, Sq) in either layout. ``attn_bwd`` takes both. Like every call here it
    records nothing for torch's autograd: the gradients are what ``attn_bwd`` returns."""
    import torch

    if layout not in LAYOUTS or rounding not in ROUNDINGS:
        raise ValueError("unknown layout or rounding mode")
    _check_bf16((("q", q), ("k", k), ("v", v)), 4, "4-D")
    B, Hq, Sq, D = _dims(q, layout)
    Bk, Hkv, Sk, Dk = _dims(k, layout)
    if (Bk, Dk) != (B, D) or tuple(v.shape) != tuple(k.shape) or Hkv < 1 or Hq % Hkv:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out(out, q)
    lse = _lse_like(lse, (B, Hq, Sq), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on_device(q.device):
        _call(load_library().attn_fwd_lse, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
              lse.data_ptr(), LAYOUTS[layout], B, Hq, Hkv, Sq, Sk, D, float(scale),
              ROUNDINGS[rounding], ATTN_FLAG_CAUSAL if causal else 0,
              _stream_of(q))
    return out, lse


def attn_fwd_varlen_lse(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, *,
                        causal: bool = False, scale: float | None = None, rounding: str = "rtne",
                        out=None, lse=None):
    """attn_fwd_varlen that also returns each query row's log-sum-exp: (out, lse), lse
    fp32 of shape (Hq, total_q). Tokens of no sequence are left as they were."""
    import torch

    if rounding not in ROUNDINGS:
        raise ValueError("unknown rounding mode")
    _check_bf16((("q", q), ("k", k), ("v", v)), 3, "(tokens, heads, d)")
    _check_offsets((("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)), q.device)
    total_q, Hq, D = q.shape
    total_k, Hkv, Dk = k.shape
    if Dk != D or tuple(v.shape) != tuple(k.shape) or Hkv < 1 or Hq % Hkv:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out(out, q)
    lse = _lse_like(lse, (Hq, total_q), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on_device(q.device):
        _call(load_library().attn_fwd_varlen_lse, q.data_ptr(), k.data_ptr(), v.data_ptr(),
              out.data_ptr(), lse.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
              cu_seqlens_q.numel() - 1, Hq, Hkv, total_q, total_k, int(max_seqlen_q), D,
              float(scale), ROUNDINGS[rounding], ATTN_FLAG_CAUSAL if causal else 0,
              _stream_of(q))
    return out, lse


def bwd_workspace_bytes(B: int, Hq: int, Hkv: int, Sq: int, Sk: int, d: int = 128) -> int:
    """Device workspace attn_bwd needs on the current device."""
    return _workspace_of(load_library(), "attn_bwd_workspace_bytes", _here(), B, Hq, Hkv, Sq, Sk, d)


def bwd_varlen_workspace_bytes(B: int, Hq: int, Hkv: int, total_q: int, total_k: int,
                               max_seqlen_q: int, max_seqlen_k: int, d: int = 128) -> int:
    """Device workspace attn_bwd_varlen needs on the current device."""
    return _workspace_of(load_library(), "attn_bwd_varlen_workspace_bytes", _here(), B, Hq, Hkv, total_q,
                         total_k, max_seqlen_q, max_seqlen_k, d)


def _grads(q, k, v, dq, dk, dv, workspace, need: int):
    """The gradients and the workspace as given (checked), or new ones."""
    import torch

    got = []
    for name, g, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if g is None:
            g = torch.empty_like(like)
        elif (not isinstance(g, torch.Tensor) or g.dtype != torch.bfloat16 or g.shape != like.shape
              or not g.is_contiguous() or g.device != like.device):
            raise ValueError(f"{name} must be a contiguous bf16 tensor shaped like {name[1:]} on its device")
        got.append(g)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _check_workspace(workspace, q.device)
    return (*got, workspace)


def attn_bwd(dout, q, k, v, out, lse, *, causal: bool = False, layout: str = "bhsd",
             scale: float | None = None, rounding: str = "rtne", dq=None, dk=None, dv=None,
             workspace=None):
    """Gradients (dq, dk, dv) of ``out, lse = attn_fwd_lse(q, k, v, ...)`` for the
    output's gradient ``dout`` (none is taken of lse), with the forward call's causal,
    layout and scale.

    ``workspace``: a CUDA tensor of at least ``bwd_workspace_bytes(...)`` bytes;
    allocated here if not given (the C entry point itself never allocates)."""
    import torch

    if layout not in LAYOUTS or rounding not in ROUNDINGS:
        raise ValueError("unknown layout or rounding mode")
    _check_bf16((("q", q), ("k", k), ("v", v), ("dout", dout), ("out", out)), 4, "4-D")
    B, Hq, Sq, D = _dims(q, layout)
    Bk, Hkv, Sk, Dk = _dims(k, layout)
    if ((Bk, Dk) != (B, D) or v.shape != k.shape or dout.shape != q.shape or out.shape != q.shape
            or Hkv < 1 or Hq % Hkv):
        raise ValueError("shape mismatch")
    if lse is None:
        raise ValueError("lse must be what attn_fwd_lse returned")
    lse = _lse_like(lse, (B, Hq, Sq), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    lib = load_library()
    with _on_device(q.device):
        dq, dk, dv, workspace = _grads(
            q, k, v, dq, dk, dv, workspace,
            _workspace_of(lib, "attn_bwd_workspace_bytes", q.get_device(), B, Hq, Hkv, Sq, Sk, D))
        _call(lib.attn_bwd, dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
              out.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
              LAYOUTS[layout], B, Hq, Hkv, Sq, Sk, D, float(scale), ROUNDINGS[rounding],
              ATTN_FLAG_CAUSAL if causal else 0, workspace.data_ptr(),
              workspace.numel() * workspace.element_size(),
              _stream_of(q))
    return dq, dk, dv


def attn_bwd_varlen(dout, q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                    max_seqlen_k: int, *, causal: bool = False, scale: float | None = None,
                    rounding: str = "rtne", dq=None, dk=None, dv=None, workspace=None):
    """Gradients (dq, dk, dv) of ``out, lse = attn_fwd_varlen_lse(q, k, v, ...)``. Tokens of
    no sequence are left as they were (unset where the gradients are allocated here).
    Invalid offsets are found on the device: check ``attn_fwd_last_error()`` after a sync."""
    import torch

    if rounding not in ROUNDINGS:
        raise ValueError("unknown rounding mode")
    _check_bf16((("q", q), ("k", k), ("v", v), ("dout", dout), ("out", out)), 3, "(tokens, heads, d)")
    _check_offsets((("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)), q.device)
    total_q, Hq, D = q.shape
    total_k, Hkv, Dk = k.shape
    if (Dk != D or v.shape != k.shape or dout.shape != q.shape or out.shape != q.shape or Hkv < 1
            or Hq % Hkv):
        raise ValueError("shape mismatch")
    if lse is None:
        raise ValueError("lse must be what attn_fwd_varlen_lse returned")
    lse = _lse_like(lse, (Hq, total_q), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    B = cu_seqlens_q.numel() - 1
    lib = load_library()
    with _on_device(q.device):
        dq, dk, dv, workspace = _grads(
            q, k, v, dq, dk, dv, workspace,
            _workspace_of(lib, "attn_bwd_varlen_workspace_bytes", q.get_device(), B, Hq, Hkv, total_q,
                          total_k, int(max_seqlen_q), int(max_seqlen_k), D))
        _call(lib.attn_bwd_varlen, dout.data_ptr(), q.data_ptr(), k.data_ptr(),
              v.data_ptr(), out.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
              dv.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, Hq, Hkv, total_q,
              total_k, int(max_seqlen_q), int(max_seqlen_k), D, float(scale), ROUNDINGS[rounding],
              ATTN_FLAG_CAUSAL if causal else 0, workspace.data_ptr(),
              workspace.numel() * workspace.element_size(),
              _stream_of(q))
    return dq, dk, dv


def prefix_workspace_bytes(B: int, Hq: int, Hkv: int, Sq: int, Sp: int, cap: int, d: int = 128) -> int:
    """Device workspace attn_fwd_prefix needs on the current device."""
    return _workspace_of(load_library(), "attn_fwd_prefix_workspace_bytes", _here(), B, Hq, Hkv, Sq, Sp, cap, d)


def attn_fwd_prefix(q, k_prefix, v_prefix, k, v, seqlens, *, causal: bool = False,
                    layout: str = "bhsd", scale: float | None = None, rounding: str = "rtne",
                    out=None, lse=None, workspace=None):
    """Attention of a batch whose sequences share a prefix (sampling many completions
    of one prompt): (out, lse).

    bf16 CUDA tensors, for "bshd": q (B, Sq, Hq, 128) new tokens, k_prefix and v_prefix
    (Sp, Hkv, 128) shared by all, k and v (B, cap, Hkv, 128) the sequences' own caches
    with ``seqlens`` (int32 CUDA, B) keys in use; for "bhsd" heads come before tokens.
    Every query sees the whole prefix and its own sequence's keys; with ``causal`` the
    Sq tokens are the sequence's last and see only what is before them. k_prefix and
    v_prefix may be None: no prefix. A length outside 0..cap is found on the device:
    check ``attn_fwd_last_error()`` after a sync."""
    import torch

    if layout not in LAYOUTS or rounding not in ROUNDINGS:
        raise ValueError("unknown layout or rounding mode")
    _check_bf16((("q", q), ("k", k), ("v", v)), 4, "4-D")
    B, Hq, Sq, D = _dims(q, layout)
    Bk, Hkv, cap, Dk = _dims(k, layout)
    if (Bk, Dk) != (B, D) or v.shape != k.shape or Hkv < 1 or Hq % Hkv:
        raise ValueError("shape mismatch")
    if (k_prefix is None) != (v_prefix is None):
        raise ValueError("k_prefix and v_prefix must be given together")
    Sp = 0
    if k_prefix is not None:
        _check_bf16((("k_prefix", k_prefix), ("v_prefix", v_prefix)), 3, "3-D")
        Sp = k_prefix.shape[0 if layout == "bshd" else 1]
        if k_prefix.device != q.device:
            raise ValueError("k_prefix must be on q's device")
        if (v_prefix.shape != k_prefix.shape or k_prefix.shape[2] != D
                or k_prefix.shape[1 if layout == "bshd" else 0] != Hkv):
            raise ValueError("shape mismatch")
    if (not isinstance(seqlens, torch.Tensor) or seqlens.dtype != torch.int32 or not seqlens.is_cuda
            or tuple(seqlens.shape) != (B,) or not seqlens.is_contiguous()):
        raise TypeError("seqlens must be a contiguous int32 CUDA tensor of B entries")
    if seqlens.device != q.device:
        raise ValueError("seqlens must be on q's device")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out(out, q)
    lse = _lse_like(lse, (B, Hq, Sq), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    lib = load_library()
    with _on_device(q.device):
        if workspace is None:
            need = _workspace_of(lib, "attn_fwd_prefix_workspace_bytes", q.get_device(), B, Hq, Hkv, Sq, Sp,
                                 cap, D)
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            _check_workspace(workspace, q.device)
        _call(lib.attn_fwd_prefix, q.data_ptr(), k_prefix.data_ptr() if Sp else None,
              v_prefix.data_ptr() if Sp else None, k.data_ptr(), v.data_ptr(), seqlens.data_ptr(),
              out.data_ptr(), lse.data_ptr(), LAYOUTS[layout], B, Hq, Hkv, Sq, Sp, cap, D,
              float(scale), ROUNDINGS[rounding], ATTN_FLAG_CAUSAL if causal else 0,
              workspace.data_ptr(), workspace.numel() * workspace.element_size(),
              _stream_of(q))
    return out, lse


def _native():
    """The compiled part of this binding (csrc/binding.cpp) and the library's entry points as it
    takes them: what checks the tensors of the calls below, whose GPU time may be a few
    microseconds."""
    lib = load_library()
    if not hasattr(lib, "entry"):
        lib.entry = {n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                     for n in ("attn_qk_norm_rope", "attn_qk_norm_rope_paged", "attn_qk_norm_rope_bwd",
                               "attn_qk_norm_rope_bwd_workspace_bytes", "attn_fwd_paged",
                               "attn_fwd_paged_workspace_bytes", "attn_cache_evict",
                               "attn_cache_evict_workspace_bytes")}
    return _binding or _load_binding(), lib.entry


_binding = None


def _load_binding():
    """``_lib/attn_binding-*.so`` for this torch and Python; raises if it has not been built."""
    global _binding
    import importlib.machinery
    import importlib.util

    import torch  # noqa: F401  (the module's symbols are torch's)

    path = binding_path()
    if not os.path.exists(path):
        raise RuntimeError(f"binding not built: {path or LIB_DIR + '/attn_binding-*.so'} is missing. Run "
                           "`python -m bf16_forward_attention_gb300.build` beside a torch with CUDA.")
    loader = importlib.machinery.ExtensionFileLoader("attn_binding", path)
    spec = importlib.util.spec_from_file_location("attn_binding", path, loader=loader)
    _binding = importlib.util.module_from_spec(spec)
    loader.exec_module(_binding)
    return _binding


def _results(got):
    """What a call of the compiled binding returned, or its nonzero status raised."""
    if got.__class__ is int:
        raise AttnError(got, status_str(got))
    return got


def attn_qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, *, eps: float = 1e-6,
                      interleaved: bool = False, layout: str = "bhsd", rounding: str = "rtne",
                      q_out=None, k_out=None):
    """Each head's queries and keys RMS-normed, weighted and rotated by position, in one pass:
    (q_out, k_out), what attn_fwd and its relatives take.

    bf16 CUDA tensors: q (tokens, Hq, 128) and k (tokens, Hkv, 128), or 4-D in ``layout``, in
    place wherever their rows lie (views of one projection's output, say); q_weight and k_weight
    128 entries; cos and sin fp32 (max_pos, rotary_dim / 2); positions int32, (tokens,) or (B, S).
    ``interleaved``: a pair is columns (2i, 2i + 1) instead of (i, i + rotary_dim / 2).
    q_out may be q and k_out k. A position outside 0..max_pos-1 is found on the device: check
    ``attn_fwd_last_error()`` after a sync. The gradients are what ``attn_qk_norm_rope_bwd``
    returns."""
    if layout not in LAYOUTS or rounding not in ROUNDINGS:
        raise ValueError("unknown layout or rounding mode")
    native, entry = _native()
    return _results(native.norm_rope(entry["attn_qk_norm_rope"], q, k, q_weight, k_weight, cos, sin, positions, q_out,
                                     k_out, eps, LAYOUTS[layout], ROUNDINGS[rounding],
                                     ATTN_FLAG_INTERLEAVED if interleaved else 0))


def attn_qk_norm_rope_paged(q, k, v, q_weight, k_weight, cos, sin, positions, slots, k_pages, v_pages, *,
                            eps: float = 1e-6, interleaved: bool = False, layout: str = "bhsd",
                            rounding: str = "rtne", q_out=None):
    """``attn_qk_norm_rope`` for tokens that are added to a paged cache: the rotated keys and the
    values v go to the cache, the rotated queries are returned.

    k_pages and v_pages: bf16 CUDA tensors (n_pages, page_size, Hkv, 128) for "bshd", (n_pages,
    Hkv, page_size, 128) for "bhsd", each page contiguous. slots: int32, one a token like
    positions, the place page * page_size + place in the page, or -1 for a token that is not
    stored (padding); the slots of a call differ. A slot out of range is found on the device."""
    if layout not in LAYOUTS or rounding not in ROUNDINGS:
        raise ValueError("unknown layout or rounding mode")
    native, entry = _native()
    return _results(native.norm_rope_paged(entry["attn_qk_norm_rope_paged"], q, k, q_weight, k_weight, cos, sin,
                                           positions, v, slots, k_pages, v_pages, q_out, eps, LAYOUTS[layout],
                                           ROUNDINGS[rounding], ATTN_FLAG_INTERLEAVED if interleaved else 0))[0]


def qk_norm_rope_bwd_workspace_bytes(B: int, S: int, Hq: int, Hkv: int, d: int = 128) -> int:
    """Device workspace attn_qk_norm_rope_bwd needs on the current device."""
    return _workspace_of(load_library(), "attn_qk_norm_rope_bwd_workspace_bytes", _here(), B, S, Hq, Hkv, d)


def attn_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions, *, eps: float = 1e-6,
                          interleaved: bool = False, layout: str = "bhsd", rounding: str = "rtne", dq=None,
                          dk=None, dq_weight=None, dk_weight=None, workspace=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of ``attn_qk_norm_rope`` for the gradients dq_out
    and dk_out of what it returned (attn_bwd's dq and dk); the weights' are fp32. dq may be dq_out
    and dk dk_out.

    ``workspace``: a CUDA tensor of at least ``qk_norm_rope_bwd_workspace_bytes(...)`` bytes;
    allocated here if not given (the C entry point itself never allocates)."""
    if layout not in LAYOUTS or rounding not in ROUNDINGS:
        raise ValueError("unknown layout or rounding mode")
    native, entry = _native()
    return _results(native.norm_rope_bwd(entry["attn_qk_norm_rope_bwd"], entry["attn_qk_norm_rope_bwd_workspace_bytes"],
                                         q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, dq, dk,
                                         dq_weight, dk_weight, workspace, eps, LAYOUTS[layout], ROUNDINGS[rounding],
                                         ATTN_FLAG_INTERLEAVED if interleaved else 0))


def paged_workspace_bytes(B: int, Hq: int, Hkv: int, Sq: int, page_size: int, max_pages: int, *,
                          with_mass: bool = False, d: int = 128) -> int:
    """Device workspace attn_fwd_paged needs on the current device (``with_mass``: whether it is
    given a mass)."""
    return _workspace_of(load_library(), "attn_fwd_paged_workspace_bytes", _here(), B, Hq, Hkv, Sq, page_size,
                         max_pages, d, int(with_mass))


def attn_fwd_paged(q, k_pages, v_pages, page_table, seqlens, *, causal: bool = False, layout: str = "bhsd",
                   scale: float | None = None, rounding: str = "rtne", out=None, lse=None, mass=None,
                   workspace=None):
    """Attention of a batch's new tokens over a paged cache: (out, lse).

    bf16 CUDA tensors, for "bshd": q (B, Sq, Hq, 128), k_pages and v_pages (n_pages, page_size,
    Hkv, 128); for "bhsd" heads come before tokens. page_table (int32 CUDA, (B, max_pages)): key j
    of sequence b is place j % page_size of page page_table[b, j // page_size]; seqlens (int32
    CUDA, B) counts each sequence's keys, the new tokens' included (``attn_qk_norm_rope_paged``
    puts them there). With ``causal`` the Sq tokens are the sequence's last and see only what is
    before them. ``mass`` (fp32, (B, Hkv, max_pages * page_size)): every key's attention weight,
    summed over the new tokens and the group's heads, is added to it. A length or page number out
    of range is found on the device: check ``attn_fwd_last_error()`` after a sync."""
    if layout not in LAYOUTS or rounding not in ROUNDINGS:
        raise ValueError("unknown layout or rounding mode")
    native, entry = _native()
    return _results(native.fwd_paged(entry["attn_fwd_paged"], entry["attn_fwd_paged_workspace_bytes"], q, k_pages,
                                     v_pages, page_table, seqlens, out, lse, mass, workspace, scale, LAYOUTS[layout],
                                     ROUNDINGS[rounding], ATTN_FLAG_CAUSAL if causal else 0))


def evict_workspace_bytes(B: int, Hkv: int, n_pages: int, page_size: int, max_pages: int, budget: int) -> int:
    """Device workspace attn_cache_evict needs."""
    return _workspace_of(load_library(), "attn_cache_evict_workspace_bytes", -1, B, Hkv, n_pages, page_size,
                         max_pages, budget)


def attn_cache_evict(k_pages, v_pages, page_table, seqlens, mass, budget: int, *, recent: int = 0,
                     layout: str = "bhsd", mass_out=None, seqlens_out=None, workspace=None):
    """A paged cache kept to ``budget`` keys a sequence: (seqlens_out, mass_out).

    Of a longer sequence, each key/value head keeps its last ``recent`` keys and the
    budget - recent of greatest mass before them (``attn_fwd_paged`` adds the masses up), moved
    together in order to the front of the sequence's pages, in place. mass_out (zero at and after
    the new lengths) may be mass, and seqlens_out seqlens. Pages and lengths out of range, and a
    page listed twice of a sequence to be cut, are found on the device: that sequence stays as it
    was; check ``attn_fwd_last_error()`` after a sync."""
    if layout not in LAYOUTS:
        raise ValueError("unknown layout")
    native, entry = _native()
    return _results(native.cache_evict(entry["attn_cache_evict"], entry["attn_cache_evict_workspace_bytes"], k_pages,
                                       v_pages, page_table, seqlens, mass, mass_out, seqlens_out, workspace,
                                       int(budget), int(recent), LAYOUTS[layout]))


def host_workspace_bytes(B: int, Hq: int, Hkv: int, Sq: int, Sk: int, d: int = 128) -> int:
    """Device workspace attn_fwd_host needs (negative: a status code)."""
    return load_library().attn_fwd_host_workspace_bytes(B, Hq, Hkv, Sq, Sk, d)


def attn_fwd_host_raw(q_ptr: int, k_ptr: int, v_ptr: int, out_ptr: int, layout: int, B: int,
                      Hq: int, Hkv: int, Sq: int, Sk: int, d: int, scale: float,
                      rounding_mode: int, flags: int, workspace_ptr: int, workspace_bytes: int,
                      stream: int) -> int:
    """Direct call of ``attn_fwd_host`` (host buffers, copies overlapped)."""
    return load_library().attn_fwd_host(q_ptr, k_ptr, v_ptr, out_ptr, layout, B, Hq, Hkv, Sq, Sk,
                                        d, ctypes.c_float(scale), rounding_mode, flags,
                                        workspace_ptr, workspace_bytes, stream)


def attn_fwd_host(q, k, v, *, causal: bool = False, layout: str = "bhsd",
                  scale: float | None = None, rounding: str = "rtne", out=None, workspace=None,
                  device=None):
    """attn_fwd_ex on CPU tensors (pinned for overlap): uploads, computes and
    downloads in overlapped chunks on ``device`` and returns ``out`` (a CPU
    tensor, pinned when allocated here). The call is asynchronous on the
    current stream: synchronize before reading ``out``, and keep q, k, v (and a
    caller-given workspace) alive until then."""
    import torch

    if layout not in LAYOUTS or rounding not in ROUNDINGS:
        raise ValueError("unknown layout or rounding mode")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CPU tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D tensor")
    B, Hq, Sq, D = _dims(q, layout)
    Bk, Hkv, Sk, Dk = _dims(k, layout)
    if (Bk, Dk) != (B, D) or tuple(v.shape) != tuple(k.shape) or Hq % Hkv:
        raise ValueError("shape mismatch")
    if out is not None:
        _check_out(out, q)
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    need = host_workspace_bytes(B, Hq, Hkv, Sq, Sk, D)
    if need < 0:
        raise AttnError(need, status_str(need))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    _check_workspace(workspace, torch.device(device))
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16).pin_memory()
    _check_out(out, q)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on_device(device):
        stream = torch.cuda.current_stream(device).cuda_stream
        st = attn_fwd_host_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                               LAYOUTS[layout], B, Hq, Hkv, Sq, Sk, D, float(scale),
                               ROUNDINGS[rounding], ATTN_FLAG_CAUSAL if causal else 0,
                               workspace.data_ptr(), workspace.numel(), stream)
    if st != ATTN_OK:
        raise AttnError(st, status_str(st))
    return out


def attn_fwd_varlen_host(q, k, v, cu_seqlens_q, cu_seqlens_k, *, causal: bool = False,
                         scale: float | None = None, rounding: str = "rtne", out=None,
                         workspace=None, device=None):
    """attn_fwd_varlen on CPU tensors (pinned for overlap): q (total_q, Hq, 128),
    k and v (total_k, Hkv, 128) bf16, cu_seqlens_q / cu_seqlens_k int32 CPU
    tensors of B + 1 offsets. Uploads, computes and downloads in overlapped chunks
    of whole sequences on ``device``; returns ``out`` (CPU). Asynchronous on the
    current stream: synchronize before reading ``out``."""
    import torch

    if rounding not in ROUNDINGS:
        raise ValueError("unknown rounding mode")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CPU tensor")
        if t.dim() != 3 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous (tokens, heads, d) tensor")
    for name, t in (("cu_seqlens_q", cu_seqlens_q), ("cu_seqlens_k", cu_seqlens_k)):
        if (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.is_cuda
                or t.dim() != 1 or not t.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous 1-D int32 CPU tensor")
    if cu_seqlens_q.numel() != cu_seqlens_k.numel() or cu_seqlens_q.numel() < 2:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both have B + 1 >= 2 entries")
    total_q, Hq, D = q.shape
    total_k, Hkv, Dk = k.shape
    if Dk != D or tuple(v.shape) != tuple(k.shape) or Hq % Hkv:
        raise ValueError("shape mismatch")
    if out is not None:
        _check_out(out, q)
    B = cu_seqlens_q.numel() - 1
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    need = load_library().attn_fwd_varlen_host_workspace_bytes(B, Hq, Hkv, total_q, total_k, D)
    if need < 0:
        raise AttnError(int(need), status_str(int(need)))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    _check_workspace(workspace, torch.device(device))
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16).pin_memory()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on_device(device):
        stream = torch.cuda.current_stream(device).cuda_stream
        st = load_library().attn_fwd_varlen_host(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), cu_seqlens_q.data_ptr(),
            cu_seqlens_k.data_ptr(), B, Hq, Hkv, total_q, total_k, D, ctypes.c_float(float(scale)),
            ROUNDINGS[rounding], ATTN_FLAG_CAUSAL if causal else 0, workspace.data_ptr(),
            workspace.numel(), stream)
    if st != ATTN_OK:
        raise AttnError(st, status_str(st))
    return out


def attn_fwd_last_error() -> int:
    return load_library().attn_fwd_last_error()


_HERE = contextlib.nullcontext()


def _on_device(device):
    """The device context for a library call: none when `device` is already the
    current CUDA device (entering torch.cuda.device costs a few microseconds, a
    noticeable share of a small call)."""
    import torch

    if torch.cuda.current_device() == device.index:
        return _HERE
    return torch.cuda.device(device)


def _dims(x, layout):
    if layout == "bhsd":
        B, H, S, D = x.shape
    else:
        B, S, H, D = x.shape
    return B, H, S, D


def _check_out(out, q):
    """The C library writes through out's pointer: it must be a contiguous bf16
    tensor shaped like q, on q's device (CUDA or host)."""
    import torch

    if (not isinstance(out, torch.Tensor) or out.dtype != torch.bfloat16
            or out.shape != q.shape or not out.is_contiguous() or out.device != q.device):
        raise ValueError("out must be a contiguous bf16 tensor shaped like q on q's device")


def _check_workspace(ws, device):
    import torch

    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {device}")


def attn_fwd(q, k, v, *, layout: str = "bhsd", scale: float | None = None,
             rounding: str = "rtne", out=None):
    """O = softmax(Q K^T * scale) V on bf16 CUDA tensors (head_dim 128).

    q: (B, H, Sq, 128) for "bhsd" or (B, Sq, H, 128) for "bshd"; k, v likewise with
    Sk. Returns ``out`` (allocated like q if not given) in the same layout, rounded
    to bf16 per ``rounding`` ("rtne", "rtna", "rtz"). Runs on the current stream.
    """
    import torch

    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}")
    if rounding not in ROUNDINGS:
        raise ValueError(f"rounding must be one of {sorted(ROUNDINGS)}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bf16 CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D tensor")
    B, H, Sq, D = _dims(q, layout)
    Bk, Hk, Sk, Dk = _dims(k, layout)
    if (Bk, Hk, Dk) != (B, H, D) or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on one device")
    if out is None:
        out = torch.empty_like(q)
    elif (out.dtype != torch.bfloat16 or out.shape != q.shape or not out.is_contiguous()
          or out.device != q.device):
        raise ValueError("out must be a contiguous bf16 tensor shaped like q on q's device")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _on_device(q.device):
        stream = torch.cuda.current_stream(q.device).cuda_stream
        st = attn_fwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                          LAYOUTS[layout], B, H, Sq, Sk, D, float(scale), ROUNDINGS[rounding],
                          stream)
    if st != ATTN_OK:
        raise AttnError(st, status_str(st))
    return out


__all__ = ["attn_fwd", "attn_fwd_raw", "attn_fwd_last_error", "attn_fwd_timeout_selftest_raw",
           "attn_fwd_splitkv", "attn_fwd_splitkv_raw", "splitkv_workspace_bytes",
           "splitkv_num_splits", "attn_fwd_splitkv_noalloc_raw", "attn_fwd_ex", "attn_fwd_ex_raw",
           "attn_fwd_varlen", "attn_fwd_varlen_raw", "ATTN_ERR_SEQLENS",
           "attn_fwd_host", "attn_fwd_host_raw", "host_workspace_bytes", "attn_fwd_varlen_host", "status_str", "load_library",
           "AttnError", "LAYOUTS", "ROUNDINGS", "lib_path", "ATTN_ERR_DEBUG_CHECK",
           "ATTN_FLAG_CAUSAL", "ATTN_FLAG_SPLIT_TAIL", "split_tail_items",
           "attn_fwd_lse", "attn_fwd_varlen_lse", "attn_bwd", "attn_bwd_varlen",
           "bwd_workspace_bytes", "bwd_varlen_workspace_bytes", "attn_fwd_prefix",
           "prefix_workspace_bytes", "ATTN_ERR_INDEX", "ATTN_FLAG_INTERLEAVED", "attn_qk_norm_rope",
           "attn_qk_norm_rope_paged", "attn_qk_norm_rope_bwd", "qk_norm_rope_bwd_workspace_bytes",
           "attn_fwd_paged", "paged_workspace_bytes", "attn_cache_evict", "evict_workspace_bytes"]
