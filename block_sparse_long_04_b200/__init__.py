"""XAttention block-sparse prefill attention for NVIDIA B200 (sm_100a).

A thin ctypes binding over libxattn.so (C ABI in include/xattn.h). Each function
has the name of the C entry point it calls and does argument marshalling only:
shapes are read from the torch tensors, pointers and the current CUDA stream are
passed through, and the status code is turned into an exception. Every step of
the computation runs in the library's CUDA kernels; there is no fallback. If the
library is missing or fails to load, the first call into it raises ImportError.

The method (page title, section):
- DuSA rebuttal (paperhub tM5mjMfFmS), Response to Q2: strided reshape of Q and K
  to (B, H, M//stride, stride*C) with a softmax over the last two dimensions.
- XAttention abstract (arXiv 2503.16428): antidiagonal sums (lower-left to
  upper-right) as the block-importance proxy.
- XAttention summary (atlas.scime.ai), Approach: keep the minimal set of blocks
  whose softmax-normalised antidiagonal mass reaches a per-head threshold.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libxattn.so")

XATTN_OK, XATTN_EINVAL, XATTN_ECAPACITY, XATTN_ECUDA, XATTN_ETIMEOUT, XATTN_EUNSUPPORTED = range(6)

# name -> (restype, argtypes); mirrors include/xattn.h
_P, _I, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "xattn_status_string": (ctypes.c_char_p, [_I]),
    "xattn_version": (_I, []),
    "xattn_score_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I]),
    "xattn_score": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _Z, _P]),
    "xattn_select_workspace_size": (_Z, [_I, _I, _I]),
    "xattn_select": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _Z, _P, _P, _Z, _P]),
    "xattn_sparse_attn": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "xattn_dense_attn": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "xattn_get_device_error": (_I, [_P]),
    "xattn_select_noalloc": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _Z, _P, _P]),
    "xattn_score_ex": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _Z, _P]),
    "xattn_select_ex": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _Z, _P, _P, _Z, _P]),
    "xattn_selftest_wait_timeout": (_I, [ctypes.c_longlong, _P, _P]),
    "xattn_selftest_exp2": (_I, [_P, _P, ctypes.c_longlong, _P]),
    "xattn_select_group_workspace_size": (_Z, [_I, _I, _I, _I]),
    "xattn_select_group": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _Z, _P, _P, _Z, _P]),
    "xattn_sparse_attn_group": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P,
                                     _P]),
    "xattn_score_select_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I]),
    "xattn_score_select": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _I, _P, _P, _P, _Z,
                                _P, _P, _Z, _P]),
}

# Structs of the decoding operators; fields mirror include/xattn.h. The wrappers pass them
# as packed bytes (made in a tenth of a ctypes.Structure's time: a decoding step is a few
# microseconds of GPU time, so the host's count); the classes name the layout.
class _Heads(ctypes.Structure):
    _fields_ = [("data", _P), ("stride_b", ctypes.c_longlong), ("stride_h", ctypes.c_longlong),
                ("stride_m", ctypes.c_longlong), ("heads", _I)]


class _Rotary(ctypes.Structure):
    _fields_ = [("pos", _P), ("inv_freq", _P), ("sections", _I * 4), ("axes", _I),
                ("interleaved", _I), ("pos_batch", _I)]


class _Cache(ctypes.Structure):
    _fields_ = [("k_pages", _P), ("v_pages", _P), ("k_scale", _P), ("v_scale", _P), ("acc", _P),
                ("ordinal", _P), ("page_table", _P), ("lens", _P), ("B", _I), ("Hkv", _I),
                ("C", _I), ("page", _I), ("num_pages", _I), ("max_pages", _I), ("kv_type", _I)]


_pack_heads = struct.Struct("Pqqqi4x").pack
_pack_rotary = struct.Struct("PP4iiii4x").pack
_pack_cache = struct.Struct("8P7i4x").pack

_S = ctypes.c_char_p     # a packed struct
SIGNATURES.update({
    "xattn_rope": (_I, [_S, _S, _S, _I, _I, _I, _I, _S, _S, _P]),
    "xattn_cache_append": (_I, [_S, _S, _S, _I, _P, _P, _P]),
    "xattn_rope_append": (_I, [_S, _S, _S, _S, _S, _I, _P, _P, _S, _P]),
    "xattn_decode_workspace_size": (_Z, [_S, _I, _I]),
    "xattn_decode_attn": (_I, [_S, _S, _F, _P, _P, _P, _P, _Z, _P]),
    "xattn_decode_attn_ex": (_I, [_S, _S, _P, _F, _P, _P, _P, _P, _Z, _P]),
    "xattn_cache_evict_workspace_size": (_Z, [_S, _I]),
    "xattn_cache_evict": (_I, [_S, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
})

XATTN_KV_BF16, XATTN_KV_E4M3 = 0, 1
XATTN_ROPE_MAX_AXES = 4

XATTN_PATTERN_ANTIDIAGONAL, XATTN_PATTERN_DIAGONAL = 0, 1
XATTN_SELECT_THRESHOLD, XATTN_SELECT_TOPK, XATTN_SELECT_RATIO = 0, 1, 2


class XAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libxattn.so not found at {LIB_PATH}; build it with "
            "`python -m block_sparse_long_04_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


class _Lazy:
    """Loads libxattn.so on first use; a missing library raises ImportError then."""
    _cdll = None

    def __getattr__(self, name):
        if _Lazy._cdll is None:
            _Lazy._cdll = _load()
        fn = getattr(_Lazy._cdll, name)
        if name in SIGNATURES:
            setattr(self, name, fn)     # the next call finds it without coming here
        return fn


_lib = _Lazy()


def status_string(status: int) -> str:
    return _lib.xattn_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != XATTN_OK:
        raise XAttnError(status, where)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def _bf16(*ts):
    for t in ts:
        if t.dtype != torch.bfloat16:
            raise TypeError("Q, K, V, O must be bfloat16")


# ------------------------------------------------------------------ sizes
def xattn_score_workspace_size(B: int, Hq: int, M: int, stride: int, causal: bool,
                               block: int = 128) -> int:
    """Bytes of the scoring workspace; sized for the `causal` flag of the call."""
    return int(_lib.xattn_score_workspace_size(B, Hq, M, stride, block, int(causal)))


def xattn_select_workspace_size(B: int, Hq: int, nb: int) -> int:
    return int(_lib.xattn_select_workspace_size(B, Hq, nb))


# ------------------------------------------------------------ entry points
def xattn_score(Q, K, stride: int, causal: bool, score_scale: float, scores, workspace,
                block: int = 128, stream=None) -> None:
    """scores[B,Hq,nb,nb] (fp32) <- strided antidiagonal block scores of Q, K."""
    _dev(Q, K, scores, workspace)
    _bf16(Q, K)
    B, Hq, M, C = Q.shape
    Hkv = K.shape[1]
    rc = _lib.xattn_score(_ptr(Q), _ptr(K), B, Hq, Hkv, M, C, stride, block, int(causal),
                          float(score_scale), _ptr(scores), _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "xattn_score")


def xattn_score_ex(Q, K, stride: int, causal: bool, pattern: int, score_scale: float, scores,
                   workspace, block: int = 128, stream=None) -> None:
    """xattn_score with a pattern: XATTN_PATTERN_ANTIDIAGONAL or XATTN_PATTERN_DIAGONAL."""
    _dev(Q, K, scores, workspace)
    _bf16(Q, K)
    B, Hq, M, C = Q.shape
    Hkv = K.shape[1]
    rc = _lib.xattn_score_ex(_ptr(Q), _ptr(K), B, Hq, Hkv, M, C, stride, block, int(causal),
                             int(pattern), float(score_scale), _ptr(scores), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "xattn_score_ex")


def xattn_select_ex(scores, param, rule: int, causal: bool, row_ptr, col_idx, nnz, workspace,
                    stream=None) -> None:
    """Selection by XATTN_SELECT_THRESHOLD (param = tau), XATTN_SELECT_TOPK (param = k)
    or XATTN_SELECT_RATIO (param = fraction of the candidates)."""
    _dev(scores, param, row_ptr, col_idx, nnz, workspace)
    B, Hq, nb, _ = scores.shape
    rc = _lib.xattn_select_ex(_ptr(scores), _ptr(param), int(rule), B, Hq, nb, int(causal),
                              _ptr(row_ptr), _ptr(col_idx), col_idx.numel(), _ptr(nnz),
                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(stream))
    _check(rc, "xattn_select_ex")


def xattn_select_group_workspace_size(B: int, Hq: int, Hkv: int, nb: int) -> int:
    return int(_lib.xattn_select_group_workspace_size(B, Hq, Hkv, nb))


def xattn_select_group(scores, param, rule: int, Hkv: int, causal: bool, row_ptr, col_idx, nnz,
                       workspace, stream=None) -> None:
    """GQA-shared kept lists (a variant): per (b, kv head, query block) the union of
    the group's per-head selections; CSR over B*Hkv*nb rows."""
    _dev(scores, param, row_ptr, col_idx, nnz, workspace)
    B, Hq, nb, _ = scores.shape
    rc = _lib.xattn_select_group(_ptr(scores), _ptr(param), int(rule), B, Hq, Hkv, nb,
                                 int(causal), _ptr(row_ptr), _ptr(col_idx), col_idx.numel(),
                                 _ptr(nnz), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "xattn_select_group")


def xattn_score_select_workspace_size(B: int, Hq: int, M: int, stride: int, causal: bool,
                                      block: int = 128) -> int:
    return int(_lib.xattn_score_select_workspace_size(B, Hq, M, stride, block, int(causal)))


def xattn_score_select(Q, K, param, rule: int, stride: int, causal: bool, score_scale: float, scores,
                       row_ptr, col_idx, nnz, workspace, block: int = 128, stream=None) -> None:
    """Scores and kept lists in one fused pass (same results as xattn_score followed
    by xattn_select_ex)."""
    _dev(Q, K, param, scores, row_ptr, col_idx, nnz, workspace)
    _bf16(Q, K)
    B, Hq, M, C = Q.shape
    Hkv = K.shape[1]
    rc = _lib.xattn_score_select(_ptr(Q), _ptr(K), B, Hq, Hkv, M, C, stride, block, int(causal),
                                 float(score_scale), _ptr(param), int(rule), _ptr(scores),
                                 _ptr(row_ptr), _ptr(col_idx), col_idx.numel(), _ptr(nnz),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    _check(rc, "xattn_score_select")


def xattn_select(scores, tau, causal: bool, row_ptr, col_idx, nnz, workspace, stream=None) -> None:
    """CSR (row_ptr, col_idx, nnz) <- per-head threshold selection of scores."""
    _dev(scores, tau, row_ptr, col_idx, nnz, workspace)
    B, Hq, nb, _ = scores.shape
    rc = _lib.xattn_select(_ptr(scores), _ptr(tau), B, Hq, nb, int(causal), _ptr(row_ptr),
                           _ptr(col_idx), col_idx.numel(), _ptr(nnz), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "xattn_select")


def xattn_select_noalloc(scores, tau, causal: bool, row_ptr, col_idx, nnz, stream=None) -> None:
    """xattn_select without a workspace, for callers that cannot allocate device
    memory while this step runs: the library keeps a fixed scratch array of
    XATTN_SELECT_NOALLOC_MAX_ROWS rows per device. Calls that overlap on the GPU
    race on that array, so issue them on one stream."""
    _dev(scores, tau, row_ptr, col_idx, nnz)
    B, Hq, nb, _ = scores.shape
    rc = _lib.xattn_select_noalloc(_ptr(scores), _ptr(tau), B, Hq, nb, int(causal), _ptr(row_ptr),
                                   _ptr(col_idx), col_idx.numel(), _ptr(nnz), _stream(stream))
    _check(rc, "xattn_select_noalloc")


XATTN_SELECT_NOALLOC_MAX_ROWS = 262144


def xattn_sparse_attn(Q, K, V, row_ptr, col_idx, causal: bool, softmax_scale: float, O,
                      lse=None, block: int = 128, stream=None) -> None:
    """O <- softmax attention of Q over the kept key blocks listed in the CSR."""
    _dev(Q, K, V, row_ptr, col_idx, O, lse)
    _bf16(Q, K, V, O)
    B, Hq, M, C = Q.shape
    Hkv = K.shape[1]
    rc = _lib.xattn_sparse_attn(_ptr(Q), _ptr(K), _ptr(V), _ptr(row_ptr), _ptr(col_idx), B, Hq,
                                Hkv, M, C, block, int(causal), float(softmax_scale), _ptr(O),
                                _ptr(lse), _stream(stream))
    _check(rc, "xattn_sparse_attn")


def xattn_sparse_attn_group(Q, K, V, row_ptr, col_idx, causal: bool, softmax_scale: float, O,
                            lse=None, block: int = 128, stream=None) -> None:
    """xattn_sparse_attn over GQA-shared lists (CSR rows per batch, KV head, query block)."""
    _dev(Q, K, V, row_ptr, col_idx, O, lse)
    _bf16(Q, K, V, O)
    B, Hq, M, C = Q.shape
    Hkv = K.shape[1]
    rc = _lib.xattn_sparse_attn_group(_ptr(Q), _ptr(K), _ptr(V), _ptr(row_ptr), _ptr(col_idx), B,
                                      Hq, Hkv, M, C, block, int(causal), float(softmax_scale),
                                      _ptr(O), _ptr(lse), _stream(stream))
    _check(rc, "xattn_sparse_attn_group")


def xattn_dense_attn(Q, K, V, causal: bool, softmax_scale: float, O, lse=None, block: int = 128,
                     stream=None) -> None:
    """O <- softmax attention of Q over every key block (dense baseline)."""
    _dev(Q, K, V, O, lse)
    _bf16(Q, K, V, O)
    B, Hq, M, C = Q.shape
    Hkv = K.shape[1]
    rc = _lib.xattn_dense_attn(_ptr(Q), _ptr(K), _ptr(V), B, Hq, Hkv, M, C, block, int(causal),
                               float(softmax_scale), _ptr(O), _ptr(lse), _stream(stream))
    _check(rc, "xattn_dense_attn")


def xattn_selftest_wait_timeout(limit_ns: int, timed_out, stream=None) -> None:
    """Diagnostic: a device wait that nothing completes must give up after
    limit_ns and raise XATTN_ETIMEOUT (read it with xattn_get_device_error)."""
    _dev(timed_out)
    _check(_lib.xattn_selftest_wait_timeout(int(limit_ns), _ptr(timed_out), _stream(stream)),
           "xattn_selftest_wait_timeout")


def xattn_selftest_exp2(x, y, stream=None) -> None:
    """y = 2^x through the FMA-pipe exponential of the attention softmax."""
    _dev(x, y)
    if x.dtype != torch.float32 or y.dtype != torch.float32 or x.numel() != y.numel():
        raise ValueError("x and y must be float32 tensors of the same size")
    _check(_lib.xattn_selftest_exp2(_ptr(x), _ptr(y), x.numel(), _stream(stream)),
           "xattn_selftest_exp2")


def xattn_get_device_error(stream=None) -> int:
    return int(_lib.xattn_get_device_error(_stream(stream)))


# ------------------------------------------------------ pipeline helpers
def max_kept(B: int, Hq: int, nb: int, causal: bool) -> int:
    """Worst-case number of kept entries (every candidate of every row)."""
    return B * Hq * (nb * (nb + 1) // 2 if causal else nb * nb)


@dataclass
class Buffers:
    """Device buffers for one prefill layer (allocated once, reused)."""
    scores: torch.Tensor
    score_ws: torch.Tensor
    select_ws: torch.Tensor
    row_ptr: torch.Tensor
    col_idx: torch.Tensor
    nnz: torch.Tensor
    O: torch.Tensor
    lse: Optional[torch.Tensor]

    @staticmethod
    def allocate(B, Hq, M, C, stride, causal, block=128, device="cuda", with_lse=False,
                 col_capacity=None):
        nb = M // block
        dev = torch.device(device)
        cap = max_kept(B, Hq, nb, causal) if col_capacity is None else col_capacity
        return Buffers(
            scores=torch.empty((B, Hq, nb, nb), dtype=torch.float32, device=dev),
            # sized for the fused score+select call, which also serves xattn_score
            score_ws=torch.empty(max(1, xattn_score_select_workspace_size(B, Hq, M, stride, causal,
                                                                          block)),
                                 dtype=torch.uint8, device=dev),
            select_ws=torch.empty(max(1, xattn_select_workspace_size(B, Hq, nb)),
                                  dtype=torch.uint8, device=dev),
            row_ptr=torch.empty(B * Hq * nb + 1, dtype=torch.int32, device=dev),
            col_idx=torch.empty(max(1, cap), dtype=torch.int32, device=dev),
            nnz=torch.zeros(1, dtype=torch.int32, device=dev),
            O=torch.empty((B, Hq, M, C), dtype=torch.bfloat16, device=dev),
            lse=torch.empty((B, Hq, M), dtype=torch.float32, device=dev) if with_lse else None,
        )


def default_score_scale(stride: int, C: int) -> float:
    """1/sqrt(stride*C): the usual attention scale for the reshaped width stride*C."""
    return 1.0 / math.sqrt(stride * C)


def xattn_prefill(Q, K, V, tau, stride: int, causal: bool, bufs: Buffers,
                  score_scale: Optional[float] = None, softmax_scale: Optional[float] = None,
                  block: int = 128, stream=None) -> torch.Tensor:
    """score -> select -> sparse attention on one stream; returns bufs.O.

    Scoring and selection run as two calls: on B200 that is faster than the fused
    xattn_score_select, whose in-kernel ranking runs on one CTA per SM behind the
    scoring tile."""
    C = Q.shape[-1]
    ss = default_score_scale(stride, C) if score_scale is None else score_scale
    sa = 1.0 / math.sqrt(C) if softmax_scale is None else softmax_scale
    xattn_score(Q, K, stride, causal, ss, bufs.scores, bufs.score_ws, block, stream)
    xattn_select(bufs.scores, tau, causal, bufs.row_ptr, bufs.col_idx, bufs.nnz, bufs.select_ws,
                 stream)
    xattn_sparse_attn(Q, K, V, bufs.row_ptr, bufs.col_idx, causal, sa, bufs.O, bufs.lse, block,
                      stream)
    return bufs.O


# ----------------------------------------------------- decoding operators
def _device_of(*ts) -> int:
    """Index of the one device of the given tensors (None entries aside)."""
    dev = -2
    for t in ts:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if i < 0:
                    raise ValueError("tensors must be CUDA tensors")
                if dev >= 0:
                    raise ValueError(f"tensors are on different devices (cuda:{dev} and cuda:{i})")
                dev = i
    return dev


def _call(fn, dev: int, stream, *args) -> None:
    """Calls a C entry point on `stream` (default: the current one of device `dev`), with
    `dev` the current device. (The raw getters avoid the objects that
    torch.cuda.current_stream() and torch.device make.)"""
    st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, st)
    if rc != XATTN_OK:
        raise XAttnError(rc, fn.__name__)


def _heads(t: torch.Tensor, what: str, shape=None) -> bytes:
    """[B, H, M, C] bf16 rows at any strides with contiguous elements, as an xattn_heads."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{what} must be bfloat16")
    size = t.shape
    if size != shape and (shape is not None or len(size) != 4):
        raise ValueError(f"{what} has shape {tuple(size)}, "
                         f"{'[B, H, M, C]' if shape is None else tuple(shape)} is wanted")
    B, H, M, C = size
    sb, sh, sm, sc = t.stride()
    if sc != 1 and C > 1:
        raise ValueError(f"the elements of a row of {what} must be contiguous")
    # the stride of a dimension of size 1 means nothing and need not be aligned
    return _pack_heads(t.data_ptr(), sb if B > 1 else 0, sh if H > 1 else 0, sm if M > 1 else 0, H)


def _workspace(t) -> tuple:
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _want(t, what: str, dtype, shape) -> None:
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, {tuple(shape)} is wanted")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


class Rotary:
    """Rotary positions: which pairs of a row turn by which axis, and how fast.

    inv_freq     fp64 CUDA tensor [pairs]
    sections     pairs of each axis, e.g. (64,) for text, (16, 24, 24) for time, height, width
    interleaved  pair p is (2p, 2p+1) instead of (p, p + pairs)
    """

    def __init__(self, inv_freq: torch.Tensor, sections, interleaved: bool = False):
        sections = tuple(int(n) for n in sections)
        if not 1 <= len(sections) <= XATTN_ROPE_MAX_AXES or min(sections) < 0:
            raise ValueError(f"sections {sections}: 1 to {XATTN_ROPE_MAX_AXES} counts are wanted")
        _want(inv_freq, "inv_freq", torch.float64, (sum(sections),))
        _device_of(inv_freq)
        self.inv_freq, self.sections, self.interleaved = inv_freq, sections, bool(interleaved)
        self._sections = sections + (0,) * (XATTN_ROPE_MAX_AXES - len(sections))

    @staticmethod
    def make(sections, base: float = 10000.0, interleaved: bool = False, device="cuda") -> "Rotary":
        """base^(-i/n) for the i-th of the n pairs of each axis."""
        f = [base ** (-torch.arange(n, dtype=torch.float64) / n) for n in sections if n]
        return Rotary(torch.cat(f).to(device), sections, interleaved)

    def _struct(self, pos: torch.Tensor, B: int, M: int) -> bytes:
        axes = len(self.sections)
        shared = pos.dim() == 2
        _want(pos, "pos", torch.int32, (M, axes) if shared else (B, M, axes))
        return _pack_rotary(pos.data_ptr(), self.inv_freq.data_ptr(), *self._sections, axes,
                            self.interleaved, 1 if shared else B)


class PagedCache:
    """A paged key-value cache: the tensors of an xattn_cache (see include/xattn.h).

    k_pages, v_pages  [num_pages, Hkv, page, C], bfloat16 or float8_e4m3fn
    page_table        int32 [B, max_pages];  lens  int32 [B], slots in use
    k_scale, v_scale  fp32 [Hkv], for float8_e4m3fn pages
    acc, ordinal      fp32 / int32 [num_pages, Hkv, page], for eviction
    The tensors are the caller's; the cache holds references and checks them once, so its
    attributes cannot be replaced (make a new PagedCache), only written into.
    """

    def __init__(self, k_pages, v_pages, page_table, lens, k_scale=None, v_scale=None, acc=None,
                 ordinal=None):
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [num_pages, Hkv, page, C]")
        if k_pages.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError("pages must be bfloat16 or float8_e4m3fn")
        P, Hkv, page, C = k_pages.shape
        B, max_pages = page_table.shape
        e4m3 = k_pages.dtype == torch.float8_e4m3fn
        _want(k_pages, "k_pages", k_pages.dtype, k_pages.shape)
        _want(v_pages, "v_pages", k_pages.dtype, k_pages.shape)
        _want(page_table, "page_table", torch.int32, (B, max_pages))
        _want(lens, "lens", torch.int32, (B,))
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to float8_e4m3fn pages")
        if e4m3:
            _want(k_scale, "k_scale", torch.float32, (Hkv,))
            _want(v_scale, "v_scale", torch.float32, (Hkv,))
        if acc is not None:
            _want(acc, "acc", torch.float32, (P, Hkv, page))
        if ordinal is not None:
            _want(ordinal, "ordinal", torch.int32, (P, Hkv, page))
        _device_of(k_pages, v_pages, page_table, lens, k_scale, v_scale, acc, ordinal)
        self.k_pages, self.v_pages, self.page_table, self.lens = k_pages, v_pages, page_table, lens
        self.k_scale, self.v_scale, self.acc, self.ordinal = k_scale, v_scale, acc, ordinal
        self.B, self.Hkv, self.C, self.page = B, Hkv, C, page
        self.num_pages, self.max_pages = P, max_pages
        self.kv_type = XATTN_KV_E4M3 if e4m3 else XATTN_KV_BF16
        self._shape = (B, Hkv, C, page, P, max_pages, self.kv_type)
        self._checked = True

    def __setattr__(self, name, value):
        # cache.lens += 1 works in place and assigns the same tensor
        if "_checked" in self.__dict__ and self.__dict__.get(name) is not value:
            raise AttributeError(f"{name}: the tensors of a PagedCache are fixed")
        self.__dict__[name] = value

    @staticmethod
    def allocate(B, Hkv, C, num_pages, max_pages, page=64, dtype=torch.bfloat16, eviction=False,
                 k_scale=None, v_scale=None, device="cuda") -> "PagedCache":
        """An empty cache (lens 0); page p of the pool is entry p of the table, row by row,
        as far as the pool goes (-1 behind)."""
        dev = torch.device(device)
        table = torch.arange(B * max_pages, dtype=torch.int32, device=dev)
        table = torch.where(table < num_pages, table, -1).view(B, max_pages)
        pool = (num_pages, Hkv, page)
        if dtype == torch.float8_e4m3fn:
            k_scale = torch.ones(Hkv, device=dev) if k_scale is None else k_scale
            v_scale = torch.ones(Hkv, device=dev) if v_scale is None else v_scale
        return PagedCache(
            torch.empty((*pool, C), dtype=dtype, device=dev),
            torch.empty((*pool, C), dtype=dtype, device=dev),
            table, torch.zeros(B, dtype=torch.int32, device=dev), k_scale, v_scale,
            torch.zeros(pool, dtype=torch.float32, device=dev) if eviction else None,
            torch.zeros(pool, dtype=torch.int32, device=dev) if eviction else None)

    def _struct(self) -> bytes:
        # the shapes are fixed; the addresses are read on every call
        return _pack_cache(self.k_pages.data_ptr(), self.v_pages.data_ptr(), _ptr(self.k_scale) or 0,
                           _ptr(self.v_scale) or 0, _ptr(self.acc) or 0, _ptr(self.ordinal) or 0,
                           self.page_table.data_ptr(), self.lens.data_ptr(), *self._shape)


def xattn_rope(Q, K, pos, rotary: Rotary, Qo, Ko, inverse: bool = False, stream=None) -> None:
    """Qo, Ko <- Q, K rotated by their positions (back, if inverse: also the gradient).

    Q, Qo [B, Hq, M, C] and K, Ko [B, Hkv, M, C] (or both None) at any strides with
    contiguous rows; pos int32 [M, axes] or [B, M, axes]. An output may be its input."""
    dev = _device_of(Q, K, pos, rotary.inv_freq, Qo, Ko)
    B, _, M, C = Q.shape
    q, qo = _heads(Q, "Q"), _heads(Qo, "Qo", Q.shape)
    if (K is None) != (Ko is None):
        raise ValueError("K and Ko go together")
    k = ko = None
    if K is not None:
        k, ko = _heads(K, "K", (B, K.shape[1], M, C)), _heads(Ko, "Ko", K.shape)
    _call(_lib.xattn_rope, dev, stream, q, k, rotary._struct(pos, B, M), int(inverse), B, M, C, qo, ko)


def _per_sequence(t, what: str, B: int):
    if t is not None:
        _want(t, what, torch.int32, (B,))
    return _ptr(t)


def xattn_cache_append(K, V, cache: PagedCache, n_new=None, seen=None, stream=None) -> None:
    """The last n_new[b] (default: all T) slots of every sequence <- K, V [B, Hkv, T, C].
    cache.lens already counts the new tokens; seen[b] (default: lens) counts every token
    of the sequence, evicted ones too."""
    dev = _device_of(K, V, cache.k_pages, n_new, seen)
    shape = (cache.B, cache.Hkv, K.shape[2], cache.C)
    _call(_lib.xattn_cache_append, dev, stream, _heads(K, "K", shape), _heads(V, "V", shape),
          cache._struct(), shape[2], _per_sequence(n_new, "n_new", cache.B),
          _per_sequence(seen, "seen", cache.B))


def xattn_rope_append(Q, K, V, pos, rotary: Rotary, cache: PagedCache, Qo, n_new=None, seen=None,
                      stream=None) -> None:
    """xattn_rope of Q (into Qo) and K, and xattn_cache_append of the rotated K and of V,
    in one launch."""
    dev = _device_of(Q, K, V, pos, rotary.inv_freq, cache.k_pages, Qo, n_new, seen)
    B, T = cache.B, K.shape[2]
    shape = (B, cache.Hkv, T, cache.C)
    _call(_lib.xattn_rope_append, dev, stream, _heads(Q, "Q", (B, Q.shape[1], T, cache.C)),
          _heads(K, "K", shape), _heads(V, "V", shape), rotary._struct(pos, B, T), cache._struct(), T,
          _per_sequence(n_new, "n_new", B), _per_sequence(seen, "seen", B),
          _heads(Qo, "Qo", Q.shape))


def xattn_decode_workspace_size(cache: PagedCache, Hq: int, weights: bool = False) -> int:
    return int(_lib.xattn_decode_workspace_size(cache._struct(), int(Hq), int(weights)))


def xattn_decode_attn(Q, cache: PagedCache, softmax_scale: float, O, workspace, lse=None,
                      weights: bool = False, acc_out=None, stream=None, n_new=None) -> None:
    """O <- attention of one query per sequence and head over the cache's slots in use.

    Q and O [B, Hq, C] or [B, Hq, 1, C]; Q at any strides, O contiguous; lse fp32 [B, Hq].
    weights adds every slot's softmax weight, summed over the query heads of its KV head,
    to cache.acc, into acc_out (default: cache.acc itself). n_new[b] is 0 for an idle
    sequence, whose O is 0 and whose weights stay, and 1 for the others (default)."""
    dev = _device_of(Q, cache.k_pages, O, workspace, lse, acc_out, n_new)
    shape = Q.shape
    if len(shape) == 3:
        B, H, C = shape
        sb, sh, sc = Q.stride()
        if Q.dtype is not torch.bfloat16:
            raise TypeError("Q must be bfloat16")
        if B != cache.B or C != cache.C or sc != 1:
            raise ValueError(f"Q has shape {tuple(shape)}, [{cache.B}, Hq, {cache.C}] with contiguous rows "
                             "is wanted")
        q = _pack_heads(Q.data_ptr(), sb if B > 1 else 0, sh if H > 1 else 0, 0, H)
    else:
        q = _heads(Q, "Q", (cache.B, shape[1], 1, cache.C))
    _want(O, "O", torch.bfloat16, shape)
    if lse is not None:
        _want(lse, "lse", torch.float32, (cache.B, shape[1]))
    if weights:
        if cache.acc is None:
            raise ValueError("weights need a cache with acc")
        if acc_out is None:
            acc_out = cache.acc
        else:
            _want(acc_out, "acc_out", torch.float32, cache.acc.shape)
    elif acc_out is not None:
        raise ValueError("acc_out needs weights=True")
    new = None if n_new is None else _per_sequence(n_new, "n_new", cache.B)
    _call(_lib.xattn_decode_attn_ex, dev, stream, q, cache._struct(), new, float(softmax_scale), O.data_ptr(),
          _ptr(lse), _ptr(acc_out), *_workspace(workspace))


def _count(n, what: str) -> int:
    n = int(n)
    if not 0 <= n < 2 ** 31:         # ctypes would cut it to 32 bits
        raise ValueError(f"{what} = {n} is not a count")
    return n


def xattn_cache_evict_workspace_size(cache: PagedCache, budget: int) -> int:
    return int(_lib.xattn_cache_evict_workspace_size(cache._struct(), _count(budget, "budget")))


def xattn_cache_evict(cache: PagedCache, budget: int, workspace, recent: int = 0, sink: int = 0,
                      seen=None, acc_out=None, ord_out=None, stream=None) -> None:
    """Keeps min(lens, budget) slots of every sequence and KV head, in slots 0..: those of the
    `recent` last and `sink` first tokens, then the largest cache.acc. acc_out and ord_out
    default to the cache's own. cache.lens is left to the caller: clamp it to budget after
    the last layer that shares it."""
    dev = _device_of(cache.k_pages, workspace, seen, acc_out, ord_out)
    if cache.acc is None or cache.ordinal is None:
        raise ValueError("eviction needs a cache with acc and ordinal")
    if acc_out is None:
        acc_out = cache.acc
    else:
        _want(acc_out, "acc_out", torch.float32, cache.acc.shape)
    if ord_out is None:
        ord_out = cache.ordinal
    else:
        _want(ord_out, "ord_out", torch.int32, cache.ordinal.shape)
    _call(_lib.xattn_cache_evict, dev, stream, cache._struct(), _count(budget, "budget"),
          _count(recent, "recent"), _count(sink, "sink"), _per_sequence(seen, "seen", cache.B), acc_out.data_ptr(), ord_out.data_ptr(),
          *_workspace(workspace))


@dataclass
class DecodeBuffers:
    """Device buffers of one layer's decoding step (allocated once, reused)."""
    Q: torch.Tensor          # rotated queries [B, Hq, 1, C]
    O: torch.Tensor
    lse: Optional[torch.Tensor]
    workspace: torch.Tensor

    @staticmethod
    def allocate(cache: PagedCache, Hq: int, weights: bool = False, with_lse: bool = False):
        dev = cache.k_pages.device
        q = torch.empty((cache.B, Hq, 1, cache.C), dtype=torch.bfloat16, device=dev)
        return DecodeBuffers(
            Q=q, O=torch.empty_like(q),
            lse=torch.empty((cache.B, Hq), dtype=torch.float32, device=dev) if with_lse else None,
            workspace=torch.empty(max(1, xattn_decode_workspace_size(cache, Hq, weights)),
                                  dtype=torch.uint8, device=dev))


def xattn_decode_step(Q, K, V, pos, rotary: Rotary, cache: PagedCache, bufs: DecodeBuffers, seen=None,
                      weights: bool = False, softmax_scale: Optional[float] = None,
                      stream=None, n_new=None) -> torch.Tensor:
    """One token per sequence through a layer after its prefill: rotate Q and K by pos, append
    K and V to the cache (cache.lens already counts the token), attend; returns bufs.O.
    weights accumulates the slots' softmax weights in cache.acc, for xattn_cache_evict. A
    batch with empty, finished or waiting sequences gives n_new: 0 for those (their rows are
    not read, their cache is left as it is, their O is 0), 1 for the others."""
    scale = 1.0 / math.sqrt(cache.C) if softmax_scale is None else softmax_scale
    xattn_rope_append(Q, K, V, pos, rotary, cache, bufs.Q, n_new, seen, stream)
    xattn_decode_attn(bufs.Q, cache, scale, bufs.O, bufs.workspace, bufs.lse, weights, n_new=n_new,
                      stream=stream)
    return bufs.O
