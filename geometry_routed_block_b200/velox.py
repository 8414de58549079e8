"""ctypes binding of libvelox (include/velox.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. PyTorch supplies device memory (output and scratch tensors are
allocated here with torch) and the current CUDA stream. Importing this module
fails loudly when libvelox.so has not been built; there is no fallback.

Camera / slice records are float32 tensors whose last dimension is 18, laid out
like velox_slice_t: R (9, row-major, world->camera), t (3), fx, fy, cx, cy,
znear, zfar.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
from typing import NamedTuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libvelox.so")

VELOX_OK = 0
VELOX_EINVAL = -1
VELOX_EUNSUPPORTED = -2
VELOX_ECUDA = -3
VELOX_ETIMEOUT = -4
VELOX_EBOUNDS = -5
VELOX_STATUS_BAD_INDEX = 1
VELOX_STATUS_TIMEOUT = 2
VELOX_STATUS_NO_SPACE = 4
VELOX_TEST_SKIP_MMA = 1
VELOX_TEST_FORCE_PAIR = 2
VELOX_BF16 = 0
VELOX_F32 = 1
CAM_FLOATS = 18
ROPE_STYLES = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "bands": 3}

_c_int, _c_size, _vp, _c_float = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
_c_i64, _c_double = ctypes.c_int64, ctypes.c_double


class _Rope(ctypes.Structure):
    """velox_rope_t"""
    _fields_ = [("freqs", _vp), ("rot", _c_int), ("style", _c_int), ("axes", _c_int),
                ("sections", _c_int * 3), ("mscale", _c_float), ("inverse", _c_int)]


# the same as bytes, which are packed in a third of the time that the structure takes
_pack_rope = struct.Struct("P6ifi").pack
assert struct.calcsize("P6ifi") == ctypes.sizeof(_Rope)


# name -> (restype, argtypes); mirrors include/velox.h
SIGNATURES = {
    "velox_version": (_c_int, []),
    "velox_strerror": (ctypes.c_char_p, [_c_int]),
    "velox_slices_build": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp]),
    "velox_block_overlap": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                     _vp, _vp]),
    "velox_route_topk_workspace_size": (_c_size, [_c_int] * 6),
    "velox_route_topk": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                  _vp, _c_float, _c_int, _vp, _vp, _c_size, _vp, _vp]),
    "velox_sparse_attn_fwd": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                       _c_int, _c_int, _c_float, _vp, _vp, _vp, _vp]),
    "velox_sparse_attn_fwd_test": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                            _c_int, _c_int, _c_int, _c_float, _vp, _vp, _vp,
                                            ctypes.c_double, _c_int, _vp]),
    "velox_depth_multiwarp_workspace_size": (_c_size, [_c_int, _c_int]),
    "velox_depth_multiwarp": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _c_float, _vp, _vp,
                                       _c_size, _vp]),
    "velox_cast_bf16": (_c_int, [_vp, _vp, _c_size, _vp]),
    "velox_depth_multiwarp_noalloc": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _c_float,
                                               _vp, _vp]),
    "velox_fp64_fma_bench": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp]),
    "velox_kbar_cache_bytes": (_c_size, [_c_int] * 6),
    "velox_kbar_append": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                   _vp, _c_int, _vp]),
    "velox_route_topk_cached": (_c_int, [_vp, _c_int, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                         _c_int, _c_int, _vp, _c_float, _c_int, _vp, _vp, _c_size,
                                         _vp, _vp]),
    "velox_rope_freqs": (_c_int, [_c_int, _c_double, _c_int, _c_double, _c_int, _c_double, _c_double,
                                  _vp, _vp]),
    "velox_rope": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _c_i64, _c_i64,
                            _vp, _vp, _vp, _vp]),
    "velox_paged_plan": (_c_int, [_vp] * 5 + [_c_int] * 5 + [_vp] * 8),
    "velox_paged_release": (_c_int, [_vp] * 5 + [_c_int] * 4 + [_vp] * 4),
    "velox_paged_append": (_c_int, [_vp] * 3 + [_c_int] * 5 + [_vp] * 5 + [_c_i64] + [_vp] * 4
                           + [_c_int, _c_int, _vp, _vp]),
    "velox_paged_attn_workspace_size": (_c_size, [_c_int] * 4),
    "velox_paged_attn": (_c_int, [_vp] * 5 + [_c_int] * 7 + [_c_float, _vp, _vp, _vp, _c_size, _vp,
                                                             _vp]),
    "velox_paged_attn_step": (_c_int, [_vp] * 6 + [_c_int] * 8 + [_c_float, _vp, _vp, _vp, _c_size,
                                                                  _vp, _vp]),
    "velox_paged_attn_test": (_c_int, [_vp] * 5 + [_c_int] * 7 + [_c_float, _vp, _vp, _vp, _c_size,
                                                                  _vp, _c_double, _c_int, _c_int, _vp]),
}


class VeloxError(RuntimeError):
    def __init__(self, what: str, code: int):
        super().__init__(f"{what} failed: {strerror(code)} ({code})")
        self.code = code


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(
            f"libvelox.so not found at {path}; build it with `python -m geometry_routed_block_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = load_library()


def strerror(code: int) -> str:
    return lib.velox_strerror(code).decode()


def _check(code: int, what: str) -> None:
    if code != VELOX_OK:
        raise VeloxError(what, code)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libvelox takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libvelox takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream: torch.cuda.Stream | None = None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _expect(t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


# ---------------------------------------------------------------- geometry

def slices_build(depth: torch.Tensor, poses: torch.Tensor, intr: torch.Tensor,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """depth [P,Hp,Wp] f32, poses [P,12] f32, intr [P,4] f32 -> slices [P,18] f32."""
    P, Hp, Wp = depth.shape
    for t, n in ((depth, "depth"), (poses, "poses"), (intr, "intr")):
        _expect(t, torch.float32, n)
    if out is None:
        out = torch.empty((P, CAM_FLOATS), dtype=torch.float32, device=depth.device)
    _check(lib.velox_slices_build(_ptr(depth), _ptr(poses), _ptr(intr), P, Hp, Wp, _ptr(out),
                                  _stream(stream)), "velox_slices_build")
    return out


def block_overlap(cur_depth: torch.Tensor, cur_cam: torch.Tensor, slices: torch.Tensor, F: int,
                  T: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """cur_depth [B,Hp,Wp] f32, cur_cam [B,18], slices [B,P,18] -> counts [B,m,P] int32."""
    B, Hp, Wp = cur_depth.shape
    P = slices.shape[1]
    m = F * Hp * Wp // T
    for t, n in ((cur_depth, "cur_depth"), (cur_cam, "cur_cam"), (slices, "slices")):
        _expect(t, torch.float32, n)
    if out is None:
        out = torch.empty((B, m, P), dtype=torch.int32, device=cur_depth.device)
    _check(lib.velox_block_overlap(_ptr(cur_depth), _ptr(cur_cam), _ptr(slices), B, P, F, Hp, Wp, T,
                                   _ptr(out), _stream(stream)), "velox_block_overlap")
    return out


def depth_multiwarp_workspace(Hp: int, Wp: int, device="cuda") -> torch.Tensor:
    n = lib.velox_depth_multiwarp_workspace_size(Hp, Wp)
    return torch.empty(n, dtype=torch.uint8, device=device)


def depth_multiwarp(past_depth: torch.Tensor, past_cams: torch.Tensor, cur_cam: torch.Tensor,
                    rel_tol: float = 0.01, ws: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """past_depth [P,Hp,Wp] f32, past_cams [P,18], cur_cam [18] -> current depth [Hp,Wp] f32."""
    P, Hp, Wp = past_depth.shape
    if ws is None:
        ws = depth_multiwarp_workspace(Hp, Wp, past_depth.device)
    if out is None:
        out = torch.empty((Hp, Wp), dtype=torch.float32, device=past_depth.device)
    _check(lib.velox_depth_multiwarp(_ptr(past_depth), _ptr(past_cams), _ptr(cur_cam), P, Hp, Wp,
                                     float(rel_tol), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "velox_depth_multiwarp")
    return out


# ---------------------------------------------------------------- routing

def route_workspace(B: int, H: int, Nq: int, Nk: int, d: int, T: int, device="cuda") -> torch.Tensor:
    n = lib.velox_route_topk_workspace_size(B, H, Nq, Nk, d, T)
    if n == 0:
        raise VeloxError("velox_route_topk_workspace_size", VELOX_EINVAL)
    return torch.empty(n, dtype=torch.uint8, device=device)


def route_topk(q: torch.Tensor, k: torch.Tensor, counts: torch.Tensor | None, alpha: float,
               topk: int, T: int, ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
               counts_ready: torch.cuda.Event | None = None, stream=None) -> torch.Tensor:
    """q [B,H,Nq,d], k [B,H,Nk,d] (bf16 or f32), counts [B,m,P] int32 or None ->
    idx [B,H,m,topk] int32 (ascending key-block indices). With `counts_ready`,
    only the selection kernel waits for that event (the counts' producer may
    still be running on another stream while the keys are pooled)."""
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if q.dtype != k.dtype:
        raise TypeError("q and k must share a dtype")
    dtype = {torch.bfloat16: VELOX_BF16, torch.float32: VELOX_F32}.get(q.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if counts is not None:
        _expect(counts, torch.int32, "counts")
    if ws is None:
        ws = route_workspace(B, H, Nq, Nk, d, T, q.device)
    if out is None:
        out = torch.empty((B, H, Nq // T, topk), dtype=torch.int32, device=q.device)
    ev = ctypes.c_void_p(counts_ready.cuda_event) if counts_ready is not None else None
    _check(lib.velox_route_topk(_ptr(q), _ptr(k), dtype, B, H, Nq, Nk, d, T, _ptr(counts),
                                float(alpha), int(topk), _ptr(out), _ptr(ws), ws.numel(), ev,
                                _stream(stream)), "velox_route_topk")
    return out


# ---------------------------------------------------------------- pooled-key cache

def kbar_cache(B: int, H: int, max_past_chunks: int, Nq: int, d: int, T: int,
               device="cuda") -> torch.Tensor:
    """An empty pooled-key cache [B, H, max_past_chunks * Nq/T, d] float32."""
    if lib.velox_kbar_cache_bytes(B, H, max_past_chunks, Nq, d, T) == 0:
        raise VeloxError("velox_kbar_cache_bytes", VELOX_EINVAL)
    return torch.empty((B, H, max_past_chunks * (Nq // T), d), dtype=torch.float32, device=device)


def kbar_append(k: torch.Tensor, Nq: int, T: int, chunk: int, kbar: torch.Tensor,
                stream=None) -> torch.Tensor:
    """Pools chunk `chunk` of the KV cache k [B,H,Nk,d] into kbar."""
    B, H, Nk, d = k.shape
    dtype = {torch.bfloat16: VELOX_BF16, torch.float32: VELOX_F32}.get(k.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {k.dtype}")
    _expect(kbar, torch.float32, "kbar")
    max_chunks = kbar.shape[2] // (Nq // T)
    _check(lib.velox_kbar_append(_ptr(k), dtype, B, H, Nk, Nq, d, T, int(chunk), _ptr(kbar),
                                 max_chunks, _stream(stream)), "velox_kbar_append")
    return kbar


def route_topk_cached(q: torch.Tensor, kbar: torch.Tensor, P: int, counts: torch.Tensor | None,
                      alpha: float, topk: int, T: int, ws: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, counts_ready: torch.cuda.Event | None = None,
                      stream=None) -> torch.Tensor:
    """route_topk over P past chunks whose pooled keys are in kbar."""
    B, H, Nq, d = q.shape
    dtype = {torch.bfloat16: VELOX_BF16, torch.float32: VELOX_F32}.get(q.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {q.dtype}")
    _expect(kbar, torch.float32, "kbar")
    if counts is not None:
        _expect(counts, torch.int32, "counts")
    max_chunks = kbar.shape[2] // (Nq // T)
    if ws is None:
        ws = route_workspace(B, H, Nq, (P + 1) * Nq, d, T, q.device)
    if out is None:
        out = torch.empty((B, H, Nq // T, topk), dtype=torch.int32, device=q.device)
    ev = ctypes.c_void_p(counts_ready.cuda_event) if counts_ready is not None else None
    _check(lib.velox_route_topk_cached(_ptr(q), dtype, _ptr(kbar), max_chunks, B, H, Nq, int(P), d,
                                       T, _ptr(counts), float(alpha), int(topk), _ptr(out),
                                       _ptr(ws), ws.numel(), ev, _stream(stream)),
           "velox_route_topk_cached")
    return out


# ---------------------------------------------------------------- attention

def sparse_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, idx: torch.Tensor | None,
                    T: int, scale: float | None = None, want_lse: bool = True,
                    status: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, stream=None):
    """q [B,H,Nq,d], k/v [B,H,Nk,d] bf16, idx [B,H,m,topk] int32 or None (dense)
    -> (O [B,H,Nq,d] bf16, lse [B,H,Nq] f32 or None)."""
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _expect(t, torch.bfloat16, n)
    topk = 0
    if idx is not None:
        _expect(idx, torch.int32, "idx")
        topk = idx.shape[-1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if not want_lse:
        lse = None
    if status is not None:
        _expect(status, torch.int32, "status")
    _check(lib.velox_sparse_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(idx), topk, B, H, Nq, Nk, d,
                                     T, float(scale), _ptr(out), _ptr(lse), _ptr(status),
                                     _stream(stream)), "velox_sparse_attn_fwd")
    return out, lse


def sparse_attn_fwd_test(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         idx: torch.Tensor | None, T: int, status: torch.Tensor,
                         wait_limit_s: float, flags: int, out: torch.Tensor | None = None,
                         lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """sparse_attn_fwd through the test entry point (bounded-wait limit and
    test-hook flags); returns O (unwritten when the waits ran out). An `lse`
    tensor [B,H,Nq] f32, when given, receives the log-sum-exp."""
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _expect(t, torch.bfloat16, n)
    _expect(status, torch.int32, "status")
    topk = 0
    if idx is not None:
        _expect(idx, torch.int32, "idx")
        topk = idx.shape[-1]
    if out is None:
        out = torch.empty_like(q)
    _check(lib.velox_sparse_attn_fwd_test(_ptr(q), _ptr(k), _ptr(v), _ptr(idx), topk, B, H, Nq, Nk,
                                          d, T, float(1.0 / math.sqrt(d)), _ptr(out), _ptr(lse),
                                          _ptr(status), float(wait_limit_s), int(flags),
                                          _stream(stream)), "velox_sparse_attn_fwd_test")
    return out


def fp64_fma_bench(out: torch.Tensor, blocks: int, threads: int, iters: int, stream=None) -> int:
    """Launches the float64 FMA throughput kernel; returns its FLOP count."""
    _expect(out, torch.float64, "out")
    _check(lib.velox_fp64_fma_bench(_ptr(out), int(blocks), int(threads), int(iters),
                                    _stream(stream)), "velox_fp64_fma_bench")
    return 16 * int(blocks) * int(threads) * int(iters)


def cast_bf16(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """float32 -> bf16 (round to nearest even) on the device."""
    _expect(x, torch.float32, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _check(lib.velox_cast_bf16(_ptr(x), _ptr(out), x.numel(), _stream(stream)), "velox_cast_bf16")
    return out


def depth_multiwarp_noalloc(past_depth: torch.Tensor, past_cams: torch.Tensor,
                            cur_cam: torch.Tensor, rel_tol: float = 0.01,
                            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """depth_multiwarp with the library's fixed scratch instead of a caller
    workspace (grids up to 65536 pixels; concurrent calls race)."""
    P, Hp, Wp = past_depth.shape
    if out is None:
        out = torch.empty((Hp, Wp), dtype=torch.float32, device=past_depth.device)
    _check(lib.velox_depth_multiwarp_noalloc(_ptr(past_depth), _ptr(past_cams), _ptr(cur_cam), P,
                                             Hp, Wp, float(rel_tol), _ptr(out), _stream(stream)),
           "velox_depth_multiwarp_noalloc")
    return out


# ---------------------------------------------------------------- tokens: rotary positions, paged cache

# These calls are short, some only a few microseconds on the GPU, so what the
# binding does per call counts: an argument is looked at once, small outputs
# share one allocation, and the raw stream handle is taken without building a
# Stream object (1.5 to 3 us each on the host of a B200).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
# pieces of an int32 buffer; no gradients run through them that would need views
_pieces = torch.unsafe_split_with_sizes
_I32, _F32, _BF16, _F64 = torch.int32, torch.float32, torch.bfloat16, torch.float64


def _elsewhere(x: torch.Tensor, stream):
    """None where a call on x can run as things stand; else the context to run it
    in: x's device, and `stream` if one is given. Outputs and scratch are then
    allocated there too."""
    index = x.get_device()
    if index < 0:
        raise ValueError("libvelox takes CUDA tensors")
    if stream is not None:
        if stream.device != x.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {x.device}")
        return torch.cuda.stream(stream)
    if index != torch.cuda.current_device():
        return torch.cuda.device(index)
    return None


def _arg(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple | None, index: int,
         dense: bool = True) -> int:
    """The address of an argument after its type, shape, device and layout have been looked at."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on the device of the other tensors")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _status(t: torch.Tensor, index: int) -> int:
    """The address of a status word."""
    at = _arg(t, "status", _I32, None, index)
    if not at:
        raise ValueError("status must have an element")
    return at


@functools.lru_cache(maxsize=256)
def _int64s(values: tuple):
    """A host array the library reads; equal values share one."""
    return (_c_i64 * len(values))(*values)


def _rows(t: torch.Tensor, name: str) -> tuple:
    """The strides of a tensor whose innermost dimension is dense."""
    stride = t.stride()
    if stride[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    return stride[:-1]


def _extent(t: torch.Tensor) -> tuple:
    """First byte and the byte behind the last of a tensor."""
    size = t.element_size()
    last = sum((n - 1) * st for n, st in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * size


def _apart(x: torch.Tensor, y: torch.Tensor) -> bool:
    """Whether two tensors of a call (an input and an output) share no element: their extents do
    not meet, or they are differently placed views of one buffer with the same strides."""
    (a, b), (c, d) = _extent(x), _extent(y)
    if b <= c or d <= a:
        return True
    if x.dtype != y.dtype or x.shape != y.shape or x.stride() != y.stride() or (c - a) % x.element_size():
        return False
    # a shared element is an index difference (di, dj, ...) that makes up for the offset. From
    # the largest stride down, only those count that the smaller ones (`rest`) can make up
    # for: at most two of a dimension that the smaller ones do not reach beyond
    dims = sorted((st, n) for n, st in zip(x.shape, x.stride()) if n > 1 and st > 0)
    rests = [0]
    for st, n in dims:
        rests.append(rests[-1] + (n - 1) * st)
    reach = {(c - a) // x.element_size()}
    for (st, n), rest in zip(reversed(dims), reversed(rests[:-1])):
        reach = {r - i * st for r in reach
                 for i in range(max(-((rest - r) // st), 1 - n), min((r + rest) // st, n - 1) + 1)}
        if len(reach) > 4096:
            return False
    return 0 not in reach


def _in_dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype is _BF16:
        return VELOX_BF16
    if t.dtype is _F32:
        return VELOX_F32
    raise TypeError(f"{name}: unsupported dtype {t.dtype}")


@functools.lru_cache(maxsize=256)
def _sections(style: str, sections: tuple):
    if style not in ROPE_STYLES:
        raise ValueError(f"style must be one of {sorted(ROPE_STYLES)}")
    if not 1 <= len(sections) <= 3 or not all(0 <= n <= 2048 for n in sections):
        raise ValueError("one to three position axes, of 0 to 2048 pairs each")
    return (ROPE_STYLES[style], len(sections), *map(int, sections), *[0] * (3 - len(sections)))


def _rope_spec(freqs: torch.Tensor, style: str, sections, mscale: float, inverse: bool,
               index: int) -> tuple:
    """A velox_rope_t and its number of axes."""
    if freqs.dim() != 1:
        raise ValueError("freqs is one-dimensional: a frequency per rotated pair")
    n = freqs.shape[0]
    layout = _sections(style, (n,) if sections is None else tuple(sections))
    return _pack_rope(_arg(freqs, "freqs", _F64, None, index), 2 * n, *layout, mscale,
                      1 if inverse else 0), layout[1]


def _pos_shape(pos: torch.Tensor, axes: int, N: int, B: int | None) -> tuple:
    """The shape that positions must have: [N] (one axis), [axes,N] or, with batches, [axes,B,N]."""
    if pos.dim() == 1 and axes == 1:
        return (N,)
    return (axes, B, N) if pos.dim() == 3 and B is not None else (axes, N)


def rope_freqs(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
               orig_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """Frequencies of `rot` rotated elements: ([rot/2] float64 radians per position,
    mscale). scaling "linear", "base" and "bands" stretch the positions `factor` times
    (include/velox.h states the formulas). For several axes, concatenate one
    call's frequencies per axis."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    out = (_c_double * max(1, rot // 2))()
    m = _c_float(1.0)
    _check(lib.velox_rope_freqs(int(rot), float(base), ROPE_SCALINGS[scaling], float(factor),
                                int(orig_len), float(beta_fast), float(beta_slow),
                                ctypes.addressof(out), ctypes.addressof(m)), "velox_rope_freqs")
    return torch.tensor(list(out), dtype=torch.float64).to(device), m.value


def rope(x: torch.Tensor, pos: torch.Tensor, freqs: torch.Tensor, style: str = "half",
         sections=None, mscale: float = 1.0, inverse: bool = False,
         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotary positions of x [B,H,N,d] (bf16 or f32; any strides, the last dimension
    dense) -> the same shape and type. pos int32 [N] (one axis), [axes,N] or
    [axes,B,N]; freqs [rot/2] float64; sections: pairs of each axis (default: one
    axis). inverse turns back (which is also the gradient of the forward call); out
    may be x itself, or share nothing with it; its strides nest."""
    B, H, N, d = shape = x.shape
    index = x.get_device()
    dt = _in_dtype(x, "x")
    spec, axes = _rope_spec(freqs, style, sections, mscale, inverse, index)
    p = _arg(pos, "pos", _I32, _pos_shape(pos, axes, N, B), index)
    xs = _rows(x, "x")
    there = _elsewhere(x, stream)
    if there is not None:
        with there:
            return rope(x, pos, freqs, style, sections, mscale, inverse, out)
    if out is None:
        out = torch.empty_like(x) if x.is_contiguous() else x.new_empty(shape)
        ys = (H * N * d, N * d, d)
    else:
        _arg(out, "out", x.dtype, shape, index, dense=False)
        ys = _rows(out, "out")
        if (out.data_ptr() != x.data_ptr() or any(
                n > 1 and i != j for n, i, j in zip(shape, xs, ys))) and not _apart(x, out):
            raise ValueError("out may be x itself, but not share some of its elements")
        reach = d  # elements up to the last of the smaller dimensions
        for st, n in sorted((st, n) for st, n in zip(ys, shape) if n > 1 and st > 0):
            if st < reach:
                raise ValueError("out lies on itself: some of its rows share elements")
            reach += (n - 1) * st
    if 0 in shape:
        return out  # nothing to turn
    batched = pos.dim() == 3
    _check(lib.velox_rope(x.data_ptr(), dt, B, H, N, d, _int64s(xs), p, B * N if batched else N,
                          N if batched else 0, spec, out.data_ptr(), _int64s(ys),
                          _raw_stream(index)), "velox_rope")
    return out


class PagedPlan(NamedTuple):
    """What a step's requests and tokens look like: cu [R+1] first token of each
    request, slots / pos / req [n_cap] of each token (-1: padding), lens [R] and
    free_count [1] after the step."""
    cu: torch.Tensor
    slots: torch.Tensor
    pos: torch.Tensor
    req: torch.Tensor
    lens: torch.Tensor
    free_count: torch.Tensor


def _pages_state(lens, table, free_list, free_count, index: int):
    """Checks the state of a paged cache; (R, max_pages, num_pages, its addresses)."""
    if lens.dim() != 1 or table.dim() != 2 or free_list.dim() != 1:
        raise ValueError("lens [R], table [R,max_pages], free_list [num_pages]")
    R = lens.shape[0]
    tr, width = table.shape
    if tr != R:
        raise ValueError(f"table has {tr} rows for {R} requests")
    return (R, width, free_list.shape[0], _arg(lens, "lens", _I32, None, index),
            _arg(table, "table", _I32, None, index), _arg(free_list, "free_list", _I32, None, index),
            _arg(free_count, "free_count", _I32, (1,), index))


def _separate(inputs: tuple, outputs: tuple) -> None:
    """Refuses int32 outputs that share elements with an input or another output, of which
    other threads may not have read or written theirs yet. Each is (name, address, elements)."""
    spans = sorted([(at, n, name, False) for name, at, n in inputs if n] +
                   [(at, n, name, True) for name, at, n in outputs if n and at])
    end_in = end_out = 0
    for at, n, name, written in spans:
        if at < end_out or (written and at < end_in):
            raise ValueError(f"{name} must not share elements of the call's other tensors")
        if written:
            end_out = at + 4 * n
        else:
            end_in = max(end_in, at + 4 * n)


def paged_plan(add: torch.Tensor, lens: torch.Tensor, table: torch.Tensor, free_list: torch.Tensor,
               free_count: torch.Tensor, page: int, n_cap: int, out: PagedPlan | None = None,
               status: torch.Tensor | None = None, stream=None) -> PagedPlan:
    """Pages for add [R] new tokens of requests with lens [R] cached ones: enters
    them in table [R,max_pages] and returns the step's PagedPlan with room for n_cap
    tokens (all int32). `out` gives the outputs' tensors; its lens and
    free_count may be the inputs (lens also add), so that a captured step carries its
    state on; else the outputs share nothing with one another or the inputs. Tensors
    allocated here are views of one buffer."""
    index = lens.get_device()
    R, width, num_pages, pl, pt, pf, pc = _pages_state(lens, table, free_list, free_count, index)
    pa = _arg(add, "add", _I32, (R,), index)
    ps = None if status is None else _status(status, index)
    page, n_cap = int(page), int(n_cap)
    if not 0 <= n_cap < 2 ** 31:
        raise ValueError("n_cap must be in [0, 2^31)")
    there = _elsewhere(lens, stream)
    if there is not None:
        with there:
            return paged_plan(add, lens, table, free_list, free_count, page, n_cap, out, status)
    if out is None:
        buf = lens.new_empty(2 * R + 2 + 3 * n_cap)
        o = buf.data_ptr()
        # slots, pos and req first: their rows then start where the buffer's alignment allows
        os_, op, oq = o, o + 4 * n_cap, o + 8 * n_cap
        oc = o + 12 * n_cap
        ol = oc + 4 * (R + 1)
        of = ol + 4 * R
        slots, pos, req, cu, lens_out, count = _pieces(buf, (n_cap, n_cap, n_cap, R + 1, R, 1))
        out = PagedPlan(cu, slots, pos, req, lens_out, count)
    else:
        oc, os_, op, oq, ol, of = [
            _arg(t, name, _I32, (size,), index) for t, name, size in
            zip(out, PagedPlan._fields, (R + 1, n_cap, n_cap, n_cap, R, 1))]
        ins, outs = [("free_list", pf, num_pages)], [
            ("cu", oc, R + 1), ("slots", os_, n_cap), ("pos", op, n_cap), ("req", oq, n_cap),
            ("lens", ol, R), ("free_count", of, 1), ("table", pt, R * width), ("status", ps, 1)]
        ins += [(name, at, R) for name, at in (("lens", pl), ("add", pa)) if at != ol]
        if of != pc:
            ins.append(("free_count", pc, 1))
        _separate(ins, outs)
    _check(lib.velox_paged_plan(pa, pl, pt, pf, pc, R, width, page, num_pages, n_cap, ol, of, oc,
                                os_, op, oq, ps, _raw_stream(index)), "velox_paged_plan")
    return out


def paged_release(done: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                  free_list: torch.Tensor, free_count: torch.Tensor, page: int,
                  lens_out: torch.Tensor | None = None, free_count_out: torch.Tensor | None = None,
                  status: torch.Tensor | None = None, stream=None):
    """The pages of the requests with done [R] != 0 go back on free_list (in
    place); returns (lens, free_count) afterwards. The outputs may be the inputs (lens_out
    also done, which may be lens itself), else they share nothing with them; those
    allocated here are views of one buffer."""
    index = lens.get_device()
    R, width, num_pages, pl, pt, pf, pc = _pages_state(lens, table, free_list, free_count, index)
    pd = _arg(done, "done", _I32, (R,), index)
    ps = None if status is None else _status(status, index)
    there = _elsewhere(lens, stream)
    if there is not None:
        with there:
            return paged_release(done, lens, table, free_list, free_count, page, lens_out,
                                 free_count_out, status)
    given = lens_out is not None or free_count_out is not None
    if lens_out is None or free_count_out is None:
        a, b = _pieces(lens.new_empty(R + 1), (R, 1))
        lens_out = a if lens_out is None else lens_out
        free_count_out = b if free_count_out is None else free_count_out
    ol = _arg(lens_out, "lens_out", _I32, (R,), index)
    of = _arg(free_count_out, "free_count_out", _I32, (1,), index)
    if given:
        ins = [(name, at, R) for name, at in (("lens", pl), ("done", pd)) if at != ol]
        ins.append(("table", pt, R * width))
        if of != pc:
            ins.append(("free_count", pc, 1))
        _separate(ins, [("lens_out", ol, R), ("free_count_out", of, 1), ("free_list", pf, num_pages),
                        ("status", ps, 1)])
    _check(lib.velox_paged_release(pd, pl, pt, pf, pc, R, width, int(page), num_pages, ol, of, ps,
                                   _raw_stream(index)), "velox_paged_release")
    return lens_out, free_count_out


@functools.lru_cache(maxsize=256)
def _strides(*strides):
    """The host arrays of several tensors' strides (None for None)."""
    return [None if s is None else _int64s(s) for s in strides]


def paged_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_pages: torch.Tensor,
                 v_pages: torch.Tensor, q: torch.Tensor | None = None,
                 pos: torch.Tensor | None = None, freqs: torch.Tensor | None = None,
                 style: str = "half", sections=None, mscale: float = 1.0,
                 out: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """Writes k, v [N,Hkv,d] (bf16 or f32; any strides, the last dimension dense)
    to their slots [N] int32 (negative: padding) of k_pages / v_pages
    [num_pages,Hkv,page,d] bf16, in place; no other tensor lies in these, nor one of them
    in the other. With freqs (see rope) k and q [N,H,d] are rotated to pos [axes,N] int32
    ([N] for one axis) on the way. Returns q as bf16 [N,H,d], or None without q; out may
    be q itself (bf16 and contiguous)."""
    N, Hkv, d = shape = k.shape
    index = k.get_device()
    dt = _in_dtype(k, "k")
    num_pages, hp, page, dp = pages = k_pages.shape
    if hp != Hkv or dp != d:
        raise ValueError(f"k has {Hkv} heads of {d}, the pages {hp} of {dp}")
    kp = _arg(k_pages, "k_pages", _BF16, None, index)
    vp = _arg(v_pages, "v_pages", _BF16, pages, index)
    pv = _arg(v, "v", k.dtype, shape, index, dense=False)
    psl = _arg(slots, "slots", _I32, (N,), index)
    ps = None if status is None else _status(status, index)
    spec = pp = None
    if freqs is not None:
        if pos is None:
            raise ValueError("freqs without pos")
        spec, axes = _rope_spec(freqs, style, sections, mscale, False, index)
        pp = _arg(pos, "pos", _I32, _pos_shape(pos, axes, N, None), index)
    H, pq, po, qs = 0, None, None, None
    if q is not None:
        H = q.shape[1]
        pq = _arg(q, "q", k.dtype, (N, H, d), index, dense=False)
        qs = _rows(q, "q")
    elif out is not None:
        raise ValueError("out without q")
    ks, vs = _rows(k, "k"), _rows(v, "v")
    there = _elsewhere(k, stream)
    if there is not None:
        with there:
            return paged_append(k, v, slots, k_pages, v_pages, q, pos, freqs, style, sections,
                                mscale, out, status)
    pk, size = k.data_ptr(), 2 if dt == VELOX_BF16 else 4
    if out is not None:
        po = _arg(out, "out", _BF16, (N, H, d), index)
        same = po == pq and dt == VELOX_BF16 and q.is_contiguous()
        if not (same or _apart(q, out)) or not _apart(k, out) or not _apart(v, out):
            raise ValueError("out may be q itself (bf16, contiguous), but not share elements of q, k or v")
    elif q is not None:
        out = q.new_empty((N, H, d)) if dt == VELOX_BF16 else q.new_empty((N, H, d), dtype=_BF16)
        po = out.data_ptr()
    # the pages are written while k, v and q are read: no other tensor reaches into them
    nbytes, m, h = 2 * k_pages.numel(), N - 1, Hkv - 1
    ke, ve = kp + nbytes, vp + nbytes
    ek = pk + (m * ks[0] + h * ks[1] + d) * size
    ev = pv + (m * vs[0] + h * vs[1] + d) * size
    shared = (kp < ve and vp < ke or pk < ke and kp < ek or pk < ve and vp < ek
              or pv < ke and kp < ev or pv < ve and vp < ev)
    if q is not None:
        eq = pq + (m * qs[0] + (H - 1) * qs[1] + d) * size
        eo = po + 2 * N * H * d
        shared = (shared or pq < ke and kp < eq or pq < ve and vp < eq
                  or po < ke and kp < eo or po < ve and vp < eo)
    if shared:
        raise ValueError("k_pages and v_pages must not share elements with each other or with q, k, v, out")
    if N == 0:
        return out  # no tokens
    qs, ks, vs = _strides(qs, ks, vs)
    _check(lib.velox_paged_append(pq, pk, pv, dt, N, H, Hkv, d, qs, ks, vs, psl, pp, N, spec, po, kp, vp,
                                  page, num_pages, ps, _raw_stream(index)),
           "velox_paged_append")
    return out


def paged_attn_workspace(R: int, H: int, Hkv: int, d: int, device="cuda") -> torch.Tensor:
    n = lib.velox_paged_attn_workspace_size(R, H, Hkv, d)
    if n == 0:
        raise VeloxError("velox_paged_attn_workspace_size", VELOX_EINVAL)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _needs_no_workspace(rows: int, longest: int) -> bool:
    """The header's rule for short histories of few rows."""
    n = 8 if rows <= 32 else 4 if rows <= 64 else 2 if rows <= 128 else 1 if rows <= 256 else 0
    return longest <= 512 * n


def paged_attn(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
               lens: torch.Tensor, scale: float | None = None, want_lse: bool = True,
               ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None,
               cu: torch.Tensor | None = None):
    """One new token per request, q [R,H,d] bf16, against its first lens [R] tokens
    in k_pages / v_pages [num_pages,Hkv,page,d] bf16 by table [R,max_pages] int32
    -> (O [R,H,d] bf16, lse [R,H] f32 or None). H is a multiple of Hkv.

    With cu [R+1] int32 of a PagedPlan, q [N,H,d] has the rows of that step's tokens, as
    paged_append returns them: a request with new tokens attends with the last of them,
    one without is idle. O and lse have the same rows; those that no request attends
    with stay as they were in out and lse (0 and -inf in tensors allocated here)."""
    N, H, d = shape = q.shape
    index = q.get_device()
    pq = _arg(q, "q", _BF16, None, index)
    num_pages, Hkv, page, dp = pages = k_pages.shape
    if dp != d:
        raise ValueError(f"q has heads of {d}, the pages of {dp}")
    kp = _arg(k_pages, "k_pages", _BF16, None, index)
    vp = _arg(v_pages, "v_pages", _BF16, pages, index)
    R, width = table.shape
    if cu is None and R != N:
        raise ValueError(f"table must be [{N},max_pages]")
    pt = _arg(table, "table", _I32, None, index)
    pl = _arg(lens, "lens", _I32, (R,), index)
    pc = None if cu is None else _arg(cu, "cu", _I32, (R + 1,), index)
    ps = None if status is None else _status(status, index)
    there = _elsewhere(q, stream)
    if there is not None:
        with there:
            return paged_attn(q, k_pages, v_pages, table, lens, scale, want_lse, ws, out, lse, status,
                              None, cu)
    if R == 0 or N == 0:
        pw, nw = None, 0
    elif ws is not None:
        pw, nw = _arg(ws, "ws", torch.uint8, None, index), ws.numel()
    elif _needs_no_workspace(R * Hkv * ((H // max(Hkv, 1) + 15) // 16), width * page):
        pw, nw = None, 0
    else:
        ws = paged_attn_workspace(R, H, Hkv, d, q.device)
        pw, nw = ws.data_ptr(), ws.numel()
    if out is None:
        out = torch.empty_like(q) if cu is None else torch.zeros_like(q)
        po = out.data_ptr()
    else:
        po = _arg(out, "out", _BF16, shape, index)
        nbytes = 2 * k_pages.numel()
        if not _apart(q, out) or any(po < p + nbytes and po + 2 * N * H * d > p for p in (kp, vp)):
            raise ValueError("out must not share elements of q or the pages: other parts still read them")
    if not want_lse:
        lse = pe = None
    elif lse is None:
        lse = q.new_empty((N, H), dtype=_F32) if cu is None else q.new_full((N, H), -math.inf, dtype=_F32)
        pe = lse.data_ptr()
    else:
        pe = _arg(lse, "lse", _F32, (N, H), index)
        nbytes, rows = 2 * k_pages.numel(), 2 * N * H * d
        if any(pe < p + n and pe + 4 * N * H > p
               for p, n in ((pq, rows), (po, rows), (kp, nbytes), (vp, nbytes))):
            raise ValueError("lse must not share elements of q, out or the pages")
    if R == 0 or N == 0:
        return out, lse  # no requests, or no tokens
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if cu is None:
        _check(lib.velox_paged_attn(pq, kp, vp, pt, pl, R, H, Hkv, d, page, num_pages, width, scale,
                                    po, pe, pw, nw, ps, _raw_stream(index)), "velox_paged_attn")
    else:
        _check(lib.velox_paged_attn_step(pq, kp, vp, pt, pl, pc, R, N, H, Hkv, d, page, num_pages, width,
                                         scale, po, pe, pw, nw, ps, _raw_stream(index)),
               "velox_paged_attn_step")
    return out, lse


def paged_attn_test(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                    table: torch.Tensor, lens: torch.Tensor, status: torch.Tensor,
                    wait_limit_s: float, skip_warps: int, ws: torch.Tensor | None = None,
                    most_cluster: int = 16):
    """paged_attn through the test entry point (bounded-wait limit, the warps that fetch
    nothing, the largest cluster); returns (O, lse), undefined where the waits ran out."""
    R, H, d = q.shape
    num_pages, Hkv, page, _ = k_pages.shape
    _expect(q, _BF16, "q")
    for t, n in ((table, "table"), (lens, "lens"), (status, "status")):
        _expect(t, _I32, n)
    out, lse = torch.empty_like(q), q.new_empty((R, H), dtype=_F32)
    _check(lib.velox_paged_attn_test(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(table), _ptr(lens), R, H, Hkv, d, page, num_pages,
        table.shape[1], 1.0 / math.sqrt(d), _ptr(out), _ptr(lse), _ptr(ws),
        0 if ws is None else ws.numel(), _ptr(status), float(wait_limit_s), int(skip_warps),
        int(most_cluster), _stream()), "velox_paged_attn_test")
    return out, lse
