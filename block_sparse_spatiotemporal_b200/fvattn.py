"""Thin Python binding of libfvattn.so (argument marshalling only).

Every step of the path runs in the library's CUDA kernels; this module only
builds the C structs, passes torch device pointers and the current CUDA
stream, and turns status codes into exceptions.  There is no fallback: if
the library is missing or the device is not an sm_100 GPU, calls raise.

Names follow the C ABI in include/fvattn.h.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

__all__ = [
    "FvattnError", "Shape", "Rope", "Blocks", "MaskCache", "lib", "library_path",
    "F32", "BF16", "RASTER_CUBE", "HILBERT", "NATURAL", "TILED",
    "make_shape", "make_rope", "num_tiles", "workspace_size", "workspace", "workspace_size_subblock",
    "pool_select_subblock",
    "tile_reorder", "pool_select", "build_worklist", "block_sparse_fwd", "forward",
    "device_status", "selftest_wait_timeout", "new_blocks", "new_cache", "profile_enable", "profile_read",
    "STAGES", "pool_select_noalloc", "noalloc_status", "profile_cta_times", "workspace_size_qkv", "qkv_rope", "workspace_size_bwd", "block_sparse_bwd",
    "augment_lists", "block_sparse_fwd_worklist", "timestep_params",
    "Norm", "Window", "View", "make_norm", "norm_workspace", "layer_norm_fwd", "layer_norm_bwd",
    "make_window", "window_workspace", "window_fwd", "window_bwd",
]

F32, BF16 = 0, 1
RASTER_CUBE, HILBERT = 0, 1
NATURAL, TILED = 0, 1

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    return os.path.join(_HERE, "libfvattn.so")


class FvattnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib().fvattn_status_string(status).decode()
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("W", ctypes.c_int32)]


class Tile(ctypes.Structure):
    _fields_ = [("t", ctypes.c_int32), ("h", ctypes.c_int32), ("w", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("enabled", ctypes.c_int32), ("dt", ctypes.c_int32), ("dh", ctypes.c_int32),
                ("dw", ctypes.c_int32), ("base", ctypes.c_float)]


class Shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("grid", Dims), ("tile", Tile), ("dtype", ctypes.c_int), ("order", ctypes.c_int),
                ("layout", ctypes.c_int), ("scale", ctypes.c_float)]


class Blocks(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("cap", ctypes.c_int32)]


class MaskCache(ctypes.Structure):
    _fields_ = [("blocks", Blocks), ("shape", Shape), ("top_p", ctypes.c_float),
                ("k_min", ctypes.c_int32), ("valid", ctypes.c_int32)]


class Norm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("gain_one", ctypes.c_int32), ("eps", ctypes.c_float),
                ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64)]


class Window(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("q_len", ctypes.c_int32), ("kv_len", ctypes.c_int32),
                ("unit", ctypes.c_int32), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float)]


class View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("head", ctypes.c_int64),
                ("token", ctypes.c_int64)]


_LIB = None

_SIGS = {
    "fvattn_num_tiles": [ctypes.POINTER(Shape), ctypes.POINTER(ctypes.c_int64)],
    "fvattn_workspace_size": [ctypes.POINTER(Shape), ctypes.POINTER(Rope), ctypes.POINTER(ctypes.c_size_t)],
    "fvattn_tile_reorder": [ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                            ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "fvattn_pool_select": [ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Rope),
                           ctypes.c_float, ctypes.c_int32, ctypes.POINTER(Blocks), ctypes.c_void_p,
                           ctypes.c_size_t, ctypes.c_void_p],
    "fvattn_workspace_size_subblock": [ctypes.POINTER(Shape), ctypes.POINTER(Rope), ctypes.POINTER(ctypes.c_size_t)],
    "fvattn_pool_select_subblock": [ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Rope),
                                    ctypes.c_float, ctypes.c_int32, ctypes.POINTER(Blocks), ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p],
    "fvattn_pool_select_noalloc": [ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Rope),
                                   ctypes.c_float, ctypes.c_int32, ctypes.POINTER(Blocks), ctypes.c_void_p],
    "fvattn_pool_select_noalloc_status": [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32)],
    "fvattn_profile_cta_times": [ctypes.POINTER(Shape), ctypes.POINTER(Rope), ctypes.c_void_p, ctypes.c_void_p,
                                 ctypes.POINTER(ctypes.c_int64), ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
    "fvattn_build_worklist": [ctypes.POINTER(Shape), ctypes.POINTER(Blocks), ctypes.c_void_p, ctypes.c_void_p,
                              ctypes.c_size_t, ctypes.c_void_p],
    "fvattn_block_sparse_fwd": [ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.POINTER(Rope), ctypes.POINTER(Blocks), ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "fvattn_forward": [ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                       ctypes.POINTER(Rope), ctypes.c_float, ctypes.c_int32, ctypes.POINTER(MaskCache),
                       ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                       ctypes.c_void_p],
    "fvattn_augment_lists": [ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Rope),
                             ctypes.POINTER(Blocks), ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                             ctypes.POINTER(Blocks), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                             ctypes.c_void_p],
    "fvattn_block_sparse_fwd_worklist": [ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.POINTER(Rope), ctypes.POINTER(Blocks), ctypes.c_void_p,
                                         ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_size_t, ctypes.c_void_p],
    "fvattn_timestep_params": [ctypes.c_int32, ctypes.c_int32, ctypes.c_float, ctypes.c_float, ctypes.c_int32,
                               ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_float),
                               ctypes.POINTER(ctypes.c_int32)],
    "fvattn_workspace_size_bwd": [ctypes.POINTER(Shape), ctypes.POINTER(ctypes.c_size_t)],
    "fvattn_block_sparse_bwd": [ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Blocks),
                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                ctypes.c_void_p],
    "fvattn_workspace_size_qkv": [ctypes.POINTER(Shape), ctypes.POINTER(Rope), ctypes.POINTER(ctypes.c_size_t)],
    "fvattn_qkv_rope": [ctypes.POINTER(Shape), ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                        ctypes.POINTER(Rope), ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "fvattn_layer_norm_fwd": [ctypes.POINTER(Norm), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p],
    "fvattn_workspace_size_norm": [ctypes.POINTER(Norm), ctypes.POINTER(ctypes.c_size_t)],
    "fvattn_layer_norm_bwd": [ctypes.POINTER(Norm)] + [ctypes.c_void_p] * 9 + [ctypes.c_size_t, ctypes.c_void_p],
    "fvattn_workspace_size_window": [ctypes.POINTER(Window), ctypes.POINTER(ctypes.c_size_t)],
    "fvattn_window_fwd": [ctypes.POINTER(Window), ctypes.POINTER(View), ctypes.POINTER(View), ctypes.POINTER(View),
                          ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(View), ctypes.c_void_p, ctypes.c_void_p,
                          ctypes.c_size_t, ctypes.c_void_p],
    "fvattn_workspace_size_window_bwd": [ctypes.POINTER(Window), ctypes.POINTER(ctypes.c_size_t)],
    "fvattn_window_bwd": [ctypes.POINTER(Window)] + [ctypes.POINTER(View)] * 5 + [ctypes.c_void_p] * 3 +
                         [ctypes.POINTER(View)] * 3 + [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
    "fvattn_get_device_status": [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32)],
    "fvattn_selftest_wait_timeout": [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_void_p],
    "fvattn_profile_enable": [ctypes.c_int],
    "fvattn_profile_read": [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)],
    "fvattn_profile_read_stages": [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64), ctypes.c_int32],
    "fvattn_status_string": [ctypes.c_int],
}

STAGES = ("tables", "reorder", "pool", "select", "schedule", "fine", "prologue", "bwd_prep", "bwd_kv", "bwd_q",
          "norm", "norm_bwd", "window", "window_prep", "window_kv", "window_q")


def lib():
    """Load libfvattn.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m block_sparse_spatiotemporal_b200.build`")
        h = ctypes.CDLL(path)
        for name, args in _SIGS.items():
            fn = getattr(h, name)
            fn.argtypes = args
            fn.restype = ctypes.c_char_p if name == "fvattn_status_string" else ctypes.c_int
        _LIB = h
    return _LIB


def _check(fn: str, status: int):
    if status != 0:
        raise FvattnError(fn, status)


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def make_shape(batch, heads, head_dim, grid, dtype=BF16, order=RASTER_CUBE, layout=NATURAL, scale=0.0) -> Shape:
    T, Hg, W = grid
    return Shape(batch, heads, head_dim, Dims(T, Hg, W), Tile(4, 4, 4), dtype, order, layout, float(scale))


def make_rope(dims=(44, 42, 42), base=10000.0, enabled=True) -> Rope:
    return Rope(1 if enabled else 0, dims[0], dims[1], dims[2], float(base))


def _rope_ptr(rope: Optional[Rope]):
    return ctypes.byref(rope) if rope is not None else None


def num_tiles(shape: Shape) -> int:
    n = ctypes.c_int64()
    _check("fvattn_num_tiles", lib().fvattn_num_tiles(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def workspace_size(shape: Shape, rope: Optional[Rope] = None) -> int:
    n = ctypes.c_size_t()
    _check("fvattn_workspace_size", lib().fvattn_workspace_size(ctypes.byref(shape), _rope_ptr(rope), ctypes.byref(n)))
    return n.value


def workspace(shape: Shape, rope: Optional[Rope] = None, device="cuda", subblock=False) -> torch.Tensor:
    """A device workspace of the size the library asks for (caller-owned);
    ``subblock`` sizes it for pool_select_subblock as well."""
    n = workspace_size_subblock(shape, rope) if subblock else workspace_size(shape, rope)
    return torch.empty(n, dtype=torch.uint8, device=device)


def workspace_size_subblock(shape: Shape, rope: Optional[Rope] = None) -> int:
    n = ctypes.c_size_t()
    _check("fvattn_workspace_size_subblock",
           lib().fvattn_workspace_size_subblock(ctypes.byref(shape), _rope_ptr(rope), ctypes.byref(n)))
    return n.value


def new_blocks(shape: Shape, device="cuda"):
    """Caller-owned block-list buffers: (counts [B,H,nT], idx [B,H,nT,nT], Blocks)."""
    nT = num_tiles(shape)
    counts = torch.empty((shape.batch, shape.heads, nT), dtype=torch.int32, device=device)
    idx = torch.empty((shape.batch, shape.heads, nT, nT), dtype=torch.int32, device=device)
    return counts, idx, Blocks(counts.data_ptr(), idx.data_ptr(), nT)


def new_cache(shape: Shape, device="cuda"):
    """A mask cache with its own block buffers: (cache, counts, idx)."""
    counts, idx, blocks = new_blocks(shape, device)
    cache = MaskCache()
    cache.blocks = blocks
    cache.valid = 0
    return cache, counts, idx


def tile_reorder(shape: Shape, x: torch.Tensor, ws: torch.Tensor, inverse=False, out=None, stream=None):
    """Permute token rows of x [B,H,N,...] between natural and tiled layout."""
    y = torch.empty_like(x) if out is None else out
    row_bytes = x[0, 0, 0].numel() * x.element_size() if x.dim() == 4 else x.element_size()
    _check("fvattn_tile_reorder", lib().fvattn_tile_reorder(ctypes.byref(shape), _ptr(x), _ptr(y), row_bytes,
                                                            1 if inverse else 0, _ptr(ws), ws.numel(),
                                                            _stream(stream)))
    return y


def pool_select(shape: Shape, q, k, ws, top_p: float, k_min: int, rope: Optional[Rope] = None, blocks=None,
                stream=None):
    """Steps 2-5: returns (counts, idx) int32 device tensors."""
    if blocks is None:
        counts, idx, b = new_blocks(shape, q.device)
    else:
        counts, idx, b = blocks
    _check("fvattn_pool_select", lib().fvattn_pool_select(ctypes.byref(shape), _ptr(q), _ptr(k), _rope_ptr(rope),
                                                          float(top_p), int(k_min), ctypes.byref(b), _ptr(ws),
                                                          ws.numel(), _stream(stream)))
    return counts, idx


def pool_select_subblock(shape: Shape, q, k, ws, top_p: float, k_min: int, rope: Optional[Rope] = None,
                         blocks=None, stream=None):
    """Steps 2-5 with hierarchical sub-block scoring (ws from
    ``workspace(..., subblock=True)``): returns (counts, idx)."""
    if blocks is None:
        counts, idx, b = new_blocks(shape, q.device)
    else:
        counts, idx, b = blocks
    _check("fvattn_pool_select_subblock",
           lib().fvattn_pool_select_subblock(ctypes.byref(shape), _ptr(q), _ptr(k), _rope_ptr(rope), float(top_p),
                                             int(k_min), ctypes.byref(b), _ptr(ws), ws.numel(), _stream(stream)))
    return counts, idx


def pool_select_noalloc(shape: Shape, q, k, top_p: float, k_min: int, rope: Optional[Rope] = None, blocks=None,
                        stream=None):
    """Steps 2-5 with the library's static scratch instead of a workspace
    (for callers that cannot allocate); returns (counts, idx)."""
    if blocks is None:
        counts, idx, b = new_blocks(shape, q.device)
    else:
        counts, idx, b = blocks
    _check("fvattn_pool_select_noalloc",
           lib().fvattn_pool_select_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _rope_ptr(rope), float(top_p),
                                            int(k_min), ctypes.byref(b), _stream(stream)))
    return counts, idx


def noalloc_status(stream=None) -> int:
    """Read and clear the device status word of pool_select_noalloc
    (synchronises the stream)."""
    v = ctypes.c_int32(0)
    _check("fvattn_pool_select_noalloc_status", lib().fvattn_pool_select_noalloc_status(_stream(stream),
                                                                                       ctypes.byref(v)))
    return int(v.value)


def _blocks_of(counts, idx):
    return Blocks(counts.data_ptr(), idx.data_ptr(), idx.shape[-1])


def build_worklist(shape: Shape, counts, idx, ws, stream=None):
    P = (num_tiles(shape) + 1) // 2
    wl = torch.empty(shape.batch * shape.heads * P, dtype=torch.int32, device=counts.device)
    b = _blocks_of(counts, idx)
    _check("fvattn_build_worklist", lib().fvattn_build_worklist(ctypes.byref(shape), ctypes.byref(b), _ptr(wl),
                                                                _ptr(ws), ws.numel(), _stream(stream)))
    return wl


def block_sparse_fwd(shape: Shape, q, k, v, counts, idx, ws, rope: Optional[Rope] = None, out=None, lse=None,
                     stream=None):
    """Step 6: returns (out, lse) in shape.layout."""
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    b = _blocks_of(counts, idx)
    _check("fvattn_block_sparse_fwd",
           lib().fvattn_block_sparse_fwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _rope_ptr(rope),
                                         ctypes.byref(b), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                         _stream(stream)))
    return out, lse


def forward(shape: Shape, q, k, v, ws, top_p: float, k_min: int, rope: Optional[Rope] = None,
            cache: Optional[MaskCache] = None, reuse_mask=False, out=None, lse=None, stream=None):
    """Whole path on natural-layout tensors: returns (out, lse)."""
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    _check("fvattn_forward",
           lib().fvattn_forward(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _rope_ptr(rope), float(top_p),
                                int(k_min), ctypes.byref(cache) if cache is not None else None,
                                1 if reuse_mask else 0, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                _stream(stream)))
    return out, lse


def augment_lists(shape: Shape, q, k, ws, counts, idx, num_ctas: int = 0, rope: Optional[Rope] = None, out=None,
                  stream=None, cta_busy_ns=None, fill_percent: int = 100):
    """Slack-aware augmentation of (counts, idx): returns (counts, idx,
    worklist) -- the augmented lists and the work list to run them with.
    cta_busy_ns: None, or one measured busy time (ns) per CTA of a run of the
    same work list on the unaugmented lists (a host sequence of ints)."""
    if out is None:
        oc, oi, ob = new_blocks(shape, q.device)
    else:
        oc, oi = out
        ob = _blocks_of(oc, oi)
    wl = torch.empty(shape.batch * shape.heads * ((num_tiles(shape) + 1) // 2), dtype=torch.int32, device=q.device)
    base = _blocks_of(counts, idx)
    busy = None
    if cta_busy_ns is not None:
        vals = [int(x) for x in cta_busy_ns]
        busy = (ctypes.c_int64 * max(1, len(vals)))(*vals)
    _check("fvattn_augment_lists",
           lib().fvattn_augment_lists(ctypes.byref(shape), _ptr(q), _ptr(k), _rope_ptr(rope), ctypes.byref(base),
                                      int(num_ctas), busy, int(fill_percent), ctypes.byref(ob), _ptr(wl), _ptr(ws),
                                      ws.numel(), _stream(stream)))
    return oc, oi, wl


def block_sparse_fwd_worklist(shape: Shape, q, k, v, counts, idx, worklist, ws, num_ctas: int = 0,
                              rope: Optional[Rope] = None, out=None, lse=None, stream=None):
    """Step 6 with a given work list and persistent grid: returns (out, lse)."""
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    b = _blocks_of(counts, idx)
    _check("fvattn_block_sparse_fwd_worklist",
           lib().fvattn_block_sparse_fwd_worklist(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _rope_ptr(rope),
                                                  ctypes.byref(b), _ptr(worklist), int(num_ctas), _ptr(out),
                                                  _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))
    return out, lse


def timestep_params(step: int, num_steps: int, p_start: float, p_end: float, k_start: int, k_end: int,
                    dense_steps: int = 0):
    """(top_p, k_min) of a diffusion step (host arithmetic in the library)."""
    p = ctypes.c_float()
    km = ctypes.c_int32()
    _check("fvattn_timestep_params",
           lib().fvattn_timestep_params(int(step), int(num_steps), float(p_start), float(p_end), int(k_start),
                                        int(k_end), int(dense_steps), ctypes.byref(p), ctypes.byref(km)))
    return p.value, km.value


def workspace_size_bwd(shape: Shape) -> int:
    n = ctypes.c_size_t()
    _check("fvattn_workspace_size_bwd", lib().fvattn_workspace_size_bwd(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def block_sparse_bwd(shape: Shape, q, k, v, out, dout, lse, counts, idx, ws, grads=None, stream=None):
    """Backward of step 6 (tiled layout, bf16): returns (dq, dk, dv)."""
    if grads is None:
        grads = tuple(torch.empty_like(q) for _ in range(3))
    dq, dk, dv = grads
    b = _blocks_of(counts, idx)
    _check("fvattn_block_sparse_bwd",
           lib().fvattn_block_sparse_bwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout),
                                         _ptr(lse), ctypes.byref(b), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                                         ws.numel(), _stream(stream)))
    return dq, dk, dv


def workspace_size_qkv(shape: Shape, rope: Optional[Rope] = None) -> int:
    n = ctypes.c_size_t()
    _check("fvattn_workspace_size_qkv",
           lib().fvattn_workspace_size_qkv(ctypes.byref(shape), _rope_ptr(rope), ctypes.byref(n)))
    return n.value


def qkv_rope(shape: Shape, x, w, ws, bias=None, rope: Optional[Rope] = None, t_offset: int = 0, out=None,
             stream=None):
    """Prologue: x [B, N, C] bf16, w [3*H*d, C] bf16, bias [3*H*d] float32
    or None -> (q, k, v) [B, H, N, d] bf16 in shape.layout, Q and K rotated
    at frame t + t_offset."""
    B, N, C = x.shape
    if out is None:
        out = tuple(torch.empty((shape.batch, shape.heads, N, shape.head_dim), dtype=torch.bfloat16,
                                device=x.device) for _ in range(3))
    q, k, v = out
    _check("fvattn_qkv_rope",
           lib().fvattn_qkv_rope(ctypes.byref(shape), _ptr(x), int(C), _ptr(w), _ptr(bias), _rope_ptr(rope),
                                 int(t_offset), _ptr(q), _ptr(k), _ptr(v), _ptr(ws), ws.numel(), _stream(stream)))
    return q, k, v


def _enter(tensors, stream: Optional[torch.cuda.Stream]):
    """(stream handle, guards to close or None): makes the tensors' device
    current and picks the stream to launch on, the given one or the device's
    current one, which new outputs then belong to.  Where that is so already,
    it only reads the stream."""
    dev = -2
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if i < 0:
                    raise ValueError("expected a CUDA tensor")
                if dev != -2:
                    raise ValueError("expected every tensor on one device")
                dev = i
    if stream is None and torch._C._cuda_getDevice() == dev:
        return torch._C._cuda_getCurrentRawStream(dev), None
    if stream is not None and stream.device.index != dev:
        raise ValueError("the stream belongs to another device than the tensors")
    guards = contextlib.ExitStack()
    guards.enter_context(torch.cuda.device(dev))
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    guards.enter_context(torch.cuda.stream(s))
    return s.cuda_stream, guards


def _typed(t: Optional[torch.Tensor], dtype, shape, what: str):
    """Pointer of a contiguous tensor of this dtype and shape (None passes)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor of shape {tuple(shape)}")
    return t.data_ptr()


_DTYPES = {F32: torch.float32, BF16: torch.bfloat16}


def make_norm(rows, channels, groups=1, dtype=BF16, eps=1e-6, gain_one=False, x_stride=0, y_stride=0) -> Norm:
    """Layer norm of `rows` rows; strides in elements (0: channels)."""
    return Norm(int(rows), int(channels), int(groups), dtype, 1 if gain_one else 0, float(eps), int(x_stride),
                int(y_stride))


def norm_workspace(norm: Norm, device="cuda") -> torch.Tensor:
    """A device workspace for layer_norm_bwd (caller-owned)."""
    n = ctypes.c_size_t()
    _check("fvattn_workspace_size_norm", lib().fvattn_workspace_size_norm(ctypes.byref(norm), ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device=device)


def _rows(t: torch.Tensor, norm: Norm, stride: int, what: str):
    """Pointer of the rows of t: contiguous [..., channels], or [rows, channels] with norm's row stride,
    16-byte aligned."""
    C, rows = norm.channels, norm.rows
    stride = stride or C
    ok = t.dtype is _DTYPES.get(norm.dtype) and t.dim() >= 1 and t.shape[-1] == C and t.numel() == rows * C
    if ok and t.is_contiguous():
        ok = stride == C or rows <= 1
    elif ok:
        ok = t.dim() == 2 and (t.stride(1) == 1 or C == 1) and (rows == 1 or t.stride(0) == stride)
    if not ok:
        raise ValueError(f"{what}: expected {rows} {_DTYPES.get(norm.dtype)} rows of {C} with row stride {stride}")
    p = t.data_ptr()
    if p & 15 and rows:
        raise ValueError(f"{what}: the rows have to start on a 16-byte boundary")
    return p


def _affine(t: Optional[torch.Tensor], norm: Norm, what: str):
    """Pointer of a weight, bias or gradient of one: float32 [groups, channels],
    or a single group's [channels]."""
    one = norm.groups == 1 and t is not None and t.dim() == 1
    return _typed(t, torch.float32, (norm.channels,) if one else (norm.groups, norm.channels), what)


def _new_rows(like: torch.Tensor, norm: Norm, stride: int):
    """An output like `like` with norm's row stride."""
    if stride in (0, norm.channels) or norm.rows <= 1:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    buf = torch.empty(norm.rows * stride, dtype=like.dtype, device=like.device)
    return buf.as_strided((norm.rows, norm.channels), (stride, 1))


def layer_norm_fwd(norm: Norm, x, weight=None, bias=None, y=None, mean=None, rstd=None, stream=None):
    """Layer norm of the rows of x ([..., channels], starting on 16 bytes) with
    weight and bias [groups, channels] float32 (a single group's may be
    [channels]; or None): returns (y, mean, rstd)."""
    per_row = (norm.rows,)
    s, guards = _enter((x, weight, bias, y, mean, rstd), stream)
    try:
        px = _rows(x, norm, norm.x_stride, "x")
        if y is None:
            y = _new_rows(x, norm, norm.y_stride)
            py = y.data_ptr()
        else:
            py = _rows(y, norm, norm.y_stride, "y")
        if mean is None and rstd is None:
            mean, rstd = torch.empty((2, norm.rows), dtype=torch.float32, device=x.device).unbind(0)
        elif mean is None:
            mean = torch.empty_like(rstd)
        elif rstd is None:
            rstd = torch.empty_like(mean)
        _check("fvattn_layer_norm_fwd",
               lib().fvattn_layer_norm_fwd(ctypes.byref(norm), px, _affine(weight, norm, "weight"),
                                           _affine(bias, norm, "bias"), py,
                                           _typed(mean, torch.float32, per_row, "mean"),
                                           _typed(rstd, torch.float32, per_row, "rstd"), s))
    finally:
        if guards is not None:
            guards.close()
    return y, mean, rstd


def layer_norm_bwd(norm: Norm, x, dy, mean, rstd, ws, weight=None, grads=None, stream=None):
    """Backward of layer_norm_fwd: returns (dx, dweight, dbias), the last two
    shaped like weight (without one: [groups, channels]).  grads: the three
    output tensors, None for a gradient that is not wanted."""
    affine, per_row = (norm.groups, norm.channels) if weight is None else weight.shape, (norm.rows,)
    s, guards = _enter((x, dy, mean, rstd, ws, weight, *(grads or ())), stream)
    try:
        px = _rows(x, norm, norm.x_stride, "x")
        if grads is None:
            grads = (_new_rows(x, norm, norm.x_stride),
                     *torch.empty((2, *affine), dtype=torch.float32, device=x.device).unbind(0))
        dx, dw, db = grads
        _check("fvattn_layer_norm_bwd",
               lib().fvattn_layer_norm_bwd(ctypes.byref(norm), px, _rows(dy, norm, norm.y_stride, "dy"),
                                           _affine(weight, norm, "weight"),
                                           _typed(mean, torch.float32, per_row, "mean"),
                                           _typed(rstd, torch.float32, per_row, "rstd"),
                                           None if dx is None else _rows(dx, norm, norm.x_stride, "dx"),
                                           _affine(dw, norm, "dweight"), _affine(db, norm, "dbias"),
                                           _ptr(ws), ws.numel(), s))
    finally:
        if guards is not None:
            guards.close()
    return dx, dw, db


def make_window(batch, heads, head_dim, q_len, kv_len, window, sinks=0, unit=1, kv_heads=None, dtype=BF16,
                scale=0.0) -> Window:
    """Sliding-window attention: `window` units of `unit` tokens (0: every
    earlier one) and the first `sinks` units."""
    return Window(int(batch), int(heads), int(heads if kv_heads is None else kv_heads), int(head_dim), int(q_len),
                  int(kv_len), int(unit), int(window), int(sinks), dtype, float(scale))


def window_workspace(win: Window, backward=False, device="cuda") -> torch.Tensor:
    """A device workspace for window_fwd, or (backward) one that serves
    window_fwd and window_bwd in turn (caller-owned)."""
    n = ctypes.c_size_t()
    _check("fvattn_workspace_size_window", lib().fvattn_workspace_size_window(ctypes.byref(win), ctypes.byref(n)))
    size = n.value
    if backward:
        _check("fvattn_workspace_size_window_bwd",
               lib().fvattn_workspace_size_window_bwd(ctypes.byref(win), ctypes.byref(n)))
        size = max(size, n.value)
    return torch.empty(size, dtype=torch.uint8, device=device)


def _view(t: torch.Tensor, batch: int, heads: int, tokens: int, d: int, what: str):
    sb, sh, st, sd = t.stride() if t.dim() == 4 else (0, 0, 0, 0)
    if t.dtype != torch.bfloat16 or t.shape != (batch, heads, tokens, d) or (sd != 1 and t.numel()):
        raise ValueError(f"{what}: expected a bfloat16 tensor [{batch}, {heads}, {tokens}, {d}] with contiguous rows")
    return ctypes.byref(View(t.data_ptr(), sb, sh, st))


def _new_heads(like: torch.Tensor, lens):
    """An output shaped and laid out like `like`; rows behind a sequence's
    length are not written by the library, so with lengths they start as 0."""
    if like.is_contiguous() or not like.transpose(1, 2).is_contiguous():
        new = torch.empty_like(like, memory_format=torch.contiguous_format)
    else:                                               # token-major
        new = torch.empty_strided(like.shape, like.stride(), dtype=like.dtype, device=like.device)
    return new if lens is None else new.zero_()


def window_fwd(win: Window, q, k, v, ws, q_lens=None, kv_lens=None, out=None, lse=None, stream=None):
    """Sliding-window attention of q [B, heads, q_len, d] over k, v
    [B, kv_heads, kv_len, d] (any strides with contiguous rows): returns
    (out, lse).  q_lens, kv_lens: int32 device tensors [B] or None."""
    B, H, Hk, D = win.batch, win.heads, win.kv_heads, win.head_dim
    s, guards = _enter((q, k, v, ws, q_lens, kv_lens, out, lse), stream)
    try:
        vq = _view(q, B, H, win.q_len, D, "q")
        if out is None:
            out = _new_heads(q, q_lens)
        if lse is None:
            lse = (torch.empty if q_lens is None else torch.zeros)((B, H, win.q_len), dtype=torch.float32,
                                                                   device=q.device)
        _check("fvattn_window_fwd",
               lib().fvattn_window_fwd(ctypes.byref(win), vq, _view(k, B, Hk, win.kv_len, D, "k"),
                                       _view(v, B, Hk, win.kv_len, D, "v"),
                                       _typed(q_lens, torch.int32, (B,), "q_lens"),
                                       _typed(kv_lens, torch.int32, (B,), "kv_lens"),
                                       _view(out, B, H, win.q_len, D, "out"),
                                       _typed(lse, torch.float32, (B, H, win.q_len), "lse"), _ptr(ws), ws.numel(), s))
    finally:
        if guards is not None:
            guards.close()
    return out, lse


def window_bwd(win: Window, q, k, v, out, dout, lse, ws, q_lens=None, kv_lens=None, grads=None, stream=None):
    """Backward of window_fwd (ws from ``window_workspace(win, backward=True)``):
    returns (dq, dk, dv).  grads: the three output tensors."""
    B, H, Hk, D = win.batch, win.heads, win.kv_heads, win.head_dim
    s, guards = _enter((q, k, v, out, dout, lse, ws, q_lens, kv_lens, *(grads or ())), stream)
    try:
        vq, vk, vv = (_view(q, B, H, win.q_len, D, "q"), _view(k, B, Hk, win.kv_len, D, "k"),
                      _view(v, B, Hk, win.kv_len, D, "v"))
        if grads is None:
            grads = (_new_heads(q, q_lens), _new_heads(k, kv_lens), _new_heads(v, kv_lens))
        dq, dk, dv = grads
        _check("fvattn_window_bwd",
               lib().fvattn_window_bwd(ctypes.byref(win), vq, vk, vv, _view(out, B, H, win.q_len, D, "out"),
                                       _view(dout, B, H, win.q_len, D, "dout"),
                                       _typed(lse, torch.float32, (B, H, win.q_len), "lse"),
                                       _typed(q_lens, torch.int32, (B,), "q_lens"),
                                       _typed(kv_lens, torch.int32, (B,), "kv_lens"),
                                       _view(dq, B, H, win.q_len, D, "dq"), _view(dk, B, Hk, win.kv_len, D, "dk"),
                                       _view(dv, B, Hk, win.kv_len, D, "dv"), _ptr(ws), ws.numel(), s))
    finally:
        if guards is not None:
            guards.close()
    return dq, dk, dv


def device_status(ws, stream=None) -> int:
    """Synchronise, read and clear the workspace status word (0 = no error)."""
    st = ctypes.c_int32()
    _check("fvattn_get_device_status", lib().fvattn_get_device_status(_ptr(ws), _stream(stream), ctypes.byref(st)))
    return st.value


def selftest_wait_timeout(ws, cap_iterations: int, stream=None):
    _check("fvattn_selftest_wait_timeout",
           lib().fvattn_selftest_wait_timeout(_ptr(ws), ws.numel(), int(cap_iterations), _stream(stream)))


def profile_enable(on: bool = True):
    """Record CUDA events around every library kernel (per-stage timing)."""
    _check("fvattn_profile_enable", lib().fvattn_profile_enable(1 if on else 0))


def profile_cta_times(shape: Shape, ws, rope: Optional[Rope] = None, stream=None):
    """(start, end) nanoseconds of every CTA of the last profiled fine-stage
    launch that used `ws`, as an [n, 2] int64 numpy array (synchronises)."""
    import numpy as np
    cap = 1024
    buf = (ctypes.c_int64 * (2 * cap))()
    n = ctypes.c_int32(0)
    _check("fvattn_profile_cta_times", lib().fvattn_profile_cta_times(ctypes.byref(shape), _rope_ptr(rope), _ptr(ws),
                                                                        _stream(stream), buf, cap, ctypes.byref(n)))
    m = min(n.value, cap)
    return np.frombuffer(buf, dtype=np.int64, count=2 * m).reshape(m, 2).copy()


def profile_read():
    """{stage: (ms, launches)} summed since the last read (synchronises)."""
    ms = (ctypes.c_double * len(STAGES))()
    n = (ctypes.c_int64 * len(STAGES))()
    _check("fvattn_profile_read_stages", lib().fvattn_profile_read_stages(ms, n, len(STAGES)))
    return {name: (ms[i], n[i]) for i, name in enumerate(STAGES)}
