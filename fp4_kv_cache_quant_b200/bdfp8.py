"""Thin ctypes binding of the 8-bit paged cache (include/bdfp8.h).

Argument checks and marshalling only: the work runs in libbdfp4.so's CUDA
kernels, on the current stream of the tensors' device.  The library and its
errors are those of the ``bdfp4`` module.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import bdfp4
from .bdfp4 import BDFP4Error, PAGE_SLOTS

E4M3, E5M2 = 0, 1
DTYPES = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
BLOCK_TOKENS = 16
ROTATE_HALVES, ROTATE_ADJACENT = 0, 1
DEV_BAD_POSITION = 16

#: names of every entry point declared in include/bdfp8.h
ENTRY_POINTS = ("bdfp8_append", "bdfp8_decode_plan", "bdfp8_decode_workspace_size", "bdfp8_decode")

_lib = None


def load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = bdfp4.load()
        i, i64, p, f, sz = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
        L.bdfp8_append.argtypes = [p, i64, p, i64, p, i64, p, p, p, p, p, i, i, i, p, p, p, i, i, i, i, i, i, i64, i, p,
                                   p, p, p, p]
        L.bdfp8_append.restype = i
        L.bdfp8_decode_plan.argtypes = [p, i, i, i, i, i, i, i, i]
        L.bdfp8_decode_plan.restype = i
        L.bdfp8_decode_workspace_size.argtypes = [i, i, i, i, i, i, i, i, i]
        L.bdfp8_decode_workspace_size.restype = sz
        L.bdfp8_decode.argtypes = [p, p, p, p, p, p, i, i, i, i, i, i, i64, i, i, i, f, i, p, sz, p, p, p]
        L.bdfp8_decode.restype = i
        _lib = L
    return _lib


def _need(ok: bool, what: str):
    if not ok:
        raise BDFP4Error(what)


def _like(t: torch.Tensor, dev: torch.device, dtype: torch.dtype, shape, what: str) -> int:
    """Data pointer of a contiguous tensor of this device, type and shape."""
    if t.device != dev or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise BDFP4Error(f"{what}: want a contiguous {dtype} tensor {tuple(shape)} on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} (strides {t.stride()}) on {t.device}")
    return t.data_ptr()


def _status(t: torch.Tensor | None, dev: torch.device):
    if t is None:
        return None
    _need(t.device == dev and t.dtype == torch.int32 and t.numel() == 1, "dev_status: want one int32 on " + str(dev))
    return t.data_ptr()


def _call(fn, dev: torch.device, stream, what: str, *args):
    """fn(*args, stream) with the tensors' device current, on `stream` or that device's current stream."""
    if dev.type != "cuda":
        raise BDFP4Error(f"{what}: tensors must be on a CUDA device, got {dev}")
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, (stream or torch.cuda.current_stream()).cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, (stream or torch.cuda.current_stream()).cuda_stream)
    if rc != 0:
        bdfp4._check(rc, what)


@dataclass
class FP8Cache:
    """The paged 8-bit KV cache arrays (layout in include/bdfp8.h)."""
    k_pages: torch.Tensor     # uint8 [num_pages, H_kv, 64 * d]
    v_pages: torch.Tensor     # uint8 [num_pages, H_kv, d * 64]
    kv_scales: torch.Tensor   # fp32 [num_pages, H_kv, 2, 4]
    num_pages: int
    H_kv: int
    d: int
    fmt: int

    @staticmethod
    def empty(num_pages: int, H_kv: int, d: int, fmt: int = E4M3, device="cuda") -> "FP8Cache":
        mk = lambda: torch.zeros((num_pages, H_kv, PAGE_SLOTS * d), dtype=torch.uint8, device=device)  # noqa: E731
        return FP8Cache(mk(), mk(), torch.ones((num_pages, H_kv, 2, 4), dtype=torch.float32, device=device), num_pages,
                        H_kv, d, fmt)

    def nbytes(self) -> int:
        return self.k_pages.numel() + self.v_pages.numel() + 4 * self.kv_scales.numel()

    def _ptrs(self, dev: torch.device):
        n = (self.num_pages, self.H_kv, PAGE_SLOTS * self.d)
        return (_like(self.k_pages, dev, torch.uint8, n, "k_pages"), _like(self.v_pages, dev, torch.uint8, n, "v_pages"),
                _like(self.kv_scales, dev, torch.float32, (self.num_pages, self.H_kv, 2, 4), "kv_scales"))


@dataclass
class OpenBlocks:
    """The tokens of each sequence's last block, kept across appends."""
    k_open: torch.Tensor   # fp32 [B, 16, H_kv, d] (rotated keys)
    v_open: torch.Tensor   # bf16 [B, 16, H_kv, d]

    @staticmethod
    def empty(B: int, H_kv: int, d: int, device="cuda") -> "OpenBlocks":
        mk = lambda t: torch.zeros((B, BLOCK_TOKENS, H_kv, d), dtype=t, device=device)  # noqa: E731
        return OpenBlocks(mk(torch.float32), mk(torch.bfloat16))


def _rows(t: torch.Tensor, dev, T, H, d, what: str):
    """(pointer, token stride) of bf16 rows [T, H, d] with contiguous heads."""
    if t.device != dev or t.dtype != torch.bfloat16 or t.dim() != 3 or t.shape[0] != T or t.shape[1] != H or \
            t.shape[2] != d or (d > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != d):
        raise BDFP4Error(f"{what}: want bf16 [{T}, {H}, {d}] on {dev} with contiguous heads, got {t.dtype} "
                         f"{tuple(t.shape)} (strides {t.stride()}) on {t.device}")
    return t.data_ptr(), (t.stride(0) if T > 1 else H * d)


def bdfp8_append(k: torch.Tensor, v: torch.Tensor, cu_tokens: torch.Tensor, seq_lens: torch.Tensor,
                 block_table: torch.Tensor, cos_sin: torch.Tensor | None, cache: FP8Cache, open_blocks: OpenBlocks,
                 q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, interleaved: bool = False,
                 dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Append the rows k, v [T, H_kv, d] of B sequences (rows cu_tokens[b] ..
    cu_tokens[b + 1] - 1 each; seq_lens counts them), rotating keys and, into q_out,
    queries q [T, H_q, d] by cos_sin [max_pos, rot_dim] (None: no rotation);
    interleaved pairs adjacent elements (bdfp8_append in bdfp8.h).  Returns q_out."""
    dev, T, H, d = k.device, k.shape[0], cache.H_kv, cache.d
    B, max_pages = block_table.shape
    kp, ks = _rows(k, dev, T, H, d, "k")
    vp, vs = _rows(v, dev, T, H, d, "v")
    H_q, qp, qs, op = H, None, 0, None
    if q is not None:
        H_q = q.shape[1]
        qp, qs = _rows(q, dev, T, H_q, d, "q")
        if q_out is None:
            q_out = torch.empty((T, H_q, d), dtype=torch.bfloat16, device=dev)
        op = _like(q_out, dev, torch.bfloat16, (T, H_q, d), "q_out")
    else:
        _need(q_out is None, "q_out without q")
    rot, max_pos, cs = 0, 0, None
    if cos_sin is not None:
        _need(cos_sin.dim() == 2, "cos_sin: want [max_pos, rot_dim]")
        max_pos, rot = cos_sin.shape
        cs = _like(cos_sin, dev, torch.float32, (max_pos, rot), "cos_sin")
    pages = cache._ptrs(dev)
    _call(load().bdfp8_append, dev, stream, "bdfp8_append", kp, ks, vp, vs, qp, qs, op,
          _like(cu_tokens, dev, torch.int32, (B + 1,), "cu_tokens"), _like(seq_lens, dev, torch.int32, (B,), "seq_lens"),
          None if positions is None else _like(positions, dev, torch.int32, (T,), "positions"), cs, rot, max_pos,
          ROTATE_ADJACENT if interleaved else ROTATE_HALVES,
          _like(open_blocks.k_open, dev, torch.float32, (B, BLOCK_TOKENS, H, d), "k_open"),
          _like(open_blocks.v_open, dev, torch.bfloat16, (B, BLOCK_TOKENS, H, d), "v_open"),
          _like(block_table, dev, torch.int32, (B, max_pages), "block_table"), B, T, H_q, H, d, max_pages,
          cache.num_pages, cache.fmt, pages[0], pages[1], pages[2], _status(dev_status, dev))
    return q_out


def bdfp8_decode_plan(host_seq_lens, T_q: int, H_q: int, H_kv: int, d: int, num_sms: int, window: int = 0,
                      sinks: int = 0) -> int:
    """Tiles per split for bdfp8_decode on these lengths."""
    import numpy as np
    sl = np.ascontiguousarray(host_seq_lens, dtype=np.int32)
    rc = load().bdfp8_decode_plan(sl.ctypes.data, sl.shape[0], T_q, H_q, H_kv, d, window, sinks, num_sms)
    if rc < 0:
        bdfp4._check(rc, "bdfp8_decode_plan")
    return rc


def bdfp8_decode_workspace_size(B: int, T_q: int, H_q: int, H_kv: int, d: int, max_pages_per_seq: int,
                                chunk_tiles: int, window: int = 0, sinks: int = 0) -> int:
    return int(load().bdfp8_decode_workspace_size(B, T_q, H_q, H_kv, d, max_pages_per_seq, window, sinks, chunk_tiles))


def workspace_for(B: int, T_q: int, H_q: int, H_kv: int, d: int, max_pages_per_seq: int, chunk_tiles: int,
                  window: int = 0, sinks: int = 0, device="cuda") -> torch.Tensor:
    n = bdfp8_decode_workspace_size(B, T_q, H_q, H_kv, d, max_pages_per_seq, chunk_tiles, window, sinks)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def bdfp8_decode(q: torch.Tensor, cache: FP8Cache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 sm_scale: float, chunk_tiles: int, workspace: torch.Tensor | None, out: torch.Tensor,
                 window: int = 0, sinks: int = 0, dev_status: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Causal attention of each sequence's T_q newest tokens, q [B, T_q, H_q, d], over
    the 8-bit cache into out; window > 0 limits each to its window newest tokens
    and the first `sinks` (bdfp8_decode in bdfp8.h)."""
    dev = q.device
    B, T_q, H_q, d = q.shape
    max_pages = block_table.shape[1]
    _need(d == cache.d, f"q: head dim {d}, the cache has {cache.d}")
    pages = cache._ptrs(dev)
    wp, wb = None, 0
    if workspace is not None:
        _need(workspace.device == dev and workspace.is_contiguous(), f"workspace: want contiguous memory on {dev}")
        wp, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(load().bdfp8_decode, dev, stream, "bdfp8_decode", _like(q, dev, torch.bfloat16, q.shape, "q"), pages[0], pages[1],
          pages[2], _like(block_table, dev, torch.int32, (B, max_pages), "block_table"),
          _like(seq_lens, dev, torch.int32, (B,), "seq_lens"), B, T_q, H_q, cache.H_kv, d, max_pages, cache.num_pages,
          cache.fmt, window, sinks, sm_scale, chunk_tiles, wp, wb, _like(out, dev, torch.bfloat16, q.shape, "out"),
          _status(dev_status, dev))
    return out
