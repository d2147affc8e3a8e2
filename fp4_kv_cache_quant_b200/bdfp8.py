"""Thin binding of the 8-bit paged cache (include/bdfp8.h).

Argument checks and marshalling only (those of the append and the decode in an
extension module, csrc/py_bdfp8.cpp, where a call costs microseconds less): the
work runs in libbdfp4.so's CUDA kernels, on the current stream of the tensors'
device.  The library and its errors are those of the ``bdfp4`` module.
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
#: names of every entry point declared in include/bdfp8_debug.h (test hooks)
DEBUG_ENTRY_POINTS = ("bdfp8_debug_decode_wait_test",)
STALL_NONE, STALL_TILE, STALL_WARP = 0, 1, 2

_lib = None
_py = None


def load() -> ctypes.CDLL:
    """Load libbdfp4.so and the extension module beside it (raises if they have not been built)."""
    global _lib, _py
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
        L.bdfp8_debug_decode_wait_test.argtypes = [p, p, p, p, p, p, i, i, i, i, i, i, i64, i, i, i, f, i, p, sz, p, p,
                                                   ctypes.c_longlong, i, p]
        L.bdfp8_debug_decode_wait_test.restype = i
        try:
            from . import _bdfp8_py
        except ImportError as e:
            raise OSError("the extension module of the 8-bit cache's calls is missing or does not load: build it with "
                          f"`python -m fp4_kv_cache_quant_b200.build` (g++, Python's and torch's headers): {e}") from e
        _bdfp8_py.set_error(BDFP4Error)
        _lib, _py = L, _bdfp8_py
    return _lib


def _calls():
    """The extension module with the calls of a serving loop."""
    if _py is None:
        load()
    return _py


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


@dataclass
class OpenBlocks:
    """The tokens of each sequence's last block, kept across appends."""
    k_open: torch.Tensor   # fp32 [B, 16, H_kv, d] (rotated keys)
    v_open: torch.Tensor   # bf16 [B, 16, H_kv, d]

    @staticmethod
    def empty(B: int, H_kv: int, d: int, device="cuda") -> "OpenBlocks":
        mk = lambda t: torch.zeros((B, BLOCK_TOKENS, H_kv, d), dtype=t, device=device)  # noqa: E731
        return OpenBlocks(mk(torch.float32), mk(torch.bfloat16))


def bdfp8_append(k: torch.Tensor, v: torch.Tensor, cu_tokens: torch.Tensor, seq_lens: torch.Tensor,
                 block_table: torch.Tensor, cos_sin: torch.Tensor | None, cache: FP8Cache, open_blocks: OpenBlocks,
                 q: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, interleaved: bool = False,
                 dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Append the rows k, v [T, H_kv, d] of B sequences (rows cu_tokens[b] ..
    cu_tokens[b + 1] - 1 each; seq_lens counts them), rotating keys and, into q_out,
    queries q [T, H_q, d] by cos_sin [max_pos, rot_dim] (None: no rotation);
    interleaved pairs adjacent elements (bdfp8_append in bdfp8.h).  Returns q_out, which
    is allocated on `stream` where it is not given (rows of no sequence are not written)."""
    if q is not None and q_out is None:
        # from the pool of the stream that writes it
        with torch.cuda.stream(stream):
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    rc = (_py or _calls()).append(
        k, v, cu_tokens, seq_lens, block_table, cos_sin, cache.k_pages, cache.v_pages, cache.kv_scales, cache.num_pages,
        cache.H_kv, cache.d, cache.fmt, open_blocks.k_open, open_blocks.v_open, q, q_out, positions,
        ROTATE_ADJACENT if interleaved else ROTATE_HALVES, dev_status, stream and stream.cuda_stream)
    if rc:
        bdfp4._check(rc, "bdfp8_append")
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
    rc = (_py or _calls()).decode(
        q, cache.k_pages, cache.v_pages, cache.kv_scales, cache.num_pages, cache.H_kv, cache.d, cache.fmt, block_table,
        seq_lens, sm_scale, chunk_tiles, workspace, out, window, sinks, dev_status, stream and stream.cuda_stream)
    if rc:
        bdfp4._check(rc, "bdfp8_decode")
    return out


def bdfp8_debug_decode_wait_test(q: torch.Tensor, cache: FP8Cache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                                 sm_scale: float, chunk_tiles: int, workspace: torch.Tensor | None, out: torch.Tensor,
                                 wait_limit_cycles: int, stall: int, window: int = 0, sinks: int = 0,
                                 dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Test hook (include/bdfp8_debug.h): bdfp8_decode with a short in-kernel wait
    bound and something (STALL_*) going wrong in every block."""
    B, T_q, H_q, d = q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ptr = bdfp4._ptr
    rc = load().bdfp8_debug_decode_wait_test(
        ptr(q), ptr(cache.k_pages), ptr(cache.v_pages), ptr(cache.kv_scales), ptr(block_table), ptr(seq_lens), B, T_q,
        H_q, cache.H_kv, d, block_table.shape[1], cache.num_pages, cache.fmt, window, sinks, float(sm_scale),
        int(chunk_tiles), ptr(workspace), ws_bytes, ptr(out), ptr(dev_status), int(wait_limit_cycles), int(stall),
        bdfp4._stream(stream))
    bdfp4._check(rc, "bdfp8_debug_decode_wait_test")
    return out
