"""Host-only checks of the 8-bit cache's entry points (include/bdfp8.h): exports,
refusals before any launch, the split plan, and the reference the GPU tests use."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import _fp8_ref as ref
from fp4_kv_cache_quant_b200 import bdfp4, bdfp8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from fp4_kv_cache_quant_b200 import build
    build.build()
    return bdfp8.load()


def test_exports_and_constants_match_the_header(lib):
    hdr = open(os.path.join(ROOT, "include", "bdfp8.h")).read()
    names = re.findall(r"BDFP4_API\s+[\w\s\*]+?\b(bdfp8_\w+)\s*\(", hdr)
    assert sorted(names) == sorted(bdfp8.ENTRY_POINTS)
    for n in names:
        assert hasattr(lib, n), n
    assert "BDFP8_E4M3 = 0, BDFP8_E5M2 = 1" in hdr and (bdfp8.E4M3, bdfp8.E5M2) == (0, 1)
    defs = dict(re.findall(r"#define (BDFP8_\w+) (\d+)", hdr))
    assert int(defs["BDFP8_DEV_BAD_POSITION"]) == bdfp8.DEV_BAD_POSITION
    assert bdfp8.DEV_BAD_POSITION not in (bdfp4.DEV_BAD_PAGE, bdfp4.DEV_BAD_SEQLEN, bdfp4.DEV_BAD_SLOT,
                                          bdfp4.DEV_TIMEOUT)
    assert (int(defs["BDFP8_ROTATE_HALVES"]), int(defs["BDFP8_ROTATE_ADJACENT"])) == (bdfp8.ROTATE_HALVES,
                                                                                     bdfp8.ROTATE_ADJACENT)


def _p(addr):
    return ctypes.c_void_p(addr)


A = _p(0x10000)


def _decode(lib, **kw):
    a = dict(q=A, kp=A, vp=A, sc=A, bt=A, sl=A, B=2, T=1, H_q=8, H_kv=2, d=128, mp=4, np=16, fmt=0, w=0, s=0, scale=0.1,
             chunk=2, ws=None, wb=0, out=A)
    a.update(kw)
    return lib.bdfp8_decode(*[a[k] for k in a], None, None)


@pytest.mark.parametrize("want, kw", [
    (-1, dict(q=None)), (-1, dict(out=None)), (-1, dict(sc=None)), (-1, dict(B=-1)), (-1, dict(T=0)), (-1, dict(mp=0)),
    (-1, dict(fmt=2)), (-1, dict(w=-1)), (-1, dict(s=-1)), (-1, dict(H_kv=0)), (-1, dict(np=-1)),
    (-2, dict(H_q=7)),
    (-3, dict(q=_p(0x10008))), (-3, dict(kp=_p(0x10040))), (-3, dict(sc=_p(0x10010))), (-3, dict(bt=_p(0x10002))),
    (-4, dict(d=96)), (-4, dict(d=256)), (-4, dict(mp=(1 << 24) + 1)), (-4, dict(T=1 << 23)), (-4, dict(np=1 << 31)),
    (-6, dict(chunk=1)),                                   # two splits want a workspace
    (-6, dict(chunk=1, ws=A, wb=16)),
    (0, dict(B=0, q=None)),
])
def test_decode_refusals(lib, want, kw):
    assert _decode(lib, **kw) == want


def _append(lib, **kw):
    a = dict(k=A, ks=256, v=A, vs=256, q=A, qs=1024, qo=A, cu=A, sl=A, pos=None, cs=A, rot=128, mpos=64, pair=0, ko=A, vo=A,
             bt=A, B=2, T=10, H_q=8, H_kv=2, d=128, mp=4, np=16, fmt=0, kp=A, vp=A, sc=A)
    a.update(kw)
    return lib.bdfp8_append(*[a[k] for k in a], None, None)


@pytest.mark.parametrize("want, kw", [
    (-1, dict(k=None)), (-1, dict(cu=None)), (-1, dict(cs=None)), (-1, dict(ko=None)), (-1, dict(q=None)),
    (-1, dict(qo=None)), (-1, dict(T=-1)), (-1, dict(B=-1)), (-1, dict(fmt=3)), (-1, dict(pair=2)), (-1, dict(rot=-16)),
    (-2, dict(H_q=7)), (-2, dict(rot=24)), (-2, dict(rot=144)), (-2, dict(ks=255)), (-2, dict(qs=512)),
    (-3, dict(k=_p(0x10008))), (-3, dict(ks=260)), (-3, dict(qs=1028)), (-3, dict(ko=_p(0x10010))),
    (-3, dict(vp=_p(0x10010))), (-3, dict(sc=_p(0x10010))), (-3, dict(cu=_p(0x10002))), (-3, dict(cs=_p(0x10008))),
    (-4, dict(d=96, ks=192, vs=192, rot=32)), (-4, dict(T=1 << 30, B=1 << 27)),
    (0, dict(T=0)), (0, dict(B=0)),
])
def test_append_refusals(lib, want, kw):
    assert _append(lib, **kw) == want


def test_binding_refuses_what_the_pointers_would_hide(lib):
    """Types, shapes, strides and devices, before the library sees an address."""
    c = bdfp8.FP8Cache.empty(2, 2, 128, device="cpu")
    bt, sl = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 128), dtype=torch.bfloat16)

    def dec(q=q, c=c, bt=bt, sl=sl, out=None, **kw):
        return bdfp8.bdfp8_decode(q, c, bt, sl, 0.1, 1, None, torch.empty_like(q) if out is None else out, **kw)
    for bad in (dict(q=q.float()), dict(q=q[..., :64]), dict(bt=bt.long()), dict(sl=sl.repeat(2)),
                dict(out=q[:, :, :2]), dict(q=q.transpose(1, 2)), dict(dev_status=torch.zeros(1))):
        with pytest.raises(bdfp4.BDFP4Error):
            dec(**bad)
    with pytest.raises(bdfp4.BDFP4Error, match="CUDA"):
        dec()
    o = bdfp8.OpenBlocks.empty(1, 2, 128, device="cpu")
    k = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32)

    def app(k=k, cu=cu, o=o, cs=None, **kw):
        return bdfp8.bdfp8_append(k, k, cu, sl, bt, cs, c, o, **kw)
    for bad in (dict(k=k.half()), dict(k=k.transpose(0, 1)), dict(cu=cu[:1]), dict(cs=torch.zeros(4, 32).double()),
                dict(q_out=k), dict(o=bdfp8.OpenBlocks.empty(2, 2, 128, device="cpu")),
                dict(positions=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(bdfp4.BDFP4Error):
            app(**bad)


def test_plan_and_workspace(lib):
    # never more tiles than a sequence has, one tile at the least
    assert bdfp8.bdfp8_decode_plan([0, 0], 1, 8, 2, 128, 148) == 1
    assert bdfp8.bdfp8_decode_plan([], 1, 8, 2, 128, 148) == 1
    for lens in ([100], [128 * 40], [32768] * 16, [131072, 5000, 1]):
        c = bdfp8.bdfp8_decode_plan(lens, 1, 32, 8, 128, 148)
        assert 1 <= c <= max(1, -(-max(lens) // 128))
    # a window bounds the tiles, whatever the length
    c = bdfp8.bdfp8_decode_plan([1 << 20], 1, 32, 8, 128, 148, window=1000, sinks=4)
    assert 1 <= c <= 10
    for bad in (dict(T_q=0), dict(H_q=7), dict(d=96), dict(num_sms=0), dict(window=-1)):
        kw = dict(T_q=1, H_q=8, H_kv=2, d=128, num_sms=148, window=0)
        kw.update(bad)
        with pytest.raises(bdfp4.BDFP4Error):
            bdfp8.bdfp8_decode_plan([100], **kw)
    # 16 pages = 8 tiles, 2 a split: 4 splits of d + 2 floats for each of the B T_q H_q rows
    rows = 2 * 3 * 4
    o = rows * 4 * 128 * 4
    assert bdfp8.bdfp8_decode_workspace_size(2, 3, 4, 1, 128, 16, 2) == (o + 255) // 256 * 256 + rows * 4 * 8
    assert bdfp8.bdfp8_decode_workspace_size(2, 3, 4, 1, 128, 16, 8) == 0
    # a window of 100 tokens spans two tiles at the most; its first tokens one more
    assert bdfp8.bdfp8_decode_workspace_size(2, 1, 4, 1, 128, 1 << 20, 3, window=100, sinks=4) == 0
    assert bdfp8.bdfp8_decode_workspace_size(2, 1, 4, 1, 128, 1 << 20, 2, window=100, sinks=4) > 0


def test_reference_codes_are_the_types():
    for fmt, t in bdfp8.DTYPES.items():
        want = torch.arange(256, dtype=torch.uint8).view(t).double().numpy()
        assert np.array_equal(ref.code_values(fmt), want, equal_nan=True)
    s = ref.scale_of(np.array([0.0, 448.0, 448.1, 224.0, 1e-45, 3e38]), bdfp8.E4M3)
    assert s.tolist()[:4] == [1.0, 1.0, 2.0, 0.5] and s[4] == 2.0 ** -126 and s[5] * 448 >= 3e38


def test_reference_layout_is_a_bijection():
    for d in (64, 128):
        for o in ref.offsets(d):
            assert np.array_equal(np.sort(o.reshape(-1)), np.arange(64 * d))


def test_wait_test_hook(lib):
    """include/bdfp8_debug.h: exports, constants, and what it refuses before a launch."""
    hdr = open(os.path.join(ROOT, "include", "bdfp8_debug.h")).read()
    names = re.findall(r"BDFP4_API\s+[\w\s\*]+?\b(bdfp8_\w+)\s*\(", hdr)
    assert tuple(names) == bdfp8.DEBUG_ENTRY_POINTS and all(hasattr(lib, n) for n in names)
    defs = dict(re.findall(r"#define (BDFP8_STALL_\w+) (\d+)", hdr))
    assert [int(defs["BDFP8_STALL_" + n]) for n in ("NONE", "TILE", "WARP")] == [bdfp8.STALL_NONE, bdfp8.STALL_TILE,
                                                                               bdfp8.STALL_WARP]

    def call(limit=1 << 20, stall=1, **kw):
        a = dict(q=A, kp=A, vp=A, sc=A, bt=A, sl=A, B=2, T=1, H_q=16, H_kv=2, d=128, mp=4, np=16, fmt=0, w=0, s=0,
                 scale=0.1, chunk=2, ws=None, wb=0, out=A)
        a.update(kw)
        return lib.bdfp8_debug_decode_wait_test(*[a[k] for k in a], None, limit, stall, None)
    assert call(limit=0) == -1 and call(stall=3) == -1 and call(stall=-1) == -1 and call(q=None) == -1
    assert call(B=0) == 0


@pytest.mark.parametrize("sinks", [2 ** 31 - 1, 2 ** 31 - 127, 2 ** 31 - 128])
def test_first_tokens_without_end(lib, sinks):
    """Any count of first tokens: they are those of the table at the most, in the plan and the workspace as in the decode."""
    mp = 64   # 4096 tokens, 32 tiles
    want = bdfp8.bdfp8_decode_workspace_size(2, 1, 8, 2, 128, mp, 2, window=100, sinks=mp * 64)
    assert want == bdfp8.bdfp8_decode_workspace_size(2, 1, 8, 2, 128, mp, 2) > 0
    assert bdfp8.bdfp8_decode_workspace_size(2, 1, 8, 2, 128, mp, 2, window=100, sinks=sinks) == want
    lens = [4096, 2000]
    assert bdfp8.bdfp8_decode_plan(lens, 1, 8, 2, 128, 148, window=100, sinks=sinks) == \
        bdfp8.bdfp8_decode_plan(lens, 1, 8, 2, 128, 148, window=100, sinks=4096)
    # the decode, which asks for the same workspace, refuses one byte less before a launch
    assert _decode(lib, mp=mp, w=100, s=sinks, ws=A, wb=want - 1) == -6
