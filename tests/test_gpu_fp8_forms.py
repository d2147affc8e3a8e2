"""GPU tests of the 8-bit decode in its other types: head dim 64 and E5M2, with several query tokens, windows, merges in
clusters and behind them, bad pages, and append and decode together."""
import numpy as np
import pytest
import torch

from fp4_kv_cache_quant_b200 import bdfp4, bdfp8
from test_gpu_fp8 import EDGES, Loop, _loop_check, _status, check, decode, make_cache, queries

pytestmark = pytest.mark.gpu

FORMS = pytest.mark.parametrize("d, fmt", [(64, bdfp8.E4M3), (64, bdfp8.E5M2), (128, bdfp8.E5M2)])


@FORMS
@pytest.mark.parametrize("chunk", [1, "plan"])
@pytest.mark.parametrize("T, G", [(2, 1), (2, 2), (3, 2), (8, 1), (4, 4), (5, 3), (2, 9), (17, 4), (70, 2)])
def test_several_query_tokens(T, G, d, fmt, chunk):
    lens = [max(n, T) for n in EDGES[1:]] + [0]
    cache, bt = make_cache(lens, 2, d, fmt, 90)
    q = queries(len(lens), T, 2 * G, d, 91)
    st = _status()
    check(decode(q, cache, bt, lens, chunk, status=st), q, cache, bt, lens)
    assert int(st) == 0


@FORMS
@pytest.mark.parametrize("chunk", [1, "plan", 0])
@pytest.mark.parametrize("T, G", [(1, 4), (1, 8), (1, 16), (3, 1), (3, 2), (3, 4), (1, 24), (40, 4)])
@pytest.mark.parametrize("window, sinks", [(1, 1), (17, 4), (100, 130), (300, 5)])
def test_windows(window, sinks, T, G, d, fmt, chunk):
    lens = [max(n, T) for n in (1, 64, 129, 385, 700)]
    cache, bt = make_cache(lens, 1, d, fmt, 92, window, sinks, T)
    q = queries(len(lens), T, G, d, 93)
    st = _status()
    check(decode(q, cache, bt, lens, chunk, window, sinks, st), q, cache, bt, lens, window, sinks)
    assert int(st) == 0


@FORMS
@pytest.mark.parametrize("T, G", [(1, 4), (1, 8), (1, 16), (2, 2), (2, 4), (2, 8), (1, 24)])
@pytest.mark.parametrize("n", [64 * 10, 64 * 14 + 9, 3000])
def test_merges(n, T, G, d, fmt):
    """Few splits, which merge in a cluster, and many; shorter sequences beside them."""
    lens = [n, n // 3, 0]
    cache, bt = make_cache(lens, 2, d, fmt, 94)
    q = queries(3, T, 2 * G, d, 95)
    for chunk in (1, 2, 1000):
        check(decode(q, cache, bt, lens, chunk), q, cache, bt, lens)


@FORMS
@pytest.mark.parametrize("T, G", [(1, 4), (3, 4), (1, 24)])
def test_bad_pages(T, G, d, fmt):
    lens = [385, 64, 200]
    cache, bt = make_cache(lens, 2, d, fmt, 96)
    bt[0, 1], bt[0, 4], bt[1, 0] = -5, cache.num_pages, 2 ** 31 - 1
    q = queries(3, T, 2 * G, d, 97)
    for chunk in (1, 4):
        st = _status()
        got = check(decode(q, cache, bt, lens, chunk, status=st), q, cache, bt, lens)
        assert int(st) == bdfp4.DEV_BAD_PAGE and np.all(got[1] == 0)


@FORMS
@pytest.mark.parametrize("T, G", [(1, 4), (1, 16), (3, 4), (1, 24)])
def test_negative_and_tiny_rows(T, G, d, fmt):
    lens = [150, 150]
    cache, bt = make_cache(lens, 1, d, fmt, 98)
    q = queries(2, T, G, d, 99)
    q[1] *= 2.0 ** -125
    for scale in (-0.09, 0.0):
        check(decode(q, cache, bt, lens, 1, scale=scale), q, cache, bt, lens, scale=scale)


@FORMS
@pytest.mark.parametrize("window, sinks", [(0, 0), (33, 3)])
def test_prompt_chunks_drafts_and_single_tokens(d, fmt, window, sinks):
    """As a server has them, one behind the other over one cache."""
    lp = Loop(2, 2, 8, d, fmt, d // 2, True, seed=100)
    for n in (70, 70, 4, 1, 4, 1):
        q, _ = lp.append([n, n], tail=0)
        lp.check()
        _loop_check(lp, q, lp.lens, window, sinks, 1 if n < 70 else 2)


@FORMS
def test_a_captured_window_step(d, fmt):
    """Append and windowed decode captured and replayed over growing lengths: the same bits as eager calls."""
    lp, twin = (Loop(2, 2, 8, d, fmt, d, False, seed=101) for _ in range(2))
    for x in (lp, twin):
        x.append([37, 120], tail=0)
    dev = dict(device="cuda")
    bt, cs = torch.from_numpy(lp.bt).cuda(), torch.from_numpy(lp.cs).cuda()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, **dev)
    qkv, lens = torch.zeros((2, 12, d), dtype=torch.bfloat16, **dev), torch.zeros(2, dtype=torch.int32, **dev)
    outs = [torch.empty((2, 1, 8, d), dtype=torch.bfloat16, **dev) for _ in range(2)]
    qo = [torch.empty((2, 8, d), dtype=torch.bfloat16, **dev) for _ in range(2)]
    wss = [bdfp8.workspace_for(2, 1, 8, 2, d, bt.shape[1], 1, 50, 3) for _ in range(2)]

    def step(x, i):
        bdfp8.bdfp8_append(qkv[:, 8:10], qkv[:, 10:], cu, lens, bt, cs, x.cache, x.open, q=qkv[:, :8], q_out=qo[i])
        bdfp8.bdfp8_decode(qo[i].view(2, 1, 8, d), x.cache, bt, lens, 0.09, 1, wss[i], outs[i], window=50, sinks=3)
    lens.copy_(torch.tensor([38, 121]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(lp, 0)
    g = torch.Generator().manual_seed(102)
    for s in range(4):
        qkv.copy_(torch.randn((2, 12, d), generator=g))
        lens.copy_(torch.tensor([38 + s, 121 + s]))
        graph.replay()
        step(twin, 1)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        check(outs[0], qo[0].view(2, 1, 8, d).cpu(), lp.cache, lp.bt, [38 + s, 121 + s], 50, 3, scale=0.09)
    for name in ("k_pages", "v_pages", "kv_scales"):
        assert torch.equal(getattr(lp.cache, name), getattr(twin.cache, name))


@FORMS
@pytest.mark.parametrize("T, G", [(5, 2), (16, 1), (40, 4), (140, 1)])
@pytest.mark.parametrize("window, sinks", [(0, 0), (7, 2)])
def test_sequences_shorter_than_their_query_tokens(T, G, d, fmt, window, sinks):
    """Rows before the first token see nothing: zeros, and the length is reported."""
    lens = [3, T - 1, T + 90, 0]
    cache, bt = make_cache(lens, 2, d, fmt, 103, window, sinks, T)
    q = queries(4, T, 2 * G, d, 104)
    for chunk in (1, 2):
        st = _status()
        got = check(decode(q, cache, bt, lens, chunk, window, sinks, st), q, cache, bt, lens, window, sinks)
        assert int(st) == bdfp4.DEV_BAD_SEQLEN and not got[0, : T - 3].any() and not got[3].any()
