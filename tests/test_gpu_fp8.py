"""GPU tests of the 8-bit paged cache (include/bdfp8.h) against the 64-bit reference of
_fp8_ref.py, which states the attention's tolerance.  Slots and blocks that no append wrote hold NaN
codes and NaN scales, pages that no query sees are -1."""
import math

import numpy as np
import pytest
import torch

import _fp8_ref as ref
from fp4_kv_cache_quant_b200 import bdfp4, bdfp8

pytestmark = pytest.mark.gpu

SMS = 148


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def make_cache(lens, H, d, fmt, seed, window=0, sinks=0, T_q=1, spread=0, extra_pages=3):
    """A cache with random codes in the tokens that exist, junk everywhere else -> (cache, block_table)."""
    rng = np.random.default_rng(seed)
    mp = max(1, max((n + 63) // 64 for n in lens)) + 1
    bt = np.full((len(lens), mp), -1, np.int32)
    used = []
    for b, n in enumerate(lens):
        lo = max(0, n - T_q - window + 1) if window else 0
        used += [(b, p) for p in range((n + 63) // 64) if p * 64 + 64 > lo or p * 64 < sinks]
    P = len(used) + extra_pages
    perm = rng.permutation(P)
    nan = 0x7F
    k = np.full((P, H, 64, d), nan, np.uint8)
    v = np.full((P, H, 64, d), nan, np.uint8)
    sc = np.full((P, H, 2, 4), np.nan, np.float32)
    for i, (b, p) in enumerate(used):
        pg = perm[i]
        bt[b, p] = pg
        n = min(64, lens[b] - p * 64)
        for x in (k, v):
            t = torch.from_numpy(rng.standard_normal((H, n, d)).astype(np.float32)).to(bdfp8.DTYPES[fmt])
            x[pg, :, :n] = t.view(torch.uint8).numpy()
        nb = (n + 15) // 16
        sc[pg, :, :, :nb] = 2.0 ** rng.uniform(-1, 1, (H, 2, nb)) if not spread else 1.0
        if spread:
            sc[pg, :, 1, :nb] = 2.0 ** rng.uniform(-spread, spread, (H, nb))
    ko, vo = ref.offsets(d)
    kp, vp = np.zeros((P, H, 64 * d), np.uint8), np.zeros((P, H, 64 * d), np.uint8)
    kp[:, :, ko] = k
    vp[:, :, vo] = v
    cache = bdfp8.FP8Cache(torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(), torch.from_numpy(sc).cuda(), P, H, d, fmt)
    return cache, bt


def queries(B, T, Hq, d, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, T, Hq, d), generator=g).to(torch.bfloat16)


def decode(q, cache, bt, lens, chunk, window=0, sinks=0, status=None, scale=None, out=None, ws=None):
    B, T, Hq, d = q.shape
    mp = bt.shape[1]
    if chunk == "plan":
        chunk = bdfp8.bdfp8_decode_plan(np.maximum(lens, 0), T, Hq, cache.H_kv, d, SMS, window, sinks)
    if ws is None:
        ws = bdfp8.workspace_for(B, T, Hq, cache.H_kv, d, mp, max(chunk, 1), window, sinks)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    bdfp8.bdfp8_decode(q.cuda(), cache, torch.from_numpy(np.asarray(bt, np.int32)).cuda(),
                       torch.tensor(list(lens), dtype=torch.int32, device="cuda"), 1 / math.sqrt(d) if scale is None else scale,
                       chunk, ws, out, window=window, sinks=sinks, dev_status=status)
    return out


def check(out, q, cache, bt, lens, window=0, sinks=0, scale=None):
    K, V = ref.values_of(cache)
    want, tol = ref.attention(q.double().numpy(), K, V, bt, lens, 1 / math.sqrt(q.shape[3]) if scale is None else scale,
                              window, sinks)
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    off = np.abs(got - want) - tol
    assert np.all(off <= 0), (float(off.max()), np.unravel_index(off.argmax(), off.shape))
    return got


EDGES = [0, 1, 15, 16, 63, 64, 65, 127, 128, 129, 200, 385]


@pytest.mark.parametrize("chunk", [1, 2, "plan", 0])
@pytest.mark.parametrize("fmt", [bdfp8.E4M3, bdfp8.E5M2])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H, G", [(1, 1), (2, 4), (2, 8), (1, 13), (1, 32), (1, 41)])
def test_decode_lengths_and_head_layouts(H, G, d, fmt, chunk):
    cache, bt = make_cache(EDGES, H, d, fmt, 1)
    q = queries(len(EDGES), 1, H * G, d, 2)
    st = _status()
    out = decode(q, cache, bt, EDGES, chunk, status=st)
    got = check(out, q, cache, bt, EDGES)
    assert int(st) == 0 and np.all(got[0] == 0)


@pytest.mark.parametrize("chunk", [1, "plan"])
@pytest.mark.parametrize("T, G", [(2, 1), (3, 2), (4, 4), (5, 3), (2, 9), (17, 4), (70, 1)])
def test_decode_several_query_tokens(T, G, chunk):
    lens = [max(n, T) for n in EDGES[1:]] + [0]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 3)
    q = queries(len(lens), T, 2 * G, 128, 4)
    st = _status()
    check(decode(q, cache, bt, lens, chunk, status=st), q, cache, bt, lens)
    assert int(st) == 0


@pytest.mark.parametrize("chunk", [1, 2, "plan", 0])
@pytest.mark.parametrize("T", [1, 3, 40])
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (17, 4), (64, 64), (100, 130), (128, 0), (300, 5), (1000, 3), (2 ** 31 - 1, 7)])
def test_window_and_first_tokens(window, sinks, T, chunk):
    lens = [max(n, T) for n in (1, 64, 129, 385, 700)]
    cache, bt = make_cache(lens, 1, 128, bdfp8.E4M3, 5, window, sinks, T)
    q = queries(len(lens), T, 4, 128, 6)
    st = _status()
    check(decode(q, cache, bt, lens, chunk, window, sinks, st), q, cache, bt, lens, window, sinks)
    assert int(st) == 0   # pages that nothing sees are -1 and were not looked up


def test_window_equals_the_whole_context_when_it_covers_it():
    lens = [300, 90]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 7)
    q = queries(2, 1, 8, 128, 8)
    a = decode(q, cache, bt, lens, 1)
    assert torch.equal(a, decode(q, cache, bt, lens, 1, window=300, sinks=0))
    assert torch.equal(a, decode(q, cache, bt, lens, 1, window=10 ** 6, sinks=10 ** 6))
    assert torch.equal(a, decode(q, cache, bt, lens, 1, window=0, sinks=9))


@pytest.mark.parametrize("G", [4, 24])
def test_bad_pages_are_left_out_and_reported(G):
    lens = [385, 64, 200]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 9)
    bt[0, 1], bt[0, 4], bt[1, 0] = -5, cache.num_pages, 2 ** 31 - 1
    q = queries(3, 1, 2 * G, 128, 10)
    for chunk in (1, 4):
        st = _status()
        got = check(decode(q, cache, bt, lens, chunk, status=st), q, cache, bt, lens)
        assert int(st) == bdfp4.DEV_BAD_PAGE and np.all(got[1] == 0)


def test_bad_lengths_give_zeros_and_are_reported():
    cache, bt = make_cache([100, 100, 100, 3], 1, 128, bdfp8.E4M3, 11)
    for lens, T in (([-1, 100, 100, 3], 1), ([100, bt.shape[1] * 64 + 1, 100, 3], 1), ([100, 100, 100, 3], 5)):
        q = queries(4, T, 4, 128, 12)
        st = _status()
        check(decode(q, cache, bt, lens, 1, status=st), q, cache, bt, lens)
        assert int(st) == bdfp4.DEV_BAD_SEQLEN


@pytest.mark.parametrize("G", [4, 8, 16, 24])
@pytest.mark.parametrize("spread", [3, 14])
def test_value_scales_far_apart(spread, G):
    lens = [500, 129]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 13, spread=spread)
    q = queries(2, 1, 2 * G, 128, 14)
    for chunk in (1, 5):
        check(decode(q, cache, bt, lens, chunk), q, cache, bt, lens)


@pytest.mark.parametrize("G", [4, 24])
def test_a_first_token_with_a_faint_crowd_behind_it(G):
    """One token with half the weight, 32767 others sharing the rest: their probabilities are
    2^-15 of the largest and must not be lost."""
    n, d = 32768, 128
    P = n // 64
    kv = torch.zeros((2, P, 1, 64, d))
    q = torch.zeros((1, 1, G, d), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    kv[0, 0, 0, 0, 0] = 10.4   # exp(10.4) = 2^15.0
    kv[1] = torch.randn(kv[1].shape, generator=torch.Generator().manual_seed(1)) * 0.1 + 1.0
    kv[1, 0, 0, 0] = -1.0
    c = kv.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    ko, vo = ref.offsets(d)
    kp, vp = np.zeros((P, 1, 64 * d), np.uint8), np.zeros((P, 1, 64 * d), np.uint8)
    kp[:, :, ko], vp[:, :, vo] = c[0], c[1]
    cache = bdfp8.FP8Cache(torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(),
                           torch.ones((P, 1, 2, 4), device="cuda"), P, 1, d, bdfp8.E4M3)
    bt = np.arange(P, dtype=np.int32)[None]
    for chunk in (32, 256):
        check(decode(q, cache, bt, [n], chunk, scale=1.0), q, cache, bt, [n], scale=1.0)


@pytest.mark.parametrize("G", [4, 24])
def test_what_is_not_a_number_reaches_the_rows_that_see_it_only(G):
    lens = [200, 200]
    cache, bt = make_cache(lens, 1, 128, bdfp8.E4M3, 15)
    q = queries(2, 3, G, 128, 16)
    q[0, 1, 2, 5] = float("nan")
    q[1, 0, 0, 7] = float("inf")
    got = decode(q, cache, bt, lens, 1).float().cpu()
    nan = torch.isnan(got).all(-1)
    want = torch.zeros_like(nan)
    want[0, 1, 2] = want[1, 0, 0] = True
    assert torch.equal(nan, want) and torch.equal(torch.isnan(got).any(-1), want)
    # a NaN scale of a visible block, for keys and for values
    for which in (0, 1):
        c2 = bdfp8.FP8Cache(cache.k_pages, cache.v_pages, cache.kv_scales.clone(), *list(vars(cache).values())[3:])
        c2.kv_scales[int(bt[0, 0]), 0, which, 2] = float("nan")
        q = queries(2, 1, G, 128, 17)
        got = decode(q, c2, bt, lens, 2).float().cpu()
        assert torch.isnan(got[0]).all() and not torch.isnan(got[1]).any()
        got = decode(q, c2, bt, lens, 2, window=100).float().cpu()   # behind the window: no influence
        assert not torch.isnan(got).any()


@pytest.mark.parametrize("G", [1, 2, 5, 40])
def test_a_block_that_only_the_newest_query_sees(G):
    """Its NaN scale, for keys and values, leaves the rows of the earlier query tokens alone."""
    lens = [193, 65]   # the last token of each begins a block
    for which in (0, 1):
        cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 24)
        for b, n in enumerate(lens):
            cache.kv_scales[int(bt[b, n // 64]), :, which, 0] = float("nan")
        q = queries(2, 3, 2 * G, 128, 25)
        got = decode(q, cache, bt, lens, 1).float().cpu()
        assert torch.isnan(got[:, 2]).all() and not torch.isnan(got[:, :2]).any()


@pytest.mark.parametrize("G", [4, 8, 24])
def test_tiny_zero_and_negative(G):
    """Rows of zeros, of subnormal size, a negative and a zero logit factor."""
    lens = [150, 150, 150]
    cache, bt = make_cache(lens, 1, 128, bdfp8.E4M3, 18)
    q = queries(3, 1, G, 128, 19)
    q[0] = 0
    q[1] *= 2.0 ** -125
    for scale in (0.09, -0.09, 0.0, 1e30):
        if scale == 1e30:
            q[2] *= 2.0 ** -100
        check(decode(q, cache, bt, lens, 1, scale=scale), q, cache, bt, lens, scale=scale)


@pytest.mark.parametrize("G", [4, 8, 16])
@pytest.mark.parametrize("n", [64 * 3, 64 * 10, 64 * 13, 64 * 14 + 9])
def test_splits_that_merge_in_a_cluster(n, G):
    """Two to eight splits of a few sequences, some of them shorter."""
    lens = [n, n // 3, 0]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 26)
    q = queries(3, 1, 2 * G, 128, 27)
    for chunk in (1, 2):
        check(decode(q, cache, bt, lens, chunk), q, cache, bt, lens)


def test_more_splits_than_a_cluster_and_odd_plans():
    lens = [3000, 1, 640]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 28)
    for G, T in ((4, 1), (8, 1), (16, 1), (24, 1), (4, 7)):
        l2 = [max(n, T) for n in lens]
        q = queries(3, T, 2 * G, 128, 29)
        for chunk in (1, 5, 1000, 2 ** 31 - 1):
            check(decode(q, cache, bt, l2 if T == 1 else lens, chunk), q, cache, bt, l2 if T == 1 else lens)


@pytest.mark.parametrize("B, G, T, d, n", [(1, 1, 1, 128, 128 * 37), (2, 4, 1, 64, 128 * 17 + 1), (3, 7, 1, 128, 128 * 9), (45, 28, 1, 128, 300), (45, 28, 1, 64, 300), (41, 30, 1, 128, 128 * 9 - 3)])
def test_merges_by_a_block_and_by_a_warp_per_row(B, G, T, d, n):
    """More splits than a block has warps, fewer, uneven ones; rows below and above those that run at once."""
    lens = [n, n // 2, 1, 0, 129] * 9
    lens = lens[:B]
    cache, bt = make_cache(lens, 1, d, bdfp8.E4M3, 34)
    q = queries(B, T, G, d, 35)
    for chunk in (1, 2):
        got = decode(q, cache, bt, lens, chunk)
        check(got, q, cache, bt, lens)
        assert torch.equal(got, decode(q, cache, bt, lens, chunk))


def test_sequences_that_share_pages():
    """A common prefix: the same pages in two sequences' tables, and twice in one's."""
    lens = [300, 300, 200]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 30)
    bt[1, :3] = bt[0, :3]
    bt[2, 1] = bt[2, 0]
    q = queries(3, 2, 8, 128, 31)
    for chunk in (1, 2):
        check(decode(q, cache, bt, lens, chunk), q, cache, bt, lens)


@pytest.mark.parametrize("d_k, d_v, Hq, H", [(128, 128, 8, 2), (576, 512, 16, 1)])
def test_behind_an_fp4_decode_of_empty_sequences_in_the_same_workspace(d_k, d_v, Hq, H):
    """The FP4 decode's query images go to the workspace that the next call's partial sums take."""
    from fp4_kv_cache_quant_b200 import bdfp4
    lens, B4 = [700, 200], 64
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 36)
    q = queries(2, 1, 8, 128, 37)
    want = decode(q, cache, bt, lens, 1)
    check(want, q, cache, bt, lens)
    ones = lambda *s: torch.ones(s, dtype=torch.float32, device="cuda")  # noqa: E731
    c4, kv = bdfp4.FP4Cache.empty(4, H, d_k, d_v, bdfp4.NVFP4), bdfp4.KVParams(ones(H, d_k), ones(H), ones(H))
    q4 = torch.randn((B4, Hq, d_k), device="cuda").bfloat16()
    table4, none = torch.full((B4, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(B4, dtype=torch.int32, device="cuda")
    out4, out, qd, btd = torch.empty((B4, Hq, d_v), dtype=torch.bfloat16, device="cuda"), torch.empty_like(want), q.cuda(), torch.from_numpy(bt).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    size = max(bdfp4.bdfp4_decode_workspace_size(B4, Hq, d_v, 4, 1), bdfp8.workspace_for(2, 1, 8, 2, 128, bt.shape[1], 1).numel())
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for _ in range(20):
        out4.fill_(1.0)
        bdfp4.bdfp4_decode(q4, c4, table4, none, kv, 0.1, 1, ws, out4)
        bdfp8.bdfp8_decode(qd, cache, btd, sl, 1 / math.sqrt(128), 1, ws, out)
        assert torch.equal(out, want) and not out4.any()


def test_a_given_stream_and_misaligned_views():
    lens = [300]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 32)
    q = queries(1, 1, 8, 128, 33)
    want = decode(q, cache, bt, lens, 1)
    st, out = torch.cuda.Stream(), torch.empty_like(want)
    qd, btd = q.cuda(), torch.from_numpy(bt).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = bdfp8.workspace_for(1, 1, 8, 2, 128, bt.shape[1], 1)
    torch.cuda.synchronize()
    bdfp8.bdfp8_decode(qd, cache, btd, sl, 1 / math.sqrt(128), 1, ws, out, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    odd = torch.empty(8 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(1, 1, 8, 128)
    with pytest.raises(bdfp4.BDFP4Error, match="align"):
        bdfp8.bdfp8_decode(odd, cache, btd, sl, 0.1, 1, ws, out)
    with pytest.raises(bdfp4.BDFP4Error, match="workspace"):
        bdfp8.bdfp8_decode(qd, cache, btd, sl, 0.1, 1, None, out)


def test_offsets_beyond_32_bits():
    """Pages at the far end of a cache of more than 4 GB per array."""
    H, d, P = 8, 128, 70000
    lens = [130, 64]
    small, bt = make_cache(lens, H, d, bdfp8.E4M3, 20, extra_pages=0)
    n = small.num_pages
    big = bdfp8.FP8Cache(torch.empty((P, H, 64 * d), dtype=torch.uint8, device="cuda"),
                         torch.empty((P, H, 64 * d), dtype=torch.uint8, device="cuda"),
                         torch.empty((P, H, 2, 4), device="cuda"), P, H, d, bdfp8.E4M3)
    for name in ("k_pages", "v_pages", "kv_scales"):
        getattr(big, name)[P - n:] = getattr(small, name)
    q = queries(2, 1, 16, d, 21)
    far = np.where(bt >= 0, bt + P - n, bt)
    assert torch.equal(decode(q, big, far, lens, 1), decode(q, small, bt, lens, 1))
    # and an append that writes there
    o = bdfp8.OpenBlocks.empty(1, H, d)
    k = torch.randn((20, H, d), device="cuda").to(torch.bfloat16)
    args = lambda c, t: (k, k, torch.tensor([0, 20], dtype=torch.int32, device="cuda"),  # noqa: E731
                         torch.tensor([20], dtype=torch.int32, device="cuda"),
                         torch.tensor([[t]], dtype=torch.int32, device="cuda"), None, c, o)
    bdfp8.bdfp8_append(*args(big, P - 1))
    bdfp8.bdfp8_append(*args(small, n - 1))
    assert torch.equal(big.k_pages[P - 1], small.k_pages[n - 1]) and torch.equal(big.v_pages[P - 1], small.v_pages[n - 1])


# ------------------------------------------------------------------------------------------------ append
class Loop:
    """Sequences that grow: the cache under test beside the reference."""

    def __init__(self, B, H, Hq, d, fmt, rot, interleaved, mp=8, seed=0, canary=0xA5):
        self.B, self.H, self.Hq, self.d, self.fmt, self.interleaved = B, H, Hq, d, fmt, interleaved
        rng = np.random.default_rng(seed)
        self.g = torch.Generator().manual_seed(seed)
        P = B * mp + 2
        self.bt = rng.permutation(P)[: B * mp].reshape(B, mp).astype(np.int32)
        self.cache = bdfp8.FP8Cache.empty(P, H, d, fmt)
        self.cache.k_pages.fill_(canary)
        self.cache.v_pages.fill_(canary)
        self.cache.kv_scales.fill_(-7.0)
        self.canary = canary
        self.open = bdfp8.OpenBlocks.empty(B, H, d)
        self.open.k_open.fill_(float("nan"))
        self.open.v_open.fill_(float("nan"))
        self.lens = np.zeros(B, np.int64)
        self.ref = ref.AppendRef(B, H, d, fmt)
        if rot:
            ang = np.arange(mp * 64)[:, None] * 1e4 ** (-np.arange(0, rot, 2) / rot)[None]
            self.cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        else:
            self.cs = None

    def append(self, new, positions=None, tail=3, status=None):
        """new[b] tokens of each sequence, `tail` rows behind the last; returns the rotated queries."""
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(cu[-1]) + tail
        H, Hq, d = self.H, self.Hq, self.d
        qkv = torch.randn((T, (Hq + 2 * H) * d), generator=self.g).to(torch.bfloat16)
        x = qkv.cuda()
        cut = lambda t, a, b: t[:, a * d: b * d].unflatten(1, (b - a, d))  # noqa: E731
        self.lens += np.asarray(new)
        q_out = torch.full((T, Hq, d), 77.0, dtype=torch.bfloat16, device="cuda")
        bdfp8.bdfp8_append(cut(x, Hq, Hq + H), cut(x, Hq + H, Hq + 2 * H), torch.from_numpy(cu).cuda(),
                           torch.tensor(self.lens.tolist(), dtype=torch.int32, device="cuda"), torch.from_numpy(self.bt).cuda(),
                           None if self.cs is None else torch.from_numpy(self.cs).cuda(), self.cache, self.open,
                           q=cut(x, 0, Hq), q_out=q_out,
                           positions=None if positions is None else torch.from_numpy(positions).cuda(),
                           interleaved=self.interleaved, dev_status=status)
        xs = qkv.double().numpy()
        want = np.full((T, Hq, d), 77.0)
        for b in range(self.B):
            r = slice(cu[b], cu[b + 1])
            n0 = len(self.ref.k[b])
            pos = np.arange(n0, n0 + new[b]) if positions is None else positions[r]
            f = lambda a, e: xs[r, a * d: e * d].reshape(-1, e - a, d)  # noqa: E731
            self.ref.append(b, f(Hq, Hq + H), f(Hq + H, Hq + 2 * H), self.cs, pos, self.interleaved)
            want[r] = f(0, Hq) if self.cs is None else ref.rotate(f(0, Hq), self.cs[pos].astype(np.float64), self.interleaved)
        got = q_out.double().cpu().numpy()
        # fp32 products and sum (three roundings of 2^-24 of |a c| + |b s| <= 1.5 max), then half a bf16 step
        lim = 2.0 ** -8 * np.abs(want) + 4.5 * 2.0 ** -24 * np.abs(xs).max()
        lim[cu[-1]:] = 0
        assert np.all(np.abs(got - want) <= lim)
        return q_out, cu

    def check(self, skip=()):
        """Every block's bytes and scales; pages and blocks that hold no token are as they were."""
        K, V = ref.codes_of(self.cache)
        sc = self.cache.kv_scales.cpu().numpy()
        k_left, v_left, s_left = np.full(K.shape, self.canary, np.uint8), np.full(V.shape, self.canary, np.uint8), np.full(sc.shape, -7.0, np.float32)
        for b in range(self.B):
            for i, (kc, ks), (vc, vs) in self.ref.blocks(b):
                pg, s = self.bt[b, i // 4], i % 4
                if pg in skip or pg < 0:
                    continue
                k_left[pg, :, 16 * s: 16 * s + 16], v_left[pg, :, 16 * s: 16 * s + 16] = kc, vc
                s_left[pg, :, 0, s], s_left[pg, :, 1, s] = ks, vs
        assert np.array_equal(sc, s_left)
        assert np.array_equal(V, v_left)
        # keys: the reference's 64-bit rotation and the kernel's may round to neighbouring fp32 values, which
        # puts a value within 2^-24 of a border between codes on its other side: in a few of 2^20
        assert np.count_nonzero(K != k_left) <= 1 + K.size * 2.0 ** -17
        t = ref.code_values(self.fmt)
        differ = K != k_left
        if differ.any():
            a, e = t[K[differ]], t[k_left[differ]]
            assert np.all(np.abs(a - e) <= np.maximum(np.abs(e), 2.0 ** -6) * 2.0 ** (-3 if self.fmt == bdfp8.E4M3 else -2))


SHAPES = [(1, 1, 128, bdfp8.E4M3, 128, False), (2, 8, 128, bdfp8.E5M2, 64, True), (3, 3, 64, bdfp8.E4M3, 16, False),
          (2, 4, 64, bdfp8.E5M2, 64, True), (2, 2, 128, bdfp8.E4M3, 0, False), (1, 16, 128, bdfp8.E4M3, 48, False)]


@pytest.mark.parametrize("H, Hq, d, fmt, rot, inter", SHAPES)
def test_append_grows_block_by_block(H, Hq, d, fmt, rot, inter):
    lp = Loop(4, H, Hq, d, fmt, rot, inter)
    st = _status()
    # prompts of odd lengths, one none; then chunks that end a block, cross it, cross several, and single tokens
    for new in ([5, 0, 64, 100], [11, 1, 0, 28], [1, 40, 16, 1], [33, 7, 15, 0], [1, 1, 1, 1], [0, 0, 0, 3]):
        lp.append(new, status=st)
        lp.check()
    assert int(st) == 0


def test_bytes_do_not_depend_on_how_the_tokens_came():
    caches = []
    for cuts in ([150], [1] * 150, [7, 9, 16, 50, 68], [149, 1]):
        lp = Loop(1, 2, 2, 128, bdfp8.E4M3, 128, False, seed=4)
        g = torch.Generator().manual_seed(9)
        kv = torch.randn((2, 150, 2, 128), generator=g).to(torch.bfloat16).cuda()
        at = 0
        for n in cuts:
            bdfp8.bdfp8_append(kv[0, at: at + n], kv[1, at: at + n], torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                               torch.tensor([at + n], dtype=torch.int32, device="cuda"), torch.from_numpy(lp.bt).cuda(),
                               torch.from_numpy(lp.cs).cuda(), lp.cache, lp.open)
            at += n
        caches.append(lp.cache)
    for c in caches[1:]:
        for name in ("k_pages", "v_pages", "kv_scales"):
            assert torch.equal(getattr(c, name), getattr(caches[0], name))


@pytest.mark.parametrize("B", [1, 31, 32, 33, 130, 1100])
def test_append_finds_its_sequence_in_any_batch(B):
    lp = Loop(B, 1, 1, 64, bdfp8.E4M3, 64, False, mp=2, seed=B)
    r = np.random.default_rng(B)
    lp.append(r.integers(0, 40, B).tolist())
    lp.append(r.integers(0, 3, B).tolist())
    lp.append([1] * B)
    lp.check()


def test_rows_before_and_behind_the_sequences_are_left_alone():
    """cu_tokens need not begin at 0 nor end at T."""
    lp = Loop(2, 1, 1, 64, bdfp8.E4M3, 0, False, seed=15)
    k = torch.randn((50, 1, 64), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    qo = torch.full((50, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    bdfp8.bdfp8_append(k.cuda(), k.cuda(), torch.tensor([17, 37, 40], dtype=torch.int32, device="cuda"),
                       torch.tensor([20, 3], dtype=torch.int32, device="cuda"), torch.from_numpy(lp.bt).cuda(), None, lp.cache,
                       lp.open, q=k.cuda(), q_out=qo)
    kn = k.double().numpy()
    lp.ref.append(0, kn[17:37], kn[17:37])
    lp.ref.append(1, kn[37:40], kn[37:40])
    lp.check()
    assert torch.equal(qo[17:40].cpu(), k[17:40]) and bool((qo[:17] == 3).all()) and bool((qo[40:] == 3).all())


def test_given_positions_and_bad_ones():
    lp = Loop(2, 2, 4, 128, bdfp8.E4M3, 128, False, seed=6)
    pos = np.array([5, 5, 300, 0, 511, 17, 2, 0, 0, 0], np.int32)
    lp.append([3, 4], positions=pos)
    lp.check()
    st = _status()
    pos = np.array([512, -1, 7, 0, 0], np.int32)
    cs, lp2 = lp.cs, Loop(1, 1, 1, 128, bdfp8.E4M3, 128, False, seed=7)
    k = torch.randn((3, 1, 128), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    bdfp8.bdfp8_append(k.cuda(), k.cuda(), torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                       torch.tensor([3], dtype=torch.int32, device="cuda"), torch.from_numpy(lp2.bt).cuda(),
                       torch.from_numpy(cs).cuda(), lp2.cache, lp2.open, positions=torch.from_numpy(pos[:3].copy()).cuda(),
                       dev_status=st)
    assert int(st) == bdfp8.DEV_BAD_POSITION
    kn = k.double().numpy()
    lp2.ref.append(0, kn[:2], kn[:2])
    lp2.ref.append(0, kn[2:], kn[2:], cs, pos[2:3])
    lp2.check()


def test_append_reports_bad_pages_and_lengths():
    lp = Loop(3, 1, 2, 128, bdfp8.E4M3, 0, False, seed=8)
    lp.bt[1, 1] = -1
    st = _status()
    lp.append([70, 100, 5], status=st)
    assert int(st) == bdfp4.DEV_BAD_PAGE
    lp.check()
    lp.append([1, 40, 1])            # page 1 of sequence 1 ends at 128: what follows is written
    lp.check()
    # a sequence shorter than its new tokens, one longer than its table: skipped, the others not
    lp = Loop(3, 1, 2, 128, bdfp8.E4M3, 0, False, seed=9)
    k = torch.randn((30, 1, 128)).to(torch.bfloat16).cuda()
    q = torch.randn((30, 2, 128)).to(torch.bfloat16).cuda()
    st, qo = _status(), torch.full((30, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    bdfp8.bdfp8_append(k, k, torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda"),
                       torch.tensor([9, 10, 513], dtype=torch.int32, device="cuda"), torch.from_numpy(lp.bt).cuda(), None,
                       lp.cache, lp.open, q=q, q_out=qo, dev_status=st)
    kn = k.double().cpu().numpy()
    lp.ref.append(1, kn[10:20], kn[10:20])
    lp.check()
    assert int(st) == bdfp4.DEV_BAD_SEQLEN
    assert torch.equal(qo[10:20], q[10:20]) and bool((qo[:10] == 5).all()) and bool((qo[20:] == 5).all())


def test_blocks_of_zeros_and_of_what_is_not_a_number():
    lp = Loop(1, 2, 2, 128, bdfp8.E4M3, 0, False, seed=10)
    k = torch.zeros((48, 2, 128), dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    k[20, 0, 3], v[33, 1, 5], k[40, 1, 1] = float("nan"), float("inf"), 2.0 ** -133
    bdfp8.bdfp8_append(k.cuda(), v.cuda(), torch.tensor([0, 48], dtype=torch.int32, device="cuda"),
                       torch.tensor([48], dtype=torch.int32, device="cuda"), torch.from_numpy(lp.bt).cuda(), None, lp.cache,
                       lp.open)
    sc = lp.cache.kv_scales[int(lp.bt[0, 0])].cpu()
    want = torch.ones(2, 2, 4)
    want[:, :, 3] = -7.0
    want[0, 0, 1] = want[1, 1, 2] = float("nan")
    want[1, 0, 2] = 2.0 ** -126
    assert torch.equal(torch.nan_to_num(sc, 99.0), torch.nan_to_num(want, 99.0))


# ------------------------------------------------------------------------------------------------ together
def _loop_check(lp, q, lens, window=0, sinks=0, chunk=1):
    out = decode(q.cpu().view(lp.B, -1, lp.Hq, lp.d), lp.cache, lp.bt, lens, chunk, window, sinks)
    check(out, q.cpu().view(lp.B, -1, lp.Hq, lp.d), lp.cache, lp.bt, lens, window, sinks)


@pytest.mark.parametrize("window, sinks", [(0, 0), (50, 4)])
def test_prompt_then_generation(window, sinks):
    """A prompt, then tokens one at a time and drafted ones four at a time, attending after each."""
    lp = Loop(3, 2, 8, 128, bdfp8.E4M3, 128, False, seed=12)
    lp.append([100, 30, 64], tail=0)
    for step in range(6):
        n = 4 if step % 3 == 2 else 1
        q, _ = lp.append([n] * 3, tail=0)
        lp.check()
        _loop_check(lp, q, lp.lens, window, sinks)


def test_a_prompt_in_chunks_that_attend_as_they_arrive():
    """Chunks of 70 tokens appended and attending causally, to everything and through a window."""
    lp = Loop(2, 2, 8, 128, bdfp8.E4M3, 128, False, seed=14)
    for step in range(3):
        q, _ = lp.append([70, 70], tail=0)
        lp.check()
        _loop_check(lp, q, lp.lens, 0, 0, 2)
        _loop_check(lp, q, lp.lens, 33, 3, 1)


def test_a_captured_step_replays_and_streams_do_not_meet():
    """Append and decode captured into a graph, replayed over growing lengths beside an eager call on
    another stream with a workspace of its own."""
    lp, twin = (Loop(2, 2, 8, 128, bdfp8.E4M3, 128, False, seed=13) for _ in range(2))
    for x in (lp, twin):
        x.append([37, 120], tail=0)
    dev = dict(device="cuda")
    bt, cs = torch.from_numpy(lp.bt).cuda(), torch.from_numpy(lp.cs).cuda()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, **dev)
    qkv = torch.zeros((2, 12, 128), dtype=torch.bfloat16, **dev)
    lens = torch.zeros(2, dtype=torch.int32, **dev)
    st = _status()
    outs = [torch.empty((2, 1, 8, 128), dtype=torch.bfloat16, **dev) for _ in range(2)]
    wss = [bdfp8.workspace_for(2, 1, 8, 2, 128, bt.shape[1], 1) for _ in range(2)]

    def step(x, i, q_out):
        bdfp8.bdfp8_append(qkv[:, 8:10], qkv[:, 10:], cu, lens, bt, cs, x.cache, x.open, q=qkv[:, :8], q_out=q_out, dev_status=st)
        bdfp8.bdfp8_decode(q_out.view(2, 1, 8, 128), x.cache, bt, lens, 0.09, 1, wss[i], outs[i], dev_status=st)

    qo = [torch.empty((2, 8, 128), dtype=torch.bfloat16, **dev) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    lens.copy_(torch.tensor([38, 121]))   # captured, not run
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(lp, 0, qo[0])
    g = torch.Generator().manual_seed(5)
    for s in range(5):
        qkv.copy_(torch.randn((2, 12, 128), generator=g))
        lens.copy_(torch.tensor([38 + s, 121 + s]))
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        graph.replay()
        with torch.cuda.stream(other):
            step(twin, 1, qo[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and int(st) == 0
        K, V = ref.values_of(lp.cache)
        q = qo[0].view(2, 1, 8, 128).double().cpu().numpy()
        want, tol = ref.attention(q, K, V, lp.bt, [38 + s, 121 + s], 0.09)
        assert np.all(np.abs(outs[0].double().cpu().numpy() - want) <= tol)
    for name in ("k_pages", "v_pages", "kv_scales"):
        assert torch.equal(getattr(lp.cache, name), getattr(twin.cache, name))


def test_the_same_call_gives_the_same_bits():
    lens = [3000, 777]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 22)
    q = queries(2, 2, 16, 128, 23)
    a = decode(q, cache, bt, lens, 3)
    for _ in range(3):
        assert torch.equal(decode(q, cache, bt, lens, 3), a)
