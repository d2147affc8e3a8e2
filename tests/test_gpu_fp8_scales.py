"""GPU tests of value scales that differ by many orders of magnitude, against the 64-bit reference of
_fp8_ref.py: what one row sees must not cost another row, or a block without weight a block with it, any bits."""
import math

import numpy as np
import pytest
import torch

import _fp8_ref as ref
from fp4_kv_cache_quant_b200 import bdfp8
from test_gpu_fp8 import _status, decode, make_cache, queries

pytestmark = pytest.mark.gpu


def check(out, q, cache, bt, lens, window=0, sinks=0):
    """Against the definition in 64 bits.  With a value block's scale c = 2^e r (1/2 < r <= 1), A = sum_t p_t |v_t|, D = max_t
    sum_i |q_i k_ti| / sqrt(d), X and E the largest |logit| (log2 units) and |e| that a row sees, a result may be off by
    half a bf16 step, 2^-8 |out|, and by A times
      2^-9 + 2^-11                    a probability's three E5M2 terms and its fp16 form
      2 (d + 8) 2^-23 D               the logits' fp32 sums (a whole step per addition), in p and in the sum of p
      2 2^-17 max|q| max_t sum_i |k_ti| / sqrt(d)   what a query's two terms leave of it, the same
      (n + 64) 2^-23                  the fp32 sums over n tokens
      4 ln 2 2^-24 (3 (X + E) + 44)   exponents x + e: three roundings (the sum, the reference, their difference), and of the
                                      22 that they are lifted by; in p and in the sum of p
      2^-19                           exponentials (2 units of 2^-22 each, twice where references meet) and the last product
    and by n 2^-28 max_t p_t 2^e max_t |code|: the terms' floor.  Blocks whose seen values are all zero have no part in it."""
    K, V = ref.values_of(cache)
    x, d, H = q.double().numpy(), q.shape[3], cache.H_kv
    G, T = q.shape[2] // H, q.shape[1]
    c = np.repeat(cache.kv_scales[:, :, 1].double().cpu().numpy(), 16, axis=2)   # [pages, H, 64]
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    for b, N in enumerate(lens):
        for i in range(T):
            p = N - T + i
            t = np.arange(p + 1)
            t = t[(t > p - window) | (t < sinks)] if window else t
            pg, slot, n = bt[b, t // 64], t % 64, len(t)
            for h in range(H):
                k, v, ct = K[pg, h, slot], V[pg, h, slot], c[pg, h, slot]
                qh = x[b, i, h * G: (h + 1) * G]
                lg = qh @ k.T / math.sqrt(d)
                e = np.exp(lg - lg.max(1, keepdims=True))
                e /= e.sum(1, keepdims=True)
                want, A = e @ v, e @ np.abs(v)
                D = (np.abs(qh) @ np.abs(k).T).max(1) / math.sqrt(d)
                left = np.abs(qh).max(1) * np.abs(k).sum(1).max() / math.sqrt(d)
                e2 = np.ceil(np.log2(np.maximum(ct, 2.0 ** -140)))
                far = 3 * (np.abs(lg).max(1) / math.log(2) + np.abs(e2).max()) + 44
                rel = (2.0 ** -9 + 2.0 ** -11 + 2 * (d + 8) * 2.0 ** -23 * D + 2.0 ** -16 * left + (n + 64) * 2.0 ** -23 +
                       4 * math.log(2) * 2.0 ** -24 * far + 2.0 ** -19)
                used = np.isin(t // 16, np.unique(t[v.any(1)] // 16))
                floor = n * 2.0 ** -28 * (e * np.where(used, 2.0 ** e2, 0)).max(1) * np.abs(v / np.maximum(ct, 2.0 ** -140)[:, None]).max()
                lim = 2.0 ** -8 * np.abs(want) + A * rel[:, None] + floor[:, None]
                off = np.abs(got[b, i, h * G: (h + 1) * G] - want) - lim
                assert np.all(off <= 0), (b, i, h, float((off / np.maximum(A, 1e-300)).max()))
    return got


FORMS = [(128, bdfp8.E4M3), (128, bdfp8.E5M2), (64, bdfp8.E4M3), (64, bdfp8.E5M2)]


@pytest.mark.parametrize("d, fmt", FORMS)
@pytest.mark.parametrize("G", [1, 2, 5, 9, 40])
@pytest.mark.parametrize("factor", [2.0 ** 20, 2.0 ** 40])
def test_a_large_block_that_only_the_newest_query_sees(factor, G, d, fmt):
    """The rows of the earlier query tokens keep their values' bits beside it in the same tile."""
    lens = [193, 65]   # the last token of each begins a block
    cache, bt = make_cache(lens, 2, d, fmt, 60)
    for b, n in enumerate(lens):
        cache.kv_scales[int(bt[b, n // 64]), :, 1, 0] *= factor
    q = queries(2, 3, 2 * G, d, 61)
    st = _status()
    for chunk in (1, 2):
        check(decode(q, cache, bt, lens, chunk, status=st), q, cache, bt, lens)
    assert int(st) == 0


@pytest.mark.parametrize("d, fmt", FORMS)
@pytest.mark.parametrize("T, G", [(2, 2), (3, 2), (9, 1), (9, 8)])
def test_a_large_block_that_only_the_oldest_window_reaches(T, G, d, fmt):
    """Its last token is the first of the oldest query token's window; the first tokens' block is small."""
    n, sinks, first = 300, 4, 175
    window = n - T - first + 1
    cache, bt = make_cache([n], 2, d, fmt, 62, window, sinks, T)
    cache.kv_scales[int(bt[0, first // 64]), :, 1, first % 64 // 16] *= 2.0 ** 30
    cache.kv_scales[int(bt[0, 0]), :, 1, 0] *= 2.0 ** -30
    q = queries(1, T, 2 * G, d, 63)
    for chunk in (1, 2):
        check(decode(q, cache, bt, [n], chunk, window, sinks), q, cache, bt, [n], window, sinks)


@pytest.mark.parametrize("G", [4, 8, 16, 24])
def test_a_large_block_without_weight(G):
    """A block of large values whose keys point away from every query: p c is small, so it costs the others nothing."""
    n, d = 400, 128
    cache, bt = make_cache([n], 1, d, bdfp8.E4M3, 64)
    q = queries(1, 1, G, d, 65)
    q[..., 0] = 20.0
    ko, _ = ref.offsets(d)
    pg = int(bt[0, 2])
    row = cache.k_pages[pg, 0].cpu().numpy()
    row[ko[16:32, 0]] = 0xE8        # E4M3 -32: a logit of about -57 for element 0 alone
    row[ko[16:32, 1:]] = 0
    cache.k_pages[pg, 0] = torch.from_numpy(row).cuda()
    cache.kv_scales[pg, 0, :, 1] = torch.tensor([1.0, 2.0 ** 40])
    for chunk in (1, 4):
        check(decode(q, cache, bt, [n], chunk), q, cache, bt, [n])


@pytest.mark.parametrize("T, G", [(1, 4), (3, 2), (1, 16), (1, 24), (3, 16)])
@pytest.mark.parametrize("where", ["all", "newest", "one"])
def test_the_largest_scales(where, T, G):
    """Up to 1.5 2^126: in every block, in the newest token's, in one that all rows see."""
    lens = [193, 65]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 66)
    top = 1.5 * 2.0 ** 126
    if where == "all":
        cache.kv_scales[:, :, 1] *= 2.0 ** 125 * 1.5
    else:
        for b, n in enumerate(lens):
            cache.kv_scales[int(bt[b, n // 64 if where == "newest" else 0]), :, 1, 0] = top
    assert float(cache.kv_scales[:, :, 1].nan_to_num(0).max()) <= 2.0 ** 127
    q = queries(2, T, 2 * G, 128, 67)
    for chunk in (1, 2):
        check(decode(q, cache, bt, lens, chunk), q, cache, bt, lens)


@pytest.mark.parametrize("G", [4, 8, 16, 24])
@pytest.mark.parametrize("low", [2.0 ** -60, 2.0 ** -91])
def test_the_smallest_scales(low, G):
    lens = [300, 17]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 68)
    cache.kv_scales[:, :, 1] *= low
    q = queries(2, 1, 2 * G, 128, 69)
    for chunk in (1, 3):
        check(decode(q, cache, bt, lens, chunk), q, cache, bt, lens)


# ------------------------------------------------------------------------------------------------ blocks of zeros
def appended(lens, H, d, fmt, std, zeros, toward, seed):
    """A cache written by bdfp8_append, values N(0, std) but zeros (of both signs) in the token ranges zeros[b], whose keys lie
    along element 0 when `toward`; whatever no append wrote holds NaN codes and scales."""
    g = torch.Generator().manual_seed(seed)
    mp = max((n + 63) // 64 for n in lens)
    P = len(lens) * mp + 1
    bt = torch.randperm(P, generator=g)[: len(lens) * mp].view(len(lens), mp).int()
    cache = bdfp8.FP8Cache.empty(P, H, d, fmt)
    cache.k_pages.fill_(0x7F)
    cache.v_pages.fill_(0x7F)
    cache.kv_scales.fill_(float("nan"))
    ks, vs = [], []
    for n, zs in zip(lens, zeros):
        k, v = torch.randn((n, H, d), generator=g), torch.randn((n, H, d), generator=g) * std
        for a, e in zs:
            v[a:e] *= 0.0
            if toward:
                k[a:e] = 0.0
                k[a:e, :, 0] = 8.0
        ks.append(k)
        vs.append(v)
    cu = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).int().cuda()
    bdfp8.bdfp8_append(torch.cat(ks).bfloat16().cuda(), torch.cat(vs).bfloat16().cuda(), cu,
                       torch.tensor(lens, dtype=torch.int32).cuda(), bt.cuda(), None, cache, bdfp8.OpenBlocks.empty(len(lens), H, d))
    return cache, bt.numpy()


@pytest.mark.parametrize("toward", [False, True])
@pytest.mark.parametrize("std", [0.1, 0.01, 0.001])
@pytest.mark.parametrize("d, fmt", FORMS)
@pytest.mark.parametrize("T, G", [(1, 4), (1, 8), (1, 16), (1, 24), (3, 2), (3, 40)])
def test_a_block_of_zero_values_among_small_ones(T, G, d, fmt, std, toward):
    """A whole block of zeros, with and without most of the weight, and an open one."""
    lens = [700, 146]
    cache, bt = appended(lens, 2, d, fmt, std, [[(48, 64), (300, 310)], [(0, 16), (144, 146)]], toward, 70)
    assert float(cache.kv_scales[int(bt[0, 0]), 0, 1, 3]) == 1.0
    q = queries(2, T, 2 * G, d, 71)
    if toward:
        q[..., 0] = q[..., 0].abs() + 4.0
    for chunk in (1, 6):
        check(decode(q, cache, bt, lens, chunk), q, cache, bt, lens)


@pytest.mark.parametrize("G", [4, 8, 16, 24])
def test_zeros_in_every_seen_slot(G):
    """Junk behind the sequence's end, and a block whose other tokens are behind the window."""
    lens, window = [133, 133], 101    # the window begins at token 32; the last block holds tokens 128 .. 132
    cache, bt = make_cache(lens, 2, 128, bdfp8.E5M2, 72, window)
    cache.kv_scales[:, :, 1] *= 2.0 ** -20
    _, vo = ref.offsets(128)
    pages = cache.v_pages.cpu().numpy()
    for pg, slots, blk in ((bt[0, 2], slice(0, 5), 0), (bt[1, 0], slice(33, 48), 2)):
        for h in range(2):
            pages[pg, h][vo[slots]] = 0x80
        cache.kv_scales[int(pg), :, 1, blk] = 1.0
    for h in range(2):
        pages[bt[1, 0], h][vo[32]] = 0
    cache.v_pages.copy_(torch.from_numpy(pages))
    q = queries(2, 1, 2 * G, 128, 73)
    for chunk in (1, 2):
        check(decode(q, cache, bt, lens, chunk, window), q, cache, bt, lens, window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [4, 8, 16, 24])
@pytest.mark.parametrize("slot, chan", [(0, 0), (15, -1), (7, 8), (8, 31), (31, 5)])
def test_one_value_makes_a_block_of_scale_one_count(slot, chan, G, d):
    cache, bt = make_cache([200], 1, d, bdfp8.E4M3, 74)
    cache.kv_scales[:, :, 1] *= 2.0 ** -20
    _, vo = ref.offsets(d)
    pages = cache.v_pages.cpu().numpy()
    for page, base in ((0, 0), (1, 32)):
        pages[bt[0, page], 0][vo[base: base + 32]] = 0
        pages[bt[0, page], 0][vo[base + slot, chan]] = 0xC0   # -2
        cache.kv_scales[int(bt[0, page]), 0, 1, base // 16: base // 16 + 2] = 1.0
    cache.v_pages.copy_(torch.from_numpy(pages))
    q = queries(1, 1, G, d, 75)
    for chunk in (1, 2):
        check(decode(q, cache, bt, [200], chunk), q, cache, bt, [200])


@pytest.mark.parametrize("G", [4, 24])
def test_nothing_but_zeros(G):
    cache, bt = appended([300], 1, 128, bdfp8.E4M3, 1.0, [[(0, 300)]], False, 76)
    got = decode(queries(1, 2, G, 128, 77), cache, bt, [300], 1)
    assert not got.any()


@pytest.mark.parametrize("zero", [0.0, -0.0])
@pytest.mark.parametrize("d, fmt", FORMS)
@pytest.mark.parametrize("T, G", [(1, 4), (1, 16), (3, 2), (1, 24), (3, 40)])
def test_scales_of_zero(T, G, d, fmt, zero):
    """Blocks whose value scale is a zero of either sign give nothing and cost nothing."""
    lens = [300, 40]
    cache, bt = make_cache(lens, 2, d, fmt, 78)
    cache.kv_scales[:, :, 1] *= 2.0 ** -20
    for b, page, blk in ((0, 0, 1), (0, 4, 0), (1, 0, 2)):
        cache.kv_scales[int(bt[b, page]), :, 1, blk] = zero
    q = queries(2, T, 2 * G, d, 79)
    for chunk in (1, 2):
        check(decode(q, cache, bt, lens, chunk), q, cache, bt, lens)
