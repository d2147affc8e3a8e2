"""GPU tests of bdfp8_append beside those of test_gpu_fp8.py: streams, tokens without a position, sequences out of order."""
import numpy as np
import pytest
import torch

import _fp8_ref as ref
from fp4_kv_cache_quant_b200 import bdfp4, bdfp8
from test_gpu_fp8 import Loop, _status

pytestmark = pytest.mark.gpu


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("given", [False, True])
def test_append_on_a_given_stream(given):
    """The same bytes as on the current stream, and rotated queries from the pool of the stream that writes them."""
    cur, side = (Loop(2, 2, 8, 128, bdfp8.E4M3, 128, False, seed=80) for _ in range(2))
    g = torch.Generator().manual_seed(81)
    k, v, q = (torch.randn((50, h, 128), generator=g).bfloat16().cuda() for h in (2, 2, 8))
    bt, cs = torch.from_numpy(cur.bt).cuda(), torch.from_numpy(cur.cs).cuda()
    cu, sl = _i32(0, 20, 50), _i32(20, 30)
    st = torch.cuda.Stream()

    def run(lp, **kw):
        return bdfp8.bdfp8_append(k, v, cu, sl, bt, cs, lp.cache, lp.open, q=q, **kw)
    want = run(cur)
    torch.cuda.synchronize()
    out = torch.empty_like(q) if given else None
    got = run(side, stream=st, q_out=out)
    st.synchronize()
    assert torch.equal(got, want) and (got is out) == given
    for name in ("k_pages", "v_pages", "kv_scales"):
        assert torch.equal(getattr(side.cache, name), getattr(cur.cache, name))
    if not given:
        at = [s for s in torch.cuda.memory_snapshot() if s["address"] <= got.data_ptr() < s["address"] + s["total_size"]]
        assert len(at) == 1 and at[0]["stream"] == st.cuda_stream


@pytest.mark.parametrize("interleaved", [False, True])
def test_tokens_of_a_bad_position_stay_as_they_are(interleaved):
    """Unrotated to the bit: infinities do not reach the elements they would be paired with, zeros keep their signs."""
    lp = Loop(1, 1, 2, 64, bdfp8.E4M3, 64, interleaved, seed=82)
    g = torch.Generator().manual_seed(83)
    k, v, q = (torch.randn((40, h, 64), generator=g).bfloat16() for h in (1, 1, 2))
    q[3, 0, 1], q[3, 1, 40], q[5, 0, 0] = float("inf"), float("-inf"), float("nan")
    q[4, :, ::3], k[4, :, ::3], k[20, :, 1::2] = -0.0, -0.0, -0.0
    pos = torch.arange(40, dtype=torch.int32)
    bad = [3, 4, 5, 20, 39]
    pos[bad] = torch.tensor([-1, 512, 2 ** 31 - 1, -2 ** 31, 513], dtype=torch.int32)
    st = _status()
    got = bdfp8.bdfp8_append(k.cuda(), v.cuda(), _i32(0, 40), _i32(40), torch.from_numpy(lp.bt).cuda(),
                             torch.from_numpy(lp.cs).cuda(), lp.cache, lp.open, q=q.cuda(), positions=pos.cuda(),
                             interleaved=interleaved, dev_status=st)
    assert int(st) == bdfp8.DEV_BAD_POSITION
    same = lambda a, b: torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))  # noqa: E731
    num = torch.tensor([i for i in range(64) if i != 0])
    for t in bad:
        assert same(got[t].cpu()[:, num], q[t][:, num])   # (a NaN's payload may change)
    assert torch.isnan(got[5, 0, 0])
    codes = ref.codes_of(lp.cache)[0][lp.bt[0, 0], 0]     # [64, 64]
    for t in (4, 20):
        zero = (k[t, 0] == 0).numpy()
        assert zero.any() and np.all(codes[t][zero] == 0x80)
    good = [t for t in range(40) if t not in bad]
    want = ref.rotate(q[good].double().numpy(), lp.cs[good].astype(np.float64), interleaved)
    assert np.all(np.abs(got[good].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 4.5 * 2.0 ** -24 * 6)


@pytest.mark.parametrize("B, swaps", [(4, [1]), (40, [3, 20, 39]), (200, [1, 100, 150, 199])])
def test_sequences_out_of_order_are_reported_and_nothing_else_is_written(B, swaps):
    """cu_tokens that falls: a block of any sequence is written as it should be, or not at all."""
    r = np.random.default_rng(B)
    new = r.integers(1, 60, B)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    for i in swaps:
        cu[i] = r.integers(0, T + 40) if i % 2 else -5
    lp = Loop(B, 1, 1, 64, bdfp8.E4M3, 0, False, mp=64, seed=84)
    lens = np.array([max(cu[b + 1] - cu[b], 1) for b in range(B)], np.int32)
    k = torch.randn((T, 1, 64), generator=torch.Generator().manual_seed(85)).bfloat16()
    st = _status()
    bdfp8.bdfp8_append(k.cuda(), k.cuda(), torch.from_numpy(cu).cuda(), torch.from_numpy(lens).cuda(), torch.from_numpy(lp.bt).cuda(),
                       None, lp.cache, lp.open, dev_status=st)
    assert int(st) == bdfp4.DEV_BAD_SEQLEN
    kn = k.double().numpy()
    K, V = ref.codes_of(lp.cache)
    sc = lp.cache.kv_scales.cpu().numpy()
    touched = np.zeros(sc.shape, bool)
    written = 0
    for b in range(B):
        if 0 <= cu[b] <= cu[b + 1] <= T and lens[b] <= 64 * lp.bt.shape[1]:   # (a longer one is skipped, too)
            lp.ref.append(b, kn[cu[b]: cu[b + 1]], kn[cu[b]: cu[b + 1]])
        for i, (kc, ks), (vc, vs) in lp.ref.blocks(b):
            pg, s = lp.bt[b, i // 4], i % 4
            if sc[pg, 0, 0, s] == -7.0:
                continue
            written += 1
            touched[pg, :, :, s] = True
            at = slice(16 * s, 16 * s + 16)
            assert np.array_equal(K[pg, :, at], kc) and np.array_equal(V[pg, :, at], vc)
            assert np.array_equal(sc[pg, :, 0, s], ks) and np.array_equal(sc[pg, :, 1, s], vs)
    assert written and np.all(sc[~touched] == -7.0)
    left = np.repeat(~touched[:, :, 0], 16, axis=2)
    assert np.all(K[left] == lp.canary) and np.all(V[left] == lp.canary)
