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
