"""The bounded in-kernel waits of the 8-bit cache's decode kernels, through the hook of
include/bdfp8_debug.h: in every block the first key tile is never announced, or one softmax warp gives
up on a tile that its neighbours see arrive.  Blocks must unwind, their warps together, report
BDFP4_DEV_TIMEOUT and leave the device usable: the next normal decode gives what it gave before.  No
fault is raised; the failure is a wait that nothing completes."""
import math

import pytest
import torch

from fp4_kv_cache_quant_b200 import bdfp4, bdfp8
from test_gpu_fp8 import check, decode, make_cache, queries

pytestmark = pytest.mark.gpu

SHORT_WAIT = 1 << 21   # clock cycles, about a millisecond


# 8 rows; 24, 48 and 140 rows of the wide kernel: one, two and four quadrants of rows, a second row group
@pytest.mark.parametrize("T, G", [(1, 8), (1, 24), (3, 16), (5, 28)])
@pytest.mark.parametrize("chunk", [1, 8])
def test_a_wait_that_runs_out_unwinds_and_reports(T, G, chunk):
    lens = [1000, 77, 129, 513]
    cache, bt = make_cache(lens, 2, 128, bdfp8.E4M3, 50)
    q = queries(len(lens), T, 2 * G, 128, 51)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = decode(q, cache, bt, lens, chunk, status=st)
    check(before, q, cache, bt, lens)
    assert int(st) == 0
    ws = bdfp8.workspace_for(len(lens), T, 2 * G, 2, 128, bt.shape[1], chunk)
    qd, btd, sl = q.cuda(), torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    for stall in (bdfp8.STALL_NONE, bdfp8.STALL_TILE, bdfp8.STALL_WARP):
        out = torch.empty_like(before)
        st.zero_()
        bdfp8.bdfp8_debug_decode_wait_test(qd, cache, btd, sl, 1 / math.sqrt(128), chunk, ws, out, SHORT_WAIT, stall,
                                           dev_status=st)
        torch.cuda.synchronize()
        if stall == bdfp8.STALL_NONE:   # the short bound alone changes nothing
            assert int(st) == 0 and torch.equal(out, before)
        else:
            assert int(st) == bdfp4.DEV_TIMEOUT
        st.zero_()
        assert torch.equal(decode(q, cache, bt, lens, chunk, status=st), before) and int(st) == 0


@pytest.mark.parametrize("T, G, d, fmt", [(1, 4, 128, bdfp8.E4M3), (2, 4, 128, bdfp8.E4M3), (1, 16, 128, bdfp8.E4M3),
                                          (1, 8, 64, bdfp8.E4M3), (1, 8, 128, bdfp8.E5M2), (1, 24, 64, bdfp8.E5M2)])
def test_the_hook_refuses_other_shapes(T, G, d, fmt):
    cache, bt = make_cache([64], 1, d, fmt, 52)
    q = queries(1, T, G, d, 53).cuda()
    sl = torch.tensor([64], dtype=torch.int32, device="cuda")
    with pytest.raises(bdfp4.BDFP4Error, match="compiled set"):
        bdfp8.bdfp8_debug_decode_wait_test(q, cache, torch.from_numpy(bt).cuda(), sl, 0.1, 1, None, torch.empty_like(q), SHORT_WAIT,
                                           bdfp8.STALL_TILE)
