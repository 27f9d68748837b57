"""Attention to another sequence's keys where items are cut and their parts joined by a kernel of its own, and
where a wait inside a kernel runs out.  Tolerances: those of test_gpu_cross."""
import pytest
import torch

import exact_io_aware_06_gb300 as fa
from gpu_util import check_status, ensure_built, scale_for
from test_gpu_cross import check_forward, forward, inputs, on_device, sizes, space
from test_gpu_window import until_a_wait_runs_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def cut_items(ws):
    """Items that the call before has cut: the workspace begins with 152 places of four ints, the first -1 where nothing
    is cut; space() leaves it so, and calls that join none do not write there."""
    return int((ws[: 152 * 16].view(torch.int32).view(152, 4)[:, 0] >= 0).sum())


@pytest.mark.parametrize("B,H,H_kv,N_q,N_kv,d,lengths", [(16, 64, 8, 1, 16384, 128, [16384] * 12 + [5] * 4),
                                                         (140, 1, 1, 200, 16384, 64, [0] * 100 + [16384] * 40)])
def test_a_wait_that_runs_out_where_items_are_cut(B, H, H_kv, N_q, N_kv, d, lengths):
    # CTAs with more segments than the ring holds: the wait for room in it is one of those that run out, and the join
    # goes by the table all the same
    q, k, v, _ = inputs(B, B, H, H_kv, N_q, N_kv, d, seed=B)
    ws = space(fa.fa_fwd_cross_workspace_size(*sizes(q, k)))
    ref = forward(q, k, v, lengths, scale_for(d), ws)
    assert cut_items(ws) > 4
    check_forward(q, k, v, lengths, *ref, scale_for(d), batches=[0, 11, B - 1])
    n, out = on_device(lengths), [torch.empty_like(t) for t in ref]
    for _ in range(3):
        ws.fill_(255)
        until_a_wait_runs_out(lambda: fa.fa_fwd_cross(q, k, v, n, *out, ws, scale_for(d)), out, ref)
