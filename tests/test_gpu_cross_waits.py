"""Waits that run out inside the kernels of cross attention: reported, and the calls that report nothing and those under
the default limit right.  (Where items are cut and joined: test_gpu_cross_joins.)"""
import pytest
import torch

import exact_io_aware_06_gb300 as fa
from gpu_util import check_status, ensure_built, scale_for
from test_gpu_cross import backward, check_backward, check_forward, forward, inputs, on_device, sizes, space
from test_gpu_window import until_a_wait_runs_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


# whole items, pairs of tiles; whole items of many short sequences, packed; a cluster of eight CTAs an item, whose
# CTAs all have to reach its barrier
@pytest.mark.parametrize("B,B_kv,H,N_q,N_kv,lengths", [(4, 4, 16, 2048, 700, None), (4, 4, 16, 2048, 700, [700, 1, 0, 300]),
                                                       (80, 40, 16, 33, 120, list(range(0, 120, 3))), (1, 1, 15, 130, 1100, [1001])])
@pytest.mark.parametrize("d", [64, 128])
def test_forward(B, B_kv, H, N_q, N_kv, lengths, d):
    q, k, v, _ = inputs(B, B_kv, H, H, N_q, N_kv, d, seed=13)
    ws = space(fa.fa_fwd_cross_workspace_size(*sizes(q, k)))
    ref = forward(q, k, v, lengths, scale_for(d), ws)
    check_forward(q, k, v, lengths, *ref, scale_for(d), batches=[B - 1])
    n, out = on_device(lengths), [torch.empty_like(t) for t in ref]
    until_a_wait_runs_out(lambda: fa.fa_fwd_cross(q, k, v, n, *out, ws, scale_for(d)), out, ref)


def step(B, H, N_q, N_kv, lengths, d):
    q, k, v, do = inputs(B, B, H, H, N_q, N_kv, d, seed=13)
    o, lse = forward(q, k, v, lengths, scale_for(d))
    ws = space(fa.fa_bwd_cross_workspace_size(*sizes(q, k)))
    ref = backward(q, k, v, lengths, o, lse, do, scale_for(d), ws)
    two = [t[:, :2].contiguous() for t in (q, k, v, do)]
    check_backward(*two[:3], lengths, two[3], [g[:, :2] for g in ref], scale_for(d), kv_batches=[0])
    n, out = on_device(lengths), [torch.empty_like(t) for t in ref]
    return lambda: fa.fa_bwd_cross(q, k, v, n, o, lse, do, *out, ws, scale_for(d)), out, ref


# many items a CTA; up to two items of dQ an SM, which run beside dK and dV, and last long
@pytest.mark.parametrize("B,H,N_q,N_kv,lengths", [(2, 8, 1024, 700, None), (4, 16, 500, 600, [600, 0, 77, 400]), (1, 100, 300, 4000, [3999])])
@pytest.mark.parametrize("d", [64, 128])
def test_backward(B, H, N_q, N_kv, lengths, d):
    until_a_wait_runs_out(*step(B, H, N_q, N_kv, lengths, d))


# few items; dK and dV in pieces; dQ in pieces; up to 32 keys
@pytest.mark.parametrize("B,H,N_q,N_kv,lengths", [(1, 2, 300, 400, [399]), (2, 2, 3000, 200, [200, 60]), (2, 2, 40, 4000, [4000, 130]),
                                                  (6, 16, 700, 30, None)])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_of_short_items(B, H, N_q, N_kv, lengths, d):
    # A wait tries its barrier 33 times, each of some hundred ns, before it looks at the limit: of items of a few
    # blocks none may run out.  What reports nothing is right, and so is what comes after.
    call, out, ref = step(B, H, N_q, N_kv, lengths, d)
    elsewhere = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    try:
        fa.fa_set_wait_timeout_ns(1)
        for _ in range(8):
            for t in out:
                t.fill_(float("nan"))
            elsewhere.zero_()  # the inputs leave L2: the first loads take longest
            call()
            status = fa.fa_last_device_error()
            assert status == fa.FA_ERR_DEVICE_TIMEOUT or status == fa.FA_OK and all(torch.equal(a, b) for a, b in zip(out, ref))
    finally:
        fa.fa_set_wait_timeout_ns(0)
    call()
    check_status()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
