"""Shared prefixes, by every way that the rows take: without lse, the same bits every time, two calls at once,
captured, tensors beyond 32-bit offsets.  Tolerances: those of test_gpu_cross."""
import pytest
import torch

import exact_io_aware_06_gb300 as fa
from gpu_util import check_status, ensure_built, scale_for
from test_gpu_cross import captured, check_forward, inputs, on_device, sizes, space
from test_gpu_cross_joins import own_attention

pytestmark = pytest.mark.gpu

# a few rows, a cluster of CTAs an item, items cut and joined, whole items
WAYS = [(2, 2, 2, 2, 1, 1500), (8, 1, 8, 2, 1, 1500), (64, 1, 8, 2, 1, 16384), (4, 4, 8, 8, 2400, 200)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


class Prefix:
    def __init__(self, B, B_kv, H, H_kv, N_q, N_kv, d, seed):
        self.q, self.k, self.v, _ = inputs(B, B_kv, H, H_kv, N_q, N_kv, d, seed)
        self.own, self.scale = own_attention(self.q, seed), scale_for(d)
        self.lengths = [N_kv - 1, N_kv // 3, 0, N_kv][:B_kv]
        self.n = on_device(self.lengths)
        self.o, self.lse = torch.full_like(self.q, float("nan")), torch.full(self.q.shape[:3], float("nan"), device="cuda")
        self.ws = space(fa.fa_fwd_prefix_workspace_size(*sizes(self.q, self.k)))

    def __call__(self, lse=True, stream=None):
        fa.fa_fwd_prefix(self.q, self.k, self.v, self.n, *self.own, self.o, self.lse if lse else None, self.ws, self.scale,
                         stream=stream)

    def check(self, lengths=None):
        batches = range(0, len(self.q), max(1, len(self.q) // 6))
        check_forward(self.q, self.k, self.v, self.lengths if lengths is None else lengths, self.o, self.lse, self.scale,
                      own=self.own, batches=batches)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("d", [64, 128])
def test_repeats_bit_for_bit_and_without_lse(way, d):
    p = Prefix(*way, d, seed=1)
    p()
    check_status()
    p.check()
    o, lse = p.o.clone(), p.lse.clone()
    for with_lse in (True, False):
        p.o.fill_(float("nan")), p.lse.fill_(7.0), p.ws.fill_(255)
        p(with_lse)
        check_status()
        assert torch.equal(p.o, o) and torch.equal(p.lse, lse if with_lse else torch.full_like(lse, 7.0))


@pytest.mark.parametrize("way", WAYS)
def test_two_calls_at_once(way):
    calls, streams = [Prefix(*way, 128, seed=20 + i) for i in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for p, s in zip(calls, streams):
            p(stream=s)
    torch.cuda.synchronize()
    check_status()
    for p in calls:
        p.check()


@pytest.mark.parametrize("way", WAYS)
def test_captured_call_follows_lengths_and_own_attention(way):
    p = Prefix(*way, 64, seed=3)
    graph = captured(p)
    for part in (1, 0, 3, 2):
        lengths = [n * part // 3 for n in p.lengths]
        p.n.copy_(torch.tensor(lengths, dtype=torch.int32))
        for mine, new in zip(p.own, own_attention(p.q, part)):
            mine.copy_(new)
        p.o.fill_(float("nan")), p.lse.fill_(float("nan"))
        graph.replay()
        check_status()
        p.check(lengths)


def test_large_offsets():
    # queries and the prefix's keys beyond 2^31 bytes from the base, of whole items, of cut ones and of a few rows
    for B, B_kv, H, N_q, N_kv in ((70, 70, 8, 16384, 64), (140, 70, 8, 5, 16384), (70, 70, 8, 1, 16384)):
        q = torch.zeros((B, H, N_q, 128), dtype=torch.bfloat16, device="cuda")
        k = torch.zeros((B_kv, H, N_kv, 128), dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        q1, k1, v1, _ = inputs(1, 1, 1, 1, N_q, N_kv, 128, seed=11)
        q[-1, -1], k[-1, -1], v[-1, -1] = q1[0, 0], k1[0, 0], v1[0, 0]
        o, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
        o[-1, -1], lse[-1, -1] = (t[0, 0] for t in own_attention(q1, 5))
        own1 = o[-1:, -1:].clone(), lse[-1:, -1:].clone()
        ws = space(fa.fa_fwd_prefix_workspace_size(*sizes(q, k)))
        fa.fa_fwd_prefix(q, k, v, None, o, lse, o, lse, ws, scale_for(128))
        check_status()
        check_forward(q1, k1, v1, None, o[-1:, -1:], lse[-1:, -1:], scale_for(128), own=own1)
        assert (o[0] == 0).all()


@pytest.mark.parametrize("way", WAYS)
def test_rows_whose_own_lse_is_the_lowest_float_have_no_keys(way):
    # as with -inf, and between them own attention that weighs next to nothing or all there is
    p = Prefix(*way, 128, seed=7)
    o, lse = p.own
    lse.view(-1)[::5] = torch.finfo(torch.float32).min
    lse.view(-1)[1::5], lse.view(-1)[2::5] = -2.0 ** 127, 2.0 ** 100
    p()
    check_status()
    low, high = lse <= -2.0 ** 127, lse == 2.0 ** 100
    own, here = p.own, torch.zeros_like(low)
    for b, n in enumerate(p.lengths):
        share = len(p.q) // len(p.lengths)
        here[b * share:(b + 1) * share] = n > 0
    out, out_lse = p.o.clone(), p.lse.clone()
    lse[low] = -float("inf")  # the prefix alone
    p()
    check_status()
    assert torch.equal(out[low & here], p.o[low & here]) and torch.equal(out_lse[low & here], p.lse[low & here])
    none = (own[0] != own[0]).any(-1) & ~here  # of neither
    assert none.sum() == 0 or (out[none] == 0).all() and (out_lse[none] == -float("inf")).all()
    assert torch.equal(out[high], o[high]) and torch.allclose(out_lse[high], lse[high], rtol=2.0 ** -22, atol=0)
