"""The layer's operators one after the other, as a layer calls them: a training step, and a prompt
followed by single tokens.  Each result is checked against the float64 form of the operator on the
tensors that it was given, with that operator's tolerance (the modules imported here)."""
import numpy as np
import pytest
import torch

import exact_io_aware_06_gb300 as fa
import plain64
import test_gpu_kv4 as kv4
import test_gpu_norm_rope as nr
import test_gpu_window as win
from gpu_util import check_status, ensure_built, f64

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def empty(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def space(nbytes):
    return torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")


def captured(call):
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    return graph


@pytest.mark.parametrize("B,H,H_kv,N,d,window,n_sink", [(2, 4, 2, 300, 64, 100, 4), (1, 6, 2, 389, 128, 130, 0),
                                                        (3, 2, 2, 1, 64, 8, 1)])
def test_training_step(B, H, H_kv, N, d, window, n_sink):
    scale, f = d ** -0.5, fa.rope_frequencies(d)
    qkv, qw, kw, _ = nr.make(B, N, H, H_kv, d, "bf16")
    do = win.rand((B, H, N, d), 5)
    q, k, v = empty(B, H, N, d), empty(B, H_kv, N, d), empty(B, H_kv, N, d)
    o, lse = empty(B, H, N, d), empty(B, H, N, dtype=torch.float32)
    dq, dk, dv, dqkv = (torch.full_like(t, float("nan")) for t in (q, k, v, qkv))
    dw = [empty(d, dtype=torch.float32) for _ in range(2)]
    # one workspace for both gradients: they follow one another on one stream
    ws = space(max(fa.fa_bwd_window_workspace_size(B, H, H_kv, N, d, window, n_sink),
                   fa.fa_qk_norm_rope_bwd_workspace_size(B, H, H_kv, N, d)))

    def step():
        fa.fa_qk_norm_rope(qkv, qw, kw, None, f, q, k, v, EPS)
        fa.fa_fwd_window(q, k, v, o, lse, scale, window, n_sink)
        fa.fa_bwd_window(q, k, v, o, lse, do, dq, dk, dv, ws, scale, window, n_sink)
        fa.fa_qk_norm_rope_bwd(qkv, qw, kw, None, f, dq, dk, dv, dqkv, *dw, ws, EPS)

    def check():
        check_status()
        nr.compare_forward(qkv, (q, k, v), qw, kw, None, f, EPS, False)
        win.check_forward(q, k, v, o, lse, scale, window, n_sink)
        win.check_backward(q, k, v, do, (dq, dk, dv), scale, window, n_sink)
        nr.compare_grad(qkv, (dq, dk, dv), dqkv, dw, qw, kw, None, f, EPS, False)

    step()
    check()
    first = [t.clone() for t in (o, lse, dqkv, *dw)]
    graph = captured(step)
    graph.replay()
    check_status()
    assert all(torch.equal(a, b) for a, b in zip(first, (o, lse, dqkv, *dw)))
    qkv.copy_(nr.make(B, N, H, H_kv, d, "bf16", seed=9)[0])
    graph.replay()
    check()


def test_two_captured_steps_at_once_on_two_streams():
    # each with its own tensors and workspaces; the same bits as one after the other
    d, H, H_kv, N, window = 64, 8, 2, 1500, 200
    f, eps = fa.rope_frequencies(d), EPS

    class Layer:
        def __init__(self, seed):
            self.qkv, self.qw, self.kw, _ = nr.make(1, N, H, H_kv, d, "bf16", seed=seed)
            self.do = win.rand((1, H, N, d), seed + 1)
            self.q, self.k, self.v = empty(1, H, N, d), empty(1, H_kv, N, d), empty(1, H_kv, N, d)
            self.o, self.lse = empty(1, H, N, d), empty(1, H, N, dtype=torch.float32)
            self.grads = [torch.full_like(t, float("nan")) for t in (self.q, self.k, self.v)]
            self.dqkv, self.dw = torch.full_like(self.qkv, float("nan")), [empty(d, dtype=torch.float32) for _ in "qk"]
            self.ws = space(max(fa.fa_bwd_window_workspace_size(1, H, H_kv, N, d, window, 4),
                                fa.fa_qk_norm_rope_bwd_workspace_size(1, H, H_kv, N, d)))
            self.c = kv4.Cache([N], H_kv, d, 32, seed=seed)
            self.first, self.n = kv4.ints([0]), kv4.ints([N])
            self.q1, self.o1 = win.rand((1, H, 1, d), seed + 2), empty(1, H, 1, d)
            self.ws1 = space(fa.fa_decode_kv4_workspace_size(1, H, H_kv, 1, d))

        def run(self):
            fa.fa_qk_norm_rope(self.qkv, self.qw, self.kw, None, f, self.q, self.k, self.v, eps)
            fa.fa_fwd_window(self.q, self.k, self.v, self.o, self.lse, 0.125, window, 4)
            fa.fa_kv4_append(self.k, self.v, *self.c.args, self.first)
            fa.fa_bwd_window(self.q, self.k, self.v, self.o, self.lse, self.do, *self.grads, self.ws, 0.125, window, 4)
            fa.fa_decode_kv4(self.q1, *self.c.args, self.n, self.o1, None, self.ws1, 0.125, window, 4)
            fa.fa_qk_norm_rope_bwd(self.qkv, self.qw, self.kw, None, f, *self.grads, self.dqkv, *self.dw, self.ws, eps)

        def results(self):
            return [self.o, self.lse, self.dqkv, *self.dw, self.o1]

    layers = [Layer(3), Layer(30)]
    for layer in layers:
        layer.run()
    check_status()
    ref = [[t.clone() for t in layer.results()] for layer in layers]
    graphs = [captured(layer.run) for layer in layers]
    for layer in layers:
        for t in layer.results():
            t.fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    check_status()
    for layer, r in zip(layers, ref):
        assert all(torch.equal(a, b) for a, b in zip(layer.results(), r))


@pytest.mark.parametrize("d,H,H_kv,page,window,n_sink", [(64, 4, 2, 16, 60, 4), (128, 6, 1, 32, 5000, 0),
                                                         (64, 3, 3, 64, 33, 40)])
def test_prompt_then_tokens(d, H, H_kv, page, window, n_sink):
    prompts, new = [150, 1, 77], 5
    B, N, scale, f = len(prompts), max(prompts), d ** -0.5, fa.rope_frequencies(d)
    c = kv4.Cache([n + new for n in prompts], H_kv, d, page)
    lengths = kv4.ints(prompts)

    # the prompts side by side, those that are shorter filled up behind their end
    qkv, qw, kw, _ = nr.make(B, N, H, H_kv, d, "bf16")
    q, k, v = empty(B, H, N, d), empty(B, H_kv, N, d), empty(B, H_kv, N, d)
    o, lse = empty(B, H, N, d), empty(B, H, N, dtype=torch.float32)
    fa.fa_qk_norm_rope(qkv, qw, kw, None, f, q, k, v, EPS)
    fa.fa_fwd_window(q, k, v, o, lse, scale, window, n_sink)
    fa.fa_kv4_append(k, v, *c.args, kv4.ints([0] * B), lengths)
    check_status()
    nr.compare_forward(qkv, (q, k, v), qw, kw, None, f, EPS, False)
    win.check_forward(q, k, v, o, lse, scale, window, n_sink)
    held = [[plain64.kv4_values(f64(t))[b, :, :n] for b, n in enumerate(prompts)] for t in (k, v)]

    # what a further piece of the prompt would attend to
    back = [torch.full_like(t, float("nan")) for t in (k, v)]
    fa.fa_kv4_read(*c.args, lengths, *back)
    check_status()
    for t, values in zip(back, held):
        for b, n in enumerate(prompts):
            assert np.array_equal(f64(t)[b, :, :n], plain64.bf16_round(values[b])) and (t[b, :, n:] == 0).all()

    # single tokens: one captured step that moves the lengths on by itself
    x = qkv[:, :1].contiguous()
    at = torch.empty((B, 1), dtype=torch.int32, device="cuda")
    q1, k1, v1 = empty(B, H, 1, d), empty(B, H_kv, 1, d), empty(B, H_kv, 1, d)
    o1, lse1 = empty(B, H, 1, d), empty(B, H, 1, dtype=torch.float32)
    ws = space(fa.fa_decode_kv4_workspace_size(B, H, H_kv, 1, d))

    def token():
        at.copy_(lengths[:, None])
        fa.fa_qk_norm_rope(x, qw, kw, at, f, q1, k1, v1, EPS)
        fa.fa_kv4_append(k1, v1, *c.args, lengths)
        lengths.add_(1)
        fa.fa_decode_kv4(q1, *c.args, lengths, o1, lse1, ws, scale, window, n_sink)

    graph = captured(token)
    for i in range(new):
        x.copy_(nr.make(B, 1, H, H_kv, d, "bf16", seed=20 + i)[0])
        graph.replay()
        check_status()
        now = [n + i + 1 for n in prompts]
        assert lengths.tolist() == now
        nr.compare_forward(x, (q1, k1, v1), qw, kw, at, f, EPS, False)
        for values, t in zip(held, (k1, v1)):
            for b in range(B):
                values[b] = np.concatenate([values[b], plain64.kv4_values(f64(t))[b]], 1)
        kv4.compare(q1, o1, lse1, *held, now, window, n_sink)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_in_two_pieces(d):
    # the second piece attends to the cache's dense prefix as one shard of keys and to itself as another
    B, H, H_kv, n0, n1 = 1, 4, 2, 140, 75
    scale, f = d ** -0.5, fa.rope_frequencies(d)
    c = kv4.Cache([n0 + n1], H_kv, d, 64)
    values = []
    for first, n in ((0, n0), (n0, n1)):
        qkv, qw, kw, _ = nr.make(B, n, H, H_kv, d, "bf16", seed=first)
        pos = torch.arange(first, first + n, dtype=torch.int32, device="cuda")[None]
        q, k, v = empty(B, H, n, d), empty(B, H_kv, n, d), empty(B, H_kv, n, d)
        fa.fa_qk_norm_rope(qkv, qw, kw, pos, f, q, k, v, EPS)
        fa.fa_kv4_append(k, v, *c.args, kv4.ints([first]))
        values.append((f64(k), f64(v)))
    pk, pv = empty(B, H_kv, n0, d), empty(B, H_kv, n0, d)
    fa.fa_kv4_read(*c.args, kv4.ints([n0]), pk, pv)
    parts, part_lse = empty(2, B, H, n1, d, dtype=torch.float32), empty(2, B, H, n1, dtype=torch.float32)
    fa.fa_fwd_kv_shard(q, pk, pv, parts[0], part_lse[0], scale, True, n0, 0)
    fa.fa_fwd_kv_shard(q, k, v, parts[1], part_lse[1], scale, True, n0, n0)
    o, lse = empty(B, H, n1, d), empty(B, H, n1, dtype=torch.float32)
    fa.fa_lse_merge(parts, part_lse, o, lse, fa.FA_BF16)
    check_status()
    keys, vals = (np.concatenate([plain64.bf16_round(plain64.kv4_values(a)), b], 2)[0]
                  for a, b in zip(values[0], values[1]))
    seen = plain64.window_mask(n1, n0 + n1, n0, 0, 0)
    for h in range(H):
        Q = f64(q)[0, h]
        ref, ref_lse, P = plain64.attention(Q, keys[h // 2], vals[h // 2], scale, seen)
        A = P @ np.abs(vals[h // 2])
        # P and o rounded to bfloat16, 2^-8 each; the row sum adds the rounded P or not, 2^-8 of lse's 1
        # (and of A) at most; float32 scores, sums and merge 2e-5
        top = 2e-5 * (1 + scale * np.abs(Q @ keys[h // 2].T).max(-1))
        assert (np.abs(f64(o)[0, h] - ref) <= 2.0 ** -8 * (2 * A + np.abs(ref)) + top[:, None] * A).all()
        assert (np.abs(f64(lse)[0, h] - ref_lse) <= 2.0 ** -8 + top).all()


def test_binding_refuses_tensors_that_kernels_would_misread():
    q, o = win.rand((1, 2, 8, 64), 1), empty(1, 2, 8, 64)
    lse = empty(1, 2, 8, dtype=torch.float32)
    bad = [(q.float(), q, q, o, lse), (q.transpose(2, 3).contiguous().transpose(2, 3), q, q, o, lse),
           (q, q[:, :, :4], q, o, lse), (q, q, q, o[:, :1], lse), (q, q, q, o, lse.double()), (q.cpu(), q, q, o, lse),
           (q[0], q, q, o, lse)]
    for args in bad:
        with pytest.raises(ValueError):
            fa.fa_fwd_window(*args, 0.125, 4, 0)
    grads = [torch.empty_like(q) for _ in range(3)]
    ws = space(fa.fa_bwd_window_workspace_size(1, 2, 2, 8, 64, 4, 0))
    for dq, w in ((grads[0][:, :, :7], ws), (grads[0], ws.cpu()), (grads[0], ws[::2])):
        with pytest.raises(ValueError):
            fa.fa_bwd_window(q, q, q, o, lse, q, dq, *grads[1:], w, 0.125, 4, 0)
    c = kv4.Cache([8], 2, 64, 16)
    n = kv4.ints([8])
    ws = space(fa.fa_decode_kv4_workspace_size(1, 4, 2, 1, 64))
    q1 = win.rand((1, 4, 1, 64), 2)
    for args in ((q1, *c.arrays, c.table.long(), n, q1, None, ws), (q1, *c.arrays, c.table, n.cpu(), q1, None, ws),
                 (q1, *c.arrays[:3], c.arrays[3].float(), c.table, n, q1, None, ws),
                 (q1, c.arrays[0][:, :, :8], *c.arrays[1:], c.table, n, q1, None, ws),
                 (q1, *c.arrays, c.table, kv4.ints([8, 8]), q1, None, ws)):
        with pytest.raises(ValueError):
            fa.fa_decode_kv4(*args, 0.125)
    for first in (n.float(), n[None], n.cpu()):
        with pytest.raises(ValueError):
            fa.fa_kv4_append(q[:, :, :1].contiguous(), q[:, :, :1].contiguous(), *c.args, first)
    assert fa.fa_last_device_error() == 0


@pytest.mark.parametrize("window,n_sink", [(2 ** 31, 0), (2 ** 32 + 1, 2), (2 ** 63, 3), (3, 2 ** 32), (5, 2 ** 40 + 1)])
def test_windows_and_sinks_beyond_32_bits(window, n_sink):
    # as any others that cover the sequence
    B, H, H_kv, N, d, scale = 1, 2, 1, 200, 64, 0.125
    q, k, v, do = win.inputs(B, H, H_kv, N, d)
    results = []
    for w, s in ((window, n_sink), (min(window, N), min(n_sink, N))):
        o, lse = win.forward(q, k, v, scale, w, s)
        grads = win.backward(q, k, v, o, lse, do, scale, w, s)
        c = kv4.Cache([N, 77], H_kv, d, 16)
        c.fill(3)
        one = kv4.decode(win.rand((2, H, 1, d), 4), c, [N, 77], w, s, scale)[:2]
        results.append((o, lse, *grads, *one))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    with pytest.raises(RuntimeError):
        fa.fa_fwd_window(q, k, v, o, lse, scale, 5 - 2 ** 32, 0)
    with pytest.raises(RuntimeError):
        fa.fa_fwd_window(q, k, v, o, lse, scale, 5, 5 - 2 ** 32)
