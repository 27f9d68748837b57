"""Layers that attend to another sequence, one operator after the other: a training step of a decoder over
encoded text with image positions, and tokens of several requests behind one shared prompt.  Each result is
checked against the float64 form of the operator on the tensors that it was given, with that operator's
tolerance (the modules imported here)."""
import numpy as np
import pytest
import torch

import exact_io_aware_06_gb300 as fa
import oracle
import plain64
import test_gpu_cross as cross
import test_gpu_kv4 as kv4
import test_gpu_norm_rope as nr
import test_gpu_rope_axes as axes
import test_gpu_window as win
from gpu_util import TOL_BF16_GRAD, TOL_BF16_O, check_status, ensure_built, f64, max_err

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def empty(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("B,B_kv,H,H_kv,N,N_kv,d,lengths", [(2, 2, 4, 2, 300, 150, 64, [150, 77]),
                                                            (4, 2, 2, 2, 130, 200, 128, [129, 24])])
def test_training_step_over_encoded_text(B, B_kv, H, H_kv, N, N_kv, d, lengths):
    # image tokens attend to one another, turned by row and column, and then to the text
    scale, (f, axis) = d ** -0.5, fa.rope_axes([d // 2, d // 2])
    qkv, qw, kw, _ = nr.make(B, N, H, H, d, "bf16")
    pos = axes.grid_positions(2, B, N)
    text_k, text_v = cross.rand((B_kv, H_kv, N_kv, d), 7), cross.rand((B_kv, H_kv, N_kv, d), 8)
    n, do = cross.on_device(lengths), cross.rand((B, H, N, d), 9)
    q, k, v, o, o2 = (empty(B, H, N, d) for _ in range(5))
    lse, lse2 = (empty(B, H, N, dtype=torch.float32) for _ in range(2))
    d_o, dq, dk, dv = (empty(B, H, N, d) for _ in range(4))
    d_text = [empty(B_kv, H_kv, N_kv, d) for _ in range(2)]
    dqkv, dw = torch.full_like(qkv, float("nan")), [empty(d, dtype=torch.float32) for _ in range(2)]
    sizes = (B, B_kv, H, H_kv, N, N_kv, d)
    # one workspace for all: they follow one another on one stream
    ws = cross.space(max(fa.fa_fwd_cross_workspace_size(*sizes), fa.fa_bwd_cross_workspace_size(*sizes),
                         fa.fa_bwd_workspace_size(B, H, N, d), fa.fa_qk_norm_rope_bwd_workspace_size(B, H, H, N, d)))

    def step():
        fa.fa_qk_norm_rope_axes(qkv, qw, kw, pos, f, axis, q, k, v, EPS)
        fa.fa_fwd(q, k, v, o, lse, scale, False, fa.FA_BF16)
        fa.fa_fwd_cross(o, text_k, text_v, n, o2, lse2, ws, scale)
        fa.fa_bwd_cross(o, text_k, text_v, n, o2, lse2, do, d_o, *d_text, ws, scale)
        fa.fa_bwd(q, k, v, o, lse, d_o, dq, dk, dv, ws, scale, False, fa.FA_BF16)
        fa.fa_qk_norm_rope_axes_bwd(qkv, qw, kw, pos, f, axis, dq, dk, dv, dqkv, *dw, ws, EPS)

    def check():
        check_status()
        ref, _ = oracle.attn_fwd(f64(q), f64(k), f64(v), scale)
        assert max_err(f64(o), ref) <= TOL_BF16_O
        cross.check_forward(o, text_k, text_v, lengths, o2, lse2, scale)
        cross.check_backward(o, text_k, text_v, lengths, do, (d_o, *d_text), scale)
        grads = oracle.attn_bwd(f64(q), f64(k), f64(v), f64(d_o), scale)
        assert all(max_err(f64(g), r) <= TOL_BF16_GRAD for g, r in zip((dq, dk, dv), grads))
        assert torch.isfinite(dqkv).all() and all(torch.isfinite(x).all() for x in dw)

    step()
    check()
    first = [t.clone() for t in (o2, lse2, *d_text, d_o)]
    graph = cross.captured(step)
    graph.replay()
    check_status()
    assert all(torch.equal(a, b) for a, b in zip(first, (o2, lse2, *d_text, d_o)))
    qkv.copy_(nr.make(B, N, H, H, d, "bf16", seed=9)[0])
    lengths[:] = [N_kv, 3]
    n.copy_(torch.tensor(lengths, dtype=torch.int32))
    graph.replay()
    check()


@pytest.mark.parametrize("d,H,H_kv", [(64, 4, 2), (128, 8, 1)])
def test_tokens_behind_a_shared_prompt(d, H, H_kv):
    # the prompt's keys and values once, the requests' own tokens in the 4-bit cache; a captured step moves the
    # requests' lengths on by itself
    own, new, N_prompt, scale, f = [3, 0, 40, 17, 1], 4, 333, d ** -0.5, fa.rope_frequencies(d)
    B = len(own)
    c = kv4.Cache([n + new for n in own], H_kv, d, 16)
    held = [[x[b][:, :n] for b, n in enumerate(own)] for x in c.fill(2)]  # K and V of the requests, as stored
    pk, pv = cross.rand((1, H_kv, N_prompt, d), 3), cross.rand((1, H_kv, N_prompt, d), 4)
    lengths, at = kv4.ints(own), torch.empty((B, 1), dtype=torch.int32, device="cuda")
    x, qw, kw, _ = nr.make(B, 1, H, H_kv, d, "bf16")
    q, k, v = empty(B, H, 1, d), empty(B, H_kv, 1, d), empty(B, H_kv, 1, d)
    o_own, lse_own = empty(B, H, 1, d), empty(B, H, 1, dtype=torch.float32)
    o, lse = empty(B, H, 1, d), empty(B, H, 1, dtype=torch.float32)
    ws = cross.space(max(fa.fa_decode_kv4_workspace_size(B, H, H_kv, 1, d),
                         fa.fa_fwd_prefix_workspace_size(B, 1, H, H_kv, 1, N_prompt, d)))

    def token():
        at.copy_(lengths[:, None] + N_prompt)
        fa.fa_qk_norm_rope(x, qw, kw, at, f, q, k, v, EPS)
        fa.fa_kv4_append(k, v, *c.args, lengths)
        lengths.add_(1)
        fa.fa_decode_kv4(q, *c.args, lengths, o_own, lse_own, ws, scale)
        fa.fa_fwd_prefix(q, pk, pv, None, o_own, lse_own, o, lse, ws, scale)

    graph = cross.captured(token)
    for i in range(new):
        x.copy_(nr.make(B, 1, H, H_kv, d, "bf16", seed=20 + i)[0])
        graph.replay()
        check_status()
        assert lengths.tolist() == [n + i + 1 for n in own]
        cross.check_forward(q, pk, pv, None, o, lse, scale, own=(o_own, lse_own))
        for values, x1 in zip(held, (k, v)):
            for b in range(B):
                values[b] = np.concatenate([values[b], plain64.kv4_values(f64(x1))[b]], 1)
    # and as one attention to prompt and own tokens together.  Of A = sum w |v|: P 2^-8 of the prompt's, the decode's
    # (test_gpu_kv4) 2^-7 and 2 e, and its result is rounded on the way (2^-8); o 2^-8; float32 scores and
    # sums of the rest and the merge 3e-5 (1 + max |score|).  lse: that and e.
    for b in range(B):
        for h in range(H):
            kv = h // (H // H_kv)
            keys, vals = (np.concatenate([f64(x0)[0, kv], values[b][kv]]) for x0, values in zip((pk, pv), held))
            Q = f64(q)[b, h]
            ref, ref_lse, P = plain64.attention(Q, keys, vals, scale, np.ones((1, len(keys)), dtype=bool))
            A, top = P @ np.abs(vals), 3e-5 * (1 + scale * np.abs(Q @ keys.T).max())
            e = 2.0 ** -21 * scale * np.abs(held[0][b][kv]).max() / 7 * 151 * np.abs(Q).sum()
            assert (np.abs(f64(o)[b, h] - ref) <= 2.0 ** -8 * (3 * A + np.abs(ref)) + (top + 2 * e) * A).all()
            assert (np.abs(f64(lse)[b, h] - ref_lse) <= top + e).all()


def test_two_captured_steps_at_once_on_two_streams():
    # each with its own tensors and workspaces; the same bits as one after the other
    d, H, H_kv, N, N_kv = 64, 8, 2, 400, 500

    class Layer:
        def __init__(self, seed):
            self.q, self.k, self.v, self.do = cross.inputs(2, 2, H, H_kv, N, N_kv, d, seed)
            self.n = cross.on_device([N_kv, 130 + seed])
            self.q1 = cross.rand((6, H, 1, d), seed + 9)
            self.o, self.lse = empty(2, H, N, d), empty(2, H, N, dtype=torch.float32)
            self.o1, self.lse1 = empty(6, H, 1, d), empty(6, H, 1, dtype=torch.float32)
            self.grads = [torch.full_like(t, float("nan")) for t in (self.q, self.k, self.v)]
            sizes = cross.sizes(self.q, self.k)
            self.ws = cross.space(max(fa.fa_fwd_cross_workspace_size(*sizes), fa.fa_bwd_cross_workspace_size(*sizes),
                                      fa.fa_fwd_cross_workspace_size(*cross.sizes(self.q1, self.k))))

        def run(self):
            fa.fa_fwd_cross(self.q, self.k, self.v, self.n, self.o, self.lse, self.ws, 0.125)
            fa.fa_bwd_cross(self.q, self.k, self.v, self.n, self.o, self.lse, self.do, *self.grads, self.ws, 0.125)
            fa.fa_fwd_cross(self.q1, self.k, self.v, self.n, self.o1, self.lse1, self.ws, 0.125)

        def results(self):
            return [self.o, self.lse, *self.grads, self.o1, self.lse1]

    layers = [Layer(3), Layer(30)]
    for layer in layers:
        layer.run()
    check_status()
    ref = [[t.clone() for t in layer.results()] for layer in layers]
    graphs = [cross.captured(layer.run) for layer in layers]
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
