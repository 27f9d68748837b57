"""Norm and rotation by positions of several axes, and their gradient, against the float64 form.
Tolerances: those of the single axis (test_gpu_norm_rope), whose arithmetic this is."""
import numpy as np
import pytest
import torch

import exact_io_aware_06_gb300 as fa
import plain64
import test_gpu_norm_rope as nr
from gpu_util import check_status, ensure_built, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def turn(x, places, inv_freq, interleaved, sign=1.0):
    """x [B, N, heads, d] with pair p turned by sign * places[..., p] * inv_freq[p]."""
    y = x.copy()
    a, b = plain64.rope_pairs(2 * len(inv_freq), interleaved)
    ang = sign * (places * inv_freq)[:, :, None]
    y[..., a] = x[..., a] * np.cos(ang) - x[..., b] * np.sin(ang)
    y[..., b] = x[..., b] * np.cos(ang) + x[..., a] * np.sin(ang)
    return y


def grid_positions(axes, B, N, seed=0):
    g = torch.Generator().manual_seed(seed)
    i = torch.arange(N) + torch.randint(0, 5000, (B, 1), generator=g)
    return torch.stack([i // (11 * 3 ** a) * (-1) ** a for a in range(axes)]).to(torch.int32).cuda()


def run_both(B, N, H, H_kv, d, dtype, sections, interleaved, pos=None, shared=False, weights=True):
    qkv, qw, kw, up = nr.make(B, N, H, H_kv, d, dtype)
    if not weights:
        qw = kw = None
    pos = grid_positions(len(sections), B, N) if pos is None else pos
    f, axis = fa.rope_axes(sections, shared=shared)
    out = nr.outputs(B, N, H, H_kv, d, qkv.dtype)
    fa.fa_qk_norm_rope_axes(qkv, qw, kw, pos, f, axis, *out, 1e-6, interleaved)
    dqkv = torch.full_like(qkv, float("nan"))
    dw = [torch.full((d,), float("nan"), device="cuda") for _ in range(2)]
    ws = torch.empty(fa.fa_qk_norm_rope_bwd_workspace_size(B, H, H_kv, N, d), dtype=torch.uint8, device="cuda")
    fa.fa_qk_norm_rope_axes_bwd(qkv, qw, kw, pos, f, axis, *up, dqkv, *dw, ws, 1e-6, interleaved)
    check_status()

    x, places = f64(qkv), pos.cpu().numpy()[axis.numpy()].transpose(1, 2, 0).astype(np.float64)
    f = f.numpy()
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    first = 0
    for i, (heads, w) in enumerate(((H, qw), (H_kv, kw))):
        sl = slice(first, first + heads)
        first += heads
        w, n = nr.f64w(w, d), x[:, :, sl] * r[:, :, sl]
        ref = turn(n * w, places, f, interleaved).swapaxes(1, 2)
        nr.check(out[i], ref, 1.5 * np.abs(ref).max(-1, keepdims=True) + 1e-30, qkv.dtype, "qk"[i])
        g = turn(f64(up[i]).swapaxes(1, 2), places, f, interleaved, -1.0)
        # the amplitudes of test_gpu_norm_rope.compare_grad
        top = np.abs(w * g).max(-1, keepdims=True)
        amp = r[:, :, sl] * (1.5 * top + 2 * np.abs(n) * np.abs(w * g * n).mean(-1, keepdims=True))
        dx = r[:, :, sl] * (w * g - n * (w * g * n).mean(-1, keepdims=True))
        nr.check(dqkv[:, :, sl], dx, amp + 1e-30, qkv.dtype, "dqkv")
        mag = (np.abs(n) * 1.5 * np.abs(g).max(-1, keepdims=True)).sum((0, 1, 2))
        assert (np.abs(f64(dw[i]) - (g * n).sum((0, 1, 2))) <= 1e-5 * mag).all()
    assert torch.equal(out[2], qkv[:, :, H + H_kv:].transpose(1, 2))
    assert torch.equal(dqkv[:, :, H + H_kv:], up[2].transpose(1, 2))
    return qkv, qw, kw, up, out, dqkv, dw


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,sections", [(64, [16, 24, 24]), (64, [16, 16]), (128, [32, 48, 48]), (128, [2, 4, 10]),
                                        (128, [64, 32]), (128, [16] * 8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_and_sections(dtype, d, sections, interleaved):
    run_both(2, 37, 6, 2, d, dtype, sections, interleaved)


@pytest.mark.parametrize("B,N,H,H_kv", [(1, 1, 1, 1), (1, 1, 32, 8), (5, 1, 7, 7), (1, 3, 5, 3), (2, 1025, 9, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_sizes_and_head_counts(B, N, H, H_kv, d):
    run_both(B, N, H, H_kv, d, "bf16", [d // 4, d // 2, d // 4], False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_one_run_of_frequencies_and_no_weights(interleaved):
    run_both(2, 50, 4, 2, 128, "f32", [16, 56, 56], interleaved, shared=True, weights=False)


def test_far_and_negative_positions():
    ends = torch.tensor([0, 1, -1, 1 << 20, 123456789, -123456789, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    pos = torch.stack([ends, ends.flip(0), ends.roll(3)])[:, None].contiguous()
    run_both(1, 8, 2, 1, 128, "f32", [32, 48, 48], False, pos)


@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("interleaved", [False, True])
def test_equal_axes_give_the_single_axis_bit_for_bit(axes, interleaved):
    B, N, H, H_kv, d = 2, 75, 6, 2, 64
    one = grid_positions(1, B, N)
    sections = [64] if axes == 1 else [16, 24, 24]
    qkv, qw, kw, up, out, dqkv, dw = run_both(B, N, H, H_kv, d, "bf16", sections, interleaved,
                                              one.expand(axes, B, N).contiguous(), shared=True)
    f = fa.rope_frequencies(d)
    out2 = nr.outputs(B, N, H, H_kv, d, qkv.dtype)
    fa.fa_qk_norm_rope(qkv, qw, kw, one[0], f, *out2, 1e-6, interleaved)
    dqkv2, dw2 = torch.empty_like(dqkv), [torch.empty_like(x) for x in dw]
    ws = torch.empty(fa.fa_qk_norm_rope_bwd_workspace_size(B, H, H_kv, N, d), dtype=torch.uint8, device="cuda")
    fa.fa_qk_norm_rope_bwd(qkv, qw, kw, one[0], f, *up, dqkv2, *dw2, ws, 1e-6, interleaved)
    # (the weights' gradients, sums over all heads and tokens in an order of each call's own, are checked by run_both)
    for a, b in zip([*out, dqkv], [*out2, dqkv2]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,N,H,H_kv,d,sections", [(3, 3335, 1, 1, 64, [16, 48]), (2, 5001, 3, 1, 128, [128]), (1, 9999, 7, 2, 64, [32]),
                                                   (5, 601, 8, 8, 128, [32, 48, 16])])
def test_many_tokens_of_few_heads(B, N, H, H_kv, d, sections, interleaved, dtype):
    # where the tokens do not fill the last group of lanes, and a group holds tokens of two batches
    qkv, qw, kw, up, out, dqkv, dw = run_both(B, N, H, H_kv, d, dtype, sections, interleaved)
    pos, (f, axis) = grid_positions(len(sections), B, N), fa.rope_axes(sections)
    for again in range(2):
        dqkv2, dw2 = torch.empty_like(dqkv), [torch.empty_like(x) for x in dw]
        ws = torch.full((fa.fa_qk_norm_rope_bwd_workspace_size(B, H, H_kv, N, d),), 255, dtype=torch.uint8, device="cuda")
        fa.fa_qk_norm_rope_axes_bwd(qkv, qw, kw, pos, f, axis, *up, dqkv2, *dw2, ws, 1e-6, interleaved)
        for a, b in zip([dqkv, *dw], [dqkv2, *dw2]):
            assert torch.equal(a, b)
    # the same rows as in another call of one batch (another place in the group)
    out2 = nr.outputs(1, N, H, H_kv, d, qkv.dtype)
    fa.fa_qk_norm_rope_axes(qkv[-1:], qw, kw, pos[:, -1:].clone(), f, axis, *out2, 1e-6, interleaved)
    assert all(torch.equal(a[-1:], b) for a, b in zip(out, out2))


def test_without_rotation():
    qkv, qw, kw, _ = nr.make(1, 9, 4, 2, 64, "f32")
    out, out2 = (nr.outputs(1, 9, 4, 2, 64, torch.float32) for _ in range(2))
    fa.fa_qk_norm_rope_axes(qkv, qw, kw, None, None, None, *out, 1e-6)
    fa.fa_qk_norm_rope(qkv, qw, kw, None, None, *out2, 1e-6)
    assert all(torch.equal(a, b) for a, b in zip(out, out2))


def test_captured_and_on_another_stream():
    B, N, H, H_kv, d = 2, 64, 8, 2, 128
    qkv, qw, kw, _ = nr.make(B, N, H, H_kv, d, "bf16")
    pos, (f, axis) = grid_positions(3, B, N), fa.rope_axes([32, 48, 48])
    eager, out = (nr.outputs(B, N, H, H_kv, d, qkv.dtype) for _ in range(2))
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        fa.fa_qk_norm_rope_axes(qkv, qw, kw, pos, f, axis, *out, 1e-6)
    torch.cuda.current_stream().wait_stream(s)
    pos += 12345  # read when the graph runs
    graph.replay()
    fa.fa_qk_norm_rope_axes(qkv, qw, kw, pos, f, axis, *eager, 1e-6)
    check_status()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_binding_refuses_wrong_tensors():
    qkv, qw, kw, _ = nr.make(1, 4, 2, 1, 64, "bf16")
    out = nr.outputs(1, 4, 2, 1, 64, torch.bfloat16)
    pos, (f, axis) = grid_positions(2, 1, 4), fa.rope_axes([32, 32])
    for args in ((pos[0], f, axis), (pos.float(), f, axis), (pos[:, :, :3], f, axis), (pos.cpu(), f, axis),
                 (None, f, axis), (pos, f, None), (pos, f, axis.long()), (pos, f, axis.cuda()), (pos, f, axis[:31]),
                 (pos, f.float(), axis)):
        with pytest.raises(ValueError):
            fa.fa_qk_norm_rope_axes(qkv, qw, kw, *args, *out, 1e-6)
    for bad in (axis + 1, axis - 1):  # an axis that positions do not have
        with pytest.raises(fa.FaError):
            fa.fa_qk_norm_rope_axes(qkv, qw, kw, pos, f, bad, *out, 1e-6)
