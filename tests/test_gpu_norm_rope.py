"""Norm and rotation of Q and K, and their gradient, against the float64 form.

Tolerances.  A value is a sum of at most two products w_a n_a cos, w_b n_b sin with n = x r:
its float32 error is at most (12 additions of the mean, halved by the root, + 2 units for
rsqrt + 3 products + cos and sin, whose angle is off by 2^-25 half turns: 2 pi 2^-25 + 2^-23)
under 2e-6 of the pair's amplitude.  bfloat16 results add half a step, 2^-8 of the value."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import exact_io_aware_06_gb300 as fa
import plain64
from gpu_util import check_status, ensure_built, f64

pytestmark = pytest.mark.gpu
F32_TOL, HALF_STEP = 2e-6, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(B, N, H, H_kv, d, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    qkv = (scale * torch.randn((B, N, H + 2 * H_kv, d), generator=g)).to(t).cuda()
    qw, kw = (1 + 0.2 * torch.randn((2, d), generator=g)).cuda().unbind()
    up = [torch.randn((B, h, N, d), generator=g).to(t).cuda() for h in (H, H_kv, H_kv)]
    return qkv, qw.contiguous(), kw.contiguous(), up


def outputs(B, N, H, H_kv, d, t):
    return [torch.full((B, h, N, d), float("nan"), dtype=t, device="cuda") for h in (H, H_kv, H_kv)]


def f64w(w, d):
    return np.ones(d) if w is None else f64(w)


def check(got, ref, amplitude, t, what):
    tol = F32_TOL * amplitude + (HALF_STEP * np.abs(ref) if t == torch.bfloat16 else 0.0)
    err = np.abs(f64(got) - ref)
    assert np.isfinite(f64(got)).all(), what
    assert (err <= tol).all(), (what, float((err / np.maximum(tol, 1e-300)).max()))


def reference_inputs(qkv, H_kv, qw, kw, pos, f):
    B, N, heads, d = qkv.shape
    p = np.broadcast_to(np.arange(N), (B, N)) if pos is None else pos.cpu().numpy()
    return f64(qkv), heads - 2 * H_kv, f64w(qw, d), f64w(kw, d), p, [] if f is None else f.numpy()


def compare_forward(qkv, out, qw, kw, pos, f, eps, interleaved):
    H_kv = out[1].shape[1]
    x, H, a, b, p, fr = reference_inputs(qkv, H_kv, qw, kw, pos, f)
    ref = plain64.norm_rope(x, H, H_kv, a, b, p, fr, eps, interleaved)
    for name, got, r in zip("qkv", out, ref):
        if name == "v":
            assert torch.equal(got, qkv[:, :, H + H_kv:].transpose(1, 2))
        else:  # the pair's amplitude is at most sqrt(2) times the row's largest |w n|
            check(got, r, 1.5 * np.abs(r).max(-1, keepdims=True) + 1e-30, qkv.dtype, name)


def compare_grad(qkv, up, dqkv, dw, qw, kw, pos, f, eps, interleaved):
    # gradient: |dx| terms are r w g and r n mean(w g n), n = x r; the mean's own error is
    # under 2e-6 of mean |w g n|
    H_kv, d = up[1].shape[1], qkv.shape[-1]
    x, H, a, b, p, fr = reference_inputs(qkv, H_kv, qw, kw, pos, f)
    rx, rqw, rkw = plain64.norm_rope_grad(x, H, H_kv, a, b, p, fr, eps, interleaved, *map(f64, up))
    w = np.concatenate([np.tile(a, (H, 1)), np.tile(b, (H_kv, 1)), np.zeros((H_kv, d))])
    g = np.concatenate([plain64.turn(f64(u).swapaxes(1, 2), p, fr, interleaved, -1.0) for u in up[:2]]
                       + [f64(up[2]).swapaxes(1, 2)], 2)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    amp = r * (1.5 * np.abs(w * g).max(-1, keepdims=True)
               + 2 * np.abs(n) * np.abs(w * g * n).mean(-1, keepdims=True))
    check(dqkv[:, :, :H + H_kv], rx[:, :, :H + H_kv], amp[:, :, :H + H_kv] + 1e-30, qkv.dtype, "dqkv")
    assert torch.equal(dqkv[:, :, H + H_kv:], up[2].transpose(1, 2))
    # a weight's gradient is a float32 sum of B N heads products, each off by 2e-6 of the pair's
    # amplitude, added in runs of at most 64 and then in trees: under 1e-5 of the sum of magnitudes
    for got, rr, sl in ((dw[0], rqw, slice(0, H)), (dw[1], rkw, slice(H, H + H_kv))):
        mag = (np.abs(n[:, :, sl]) * 1.5 * np.abs(g[:, :, sl]).max(-1, keepdims=True)).sum((0, 1, 2))
        assert (np.abs(f64(got) - rr) <= 1e-5 * mag).all()


def run_both(B, N, H, H_kv, d, dtype, rot, interleaved, pos, weights=True, eps=1e-6, scale=1.0):
    qkv, qw, kw, up = make(B, N, H, H_kv, d, dtype, scale=scale)
    t = qkv.dtype
    if not weights:
        qw = kw = None
    f = fa.rope_frequencies(rot) if rot else None
    out = outputs(B, N, H, H_kv, d, t)
    fa.fa_qk_norm_rope(qkv, qw, kw, pos, f, *out, eps, interleaved)
    dqkv = torch.full_like(qkv, float("nan"))
    dw = [torch.full((d,), float("nan"), device="cuda") for _ in range(2)]
    ws = torch.empty(fa.fa_qk_norm_rope_bwd_workspace_size(B, H, H_kv, N, d), dtype=torch.uint8, device="cuda")
    fa.fa_qk_norm_rope_bwd(qkv, qw, kw, pos, f, *up, dqkv, *dw, ws, eps, interleaved)
    check_status()

    compare_forward(qkv, out, qw, kw, pos, f, eps, interleaved)
    compare_grad(qkv, up, dqkv, dw, qw, kw, pos, f, eps, interleaved)
    return qkv, out, dqkv, dw


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 96), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_and_rotations(dtype, d, rot, interleaved):
    B, N, H, H_kv = 2, 37, 6, 2
    pos = torch.arange(B * N, dtype=torch.int32, device="cuda").view(B, N) * 3
    run_both(B, N, H, H_kv, d, dtype, rot, interleaved, pos)


@pytest.mark.parametrize("B,N,H,H_kv", [(1, 1, 1, 1), (1, 1, 32, 8), (5, 1, 7, 7), (1, 3, 5, 3), (3, 131, 3, 1),
                                        (2, 1025, 9, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_sizes_and_head_counts(B, N, H, H_kv, d):
    run_both(B, N, H, H_kv, d, "bf16", d, False, None)


def test_no_weights_and_zero_rows():
    B, N, H, H_kv, d = 1, 9, 4, 2, 64
    run_both(B, N, H, H_kv, d, "f32", d, False, None, weights=False)
    qkv = torch.zeros((B, N, H + 2 * H_kv, d), device="cuda")
    out = outputs(B, N, H, H_kv, d, torch.float32)
    fa.fa_qk_norm_rope(qkv, None, None, None, fa.rope_frequencies(d), *out, 1e-6)
    assert all((x == 0).all() for x in out)


@pytest.mark.parametrize("scale", [1e-6, 1e6])
def test_small_and_large_values(scale):
    run_both(1, 17, 3, 1, 128, "f32", 128, False, None, scale=scale)


def test_far_and_negative_positions():
    # the angle's error is 2^-25 half turns at any position: also at the ends of int32
    pos = torch.tensor([[0, 1, -1, 1 << 20, (1 << 20) + 1, 123456789, -123456789, 2 ** 31 - 1, -2 ** 31]],
                       dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        run_both(1, pos.shape[1], 2, 1, 128, "f32", 128, interleaved, pos)


def test_gradient_without_weight_gradients_and_repeatable():
    B, N, H, H_kv, d = 3, 700, 8, 2, 128
    qkv, _, dqkv, dw = run_both(B, N, H, H_kv, d, "bf16", d, False, None)
    _, qw, kw, up = make(B, N, H, H_kv, d, "bf16")
    again, dw2 = torch.empty_like(dqkv), [torch.empty_like(x) for x in dw]
    f = fa.rope_frequencies(d)
    ws = torch.empty(fa.fa_qk_norm_rope_bwd_workspace_size(B, H, H_kv, N, d), dtype=torch.uint8, device="cuda")
    fa.fa_qk_norm_rope_bwd(qkv, qw, kw, None, f, *up, again, *dw2, ws, 1e-6)
    assert torch.equal(again, dqkv) and torch.equal(dw2[0], dw[0]) and torch.equal(dw2[1], dw[1])
    again.fill_(float("nan"))
    fa.fa_qk_norm_rope_bwd(qkv, qw, kw, None, f, *up, again, None, None, None, 1e-6)
    assert torch.equal(again, dqkv)
    k_only = torch.full_like(dw[0], float("nan"))
    fa.fa_qk_norm_rope_bwd(qkv, qw, kw, None, f, *up, again, None, k_only, ws, 1e-6)
    assert torch.equal(k_only, dw[1])


def test_binding_refuses_wrong_tensors():
    qkv, qw, kw, _ = make(1, 4, 2, 1, 64, "bf16")
    out = outputs(1, 4, 2, 1, 64, torch.bfloat16)
    f = fa.rope_frequencies(64)
    for args in ((qkv[:, :, :3].contiguous(), qw, kw, None, f, *out), (qkv.transpose(0, 1), qw, kw, None, f, *out),
                 (qkv, qw.double(), kw, None, f, *out), (qkv, qw, kw, torch.zeros((1, 4), device="cuda"), f, *out),
                 (qkv, qw, kw, None, f.cuda(), *out), (qkv, qw, kw, None, f.float(), *out),
                 (qkv.half(), qw, kw, None, f, *out), (qkv.cpu(), qw, kw, None, f, *out),
                 (qkv, qw, kw, None, f, out[0].float(), out[1], out[2])):
        with pytest.raises(ValueError):
            fa.fa_qk_norm_rope(*args, 1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (3, 1), (6, 3), (5, 6)])
def test_without_eps(H, H_kv, d, dtype):
    # heads that do not fill a warp's pass: what has no head adds nothing to the weight gradients
    run_both(2, 19, H, H_kv, d, dtype, d, False, None, eps=0.0)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("exponent", [-57, 57])
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_magnitudes_at_the_ends_of_the_range(exponent, eps, dtype, d):
    # rows whose largest value is near 2^-56 or 2^59: squares and their sums stay within float32
    run_both(1, 9, 3, 1, d, dtype, d, False, None, eps=eps, scale=2.0 ** exponent)


def exact_angles(positions, inv_freq):
    """positions [n] times frequencies [p], less whole turns, from integers: float64 in [-pi, pi]."""
    bits = 1400
    atan = lambda x: sum((-1) ** k * ((1 << bits) // ((2 * k + 1) * x ** (2 * k + 1))) for k in range(bits // 4))  # noqa: E731
    two_pi = 8 * (4 * atan(5) - atan(239))  # Machin; off by under 2^-1380
    out = np.empty((len(positions), len(inv_freq)))
    for i, t in enumerate(positions):
        for j, f in enumerate(inv_freq):
            m, e = Fraction(float(f)).as_integer_ratio()
            rest = (int(t) * m << bits) // e % two_pi
            out[i, j] = float(Fraction(rest - (two_pi if 2 * rest > two_pi else 0), 1 << bits))
    return out


@pytest.mark.parametrize("interleaved", [False, True])
def test_frequencies_of_any_size_at_far_positions(interleaved):
    # the angle's error does not grow with the frequency
    B, H, H_kv, d, eps = 1, 2, 1, 64, 1e-6
    positions = [0, 1, -1, 7, 4099, -123456789, 2 ** 31 - 1, -2 ** 31]
    N = len(positions)
    f = torch.tensor([2.0 ** 64, -2.0 ** 64, 1.7e19, 1e12 + 0.1, 2.0 ** 53 + 2, 1e6, -54321.098, 4096.0, 1234.5, 100.0, 10.0,
                      2 * np.pi, 3.7, 1.0, 0.99, -0.5, 1 / 3, 0.1, 1e-3, 1e-6, 1e-9, -1e-12, 1e-20, 1e-30, 5e-324, -5e-324,
                      0.0, 2.2250738585072014e-308, 50.0, 20.0, 5.0, 2.0], dtype=torch.float64)
    qkv, qw, kw, up = make(B, N, H, H_kv, d, "f32")
    pos = torch.tensor([positions], dtype=torch.int32, device="cuda")
    out = outputs(B, N, H, H_kv, d, torch.float32)
    fa.fa_qk_norm_rope(qkv, qw, kw, pos, f, *out, eps, interleaved)
    dqkv = torch.full_like(qkv, float("nan"))
    fa.fa_qk_norm_rope_bwd(qkv, qw, kw, pos, f, *up, dqkv, None, None, None, eps, interleaved)
    check_status()
    angles = exact_angles(positions, f.numpy())
    for n in range(N):
        one = lambda x: x[:, :, n:n + 1].contiguous()  # noqa: E731
        x, first = qkv[:, n:n + 1].contiguous(), torch.ones((1, 1), dtype=torch.int32)
        angle = torch.from_numpy(angles[n].copy())
        compare_forward(x, [one(t) for t in out], qw, kw, first, angle, eps, interleaved)
        ref = plain64.norm_rope_grad(f64(x), H, H_kv, f64(qw), f64(kw), first.numpy(), angle.numpy(), eps, interleaved,
                                     *(f64(one(u)) for u in up))[0]
        g = np.concatenate([f64(one(u)).swapaxes(1, 2) for u in up[:2]], 2)
        w = np.concatenate([np.tile(f64(qw), (H, 1)), np.tile(f64(kw), (H_kv, 1))])
        r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + eps)[:, :, :H + H_kv]
        xn = f64(x)[:, :, :H + H_kv] * r
        # as in compare_grad, with |g| before its turn: a turn makes it sqrt(2) larger at most
        top = 2.2 * np.abs(w).max() * np.abs(g).max(-1, keepdims=True)
        check(dqkv[:, n:n + 1, :H + H_kv], ref[:, :, :H + H_kv], r * (top + 2 * np.abs(xn) * top * np.abs(xn).mean(-1, keepdims=True)),
              torch.float32, "dqkv")
