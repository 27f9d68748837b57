"""Gradients of attention to another sequence's keys against differences of the loss sum(o dO), in float64.

Each gradient g is taken along a direction with the signs of the float64 gradient r, so that the slope there is
sum |r| |direction| and what g lacks, has too much of or has in the wrong place changes it by its whole size:
of a direction without regard to r the terms cancel to 1 or 2% of that sum.  The tolerance comes from the
float64 form alone: that of test_gpu_cross for each entry (P and dS in bfloat16, delta from the o that the
forward rounded, each gradient's own rounding), weighted by the direction, and 1e-6 of the slope for the differences
(a step of 1e-4: the second-order term of two-sided differences is 1e-8 of the third derivative)."""
import numpy as np

import plain64

NAMES = ("dq", "dk", "dv")


def pairs(q, k, lengths):
    share, G = q.shape[0] // k.shape[0], q.shape[1] // k.shape[1]
    for b in range(q.shape[0]):
        for h in range(q.shape[1]):
            yield (b, h), (b // share, h // G), lengths[b // share]


def loss(q, k, v, do, lengths, scale):
    total = 0.0
    for qh, kh, n in pairs(q, k, lengths):
        seen = np.ones((q.shape[2], n), dtype=bool)
        total += (plain64.attention(q[qh], k[kh][:n], v[kh][:n], scale, seen)[0] * do[qh]).sum()
    return total


def reference(q, k, v, do, lengths, scale, few=24):
    """Float64 gradients and the tolerance of each entry."""
    ref, tol = ([np.zeros_like(t) for t in (q, k, v)] for _ in range(2))
    for qh, kh, n in pairs(q, k, lengths):
        Q, K, V, dO, seen = q[qh], k[kh][:n], v[kh][:n], do[qh], np.ones((q.shape[2], n), dtype=bool)
        o, _, P = plain64.attention(Q, K, V, scale, seen)
        gq, gk, gv = plain64.attention_grad(Q, K, V, dO, scale, seen)
        ref[0][qh] = gq
        ref[1][kh][:n] += gk
        ref[2][kh][:n] += gv
        t = 1e-5 * (1 + np.abs(scale) * np.abs(Q @ K.T).max(initial=0))
        A, dP = P @ np.abs(V), dO @ V.T
        if n <= few:
            d_delta = (t + 1e-6) * (np.abs(dO) * A).sum(-1, keepdims=True)
        else:
            d_delta = (np.abs(dO) * (2.0 ** -8 * (A + np.abs(o)) + t * A)).sum(-1, keepdims=True)
        delta = (dO * o).sum(-1, keepdims=True)
        d_dS = P * (d_delta + 1e-6 * (np.abs(dO) @ np.abs(V).T) + (2.0 ** -8 + t) * (np.abs(dP - delta) + d_delta))
        tol[0][qh] = np.abs(scale) * d_dS @ np.abs(K)
        tol[1][kh][:n] += np.abs(scale) * d_dS.T @ np.abs(Q)
        tol[2][kh][:n] += (2.0 ** -8 + t) * P.T @ np.abs(dO)
    return ref, [t + 2.0 ** -8 * np.abs(r) for t, r in zip(tol, ref)]


class Differences:
    """Slopes of the loss along one direction for each of q, k and v."""

    def __init__(self, q, k, v, do, lengths, scale, seed=0, eps=1e-4):
        base = [q, k, v]
        self.ref, tol = reference(q, k, v, do, lengths, scale)
        rng = np.random.default_rng(seed)
        self.directions = [np.sign(r) * np.abs(rng.standard_normal(r.shape)) for r in self.ref]
        self.slopes, self.tolerances = [], []
        for i, u in enumerate(self.directions):
            sides = [loss(*[t + sign * eps * u if j == i else t for j, t in enumerate(base)], do, lengths, scale) for sign in (1, -1)]
            slope = (sides[0] - sides[1]) / (2 * eps)
            self.slopes.append(slope)
            self.tolerances.append((tol[i] * np.abs(u)).sum() + 1e-6 * abs(slope))

    def off(self, i, grad):
        """How far gradient i is from the difference, in tolerances."""
        return abs((grad * self.directions[i]).sum() - self.slopes[i]) / self.tolerances[i]
