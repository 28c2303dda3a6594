"""Differential attention layer in float64: rotary positions, the learned
difference weight, differential attention of a packed stream (forward and
analytic backward) and the norm of each head's row.

Plain restatements of the definitions in include/nsp.h, written row by row or
document by document with numpy; they share no code with the CUDA path.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

# pi to 60 digits: whole turns are taken off far positions exactly
_TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")


def rope_positions(cu, n, start=0):
    """Position of stream rows start .. start + n - 1 in their documents; -1
    for a row past the last document."""
    cu = np.asarray(cu, np.int64)
    rows = np.arange(start, start + n)
    doc = np.searchsorted(cu, rows, side="right") - 1
    pos = rows - cu[np.minimum(doc, len(cu) - 1)]
    return np.where(rows < cu[-1], pos, -1)


def rope_angles(positions, freqs):
    """Angles in (-2 pi, 2 pi) congruent to position x frequency, by exact
    rational arithmetic."""
    out = np.empty((len(positions), len(freqs)))
    for i, p in enumerate(positions):
        for j, f in enumerate(freqs):
            a = Fraction(int(p)) * Fraction(float(f))
            out[i, j] = float(a - _TWO_PI * int(a / _TWO_PI))
    return out


def rope(x, angles, rot, interleaved=False, mscale=1.0, inverse=False):
    """x [T, H, d] rotated by angles [T, rot / 2]."""
    y = np.array(x, np.float64)
    c, s = mscale * np.cos(angles)[:, None], mscale * np.sin(angles)[:, None]
    if inverse:
        s = -s
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def diff_lambda(q1, k1, q2, k2, heads, init):
    lam = np.exp((q1 * k1).sum(-1)) - np.exp((q2 * k2).sum(-1)) + init
    return np.broadcast_to(lam, (heads,)).copy()


def diff_lambda_bwd(dlam, q1, k1, q2, k2):
    g = np.asarray(dlam, np.float64).reshape(-1)
    if q1.shape[0] == 1:
        g = g.sum(keepdims=True)
    e1, e2 = np.exp((q1 * k1).sum(-1)) * g, np.exp((q2 * k2).sum(-1)) * g
    return e1[:, None] * k1, e1[:, None] * q1, -e2[:, None] * k2, -e2[:, None] * q2


def _documents(cu, T):
    cu = np.asarray(cu, np.int64)
    for b in range(len(cu) - 1):
        lo, hi = min(cu[b], T), min(cu[b + 1], T)
        if hi > lo:
            yield slice(int(lo), int(hi))


def diff_maps(q, k, cu, scale, causal):
    """Both maps' probabilities [2, Hq, T, T] and lse [Hq, 2, T] of a stream."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    P = np.zeros((2, Hq, T, T))
    lse = np.full((Hq, 2, T), -np.inf)
    for h in range(Hq):
        g = h // (Hq // Hkv)
        for m in range(2):
            cols = slice(m * d // 2, (m + 1) * d // 2)
            for doc in _documents(cu, T):
                x = scale * q[doc, h, cols] @ k[doc, g, cols].T
                if causal:
                    x = np.where(np.tril(np.ones(x.shape, bool)), x, -np.inf)
                top = x.max(-1, keepdims=True)
                e = np.exp(x - top)
                z = e.sum(-1, keepdims=True)
                P[m, h, doc, doc] = e / z
                lse[h, m, doc] = (top + np.log(z))[:, 0]
    return P, lse


def diff_attn_fwd(q, k, v, lam, cu, scale, causal=True):
    """out, out2 [T, Hq, d] and lse [Hq, 2, T]; lam [Hq, 1] or [Hq, T]."""
    T, Hq, d = q.shape
    P, lse = diff_maps(q, k, cu, scale, causal)
    V = np.repeat(v, Hq // k.shape[1], axis=1)
    o1, o2 = (np.einsum("hij,jhd->ihd", P[m], V) for m in range(2))
    w = np.broadcast_to(lam, (Hq, T)).T[:, :, None]
    return o1 - w * o2, o2, lse


def diff_attn_bwd(q, k, v, lam, dout, cu, scale, causal=True):
    """dq, dk, dv and dlam (lam's shape)."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    P, _ = diff_maps(q, k, cu, scale, causal)
    w = np.broadcast_to(lam, (Hq, T))
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dlam = np.zeros((Hq, T))
    for h in range(Hq):
        g = h // G
        dp = dout[:, h] @ v[:, g].T
        dv[:, g] += (P[0, h] - w[h][:, None] * P[1, h]).T @ dout[:, h]
        dlam[h] = -(P[1, h] * dp).sum(-1)
        for m, sign in ((0, np.ones(T)), (1, -w[h])):
            cols = slice(m * d // 2, (m + 1) * d // 2)
            ds = sign[:, None] * P[m, h] * (dp - (P[m, h] * dp).sum(-1, keepdims=True))
            dq[:, h, cols] = scale * ds @ k[:, g, cols]
            dk[:, g, cols] += scale * ds.T @ q[:, h, cols]
    return dq, dk, dv, dlam if np.shape(lam)[-1] == T and T > 1 else dlam.sum(-1, keepdims=True)


def head_norm(x, weight=None, gate=None, eps=1e-6, scale=1.0):
    y = scale * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight
    if gate is not None:
        y = y / (1 + np.exp(-gate))
    return y


def head_norm_bwd(x, dy, weight=None, gate=None, eps=1e-6, scale=1.0):
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    w = 1.0 if weight is None else weight
    s = 1.0 if gate is None else 1 / (1 + np.exp(-gate))
    u = scale * dy * w * s
    dx = r * (u - n * (u * n).mean(-1, keepdims=True))
    dw = None if weight is None else (scale * dy * n * s).sum((0, 1))
    dg = None if gate is None else scale * dy * w * n * s * (1 - s)
    return dx, dw, dg
