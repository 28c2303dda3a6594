"""Differential attention layer on the GPU against the float64 oracle.

Tolerances are derived, element by element, from roundings: u is half a step
of the output's type (bf16 2^-8, float32 2^-24, relative to the value), e =
2^-24 that of the float32 arithmetic in between.  A product with bf16
probabilities or dS (the tensor-core path rounds both once) is off by at most
u times the sum of the terms' magnitudes, plus the float32 terms.
"""
import numpy as np
import pytest
import torch

import oracle
import oracle.layer as L

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def half_step(dt):
    return torch.finfo(dt).eps / 2


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def randn(seed, *shape, dt=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dt).cuda()


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def assert_within(got, ref, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - tol
    i = np.unravel_index(int(np.argmax(over)), over.shape)
    assert over[i] <= 0, f"{what} at {i}: {got[i]} against {ref[i]}, off by more than {np.broadcast_to(tol, ref.shape)[i]}"


# ----------------------------------------------------------------------------- rotary positions

def check_rope(got, x, angles, rot, inter, m, inverse, dt, what, angle_err=0.0):
    x = f64(x) if isinstance(x, torch.Tensor) else x
    ref = L.rope(x, angles, rot, inter, m, inverse)
    # sine and cosine: 2 ulp of sincospi, the angle's float32 rounding (pi e) and
    # its 2^-32 turns; the factor, two products and the sum: 16 e in all of m (|a| + |b|)
    a = np.abs(x)
    pair = a.copy()
    ia = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
    ib = ia + 1 if inter else ia + rot // 2
    pair[..., ia] = pair[..., ib] = a[..., ia] + a[..., ib]
    pair[..., rot:] = 0
    assert_within(got, ref, half_step(dt) * np.abs(ref) + (16 * E + angle_err) * abs(m) * pair, what)
    if rot < x.shape[-1]:
        np.testing.assert_array_equal(f64(got)[..., rot:], x[..., rot:])


LENS = [3, 0, 1, 70, 0, 26]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("d,rot,hq,hkv", [(128, 128, 8, 2), (64, 32, 3, 1), (96, 96, 2, 2), (128, 64, 33, 4),
                                          (64, 64, 1, 1), (80, 20, 2, 1), (7, 6, 3, 2)])
def test_rope(nsp, dt, inter, inverse, d, rot, hq, hkv):
    T = sum(LENS)
    q, k = randn(1, T, hq, d, dt=dt), randn(2, T, hkv, d, dt=dt)
    fr = nsp.rope_freqs(rot, base=500.0, device="cuda")
    cu = cu_of(LENS)
    a = L.rope_angles(L.rope_positions(cu.cpu().numpy(), T), fr.cpu().numpy())
    qo, ko = nsp.rope(q, k, cu, fr, layout="interleaved" if inter else "half", mscale=1.25,
                      inverse=inverse)
    check_rope(qo, q, a, rot, inter, 1.25, inverse, dt, "q")
    check_rope(ko, k, a, rot, inter, 1.25, inverse, dt, "k")


def test_rope_far_positions(nsp):
    """Explicit positions to the end of int32, negative ones too: the angle
    error is that of the float64 frequency (2^-52 turns a turn) alone."""
    pos = torch.tensor([0, 1, 399999, 2 ** 30 + 7, 2 ** 31 - 1, -1, -2 ** 31], dtype=torch.int32, device="cuda")
    fr = nsp.rope_freqs(64, base=1e6, device="cuda")
    x = randn(3, 7, 2, 64, dt=F32)
    got, none = nsp.rope(x, None, None, fr, positions=pos)
    assert none is None
    err = np.abs(pos.cpu().numpy().astype(np.float64))[:, None] * fr.cpu().numpy() * 2.0 ** -51
    err = np.concatenate([err, err], -1)[:, None]
    check_rope(got, x, L.rope_angles(pos.cpu().numpy(), fr.cpu().numpy()), 64, False, 1.0, False, F32,
               "far", err)


@pytest.mark.parametrize("d", [64, 6])
@pytest.mark.parametrize("sign", [1, -1])
def test_rope_angle(nsp, d, sign):
    """Sine and cosine themselves, of pairs (1, 0): off by the angle's 2^-26 turns and
    2^-52 of the whole angle, whichever way a frequency turns, and by 4 e (2 ulp of
    sincospi)."""
    pos = np.array([0, 1, 399999, 2 ** 30 + 7, 2 ** 31 - 1, -5, -2 ** 31], np.int64)
    fr = sign * np.logspace(-8, 0.5, d // 2)
    x = torch.zeros((len(pos), 1, d), device="cuda")
    x[..., :d // 2] = 1
    got, _ = nsp.rope(x, None, None, torch.from_numpy(fr).cuda(), positions=torch.from_numpy(pos).int().cuda())
    a = L.rope_angles(pos, fr)
    tol = 4 * E + 2 * np.pi * 2.0 ** -26 + np.abs(pos[:, None] * fr) * 2.0 ** -52
    ref = np.concatenate([np.cos(a), np.sin(a)], -1)[:, None]
    assert_within(got, ref, np.concatenate([tol, tol], -1)[:, None], "angle")


@pytest.mark.parametrize("inter", [False, True])
def test_rope_fused_views_in_place_groups(nsp, inter):
    """Columns of a fused projection in, packed, head-grouped and in-place out;
    every form the same bits; the columns in between untouched."""
    T, hq, hkv, d = sum(LENS), 8, 2, 128
    lay = "interleaved" if inter else "half"
    cu, fr = cu_of(LENS), nsp.rope_freqs(d, device="cuda")
    qkv = randn(4, T, hq + 2 * hkv, d)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    ref_q, ref_k = nsp.rope(q.contiguous(), k.contiguous(), cu, fr, layout=lay)
    got_q, got_k = nsp.rope(q, k, cu, fr, layout=lay)
    assert torch.equal(got_q, ref_q) and torch.equal(got_k, ref_k)
    for p in (2, 4):
        gq, _ = nsp.rope(q, k, cu, fr, layout=lay, q_groups=p)
        assert torch.equal(gq, nsp.seq2head(ref_q, p))
        back, _ = nsp.rope(gq, ref_k, cu, fr, layout=lay, q_groups=p, inverse=True)
        plain, _ = nsp.rope(ref_q, ref_k, cu, fr, layout=lay, inverse=True)
        assert torch.equal(back, plain)
    before = qkv.clone()
    nsp.rope(q, k, cu, fr, layout=lay, out=(q, k))
    assert torch.equal(qkv[:, :hq], ref_q) and torch.equal(qkv[:, hq:hq + hkv], ref_k)
    assert torch.equal(qkv[:, hq + hkv:], before[:, hq + hkv:])


def test_rope_odd_addresses(nsp):
    """Strides and addresses that are no whole 16 bytes give the same bits."""
    T, h, d = 29, 3, 64
    cu, fr = cu_of([29]), nsp.rope_freqs(d, device="cuda")
    x = randn(5, T, h, d)
    ref, _ = nsp.rope(x, None, cu, fr)
    wide = torch.zeros((T, h * d + 3), dtype=BF16, device="cuda")
    view = wide[:, 1:1 + h * d].unflatten(1, (h, d))
    view.copy_(x)
    got, _ = nsp.rope(view, None, cu, fr)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("d,rot,inter", [(1024, 8, True), (1024, 8, False), (1024, 1024, True),
                                         (1024, 1024, False), (516, 4, True)])
def test_rope_wide_heads(nsp, d, rot, inter):
    """More 16-byte pieces in a head than half a block has threads."""
    T, h = 9, 3
    fr = nsp.rope_freqs(rot, base=500.0, device="cuda")
    cu, x = cu_of([5, 4]), randn(30, T, h, d, dt=F32)
    got, _ = nsp.rope(x, None, cu, fr, layout="interleaved" if inter else "half")
    a = L.rope_angles(L.rope_positions(cu.cpu().numpy(), T), fr.cpu().numpy())
    check_rope(got, x, a, rot, inter, 1.0, False, F32, "wide")


@pytest.mark.parametrize("T,h,hkv,groups", [(1, 36, 4, 4), (2, 40, 1, 8), (20011, 39, 13, 3),
                                            (700, 64, 64, 1)])
def test_rope_parts_of_heads(nsp, T, h, hkv, groups):
    """However a token's heads are split over the blocks, within a tensor, over
    two and over head groups: the bits of every head alone."""
    cu, fr = cu_of([T]), nsp.rope_freqs(64, device="cuda")
    q, k = randn(31, T, h, 64), randn(32, T, hkv, 64)
    whole_q, whole_k = nsp.rope(q, k, cu, fr, q_groups=groups)
    if groups > 1:
        whole_q = whole_q.permute(1, 0, 2, 3).reshape(T, h, 64)
    for i in (0, h // groups - 1, h // groups % h, h // 2, h - 1):
        assert torch.equal(whole_q[:, i:i + 1], nsp.rope(q[:, i:i + 1], None, cu, fr)[0]), i
    for i in (0, hkv - 1):
        assert torch.equal(whole_k[:, i:i + 1], nsp.rope(k[:, i:i + 1], None, cu, fr)[0]), i


def test_rope_rows_behind_the_last_document_and_shards(nsp):
    T, h, d = 100, 4, 64
    cu, fr = cu_of([40, 30]), nsp.rope_freqs(d, device="cuda")
    x = randn(6, T, h, d)
    out = torch.full_like(x, 7.0)
    nsp.rope(x, None, cu, fr, out=(out, None))
    assert (out[70:] == 7).all()
    ref, _ = nsp.rope(x[:70].contiguous(), None, cu, fr)
    assert torch.equal(out[:70], ref)
    for s, e in ((0, 33), (33, 70)):                 # a sequence shard's own rows
        part, _ = nsp.rope(x[s:e], None, cu, fr, start=s)
        assert torch.equal(part, ref[s:e])
    one, _ = nsp.rope(x[:1], None, cu, fr)
    assert torch.equal(one, ref[:1])
    none, _ = nsp.rope(x[:0], None, cu, fr)
    assert none.shape == (0, h, d)


# ----------------------------------------------------------------------------- difference weight

@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("n,heads,dl", [(1, 1, 1), (1, 37, 64), (16, 16, 64), (5, 5, 33), (3, 3, 300)])
def test_diff_lambda(nsp, dt, n, heads, dl):
    vec = [randn(10 + i, n, dl, dt=dt, scale=0.1) for i in range(4)]
    ref = [f64(x) for x in vec]
    lam = nsp.diff_lambda(*vec, heads=heads, lambda_init=0.8)
    # a dot product of dl terms and exp (2 ulp): the exponentials are off by
    # (dl + 4) e of themselves at most
    e1, e2 = (np.exp((ref[2 * i] * ref[2 * i + 1]).sum(-1)) for i in range(2))
    dot = sum(np.abs(ref[2 * i] * ref[2 * i + 1]).sum(-1) for i in range(2)) * dl + 6
    want = L.diff_lambda(*ref, heads, 0.8)
    assert_within(lam, want, half_step(dt) * np.abs(want) + E * dot * (e1 + e2 + 1), "lambda")
    g = randn(20, heads, dt=dt)
    grads = nsp.diff_lambda_bwd(g, *vec)
    gs = np.abs(f64(g)).sum() if n == 1 else np.abs(f64(g))
    for i, (a, b) in enumerate(zip(grads, L.diff_lambda_bwd(f64(g), *ref))):
        other = np.abs(ref[i ^ 1]) * ((e1, e2)[i // 2] * gs * (dot + heads + 4))[:, None]
        assert_within(a, b, half_step(dt) * np.abs(b) + E * other, f"gradient {i}")
        assert a.shape == vec[i].shape


# ----------------------------------------------------------------------------- head norm

@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("gate,weight", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("tokens,heads,d", [(1, 1, 128), (37, 3, 64), (129, 5, 128), (300, 2, 512), (11, 7, 8),
                                            (50, 4, 96), (1000, 16, 256)])
def test_head_norm(nsp, dt, gate, weight, tokens, heads, d):
    x, dy = randn(30, tokens, heads, d, dt=dt), randn(31, tokens, heads, d, dt=dt)
    g = randn(32, tokens, heads, d, dt=dt) if gate else None
    w = randn(33, d, dt=dt) if weight else None
    kw = dict(eps=1e-5, scale=0.2)
    rx, rdy = f64(x), f64(dy)
    rw, rg = (None if t is None else f64(t) for t in (w, g))
    y = nsp.head_norm(x, w, g, **kw)
    ref = L.head_norm(rx, rw, rg, 1e-5, 0.2)
    # the sum of d squares (16 partial sums and 5 shuffles at most: 40 e), rsqrt
    # 2 ulp, sigmoid (exp 2 + 1.2 |g| ulp, sum, quotient) and four products
    c = (64 + 4 * (np.abs(rg).max() if gate else 0)) * E
    assert_within(y, ref, (half_step(dt) + c) * np.abs(ref), "y")
    dx, dw, dg = nsp.head_norm_bwd(x, dy, w, g, **kw)
    rdx, rdw, rdg = L.head_norm_bwd(rx, rdy, rw, rg, 1e-5, 0.2)
    r = 1 / np.sqrt((rx * rx).mean(-1, keepdims=True) + 1e-5)
    s = 1.0 if rg is None else 1 / (1 + np.exp(-rg))
    u = np.abs(0.2 * rdy * (1.0 if rw is None else rw) * s)
    n = np.abs(rx * r)
    terms = r * (u + n * (u * n).mean(-1, keepdims=True))
    assert_within(dx, rdx, half_step(dt) * np.abs(rdx) + c * terms, "dx")
    if weight:
        # a column's terms pass through at most 32 + 16 + 76 + 8 sums here
        mag = (np.abs(0.2 * rdy * rx * r) * s).sum((0, 1))
        assert_within(dw, rdw, half_step(dt) * np.abs(rdw) + (c + 132 * E) * mag, "dw")
    else:
        assert dw is None
    if gate:
        # 1 - sigmoid of a large gate keeps only sigmoid's absolute error
        big = np.abs(0.2 * rdy * rx * r * (1.0 if rw is None else rw)) * s
        assert_within(dg, rdg, half_step(dt) * np.abs(rdg) + c * big, "dgate")
    else:
        assert dg is None


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 512])
def test_head_norm_far_gates(nsp, dt, d):
    """Gates far from zero, on both sides: sigmoid and 1 - sigmoid are exact to
    float32's roundings of their own values, however small they are (and bf16's exp to
    2 + 1.2 |g| ulp more)."""
    T, H = 65, 3
    x, dy, w = randn(34, T, H, d, dt=dt), randn(35, T, H, d, dt=dt), randn(36, d, dt=dt)
    g = (torch.linspace(-60, 60, T * H * d).view(T, H, d)).to(dt).cuda()
    kw = dict(eps=1e-5, scale=0.2)
    rx, rdy, rw, rg = (f64(t) for t in (x, dy, w, g))
    # as in the test above: 64 e for the norm and the products, exp 2 ulp, the sum,
    # the reciprocal and the product of the rest: 8 e
    c = (72 + (4 * np.abs(rg) if dt == BF16 else 0)) * E
    y = nsp.head_norm(x, w, g, **kw)
    ref = L.head_norm(rx, rw, rg, 1e-5, 0.2)
    assert_within(y, ref, (half_step(dt) + c) * np.abs(ref), "y")
    dg = nsp.head_norm_bwd(x, dy, w, g, **kw)[2]
    # (the oracle's 1 - s cancels for a large gate as well: sigmoid(-g) does not)
    s, rest = 1 / (1 + np.exp(-rg)), 1 / (1 + np.exp(rg))
    ref = 0.2 * rdy * rw * rx / np.sqrt((rx * rx).mean(-1, keepdims=True) + 1e-5) * s * rest
    assert_within(dg, ref, (half_step(dt) + 2 * c) * np.abs(ref), "dgate")


def test_head_norm_infinite_gates(nsp):
    """A gate of minus infinity closes, one of plus infinity opens; neither has a gradient,
    and a NaN stays one."""
    x = randn(37, 5, 2, 64, dt=F32)
    dy, g = randn(38, 5, 2, 64, dt=F32), torch.zeros_like(x)
    g[0], g[1], g[2, 0, 0] = float("-inf"), float("inf"), float("nan")
    y, (dx, _, dg) = nsp.head_norm(x, gate=g), nsp.head_norm_bwd(x, dy, gate=g)
    assert (y[0] == 0).all() and torch.equal(y[1], nsp.head_norm(x)[1])
    assert (dg[:2] == 0).all() and (dx[0] == 0).all() and torch.isfinite(dx[1]).all()
    assert torch.isnan(y[2, 0, 0]) and torch.isnan(dg[2, 0, 0]) and torch.isfinite(y[3:]).all()


def test_head_norm_views_and_edges(nsp):
    """Columns of a fused tensor; zero rows and extreme gates; no rows; results
    the same bits twice."""
    qkv = randn(40, 65, 10, 64)
    x, w = qkv[:, 2:6], randn(41, 64)
    dy, g = randn(42, 65, 4, 64), randn(43, 65, 4, 64)
    assert torch.equal(nsp.head_norm(x, w, g), nsp.head_norm(x.contiguous(), w, g))
    for a, b in zip(nsp.head_norm_bwd(x, dy, w, g), nsp.head_norm_bwd(x.contiguous(), dy, w, g)):
        assert torch.equal(a, b)
    z = torch.zeros(3, 2, 64, device="cuda")
    far = torch.full_like(z, 200.0)
    assert (nsp.head_norm(z) == 0).all() and (nsp.head_norm(z + 1, gate=-far) == 0).all()
    np.testing.assert_allclose(f64(nsp.head_norm(z + 1, gate=far, eps=1e-12)), 1, rtol=1e-6)
    dx, _, dg = nsp.head_norm_bwd(z + 1, z + 1, gate=far)
    assert torch.isfinite(dx).all() and (dg == 0).all()
    e = x[:0]
    assert nsp.head_norm(e, w).shape == (0, 4, 64)
    dx, dw, _ = nsp.head_norm_bwd(e, dy[:0], w)
    assert dx.shape == (0, 4, 64) and (dw == 0).all()


# ----------------------------------------------------------------------------- differential attention

def diff_inputs(seed, lens, hq, hkv, d, dt, tokens, scale=1.0):
    T = sum(lens)
    g = torch.Generator().manual_seed(seed)
    lam = (torch.rand((hq, T if tokens else 1), generator=g) * 1.2 - 0.3).to(dt).cuda()
    return (randn(seed + 1, T, hq, d, dt=dt, scale=scale), randn(seed + 2, T, hkv, d, dt=dt, scale=scale),
            randn(seed + 3, T, hkv, d, dt=dt), lam, randn(seed + 4, T, hq, d, dt=dt), cu_of(lens))


def diff_bounds(q, k, v, lam, do, cu, scale, causal, dt):
    """The oracle's results and how far each may be off, element by element."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    P, lse = L.diff_maps(q, k, cu, scale, causal)
    out, out2, _ = L.diff_attn_fwd(q, k, v, lam, cu, scale, causal)
    w = np.broadcast_to(lam, (Hq, T))
    V, K = np.repeat(v, G, 1), np.repeat(k, G, 1)
    h = half_step(dt)
    u = h if dt == BF16 else 0.0                      # one rounding of P and of dS
    # a score is off by d/2 + 2 float32 roundings of its terms' magnitudes; exp
    # turns that into a relative error of P
    mag = np.zeros((Hq, 2, T))
    for m in range(2):
        c = slice(m * d // 2, (m + 1) * d // 2)
        s = scale * np.einsum("ihc,jhc->hij", np.abs(q[..., c]), np.abs(K[..., c]))
        mag[:, m] = np.where(P[m] > 0, s, 0).max(-1)
    rel = E * ((d // 2 + 2) * mag + 64)               # of P, per row
    tol_lse = rel + 4 * E * np.abs(lse)
    A1, A2 = (np.einsum("hij,jhd->ihd", P[m], np.abs(V)) for m in range(2))
    r1, r2 = rel[:, 0].T[..., None], rel[:, 1].T[..., None]
    lw = np.abs(w).T[..., None]
    # a row's sum of exponentials adds as much again, float32 sums over the keys e each
    acc = T * E
    tol_o2 = (u + 2 * r2 + acc) * A2 + h * np.abs(out2)
    tol_out = (u + 2 * r1 + acc) * A1 + lw * (u + 2 * r2 + acc) * A2 + h * np.abs(out)
    if do is None:
        return (out, out2, lse), (tol_out, tol_o2, tol_lse)
    grads = L.diff_attn_bwd(q, k, v, lam, do, cu, scale, causal)
    ado = np.abs(do)
    d2_err = (ado * (tol_o2 + d * E * np.abs(out2))).sum(-1).T                # [Hq, T]
    d1_err = (ado * (tol_out + d * E * np.abs(out))).sum(-1).T + np.abs(w) * d2_err
    tq, tk, tv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for hh in range(Hq):
        g = hh // G
        dp = do[:, hh] @ v[:, g].T
        dp_err = d * E * ado[:, hh] @ np.abs(v[:, g]).T
        pc = (u + acc) * (P[0, hh] + np.abs(w[hh])[:, None] * P[1, hh])
        pc += rel[hh, 0][:, None] * P[0, hh] + (rel[hh, 1] * np.abs(w[hh]))[:, None] * P[1, hh]
        tv[:, g] += pc.T @ ado[:, hh]
        for m, sign, derr in ((0, np.ones(T), d1_err[hh]), (1, np.abs(w[hh]), d2_err[hh])):
            c = slice(m * d // 2, (m + 1) * d // 2)
            diff = np.abs(dp - (P[m, hh] * dp).sum(-1, keepdims=True))
            # P's own error, P and dS rounded (u each), delta's and dP's errors
            es = sign[:, None] * P[m, hh] * ((2 * u + 2 * rel[hh, m][:, None] + acc) * diff
                                             + derr[:, None] + dp_err)
            tq[:, hh, c] += scale * es @ np.abs(k[:, g, c])
            tk[:, g, c] += scale * es.T @ np.abs(q[:, hh, c])
    tl = d2_err + T * E * np.abs(out2 * do).sum(-1).T
    if grads[3].shape[1] != T or T == 1:
        tl = tl.sum(-1, keepdims=True)
    tols = [t + h * np.abs(g) for t, g in zip((tq, tk, tv, tl), grads)]
    return (out, out2, lse) + tuple(grads), (tol_out, tol_o2, tol_lse) + tuple(tols)


DIFF_CASES = [
    ([1], 1, 1, 128), ([1], 2, 1, 64), ([5, 0, 1, 130], 4, 2, 128), ([128, 129], 2, 2, 64),
    ([127, 1, 128, 2], 6, 2, 128), ([33] * 9, 5, 1, 64), ([300], 3, 3, 128), ([40, 0, 0, 333, 27], 4, 1, 128),
]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tokens", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,d", DIFF_CASES)
def test_diff_attention(nsp, dt, causal, tokens, lens, hq, hkv, d):
    q, k, v, lam, do, cu = diff_inputs(50, lens, hq, hkv, d, dt, tokens)
    scale = (d // 2) ** -0.5
    ref, tol = diff_bounds(*(f64(t) for t in (q, k, v, lam, do)), cu.cpu().numpy(), scale, causal, dt)
    out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, causal=causal, save=True)
    assert torch.equal(out, nsp.diff_attn_fwd(q, k, v, lam, cu, causal=causal))
    grads = nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu, causal=causal)
    for name, a, b, t in zip(("out", "out2", "lse", "dq", "dk", "dv", "dlam"),
                             (out, out2, lse) + grads, ref, tol):
        assert_within(a, b, t, name)
        # as a whole within the library's bar for gradients, where roundings do
        # not outweigh the result: one token alone has P = 1 and dP = delta, so
        # its dq and dk are zero and what comes out is delta's rounding (within
        # the elements' tolerance above, which no multiple of zero can be)
        if np.linalg.norm(b) > np.linalg.norm(t):
            assert np.linalg.norm(f64(a) - b) <= 1e-2 * np.linalg.norm(b), name
    for a, b in zip(grads, nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu, causal=causal)):
        assert torch.equal(a, b)                      # one fixed order of sums


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,hq,hkv,d", [
    ([1], 8, 1, 64), ([17, 1, 0, 140, 3, 30], 8, 1, 128), ([9, 8, 7, 6, 5, 4, 3, 2, 1], 16, 2, 128),
    ([130, 200], 16, 1, 64), ([70, 77], 6, 1, 128), ([250, 7], 24, 2, 64), ([16, 16, 15, 1, 81, 127], 8, 1, 64),
])
def test_diff_attention_heads_of_a_group(nsp, lens, hq, hkv, d, causal):
    """Groups whose heads go into one query tile, 2, 4 or 8 at a time, with documents
    that begin and end inside its few tokens."""
    test_diff_attention(nsp, BF16, causal, True, lens, hq, hkv, d)


def lambda_grad_bounds(q, k, v, lam, do, cu, scale, causal, dt):
    """-sum_j P_2 dP of every token and head [Hq, T], how far each may be off in
    float32, and how far their sum over the tokens may be, by roundings that are
    independent of one another (eight standard deviations): a score is a sum of d/2
    products and dP one of d, each off by e times the square root of their number
    and the terms' magnitudes; exp and the row's lse are off by 16 e and 8 e |lse|, the
    same for a whole row; T sums of a row add e of its terms' magnitudes each."""
    T, Hq, d = q.shape
    P, lse = L.diff_maps(q, k, cu, scale, causal)
    val, var, common = (np.zeros((Hq, T)) for _ in range(3))
    for h in range(Hq):
        g = h // (Hq // k.shape[1])
        p, dp = P[1, h], do[:, h] @ v[:, g].T
        mag = scale * np.abs(q[:, h, d // 2:]) @ np.abs(k[:, g, d // 2:]).T
        each = (p * dp * E * (np.sqrt(d // 2 + 2) * mag + 8)) ** 2
        each += (p * E * np.sqrt(d) * (np.abs(do[:, h]) @ np.abs(v[:, g]).T)) ** 2
        val[h] = -(p * dp).sum(-1)
        var[h] = each.sum(-1) + T * (E * np.abs(p * dp).sum(-1)) ** 2
        common[h] = E * (16 + 8 * np.abs(np.where(np.isfinite(lse[h, 1]), lse[h, 1], 0))) * np.abs(val[h])
    one = 8 * np.sqrt(var) + common
    total = 8 * np.sqrt(var.sum(-1)) + (common + 32 * E * np.abs(val)).sum(-1)
    h = half_step(dt)
    return val, one + h * np.abs(val), total + h * np.abs(val.sum(-1))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("lens,hq,d", [([300], 4, 128), ([170, 131, 40], 4, 128), ([600], 3, 64), ([33] * 9, 8, 128)])
def test_diff_attention_lambda_gradient_cancels(nsp, lens, hq, d, dt):
    """A head's gradient of lambda is a sum over the tokens whose terms cancel: with
    either type it is as exact as float32 arithmetic and one rounding to the type."""
    cu = cu_of(lens)
    for seed in range(300, 380, 10):
        q, k, v, lam, do, _ = diff_inputs(seed, lens, hq, 1, d, dt, False)
        ref = [f64(t) for t in (q, k, v, lam, do)]
        val, one, total = lambda_grad_bounds(*ref, cu.cpu().numpy(), (d // 2) ** -0.5, True, dt)
        want = val.sum(-1)
        assert (np.abs(want) > 2 * total).mean() > 0.9            # (zeros would not pass)
        out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
        got = nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu)[3]
        assert_within(got, want[:, None], total[:, None], f"dlam {seed}")
        if dt == BF16:
            # and of each token
            many = lam.expand(hq, sum(lens)).contiguous()
            got = nsp.diff_attn_bwd(q, k, v, many, out, out2, do, lse, cu)[3]
            assert_within(got, val, one, f"dlam of tokens {seed}")


@pytest.mark.parametrize("lens", [[2500], [300, 1, 900, 0, 60]])
def test_diff_attention_split_key_tiles(nsp, lens):
    """Few key tiles: each is split in parts, whose float32 shares lie in a workspace
    with no more than its documented 16-byte alignment."""
    hq, hkv, d, T = 8, 1, 128, sum(lens)
    q, k, v, lam, do, cu = diff_inputs(160, lens, hq, hkv, d, BF16, False)
    out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
    n = nsp.load().nsp_diff_attn_bwd_workspace_size(T, hq, hkv, d, nsp.NSP_BF16)
    ws = torch.empty(n + 16, dtype=torch.uint8, device="cuda")[16:]
    assert ws.data_ptr() % 32 == 16
    grads = nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu, workspace=ws)
    ref = L.diff_attn_bwd(*(f64(t) for t in (q, k, v, lam, do)), cu.cpu().numpy(), (d // 2) ** -0.5, True)
    for name, a, b in zip(("dq", "dk", "dv", "dlam"), grads, ref):
        assert np.linalg.norm(f64(a) - b) <= 1e-2 * np.linalg.norm(b), name
    for a, b in zip(grads, nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu)):
        assert torch.equal(a, b)


def test_diff_attention_split_captured_and_on_two_streams(nsp):
    """The split backward replayed from a graph on new values, and two of them in
    flight at once."""
    lens = [1200, 77]
    ins = [diff_inputs(163 + i, lens, 8, 2, 64, BF16, True) for i in range(2)]

    def step(x):
        q, k, v, lam, do, cu = x
        out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
        return (out,) + nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu)

    want = [step(x) for x in ins]
    held = tuple(t.clone() for t in ins[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(held)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held)
    for i in (1, 0, 1):
        for a, b in zip(held, ins[i]):
            a.copy_(b)
        graph.replay()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    streams, both = [torch.cuda.Stream() for _ in ins], [None, None]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                both[i] = step(ins[i])
    torch.cuda.synchronize()
    for a, b in zip(want, both):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_diff_attention_heads_many_documents(nsp):
    """Every head of a packed group alone (one head a group, whole tiles of tokens):
    the same values to the rounding of sums in another order of keys."""
    rng = np.random.default_rng(11)
    lens = [int(n) for n in rng.choice([0, 1, 2, 5, 16, 40, 131], size=400)]
    q, k, v, lam, do, cu = diff_inputs(145, lens, 8, 1, 128, BF16, True)
    out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
    dq, dk, dv, dlam = nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu)
    kv = [np.zeros(k.shape) for _ in range(2)]
    for h in range(8):
        one = [t[:, h:h + 1].contiguous() for t in (q, do)]
        o, o2, ls = nsp.diff_attn_fwd(one[0], k, v, lam[h:h + 1].clone(), cu, save=True)
        g = nsp.diff_attn_bwd(one[0], k, v, lam[h:h + 1].clone(), o, o2, one[1], ls, cu)
        # P, dS and the outputs are rounded to bf16 on both sides, sums of bf16 products in float32
        for a, b in ((out[:, h], o[:, 0]), (out2[:, h], o2[:, 0]), (dq[:, h], g[0][:, 0]), (dlam[h], g[3][0])):
            a, b = f64(a), f64(b)
            assert np.linalg.norm(a - b) <= 4 * half_step(BF16) * np.linalg.norm(b)
        np.testing.assert_allclose(f64(lse[h]), f64(ls[0]), rtol=0, atol=2e-5)
        for t, x in zip(kv, g[1:3]):
            t += f64(x)
    for a, b in zip((dk, dv), kv):                    # eight rounded shares against one rounded sum
        a = f64(a)
        assert np.linalg.norm(a - b) <= 4 * half_step(BF16) * np.linalg.norm(b)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_diff_attention_growing_scores(nsp, dt):
    """Scores that climb along the document (the running maximum is replaced
    again and again) and lambda of both signs."""
    lens, d = [700], 128
    q, k, v, lam, do, cu = diff_inputs(60, lens, 2, 1, d, dt, True)
    ramp = torch.linspace(0, 6, 700, device="cuda")[:, None]
    k[:, :, 0] = (k[:, :, 0].float() + 4 * ramp).to(dt)
    k[:, :, 64] = (k[:, :, 64].float() - 4 * ramp).to(dt)
    q[:, :, 0] = (q[:, :, 0].float().abs() + 1).to(dt)
    q[:, :, 64] = (q[:, :, 64].float().abs() + 1).to(dt)
    ref, tol = diff_bounds(*(f64(t) for t in (q, k, v, lam, do)), [0, 700], 0.125, True, dt)
    out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
    grads = nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu)
    for name, a, b, t in zip(("out", "out2", "lse", "dq", "dk", "dv", "dlam"),
                             (out, out2, lse) + grads, ref, tol):
        assert_within(a, b, t, name)


def test_diff_attention_equals_attention(nsp):
    """lambda = 0 leaves the first map: ordinary attention of 64-column heads
    on v's column halves."""
    lens = [200, 3, 57]
    q, k, v, lam, do, cu = diff_inputs(70, lens, 4, 2, 128, BF16, False)
    out = nsp.diff_attn_fwd(q, k, v, torch.zeros_like(lam), cu)
    for half in range(2):
        o, _ = nsp.attn_fwd(q[..., :64].contiguous(), k[..., :64].contiguous(),
                            v[..., 64 * half:64 * half + 64].contiguous(), cu, scale=0.125)
        # both round P (u each) and the result
        assert (f64(out[..., 64 * half:64 * half + 64]) - f64(o)).max() <= 4 * 2.0 ** -8 * 4


@pytest.mark.parametrize("causal", [True, False])
def test_diff_attention_equals_attention_on_both_sides(nsp, causal):
    """The same, neither larger nor smaller than the roundings allow: both round P (u of
    the terms each) and the result, element by element."""
    lens, scale = [200, 3, 57], 0.125
    q, k, v, lam, do, cu = diff_inputs(70, lens, 4, 2, 128, BF16, False)
    lam = torch.zeros_like(lam)
    out = f64(nsp.diff_attn_fwd(q, k, v, lam, cu, causal=causal))
    (ref, _, _), (tol, _, _) = diff_bounds(*(f64(t) for t in (q, k, v, lam)), None, cu.cpu().numpy(), scale, causal,
                                           BF16)
    assert np.linalg.norm(tol) < 0.05 * np.linalg.norm(ref)
    for half in range(2):
        c = slice(64 * half, 64 * half + 64)
        o, _ = nsp.attn_fwd(q[..., :64].contiguous(), k[..., :64].contiguous(), v[..., c].contiguous(), cu,
                            scale=scale, causal=causal)
        assert_within(out[..., c], f64(o), 2 * tol[..., c], "out")


def test_diff_attention_differences(nsp):
    """Directional differences of the float32 forward: the step h leaves an
    h^2 / 6 third-derivative term (third derivatives of this loss along a unit
    direction are below its norm), the two losses e of their terms' sum."""
    lens = [40, 0, 77]
    q, k, v, lam, do, cu = diff_inputs(80, lens, 4, 2, 64, F32, True)
    out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
    grads = nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu)
    for i, g in enumerate(grads):
        dirn = randn(90 + i, *g.shape, dt=F32)
        dirn /= dirn.norm()
        step, f = 1e-2, []
        for e in (step, -step):
            x = [q, k, v, lam]
            x[i] = x[i] + e * dirn
            o = nsp.diff_attn_fwd(*x, cu)
            f.append((o.double() * do.double()).sum().item())
        noise = 64 * E * (out.double() * do.double()).norm().item() / step
        want = (g.double() * dirn.double()).sum().item()
        assert abs((f[0] - f[1]) / (2 * step) - want) <= noise + step ** 2 * g.norm().item(), i


def test_diff_attention_status(nsp):
    """cu_seqlens shorter than the stream, or decreasing: recorded, nothing written."""
    q, k, v, lam, do, _ = diff_inputs(100, [100], 2, 1, 64, BF16, False)
    good = cu_of([100])
    _, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, good, save=True)
    for bad in ([0, 60], [0, 70, 50, 100], [1, 100]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        ws = torch.empty(nsp.load().nsp_diff_attn_fwd_workspace_size(100), dtype=torch.uint8, device="cuda")
        nsp.diff_attn_fwd(q, k, v, lam, cu, workspace=ws)
        assert nsp.nsp_status_query(ws) == nsp.NSP_ERR_INVALID
        ws = torch.empty(nsp.load().nsp_diff_attn_bwd_workspace_size(100, 2, 1, 64, nsp.NSP_BF16), dtype=torch.uint8,
                         device="cuda")
        nsp.diff_attn_bwd(q, k, v, lam, q, out2, do, lse, cu, workspace=ws)
        assert nsp.nsp_status_query(ws) == nsp.NSP_ERR_INVALID
    # a longer cu_seqlens: the stream is the start of it
    cu = torch.tensor([0, 30, 170], dtype=torch.int32, device="cuda")
    a = nsp.diff_attn_fwd(q, k, v, lam, cu, causal=False)
    assert torch.equal(a, nsp.diff_attn_fwd(q, k, v, lam, cu_of([30, 70]), causal=False))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("T,hq,hkv,d", [(100, 2, 1, 64), (333, 8, 1, 128), (1000, 8, 2, 64), (129, 5, 5, 128),
                                        (20000, 8, 1, 64)])
@pytest.mark.parametrize("past", [1, 1000, 2 ** 31 - 1])
def test_diff_attention_stream_ends_inside_a_document(nsp, dt, causal, T, hq, hkv, d, past):
    """cu_seqlens longer than the stream: its start, bit for bit, with key tiles whole
    and in parts, heads of a group together and alone, and nothing written around the
    workspace."""
    if dt == F32 and T > 1000:
        T = 1500
    first = T // 3
    cut = cu_of([first, T - first])
    long = torch.tensor([0, first, min(T + past, 2 ** 31 - 1), 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    q, k, v, lam, do, _ = diff_inputs(190, [T], hq, hkv, d, dt, False)
    n = nsp.load().nsp_diff_attn_bwd_workspace_size(T, hq, hkv, d, nsp._DTYPES[dt])
    got = []
    for cu in (cut, long):
        out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, causal=causal, save=True)
        buf = torch.full((n + 2 * 65536,), 0xA5, dtype=torch.uint8, device="cuda")
        ws = buf[65536:65536 + n]
        grads = nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu, causal=causal, workspace=ws)
        assert nsp.nsp_status_query(ws) == nsp.NSP_OK
        assert (buf[:65536] == 0xA5).all() and (buf[65536 + n:] == 0xA5).all()
        got.append((out, out2, lse) + grads)
    for a, b in zip(*got):
        assert torch.equal(a, b)
    if T <= 333:
        scale = (d // 2) ** -0.5
        ref, tol = diff_bounds(*(f64(t) for t in (q, k, v, lam, do)), cut.cpu().numpy(), scale, causal, dt)
        for name, a, b, t in zip(("out", "out2", "lse", "dq", "dk", "dv", "dlam"), got[1], ref, tol):
            assert_within(a, b, t, name)


def test_diff_attention_empty_stream(nsp):
    q, k, v, lam, do, _ = diff_inputs(110, [0], 2, 1, 64, BF16, False)
    cu = cu_of([0])
    out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
    assert out.shape == (0, 2, 64) and lse.shape == (2, 2, 0)
    dq, dk, dv, dl = nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu)
    assert dq.shape == (0, 2, 64) and (dl == 0).all()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_diff_attention_guard_zones(nsp, dt):
    """Nothing around the outputs and the workspaces is written."""
    lens, hq, hkv, d = [70, 1, 130], 4, 2, 128
    q, k, v, lam, do, cu = diff_inputs(120, lens, hq, hkv, d, dt, False)
    T, lib = sum(lens), nsp.load()
    pad = 4096

    def guarded(nbytes):
        buf = torch.full((pad + (nbytes + 255) // 256 * 256 + pad,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[pad:pad + nbytes]

    def check(buf, n):
        assert (buf[:pad] == 0xA5).all() and (buf[pad + n:] == 0xA5).all()

    es = q.element_size()
    sizes = [T * hq * d * es, T * hq * d * es, hq * 2 * T * 4, lib.nsp_diff_attn_fwd_workspace_size(T),
             T * hq * d * es, T * hkv * d * es, T * hkv * d * es, hq * es,
             lib.nsp_diff_attn_bwd_workspace_size(T, hq, hkv, d, nsp._DTYPES[dt])]
    bufs = [guarded(n) for n in sizes]
    p = [b[1].data_ptr() for b in bufs]
    io, st = nsp._DTYPES[dt], torch.cuda.current_stream().cuda_stream
    assert lib.nsp_diff_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), lam.data_ptr(), 1, cu.data_ptr(),
                                 len(lens), T, hq, hkv, d, 0.125, 1, io, p[0], p[1], p[2], p[3], sizes[3],
                                 st) == 0
    assert lib.nsp_diff_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), lam.data_ptr(), 1, p[0], p[1],
                                 do.data_ptr(), p[2], cu.data_ptr(), len(lens), T, hq, hkv, d, 0.125, 1, io,
                                 p[4], p[5], p[6], p[7], p[8], sizes[8], st) == 0
    torch.cuda.synchronize()
    for (buf, _), n in zip(bufs, sizes):
        check(buf, n)


def test_diff_attention_grids(nsp, monkeypatch):
    """1, 7 and 152 persistent blocks: the same bits (each item is computed whole
    by one block, each sum has one order)."""
    q, k, v, lam, do, cu = diff_inputs(130, [300, 1, 0, 77, 129, 500], 4, 2, 128, BF16, True)

    def step():
        out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
        return (out, out2, lse) + nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu)

    monkeypatch.setenv("NSP_PERSISTENT_CTAS", "152")
    want = step()
    for n in ("1", "7"):
        monkeypatch.setenv("NSP_PERSISTENT_CTAS", n)
        for a, b in zip(want, step()):
            assert torch.equal(a, b)


def test_diff_attention_many_documents(nsp):
    """More documents than one look of the document search (32 starts a warp,
    empty ones among them) against one document at a time."""
    rng = np.random.default_rng(7)
    lens = [int(n) for n in rng.choice([0, 0, 1, 1, 2, 3, 40], size=700)]
    q, k, v, lam, do, cu = diff_inputs(140, lens, 2, 1, 64, BF16, False)
    out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
    dq, dk, dv, _ = nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu)
    ref, tol = diff_bounds(*(f64(t) for t in (q, k, v, lam, do)), cu.cpu().numpy(), 32 ** -0.5, True, BF16)
    for name, a, i in (("out", out, 0), ("out2", out2, 1), ("lse", lse, 2), ("dq", dq, 3), ("dk", dk, 4),
                       ("dv", dv, 5)):
        assert_within(a, ref[i], tol[i], name)


def test_diff_attention_masked_neighbours(nsp):
    """Infinite and NaN keys of one document leave its neighbours in the tile as
    they are (scores outside a row's document are dropped, not multiplied)."""
    lens = [50, 30, 60]
    q, k, v, lam, do, cu = diff_inputs(150, lens, 2, 1, 128, BF16, False)
    want = nsp.diff_attn_fwd(q, k, v, lam, cu)
    k[50:65] = float("nan")
    k[65:80] = float("inf")
    got = nsp.diff_attn_fwd(q, k, v, lam, cu)
    assert torch.equal(got[:50], want[:50]) and torch.equal(got[80:], want[80:])
    assert torch.isnan(got[50:80]).any()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (8, 1, 64), (3, 3, 64)])
def test_diff_attention_non_finite_queries_and_keys(nsp, dt, hq, hkv, d):
    """A NaN query is its own row's, a NaN or infinite key those rows' that see it: rows
    before it in its document and all other documents keep their bits.  Whatever a stream
    holds, the call ends without an error and leaves nothing behind for the next."""
    lens = [150, 300, 40]
    q, k, v, lam, do, cu = diff_inputs(155, lens, hq, hkv, d, dt, True)
    n = nsp.load().nsp_diff_attn_bwd_workspace_size(sum(lens), hq, hkv, d, nsp._DTYPES[dt])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step(x):
        out, out2, lse = nsp.diff_attn_fwd(*x, lam, cu, save=True, workspace=ws)
        assert nsp.nsp_status_query(ws) == nsp.NSP_OK
        grads = nsp.diff_attn_bwd(*x, lam, out, out2, do, lse, cu, workspace=ws)
        assert nsp.nsp_status_query(ws) == nsp.NSP_OK
        return (out, out2, lse) + grads

    want = step((q, k, v))
    keys, queries = k.clone(), q.clone()
    keys[290], keys[300, :, ::2] = float("nan"), float("inf")
    queries[200] = float("nan")
    out, out2, lse = step((queries, keys, v))[:3]
    same = [r for r in range(sum(lens)) if r != 200 and not 290 <= r < 450]
    for a, b in zip((out, out2, lse.permute(2, 0, 1)), (want[0], want[1], want[2].permute(2, 0, 1))):
        assert torch.equal(a[same], b[same])
        assert torch.isnan(a[200]).all() and torch.isnan(a[290:450]).all()
    bad = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    assert torch.isnan(step(bad)[0]).all()
    for a, b in zip(step((q, k, v)), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("backward", [False, True])
def test_diff_attention_timeout(nsp, backward):
    """A wait that runs out is recorded, the context stays usable and the same
    workspace works again."""
    lens = [700, 300]
    q, k, v, lam, do, cu = diff_inputs(160, lens, 8, 2, 128, BF16, False)
    T, lib = sum(lens), nsp.load()
    out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
    n = (lib.nsp_diff_attn_bwd_workspace_size(T, 8, 2, 128, nsp.NSP_BF16) if backward
         else lib.nsp_diff_attn_fwd_workspace_size(T))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call():
        if backward:
            return nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu, workspace=ws)
        return nsp.diff_attn_fwd(q, k, v, lam, cu, save=True, workspace=ws)

    want = call()
    torch.cuda.synchronize()
    old = nsp.nsp_set_wait_timeout_cycles(100)
    try:
        call()
        assert nsp.nsp_status_query(ws) == nsp.NSP_ERR_TIMEOUT
    finally:
        nsp.nsp_set_wait_timeout_cycles(old)
    got = call()
    assert nsp.nsp_status_query(ws) == nsp.NSP_OK
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_two_streams_at_once(nsp):
    """Two steps in flight at the same time on their own workspaces."""
    ins = [diff_inputs(170 + 10 * i, [900, 33, 600], 4, 2, 128, BF16, False) for i in range(2)]

    def step(x):
        q, k, v, lam, do, cu = x
        out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
        return (out, nsp.head_norm(out)) + nsp.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, cu)

    want = [step(x) for x in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step(ins[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_offsets_past_32_bits(nsp):
    """More than 2^31 elements in q: the last documents equal the same documents
    alone (they start on a tile's edge, so the same tiles are summed)."""
    d, hq, n = 128, 256, 66048                        # 2.16e9 elements
    tail = 256
    q = torch.empty((n, hq, d), dtype=BF16, device="cuda")
    q[:n - tail] = 0.5
    q[n - tail:] = randn(180, tail, hq, d)
    cu = torch.arange(0, n + 1, 64, dtype=torch.int32, device="cuda")
    cu2 = torch.arange(0, tail + 1, 64, dtype=torch.int32, device="cuda")
    qt = q[n - tail:].clone()
    assert q.numel() > 2 ** 31
    fr = nsp.rope_freqs(d, device="cuda")
    r, _ = nsp.rope(q, None, cu, fr)
    assert torch.equal(r[n - tail:], nsp.rope(qt, None, cu2, fr)[0])
    del r
    y = nsp.head_norm(q)
    assert torch.equal(y[n - tail:], nsp.head_norm(qt))
    del y
    k = randn(181, n, 1, d)
    v = randn(182, n, 1, d)
    lam = torch.full((hq, 1), 0.5, dtype=BF16, device="cuda")
    out, out2, lse = nsp.diff_attn_fwd(q, k, v, lam, cu, save=True)
    o, o2, l = nsp.diff_attn_fwd(qt, k[n - tail:].contiguous(), v[n - tail:].contiguous(), lam, cu2, save=True)
    assert torch.equal(out[n - tail:], o) and torch.equal(out2[n - tail:], o2)
    assert torch.equal(lse[:, :, n - tail:], l)
    dq, dk, dv, _ = nsp.diff_attn_bwd(q, k, v, lam, out, out2, q, lse, cu)
    eq, ek, ev, _ = nsp.diff_attn_bwd(qt, k[n - tail:].contiguous(), v[n - tail:].contiguous(), lam, o, o2,
                                      qt, l, cu2)
    assert torch.equal(dq[n - tail:], eq) and torch.equal(dk[n - tail:], ek) and torch.equal(dv[n - tail:], ev)
    dx, _, _ = nsp.head_norm_bwd(q, dq)
    assert torch.equal(dx[n - tail:], nsp.head_norm_bwd(qt, eq)[0])


# ----------------------------------------------------------------------------- together

def layer_forward(nsp, x, cu, fr):
    q, k = nsp.rope(x["q"], x["k"], cu, fr)
    lam = nsp.diff_lambda(*x["vec"], heads=q.shape[1], lambda_init=0.5)
    out, out2, lse = nsp.diff_attn_fwd(q, k, x["v"], lam, cu, save=True)
    return q, k, lam, out, out2, lse, nsp.head_norm(out, x["w"], x["gate"], scale=0.5)


def layer_backward(nsp, x, saved, dy, cu, fr):
    q, k, lam, out, out2, lse, _ = saved
    dout, dw, dg = nsp.head_norm_bwd(out, dy, x["w"], x["gate"], scale=0.5)
    dq, dk, dv, dl = nsp.diff_attn_bwd(q, k, x["v"], lam, out, out2, dout, lse, cu)
    dvec = nsp.diff_lambda_bwd(dl, *x["vec"])
    dq, dk = nsp.rope(dq, dk, cu, fr, inverse=True)
    return (dq, dk, dv, dw, dg) + dvec


def layer_inputs(lens, hq, hkv, d, dt):
    T = sum(lens)
    qkv = randn(200, T, hq + 2 * hkv, d, dt=dt)
    return {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:].contiguous(),
            "vec": [randn(201 + i, hq, d // 2, dt=dt, scale=0.1) for i in range(4)],
            "w": randn(210, d, dt=dt), "gate": randn(211, T, hq, d, dt=dt)}


def test_layer_forward_and_gradients(nsp):
    """The whole layer in float32 against the oracle's chain: the gradients
    pass five operators, each within a few e of its terms; 2e-5 of each
    tensor's norm leaves a factor of ten over the measured float32 chains of
    the separate tests."""
    lens, hq, hkv, d = [50, 0, 1, 90], 4, 2, 64
    x, cu = layer_inputs(lens, hq, hkv, d, F32), cu_of(lens)
    fr = nsp.rope_freqs(d, device="cuda")
    saved = layer_forward(nsp, x, cu, fr)
    dy = randn(220, sum(lens), hq, d, dt=F32)
    got = (saved[-1],) + layer_backward(nsp, x, saved, dy, cu, fr)

    c = cu.cpu().numpy()
    a = L.rope_angles(L.rope_positions(c, sum(lens)), fr.cpu().numpy())
    rq, rk = (L.rope(f64(x[n]), a, d) for n in ("q", "k"))
    vec, v, w, g = [f64(t) for t in x["vec"]], f64(x["v"]), f64(x["w"]), f64(x["gate"])
    lam = L.diff_lambda(*vec, hq, 0.5)[:, None]
    s = (d // 2) ** -0.5
    out, _, _ = L.diff_attn_fwd(rq, rk, v, lam, c, s)
    y = L.head_norm(out, w, g, 1e-6, 0.5)
    dout, dw, dg = L.head_norm_bwd(out, f64(dy), w, g, 1e-6, 0.5)
    dq, dk, dv, dl = L.diff_attn_bwd(rq, rk, v, lam, dout, c, s)
    ref = (y, L.rope(dq, a, d, inverse=True), L.rope(dk, a, d, inverse=True), dv, dw, dg) + \
        L.diff_lambda_bwd(dl, *vec)
    for i, (p, r) in enumerate(zip(got, ref)):
        assert np.linalg.norm(f64(p) - r) <= 2e-5 * np.linalg.norm(r), i


@pytest.mark.parametrize("dt", [BF16, F32])
def test_layer_captured_and_on_another_stream(nsp, dt):
    """Captured into a graph and replayed on new inputs, and run on a side
    stream: the same bits as eager calls."""
    lens, hq, hkv, d = [64, 3, 150], 4, 2, 128
    x, cu = layer_inputs(lens, hq, hkv, d, dt), cu_of(lens)
    fr = nsp.rope_freqs(d, device="cuda")
    dy = randn(230, sum(lens), hq, d, dt=dt)

    def step():
        saved = layer_forward(nsp, x, cu, fr)
        return (saved[-1],) + layer_backward(nsp, x, saved, dy, cu, fr)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    y = nsp.head_norm(x["gate"], x["w"], stream=side)
    side.synchronize()
    for a, b in zip(want, other):
        assert torch.equal(a, b)
    assert torch.equal(y, nsp.head_norm(x["gate"], x["w"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    x["v"].mul_(-0.5)
    x["gate"].neg_()
    want = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_layer_refusals_on_the_gpu(nsp):
    q, k, v, lam, do, cu = diff_inputs(240, [20], 4, 2, 64, BF16, False)
    with pytest.raises(ValueError):
        nsp.diff_attn_fwd(q.transpose(0, 1), k, v, lam, cu)
    with pytest.raises(ValueError):
        nsp.diff_attn_fwd(q, k, v[:-1], lam, cu)
    with pytest.raises(TypeError):
        nsp.diff_attn_fwd(q, k.float(), v, lam, cu)
    with pytest.raises(TypeError):
        nsp.diff_attn_fwd(q, k, v, lam, cu.long())
    with pytest.raises(ValueError):
        nsp.diff_attn_fwd(q, k, v, lam[:2], cu)
    with pytest.raises(ValueError):
        nsp.diff_attn_fwd(q, k, v, lam.cpu(), cu)
    with pytest.raises(nsp.NspError):
        nsp.diff_attn_fwd(q, k, v, lam, cu, scale=-1.0)
    with pytest.raises(nsp.NspError):
        nsp.diff_attn_fwd(q, k, v, lam, cu, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    fr = nsp.rope_freqs(64, device="cuda")
    with pytest.raises(ValueError):
        nsp.rope(q, k, None, fr)
    with pytest.raises(ValueError):
        nsp.rope(q, k, cu, fr, q_groups=3)
    with pytest.raises(TypeError):
        nsp.rope(q, k, cu, fr.float())
    with pytest.raises(ValueError):
        nsp.rope(q.transpose(1, 2), k, cu, fr)
    with pytest.raises(nsp.NspError):                 # overlapping, not in place
        nsp.rope(q[:-1], None, cu, fr, out=(q[1:], None))
    with pytest.raises(nsp.NspError):
        nsp.head_norm(q, eps=0.0)
    with pytest.raises(ValueError):
        nsp.head_norm(q, weight=lam[:, 0])
