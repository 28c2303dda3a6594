"""Post-training step on the GPU against the float64 oracle.

Tolerances are derived, element by element, from roundings: u is half a step
of the output's type (bf16 2^-8, float32 2^-24, relative to the value), E =
2^-24 that of the float32 arithmetic in between.
"""
import numpy as np
import pytest
import torch

import oracle.layer as L
import oracle.step as S

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
    got = f64(got) if isinstance(got, torch.Tensor) else np.asarray(got)
    ref = np.asarray(ref)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if got.size == 0:
        return
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - tol
    i = np.unravel_index(int(np.argmax(over)), over.shape)
    assert over[i] <= 0, f"{what} at {i}: {got[i]} against {ref[i]}, off by more than {np.broadcast_to(tol, ref.shape)[i]}"


# ----------------------------------------------------------------------------- head norm with rotation

LENS = [3, 0, 1, 70, 0, 26]


def pair_sum(a, rot, inter, m):
    """m (|a| + |b|) of each rotated pair in both its columns, |a| of the others."""
    out = np.abs(a)
    ia = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
    ib = ia + 1 if inter else ia + rot // 2
    both = abs(m) * (out[..., ia] + out[..., ib])
    out[..., ia] = out[..., ib] = both
    return out


def check_qk(x, w, dy, y, dx, dw, ang, rot, inter, m, eps, dt):
    x, dy = f64(x), f64(dy)
    w = None if w is None else f64(w)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n, ww = x * r, (1.0 if w is None else w)
    # the norm: a sum of d squares (at most 40 sums on the way), rsqrt 2 ulp, products: 64 E;
    # the rotation: 2 ulp of sine and cosine, its angle (pi E), products and sum: 16 E
    ref = S.qk_norm_rope(x, w, ang, rot, inter, m, eps)
    assert_within(y, ref, half_step(dt) * np.abs(ref) + 84 * E * pair_sum(n * ww, rot, inter, m), "y")
    rdx, rdw = S.qk_norm_rope_bwd(x, w, dy, ang, rot, inter, m, eps)
    z = pair_sum(dy, rot, inter, m)
    u = np.abs(ww) * z
    # z 16 E, the mean of u n another 64 E (d terms, 40 sums on the way), n 64 E
    terms = r * (u + np.abs(n) * (u * np.abs(n)).mean(-1, keepdims=True))
    assert_within(dx, rdx, half_step(dt) * np.abs(rdx) + 160 * E * terms, "dx")
    if w is None:
        assert dw is None
    else:
        # a column's terms pass through at most 132 sums at these sizes
        assert_within(dw, rdw, half_step(dt) * np.abs(rdw) + 232 * E * (np.abs(n) * z).sum((0, 1)), "dw")


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("d,rot,hq,hkv", [(128, 128, 8, 2), (64, 32, 3, 1), (96, 96, 2, 2), (128, 64, 33, 4),
                                          (256, 256, 4, 1), (512, 512, 2, 1), (80, 20, 2, 1), (7, 6, 3, 2),
                                          (96, 48, 2, 1), (24, 16, 5, 1), (40, 8, 2, 2), (512, 256, 3, 1)])
def test_qk_norm_rope(nsp, dt, inter, weight, d, rot, hq, hkv):
    T = sum(LENS)
    q, k = randn(1, T, hq, d, dt=dt), randn(2, T, hkv, d, dt=dt, scale=3.0)
    gq, gk = randn(3, T, hq, d, dt=dt), randn(4, T, hkv, d, dt=dt)
    wq, wk = (randn(5 + i, d, dt=dt) if weight else None for i in range(2))
    fr, cu = nsp.rope_freqs(rot, base=500.0, device="cuda"), cu_of(LENS)
    ang = L.rope_angles(L.rope_positions(cu.cpu().numpy(), T), fr.cpu().numpy())
    kw = dict(layout="interleaved" if inter else "half", mscale=1.25, eps=1e-5)
    yq, yk = nsp.qk_norm_rope(q, k, cu, fr, wq, wk, **kw)
    dq, dk, dwq, dwk = nsp.qk_norm_rope_bwd(q, k, gq, gk, cu, fr, wq, wk, **kw)
    check_qk(q, wq, gq, yq, dq, dwq, ang, rot, inter, 1.25, 1e-5, dt)
    check_qk(k, wk, gk, yk, dk, dwk, ang, rot, inter, 1.25, 1e-5, dt)


@pytest.mark.parametrize("T,h,hkv", [(1, 1, 1), (1, 40, 1), (2, 36, 4), (700, 64, 64), (5000, 6, 2), (3, 128, 8)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_qk_norm_rope_sizes(nsp, dt, T, h, hkv):
    """However rows are spread over the blocks: every head's bits alone, sums of
    the weights' gradients against the oracle, the same bits twice."""
    cu, fr = cu_of([T]), nsp.rope_freqs(64, device="cuda")
    q, k, gq, gk = (randn(10 + i, T, n, 64, dt=dt) for i, n in enumerate((h, hkv, h, hkv)))
    wq, wk = randn(15, 64, dt=dt), randn(16, 64, dt=dt)
    yq, yk = nsp.qk_norm_rope(q, k, cu, fr, wq, wk)
    got = nsp.qk_norm_rope_bwd(q, k, gq, gk, cu, fr, wq, wk)
    for a, b in zip(got, nsp.qk_norm_rope_bwd(q, k, gq, gk, cu, fr, wq, wk)):
        assert torch.equal(a, b)
    for i in (0, h // 2, h - 1):
        one = q[:, i:i + 1]
        assert torch.equal(yq[:, i:i + 1], nsp.qk_norm_rope(one, None, cu, fr, wq)[0]), i
        dx = nsp.qk_norm_rope_bwd(one, None, gq[:, i:i + 1], None, cu, fr, wq)[0]
        assert torch.equal(got[0][:, i:i + 1], dx), i
    assert torch.equal(yk[:, -1:], nsp.qk_norm_rope(k[:, -1:], None, cu, fr, wk)[0])
    x, z = f64(q), S.rope(f64(gq), L.rope_angles(np.arange(T), fr.cpu().numpy()), 64, inverse=True)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    mag = (np.abs(n) * pair_sum(f64(gq), 64, False, 1.0)).sum((0, 1))
    # rows of a warp one after the other (2432 warps at most), and 160 more sums
    sums = T * h / 1216 + 260
    ref = (n * z).sum((0, 1))
    assert_within(got[2], ref, half_step(dt) * np.abs(ref) + sums * E * mag, "dw")


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_qk_norm_rope_views_in_place_groups(nsp, dt, inter):
    """Columns of a fused projection in, packed, head-grouped and in-place out, both
    directions; the columns in between untouched."""
    T, hq, hkv, d = sum(LENS), 8, 2, 128
    kw = dict(layout="interleaved" if inter else "half")
    cu, fr = cu_of(LENS), nsp.rope_freqs(d, device="cuda")
    qkv, wq, wk = randn(20, T, hq + 2 * hkv, d, dt=dt), randn(21, d, dt=dt), randn(22, d, dt=dt)
    gq, gk = randn(23, T, hq, d, dt=dt), randn(24, T, hkv, d, dt=dt)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    ref = nsp.qk_norm_rope(q.contiguous(), k.contiguous(), cu, fr, wq, wk, **kw)
    back = nsp.qk_norm_rope_bwd(q.contiguous(), k.contiguous(), gq, gk, cu, fr, wq, wk, **kw)
    for a, b in zip(nsp.qk_norm_rope(q, k, cu, fr, wq, wk, **kw), ref):
        assert torch.equal(a, b)
    for p in (2, 4):
        grouped, _ = nsp.qk_norm_rope(q, k, cu, fr, wq, wk, q_groups=p, **kw)
        assert torch.equal(grouped, nsp.seq2head(ref[0], p))
        got = nsp.qk_norm_rope_bwd(q, k, nsp.seq2head(gq, p), gk, cu, fr, wq, wk, q_groups=p, **kw)
        for a, b in zip(got, back):
            assert torch.equal(a, b)
    # gradients into columns of the fused projection's gradient, over dy, over x
    fused = torch.full_like(qkv, 7.0)
    got = nsp.qk_norm_rope_bwd(q, k, gq, gk, cu, fr, wq, wk, out=(fused[:, :hq], fused[:, hq:hq + hkv]), **kw)
    assert torch.equal(fused[:, :hq], back[0]) and torch.equal(fused[:, hq:hq + hkv], back[1])
    assert (fused[:, hq + hkv:] == 7).all() and torch.equal(got[2], back[2])
    a, b = gq.clone(), gk.clone()
    nsp.qk_norm_rope_bwd(q, k, a, b, cu, fr, wq, wk, out=(a, b), **kw)
    assert torch.equal(a, back[0]) and torch.equal(b, back[1])
    over = qkv.clone()
    got = nsp.qk_norm_rope_bwd(over[:, :hq], over[:, hq:hq + hkv], gq, gk, cu, fr, wq, wk,
                               out=(over[:, :hq], over[:, hq:hq + hkv]), **kw)
    assert torch.equal(over[:, :hq], back[0]) and torch.equal(over[:, hq:hq + hkv], back[1])
    for i in (2, 3):
        assert torch.equal(got[i], back[i])
    before = qkv.clone()
    nsp.qk_norm_rope(q, k, cu, fr, wq, wk, out=(q, k), **kw)
    assert torch.equal(qkv[:, :hq], ref[0]) and torch.equal(qkv[:, hq:hq + hkv], ref[1])
    assert torch.equal(qkv[:, hq + hkv:], before[:, hq + hkv:])


@pytest.mark.parametrize("dt", [BF16, F32])
def test_qk_norm_rope_odd_addresses(nsp, dt):
    """Strides and addresses that are no whole 16 bytes: within two roundings of the
    output of the same rows elsewhere (sums of squares in another order)."""
    T, h, d = 29, 3, 64
    cu, fr, w = cu_of([29]), nsp.rope_freqs(d, device="cuda"), randn(31, d, dt=dt)
    x, g = randn(30, T, h, d, dt=dt), randn(32, T, h, d, dt=dt)
    ang = L.rope_angles(np.arange(T), fr.cpu().numpy())
    wide = torch.zeros((T, h * d + 3), dtype=dt, device="cuda")
    view = wide[:, 1:1 + h * d].unflatten(1, (h, d))
    view.copy_(x)
    y, _ = nsp.qk_norm_rope(view, None, cu, fr, w)
    dx, _, dw, _ = nsp.qk_norm_rope_bwd(view, None, g, None, cu, fr, w)
    check_qk(x, w, g, y, dx, dw, ang, d, False, 1.0, 1e-6, dt)


def test_qk_norm_rope_rows_behind_and_positions(nsp):
    """Rows behind the last document: left as they were, and nothing of theirs in the
    weights' gradients, whatever they hold; shards of a stream; given positions;
    no rows; a row of NaN."""
    T, h, d = 100, 4, 64
    cu, fr, w = cu_of([40, 30]), nsp.rope_freqs(d, device="cuda"), randn(41, d)
    x, g = randn(40, T, h, d), randn(42, T, h, d)
    x[70:], g[70:] = float("nan"), float("inf")
    out, dx = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    nsp.qk_norm_rope(x, None, cu, fr, w, out=(out, None))
    dw = nsp.qk_norm_rope_bwd(x, None, g, None, cu, fr, w, out=(dx, None))[2]
    assert (out[70:] == 7).all() and (dx[70:] == 7).all()
    ref, _ = nsp.qk_norm_rope(x[:70].contiguous(), None, cu, fr, w)
    rdx, _, rdw, _ = nsp.qk_norm_rope_bwd(x[:70].contiguous(), None, g[:70].contiguous(), None, cu, fr, w)
    assert torch.equal(out[:70], ref) and torch.equal(dx[:70], rdx)
    np.testing.assert_allclose(f64(dw), f64(rdw), rtol=2 ** -7, atol=1e-3)
    for s, e in ((0, 33), (33, 70)):
        part, _ = nsp.qk_norm_rope(x[s:e], None, cu, fr, w, start=s)
        assert torch.equal(part, ref[s:e])
        part = nsp.qk_norm_rope_bwd(x[s:e], None, g[s:e], None, cu, fr, w, start=s)[0]
        assert torch.equal(part, rdx[s:e])
    pos = torch.tensor([5, 399999, 0], dtype=torch.int32, device="cuda")
    y, _ = nsp.qk_norm_rope(x[:3], None, None, fr, w, positions=pos)
    ang = L.rope_angles(pos.cpu().numpy(), fr.cpu().numpy())
    xs = f64(x[:3])
    want = S.qk_norm_rope(xs, f64(w), ang, d)
    n = xs / np.sqrt((xs * xs).mean(-1, keepdims=True) + 1e-6) * f64(w)
    far = np.concatenate([np.abs(pos.cpu().numpy()[:, None] * fr.cpu().numpy()) * 2.0 ** -51] * 2, -1)[:, None]
    assert_within(y, want, 2 ** -8 * np.abs(want) + (84 * E + far) * pair_sum(n, d, False, 1.0), "far")
    assert nsp.qk_norm_rope(x[:0], None, cu, fr, w)[0].shape == (0, h, d)
    none = nsp.qk_norm_rope_bwd(x[:0], None, g[:0], None, cu, fr, w)
    assert none[0].shape == (0, h, d) and (none[2] == 0).all()
    x[1, 2, 5] = float("nan")
    y, _ = nsp.qk_norm_rope(x[:70], None, cu, fr, w)
    bad = torch.isnan(y)
    assert bad[1, 2].all() and int(bad.sum()) == d
    z = torch.zeros((2, 1, d), device="cuda")
    assert (nsp.qk_norm_rope(z, None, cu_of([2]), fr)[0] == 0).all()


def test_qk_norm_rope_is_norm_then_rope(nsp):
    """Float32: the two operators after one another, up to roundings."""
    T, h, d = sum(LENS), 6, 128
    cu, fr, w = cu_of(LENS), nsp.rope_freqs(d, device="cuda"), randn(51, d, dt=F32)
    x, g = randn(50, T, h, d, dt=F32), randn(52, T, h, d, dt=F32)
    y, _ = nsp.qk_norm_rope(x, None, cu, fr, w)
    two, _ = nsp.rope(nsp.head_norm(x, w), None, cu, fr)
    torch.testing.assert_close(y, two, rtol=0, atol=200 * E * float(two.abs().max()))
    dx, _, dw, _ = nsp.qk_norm_rope_bwd(x, None, g, None, cu, fr, w)
    rdx, rdw, _ = nsp.head_norm_bwd(x, nsp.rope(g, None, cu, fr, inverse=True)[0], w)
    torch.testing.assert_close(dx, rdx, rtol=0, atol=400 * E * float(rdx.abs().max()))
    torch.testing.assert_close(dw, rdw, rtol=0, atol=400 * E * float((x.abs() * g.abs()).sum((0, 1)).max()) * 3)


# ----------------------------------------------------------------------------- log-probabilities

SCALE = 0.75                     # (exact in float32)


def logits_of(seed, T, V, dt, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, V), generator=g) * spread).to(dt)
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    y[torch.rand(T, generator=g) < 0.25] = -1
    return x.cuda(), y.cuda()


def lse_error(x, scale=SCALE):
    """Absolute error of a row's log sum: an argument's roundings (of the scaled maximum,
    the scale and the difference: 8 E of the largest magnitude), exp 2 ulp, the
    terms' sums (a thread's terms one after the other, of 512 threads at least, then 40
    more), log."""
    top = scale * np.abs(np.where(np.isfinite(x), x, 0)).max(-1)
    return E * (8 * top + 64 + x.shape[-1] / 512)


def check_logp(x, y, logp, lse, scale=SCALE):
    x, y = f64(x), y.cpu().numpy()
    rl, rs = S.token_logp(x, y, scale)
    err = np.where(y >= 0, lse_error(x, scale), 0)
    assert_within(logp, rl, err + 2 * E * np.abs(rl), "logp")
    if lse is not None:
        assert_within(lse, rs, err + 2 * E * np.abs(rs), "lse")


def check_dlogits(x, y, dlogp, got, dt, scale=SCALE, dlogp_err=0.0):
    x, y = f64(x), y.cpu().numpy()
    g = f64(dlogp) if isinstance(dlogp, torch.Tensor) else dlogp
    ref = S.token_logp_bwd(x, y, g, scale)
    p = np.abs(S.token_logp_bwd(x, y, np.ones(len(y)), scale)) / scale       # p, or 1 - p of the target
    c = (lse_error(x, scale) + 8 * E)[:, None]
    # the target's own column is 1 - p: p's error there is c (1 - (1 - p))
    col = np.where(np.arange(x.shape[1])[None] == y[:, None], 1.0, p)
    # (a power of two below 2^-126 is zero; the sum that divides it is 1/2 or more, as its
    # largest term's exponent is in (-1, 0]: a p below 2^-125 may be zero)
    tol = half_step(dt) * np.abs(ref) + np.abs(scale * g)[:, None] * (c * col + 4 * E * p + 2.0 ** -125)
    tol = tol + np.broadcast_to(np.asarray(dlogp_err), (len(y),))[:, None] * p
    assert_within(got, ref, np.where(y[:, None] >= 0, tol, 0), "dlogits")


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (7, 8), (5, 31), (4, 257), (9, 1000), (3, 1024), (6, 4096), (5, 4103),
                                 (2, 16384), (3, 32003), (2, 65536), (2, 100001), (1, 131072), (2, 200000),
                                 (1, 1 << 20), (700, 264), (400, 1001)])
def test_token_logp(nsp, dt, T, V):
    x, y = logits_of(60, T, V, dt)
    y[0] = V - 1
    logp, lse = nsp.token_logp(x, y, scale=SCALE)
    check_logp(x, y, logp, lse)
    g = randn(61, T, dt=F32)
    dx = nsp.token_logp_bwd(x, y, lse, g, scale=SCALE)
    check_dlogits(x, y, g, dx, dt)
    again, _ = nsp.token_logp(x, y, scale=SCALE)
    assert torch.equal(again, logp)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("V,stride,shift", [(1000, 1024, 0), (1000, 1001, 0), (999, 1024, 8), (1001, 1003, 1), (40000, 40008, 3),
                                            (40001, 40001, 5)])
def test_token_logp_strides(nsp, dt, V, stride, shift):
    """Padded vocabularies, rows at any distance from a 16-byte border, outputs at the
    same or at another one, in place: columns behind the vocabulary stay as they were."""
    T = 6
    x, y = logits_of(62, T, V, dt)
    flat = torch.full((T * stride + shift + 64,), float("nan"), dtype=dt, device="cuda")
    wide = flat[shift:shift + T * stride].view(T, stride)
    wide[:, :V] = x
    view = wide[:, :V]
    logp, lse = nsp.token_logp(view, y, scale=SCALE)
    check_logp(x, y, logp, lse)
    g = randn(63, T, dt=F32)
    for off in (shift, shift + 1):
        out = torch.full((T * stride + 72,), 7.0, dtype=dt, device="cuda")
        ov = out[off:off + T * stride].view(T, stride)[:, :V]
        nsp.token_logp_bwd(view, y, lse, g, scale=SCALE, out=ov)
        check_dlogits(x, y, g, ov, dt)
        ov[:] = 7.0
        assert (out == 7).all()
    ref = nsp.token_logp_bwd(view, y, lse, g, scale=SCALE)
    nsp.token_logp_bwd(view, y, lse, g, scale=SCALE, out=view)
    assert torch.equal(view, ref)
    view[:] = float("nan")
    assert torch.isnan(flat).all()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("V", [40, 1001, 70000])
def test_token_logp_masked_logits(nsp, dt, V):
    """Minus infinity has probability zero, wherever it stands (all but one, the
    target's own); rows without a target may hold anything; NaN, plus infinity and a
    target past the vocabulary give NaN in their row alone; large magnitudes do not
    overflow."""
    x, y = logits_of(64, 8, V, dt)
    y[:] = torch.arange(8, dtype=torch.int32)
    inf = float("inf")
    x[0, 1:] = -inf                       # only the target
    x[1, 5:] = -inf
    x[2, 2], x[2, 9:30] = -inf, -inf      # the target itself
    x[3] = float("nan")
    y[3] = -1
    x[4] *= 3e4
    x[5, 3], x[6, V - 1] = float("nan"), inf
    y[7] = V
    logp, lse = nsp.token_logp(x, y, scale=SCALE)
    g = torch.full((8,), 0.5, device="cuda")
    g[3] = float("nan")
    dx = nsp.token_logp_bwd(x, y, lse, g, scale=SCALE)
    good = [0, 1, 4]
    check_logp(x[good], y[good], logp[good], lse[good])
    check_dlogits(x[good], y[good], g[good], dx[good], dt)
    # (1 - p of a certain target: x_y - lse is off by lse's own rounding)
    assert logp[0] <= 0 and (dx[0, 1:] == 0).all() and abs(float(dx[0, 0])) <= E * (2 * abs(float(x[0, 0])) + 4)
    assert logp[2] == -inf and torch.isfinite(lse[2]) and torch.isfinite(dx[2]).all()
    assert logp[3] == 0 and lse[3] == 0 and (dx[3] == 0).all()
    assert torch.isnan(logp[5:]).all() and torch.isnan(dx[7]).all()
    assert torch.isnan(lse[5]) and torch.isnan(lse[6]) and torch.isfinite(lse[7])
    x[0] = -inf
    assert torch.isnan(nsp.token_logp(x, y)[0][0])


def test_token_logp_no_rows_and_far_rows(nsp):
    """No rows; offsets past 32 bits."""
    x = torch.empty((0, 50), device="cuda")
    y = torch.empty(0, dtype=torch.int32, device="cuda")
    logp, lse = nsp.token_logp(x, y)
    assert logp.shape == (0,) and nsp.token_logp_bwd(x, y, lse, logp).shape == (0, 50)
    T, V = 34000, 65536                   # 2.2e9 elements
    big = torch.zeros((T, V), dtype=BF16, device="cuda")
    few, y5 = logits_of(65, 5, V, BF16)
    big[-5:] = few
    y = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    y[-5:] = y5
    logp, lse = nsp.token_logp(big, y, scale=SCALE)
    assert (logp[:-5] == 0).all()
    check_logp(few, y5, logp[-5:], lse[-5:])
    g = randn(66, T, dt=F32)
    nsp.token_logp_bwd(big, y, lse, g, scale=SCALE, out=big)
    check_dlogits(few, y5, g[-5:], big[-5:], BF16)
    assert not big[:-5].any()


# ----------------------------------------------------------------------------- losses

# (an empty document, ones without a scored row, a row behind the last one)
DOCS = [5, 0, 1, 40, 33, 1, 300, 2, 0, 64]


def step_inputs(seed, lens, behind=3, T=None):
    """Targets, log-probabilities and what a policy loss reads, off the clip's borders."""
    T = sum(lens) + behind if T is None else T
    rng = np.random.default_rng(seed)
    y = rng.integers(0, 50, T)
    y[rng.random(T) < 0.3] = -1
    logp = -rng.uniform(0.01, 6, T)
    d = rng.normal(size=T) * 0.3          # log of the ratio
    for border in (np.log(0.8), np.log(1.25)):
        d = np.where(np.abs(d - border) < 1e-3, border + 2e-3, d)
    cuda = lambda a: torch.tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
    return (torch.tensor(y, dtype=torch.int32, device="cuda"), cuda(logp), cuda(logp - d),
            cuda(logp + rng.normal(size=T) * 0.5), rng)


def check_policy(logp, y, old, ref, adv, cu, stats, dlogp, kw, logp_err=0.0):
    """logp_err: of each log-probability."""
    l, o, a = f64(logp), f64(old), f64(adv)
    r = None if ref is None else f64(ref)
    y, cu = y.cpu().numpy(), cu.cpu().numpy()
    args = dict(clip_low=float(np.float32(kw["clip_low"])), clip_high=float(np.float32(kw["clip_high"])),
                kl_coef=float(np.float32(kw["kl_coef"])), mean=kw["mean"], total=kw.get("total", 0.0))
    rs, rg = S.policy_loss(l, o, r, a, y, cu, **args)
    # one row's terms without their weights: sums of magnitudes times their roundings (the
    # log ratio's own and its exp: (|d| + 8) E; the weight 3 E)
    d = np.where(y >= 0, l - o, 0)
    T = len(l)
    weight = np.zeros(T)
    rows_adv = np.zeros(T)
    live = [[t for t in range(min(cu[b], T), min(cu[b + 1], T)) if y[t] >= 0] for b in range(len(cu) - 1)]
    nt, nd = sum(map(len, live)), sum(len(x) > 0 for x in live)
    for b, rows in enumerate(live):
        for t in rows:
            n = args["total"] or (nt if args["mean"] == "tokens" else nd)
            weight[t] = 1 / n if args["mean"] == "tokens" else 1 / (n * len(rows))
            rows_adv[t] = a[t] if len(a) == T and len(a) != len(live) else a[b]
    g = np.abs(rows_adv) * np.exp(d)
    e_rel = (np.abs(d) + 12) * E + logp_err
    tol = weight * g * e_rel
    kl_tol = 0.0
    if r is not None:
        z = np.where(y >= 0, r - l, 0)
        big = np.exp(z) + 1 + np.abs(z)
        kl_tol = weight * big * ((np.abs(z) + 12) * E + logp_err)
        tol = tol + args["kl_coef"] * kl_tol
    assert_within(dlogp, rg, tol + 2 * E * np.abs(rg), "dlogp")
    pg_tol = (weight * g * e_rel).sum()
    k = np.sum(kl_tol)
    assert_within(stats, rs, np.array([pg_tol + args["kl_coef"] * k, pg_tol, k, 6 * E * rs[3]]) + 2 * E * np.abs(rs),
                  "stats")


@pytest.mark.parametrize("mean", ["tokens", "documents"])
@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("kl", [0.0, 0.07])
@pytest.mark.parametrize("lens", [DOCS, [1], [2000], [3] * 700, [0, 0, 40000, 0, 17]])
def test_policy_loss(nsp, mean, per_token, kl, lens):
    y, logp, old, ref, rng = step_inputs(70, lens)
    cu = cu_of(lens)
    T = len(y)
    adv = torch.tensor(rng.normal(size=T if per_token else len(lens)), dtype=torch.float32, device="cuda")
    kw = dict(clip_low=0.2, clip_high=0.25, kl_coef=kl, mean=mean)
    # rows without a score may hold anything
    out = (y < 0) | (torch.arange(T, device="cuda") >= int(cu[-1]))
    for t in (logp, old, ref) + ((adv,) if per_token else ()):
        t[out] = float("nan")
    r = ref if kl else None
    stats, dlogp = nsp.policy_loss(logp, y, old, adv, cu, ref=r, **kw)
    clean = [t.clone() for t in (logp, old, ref, adv)]
    for t in clean[:3] + ([clean[3]] if per_token else []):
        t[out] = 0.0
    c_logp, c_old, c_ref, c_adv = clean
    check_policy(c_logp, y, c_old, c_ref if kl else None, c_adv, cu, stats, dlogp, kw)
    assert (dlogp[out] == 0).all()
    again, d2 = nsp.policy_loss(logp, y, old, adv, cu, ref=r, **kw)
    assert torch.equal(again, stats) and torch.equal(d2, dlogp)


@pytest.mark.parametrize("mean", ["tokens", "documents"])
def test_policy_loss_total_and_parts(nsp, mean):
    """Two calls over halves of the documents with the whole's number are the whole."""
    y, logp, old, ref, rng = step_inputs(71, DOCS, behind=0)
    cu = cu_of(DOCS)
    adv = torch.tensor(rng.normal(size=len(DOCS)), dtype=torch.float32, device="cuda")
    kw = dict(clip_low=0.2, clip_high=0.25, kl_coef=0.1, mean=mean)
    stats, dlogp = nsp.policy_loss(logp, y, old, adv, cu, ref=ref, **kw)
    at = int(cu[5])
    yh = y.cpu().numpy()
    cuh = cu.cpu().numpy()
    total = float((yh >= 0).sum() if mean == "tokens" else sum((yh[a:b] >= 0).any() for a, b in zip(cuh, cuh[1:])))
    parts = [nsp.policy_loss(logp[s], y[s], old[s], adv[d], c, ref=ref[s], total=total, **kw)
             for s, d, c in ((slice(0, at), slice(0, 5), cu[:6]), (slice(at, None), slice(5, None), cu[5:] - cu[5]))]
    assert torch.equal(torch.cat([p[1] for p in parts]), dlogp)
    torch.testing.assert_close(parts[0][0] + parts[1][0], stats, rtol=0, atol=8 * E * float(stats.abs().max()) + 1e-7)


def test_policy_loss_nothing_scored(nsp):
    cu = cu_of([4, 0, 3])
    y = torch.full((7,), -1, dtype=torch.int32, device="cuda")
    nan = torch.full((7,), float("nan"), device="cuda")
    x = torch.full((7, 33), float("nan"), device="cuda")
    for mean in ("tokens", "documents"):
        stats, dlogp = nsp.policy_loss(nan, y, nan, nan[:3], cu, ref=nan, kl_coef=0.1, mean=mean)
        assert (stats == 0).all() and (dlogp == 0).all()
        stats, logp, dx = nsp.policy_loss_logits(x, y, nan, nan[:3], cu, ref=nan, kl_coef=0.1, mean=mean)
        assert (stats == 0).all() and (logp == 0).all() and (dx == 0).all()
    e = x[:0]
    stats, logp, dx = nsp.policy_loss_logits(e, y[:0], nan[:0], nan[:3], cu)
    assert (stats == 0).all() and logp.shape == (0,) and dx.shape == (0, 33)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("V,lens,kl,mean", [(50, DOCS, 0.07, "documents"), (1003, [5, 0, 7, 1], 0.0, "tokens"),
                                            (32768, [3, 9], 0.07, "tokens"), (131072, [4], 0.07, "documents"),
                                            (70001, [2, 5], 0.07, "documents"), (300000, [3], 0.07, "tokens"),
                                            (8, [1000, 1000], 0.1, "tokens")])
def test_policy_loss_logits(nsp, dt, V, lens, kl, mean):
    """Against the oracle, and the three calls that it does in one."""
    y, _, _, _, rng = step_inputs(72, lens)
    T, cu = len(y), cu_of(lens)
    x, _ = logits_of(73, T, V, dt)
    y = torch.where(y >= 0, torch.tensor(rng.integers(0, V, T), dtype=torch.int32, device="cuda"), y)
    logp64, _ = S.token_logp(f64(x), y.cpu().numpy(), SCALE)
    d = rng.normal(size=T) * 0.3
    for border in (np.log(0.8), np.log(1.25)):
        d = np.where(np.abs(d - border) < 1e-3, border + 2e-3, d)
    old, ref = (torch.tensor(logp64 + o, dtype=torch.float32, device="cuda") for o in (-d, rng.normal(size=T) * 0.5))
    adv = torch.tensor(rng.normal(size=len(lens)), dtype=torch.float32, device="cuda")
    kw = dict(clip_low=0.2, clip_high=0.25, kl_coef=kl, mean=mean)
    r = ref if kl else None
    behind = torch.arange(T, device="cuda") >= int(cu[-1])
    x[y < 0], x[behind] = float("nan"), float("nan")
    stats, logp, dx = nsp.policy_loss_logits(x, y, old, adv, cu, ref=r, scale=SCALE, **kw)
    scored = torch.where(behind, torch.full_like(y, -1), y)
    x0 = torch.nan_to_num(x, nan=0.0)
    check_logp(x0, scored, logp, None)
    err = lse_error(f64(x0)) + 2 * E * np.abs(logp64)
    lw = torch.tensor(np.where(scored.cpu().numpy() >= 0, logp64, 0), device="cuda")
    dl_ref = S.policy_loss(f64(lw), f64(old), None if r is None else f64(r), f64(adv), scored.cpu().numpy(),
                           cu.cpu().numpy(), float(np.float32(0.2)), 0.25, float(np.float32(kl)), mean)[1]
    two, dl = nsp.policy_loss(logp, y, old, adv, cu, ref=r, **kw)
    check_policy(lw, scored, old, r, adv, cu, stats, dl, kw, logp_err=err)
    dl_err = np.abs(f64(dl) - dl_ref) + 4 * E * np.abs(dl_ref)
    check_dlogits(x0, scored, dl_ref, dx, dt, dlogp_err=SCALE * dl_err)
    torch.testing.assert_close(stats, two, rtol=8 * E, atol=8 * E * float(two.abs().max()))
    # in place, into padded rows, and twice: the same bits
    wide = torch.full((T, V + 16 // x.element_size()), 7.0, dtype=dt, device="cuda")
    wide[:, :V] = x
    s2, l2, d2 = nsp.policy_loss_logits(wide[:, :V], y, old, adv, cu, ref=r, scale=SCALE, out=wide[:, :V], **kw)
    assert torch.equal(s2, stats) and torch.equal(l2, logp) and torch.equal(d2, dx) and (wide[:, V:] == 7).all()
    s3, _, d3 = nsp.policy_loss_logits(x, y, old, adv, cu, ref=r, scale=SCALE, **kw)
    assert torch.equal(s3, stats) and torch.equal(d3, dx)


@pytest.mark.parametrize("bad", [[1, 3, 6], [0, 5, 3], [0, -1, 6], [0, 3, 2]])
def test_losses_bad_documents(nsp, bad):
    """The status word says so, and the next call is a clean one."""
    T = 6
    cu, good = torch.tensor(bad, dtype=torch.int32, device="cuda"), cu_of([3, 3])
    y = torch.tensor([0, 1, -1, 2, 0, 1], dtype=torch.int32, device="cuda")
    v, x = randn(80, T, dt=F32), randn(81, T, 9, dt=F32)
    ws = torch.empty(8192, dtype=torch.uint8, device="cuda")
    for call in (lambda c: nsp.policy_loss(v, y, v, v[:2], c, workspace=ws),
                 lambda c: nsp.policy_loss_logits(x, y, v, v[:2], c, workspace=ws),
                 lambda c: nsp.preference_loss(v, y, c, workspace=ws)):
        call(cu)
        assert nsp.nsp_status_query(ws) == nsp.NSP_ERR_INVALID
        first = call(good)
        assert nsp.nsp_status_query(ws) == nsp.NSP_OK
        for a, b in zip(first, call(good)):
            assert torch.equal(a, b)
    # a cu_seqlens that reaches past the rows is cut there
    long = cu_of([3, 300])
    for a, b in zip(nsp.policy_loss(v, y, v, v[:2], long, workspace=ws), nsp.policy_loss(v, y, v, v[:2], good)):
        assert torch.equal(a, b)
    for a, b in zip(nsp.preference_loss(v, y, long, workspace=ws), nsp.preference_loss(v, y, good)):
        assert torch.equal(a, b)
    assert nsp.nsp_status_query(ws) == nsp.NSP_OK


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "square"])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("lens", [DOCS, [1, 1], [0, 0], [3000, 4097], [3] * 900, [0, 70000, 3, 1], [20000, 1, 1, 20000]])
def test_preference_loss(nsp, kind, average, lens):
    y, logp, _, ref, _ = step_inputs(74, lens, behind=5)
    cu, T = cu_of(lens), len(y)
    out = (y < 0) | (torch.arange(T, device="cuda") >= int(cu[-1]))
    logp[out], ref[out] = float("nan"), float("nan")
    kw = dict(kind=kind, beta=0.125, smoothing=0.0625, margin=0.25, average=average)     # (exact in float32)
    for r in (ref, None):
        stats, rewards, dlogp = nsp.preference_loss(logp, y, cu, ref=r, **kw)
        l0 = torch.where(out, 0.0, logp)
        r0 = None if r is None else f64(torch.where(out, 0.0, r))
        scored = torch.where(out, torch.full_like(y, -1), y).cpu().numpy()
        rs, rr, rg = S.preference_loss(f64(l0), r0, scored, cu.cpu().numpy(), **kw)
        # scores are exact to 2^-40 of their terms' magnitudes, the rest is float64
        mag = np.abs(f64(l0)).sum() * 2.0 ** -38
        assert_within(rewards, rr, 2 * E * np.abs(rr) + mag, "rewards")
        # the loss's slope in h is at most 1, or (square) 2 |off| / beta^2
        slope = 1.0 if kind != "square" else 2 * (np.abs(rr).max() * 2 + 5) / 0.125 ** 2
        assert_within(stats[:1], rs[:1], 4 * E * np.abs(rs[:1]) + slope * mag, "loss")
        assert stats[1] == np.float32(rs[1])
        assert_within(dlogp, rg, 3 * E * np.abs(rg) + slope * mag, "dlogp")
        assert (dlogp[out] == 0).all()
        for a, b in zip(nsp.preference_loss(logp, y, cu, ref=r, **kw), (stats, rewards, dlogp)):
            assert torch.equal(a, b)


def test_preference_loss_far_scores(nsp):
    """Scores that differ by thousands: the sigmoid's tails keep their own precision."""
    cu = cu_of([1, 1, 1, 1, 1, 1])
    y = torch.zeros(6, dtype=torch.int32, device="cuda")
    logp = torch.tensor([-1.0, -4001.0, -4001.0, -1.0, -1.0, -301.0], device="cuda")
    stats, rewards, dlogp = nsp.preference_loss(logp, y, cu, beta=0.125)
    rs, rr, rg = S.preference_loss(f64(logp), None, np.zeros(6), cu.cpu().numpy(), beta=0.125)
    np.testing.assert_allclose(f64(rewards), rr, rtol=2e-7)
    np.testing.assert_allclose(f64(stats), rs, rtol=2e-7)
    np.testing.assert_allclose(f64(dlogp), rg, rtol=4e-7, atol=1e-38)


# ----------------------------------------------------------------------------- many gradients

def grads_of(seed, sizes, types, shift=0, scale=1.0):
    out = []
    for i, n in enumerate(sizes):
        dt = types[i % len(types)]
        base = torch.zeros(n + 16, dtype=dt, device="cuda")
        t = base[shift * i % 9:][:n]
        t.copy_(randn(seed + i, n, dt=F32, scale=scale))
        out.append(t)
    return out


def check_norm(grads, norm, unscale=1.0, kind=2):
    ref = S.grad_norm([f64(g) for g in grads], unscale, kind)
    # a square's rounding and at most 126 float32 sums of squares, halved by the root
    assert_within(norm, [ref], (64 if kind == 2 else 1) * E * ref, "norm")
    return ref


SIZES = [[1], [7, 0, 300], [32768], [32769, 5], [40000, 1, 1, 1, 65536, 3000], [1000003], [17] * 70, [5] * 900 + [40001] * 3]


@pytest.mark.parametrize("types", [[BF16], [F32], [BF16, F32]])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("sizes", SIZES)
def test_grad_norm_and_clip(nsp, types, shift, sizes):
    grads = grads_of(90, sizes, types, shift)
    norm = nsp.grad_norm(grads, unscale=-0.25)
    ref = check_norm(grads, norm, -0.25)
    assert torch.equal(nsp.grad_norm(grads, unscale=-0.25), norm)
    check_norm(grads, nsp.grad_norm(grads, float("inf"), unscale=0.5), 0.5, np.inf)
    max_norm = float(np.float32(0.3 * ref))
    factor = -0.25 * max_norm / (ref + 1e-6)
    for other in (False, True):
        out = [torch.full((n + 8,), 7.0, dtype=types[(i + other) % len(types)], device="cuda") for i, n in enumerate(sizes)]
        views = [o[1 + shift * (i % 3):][:n] for i, (o, n) in enumerate(zip(out, sizes))]
        got = nsp.clip_grads(grads, max_norm, unscale=-0.25, out=views)
        assert torch.equal(got, norm)
        for i, (g, v) in enumerate(zip(grads, views)):
            want = f64(g) * factor
            # (float32 values below 2^-126 aside)
            assert_within(v, want, (half_step(v.dtype) + 80 * E) * np.abs(want) + 2.0 ** -126, i)
            v[:] = 7.0
        assert all([(o == 7).all() for o in out])
    keep = [g.clone() for g in grads]
    assert torch.equal(nsp.clip_grads(grads, max_norm, unscale=-0.25), norm)
    for g, k in zip(grads, keep):
        want = f64(k) * factor
        assert_within(g, want, (half_step(g.dtype) + 80 * E) * np.abs(want) + 2.0 ** -126, "in place")


def test_clip_does_nothing_below_the_norm(nsp):
    grads = grads_of(91, [1000, 77], [F32, BF16])
    keep = [g.clone() for g in grads]
    norm = nsp.clip_grads(grads, 1e6)
    check_norm(grads, norm)
    for g, k in zip(grads, keep):
        assert torch.equal(g, k)
    nsp.clip_grads(grads, 1e6, unscale=0.5)
    for g, k in zip(grads, keep):
        assert torch.equal(g, k * 0.5)
    nsp.clip_grads(grads, 0.0)
    assert all([(g == 0).all() for g in grads])


def test_grad_norm_special_values(nsp):
    """NaN and infinity anywhere; zeros; no elements; magnitudes near the ends."""
    for kind in (2, float("inf")):
        for at in (0, 999, 40000):
            g = grads_of(92, [40001, 30], [F32])
            g[0][at] = float("inf")
            assert nsp.grad_norm(g, kind) == float("inf")
            keep = g[1].clone()
            assert nsp.clip_grads(g, 1.0, kind) == float("inf")
            assert torch.isnan(g[0][at]) and (g[1] == 0).all() and keep.any()
            g[1][3] = float("nan")
            assert torch.isnan(nsp.grad_norm(g, kind))
            nsp.clip_grads(g, 1.0, kind)
            assert all([torch.isnan(t).all() for t in g])
    z = [torch.zeros(500, device="cuda"), torch.zeros(0, device="cuda")]
    assert nsp.grad_norm(z) == 0 and nsp.grad_norm(z[1:]) == 0 and nsp.clip_grads(z, 1.0) == 0
    big = [torch.full((4,), 1e18, device="cuda"), torch.full((4,), 1e-18, device="cuda")]
    check_norm(big[:1], nsp.grad_norm(big[:1]))
    check_norm(big[1:], nsp.grad_norm(big[1:]))
    check_norm(big, nsp.grad_norm(big))


def test_grad_norm_far_elements(nsp):
    """Offsets past 32 bits in one tensor."""
    n = (1 << 31) + 5000
    t = torch.zeros(n, dtype=BF16, device="cuda")
    t[-3:] = 4.0
    t[0] = 1.0
    assert nsp.grad_norm([t]) == 7.0
    nsp.clip_grads([t], 3.5)
    assert abs(float(t[-1]) - 2.0) < 0.01 and abs(float(t[0]) - 0.5) < 0.01 and not t[1:-3].any()


# ----------------------------------------------------------------------------- many long rows

def scattered(seed, T, V, every=1):
    """Targets of about half of every `every`-th row: runs of scored and other rows, single ones."""
    rng = np.random.default_rng(seed)
    y = np.full(T, -1)
    at = np.arange(0, T, every)
    on = np.repeat(rng.random(len(at) // 7 + 1) < 0.6, 7)[:len(at)] ^ (rng.random(len(at)) < 0.1)
    y[at[on]] = rng.integers(0, V, on.sum())
    y[at[0]], y[at[-1]] = 0, V - 1
    return torch.tensor(y, dtype=torch.int32, device="cuda")


def logits_on(seed, y, V, dt, stride=None, shift=0):
    """Logits whose rows without a target are NaN, rows `stride` apart."""
    T, stride = len(y), stride or V
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.full((T * stride + shift + 64,), float("nan"), dtype=dt, device="cuda")
    x = flat[shift:shift + T * stride].view(T, stride)[:, :V]
    rows = torch.nonzero(y >= 0)[:, 0]
    x[rows] = (torch.randn((len(rows), V), generator=g, device="cuda") * 2.5).to(dt)
    return x, rows


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T,V,stride,shift", [(609, 4200, None, 0), (700, 4111, None, 3), (1300, 8192, 8200, 0),
                                              (640, 20001, None, 1), (650, 33000, None, 0), (5000, 5003, None, 0),
                                              (609, 500, None, 0), (620, 1000, 1016, 5), (612, 6001, None, 0),
                                              (611, 12000, None, 0), (610, 24000, None, 0), (640, 66000, None, 0),
                                              (800, 40001, 40016, 2)])
def test_token_logp_many_rows(nsp, dt, T, V, stride, shift):
    y = scattered(100, T, V)
    x, rows = logits_on(101, y, V, dt, stride, shift)
    logp, lse = nsp.token_logp(x, y, scale=SCALE)
    assert (logp[y < 0] == 0).all() and (lse[y < 0] == 0).all()
    check_logp(x[rows], y[rows], logp[rows], lse[rows])
    again = nsp.token_logp(x, y, scale=SCALE)
    assert torch.equal(again[0], logp) and torch.equal(again[1], lse)
    # whatever the way: one row alone
    for r in (int(rows[0]), int(rows[-1])):
        one, _ = nsp.token_logp(x[r:r + 1], y[r:r + 1], scale=SCALE)
        err = 2 * float(lse_error(f64(x[r:r + 1]))[0]) + 4 * E * abs(float(one[0]))
        assert abs(float(one[0]) - float(logp[r])) <= err
    g = randn(102, T, dt=F32)
    dx = nsp.token_logp_bwd(x, y, lse, g, scale=SCALE)
    assert not dx[y < 0].any()
    check_dlogits(x[rows], y[rows], g[rows], dx[rows], dt)
    none = torch.full_like(y, -1)
    logp, lse = nsp.token_logp(x, none)
    assert not logp.any() and not lse.any()


@pytest.mark.parametrize("scale", [1.0, 0.8, float(np.log(2)), 2 * float(np.log(2)), 0.1, 1 / 3, 1.7, 3.0, 1e-3, 40.0])
@pytest.mark.parametrize("T,V", [(5, 999), (2, 20000), (620, 4999), (610, 16500)])
def test_token_logp_scales(nsp, scale, T, V):
    """Any temperature, whichever way its factor rounds; masked logits; forward and backward."""
    x = randn(105, T, V, dt=F32, scale=2.0)
    x[:, 7:40] = float("-inf")
    y = torch.randint(0, V - 40, (T,), generator=torch.Generator().manual_seed(106), dtype=torch.int32).cuda()
    y = torch.where(y < 7, y, y + 33)
    logp, lse = nsp.token_logp(x, y, scale=scale)
    check_logp(x, y, logp, lse, scale)
    g = randn(107, T, dt=F32)
    check_dlogits(x, y, g, nsp.token_logp_bwd(x, y, lse, g, scale=scale), F32, scale)
    cu = cu_of([T])
    stats, lp, dx = nsp.policy_loss_logits(x, y, logp, torch.ones(1, device="cuda"), cu, scale=scale)
    check_logp(x, y, lp, None, scale)
    # rho = 1 but for the log-probabilities' own errors: the gradient of -mean(logp)
    err = 2 * lse_error(f64(x), scale) + 8 * E * np.abs(f64(lp))
    check_dlogits(x, y, np.full(T, -1.0 / T), dx, F32, scale, dlogp_err=scale * err / T)


def test_token_logp_errors_do_not_lean(nsp):
    """The mean error of thousands of log-probabilities, which a document's sum multiplies by
    their number, is below one's own.  One is off by 3e-7 rms (the roundings of values near
    10); what is the same for all is ex2's mean error, which is taken off as it is over
    uniform arguments, and differs from that by at most its whole, 1e-7, elsewhere.  (One-
    sided roundings of the scale or of the powers of two gave 2e-7 to 3e-7.)"""
    T, V = 3000, 5001
    x, _ = logits_of(108, T, V, BF16)
    y = torch.arange(T, dtype=torch.int32, device="cuda")
    for scale in (1.0, 0.8, 1 / 3, 0.9):
        ref = S.token_logp(f64(x), y.cpu().numpy(), scale)[0]
        for part in (slice(0, T), slice(0, 500)):
            got = nsp.token_logp(x[part], y[part], scale=scale)[0]
            lean = np.mean(f64(got) - ref[part])
            assert abs(lean) <= 1e-7 + 3 * 3e-7 / np.sqrt(len(got)), (scale, part, lean)


def test_token_logp_many_rows_special(nsp):
    """NaN, infinities and targets past the vocabulary stay in their rows, also where many
    rows are on their way at once."""
    T, V = 700, 17000
    x = randn(103, T, V, dt=F32)
    y = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(104), dtype=torch.int32).cuda()
    x[10, 5] = x[200, V - 1] = float("nan")
    x[11, 17] = float("inf")
    x[12] = float("-inf")
    x[13, 40:] = float("-inf")
    y[13] = 3
    y[14] = V
    y[600] = 2 ** 31 - 1
    logp, lse = nsp.token_logp(x, y)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[10, 11, 12, 14, 200, 600]] = True
    assert torch.isnan(logp[bad]).all() and torch.isfinite(logp[~bad]).all() and torch.isfinite(lse[14])
    check_logp(x[~bad], y[~bad], logp[~bad], lse[~bad], 1.0)


@pytest.mark.parametrize("dt,T,V,stride,shift,every", [
    (BF16, 612, 4200, None, 0, 1), (F32, 700, 4111, None, 3, 1), (BF16, 640, 20001, None, 1, 1),
    (F32, 620, 12288, None, 0, 1), (BF16, 1000, 33000, 33008, 0, 3), (F32, 310, 50001, None, 0, 2),
    (BF16, 330, 131072, None, 0, 4), (BF16, 320, 140001, None, 1, 5), (F32, 200, 140000, None, 0, 3),
    (BF16, 160, 300001, None, 0, 4), (F32, 100, 200000, None, 0, 2), (BF16, 620, 49999, None, 0, 2),
    (F32, 640, 16389, None, 1, 3), (BF16, 620, 500, None, 0, 1), (BF16, 700, 1001, 1016, 3, 1),
    (F32, 610, 1000, None, 0, 1), (F32, 612, 3001, None, 2, 1), (BF16, 615, 8190, None, 0, 1),
    (F32, 612, 6002, None, 0, 2), (BF16, 611, 24001, 24008, 1, 2), (F32, 609, 16000, None, 0, 3)])
@pytest.mark.parametrize("mean", ["documents", "tokens"])
def test_policy_loss_logits_many_rows(nsp, dt, T, V, stride, shift, every, mean):
    """Rows shared by up to eight blocks, odd vocabularies at any distance from a 16-byte
    border; rows behind the last document; outputs whole, in place the same bits."""
    lens = [T // 3, 0, 1, T // 2, T - T // 3 - T // 2 - 4]
    cu, y = cu_of(lens), scattered(110, T, V, every)
    x, _ = logits_on(111, y, V, dt, stride, shift)
    scored = y.clone()
    scored[sum(lens):] = -1
    rows = torch.nonzero(scored >= 0)[:, 0]
    rng = np.random.default_rng(112)
    lp = np.zeros(T)
    r = rows.cpu().numpy()
    lp[r] = S.token_logp(f64(x[rows]), scored[rows].cpu().numpy(), SCALE)[0]
    d = rng.normal(size=T) * 0.3
    for border in (np.log(0.8), np.log(1.25)):
        d = np.where(np.abs(d - border) < 1e-3, border + 2e-3, d)
    old, ref = (torch.tensor(lp + o, dtype=torch.float32, device="cuda") for o in (-d, rng.normal(size=T) * 0.5))
    adv = torch.tensor(rng.normal(size=len(lens)), dtype=torch.float32, device="cuda")
    kw = dict(clip_low=0.2, clip_high=0.25, kl_coef=0.07, mean=mean)
    out = torch.full((T * (stride or V) + shift + 64,), 7.0, dtype=dt, device="cuda")
    view = out[shift:shift + T * (stride or V)].view(T, stride or V)[:, :V]
    stats, logp, dx = nsp.policy_loss_logits(x, y, old, adv, cu, ref=ref, scale=SCALE, out=view, **kw)
    assert (logp[scored < 0] == 0).all()
    check_logp(x[rows], scored[rows], logp[rows], None)
    dl_ref = S.policy_loss(lp, f64(old), f64(ref), f64(adv), scored.cpu().numpy(), cu.cpu().numpy(),
                           float(np.float32(0.2)), 0.25, float(np.float32(0.07)), mean)[1]
    two, dl = nsp.policy_loss(logp, y, old, adv, cu, ref=ref, **kw)
    err = np.zeros(T)
    err[r] = lse_error(f64(x[rows])) + 2 * E * np.abs(lp[r])
    lw = torch.tensor(lp, device="cuda")
    check_policy(lw, scored, old, ref, adv, cu, stats, dl, kw, logp_err=err)
    torch.testing.assert_close(stats, two, rtol=8 * E, atol=8 * E * float(two.abs().max()))
    dl_err = np.abs(f64(dl) - dl_ref) + 4 * E * np.abs(dl_ref)
    check_dlogits(x[rows], scored[rows], dl_ref[r], dx[rows], dt, dlogp_err=SCALE * dl_err[r])
    assert not dx[scored < 0].any()
    keep = view.clone()
    view[:] = 7.0
    assert (out == 7).all()
    # another distance from the border, and in place
    two, _, other = nsp.policy_loss_logits(x, y, old, adv, cu, ref=ref, scale=SCALE,
                                           out=torch.empty(T * V + 1, dtype=dt, device="cuda")[1:].view(T, V), **kw)
    assert torch.equal(other, keep) and torch.equal(two, stats)
    _, _, same = nsp.policy_loss_logits(x, y, old, adv, cu, ref=ref, scale=SCALE, out=x, **kw)
    assert torch.equal(same, keep)


def test_policy_loss_logits_many_rows_edges(nsp):
    """Nothing scored, a bad cu_seqlens, a target past the vocabulary."""
    T, V = 700, 33000
    x = randn(120, T, V)
    y = scattered(121, T, V)
    old, adv = -torch.rand(T, device="cuda"), torch.ones(2, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    none = torch.full_like(y, -1)
    stats, logp, dx = nsp.policy_loss_logits(x, none, old, adv, cu_of([300, 400]), workspace=ws)
    assert not stats.any() and not logp.any() and not dx.any()
    keep = x.clone()
    bad = torch.tensor([0, 500, 400], dtype=torch.int32, device="cuda")
    nsp.policy_loss_logits(x, y, old, adv, bad, workspace=ws, out=x)
    assert nsp.nsp_status_query(ws) == nsp.NSP_ERR_INVALID and torch.equal(x, keep)
    good, _, dgood = nsp.policy_loss_logits(x, y, old, adv, cu_of([300, 400]), workspace=ws)
    assert nsp.nsp_status_query(ws) == nsp.NSP_OK
    y2, row = y.clone(), int(torch.nonzero(y >= 0)[5, 0])
    y2[row] = V + 3
    stats, logp, dx = nsp.policy_loss_logits(x, y2, old, adv, cu_of([300, 400]), workspace=ws)
    assert torch.isnan(stats[0]) and torch.isnan(logp[row]) and torch.isnan(dx[row]).all()
    rest = torch.arange(T, device="cuda") != row
    assert torch.equal(dx[rest], dgood[rest])


def test_qk_norm_rope_far_rows(nsp):
    """Offsets past 32 bits, both directions, in place."""
    T, h, d = 270000, 64, 128                 # 2.2e9 elements
    cu, fr, w = cu_of([T - 7, 7]), nsp.rope_freqs(d, device="cuda"), randn(60, d)
    x = torch.zeros((T, h, d), dtype=BF16, device="cuda")
    x[-9:] = few = randn(61, 9, h, d)
    pos = torch.tensor([T - 9, T - 8, 0, 1, 2, 3, 4, 5, 6], dtype=torch.int32, device="cuda")
    y, _ = nsp.qk_norm_rope(x, None, cu, fr, w)
    ref, _ = nsp.qk_norm_rope(few, None, None, fr, w, positions=pos)
    assert torch.equal(y[-9:], ref) and not y[:-9].any()
    dx = nsp.qk_norm_rope_bwd(x, None, y, None, cu, fr, w, out=(y, None))[0]
    ref = nsp.qk_norm_rope_bwd(few, None, ref, None, None, fr, w, positions=pos)[0]
    assert torch.equal(dx[-9:], ref) and not dx[:-9].any()


# ----------------------------------------------------------------------------- all of them

def step_calls(nsp, seed, T=700, V=33000, ws=None, stream=None):
    """The operators on one set of inputs: [(name, call, outputs' number)]; ws: a workspace for each."""
    lens = [T // 2, 0, T // 4, T - T // 2 - T // 4]
    cu = cu_of(lens)
    q, k = randn(seed, T, 6, 64), randn(seed + 1, T, 2, 64)
    gq, gk, wq, wk = randn(seed + 2, T, 6, 64), randn(seed + 3, T, 2, 64), randn(seed + 4, 64), randn(seed + 5, 64)
    fr = nsp.rope_freqs(64, device="cuda")
    y = scattered(seed + 6, T, V)
    x, few = randn(seed + 7, T, V), randn(seed + 8, 40, V)
    y40, cu40 = y[:40].clone(), cu_of([13, 20])
    logp = -torch.rand(T, generator=torch.Generator().manual_seed(seed)).cuda()
    adv = randn(seed + 9, 4, dt=F32)
    grads = [randn(seed + 10 + i, n, dt=(F32, BF16)[i % 2]) for i, n in enumerate((70000, 5, 4097, 33))]
    st = dict(stream=stream)

    def w(i):
        return dict(st, workspace=None if ws is None else ws[i])
    lse = nsp.token_logp(x, y)[1]
    torch.cuda.synchronize()
    return [lambda: nsp.qk_norm_rope(q, k, cu, fr, wq, wk, **st),
            lambda: nsp.qk_norm_rope_bwd(q, k, gq, gk, cu, fr, wq, wk, **w(0)),
            lambda: nsp.token_logp(x, y, **w(1)),
            lambda: nsp.token_logp(few, y40, **w(2)),
            lambda: (nsp.token_logp_bwd(x, y, lse, logp, **st),),
            lambda: nsp.policy_loss(logp, y, logp * 0.9, adv, cu, ref=logp * 1.1, kl_coef=0.1, **w(3)),
            lambda: nsp.policy_loss_logits(x, y, logp, adv, cu, ref=logp, kl_coef=0.1, **w(4)),
            lambda: nsp.policy_loss_logits(few, y40, logp[:40], adv[:2], cu40, **w(5)),
            lambda: nsp.preference_loss(logp, y, cu, ref=logp * 0.5, **w(6)),
            lambda: (nsp.grad_norm(grads, **w(7)),),
            lambda: (lambda o: (nsp.clip_grads(grads, 0.5, out=o, **w(8)), *o))([torch.empty_like(g) for g in grads])]


def test_step_guard_zones(nsp):
    """Workspaces of exactly the asked size, and what lies behind them and the outputs, in
    arrays of one buffer one behind the other, stays as it was."""
    import ctypes as C
    lib = nsp.load()
    T, V, lens = 700, 33000, [350, 0, 175, 175]
    cu, y, x = cu_of(lens), scattered(130, T, V), randn(131, T, V)
    logp, adv = -torch.rand(T, device="cuda"), torch.ones(4, device="cuda")
    zone = 4096

    def guarded(nbytes):
        buf = torch.full((nbytes + 2 * zone,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[zone:zone + nbytes]

    def intact(buf):
        return bool((buf[:zone] == 0xA5).all()) and bool((buf[-zone:] == 0xA5).all())

    q, gq, w = randn(132, T, 6, 64), randn(133, T, 6, 64), randn(134, 64)
    fr = nsp.rope_freqs(64, device="cuda")
    desc = (nsp.QkTensor * 1)(nsp.QkTensor(heads=6))
    sizes = {"qk": lib.nsp_qk_norm_rope_bwd_workspace_size(C.addressof(desc), 1, T, 64),
             "logp": lib.nsp_token_logp_workspace_size(T),
             "policy": lib.nsp_policy_loss_workspace_size(T, 4, 0), "logits": lib.nsp_policy_loss_workspace_size(T, 4, 1),
             "preference": lib.nsp_preference_loss_workspace_size(4)}
    ws = {n: guarded(s) for n, s in sizes.items()}
    ob, o = guarded(T * V * 2)
    dx = o.view(torch.bfloat16).view(T, V)
    qb, qo = guarded(T * 6 * 64 * 2)
    dq = qo.view(torch.bfloat16).view(T, 6, 64)
    nsp.qk_norm_rope_bwd(q, None, gq, None, cu, fr, w, out=(dq, None), workspace=ws["qk"][1])
    nsp.token_logp(x, y, workspace=ws["logp"][1])
    nsp.policy_loss(logp, y, logp, adv, cu, workspace=ws["policy"][1])
    nsp.policy_loss_logits(x, y, logp, adv, cu, out=dx, workspace=ws["logits"][1])
    nsp.preference_loss(logp, y, cu, workspace=ws["preference"][1])
    grads = [randn(135, n) for n in (3, 5000, 40001)]
    counts = (C.c_int64 * 3)(3, 5000, 40001)
    ws["grad"] = guarded(lib.nsp_grad_norm_workspace_size(counts, 3))
    outs = [guarded(g.numel() * 2) for g in grads]
    nsp.clip_grads(grads, 0.1, out=[v.view(torch.bfloat16) for _, v in outs], workspace=ws["grad"][1])
    torch.cuda.synchronize()
    assert all([intact(b) for b, _ in list(ws.values()) + outs]) and intact(ob) and intact(qb)


def test_step_captured_and_replayed(nsp):
    """Every operator in one captured graph, replayed while eager calls run between: the
    bits of the eager calls, as often as it is replayed."""
    calls = step_calls(nsp, 140)
    eager = [c() for c in calls]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for c in calls:
            c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [c() for c in calls]
    for _ in range(3):
        for o in outs:
            for t in o:
                if t is not None:
                    t.fill_(-3.0)
        graph.replay()
        for c in calls:
            c()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, eager)):
            for s, t in zip(a, b):
                assert (s is None and t is None) or torch.equal(s, t), i


def test_step_two_streams(nsp):
    """Two sets of inputs on two streams at once, each with its own workspaces, several times:
    the bits of each alone."""
    sets = [step_calls(nsp, 150), step_calls(nsp, 180, T=900, V=33001)]
    alone = [[c() for c in calls] for calls in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [[], []]
        for i in range(len(sets[0])):
            for j in (0, 1):
                with torch.cuda.stream(streams[j]):
                    got[j].append(sets[j][i]())
        torch.cuda.synchronize()
        for j in (0, 1):
            for i, (a, b) in enumerate(zip(got[j], alone[j])):
                for s, t in zip(a, b):
                    assert (s is None and t is None) or torch.equal(s, t), (j, i)


def test_step_stream_argument(nsp):
    """A given stream in place of the current one."""
    side = torch.cuda.Stream()
    alone = [c() for c in step_calls(nsp, 200)]
    torch.cuda.synchronize()
    got = [c() for c in step_calls(nsp, 200, stream=side)]
    side.synchronize()
    for a, b in zip(got, alone):
        for s, t in zip(a, b):
            assert (s is None and t is None) or torch.equal(s, t)


FIRST_CALL_CAPTURED = """
import torch
import test_step_gpu as t
from variable_length_sequence_gb300 import nsp
g = torch.cuda.CUDAGraph()
q, w = t.randn(1, 300, 4, 64), t.randn(2, 64)
cu, fr = t.cu_of([200, 100]), nsp.rope_freqs(64, device="cuda")
x, y = t.randn(3, 700, 33000), t.scattered(4, 700, 33000)
logp, adv, docs = -torch.rand(700, device="cuda"), torch.ones(2, device="cuda"), t.cu_of([300, 400])
grads = [t.randn(5, 5000)]
torch.cuda.synchronize()
with torch.cuda.graph(g):
    a = nsp.qk_norm_rope_bwd(q, None, q, None, cu, fr, w)[0]
    b = nsp.token_logp(x, y)[0]
    c = nsp.policy_loss_logits(x, y, logp, adv, docs)[2]
    d = nsp.preference_loss(logp, y, docs)[2]
    e = nsp.grad_norm(grads)
g.replay()
torch.cuda.synchronize()
assert torch.equal(a, nsp.qk_norm_rope_bwd(q, None, q, None, cu, fr, w)[0])
assert torch.equal(b, nsp.token_logp(x, y)[0])
assert torch.equal(c, nsp.policy_loss_logits(x, y, logp, adv, docs)[2])
assert torch.equal(d, nsp.preference_loss(logp, y, docs)[2])
assert torch.equal(e, nsp.grad_norm(grads))
print("same bits")
"""


def test_step_first_call_captured():
    """A process whose first call of an operator is a captured one."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stderr[-2000:]


def model64(p, tokens, lens, heads, loss):
    """An attention layer and its logits in float64; loss(logits) and its gradients."""
    p = {n: v.detach().cpu().double().requires_grad_() for n, v in p.items()}
    hq, hkv, d = heads
    x = p["embed"][tokens]
    T = len(tokens)
    qkv = (x @ p["qkv"]).view(T, hq + 2 * hkv, d)
    pos = torch.cat([torch.arange(n, dtype=torch.float64) for n in lens])
    freqs = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    turn = torch.polar(torch.ones(T, d // 2, dtype=torch.float64), torch.outer(pos, freqs))[:, None]

    def norm_rope(v, w):
        n = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w
        z = torch.complex(n[..., :d // 2], n[..., d // 2:]) * turn
        return torch.cat([z.real, z.imag], -1)
    q, k, v = norm_rope(qkv[:, :hq], p["wq"]), norm_rope(qkv[:, hq:hq + hkv], p["wk"]), qkv[:, hq + hkv:]
    k, v = (t.repeat_interleave(hq // hkv, 1) for t in (k, v))
    doc = torch.cat([torch.full((n,), i) for i, n in enumerate(lens)])
    seen = (doc[:, None] == doc[None]) & torch.ones(T, T).tril().bool()
    a = torch.einsum("thd,jhd->htj", q, k) * d ** -0.5
    a = torch.softmax(a.masked_fill(~seen, float("-inf")), -1)
    o = torch.einsum("htj,jhd->thd", a, v).reshape(T, hq * d)
    value = loss((x + o @ p["out"]) @ p["embed"].T)
    return value, dict(zip(p, torch.autograd.grad(value, list(p.values()))))


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_step_of_a_model(nsp, kind):
    """A training step as it would be run, float32: fused projection, norm and rotation from
    its columns, attention, logits, loss, all the way back into the fused projection's
    gradient, and all gradients clipped: against float64 autograd of the whole, and against
    differences of the float64 loss.  Everything is float32 with sums of at most 500 terms,
    six matrix products deep: 1e-4 of each gradient's norm is 50 times the roundings of
    such a sum of random terms (sqrt(500) E a product)."""
    torch.backends.cuda.matmul.allow_tf32 = False
    hq, hkv, d, D, V, lens = 4, 2, 64, 96, 300, [40, 1, 70, 33]
    T = sum(lens)
    gen = torch.Generator().manual_seed(7)
    rand = lambda *s, scale=1.0: (torch.randn(s, generator=gen) * scale).cuda()  # noqa: E731
    p = {"embed": rand(V, D), "qkv": rand(D, (hq + 2 * hkv) * d, scale=D ** -0.5), "out": rand(hq * d, D, scale=(hq * d) ** -0.5),
         "wq": 1 + rand(d, scale=0.1), "wk": 1 + rand(d, scale=0.1)}
    tokens = torch.randint(0, V, (T,), generator=gen)
    cu = cu_of(lens)
    targets = torch.cat([tokens[1:], tokens[:1]]).to(torch.int32)
    first = 0
    for n in lens:                          # prompts, and rows without a next token
        targets[first:first + n // 3] = -1
        targets[first + n - 1] = -1
        first += n
    fr = nsp.rope_freqs(d, device="cuda")
    old, ref = rand(T, scale=0.1) - 6, rand(T, scale=0.3) - 6
    adv = rand(len(lens))

    x = p["embed"][tokens.cuda()]
    qkv = (x @ p["qkv"]).view(T, hq + 2 * hkv, d)
    q, k = nsp.qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], cu, fr, p["wq"], p["wk"])
    v = qkv[:, hq + hkv:].contiguous()
    out, lse = nsp.attn_fwd(q, k, v, cu)
    h = x + out.view(T, -1) @ p["out"]
    logits = h @ p["embed"].T
    y = targets.cuda()
    if kind == "policy":
        old = nsp.token_logp(logits, y)[0] + 0.1 * (old + 6)
        ref = old + 0.3 * (ref + 6)
        stats, _, dlogits = nsp.policy_loss_logits(logits, y, old, adv, cu, ref=ref, kl_coef=0.1, mean="documents")
    else:
        logp, row_lse = nsp.token_logp(logits, y)
        stats, _, dlogp = nsp.preference_loss(logp, y, cu, ref=ref, beta=0.1, smoothing=0.1)
        dlogits = nsp.token_logp_bwd(logits, y, row_lse, dlogp)
    dh = dlogits @ p["embed"]
    grads = {"embed": dlogits.T @ h, "out": out.view(T, -1).T @ dh}
    dout = (dh @ p["out"].T).view(T, hq, d).contiguous()
    dq, dk, dv = nsp.attn_bwd(q, k, v, out, dout, lse, cu)
    dqkv = torch.empty_like(qkv)
    dqkv[:, hq + hkv:] = dv
    _, _, grads["wq"], grads["wk"] = nsp.qk_norm_rope_bwd(
        qkv[:, :hq], qkv[:, hq:hq + hkv], dq, dk, cu, fr, p["wq"], p["wk"], out=(dqkv[:, :hq], dqkv[:, hq:hq + hkv]))
    dqkv = dqkv.view(T, -1)
    grads["qkv"] = x.T @ dqkv
    grads["embed"].index_add_(0, tokens.cuda(), dh + dqkv @ p["qkv"].T)
    norm = nsp.clip_grads(list(grads.values()), 0.25, unscale=0.5)

    yc, o64, r64, a64 = targets.long(), old.cpu().double(), ref.cpu().double(), adv.cpu().double()

    def loss(z):
        lp = torch.log_softmax(z, -1).gather(1, yc.clamp(min=0)[:, None])[:, 0]
        parts, first, scores = [], 0, []
        for b, n in enumerate(lens):
            rows = [t for t in range(first, first + n) if yc[t] >= 0]
            first += n
            scores.append((lp[rows] - r64[rows]).sum())
            if rows:
                rho = torch.exp(lp[rows] - o64[rows])
                far = r64[rows] - lp[rows]
                pg = -torch.min(rho * a64[b], rho.clamp(0.8, 1.2) * a64[b])
                parts.append((pg + 0.1 * (torch.exp(far) - far - 1)).mean())
        if kind == "policy":
            return torch.stack(parts).mean()
        hs = 0.1 * (torch.stack(scores[0::2]) - torch.stack(scores[1::2]))
        ls = torch.nn.functional.logsigmoid
        return -(0.9 * ls(hs) + 0.1 * ls(-hs)).mean()

    heads = (hq, hkv, d)
    value, want = model64(p, tokens, lens, heads, loss)
    value = float(value.detach())
    assert abs(float(stats[0]) - value) <= 1e-4 * max(1.0, abs(value))
    total = 0.5 * float(torch.sqrt(sum((g ** 2).sum() for g in want.values())))
    assert abs(float(norm) - total) <= 1e-4 * total
    factor = 0.5 * min(1.0, 0.25 / (total + 1e-6))
    for n, g in want.items():
        off = (grads[n].cpu().double() - factor * g).norm() / (factor * g).norm()
        assert off <= 1e-4, (n, float(off))
    # differences of the whole along a random direction of all parameters
    dirs = {n: torch.randn(v.shape, generator=gen).double() for n, v in p.items()}
    f = [float(model64({n: v.cpu().double() + s * dirs[n] for n, v in p.items()}, tokens, lens, heads, loss)[0])
         for s in (1e-6, -1e-6)]
    along = sum(float((grads[n].cpu().double() * dirs[n]).sum()) for n in p) / factor
    size = sum(float((grads[n].cpu().double() * dirs[n]).norm()) for n in p) / factor
    assert abs((f[0] - f[1]) / 2e-6 - along) <= 1e-3 * size
