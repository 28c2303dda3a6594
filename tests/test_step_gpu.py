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
