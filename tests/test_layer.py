"""Differential attention layer on the host: the float64 oracle against torch
autograd and differences, the frequency helper, and every refusal of the new
entry points (made before any CUDA call)."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import oracle.layer as L
from variable_length_sequence_gb300 import build as nsp_build
from variable_length_sequence_gb300 import nsp


@pytest.fixture(scope="module")
def lib():
    nsp_build.build()
    return nsp.load()


# ----------------------------------------------------------------------------- oracle

CU = [0, 4, 4, 5, 12]


def _diff_inputs(seed, T=12, Hq=4, Hkv=2, d=8, tokens=False):
    rng = np.random.default_rng(seed)
    return (rng.normal(size=(T, Hq, d)), rng.normal(size=(T, Hkv, d)), rng.normal(size=(T, Hkv, d)),
            rng.uniform(-0.3, 0.9, size=(Hq, T if tokens else 1)), rng.normal(size=(T, Hq, d)))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tokens", [True, False])
def test_oracle_diff_attention_against_autograd(causal, tokens):
    q, k, v, lam, do = _diff_inputs(1, tokens=tokens)
    T, Hq, d = q.shape
    leaves = [torch.tensor(x, requires_grad=True) for x in (q, k, v, lam)]
    tq, tk, tv, tl = leaves
    doc = np.searchsorted(CU, np.arange(T), side="right")
    mask = doc[:, None] == doc[None]
    if causal:
        mask &= np.tril(np.ones((T, T), bool))
    bias = torch.tensor(np.where(mask, 0.0, -np.inf))
    rep = Hq // 2

    def one(m):
        c = slice(m * d // 2, (m + 1) * d // 2)
        x = torch.einsum("ihc,jhc->hij", tq[..., c], tk[..., c].repeat_interleave(rep, 1)) * 0.5
        return torch.einsum("hij,jhc->ihc", torch.softmax(x + bias, -1), tv.repeat_interleave(rep, 1))

    out = one(0) - tl.expand(Hq, T).T[..., None] * one(1)
    grads = torch.autograd.grad(out, leaves, torch.tensor(do))
    ro, ro2, _ = L.diff_attn_fwd(q, k, v, lam, CU, 0.5, causal)
    np.testing.assert_allclose(ro, out.detach(), atol=1e-13)
    np.testing.assert_allclose(ro2, one(1).detach(), atol=1e-13)
    for a, b in zip(L.diff_attn_bwd(q, k, v, lam, do, CU, 0.5, causal), grads):
        np.testing.assert_allclose(a, b, atol=1e-12)


def test_oracle_diff_attention_against_differences():
    q, k, v, lam, do = _diff_inputs(2)
    grads = L.diff_attn_bwd(q, k, v, lam, do, CU, 0.5)
    rng = np.random.default_rng(3)
    for i, g in enumerate(grads):
        dirn = rng.normal(size=g.shape)
        f = []
        for e in (1e-6, -1e-6):
            x = [q, k, v, lam]
            x[i] = x[i] + e * dirn
            f.append((L.diff_attn_fwd(*x, CU, 0.5)[0] * do).sum())
        assert abs((f[0] - f[1]) / 2e-6 - (g * dirn).sum()) < 1e-6


def test_oracle_lambda_and_norm_against_autograd():
    rng = np.random.default_rng(4)
    for n in (1, 5):
        vec = [rng.normal(size=(n, 7)) * 0.3 for _ in range(4)]
        t = [torch.tensor(x, requires_grad=True) for x in vec]
        lam = ((t[0] * t[1]).sum(-1).exp() - (t[2] * t[3]).sum(-1).exp() + 0.4).expand(5)
        np.testing.assert_allclose(L.diff_lambda(*vec, 5, 0.4), lam.detach(), rtol=1e-13)
        g = rng.normal(size=5)
        for a, b in zip(L.diff_lambda_bwd(g, *vec), torch.autograd.grad(lam, t, torch.tensor(g))):
            np.testing.assert_allclose(a, b, rtol=1e-12)
    x, gate, dy, w = (rng.normal(size=s) for s in ((3, 2, 8), (3, 2, 8), (3, 2, 8), (8,)))
    tx, tg, tw = (torch.tensor(a, requires_grad=True) for a in (x, gate, w))
    y = 0.3 * tx * torch.rsqrt(tx.square().mean(-1, keepdim=True) + 1e-3) * tw * torch.sigmoid(tg)
    np.testing.assert_allclose(L.head_norm(x, w, gate, 1e-3, 0.3), y.detach(), rtol=1e-13)
    ref = torch.autograd.grad(y, (tx, tw, tg), torch.tensor(dy))
    for a, b in zip(L.head_norm_bwd(x, dy, w, gate, 1e-3, 0.3), ref):
        np.testing.assert_allclose(a, b, rtol=1e-11, atol=1e-14)


def test_oracle_rope():
    freqs = np.array([1.0, 0.25, 1e-3])
    a = L.rope_angles([0, 1, 7, 399999], freqs)
    pos = np.array([0, 1, 7, 399999.0])[:, None]
    np.testing.assert_allclose(np.cos(a), np.cos(pos * freqs), atol=1e-9)
    x = np.random.default_rng(5).normal(size=(4, 2, 8))
    for inter in (False, True):
        y = L.rope(x, a, 6, inter)
        np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        np.testing.assert_allclose(L.rope(y, a, 6, inter, inverse=True), x, atol=1e-14)
        np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
        z = x[..., 0:6:2] + 1j * x[..., 1:6:2] if inter else x[..., :3] + 1j * x[..., 3:6]
        z = z * np.exp(1j * a)[:, None]
        got = y[..., 0:6:2] + 1j * y[..., 1:6:2] if inter else y[..., :3] + 1j * y[..., 3:6]
        np.testing.assert_allclose(got, z, atol=1e-14)
    np.testing.assert_array_equal(L.rope_positions([0, 2, 2, 5], 6, 1), [1, 0, 1, 2, -1, -1])


# ----------------------------------------------------------------------------- frequencies

def test_rope_freqs(lib):
    i = np.arange(0, 64, 2)
    f = 1e4 ** (-i / 64)
    np.testing.assert_allclose(nsp.rope_freqs(64), f, rtol=1e-15)
    np.testing.assert_allclose(nsp.rope_freqs(64, scaling="linear", factor=4), f / 4, rtol=1e-15)
    b = nsp.rope_freqs(64, scaling="base", factor=8).numpy()
    np.testing.assert_allclose(b, (1e4 * 8 ** (64 / 62)) ** (-i / 64), rtol=1e-14)
    assert b[0] == 1 and abs(b[-1] / (f[-1] / 8) - 1) < 1e-12
    p = nsp.rope_freqs(64, scaling="parts", factor=8, low=1, high=32, orig_len=4096).numpy()
    turns = 4096 * f / (2 * math.pi)
    k = np.clip((turns - 1) / 31, 0, 1)
    np.testing.assert_allclose(p, k * f + (1 - k) * f / 8, rtol=1e-14)
    assert p[0] == f[0] and abs(p[-1] / (f[-1] / 8) - 1) < 1e-12
    for kw in ({"rot": 63}, {"rot": 0}, {"rot": 2048}, {"base": 0.0}, {"base": float("nan")},
               {"scaling": "linear", "factor": 0.5}, {"scaling": "parts", "factor": 2},
               {"scaling": "parts", "factor": 2, "low": 3, "high": 3, "orig_len": 10},
               {"scaling": "base", "factor": 2, "rot": 2}):
        with pytest.raises(nsp.NspError):
            nsp.rope_freqs(**{"rot": 64, **kw})
    with pytest.raises(ValueError):
        nsp.rope_freqs(64, scaling="other")


# ----------------------------------------------------------------------------- refusals

A = 1 << 24          # made-up aligned addresses: every call below is refused before any launch


def _rope(lib, tensors=None, **kw):
    a = dict(n=None, cu=A, ndoc=2, pos=None, start=0, len=10, d=128, rot=128, freqs=A + 4096, inter=0,
             m=1.0, inverse=0, io=nsp.NSP_BF16)
    a.update(kw)
    tensors = [(A + (1 << 20), A + (2 << 20), 0, 0, 4, 1)] if tensors is None else tensors
    arr = (nsp.RopeTensor * max(1, len(tensors)))(*[nsp.RopeTensor(*t) for t in tensors])
    return lib.nsp_rope(C.addressof(arr), len(tensors) if a["n"] is None else a["n"], a["cu"],
                        a["ndoc"], a["pos"], a["start"], a["len"], a["d"], a["rot"], a["freqs"],
                        a["inter"], a["m"], a["inverse"], a["io"], None)


X, Y = A + (1 << 20), A + (2 << 20)
INVALID, UNSUPPORTED, ALIGN = nsp.NSP_ERR_INVALID, nsp.NSP_ERR_UNSUPPORTED, nsp.NSP_ERR_ALIGN


@pytest.mark.parametrize("kw", [
    {"pos": Y + 64}, {"pos": Y - 36}, {"pos": Y + 10 * 1024 - 4}, {"freqs": Y}, {"freqs": Y - 504}, {"cu": Y + 4},
    {"cu": Y - 8}, {"cu": Y + 2048 * 9, "tensors": [(X, Y, 0, 1024, 4, 1)]},
    {"freqs": Y, "tensors": [(Y, Y, 0, 0, 4, 1)]},                      # (in place as well)
])
def test_rope_outputs_over_what_it_reads(lib, kw):
    """An output over the positions, the frequencies or the documents is refused."""
    assert _rope(lib, **kw) == INVALID


def test_rope_outputs_beside_what_it_reads(lib):
    """Neighbours are not (checked with no rows, which launches nothing)."""
    assert _rope(lib, len=0, pos=Y, freqs=Y, cu=Y) == nsp.NSP_OK


@pytest.mark.parametrize("kw,expect", [
    ({"n": 0}, INVALID), ({"n": 5}, INVALID), ({"cu": None}, INVALID), ({"ndoc": 0}, INVALID),
    ({"len": -1}, INVALID), ({"start": -1}, INVALID), ({"rot": 63}, INVALID), ({"rot": 130}, INVALID),
    ({"rot": 0}, INVALID), ({"d": 2000}, UNSUPPORTED), ({"freqs": None}, INVALID),
    ({"inter": 2}, INVALID), ({"inverse": -1}, INVALID), ({"io": 5}, INVALID),
    ({"m": float("inf")}, INVALID), ({"len": 1 << 31}, UNSUPPORTED),
    ({"start": (1 << 30) - 5}, UNSUPPORTED), ({"freqs": A + 4}, ALIGN), ({"cu": A + 2}, ALIGN),
    ({"tensors": [(X, X + 256, 0, 0, 4, 1)]}, INVALID),                 # overlaps itself
    ({"tensors": [(X, X, 0, 0, 4, 2)]}, INVALID),                       # regrouped in place
    ({"tensors": [(X, X, 1024, 512, 4, 1)]}, INVALID),                  # in place, other stride
    ({"tensors": [(X, Y, 0, 0, 4, 3)]}, INVALID), ({"tensors": [(X, Y, 0, 0, 0, 1)]}, INVALID),
    ({"tensors": [(X, Y, 500, 0, 4, 1)]}, INVALID),                     # stride below a row
    ({"tensors": [(X, Y, 0, 1024, 4, 2)]}, INVALID),                    # grouped side packed
    ({"tensors": [(0, Y, 0, 0, 4, 1)]}, INVALID), ({"tensors": [(X + 1, Y, 0, 0, 4, 1)]}, ALIGN),
    ({"tensors": [(X, Y, 0, 0, 1 << 20, 1)]}, UNSUPPORTED),
    # q's output over k's input columns of one fused tensor
    ({"tensors": [(X, X + 1024, 1024, 1024, 4, 1), (X + 1024, Y, 1024, 0, 4, 1)]}, INVALID),
    ({"tensors": [(X, Y, 0, 0, 4, 1), (X, Y, 0, 0, 4, 1)]}, INVALID),   # the same output twice
    ({"len": 0}, nsp.NSP_OK),
    ({"len": 0, "tensors": [(0, 0, 0, 0, 4, 1)]}, nsp.NSP_OK),
])
def test_rope_refusals(lib, kw, expect):
    assert _rope(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"n": 2}, INVALID), ({"dl": 0}, INVALID), ({"heads": 0}, INVALID), ({"io": 9}, INVALID),
    ({"q1": None}, INVALID), ({"k2": A + 1}, ALIGN), ({"lam": None}, INVALID),
    ({"init": float("nan")}, INVALID), ({"heads": 1 << 20, "n": 1}, UNSUPPORTED),
])
def test_lambda_refusals(lib, kw, expect):
    a = dict(q1=A, k1=A + 4096, q2=A + 8192, k2=A + 12288, n=4, dl=64, heads=4, init=0.8,
             io=nsp.NSP_BF16, lam=A + 16384)
    a.update(kw)
    vec = [a[x] for x in ("q1", "k1", "q2", "k2")]
    assert lib.nsp_diff_lambda_fwd(*vec, a["n"], a["dl"], a["heads"], a["init"], a["io"], a["lam"],
                                   None) == expect
    if "init" not in kw:
        assert lib.nsp_diff_lambda_bwd(a["lam"], *vec, a["n"], a["dl"], a["heads"], a["io"],
                                       A + 20480, A + 24576, A + 28672, A + 32768, None) == expect


@pytest.mark.parametrize("lam", [A, A + 508, A + 4096 + 64, A + 8192 + 510, A + 12288 - 6])
def test_lambda_over_a_vector(lib, lam):
    """Vectors of 4 x 64 bf16 (512 bytes), lambda of 4 (8 bytes)."""
    assert lib.nsp_diff_lambda_fwd(A, A + 4096, A + 8192, A + 12288, 4, 64, 4, 0.8, nsp.NSP_BF16, lam,
                                   None) == INVALID


@pytest.mark.parametrize("kw,expect", [
    ({"heads": 0}, INVALID), ({"d": 0}, INVALID), ({"d": 60}, UNSUPPORTED), ({"d": 1024}, UNSUPPORTED),
    ({"tokens": -1}, INVALID), ({"tokens": 1 << 31}, UNSUPPORTED), ({"eps": 0.0}, INVALID),
    ({"scale": float("inf")}, INVALID), ({"io": 3}, INVALID), ({"x": None}, INVALID),
    ({"x": A + 8}, ALIGN), ({"gate": A + 8}, ALIGN), ({"y": None}, INVALID), ({"y": A + 8}, ALIGN),
    ({"stride": 100}, INVALID), ({"stride": 1027}, ALIGN), ({"w": A + 2}, ALIGN),
])
def test_norm_refusals(lib, kw, expect):
    a = dict(x=A, stride=0, w=A + (1 << 20), gate=A + (2 << 20), tokens=10, heads=4, d=128, eps=1e-6,
             scale=1.0, io=nsp.NSP_BF16, y=A + (3 << 20))
    a.update(kw)
    assert lib.nsp_head_norm_fwd(a["x"], a["stride"], a["w"], a["gate"], a["tokens"], a["heads"],
                                 a["d"], a["eps"], a["scale"], a["io"], a["y"], None) == expect
    ws = nsp.load().nsp_head_norm_bwd_workspace_size(10, 4, 128)
    call = lambda ws_ptr, n, dg=A + (4 << 20), gate=a["gate"]: lib.nsp_head_norm_bwd(  # noqa: E731
        a["x"], a["stride"], a["w"], gate, A + (5 << 20), a["tokens"], a["heads"], a["d"], a["eps"],
        a["scale"], a["io"], a["y"], dg, A + (6 << 20), ws_ptr, n, None)
    assert call(A + (7 << 20), max(ws, 1 << 22)) == expect


def test_norm_backward_refusals(lib):
    ws = lib.nsp_head_norm_bwd_workspace_size(10, 4, 128)
    assert ws > 0 and lib.nsp_head_norm_bwd_workspace_size(-1, 4, 128) == 0

    def call(ws_ptr=A + (7 << 20), n=ws, w=A + (1 << 20), gate=A + (2 << 20), dg=A + (4 << 20),
             dw=A + (6 << 20)):
        return lib.nsp_head_norm_bwd(A, 0, w, gate, A + (5 << 20), 10, 4, 128, 1e-6, 1.0,
                                     nsp.NSP_BF16, A + (3 << 20), dg, dw, ws_ptr, n, None)

    assert call(ws_ptr=None) == nsp.NSP_ERR_WORKSPACE
    assert call(n=ws - 1) == nsp.NSP_ERR_WORKSPACE
    assert call(dg=None) == INVALID                     # a gate without its gradient
    assert call(gate=None) == INVALID                   # a gradient without its gate
    assert call(w=None) == INVALID


def test_norm_overlap_refusals(lib):
    """10 tokens of 4 heads of 128 bf16 columns: 10240 bytes an array."""
    x, w, gate, y = A, A + (1 << 20), A + (2 << 20), A + (3 << 20)

    def fwd(y=y, stride=0, gate=gate):
        return lib.nsp_head_norm_fwd(x, stride, w, gate, 10, 4, 128, 1e-6, 1.0, nsp.NSP_BF16, y, None)

    # rows of x 1024 elements apart leave 1024 bytes between them: y fits none of them
    assert fwd(y=x + 1024) == INVALID and fwd(y=gate + 1024) == INVALID and fwd(y=w) == INVALID
    assert fwd(y=x, stride=1024) == INVALID and fwd(y=x - 10240 + 16) == INVALID
    assert fwd(y=x + 1024, stride=1024) == INVALID

    def bwd(dy=A + (5 << 20), dx=y, dg=A + (4 << 20), dw=A + (6 << 20), ws=A + (7 << 20)):
        n = lib.nsp_head_norm_bwd_workspace_size(10, 4, 128)
        return lib.nsp_head_norm_bwd(x, 0, w, gate, dy, 10, 4, 128, 1e-6, 1.0, nsp.NSP_BF16, dx, dg, dw,
                                     ws, n, None)

    for kw in (dict(dx=x), dict(dx=gate), dict(dx=w), dict(dg=y), dict(dg=x), dict(dg=A + (5 << 20)),
               dict(dw=w), dict(dw=gate + 256), dict(ws=y), dict(ws=A + (6 << 20)),
               dict(dx=A + (5 << 20) + 1024)):
        assert bwd(**kw) == INVALID, kw


def test_lambda_overlap_refusals(lib):
    """4 heads of 64 bf16 columns: 512 bytes an array."""
    a = [A + 4096 * i for i in range(9)]                # dlambda, four vectors, four gradients

    def call(**kw):
        p = list(a)
        for i, x in kw.items():
            p[int(i[1:])] = x
        return lib.nsp_diff_lambda_bwd(*p[:5], 4, 64, 4, nsp.NSP_BF16, *p[5:], None)

    for kw in (dict(p5=a[1]), dict(p6=a[1] + 510), dict(p7=a[0] + 6), dict(p8=a[7] - 510), dict(p8=a[5])):
        assert call(**kw) == INVALID, kw


def _diff(lib, back, **kw):
    n = (lib.nsp_diff_attn_bwd_workspace_size(300, 4, 2, 128, nsp.NSP_F32) if back
         else lib.nsp_diff_attn_fwd_workspace_size(300))
    a = dict(q=A, k=A + (1 << 20), v=A + (2 << 20), lam=A + (3 << 20), n_lambda=1, cu=A + (4 << 20),
             ndoc=3, T=300, Hq=4, Hkv=2, d=128, scale=0.125, causal=1, io=nsp.NSP_BF16,
             out=A + (5 << 20), out2=A + (6 << 20), lse=A + (7 << 20), dout=A + (8 << 20),
             dq=A + (9 << 20), dk=A + (10 << 20), dv=A + (11 << 20), dlam=A + (12 << 20),
             ws=A + (13 << 20), ws_bytes=n)
    a.update(kw)
    head = [a[x] for x in ("q", "k", "v", "lam", "n_lambda")]
    mid = [a[x] for x in ("cu", "ndoc", "T", "Hq", "Hkv", "d", "scale", "causal", "io")]
    if back:
        return lib.nsp_diff_attn_bwd(*head, a["out"], a["out2"], a["dout"], a["lse"], *mid, a["dq"],
                                     a["dk"], a["dv"], a["dlam"], a["ws"], a["ws_bytes"], None)
    return lib.nsp_diff_attn_fwd(*head, *mid, a["out"], a["out2"], a["lse"], a["ws"], a["ws_bytes"],
                                 None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,expect", [
    ({"Hq": 5}, INVALID), ({"Hkv": 0}, INVALID), ({"ndoc": 0}, INVALID), ({"d": 96}, UNSUPPORTED),
    ({"causal": 2}, INVALID), ({"io": 2}, INVALID), ({"T": -1}, INVALID), ({"n_lambda": 2}, INVALID),
    ({"scale": 0.0}, INVALID), ({"scale": float("nan")}, INVALID), ({"cu": None}, INVALID),
    ({"T": (1 << 30) + 1, "n_lambda": 1}, UNSUPPORTED), ({"q": None}, INVALID), ({"lam": None}, INVALID),
    ({"k": A + 8}, ALIGN), ({"lam": A + 2}, ALIGN), ({"lse": A + 4}, ALIGN),
    ({"ws": None}, nsp.NSP_ERR_WORKSPACE), ({"ws_bytes": 300}, nsp.NSP_ERR_WORKSPACE),
    ({"Hq": 1 << 16, "Hkv": 1}, UNSUPPORTED),
])
def test_diff_refusals(lib, back, kw, expect):
    assert _diff(lib, back, **kw) == expect


def test_diff_output_alignment(lib):
    for name in ("out", "out2"):
        assert _diff(lib, False, **{name: A + (5 << 20) + 16}) == ALIGN
    for name in ("dq", "dk", "dv"):
        assert _diff(lib, True, **{name: A + (9 << 20) + 16}) == ALIGN
    for name in ("out", "out2", "dout", "lse", "dq", "dk", "dv", "dlam"):
        assert _diff(lib, True, **{name: None}) == INVALID
    assert _diff(lib, False, out=None) == INVALID
    assert lib.nsp_diff_attn_fwd_workspace_size(-1) == 0
    assert lib.nsp_diff_attn_bwd_workspace_size(10, 0, 1, 128, 1) == 0
    assert lib.nsp_diff_attn_bwd_workspace_size((1 << 30) + 1, 4, 4, 128, 1) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        nsp.rope(x, x, cu, torch.ones(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        nsp.head_norm(x)
    with pytest.raises(ValueError):
        nsp.diff_attn_fwd(x, x, x, x[0, :, :1], cu)
    with pytest.raises(ValueError):
        nsp.diff_lambda(x[0], x[0], x[0], x[0], 2, 0.8)
    with pytest.raises(TypeError):
        nsp.head_norm(x.to(torch.float16))
