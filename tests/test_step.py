"""Post-training step on the host: the float64 oracle against torch autograd and
differences, and every refusal of the new entry points (made before any CUDA
call)."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle.layer as L
import oracle.step as S
from variable_length_sequence_gb300 import build as nsp_build
from variable_length_sequence_gb300 import nsp

A = 1 << 24          # made-up aligned addresses: every call below is refused before any launch
INVALID, UNSUPPORTED, ALIGN = nsp.NSP_ERR_INVALID, nsp.NSP_ERR_UNSUPPORTED, nsp.NSP_ERR_ALIGN
WORKSPACE = nsp.NSP_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    nsp_build.build()
    return nsp.load()


# ----------------------------------------------------------------------------- head norm with rotation

@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("weight", [False, True])
def test_oracle_qk_norm_rope_against_autograd(inter, weight):
    rng = np.random.default_rng(1)
    x, dy, w = rng.normal(size=(5, 3, 10)), rng.normal(size=(5, 3, 10)), rng.normal(size=10)
    ang = rng.normal(size=(5, 3))
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    n = tx / torch.sqrt((tx * tx).mean(-1, keepdim=True) + 1e-3)
    if weight:
        n = n * tw
    ia = list(range(0, 6, 2)) if inter else [0, 1, 2]
    ib = list(range(1, 6, 2)) if inter else [3, 4, 5]
    z = torch.complex(n[..., ia], n[..., ib]) * torch.tensor(1.3 * np.exp(1j * ang))[:, None]
    y = n.clone()
    y[..., ia], y[..., ib] = z.real, z.imag
    ref = torch.autograd.grad(y, (tx, tw) if weight else (tx,), torch.tensor(dy))
    rw = w if weight else None
    np.testing.assert_allclose(S.qk_norm_rope(x, rw, ang, 6, inter, 1.3, 1e-3), y.detach(), rtol=1e-12)
    dx, dw = S.qk_norm_rope_bwd(x, rw, dy, ang, 6, inter, 1.3, 1e-3)
    np.testing.assert_allclose(dx, ref[0], rtol=1e-10, atol=1e-13)
    if weight:
        np.testing.assert_allclose(dw, ref[1], rtol=1e-10, atol=1e-13)
    else:
        assert dw is None
    e = 1e-6 * rng.normal(size=x.shape)
    f = [(S.qk_norm_rope(x + s * e, rw, ang, 6, inter, 1.3, 1e-3) * dy).sum() for s in (1, -1)]
    assert abs((f[0] - f[1]) / 2 - (dx * e).sum()) < 1e-11


X, Y = A + (1 << 20), A + (2 << 20)
W, DY, DX, DW = A + (3 << 20), A + (4 << 20), A + (5 << 20), A + (6 << 20)


def _qk(lib, back=False, tensor=None, more=(), **kw):
    """One tensor of 10 tokens x 4 heads x 128 bf16 columns: 10240 bytes an array."""
    a = dict(n=None, cu=A, ndoc=2, pos=None, start=0, len=10, d=128, rot=128, freqs=A + 4096, inter=0,
             m=1.0, eps=1e-6, io=nsp.NSP_BF16, ws=A + (9 << 20), ws_bytes=1 << 20)
    a.update(kw)
    t = dict(x=X, weight=W, y=Y, dy=DY, dx=DX, dweight=DW, x_stride=0, y_stride=0, dx_stride=0,
             heads=4, groups=1)
    t.update(tensor or {})
    every = [t] + [{**t, **m} for m in more]
    arr = (nsp.QkTensor * len(every))(*[nsp.QkTensor(**e) for e in every])
    args = (C.addressof(arr), len(every) if a["n"] is None else a["n"], a["cu"], a["ndoc"], a["pos"],
            a["start"], a["len"], a["d"], a["rot"], a["freqs"], a["inter"], a["m"], a["eps"], a["io"])
    if back:
        return lib.nsp_qk_norm_rope_bwd(*args, a["ws"], a["ws_bytes"], None)
    return lib.nsp_qk_norm_rope_fwd(*args, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,expect", [
    ({"n": 0}, INVALID), ({"n": 5}, INVALID), ({"cu": None}, INVALID), ({"ndoc": 0}, INVALID),
    ({"len": -1}, INVALID), ({"start": -1}, INVALID), ({"rot": 63}, INVALID), ({"rot": 130}, INVALID),
    ({"rot": 0}, INVALID), ({"d": 514, "rot": 64}, UNSUPPORTED), ({"d": 1}, INVALID),
    ({"freqs": None}, INVALID), ({"inter": 2}, INVALID), ({"io": 5}, INVALID),
    ({"m": float("inf")}, INVALID), ({"eps": 0.0}, INVALID), ({"eps": float("nan")}, INVALID),
    ({"len": 1 << 31}, UNSUPPORTED), ({"start": (1 << 30) - 5}, UNSUPPORTED),
    ({"freqs": A + 4}, ALIGN), ({"cu": A + 2}, ALIGN),
    ({"tensor": {"x": 0}}, INVALID), ({"tensor": {"x": X + 1}}, ALIGN), ({"tensor": {"weight": W + 1}}, ALIGN),
    ({"tensor": {"heads": 0}}, INVALID), ({"tensor": {"heads": 1 << 20}}, UNSUPPORTED),
    ({"tensor": {"groups": 3}}, INVALID), ({"tensor": {"x_stride": 500}}, INVALID),
    ({"tensor": {"y_stride": 500}}, INVALID), ({"tensor": {"groups": 2, "y_stride": 1024}}, INVALID),
    ({"tensor": {"x_stride": (1 << 31) + 8}}, UNSUPPORTED),
])
def test_qk_refusals(lib, back, kw, expect):
    assert _qk(lib, back, **kw) == expect


@pytest.mark.parametrize("back,kw", [
    (False, {"tensor": {"y": X + 256}}), (False, {"tensor": {"y": X, "groups": 2}}),
    (False, {"tensor": {"y": X, "x_stride": 1024}}), (False, {"tensor": {"y": W}}),
    (False, {"tensor": {"y": None}}), (False, {"pos": Y + 64}), (False, {"freqs": Y}), (False, {"cu": Y + 8}),
    (False, {"more": [{"x": DX}]}), (False, {"more": [{"x": Y + 512, "y": DX}]}),
    (True, {"tensor": {"dx": X + 256}}), (True, {"tensor": {"dx": DY + 16}}),
    (True, {"tensor": {"dx": DY, "groups": 2}}), (True, {"tensor": {"dx": DW}}),
    (True, {"tensor": {"dx": W}}), (True, {"tensor": {"dweight": W}}), (True, {"tensor": {"dweight": X}}),
    (True, {"tensor": {"weight": None}}), (True, {"tensor": {"dx": None}}), (True, {"tensor": {"dy": None}}),
    (True, {"ws": X}), (True, {"ws": W - 256}), (True, {"ws": DX + 512}), (True, {"pos": DX}),
    (True, {"ws": A - 1024}), (True, {"more": [{"x": Y, "dy": A + (7 << 20), "dx": A + (8 << 20)}]}),
])
def test_qk_overlaps_and_missing(lib, back, kw):
    assert _qk(lib, back, **kw) == INVALID


def test_qk_workspace_and_no_rows(lib):
    assert _qk(lib, True, ws=None) == WORKSPACE and _qk(lib, True, ws_bytes=256) == WORKSPACE
    assert _qk(lib, True, ws=A + (9 << 20) + 8) == ALIGN
    assert _qk(lib, False, len=0) == nsp.NSP_OK
    assert _qk(lib, False, len=0, tensor={"x": 0, "y": 0}) == nsp.NSP_OK
    arr = (nsp.QkTensor * 1)(nsp.QkTensor(heads=4))
    size = lib.nsp_qk_norm_rope_bwd_workspace_size
    assert size(C.addressof(arr), 1, 10, 128) > 0 and size(C.addressof(arr), 1, -1, 128) == 0
    assert size(None, 1, 10, 128) == 0 and size(C.addressof(arr), 1, 10, 513) == 0
    arr[0].heads = 0
    assert size(C.addressof(arr), 1, 10, 128) == 0


def test_qk_binding_refusals():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu, fr = torch.tensor([0, 4], dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        nsp.qk_norm_rope(x, x, cu, fr)
    with pytest.raises(TypeError):
        nsp.qk_norm_rope(x.half(), x.half(), cu, fr)
    with pytest.raises(ValueError):
        nsp.qk_norm_rope_bwd(x, x, x, x, cu, fr)


# ----------------------------------------------------------------------------- log-probabilities and losses

CU = [0, 4, 4, 5, 12, 13, 14]
TARGETS = np.array([-1, 2, 0, 5, 1, -1, -1, 4, 3, 2, -1, 0, -1, 5, 5])      # (the last row in no document)


def test_oracle_token_logp_against_autograd():
    rng = np.random.default_rng(2)
    x, g = rng.normal(size=(15, 6)) * 4, rng.normal(size=15)
    x[2, 3] = -np.inf
    leaf = torch.tensor(x, requires_grad=True)
    rows = np.flatnonzero(TARGETS >= 0)
    ref = torch.log_softmax(0.7 * leaf[rows], -1)[torch.arange(len(rows)), TARGETS[rows]]
    (dx,) = torch.autograd.grad(ref, leaf, torch.tensor(g[rows]))
    logp, lse = S.token_logp(x, TARGETS, 0.7)
    np.testing.assert_allclose(logp[rows], ref.detach(), rtol=1e-12)
    np.testing.assert_allclose(lse[rows], torch.logsumexp(0.7 * leaf.detach(), -1)[rows], rtol=1e-12)
    assert (logp[TARGETS < 0] == 0).all() and (lse[TARGETS < 0] == 0).all()
    np.testing.assert_allclose(S.token_logp_bwd(x, TARGETS, g, 0.7), dx, atol=1e-14)


@pytest.mark.parametrize("mean", ["tokens", "documents"])
@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("total", [0.0, 40.0])
def test_oracle_policy_loss_against_autograd(mean, per_token, total):
    rng = np.random.default_rng(3)
    logp, T = -rng.uniform(0.1, 3, 15), 15
    old, ref = logp + rng.normal(size=T) * 0.4, logp + rng.normal(size=T) * 0.5
    adv = rng.normal(size=T if per_token else 6)
    leaf = torch.tensor(logp, requires_grad=True)
    docs = [[t for t in range(CU[b], CU[b + 1]) if TARGETS[t] >= 0] for b in range(6)]
    n_tokens, n_docs = sum(map(len, docs)), sum(len(d) > 0 for d in docs)
    parts = []
    for b, d in enumerate(docs):
        for t in d:
            a = adv[t] if per_token else adv[b]
            r = torch.exp(leaf[t] - old[t])
            pg = -torch.min(r * a, torch.clamp(r, 0.8, 1.3) * a)
            kl = torch.exp(ref[t] - leaf[t]) - (ref[t] - leaf[t]) - 1
            w = 1 / (total or n_tokens) if mean == "tokens" else 1 / ((total or n_docs) * len(d))
            parts.append(w * torch.stack([pg + 0.3 * kl, pg, kl]))
    loss = torch.stack(parts).sum(0)
    (g,) = torch.autograd.grad(loss[0], leaf)
    stats, dlogp = S.policy_loss(logp, old, ref, adv, TARGETS, CU, 0.2, 0.3, 0.3, mean, total)
    np.testing.assert_allclose(stats[:3], loss.detach(), rtol=1e-12)
    np.testing.assert_allclose(dlogp, g, atol=1e-14)
    d = rng.normal(size=T) * 1e-6
    f = [S.policy_loss(logp + s * d, old, ref, adv, TARGETS, CU, 0.2, 0.3, 0.3, mean, total)[0][0] for s in (1, -1)]
    assert abs((f[0] - f[1]) / 2 - (dlogp * d).sum()) < 1e-12
    # without anything scored
    stats, dlogp = S.policy_loss(logp, old, ref, adv, np.full(T, -1), CU, mean=mean)
    assert (stats == 0).all() and (dlogp == 0).all()


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "square"])
@pytest.mark.parametrize("average", [False, True])
def test_oracle_preference_loss_against_autograd(kind, average):
    rng = np.random.default_rng(4)
    T = 15
    logp = -rng.uniform(0.1, 3, T)
    ref = logp + rng.normal(size=T)
    leaf = torch.tensor(logp, requires_grad=True)
    score = []
    for b in range(6):
        rows = [t for t in range(CU[b], CU[b + 1]) if TARGETS[t] >= 0]
        x = (leaf[rows] - torch.tensor(ref[rows])).sum()
        score.append(x / max(1, len(rows)) if average else x)
    r = 0.6 * torch.stack(score)
    h = r[0::2] - r[1::2] - 0.1
    if kind == "sigmoid":
        loss = -0.9 * torch.nn.functional.logsigmoid(h) - 0.1 * torch.nn.functional.logsigmoid(-h)
    elif kind == "hinge":
        loss = torch.relu(1 - h)
    else:
        loss = (h / 0.6 - 1 / 1.2) ** 2
    (g,) = torch.autograd.grad(loss.mean(), leaf)
    kw = dict(kind=kind, beta=0.6, smoothing=0.1, margin=0.1, average=average)
    stats, rewards, dlogp = S.preference_loss(logp, ref, TARGETS, CU, **kw)
    np.testing.assert_allclose(stats[0], loss.mean().item(), rtol=1e-12)
    np.testing.assert_allclose(rewards, r.detach(), rtol=1e-12, atol=1e-15)
    np.testing.assert_allclose(dlogp, g, atol=1e-14)
    assert stats[1] == (r[0::2] > r[1::2]).double().mean().item()


def test_oracle_grad_norm():
    rng = np.random.default_rng(5)
    g = [rng.normal(size=n) for n in (3, 0, 17)]
    assert abs(S.grad_norm(g, 0.5) - 0.5 * np.linalg.norm(np.concatenate(g))) < 1e-14
    assert S.grad_norm(g, -2.0, np.inf) == 2 * np.abs(np.concatenate(g)).max()


LG, TG, LP, LS, DL, GO = (A + (i << 20) for i in range(1, 7))


def _fwd(lib, **kw):
    """10 rows of 100 bf16 logits."""
    a = dict(x=LG, stride=0, y=TG, rows=10, vocab=100, scale=1.0, io=nsp.NSP_BF16, logp=LP, lse=LS, ws=A + (14 << 20),
             n=4096)
    a.update(kw)
    return lib.nsp_token_logp_fwd(a["x"], a["stride"], a["y"], a["rows"], a["vocab"], a["scale"], a["io"],
                                  a["logp"], a["lse"], a["ws"], a["n"], None)


def _bwd(lib, **kw):
    a = dict(x=LG, stride=0, y=TG, lse=LS, dlogp=DL, rows=10, vocab=100, scale=1.0, io=nsp.NSP_BF16, out=GO,
             out_stride=0)
    a.update(kw)
    return lib.nsp_token_logp_bwd(a["x"], a["stride"], a["y"], a["lse"], a["dlogp"], a["rows"], a["vocab"],
                                  a["scale"], a["io"], a["out"], a["out_stride"], None)


@pytest.mark.parametrize("kw,expect", [
    ({"x": None}, INVALID), ({"y": None}, INVALID), ({"rows": -1}, INVALID), ({"vocab": 0}, INVALID),
    ({"vocab": (1 << 20) + 1}, UNSUPPORTED), ({"rows": (1 << 30) + 1}, UNSUPPORTED), ({"scale": 0.0}, INVALID),
    ({"scale": float("nan")}, INVALID), ({"scale": float("inf")}, INVALID), ({"io": 2}, INVALID),
    ({"stride": 99}, INVALID), ({"stride": (1 << 31) + 1}, UNSUPPORTED), ({"x": LG + 1}, ALIGN), ({"y": TG + 2}, ALIGN),
    ({"rows": 0}, nsp.NSP_OK), ({"rows": 0, "x": None, "y": None}, nsp.NSP_OK),
])
def test_token_logp_refusals(lib, kw, expect):
    assert _fwd(lib, **kw) == expect and _bwd(lib, **kw) == expect


def test_token_logp_outputs(lib):
    assert _fwd(lib, logp=None) == INVALID and _fwd(lib, logp=LP + 2) == ALIGN
    assert _fwd(lib, ws=None) == WORKSPACE and _fwd(lib, n=300) == WORKSPACE and _fwd(lib, ws=A + 8) == ALIGN
    assert _fwd(lib, ws=LG + 1600) == INVALID and _fwd(lib, ws=LP - 320) == INVALID
    assert lib.nsp_token_logp_workspace_size(-1) == 0 and lib.nsp_token_logp_workspace_size(0) > 0
    for kw in (dict(logp=LG + 1996), dict(lse=LP + 36), dict(lse=TG), dict(logp=LG + 200, stride=108)):
        assert _fwd(lib, **kw) == INVALID, kw
    for kw in (dict(lse=None), dict(dlogp=None), dict(out=None), dict(out=LG + 2), dict(out=LG, out_stride=108),
               dict(out=LS), dict(out=DL + 36), dict(out=TG - 1996), dict(out_stride=99)):
        assert _bwd(lib, **kw) == INVALID, kw
    assert _bwd(lib, out=GO + 1) == ALIGN and _bwd(lib, out_stride=(1 << 31) + 2) == UNSUPPORTED


POLICY = dict(old_logp=A + (10 << 20), ref_logp=A + (11 << 20), advantages=A + (12 << 20), per_token=0, mean=0,
              clip_low=0.2, clip_high=0.2, kl_coef=0.1, total=0.0)


def _policy(lib, logits=False, policy=(), **kw):
    p = nsp.Policy(**{**POLICY, **dict(policy)})
    size = lib.nsp_policy_loss_workspace_size(10, 3, int(logits))
    a = dict(logp=LP, x=LG, y=TG, cu=A, ndoc=3, rows=10, p=C.addressof(p), stats=A + (13 << 20), out=GO, ws=A + (14 << 20),
             n=size, vocab=100, stride=0, out_stride=0)
    a.update(kw)
    if logits:
        return lib.nsp_policy_loss_logits(a["x"], a["stride"], a["y"], a["cu"], a["ndoc"], a["rows"], a["vocab"], 1.0,
                                          nsp.NSP_BF16, a["p"], a["stats"], a["logp"], a["out"], a["out_stride"],
                                          a["ws"], a["n"], None)
    return lib.nsp_policy_loss(a["logp"], a["y"], a["cu"], a["ndoc"], a["rows"], a["p"], a["stats"], a["out"],
                               a["ws"], a["n"], None)


@pytest.mark.parametrize("logits", [False, True])
@pytest.mark.parametrize("kw,expect", [
    ({"cu": None}, INVALID), ({"ndoc": 0}, INVALID), ({"rows": -1}, INVALID), ({"p": None}, INVALID),
    ({"stats": None}, INVALID), ({"y": None}, INVALID), ({"out": None}, INVALID), ({"ws": None}, WORKSPACE),
    ({"n": 300}, WORKSPACE), ({"ws": A + (14 << 20) + 4}, ALIGN), ({"stats": A + (13 << 20) + 2}, ALIGN),
    ({"rows": (1 << 30) + 1}, UNSUPPORTED), ({"policy": {"clip_low": -0.1}}, INVALID),
    ({"policy": {"clip_low": 1.5}}, INVALID), ({"policy": {"clip_high": float("inf")}}, INVALID),
    ({"policy": {"kl_coef": float("nan")}}, INVALID), ({"policy": {"total": -1.0}}, INVALID),
    ({"policy": {"mean": 2}}, INVALID), ({"policy": {"per_token": 2}}, INVALID),
    ({"policy": {"advantages": None}}, INVALID), ({"policy": {"old_logp": None}}, INVALID),
    ({"policy": {"ref_logp": None}}, INVALID), ({"policy": {"old_logp": A + 2}}, ALIGN),
    # overlaps
    ({"stats": TG + 36}, INVALID), ({"out": TG}, INVALID), ({"out": A - 4}, INVALID), ({"ws": TG - 64}, INVALID),
    ({"stats": GO}, INVALID), ({"out": POLICY["old_logp"]}, INVALID), ({"out": POLICY["ref_logp"] - 16}, INVALID),
    ({"stats": POLICY["advantages"] + 8}, INVALID), ({"policy": {"per_token": 1}, "stats": POLICY["advantages"] + 36}, INVALID),
    ({"ws": POLICY["advantages"]}, INVALID),
])
def test_policy_refusals(lib, logits, kw, expect):
    assert _policy(lib, logits, **kw) == expect


def test_policy_logits_refusals(lib):
    for kw in (dict(x=None), dict(logp=LG + 64), dict(out=LG + 2), dict(out=LG, out_stride=108), dict(stats=LG + 32),
               dict(logp=GO + 8), dict(vocab=0), dict(ws=LG + 64)):
        assert _policy(lib, True, **kw) == INVALID, kw
    assert _policy(lib, True, logp=LP + 2) == ALIGN
    assert _policy(lib, False, logp=None) == INVALID
    size = lib.nsp_policy_loss_workspace_size
    assert size(-1, 3, 0) == 0 and size(10, 0, 0) == 0 and size(10, 3, 2) == 0 and size(10, 3, 1) > 256


def _preference(lib, **kw):
    a = dict(logp=LP, ref=LS, y=TG, cu=A, ndoc=4, rows=10, kind=0, beta=0.1, smoothing=0.0, margin=0.0, average=0,
             stats=A + (13 << 20), rewards=A + (12 << 20), out=DL, ws=A + (14 << 20), n=1024)
    a.update(kw)
    return lib.nsp_preference_loss(*[a[k] for k in ("logp", "ref", "y", "cu", "ndoc", "rows", "kind", "beta",
                                                    "smoothing", "margin", "average", "stats", "rewards", "out",
                                                    "ws", "n")], None)


@pytest.mark.parametrize("kw,expect", [
    ({"ndoc": 3}, INVALID), ({"ndoc": 0}, INVALID), ({"rows": -1}, INVALID), ({"rows": 1 << 31}, UNSUPPORTED),
    ({"kind": 3}, INVALID), ({"kind": -1}, INVALID), ({"beta": 0.0}, INVALID), ({"beta": float("inf")}, INVALID),
    ({"smoothing": -0.1}, INVALID), ({"smoothing": 1.1}, INVALID), ({"margin": float("nan")}, INVALID),
    ({"average": 2}, INVALID), ({"logp": None}, INVALID), ({"y": None}, INVALID), ({"cu": None}, INVALID),
    ({"stats": None}, INVALID), ({"rewards": None}, INVALID), ({"out": None}, INVALID), ({"ws": None}, WORKSPACE),
    ({"n": 256}, WORKSPACE), ({"ws": A + (14 << 20) + 8}, ALIGN), ({"logp": LP + 1}, ALIGN),
    ({"out": LP}, INVALID), ({"out": LS + 36}, INVALID), ({"rewards": A + 16}, INVALID), ({"stats": TG}, INVALID),
    ({"ws": DL}, INVALID), ({"rewards": A + (13 << 20) + 4}, INVALID),
])
def test_preference_refusals(lib, kw, expect):
    assert _preference(lib, **kw) == expect
    assert lib.nsp_preference_loss_workspace_size(3) == 0 and lib.nsp_preference_loss_workspace_size(0) == 0


def _grads(lib, clip, ptrs=(LG, TG), counts=(100, 50), types=(0, 1), out=None, out_types=None, **kw):
    n = len(ptrs)
    a = dict(n=n, kind=0, unscale=1.0, max_norm=1.0, eps=1e-6, norm=A + (13 << 20), ws=A + (14 << 20), size=1 << 16)
    a.update(kw)
    vp, i64, i32 = C.c_void_p * n, C.c_int64 * n, C.c_int32 * n
    out = ptrs if out is None else out
    out_types = types if out_types is None else out_types
    if clip:
        return lib.nsp_grad_clip(vp(*ptrs), vp(*out), i64(*counts), i32(*types), i32(*out_types), a["n"], a["kind"],
                                 a["unscale"], a["max_norm"], a["eps"], a["norm"], a["ws"], a["size"], None)
    return lib.nsp_grad_norm(vp(*ptrs), i64(*counts), i32(*types), a["n"], a["kind"], a["unscale"], a["norm"], a["ws"],
                             a["size"], None)


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("kw,expect", [
    ({"n": 0}, INVALID), ({"n": 1 << 20}, UNSUPPORTED), ({"kind": 2}, INVALID), ({"unscale": float("inf")}, INVALID),
    ({"norm": None}, INVALID), ({"norm": A + 2}, ALIGN), ({"ws": None}, WORKSPACE), ({"size": 8}, WORKSPACE),
    ({"ws": A + 8}, ALIGN), ({"types": (0, 2)}, INVALID), ({"counts": (100, -1)}, INVALID),
    ({"counts": (100, (1 << 40) + 1)}, UNSUPPORTED), ({"ptrs": (LG, 0)}, INVALID), ({"ptrs": (LG + 2, TG)}, ALIGN),
    ({"norm": LG + 396}, INVALID), ({"ws": TG + 96}, INVALID), ({"norm": A + (14 << 20) + 8}, INVALID),
])
def test_grad_refusals(lib, clip, kw, expect):
    assert _grads(lib, clip, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    ({"max_norm": -1.0}, INVALID), ({"max_norm": float("nan")}, INVALID), ({"max_norm": float("inf")}, INVALID),
    ({"eps": 0.0}, INVALID), ({"ptrs": (LG, LG), "counts": (100, 100), "types": (0, 0)}, INVALID),      # twice
    ({"ptrs": (LG, LG + 396), "types": (0, 0)}, INVALID), ({"out": (LG + 4, GO)}, INVALID),
    ({"out": (GO, GO + 399)}, ALIGN), ({"out": (GO, GO + 398)}, INVALID), ({"out": (TG, GO)}, INVALID),
    ({"out": (GO, 0)}, INVALID), ({"out": (LG, TG), "out_types": (1, 1)}, INVALID), ({"out_types": (0, 3)}, INVALID),
    ({"out": (GO, LG + 100)}, INVALID),
])
def test_clip_refusals(lib, kw, expect):
    assert _grads(lib, True, **kw) == expect


def test_grad_workspace(lib):
    size = lib.nsp_grad_norm_workspace_size
    assert size((C.c_int64 * 2)(5, 0), 2) > 0 and size((C.c_int64 * 1)(-5), 1) == 0 and size(None, 1) == 0
    assert size((C.c_int64 * 1)(5), 0) == 0


def test_step_binding_refusals():
    x, y = torch.zeros((4, 6)), torch.zeros(4, dtype=torch.int32)
    cu = torch.tensor([0, 2, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        nsp.token_logp(x, y)
    with pytest.raises(TypeError):
        nsp.token_logp(x.double(), y)
    with pytest.raises(ValueError):
        nsp.policy_loss(x[:, 0], y, x[:, 0], x[:2, 0], cu)
    with pytest.raises(ValueError):
        nsp.policy_loss_logits(x, y, x[:, 0], x[:2, 0], cu)
    with pytest.raises(ValueError):
        nsp.preference_loss(x[:, 0], y, cu)
    with pytest.raises(ValueError):
        nsp.grad_norm([x])
    with pytest.raises(ValueError):
        nsp.clip_grads([], 1.0)
    with pytest.raises(ValueError):
        nsp.grad_norm([x], norm_type=1)
