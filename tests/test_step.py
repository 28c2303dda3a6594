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
