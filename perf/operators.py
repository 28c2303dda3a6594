"""Cases of the operators between the projections of a differential attention
layer on a packed token stream: rotary positions, the learned difference
weight, differential attention forward and backward, and the norm of each
head's output.

``run`` computes them in their plain form (elementary torch operations in
float32), or, with ``own`` set, through this package's entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_BF16, _F32 = "bf16", "f32"


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of each of 7 running sequences, far positions given by the
        # caller: the smallest rotation, latency only
        {"name": "rope tokens", "op": "rope", "tokens": 7, "hq": 32, "hkv": 4, "d": 128, "rot": 128,
         "layout": "half", "base": 1e6, "inverse": False, "groups": 1, "fused": False,
         "explicit": True, "docs": "mixed", "dtype": _BF16},
        # a packed training batch, q and k read from the fused projection
        {"name": "rope stream", "op": "rope", "tokens": 32768, "hq": 32, "hkv": 4, "d": 128,
         "rot": 128, "layout": "half", "base": 5e5, "inverse": False, "groups": 1, "fused": True,
         "explicit": False, "docs": "mixed", "dtype": _BF16},
        # the rotation's backward: gradients of q come head-grouped from an
        # all-to-all, half of each head was rotated, pairs interleaved
        {"name": "rope back f32", "op": "rope", "tokens": 8191, "hq": 16, "hkv": 4, "d": 64,
         "rot": 32, "layout": "interleaved", "base": 1e4, "inverse": True, "groups": 4,
         "fused": False, "explicit": False, "docs": "mixed", "dtype": _F32},
        # the difference weight of a layer's heads, and its gradient
        {"name": "lambda", "op": "lambda", "heads": 16, "n": 16, "dl": 64, "back": False,
         "dtype": _BF16},
        {"name": "lambda back shared", "op": "lambda", "heads": 40, "n": 1, "dl": 128, "back": True,
         "dtype": _F32},
        # a few short documents: the smallest call
        {"name": "diff few tokens", "op": "diff", "tokens": 197, "hq": 4, "hkv": 2, "d": 128,
         "docs": "few", "causal": True, "back": False, "token_lambda": False, "dtype": _BF16},
        # many documents of 32 to 256 tokens (a short-document fine-tuning batch)
        {"name": "diff short documents", "op": "diff", "tokens": 65536, "hq": 16, "hkv": 2, "d": 128,
         "docs": "short", "causal": True, "back": False, "token_lambda": False, "dtype": _BF16},
        # one long document (long-context training), lambda of each token
        {"name": "diff long document", "op": "diff", "tokens": 20001, "hq": 8, "hkv": 4, "d": 128,
         "docs": "one", "causal": True, "back": False, "token_lambda": True, "dtype": _BF16},
        # a training step over the long-tailed mix of document lengths
        {"name": "diff step mixed", "op": "diff", "tokens": 16384, "hq": 16, "hkv": 4, "d": 128,
         "docs": "mixed", "causal": True, "back": True, "token_lambda": False, "dtype": _BF16},
        # a bidirectional float32 training step (a numerics run), odd sizes
        {"name": "diff step f32", "op": "diff", "tokens": 3001, "hq": 6, "hkv": 2, "d": 64,
         "docs": "mixed", "causal": False, "back": True, "token_lambda": True, "dtype": _F32},
        # the gated norm of each head's output, and its backward
        {"name": "head norm", "op": "norm", "tokens": 32768, "heads": 16, "d": 128, "gate": True,
         "weight": True, "back": False, "dtype": _BF16},
        {"name": "head norm back", "op": "norm", "tokens": 16383, "heads": 16, "d": 128, "gate": True,
         "weight": True, "back": True, "dtype": _BF16},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "diff", "diff", "diff", "diff", "norm", "norm", "lambda"])
    dtype = rng.choice([_BF16, _BF16, _F32])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4])
    hq = hkv * rng.choice([1, 2, 3, 4])
    if op == "rope":
        return {"op": op, "tokens": _log_int(rng, 1, 40000), "hq": hq * 2, "hkv": hkv, "d": d,
                "rot": rng.choice([d, d, d // 2]), "layout": rng.choice(["half", "interleaved"]),
                "base": rng.choice([1e4, 5e5, 1e6]), "inverse": rng.random() < 0.5,
                "groups": rng.choice([1, 1, 2]), "fused": rng.random() < 0.5,
                "explicit": rng.random() < 0.3, "docs": rng.choice(["mixed", "short", "one"]),
                "dtype": dtype}
    if op == "lambda":
        heads = rng.randint(1, 64)
        return {"op": op, "heads": heads, "n": rng.choice([1, heads]), "dl": rng.choice([32, 64, 128]),
                "back": rng.random() < 0.5, "dtype": dtype}
    if op == "norm":
        return {"op": op, "tokens": _log_int(rng, 1, 30000), "heads": rng.randint(1, 16),
                "d": rng.choice([64, 128, 256]), "gate": rng.random() < 0.6,
                "weight": rng.random() < 0.8, "back": rng.random() < 0.5, "dtype": dtype}
    back = rng.random() < 0.5
    docs = rng.choice(["mixed", "short", "one", "few"])
    most = {"mixed": 8000, "short": 30000, "one": 4000, "few": 600}[docs]
    if dtype == _F32:
        most = min(most, 2500)
    return {"op": op, "tokens": _log_int(rng, 20, most), "hq": hq, "hkv": hkv, "d": d, "docs": docs,
            "causal": rng.random() < 0.75, "back": back, "token_lambda": rng.random() < 0.4,
            "dtype": dtype}


def _lengths(case):
    """Document lengths of a case, drawn from its own size alone."""
    total, kind = case["tokens"], case["docs"]
    rng = random.Random(total * 7 + len(kind))
    if kind == "one":
        return [total]
    lens, left = [], total
    while left > 0:
        if kind == "few":
            n = rng.choice([1, 2, 45, 130])
        elif kind == "short":
            n = rng.randint(32, 256)
        else:
            n = min(4096, max(1, round(math.exp(rng.gauss(math.log(1024), 1.0)))))
        n = min(n, left)
        lens.append(n)
        left -= n
    return lens


# ----------------------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == _BF16 else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _dtype(case)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = {"case": case}
    op = case["op"]
    if op in ("rope", "diff"):
        lens = _lengths(case)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["longest"] = max(lens)
    if op == "rope":
        t, hq, hkv, d, rot = (case[n] for n in ("tokens", "hq", "hkv", "d", "rot"))
        if case["fused"] and not case["inverse"]:
            qkv = randn(t, hq + 2 * hkv, d)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            p = case["groups"]
            s["q"] = randn(p, t, hq // p, d) if case["inverse"] and p > 1 else randn(t, hq, d)
            s["k"] = randn(t, hkv, d)
        i = torch.arange(0, rot, 2, dtype=torch.float64)
        s["freqs"] = (case["base"] ** (-i / rot)).cuda()
        s["positions"] = None
        if case["explicit"]:
            s["positions"] = torch.randint(0, 400000, (t,), generator=g, device="cuda",
                                           dtype=torch.int32)
    elif op == "lambda":
        n, dl = case["n"], case["dl"]
        # learned vectors start at a standard deviation of 0.1
        s["vectors"] = [(randn(n, dl).float() * 0.1).to(dt) for _ in range(4)]
        s["dlam"] = randn(case["heads"])
    elif op == "norm":
        t, h, d = case["tokens"], case["heads"], case["d"]
        s["x"] = randn(t, h, d)
        s["gate"] = randn(t, h, d) if case["gate"] else None
        s["weight"] = (1 + 0.1 * randn(d).float()).to(dt) if case["weight"] else None
        s["dy"] = randn(t, h, d) if case["back"] else None
    else:
        t, hq, hkv, d = (case[n] for n in ("tokens", "hq", "hkv", "d"))
        s["q"], s["k"], s["v"] = randn(t, hq, d), randn(t, hkv, d), randn(t, hkv, d)
        n = t if case["token_lambda"] else 1
        s["lam"] = torch.rand((hq, n), generator=g, device="cuda").mul_(0.6).add_(0.2).to(dt)
        s["dout"] = randn(t, hq, d) if case["back"] else None
    return s


_NORM_SCALE, _EPS, _LAMBDA_INIT, _ATTN_FACTOR = 0.2, 1e-5, 0.8, 1.1


# ----------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"rope": _plain_rope, "lambda": _plain_lambda, "norm": _plain_norm,
            "diff": _plain_diff}[case["op"]](state, case)


def _own(s, case):
    from variable_length_sequence_gb300 import nsp
    op = case["op"]
    if op == "rope":
        return nsp.rope(s["q"], s["k"], s["cu"], s["freqs"], layout=case["layout"],
                        mscale=_ATTN_FACTOR, inverse=case["inverse"], positions=s["positions"],
                        q_groups=case["groups"])
    if op == "lambda":
        if case["back"]:
            return nsp.diff_lambda_bwd(s["dlam"], *s["vectors"])
        return nsp.diff_lambda(*s["vectors"], heads=case["heads"], lambda_init=_LAMBDA_INIT)
    if op == "norm":
        if case["back"]:
            return nsp.head_norm_bwd(s["x"], s["dy"], s["weight"], s["gate"], eps=_EPS,
                                     scale=_NORM_SCALE)
        return nsp.head_norm(s["x"], s["weight"], s["gate"], eps=_EPS, scale=_NORM_SCALE)
    if not case["back"]:
        return nsp.diff_attn_fwd(s["q"], s["k"], s["v"], s["lam"], s["cu"], causal=case["causal"])
    out, out2, lse = nsp.diff_attn_fwd(s["q"], s["k"], s["v"], s["lam"], s["cu"],
                                       causal=case["causal"], save=True)
    return (out,) + nsp.diff_attn_bwd(s["q"], s["k"], s["v"], s["lam"], out, out2, s["dout"], lse,
                                      s["cu"], causal=case["causal"])


# ----------------------------------------------------------------------------- plain forms

def _document_of(cu, t):
    return torch.searchsorted(cu[1:].contiguous(), torch.arange(t, device=cu.device), right=True)


def _plain_rope(s, case):
    t, rot, dt = case["tokens"], case["rot"], _dtype(case)
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(t, device="cuda") - s["cu"].long()[_document_of(s["cu"], t)]
    angle = pos.double()[:, None] * s["freqs"][None]
    cos = (angle.cos() * _ATTN_FACTOR).float()[:, None]
    sin = (angle.sin() * _ATTN_FACTOR).float()[:, None]
    if case["inverse"]:
        sin = -sin

    def rotate(x):
        y = x.float()
        part = y[..., :rot]
        if case["layout"] == "half":
            a, b = part[..., :rot // 2], part[..., rot // 2:]
        else:
            a, b = part[..., 0::2], part[..., 1::2]
        u, w = a * cos - b * sin, a * sin + b * cos
        if case["layout"] == "half":
            turned = torch.cat([u, w], -1)
        else:
            turned = torch.stack([u, w], -1).flatten(-2)
        return torch.cat([turned, y[..., rot:]], -1).to(dt)

    q, k, p = s["q"], s["k"], case["groups"]
    if case["inverse"] and p > 1:
        q = q.transpose(0, 1).reshape(t, case["hq"], case["d"])
    q = rotate(q)
    if not case["inverse"] and p > 1:
        q = q.view(t, p, case["hq"] // p, case["d"]).transpose(0, 1).contiguous()
    return q, rotate(k)


def _plain_lambda(s, case):
    dt = _dtype(case)
    q1, k1, q2, k2 = (x.float() for x in s["vectors"])
    e1 = (q1 * k1).sum(-1, keepdim=True).exp()
    e2 = (q2 * k2).sum(-1, keepdim=True).exp()
    if not case["back"]:
        return (e1 - e2 + _LAMBDA_INIT)[:, 0].expand(case["heads"]).to(dt)
    g = s["dlam"].float()[:, None]
    if case["n"] == 1:
        g = g.sum(0, keepdim=True)
    e1, e2 = g * e1, g * e2
    return tuple(x.to(dt) for x in (e1 * k1, e1 * q1, -e2 * k2, -e2 * q2))


def _plain_norm(s, case):
    dt = _dtype(case)
    x = s["x"].float()
    r = (x.square().mean(-1, keepdim=True) + _EPS).rsqrt()
    xn = x * r
    w = _NORM_SCALE if s["weight"] is None else _NORM_SCALE * s["weight"].float()
    if s["gate"] is None:
        c = w
    else:
        sig = 1 / (1 + (-s["gate"].float()).exp())
        c = w * sig
    if not case["back"]:
        return (xn * c).to(dt)
    dy = s["dy"].float()
    u = dy * c
    dx = r * (u - xn * (u * xn).mean(-1, keepdim=True))
    dw = dgate = None
    if s["weight"] is not None:
        dyg = dy if s["gate"] is None else dy * sig
        dw = (_NORM_SCALE * dyg * xn).sum((0, 1)).to(dt)
    if s["gate"] is not None:
        dgate = (dy * xn * w * sig * (1 - sig)).to(dt)
    return dx.to(dt), dw, dgate


def _plain_diff(s, case):
    """Documents padded to the longest one: [documents, kv heads, maps, heads x
    rows, keys] scores, softmax and products over whole rows."""
    t, hq, hkv, d, dt = case["tokens"], case["hq"], case["hkv"], case["d"], _dtype(case)
    g, half, scale = hq // hkv, d // 2, (d // 2) ** -0.5
    cu, longest = s["cu"].long(), s["longest"]
    docs = cu.numel() - 1
    ar = torch.arange(longest, device="cuda")
    index = (cu[:-1, None] + ar).clamp_(max=t - 1)
    inside = ar[None] < (cu[1:] - cu[:-1])[:, None]
    doc = _document_of(s["cu"], t)
    back_index = doc * longest + (torch.arange(t, device="cuda") - cu[doc])

    def padded(x, heads):                   # [docs, longest, heads, d], rows past a document zero
        return x[index].float() * inside[:, :, None, None]

    q = padded(s["q"], hq).view(docs, longest, hkv, g, 2, half).permute(0, 2, 4, 3, 1, 5)
    q = q.reshape(docs, hkv, 2, g * longest, half)
    k = padded(s["k"], hkv).view(docs, longest, hkv, 2, half).permute(0, 2, 3, 1, 4)
    v = padded(s["v"], hkv).permute(0, 2, 1, 3)[:, :, None]
    seen = inside[:, None, :]
    if case["causal"]:
        seen = seen & (ar[None] <= ar[:, None])[None]
    hidden = ~seen[:, None, None, None]
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    p.view(docs, hkv, 2, g, longest, longest).masked_fill_(hidden, -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    o = torch.matmul(p, v)                  # [docs, hkv, 2, g longest, d]
    lam = s["lam"].float()
    if case["token_lambda"]:
        lam = lam[:, index].view(hkv, g, docs, longest).permute(2, 0, 1, 3)
    else:
        lam = lam.view(1, hkv, g, 1).expand(docs, hkv, g, longest)
    lam = lam.reshape(docs, hkv, g * longest, 1)

    def packed(x, heads):                   # [docs, hkv, heads / hkv x longest, d] -> stream rows
        x = x.view(docs, hkv, heads // hkv, longest, -1).permute(0, 3, 1, 2, 4)
        return x.reshape(docs * longest, heads, -1)[back_index].to(dt)

    out = packed(o[:, :, 0] - lam * o[:, :, 1], hq)
    if not case["back"]:
        return out
    do = padded(s["dout"], hq).view(docs, longest, hkv, g, d).permute(0, 2, 3, 1, 4)
    do = do.reshape(docs, hkv, g * longest, d)
    delta = (do[:, :, None] * o).sum(-1, keepdim=True)
    dv = torch.matmul((p[:, :, 0] - lam * p[:, :, 1]).transpose(-1, -2), do)
    dp = torch.matmul(do, v[:, :, 0].transpose(-1, -2))
    p[:, :, 0].mul_(dp - delta[:, :, 0])
    p[:, :, 1].mul_(dp.sub_(delta[:, :, 1]).mul_(-lam))
    dq = torch.matmul(p, k).mul_(scale)
    dk = torch.matmul(p.transpose(-1, -2), q).mul_(scale)
    dq = dq.view(docs, hkv, 2, g, longest, half).permute(0, 1, 3, 4, 2, 5)
    dq = packed(dq.reshape(docs, hkv, g * longest, d), hq)
    dk = packed(dk.permute(0, 1, 3, 2, 4).reshape(docs, hkv, longest, d), hkv)
    dlam = -delta[:, :, 1].view(docs, hkv, g, longest).permute(1, 2, 0, 3).reshape(hq, docs * longest)
    dlam = dlam[:, back_index]
    if not case["token_lambda"]:
        dlam = dlam.sum(-1, keepdim=True)
    return out, dq, dk, packed(dv, hkv), dlam.to(dt)


# ----------------------------------------------------------------------------- what a pass needs

def work(case):
    es = 2 if case["dtype"] == _BF16 else 4
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": 2 * n * case["d"] * es, "flops": 3 * n * case["rot"]}
    if op == "lambda":
        n = 4 * case["n"] * case["dl"]
        return {"bytes": (n * (2 if case["back"] else 1) + case["heads"]) * es, "flops": 2 * n}
    if op == "norm":
        n = case["tokens"] * case["heads"] * case["d"]
        arrays = 2 + case["gate"] + (1 + case["gate"] if case["back"] else 0)
        return {"bytes": arrays * n * es, "flops": n * (14 if case["back"] else 6)}
    lens, d = _lengths(case), case["d"]
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
    t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
    lam = hq * (t if case["token_lambda"] else 1)
    n = 2 * t * hq * d + 2 * t * hkv * d + lam
    if case["back"]:
        n += 2 * t * hq * d + 2 * t * hkv * d + lam
    return {"bytes": n * es, "flops": pairs * hq * d * (14 if case["back"] else 6)}


# ----------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "lambda": _exact_lambda, "norm": _exact_norm,
            "diff": _exact_diff}[case["op"]](s, case)


def _exact_rope(s, case):
    t, rot = case["tokens"], case["rot"]
    if s["positions"] is not None:
        pos = s["positions"].double()
    else:
        pos = torch.cat([torch.arange(n, device="cuda", dtype=torch.float64)
                         for n in _lengths(case)])
    turn = torch.polar(torch.full((t, rot // 2), _ATTN_FACTOR, dtype=torch.float64, device="cuda"),
                       torch.outer(pos, s["freqs"]))[:, None, :]
    if case["inverse"]:
        turn = turn.conj()

    def rotate(x):
        y = x.double().clone()
        if case["layout"] == "half":
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        else:
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        return y

    q, p = s["q"], case["groups"]
    if p > 1 and case["inverse"]:
        q = torch.cat(list(q), dim=1)
    q = rotate(q)
    if p > 1 and not case["inverse"]:
        q = torch.stack(q.chunk(p, dim=1))
    return q, rotate(s["k"])


def _exact_lambda(s, case):
    v = [x.double().requires_grad_() for x in s["vectors"]]
    lam = torch.exp(torch.einsum("nd,nd->n", v[0], v[1])) - torch.exp(
        torch.einsum("nd,nd->n", v[2], v[3])) + _LAMBDA_INIT
    lam = lam.expand(case["heads"])
    if not case["back"]:
        return lam.detach()
    return torch.autograd.grad(lam, v, s["dlam"].double())


def _exact_norm(s, case):
    x = s["x"].double().requires_grad_()
    w = None if s["weight"] is None else s["weight"].double().requires_grad_()
    gate = None if s["gate"] is None else s["gate"].double().requires_grad_()
    y = _NORM_SCALE * x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + _EPS)
    if w is not None:
        y = y * w
    if gate is not None:
        y = y * torch.special.expit(gate)
    if not case["back"]:
        return y.detach()
    leaves = [v for v in (x, w, gate) if v is not None]
    grads = iter(torch.autograd.grad(y, leaves, s["dy"].double()))
    return tuple(None if v is None else next(grads) for v in (x, w, gate))


def _exact_diff(s, case):
    """Document by document, head by head, rows in slices."""
    t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    half, back = d // 2, case["back"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    lam = s["lam"].double().expand(hq, t)
    out = torch.zeros_like(q)
    if back:
        do = s["dout"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dlam = torch.zeros(hq, t, dtype=torch.float64, device="cuda")
    groups = torch.arange(hq, device="cuda") // (hq // hkv)
    first = 0
    for n in _lengths(case):
        # heads first: [hq, n, d]
        kd, vd = (x[first:first + n].transpose(0, 1)[groups] for x in (k, v))
        for r0 in range(0, n, 2048):
            r1 = min(n, r0 + 2048)
            rows = slice(first + r0, first + r1)
            qd = q[rows].transpose(0, 1)
            allowed = None
            if case["causal"]:
                allowed = (torch.arange(r0, r1, device="cuda")[:, None]
                           >= torch.arange(n, device="cuda")[None])
            maps = []
            for cols in (slice(0, half), slice(half, d)):
                z = torch.einsum("hrc,hjc->hrj", qd[..., cols], kd[..., cols]) / math.sqrt(half)
                if allowed is not None:
                    z = torch.where(allowed, z, -math.inf)
                maps.append(torch.softmax(z, dim=-1))
            a, b = maps
            w = lam[:, rows, None]
            c = a - w * b
            out[rows] = (c @ vd).transpose(0, 1)
            if not back:
                continue
            dod = do[rows].transpose(0, 1)
            dc = dod @ vd.transpose(1, 2)
            dlam[:, rows] = -(dc * b).sum(-1)
            gv = c.transpose(1, 2) @ dod
            dv[first:first + n].index_add_(1, groups, gv.transpose(0, 1))
            for m, cols, up in ((a, slice(0, half), dc), (b, slice(half, d), -w * dc)):
                z = m * (up - (up * m).sum(-1, keepdim=True)) / math.sqrt(half)
                dq[rows, :, cols] = (z @ kd[..., cols]).transpose(0, 1)
                gk = (z.transpose(1, 2) @ qd[..., cols]).transpose(0, 1)
                full = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
                full[..., cols] = gk
                dk[first:first + n].index_add_(1, groups, full)
        first += n
    if not back:
        return out
    if not case["token_lambda"]:
        dlam = dlam.sum(-1, keepdim=True)
    return out, dq, dk, dv, dlam
