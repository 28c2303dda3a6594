"""Cases of the operators of a packed post-training step next to attention: the
norm of every query and key head with the position rotation in the same pass,
the log-probability of given tokens under their logits, the clipped policy loss
with its KL term, the preference loss over pairs of documents, and the global
norm of many gradients with their clipping.

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
        # one token of each of 7 running sequences, positions given by the
        # caller: the smallest norm and rotation, latency only
        {"name": "qk tokens", "op": "qk", "tokens": 7, "hq": 32, "hkv": 4, "d": 128, "rot": 128,
         "layout": "half", "base": 1e6, "back": False, "groups": 1, "fused": True, "explicit": True,
         "docs": "mixed", "dtype": _BF16},
        # a packed training batch, q and k read from the fused projection
        {"name": "qk stream", "op": "qk", "tokens": 32768, "hq": 32, "hkv": 4, "d": 128, "rot": 128,
         "layout": "half", "base": 5e5, "back": False, "groups": 1, "fused": True, "explicit": False,
         "docs": "mixed", "dtype": _BF16},
        # the backward of that batch: gradients of q, k and both weights
        {"name": "qk stream back", "op": "qk", "tokens": 32768, "hq": 32, "hkv": 4, "d": 128,
         "rot": 128, "layout": "half", "base": 5e5, "back": True, "groups": 1, "fused": True,
         "explicit": False, "docs": "mixed", "dtype": _BF16},
        # the tokens that 5 running sequences sampled: the smallest scoring call
        {"name": "logp tokens", "op": "logp", "tokens": 5, "vocab": 131072, "docs": "token",
         "dtype": _BF16},
        # the reference pass of a packed batch: scores alone
        {"name": "logp stream", "op": "logp", "tokens": 8192, "vocab": 65536, "docs": "mixed",
         "dtype": _BF16},
        # a float32 numerics run over a few short answers, odd vocabulary
        {"name": "policy f32", "op": "policy", "tokens": 301, "vocab": 32003, "docs": "few",
         "advantages": "tokens", "mean": "tokens", "kl": True, "dtype": _F32},
        # a policy step over the long-tailed mix of answers, from logits to their gradient
        {"name": "policy step", "op": "policy", "tokens": 8192, "vocab": 131072, "docs": "mixed",
         "advantages": "documents", "mean": "documents", "kl": True, "dtype": _BF16},
        # the loss over pairs alone, log-probabilities in hand: the smallest call
        {"name": "preference pairs", "op": "preference", "tokens": 4099, "vocab": 0, "docs": "pairs",
         "kind": "sigmoid", "average": False, "dtype": _F32},
        # a preference step from logits to their gradient, odd vocabulary
        {"name": "preference step", "op": "preference", "tokens": 6000, "vocab": 49999,
         "docs": "pairs", "kind": "sigmoid", "average": False, "dtype": _BF16},
        # the gradients of a small layer, clipped
        {"name": "clip layer", "op": "clip", "tensors": 11, "elements": 300007, "flat": False,
         "types": _F32, "write": True},
        # a model's gradients, matrices and vectors in both types, clipped
        {"name": "clip model", "op": "clip", "tensors": 60, "elements": 500000000, "flat": False,
         "types": "mixed", "write": True},
        # the norm alone, of many views of one flat float32 buffer at any offset
        {"name": "norm flat", "op": "clip", "tensors": 400, "elements": 300000001, "flat": True,
         "types": _F32, "write": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "qk", "qk", "logp", "policy", "policy", "preference", "preference",
                     "clip", "clip"])
    dtype = rng.choice([_BF16, _BF16, _F32])
    if op == "qk":
        hkv = rng.choice([1, 2, 4, 5])
        hq = hkv * 2 * rng.choice([1, 2, 3, 4])
        d = rng.choice([64, 128, 128, 256, 96])
        back = rng.random() < 0.5
        return {"op": op, "tokens": _log_int(rng, 1, 20000 if dtype == _F32 or d > 128 else 32000),
                "hq": hq, "hkv": hkv, "d": d, "rot": rng.choice([d, d, d // 2]),
                "layout": rng.choice(["half", "interleaved"]), "base": rng.choice([1e4, 5e5, 1e6]),
                "back": back, "groups": rng.choice([1, 1, 2]), "fused": rng.random() < 0.6,
                "explicit": rng.random() < 0.3, "docs": rng.choice(["mixed", "few", "one"]),
                "dtype": dtype}
    if op == "clip":
        return {"op": op, "tensors": rng.randint(1, 60), "elements": _log_int(rng, 1000, 400000000),
                "flat": rng.random() < 0.4, "types": rng.choice([_BF16, _F32, "mixed"]),
                "write": rng.random() < 0.6}
    vocab = _log_int(rng, 257, 131072)
    if rng.random() < 0.5:
        vocab = (vocab + 7) // 8 * 8
    most = min(30000, 400000000 // vocab)
    case = {"op": op, "tokens": _log_int(rng, 2, most), "vocab": vocab, "dtype": dtype}
    if op == "logp":
        return {**case, "docs": rng.choice(["mixed", "token", "one"])}
    if op == "policy":
        return {**case, "docs": rng.choice(["mixed", "few", "one"]),
                "advantages": rng.choice(["documents", "tokens"]),
                "mean": rng.choice(["documents", "tokens"]), "kl": rng.random() < 0.7}
    if rng.random() < 0.4:
        case["vocab"], case["dtype"], case["tokens"] = 0, _F32, _log_int(rng, 4, 300000)
    return {**case, "docs": "pairs", "kind": rng.choice(["sigmoid", "hinge", "square"]),
            "average": rng.random() < 0.4}


def _lengths(case):
    """Document lengths of a case, drawn from its own size alone (pairs: an even
    number of documents)."""
    total, kind = case["tokens"], case["docs"]
    rng = random.Random(total * 7 + len(kind))
    if kind == "one":
        return [total]
    if kind == "token":
        return [2] * (total // 2) + [1] * (total % 2)
    lens, left = [], total
    while left > 0:
        if kind == "few":
            n = rng.choice([1, 2, 45, 130])
        else:
            n = min(4096, max(1, round(math.exp(rng.gauss(math.log(400), 1.2)))))
        n = min(n, left)
        lens.append(n)
        left -= n
    if kind == "pairs" and len(lens) % 2:
        lens.append(0)
    return lens


def _answers(case):
    """For each document the first of its rows with a token to score, and one past
    the last: the prompt before them has none, nor has a document's last row (a
    running sequence's one row has)."""
    if case["docs"] == "token":
        return [(0, n) for n in _lengths(case)]
    return [(int(0.3 * n), max(int(0.3 * n), n - 1)) for n in _lengths(case)]


def _sizes(case):
    """Elements of a case's tensors: three in four are matrices, the rest vectors,
    odd ones among them."""
    n, total = case["tensors"], case["elements"]
    rng = random.Random(total + 31 * n)
    share = [math.exp(rng.uniform(0, 3)) if rng.random() < 0.75 else 1e-3 for _ in range(n)]
    sizes = [max(1, int(total * s / sum(share))) for s in share]
    sizes[0] += max(0, total - sum(sizes))
    return sizes


# ----------------------------------------------------------------------------- inputs

_EPS, _ATTN_FACTOR = 1e-6, 1.1
_CLIP_LOW, _CLIP_HIGH, _KL = 0.2, 0.28, 0.05
_BETA, _SMOOTHING = 0.1, 0.05
_TEMPERATURE = 1.25                       # the sampler's: logits are divided by it
_MAX_NORM, _UNSCALE = 1.0, 0.125          # (gradients summed over 8 micro-batches)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == _BF16 else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] == "clip":
        sizes = _sizes(case)
        kinds = {_BF16: [torch.bfloat16], _F32: [torch.float32],
                 "mixed": [torch.bfloat16, torch.bfloat16, torch.float32]}[case["types"]]
        # a norm of 2.5 to 7.5 after the division by the number of micro-batches, another
        # one each step
        sigma = random.Random(seed).uniform(2.5, 7.5) / _UNSCALE / math.sqrt(sum(sizes))
        if case["flat"]:
            # each type's gradients one behind the other, as a bucket holds them
            of = [kinds[i % len(kinds)] for i in range(len(sizes))]
            grads = [None] * len(sizes)
            for dt in set(of):
                at = [i for i, o in enumerate(of) if o == dt]
                flat = (randn(sum(sizes[i] for i in at)) * sigma).to(dt)
                for i, t in zip(at, flat.split([sizes[i] for i in at])):
                    grads[i] = t
        else:
            grads = [(randn(n) * sigma).to(kinds[i % len(kinds)]) for i, n in enumerate(sizes)]
        s["grads"] = grads
        s["out"] = [torch.empty_like(t) for t in grads] if case["write"] else None
        return s

    dt = _dtype(case)
    lens = _lengths(case)
    t = case["tokens"]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] == "qk":
        hq, hkv, d, rot = (case[n] for n in ("hq", "hkv", "d", "rot"))
        if case["fused"]:
            qkv = randn(t, hq + 2 * hkv, d).to(dt)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            s["q"], s["k"] = randn(t, hq, d).to(dt), randn(t, hkv, d).to(dt)
        s["wq"], s["wk"] = ((1 + 0.1 * randn(d)).to(dt) for _ in range(2))
        i = torch.arange(0, rot, 2, dtype=torch.float64)
        s["freqs"] = (case["base"] ** (-i / rot)).cuda()
        s["positions"] = None
        if case["explicit"]:
            s["positions"] = torch.randint(0, 400000, (t,), generator=g, device="cuda",
                                           dtype=torch.int32)
        if case["back"]:
            p = case["groups"]
            s["dq"] = randn(p, t, hq // p, d).to(dt) if p > 1 else randn(t, hq, d).to(dt)
            s["dk"] = randn(t, hkv, d).to(dt)
        return s

    vocab = case["vocab"]
    targets = torch.randint(0, max(1, vocab), (t,), generator=g, device="cuda", dtype=torch.int32)
    scored = torch.zeros(t, dtype=torch.bool)
    for first, (a, b) in zip(cu, _answers(case)):
        scored[first + a:first + b] = True
    scored = scored.cuda()
    s["targets"] = targets.masked_fill(~scored, -1)
    if vocab:
        # a spread of 2.5, the sampled tokens among the likely ones
        s["logits"] = torch.randn((t, vocab), generator=g, device="cuda", dtype=dt).mul_(2.5)
        rows = torch.arange(t, device="cuda")
        s["logits"][rows, targets.long()] = (8 + 3 * randn(t)).to(dt)
        logp = _scores(s["logits"], targets)
    else:
        logp = -randn(t).abs()
        s["logp"] = logp
    if case["op"] == "policy":
        # the policy that sampled is some updates old; a log ratio within 1e-4 of a
        # border of the clip, whose side would be a matter of rounding, is moved off it
        old = logp + 0.15 * randn(t)
        for border in (math.log(1 - _CLIP_LOW), math.log(1 + _CLIP_HIGH)):
            old = torch.where((logp - old - border).abs() < 1e-4, old - 1e-3, old)
        s["old"] = old
        s["ref"] = logp + 0.3 * randn(t) if case["kl"] else None
        s["advantages"] = randn(len(lens) if case["advantages"] == "documents" else t)
    if case["op"] == "preference":
        s["ref"] = logp + 0.5 * randn(t)
    return s


def _scores(logits, targets):
    """Log-probability of the targets, some rows at a time."""
    out = []
    for i in range(0, logits.shape[0], 1024):
        x = logits[i:i + 1024].float() / _TEMPERATURE
        out.append(x.gather(1, targets[i:i + 1024, None].long())[:, 0] - x.logsumexp(-1))
    return torch.cat(out)


# ----------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"qk": _plain_qk, "logp": _plain_logp, "policy": _plain_policy,
            "preference": _plain_preference, "clip": _plain_clip}[case["op"]](state, case)


def _own(s, case):
    from variable_length_sequence_gb300 import nsp
    op = case["op"]
    if op == "qk":
        kw = dict(layout=case["layout"], mscale=_ATTN_FACTOR, eps=_EPS, positions=s["positions"],
                  q_groups=case["groups"])
        if case["back"]:
            return nsp.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["cu"], s["freqs"],
                                        s["wq"], s["wk"], **kw)
        return nsp.qk_norm_rope(s["q"], s["k"], s["cu"], s["freqs"], s["wq"], s["wk"], **kw)
    if op == "logp":
        return nsp.token_logp(s["logits"], s["targets"], scale=1 / _TEMPERATURE)
    if op == "policy":
        return nsp.policy_loss_logits(s["logits"], s["targets"], s["old"], s["advantages"], s["cu"],
                                      ref=s["ref"], clip_low=_CLIP_LOW, clip_high=_CLIP_HIGH,
                                      kl_coef=_KL, mean=case["mean"], scale=1 / _TEMPERATURE)
    if op == "preference":
        kw = dict(ref=s["ref"], kind=case["kind"], beta=_BETA, smoothing=_SMOOTHING,
                  average=case["average"])
        if not case["vocab"]:
            return nsp.preference_loss(s["logp"], s["targets"], s["cu"], **kw)
        logp, lse = nsp.token_logp(s["logits"], s["targets"], scale=1 / _TEMPERATURE)
        stats, rewards, dlogp = nsp.preference_loss(logp, s["targets"], s["cu"], **kw)
        dlogits = nsp.token_logp_bwd(s["logits"], s["targets"], lse, dlogp, scale=1 / _TEMPERATURE)
        return stats, rewards, dlogits
    if case["write"]:
        norm = nsp.clip_grads(s["grads"], _MAX_NORM, unscale=_UNSCALE, out=s["out"])
        return [norm] + s["out"]
    return nsp.grad_norm(s["grads"], unscale=_UNSCALE)


# ----------------------------------------------------------------------------- plain forms

def _document_of(cu, t):
    return torch.searchsorted(cu[1:].contiguous(), torch.arange(t, device=cu.device), right=True)


def _plain_qk(s, case):
    t, rot, dt, p = case["tokens"], case["rot"], _dtype(case), case["groups"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(t, device="cuda") - s["cu"].long()[_document_of(s["cu"], t)]
    angle = pos.double()[:, None] * s["freqs"][None]
    cos = (angle.cos() * _ATTN_FACTOR).float()[:, None]
    sin = (angle.sin() * _ATTN_FACTOR).float()[:, None]

    def rotate(y, sin):
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
        return torch.cat([turned, y[..., rot:]], -1)

    def normed(x):
        x = x.float()
        r = (x.square().mean(-1, keepdim=True) + _EPS).rsqrt()
        return x * r, r

    if not case["back"]:
        q = rotate(normed(s["q"])[0] * s["wq"].float(), sin).to(dt)
        k = rotate(normed(s["k"])[0] * s["wk"].float(), sin).to(dt)
        if p > 1:
            q = q.view(t, p, case["hq"] // p, case["d"]).transpose(0, 1).contiguous()
        return q, k

    def back(x, weight, dy):
        n, r = normed(x)
        dn = rotate(dy.float(), -sin)
        u = dn * weight.float()
        dx = r * (u - n * (u * n).mean(-1, keepdim=True))
        return dx.to(dt), (dn * n).sum((0, 1)).to(dt)

    dq = s["dq"]
    if p > 1:
        dq = dq.transpose(0, 1).reshape(t, case["hq"], case["d"])
    dq, dwq = back(s["q"], s["wq"], dq)
    dk, dwk = back(s["k"], s["wk"], s["dk"])
    return dq, dk, dwq, dwk


def _log_probabilities(s):
    """Of the targets (0 where there is none), the scaled logits and their log sums."""
    x = s["logits"].float() / _TEMPERATURE
    top = x.amax(-1, keepdim=True)
    lse = top[:, 0] + (x - top).exp().sum(-1).log()
    logp = x.gather(1, s["targets"].clamp(min=0).long()[:, None])[:, 0] - lse
    there = s["targets"] >= 0
    return torch.where(there, logp, 0.0), x, torch.where(there, lse, 0.0)


def _logits_gradient(s, case, x, lse, dlogp):
    p = (x - lse[:, None]).exp()
    dx = p * -dlogp[:, None]
    dx.scatter_add_(1, s["targets"].clamp(min=0).long()[:, None], dlogp[:, None])
    dx = torch.where((s["targets"] >= 0)[:, None], dx, 0.0)
    return (dx / _TEMPERATURE).to(_dtype(case))


def _plain_logp(s, case):
    logp, _, lse = _log_probabilities(s)
    return logp, lse


def _plain_policy(s, case):
    t, there = case["tokens"], s["targets"] >= 0
    logp, x, lse = _log_probabilities(s)
    doc = _document_of(s["cu"], t)
    counts = torch.zeros(s["cu"].numel() - 1, device="cuda").index_add_(0, doc, there.float())
    if case["mean"] == "tokens":
        weight = there.float() / counts.sum().clamp(min=1)
    else:
        weight = there.float() / (counts[doc].clamp(min=1) * (counts > 0).sum().clamp(min=1))
    a = s["advantages"] if case["advantages"] == "tokens" else s["advantages"][doc]
    ratio = (logp - s["old"]).exp()
    surrogate = -torch.minimum(ratio * a, ratio.clamp(1 - _CLIP_LOW, 1 + _CLIP_HIGH) * a)
    clipped = ((a > 0) & (ratio > 1 + _CLIP_HIGH)) | ((a < 0) & (ratio < 1 - _CLIP_LOW))
    dlogp = torch.where(clipped, 0.0, -ratio * a)
    kl = torch.zeros_like(logp)
    if s["ref"] is not None:
        far = s["ref"] - logp
        kl = far.exp() - far - 1
        dlogp = dlogp + _KL * (1 - far.exp())
    dlogp = dlogp * weight

    def mean(v):
        return torch.where(there, v.double() * weight.double(), 0.0).sum()

    stats = torch.stack([mean(surrogate) + _KL * mean(kl), mean(surrogate), mean(kl),
                         mean(clipped)]).float()
    return stats, torch.where(there, logp, 0.0), _logits_gradient(s, case, x, lse, dlogp)


def _plain_preference(s, case):
    t, there = case["tokens"], s["targets"] >= 0
    if case["vocab"]:
        logp, x, lse = _log_probabilities(s)
    else:
        logp = s["logp"]
    doc = _document_of(s["cu"], t)
    docs = s["cu"].numel() - 1

    def total(v):                           # of each document, long sums in 64 bits
        v = torch.where(there, v.double(), 0.0)
        return torch.zeros(docs, dtype=torch.float64, device="cuda").index_add_(0, doc, v)

    count = total(torch.ones(t, device="cuda")).clamp(min=1)
    score = total(logp.double() - s["ref"].double())
    if case["average"]:
        score = score / count
    rewards = _BETA * score
    h = rewards[0::2] - rewards[1::2]
    n = h.numel()
    if case["kind"] == "sigmoid":
        softplus = (-h).clamp(min=0) + (1 + (-h.abs()).exp()).log()
        loss = softplus + _SMOOTHING * h
        dh = _SMOOTHING - 1 / (1 + h.exp())
    elif case["kind"] == "hinge":
        loss, dh = (1 - h).clamp(min=0), -(h < 1).double()
    else:
        off = h / _BETA - 1 / (2 * _BETA)
        loss, dh = off.square(), 2 * off / _BETA
    stats = torch.stack([loss.mean(), (h > 0).double().mean()]).float()
    dscore = torch.stack([dh, -dh], 1).flatten() * _BETA / n
    if case["average"]:
        dscore = dscore / count
    dlogp = torch.where(there, dscore[doc], 0.0).float()
    if not case["vocab"]:
        return stats, rewards.float(), dlogp
    return stats, rewards.float(), _logits_gradient(s, case, x, lse, dlogp)


def _plain_clip(s, case):
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]])
    norm = squares.sum().sqrt() * _UNSCALE
    if not case["write"]:
        return norm.float()[None]
    factor = ((_MAX_NORM / (norm + _EPS)).clamp(max=1.0) * _UNSCALE).float()
    return [norm.float()[None]] + [(g.float() * factor).to(g.dtype) for g in s["grads"]]


# ----------------------------------------------------------------------------- what a pass needs

def work(case):
    if case["op"] == "clip":
        sizes = _sizes(case)
        each = {_BF16: [2], _F32: [4], "mixed": [2, 2, 4]}[case["types"]]
        n = sum(size * each[i % len(each)] for i, size in enumerate(sizes))
        return {"bytes": n * (2 if case["write"] else 1),
                "flops": (3 if case["write"] else 2) * sum(sizes)}
    es = 2 if case["dtype"] == _BF16 else 4
    t = case["tokens"]
    if case["op"] == "qk":
        n = t * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": (3 if case["back"] else 2) * n * es, "flops": n * (14 if case["back"] else 7)}
    rows, vocab = sum(b - a for a, b in _answers(case)), case["vocab"]
    if case["op"] == "logp":
        return {"bytes": rows * (vocab * es + 8) + 4 * t, "flops": 4 * rows * vocab}
    vectors = 4 * t * (4 if case["op"] == "policy" else 3)
    return {"bytes": (rows + t) * vocab * es + vectors, "flops": rows * (8 * vocab + 20)}


# ----------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"qk": _exact_qk, "logp": _exact_logp, "policy": _exact_policy,
            "preference": _exact_preference, "clip": _exact_clip}[case["op"]](s, case)


def _exact_qk(s, case):
    t, rot, p = case["tokens"], case["rot"], case["groups"]
    if s["positions"] is not None:
        pos = s["positions"].double()
    else:
        pos = torch.cat([torch.arange(n, device="cuda", dtype=torch.float64) for n in _lengths(case)])
    turn = torch.polar(torch.full((t, rot // 2), _ATTN_FACTOR, dtype=torch.float64, device="cuda"),
                       torch.outer(pos, s["freqs"]))[:, None, :]

    def forward(x, w):
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + _EPS) * w
        if case["layout"] == "half":
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            z = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_real(torch.view_as_complex(
                y[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * turn).flatten(-2)
        return torch.cat([z, y[..., rot:]], -1)

    if not case["back"]:
        q, k = forward(s["q"].double(), s["wq"].double()), forward(s["k"].double(), s["wk"].double())
        return (torch.stack(q.chunk(p, dim=1)) if p > 1 else q), k
    grads = []
    for x, w, dy in ((s["q"], s["wq"], s["dq"]), (s["k"], s["wk"], s["dk"])):
        if dy.dim() == 4:
            dy = torch.cat(list(dy), dim=1)
        x, w = x.double().requires_grad_(), w.double().requires_grad_()
        grads.append(torch.autograd.grad(forward(x, w), (x, w), dy.double()))
    return grads[0][0], grads[1][0], grads[0][1], grads[1][1]


def _exact_scores(s, case, dlogp=None):
    """Log-probabilities and log sums of the scored rows, or, given the gradient of
    the former, the gradient of the logits: some rows at a time."""
    t, vocab = case["tokens"], case["vocab"]
    logp, lse = (torch.zeros(t, dtype=torch.float64, device="cuda") for _ in range(2))
    grad = None
    if dlogp is not None:
        grad = torch.zeros(t, vocab, dtype=torch.float64, device="cuda")
    for rows in torch.nonzero(s["targets"] >= 0)[:, 0].split(512):
        x = s["logits"][rows].double() / _TEMPERATURE
        at = s["targets"][rows].long()
        if grad is None:
            lse[rows] = torch.logsumexp(x, -1)
            logp[rows] = torch.log_softmax(x, -1)[torch.arange(len(rows), device="cuda"), at]
        else:
            one = torch.nn.functional.one_hot(at, vocab).double()
            grad[rows] = (one - torch.softmax(x, -1)) * dlogp[rows, None] / _TEMPERATURE
    return grad if grad is not None else (logp, lse)


def _exact_logp(s, case):
    return _exact_scores(s, case)


def _spans(case):
    """First and one past the last scored row of each document, in the stream."""
    at, spans = 0, []
    for n, (a, b) in zip(_lengths(case), _answers(case)):
        spans.append((at + a, at + b))
        at += n
    return spans


def _exact_policy(s, case):
    logp, _ = _exact_scores(s, case)
    leaf = logp.clone().requires_grad_()
    spans = [(i, a, b) for i, (a, b) in enumerate(_spans(case)) if b > a]
    scored = sum(b - a for _, a, b in spans)
    parts = torch.zeros(3, dtype=torch.float64, device="cuda")
    for i, a, b in spans:
        adv = s["advantages"].double()
        adv = adv[a:b] if case["advantages"] == "tokens" else adv[i]
        rho = torch.exp(leaf[a:b] - s["old"][a:b].double())
        bounded = torch.clip(rho, 1 - _CLIP_LOW, 1 + _CLIP_HIGH)
        gain = torch.where(rho * adv <= bounded * adv, rho * adv, bounded * adv)
        kl = torch.zeros_like(rho)
        if s["ref"] is not None:
            z = s["ref"][a:b].double() - leaf[a:b]
            kl = torch.expm1(z) - z
        cut = (bounded * adv < rho * adv).double()
        terms = torch.stack([-gain.sum(), kl.sum(), cut.sum()])
        parts = parts + terms / (scored if case["mean"] == "tokens" else (b - a) * len(spans))
    loss = parts[0] + _KL * parts[1]
    dlogp = torch.zeros_like(logp)
    if spans:
        dlogp = torch.autograd.grad(loss, leaf)[0]
    stats = torch.stack([loss, *parts]).detach()
    return stats, logp, _exact_scores(s, case, dlogp)


def _exact_preference(s, case):
    logp = _exact_scores(s, case)[0] if case["vocab"] else s["logp"].double()
    leaf = logp.clone().requires_grad_()
    rewards = []
    for a, b in _spans(case):
        score = leaf[a:b].sum() - s["ref"][a:b].double().sum()
        rewards.append(_BETA * (score / max(1, b - a) if case["average"] else score))
    rewards = torch.stack(rewards)
    h = rewards[0::2] - rewards[1::2]
    if case["kind"] == "sigmoid":
        ls = torch.nn.functional.logsigmoid
        loss = -(1 - _SMOOTHING) * ls(h) - _SMOOTHING * ls(-h)
    elif case["kind"] == "hinge":
        loss = torch.relu(1 - h)
    else:
        loss = (h / _BETA - 0.5 / _BETA) ** 2
    dlogp = torch.autograd.grad(loss.mean(), leaf)[0]
    stats = torch.stack([loss.mean(), (h > 0).double().mean()]).detach()
    if not case["vocab"]:
        return stats, rewards.detach(), dlogp
    return stats, rewards.detach(), _exact_scores(s, case, dlogp)


def _exact_clip(s, case):
    norm = torch.linalg.vector_norm(torch.stack(
        [torch.linalg.vector_norm(g.double()) for g in s["grads"]])) * _UNSCALE
    if not case["write"]:
        return norm[None]
    factor = torch.minimum(torch.ones_like(norm), _MAX_NORM / (norm + _EPS)) * _UNSCALE
    return [norm[None]] + [g.double() * factor for g in s["grads"]]
