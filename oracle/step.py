"""Operators of a packed post-training step in float64: head norm with rotation,
log-probabilities of given tokens, the clipped policy loss with its KL term, the
preference loss over pairs of documents, the norm of many gradients.

Plain restatements of the definitions in include/nsp.h, document by document
with numpy; they share no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from .layer import head_norm, head_norm_bwd, rope


def qk_norm_rope(x, weight, angles, rot, interleaved=False, mscale=1.0, eps=1e-6):
    return rope(head_norm(x, weight, None, eps), angles, rot, interleaved, mscale)


def qk_norm_rope_bwd(x, weight, dy, angles, rot, interleaved=False, mscale=1.0, eps=1e-6):
    """dx and dweight (None without a weight)."""
    z = rope(dy, angles, rot, interleaved, mscale, inverse=True)
    # the factor of the rotated columns is in z; the unrotated ones have none
    return head_norm_bwd(x, z, weight, None, eps)[:2]


def token_logp(logits, targets, scale=1.0):
    """logp and lse [T], zero for a row without a target (a negative one)."""
    T = len(targets)
    logp, lse = np.zeros(T), np.zeros(T)
    for t in range(T):
        if targets[t] < 0:
            continue
        x = scale * np.asarray(logits[t], np.float64)
        top = x.max()
        e = x - top
        lse[t] = top + np.log(np.exp(e).sum())
        logp[t] = e[targets[t]] - np.log(np.exp(e).sum())
    return logp, lse


def token_logp_bwd(logits, targets, dlogp, scale=1.0):
    out = np.zeros(np.shape(logits))
    for t in range(len(targets)):
        if targets[t] < 0:
            continue
        x = scale * np.asarray(logits[t], np.float64)
        p = np.exp(x - x.max())
        p /= p.sum()
        out[t] = -scale * dlogp[t] * p
        out[t, targets[t]] += scale * dlogp[t]
    return out


def _documents(cu, T):
    cu = np.asarray(cu, np.int64)
    return [np.arange(min(cu[b], T), min(cu[b + 1], T)) for b in range(len(cu) - 1)]


def policy_loss(logp, old, ref, advantages, targets, cu, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                mean="tokens", total=0.0):
    """stats (loss, surrogate, kl, clipped share) and dlogp [T]; advantages of each
    document or each token; ref may be None; total > 0 takes the place of the
    number of scored tokens or of documents that have one."""
    T = len(logp)
    docs = [d[np.asarray(targets)[d] >= 0] for d in _documents(cu, T)]
    n_tokens, n_docs = sum(len(d) for d in docs), sum(len(d) > 0 for d in docs)
    stats, dlogp = np.zeros(4), np.zeros(T)
    for b, rows in enumerate(docs):
        for t in rows:
            if mean == "tokens":
                w = 1 / (total if total > 0 else n_tokens)
            else:
                w = 1 / ((total if total > 0 else n_docs) * len(rows))
            a = advantages[t] if len(advantages) == T and len(advantages) != len(docs) else advantages[b]
            r = np.exp(logp[t] - old[t])
            cut = (a > 0 and r > 1 + clip_high) or (a < 0 and r < 1 - clip_low)
            pg = -a * (min(max(r, 1 - clip_low), 1 + clip_high) if cut else r)
            g = 0.0 if cut else -a * r
            kl = 0.0
            if ref is not None:
                z = ref[t] - logp[t]
                kl = np.expm1(z) - z
                g -= kl_coef * np.expm1(z)
            stats += w * np.array([pg + kl_coef * kl, pg, kl, float(cut)])
            dlogp[t] = w * g
    return stats, dlogp


def preference_loss(logp, ref, targets, cu, kind="sigmoid", beta=0.1, smoothing=0.0, margin=0.0,
                    average=False):
    """stats (loss, share of pairs whose chosen one is ahead), rewards [documents]
    and dlogp [T]; documents 2 i and 2 i + 1 are the chosen and rejected one."""
    T = len(logp)
    docs = [d[np.asarray(targets)[d] >= 0] for d in _documents(cu, T)]
    score = np.array([sum(logp[t] - (0.0 if ref is None else ref[t]) for t in d) for d in docs])
    if average:
        score = score / np.array([max(1, len(d)) for d in docs])
    rewards = beta * score
    n = len(docs) // 2
    stats, dlogp = np.zeros(2), np.zeros(T)
    for i in range(n):
        h = rewards[2 * i] - rewards[2 * i + 1] - margin
        if kind == "sigmoid":
            loss = (1 - smoothing) * np.logaddexp(0, -h) + smoothing * np.logaddexp(0, h)
            dh = smoothing - np.exp(-np.logaddexp(0, h))
        elif kind == "hinge":
            loss, dh = max(0.0, 1 - h), -1.0 if h < 1 else 0.0
        else:
            off = h / beta - 1 / (2 * beta)
            loss, dh = off * off, 2 * off / beta
        stats += np.array([loss, float(rewards[2 * i] > rewards[2 * i + 1])]) / n
        for d, sign in ((docs[2 * i], 1), (docs[2 * i + 1], -1)):
            dlogp[d] = sign * dh * beta / n / (max(1, len(d)) if average else 1)
    return stats, rewards, dlogp


def grad_norm(grads, unscale=1.0, kind=2):
    if kind == 2:
        return np.sqrt(sum((np.asarray(g, np.float64) ** 2).sum() for g in grads)) * abs(unscale)
    return max([np.abs(np.asarray(g, np.float64)).max() for g in grads if np.size(g)], default=0.0) * abs(unscale)
