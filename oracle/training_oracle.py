"""fp64 oracle of the router's losses and of orthogonalised updates.

Definitions (include/moe.h prints them in full):

* router's losses: p = softmax(logits) over the experts; sequence s with N_s
  counted tokens, c[s,e] of its (token, slot) pairs on expert e; f = E c/(k N_s),
  P = mean p; balance = sum_s N_s/N sum_e f P, z = mean logsumexp^2; the gradient
  holds f fixed.
* orthogonalised update: m' = momentum*m + (1-dampening)*g, U = m' or with
  nesterov (1-dampening)*g + momentum*m', X = U/(|U|+eps) and steps times
  X <- a X + b (X X^T) X + c (X X^T)^2 X.

The functions that a kernel is held against also return the magnitudes of what
each value is added up from, or have a form with the kernel's roundings.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24          # half a step of fp32
DEFAULT = (3.4445, -4.7750, 2.0315)


# ------------------------------------------------------- router's losses
def softmax(logits):
    """p, logsumexp; a row without a logit above -inf gives zeros."""
    top = logits.max(axis=1, keepdims=True)
    empty = np.isneginf(top)
    with np.errstate(invalid="ignore"):
        e = np.where(empty, 0.0, np.exp(logits - np.where(empty, 0.0, top)))
        total = np.where(empty, 1.0, e.sum(axis=1, keepdims=True))
        lse = np.where(empty, 0.0, top + np.log(total))
    return e / total, lse[:, 0]


def segments(T, S, mask=None, offsets=None):
    """[S, T]: 1 where token t counts in sequence s."""
    t = np.arange(T)
    live = np.ones(T) if mask is None else (np.asarray(mask) != 0).astype(np.float64)
    offsets = np.array([0, T]) if offsets is None else np.asarray(offsets)
    return np.stack([live * ((t >= offsets[s]) & (t < offsets[s + 1])) for s in range(S)])


def router_loss(logits, topk_idx, S, balance_coef, z_coef, mask=None, offsets=None):
    """counts, tokens, probs, loss[3], and z's magnitude with its derivative's."""
    T, E = logits.shape
    k = topk_idx.shape[1]
    p, lse = softmax(logits)
    seg = segments(T, S, mask, offsets)
    hot = np.zeros((T, E))
    for i in range(k):
        np.add.at(hot, (np.arange(T), topk_idx[:, i]), 1.0)
    counts = seg @ hot
    n = seg.sum(axis=1)
    N = max(n.sum(), 1.0)
    some = np.maximum(n, 1.0)[:, None]
    probs = (seg @ p) / some
    f = counts * E / (k * some)
    balance = (n[:, None] * f * probs).sum() / N
    w = seg.sum(axis=0)
    z = (w * lse * lse).sum() / N
    loss = np.array([balance_coef * balance + z_coef * z, balance, z])
    tokens = np.concatenate([n, [n.sum()]])
    return counts.astype(np.int64), tokens.astype(np.int64), probs, loss, (w * np.abs(lse)).sum() / N


def router_loss_grad(logits, k, S, counts, tokens, balance_coef, z_coef, mask=None, offsets=None,
                     dloss=1.0, routed=None):
    """dlogits and the magnitude of the terms that each is added up from;
    routed: (dw, topk_w, topk_idx)."""
    T, E = logits.shape
    p, lse = softmax(logits)
    seg = segments(T, S, mask, offsets)
    f = seg.T @ (counts * E / (k * np.maximum(tokens[:S], 1.0)[:, None]))        # [T, E]
    scale = (dloss / max(tokens[S], 1.0)) * seg.sum(axis=0)[:, None]
    dot = (f * p).sum(axis=1, keepdims=True)
    out = scale * p * (balance_coef * (f - dot) + 2 * z_coef * lse[:, None])
    mag = np.abs(scale) * p * (abs(balance_coef) * (f + 1 + dot + 1) +
                               2 * abs(z_coef) * np.abs(lse)[:, None])
    if routed is not None:
        dw, w, idx = routed
        share = w * (dw - (w * dw).sum(axis=1, keepdims=True))
        size = np.abs(w) * (np.abs(dw) + np.abs(w * dw).sum(axis=1, keepdims=True))
        for i in range(k):
            at = (np.arange(T), idx[:, i])
            np.add.at(out, at, share[:, i])
            np.add.at(mag, at, size[:, i])
    return out, mag


# ------------------------------------------------- orthogonalised updates
def momentum_update(g, m, momentum, dampening=0.0, nesterov=False):
    """m', U (m None: no momentum)."""
    if m is None:
        return None, g
    m = momentum * m + (1 - dampening) * g
    return m, (1 - dampening) * g + momentum * m if nesterov else m


def orthogonalize(u, steps=5, coefficients=DEFAULT, eps=1e-7, scale=1.0):
    """One matrix [rows, cols]."""
    a, b, c = coefficients
    x = u / (np.linalg.norm(u) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(steps):
        A = x @ x.T
        x = a * x + (b * A + c * (A @ A)) @ x
    return scale * (x.T if tall else x)


def orthogonalize_rounded(u, steps=5, coefficients=DEFAULT, eps=1e-7, scale=1.0, joined=False):
    """The same with the roundings that the kernels make: the products' operands as
    fp16 of values times powers of two; joined: the first two steps as one, by
    polynomials of A."""
    a, b, c = coefficients

    def half(v, by):
        return (v * by).astype(np.float16).astype(np.float64) / by

    xs = 2.0 ** round(0.5 * np.log2(u.size))
    x = u / (np.linalg.norm(u) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for step in range(1 if joined else 0, steps):
        hi = half(x, xs)
        A = half(hi @ hi.T, 4096.0)
        B = b * A + c * (A @ A)
        if joined and step == 1:
            B = half(B, 1.0)
            N = half(2 * a * B + B @ B, 1.0)
            A2 = half(a * a * A + N @ A, 4096.0)
            B2 = half(b * A2 + c * (A2 @ A2), 1.0)
            x = a * a * x + half(a * (B + B2) + B2 @ B, 1.0) @ hi
            continue
        s = 0.0
        if step >= steps - 2:
            s = (b * np.trace(A) + c * (A * A).sum()) / len(A)
            B = B - s * np.eye(len(A))
        x = (a + s) * x + half(B, 1.0) @ hi
    return scale * (x.T if tall else x)
