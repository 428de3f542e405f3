"""fp64 oracle of the residual block's norms and of gradient clipping.

Definitions (v a row of d channels):

* RMS norm: xhat = v / sqrt(mean(v^2) + eps); layer norm: xhat = (v - mean(v))
  / sqrt(mean((v - mean(v))^2) + eps); both N(v) = xhat*(offset + w) + b.
* pre norm x = N1(r); post norm r' = res_scale*r + branch_scale * G * N2(y),
  then x' = N1(r'); G = act(gate).
* gradients by the chain rule, row by row.
* norm of a gradient list: sqrt of the sum of squares, or the largest
  magnitude; clipped: g * min(1, max_norm / (norm + eps)).

Every function returns, beside each value, the sum of the magnitudes of the
terms it is added up from.  A sum taken in another order or in 32 bits may be
off by a small multiple of 2^-24 times that magnitude, so tests can hold a
kernel to a bound that follows from its arithmetic.
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import numpy as np


@dataclasses.dataclass(frozen=True)
class NormSpec:
    kind: Optional[str]          # "rms" | "layer" | None
    eps: float = 1e-6
    offset: float = 0.0


def _weight(spec, w):
    return 1.0 if w is None else w + spec.offset


def norm_stats(v, spec):
    """xhat, its magnitude, 1/sqrt(...) [T,1]."""
    if spec.kind == "layer":
        mu = v.mean(axis=1, keepdims=True)
        mag_v = np.abs(v) + np.abs(v).mean(axis=1, keepdims=True)
        c = v - mu
    else:
        c, mag_v = v, np.abs(v)
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + spec.eps)
    return c * rstd, mag_v * rstd, rstd


def norm_fwd(v, spec, w=None, b=None):
    if spec.kind is None:
        return v, np.abs(v)
    xh, mag, _ = norm_stats(v, spec)
    ww, bb = _weight(spec, w), (0.0 if b is None else b)
    return xh * ww + bb, mag * np.abs(ww) + np.abs(bb)


def norm_bwd(dn, mag_dn, v, spec, w=None):
    """Gradients of N by v, w and b: three (value, magnitude) pairs."""
    if spec.kind is None:
        return (dn, mag_dn), None, None
    xh, mag_x, rstd = norm_stats(v, spec)
    ww = _weight(spec, w)
    dxh, mag = dn * ww, mag_dn * np.abs(ww)
    dv = dxh - xh * (dxh * xh).mean(axis=1, keepdims=True)
    mag_dv = mag + mag_x * (mag * mag_x).mean(axis=1, keepdims=True)
    if spec.kind == "layer":
        dv = dv - dxh.mean(axis=1, keepdims=True)
        mag_dv = mag_dv + mag.mean(axis=1, keepdims=True)
    return ((dv * rstd, mag_dv * rstd),
            ((dn * xh).sum(axis=0), (mag_dn * mag_x).sum(axis=0)),
            (dn.sum(axis=0), mag_dn.sum(axis=0)))


def gate_value(gate, kind, act):
    """Gate and the derivative of its activation, shaped to broadcast over [T,d]."""
    if kind is None:
        return 1.0, None
    g = gate[:, None] if kind == "token" else gate
    if act == "sigmoid":
        v = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
        return v, v * (1 - v)
    if act == "tanh":
        v = np.tanh(g)
        return v, 1 - v * v
    return g, np.ones_like(g)


def combine_rows(Y, row_of, topk_w):
    picked = Y[row_of] * topk_w[:, :, None].astype(np.float64)
    return picked.sum(axis=1), np.abs(picked).sum(axis=1)


def post_fwd(res, y, mag_y, spec, w=None, b=None, gate=None, gate_kind=None, gate_act=None,
             res_scale=1.0, branch_scale=1.0):
    """r' and its magnitude; mag_y: magnitude of y (|y| for a given tensor)."""
    n, mag = norm_fwd(y, spec, w, b)
    # y's own error reaches n through the statistics and the element itself
    if spec.kind is None:
        mag = np.maximum(mag, mag_y)
    else:
        rstd = norm_stats(y, spec)[2]
        mag = mag + (mag_y - np.abs(y)) * rstd * np.abs(_weight(spec, w))
        mag = mag + np.abs(n) * (mag_y * np.abs(y)).mean(axis=1, keepdims=True) * rstd ** 2
    G, _ = gate_value(gate, gate_kind, gate_act)
    return (res_scale * res + branch_scale * G * n,
            np.abs(res_scale * res) + np.abs(branch_scale * G) * mag)


def norm_fwd_of(v, mag_v, spec, w=None, b=None):
    """N(v) for a v that itself carries the magnitude mag_v."""
    n, mag = norm_fwd(v, spec, w, b)
    rstd = norm_stats(v, spec)[2]
    ww = np.abs(_weight(spec, w))
    extra = (mag_v + (mag_v.mean(axis=1, keepdims=True) if spec.kind == "layer" else 0.0)) * rstd * ww
    spread = (mag_v * np.abs(v)).mean(axis=1, keepdims=True) * rstd ** 2
    return n, mag + extra + np.abs(n) * spread


def join_grads(dres_in, dx, r, spec, w=None, dres_scale=1.0):
    """D = dres_scale*dres_in + N1^T(dx; r): (D, mag), (dw, mag), (db, mag)."""
    D, mag, dw, db = 0.0, 0.0, None, None
    if dres_in is not None:
        D, mag = dres_scale * dres_in, np.abs(dres_scale * dres_in)
    if dx is not None:
        (dv, mag_dv), dw, db = norm_bwd(dx, np.abs(dx), r, spec, w)
        D, mag = D + dv, mag + mag_dv
    return (D, mag), dw, db


def post_bwd(D, mag_D, y, spec, w=None, b=None, gate=None, gate_kind=None, gate_act=None,
             branch_scale=1.0):
    """dict of (value, magnitude): dy, dw, db (with a norm), dgate (with a gate)."""
    n, mag_n = norm_fwd(y, spec, w, b)
    G, slope = gate_value(gate, gate_kind, gate_act)
    out = {}
    if gate_kind is not None:
        dg = branch_scale * D * n * slope
        mag = np.abs(branch_scale * slope) * mag_D * mag_n
        if gate_act == "sigmoid":         # 1 - v in 32 bits
            mag = mag + np.abs(branch_scale) * mag_D * mag_n * np.abs(G)
        elif gate_act == "tanh":
            mag = mag + np.abs(branch_scale) * mag_D * mag_n
        axis = {"channel": 0, "token": 1, "full": None}[gate_kind]
        out["gate"] = (dg, mag) if axis is None else (dg.sum(axis=axis), mag.sum(axis=axis))
    dn, mag_dn = branch_scale * G * D, np.abs(branch_scale * G) * mag_D
    out["dy"], dw, db = norm_bwd(dn, mag_dn, y, spec, w)
    if spec.kind is not None:
        out["dw"], out["db"] = dw, db
    return out


def grad_norm(grads, kind="l2"):
    """Total and each tensor's norm."""
    each = []
    for g in grads:
        g = np.asarray(g, dtype=np.float64).ravel()
        if g.size == 0:
            each.append(0.0)
        elif kind == "inf":
            each.append(np.abs(g).max())
        else:
            top = np.abs(g).max()
            scale = top if np.isfinite(top) and top > 0 else 1.0
            each.append(scale * np.sqrt(((g / scale) ** 2).sum()))
    each = np.array(each)
    if each.size == 0:
        return 0.0, each
    if kind == "inf":
        return each.max(), each
    top = each.max()
    scale = top if np.isfinite(top) and top > 0 else 1.0
    return scale * np.sqrt(((each / scale) ** 2).sum()), each


def clip_factor(norm, max_norm, eps):
    f = max_norm / (norm + eps)
    return 1.0 if f >= 1.0 else f
