"""Plain CPU float64 reference of the operators on causal sequences: rotary positions, head norms and
causal attention with grouped heads, forward and gradient.

Written from the definitions with numpy, one head at a time; it shares no code with the CUDA path.

  rotation   pair (a, b) of a head at angle t f: (a cos - b sin, b cos + a sin) * amplitude
  norm       y = x w / sqrt(mean(x^2) + eps)
  attention  query i of n sees keys j <= m - n + i of m; S = scale q k^T, O = softmax(S) V,
             LSE = ln sum exp S; no visible key: O = 0, LSE = -inf
"""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------- rotation and norm
def angles(positions, radians, axis_pairs):
    """[tokens, pairs] angles; positions [tokens, axes]."""
    axis = np.repeat(np.arange(len(axis_pairs)), axis_pairs)
    return positions.astype(np.float64)[:, axis] * np.asarray(radians, dtype=np.float64)


def rotate(x, angle, half, amplitude=1.0):
    """x [tokens, heads, d], the first 2 * pairs channels rotated."""
    x = np.asarray(x, dtype=np.float64)
    pairs = angle.shape[1]
    first = np.arange(pairs)
    a, b = (first, first + pairs) if half else (2 * first, 2 * first + 1)
    cos, sin = (np.cos(angle) * amplitude)[:, None], (np.sin(angle) * amplitude)[:, None]
    out = x.copy()
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out


def rms_norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * weight


def rms_norm_grad(x, weight, eps, dy):
    """(dx, dweight) of <dy, rms_norm(x)>."""
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    n = x * r
    dn = dy * weight
    dx = r * (dn - n * np.mean(dn * n, -1, keepdims=True))
    return dx, np.sum(dy * n, axis=(0, 1))


# ---------------------------------------------------------------- attention
def visible(n, m):
    """[n, m] truth values: query i sees key j."""
    return np.arange(m)[None, :] <= m - n + np.arange(n)[:, None]


def attend_head(q, k, v, scale):
    """(P, O, LSE) of one head's rows q [n, d], k, v [m, d]."""
    n, m = len(q), len(k)
    s = np.where(visible(n, m), scale * (q @ k.T), -np.inf) if m else np.zeros((n, 0))
    top = s.max(1, keepdims=True, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(1, keepdims=True)
    p = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
    with np.errstate(divide="ignore"):
        lse = (np.where(np.isfinite(top), top, 0.0) + np.log(total))[:, 0]
    return p, p @ v, lse


def attend(q, k, v, seqs, scale):
    """(O [Tq, Hq, d], LSE [Tq, Hq]); rows of no sequence are NaN."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    hq, hk = q.shape[1], k.shape[1]
    o, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    for q0, n, k0, m in seqs:
        for h in range(hq):
            c = h // (hq // hk)
            _, o[q0:q0 + n, h], lse[q0:q0 + n, h] = attend_head(q[q0:q0 + n, h], k[k0:k0 + m, c], v[k0:k0 + m, c], scale)
    return o, lse


def attend_grad(q, k, v, d_o, seqs, scale):
    """(dq, dk, dv) of <d_o, O>; rows of no sequence are NaN."""
    q, k, v, d_o = (np.asarray(x, dtype=np.float64) for x in (q, k, v, d_o))
    hq, hk = q.shape[1], k.shape[1]
    dq, dk, dv = (np.full(x.shape, np.nan) for x in (q, k, v))
    for q0, n, k0, m in seqs:
        dk[k0:k0 + m] = dv[k0:k0 + m] = 0.0
        for h in range(hq):
            c = h // (hq // hk)
            qh, kh, vh, g = q[q0:q0 + n, h], k[k0:k0 + m, c], v[k0:k0 + m, c], d_o[q0:q0 + n, h]
            p, o, _ = attend_head(qh, kh, vh, scale)
            ds = p * (g @ vh.T - np.sum(g * o, 1, keepdims=True))
            dq[q0:q0 + n, h] = scale * (ds @ kh)
            dk[k0:k0 + m, c] += scale * (ds.T @ qh)
            dv[k0:k0 + m, c] += p.T @ g
    return dq, dk, dv
