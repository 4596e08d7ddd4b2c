"""Plain fp64 NumPy definitions of the dense-attention operators: causal attention
over whole prompts and its gradients, attention of a tree of drafted tokens over a
cache, and the norm and rotation of heads with their gradients.

Test infrastructure only; shares no code with the GPU path.  Next to each result
stand the sums of magnitudes that the tests' error bounds are made of.
"""
from __future__ import annotations

import math
from typing import Optional

import numpy as np


def _f64(x) -> np.ndarray:
    if hasattr(x, "detach"):
        x = x.detach().double().cpu().numpy()
    return np.asarray(x, dtype=np.float64)


def attend_head(q, k, v, sees, scale: float):
    """One head: q [n, D], k, v [m, D], sees [n, m] truth values.  Returns (P [n, m],
    out [n, D], lse [n]); a row that sees nothing has P = 0, out = 0, lse = -inf.
    Hidden keys and values take no part, whatever they hold."""
    n, m = sees.shape
    p = np.zeros((n, m))
    out = np.zeros((n, v.shape[1]))
    lse = np.full(n, -np.inf)
    for i in range(n):
        cols = np.flatnonzero(sees[i])
        if cols.size == 0:
            continue
        s = scale * (k[cols] @ q[i])
        top = s.max()
        e = np.exp(s - top)
        p[i, cols] = e / e.sum()
        out[i] = p[i, cols] @ v[cols]
        lse[i] = top + math.log(e.sum())
    return p, out, lse


def causal(n: int, m: int, pos0: int) -> np.ndarray:
    """Row i, at position pos0 + i, sees keys 0 .. pos0 + i."""
    return np.arange(m)[None, :] <= pos0 + np.arange(n)[:, None]


def dense_attend(q, k, v, pos0: int, scale: Optional[float] = None, dout=None):
    """One sequence: q [n, Hq, D], k, v [m, Hkv, D]; dout like q for the gradients.

    Returns a dict: out, lse, and out_mag = sum_j P_j |v_j|; with dout also dq, dk, dv,
    their error weights dv_mag = sum P |dout|, dq_mag, dk_mag (sums of |dS| times |k|,
    |q|), dq_p, dk_p (the same with P times the row's error scale of delta, sum_d
    |dout_d| (out_mag_d + |out_d|), in place of |dS|) and dq_f, dk_f (that of delta and of
    dout . v, sum_d |dout_d| |v_d|, together)."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    n, hq, d = q.shape
    m, hkv, _ = k.shape
    g = hq // hkv
    scale = 1.0 / math.sqrt(d) if not scale else scale
    sees = causal(n, m, pos0)
    r = {"out": np.zeros_like(q), "lse": np.zeros((n, hq)), "out_mag": np.zeros_like(q)}
    if dout is not None:
        dout = _f64(dout)
        for name in ("dq", "dq_mag", "dq_p", "dq_f"):
            r[name] = np.zeros_like(q)
        for name in ("dk", "dk_mag", "dk_p", "dk_f", "dv", "dv_mag"):
            r[name] = np.zeros_like(k)
    for h in range(hq):
        c = h // g
        p, o, lse = attend_head(q[:, h], k[:, c], v[:, c], sees, scale)
        r["out"][:, h], r["lse"][:, h] = o, lse
        r["out_mag"][:, h] = p @ np.abs(v[:, c])
        if dout is None:
            continue
        do = dout[:, h]
        delta = (do * o).sum(1, keepdims=True)
        dp = do @ v[:, c].T
        ds = p * (dp - delta)
        r["dq"][:, h] = scale * ds @ k[:, c]
        r["dk"][:, c] += scale * ds.T @ q[:, h]
        r["dv"][:, c] += p.T @ do
        r["dv_mag"][:, c] += p.T @ np.abs(do)
        r["dq_mag"][:, h] = scale * np.abs(ds) @ np.abs(k[:, c])
        r["dk_mag"][:, c] += scale * np.abs(ds).T @ np.abs(q[:, h])
        w = p * (np.abs(do) * (r["out_mag"][:, h] + np.abs(o))).sum(1, keepdims=True)
        r["dq_p"][:, h] = scale * w @ np.abs(k[:, c])
        r["dk_p"][:, c] += scale * w.T @ np.abs(q[:, h])
        w = w + p * (np.abs(do) @ np.abs(v[:, c]).T)
        r["dq_f"][:, h] = scale * w @ np.abs(k[:, c])
        r["dk_f"][:, c] += scale * w.T @ np.abs(q[:, h])
    return r


def tree_attend(q, k, v, mask, kept: int, scale: Optional[float] = None):
    """One sequence: q [n, Hq, D], the cache's rows k, v [>= kept + n, Hkv, D], mask
    [n, n] truth values.  Returns out, lse and out_mag as :func:`dense_attend`."""
    q, k, v = _f64(q), _f64(k)[:kept + len(q)], _f64(v)[:kept + len(q)]
    n, hq, d = q.shape
    g = hq // k.shape[1]
    scale = 1.0 / math.sqrt(d) if not scale else scale
    sees = np.concatenate([np.ones((n, kept), bool), np.asarray(mask, bool)], 1)
    out, mag, lse = np.zeros_like(q), np.zeros_like(q), np.zeros((n, hq))
    for h in range(hq):
        p, o, z = attend_head(q[:, h], k[:, h // g], v[:, h // g], sees, scale)
        seen = sees.any(0)
        out[:, h], lse[:, h] = o, z
        mag[:, h] = p[:, seen] @ np.abs(v[seen, h // g])
    return {"out": out, "lse": lse, "out_mag": mag}


def rotate(y, positions, inv_freq, interleaved: bool, back: bool = False):
    """Turns the first 2 len(inv_freq) elements of y [rows, H, D] by positions *
    inv_freq (back: by the negative angle)."""
    y = _f64(y).copy()
    inv_freq, positions = _f64(inv_freq), np.asarray(positions, dtype=np.float64)
    half = len(inv_freq)
    for i in range(half):
        f = positions * inv_freq[i] * (-1.0 if back else 1.0)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(f)[:, None], np.sin(f)[:, None]
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a] = ya * c - yb * s
        y[..., b] = yb * c + ya * s
    return y


def norm_rope(x, w, inv_freq, positions, eps: float, interleaved: bool):
    """x [rows, H, D] -> rotated w x / sqrt(mean(x^2) + eps)."""
    x, w = _f64(x), _f64(w)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(w * x * r, positions, inv_freq, interleaved)


def norm_rope_backward(dy, x, w, inv_freq, positions, eps: float, interleaved: bool):
    """(dx, dw, dw_mag): gradients of :func:`norm_rope` and the sum of the magnitudes
    that dw adds up."""
    x, w = _f64(x), _f64(w)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = rotate(dy, positions, inv_freq, interleaved, back=True)
    u = r * x
    t = w * g
    dx = r * (t - u * (t * u).mean(-1, keepdims=True))
    return dx, (g * u).sum((0, 1)), np.abs(g * u).sum((0, 1))
