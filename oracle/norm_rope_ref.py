"""Reference for the head norms with rotation and the rotated cache append -- TEST INFRASTRUCTURE ONLY.

Plain definitions in float64:

* ``rms(x, w, eps)``: w x / sqrt(mean(x^2) + eps) over the last axis; x itself where w is None.
* ``rotate(x, pos, inv_freq, interleaved)``: pair i of the last axis -- columns (2i, 2i+1), or
  (i, i + n/2) -- turned by pos * inv_freq[i] radians.
* ``qk_norm_rope``: queries and keys, the nope and the rope part of each head normalised on
  their own, the rope part then rotated.
* ``qk_norm_rope_backward``: the chain rule of that, written out: with g the upstream gradient
  (turned back for the rope part) and r = 1 / sqrt(mean(x^2) + eps),
  dx = r (w g - x r^2 mean(x w g)) and dw = sum g x r.
* ``rope_append_rows``: the finished cache rows of raw rows; ``rope_append`` puts them into a copy
  of the cache.
"""
from __future__ import annotations

import numpy as np


def rms(x, w, eps):
    x = np.asarray(x, dtype=np.float64)
    if w is None:
        return x
    return w * x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def rms_backward(x, w, eps, g):
    """(dx, dw) for the upstream gradient g of rms(x, w, eps); dw summed over all but the last axis."""
    if w is None:
        return g, None
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    dx = r * (w * g - x * r * r * np.mean(x * w * g, axis=-1, keepdims=True))
    return dx, (g * x * r).reshape(-1, x.shape[-1]).sum(axis=0)


def rotate(x, pos, inv_freq, interleaved):
    """x [..., n]; pos broadcastable to x's leading axes."""
    x = np.asarray(x, dtype=np.float64)
    ang = np.asarray(pos, dtype=np.float64)[..., None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang), np.sin(ang)
    n = x.shape[-1]
    first, second = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n))
    y = np.empty_like(x)
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def qk_norm_rope(q, k_nope, k_rope, pos, inv_freq, weights, eps, interleaved):
    """q [B,S,H,dn+dr], k_nope [B,S,H,dn], k_rope [B,S,dr] (each may be None), pos [B,S], weights
    (q_nope, q_rope, k_nope, k_rope).  Returns the four outputs (None where not given)."""
    w_qn, w_qr, w_kn, w_kr = weights
    pos = np.asarray(pos)
    dr = 2 * len(inv_freq)
    qn = qr = kn = kr = None
    if q is not None:
        qn = rms(q[..., :-dr], w_qn, eps)
        qr = rotate(rms(q[..., -dr:], w_qr, eps), pos[..., None], inv_freq, interleaved)
    if k_nope is not None:
        kn = rms(k_nope, w_kn, eps)
    if k_rope is not None:
        kr = rotate(rms(k_rope, w_kr, eps), pos, inv_freq, interleaved)
    return qn, qr, kn, kr


def qk_norm_rope_backward(dqn, dqr, dkn, dkr, q, k_nope, k_rope, pos, inv_freq, weights, eps, interleaved):
    """(dq, dk_nope, dk_rope, dw_qn, dw_qr, dw_kn, dw_kr); None where not given."""
    w_qn, w_qr, w_kn, w_kr = weights
    pos = np.asarray(pos)
    dr = 2 * len(inv_freq)
    res = [None] * 7
    if q is not None:
        a, res[3] = rms_backward(q[..., :-dr], w_qn, eps, dqn)
        b, res[4] = rms_backward(q[..., -dr:], w_qr, eps, rotate(dqr, -pos[..., None], inv_freq, interleaved))
        res[0] = np.concatenate([a, b], axis=-1)
    if k_nope is not None:
        res[1], res[5] = rms_backward(k_nope, w_kn, eps, dkn)
    if k_rope is not None:
        res[2], res[6] = rms_backward(k_rope, w_kr, eps, rotate(dkr, -pos, inv_freq, interleaved))
    return tuple(res)


def append_places(lens, new_lens, T):
    """Place of every row in its sequence, [B, T]; -1 where nothing is written."""
    lens, n = np.asarray(lens, dtype=np.int64), np.asarray(new_lens, dtype=np.int64)
    t = np.arange(T)[None]
    place = lens[:, None] - n[:, None] + t
    return np.where((t < n[:, None]) & (n[:, None] <= T) & (place >= 0), place, -1)


def rope_append_rows(c_new, pos, inv_freq, w, eps, interleaved):
    """Finished rows [B, T, dl + dr] (float64, not rounded) of the raw rows c_new."""
    dr = 2 * len(inv_freq)
    return np.concatenate([rms(c_new[..., :-dr], w, eps), rotate(c_new[..., -dr:], pos, inv_freq, interleaved)],
                          axis=-1)
