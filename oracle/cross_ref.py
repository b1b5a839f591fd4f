"""Reference for cross attention and its gradient -- TEST INFRASTRUCTURE ONLY.

Plain definitions in float64 (torch tensors of any floating type, on any device), one sequence and one head at
a time, over the keys that exist:

* ``forward``: s = scale (qn kn' + qr kr'), lse = logsumexp(s), o = exp(s - lse) v; no key: o = 0, lse = -inf.
  Also the sums that bounds of rounding errors are made of: a = exp(s - lse) |v| and, a row, the largest
  sum of |q k| scale.
* ``backward``: P = exp(s - lse), dV = P' dO, dS = P * (dO V' - rowsum(dO * O)), dQ = scale dS K,
  dK = scale dS' Q, the rope key's over all heads, for given out and lse.  ``bounds`` has, for each
  gradient, what bf16 roundings of P and dS and fp32 sums can be off by, before the gradient's own rounding.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8     # half a step of bf16, relative
E32 = 2.0 ** -16  # fp32 sums of up to 192 products, and the roundings of an exponent's argument, relative


def counts(k_nope, key_lens):
    B, Sk = k_nope.shape[:2]
    return [Sk] * B if key_lens is None else [min(max(int(n), 0), Sk) for n in key_lens]


def _operands(q_nope, q_rope, k_nope, k_rope, v, b, h, n):
    q = torch.cat((q_nope[b, :, h], q_rope[b, :, h]), -1).double()
    k = torch.cat((k_nope[b, :n, h], k_rope[b, :n]), -1).double()
    return q, k, v[b, :n, h].double()


def forward(q_nope, q_rope, k_nope, k_rope, v, key_lens, scale):
    """(o [B,Sq,H,dv], lse [B,H,Sq], a as o, sum |q k| scale [B,H,Sq])."""
    B, Sq, H, _ = q_nope.shape
    o = torch.zeros(B, Sq, H, v.shape[-1], dtype=torch.float64, device=v.device)
    a, lse = o.clone(), torch.full((B, H, Sq), -math.inf, dtype=torch.float64, device=v.device)
    e = torch.zeros(B, H, Sq, dtype=torch.float64, device=v.device)
    for b, n in enumerate(counts(k_nope, key_lens)):
        for h in range(H if n else 0):
            q, k, vv = _operands(q_nope, q_rope, k_nope, k_rope, v, b, h, n)
            s = (q @ k.T) * scale
            lse[b, h] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[b, h][:, None])
            o[b, :, h], a[b, :, h] = p @ vv, p @ vv.abs()
            e[b, h] = ((q.abs() @ k.abs().T) * scale).amax(-1)
    return o, lse, a, e


def backward(q_nope, q_rope, k_nope, k_rope, v, key_lens, scale, out, lse, d_out):
    """(grads, bounds): dq_nope, dq_rope, dk_nope, dk_rope, dv and what each may be off by, float64."""
    dn = q_nope.shape[-1]
    shapes = [q_nope.shape, q_rope.shape, k_nope.shape, k_rope.shape, v.shape]
    g = [torch.zeros(s, dtype=torch.float64, device=v.device) for s in shapes]
    w = [torch.zeros(s, dtype=torch.float64, device=v.device) for s in shapes]
    for b, n in enumerate(counts(k_nope, key_lens)):
        for h in range(q_nope.shape[2] if n else 0):
            q, k, vv = _operands(q_nope, q_rope, k_nope, k_rope, v, b, h, n)
            do, o, l = d_out[b, :, h].double(), out[b, :, h].double(), lse[b, h].double()[:, None]
            p = torch.exp((q @ k.T) * scale - l)
            dp, d = do @ vv.T, (do * o).sum(-1, keepdim=True)
            ds = p * (dp - d)
            dq, dk = scale * ds @ k, scale * ds.T @ q
            for i, x in ((0, dq[:, :dn]), (1, dq[:, dn:]), (2, dk[:, :dn]), (3, dk[:, dn:]), (4, p.T @ do)):
                _add(g, i, b, h, n, x)
            # a weight is off by 4 E32 sum |q k| scale and E32 |lse|, dP - D by E32 of its terms' sum
            p_err = p * (4 * E32 * ((q.abs() @ k.abs().T) * scale + l.abs()) + E32)
            ds_err = U * ds.abs() + p_err * (dp - d).abs() + p * E32 * (do.abs() @ vv.abs().T + (do * o).abs().sum(-1, keepdim=True))
            eq, ek = scale * ds_err @ k.abs(), scale * ds_err.T @ q.abs()
            ev = (U * p + p_err).T @ do.abs()
            # (and E32 of the terms' sum for the accumulation)
            eq, ek = eq + E32 * scale * ds.abs() @ k.abs(), ek + E32 * scale * ds.abs().T @ q.abs()
            for i, x in ((0, eq[:, :dn]), (1, eq[:, dn:]), (2, ek[:, :dn]), (3, ek[:, dn:]), (4, ev + E32 * p.T @ do.abs())):
                _add(w, i, b, h, n, x)
    return g, w


def _add(to, i, b, h, n, x):
    if i < 2:
        to[i][b, :, h] = x
    elif i == 3:  # one rope key for all heads
        to[i][b, :n] += x
    else:
        to[i][b, :n, h] = x
