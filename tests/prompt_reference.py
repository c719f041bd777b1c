"""Plain 64-bit forms of the prompt path's operators, and the error bounds its tests allow.

Bounds count roundings. u is half a step of the type (torch.finfo(t).eps / 2,
relative). An attention output sum_t p_t v_t / sum_t p_t carries
  * its own rounding                            u |out|
  * each weight's rounding to the type          u A,  A = sum_t p_t |v_t| / sum_t p_t
  * the scores' 32-bit sums of D products, their scaling and the exponential:
    a score moves by at most D 2^-24 sum_d |q_d k_d| scale (below 2^-13 for the
    inputs here), which moves the weighted mean by at most twice that times A
  * weights and outputs below the type's normal range (fp16: 2^-14), which are
    off by 2^-25 each instead: n 2^-25 max |v|.
"""
from __future__ import annotations

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def attention(q, k, v, scale, first):
    """(out, bound) in 64 bits of q [n][H][D] over k, v [m][Hkv][D]; row i sees keys 0 .. first + i."""
    n, H, D = q.shape
    m, Hkv, _ = k.shape
    G = H // Hkv
    u = U[q.dtype]
    if m == 0:
        return q.double() * 0.0, q.double() * 0.0
    q, k, v = q.double(), k.double(), v.double()
    z = torch.einsum("ngjd,mgd->gjnm", q.view(n, Hkv, G, D), k) * scale
    seen = torch.arange(m, device=q.device)[None, :] <= first + torch.arange(n, device=q.device)[:, None]
    z = z.masked_fill(~seen, float("-inf"))
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top)
    p = torch.where(seen, p, 0.0)
    p = p / p.sum(-1, keepdim=True)

    def weigh(x):
        return torch.einsum("gjnm,mgd->ngjd", p, x).reshape(n, H, D)

    out, a = weigh(v), weigh(v.abs())
    small = m * 2.0 ** -25 * (v.abs().nan_to_num(0.0, 0.0).amax() if m else 0.0)
    bound = u * out.abs() + (u + 2 * D * 2.0 ** -24 * 8.0 + 2.0 ** -20) * a + small + 2.0 ** -25
    if first < 0:  # rows that see nothing are zero
        empty = (first + torch.arange(n, device=q.device)) < 0
        out[empty] = 0.0
        bound[empty] = 0.0
    return out, bound


def gather(pool, row, n):
    """The first n cached rows [n][Hkv][D] of a table row."""
    bs = pool.shape[2]
    ids = row[:-(-n // bs)].long()
    return pool[ids].transpose(1, 2).flatten(0, 1)[:n]


def rope(x, positions, inv_freq, mscale, interleaved):
    """x [T][h][D] turned, in 64 bits."""
    y = x.double().clone()
    half = inv_freq.numel()
    a = positions.double()[:, None, None] * inv_freq
    c, s = torch.cos(a) * mscale, torch.sin(a) * mscale
    i = torch.arange(half, device=x.device)
    e, o = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    p, r = x.double()[..., e], x.double()[..., o]
    y[..., e], y[..., o] = p * c - r * s, r * c + p * s
    return y
