"""CPU float64 oracles of what a model step does around the attention: the plan
of a serving step, the head norm with rotary positions and its gradient, and
the attention of several new tokens over a paged cache.

TEST INFRASTRUCTURE ONLY -- never imported by the product path.  Pinned in
tests/test_oracle_step_pins.py against automatic differentiation, complex
arithmetic, closed forms and the main attention oracle.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def oracle_plan(cached, new, free, table, page: int, max_tokens: int):
    """The plan of a step, one token at a time.  cached, new, free: lists; table:
    list of lists, changed in place.  Returns slots, positions, cu, lens, needed."""
    slots, positions, cu, lens, taken = [], [], [0], [], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        have, end = -(-c // page), -(-(c + n) // page)
        for col in range(have, end):
            table[b][col] = free[taken] if taken < len(free) else -1
            taken += 1
        for pos in range(c, c + n):
            pg = table[b][pos // page]
            slots.append(pg * page + pos % page if pg >= 0 else -1)
            positions.append(pos)
        cu.append(min(len(slots), max_tokens))
        lens.append(c + n)
    pad = max_tokens - len(slots)
    return ((slots + [-1] * pad)[:max_tokens], (positions + [0] * pad)[:max_tokens], cu, lens,
            taken)


def pair_dims(rotary: int, interleaved: bool):
    """First and second dimension of every rotated pair."""
    i = torch.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def rope_angles(positions, inv_freq, pair_axis):
    """[T, pairs] in float64; positions [axes, T]."""
    return positions.double()[torch.as_tensor(pair_axis, dtype=torch.long)].T * inv_freq.double()


def oracle_rope(x, weight, angles, *, eps: float, interleaved: bool, amplitude: float):
    """Norm (weight None: none) and rotation of x [T, heads, 64]."""
    u = x.to(F64)
    if weight is not None:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * weight.to(F64)
    a, b = pair_dims(2 * angles.shape[1], interleaved)
    cos, sin = amplitude * torch.cos(angles)[:, None], amplitude * torch.sin(angles)[:, None]
    y = u.clone()
    y[..., a] = u[..., a] * cos - u[..., b] * sin
    y[..., b] = u[..., b] * cos + u[..., a] * sin
    return y


def oracle_rope_bwd(x, weight, angles, dy, *, eps: float, interleaved: bool, amplitude: float):
    """(dx, dweight or None) of oracle_rope, from the formula."""
    g = dy.to(F64).clone()
    a, b = pair_dims(2 * angles.shape[1], interleaved)
    cos, sin = amplitude * torch.cos(angles)[:, None], amplitude * torch.sin(angles)[:, None]
    da, db = dy.to(F64)[..., a], dy.to(F64)[..., b]
    g[..., a] = da * cos + db * sin
    g[..., b] = db * cos - da * sin
    if weight is None:
        return g, None
    x = x.to(F64)
    inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    h = g * weight.to(F64)
    dx = inv * (h - x * inv * inv * (h * x).mean(-1, keepdim=True))
    return dx, (g * x * inv).sum((0, 1))


def oracle_extend(q, k_cache, v_cache, table, seq_lens, cu, sink, *, scale: float,
                  window: int = 0):
    """(out [T, H_q, d], lse [H_q, T], spread) in float64; rows behind cu[-1] are
    NaN.  Keys whose table entry is outside the cache are skipped.  spread =
    sum_j P_ij |v_j|, what the rounding of P can move."""
    t, hq, d = q.shape
    pages, page, hkv = k_cache.shape[:3]
    out = torch.full((t, hq, d), math.nan, dtype=F64)
    lse = torch.full((hq, t), math.nan, dtype=F64)
    spread = torch.full((t, hq, d), math.nan, dtype=F64)
    kf, vf = k_cache.reshape(-1, hkv, d), v_cache.reshape(-1, hkv, d)
    for b in range(len(seq_lens)):
        q0, n, length = int(cu[b]), int(cu[b + 1]) - int(cu[b]), int(seq_lens[b])
        pos = torch.arange(length - n, length)
        j = torch.arange(length)
        seen = j[None] <= pos[:, None]
        if window > 0:
            seen &= j[None] > pos[:, None] - window
        entry = table[b].long()[j // page] if length else j
        seen &= ((entry >= 0) & (entry < pages))[None]
        used = seen.any(0)
        rows = (entry * page + j % page)[used]
        k, v = kf[rows].to(F64), vf[rows].to(F64)
        for h in range(hq):
            s = scale * q[q0:q0 + n, h].to(F64) @ k[:, h // (hq // hkv)].T
            s = s.masked_fill(~seen[:, used], -math.inf)
            z = torch.logsumexp(torch.cat([s, sink[h].to(F64).expand(n, 1)], 1), 1)
            p = torch.exp(s - torch.where(torch.isinf(z), 0.0, z)[:, None])
            vv = v[:, h // (hq // hkv)]
            out[q0:q0 + n, h] = p @ vv
            spread[q0:q0 + n, h] = p @ vv.abs()
            lse[h, q0:q0 + n] = z
    return out, lse, spread
