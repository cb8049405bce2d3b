"""Float64 definitions of what reads and keeps less of a long paged cache, on the CPU:
attention over chosen keys, bounds of pages and the choice by them, the weight of keys
and their eviction.  Written from the formulas, one sequence and head at a time."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def cache_rows(table_row, keys, page: int, pages: int):
    """(rows of the cache, which of them there are) of these keys of a sequence."""
    keys = torch.as_tensor(keys, dtype=torch.long)
    if keys.numel() == 0:
        return keys, keys.bool()
    entry = table_row.long()[keys // page]
    ok = (entry >= 0) & (entry < pages)
    return torch.where(ok, entry, 0) * page + keys % page, ok


def oracle_attend(q, k_cache, v_cache, table, keys_of, sink, *, scale: float):
    """(out [B, H_q, d], lse [H_q, B], spread) of one new token a sequence over the
    keys keys_of(b, h) of each kv head; spread = sum_j P_j |v_j|."""
    b, hq, d = q.shape
    pages, page, hkv = k_cache.shape[:3]
    kf, vf = k_cache.reshape(-1, hkv, d), v_cache.reshape(-1, hkv, d)
    out, spread = torch.zeros(b, hq, d, dtype=F64), torch.zeros(b, hq, d, dtype=F64)
    lse = torch.zeros(hq, b, dtype=F64)
    for i in range(b):
        for e in range(hq):
            h = e // (hq // hkv)
            rows, ok = cache_rows(table[i], keys_of(i, h), page, pages)
            rows = rows[ok]
            s = scale * (kf[rows, h].to(F64) @ q[i, e].to(F64))
            z = torch.logsumexp(torch.cat([s, sink[e].to(F64).reshape(1)]), 0)
            p = torch.exp(s - z) if not torch.isinf(z) else torch.zeros_like(s)
            v = vf[rows, h].to(F64)
            out[i, e], spread[i, e], lse[e, i] = p @ v, p @ v.abs(), z
    return out, lse, spread


def oracle_bounds(k_cache, table, cached, lens, bounds):
    """bounds [pages, H_kv, 2, d] after the keys [cached, lens) were written."""
    pages, page = k_cache.shape[:2]
    want = bounds.clone()
    for b, (c, n) in enumerate(zip(cached, lens)):
        for col in range(c // page, -(-n // page) if n > c else 0):
            e = int(table[b, col])
            if 0 <= e < pages:
                k = k_cache[e, : min(page, n - col * page)]
                want[e, :, 0], want[e, :, 1] = k.amin(0), k.amax(0)
    return want


def page_scores(q, bounds, entries, group: int, h: int):
    """Scores [pages of the list] of one sequence's kv head; q [H_q, d]."""
    x = q[h * group:(h + 1) * group].to(F64)
    e = torch.as_tensor(entries, dtype=torch.long)
    ok = (e >= 0) & (e < bounds.shape[0])
    b = bounds[torch.where(ok, e, 0), h].to(F64)
    s = (x.clamp(min=0)[:, None] * b[None, :, 1] + x.clamp(max=0)[:, None] * b[None, :, 0]).sum(-1)
    s = s.nan_to_num(nan=math.inf, posinf=math.inf, neginf=-math.inf) if s.isnan().any() else s
    return torch.where(ok, s.amax(0), -math.inf)


def oracle_select(q, bounds, table, lens, *, page: int, count: int, first: int, last: int):
    """selected [B, H_kv, count] int32."""
    hkv = bounds.shape[1]
    group = q.shape[1] // hkv
    sel = torch.full((len(lens), hkv, count), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        have = -(-n // page)
        for h in range(hkv):
            if have <= count:
                take = list(range(have))
            else:
                s = page_scores(q[b], bounds, table[b, :have], group, h).tolist()
                middle = sorted(range(first, have - last), key=lambda c: (-s[c], c))
                take = sorted([*range(first), *range(have - last, have),
                               *middle[:count - first - last]])
            sel[b, h, :len(take)] = torch.tensor(take, dtype=torch.int32)
    return sel


def oracle_mass(q, k_cache, table, lens, cu, lse, mass, *, scale: float):
    """mass [B, H_kv, C] in float64 with the new tokens' weights added."""
    pages, page, hkv, d = k_cache.shape
    group = q.shape[1] // hkv
    got = mass.to(F64).clone()
    kf = k_cache.reshape(-1, hkv, d)
    for b, n in enumerate(lens):
        t0, new = int(cu[b]), int(cu[b + 1]) - int(cu[b])
        rows, ok = cache_rows(table[b], range(n), page, pages)
        m = min(n, got.shape[2])
        pos = torch.arange(n - new, n)[:, None]
        seen = (torch.arange(n)[None] <= pos) & ok[None]
        for e in range(q.shape[1]):
            s = scale * (q[t0:t0 + new, e].to(F64) @ kf[rows, e // group].to(F64).T)
            z = lse[e, t0:t0 + new].to(F64)[:, None]
            w = torch.where(seen & ~torch.isinf(z), torch.exp(s - z), 0.0)
            got[b, e // group, :m] += w.sum(0)[:m]
    return got


def oracle_evict(k_cache, v_cache, table, lens, mass, *, budget: int, first: int, last: int):
    """(k_cache, v_cache, mass, lens, freed pages) after the eviction."""
    pages, page, hkv, d = k_cache.shape
    k, v = k_cache.clone(), v_cache.clone()
    kf, vf = k.view(-1, hkv, d), v.view(-1, hkv, d)
    out, fewer, freed = torch.zeros_like(mass), [], []
    for b, n in enumerate(lens):
        keep = min(n, budget)
        fewer.append(keep)
        freed += [int(x) for x in table[b, -(-keep // page):-(-n // page)] if 0 <= x < pages]
        for h in range(hkv):
            if n <= budget:
                out[b, h, :n] = mass[b, h, :n]
                continue
            w = [math.inf if math.isnan(x) else x for x in mass[b, h, :n].tolist()]
            nan = [math.isnan(x) for x in mass[b, h, :n].tolist()]
            middle = sorted(range(first, n - last), key=lambda j: (not nan[j], -w[j], j))
            kept = {*range(first), *range(n - last, n), *middle[:budget - first - last]}
            holes = [j for j in range(keep) if j not in kept]
            come = sorted(j for j in kept if j >= keep)
            assert len(holes) == len(come)
            out[b, h, :keep] = mass[b, h, :keep]
            for to, src in zip(holes, come):
                out[b, h, to] = mass[b, h, src]
                (a, c), ok = cache_rows(table[b], [src, to], page, pages)
                if bool(ok.all()):
                    kf[c, h], vf[c, h] = k_cache.view(-1, hkv, d)[a, h], v_cache.view(-1, hkv, d)[a, h]
    return k, v, out, fewer, freed
