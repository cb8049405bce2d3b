"""Cases of the operators that read and keep less of a long paged key/value cache.

  shared   decode step of groups of sequences that share a prefix, whose keys are read once a group
  bounds   elementwise minimum and maximum of the keys of every page that new tokens went to
  select   the pages whose bounds promise the largest scores, for every sequence and kv head
  pages    decode step over the selected pages alone
  mass     the weight that every cached key received from the new tokens, accumulated
  evict    the keys with the least weight leave the cache, the others move together

``run`` computes the plain form with elementary torch operations, or, where ``own`` is true, calls
the framework.
"""
import math
import random

import torch

own = False

HEAD = 64


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # a few chats behind one system prompt: the smallest step
        dict(name="shared_chat", op="shared", batch=8, groups=1, prefix=1024, keys=200, heads_q=64, heads_kv=8,
             page=16),
        # samples of three long prompts, decoded together
        dict(name="shared_samples", op="shared", batch=192, groups=3, prefix=8192, keys=1024, heads_q=64, heads_kv=8,
             page=64),
        # the bounds after one decode step of 128 requests
        dict(name="bounds_decode", op="bounds", batch=128, new=1, cached=8192, heads_kv=8, page=16),
        # and after a wave of prompts, some of them on cached prefixes
        dict(name="bounds_prompts", op="bounds", batch=16, new=2047, cached=2000, heads_kv=8, page=16),
        # one request alone at a very long context: 4096 of its 131072 keys
        dict(name="select_single", op="select", batch=1, keys=131072, heads_q=64, heads_kv=8, page=16, count=256),
        # a batch of long conversations, an eighth of the pages
        dict(name="select_batch", op="select", batch=64, keys=16383, heads_q=64, heads_kv=8, page=16, count=128),
        # the attention of the two selections
        dict(name="pages_single", op="pages", batch=1, keys=131072, heads_q=64, heads_kv=8, page=16, count=256),
        dict(name="pages_batch", op="pages", batch=64, keys=16383, heads_q=64, heads_kv=8, page=16, count=128),
        # every decode step of a cache that evicts
        dict(name="mass_decode", op="mass", batch=32, new=1, keys=8192, heads_q=64, heads_kv=8, page=16),
        # the last tokens of four long prompts say what is kept of them
        dict(name="mass_prompt", op="mass", batch=4, new=512, keys=16384, heads_q=64, heads_kv=8, page=64),
        # those prompts cut down to an eighth
        dict(name="evict_prompt", op="evict", batch=4, keys=16384, budget=2048, heads_kv=8, page=64),
        # conversations that have grown past their budget by a few pages
        dict(name="evict_grown", op="evict", batch=64, keys=4351, budget=4096, heads_kv=8, page=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "bounds", "select", "pages", "mass", "evict"])
    heads_kv = rng.choice([1, 2, 4, 8])
    heads_q = heads_kv * rng.choice([1, 2, 4, 8])
    page = rng.choice([1, 8, 16, 16, 24, 64, 128])
    if op == "shared":
        groups = rng.choice([1, 1, 2, 3, 7])
        batch = _log(rng, groups, 192)
        most = 192 * (8192 + 1024) // batch                     # the largest listed case's keys
        prefix = _log(rng, 1, min(16384, most // 2))
        return dict(op=op, batch=batch, groups=groups, prefix=prefix, keys=_log(rng, 1, min(4096, most // 2)),
                    heads_q=heads_q, heads_kv=heads_kv, page=page)
    if op == "bounds":
        batch, new = _log(rng, 1, 128), _log(rng, 1, 2047)
        new = max(1, min(new, 16 * 2047 // batch))
        return dict(op=op, batch=batch, new=new, cached=_log(rng, 1, 16 * 4096 // batch), heads_kv=heads_kv, page=page)
    if op in ("select", "pages"):
        page = rng.choice([8, 16, 16, 32, 64])
        batch = _log(rng, 1, 64)
        most = 64 * 16384 // batch if batch > 8 else 131072
        keys = _log(rng, 64 * page if op == "select" else 1, most)          # at least 32 pages of each sequence
        return dict(op=op, batch=batch, keys=keys, heads_q=heads_q, heads_kv=heads_kv, page=page,
                    count=_log(rng, 4, 24 if keys < 512 * page else 256))
    if op == "mass":
        batch, new = _log(rng, 1, 32), _log(rng, 1, 512)
        most = 4 * 512 * 16384 * 64 // (batch * new * heads_q)   # the largest listed case's scores
        keys = _log(rng, new, max(new + 1, min(32768, most, 32 * 8192 // batch)))
        if batch * new * keys * heads_q > 4 * 512 * 16384 * 64:
            batch = max(1, 4 * 512 * 16384 * 64 // (new * keys * heads_q))
        return dict(op=op, batch=batch, new=new, keys=keys, heads_q=heads_q, heads_kv=heads_kv, page=page)
    batch = _log(rng, 1, 64)
    keys = _log(rng, 40, min(32768, 64 * 4351 // batch))
    return dict(op=op, batch=batch, keys=keys, budget=max(36, int(keys * rng.uniform(0.05, 1.0))), heads_kv=heads_kv,
                page=page)


# ----------------------------------------------------------------------------- lengths of a case
def _lengths(case):
    """(what comes first, the lengths) of every sequence: ragged, the same for every seed; the first
    sequence has the full sizes."""
    r = random.Random(1000003 * case["batch"] + 1009 * case["page"] + case.get("keys", case.get("cached", 0)))
    rest = range(case["batch"] - 1)
    if case["op"] == "bounds":
        new = [case["new"]] + [r.randint((case["new"] + 1) // 2, case["new"]) for _ in rest]
        cached = [case["cached"]] + [r.choice([0, r.randint(0, case["cached"])]) if case["new"] > 1 else
                                     r.randint(case["cached"] // 2, case["cached"]) for _ in rest]
        return cached, [c + n for c, n in zip(cached, new)]
    if case["op"] == "shared":
        # the groups' first sequences, and the prefix of every sequence: whole pages
        cut = sorted(r.sample(range(1, case["batch"]), min(case["groups"], case["batch"]) - 1))
        starts = [0] + cut + [case["batch"]]
        whole = case["prefix"] // case["page"] * case["page"]
        prefix = [whole] + [r.randint(whole // case["page"] // 2, whole // case["page"]) * case["page"]
                            for _ in starts[2:]]
        group = [p for p in range(len(prefix)) for _ in range(starts[p + 1] - starts[p])]
        lens = [prefix[p] + (case["keys"] if i == 0 else r.randint((case["keys"] + 1) // 2, case["keys"]))
                for i, p in enumerate(group)]
        return (starts, prefix), lens
    if case["op"] == "mass":
        new = [case["new"]] + [r.randint((case["new"] + 1) // 2, case["new"]) for _ in rest]
        return new, [case["keys"]] + [max(n, r.randint(case["keys"] // 2, case["keys"])) for n in new[1:]]
    return None, [case["keys"]] + [r.randint((case["keys"] + 1) // 2, case["keys"]) for _ in rest]


def _gen(seed, salt=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * int(seed) + salt)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(g, counts, spare=8):
    """Block table of sequences with so many pages each, at random places of the cache, one column
    more than the longest needs; and the pages of that cache."""
    pages = sum(counts) + spare
    perm = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    have = torch.tensor(counts, device="cuda")
    first = torch.cumsum(have, 0) - have
    col = torch.arange(max(counts) + 1, device="cuda")
    return torch.where(col[None] < have[:, None],
                       perm[(first[:, None] + col[None]).clamp(max=pages - 1)], -1).to(torch.int32), pages


def prepare(case, seed):
    g = _gen(seed)
    page, hkv = case["page"], case["heads_kv"]
    first, lens = _lengths(case)
    table, pages = _table(g, [-(-n // page) for n in lens])
    s = dict(case=case, table=table, pages=pages, lens=_ints(lens), scale=HEAD ** -0.5)
    if case["op"] == "shared":
        starts, prefix = first
        col = torch.arange(table.shape[1], device="cuda")
        shared = torch.tensor([prefix[p] // page for p in range(len(prefix)) for _ in range(starts[p + 1] - starts[p])],
                              device="cuda")
        head = torch.tensor([starts[p] for p in range(len(prefix)) for _ in range(starts[p + 1] - starts[p])],
                            device="cuda")
        s["table"] = torch.where(col[None] < shared[:, None], table[head], table).contiguous()
        s["groups"], s["prefix"] = _ints(starts), _ints(prefix)
    if case["op"] in ("shared", "bounds", "pages", "mass", "evict"):
        s["k_cache"] = _randn(g, pages, page, hkv, HEAD)
    if case["op"] in ("shared", "pages", "evict"):
        s["v_cache"] = _randn(g, pages, page, hkv, HEAD)
    if case["op"] in ("shared", "pages"):
        s["q"] = _randn(g, case["batch"], case["heads_q"], HEAD)
        s["sink"] = torch.randn(case["heads_q"], device="cuda", generator=g)
    if case["op"] == "bounds":
        s["cached"] = _ints(first)
        s["bounds"] = _randn(g, pages, hkv, 2, HEAD)
    if case["op"] == "select":
        # the spread of a page's keys around what they have in common
        middle = 0.7 * torch.randn(pages, hkv, 1, HEAD, device="cuda", generator=g)
        reach = 0.6 + 0.5 * torch.rand(pages, hkv, 2, HEAD, device="cuda", generator=g)
        sign = torch.tensor([-1.0, 1.0], device="cuda")[:, None]
        s["bounds"] = (middle + sign * reach * math.sqrt(2 * math.log(page + 1))).to(torch.bfloat16)
        s["q"] = _randn(g, case["batch"], case["heads_q"], HEAD)
    if case["op"] == "pages":
        have = torch.tensor([-(-n // page) for n in lens], device="cuda")
        rank = torch.rand(case["batch"], hkv, table.shape[1], device="cuda", generator=g)
        col = torch.arange(table.shape[1], device="cuda")
        rank = torch.where(col < have[:, None, None], rank, 2.0)
        rank[:, :, 0] = -1.0                                    # the first and the last page are always there
        rank.scatter_(2, (have - 1)[:, None, None].expand(-1, hkv, 1), -1.0)
        few = rank.argsort(2)[:, :, : case["count"]]
        few = torch.where(torch.arange(few.shape[2], device="cuda") < have[:, None, None], few, table.shape[1])
        few = few.sort(2).values
        sel = torch.full((case["batch"], hkv, case["count"]), -1, dtype=torch.int32, device="cuda")
        sel[:, :, : few.shape[2]] = torch.where(few < table.shape[1], few, -1).to(torch.int32)
        s["selected"] = sel
    if case["op"] == "mass":
        s["cu"] = torch.tensor([0] + first, device="cuda").cumsum(0).to(torch.int32)
        s["max_new"], s["max_keys"] = max(first), max(lens)
        s["q"] = _randn(g, sum(first), case["heads_q"], HEAD)
        sink = torch.randn(case["heads_q"], device="cuda", generator=g)
        s["lse"] = _lse(s, first, lens, sink)
        s["mass"] = torch.zeros(case["batch"], hkv, table.shape[1] * page, device="cuda")
        rand = torch.rand(s["mass"].shape, device="cuda", generator=g)
        key = torch.arange(s["mass"].shape[2], device="cuda")
        s["mass"] = torch.where(key < s["lens"][:, None, None], rand, 0.0)
    if case["op"] == "evict":
        # few keys have most of the weight
        s["mass"] = torch.exp(2 * torch.randn(case["batch"], hkv, table.shape[1] * page, device="cuda", generator=g))
    return s


def _lse(s, new, lens, sink):
    """What the attention of the new tokens left: lse [H_q, T], the sink included."""
    case, t0, got = s["case"], 0, []
    page, hkv = case["page"], case["heads_kv"]
    for b, (n, m) in enumerate(zip(new, lens)):
        rows = s["table"][b, : -(-m // page)].long()
        k = s["k_cache"][rows].view(-1, hkv, HEAD)[:m].float().permute(1, 2, 0)          # [hkv, 64, m]
        q = s["q"][t0 : t0 + n].float().view(n, hkv, -1, HEAD).permute(1, 2, 0, 3).reshape(hkv, -1, HEAD)
        a = (q @ k).mul_(s["scale"]).view(case["heads_q"], n, m)
        hidden = torch.arange(m, device="cuda")[None] > torch.arange(m - n, m, device="cuda")[:, None]
        a.masked_fill_(hidden, -math.inf)
        got.append(torch.logaddexp(torch.logsumexp(a, 2), sink[:, None]))
        t0 += n
    return torch.cat(got, 1).contiguous()


# ----------------------------------------------------------------------------- the plain forms
def _rows(s, j):
    """Cache rows [B, ...] of the keys j of every sequence (a missing page: page 0)."""
    page = s["case"]["page"]
    batch = torch.arange(s["lens"].numel(), device="cuda").view(-1, *[1] * (j.dim() - 1))
    return s["table"].long()[batch, j // page].clamp(min=0) * page + j % page


def _attend(q, k, v, seen, s):
    """q [B, hkv, G, 64], k and v [B, hkv, m, 64], seen [B, hkv or 1, m]: out [B, H_q, 64], lse [H_q, B]."""
    scores = (q @ k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~seen[:, :, None], -math.inf)
    sink = s["sink"].view(1, q.shape[1], q.shape[2], 1)
    top = torch.maximum(scores.amax(-1, keepdim=True), sink)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True) + torch.exp(sink - top)
    out = (weights @ v) / total
    lse = (top + total.log()).flatten(1).t()
    return dict(out=out.flatten(1, 2).to(torch.bfloat16), lse=lse.contiguous())


def _shared(s):
    case, hkv = s["case"], s["case"]["heads_kv"]
    j = torch.arange(s["table"].shape[1] * case["page"], device="cuda")[None]
    rows = _rows(s, j)
    k, v = (s[c].view(-1, hkv, HEAD)[rows].float().transpose(1, 2) for c in ("k_cache", "v_cache"))
    q = s["q"].float().view(case["batch"], hkv, -1, HEAD)
    return _attend(q, k, v, (j < s["lens"][:, None])[:, None], s)


def _bounds(s):
    case, page = s["case"], s["case"]["page"]
    col = torch.arange(s["table"].shape[1], device="cuda")[None]
    lens = s["lens"].long()[:, None]
    b, c = ((col >= s["cached"].long()[:, None] // page) & (col * page < lens)).nonzero(as_tuple=True)
    entry = s["table"][b, c].long()
    k = s["k_cache"][entry].float()                             # [pages, page, hkv, 64]
    gone = (c[:, None] * page + torch.arange(page, device="cuda") >= lens[b])[:, :, None, None]
    least = k.masked_fill(gone, math.inf).amin(1)
    most = k.masked_fill(gone, -math.inf).amax(1)
    s["bounds"][entry] = torch.stack([least, most], 2).to(torch.bfloat16)
    return dict(bounds=s["bounds"])


def _select(s):
    case, cols = s["case"], s["table"].shape[1]
    have = -(-s["lens"].long() // case["page"])[:, None, None]
    b = s["bounds"][s["table"].long().clamp(min=0)].double()    # values next to the border need 64 bits
    q = s["q"].double().view(case["batch"], case["heads_kv"], -1, HEAD)
    score = q.clamp(min=0) @ b[:, :, :, 1].permute(0, 2, 3, 1) + q.clamp(max=0) @ b[:, :, :, 0].permute(0, 2, 3, 1)
    score = score.amax(2)                                       # [B, hkv, cols]
    col = torch.arange(cols, device="cuda")
    score = torch.where((col == 0) | (col == have - 1), math.inf, score)
    score = torch.where(col < have, score, -math.inf)
    order = score.sort(dim=2, descending=True, stable=True).indices
    few = order[:, :, : case["count"]]
    few = torch.where(torch.arange(few.shape[2], device="cuda") < have, few, cols).sort(2).values
    sel = torch.full((*few.shape[:2], case["count"]), -1, dtype=torch.int32, device="cuda")
    sel[:, :, : few.shape[2]] = torch.where(few < cols, few, -1).to(torch.int32)
    return dict(selected=sel)


def _pages(s):
    case, page, hkv = s["case"], s["case"]["page"], s["case"]["heads_kv"]
    sel = s["selected"].long()
    j = (sel[..., None] * page + torch.arange(page, device="cuda")).flatten(2)          # [B, hkv, keys]
    seen = (j >= 0) & (j < s["lens"].long()[:, None, None])
    rows = _rows(s, j.clamp(min=0))
    head = torch.arange(hkv, device="cuda")[None, :, None]
    k, v = (s[c].view(-1, hkv, HEAD)[rows, head].float() for c in ("k_cache", "v_cache"))
    q = s["q"].float().view(case["batch"], hkv, -1, HEAD)
    return _attend(q, k, v, seen, s)


def _mass(s):
    case, cu, lens = s["case"], s["cu"].long(), s["lens"].long()
    hq, hkv, n, m = case["heads_q"], case["heads_kv"], s["max_new"], s["max_keys"]
    g, batch = hq // hkv, lens.numel()
    new = cu[1:] - cu[:-1]
    i, j = torch.arange(n, device="cuda"), torch.arange(m, device="cuda")
    k = s["k_cache"].view(-1, hkv, HEAD)[_rows(s, j[None])].float().permute(0, 2, 3, 1)
    t = (cu[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)                        # [B, n]
    q = s["q"][t].float().view(batch, n, hkv, g, HEAD).permute(0, 2, 3, 1, 4).reshape(batch, hkv, g * n, HEAD)
    lse = s["lse"][:, t].view(hkv, g, batch, n).permute(2, 0, 1, 3)
    weight = (q @ k).mul_(s["scale"]).view(batch, hkv, g, n, m).sub_(lse[..., None]).exp_()
    seen = (j[None] <= (i[None] + (lens - new)[:, None])[:, :, None]) & (i[None] < new[:, None])[:, :, None]
    weight *= seen[:, None, None]
    s["mass"][:, :, :m] += weight.sum((2, 3))
    return dict(mass=s["mass"])


KEEP_FIRST, KEEP_LAST = 4, 32


def _kept(score, lens, budget):
    """Which keys [B, hkv, C] stay, from the scores and the lengths."""
    j = torch.arange(score.shape[2], device="cuda")
    lens = lens.long()[:, None, None]
    score = torch.where((j < KEEP_FIRST) | (j >= lens - KEEP_LAST), math.inf, score)
    score = torch.where(j < lens, score, -math.inf)
    order = score.sort(dim=2, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, j.expand_as(order))
    return rank < lens.clamp(max=budget)


def _evict(s):
    case, page, hkv, budget = s["case"], s["case"]["page"], s["case"]["heads_kv"], s["case"]["budget"]
    mass, lens = s["mass"], s["lens"].long()
    kept = _kept(mass, lens, budget)
    fewer = lens.clamp(max=budget)
    j = torch.arange(mass.shape[2], device="cuda")
    below = j < fewer[:, None, None]
    # the n-th kept key behind the budget goes to the n-th hole below it
    behind = torch.where(kept & ~below, j, mass.shape[2]).sort(2).values
    hole = ~kept & below
    b, h, to = hole.nonzero(as_tuple=True)
    come = behind[b, h, hole.cumsum(2)[b, h, to] - 1]
    table = s["table"].long()
    src = table[b, come // page] * page + come % page
    dst = table[b, to // page] * page + to % page
    for c in ("k_cache", "v_cache"):
        rows = s[c].view(-1, hkv, HEAD)
        rows[dst, h] = rows[src, h]
    out = torch.where(below, mass, 0.0)
    out[b, h, to] = mass[b, h, come]
    col = torch.arange(table.shape[1], device="cuda")[None]
    free = (col >= -(-fewer // page)[:, None]) & (col < -(-lens // page)[:, None])
    place = torch.where(free.flatten(), free.flatten().cumsum(0) - 1, free.numel())
    freed = torch.full((free.numel() + 1,), -1, dtype=torch.int32, device="cuda")
    freed[place] = s["table"].flatten()
    freed[-1] = -1
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], mass=out, lens=fewer.int(), freed=freed[:-1],
                count=free.sum().int().reshape(1))


def _own(s):
    from attention_learnable_head_gb300 import binding
    case = s["case"]
    if case["op"] == "shared":
        out, lse = binding.decode_shared(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["groups"],
                                         s["prefix"], s["sink"], softmax_scale=s["scale"])
        return dict(out=out, lse=lse)
    if case["op"] == "bounds":
        binding.page_bounds(s["k_cache"], s["table"], s["cached"], s["lens"], s["bounds"])
        return dict(bounds=s["bounds"])
    if case["op"] == "select":
        return dict(selected=binding.select_pages(s["q"], s["bounds"], s["table"], s["lens"], count=case["count"],
                                                  page_size=case["page"], keep_first=1, keep_last=1))
    if case["op"] == "pages":
        out, lse = binding.decode_pages(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["selected"],
                                        s["sink"], softmax_scale=s["scale"])
        return dict(out=out, lse=lse)
    if case["op"] == "mass":
        return dict(mass=binding.key_mass(s["q"], s["k_cache"], s["table"], s["lens"], s["cu"], s["lse"], s["mass"],
                                          softmax_scale=s["scale"]))
    r = binding.evict(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["mass"], budget=case["budget"],
                      keep_first=KEEP_FIRST, keep_last=KEEP_LAST)
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], mass=r.mass, lens=r.seq_lens, freed=r.freed_pages,
                count=r.num_freed)


def run(state):
    if own:
        return _own(state)
    return dict(shared=_shared, bounds=_bounds, select=_select, pages=_pages, mass=_mass,
                evict=_evict)[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    first, lens = _lengths(case)
    page, hkv, batch = case["page"], case["heads_kv"], case["batch"]
    hq = case.get("heads_q", 0)
    row = HEAD * 2                                              # one key of one head
    ends = 2 * batch * hq * row + 4 * batch * hq                # q, out and lse of single tokens
    if case["op"] == "shared":
        starts, prefix = first
        keys = sum(lens) - sum(prefix[p] * (starts[p + 1] - starts[p] - 1) for p in range(len(prefix)))
        return dict(bytes=2 * keys * hkv * row + ends + 4 * -(-keys // page), flops=4 * HEAD * hq * sum(lens))
    if case["op"] == "bounds":
        keys = sum(n - c // page * page for c, n in zip(first, lens))
        some = sum(-(-n // page) - c // page for c, n in zip(first, lens))
        return dict(bytes=keys * hkv * row + some * (2 * hkv * row + 4), flops=0)
    if case["op"] == "select":
        some = sum(-(-n // page) for n in lens)
        return dict(bytes=some * (2 * hkv * row + 4) + batch * hq * row + 4 * batch * hkv * case["count"],
                    flops=4 * HEAD * hq * some)
    if case["op"] == "pages":
        keys = sum(n if -(-n // page) <= case["count"] else case["count"] * page - (-n % page) for n in lens)
        return dict(bytes=2 * keys * hkv * row + ends + 4 * batch * hkv * case["count"], flops=4 * HEAD * hq * keys)
    if case["op"] == "mass":
        keys, t = sum(lens), sum(first)
        pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(first, lens))
        return dict(bytes=keys * hkv * (row + 8) + t * hq * (row + 4) + 4 * -(-keys // page),
                    flops=2 * HEAD * hq * pairs)
    # the keys that are kept behind the budget, as many as it takes on average
    budget, moved = case["budget"], 0.0
    for n in lens:
        if n > budget:
            last = min(KEEP_LAST, n - budget)
            moved += last + (n - budget - last) * max(0, budget - KEEP_FIRST - KEEP_LAST) / (n - KEEP_FIRST - KEEP_LAST)
    space = (max(-(-n // page) for n in lens) + 1) * page
    return dict(bytes=hkv * (moved * 4 * row + 4 * sum(lens) + 4 * batch * space), flops=0)


# ----------------------------------------------------------------------------- the definitions in 64 bits
def _softmax_sink(q, k, v, sink, scale):
    """q [G, 64], k and v [m, 64] in 64 bits, sink [G]: out [G, 64] and lse [G]."""
    a = torch.cat([scale * (q @ k.t()), sink[:, None]], 1)
    lse = torch.logsumexp(a, 1)
    return torch.exp(a[:, :-1] - lse[:, None]) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    page, hkv = case["page"], case["heads_kv"]
    first, lens = _lengths(case)
    if case["op"] == "select":
        return None                                             # whole numbers: they have to be equal
    if case["op"] in ("shared", "pages"):
        g = case["heads_q"] // hkv
        outs, lses = [], []
        for b, n in enumerate(lens):
            used = s["table"][b, : -(-n // page)].long()
            kb = s["k_cache"][used].view(-1, hkv, HEAD)[:n]
            vb = s["v_cache"][used].view(-1, hkv, HEAD)[:n]
            for h in range(hkv):
                at = slice(None)
                if case["op"] == "pages":
                    mark = torch.zeros(used.numel() + 1, dtype=torch.bool, device="cuda")
                    mark[s["selected"][b, h].long()] = True     # -1: the last mark, of no page
                    at = mark[:-1].repeat_interleave(page)[:n]
                e = slice(h * g, (h + 1) * g)
                o, z = _softmax_sink(s["q"][b, e].double(), kb[at, h].double(), vb[at, h].double(),
                                     s["sink"][e].double(), s["scale"])
                outs.append(o)
                lses.append(z)
        out = torch.stack(outs).view(case["batch"], case["heads_q"], HEAD)
        return dict(out=out, lse=torch.stack(lses).view(case["batch"], case["heads_q"]).t().contiguous())
    if case["op"] == "bounds":
        want = s["bounds"].double()
        for b, (c, n) in enumerate(zip(first, lens)):
            cols = torch.arange(c // page, -(-n // page), device="cuda")
            entry = s["table"][b, cols].long()
            k = s["k_cache"][entry].double()
            if n % page:                                        # the last key stands for those that are not there
                k[-1, n % page :] = k[-1, n % page - 1].clone()
            want[entry, :, 0] = k.min(1).values
            want[entry, :, 1] = k.max(1).values
        return dict(bounds=want)
    if case["op"] == "mass":
        mass, g, t0 = s["mass"].double(), case["heads_q"] // hkv, 0
        for b, (n, m) in enumerate(zip(first, lens)):
            k = s["k_cache"][s["table"][b, : -(-m // page)].long()].view(-1, hkv, HEAD)[:m]
            pos = torch.arange(m - n, m, device="cuda")[:, None]
            key = torch.arange(m, device="cuda")[None]
            for e in range(case["heads_q"]):
                a = s["scale"] * (s["q"][t0 : t0 + n, e].double() @ k[:, e // g].double().t())
                w = torch.exp(a - s["lse"][e, t0 : t0 + n].double()[:, None])
                mass[b, e // g, :m] += w.masked_fill(key > pos, 0.0).sum(0)
            t0 += n
        return dict(mass=mass)
    # one sequence and head after the other, from the ranks of its keys
    k, v = s["k_cache"].double().view(-1, hkv, HEAD), s["v_cache"].double().view(-1, hkv, HEAD)
    out = torch.zeros(s["mass"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        keep = min(n, case["budget"])
        key = torch.arange(n, device="cuda")
        row = s["table"][b, key // page].long() * page + key % page
        for h in range(hkv):
            score = s["mass"][b, h, :n].double()
            score[:KEEP_FIRST] = math.inf
            score[max(0, n - KEEP_LAST) :] = math.inf
            stay = torch.sort(-score, stable=True).indices[:keep].sort().values
            mark = torch.zeros(n, dtype=torch.bool, device="cuda")
            mark[stay] = True
            to = (~mark[:keep]).nonzero().flatten()
            come = stay[keep - to.numel() :]
            k[row[to], h], v[row[to], h] = k[row[come], h], v[row[come], h]
            out[b, h, :keep] = s["mass"][b, h, :keep].double()
            out[b, h, to] = s["mass"][b, h, come].double()
    return dict(k_cache=k.view(s["k_cache"].shape), v_cache=v.view(s["v_cache"].shape), mass=out, lens=None,
                freed=None, count=None)
