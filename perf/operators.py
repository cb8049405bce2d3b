"""Cases of the operators around the paged key/value cache and the head rotation.

  page_plan   block tables, slot map and positions of a serving step, from request lengths
  rope        per-head RMS norm and rotary positions of q and k (several position axes), with v
              passed through; in serving k and v go straight into the pages of the cache
  rope_bwd    its gradient: the packed projection's and the two norm weights'
  extend      attention of several new tokens per sequence over a paged cache, with the sink

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
        # one decode step of a serving batch of 128 requests: the smallest plan
        dict(name="plan_decode", op="plan", batch=128, new=1, cached=8192, page=16),
        # admission of a wave of 1024 short prompts, some of them on cached prefixes
        dict(name="plan_prompts", op="plan", batch=1024, new=128, cached=512, page=16),
        # decode step of 128 sequences: q rotated, k and v written into the paged cache
        dict(name="rope_decode", op="rope", tokens=128, heads_q=64, heads_kv=8, rotary=64, norm=True,
             axes=1, interleaved=False, far=131072, page=16),
        # images and video: three position axes, pairs side by side, an odd number of tokens
        dict(name="rope_axes", op="rope", tokens=4099, heads_q=16, heads_kv=2, rotary=64, norm=True,
             axes=3, interleaved=True, far=1024, page=0),
        # training on the long batch: 4 sequences of 16384 tokens
        dict(name="rope_train", op="rope", tokens=65536, heads_q=64, heads_kv=8, rotary=64, norm=True,
             axes=1, interleaved=False, far=16384, page=0),
        # the smallest training step: 128 tokens, two heads
        dict(name="rope_bwd_tiny", op="rope_bwd", tokens=128, heads_q=2, heads_kv=2, rotary=64, norm=True,
             axes=1, interleaved=False, far=128, fp32=False),
        # one 4096-token layer without norms, rotating half of each head, fp32 gradients coming in
        dict(name="rope_bwd_layer", op="rope_bwd", tokens=4096, heads_q=64, heads_kv=8, rotary=32,
             norm=False, axes=1, interleaved=False, far=4096, fp32=True),
        # the backward of rope_train
        dict(name="rope_bwd_train", op="rope_bwd", tokens=65536, heads_q=64, heads_kv=8, rotary=64,
             norm=True, axes=1, interleaved=False, far=16384, fp32=False),
        # drafted tokens verified against 32 long conversations
        dict(name="extend_verify", op="extend", batch=32, new=5, keys=8192, heads_q=64, heads_kv=8,
             window=0, page=16),
        # one request alone at a very long context, a handful of new tokens
        dict(name="extend_single", op="extend", batch=1, new=17, keys=131072, heads_q=64, heads_kv=8,
             window=0, page=64),
        # the next chunk of four prompts, up to 16384 keys each with the cached ones
        dict(name="extend_chunk", op="extend", batch=4, new=1024, keys=16384, heads_q=64, heads_kv=8,
             window=0, page=128),
        # the same step in a sliding-window layer
        dict(name="extend_window", op="extend", batch=8, new=513, keys=8192, heads_q=64, heads_kv=8,
             window=128, page=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope_bwd", "extend", "extend"])
    if op == "plan":
        return dict(op=op, batch=_log(rng, 1, 1024), new=_log(rng, 1, 128), cached=_log(rng, 1, 8192),
                    page=rng.choice([1, 16, 24, 64, 128]))
    heads_kv = rng.choice([1, 2, 4, 8])
    heads_q = heads_kv * rng.choice([1, 2, 4, 5, 8])
    if op in ("rope", "rope_bwd"):
        axes = rng.choice([1, 1, 2, 3])
        case = dict(op=op, tokens=_log(rng, 1, 65536), heads_q=heads_q, heads_kv=heads_kv,
                    rotary=rng.choice([16, 32, 48, 64, 64]), norm=rng.random() < 0.7, axes=axes,
                    interleaved=rng.random() < 0.5, far=_log(rng, 64, 1000000))
        if op == "rope":
            case["page"] = rng.choice([0, 0, 1, 16, 24, 128])
        else:
            case["fp32"] = rng.random() < 0.5
        return case
    batch, new = _log(rng, 1, 48), _log(rng, 1, 1024)
    most = 4 * 1024 * 64 * 16384 // (batch * new * heads_q)   # the largest listed case's scores
    keys = _log(rng, new, max(new + 1, min(32768, most)))
    if batch * new * keys * heads_q > 4 * 1024 * 64 * 16384:
        batch = max(1, 4 * 1024 * 64 * 16384 // (new * keys * heads_q))
    return dict(op=op, batch=batch, new=new, keys=keys, heads_q=heads_q, heads_kv=heads_kv,
                window=rng.choice([0, 0, 0, 1, 100, 128, 1000]), page=rng.choice([1, 8, 16, 24, 64, 128]))


# ----------------------------------------------------------------------------- lengths of a case
def _lengths(case):
    """(new tokens, keys or cached tokens) of every sequence: ragged, the same for every seed; the
    first sequence has the full sizes."""
    r = random.Random(1000003 * case["batch"] + 1009 * case["new"] + case.get("keys", case.get("cached", 0)))
    new = [case["new"]] + [r.randint((case["new"] + 1) // 2, case["new"]) for _ in range(case["batch"] - 1)]
    if case["op"] == "plan":
        rest = [case["cached"]] + [r.choice([0, r.randint(0, case["cached"])]) if case["new"] > 1 else
                                   r.randint(case["cached"] // 2, case["cached"]) for _ in range(case["batch"] - 1)]
    else:
        rest = [case["keys"]] + [max(n, r.randint(case["keys"] // 2, case["keys"])) for n in new[1:]]
    return new, rest


def _gen(seed, salt=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 * int(seed) + salt)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


def _pair_axis(case):
    """The position axis of each rotated pair: whole sections of the pairs, the first the largest."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    small = pairs // (axes + 1) if axes > 1 else 0
    return [0] * (pairs - (axes - 1) * small) + [a for a in range(1, axes) for _ in range(small)]


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "plan":
        new, cached = _lengths(case)
        page = case["page"]
        cols = max(-(-(n + c) // page) for n, c in zip(new, cached)) + 1
        held = sum(-(-c // page) for c in cached)
        need = sum(-(-(n + c) // page) + (-c // page) for n, c in zip(new, cached))
        pages = held + need + 64
        perm = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        have = torch.tensor([-(-c // page) for c in cached], device="cuda")
        first = torch.cumsum(have, 0) - have
        col = torch.arange(cols, device="cuda")
        table = torch.where(col[None] < have[:, None],
                            perm[(first[:, None] + col[None]).clamp(max=pages - 1)], -1).to(torch.int32)
        return dict(case=case, cached=torch.tensor(cached, dtype=torch.int32, device="cuda"),
                    new=torch.tensor(new, dtype=torch.int32, device="cuda"), free=perm[held:].contiguous(),
                    table=table, pages=pages, tokens=-(-sum(new) // 64) * 64)
    if case["op"] in ("rope", "rope_bwd"):
        t, hq, hkv, pairs = case["tokens"], case["heads_q"], case["heads_kv"], case["rotary"] // 2
        s = dict(case=case, pair_axis=_pair_axis(case), eps=1e-6)
        s["qkv"] = _randn(g, t, hq + 2 * hkv, HEAD)
        start = torch.randint(0, max(1, case["far"] - t + 1), (case["axes"], 1), device="cuda", generator=g)
        step = torch.arange(t, device="cuda")[None] if case["axes"] == 1 else torch.randint(
            0, min(t, 64), (case["axes"], t), device="cuda", generator=g)
        s["positions"] = (start + step).to(torch.int32).contiguous()
        s["inv_freq"] = (150000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))).float().cuda()
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = 1 + 0.1 * torch.randn(HEAD, device="cuda", generator=g)
            s["k_weight"] = 1 + 0.1 * torch.randn(HEAD, device="cuda", generator=g)
        s["amplitude"] = 1.0 if case["norm"] else 1.34657359
        if case["op"] == "rope_bwd":
            kind = torch.float32 if case["fp32"] else torch.bfloat16
            s["dq"], s["dk"], s["dv"] = (_randn(g, t, h, HEAD).to(kind) for h in (hq, hkv, hkv))
        elif case["page"]:
            page = case["page"]
            pages = -(-t // page) + 8
            s["k_cache"], s["v_cache"] = _randn(g, pages, page, hkv, HEAD), _randn(g, pages, page, hkv, HEAD)
            s["slots"] = torch.randperm(pages * page, device="cuda", generator=g)[:t].contiguous()
        return s
    new, keys = _lengths(case)
    page, hkv = case["page"], case["heads_kv"]
    count = [-(-k // page) for k in keys]
    cols, pages = max(count), sum(count) + 8
    perm = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    have = torch.tensor(count, device="cuda")
    first = torch.cumsum(have, 0) - have
    col = torch.arange(cols, device="cuda")
    table = torch.where(col[None] < have[:, None],
                        perm[(first[:, None] + col[None]).clamp(max=pages - 1)], -1).to(torch.int32)
    cu = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    return dict(case=case, q=_randn(g, sum(new), case["heads_q"], HEAD), k_cache=_randn(g, pages, page, hkv, HEAD),
                v_cache=_randn(g, pages, page, hkv, HEAD), table=table, cu=cu, max_new=max(new), max_keys=max(keys),
                keys=torch.tensor(keys, dtype=torch.int32, device="cuda"),
                sink=torch.randn(case["heads_q"], device="cuda", generator=g), scale=HEAD ** -0.5)


# ----------------------------------------------------------------------------- the plain forms
def _plan(s):
    page, table, free = s["case"]["page"], s["table"], s["free"].long()
    cached, new = s["cached"].long(), s["new"].long()
    have = (cached + page - 1) // page
    need = (cached + new + page - 1) // page - have
    base = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device="cuda")[None]
    fresh = free[(base[:, None] + col - have[:, None]).clamp(0, free.numel() - 1)]
    table.copy_(torch.where((col >= have[:, None]) & (col < (have + need)[:, None]), fresh, table.long()))
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=new.numel() - 1)
    inside = t < cu[-1]
    pos = cached[b] + t - cu[b]
    row = table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    return dict(table=table, slots=torch.where(inside, row, -1), positions=torch.where(inside, pos, 0).int(),
                cu=cu.int(), lens=(cached + new).int(), needed=need.sum().int().reshape(1))


def _angles(s):
    """cos and sin [T, 1, pairs] of every token's angles, times the amplitude: the angles of far
    positions need 64 bits."""
    axis = torch.tensor(s["pair_axis"], device="cuda")
    angle = s["positions"].double()[axis].t() * s["inv_freq"].double()[None]
    return ((torch.cos(angle) * s["amplitude"]).float()[:, None], (torch.sin(angle) * s["amplitude"]).float()[:, None])


def _split(x, case):
    """The first and the second numbers of the rotated pairs, and the dimensions that are not rotated."""
    r = case["rotary"]
    if case["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., : r // 2], x[..., r // 2 : r], x[..., r:]


def _join(a, b, rest, case):
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1), rest], -1)


def _rotate(x, cos, sin, case):
    a, b, rest = _split(x, case)
    return _join(a * cos - b * sin, b * cos + a * sin, rest, case)


def _norm_rotate(x, weight, cos, sin, s):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight
    return _rotate(x, cos, sin, s["case"]).to(torch.bfloat16)


def _rope(s):
    case = s["case"]
    q, k, v = s["qkv"].split([case["heads_q"], case["heads_kv"], case["heads_kv"]], 1)
    cos, sin = _angles(s)
    q, k = _norm_rotate(q, s["q_weight"], cos, sin, s), _norm_rotate(k, s["k_weight"], cos, sin, s)
    if not case["page"]:
        return dict(q=q, k=k, v=v.contiguous())
    s["k_cache"].view(-1, case["heads_kv"], HEAD)[s["slots"]] = k
    s["v_cache"].view(-1, case["heads_kv"], HEAD)[s["slots"]] = v
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _norm_rotate_bwd(x, dy, weight, cos, sin, s):
    dy = _rotate(dy.float(), cos, -sin, s["case"])
    if weight is None:
        return dy, None
    x = x.float()
    inv = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
    unit = x * inv
    dunit = dy * weight
    return inv * (dunit - unit * (dunit * unit).mean(-1, keepdim=True)), (dy * unit).sum((0, 1))


def _rope_bwd(s):
    case = s["case"]
    q, k, _ = s["qkv"].split([case["heads_q"], case["heads_kv"], case["heads_kv"]], 1)
    cos, sin = _angles(s)
    dq, dwq = _norm_rotate_bwd(q, s["dq"], s["q_weight"], cos, sin, s)
    dk, dwk = _norm_rotate_bwd(k, s["dk"], s["k_weight"], cos, sin, s)
    return dict(dqkv=torch.cat([dq, dk, s["dv"].float()], 1).to(torch.bfloat16), dq_weight=dwq, dk_weight=dwk)


def _extend(s):
    case, cu, lens = s["case"], s["cu"].long(), s["keys"].long()
    hq, hkv, page = case["heads_q"], case["heads_kv"], case["page"]
    g, n, m = hq // hkv, s["max_new"], s["max_keys"]
    new, batch = cu[1:] - cu[:-1], lens.numel()
    i, j = torch.arange(n, device="cuda"), torch.arange(m, device="cuda")
    rows = s["table"].long()[:, j // page].clamp(min=0) * page + j % page
    k = s["k_cache"].view(-1, hkv, HEAD)[rows].float().permute(0, 2, 3, 1)
    q = s["q"][(cu[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.view(batch, n, hkv, g, HEAD).permute(0, 2, 3, 1, 4).reshape(batch, hkv, g * n, HEAD)
    scores = (q @ k).mul_(s["scale"]).view(batch, hkv, g, n, m)
    at = (i[None] + (lens - new)[:, None])[:, :, None]          # the key position of each new token
    seen = (j <= at) & (j < lens[:, None, None])
    if case["window"]:
        seen &= j > at - case["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    sink = s["sink"].view(1, hkv, g, 1, 1)
    top = torch.maximum(scores.amax(-1, keepdim=True), sink)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True) + torch.exp(sink - top)
    v = s["v_cache"].view(-1, hkv, HEAD)[rows].float().permute(0, 2, 1, 3)
    out = (weights.view(batch, hkv, g * n, m) @ v).view(batch, hkv, g, n, HEAD) / total
    lse = (top + total.log()).squeeze(-1)
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    r = t - cu[b]
    return dict(out=out.permute(0, 3, 1, 2, 4).reshape(batch, n, hq, HEAD)[b, r].to(torch.bfloat16),
                lse=lse.permute(1, 2, 0, 3).reshape(hq, batch, n)[:, b, r].contiguous())


def _own(s):
    from attention_learnable_head_gb300 import binding
    case = s["case"]
    if case["op"] == "plan":
        p = binding.page_plan(s["cached"], s["new"], s["free"], s["table"], page_size=case["page"],
                              num_pages=s["pages"], max_tokens=s["tokens"])
        return dict(table=s["table"], slots=p.slots, positions=p.positions, cu=p.cu_seqlens_q, lens=p.seq_lens,
                    needed=p.pages_needed)
    if case["op"] == "extend":
        out, lse = binding.extend(s["q"], s["k_cache"], s["v_cache"], s["table"], s["keys"], s["cu"], s["sink"],
                                  window=case["window"], softmax_scale=s["scale"])
        return dict(out=out, lse=lse)
    kw = dict(heads_q=case["heads_q"], heads_kv=case["heads_kv"], q_weight=s["q_weight"], k_weight=s["k_weight"],
              eps=s["eps"], pair_axis=s["pair_axis"], interleaved=case["interleaved"], amplitude=s["amplitude"])
    if case["op"] == "rope_bwd":
        dqkv, dwq, dwk = binding.qkv_rope_backward(s["qkv"], s["positions"], s["inv_freq"], s["dq"], s["dk"],
                                                   s["dv"], **kw)
        return dict(dqkv=dqkv, dq_weight=dwq, dk_weight=dwk)
    if case["page"]:
        q, _, _ = binding.qkv_rope(s["qkv"], s["positions"], s["inv_freq"], slots=s["slots"], k_cache=s["k_cache"],
                                   v_cache=s["v_cache"], **kw)
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    q, k, v = binding.qkv_rope(s["qkv"], s["positions"], s["inv_freq"], **kw)
    return dict(q=q, k=k, v=v)


def run(state):
    if own:
        return _own(state)
    return dict(plan=_plan, rope=_rope, rope_bwd=_rope_bwd, extend=_extend)[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "plan":
        new, cached = _lengths(case)
        page, b = case["page"], case["batch"]
        need = sum(-(-(n + c) // page) + (-c // page) for n, c in zip(new, cached))
        half = sum(1 for c in cached if c % page)               # pages that are filled up first
        tokens = -(-sum(new) // 64) * 64
        return dict(bytes=8 * b + 8 * need + 4 * half + 12 * tokens + 4 * (2 * b + 2), flops=0)
    if case["op"] in ("rope", "rope_bwd"):
        t, hq, hkv, r = case["tokens"], case["heads_q"], case["heads_kv"], case["rotary"]
        x = t * HEAD * 2                                        # one head of every token in bf16
        extra = t * 4 * case["axes"] + 2 * r + (2 * HEAD * 4 if case["norm"] else 0)
        per = 3 * (r / HEAD) + (4 if case["norm"] else 0)
        if case["op"] == "rope":
            slots = 8 * t if case["page"] else 0
            return dict(bytes=2 * x * (hq + 2 * hkv) + extra + slots, flops=per * t * HEAD * (hq + hkv))
        come = x * (hq + 2 * hkv) * (2 if case["fp32"] else 1)
        saved = x * (hq + hkv) if case["norm"] else 0           # without norms the inputs are not needed
        grads = 2 * HEAD * 4 if case["norm"] else 0
        return dict(bytes=come + saved + x * (hq + 2 * hkv) + extra + grads, flops=2.5 * per * t * HEAD * (hq + hkv))
    new, keys = _lengths(case)
    hq, hkv, w = case["heads_q"], case["heads_kv"], case["window"]
    pairs = read = 0
    for n, m in zip(new, keys):
        span = m if not w else min(m, n + w - 1)                # keys that some new token sees
        read += span
        if not w:
            pairs += n * m - n * (n - 1) // 2
        else:
            pairs += sum(min(w, m - n + i + 1) for i in range(n))
    t = sum(new)
    table = 4 * sum(-(-m // case["page"]) for m in keys)
    return dict(bytes=2 * read * hkv * HEAD * 2 + 2 * t * hq * HEAD * 2 + 4 * t * hq + table, flops=4 * HEAD * hq * pairs)


# ----------------------------------------------------------------------------- the definitions in 64 bits
def _turned(x, weight, s):
    """The norm and the rotation of x [T, heads, 64] in 64 bits, pair by pair from the definition
    (the pair as a complex number, times amplitude * e^(i angle))."""
    case = s["case"]
    y = x
    if weight is not None:
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / HEAD + s["eps"]) * weight
    pairs = case["rotary"] // 2
    one = torch.arange(pairs, device="cuda") * (2 if case["interleaved"] else 1)
    two = one + (1 if case["interleaved"] else pairs)
    axis = torch.tensor(s["pair_axis"], device="cuda")
    angle = s["inv_freq"].double() * s["positions"].double().index_select(0, axis).transpose(0, 1)
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), angle).unsqueeze(1)
    z = torch.complex(y.index_select(-1, one), y.index_select(-1, two)) * turn
    out = y.clone()
    out = out.index_copy(-1, one, z.real).index_copy(-1, two, z.imag)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                                             # whole numbers: they have to be equal
    if case["op"] == "extend":
        hq, hkv, page, w = case["heads_q"], case["heads_kv"], case["page"], case["window"]
        new, keys = _lengths(case)
        g, t0, outs, lses = hq // hkv, 0, [], []
        for b, (n, m) in enumerate(zip(new, keys)):
            used = s["table"][b, : -(-m // page)].long()
            out = torch.empty(n, hq, HEAD, dtype=torch.float64, device="cuda")
            lse = torch.empty(hq, n, dtype=torch.float64, device="cuda")
            pos = torch.arange(m - n, m, device="cuda")[:, None]
            key = torch.arange(m, device="cuda")[None]
            hidden = key > pos
            if w:
                hidden = hidden | (key <= pos - w)
            for h in range(hkv):
                k = s["k_cache"][used, :, h].reshape(-1, HEAD)[:m].double()
                v = s["v_cache"][used, :, h].reshape(-1, HEAD)[:m].double()
                for e in range(h * g, (h + 1) * g):
                    a = torch.addmm(k.new_zeros(1, 1), s["q"][t0 : t0 + n, e].double(), k.t(), alpha=s["scale"], beta=0)
                    a = torch.cat([a.masked_fill(hidden, -math.inf), s["sink"][e].double().expand(n, 1)], 1)
                    lse[e] = torch.logsumexp(a, 1)
                    out[:, e] = torch.exp(a - lse[e][:, None])[:, :m] @ v
            outs.append(out)
            lses.append(lse)
            t0 += n
        return dict(out=torch.cat(outs), lse=torch.cat(lses, 1))
    hq, hkv = case["heads_q"], case["heads_kv"]
    x = s["qkv"].double()
    if case["op"] == "rope":
        q = _turned(x[:, :hq], None if s["q_weight"] is None else s["q_weight"].double(), s)
        k = _turned(x[:, hq : hq + hkv], None if s["k_weight"] is None else s["k_weight"].double(), s)
        v = x[:, hq + hkv :]
        if not case["page"]:
            return dict(q=q, k=k, v=v)
        caches = [c.double().view(-1, hkv, HEAD) for c in (s["k_cache"], s["v_cache"])]
        for c, rows in zip(caches, (k, v)):
            c.index_copy_(0, s["slots"], rows)
        return dict(q=q, k_cache=caches[0].view(s["k_cache"].shape), v_cache=caches[1].view(s["v_cache"].shape))
    # the gradient by automatic differentiation of the definition, some tokens at a time
    wq = wk = None
    dwq = dwk = None
    if case["norm"]:
        wq, wk = s["q_weight"].double().requires_grad_(), s["k_weight"].double().requires_grad_()
        dwq, dwk = torch.zeros_like(wq), torch.zeros_like(wk)
    dqkv = torch.empty_like(x)
    every = s["positions"]
    for t in range(0, case["tokens"], 8192):
        part = slice(t, t + 8192)
        a, b = x[part, :hq].clone().requires_grad_(), x[part, hq : hq + hkv].clone().requires_grad_()
        p = dict(s, positions=every[:, part])
        y, z = _turned(a, wq, p), _turned(b, wk, p)
        leaves = [a, b] + ([wq, wk] if case["norm"] else [])
        got = torch.autograd.grad([y, z], leaves, [s["dq"][part].double(), s["dk"][part].double()])
        dqkv[part, :hq], dqkv[part, hq : hq + hkv] = got[0], got[1]
        dqkv[part, hq + hkv :] = s["dv"][part].double()
        if case["norm"]:
            dwq += got[2].detach()
            dwk += got[3].detach()
    return dict(dqkv=dqkv, dq_weight=dwq, dk_weight=dwk)
