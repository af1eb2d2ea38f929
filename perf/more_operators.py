"""What a serving step does between its matrix products: the cases that these operators are timed on.

Four groups of calls, in the order of a step.  "plan": from the sequences' lengths, the pages that each one holds and a
stack of free pages, the step's rows, slots and positions, with pages taken and given back (`ft_kv_plan`).  "rotate":
the norm of each query's and key's head, the rotation by position, and the keys and values quantised into the cache
(`ft_kv_append_rotated`), which are then read back.  "route": router logits to expert ids and weights (`ft_moe_route`).
"logprobs": the log probability of a given token, the entropy and the most likely tokens of each row of logits
(`ft_logprobs`).

The plain forms below are elementary torch operations; what decides an order or a rounding of stored values is in 64
bits, the rest in 32.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LARGEST = torch.finfo(torch.float32).max


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the next token of 16 streams: one new slot each, now and then a page
        {"name": "plan step", "op": "plan", "kind": "step", "s": 16, "q": 1, "ctx": 8192, "page": 64},
        # a server's mixed step: sequences that end, wait, go on by a token or by a chunk of their prompt
        {"name": "plan mix", "op": "plan", "kind": "mix", "s": 200, "q": 300, "ctx": 4000, "page": 16},
        # one layer's projections of a single token, heads of 256 of which the first quarter turns
        {"name": "rotate step", "op": "rotate", "fmt": "nvfp4", "n": 1, "hq": 16, "hkv": 2, "d": 256, "rope": 64, "inter": 0, "norm": 1,
         "page": 64, "places": 32768, "skip": 0},
        # the prefill workload's 8192 tokens
        {"name": "rotate chunk", "op": "rotate", "fmt": "nvfp4", "n": 8192, "hq": 32, "hkv": 8, "d": 128, "rope": 128, "inter": 0, "norm": 1,
         "page": 64, "places": 16384, "skip": 0},
        # an odd number of tokens with padding among them, pairs of neighbours, no norms, 8-bit cache
        {"name": "rotate odd", "op": "rotate", "fmt": "fp8", "n": 3001, "hq": 20, "hkv": 4, "d": 64, "rope": 32, "inter": 1, "norm": 0,
         "page": 16, "places": 100003, "skip": 7},
        # the decode workload's router: one token, 8 of 256 experts
        {"name": "route one", "op": "route", "t": 1, "e": 256, "k": 8, "score": "softmax", "bias": 0, "groups": 1, "keep": 1, "best": 1,
         "renorm": 1, "fp32": 0},
        # a decode batch whose router has sigmoid scores, a bias that balances the experts, and groups of them
        {"name": "route batch", "op": "route", "t": 16, "e": 256, "k": 6, "score": "sigmoid", "bias": 1, "groups": 8, "keep": 4, "best": 2,
         "renorm": 1, "fp32": 1},
        # the prefill workload's router
        {"name": "route chunk", "op": "route", "t": 8192, "e": 256, "k": 8, "score": "softmax", "bias": 0, "groups": 1, "keep": 1, "best": 1,
         "renorm": 1, "fp32": 0},
        # a prompt of odd length, experts that are no power of two, balanced
        {"name": "route odd", "op": "route", "t": 5003, "e": 160, "k": 6, "score": "softmax", "bias": 1, "groups": 8, "keep": 3, "best": 1,
         "renorm": 0, "fp32": 0},
        # the answer of one stream
        {"name": "logprobs one", "op": "logprobs", "n": 1, "v": 131072, "k": 8, "fp32": 0, "cool": 1.0},
        # a tree of 48 drafted tokens, rows of an odd number of fp32 logits
        {"name": "logprobs tree", "op": "logprobs", "n": 48, "v": 100003, "k": 20, "fp32": 1, "cool": 0.7},
        # the tokens of a prompt's chunk, scored
        {"name": "logprobs chunk", "op": "logprobs", "n": 2048, "v": 131072, "k": 5, "fp32": 0, "cool": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("plan", "rotate", "route", "logprobs"))
    if op == "plan":
        kind = rng.choice(("step", "tree", "mix"))
        s = _log(rng, 1, 1024)
        q = {"step": 1, "tree": rng.randint(2, 64), "mix": _log(rng, 2, 8192)}[kind]
        q = max(1, min(q, 65536 // s))
        return {"op": op, "kind": kind, "s": s, "q": q, "ctx": _log(rng, 1, min(131072, 2 ** 21 // s)), "page": rng.choice((16, 32, 64, 128, 256))}
    if op == "rotate":
        d, hkv = rng.choice((64, 128, 256)), rng.choice((1, 2, 4, 8))
        hq = hkv * rng.choice((1, 2, 4, 5, 8))
        return {"op": op, "fmt": rng.choice(("nvfp4", "fp8")), "n": _log(rng, 1, min(8192, 8192 * 48 * 128 // ((hq + 2 * hkv) * d))), "hq": hq,
                "hkv": hkv, "d": d, "rope": rng.choice([r for r in (32, 64, 96, 128, 256) if r <= d]), "inter": rng.randint(0, 1),
                "norm": rng.randint(0, 1), "page": rng.choice((16, 64, 256)), "places": _log(rng, 1000, 131072), "skip": rng.choice((0, 0, 5))}
    if op == "route":
        e = rng.choice((8, 16, 60, 64, 72, 128, 160, 256, 384, 512))
        groups = rng.choice([g for g in (1, 1, 4, 8) if e % g == 0 and e // g >= 2])
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(10, keep * (e // groups)))
        return {"op": op, "t": _log(rng, 1, 32768 * 64 // max(64, e)), "e": e, "k": k, "score": rng.choice(("softmax", "sigmoid")),
                "bias": rng.randint(0, 1), "groups": groups, "keep": keep, "best": rng.randint(1, 2), "renorm": rng.randint(0, 1),
                "fp32": rng.randint(0, 1)}
    v, fp32 = _log(rng, 1000, 262144), rng.randint(0, 1)
    return {"op": op, "n": _log(rng, 1, min(2048, 2 ** (27 - fp32) // v)), "v": v, "k": rng.choice((0, 1, 5, 20, 32)), "fp32": fp32,
            "cool": rng.choice((0.5, 1.0, 1.3))}


def _token_bytes(c):
    return 2 * c["hkv"] * (c["d"] if c["fmt"] == "fp8" else c["d"] // 2 + c["d"] // 16)


def work(case):
    c = case
    if c["op"] == "plan":
        tokens = c["s"] * c["q"]
        # lengths, pages held and new tokens in, both out again with the rows; slots and positions; the tokens' pages
        return {"bytes": c["s"] * 32 + tokens * (16 if c["kind"] == "tree" else 8) + tokens // c["page"] * 8, "flops": 0}
    if c["op"] == "rotate":
        live = c["n"] - (c["n"] // c["skip"] if c["skip"] else 0)
        row = c["d"] * 2
        # q, k and v in, turned q and k out, codes; the angles; then codes in and both out
        return {"bytes": live * (row * (2 * c["hq"] + 3 * c["hkv"]) + 2 * _token_bytes(c) + 4 * c["rope"] + 4) + c["n"] * (row * 2 * c["hkv"] + 8),
                "flops": live * c["d"] * (c["hq"] + c["hkv"]) * 6}
    if c["op"] == "route":
        return {"bytes": c["t"] * (c["e"] * (4 if c["fp32"] else 2) + 8 * c["k"]), "flops": 4 * c["t"] * c["e"]}
    return {"bytes": c["n"] * (c["v"] * (4 if c["fp32"] else 2) + 12 + 8 * c["k"]), "flops": 6 * c["n"] * c["v"]}


# ------------------------------------------------------------------------------ prepare

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"plan": _prepare_plan, "rotate": _prepare_rotate, "route": _prepare_route, "logprobs": _prepare_logprobs}[case["op"]](dict(case), gen)


def _ints(*shape):
    return torch.empty(*shape, dtype=torch.int32, device="cuda")


def _prepare_plan(c, gen):
    s, q, ctx, page = c["s"], c["q"], c["ctx"], c["page"]

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    # lengths over their logarithm; some tokens at the end of the pages held are drafts that were not accepted
    length = torch.exp(uniform(s) * math.log(ctx + 0.49)).round().long().clamp(1, ctx)
    drop = (uniform(s) * 8).long() if c["kind"] != "step" else torch.zeros(s, dtype=torch.int64, device="cuda")
    held = (length + page - 1) // page
    length = (length - drop).clamp(min=0)
    if c["kind"] == "step":
        n_new = torch.ones(s, dtype=torch.int64, device="cuda")
    elif c["kind"] == "tree":
        n_new = 1 + (uniform(s) * q).long().clamp(max=q - 1)
    else:
        u = uniform(s)                           # a few end, a few wait, half go on by one token, the rest by a chunk
        n_new = torch.where(u < 0.1, -1, torch.where(u < 0.2, 0, torch.where(u < 0.6, 1, 1 + (uniform(s) * q).long().clamp(max=q - 1))))
    per = -(-(ctx + q) // page)
    n_pages = s * per + 5
    order = torch.randperm(n_pages, generator=gen, device="cuda").int()
    at = held.cumsum(0) - held
    j = torch.arange(per + 1, device="cuda")
    table = torch.where(j < held[:, None], order[(at[:, None] + j).clamp(max=n_pages - 1)], -1)
    i = torch.arange(n_pages, device="cuda")
    n_free = n_pages - held.sum()
    free = torch.where(i < n_free, order[(i + held.sum()).clamp(max=n_pages - 1)], -1)
    tokens = s * q
    st = {"case": c, "n_new": n_new.int(), "len": length.int(), "held": held.int(), "table": table.contiguous(), "free": free.contiguous(),
          "n_free": n_free.int().reshape(1), "n_pages": n_pages, "tokens": tokens, "q_start": _ints(s + 1), "kv_len": _ints(s),
          "len_out": _ints(s), "held_out": _ints(s), "n_free_out": _ints(1), "slots": _ints(tokens), "positions": _ints(tokens), "tree": None}
    if c["kind"] == "tree":                      # every drafted token under one of the few before it, or under the context
        start = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), n_new.cumsum(0)))
        t = torch.arange(tokens, device="cuda")
        seq = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=s - 1)
        bit = (t - start[seq]).clamp(0, 63)
        st["tree"] = (torch.randint(0, 2 ** 62, (tokens,), generator=gen, device="cuda") & ((1 << bit) - 1)) | (1 << bit)
    if own:                                      # the handle over its pool that a program keeps
        import expert_cache_gb300 as ft
        st["kv"] = ft.KVCache(L=1, n_pages=n_pages, page_size=page, n_kv_heads=1, head_dim=64, n_q_heads=1, max_seqs=s)
    return st


def _prepare_rotate(c, gen):
    n, hq, hkv, d, page, rope = (c[x] for x in ("n", "hq", "hkv", "d", "page", "rope"))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    # q, k and v lie side by side in the fused projection's output; a few of a key's channels are much larger than the rest
    qkv = normal(n, (hq + 2 * hkv) * d)
    qkv[:, hq * d:(hq + hkv) * d] *= torch.exp(0.6 * normal(hkv * d))
    qkv = qkv.to(torch.bfloat16)
    n_pages = -(-n // page) + 3
    i = torch.arange(n, device="cuda")
    order = torch.randperm(n_pages, generator=gen, device="cuda")
    slots = order[i // page] * page + i % page
    if c["skip"]:
        slots[c["skip"] - 1::c["skip"]] = -1
    first = torch.randint(0, max(1, c["places"] - n), (1,), generator=gen, device="cuda")
    places = max(c["places"], n)
    angle = torch.arange(places, device="cuda", dtype=torch.float64)[:, None] * 1e6 ** (
        -torch.arange(rope // 2, device="cuda", dtype=torch.float64) / (rope // 2))
    st = {"case": c, "q": qkv[:, :hq * d], "k": qkv[:, hq * d:(hq + hkv) * d], "v": qkv[:, (hq + hkv) * d:], "slots": slots.int(),
          "positions": (first + i).int(), "rope": torch.cat((torch.cos(angle), torch.sin(angle)), 1).float(), "places": places,
          "q_norm": None, "k_norm": None, "eps": 1e-6, "k_scale": 0.0625, "v_scale": 0.015625}
    if c["norm"]:
        st["q_norm"], st["k_norm"] = ((1 + 0.2 * normal(d)).to(torch.bfloat16).float() for _ in range(2))
    st["q_out"] = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    st["k_out"] = torch.zeros(n, hkv, d, dtype=torch.bfloat16, device="cuda")
    st["k_back"], st["v_back"] = torch.empty_like(st["k_out"]), torch.empty_like(st["k_out"])
    pool = torch.zeros(n_pages * page * _token_bytes(c), dtype=torch.uint8, device="cuda")
    if own:                                      # the handle over its pool that a program keeps
        import expert_cache_gb300 as ft
        st["kv"] = ft.KVCache(L=1, n_pages=n_pages, page_size=page, n_kv_heads=hkv, head_dim=d, n_q_heads=hq, max_seqs=1, fmt=c["fmt"],
                              k_scale=st["k_scale"], v_scale=st["v_scale"], pool=pool)
    return st


def _prepare_route(c, gen):
    t, e, k = c["t"], c["e"], c["k"]
    logits = 1.5 * torch.randn(t, e, generator=gen, device="cuda")
    return {"case": c, "logits": logits if c["fp32"] else logits.to(torch.bfloat16),
            "bias": 0.05 * torch.randn(e, generator=gen, device="cuda") if c["bias"] else None,
            "scale": 1.0 if c["renorm"] else 2.5, "ids": _ints(t, k), "w": torch.empty(t, k, device="cuda")}


def _prepare_logprobs(c, gen):
    n, v, k = c["n"], c["v"], c["k"]
    logits = torch.empty(n, v, dtype=torch.float32 if c["fp32"] else torch.bfloat16, device="cuda")
    logits.normal_(0.0, 3.0, generator=gen)
    # the token asked for is a likely one in half of the rows
    tokens = torch.randint(0, v, (n,), generator=gen, device="cuda")
    likely = torch.rand(n, generator=gen, device="cuda") < 0.5
    i = torch.arange(n, device="cuda")
    logits[i, tokens] = torch.where(likely, 13.0, logits[i, tokens].float()).to(logits.dtype)
    return {"case": c, "logits": logits, "tokens": tokens.int(), "logp": torch.empty(n, device="cuda"), "entropy": torch.empty(n, device="cuda"),
            "ids": _ints(n, k), "top": torch.empty(n, k, device="cuda")}


# ------------------------------------------------------------------------------ run

def run(state):
    st, c = state, state["case"]
    if own:
        return {"plan": _own_plan, "rotate": _own_rotate, "route": _own_route, "logprobs": _own_logprobs}[c["op"]](st, c)
    return {"plan": _plain_plan, "rotate": _plain_rotate, "route": _plain_route, "logprobs": _plain_logprobs}[c["op"]](st, c)


def _own_plan(st, c):
    import expert_cache_gb300 as ft
    ft.ft_kv_plan(st["kv"].handle, st["n_new"], st["len"], st["held"], st["table"], st["table"].stride(0), st["free"], st["n_free"], c["s"],
                  st["tokens"], st["q_start"], st["kv_len"], st["slots"], st["len_out"], st["held_out"], st["n_free_out"],
                  positions=st["positions"], tree_mask=st["tree"])
    return {x: st[x] for x in ("q_start", "kv_len", "slots", "positions", "len_out", "held_out", "n_free_out", "table", "free")}


def _own_rotate(st, c):
    import expert_cache_gb300 as ft
    h = st["kv"].handle
    ft.ft_kv_append_rotated(h, 0, st["q"], st["k"], st["v"], st["slots"], c["n"], st["q_out"], st["positions"], st["rope"], c["rope"],
                            st["places"], k_out=st["k_out"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=st["eps"], interleaved=c["inter"])
    ft.ft_kv_read(h, 0, st["slots"], c["n"], st["k_back"], st["v_back"])
    return {x: st[x] for x in ("q_out", "k_out", "k_back", "v_back")}


def _own_route(st, c):
    import expert_cache_gb300 as ft
    ft.ft_moe_route(st["logits"], c["t"], c["e"], c["k"], st["ids"], st["w"], score=c["score"], bias=st["bias"], n_group=c["groups"],
                    topk_group=c["keep"], group_best=c["best"], renormalise=c["renorm"], scale=st["scale"])
    return {"ids": st["ids"], "w": st["w"]}


def _own_logprobs(st, c):
    import expert_cache_gb300 as ft
    ft.ft_logprobs(st["logits"], c["n"], c["v"], st["tokens"], st["logp"], st["entropy"], st["ids"], st["top"], c["k"], scale=c["cool"])
    return {"logp": st["logp"], "entropy": st["entropy"], "ids": st["ids"], "top": st["top"]}


# ------------------------------------------------------------------------------ plain forms

def _plain_plan(st, c):
    page, s = c["page"], c["s"]
    n_new, length, held, n_free = st["n_new"].long(), st["len"].long(), st["held"].long(), st["n_free"].long()
    ends, rows = n_new < 0, n_new.clamp(min=0)
    length = torch.where(ends, 0, length)
    after = length + rows
    want = (after + page - 1) // page
    gives, takes = (held - want).clamp(min=0), (want - held).clamp(min=0)
    first = torch.cat((rows.new_zeros(1), rows.cumsum(0)))
    given, taken = gives.cumsum(0), takes.cumsum(0)
    # the stack with what is given back on top of it
    i = torch.arange(st["n_pages"], device="cuda")
    g = i - n_free
    of = torch.searchsorted(given, g, right=True).clamp(max=s - 1)
    back = st["table"].flatten()[(of * st["table"].stride(0) + want[of] + g - (given - gives)[of]).clamp(0, st["table"].numel() - 1)]
    avail = n_free + given[-1]
    stack = torch.where(i < n_free, st["free"], back)
    left = avail - taken[-1]
    free = torch.where((i >= n_free) & (i < left), stack, st["free"])
    # pages taken stand behind those held
    j = torch.arange(st["table"].shape[1], device="cuda")
    rank = (taken - takes)[:, None] + j - held[:, None]
    mine = stack[(avail - 1 - rank).clamp(0, st["n_pages"] - 1)]
    table = torch.where((j >= held[:, None]) & (j < want[:, None]), mine, st["table"])
    t = torch.arange(st["tokens"], device="cuda")
    seq = torch.searchsorted(first[1:].contiguous(), t, right=True)
    live, seq = seq < s, seq.clamp(max=s - 1)
    pos = length[seq] + t - first[seq]
    slots = table[seq, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    if st["tree"] is not None:
        bits = (st["tree"][:, None] >> torch.arange(64, device="cuda")) & 1
        pos = length[seq] + bits.sum(1) - 1
    out = {"q_start": first, "kv_len": after, "slots": torch.where(live, slots, -1), "positions": torch.where(live, pos, 0), "len_out": after,
           "held_out": want, "n_free_out": left, "table": table, "free": free}
    return {x: v.int() for x, v in out.items()}


def _turn(x, weight, eps, cos, sin, inter):
    """Norm of each head and rotation by position, in the type of x [n, heads, D]."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.to(x.dtype)
    cos, sin, r = cos.to(x.dtype)[:, None], sin.to(x.dtype)[:, None], cos.shape[-1]
    a, b = (x[..., 0:2 * r:2], x[..., 1:2 * r:2]) if inter else (x[..., :r], x[..., r:2 * r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., 2 * r:]), -1)


def _e4m3_round(x):
    """Nearest E4M3 value of |x|, ties to even, at most 448."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(-6, 8)
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -6), e - 1, e)       # log2 may round up
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, e).clamp(-6, 8)          # or down
    step = torch.exp2(e - 3)
    return (torch.round(a / step) * step).clamp(max=448.0)


def _stored(x, fmt, st):
    """The values that the codes of x [.., D] (bf16) stand for."""
    x = x.float()
    if fmt == "fp8":
        y = x / st
        return torch.where(y < 0, -_e4m3_round(y), _e4m3_round(y)) * st
    b = x.unflatten(-1, (-1, 16))
    sc = _e4m3_round(b.abs().amax(-1, keepdim=True) / 6.0 / st)
    den = sc * st
    y = torch.where(den > 0, b / torch.where(den > 0, den, 1.0), 0.0)
    a = y.abs()
    mag = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    val = torch.tensor(E2M1, device=x.device)[mag]
    return ((torch.where(y < 0, -val, val) * sc) * st).flatten(-2)


def _plain_rotate(st, c):
    n, hq, hkv, d, r = c["n"], c["hq"], c["hkv"], c["d"], c["rope"] // 2
    at = st["rope"][st["positions"].long()]
    cos, sin = at[:, :r], at[:, r:]
    q = _turn(st["q"].float().reshape(n, hq, d), st["q_norm"], st["eps"], cos, sin, c["inter"]).to(torch.bfloat16)
    # a key is rounded to the cache's few bits: the values before that in 64
    k = _turn(st["k"].double().reshape(n, hkv, d), st["k_norm"], st["eps"], cos, sin, c["inter"]).float().to(torch.bfloat16)
    live = (st["slots"] >= 0)[:, None, None]
    back = [_stored(x, c["fmt"], st[s]).to(torch.bfloat16) for x, s in ((k, "k_scale"), (st["v"].reshape(n, hkv, d), "v_scale"))]
    return {x: torch.where(live, v, 0) for x, v in (("q_out", q), ("k_out", k), ("k_back", back[0]), ("v_back", back[1]))}


def _plain_route(st, c):
    t, e, k = c["t"], c["e"], c["k"]
    # the order of scores that lie close together: in 64 bits
    x = torch.where(torch.isnan(st["logits"]), -float("inf"), st["logits"].double()).clamp(max=LARGEST)
    if c["score"] == "softmax":
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(top == -float("inf"), 0.0, top))
        total = p.sum(-1, keepdim=True)
        score = p / torch.where(total > 0, total, 1.0)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    choice = score if st["bias"] is None else score + st["bias"].double()
    choice = torch.where((x == -float("inf")) | torch.isnan(choice), -float("inf"), choice)
    if c["groups"] > 1:
        g = choice.reshape(t, c["groups"], -1)
        best = g.sort(dim=-1, descending=True).values[..., :c["best"]]
        best = torch.where(best[..., :1] == -float("inf"), -float("inf"), torch.where(best == -float("inf"), 0.0, best)).sum(-1)
        order = best.sort(dim=-1, descending=True, stable=True).indices
        kept = torch.zeros_like(best, dtype=torch.bool).scatter(1, order[:, :c["keep"]], True)
        choice = torch.where(kept[..., None], g, -float("inf")).reshape(t, e)
    order = choice.sort(dim=-1, descending=True, stable=True)
    ids, some = order.indices[:, :k], order.values[:, :k] > -float("inf")
    w = torch.where(some, torch.gather(score, 1, ids), 0.0)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return {"ids": torch.where(some, ids, -1).int(), "w": (w * st["scale"]).float()}


def _plain_logprobs(st, c):
    n, v, k = c["n"], c["v"], c["k"]
    x = st["logits"].float()
    x = torch.where(torch.isnan(x), -float("inf"), x).clamp(max=LARGEST)
    top = x.amax(-1, keepdim=True)
    y = (x - torch.where(top == -float("inf"), 0.0, top)) * c["cool"]
    p = torch.exp(y)
    total = p.sum(-1, dtype=torch.float64)                # 100,000 terms
    log_total = torch.log(total)
    entropy = log_total - torch.where(p > 0, p * y, 0.0).sum(-1, dtype=torch.float64) / total
    logp = torch.gather(y, 1, st["tokens"].long()[:, None])[:, 0] - log_total
    # the largest, the lower index first among equals: as whole numbers in that order
    bits = x.view(torch.int32).long() if c["k"] else None
    if k:
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * 2 ** 20 + (v - 1 - torch.arange(v, device="cuda"))
        ids = v - 1 - torch.topk(key, k, -1).values % 2 ** 20
        tops = torch.gather(y, 1, ids) - log_total[:, None]
    else:
        ids, tops = st["ids"], st["top"]
    return {"logp": logp.float(), "entropy": entropy.float(), "ids": ids.int(), "top": tops.float()}


# ------------------------------------------------------------------------------ in 64 bits

def _prepared(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def exact(case, seed):
    if case["op"] == "plan":
        return None                              # whole numbers
    st = _prepared(case, seed)
    return {"rotate": _exact_rotate, "route": _exact_route, "logprobs": _exact_logprobs}[case["op"]](st, st["case"])


def _exact_e4m3(a):
    """|a| on the E4M3 grid by its table of 127 values: nearest, ties to the even code."""
    grid = torch.tensor([m / 512.0 for m in range(8)] + [(1 + m / 8.0) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:119],
                        dtype=torch.float64, device=a.device)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 126)
    dl, dh = a - grid[hi - 1], grid[hi] - a
    return grid[torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, hi - 1)]


def _exact_rotate(st, c):
    n, d, r = c["n"], c["d"], c["rope"] // 2
    row = st["rope"].double()[st["positions"].long()]
    turn = torch.complex(row[:, :r], row[:, r:])[:, None]
    live = st["slots"] >= 0
    out = {}
    for name, w in (("q", st["q_norm"]), ("k", st["k_norm"])):
        x = st[name].double().reshape(n, -1, d)
        if w is not None:
            x = w.double() * x / torch.sqrt(torch.einsum("nhd,nhd->nh", x, x) / d + st["eps"])[..., None]
        even, odd = (torch.arange(r, device="cuda") * 2, torch.arange(r, device="cuda") * 2 + 1) if c["inter"] else (
            torch.arange(r, device="cuda"), torch.arange(r, device="cuda") + r)
        z = torch.complex(x[..., even], x[..., odd]) * turn
        x[..., even], x[..., odd] = z.real, z.imag
        x[~live] = 0
        out[name + "_out"] = x
    # what is stored is the key's bf16 value in few bits
    for name, x, s in (("k", out["k_out"].float().to(torch.bfloat16), st["k_scale"]), ("v", st["v"].reshape(n, -1, d), st["v_scale"])):
        s = torch.tensor(s, dtype=torch.float32).double().item()
        x = x.double()
        if c["fmt"] == "fp8":
            val = torch.sign(x) * _exact_e4m3((x / s).abs()) * s
        else:
            b = x.reshape(-1, 16)
            sc = _exact_e4m3(b.abs().amax(1, keepdim=True) / 6 / s) * s
            y = torch.where(sc > 0, b / torch.where(sc > 0, sc, 1.0), 0.0)
            grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
            a = y.abs().clamp(max=6.0).contiguous()
            hi = torch.searchsorted(grid, a).clamp(1, 7)
            dl, dh = a - grid[hi - 1], grid[hi] - a
            val = (grid[torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, hi - 1)] * torch.sign(y) * sc).reshape(x.shape)
        val[~live] = 0
        out[name + "_back"] = val
    return out


def _exact_route(st, c):
    """Each row's experts by repeated search for the largest, in 64 bits."""
    x = st["logits"].double()
    score = torch.softmax(x, -1) if c["score"] == "softmax" else torch.sigmoid(x)
    choice = score.clone() if st["bias"] is None else score + st["bias"].double()
    rows = torch.arange(c["t"], device="cuda")
    size = c["e"] // c["groups"]
    if c["groups"] > 1:
        worth = choice.view(c["t"], c["groups"], size).topk(min(c["best"], size), -1).values.sum(-1)
        out = torch.ones(c["t"], c["groups"], dtype=torch.bool, device="cuda")
        for _ in range(c["keep"]):
            g = worth.argmax(-1)
            worth[rows, g] = -float("inf")
            out[rows, g] = False
        choice[out.repeat_interleave(size, 1)] = -float("inf")
    w = torch.zeros(c["t"], c["k"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        best = choice.amax(-1, keepdim=True)
        i = torch.where(choice == best, torch.arange(c["e"], device="cuda"), c["e"]).amin(-1)
        choice[rows, i] = -float("inf")
        w[:, j] = score[rows, i]
    if c["renorm"]:
        w /= w.sum(-1, keepdim=True)
    return {"ids": None, "w": w * st["scale"]}


def _exact_logprobs(st, c):
    logp, entropy, top = [], [], []
    for a in range(0, c["n"], 256):              # 256 rows at a time
        z = st["logits"][a:a + 256].double() * c["cool"]
        z = z - torch.logsumexp(z, -1, keepdim=True)
        logp.append(torch.gather(z, 1, st["tokens"][a:a + 256].long()[:, None])[:, 0])
        entropy.append(-(torch.exp(z) * z).sum(-1))
        top.append(z.topk(c["k"], -1).values if c["k"] else st["top"][a:a + 256].double())
    return {"logp": torch.cat(logp), "entropy": torch.cat(entropy), "ids": None, "top": torch.cat(top)}
