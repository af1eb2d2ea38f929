"""The quantised key/value cache and the attention over it: the cases they are timed on.

Two groups of calls.  "write": a layer's new keys and values are quantised into the pages of the
cache (`ft_kv_append`) and read back as bf16 (`ft_kv_read`).  "attend": attention of the new tokens of
a batch of sequences over the paged cache (`ft_kv_attention`), for one new token, for a tree of
drafted tokens and for a chunk of a prompt, with or without a sliding window and first tokens that
stay visible.

The plain forms below are elementary torch operations in 32 bits.  The cache is one uint8 pool of
pages; a page holds, for each kv head, page_size / 16 tiles of 16 tokens.  Bytes of a tile (D = head
dim; lane = 4 g + t, g in 0..7, t in 0..3; a lane's bytes come in 16-byte vectors, vector-major):
  K codes   lane's bytes [v 2][D/4 dims]: token 8 v + g, dims t D/4 ..
  V codes   lane's bytes [q 4][D/8 dims]: token 8 (q >> 1) + 2 t + (q & 1), dims g D/8 ..
  K scales  [lane][v 2][D/64 blocks]          (NVFP4 only: UE4M3 per 16 dims of a token)
  V scales  [block D/16][t 4][q 4]
NVFP4: two E2M1 codes per byte, the even dim in the low nibble; FP8: one E4M3 code per byte.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 16 sequences: every layer stores 16 tokens; launch latency counts
        {"name": "write step", "op": "write", "fmt": "nvfp4", "n": 16, "hkv": 8, "d": 128, "page": 64, "skip": 0},
        # one 8192-token prefill chunk (the prefill workload's T)
        {"name": "write chunk", "op": "write", "fmt": "nvfp4", "n": 8192, "hkv": 8, "d": 128, "page": 64, "skip": 0},
        # an odd number of tokens with some of them padding (slot -1), wide heads, 8-bit cache
        {"name": "write odd", "op": "write", "fmt": "fp8", "n": 5003, "hkv": 2, "d": 256, "page": 16, "skip": 7},
        # single-stream decode at an ordinary context: the latency of one layer's attention
        {"name": "decode one", "op": "attend", "fmt": "nvfp4", "kind": "step", "s": 1, "q": 1, "ctx": 4096, "ragged": 0,
         "hq": 16, "hkv": 2, "d": 256, "page": 64, "window": 0, "sink": 0},
        # batched serving, contexts from a few tokens to 32768
        {"name": "decode batch", "op": "attend", "fmt": "fp8", "kind": "step", "s": 32, "q": 1, "ctx": 32768, "ragged": 1,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "window": 0, "sink": 0},
        # one long conversation
        {"name": "decode long", "op": "attend", "fmt": "nvfp4", "kind": "step", "s": 1, "q": 1, "ctx": 262145, "ragged": 0,
         "hq": 16, "hkv": 2, "d": 256, "page": 64, "window": 0, "sink": 0},
        # a sliding-window layer in a larger batch, four sink tokens
        {"name": "decode window", "op": "attend", "fmt": "nvfp4", "kind": "step", "s": 64, "q": 1, "ctx": 8192, "ragged": 1,
         "hq": 64, "hkv": 8, "d": 64, "page": 32, "window": 1024, "sink": 4},
        # a few drafted tokens per sequence over short, windowed contexts
        {"name": "tree small", "op": "attend", "fmt": "fp8", "kind": "tree", "s": 4, "q": 7, "ctx": 1000, "ragged": 1,
         "hq": 16, "hkv": 4, "d": 64, "page": 16, "window": 300, "sink": 2},
        # one stream verifying a tree of 48 drafted tokens
        {"name": "tree one", "op": "attend", "fmt": "nvfp4", "kind": "tree", "s": 1, "q": 48, "ctx": 8192, "ragged": 0,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "window": 0, "sink": 0},
        # a batch of streams verifying trees of up to 64 tokens
        {"name": "tree batch", "op": "attend", "fmt": "nvfp4", "kind": "tree", "s": 16, "q": 64, "ctx": 16384, "ragged": 1,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "window": 0, "sink": 0},
        # a chunk of a long prompt over what the cache holds already
        {"name": "chunk", "op": "attend", "fmt": "nvfp4", "kind": "chunk", "s": 1, "q": 2048, "ctx": 8192, "ragged": 0,
         "hq": 32, "hkv": 8, "d": 128, "page": 64, "window": 0, "sink": 0},
        # ragged prompts through a sliding-window layer
        {"name": "chunk window", "op": "attend", "fmt": "fp8", "kind": "chunk", "s": 5, "q": 1500, "ctx": 5000, "ragged": 1,
         "hq": 16, "hkv": 2, "d": 256, "page": 32, "window": 512, "sink": 8},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    fmt = rng.choice(("nvfp4", "fp8"))
    d = rng.choice((64, 128, 256))
    page = rng.choice((16, 32, 64, 128))
    if rng.random() < 0.25:
        hkv = rng.choice((1, 2, 4, 8))
        n = _log(rng, 1, 8192 * 8 * 128 // (hkv * d) // 2)
        return {"op": "write", "fmt": fmt, "n": n, "hkv": hkv, "d": d, "page": page, "skip": rng.choice((0, 0, 5, 11))}
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.choice((1, 2, 4, 5, 8))
    window, sink = rng.choice(((0, 0), (0, 0), (_log(rng, 16, 4096), rng.randint(0, 16))))
    kind = rng.choice(("step", "tree", "chunk"))
    if kind == "step":
        s = _log(rng, 1, 64)
        ctx = _log(rng, 1, min(262144, 2 ** 28 // (s * hkv * d)))
        q = 1
    elif kind == "tree":
        s = _log(rng, 1, 16)
        q = rng.randint(2, 64)
        ctx = _log(rng, q, min(32768, 2 ** 27 // (s * hkv * d)))
    else:
        s = _log(rng, 1, 6)
        q = _log(rng, 65, min(2048, math.isqrt(2 ** 36 // (s * hq * d))))
        ctx = _log(rng, q, min(16384, 2 ** 36 // (s * q * hq * d)))
    return {"op": "attend", "fmt": fmt, "kind": kind, "s": s, "q": q, "ctx": ctx, "ragged": int(s > 1 and rng.random() < 0.7),
            "hq": hq, "hkv": hkv, "d": d, "page": page, "window": window, "sink": sink}


# ------------------------------------------------------------------------------ what a case fixes

def _plan(c):
    """New tokens and cached length of each sequence, and the drafted tokens' parents: fixed by the case."""
    rng = random.Random("%s %s %s %s" % (c["s"], c["q"], c["ctx"], c["hkv"]))
    nq, kv, parents = [], [], []
    for i in range(c["s"]):
        n = c["q"] if not c["ragged"] or c["q"] == 1 else rng.randint(1, c["q"])
        length = c["ctx"] if not c["ragged"] or i == 0 else _log(rng, min(n, c["ctx"]), c["ctx"])
        nq.append(n)
        kv.append(max(n, length))
        # a drafted token hangs under one of the last few before it; the first under the context
        parents.append([rng.randint(max(-1, j - 6), j - 1) for j in range(n)] if c["kind"] == "tree" else None)
    return nq, kv, parents


def _masks(parents):
    """Ancestors of each drafted token, itself included, as 64-bit masks."""
    out = []
    for j, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | (1 << j))
    return out


def _signed(m):
    return m - (1 << 64) if m >> 63 else m


def _token_bytes(c):
    return 2 * c["hkv"] * (c["d"] if c["fmt"] == "fp8" else c["d"] // 2 + c["d"] // 16)


def _tile_bytes(c):
    return 16 * _token_bytes(c) // c["hkv"]


def work(case):
    c = case
    if c["op"] == "write":
        live = c["n"] - (c["n"] // c["skip"] if c["skip"] else 0)
        moved = 2 * c["hkv"] * c["d"] * 2
        # k and v in, codes out; codes in, bf16 out (zeros for the padding); the slots twice
        return {"bytes": live * (moved + 2 * _token_bytes(c)) + c["n"] * (moved + 8), "flops": 0}
    nq, kv, parents = _plan(c)
    pairs = keys = 0
    for n, length, par in zip(nq, kv, parents):
        base, w, sink = length - n, c["window"], c["sink"]
        masks = _masks(par) if par else None
        low = length
        for i in range(n):
            if par:
                depth = bin(masks[i]).count("1") - 1
                top = base
                first = max(0, base + depth - w + 1) if w else 0
                new = depth + 1
                if w and depth >= w:          # ancestors that the window has left behind
                    new = w
                seen = max(0, top - first) + new + max(0, min(sink, first, top))
            else:
                top = base + i + 1
                first = max(0, top - w) if w else 0
                seen = top - first + min(sink, first)
            low = min(low, first)
            pairs += seen
        keys += length - low + min(sink, low)
    tokens = sum(nq)
    return {"bytes": tokens * c["hq"] * (c["d"] * 4 + 4) + keys * _token_bytes(c),
            "flops": 4 * c["d"] * c["hq"] * pairs}


# ------------------------------------------------------------------------------ number formats, plain

def _e4m3_round(x):
    """Nearest E4M3 value of |x|, ties to even, at most 448."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(-6, 8)
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -6), e - 1, e)       # log2 may round up
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, e).clamp(-6, 8)          # or down
    step = torch.exp2(e - 3)
    return (torch.round(a / step) * step).clamp(max=448.0)


def _quantise(x, fmt, st):
    """Codes (one per element), UE4M3 scale values (NVFP4) and the values that they stand for."""
    x = x.float()
    if fmt == "fp8":
        y = torch.nan_to_num(x / st, nan=0.0, posinf=448.0, neginf=-448.0)
        r = _e4m3_round(y)
        val = torch.where(y < 0, -r, r)
        return val, None, val * st
    b = x.unflatten(-1, (-1, 16))
    sc = _e4m3_round(torch.nan_to_num(b.abs(), nan=0.0, posinf=float("inf")).amax(-1, keepdim=True) / 6.0 / st)
    den = sc * st
    y = torch.where(den > 0, torch.nan_to_num(b / torch.where(den > 0, den, 1.0), nan=0.0), 0.0)
    a = y.abs()
    mag = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() +
           (a >= 3.5).int() + (a > 5.0).int())
    code = torch.where((y < 0) & (mag > 0), mag + 8, mag)
    table = torch.tensor(E2M1, device=x.device)
    val = torch.where(y < 0, -table[mag], table[mag])
    return code.flatten(-2), sc.squeeze(-1), ((val * sc) * st).flatten(-2)


def _e4m3_byte(v):
    """Byte of a value that E4M3 holds exactly."""
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -6), e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, e)
    m = torch.where(a < 2.0 ** -6, a * 512.0, (a / torch.exp2(e) - 1.0) * 8.0 + 8.0 * (e + 7.0))
    return (m.to(torch.int32) | ((v < 0) & (a > 0)).int() * 128).to(torch.uint8)


def _e4m3_value(b):
    b = b.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).float()
    a = torch.where(e == 0, m / 512.0, (1.0 + m / 8.0) * torch.exp2((e - 7).float()))
    return torch.where(b >= 128, -a, a)


# ------------------------------------------------------------------------------ tiles, plain

def _pack_tiles(k, v, c):
    """[.., 16, D] keys and values -> [.., tile bytes]."""
    d, fmt = c["d"], c["fmt"]
    lead = k.shape[:-2]
    parts = []
    kc, ks, _ = _quantise(k, fmt, c["k_scale"])
    vc, vs, _ = _quantise(v, fmt, c["v_scale"])
    for what, codes in (("k", kc), ("v", vc)):
        b = _e4m3_byte(codes) if fmt == "fp8" else (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)
        w = b.shape[-1]
        if what == "k":        # [v, g][t, w/4] -> [g, t][v, w/4]
            b = b.reshape(*lead, 2, 8, 4, w // 4).movedim(-4, -2)
        else:                  # [q>>1, t, q&1][g, w/8] -> [g, t][q>>1, q&1, w/8]
            b = b.reshape(*lead, 2, 4, 2, 8, w // 8).movedim(-2, -5).movedim(-3, -4)
        b = b.reshape(*lead, 32, -1, 16).transpose(-3, -2)
        parts.append(b.reshape(*lead, -1))
    if fmt == "nvfp4":
        s = _e4m3_byte(ks).reshape(*lead, 2, 8, 4, d // 64).movedim(-4, -2)
        parts.append(s.reshape(*lead, -1))
        s = _e4m3_byte(vs).reshape(*lead, 2, 4, 2, d // 16).movedim(-1, -4).transpose(-3, -2)
        parts.append(s.reshape(*lead, -1))
    return torch.cat(parts, -1)


def _unpack_tiles(t, c):
    """[.., tile bytes] -> fp32 keys and values [.., 16, D]."""
    d, fmt = c["d"], c["fmt"]
    lead = t.shape[:-1]
    size = 16 * d if fmt == "fp8" else 8 * d
    w = size // 16
    out = []
    for what, b in (("k", t[..., :size]), ("v", t[..., size:2 * size])):
        b = b.reshape(*lead, -1, 32, 16).transpose(-3, -2)
        if what == "k":
            b = b.reshape(*lead, 8, 4, 2, w // 4).movedim(-2, -4)
        else:
            b = b.reshape(*lead, 8, 4, 2, 2, w // 8).transpose(-4, -3).movedim(-5, -2)
        b = b.reshape(*lead, 16, w)
        if fmt == "fp8":
            out.append(_e4m3_value(b))
        else:
            n = torch.stack((b & 15, b >> 4), -1).reshape(*lead, 16, d).int()
            mag = torch.tensor(E2M1, device=t.device)[(n & 7)]
            out.append(torch.where(n >= 8, -mag, mag))
    if fmt == "nvfp4":
        s = _e4m3_value(t[..., 2 * size:2 * size + d])
        s = s.reshape(*lead, 8, 4, 2, d // 64).movedim(-2, -4).reshape(*lead, 16, d // 16, 1)
        out[0] = (out[0].unflatten(-1, (-1, 16)) * s).flatten(-2)
        s = _e4m3_value(t[..., 2 * size + d:])
        s = s.reshape(*lead, d // 16, 4, 2, 2).transpose(-3, -2).movedim(-4, -1).reshape(*lead, 16, d // 16, 1)
        out[1] = (out[1].unflatten(-1, (-1, 16)) * s).flatten(-2)
    return out[0] * c["k_scale"], out[1] * c["v_scale"]


# ------------------------------------------------------------------------------ prepare

def prepare(case, seed):
    c = dict(case)
    c["k_scale"], c["v_scale"] = 0.5, 0.25
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    d, hkv, page = c["d"], c["hkv"], c["page"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    # keys have a few channels that are much larger than the rest, values do not
    channel = torch.exp(0.6 * normal(hkv, d))
    st = {"case": c}
    if c["op"] == "write":
        n = c["n"]
        n_pages = -(-n // page) + 3
        # k and v lie in the fused projection's output
        width = (2 * hkv + 2) * d
        qkv = normal(n, width).to(torch.bfloat16)
        qkv[:, 2 * d:2 * d + hkv * d] *= channel.reshape(-1).to(torch.bfloat16)
        k, v = qkv[:, 2 * d:(2 + hkv) * d], qkv[:, (2 + hkv) * d:]
        order = torch.randperm(n_pages, generator=gen, device="cuda")
        i = torch.arange(n, device="cuda")
        slots = order[i // page] * page + i % page
        if c["skip"]:
            slots[c["skip"] - 1::c["skip"]] = -1
        st.update(k=k, v=v, slots=slots.int(), k_out=torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda"),
                  v_out=torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda"))
        pool = torch.zeros(n_pages * hkv * (page // 16) * _tile_bytes(c), dtype=torch.uint8, device="cuda")
        hq, s = hkv, 1
    else:
        s, hq = c["s"], c["hq"]
        nq, kv, parents = _plan(c)
        per = [-(-length // page) for length in kv]
        n_pages = sum(per) + 2
        stride = max(per) + 1
        order = torch.randperm(n_pages, generator=gen, device="cuda").int()
        table = torch.zeros(s, stride, dtype=torch.int32, device="cuda")
        at = 0
        for i, p in enumerate(per):
            table[i, :p] = order[at:at + p]
            at += p
        pool = torch.empty(n_pages, hkv, page // 16, _tile_bytes(c), dtype=torch.uint8, device="cuda")
        step = max(1, 2 ** 26 // (hkv * page * d))
        for a in range(0, n_pages, step):                       # every token of every page is a written one
            m = min(step, n_pages - a)
            k = (normal(m, hkv, page // 16, 16, d) * channel[:, None, None]).to(torch.bfloat16)
            v = normal(m, hkv, page // 16, 16, d).to(torch.bfloat16)
            pool[a:a + m] = _pack_tiles(k, v, c)
        pool = pool.reshape(-1)
        tokens = sum(nq)
        start = torch.tensor([sum(nq[:i]) for i in range(s + 1)], dtype=torch.int32, device="cuda")
        masks = None
        if c["kind"] == "tree":
            masks = torch.tensor([_signed(m) for par in parents for m in _masks(par)], dtype=torch.int64, device="cuda")
        # a query that finds some keys: logits of a few units, as trained heads have
        st.update(q=normal(tokens, hq, d).to(torch.bfloat16), start=start, tokens=tokens, max_q=max(nq), max_kv=max(kv),
                  kv_len=torch.tensor(kv, dtype=torch.int32, device="cuda"), table=table, masks=masks,
                  scale=1.0 / math.sqrt(d), o=torch.empty(tokens, hq, d, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.empty(tokens, hq, dtype=torch.float32, device="cuda"))
    st["pool"], st["n_pages"] = pool, n_pages
    if own:                                                     # the handle over the pool that a program keeps
        import expert_cache_gb300 as ft
        st["kv"] = ft.KVCache(L=1, n_pages=n_pages, page_size=page, n_kv_heads=hkv, head_dim=d, n_q_heads=hq, max_seqs=s,
                              fmt=c["fmt"], k_scale=c["k_scale"], v_scale=c["v_scale"], pool=pool)
    return st


# ------------------------------------------------------------------------------ run

def run(state):
    st, c = state, state["case"]
    if own:
        import expert_cache_gb300 as ft
        h = st["kv"].handle
        if c["op"] == "write":
            ft.ft_kv_append(h, 0, st["k"], st["v"], st["slots"], c["n"], k_stride=st["k"].stride(0), v_stride=st["v"].stride(0))
            ft.ft_kv_read(h, 0, st["slots"], c["n"], st["k_out"], st["v_out"])
            return {"k": st["k_out"], "v": st["v_out"]}
        ft.ft_kv_attention(h, 0, st["q"], st["start"], st["kv_len"], st["table"], st["table"].stride(0), c["s"], st["tokens"],
                           st["max_q"], st["o"], tree_mask=st["masks"], window=c["window"], n_sink=c["sink"],
                           sm_scale=st["scale"], lse=st["lse"])
        return {"o": st["o"], "lse": st["lse"]}
    if c["op"] == "write":
        return _plain_write(st, c)
    return _plain_attend(st, c)


def _plain_write(st, c):
    n, hkv, d = c["n"], c["hkv"], c["d"]
    live = (st["slots"] >= 0)[:, None, None]
    out = {}
    for name, sc in (("k", c["k_scale"]), ("v", c["v_scale"])):
        val = _quantise(st[name].reshape(n, hkv, d), c["fmt"], sc)[2]
        out[name] = torch.where(live, val, 0.0).to(torch.bfloat16)
    return out


def _plain_attend(st, c):
    s, hq, hkv, d, page = c["s"], c["hq"], c["hkv"], c["d"], c["page"]
    g = hq // hkv
    nq, nk = st["max_q"], st["max_kv"]
    start, kv_len = st["start"].long(), st["kv_len"].long()
    # the sequences' keys and values, padded to the longest
    pages = st["table"][:, :-(-nk // page)].long()
    tiles = st["pool"].reshape(st["n_pages"], hkv, page // 16, -1)[pages]            # [s, pages, hkv, tiles, bytes]
    k, v = _unpack_tiles(tiles, c)
    k = k.movedim(2, 1).reshape(s, hkv, -1, d)[:, :, :nk]
    v = v.movedim(2, 1).reshape(s, hkv, -1, d)[:, :, :nk]
    # the queries, padded likewise
    n = start[1:] - start[:-1]
    i = torch.arange(nq, device="cuda")
    row = (start[:-1, None] + i).clamp(max=st["tokens"] - 1)
    q = st["q"].float()[row].reshape(s, nq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(s, hkv, g * nq, d)
    logits = torch.matmul(q, k.transpose(-1, -2)).reshape(s, hkv, g, nq, nk) * st["scale"]
    # who sees whom
    base = (kv_len - n)[:, None, None]
    j = torch.arange(nk, device="cuda")[None, None, :]
    if st["masks"] is None:
        seen = j <= base + i[None, :, None]
        pos_q = (base + i[None, :, None])
        pos_k = j.expand(s, 1, nk)
    else:
        m = st["masks"][row]                                                         # [s, nq]
        bits = (m[:, :, None] >> torch.arange(64, device="cuda")) & 1
        depth = bits.sum(-1) - 1
        jj = (j - base).clamp(0, 63)
        mine = torch.gather(bits, 2, jj.expand(s, nq, nk)) == 1
        seen = (j < base) | ((j - base < n[:, None, None]) & mine)
        pos_q = base + depth[:, :, None]
        pos_k = torch.where(j < base, j, base + torch.gather(depth[:, None, :].expand(s, 1, nq), 2, jj.clamp(max=nq - 1)))
    seen = seen & (j < kv_len[:, None, None])
    if c["window"]:
        seen = seen & ((j < c["sink"]) | (pos_q - pos_k < c["window"]))
    logits = torch.where(seen[:, None, None], logits, -float("inf"))
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -float("inf"), 0.0, top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(s, hkv, g * nq, nk), v).reshape(s, hkv, g, nq, d)
    o = o / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + top).squeeze(-1)
    # back to the packed rows
    seq = torch.searchsorted(start[1:].contiguous(), torch.arange(st["tokens"], device="cuda"), right=True)
    at = torch.arange(st["tokens"], device="cuda") - start[seq]
    o = o.permute(0, 3, 1, 2, 4).reshape(s, nq, hq, d)[seq, at]
    lse = lse.permute(0, 3, 1, 2).reshape(s, nq, hq)[seq, at]
    return {"o": o.to(torch.bfloat16), "lse": lse}


# ------------------------------------------------------------------------------ in 64 bits

def _exact_e4m3(a):
    """|a| on the E4M3 grid by its table of 127 values: nearest, ties to the even code."""
    grid = torch.tensor([m / 512.0 for m in range(8)] + [(1 + m / 8.0) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:119],
                        dtype=torch.float64, device=a.device)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return grid[pick]


def _exact_write(st, c):
    out = {}
    for name, sc in (("k", c["k_scale"]), ("v", c["v_scale"])):
        x = st[name].double().reshape(-1, 16)
        if c["fmt"] == "fp8":
            y = x / sc
            val = torch.sign(y) * _exact_e4m3(y.abs()) * sc
        else:
            s = _exact_e4m3(x.abs().amax(1, keepdim=True) / 6 / sc) * sc
            y = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0)
            grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
            a = y.abs().clamp(max=6.0).contiguous()
            hi = torch.searchsorted(grid, a).clamp(1, 7)
            dl, dh = a - grid[hi - 1], grid[hi] - a
            val = grid[torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, hi - 1)] * torch.sign(y) * s
        val = val.reshape(c["n"], c["hkv"], c["d"])
        val[st["slots"] < 0] = 0
        out[name] = val
    return out


def _exact_rows(st, c, seq, length, head):
    """Keys and values [length, D] of one head in 64 bits, by the byte address of every element."""
    d, page = c["d"], c["page"]
    tok = torch.arange(length, device="cuda")
    tile = (st["table"][seq].long()[tok // page] * c["hkv"] + head) * (page // 16) + tok % page // 16
    at = tile * _tile_bytes(c)
    r = (tok % 16)[:, None]
    x = torch.arange(d, device="cuda")[None, :]
    pool, four = st["pool"], c["fmt"] == "nvfp4"
    size = 8 * d if four else 16 * d
    out = []
    for what in ("k", "v"):
        if what == "k":
            lane, within = 4 * (r % 8) + x // (d // 4), (r // 8) * (d // 4) + x % (d // 4)
        else:
            q = 2 * (r // 8) + r % 2
            lane, within = 4 * (x // (d // 8)) + r % 8 // 2, q * (d // 8) + x % (d // 8)
        b = within // 2 if four else within
        byte = pool[at[:, None] + (size if what == "v" else 0) + b // 16 * 512 + lane * 16 + b % 16].long()
        if four:
            n = torch.where(within % 2 == 1, byte >> 4, byte & 15)
            val = torch.tensor(E2M1 + tuple(-e for e in E2M1), dtype=torch.float64, device="cuda")[n]
            blk = x // 16
            if what == "k":
                o = (4 * (r % 8) + blk // (d // 64)) * (d // 32) + (r // 8) * (d // 64) + blk % (d // 64)
            else:
                o = d + (blk * 4 + r % 8 // 2) * 4 + 2 * (r // 8) + r % 2
            byte = pool[at[:, None] + 2 * size + o].long()
        e, m = byte // 8 % 16, (byte % 8).double()
        f = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2((e - 7).double()))
        f = torch.where(byte >= 128, -f, f)
        out.append((val * f if four else f) * c["k_scale" if what == "k" else "v_scale"])
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    c = st["case"]
    if c["op"] == "write":
        return _exact_write(st, c)
    nq, kv, parents = _plan(c)
    g, first = c["hq"] // c["hkv"], 0
    o = torch.zeros(st["tokens"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((st["tokens"], c["hq"]), -float("inf"), dtype=torch.float64, device="cuda")
    for s, (n, length, par) in enumerate(zip(nq, kv, parents)):
        base = length - n
        j = torch.arange(length, device="cuda")
        i = torch.arange(n, device="cuda")[:, None]
        pos_k, pos_q, seen = j, base + i, j <= base + i
        if par:
            new = torch.zeros(n, n, dtype=torch.bool)
            for a, p in enumerate(par):
                if p >= 0:
                    new[a] = new[p]
                new[a, a] = True
            depth = new.sum(1).cuda() - 1
            seen = torch.cat((torch.ones(n, base, dtype=torch.bool, device="cuda"), new.cuda()), 1)
            pos_q = base + depth[:, None]
            pos_k = torch.cat((j[:base], base + depth))
        if c["window"]:
            seen = seen & ((j < c["sink"]) | (pos_q - pos_k < c["window"]))
        for h in range(c["hkv"]):
            k, v = _exact_rows(st, c, s, length, h)
            for hq in range(h * g, (h + 1) * g):
                z = (st["q"][first:first + n, hq].double() @ k.T) * st["scale"]
                z = z.masked_fill(~seen, -float("inf"))
                lse[first:first + n, hq] = torch.logsumexp(z, 1)
                o[first:first + n, hq] = torch.softmax(z, 1) @ v
        first += n
    return {"o": o, "lse": lse}
