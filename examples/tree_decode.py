"""A small decoder whose layers keep their keys and values in a quantised cache and their experts in the
expert cache, run three ways over the same text: one token per step, the prompt in chunks, and trees
of drafted tokens verified in one step.

    python examples/tree_decode.py [--fmt nvfp4|fp8] [--tokens N]

Every layer call is the order a serving loop has: ft_kv_append stores the step's new tokens,
ft_kv_attention reads the cache (the odd layers through a sliding window with two sink tokens),
ft_moe_decode adds the routed experts.  Weights are random; a drafter is stood in for by the tokens
of a first run among wrong ones.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import expert_cache_gb300 as ft  # noqa: E402
from expert_cache_gb300.workloads import SHAPES, build_pool  # noqa: E402

PAGE, VOCAB, BATCH = 16, 64, 32
WINDOW, SINKS = 24, 2


class Decoder:
    """One sequence over both caches."""

    def __init__(self, fmt="nvfp4", head_dim=64, n_q_heads=8, n_kv_heads=2, most=1024, seed=0):
        s = self.shape = SHAPES["tiny"]
        self.head_dim, self.n_q, self.n_kv = head_dim, n_q_heads, n_kv_heads
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols, scale=1.0):
            return (torch.randn(rows, cols, generator=g) * scale * rows ** -0.5).to(torch.bfloat16).cuda()

        self.embed = weight(VOCAB, s.H, VOCAB ** 0.5)
        self.place = weight(most, s.H, 0.5 * most ** 0.5)
        self.layers = [dict(q=weight(s.H, n_q_heads * head_dim), k=weight(s.H, n_kv_heads * head_dim),
                            v=weight(s.H, n_kv_heads * head_dim), o=weight(n_q_heads * head_dim, s.H),
                            r=weight(s.H, s.E)) for _ in range(s.L)]
        self.head = weight(s.H, VOCAB)
        # scales of the stored tensors: normalised activations through these weights stay within +-6
        self.kv = ft.KVCache(s.L, most // PAGE, PAGE, n_kv_heads, head_dim, n_q_heads, 1, fmt, 6 / 448, 6 / 448)
        self.pool = build_pool(seed, s.L, s.E, s.H, s.I)
        self.experts = ft.ExpertCache(s.L, s.E, s.H, s.I, s.k, BATCH, s.L * s.E, self.pool.ptr)
        # the sequence's pages in any order; a cached token's slot is its page times the page size plus its place
        self.table = torch.randperm(most // PAGE, generator=g).to(torch.int32).cuda()[None]
        self.len = 0

    def slots(self, at):
        return (self.table[0, at // PAGE] * PAGE + at % PAGE).to(torch.int32)

    def step(self, tokens, places, masks=None):
        """Logits of new tokens that follow the cached ones; masks: their ancestors and themselves (a tree of
        drafted tokens), else each sees those before it.  They are cached when the call returns; returns also
        their keys and values by layer."""
        s, n = self.shape, len(tokens)
        x = (self.embed[tokens] + self.place[places]).float()
        slots = self.slots(torch.arange(self.len, self.len + n, device="cuda"))
        start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        length = torch.tensor([self.len + n], dtype=torch.int32, device="cuda")
        tree = None if masks is None else torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).cuda()
        y = torch.empty(n, s.H, device="cuda")
        deferred = torch.empty(n, s.k, dtype=torch.int32, device="cuda")
        kept = []
        for l, w in enumerate(self.layers):
            h = torch.nn.functional.normalize(x, dim=-1).mul(s.H ** 0.5).to(torch.bfloat16)
            q = (h @ w["q"]).view(n, self.n_q, self.head_dim)
            k, v = ((h @ w[i]).view(n, self.n_kv, self.head_dim) for i in "kv")
            ft.ft_kv_append(self.kv.handle, l, k, v, slots, n)
            o = torch.empty_like(q)
            ft.ft_kv_attention(self.kv.handle, l, q, start, length, self.table, self.table.stride(0), 1, n, n, o,
                               tree_mask=tree, window=WINDOW if l % 2 else 0, n_sink=SINKS if l % 2 else 0,
                               sm_scale=self.head_dim ** -0.5)
            x = x + (o.view(n, -1) @ w["o"]).float()
            h = torch.nn.functional.normalize(x, dim=-1).mul(s.H ** 0.5).to(torch.bfloat16)
            gate, ids = torch.topk((h @ w["r"]).float(), s.k)
            ft.ft_moe_decode(self.experts.handle, l, h, ids.to(torch.int32), torch.softmax(gate, -1), n, s.k, y, deferred)
            x = x + y
            kept.append((k, v))
        self.len += n
        return (torch.nn.functional.normalize(x, dim=-1).mul(s.H ** 0.5).to(torch.bfloat16) @ self.head).float(), kept

    def chunk(self, tokens):
        """Logits after each token of a prompt's chunk (at most 32)."""
        return self.step(tokens, list(range(self.len, self.len + len(tokens))))[0]

    def keep(self, n_new, path, kept):
        """Of the last n_new cached tokens, only those of the path stay, moved to the front of their range."""
        base = self.len - n_new
        pick = torch.tensor(path, device="cuda")
        slots = self.slots(torch.arange(base, base + len(path), device="cuda"))
        for l, (k, v) in enumerate(kept):
            ft.ft_kv_append(self.kv.handle, l, k[pick], v[pick], slots, len(path))
        self.len = base + len(path)

    def verify(self, last, drafts):
        """One step over a tree: the last token and drafted ones, (token, parent's index; 0 is the last
        token).  Returns the tokens that greedy decoding would emit, and the logits along its path."""
        tokens, masks, places = [last], [1], [self.len]
        for j, (token, parent) in enumerate(drafts, 1):
            tokens.append(token)
            masks.append(masks[parent] | 1 << j)
            places.append(places[parent] + 1)
        logits, kept = self.step(tokens, places, masks)
        best = logits.argmax(-1).tolist()
        path = [0]
        while True:
            follow = [j for j, (token, parent) in enumerate(drafts, 1) if parent == path[-1] and token == best[path[-1]]]
            if not follow:
                break
            path.append(follow[0])
        self.keep(len(tokens), path, kept)
        return [best[j] for j in path], logits[path]

    def close(self):
        torch.cuda.synchronize()
        if ft.ft_kv_status(self.kv.handle):
            raise RuntimeError("the key/value cache reports an error")
        self.kv.close()
        self.experts.close()


def plain(prompt, n, **kw):
    """n tokens after the prompt, one per step, and the logits that gave them."""
    d = Decoder(**kw)
    out = [d.chunk([t]) for t in prompt][-1:]
    tokens = [int(out[0][-1].argmax())]
    while len(tokens) < n:
        out.append(d.chunk([tokens[-1]]))
        tokens.append(int(out[-1][-1].argmax()))
    d.close()
    return tokens, torch.cat(out)


def by_trees(prompt, n, guess, rng, depth=6, **kw):
    """The same by chunks and trees: a branch of the guess's next tokens, wrong ones hanging from it.
    Returns the tokens, their logits and the number of verifying steps."""
    d = Decoder(**kw)
    for at in range(0, len(prompt), BATCH):
        logits = d.chunk(prompt[at:at + BATCH])
    tokens, out, steps = [int(logits[-1].argmax())], [logits[-1:]], 0
    while len(tokens) < n:
        drafts, parent = [], 0
        for t in guess[len(tokens):len(tokens) + depth]:
            for _ in range(int(rng.integers(0, 4))):
                drafts.append(((t + int(rng.integers(1, VOCAB))) % VOCAB, parent))
            drafts.append((t, parent))
            parent = len(drafts)
        got, logits = d.verify(tokens[-1], drafts)
        tokens += got
        out.append(logits)
        steps += 1
    d.close()
    return tokens[:n], torch.cat(out)[:n], steps


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--fmt", default="nvfp4", choices=["nvfp4", "fp8"])
    p.add_argument("--tokens", type=int, default=96)
    args = p.parse_args()
    rng = np.random.default_rng(0)
    prompt = rng.integers(0, VOCAB, 50).tolist()
    a, la = plain(prompt, args.tokens, fmt=args.fmt)
    b, lb, steps = by_trees(prompt, args.tokens, a, rng, fmt=args.fmt)
    same = next((i for i in range(len(a)) if a[i] != b[i]), len(a))
    print(f"{args.tokens} tokens: {args.tokens} steps one by one, {steps} steps by trees; the same up to token {same}; "
          f"logits differ by {((la - lb)[:same].norm() / la[:same].norm()).item():.1e} of their norm")


if __name__ == "__main__":
    main()
