"""What a serving step does around the caches, in fp64 and whole numbers (oracle side).

TEST INFRASTRUCTURE: see the package docstring for who may import this.

The pages give no kernels for these; this module restates the rules that the C ABI's header gives, one sequence,
head or row after the other: pages taken and given back, the norm of a head and its rotation, the router, and the log
probabilities of a row of logits.
"""
from __future__ import annotations

import numpy as np

BAD_ID, NO_PAGES = 0x1, 0x8
F32_MAX = float(np.finfo(np.float32).max)


def plan(n_new, length, held, table, free, n_free, n_pages, page, n_tokens, masks=None):
    """The state and the rows after a step (every array of ft_kv_step by its name) and the status bits."""
    S, stride = table.shape
    table, free = table.copy(), free.copy()
    out = dict(q_start=[0], kv_len=[], slots=np.full(n_tokens, -1, np.int64), positions=np.zeros(n_tokens, np.int64), len_out=[], held_out=[])
    status = 0
    if not 0 <= n_free <= n_pages:
        status |= BAD_ID
        n_free = min(max(n_free, 0), n_pages)
    stack = [int(x) for x in free[:n_free]]
    row, todo = 0, []
    for s in range(S):
        n, l, h = int(n_new[s]), int(length[s]), int(held[s])
        ends, rows = n < 0, max(n, 0)
        after = (0 if ends else l) + rows
        want = -(-after // page)
        fine = 0 <= h <= min(stride, n_pages)
        if not ends:
            fine = (fine and l >= 0 and -(-l // page) <= h and want <= stride and after < 1 << 31 and (masks is None or rows <= 64)
                    and (rows == 0 or row + rows <= n_tokens))
        if not fine:
            status |= BAD_ID
        todo.append((s, row, rows, 0 if ends else l, h, after, want, fine))
        row += rows
        out["q_start"].append(min(row, n_tokens))
    for s, _, _, _, h, _, want, fine in todo:                      # given back first
        if fine and h > want:
            stack += [int(x) for x in table[s, want:h]]
    avail, asked = len(stack), 0
    for s, first, rows, l, h, after, want, fine in todo:
        served = fine
        if fine and want > h:
            asked += want - h
            if asked > avail:
                served = False
                status |= NO_PAGES
            else:
                for j in range(h, want):
                    table[s, j] = stack.pop()
        out["kv_len"].append(after if served else 0)
        out["len_out"].append(after if served else int(length[s]))
        out["held_out"].append(want if served else int(held[s]))
        if not served:
            continue
        for i in range(rows):
            p, t = l + i, first + i
            pg = int(table[s, p // page])
            if 0 <= pg < n_pages:
                out["slots"][t] = pg * page + p % page
            else:
                status |= BAD_ID
            out["positions"][t] = p if masks is None else l + bin(int(masks[t]) & ~(1 << i)).count("1")
    if len(stack) > n_pages:
        status |= BAD_ID
        stack = stack[:n_pages]
    if len(stack) > n_free:
        free[n_free:len(stack)] = stack[n_free:]
    out.update(block_table=table, free_pages=free, n_free_out=len(stack))
    return {k: np.asarray(v) for k, v in out.items()}, status


def turn(x, norm, eps, cos, sin, interleaved):
    """Heads x [n, heads, D] normalised and turned; cos and sin [n, pairs]."""
    x = np.asarray(x, np.float64)
    if norm is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * np.asarray(norm, np.float64)
    out = x.copy()
    for i in range(cos.shape[1]):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + cos.shape[1])
        c, s = (np.asarray(t[:, i], np.float64)[:, None] for t in (cos, sin))
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def _logits(x):
    x = np.asarray(x, np.float64)
    return np.where(np.isnan(x), -np.inf, np.minimum(x, F32_MAX))


def route(x, k, score, bias=None, n_group=1, topk_group=1, group_best=1, renormalise=True, scale=1.0):
    """One row: (ids, weights, the smallest difference of choices that the order rests on)."""
    x = _logits(x)
    E = x.size
    top = x.max()
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "softmax":
            p = np.exp(x - (0.0 if np.isneginf(top) else top))
            sc = p / p.sum() if p.sum() > 0 else p
        else:
            sc = 1.0 / (1.0 + np.exp(-x))
        choice = sc if bias is None else sc + np.asarray(bias, np.float64)
        # without a bias the order is the logits' own, also where their scores are equal in 64 bits
        key = x.copy() if bias is None and (n_group == 1 or group_best == 1) else choice.copy()
    key[np.isneginf(x) | np.isnan(key)] = -np.inf
    if n_group > 1:
        size = E // n_group
        worth = []
        for g in range(n_group):
            best = sorted(key[g * size:(g + 1) * size], reverse=True)[:group_best]
            worth.append(best[0] if len(best) == 1 or np.isneginf(best[1]) else best[0] + best[1])
        for g in sorted(range(n_group), key=lambda g: (-worth[g], g))[topk_group:]:
            key[g * size:(g + 1) * size] = -np.inf
    ids = [e for e in sorted(range(E), key=lambda e: (-key[e], e))[:k] if not np.isneginf(key[e])]
    if renormalise and ids:
        if score == "softmax":
            w = np.exp(x[ids] - x[ids].max())
        else:
            lo = np.minimum(x[ids], 0.0)
            w = np.exp(lo - lo.max()) / (1.0 + np.exp(-np.abs(x[ids])))
        w = w / w.sum()
    else:
        w = sc[ids]
    pad = k - len(ids)
    return np.array(ids + [-1] * pad), np.concatenate([w * float(np.float32(scale)), np.zeros(pad)])


def logprobs(x, token, k, scale=1.0):
    """One row: (logp, entropy, top ids, their log probabilities)."""
    x = _logits(x)
    top = x.max()
    if np.isneginf(top):
        return -np.inf, 0.0, np.full(k, -1), np.full(k, -np.inf)
    y = (x - top) * float(np.float32(scale))
    p = np.exp(y)
    log_sum = np.log(p.sum())
    some = p > 0
    entropy = log_sum - (p[some] * y[some]).sum() / p.sum()
    order = np.lexsort((np.arange(x.size), -x))[:k]
    order = order[~np.isneginf(x[order])]
    ids = np.concatenate([order, np.full(k - order.size, -1, np.int64)]).astype(np.int64)
    return (y[token] - log_sum if 0 <= token < x.size else -np.inf, entropy, ids,
            np.concatenate([y[order] - log_sum, np.full(k - order.size, -np.inf)]))
