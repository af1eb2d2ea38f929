"""Quantised key/value cache and attention over it, in fp64 (oracle side).

TEST INFRASTRUCTURE: see the package docstring for who may import this.

The pages give no kernel for the attention layers; this module restates the rules that
the C ABI's header gives: the two cache formats (the quantisers' fp32 IEEE steps, so a
device that does the same steps is bit-exact), the place of every byte in a tile, and
masked softmax attention with the keys that a row sees taken from the definition.
"""
from __future__ import annotations

import numpy as np

from .formats import e2m1_decode, e2m1_encode, e4m3_decode, e4m3_encode_unsigned

F32 = np.float32
E2M1_MAX, E4M3_MAX = 6.0, 448.0


def quantise(x, fmt: str, st: float):
    """x [.., D] -> (codes uint8 [.., D], scale bytes uint8 [.., D/16] or None).
    NaN counts as 0, infinities saturate."""
    x = np.asarray(x, F32)
    st = F32(st)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if fmt == "fp8":
            y = np.nan_to_num((x / st).astype(F32), nan=0.0, posinf=E4M3_MAX, neginf=-E4M3_MAX)
            mag = e4m3_encode_unsigned(np.abs(y))
            return (mag | (((y < 0) & (mag != 0)).astype(np.uint8) << 7)).astype(np.uint8), None
        b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
        amax = np.max(np.where(np.isnan(b), F32(0), np.abs(b)), axis=-1).astype(F32)
        t = ((amax / F32(6.0)).astype(F32) / st).astype(F32)
        sc = e4m3_encode_unsigned(np.minimum(t, F32(E4M3_MAX)))
        den = (e4m3_decode(sc).astype(F32) * st).astype(F32)[..., None]
        y = np.where(den == 0, F32(0), (b / np.where(den == 0, F32(1), den)).astype(F32))
        y = np.nan_to_num(y, nan=0.0, posinf=E2M1_MAX, neginf=-E2M1_MAX)
    sc = np.where(den[..., 0] == 0, np.uint8(0), sc)
    return e2m1_encode(y).reshape(x.shape), sc


def values(codes, scales, fmt: str, st: float) -> np.ndarray:
    """fp64 values of the codes, exact up to the product with the fp32 tensor scale."""
    if fmt == "fp8":
        return e4m3_decode(codes) * float(F32(st))
    v = e2m1_decode(codes).reshape(*codes.shape[:-1], codes.shape[-1] // 16, 16) * e4m3_decode(scales)[..., None]
    return v.reshape(codes.shape) * float(F32(st))


def tile_bytes(D: int, fmt: str) -> int:
    return 32 * D if fmt == "fp8" else 18 * D


def code_place(r: int, d: int, D: int, fmt: str, value: bool) -> tuple[int, int]:
    """(byte of the tile, nibble) of dim d of token r's key or value."""
    if value:
        lane, at = 4 * (d // (D // 8)) + (r % 8) // 2, (2 * (r // 8) + r % 2) * (D // 8) + d % (D // 8)
    else:
        lane, at = 4 * (r % 8) + d // (D // 4), (r // 8) * (D // 4) + d % (D // 4)
    byte, nib = (at, 0) if fmt == "fp8" else (at // 2, at % 2)
    first = (16 * D if fmt == "fp8" else 8 * D) if value else 0
    return first + byte // 16 * 512 + lane * 16 + byte % 16, nib


def scale_place(r: int, b: int, D: int, value: bool) -> int:
    """Byte of the tile of block b's scale (NVFP4)."""
    if value:
        return 17 * D + (4 * b + (r % 8) // 2) * 4 + 2 * (r // 8) + r % 2
    return 16 * D + (4 * (r % 8) + b // (D // 64)) * (D // 32) + (r // 8) * (D // 64) + b % (D // 64)


def seen(n: int, kv_len: int, window: int = 0, n_sink: int = 0, masks=None) -> np.ndarray:
    """bool [n, kv_len]: the keys that each new token sees."""
    base = kv_len - n
    out = np.zeros((n, kv_len), bool)

    def pos(j):
        if masks is None or j < base:
            return j
        m = int(masks[j - base]) & ~(1 << (j - base))
        return base + bin(m).count("1")

    for i in range(n):
        p = pos(base + i) if base + i >= 0 or masks is not None else base + i
        for j in range(kv_len):
            if masks is None:
                ok = j <= base + i
            else:
                ok = j < base or (j - base < 64 and (int(masks[i]) >> (j - base)) & 1 == 1)
            if ok and window > 0:
                ok = j < n_sink or p - pos(j) < window
            out[i, j] = ok
    return out


def attention(q, k, v, vis, scale: float):
    """q [n, D], k and v [len, D], vis [n, len] -> (o [n, D], lse [n], sum_j p_j |v_j| [n, D],
    max_j sum_d |q_d k_jd| [n]) in fp64; the last two are what error bounds are made of."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    n = q.shape[0]
    o, av = np.zeros((n, v.shape[1])), np.zeros((n, v.shape[1]))
    lse, mag = np.full(n, -np.inf), np.zeros(n)
    for i in range(n):
        js = np.flatnonzero(vis[i])
        if js.size == 0:
            continue
        z = k[js] @ q[i] * scale
        top = z.max()
        p = np.exp(z - top)
        lse[i] = top + np.log(p.sum())
        p /= p.sum()
        o[i], av[i] = p @ v[js], p @ np.abs(v[js])
        mag[i] = (np.abs(k[js]) @ np.abs(q[i])).max()
    return o, lse, av, mag
