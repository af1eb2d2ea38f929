"""Pins for oracle.kv: the cache's formats, its tile layout, who sees whom, attention.
Also the host-side refusals of the cache's C ABI (nothing here reaches a CUDA call)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import kv as K


@pytest.mark.parametrize("st", [1.0, 0.5, 0.0371])
def test_nvfp4_is_nearest_under_its_scale(st):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 64)) * np.exp(rng.standard_normal((40, 1)))).astype(np.float32)
    codes, sc = K.quantise(x, "nvfp4", st)
    val = K.values(codes, sc, "nvfp4", st).reshape(40, 4, 16)
    grid = np.concatenate([F.e2m1_decode(np.arange(8)), -F.e2m1_decode(np.arange(8))])
    den = F.e4m3_decode(sc) * float(np.float32(st))
    best = np.abs(x.reshape(40, 4, 16, 1) - den[..., None, None] * grid).min(-1)
    # nearest up to the fp32 rounding of the quotient
    assert np.all(np.abs(x.reshape(40, 4, 16) - val) <= best + 1e-6 * np.abs(x.reshape(40, 4, 16)))


def test_fp8_matches_torch_rounding_and_non_finite_rules():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((64, 32)) * 30).astype(np.float32)
    codes, none = K.quantise(x, "fp8", 0.25)
    assert none is None
    y = torch.from_numpy(x / np.float32(0.25)).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert np.array_equal(K.values(codes, None, "fp8", 0.25), y.double().numpy() * 0.25)
    bad = np.array([[np.nan, np.inf, -np.inf, -0.0] + [1.0] * 12], np.float32)
    assert K.values(K.quantise(bad, "fp8", 1.0)[0], None, "fp8", 1.0)[0, :4].tolist() == [0, 448, -448, 0]
    codes, sc = K.quantise(bad, "nvfp4", 1.0)
    assert K.values(codes, sc, "nvfp4", 1.0)[0, :4].tolist() == [0, 2688, -2688, 0]
    codes, sc = K.quantise(np.zeros((1, 16), np.float32), "nvfp4", 1.0)
    assert not codes.any() and not sc.any()


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tile_layout_is_a_bijection(D, fmt):
    places = [K.code_place(r, d, D, fmt, v) for v in (False, True) for r in range(16) for d in range(D)]
    assert len(set(places)) == len(places)
    used = {b for b, _ in places}
    if fmt == "nvfp4":
        scales = [K.scale_place(r, b, D, v) for v in (False, True) for r in range(16) for b in range(D // 16)]
        assert len(set(scales)) == len(scales) and not used & set(scales)
        used |= set(scales)
    assert used == set(range(K.tile_bytes(D, fmt)))


def test_seen_by_hand():
    # causal: 2 new of 4
    assert K.seen(2, 4).tolist() == [[True, True, True, False], [True] * 4]
    # fewer cached than new: the first rows see nothing
    assert K.seen(3, 1).tolist() == [[False], [False], [True]]
    # window 2 and one sink
    assert K.seen(1, 5, window=2, n_sink=1).tolist() == [[True, False, False, True, True]]
    # a tree of three: 0 and 1 under the context, 2 under 0; row 1 empty but for the context
    m = [0b001, 0b010, 0b101]
    assert K.seen(3, 5, masks=m).tolist() == [[True, True, True, False, False], [True, True, False, True, False],
                                              [True, True, True, False, True]]
    # 2 stands at depth 1: with a window of 2 it sees its parent and itself only
    assert K.seen(3, 5, window=2, masks=m)[2].tolist() == [False, False, True, False, True]
    assert K.seen(2, 2, masks=[0, 0]).any() == False  # noqa: E712


def test_attention_against_torch():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, 64, generator=g, dtype=torch.float64) for n in (3, 9, 9))
    vis = K.seen(3, 9)
    o, lse, av, mag = K.attention(q, k, v, vis, 0.3)
    z = (q @ k.T * 0.3).masked_fill(~torch.from_numpy(vis), -float("inf"))
    assert np.allclose(o, torch.softmax(z, 1) @ v, atol=1e-13)
    assert np.allclose(lse, torch.logsumexp(z, 1), atol=1e-13)
    assert np.all(av >= np.abs(o) - 1e-12) and np.all(mag * 0.3 >= z[:, 0].abs().numpy() - 1e-12)
    o, lse, _, _ = K.attention(q, k, v, np.zeros((3, 9), bool), 0.3)
    assert not o.any() and np.all(np.isneginf(lse))


# ------------------------------------------------------------------ refusals without a GPU

@pytest.fixture(scope="module")
def ft():
    import __graft_entry__ as entry
    entry.build()
    import expert_cache_gb300
    return expert_cache_gb300


def _desc(ft, **kw):
    base = dict(L=2, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, n_q_heads=4, max_seqs=3, format=0,
                k_scale=1.0, v_scale=1.0)
    base.update(kw)
    return ft.FtKvDesc(*base.values(), None, None)


def test_required_sizes(ft):
    for fmt, name in ((ft.FT_KV_NVFP4, "nvfp4"), (ft.FT_KV_FP8, "fp8")):
        for D in (64, 128, 256):
            for page in (16, 32, 64, 128, 256):
                pool, ws = ft.ft_kv_required_sizes(_desc(ft, head_dim=D, page_size=page, format=fmt))
                assert pool == 2 * 8 * 2 * (page // 16) * K.tile_bytes(D, name) and ws > 0 and ws % 256 == 0


@pytest.mark.parametrize("bad", [dict(L=0), dict(n_pages=0), dict(page_size=24), dict(page_size=8), dict(page_size=512),
                                 dict(n_kv_heads=0), dict(head_dim=96), dict(head_dim=32), dict(n_q_heads=3),
                                 dict(n_q_heads=0), dict(max_seqs=0), dict(max_seqs=5000), dict(format=2),
                                 dict(k_scale=0.0), dict(v_scale=-1.0), dict(k_scale=float("nan")),
                                 dict(v_scale=float("inf")), dict(n_pages=1 << 27, page_size=16)])
def test_descriptor_refusals(ft, bad):
    with pytest.raises(ft.FtError) as ei:
        ft.ft_kv_required_sizes(_desc(ft, **bad))
    assert ei.value.status == ft.FT_ERR_ARG


def test_create_and_calls_without_memory(ft):
    with pytest.raises(ft.FtError) as ei:
        ft.ft_kv_create(_desc(ft))
    assert ei.value.status == ft.FT_ERR_ARG
    for call in (lambda: ft.ft_kv_append(None, 0, 0, 0, 0, 1, 128, 128, stream=0),
                 lambda: ft.ft_kv_read(None, 0, 0, 1, 0, 0, stream=0),
                 lambda: ft.ft_kv_attention(None, 0, 0, 0, 0, 0, 1, 1, 1, 1, 0, q_stride=256, o_stride=256, stream=0)):
        with pytest.raises(ft.FtError) as ei:
            call()
        assert ei.value.status == ft.FT_ERR_ARG
    assert ctypes.sizeof(ft.FtKvDesc) == 56


def test_binding_matches_the_header(ft, tmp_path):
    """The layout that the binding packs is the C compiler's."""
    fields = ["q", "o", "lse", "q_stride", "o_stride", "q_start", "kv_len", "block_table", "tree_mask", "layer",
              "table_stride", "n_seqs", "n_tokens", "max_q", "window", "n_sink", "sm_scale"]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ft.h"\nint main(void) {\n'
                   '    printf("%zu %zu", sizeof(ft_kv_desc), sizeof(ft_kv_attn));\n' +
                   "".join(f'    printf(" %zu", offsetof(ft_kv_attn, {f}));\n' for f in fields) + "    return 0;\n}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()]
    at, want = 0, []
    for size in [8] * 9 + [4] * 8:
        want.append(at)
        at += size
    assert got == [ctypes.sizeof(ft.FtKvDesc), ft._KV_ATTN.size] + want
    one = ft._KV_ATTN.unpack(ft._KV_ATTN.pack(*range(1, 17), 0.5))
    assert one == (*range(1, 17), 0.5)


def test_pools_past_the_address_space_are_refused(ft):
    """Layers whose bytes together pass 2^64 would come out as a small pool."""
    wide = dict(n_pages=(1 << 27) - 1, n_kv_heads=1024, n_q_heads=1024, head_dim=256, format=ft.FT_KV_FP8)
    pool, _ = ft.ft_kv_required_sizes(_desc(ft, **wide, L=1 << 12))
    assert pool == (1 << 12) * ((1 << 27) - 1) * 1024 * K.tile_bytes(256, "fp8")
    for L in (1 << 13, 1 << 14, (1 << 14) + 1, (1 << 31) - 1):
        if L * ((1 << 27) - 1) * 1024 * K.tile_bytes(256, "fp8") < 1 << 63:
            continue
        with pytest.raises(ft.FtError) as ei:
            ft.ft_kv_required_sizes(_desc(ft, **wide, L=L))
        assert ei.value.status == ft.FT_ERR_ARG
