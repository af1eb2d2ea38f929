"""The oracle of a serving step against cases worked by hand and closed forms, the calls' refusals, and the binding's
layouts against the C compiler's (no GPU)."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import step as S


@pytest.fixture(scope="module")
def ft():
    import __graft_entry__ as entry
    entry.build()
    import expert_cache_gb300
    return expert_cache_gb300


# ------------------------------------------------------------------------------ oracle

def test_plan_by_hand():
    """Pages of 16.  Sequence 0 goes on over a page's end, 1 ends (pages 7, 2 go back), 2 starts with 20 tokens, 3 rejected
    drafts down to 10 tokens and holds one page too many (5), 4 waits."""
    table = np.array([[4, -1, -1], [7, 2, -1], [-1, -1, -1], [3, 5, -1], [6, -1, -1]])
    out, status = S.plan([3, -1, 20, 1, 0], [15, 20, 0, 10, 16], [1, 2, 0, 2, 1], table, np.array([0, 1, 8, -1, -1, -1, -1, -1, -1]), 3, 9, 16, 30)
    assert status == 0
    # the stack: 0 1 8, then 7 2 (sequence 1), 5 (3); taken from the top: 5 by 0, 2 and 7 by 2
    assert out["block_table"].tolist() == [[4, 5, -1], [7, 2, -1], [2, 7, -1], [3, 5, -1], [6, -1, -1]]
    assert out["n_free_out"] == 3 and out["free_pages"][:3].tolist() == [0, 1, 8]
    assert out["q_start"].tolist() == [0, 3, 3, 23, 24, 24] and out["kv_len"].tolist() == [18, 0, 20, 11, 16]
    assert out["len_out"].tolist() == [18, 0, 20, 11, 16] and out["held_out"].tolist() == [2, 0, 2, 1, 1]
    assert out["slots"][:4].tolist() == [4 * 16 + 15, 5 * 16, 5 * 16 + 1, 2 * 16] and out["slots"][22:].tolist() == [7 * 16 + 3, 3 * 16 + 10] + [-1] * 6
    assert out["positions"][:4].tolist() == [15, 16, 17, 0] and out["positions"][23:].tolist() == [10] + [0] * 6


def test_plan_refuses_in_order():
    table = np.full((4, 4), -1)
    out, status = S.plan([16, 40, 16, 0], [0, 0, 0, 0], [0, 0, 0, 0], table, np.array([3, 1, 2, 0]), 2, 4, 16, 100)
    assert status == S.NO_PAGES
    # one of two pages for sequence 0; 1 wants three more than there are, and 2 asks after it
    assert out["kv_len"].tolist() == [16, 0, 0, 0] and out["held_out"].tolist() == [1, 0, 0, 0] and out["n_free_out"] == 1
    assert out["q_start"].tolist() == [0, 16, 56, 72, 72] and (out["slots"][16:] == -1).all()
    for bad in (dict(length=[-1]), dict(held=[5]), dict(held=[-1]), dict(length=[17], held=[1]), dict(n_new=[101])):
        kw = dict(n_new=[1], length=[0], held=[0], **{}) | bad
        out, status = S.plan(kw["n_new"], kw["length"], kw["held"], np.zeros((1, 4), int), np.arange(9), 5, 9, 16, 100)
        assert status & S.BAD_ID and out["kv_len"].tolist() == [0] and out["len_out"].tolist() == kw["length"]


def test_plan_keeps_every_page_once():
    """Whatever happens, the tables of the served sequences and the stack hold every page exactly once."""
    rng = np.random.default_rng(0)
    S_, n_pages, page, stride = 9, 60, 16, 12
    length, held, table = np.zeros(S_, int), np.zeros(S_, int), np.full((S_, stride), -1)
    free, n_free = rng.permutation(n_pages), n_pages
    for _ in range(200):
        n_new = rng.choice([-1, 0, 1, 1, 5, 33, 90], S_)
        length = np.maximum(0, length - rng.integers(0, 20, S_) * (rng.random(S_) < 0.3))
        out, status = S.plan(n_new, length, held, table, free, n_free, n_pages, page, 2000)
        length, held, table, free, n_free = (out[k] for k in ("len_out", "held_out", "block_table", "free_pages", "n_free_out"))
        n_free = int(n_free)
        have = [int(p) for s in range(S_) for p in table[s, :held[s]]] + [int(p) for p in free[:n_free]]
        assert sorted(have) == list(range(n_pages))             # also where a sequence outgrows its table and is refused
        used = out["slots"][out["slots"] >= 0]
        assert len(set(used.tolist())) == used.size


def test_turn_is_a_rotation_of_the_normalised_head():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 64))
    p = np.array([0.0, 1.0, 500.0])
    f = 1e4 ** (-np.arange(16) / 16)
    cos, sin = np.cos(p[:, None] * f), np.sin(p[:, None] * f)
    for inter in (False, True):
        y = S.turn(x, np.ones(64), 1e-6, cos, sin, inter)
        assert np.allclose((y * y).mean(-1), 1, atol=1e-5)                       # the norm, and rotations keep it
        assert np.allclose(y[0], x[0] / np.sqrt((x[0] ** 2).mean(-1, keepdims=True) + 1e-6))          # position 0
        assert np.allclose(y[..., 32:] * np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6), x[..., 32:])  # dims that do not turn
        # the product of a query and a key depends on the distance only
        a, b = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))

        def at(x, p):
            return S.turn(x, None, 0, np.cos(p * f)[None], np.sin(p * f)[None], inter).ravel()
        assert np.isclose(at(a, 7.0) @ at(b, 3.0), at(a, 104.0) @ at(b, 100.0))
    # the order of a pair's two dims
    one = np.zeros((1, 1, 64))
    one[..., 3] = 1
    y = S.turn(one, None, 0, np.full((1, 16), 0.6), np.full((1, 16), 0.8), False).ravel()
    assert y[3] == 0.6 and y[19] == 0.8 and np.count_nonzero(y) == 2
    y = S.turn(one, None, 0, np.full((1, 16), 0.6), np.full((1, 16), 0.8), True).ravel()
    assert y[3] == 0.6 and y[2] == -0.8 and np.count_nonzero(y) == 2


def test_route_by_hand():
    x = np.log([1.0, 2.0, 4.0, 1.0])                                             # softmax: 1/8, 1/4, 1/2, 1/8
    assert S.route(x, 2, "softmax", renormalise=False)[0].tolist() == [2, 1]
    assert np.allclose(S.route(x, 2, "softmax", renormalise=False)[1], [0.5, 0.25])
    assert np.allclose(S.route(x, 2, "softmax", scale=3.0)[1], [2.0, 1.0])
    assert S.route(x, 4, "softmax")[0].tolist() == [2, 1, 0, 3]                  # equal: the lower index
    ids, w = S.route(x, 2, "softmax", bias=[0.5, 0, 0, 0.5], renormalise=False)
    assert ids.tolist() == [0, 3] and np.allclose(w, [0.125, 0.125])            # the bias chooses, the score weighs
    ids, w = S.route([0.0, np.log(3.0), -np.inf, np.nan], 4, "sigmoid", renormalise=False)
    assert ids.tolist() == [1, 0, -1, -1] and np.allclose(w, [0.75, 0.5, 0, 0])
    # groups (0, 1), (2, 3), (4, 5): best 1 keeps the largest expert's group, best 2 the largest sum's
    y = np.log([0.9, 0.01, 0.6, 0.55, 0.3, 0.2])
    s = np.exp(y) / (1 + np.exp(y))
    assert S.route(y, 2, "sigmoid", n_group=3, topk_group=1, group_best=1)[0].tolist() == [0, 1]
    assert s[2] + s[3] > s[0] + s[1]
    assert S.route(y, 2, "sigmoid", n_group=3, topk_group=1, group_best=2)[0].tolist() == [2, 3]
    assert S.route([-np.inf] * 3, 2, "softmax")[0].tolist() == [-1, -1]
    assert np.allclose(S.route([-800.0, -801.0, -900.0], 2, "sigmoid")[1], [1 / (1 + math.exp(-1)), 1 / (1 + math.e)])


def test_logprobs_closed_forms():
    lp, h, ids, top = S.logprobs(np.zeros(8), 3, 3)
    assert np.isclose(lp, -np.log(8)) and np.isclose(h, np.log(8)) and ids.tolist() == [0, 1, 2] and np.allclose(top, -np.log(8))
    lp, h, ids, top = S.logprobs([np.log(3.0), -np.inf, 0.0, np.nan], 1, 4, 1.0)
    assert np.isneginf(lp) and np.isclose(h, -(0.75 * np.log(0.75) + 0.25 * np.log(0.25)))
    assert ids.tolist() == [0, 2, -1, -1] and np.allclose(top[:2], np.log([0.75, 0.25])) and np.isneginf(top[2:]).all()
    lp, h, ids, _ = S.logprobs([np.inf, 1.0, np.inf], 2, 2)
    assert np.isclose(lp, -np.log(2)) and np.isclose(h, np.log(2)) and ids.tolist() == [0, 2]
    lp, h, ids, top = S.logprobs([-np.inf, np.nan], 0, 1)
    assert np.isneginf(lp) and h == 0 and ids.tolist() == [-1]
    x = np.random.default_rng(0).standard_normal(50)
    for t in (0.5, 1.0, 2.0):
        z = torch.log_softmax(torch.from_numpy(x * t), 0).numpy()
        lp, h, _, top = S.logprobs(x, 7, 50, t)
        assert np.isclose(lp, z[7]) and np.isclose(h, -(np.exp(z) * z).sum()) and np.allclose(top, np.sort(z)[::-1])


# ------------------------------------------------------------------------------ refusals

def refused(ft, f):
    with pytest.raises(ft.FtError) as ei:
        f()
    assert ei.value.status == ft.FT_ERR_ARG


ROUTE = dict(logits=4096, T=4, E=64, k=4, topk_ids=8192, topk_w=8192, stride=64, stream=0)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(E=0), dict(E=4097, stride=5000), dict(k=0), dict(k=33), dict(E=3, k=4), dict(stride=63),
                                 dict(n_group=0), dict(n_group=33, E=66, stride=66), dict(n_group=5), dict(n_group=4, topk_group=0),
                                 dict(n_group=4, topk_group=5), dict(group_best=0), dict(group_best=3), dict(scale=float("inf")),
                                 dict(scale=float("nan")), dict(logits=None), dict(logits=4097), dict(topk_ids=None), dict(topk_w=None),
                                 dict(topk_w=8194), dict(topk_ids=8193), dict(bias=8194), dict(logits=4098, dtype="fp32")])
def test_route_refusals(ft, bad):
    refused(ft, lambda: ft.ft_moe_route(**(ROUTE | bad)))


def test_route_of_nothing(ft):
    ft.ft_moe_route(**(ROUTE | dict(T=0, logits=None, topk_ids=None, topk_w=None)))
    assert ft._f["ft_moe_route"](None, None) == ft.FT_ERR_ARG
    good = [4096, 0, 8192, 8192, 64, 0, 64, 4, 0, 0, 1, 1, 1, 1, 1.0]            # T = 0: only the arguments are looked at
    assert ft._moe_route(ft._ROUTE.pack(*good), None) == ft.FT_OK
    for at, value in ((8, 2), (8, -1), (9, 2), (9, -1), (13, 2), (13, -1)):
        assert ft._moe_route(ft._ROUTE.pack(*good[:at], value, *good[at + 1:]), None) == ft.FT_ERR_ARG
    with pytest.raises(KeyError):
        ft.ft_moe_route(**(ROUTE | dict(score="tanh")))
    with pytest.raises(TypeError, match="stride"):
        ft.ft_moe_route(**(ROUTE | dict(stride=None)))


LOGP = dict(logits=4096, n=4, V=64, tokens=8192, logp=8192, entropy=8192, top_ids=8192, top_logp=8192, k=4, stride=64, stream=0)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(V=0), dict(V=(1 << 30) + 1, stride=1 << 31), dict(k=-1), dict(k=33), dict(V=3), dict(stride=63),
                                 dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(logits=None),
                                 dict(logits=4097), dict(logits=4098, dtype="fp32"), dict(tokens=None), dict(top_ids=None), dict(top_logp=None),
                                 dict(tokens=8193), dict(logp=8194), dict(entropy=8190), dict(top_ids=8194), dict(top_logp=8193)])
def test_logprobs_refusals(ft, bad):
    refused(ft, lambda: ft.ft_logprobs(**(LOGP | bad)))


def test_logprobs_of_nothing(ft):
    ft.ft_logprobs(**(LOGP | dict(n=0, logits=None)))
    assert ft._f["ft_logprobs"](None, None) == ft.FT_ERR_ARG
    with pytest.raises(TypeError, match="stride"):
        ft.ft_logprobs(**(LOGP | dict(stride=None)))


def test_rope_table_refusals(ft):
    good = dict(inv_freq=4096, rope_dim=64, n_positions=10, table=8192, stream=0)
    for bad in (dict(rope_dim=0), dict(rope_dim=3), dict(rope_dim=258), dict(n_positions=0), dict(table=None), dict(inv_freq=None),
                dict(inv_freq=4100), dict(table=8193), dict(mscale=float("nan")), dict(inv_freq=torch.zeros(32)), dict(table=torch.zeros(10, 64).double())):
        refused(ft, lambda: ft.ft_rope_table(**(good | bad)))


def test_calls_without_a_handle(ft):
    z = dict(stream=0)
    refused(ft, lambda: ft.ft_kv_plan(None, 0, 0, 0, 0, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, **z))
    refused(ft, lambda: ft.ft_kv_append_rotated(None, 0, 0, 0, 0, 0, 1, 0, 0, 0, 0, 0, q_stride=64, k_stride=64, v_stride=64, q_out_stride=64, **z))


# ------------------------------------------------------------------------------ binding

def test_binding_matches_the_header(ft, tmp_path):
    """The layouts that the binding packs are the C compiler's."""
    structs = {
        "ft_kv_step": (ft._KV_STEP, "n_new len held n_free block_table free_pages tree_mask q_start kv_len slots positions len_out held_out "
                                    "n_free_out n_seqs table_stride n_tokens"),
        "ft_kv_qkv": (ft._KV_QKV, "q k v q_out k_out q_stride k_stride v_stride q_out_stride k_out_stride q_norm k_norm rope positions slots layer n "
                                  "rope_dim n_positions interleaved eps"),
        "ft_route": (ft._ROUTE, "logits bias topk_ids topk_w stride T E k dtype score n_group topk_group group_best renormalise scale"),
        "ft_logprob": (ft._LOGPROB, "logits tokens logp entropy top_ids top_logp stride n V k dtype scale")}
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ft.h"\nint main(void) {\n' + "".join(
        f'    printf("%zu ", sizeof({t}));\n' + "".join(f'    printf("%zu ", offsetof({t}, {f}));\n' for f in fields.split())
        for t, (_, fields) in structs.items()) + "    return 0;\n}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for name, (packed, fields) in structs.items():
        want.append(packed.size)
        kinds = "".join(int(n or 1) * c for n, c in __import__("re").findall(r"(\d*)([Pqif])", packed.format.replace("4x", "")))
        assert len(kinds) == len(fields.split()), name
        at = 0
        for c in kinds:
            want.append(at)
            at += 8 if c in "Pq" else 4
    assert got == want
    assert ctypes.sizeof(ctypes.c_void_p) == 8


@pytest.fixture
def calls(ft, monkeypatch):
    ft._load_types()
    got = {}

    def catch(name):
        def call(*args):
            got[name] = args
            return 0
        return call

    for name in ("kv_plan", "kv_append_rotated", "moe_route", "logprobs"):
        monkeypatch.setattr(ft, f"_{name}", catch(name))
    return got


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def misread(ft, what, f):
    with pytest.raises(ft.FtError, match=what) as ei:
        f()
    assert ei.value.status == ft.FT_ERR_ARG


def test_plan_looks_at_its_arrays(ft, calls):
    names = ("n_new", "len", "held", "n_free", "block_table", "free_pages", "tree_mask", "q_start", "kv_len", "slots", "positions", "len_out", "held_out",
             "n_free_out")
    good = dict(n_new=i32(3), len=i32(3), held=i32(3), block_table=i32(3, 5), table_stride=5, free_pages=i32(9), n_free=i32(1), n_seqs=3, n_tokens=7,
                q_start=i32(4), kv_len=i32(3), slots=i32(7), len_out=i32(3), held_out=i32(3), n_free_out=i32(1), positions=i32(7),
                tree_mask=torch.zeros(7, dtype=torch.int64), stream=0)
    ft.ft_kv_plan(7, **good)
    assert ft._KV_STEP.unpack(calls["kv_plan"][1]) == (*(good[n].data_ptr() for n in names), 3, 5, 7)
    wide = i32(3, 9)[:, :5]
    ft.ft_kv_plan(7, **(good | dict(block_table=wide, table_stride=9, positions=None, tree_mask=None)))
    got = ft._KV_STEP.unpack(calls.pop("kv_plan")[1])
    assert got[4] == wide.data_ptr() and got[6] == got[10] == 0 and got[15] == 9
    ft.ft_kv_plan(7, **(good | dict(tree_mask=torch.zeros(7, dtype=torch.uint64))))
    calls.clear()
    for n in names:
        for t in (good[n].float(), torch.zeros(14, dtype=good[n].dtype)[::2]):
            if n == "block_table" and t.dtype is torch.int32:
                t = i32(3, 10)[:, ::2]
            misread(ft, f"plan: {n}", lambda: ft.ft_kv_plan(7, **(good | {n: t})))
    assert not calls


def test_append_rotated_looks_at_its_arrays(ft, calls):
    wide = bf16(5, 8 * 64)
    good = dict(layer=1, q=wide[:, :256], k=wide[:, 256:384], v=wide[:, 384:], slots=i32(5), n=5, q_out=bf16(5, 4, 64), positions=i32(5),
                rope=torch.zeros(9, 32), rope_dim=32, n_positions=9, k_out=bf16(5, 2, 64), q_norm=torch.zeros(64), k_norm=torch.zeros(64), stream=0)
    ft.ft_kv_append_rotated(7, **good)
    got = ft._KV_QKV.unpack(calls["kv_append_rotated"][1])
    assert got[:10] == (*(good[n].data_ptr() for n in ("q", "k", "v", "q_out", "k_out")), 512, 512, 512, 256, 128)
    assert got[10:15] == tuple(good[n].data_ptr() for n in ("q_norm", "k_norm", "rope", "positions", "slots"))
    assert got[15:20] == (1, 5, 32, 9, 0) and abs(got[20] - 1e-6) < 1e-12
    ft.ft_kv_append_rotated(7, **(good | dict(k_out=None, q_norm=None, k_norm=None, rope=None, positions=None, rope_dim=0, interleaved=True)))
    got = ft._KV_QKV.unpack(calls["kv_append_rotated"][1])
    assert got[4] == got[9] == got[10] == got[11] == got[12] == got[13] == 0 and got[17] == 0 and got[19] == 1
    one = {x: good[x][:1] for x in ("q", "k", "v", "q_out", "k_out", "slots", "positions")}
    ft.ft_kv_append_rotated(7, **(good | one | dict(n=1, q_out=bf16(64, 4).t().reshape(1, 64, 4).transpose(1, 2).contiguous())))
    assert all(x % 8 == 0 and x >= 256 for x in ft._KV_QKV.unpack(calls["kv_append_rotated"][1])[5:10])
    with pytest.raises(TypeError, match="stride"):
        ft.ft_kv_append_rotated(7, **(good | dict(q=good["q"].data_ptr())))
    calls.clear()
    for n in ("q", "k", "v", "q_out", "k_out"):
        for t in (good[n].float(), bf16(5, 4, 2, 64)[:, :, 0], bf16(5, 64, 2).transpose(1, 2)):
            misread(ft, f"append_rotated: {n}", lambda: ft.ft_kv_append_rotated(7, **(good | {n: t})))
        misread(ft, f"append_rotated: {n}", lambda: ft.ft_kv_append_rotated(7, **(good | one | dict(n=1) | {n: bf16(1, 4, 2, 64)[:, :, 0]})))
    for n in ("slots", "positions", "rope", "q_norm", "k_norm"):
        for t in (good[n].double(), good[n].repeat(2, *[1] * (good[n].dim() - 1))[::2]):
            misread(ft, f"append_rotated: {n}", lambda: ft.ft_kv_append_rotated(7, **(good | {n: t})))
    assert not calls


def test_route_and_logprobs_look_at_their_arrays(ft, calls):
    wide = torch.zeros(6, 80)[:, :64]
    good = dict(logits=wide, T=6, E=64, k=4, topk_ids=i32(6, 4), topk_w=torch.zeros(6, 4), bias=torch.zeros(64), stream=0)
    ft.ft_moe_route(**good)
    got = ft._ROUTE.unpack(calls["moe_route"][0])
    assert got == (wide.data_ptr(), good["bias"].data_ptr(), good["topk_ids"].data_ptr(), good["topk_w"].data_ptr(), 80, 6, 64, 4, ft.FT_DTYPE_F32,
                   ft.FT_ROUTE_SOFTMAX, 1, 1, 1, 1, 1.0)
    ft.ft_moe_route(**(good | dict(logits=bf16(1, 64), T=1, score="sigmoid", bias=None, renormalise=False)))
    got = ft._ROUTE.unpack(calls.pop("moe_route")[0])
    assert got[1] == 0 and got[4:15] == (64, 1, 64, 4, ft.FT_DTYPE_BF16, ft.FT_ROUTE_SIGMOID, 1, 1, 1, 0, 1.0)
    one = torch.zeros(8, 64)[:1].as_strided((1, 64), (0, 1))                     # the stride of a single row says nothing
    ft.ft_moe_route(**(good | dict(logits=one, T=1)))
    assert ft._ROUTE.unpack(calls.pop("moe_route")[0])[4] == 64
    ft.ft_moe_route(**(good | dict(logits=torch.zeros(6, 100))))                 # more columns than experts
    assert ft._ROUTE.unpack(calls.pop("moe_route")[0])[4] == 100
    for n, ts in dict(logits=[torch.zeros(3, 2, 64), torch.zeros(64), torch.zeros(()), wide.half(), wide.double(), torch.zeros(64, 6).t(), torch.zeros(6, 128)[:, ::2]], topk_ids=[i32(6, 8)[:, ::2], i32(6, 4).long()],
                      topk_w=[bf16(6, 4), torch.zeros(4, 6).t()], bias=[bf16(64), torch.zeros(128)[::2]]).items():
        for t in ts:
            misread(ft, f"route: {n}", lambda: ft.ft_moe_route(**(good | {n: t})))
    good = dict(logits=bf16(6, 70)[:, :64], n=6, V=64, tokens=i32(6), logp=torch.zeros(6), entropy=torch.zeros(6), top_ids=i32(6, 4),
                top_logp=torch.zeros(6, 4), k=4, scale=0.5, stream=0)
    ft.ft_logprobs(**good)
    got = ft._LOGPROB.unpack(calls.pop("logprobs")[0])
    assert got == (*(good[n].data_ptr() for n in ("logits", "tokens", "logp", "entropy", "top_ids", "top_logp")), 70, 6, 64, 4, ft.FT_DTYPE_BF16, 0.5)
    for n, ts in dict(logits=[torch.zeros(3, 2, 64), torch.zeros(64), torch.zeros(()), wide.half(), torch.zeros(64, 6).t()], tokens=[i32(12)[::2], i32(6).long()], logp=[bf16(6)], entropy=[torch.zeros(12)[::2]],
                      top_ids=[i32(6, 4).long()], top_logp=[torch.zeros(4, 6).t()]).items():
        for t in ts:
            misread(ft, f"logprobs: {n}", lambda: ft.ft_logprobs(**(good | {n: t})))
    assert not calls
