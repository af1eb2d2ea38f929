"""A serving step's calls together, as they would be used: planned, turned, stored, attended, routed, computed, scored.

Attention's bound is the one of its own tests (head of test_gpu_kv.py), with q as the call wrote it; the experts' is the
stated parity tolerance."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import kv as K
from oracle import step as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ft():
    import __graft_entry__ as entry
    entry.build()
    import expert_cache_gb300
    return expert_cache_gb300


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tree_decode", os.path.join(os.path.dirname(os.path.dirname(
        os.path.abspath(__file__))), "examples", "tree_decode.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_served_decoder(ft, example, fmt, seed):
    """The example, by single tokens and by chunks and verified trees: the two ways agree as far as the plain one's do
    (test_layers_together) until they part at a tie of two tokens' bf16 logits, which may come at any token."""
    ex, rng = example, np.random.default_rng(seed)
    prompt = rng.integers(0, ex.VOCAB, 45).tolist()
    a, la = ex.plain(prompt, 60, ex.Served, fmt=fmt)
    b, lb, steps = ex.by_trees(prompt, 60, a, rng, cls=ex.Served, fmt=fmt)
    same = next((i for i in range(60) if a[i] != b[i]), 60)
    gap = la.topk(2).values
    assert same == 60 or (gap[same, 0] - gap[same, 1]) < 2.0 ** -4 * la[same].abs().max(), "a token that is no tie"
    assert same >= 1 and steps <= -(-same // 7) + 60 - same + 1
    assert ((la - lb)[:same].norm() / la[:same].norm()).item() < 2.0 ** -4
    assert a == la.argmax(-1).tolist()


class Step:
    """Three sequences of one attention layer and one of experts, over fixed buffers: a step by a call of each."""

    HQ, HKV, D, ROPE, PAGE, PLACES, V = 8, 2, 64, 32, 16, 512, 1000

    def __init__(self, ft, n_tokens, pool, shape, seed=0):
        self.ft, self.n, self.shape = ft, n_tokens, shape
        g = torch.Generator().manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.kv = ft.KVCache(1, 40, self.PAGE, self.HKV, self.D, self.HQ, 3, "nvfp4", 0.0625, 0.0625)
        self.experts = ft.ExpertCache(shape.L, shape.E, shape.H, shape.I, shape.k, 32, shape.L * shape.E, pool.ptr)
        self.t = dict(n_new=torch.zeros(3, **i32), len=torch.zeros(3, **i32), held=torch.zeros(3, **i32), table=torch.zeros(3, 30, **i32),
                      free=torch.randperm(40, generator=g).to(torch.int32).cuda(), n_free=torch.tensor([40], **i32), start=torch.zeros(4, **i32),
                      kv_len=torch.zeros(3, **i32), slots=torch.zeros(n_tokens, **i32), at=torch.zeros(n_tokens, **i32),
                      ids=torch.zeros(n_tokens, shape.k, **i32), deferred=torch.zeros(n_tokens, shape.k, **i32), tops=torch.zeros(n_tokens, 4, **i32),
                      tokens=torch.zeros(n_tokens, **i32))
        self.x = {name: torch.zeros(n_tokens, width, dtype=torch.bfloat16, device="cuda") for name, width in (
            ("qkv", (self.HQ + 2 * self.HKV) * self.D), ("h", shape.H), ("router", shape.E), ("logits", self.V))}
        self.q, self.o = (torch.zeros(n_tokens, self.HQ, self.D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.k = torch.zeros(n_tokens, self.HKV, self.D, dtype=torch.bfloat16, device="cuda")
        self.f = {name: torch.zeros(n_tokens, *width, device="cuda") for name, width in (
            ("w", (shape.k,)), ("y", (shape.H,)), ("logp", ()), ("entropy", ()), ("top", (4,)))}
        self.norms = [(1 + 0.2 * torch.randn(self.D, generator=g)).cuda() for _ in range(2)]
        self.rope = torch.empty(self.PLACES, self.ROPE, device="cuda")
        ft.ft_rope_table((1e4 ** (-torch.arange(self.ROPE // 2, dtype=torch.float64) / (self.ROPE // 2))).cuda(), self.ROPE, self.PLACES, self.rope)

    def run(self, stream=None):
        ft, t, s, n, D = self.ft, self.t, self.shape, self.n, self.D
        ft.ft_kv_plan(self.kv.handle, t["n_new"], t["len"], t["held"], t["table"], 30, t["free"], t["n_free"], 3, n, t["start"], t["kv_len"], t["slots"],
                      t["len"], t["held"], t["n_free"], positions=t["at"], stream=stream)
        q, k, v = self.x["qkv"].split([self.HQ * D, self.HKV * D, self.HKV * D], 1)
        ft.ft_kv_append_rotated(self.kv.handle, 0, q, k, v, t["slots"], n, self.q, t["at"], self.rope, self.ROPE, self.PLACES, k_out=self.k,
                                q_norm=self.norms[0], k_norm=self.norms[1], stream=stream)
        ft.ft_kv_attention(self.kv.handle, 0, self.q, t["start"], t["kv_len"], t["table"], 30, 3, n, n, self.o, sm_scale=D ** -0.5, stream=stream)
        ft.ft_moe_route(self.x["router"], n, s.E, s.k, t["ids"], self.f["w"], n_group=4, topk_group=2, group_best=2, stream=stream)
        ft.ft_moe_decode(self.experts.handle, 0, self.x["h"], t["ids"], self.f["w"], n, s.k, self.f["y"], t["deferred"], stream=stream)
        ft.ft_logprobs(self.x["logits"], n, self.V, t["tokens"], self.f["logp"], self.f["entropy"], t["tops"], self.f["top"], 4, stream=stream)

    def feed(self, n_new, seed):
        """A step's inputs."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.t["n_new"].copy_(torch.tensor(n_new, dtype=torch.int32))
        for x in self.x.values():
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        self.t["tokens"].copy_(torch.randint(0, self.V, (self.n,), generator=g, device="cuda"))


STEPS = [[5, 20, 1], [1, 1, 1], [0, 7, 3], [1, 1, -1], [16, 1, 0], [1, 1, 12], [1, -1, 1], [1, 24, 1]]


def test_steps_in_a_graph(ft):
    """A step captured once and replayed, its sequences growing, waiting, ending and starting; against oracles step by step."""
    from expert_cache_gb300.workloads import SHAPES, build_pool
    from oracle.formats import encode_record
    from oracle.moe import RecordSource, decode_layer
    import synth
    shape, n = SHAPES["tiny"], 28
    pool = build_pool(5, shape.L, shape.E, shape.H, shape.I)
    s = Step(ft, n, pool, shape)
    recs = RecordSource(lambda f: encode_record(*[w.numpy() for w in synth.expert_weights(5, f, shape.H, shape.I)]), shape.H, shape.I)
    state = dict(length=np.zeros(3, int), held=np.zeros(3, int), table=np.zeros((3, 30), int), free=s.t["free"].cpu().numpy().astype(int), n_free=40)
    s.feed([0, 0, 0], 99)                                        # before any capture: the kernels are loaded
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    keys, values = [[] for _ in range(3)], [[] for _ in range(3)]
    table = s.rope.double().cpu().numpy()
    for i, n_new in enumerate(STEPS):
        s.feed(n_new, i)
        s.o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert ft.ft_kv_status(s.kv.handle) == 0
        plan, _ = S.plan(n_new, state["length"], state["held"], state["table"], state["free"], state["n_free"], 40, s.PAGE, n)
        for name, key in (("start", "q_start"), ("kv_len", "kv_len"), ("slots", "slots"), ("at", "positions"), ("len", "len_out"), ("held", "held_out"),
                          ("table", "block_table"), ("free", "free_pages")):
            assert np.array_equal(s.t[name].cpu().numpy(), plan[key]), (i, name)
        assert s.t["n_free"].item() == plan["n_free_out"]
        state = dict(length=plan["len_out"], held=plan["held_out"], table=plan["block_table"], free=plan["free_pages"], n_free=int(plan["n_free_out"]))
        live = plan["slots"] >= 0
        row = table[plan["positions"]]
        qkv = s.x["qkv"].double().cpu().numpy().reshape(n, -1, s.D)
        k = S.turn(qkv[:, s.HQ:s.HQ + s.HKV], s.norms[1].double().cpu().numpy(), 1e-6, row[:, :16], row[:, 16:], False)
        k = torch.from_numpy(k.astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(s.k.cpu()[live], k[live])
        kq = K.values(*K.quantise(k.float().numpy(), "nvfp4", 0.0625), "nvfp4", 0.0625)
        vq = K.values(*K.quantise(qkv[:, s.HQ + s.HKV:].astype(np.float32), "nvfp4", 0.0625), "nvfp4", 0.0625)
        o, q = s.o.double().cpu().numpy(), s.q.double().cpu().numpy()
        for seq, m in enumerate(n_new):
            if m < 0:
                keys[seq], values[seq] = [], []
                continue
            a = plan["q_start"][seq]
            keys[seq] += list(kq[a:a + m])
            values[seq] += list(vq[a:a + m])
            length = len(keys[seq])
            assert length == plan["kv_len"][seq]
            for h in range(s.HQ if m else 0):
                kk, vv = (np.array(x)[:, h // (s.HQ // s.HKV)] for x in (keys[seq], values[seq]))
                ro, _, av, mag = K.attention(q[a:a + m, h], kk, vv, K.seen(m, length), s.D ** -0.5)
                e = (s.D ** -0.5 * (s.D + 16) * 2.0 ** -23 * mag)[:, None]
                tol = 2.0 ** -8 * np.abs(ro) + (2 * e + 2.0 ** -10) * av + length * 2.0 ** -24 * np.abs(vv).max()
                assert np.all(np.abs(o[a:a + m, h] - ro) <= tol), (i, seq, h)
        assert (o[plan["q_start"][-1]:] == 7).all()              # rows behind the last sequence
        z = s.x["router"].double().cpu().numpy()
        for r in range(n):
            ids, w = S.route(z[r], shape.k, "softmax", n_group=4, topk_group=2, group_best=2)
            assert s.t["ids"][r].tolist() == ids.tolist()
            assert np.allclose(s.f["w"][r].cpu().numpy(), w, rtol=2.0 ** -18)          # 64 roundings of 2^-24
            lp, _, tops, _ = S.logprobs(s.x["logits"][r].double().cpu().numpy(), int(s.t["tokens"][r]), 4)
            assert s.t["tops"][r].tolist() == tops.tolist() and abs(s.f["logp"][r].item() - lp) < 2.0 ** -16 * abs(lp)      # 70 of them and 2^-22
        ref = decode_layer(s.x["h"].float().cpu().numpy(), s.t["ids"].cpu().numpy(), s.f["w"].cpu().numpy(), 0, shape.E, recs)
        y = s.f["y"].double().cpu().numpy()
        assert np.linalg.norm(y - ref) <= 5e-3 * np.linalg.norm(ref)
    s.experts.close()
    s.kv.close()
    pool.free()


def test_refused_sequences_are_harmless(ft):
    """A sequence that gets no pages: its rows are not stored, attend to nothing and go on once there is room."""
    from expert_cache_gb300.workloads import SHAPES, build_pool
    shape = SHAPES["tiny"]
    pool = build_pool(5, shape.L, shape.E, shape.H, shape.I)
    s = Step(ft, 32, pool, shape)
    s.t["n_free"].fill_(1)
    s.feed([4, 17, 2], 0)
    s.run()
    assert ft.ft_kv_status(s.kv.handle) == ft.FT_DEV_NO_PAGES
    assert s.t["slots"].tolist()[4:] == [-1] * 28 and s.t["kv_len"].tolist() == [4, 0, 0] and s.t["len"].tolist() == [4, 0, 0]
    assert torch.isfinite(s.o[:4].float()).all() and s.o[:4].any() and not s.o[4:23].any()
    s.t["n_free"].fill_(30)
    s.t["free"].copy_(torch.arange(40, dtype=torch.int32)[torch.arange(40) != s.t["table"][0, 0].cpu()].repeat(2)[:40])
    s.feed([1, 17, 2], 1)
    s.run()
    assert ft.ft_kv_status(s.kv.handle) == 0 and s.t["kv_len"].tolist() == [5, 17, 2] and (s.t["slots"][:20] >= 0).all() and s.o[:20].any(-1).all()
    s.experts.close()
    s.kv.close()
    pool.free()


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_served_decoder_over_a_given_text(ft, example, fmt, seed):
    """The same text by single tokens, by chunks and by trees whose branch it is, so that no tie of two tokens parts the ways: the
    logits of every place, within the plain decoder's bound (test_layers_together)."""
    ex, rng = example, np.random.default_rng(seed)
    text = rng.integers(0, ex.VOCAB, 130).tolist()
    d = ex.Served(fmt=fmt)
    one = torch.cat([d.chunk([t]) for t in text])
    d.close()
    d, chunks, at = ex.Served(fmt=fmt), [], 0
    while at < len(text):
        n = int(rng.integers(1, ex.BATCH + 1))
        chunks.append(d.chunk(text[at:at + n]))
        at += n
    d.close()
    d, trees, at = ex.Served(fmt=fmt), [], 0
    while at < len(text):
        tokens, masks, path = [text[at]], [1], [0]
        for t in text[at + 1:at + 1 + int(rng.integers(0, 7))]:
            for wrong in range(int(rng.integers(0, 3))):           # siblings that are not the text's
                masks.append(masks[path[-1]] | 1 << len(tokens))
                tokens.append((t + 1 + wrong) % ex.VOCAB)
            masks.append(masks[path[-1]] | 1 << len(tokens))
            path.append(len(tokens))
            tokens.append(t)
        logits, kept = d.step(tokens, None, masks)
        d.keep(len(tokens), path, kept)
        trees.append(logits[path])
        at += len(path)
    d.close()
    for other in (torch.cat(chunks), torch.cat(trees)):
        assert other.shape == one.shape and ((other - one).norm() / one.norm()).item() < 2.0 ** -4
