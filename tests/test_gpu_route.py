"""ft_moe_route against oracle.step: ids equal, weights within their roundings.

A weight is e / sum e (or a score, or a renormalised score) times the scale, in fp32: two roundings of the exponential's
argument (2^-24 |x - top| each), 2 units in the last place of the function (2^-22), at most E / 32 + 5 additions and three more
operations of 2^-24 each, on the term and on the sum: relative 2^-24 (4 |x - top| + E / 32 + 24)."""
import numpy as np
import pytest
import torch

from oracle import step as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ft():
    import __graft_entry__ as entry
    entry.build()
    import expert_cache_gb300
    return expert_cache_gb300


def run(ft, x, k, stream=None, out=None, **kw):
    T, E = x.shape
    bias = kw.pop("bias", None)
    ids, w = out or (torch.full((T, k), -9, dtype=torch.int32, device="cuda"), torch.full((T, k), float("nan"), device="cuda"))
    ft.ft_moe_route(x, T, E, k, ids, w, bias=None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda(), stream=stream, **kw)
    return ids, w


def check(x, ids, w, k, rows=None, **kw):
    torch.cuda.synchronize()
    ids, w, x = ids.cpu().numpy(), w.double().cpu().numpy(), x.double().cpu().numpy()
    E = x.shape[1]
    for t in range(len(x)) if rows is None else rows:
        want, ww = S.route(x[t], k, **kw)
        assert ids[t].tolist() == want.tolist(), (t, ids[t], want)
        z = np.where(want >= 0, np.minimum(x[t][want], S.F32_MAX), 0)
        fin = np.isfinite(x[t])
        far = np.abs(z - (x[t][fin].max() if fin.any() else 0)) if kw["score"] == "softmax" else np.abs(z) + 1
        assert np.all(np.abs(w[t] - ww) <= np.abs(ww) * 2.0 ** -24 * (4 * np.minimum(far, 200) + E / 32 + 24) + 2.0 ** -120), (t, w[t], ww)


def logits(seed, T, E, dtype=torch.float32, spread=1.5, pad=0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((T, E + pad)) * spread).astype(np.float32)).to(dtype).cuda()
    return x[:, :E]


SHAPES = [(1, 1, 1, 1), (3, 2, 2, 1), (5, 7, 3, 1), (4, 8, 8, 4), (33, 16, 2, 1), (9, 60, 4, 6), (6, 64, 6, 8), (17, 96, 9, 3), (130, 256, 8, 8), (7, 256, 32, 1),
          (21, 160, 6, 8), (5, 320, 10, 32), (3, 1000, 7, 5), (3, 1024, 32, 16), (2, 1025, 8, 1), (2, 1920, 9, 30), (2, 4096, 32, 32), (1, 4095, 5, 3)]


@pytest.mark.parametrize("T,E,k,groups", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [None, 0.05, 3.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shapes(ft, T, E, k, groups, score, bias, dtype):
    rng = np.random.default_rng(E)
    x = logits(E + T, T, E, dtype, pad=3 * (k % 2))
    b = None if bias is None else (rng.standard_normal(E) * bias).astype(np.float32)
    kw = dict(score=score, bias=b, renormalise=True, scale=2.5)
    check(x, *run(ft, x, k, **kw), k, **kw)
    kw["renormalise"] = False
    check(x, *run(ft, x, k, **kw), k, **kw)
    for best in (1, 2):
        for keep in {1, (groups + 1) // 2, groups}:
            kw = dict(score=score, bias=b, n_group=groups, topk_group=keep, group_best=best)
            check(x, *run(ft, x, k, **kw), k, **kw)                # may leave fewer than k experts


@pytest.mark.parametrize("E", [31, 32, 33, 63, 65, 127, 129, 255, 257, 511, 512, 513, 1023, 1025])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sizes_around_the_variants(ft, E, dtype):
    """Numbers of experts at which another variant takes over, with one expert chosen and with as many as there may be."""
    x = logits(E, 5, E, dtype, pad=E % 2)
    b = np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.1
    for k in (1, 31, min(E, 32)):
        for bias in (None, b):
            kw = dict(score="sigmoid" if E % 2 else "softmax", bias=bias)
            check(x, *run(ft, x, k, **kw), k, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_experts_that_come_out_on_top_together(ft, dtype):
    """The chosen ones are neighbours: rising and falling rows and biases."""
    for E in (40, 160, 256, 500):
        x = torch.stack([torch.arange(E) * 0.5, -torch.arange(E) * 0.5, torch.zeros(E), (torch.arange(E) // 8) * 1.0]).to(dtype).cuda()
        for bias in (None, np.arange(E, dtype=np.float32) * 10, -np.arange(E, dtype=np.float32)):
            for groups in (1, 4):
                kw = dict(score="softmax", bias=bias, n_group=groups, topk_group=2 if groups > 1 else 1, group_best=2)
                check(x, *run(ft, x, 9, **kw), 9, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 100, 256, 2048])
def test_ties_take_the_lower_index(ft, score, E):
    rng = np.random.default_rng(E)
    x = torch.from_numpy(rng.choice([0.5, 1.0, 1.0, 2.0], (20, E)).astype(np.float32)).cuda()
    x[3] = 1.0
    for bias in (None, np.zeros(E, np.float32), rng.choice([0.0, 0.125], E).astype(np.float32)):
        for groups, best in ((1, 1), (4, 1), (4, 2)):
            kw = dict(score=score, bias=bias, n_group=groups, topk_group=min(2, groups), group_best=best)
            check(x, *run(ft, x, 4, **kw), 4, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choices_closer_than_fp32_tells(ft, score):
    """Biases that bring the choices of neighbours within one fp32 step of each other, on either side."""
    rng = np.random.default_rng(7)
    E, T = 64, 200
    x = rng.standard_normal((T, E)).astype(np.float32)
    p = np.exp(x.astype(np.float64))
    sc = p / p.sum(1, keepdims=True) if score == "softmax" else p / (1 + p)
    # every choice of row 0 lies within a rounding of 0.75, and those of the others spread out from there
    bias = (0.75 - sc[0]).astype(np.float32)
    t = torch.from_numpy(x).cuda()
    for groups, keep, best in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
        kw = dict(score=score, bias=bias, n_group=groups, topk_group=keep, group_best=best)
        check(t, *run(ft, t, 6, **kw), 6, **kw)
    # logits that differ in their last bit, without a bias: no rounding of scores decides
    y = np.ones((4, E), np.float32)
    y[:, 40:44] = np.nextafter(np.float32(1), np.float32(2))
    y[2] *= 30
    t = torch.from_numpy(y).cuda()
    for groups, keep, best in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
        kw = dict(score=score, n_group=groups, topk_group=keep, group_best=best)
        check(t, *run(ft, t, 6, **kw), 6, **kw)


@pytest.mark.parametrize("E", [64, 600])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_large_score_passes_between_two_small_ones(ft, score, E):
    """A large score with a bias far below it, and so a larger error, rises past the last that is chosen and the first that is
    not, which lie further apart than their own errors."""
    T = 2000
    x = np.full((T, E), -4.0, np.float32)
    x[:, 1], x[:, 2], x[:, 3] = 0.0, -1.0, -2.0
    x[:, 0] = 2.2 + (np.arange(T) - T / 2) * 2.0 ** -21
    p = np.exp(x[T // 2].astype(np.float64))
    sc = p / p.sum() if score == "softmax" else p / (1 + p)
    bias = np.full(E, -1.0, np.float32)
    bias[1], bias[2], bias[3] = 0.5 - sc[1], 0.3 - sc[2], 0.3 - 5e-7 - sc[3]
    bias[0] = 0.3 - 2.5e-7 - sc[0]
    t = torch.from_numpy(x).cuda()
    kw = dict(score=score, bias=bias)
    check(t, *run(ft, t, 2, **kw), 2, rows=range(T // 2 - 150, T // 2 + 150), **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 544])
def test_groups_worth_more_than_fp32_holds(ft, score, E):
    """Biases of the type's lowest value (a mask), two of which have a sum in 64 bits only: such a group comes before one without
    experts, and one of two lesser values before it."""
    groups = 4 if E == 64 else 32
    size = E // groups
    rng = np.random.default_rng(E)
    x = rng.standard_normal((6, E)).astype(np.float32)
    x[:, 4 * size:] = np.nan                                       # only the first four groups have experts
    x[:3, :size] = np.nan                                          # in these rows without the first
    bias = rng.standard_normal(E).astype(np.float32)
    bias[size:2 * size] = np.finfo(np.float32).min
    bias[2 * size:3 * size] = -3e38
    t = torch.from_numpy(x).cuda()
    for topk_group in (1, 2, 3, 4):
        kw = dict(score=score, bias=bias, n_group=groups, topk_group=topk_group, group_best=2, renormalise=False)
        check(t, *run(ft, t, 32, **kw), 32, **kw)
    most = np.finfo(np.float32).max
    bias[size:2 * size], bias[2 * size:3 * size] = most, 3e38
    for topk_group in (1, 2):
        kw = dict(score=score, bias=bias, n_group=groups, topk_group=topk_group, group_best=2, renormalise=False)
        check(t, *run(ft, t, 32, **kw), 32, **kw)


@pytest.mark.parametrize("E", [40, 256, 640])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_logits_around_the_last_place(ft, E, dtype):
    """The k-th, the next and more are equal, and behind them stand larger ones that fp32 does not tell from them."""
    x = torch.linspace(-3, 1, E, dtype=torch.float32).repeat(2, 1)
    x[0, :10], x[0, E - 1], x[0, E - 5] = 20.0, 25.0, 22.0        # a sigmoid of 1 in fp32
    x[1, E - 20:E - 5], x[1, E - 1], x[1, E - 3] = 18.0, 18.5, 19.0
    t = x.to(dtype).cuda()
    kw = dict(score="sigmoid", bias=np.zeros(E, np.float32))
    for k in (1, 3, 4, 8):
        check(t, *run(ft, t, k, **kw), k, **kw)
    kw = dict(score="softmax", bias=np.full(E, 1e7, np.float32))  # any score is lost in the sum
    for k in (1, 3, 4, 8):
        check(t, *run(ft, t, k, **kw), k, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [96, 640])
def test_scores_at_the_end_of_64_bits(ft, score, E):
    """Scores of e^-690 to e^-709 (and, softmax, to e^-740, which numbers of 64 bits below the normal ones hold) are in order; below
    e^-746 they are all 0 and the lower index comes first."""
    rng = np.random.default_rng(E)
    last = -740.0 if score == "softmax" else -709.0
    x = np.full((4, E), -800.0, np.float32)
    for row in x:
        at = rng.permutation(E - 1)[:9]
        row[at] = np.linspace(-690.0, last, 9)
    x[:, E - 1] = 0.0                                              # the largest
    x[3, :] = np.where(np.arange(E) < E - 1, -760.0 - rng.permutation(E), 0.0)
    bias = np.zeros(E, np.float32)
    t = torch.from_numpy(x).cuda()
    kw = dict(score=score, bias=bias, renormalise=False)
    check(t, *run(ft, t, 12, **kw), 12, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_what_is_masked(ft, score, dtype):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    rows = torch.randn(12, 40, generator=torch.Generator().manual_seed(0))
    rows[0] = -inf
    rows[1] = nan
    rows[2, 1:] = -inf
    rows[3, ::2] = nan
    rows[4, 7] = inf
    rows[5, 7], rows[5, 30] = inf, inf
    rows[6] = low
    rows[7, 3:] = low
    rows[8] = inf
    rows[9, :38] = -inf
    rows[10, 5:9] = -200.0
    rows[11] = -300.0
    x = rows.to(dtype).cuda()
    bias = np.random.default_rng(0).standard_normal(40).astype(np.float32)
    odd = bias.copy()
    odd[0], odd[3], odd[11], odd[12] = -np.inf, np.nan, np.inf, 1e30
    for b in (None, bias, odd):
        for groups, keep, best in ((1, 1, 1), (5, 2, 1), (5, 2, 2)):
            for renorm in (True, False):
                kw = dict(score=score, bias=b, n_group=groups, topk_group=keep, group_best=best, renormalise=renorm)
                ids, w = run(ft, x, 5, **kw)
                assert torch.isfinite(w).all()
                check(x, ids, w, 5, **kw)


def test_weights_do_not_underflow_together(ft):
    x = torch.full((2, 8), -150.0, device="cuda")
    x[:, 3] = -149.0
    x[1, 0] = 500.0
    bias = np.zeros(8, np.float32)
    bias[0] = -1000
    for score in ("softmax", "sigmoid"):
        kw = dict(score=score, bias=bias)
        check(x, *run(ft, x, 3, **kw), 3, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_wherever_they_stand(ft, dtype):
    """Row strides and starts of every alignment; what lies between the rows is not read, rows of the output behind the call's stay."""
    for E, pad, at in ((256, 8, 8), (256, 3, 1), (64, 1, 5), (31, 2, 3)):
        flat = torch.full((12 * (E + pad) + at,), float("inf"), dtype=dtype, device="cuda")
        x = flat[at:at + 11 * (E + pad)].view(11, E + pad)[:, :E]
        x.copy_(logits(E, 11, E, dtype))
        ids, w = torch.full((13, 4), -9, dtype=torch.int32, device="cuda"), torch.full((13, 4), 7.0, device="cuda")
        run(ft, x, 4, out=(ids, w))
        check(x, ids, w, 4, score="softmax")
        assert (ids[11:] == -9).all() and (w[11:] == 7).all()
    x = logits(1, 1, 64, dtype)
    check(x, *run(ft, x, 4), 4, score="softmax")
    ids, w = torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda")
    ft.ft_moe_route(x[:0], 0, 64, 4, ids, w)


def test_many_rows_streams_and_graphs(ft):
    x = logits(5, 40000, 128, torch.bfloat16)
    ids, w = run(ft, x, 6)
    rows = np.random.default_rng(0).integers(0, 40000, 100).tolist() + [0, 39999]
    check(x, ids, w, 6, rows=rows, score="softmax")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run(ft, x, 6, stream=side)
    side.synchronize()
    assert torch.equal(ids, again[0]) and torch.equal(w, again[1])
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(ids), torch.empty_like(w)
    with torch.cuda.graph(g):
        run(ft, x, 6, out=out)
    x.copy_(logits(6, 40000, 128, torch.bfloat16))
    g.replay()
    check(x, *out, 6, rows=rows, score="softmax")


def test_what_is_routed_is_what_the_experts_take(ft):
    """ids and weights go to ft_moe_decode as they are."""
    from expert_cache_gb300.workloads import SHAPES as W, build_pool
    from oracle.formats import encode_record
    from oracle.moe import RecordSource, decode_layer
    import synth
    s = W["tiny"]
    pool = build_pool(3, s.L, s.E, s.H, s.I)
    cache = ft.ExpertCache(s.L, s.E, s.H, s.I, s.k, 8, s.L * s.E, pool.ptr)
    x = torch.randn(8, s.H, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    z = logits(4, 8, s.E)
    ids, w = run(ft, z, s.k, score="sigmoid", n_group=4, topk_group=2, group_best=2, scale=1.5)
    y, deferred = torch.empty(8, s.H, device="cuda"), torch.empty(8, s.k, dtype=torch.int32, device="cuda")
    ft.ft_moe_decode(cache.handle, 1, x, ids, w, 8, s.k, y, deferred)
    recs = RecordSource(lambda f: encode_record(*[t.numpy() for t in synth.expert_weights(3, f, s.H, s.I)]), s.H, s.I)
    torch.cuda.synchronize()
    ref = decode_layer(x.float().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), 1, s.E, recs)
    assert np.linalg.norm(y.double().cpu().numpy() - ref) <= 5e-3 * np.linalg.norm(ref)
    cache.close()
    pool.free()
