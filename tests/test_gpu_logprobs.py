"""ft_logprobs against oracle.step: indices equal, values within their roundings.

With d = x - max and y = scale d: d and y are rounded once each (2^-24 |y| each, 2^-23 more for the exponential's base), the
exponential to 2 units in the last place (2^-22), and of the sum S every term passes at most n = V / 256 + 64 additions: relative
error of S at most s = 2^-24 (n + 4 max_i |y_i| e^y_i + 4) <= 2^-24 (n + 6).  So
  |d logp| <= 2^-22 |y| + s + 2^-23 |log S| + 2^-149
  |d entropy| <= s (1 + |log S|) + 2 s sum e^y |y| / S + 2^-22 sum e^y y^2 / S + 2^-22."""
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


def run(ft, x, tokens, k, scale=1.0, stream=None, out=None, **kw):
    n, V = x.shape
    logp, h, ids, top = out or (torch.full((n,), float("nan"), device="cuda"), torch.full((n,), float("nan"), device="cuda"),
                                torch.full((n, k), -9, dtype=torch.int32, device="cuda"), torch.full((n, k), float("nan"), device="cuda"))
    ft.ft_logprobs(x, n, V, tokens, logp, h, ids, top, k, scale=scale, stream=stream, **kw)
    return logp, h, ids, top


def check(x, tokens, got, k, scale=1.0, rows=None):
    torch.cuda.synchronize()
    logp, h, ids, top = (None if t is None else t.double().cpu().numpy() for t in got)
    tokens = tokens.cpu().numpy()
    V = x.shape[1]
    s = 2.0 ** -24 * (V / 256 + 70)
    for r in range(len(x)) if rows is None else rows:
        row = x[r].double().cpu().numpy()
        lp, e, want, wtop = S.logprobs(row, int(tokens[r]), k, scale)
        z = S._logits(row)
        if np.isneginf(z.max()):
            log_s = far = dot = sq = 0.0
        else:
            y = (z - z.max()) * float(np.float32(scale))
            p = np.exp(y)
            log_s = np.log(p.sum())
            some = p > 0
            dot, sq = (p[some] * -y[some]).sum() / p.sum(), (p[some] * y[some] ** 2).sum() / p.sum()
            far = 0.0

        def close(a, b):
            if b < -S.F32_MAX * (1 + 2.0 ** -25):                  # past fp32's range such a value rounds to -inf (IEEE 754, 7.4)
                return np.isneginf(a)
            far = abs(b + log_s)
            return abs(a - b) <= 2.0 ** -22 * far + s + 2.0 ** -23 * abs(log_s) + 2.0 ** -149
        if logp is not None:
            assert close(logp[r], lp), (r, logp[r], lp)
        if h is not None:
            assert abs(h[r] - e) <= s * (1 + abs(log_s)) + 2 * s * dot + 2.0 ** -22 * sq + 2.0 ** -22, (r, h[r], e)
        if k:
            assert ids[r].tolist() == want.tolist(), (r, ids[r], want)
            assert all(close(a, b) for a, b in zip(top[r], wtop)), (r, top[r], wtop)


def logits(seed, n, V, dtype=torch.float32, spread=3.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, V + pad, generator=g, device="cuda") * spread).to(dtype)[:, :V]


def tokens_of(seed, n, V):
    return torch.from_numpy(np.random.default_rng(seed).integers(0, V, n).astype(np.int32)).cuda()


@pytest.mark.parametrize("n,V", [(1, 1), (3, 2), (2, 7), (5, 31), (4, 64), (3, 257), (9, 1000), (2, 4095), (3, 8200), (2, 30011), (1, 65536), (3, 100003), (1, 131072),
                                 (2, 200000), (1, 262147), (700, 500), (160, 5000), (330, 33000), (70000, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [0, 1, 5, 20, 32])
def test_sizes(ft, n, V, dtype, k):
    k = min(k, V)
    x, t = logits(n + V, n, V, dtype, pad=k % 3), tokens_of(V, n, V)
    scale = [1.0, 0.7, 1.3][k % 3]
    rows = None if n < 10 else [0, 1, n // 2, n - 1]
    check(x, t, run(ft, x, t, k, scale), k, scale, rows)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_wherever_they_stand(ft, dtype):
    """Rows that start at every alignment; what lies around them is not read, outputs behind the call's stay."""
    for V in (5, 100, 1003, 20001, 70007):
        for at in range(0, 9, 1 if V < 2000 else 3):
            flat = torch.full((4 * (V + 1) + 32,), float("inf"), dtype=dtype, device="cuda")
            x = flat[at:at + 3 * (V + 1)].view(3, V + 1)[:, :V]
            x.copy_(logits(V + at, 3, V, dtype))
            t = tokens_of(at, 3, V)
            out = (torch.full((5,), 7.0, device="cuda"), torch.full((5,), 7.0, device="cuda"), torch.full((5, 4), -9, dtype=torch.int32, device="cuda"),
                   torch.full((5, 4), 7.0, device="cuda"))
            run(ft, x, t, 4, out=out)
            check(x, t, [o[:3] for o in out], 4)
            assert all((o[3:] == (-9 if o.dtype == torch.int32 else 7)).all() for o in out)


@pytest.mark.parametrize("V", [40, 3000, 50000, 140000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orders_that_are_hard(ft, V, dtype):
    """Ties, rising and falling rows, one value everywhere, the largest last: whatever is looked at first."""
    n = 10
    x = logits(V, n, V, dtype)
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    x[0] = 1.5
    x[1] = (i / V * 40).to(dtype)
    x[2] = (-i / V * 40).to(dtype)
    x[3] = (i % 7).to(dtype)
    x[4] = torch.where(i < V - 40, 0.0, 5.0).to(dtype)
    x[5] = torch.where(i % 13 == 3, 9.0, -9.0).to(dtype)
    x[6] = torch.where(i == V - 1, 100.0, 0.0).to(dtype)
    x[7] = (torch.round(x[7].float()) * 2).to(dtype)
    x[8] = torch.where(i < V // 2, -30.0, 0.0).to(dtype)
    x[9] = 0.0
    x[9, 1::2] = -0.0                                              # equal
    t = tokens_of(1, n, V)
    for k in (1, 7, 32):
        check(x, t, run(ft, x, t, k), k)


@pytest.mark.parametrize("V", [33, 5000, 131072])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_what_is_masked(ft, V, dtype):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    x = logits(V, 14, V, dtype)
    x[0] = -inf
    x[1] = nan
    x[2, 1:] = -inf
    x[3, :-1] = nan
    x[4, V // 2] = inf
    x[5, 3], x[5, V - 2] = inf, inf
    x[6] = low
    x[7, 5:] = low
    x[8] = inf
    x[9, 20:] = -inf
    x[10, ::2] = nan
    x[11, :-3] = -inf
    x[12] = -5000.0
    x[12, 7] = -4999.0
    x[13] = torch.finfo(dtype).max
    x[13, 9] = inf
    t = tokens_of(0, 14, V)
    t[2], t[3], t[4], t[7] = 0, V - 1, V // 2, 5
    for k, scale in ((4, 1.0), (25, 0.3), (1, 4.0), (0, 1.0), (3, 1e-37), (3, 1e-42), (0, 1e-37), (2, 1e30), (2, 3e38)):
        got = run(ft, x, t, k, scale)
        assert not any(torch.isnan(g).any() for g in got)
        check(x, t, got, k, scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_rising_rows(ft, dtype):
    """Rows whose every part is larger than the one before, in steps that the type tells apart: a bound from the front says nothing."""
    n, V = 3, 400000
    x = torch.arange(V, device="cuda", dtype=torch.float32)[None].repeat(n, 1) * torch.tensor([1e-4, 1e-3, 0.1], device="cuda")[:, None]
    x, t = x.to(dtype), tokens_of(3, n, V)
    for k in (1, 32):
        check(x, t, run(ft, x, t, k), k)


@pytest.mark.parametrize("V,dtype", [(33, torch.bfloat16), (4099, torch.float32), (20000, torch.bfloat16), (50305, torch.float32), (57001, torch.float32),
                                     (112503, torch.bfloat16)])
def test_more_rows_than_the_gpu_holds(ft, V, dtype):
    """Hard rows among many others, k on both sides of what decides how many threads a row gets."""
    n = 2 * torch.cuda.get_device_properties(0).multi_processor_count + 17
    x = logits(V, n, V, dtype, pad=3)
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    x[0], x[1], x[2] = 1.5, (i / V * 40).to(dtype), (-i / V * 40).to(dtype)
    x[3], x[4] = torch.where(i < V - 40, 0.0, 5.0).to(dtype), float("nan")
    x[5, 1:], x[6, ::2], x[7] = float("-inf"), float("nan"), torch.finfo(dtype).min
    x[8, V // 2], x[n - 1, V - 1] = float("inf"), 50.0
    t = tokens_of(2, n, V)
    for k in (0, 1, 4, 16, 32):
        check(x, t, run(ft, x, t, k), k, rows=[0, 1, 2, 3, 4, 5, 6, 7, 8, 9, n // 2, n - 2, n - 1])


def test_temperatures_and_tokens(ft):
    x = logits(3, 6, 40000)
    t = tokens_of(0, 6, 40000)
    t[1], t[2], t[3] = -1, 40000, -(1 << 31)                      # no tokens of the row
    for scale in (1e-6, 1e-3, 0.05, 1.0, 20.0, 1e4, 1e30):
        check(x, t, run(ft, x, t, 6, scale), 6, scale)
    got = run(ft, x, t, 0)
    assert torch.isneginf(got[0][1:4]).all() and torch.isfinite(got[0][[0, 4, 5]]).all()
    # only what is asked for
    full = run(ft, x, t, 5)
    for keep in ((0,), (1,), (2, 3), (0, 1)):
        out = [torch.full_like(f, -3) for f in full]
        ft.ft_logprobs(x, 6, 40000, tokens=t if 0 in keep else None, logp=out[0] if 0 in keep else None, entropy=out[1] if 1 in keep else None,
                       top_ids=out[2] if 2 in keep else None, top_logp=out[3] if 3 in keep else None, k=5 if 2 in keep else 0)
        for i, (a, b) in enumerate(zip(out, full)):
            assert torch.equal(a, b if i in keep else torch.full_like(b, -3))


def test_two_calls_at_once(ft):
    xs, t = [logits(i, 300, 50000, torch.bfloat16) for i in range(2)], tokens_of(0, 300, 50000)
    alone = [run(ft, x, t, 7) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [run(ft, x, t, 7, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_far_rows_streams_and_graphs(ft):
    """Rows whose offsets pass 2^32 bytes; the same bits on another stream and again; a captured call on new logits."""
    n, V = 9000, 262144
    x = torch.empty(n, V, dtype=torch.bfloat16, device="cuda")
    x[::997] = logits(0, len(range(0, n, 997)), V, torch.bfloat16)
    x[-1] = logits(1, 1, V, torch.bfloat16)[0]
    t = tokens_of(2, n, V)
    got = run(ft, x[997::997], t[997::997].contiguous(), 5)        # a row stride of 2^28 elements
    check(x[997::997], t[997::997], got, 5, rows=[0, 8])
    rest = run(ft, x[8192:], t[8192:], 5)
    check(x[8192:], t[8192:], rest, 5, rows=[n - 1 - 8192, 997 * 9 - 8192])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run(ft, x[997::997], t[997::997].contiguous(), 5, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    y, out = x[:3].clone(), [torch.empty_like(g[:3]) for g in got]
    g = torch.cuda.CUDAGraph()
    u = t[:3].clone()
    with torch.cuda.graph(g):
        run(ft, y, u, 5, out=out)
    y.copy_(logits(9, 3, V, torch.bfloat16))
    g.replay()
    check(y, u, out, 5)


def test_results_do_not_depend_on_the_run_or_the_other_rows(ft):
    x, t = logits(4, 40, 60000, torch.bfloat16), tokens_of(4, 40, 60000)
    a = run(ft, x, t, 9)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, run(ft, x, t, 9)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V", [(2, 131072), (200, 20000), (330, 60001)])
def test_scales_by_decades(ft, n, V, dtype):
    """Temperatures down to 1e-20: scale times the largest logit through every power of two from 2^16 to 2^70.  (Where it is kept as a
    rounded product, an offset of at most 2 in the base-2 exponents costs the entropy 2 log 2 of the n roundings of s that are not
    made: V / 256 counts twice the additions of a term.)"""
    x, t = logits(n + V, n, V, dtype), tokens_of(V, n, V)
    t[0] = int(x[0].float().argmax())
    for e in range(4, 21):
        for k in (0, 5):
            check(x, t, run(ft, x, t, k, 10.0 ** e), k, 10.0 ** e, rows=[0, n // 2, n - 1])


@pytest.mark.parametrize("k", [0, 4])
@pytest.mark.parametrize("n,V", [(2, 131072), (200, 60001)])
def test_neighbours_far_from_zero(ft, n, V, k):
    """Logits a few steps of fp32 apart around 2^10 to 2^100, a step worth 1/4 to 140: first the lower ones, so that the later ones lie above
    every thread's reference.  The same bound as in test_scales_by_decades."""
    g = torch.Generator(device="cuda").manual_seed(V)
    step = torch.randint(0, 4, (n, V), generator=g, device="cuda")
    step[:, V // 4 * 3:] += 1
    step[n - 1, V - 1] += 2
    t = tokens_of(k, n, V)
    for e in (10, 26, 30, 31, 40, 60, 100):
        x = (1 + step * 2.0 ** -23) * 2.0 ** e
        for worth in (0.25, 1.0, 2.0, 5.0, 16.0, 70.0, 100.0, 140.0):
            scale = worth * 2.0 ** (23 - e)
            check(x, t, run(ft, x, t, k, scale), k, scale, rows=[0, n - 1])
            check(-x, t, run(ft, -x, t, k, scale), k, scale, rows=[0, n - 1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V", [(9, 131072), (200, 20000), (330, 60001)])
def test_infinities_at_every_scale(ft, n, V, dtype):
    """+inf counts as the largest fp32 value, first, last, alone, beside numbers that lie within the exponentials' range of it, and everywhere."""
    inf, x, t = float("inf"), logits(n + V, n, V, dtype), tokens_of(V, n, V)
    x[0, 3] = inf
    x[1, V - 1] = inf
    x[2, 9], x[2, V - 1] = 2.5e38, inf                            # the span may pass the largest number
    x[3, 9], x[3, V // 2] = 3.3e38, inf
    x[4, ::5] = inf
    x[5] = inf
    x[6, V // 2:] = inf
    x[7] = -inf
    x[7, V - 2] = inf
    t[0], t[1], t[2], t[3] = 3, V - 1, 9, 9
    for scale in (1e-36, 6e-37, 5.5e-37, 4e-37, 3e-36, 1e-33, 1e-30, 1e-25, 1e-22, 2e-21, 1e-20, 1e-15, 1e-10, 1e-5, 1.0, 1e5, 1e15, 1e25):
        for k in (0, 3):
            check(x, t, run(ft, x, t, k, scale), k, scale, rows=range(9))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V", [(9, 131072), (200, 20000), (330, 60001)])
def test_differences_past_the_range(ft, n, V, dtype):
    """Rows over the whole range of the type at scales that leave their exponentials numbers.  (Below 1.2e-38 the scale in base 2 is
    rounded to a step of 2^-149, which moves an exponent by at most 2^-150 times 2^129, half of the 70 roundings of s that no row makes.)"""
    x, t = torch.empty(n, V, dtype=dtype, device="cuda"), tokens_of(V, n, V)
    most, low = torch.finfo(dtype).max, torch.finfo(dtype).min
    g = torch.Generator(device="cuda").manual_seed(V)
    x.copy_((torch.rand(n, V, generator=g, device="cuda") * 2 - 1) * 3.38e38)
    x[0, :V // 2], x[0, V // 2:] = low, most                      # every thread's reference is the lowest value at first
    x[1, :V // 2], x[1, V // 2:] = most, low
    x[2] = low
    x[2, V - 1] = float("inf")
    x[3] = low
    x[3, 0] = float("inf")
    x[4, V // 4 * 3:] = most
    x[5, ::2] = float("-inf")
    t[0], t[1], t[2], t[3] = 0, V - 1, 0, V - 1
    for scale in (1e-42, 1e-40, 4e-39, 1e-38, 5e-38, 1e-37, 1.9e-37, 2.5e-37, 3e-37, 1e-36, 1e-35):
        for k in (0, 3):
            check(x, t, run(ft, x, t, k, scale), k, scale, rows=range(9))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V", [(6, 131072), (200, 20000), (330, 60001), (3, 29)])
def test_nan_among_equal_logits(ft, n, V, dtype):
    """NaN counts for nothing wherever the sums are taken apart: large scales, large logits, the ends of both; many logits share the
    largest value, so that the entropy is no zero."""
    g = torch.Generator(device="cuda").manual_seed(V)
    hit = torch.rand(n, V, generator=g, device="cuda")
    t = tokens_of(V, n, V)
    for top in (3.0, 1e12, -1e12, 2e38, float("inf")):
        x = torch.where(hit < 0.3, top, logits(V, n, V) - 20 if top == 3.0 else float("-inf")).to(dtype)
        x[hit > 0.6] = float("nan")
        x[0, 0], x[1, -1] = float("nan"), float("nan")
        x[2, V // 2] = top
        for scale in (1e-42, 1e-37, 1e-25, 1e-3, 1.0, 50.0, 1e8, 1e12, 1e19, 1e30, 3e38):
            for k in (0, 3):
                check(x, t, run(ft, x, t, k, scale), k, scale, rows=range(3))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [12, 30, 318, 1003, 2041])
def test_a_largest_logit_that_comes_late(ft, V, dtype):
    """The largest stands behind what the references are taken from, 1 to 200 above the others.  (A thread's terms lie up to 2^64 above its
    reference.  The exponent's rounding is then 22 of the 2^-24 of which s has 70 or more, that of the factor back to the largest another 22,
    the exponentials 8; a term of these short rows passes fewer than 16 additions.)"""
    gaps = [1, 3, 8, 11, 12, 13, 20, 33, 41, 55, 60, 66, 68, 70, 90, 120, 200]
    n = 2 * len(gaps)
    x = logits(V, n, V, dtype, spread=1.0)
    for i, gap in enumerate(gaps):
        x[2 * i, V - 1] = x[2 * i].float().max() + gap
        x[2 * i + 1, V - 1] = x[2 * i + 1].float().max() + gap + 0.37
        x[2 * i + 1, V - 2] = x[2 * i + 1, V - 1].float() - 1
    t = torch.full((n,), V - 1, dtype=torch.int32, device="cuda")
    for scale in (1.0, 0.9, 1.2587579488754272):
        for k in (0, 2):
            check(x, t, run(ft, x, t, k, scale), k, scale)
