"""ft_kv_append_rotated and ft_rope_table against oracle.step and oracle.kv.

Keys are carried to some 2^-40 and rounded twice as the oracle does, so k_out and the stored codes are the oracle's exactly.  A
query is fp32 until its rounding to bf16 (2^-8 of its value, half a step of 8 bits being 2^-9 to 2^-8): with A = |a c|, B = |b s| of
the normalised pair, the products' and their sum's roundings, the folded factors' and the norm's (D / 16 + 6 additions, a
root of 2 units) come to less than 2^-24 (D / 16 + 24) (A + B) before."""
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


def table(ft, rope, n, theta=1e4, mscale=1.0):
    f = torch.from_numpy(theta ** (-np.arange(rope // 2) / (rope // 2))).cuda()
    t = torch.full((n, rope), float("nan"), device="cuda")
    ft.ft_rope_table(f, rope, n, t, mscale=mscale)
    return t


class Case:
    def __init__(self, ft, fmt="nvfp4", D=128, hq=4, hkv=2, n=9, rope=None, norm=True, inter=False, seed=0, page=16, skip=(), L=2, layer=1,
                 k_scale=0.5, v_scale=0.25, n_positions=300, eps=1e-6, extra=0, n_pages=None):
        rng = np.random.default_rng(seed)
        self.ft, self.fmt, self.D, self.hq, self.hkv, self.n, self.layer = ft, fmt, D, hq, hkv, n, layer
        self.rope = D if rope is None else rope
        self.inter, self.eps, self.n_positions, self.scales = inter, eps, n_positions, (k_scale, v_scale)
        width = (hq + 2 * hkv) * D + extra
        qkv = rng.standard_normal((n, width)).astype(np.float32)
        qkv[:, hq * D:(hq + hkv) * D] *= np.exp(0.6 * rng.standard_normal(hkv * D))
        self.qkv = torch.from_numpy(qkv).to(torch.bfloat16).cuda()
        self.q, self.k, self.v = self.qkv[:, :hq * D], self.qkv[:, hq * D:(hq + hkv) * D], self.qkv[:, (hq + hkv) * D:(hq + 2 * hkv) * D]
        self.norms = [torch.from_numpy((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)).cuda() for _ in range(2)] if norm else [None, None]
        n_pages = n_pages or -(-n // page) + 3
        self.page = page
        self.slots_np = rng.permutation(n_pages * page)[:n].astype(np.int32)
        for i in skip:
            self.slots_np[i] = -1
        self.slots = torch.from_numpy(self.slots_np).cuda()
        self.pos_np = rng.integers(0, n_positions, n).astype(np.int32)
        self.positions = torch.from_numpy(self.pos_np).cuda()
        self.table = table(ft, self.rope, n_positions) if self.rope else None
        pool = torch.full((L * n_pages * page * K.tile_bytes(D, fmt) * hkv // 16,), 0xEE, dtype=torch.uint8, device="cuda")
        self.kv = ft.KVCache(L, n_pages, page, hkv, D, hq, 1, fmt, k_scale, v_scale, pool=pool)

    def run(self, q_out=None, k_out=True, stream=None, **kw):
        n = self.n
        if q_out is None:
            q_out = torch.full((n, self.hq, self.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        if k_out is True:
            k_out = torch.full((n, self.hkv, self.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        a = dict(q=self.q, k=self.k, v=self.v, slots=self.slots, n=n, q_out=q_out, positions=self.positions if self.rope else None, rope=self.table,
                 rope_dim=self.rope, n_positions=self.n_positions, k_out=k_out, q_norm=self.norms[0], k_norm=self.norms[1], eps=self.eps,
                 interleaved=self.inter, stream=stream) | kw
        self.ft.ft_kv_append_rotated(self.kv.handle, self.layer, **a)
        return q_out, k_out

    def want(self):
        """The oracle's q, its bound, k rounded to bf16, v."""
        n, D, r = self.n, self.D, self.rope // 2
        row = np.zeros((n, 2 * r)) if not r else self.table.double().cpu().numpy()[np.clip(self.pos_np, 0, self.n_positions - 1)]
        cos, sin = row[:, :r], row[:, r:]
        q, k, v = (t.double().cpu().numpy().reshape(n, -1, D) for t in (self.q, self.k, self.v))
        wq, wk = (None if w is None else w.double().cpu().numpy() for w in self.norms)
        oq, ok = S.turn(q, wq, self.eps, cos, sin, self.inter), S.turn(k, wk, self.eps, cos, sin, self.inter)
        size = np.abs(q if wq is None else S.turn(q, wq, self.eps, cos[:, :0], sin[:, :0], self.inter))
        mag = size.copy()
        for i in range(r):
            a, b = (2 * i, 2 * i + 1) if self.inter else (i, i + r)
            c, s = np.abs(cos[:, i])[:, None], np.abs(sin[:, i])[:, None]
            mag[..., a] = size[..., a] * c + size[..., b] * s
            mag[..., b] = size[..., b] * c + size[..., a] * s
        with np.errstate(over="ignore", invalid="ignore"):
            ok = torch.from_numpy(ok.astype(np.float32)).to(torch.bfloat16)
        return oq, 2.0 ** -8 * np.abs(oq) + 2.0 ** -24 * (D / 16 + 24) * mag, ok, v

    def check(self, q_out, k_out, dead=()):
        torch.cuda.synchronize()
        oq, tol, ok, v = self.want()
        live = np.array([i for i in range(self.n) if self.slots_np[i] >= 0 and i not in dead], np.int64)
        got = q_out.double().cpu().numpy().reshape(self.n, self.hq, self.D)
        assert np.all(np.abs(got[live] - oq[live]) <= tol[live]), np.max(np.abs(got[live] - oq[live]) / tol[live])
        if k_out is not None:
            assert torch.equal(k_out.cpu().reshape(self.n, self.hkv, self.D)[live], ok[live])
        back = [torch.empty(self.n, self.hkv, self.D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        slots = torch.from_numpy(np.where(np.isin(np.arange(self.n), live), self.slots_np, -1).astype(np.int32)).cuda()
        self.ft.ft_kv_read(self.kv.handle, self.layer, slots, self.n, *back)
        for b, x, st in zip(back, (ok.float().numpy(), v.astype(np.float32)), self.scales):
            val = K.values(*K.quantise(x, self.fmt, st), self.fmt, st)
            assert torch.equal(b.cpu()[live], torch.from_numpy(val.astype(np.float32)).to(torch.bfloat16)[live])
        return live


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (20, 4), (7, 7)])
@pytest.mark.parametrize("n", [1, 2, 3, 9, 100])
def test_shapes(ft, fmt, D, hq, hkv, n):
    for rope, inter, norm in ((D, False, True), (32, True, True), (64, False, False), (32, False, True), (0, False, True), (D, True, False), (0, True, False)):
        c = Case(ft, fmt, D, hq, hkv, n, rope, norm, inter, seed=n + rope)
        c.check(*c.run())
        assert ft.ft_kv_status(c.kv.handle) == 0


@pytest.mark.parametrize("fmt,D,rope", [("nvfp4", 128, 96), ("fp8", 256, 160), ("nvfp4", 256, 192), ("fp8", 256, 224)])
@pytest.mark.parametrize("inter", [False, True])
def test_dims_that_turn_in_part(ft, fmt, D, rope, inter):
    c = Case(ft, fmt, D, 6, 3, 40, rope, True, inter)
    c.check(*c.run())


@pytest.mark.parametrize("fmt,D,hq,hkv,n", [("nvfp4", 128, 32, 8, 1500), ("fp8", 64, 20, 4, 3001), ("nvfp4", 256, 16, 2, 1001), ("fp8", 128, 5, 1, 5003)])
def test_many_tokens(ft, fmt, D, hq, hkv, n):
    c = Case(ft, fmt, D, hq, hkv, n, 64, skip=range(6, n, 7), page=64, n_positions=5000)
    q, k = c.run()
    live = c.check(q, k)
    dead = np.setdiff1d(np.arange(n), live)
    assert torch.isnan(q[dead]).all() and torch.isnan(k[dead]).all()              # padding is left as it was


def test_stored_as_append_stores(ft):
    """The bytes of the pool are those that ft_kv_append writes of k_out and v, and no other byte changes."""
    for fmt, D in (("nvfp4", 64), ("fp8", 128), ("nvfp4", 256)):
        c = Case(ft, fmt, D, 4, 2, 50, 64, skip=(0, 9, 49))
        _, k = c.run()
        other = Case(ft, fmt, D, 4, 2, 50, 64, skip=(0, 9, 49))
        ft.ft_kv_append(other.kv.handle, other.layer, k.nan_to_num(), other.v, other.slots, 50)
        torch.cuda.synchronize()
        assert torch.equal(c.kv.pool, other.kv.pool)


def test_only_one_norm_and_no_k_out(ft):
    for which in (0, 1):
        c = Case(ft, n=20)
        c.norms[which] = None
        q, k = c.run(k_out=None)
        c.check(q, k)


def test_in_place_and_strides(ft):
    """q and k turned where they stand, in the projection's output; outputs among other data; the rest untouched."""
    c = Case(ft, "fp8", 64, 4, 2, 30, 32, extra=8)
    ref, keep = Case(ft, "fp8", 64, 4, 2, 30, 32, extra=8), c.qkv.clone()
    a = ref.run()
    c.run(q_out=c.q, k_out=c.k)
    torch.cuda.synchronize()
    assert torch.equal(c.q.reshape(30, 4, 64), a[0]) and torch.equal(c.k.reshape(30, 2, 64), a[1]) and torch.equal(c.qkv[:, 384:], keep[:, 384:])
    assert torch.equal(c.kv.pool, ref.kv.pool)
    wide = torch.full((30, 1000), 3.0, dtype=torch.bfloat16, device="cuda")
    ref.run(q_out=wide[:, 8:264], k_out=wide[:, 272:400])
    torch.cuda.synchronize()
    assert torch.equal(wide[:, 8:264].reshape(30, 4, 64), a[0]) and torch.equal(wide[:, 272:400].reshape(30, 2, 64), a[1])
    assert (wide[:, :8] == 3).all() and (wide[:, 264:272] == 3).all() and (wide[:, 400:] == 3).all()


@pytest.mark.parametrize("D,fmt", [(64, "fp8"), (128, "nvfp4"), (256, "nvfp4")])
def test_values_that_are_hard(ft, D, fmt):
    """Zero heads, one large dim, tiny and huge values, NaN and infinities: nothing leaves its token and head."""
    c = Case(ft, fmt, D, 4, 2, 24, 64 if D > 64 else 32)
    for t, base in ((c.q, 4), (c.k, 2)):
        x = t.view(24, base, D)
        x[0] = 0
        x[1] = 0
        x[1, :, D - 1] = 100.0
        x[2] *= 1e-18
        x[3] *= 1e15
        x[4, 0] = 1e-30
        x[5, 0] *= 2.0 ** -60
    c.check(*c.run())
    inf, nan = float("inf"), float("nan")
    for t, base in ((c.q, 4), (c.k, 2)):
        x = t.view(24, base, D)
        x[6, 0, 3], x[7, 0, 5], x[8, 0, D - 1], x[9, 0] = nan, inf, -inf, 3e38
    c.v.view(24, 2, D)[6, 0, 3], c.v.view(24, 2, D)[7, 1, 5] = nan, inf
    q, k = c.run()
    torch.cuda.synchronize()
    clean = [i for i in range(24) if i not in (6, 7, 8, 9)]
    oq, tol, ok, _ = c.want()
    got = q.double().cpu().numpy()
    assert np.all(np.abs(got[clean] - oq[clean]) <= tol[clean]) and torch.equal(k.cpu()[clean], ok[clean])
    for i in (6, 7, 8, 9):                                       # the other heads of those tokens
        assert np.all(np.abs(got[i, 1:] - oq[i, 1:]) <= tol[i, 1:]) and torch.equal(k.cpu()[i, 1:], ok[i, 1:])
    assert (got[9, 0] == 0).all() and (k[9, 0] == 0).all()       # squares past fp32's range
    back = [torch.empty(24, 2, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ft.ft_kv_read(c.kv.handle, 1, c.slots, 24, *back)
    assert all(torch.isfinite(b).all() for b in back)
    # without a norm an infinity that does not turn stays one, and is stored as the largest value
    if D > 64:
        c = Case(ft, fmt, D, 4, 2, 3, 64, norm=False)
        c.q.view(3, 4, D)[0, 1, 70], c.k.view(3, 2, D)[0, 1, 70] = inf, -inf
        q, k = c.run()
        assert torch.isposinf(q[0, 1, 70]) and torch.isneginf(k[0, 1, 70]) and torch.isfinite(q[1:]).all()
        assert torch.isfinite(q[0, 1]).sum() == D - 1 and torch.isfinite(k[0, 1]).sum() == D - 1


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rope,fmt", [(64, 64, "fp8"), (128, 128, "nvfp4"), (256, 128, "nvfp4")])
def test_keys_at_the_end_of_the_range(ft, D, rope, fmt, inter):
    """Keys without a norm whose turn may leave fp32's range: an infinity then, stored as the largest value, not a NaN, and numbers
    where the formula gives one although its terms are larger."""
    c = Case(ft, fmt, D, 3, 3, 40, rope, norm=False, inter=inter)
    c.table *= 1.375                                               # as a mscale does, in numbers that fp32 holds
    rng = np.random.default_rng(D)
    x = rng.choice([-1.0, 1.0], (40, 3, D)) * np.exp2(rng.uniform(110, 127.99, (40, 3, D)))
    x[:10, 1] *= 2.0 ** -8                                         # these do not leave it
    x[10:20, 2] = np.where(rng.random((10, D)) < 0.9, 3.3e38, x[10:20, 2])
    c.k.copy_(torch.from_numpy(x.reshape(40, 3 * D).astype(np.float32)).to(torch.bfloat16))
    ok = c.want()[2]
    assert torch.isinf(ok).any() and not torch.isnan(ok).any()
    c.check(*c.run())


def test_places_that_are_none(ft):
    """Slots outside the cache, positions outside the table: skipped, reported, the rest served."""
    c = Case(ft, "nvfp4", 128, 4, 2, 12, 64)
    before = c.kv.pool.clone()
    c.slots[2], c.slots[5], c.positions[7], c.positions[8] = -2, 1 << 30, -1, c.n_positions
    c.slots_np[2], c.slots_np[5] = -1, -1
    q, k = c.run()
    live = c.check(q, k, dead=(7, 8))
    assert ft.ft_kv_status(c.kv.handle) == ft.FT_DEV_BAD_ID and ft.ft_kv_status(c.kv.handle) == 0
    dead = np.setdiff1d(np.arange(12), live)
    assert dead.tolist() == [2, 5, 7, 8] and torch.isnan(q[dead]).all() and torch.isnan(k[dead]).all()
    c.slots[:] = -1
    now = c.kv.pool.clone()
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(now, c.kv.pool) and not torch.equal(before, now) and ft.ft_kv_status(c.kv.handle) == 0
    c.run(n=0, q=None, k=None, v=None, slots=None, q_out=None, q_stride=512, k_stride=256, v_stride=256, q_out_stride=512, k_out=None)


def test_far_slots(ft):
    """A pool past 4 GiB."""
    c = Case(ft, "fp8", 256, 8, 8, 6, 64, page=256, n_pages=4300, L=1, layer=0)
    c.slots_np[:] = [0, 1100799, 1100000, 524288, 524287, 1048576]
    c.slots.copy_(torch.from_numpy(c.slots_np))
    assert c.kv.pool_bytes > 1 << 32
    c.check(*c.run())


def test_streams_and_graphs(ft):
    c = Case(ft, "nvfp4", 128, 8, 2, 64, 128)
    a = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = c.run(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    g = torch.cuda.CUDAGraph()
    out = [torch.zeros_like(x) for x in a]
    with torch.cuda.graph(g):
        c.run(q_out=out[0], k_out=out[1])
    d = Case(ft, "nvfp4", 128, 8, 2, 64, 128, seed=5)
    c.qkv.copy_(d.qkv)
    c.positions.copy_(d.positions)
    c.pos_np = d.pos_np
    g.replay()
    c.check(*out)


@pytest.mark.parametrize("rope,n,theta,mscale", [(2, 5, 1e4, 1.0), (64, 1000, 1e4, 1.0), (128, 300000, 1e6, 1.2), (256, 7, 5e5, 0.5)])
def test_rope_table(ft, rope, n, theta, mscale):
    """Each entry within half a step of fp32 of the function of the fp64 angle (whose own error is 2^-53 of it)."""
    t = table(ft, rope, n, theta, mscale).double().cpu().numpy()
    f = theta ** (-np.arange(rope // 2) / (rope // 2))
    pick = np.unique(np.concatenate([np.arange(min(n, 50)), np.random.default_rng(0).integers(0, n, 500), [n - 1]]))
    a = pick[:, None] * f
    want = mscale * np.concatenate([np.cos(a), np.sin(a)], 1)
    assert np.all(np.abs(t[pick] - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -50 * np.concatenate([a, a], 1) + 2.0 ** -50) and np.isfinite(t).all()


def test_refusals(ft):
    c = Case(ft, "nvfp4", 128, 4, 2, 5, 64)
    raw = c.q.data_ptr()
    for bad in (dict(n=-1), dict(rope_dim=-32), dict(rope_dim=16), dict(rope_dim=160), dict(n_positions=0), dict(interleaved=2), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(q=None, q_stride=512), dict(k=None, k_stride=512), dict(v=None, v_stride=512),
                dict(slots=None), dict(rope=None), dict(q=raw + 2, q_stride=1024), dict(k=raw + 8, k_stride=1024), dict(v=raw + 4, v_stride=1024),
                dict(q_norm=c.norms[0].data_ptr() + 4), dict(k_norm=c.norms[1].data_ptr() + 8), dict(rope=c.table.data_ptr() + 4),
                dict(q_stride=504), dict(q_stride=1020), dict(k_stride=248), dict(v_stride=1028), dict(q_out_stride=508), dict(q_out_stride=496),
                dict(k_out_stride=255), dict(k_out_stride=240)):
        with pytest.raises(ft.FtError, match="append_rotated") as ei:
            c.run(**bad)
        assert ei.value.status == ft.FT_ERR_ARG, bad
    for layer in (-1, 2):
        c.layer = layer
        with pytest.raises(ft.FtError):
            c.run()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rope,fmt", [(64, 32, "fp8"), (64, 64, "nvfp4"), (128, 128, "nvfp4"), (128, 64, "fp8"), (256, 0, "nvfp4"), (256, 160, "fp8")])
def test_a_norm_of_a_nan_or_an_infinity(ft, D, rope, fmt, inter):
    """A NaN makes every dim of its head one; an infinity leaves zeros and, where it and its partner stand, NaN.  Both are stored as
    such, in whichever lane they stand."""
    c = Case(ft, fmt, D, 3, 3, 60, rope, inter=inter)
    rng = np.random.default_rng(D + rope)
    q, k = c.q.view(60, 3, D), c.k.view(60, 3, D)
    for i in range(60):
        d = i * D // 60 if i < 50 else int(rng.integers(0, D))
        value = [float("nan"), float("inf"), float("-inf")][i % 3]
        q[i, i % 2, d] = value
        k[i, i % 2, d] = value
    q_out, k_out = c.run()
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        oq, tol, ok, _ = c.want()
    got = q_out.double().cpu().numpy()
    none = np.isnan(oq)
    assert np.array_equal(np.isnan(got), none) and np.all(np.abs(got - oq)[~none] <= tol[~none])
    assert torch.equal(k_out.cpu().isnan(), ok.isnan()) and torch.equal(k_out.cpu().nan_to_num(), ok.nan_to_num())
    assert ok[0, 0].isnan().all() and not ok[1, 1].isnan().all()
    back = torch.empty(60, 3, D, dtype=torch.bfloat16, device="cuda")
    ft.ft_kv_read(c.kv.handle, c.layer, c.slots, 60, back, torch.empty_like(back))
    val = K.values(*K.quantise(ok.float().numpy(), fmt, c.scales[0]), fmt, c.scales[0])
    assert torch.equal(back.cpu(), torch.from_numpy(val.astype(np.float32)).to(torch.bfloat16))


@pytest.mark.parametrize("D,rope,fmt", [(64, 32, "fp8"), (128, 128, "nvfp4"), (256, 96, "nvfp4")])
@pytest.mark.parametrize("eps", [1.5e-45, 1e-42, 3e-39, 1.2e-38, 1e-30, 1e-3, 1e30, 3.4e38])
def test_norms_at_the_ends_of_the_range(ft, D, rope, fmt, eps):
    """Any positive eps, with heads of zeros and of values up to 2^60: the norm stays good to 2^-40 as long as eps or the squares do not
    lie below some 2^-100 (other heads are left out here where eps is)."""
    c = Case(ft, fmt, D, 3, 3, 200, rope, eps=eps)
    rng = np.random.default_rng(D)
    for t in (c.q, c.k):
        x = t.view(200, 3, D)
        x[:150] *= torch.from_numpy(np.exp2(rng.uniform(-40 if eps < 1e-30 else -60, 58, (150, 3, 1))).astype(np.float32)).to(torch.bfloat16).cuda()
        x[::7] = 0
        x[1::7, 1] = 0
        x[3, :, 1:] = 0                                            # one dim of a head
    q_out, k_out = c.run()
    # a number of bf16 below 2^-126 is a multiple of 2^-133, so its rounding may be off by 2^-134 (and the two products' and the sum's before
    # it, below fp32's 2^-126, by 3 times 2^-150)
    oq, tol, _, _ = c.want()
    got = q_out.double().cpu().numpy()
    assert np.all(np.abs(got - oq) <= tol + 2.0 ** -134 + 2.0 ** -148)
    small = np.abs(oq) < 2.0 ** -125
    c.check(torch.where(torch.from_numpy(small).cuda(), torch.from_numpy(oq).cuda(), q_out.double()), k_out)
