"""The quantised key/value cache and its attention against oracle.kv (fp64).

Tolerances (derived, not fitted).  With s = sm_scale q.k: products of stored values and q are
exact and summed in fp32, so |ds| <= e = sm_scale (D + 16) 2^-23 max_j sum_d |q_d k_jd| (the 16:
the roundings of the folded scales and of the exponent's argument).  The weights are rounded to
f16 (2^-11 relative, 2^-24 absolute against the row's largest) and the output to bf16 (2^-9):
  |do| <= 2^-8 |o| + (2 e + 2^-10) sum_j p_j |v_j| + len 2^-24 max |v|
  |dlse| <= e + len 2^-23 + 2^-20 + 2^-22 |lse|."""
import numpy as np
import pytest
import torch

from oracle import kv as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ft():
    import __graft_entry__ as entry
    entry.build()
    import expert_cache_gb300
    return expert_cache_gb300


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


@pytest.fixture(autouse=True, params=[0, 980], ids=["alone", "crowd"])
def crowd(request):
    """Empty sequences behind every call's own: with many of them the host has to expect much work, so the same
    small cases go by the kernels of large calls."""
    Case.crowd = request.param


class Case:
    """A cache filled through ft_kv_append (the rest of the pool holds 0xFF bytes) and the
    oracle's values of every token."""

    def __init__(self, ft, fmt="nvfp4", D=128, hkv=2, G=4, page=16, lens=(40,), nq=(1,), seed=0, L=2, layer=1,
                 k_scale=0.5, v_scale=0.25, masks=None, kmul=1.0, spare=1):
        rng = np.random.default_rng(seed)
        self.ft, self.fmt, self.D, self.hkv, self.G, self.layer = ft, fmt, D, hkv, G, layer
        self.lens, self.nq, self.masks, self.page = list(lens), list(nq), masks, page
        per = [-(-n // page) for n in lens]
        n_pages = sum(per) + 3
        order = rng.permutation(n_pages)
        stride = max(per + [1]) + spare                      # spare columns: the longest sequence the host can expect
        table = np.full((len(lens), stride), -1, np.int32)              # never read past the keys
        self.kv = ft.KVCache(L, n_pages, page, hkv, D, hkv * G, max(len(lens), 1) + self.crowd, fmt, k_scale, v_scale,
                             pool=torch.full((ft.ft_kv_required_sizes(ft.FtKvDesc(
                                 L, n_pages, page, hkv, D, hkv * G, len(lens), ft.KV_FORMATS[fmt], k_scale, v_scale,
                                 None, None))[0],), 255, dtype=torch.uint8, device="cuda"))
        self.kval, self.vval, at, slots, ks, vs = [], [], 0, [], [], []
        for s, n in enumerate(lens):
            table[s, :per[s]] = order[at:at + per[s]]
            at += per[s]
            k, v = bf16(rng, n, hkv, D, scale=kmul), bf16(rng, n, hkv, D)
            j = np.arange(n)
            slots.append(table[s, j // page] * page + j % page)
            ks.append(k)
            vs.append(v)
            for vals, x, st in ((self.kval, k, k_scale), (self.vval, v, v_scale)):
                vals.append(K.values(*K.quantise(x.float().numpy(), fmt, st), fmt, st))
        slots = np.concatenate(slots).astype(np.int32)
        if slots.size:
            ft.ft_kv_append(self.kv.handle, layer, torch.cat(ks).cuda(), torch.cat(vs).cuda(),
                            torch.from_numpy(slots).cuda(), slots.size)
        self.table_np, self.slots = table, slots
        self.table = torch.from_numpy(np.concatenate([table, np.full((self.crowd, stride), -1, np.int32)])).cuda()[:len(lens)]
        self.start_np = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        self.start = torch.from_numpy(np.concatenate([self.start_np, np.repeat(self.start_np[-1:], self.crowd)])).cuda()
        self.len_dev = torch.tensor(self.lens + [0] * self.crowd, dtype=torch.int32, device="cuda")[:len(lens)]
        self.T = int(self.start_np[-1])
        self.q = bf16(rng, self.T, hkv * G, D)
        self.scale = 1.0 / np.sqrt(D)
        self.tree = None
        if masks is not None:
            flat = np.array([m for ms in masks for m in ms], np.uint64).view(np.int64)
            self.tree = torch.from_numpy(flat).cuda()

    def run(self, window=0, n_sink=0, lse=True, max_q=None, q=None, o=None, stream=None):
        q = self.q.cuda() if q is None else q
        o = torch.full((self.T, self.hkv * self.G, self.D), float("nan"), dtype=torch.bfloat16, device="cuda") if o is None else o
        z = torch.full((self.T, self.hkv * self.G), float("nan"), device="cuda") if lse else None
        self.ft.ft_kv_attention(self.kv.handle, self.layer, q, self.start, self.len_dev, self.table, self.table.stride(0),
                                len(self.lens) + self.crowd, self.T, max_q or max(self.nq), o, tree_mask=self.tree, window=window,
                                n_sink=n_sink, sm_scale=self.scale, lse=z, stream=stream)
        return o, z

    def check(self, o, z, window=0, n_sink=0, rows=None):
        torch.cuda.synchronize()
        o = o.double().cpu().numpy()
        z = None if z is None else z.double().cpu().numpy()
        q = self.q.double().numpy()
        for s, (n, length) in enumerate(zip(self.nq, self.lens)):
            vis = K.seen(n, length, window, n_sink, None if self.masks is None else self.masks[s])
            at = self.start_np[s]
            pick = range(n) if rows is None else [r for r in rows if r < n]
            for h in range(self.hkv * self.G):
                k, v = self.kval[s][:, h // self.G], self.vval[s][:, h // self.G]
                ro, rl, av, mag = K.attention(q[at + np.array(pick, int), h] if len(pick) else q[:0, h], k, v, vis[list(pick)],
                                              self.scale)
                for x, i in enumerate(pick):
                    got = o[at + i, h]
                    if not vis[i].any():
                        assert not got.any(), (s, i, h)
                        assert z is None or np.isneginf(z[at + i, h])
                        continue
                    e = self.scale * (self.D + 16) * 2.0 ** -23 * mag[x]
                    tol = 2.0 ** -8 * np.abs(ro[x]) + (2 * e + 2.0 ** -10) * av[x] + length * 2.0 ** -24 * np.abs(v).max()
                    assert np.all(np.abs(got - ro[x]) <= tol), (s, i, h, np.max(np.abs(got - ro[x]) / tol))
                    if z is not None:
                        assert abs(z[at + i, h] - rl[x]) <= e + length * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22 * abs(rl[x])

    def both(self, **kw):
        o, z = self.run(**kw)
        self.check(o, z, **kw)
        return o, z


def tree(rng, n):
    out = []
    for j in range(n):
        p = int(rng.integers(max(-1, j - 4), j)) if j else -1
        out.append((out[p] if p >= 0 else 0) | 1 << j)
    return out


# ------------------------------------------------------------------------------ write and read

@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
@pytest.mark.parametrize("D,hkv,page,n", [(64, 1, 16, 1), (128, 3, 32, 37), (256, 2, 64, 130), (64, 8, 256, 515), (128, 1, 128, 16)])
def test_append_is_bit_exact_and_reads_back(ft, fmt, D, hkv, page, n):
    rng = np.random.default_rng(n)
    n_pages, L = -(-n // page) + 2, 2
    kv = ft.KVCache(L, n_pages, page, hkv, D, hkv, 1, fmt, 0.37, 1.9)
    kv.pool.fill_(0xA5)
    x = rng.standard_normal((2, n, hkv, D)).astype(np.float32) * np.exp(2 * rng.standard_normal((2, n, hkv, 1)))
    x[:, 0, :, :16] = 0.0                                  # a zero block
    x[0, n // 2, 0, 16:20] = [np.nan, np.inf, -np.inf, -0.0]
    x[1, n // 3, 0, :4] = [3e38, -3e38, 1e-38, np.nan]     # saturation, underflow
    x[0, n - 1, hkv - 1, 32:48] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 2     # ties of a scale of 1 / st
    x = torch.from_numpy(x).to(torch.bfloat16)
    slots = rng.permutation(n_pages * page)[:n].astype(np.int32)
    if n > 2:
        slots[1] = -1
    # rows inside a wider buffer
    wide = torch.zeros(n, 2 * hkv * D + 8, dtype=torch.bfloat16)
    wide[:, :hkv * D], wide[:, hkv * D + 8:] = x[0].reshape(n, -1), x[1].reshape(n, -1)
    wide, sd = wide.cuda(), torch.from_numpy(slots).cuda()
    before = kv.pool.clone()
    ft.ft_kv_append(kv.handle, 1, wide, wide[:, hkv * D + 8:], sd, n)
    torch.cuda.synchronize()
    pool = kv.pool.cpu().numpy().reshape(L, -1)
    assert np.array_equal(pool[0], before.cpu().numpy().reshape(L, -1)[0])      # the other layer is untouched
    want = before.cpu().numpy().reshape(L, n_pages, hkv, page // 16, K.tile_bytes(D, fmt))[1].copy()
    vals = []
    for which, st in ((0, 0.37), (1, 1.9)):
        codes, sc = K.quantise(x[which].float().numpy(), fmt, st)
        val = K.values(codes, sc, fmt, st)
        val[slots < 0] = 0
        vals.append(val)
        for i in np.flatnonzero(slots >= 0):
            page_i, r = divmod(int(slots[i]), page)
            for h in range(hkv):
                tile = want[page_i, h, r // 16]
                for d in range(D):
                    byte, nib = K.code_place(r % 16, d, D, fmt, which == 1)
                    c = int(codes[i, h, d])
                    tile[byte] = c if fmt == "fp8" else (tile[byte] & (0x0F if nib else 0xF0)) | c << (4 * nib)
                if fmt == "nvfp4":
                    for b in range(D // 16):
                        tile[K.scale_place(r % 16, b, D, which == 1)] = sc[i, h, b]
    assert np.array_equal(pool[1].reshape(want.shape), want)
    ko, vo = (torch.full((n, hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ft.ft_kv_read(kv.handle, 1, sd, n, ko, vo)
    torch.cuda.synchronize()
    for got, val in ((ko, vals[0]), (vo, vals[1])):
        ref = torch.from_numpy(val.astype(np.float32)).to(torch.bfloat16)       # one fp32 rounding, then bf16
        assert torch.equal(got.cpu(), ref)
    assert ft.ft_kv_status(kv.handle) == 0


def test_slots_outside_the_cache_are_skipped_and_reported(ft):
    kv = ft.KVCache(1, 2, 16, 1, 64, 1, 1)
    kv.pool.zero_()
    one = float(K.values(*K.quantise(np.ones((1, 64), np.float32), "nvfp4", 1.0), "nvfp4", 1.0)[0, 0])
    k = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (32, 2 ** 31 - 1, -2):
        slots = torch.tensor([bad, 5, -1], dtype=torch.int32, device="cuda")
        ft.ft_kv_append(kv.handle, 0, k, k, slots, 3)
        assert ft.ft_kv_status(kv.handle) == ft.FT_DEV_BAD_ID
        assert ft.ft_kv_status(kv.handle) == 0
        ko, vo = torch.full_like(k, 9.0), torch.full_like(k, 9.0)
        ft.ft_kv_read(kv.handle, 0, slots, 3, ko, vo)
        assert ft.ft_kv_status(kv.handle) == ft.FT_DEV_BAD_ID
        assert ko[:, 0, 0].tolist() == [0, one, 0] and vo[:, 0, 0].tolist() == [0, one, 0]
    kv.close()


def test_pool_past_four_gigabytes(ft):
    D, page, hkv = 128, 16, 1
    n_pages = (5 << 30) // K.tile_bytes(D, "fp8")
    kv = ft.KVCache(1, n_pages, page, hkv, D, 2, 1, "fp8")
    rng = np.random.default_rng(4)
    n = 40
    k, v = bf16(rng, n, hkv, D), bf16(rng, n, hkv, D)
    table = np.array([[n_pages - 1, 0, n_pages // 2 + 3]], np.int32)
    slots = np.array([table[0, j // page] * page + j % page for j in range(n)], np.int32)
    ft.ft_kv_append(kv.handle, 0, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), n)
    q = bf16(rng, 1, 2, D)
    o, z = torch.empty(1, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 2, device="cuda")
    ft.ft_kv_attention(kv.handle, 0, q.cuda(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), torch.from_numpy(table).cuda(), 3, 1, 1, 1, o,
                       sm_scale=0.1, lse=z)
    kk, vv = (K.values(*K.quantise(x.float().numpy(), "fp8", 1.0), "fp8", 1.0)[:, 0] for x in (k, v))
    for h in range(2):
        ro, rl, _, _ = K.attention(q.double().numpy()[:, h], kk, vv, np.ones((1, n), bool), 0.1)
        assert np.allclose(o[:, h].double().cpu().numpy(), ro, rtol=2 ** -8, atol=2 ** -9)
        assert np.allclose(z[:, h].double().cpu().numpy(), rl, atol=1e-5)
    assert ft.ft_kv_status(kv.handle) == 0


# ------------------------------------------------------------------------------ attention

@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 5, 8, 20])
def test_one_new_token(ft, fmt, D, G):
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 100, 257, 700]
    Case(ft, fmt, D, 2, G, 16 if G < 8 else 64, lens, [1] * len(lens), seed=G).both()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(ft, page):
    lens = [page - 1, page, page + 1, 3 * page + 5]
    Case(ft, "nvfp4", 128, 1, 4, page, lens, [1, 2, 1, 3], seed=page).both()


@pytest.mark.parametrize("fmt,D,hkv,G", [("nvfp4", 128, 1, 2), ("fp8", 64, 2, 3), ("nvfp4", 256, 1, 8), ("fp8", 128, 1, 1)])
def test_chunks_of_every_length(ft, fmt, D, hkv, G):
    nq = [1, 3, 16, 33, 65, 130, 7, 1]
    lens = [1, 3, 40, 33, 200, 131, 300, 90]
    Case(ft, fmt, D, hkv, G, 32, lens, nq, seed=D).both()


@pytest.mark.parametrize("fmt,D", [("nvfp4", 64), ("fp8", 256)])
def test_long_chunk(ft, fmt, D):
    Case(ft, fmt, D, 1, 4, 64, [900], [300], seed=3).both()


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 3), (16, 0), (17, 4), (50, 16), (64, 100), (10 ** 9, 5), (0, 7), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_window_and_sinks(ft, window, n_sink):
    Case(ft, "nvfp4", 64, 2, 4, 16, [1, 30, 300, 77, 200], [1, 9, 1, 77, 40], seed=9).both(window=window, n_sink=n_sink)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (1, 0), (3, 2), (40, 4)])
@pytest.mark.parametrize("fmt,D,G", [("nvfp4", 128, 4), ("fp8", 64, 1), ("nvfp4", 256, 8)])
def test_trees(ft, fmt, D, G, window, n_sink):
    rng = np.random.default_rng(11)
    nq, lens = [1, 7, 64, 20, 64], [50, 7, 64, 333, 300]
    masks = [tree(rng, n) for n in nq]
    masks[1][3] = 0                                          # sees nothing: 7 cached, 7 drafted
    masks[3][5] = 0                                          # sees the context only
    masks[3][2] |= 1 << 63 | 1 << 40                         # bits past the drafted tokens
    Case(ft, fmt, D, 2, G, 16, lens, nq, seed=5, masks=masks).both(window=window, n_sink=n_sink)


def test_rows_that_see_nothing(ft):
    # nothing cached; fewer cached than new
    Case(ft, "nvfp4", 128, 2, 4, 16, [0, 3, 20, 0], [1, 9, 2, 5]).both()
    Case(ft, "fp8", 64, 1, 2, 16, [0, 3, 100], [1, 64, 70]).both(window=5, n_sink=1)
    c = Case(ft, "fp8", 64, 1, 2, 16, [0], [2], masks=[[1, 3]])
    c.both()


@pytest.mark.parametrize("nq", [1, 40])
def test_no_rows_and_empty_batches(ft, nq):
    c = Case(ft, "nvfp4", 64, 1, 4, 16, [30, 20, 40], [nq, 0, nq], seed=1)
    c.both()
    o = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    c.ft.ft_kv_attention(c.kv.handle, 0, c.q.cuda(), c.start, c.len_dev, c.table, c.table.stride(0), 0, 0, 1, o)
    torch.cuda.synchronize()


@pytest.mark.parametrize("mul", [0.01, 8.0, 40.0])
def test_flat_and_peaked_logits(ft, mul):
    for n in (1, 40):
        Case(ft, "nvfp4", 128, 1, 8, 64, [500, 90], [n, n], seed=2, kmul=mul, k_scale=0.02 * mul).both()


def test_large_and_small_queries(ft):
    c = Case(ft, "fp8", 64, 1, 4, 16, [120, 90], [1, 50], seed=6, k_scale=1.0)
    mul = torch.tensor([1e-30, 1.0, 1e4, 1e30]).to(torch.bfloat16)[None, :, None]
    c.q = (c.q * mul).to(torch.bfloat16)
    c.scale = 1e-4
    o, z = c.run()
    torch.cuda.synchronize()
    q = c.q.double().numpy()
    for s, n in enumerate(c.nq):
        vis = K.seen(n, c.lens[s])
        for h in range(4):
            at = c.start_np[s]
            ro, rl, av, mag = K.attention(q[at:at + n, h], c.kval[s][:, 0], c.vval[s][:, 0], vis, c.scale)
            got = o[at:at + n, h].double().cpu().numpy()
            e = np.minimum(c.scale * (c.D + 16) * 2.0 ** -23 * mag, 1.0)[:, None]
            if h < 3:
                assert np.all(np.abs(got - ro) <= 2.0 ** -8 * np.abs(ro) + (2 * e + 2.0 ** -10) * av + 1e-4), (s, h)
            else:                                            # one key takes all, and ties are far apart
                assert np.all(np.isfinite(got)) and np.all(np.abs(got) <= np.abs(c.vval[s]).max() * 1.01)


def test_non_finite_queries_stay_in_their_row(ft):
    for n in (1, 30):
        c = Case(ft, "nvfp4", 128, 1, 4, 16, [60, 50], [n, n], seed=8)
        o, z = c.run()
        q = c.q.clone()
        q[0, 1, 5], q[0, 2, 0], q[n, 3, 9] = float("nan"), float("inf"), float("nan")
        o2, z2 = c.run(q=q.cuda())
        torch.cuda.synchronize()
        keep = torch.ones(c.T, 4, dtype=torch.bool)
        keep[0, 1] = keep[0, 2] = keep[n, 3] = False
        assert torch.equal(o.cpu()[keep], o2.cpu()[keep]) and torch.equal(z.cpu()[keep], z2.cpu()[keep])
        assert not torch.isfinite(o2[0, 1].float()).any() and not torch.isfinite(o2[n, 3].float()).any()


@pytest.mark.parametrize("nq", [1, 3, 40])
def test_strides_streams_and_runs(ft, nq):
    c = Case(ft, "nvfp4", 128, 2, 4, 16, [300, 77], [nq, nq], seed=7)
    o, z = c.both()
    wide_q = torch.full((c.T, 8 * 128 + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_q[:, :1024] = c.q.reshape(c.T, -1).cuda()
    wide_o = torch.full((c.T, 8 * 128 + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(q=wide_q, o=wide_o, lse=False)
    torch.cuda.synchronize()
    assert torch.equal(wide_o[:, :1024].reshape(o.shape), o)
    assert torch.all(wide_o[:, 1024:] == 5.0)
    for _ in range(3):                                       # the same bits every time
        o2, z2 = c.run()
        assert torch.equal(o, o2) and torch.equal(z, z2)
    g = torch.cuda.CUDAGraph()                               # captured, with other lengths at replay
    q, buf = c.q.cuda(), torch.empty_like(o)
    c.run(q=q, o=buf, lse=False)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.run(q=q, o=buf, lse=False, stream=torch.cuda.current_stream())
    c.len_dev.copy_(torch.tensor([123, 60], dtype=torch.int32))
    g.replay()
    c.lens = [123, 60]
    c.kval, c.vval = [x[:n] for x, n in zip(c.kval, c.lens)], [x[:n] for x, n in zip(c.vval, c.lens)]
    c.check(buf, None)


@pytest.mark.parametrize("nq", [1, 40])
def test_what_the_host_cannot_see_is_bounded(ft, nq):
    def fresh():
        return Case(ft, "fp8", 64, 1, 2, 16, [100, 60], [nq, nq], seed=3)
    c = fresh()                                              # a page outside the cache: its keys are not seen
    c.table[0, 2] = 10 ** 6
    o, z = c.run()
    assert ft.ft_kv_status(c.kv.handle) == ft.FT_DEV_BAD_ID
    q = c.q.double().numpy()
    vis = K.seen(nq, 100)
    vis[:, 32:48] = False
    for h in range(2):
        ro, rl, av, _ = K.attention(q[:nq, h], c.kval[0][:, 0], c.vval[0][:, 0], vis, c.scale)
        assert np.all(np.abs(o[:nq, h].double().cpu().numpy() - ro) <= 2.0 ** -8 * np.abs(ro) + 2.0 ** -9 * av)
    c = fresh()                                              # a length past the table: as far as the table goes
    c.len_dev[1] = 10 ** 9
    c.run()
    assert ft.ft_kv_status(c.kv.handle) & ft.FT_DEV_BAD_ID
    c = fresh()                                              # rows past the tensors
    c.start[2] = 10 ** 6
    o, _ = c.run()
    assert ft.ft_kv_status(c.kv.handle) == ft.FT_DEV_BAD_ID
    c = fresh()
    c.start[0] = -5
    c.run()
    assert ft.ft_kv_status(c.kv.handle) == ft.FT_DEV_BAD_ID
    if nq > 1:                                               # more rows than max_q: the rest stay as they are
        c = fresh()
        o, _ = c.run(max_q=nq - 1)
        assert ft.ft_kv_status(c.kv.handle) == ft.FT_DEV_BAD_ID
        assert torch.isnan(o[nq - 1].float()).all() and torch.isfinite(o[:nq - 1].float()).all()


def test_refusals(ft):
    c = Case(ft, "fp8", 64, 1, 2, 16, [30], [1], seed=3)
    h, q = c.kv.handle, c.q.cuda()
    o = torch.empty(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    good = dict(layer=0, q=q, q_start=c.start, kv_len=c.len_dev, block_table=c.table, table_stride=c.table.stride(0),
                n_seqs=1, n_tokens=1, max_q=1, o=o)
    ft.ft_kv_attention(h, **good)
    bad = [dict(layer=-1), dict(layer=2), dict(n_seqs=-1), dict(n_seqs=c.crowd + 2), dict(n_tokens=-1), dict(table_stride=0),
           dict(max_q=0), dict(max_q=65, tree_mask=c.start), dict(max_q=(1 << 29) + 1), dict(window=-1), dict(n_sink=-1), dict(sm_scale=float("nan")),
           dict(sm_scale=float("inf")), dict(q=None, q_stride=128), dict(o=None, o_stride=128), dict(kv_len=None),
           dict(block_table=None), dict(q_start=None), dict(q_stride=120), dict(q_stride=132), dict(o_stride=64),
           dict(q=q.data_ptr() + 2, q_stride=128), dict(o=o.data_ptr() + 8, o_stride=128)]
    for b in bad:
        with pytest.raises(ft.FtError) as ei:
            ft.ft_kv_attention(h, **{**good, **b})
        assert ei.value.status == ft.FT_ERR_ARG and "attention" in str(ei.value)
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    sl = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    ft.ft_kv_append(h, 0, k, k, sl, 0)
    ft.ft_kv_read(h, 0, sl, 0, k, k)
    for b in (dict(layer=2), dict(n=-1), dict(k=None, k_stride=64), dict(slots=None), dict(k_stride=56), dict(v_stride=66),
              dict(v=k.data_ptr() + 2, v_stride=64)):
        with pytest.raises(ft.FtError) as ei:
            ft.ft_kv_append(h, **{**dict(layer=0, k=k, v=k, slots=sl, n=2), **b})
        assert ei.value.status == ft.FT_ERR_ARG
    for b in (dict(layer=-1), dict(n=-1), dict(k_out=None), dict(v_out=k.data_ptr() + 2), dict(slots=None)):
        with pytest.raises(ft.FtError) as ei:
            ft.ft_kv_read(h, **{**dict(layer=0, slots=sl, n=2, k_out=k, v_out=k), **b})
        assert ei.value.status == ft.FT_ERR_ARG
    d = ft.FtKvDesc(1, 2, 16, 1, 64, 2, 1, 0, 1.0, 1.0, c.kv.pool.data_ptr(), torch.zeros(256, dtype=torch.uint8).data_ptr())
    with pytest.raises(ft.FtError) as ei:                   # host workspace
        ft.ft_kv_create(d)
    assert ei.value.status == ft.FT_ERR_ARG
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_whole_tiles_and_loose_tokens(ft, fmt, D):
    """Many tokens in one call: tiles in order, tiles cut by padding or by a jump, tokens in
    reverse, a start inside a tile, an odd end; bit-exact like the calls of few tokens."""
    rng = np.random.default_rng(D)
    hkv, page, n_pages, st = 8, 32, 40, (0.37, 1.9)
    runs = [np.arange(5, 5 + 70), np.arange(200, 264), np.array([-1]), np.arange(320, 352)[::-1], np.arange(400, 416),
            np.array([640]), np.arange(417, 431), np.arange(801, 801 + 300)]
    slots = np.concatenate(runs).astype(np.int32)
    assert len(set(slots)) == slots.size
    slots[100] = -1
    while slots.size * hkv < 5000:                           # enough rows for the calls by tiles
        slots = np.concatenate([slots, np.arange(1104, 1104 + 160, dtype=np.int32)])
    n = slots.size
    assert len(set(slots[slots >= 0])) == (slots >= 0).sum()
    x = rng.standard_normal((2, n, hkv, D)).astype(np.float32) * np.exp(rng.standard_normal((2, n, hkv, 1)))
    x[0, ::7, 0, :4] = [np.nan, np.inf, -np.inf, -0.0]
    x[1, ::5, 1, 16:20] = [3e38, -1e-38, 1e-30, np.nan]
    x = torch.from_numpy(x).to(torch.bfloat16)
    dev = x.cuda()
    sd = torch.from_numpy(slots).cuda()
    a, b = (ft.KVCache(1, n_pages, page, hkv, D, hkv, 1, fmt, *st) for _ in range(2))
    a.pool.fill_(0x5A)
    b.pool.fill_(0x5A)
    ft.ft_kv_append(a.handle, 0, dev[0], dev[1], sd, n)
    for i in range(0, n, 300):                               # the same tokens in calls of few
        m = min(300, n - i)
        ft.ft_kv_append(b.handle, 0, dev[0, i:i + m], dev[1, i:i + m], sd[i:i + m], m)
    torch.cuda.synchronize()
    assert torch.equal(a.pool, b.pool)
    ko, vo = (torch.full((n, hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ft.ft_kv_read(a.handle, 0, sd, n, ko, vo)
    torch.cuda.synchronize()
    for got, which in ((ko, 0), (vo, 1)):
        val = K.values(*K.quantise(x[which].float().numpy(), fmt, st[which]), fmt, st[which])
        val[slots < 0] = 0
        assert torch.equal(got.cpu(), torch.from_numpy(val.astype(np.float32)).to(torch.bfloat16))
    assert ft.ft_kv_status(a.handle) == 0
    sd[3], sd[50] = -7, n_pages * page
    ft.ft_kv_append(a.handle, 0, dev[0], dev[1], sd, n)
    assert ft.ft_kv_status(a.handle) == ft.FT_DEV_BAD_ID
    ft.ft_kv_read(a.handle, 0, sd, n, ko, vo)
    assert ft.ft_kv_status(a.handle) == ft.FT_DEV_BAD_ID
    assert not ko[3].any() and not vo[50].any()


@pytest.mark.parametrize("n", [1, 5, 40])
def test_negative_and_zero_scale(ft, n):
    for scale in (-0.2, 0.0):
        c = Case(ft, "nvfp4", 128, 1, 4, 16, [150, 60], [n, n], seed=12)
        c.scale = scale
        o, z = c.run()
        torch.cuda.synchronize()
        q = c.q.double().numpy()
        for s, length in enumerate(c.lens):
            at = c.start_np[s]
            for h in range(4):
                ro, rl, av, mag = K.attention(q[at:at + n, h], c.kval[s][:, 0], c.vval[s][:, 0], K.seen(n, length), scale)
                e = (abs(scale) * (c.D + 16) * 2.0 ** -23 * mag)[:, None]
                got = o[at:at + n, h].double().cpu().numpy()
                assert np.all(np.abs(got - ro) <= 2.0 ** -8 * np.abs(ro) + (2 * e + 2.0 ** -10) * av + length * 2.0 ** -24 * np.abs(c.vval[s]).max())
                assert np.allclose(z[at:at + n, h].double().cpu().numpy(), rl, rtol=1e-6, atol=1e-5)


@pytest.mark.parametrize("fmt,D,G,page", [("nvfp4", 128, 4, 16), ("fp8", 64, 1, 64), ("nvfp4", 256, 8, 32), ("fp8", 256, 3, 16),
                                          ("fp8", 128, 16, 16), ("nvfp4", 64, 16, 128)])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (33, 5)])
def test_long_tables(ft, fmt, D, G, page, window, n_sink):
    """Tables wide enough for sequences far longer than the present ones: the same answers."""
    rng = np.random.default_rng(21)
    lens = [1, 700, 15, 0, 64, 129, 300, 17, 16, 40] + [int(x) for x in rng.integers(1, 60, 30)]
    nq = [1, 1, 1, 2, 1, 2, 1, 1, 0, 1] + [1] * 30
    kw = dict(seed=D, spare=(1 << 17) // page)
    Case(ft, fmt, D, 2, G, page, lens, nq, **kw).both(window=window, n_sink=n_sink)
    if G <= 8:
        masks = [tree(rng, n) for n in (4, 3, 1)]
        Case(ft, fmt, D, 1, G, page, [4, 260, 90], [4, 3, 1], masks=masks, **kw).both(window=window, n_sink=n_sink)
    Case(ft, fmt, D, 1, G, page, [5000], [1], **kw).both(window=window, n_sink=n_sink)


@pytest.mark.parametrize("fmt,D", [("nvfp4", 64), ("fp8", 64), ("nvfp4", 128), ("fp8", 128), ("nvfp4", 256)])
@pytest.mark.parametrize("hkv,seqs,tokens", [(4, 1, 2100), (2, 6, 2100), (4, 12, 1000)])
@pytest.mark.parametrize("kind,window,n_sink", [("causal", 0, 0), ("tree", 0, 0), ("tree", 900, 3)])
def test_units_of_many_rows_over_short_tables(ft, fmt, D, hkv, seqs, tokens, kind, window, n_sink):
    """Up to 512 rows a unit over tables of 1000 and 2100 tokens: a unit's blocks divided among a few CTAs or in one,
    some of them without a block, sequences much shorter than the table, of no rows and of no tokens."""
    rng = np.random.default_rng(D + seqs)
    lens = [tokens - 40, 64, 0, 129, 700, 3, 64, 65, 500, 1, 0, 260][:seqs]
    nq = [64, 5, 2, 64, 33, 3, 64, 17, 0, 1, 0, 50][:seqs]
    masks = [tree(rng, n) for n in nq] if kind == "tree" else None
    c = Case(ft, fmt, D, hkv, 8, 16, lens, nq, seed=hkv, masks=masks, spare=2)
    o, z = c.run(window=window, n_sink=n_sink)
    c.check(o, z, window=window, n_sink=n_sink, rows=[0, 1, 2, 4, 15, 16, 31, 32, 40, 49, 62, 63])
    assert torch.isfinite(o.float()).all() and ft.ft_kv_status(c.kv.handle) == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
def test_layers_together(ft, fmt):
    """The example: a decoder over both caches, by single tokens and by chunks and trees.  The two ways differ by
    attention's roundings (2^-8) and the order of the experts' sums; a rounding that flips in a stored key or
    an expert's input moves it by a step of its format (up to 2^-3 of an element), one in a few dozen."""
    import importlib.util
    import os
    spec = importlib.util.spec_from_file_location("tree_decode", os.path.join(os.path.dirname(os.path.dirname(
        os.path.abspath(__file__))), "examples", "tree_decode.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    rng = np.random.default_rng(1)
    prompt = rng.integers(0, ex.VOCAB, 45).tolist()
    a, la = ex.plain(prompt, 60, fmt=fmt)
    b, lb, steps = ex.by_trees(prompt, 60, a, rng, fmt=fmt)
    same = next((i for i in range(60) if a[i] != b[i]), 60)
    gap = la.topk(2).values
    assert same == 60 or (gap[same, 0] - gap[same, 1]) < 2.0 ** -4 * la[same].abs().max(), "a token that is no tie"
    # a right guess gives depth + 1 = 7 tokens a step, a wrong one still one
    assert same >= 10 and steps <= -(-same // 7) + 60 - same + 1
    assert ((la - lb)[:same].norm() / la[:same].norm()).item() < 2.0 ** -4
