"""Who sees whom at the edges: keys that no row sees, what their slots hold and where they have no page, masks with bits past the drafted
tokens, rows and lengths past what the call says.  Against oracle.kv, with test_gpu_kv's derived bounds."""
import numpy as np
import pytest
import torch

from oracle import kv as K
from test_gpu_kv import Case, crowd, ft, tree  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

SHAPES = [("nvfp4", 64, 4), ("fp8", 64, 5), ("nvfp4", 128, 4), ("fp8", 128, 8), ("nvfp4", 256, 8), ("fp8", 256, 3)]


def forget(c, s, js):
    """The bytes of sequence s's tokens js back to 0xFF, as if they had never been written."""
    pool = c.kv.pool.view(c.kv.desc.L, -1)[c.layer].view(-1, c.hkv, c.page // 16, K.tile_bytes(c.D, c.fmt))
    d = np.arange(c.D)
    for j in js:
        at = pool[int(c.table_np[s, j // c.page]), :, j % c.page // 16]
        for value in (False, True):
            where = np.unique(K.code_place(j % 16, d, c.D, c.fmt, value)[0])
            if c.fmt == "nvfp4":
                where = np.concatenate([where, [K.scale_place(j % 16, b, c.D, value) for b in range(c.D // 16)]])
            at[:, torch.from_numpy(where).cuda()] = 255


def check_rows(c, o, s, rows, vis):
    """Rows of sequence s against the oracle; vis [rows, keys] may end before or after the cached tokens."""
    n = min(vis.shape[1], c.lens[s])
    at = int(c.start_np[s]) + rows
    q = c.q.double().numpy()[at]
    for h in range(c.hkv * c.G):
        k, v = c.kval[s][:n, h // c.G], c.vval[s][:n, h // c.G]
        ro, _, av, mag = K.attention(q[:, h], k, v, vis[:, :n], c.scale)
        e = (c.scale * (c.D + 16) * 2.0 ** -23 * mag)[:, None]
        got = o[at, h].double().cpu().numpy()
        assert np.all(np.abs(got - ro) <= 2.0 ** -8 * np.abs(ro) + (2 * e + 2.0 ** -10) * av + n * 2.0 ** -24 * np.abs(v).max())


# ------------------------------------------------------------------------------ rows and lengths past the call's

@pytest.mark.parametrize("fmt,D,G", SHAPES)
@pytest.mark.parametrize("kind,window,n_sink", [("causal", 0, 0), ("causal", 40, 3), ("tree", 0, 0), ("tree", 90, 2)])
def test_the_rows_up_to_max_q_see_what_they_should(ft, fmt, D, G, kind, window, n_sink):
    rng = np.random.default_rng(D)
    for nq, most in (([9, 3], 5), ([50, 64], 33), ([100, 7], 64)):
        masks = None
        if kind == "tree":                                   # rows past the 64th are never computed
            masks = [tree(rng, min(n, 64)) + [0] * max(n - 64, 0) for n in nq]
        c = Case(ft, fmt, D, 2, G, 32, [170, 90], nq, seed=G, masks=masks)
        o, z = c.run(window=window, n_sink=n_sink, max_q=most)
        c.check(o, z, window=window, n_sink=n_sink, rows=range(most))
        assert ft.ft_kv_status(c.kv.handle) == ft.FT_DEV_BAD_ID
        for s, n in enumerate(nq):
            rest = slice(c.start_np[s] + most, c.start_np[s] + max(n, most))
            assert torch.isnan(o[rest].float()).all() and torch.isnan(z[rest]).all()


@pytest.mark.parametrize("nq", [1, 40])
def test_a_length_past_the_table_keeps_the_rows_places(ft, nq):
    c = Case(ft, "fp8", 128, 1, 4, 16, [96, 64], [nq, nq], seed=1, spare=0)
    c.len_dev[0] = 96 + 37                                   # 37 keys have no page
    for window, n_sink in ((0, 0), (60, 0), (10, 0), (10, 3), (10, 20)):
        o, _ = c.run(window=window, n_sink=n_sink)
        assert ft.ft_kv_status(c.kv.handle) == ft.FT_DEV_BAD_ID
        check_rows(c, o, 0, np.arange(nq), K.seen(nq, 96 + 37, window, n_sink))


def test_a_sequence_that_ends_past_the_rows(ft):
    """q_start[s + 1] above n_tokens: the rows that there are have their places; a start outside: no rows."""
    c = Case(ft, "nvfp4", 64, 1, 4, 16, [100, 80], [3, 20], seed=2)
    c.start[2] = 3 + 30                                      # 30 new tokens, 20 of them in the tensors
    o, z = c.run(max_q=30)
    assert ft.ft_kv_status(c.kv.handle) == ft.FT_DEV_BAD_ID
    check_rows(c, o, 1, np.arange(20), K.seen(30, 80)[:20])
    c.start[2] = 23
    c.start[0] = -5
    o, z = c.run()
    assert ft.ft_kv_status(c.kv.handle) == ft.FT_DEV_BAD_ID
    assert torch.isnan(o[:3].float()).all() and torch.isfinite(o[3:].float()).all()


# ------------------------------------------------------------------------------ bits past the drafted tokens

@pytest.mark.parametrize("fmt,D,G", SHAPES)
@pytest.mark.parametrize("n,length,window", [(40, 1524, 512), (12, 700, 300), (64, 1000, 256)])
def test_stray_bits_move_the_window_of_their_row_alone(ft, fmt, D, G, n, length, window):
    """A row stands at base + the number of its mask's other bits, whichever they are."""
    rng = np.random.default_rng(n)
    masks = tree(rng, n)
    for i in (0, 5, n - 1):
        masks[i] |= ((1 << 64) - 1) ^ ((1 << n) - 1)
    masks[7] = (1 << 64) - 1
    c = Case(ft, fmt, D, 1, G, 64, [length, 50], [n, 3], seed=n, masks=[masks, tree(rng, 3)])
    for n_sink in (0, 5):
        o, z = c.run(window=window, n_sink=n_sink)
        c.check(o, z, window=window, n_sink=n_sink, rows=[0, 1, 2, 5, 6, 7, 8, n - 2, n - 1])
    assert ft.ft_kv_status(c.kv.handle) == 0


@pytest.mark.parametrize("fmt,D,G", SHAPES)
@pytest.mark.parametrize("window", [1, 3, 20, 64, 100])
def test_trees_of_more_tokens_than_are_cached(ft, fmt, D, G, window):
    """The first drafted tokens then stand before the sequence's start, at places below 0, as do some of the keys."""
    rng = np.random.default_rng(window)
    lens, nq = [4, 20, 63, 1], [46, 24, 64, 2]
    masks = [tree(rng, n) for n in nq]
    for ms in masks:
        for i in range(0, len(ms), 3):                       # any bits
            ms[i] |= int(rng.integers(0, 1 << 62)) << 2
    c = Case(ft, fmt, D, 2, G, 16, lens, nq, seed=window, masks=masks)
    for n_sink in (0, 2):
        c.both(window=window, n_sink=n_sink)
    assert ft.ft_kv_status(c.kv.handle) == 0


# ------------------------------------------------------------------------------ keys that no row sees

@pytest.mark.parametrize("fmt,D,G", SHAPES)
@pytest.mark.parametrize("n", [1, 6, 40])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (50, 0), (50, 3), (130, 20)])
def test_keys_that_the_window_has_left_may_never_have_been_written(ft, fmt, D, G, n, window, n_sink):
    """A sequence whose cache was filled from its last tokens (and the first ones that stay): bytes of 0xFF before."""
    lens = [300, n + 11, 190]
    c = Case(ft, fmt, D, 2, G, 32, lens, [n] * 3, seed=n)
    for s, length in enumerate(lens):
        forget(c, s, np.flatnonzero(~K.seen(n, length, window, n_sink).any(0)))
    c.both(window=window, n_sink=n_sink)


@pytest.mark.parametrize("fmt,D,G", SHAPES)
@pytest.mark.parametrize("pad,window,n_sink", [("nothing", 0, 0), ("itself", 0, 0), ("nothing", 60, 2), ("itself", 2, 0)])
def test_trees_padded_to_a_fixed_size(ft, fmt, D, G, pad, window, n_sink):
    """Padding tokens have no slot, so their keys were never written; no other row has them in its mask.  A padding row
    that has itself there gets what its bytes give, and nobody else does."""
    rng = np.random.default_rng(3)
    real, nq, lens, masks = [5, 1, 40, 17], [8, 8, 64, 17], [40, 8, 164, 64], []
    for n, r in zip(nq, real):
        masks.append(tree(rng, r) + [1 << j if pad == "itself" else 0 for j in range(r, n)])
    c = Case(ft, fmt, D, 2, G, 16, lens, nq, seed=4, masks=masks)
    for s, (n, r, length) in enumerate(zip(nq, real, lens)):
        forget(c, s, range(length - n + r, length))
        if window:
            forget(c, s, np.flatnonzero(~K.seen(n, length, window, n_sink, masks[s]).any(0)))
    o, z = c.run(window=window, n_sink=n_sink)
    c.check(o, z, window=window, n_sink=n_sink, rows=None if pad == "nothing" else [0])
    if pad == "itself":
        keep = np.concatenate([np.arange(n) < r for n, r in zip(nq, real)])
        assert torch.isfinite(o.float()[torch.from_numpy(keep).cuda()]).all()
        for s, r in enumerate(real):
            check_rows(c, o, s, np.arange(r), K.seen(nq[s], lens[s], window, n_sink, masks[s])[:r])


@pytest.mark.parametrize("fmt,D,G", SHAPES)
@pytest.mark.parametrize("window,n_sink", [(0, 0), (30, 2)])
def test_prompts_padded_to_a_fixed_size(ft, fmt, D, G, window, n_sink):
    """Causal rows behind the prompt's end have no slot: they see keys that were never written, the prompt's rows do
    not, though they share blocks and products."""
    real, nq, lens = [5, 1, 40, 90], [8, 8, 64, 96], [40, 8, 164, 96]
    c = Case(ft, fmt, D, 2, G, 16, lens, nq, seed=4)
    for s, (n, r, length) in enumerate(zip(nq, real, lens)):
        forget(c, s, range(length - n + r, length))
    o, _ = c.run(window=window, n_sink=n_sink)
    torch.cuda.synchronize()
    for s, r in enumerate(real):
        check_rows(c, o, s, np.arange(r), K.seen(nq[s], lens[s], window, n_sink)[:r])


@pytest.mark.parametrize("fmt,D,G", SHAPES)
@pytest.mark.parametrize("kind", ["step", "chunk", "tree", "padded"])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (40, 0), (40, 20), (3, 17)])
def test_pages_that_no_row_needs_may_be_missing(ft, fmt, D, G, kind, window, n_sink):
    """Table entries of -1 where no row sees a key of the page: behind the window, and where only padding of a tree
    stands.  No status, and the same results."""
    rng = np.random.default_rng(5)
    lens = [300, 77, 190]
    nq = [1, 1, 1] if kind == "step" else [40, 9, 33]
    masks = None
    if kind in ("tree", "padded"):
        masks = [tree(rng, n) for n in nq]
        if kind == "padded":
            masks = [[m if j < n // 4 else 0 for j, m in enumerate(ms)] for n, ms in zip(nq, masks)]
    c = Case(ft, fmt, D, 2, G, 16, lens, nq, seed=6, masks=masks)
    gone = 0
    for s, (n, length) in enumerate(zip(nq, lens)):
        seen = K.seen(n, length, window, n_sink, None if masks is None else masks[s]).any(0)
        for p in range(-(-length // c.page)):
            if not seen[p * c.page:(p + 1) * c.page].any():
                c.table[s, p] = -1
                gone += 1
    assert gone or not window and kind != "padded"
    c.both(window=window, n_sink=n_sink)
    assert ft.ft_kv_status(c.kv.handle) == 0
    if masks is not None:                                    # a page that some row does need
        s = 0
        c.table[s, int(np.flatnonzero(K.seen(nq[s], lens[s], window, n_sink, masks[s]).any(0))[-1]) // c.page] = 10 ** 6
        c.run(window=window, n_sink=n_sink)
        assert ft.ft_kv_status(c.kv.handle) == ft.FT_DEV_BAD_ID
