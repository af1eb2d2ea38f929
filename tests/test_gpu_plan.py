"""ft_kv_plan against oracle.step (whole numbers: equal)."""
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


class State:
    """Sequences of given lengths over a pool, their pages in any order; runs a step both ways and compares."""

    def __init__(self, ft, length, page=16, stride=None, n_pages=None, held=None, seed=0, max_seqs=None, spare=4):
        rng = np.random.default_rng(seed)
        self.ft, self.page, s = ft, page, len(length)
        self.length = np.array(length, np.int64)
        self.held = np.array([-(-int(n) // page) for n in length] if held is None else held, np.int64)
        self.stride = stride or int(max([0, *self.held])) + spare
        self.n_pages = n_pages or int(self.held.sum()) + 50
        order = rng.permutation(self.n_pages)
        self.table, at = np.full((s, self.stride), -1, np.int64), 0
        for i, h in enumerate(self.held):
            self.table[i, :h] = order[at:at + h]
            at += h
        self.free = np.concatenate([order[at:], np.full(at, -7)])
        self.n_free = self.n_pages - at
        self.kv = ft.KVCache(1, self.n_pages, page, 1, 64, 1, max_seqs or max(s, 1))

    def step(self, n_new, n_tokens, masks=None, in_place=False, stream=None, positions=True):
        """Both ways; the state goes on."""
        s = len(self.length)
        want, status = S.plan(n_new, self.length, self.held, self.table, self.free, self.n_free, self.n_pages, self.page, n_tokens, masks)
        t = dict(n_new=dev(n_new), len=dev(self.length), held=dev(self.held), block_table=dev(self.table), free_pages=dev(self.free),
                 n_free=dev([self.n_free]), q_start=dev([-9] * (s + 1)), kv_len=dev([-9] * s), slots=dev([-9] * n_tokens))
        t |= dict(len_out=t["len"], held_out=t["held"], n_free_out=t["n_free"]) if in_place else dict(
            len_out=dev([-9] * s), held_out=dev([-9] * s), n_free_out=dev([-9]))
        t["positions"] = dev([-9] * n_tokens) if positions else None
        tree = None if masks is None else torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).cuda()
        torch.cuda.synchronize()
        self.ft.ft_kv_plan(self.kv.handle, n_seqs=s, n_tokens=n_tokens, table_stride=self.stride, tree_mask=tree, stream=stream, **t)
        got = self.ft.ft_kv_status(self.kv.handle)                # synchronises
        for name in ("q_start", "kv_len", "slots", "positions", "len_out", "held_out", "block_table", "free_pages"):
            if t[name] is not None:
                assert np.array_equal(t[name].cpu().numpy(), want[name]), name
        assert t["n_free_out"].item() == want["n_free_out"] and got == status
        if not in_place:
            assert np.array_equal(t["len"].cpu().numpy(), self.length) and np.array_equal(t["n_new"].cpu().numpy(), n_new)
        self.length, self.held, self.table, self.free, self.n_free = (want[k] for k in ("len_out", "held_out", "block_table", "free_pages", "n_free_out"))
        self.n_free = int(self.n_free)
        return want, status


def test_by_hand(ft):
    c = State(ft, [15, 20, 0, 30, 16], stride=3, n_pages=9)
    c.length[3] = 10                                              # drafts that were rejected
    want, status = c.step([3, -1, 20, 1, 0], 30)
    assert status == 0 and want["kv_len"].tolist() == [18, 0, 20, 11, 16] and want["held_out"].tolist() == [2, 0, 2, 1, 1]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("s,page,n_tokens", [(1, 16, 1), (1, 256, 300), (7, 32, 100), (40, 16, 3000), (300, 64, 5000), (1024, 16, 9000), (1023, 128, 40000)])
def test_many_steps(ft, s, page, n_tokens, in_place):
    """Growing, waiting, ending and starting again, drafts rejected; pages run out now and then."""
    rng = np.random.default_rng(s + page)
    most = max(1, n_tokens // s)
    c = State(ft, rng.integers(0, 5 * page, s), page, stride=12, n_pages=8 * s + 3, seed=s)
    seen = 0
    for i in range(12):
        kind = rng.random(s)
        n = np.where(kind < 0.15, -rng.integers(1, 1 << 30, s), np.where(kind < 0.3, 0, np.where(kind < 0.6, 1, rng.integers(1, most + 1, s))))
        _, status = c.step(n, n_tokens, in_place=in_place, positions=i % 4 != 3)
        seen |= status
        back = np.minimum(rng.integers(0, 20, s) * (rng.random(s) < 0.4), c.length)
        c.length = c.length - back
    c.step(np.full(s, -1), n_tokens, in_place=in_place)           # all end: every page is free
    assert c.n_free == c.n_pages and sorted(c.free.tolist()) == list(range(c.n_pages))


def test_trees(ft):
    rng = np.random.default_rng(3)
    n = [1, 64, 0, 17, -1, 33, 2]
    masks = []
    for x in n:
        for j in range(max(x, 0)):
            masks.append(int(rng.integers(0, 1 << 62)) & ((1 << j) - 1) | 1 << j)
    c = State(ft, [5, 0, 9, 100, 7, 31, 16])
    c.step(n, len(masks) + 5, masks + [0] * 5)
    want, status = c.step([65, 64, 1, 0, 0, 0, 0], 130, [(1 << 64) - 1] * 130)       # 65 under a mask: refused; bits past the drafts count
    assert status == S.BAD_ID and want["kv_len"][0] == 0 and want["positions"][65] == c.length[1] - 64 + 63


@pytest.mark.parametrize("free", [0, 1, 2, 3, 5, 8])
def test_pages_run_out(ft, free):
    """The sequences that what is left is enough for are served, in order; the others keep what they have."""
    c = State(ft, [16, 3, 16, 0, 40, 16], n_pages=sum([1, 1, 1, 0, 3, 1]) + free)
    want, status = c.step([1, 5, 17, 0, -1, 30], 60)
    assert (status == S.NO_PAGES) == (free + 3 < 1 + 2 + 2)
    c.step([0, 0, 0, -1, -1, -1], 0)


def test_bad_descriptions(ft):
    """Each is refused by itself, and the others are served."""
    base = dict(length=[20, 20, 20], held=[2, 2, 2], n_new=[1, 1, 1])
    for at, name, value in ((0, "length", -1), (1, "length", 33), (2, "length", 1 << 30), (0, "held", -1), (1, "held", 1 << 30), (2, "held", 1),
                            (0, "n_new", 61), (1, "n_new", (1 << 31) - 1), (2, "n_new", 100)):
        c = State(ft, [20, 20, 20], stride=5)
        vals = {k: list(v) for k, v in base.items()}
        vals[name][at] = value
        c.length, c.held = np.array(vals["length"]), np.array(vals["held"])
        want, status = c.step(vals["n_new"], 64)
        assert status == S.BAD_ID and want["kv_len"][at] == 0 and want["len_out"][at] == vals["length"][at]
        assert name == "n_new" or sum(x > 0 for x in want["kv_len"]) == 2
    c = State(ft, [20, 20], stride=5)
    c.held[1] = 9                                                 # more than the table has: it cannot end either
    _, status = c.step([-1, -1], 0)
    assert status == S.BAD_ID
    c = State(ft, [20, 20, 5], stride=5)
    c.table[0, 1], c.table[1, 0], c.free[c.n_free - 1] = c.n_pages, -1, -5
    c.step([1, 1, 20], 64)                                        # pages that are none: their tokens get no slot
    for n_free in (-3, 1000):
        c = State(ft, [20, 20], n_pages=12, stride=5)
        c.free[:] = np.arange(12) % 7
        c.n_free = n_free
        assert c.step([-1, 9], 64)[1] & S.BAD_ID


def test_states_of_more_pages_than_there_are(ft):
    """Every sequence claims all pages, or wants more than any table may have: sums that 32 bits do not hold are cut, nothing is read
    outside its row."""
    c = State(ft, [0] * 1000, n_pages=5000, stride=5000, held=[0] * 1000)
    c.held[:] = 5000
    c.table[:] = np.arange(5000)
    want, status = c.step([1] + [-1] * 999, 4)
    assert status == S.BAD_ID and want["n_free_out"] == 5000
    c = State(ft, [0] * 1000, n_pages=200, stride=1 << 16, page=256, held=[0] * 1000)
    want, status = c.step([1 << 23] * 1000, 1 << 10)
    assert status == S.BAD_ID and not want["kv_len"].any()
    c = State(ft, [0] * 3, n_pages=200, stride=1 << 16, page=16, held=[0] * 3)
    want, status = c.step([5, 1 << 20, 5], (1 << 20) + 10)
    assert status == S.NO_PAGES and want["kv_len"].tolist() == [5, 0, 0]


def test_rows_past_the_tokens(ft):
    c = State(ft, [16, 16, 16, 16])
    want, status = c.step([5, 6, 0, -1], 8)                       # the second's rows do not all fit
    assert status == S.BAD_ID and want["q_start"].tolist() == [0, 5, 8, 8, 8] and want["kv_len"].tolist() == [21, 0, 16, 0]


def test_nothing_to_do(ft):
    c = State(ft, [], max_seqs=4, stride=1)
    want, _ = c.step([], 5)
    assert want["q_start"].tolist() == [0]
    c = State(ft, [4, 5])
    c.step([0, 0], 0)
    c.step([0, 0], 3)


def test_refusals(ft):
    c = State(ft, [4, 5])
    t = dict(n_new=dev([1, 1]), len=dev([4, 5]), held=dev([1, 1]), block_table=dev(c.table), table_stride=c.stride, free_pages=dev(c.free), n_free=dev([3]),
             n_seqs=2, n_tokens=4, q_start=dev([0, 0, 0]), kv_len=dev([0, 0]), slots=dev([0] * 4), len_out=dev([0, 0]), held_out=dev([0, 0]),
             n_free_out=dev([0]))
    for bad in (dict(n_seqs=-1), dict(n_seqs=3), dict(n_tokens=-1), dict(n_tokens=1 << 30), dict(table_stride=0), *({k: None} for k in (
            "n_new", "len", "held", "block_table", "free_pages", "n_free", "q_start", "kv_len", "slots", "len_out", "held_out", "n_free_out"))):
        with pytest.raises(ft.FtError, match="plan") as ei:
            ft.ft_kv_plan(c.kv.handle, **(t | bad))
        assert ei.value.status == ft.FT_ERR_ARG
    with pytest.raises(ft.FtError, match="tree_mask"):
        ft.ft_kv_plan(c.kv.handle, **(t | dict(tree_mask=t["slots"].data_ptr() + 4)))
    assert t["slots"].tolist() == [0] * 4


def test_graph_goes_on_in_place(ft):
    """A captured step that updates its state in place, replayed, is as many steps."""
    c = State(ft, [15, 0, 33], n_pages=40, stride=12)
    t = dict(n_new=dev([1, 2, 0]), len=dev(c.length), held=dev(c.held), block_table=dev(c.table), free_pages=dev(c.free), n_free=dev([c.n_free]),
             q_start=dev([0] * 4), kv_len=dev([0] * 3), slots=dev([0] * 4), positions=dev([0] * 4))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ft.ft_kv_plan(c.kv.handle, n_seqs=3, n_tokens=4, table_stride=12, len_out=t["len"], held_out=t["held"], n_free_out=t["n_free"],
                      stream=torch.cuda.current_stream(), **t)
    for i in range(40):
        g.replay()
        torch.cuda.synchronize()
        want, _ = S.plan([1, 2, 0], c.length, c.held, c.table, c.free, c.n_free, 40, 16, 4)
        for name in ("q_start", "kv_len", "slots", "positions", "block_table", "free_pages"):
            assert np.array_equal(t[name].cpu().numpy(), want[name]), (i, name)
        c.length, c.held, c.table, c.free, c.n_free = (want[k] for k in ("len_out", "held_out", "block_table", "free_pages", "n_free_out"))
        c.n_free = int(c.n_free)
        assert t["n_free"].item() == c.n_free and np.array_equal(t["len"].cpu().numpy(), c.length)
    assert ft.ft_kv_status(c.kv.handle) == 0


def test_two_streams(ft):
    """Steps of two sets of sequences under one handle at the same time: nothing is shared between them."""
    a = State(ft, [40] * 200, n_pages=3000, stride=40)
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = []
    for i in range(2):
        n = np.full(200, 20 + i)
        t = dict(n_new=dev(n), len=dev(a.length), held=dev(a.held), block_table=dev(a.table), free_pages=dev(a.free), n_free=dev([a.n_free]), q_start=dev([0] * 201),
                 kv_len=dev([0] * 200), slots=dev([0] * 5000), len_out=dev([0] * 200), held_out=dev([0] * 200), n_free_out=dev([0]))
        sets.append((n, t))
    torch.cuda.synchronize()
    for _ in range(20):
        for (n, t), s in zip(sets, streams):
            ft.ft_kv_plan(a.kv.handle, n_seqs=200, n_tokens=5000, table_stride=40, stream=s, **t)
    torch.cuda.synchronize()
    for n, t in sets:
        want, _ = S.plan(n, a.length, a.held, a.table, a.free, a.n_free, 3000, 16, 5000)
        for name in ("q_start", "kv_len", "slots", "len_out", "held_out", "block_table", "free_pages"):
            assert np.array_equal(t[name].cpu().numpy(), want[name]), name
