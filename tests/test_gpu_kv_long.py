"""Attention at the sizes where index paths change: units of more than 32 row tiles, sequences of more than 100,000 keys, many
sequences.  Against oracle.kv on some of the rows, with test_gpu_kv's derived bounds."""
import numpy as np
import pytest
import torch

from oracle import kv as K
from test_gpu_kv import Case, ft  # noqa: F401  (fixture)
from test_gpu_kv_masks import check_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def alone():
    """No empty sequences behind the calls' own: these are calls of many or long ones already."""
    Case.crowd = 0


def causal(rows, n, length, window=0, n_sink=0):
    j, p = np.arange(length)[None, :], (length - n + rows)[:, None]
    return (j <= p) & ((window == 0) | (j < n_sink) | (p - j < window))


@pytest.mark.parametrize("fmt,D", [("nvfp4", 64), ("fp8", 128), ("fp8", 256)])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (200, 4)])
def test_chunks_of_more_than_32_row_tiles(ft, fmt, D, window, n_sink):
    """Over 8192 rows a sequence and kv head (32 tiles of 256, 64 of 128), beside a short chunk and a single token."""
    nq, lens = [1100, 5, 1, 1040], [1300, 40, 700, 1040]
    c = Case(ft, fmt, D, 1, 8, 64, lens, nq, seed=D)
    o, _ = c.run(window=window, n_sink=n_sink)
    torch.cuda.synchronize()
    assert torch.isfinite(o.float()).all() and ft.ft_kv_status(c.kv.handle) == 0
    for s, (n, length) in enumerate(zip(nq, lens)):
        rows = np.unique(np.clip([0, 1, 15, 16, 31, 32, 500, 1022, 1023, 1024, 1025, 1039, 1055, 1056, n - 2, n - 1], 0, n - 1))
        check_rows(c, o, s, rows, causal(rows, n, length, window, n_sink))


@pytest.mark.parametrize("fmt,D,G", [("nvfp4", 64, 8), ("fp8", 128, 1), ("nvfp4", 256, 2)])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_more_than_a_hundred_thousand_keys(ft, fmt, D, G, n):
    lens, nq = [131077, 65, 2], [n, n, 1]
    c = Case(ft, fmt, D, 1, G, 128, lens, nq, seed=n)
    for window, n_sink in ((0, 0), (70000, 33)):
        o, _ = c.run(window=window, n_sink=n_sink)
        torch.cuda.synchronize()
        assert ft.ft_kv_status(c.kv.handle) == 0
        for s, (m, length) in enumerate(zip(nq, lens)):
            rows = np.unique([0, m - 1])
            check_rows(c, o, s, rows, causal(rows, m, length, window, n_sink))


@pytest.mark.parametrize("fmt,D,G", [("fp8", 64, 4), ("nvfp4", 128, 8)])
@pytest.mark.parametrize("empty", [0, 724])
def test_several_hundred_sequences(ft, fmt, D, G, empty):
    """Ragged lengths and numbers of new tokens, some of none; with the empty ones as many as a call takes."""
    Case.crowd = empty
    rng = np.random.default_rng(2)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(400), 300))]
    for most in (1, 30):
        nq = [int(rng.integers(0, most + 1)) for _ in lens]
        c = Case(ft, fmt, D, 2, G, 16, lens, nq, seed=most)
        o, _ = c.run(max_q=most)
        torch.cuda.synchronize()
        assert ft.ft_kv_status(c.kv.handle) == 0
        for s in range(0, 300, 7):
            rows = np.arange(nq[s])
            check_rows(c, o, s, rows, causal(rows, nq[s], lens[s]))
