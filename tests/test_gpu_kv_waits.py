"""The bounded waits of the attention kernels give up when nothing will satisfy them, and the context stays usable."""
import pytest
import torch

from test_gpu_kv import Case, ft  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def test_bounded_waits_expire_and_attention_runs_afterwards(ft):  # noqa: F811
    assert ft.ft_kv_check_bounded_waits() == 0xF             # a tile's copy, a role, one that was told, the products
    Case.crowd = 0
    for n in (1, 40):
        c = Case(ft, "nvfp4", 128, 2, 4, 16, [300, 77], [n, n], seed=n)
        c.both()
        assert ft.ft_kv_status(c.kv.handle) == 0
    torch.cuda.synchronize()
