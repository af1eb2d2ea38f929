"""The key/value calls of the binding look at the types and strides of the tensors that they are given: what the kernels would
misread is refused, and what they can read reaches them with the right strides.  No GPU: the C calls are caught."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def ft():
    import __graft_entry__ as entry
    entry.build()
    import expert_cache_gb300
    expert_cache_gb300._load_types()                         # as the first handle does
    return expert_cache_gb300


@pytest.fixture
def calls(ft, monkeypatch):
    got = {}

    def catch(name):
        def call(*args):
            got[name] = args
            return 0
        return call

    for name in ("append", "read", "attention"):
        monkeypatch.setattr(ft, f"_kv_{name}", catch(name))
    return got


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def refused(ft, what, f):
    with pytest.raises(ft.FtError, match=what) as ei:
        f()
    assert ei.value.status == ft.FT_ERR_ARG


def test_append_takes_rows_wherever_they_stand(ft, calls):
    wide = bf16(5, 3 * 2 * 64 + 8)
    k, v = wide[:, 8:136], wide[:, 136:264]                  # slices of a projection's output
    heads = wide[:, 8:].view(5, 3, 2, 64)[:, 1]              # [5, 2, 64], dense within a token
    sl = i32(5)
    for a, b in ((k, v), (heads, v), (bf16(5, 2, 64), k)):
        ft.ft_kv_append(7, 1, a, b, sl, 5, stream=0)
        assert calls["append"] == (7, 1, a.data_ptr(), b.data_ptr(), a.stride(0), b.stride(0), sl.data_ptr(), 5, 0)
    ft.ft_kv_append(7, 1, k.data_ptr(), v.data_ptr(), sl.data_ptr(), 5, k_stride=392, v_stride=400, stream=0)
    assert calls["append"][2:7] == (k.data_ptr(), v.data_ptr(), 392, 400, sl.data_ptr())


@pytest.mark.parametrize("one", [lambda: bf16(2, 1, 64).transpose(0, 1), lambda: bf16(64, 2).view(2, 64)[None], lambda: bf16(3, 128)[1:2],
                                 lambda: bf16(1, 128).as_strided((1, 2, 64), (0, 64, 1))])
def test_a_single_token_has_no_stride_to_refuse(ft, calls, one):
    k = one()
    assert k.is_contiguous()
    ft.ft_kv_append(7, 0, k, k, i32(1), 1, stream=0)
    assert calls["append"][4:6] == (128, 128)
    ft.ft_kv_attention(7, 0, k, i32(2), i32(1), i32(1, 3), 3, 1, 1, 1, k, stream=0)
    assert ft._KV_ATTN.unpack(calls["attention"][1])[3:5] == (128, 128)


def test_append_and_read_refuse_what_they_would_misread(ft, calls):
    k, sl = bf16(4, 2, 64), i32(4)
    gaps = bf16(4, 2, 2, 64)[:, :, 0]                        # every other head
    turned = bf16(4, 64, 2).transpose(1, 2)
    for bad in (gaps, turned, k.float(), k.half()):
        refused(ft, "append: k", lambda: ft.ft_kv_append(7, 0, bad, k, sl, 4, stream=0))
        refused(ft, "append: v", lambda: ft.ft_kv_append(7, 0, k, bad, sl, 4, stream=0))
        refused(ft, "read: k_out", lambda: ft.ft_kv_read(7, 0, sl, 4, bad, k, stream=0))
        refused(ft, "read: v_out", lambda: ft.ft_kv_read(7, 0, sl, 4, k, bad, stream=0))
    for bad in (sl.long(), i32(8)[::2], sl.float()):
        refused(ft, "append: slots", lambda: ft.ft_kv_append(7, 0, k, k, bad, 4, stream=0))
        refused(ft, "read: slots", lambda: ft.ft_kv_read(7, 0, bad, 4, k, k, stream=0))
    refused(ft, "read: k_out", lambda: ft.ft_kv_read(7, 0, sl, 4, bf16(4, 4, 64)[:, :2], k, stream=0))
    assert not calls


def test_attention_refuses_what_it_would_misread(ft, calls):
    good = dict(layer=0, q=bf16(6, 4, 64), q_start=i32(3), kv_len=i32(2), block_table=i32(2, 5), table_stride=5, n_seqs=2, n_tokens=6,
                max_q=3, o=bf16(6, 4, 64), tree_mask=torch.zeros(6, dtype=torch.int64), lse=torch.zeros(6, 4), stream=0)
    ft.ft_kv_attention(7, **good)
    got = ft._KV_ATTN.unpack(calls.pop("attention")[1])
    assert got == (*(good[n].data_ptr() for n in ("q", "o", "lse")), 256, 256,
                   *(good[n].data_ptr() for n in ("q_start", "kv_len", "block_table", "tree_mask")), 0, 5, 2, 6, 3, 0, 0, 1.0)
    fine = dict(block_table=i32(2, 9)[:, :5], tree_mask=torch.zeros(6, dtype=torch.uint64), q=bf16(6, 300)[:, :256], lse=None)
    for name, t in fine.items():
        ft.ft_kv_attention(7, **{**good, name: t})
    calls.clear()
    bad = dict(q=[bf16(6, 8, 64)[:, ::2], good["q"].float(), bf16(6, 64, 4).transpose(1, 2)], o=[bf16(6, 8, 64)[:, ::2], good["q"].half()],
               q_start=[i32(6)[::2], i32(3).long()], kv_len=[i32(4)[::2], i32(2).long()],
               block_table=[i32(2, 10)[:, ::2], i32(5, 2).t(), i32(2, 5).long()],
               tree_mask=[i32(6), torch.zeros(12, dtype=torch.int64)[::2]], lse=[bf16(6, 4), torch.zeros(4, 6).t()])
    for name, ts in bad.items():
        for t in ts:
            refused(ft, f"attention: {name}", lambda: ft.ft_kv_attention(7, **{**good, name: t}))
    assert not calls
    with pytest.raises(TypeError, match="stride"):
        ft.ft_kv_attention(7, **{**good, "q": good["q"].data_ptr()})


@pytest.fixture
def rotated(ft, monkeypatch):
    got = []
    monkeypatch.setattr(ft, "_kv_append_rotated", lambda *args: got.append(args) or 0)
    return got


def test_rows_that_are_no_tokens(ft, calls, rotated):
    """A batch of sequences is not taken for its tokens: their stride would be a sequence's, and most of them lie behind the tensor."""
    n = 12
    fine = dict(q=bf16(n, 4, 64), k=bf16(n, 2, 64), v=bf16(n, 2, 64), q_out=bf16(n, 4, 64), k_out=bf16(n, 2, 64), slots=i32(n))
    attn = dict(layer=0, q=bf16(n, 4, 64), q_start=i32(3), kv_len=i32(2), block_table=i32(2, 5), table_stride=5, n_seqs=2, n_tokens=n, max_q=n,
                o=bf16(n, 4, 64), stream=0)

    def rotate(n=n, **kw):
        ft.ft_kv_append_rotated(7, 0, n=n, positions=None, rope=None, rope_dim=0, n_positions=0, stream=0, **(fine | kw))

    rotate()
    for name, t in list(fine.items())[:5]:
        h = t.shape[1]
        for batch in (t[None], t.view(3, 4, h, 64), t.view(3, 4, h * 64), t.view(1, n * h * 64), bf16(3, 4, 2 * h, 64)[:, :, :h].contiguous(),
                      bf16(3, 4, h * 64 + 8)[:, :, :h * 64], t[:n - 1]):
            refused(ft, f"append_rotated: {name}", lambda: rotate(**{name: batch}))
    assert len(rotated) == 1
    for batch in (fine["k"][None], fine["k"].view(3, 4, 128), fine["k"][:5], fine["k"][:0], bf16(())):
        refused(ft, "append: k", lambda: ft.ft_kv_append(7, 0, batch, fine["v"], fine["slots"], n, stream=0))
        refused(ft, "append: v", lambda: ft.ft_kv_append(7, 0, fine["k"], batch, fine["slots"], n, stream=0))
    for name in ("q", "o"):
        for batch in (attn[name][None], attn[name].view(3, 4, 256), attn[name][:5]):
            refused(ft, f"attention: {name}", lambda: ft.ft_kv_attention(7, **(attn | {name: batch})))
    assert not calls
    # more rows than tokens, one token in any shape, a stride that is given
    rotate(n=5)
    rotate(**{name: t[:1][None] for name, t in fine.items()}, n=1)
    rotate(q=fine["q"][None], q_stride=256)
    assert ft._KV_QKV.unpack(rotated[1][1])[5:10] == (256, 128, 128, 256, 128) == ft._KV_QKV.unpack(rotated[3][1])[5:10]
    assert len(rotated) == 4 and all(x >= 256 and x % 8 == 0 for x in ft._KV_QKV.unpack(rotated[2][1])[5:10])
    ft.ft_kv_append(7, 0, fine["k"], fine["v"], fine["slots"], 5, stream=0)
    ft.ft_kv_attention(7, **(attn | dict(n_tokens=5)))
    assert calls["append"][4:6] == (128, 128) and ft._KV_ATTN.unpack(calls["attention"][1])[3:5] == (256, 256)


def test_arrays_at_odd_addresses(ft):
    """Arrays of 32-bit elements that do not start at one are refused by the calls themselves, before anything is launched.  The handle's
    fields stand in host memory here; a call that is not refused finds no GPU, or no work."""
    class Handle(ctypes.Structure):
        _fields_ = [("d", ft.FtKvDesc), ("layer_bytes", ctypes.c_size_t), ("page_shift", ctypes.c_int), ("err", ctypes.c_char * 256)]

    h = Handle(ft.FtKvDesc(1, 8, 16, 2, 64, 4, 2, ft.FT_KV_FP8, 1.0, 1.0, None, None), 8 * 16 * 2 * 128, 4, b"")
    handle, at = ctypes.addressof(h), 1 << 12

    def misaligned(what, f):
        with pytest.raises(ft.FtError, match=f"{what}: .*misaligned") as ei:
            f()
        assert ei.value.status == ft.FT_ERR_ARG

    for odd in (1, 2, 3):
        misaligned("append", lambda: ft.ft_kv_append(handle, 0, at, at, at + odd, 2, k_stride=128, v_stride=128, stream=0))
        misaligned("read", lambda: ft.ft_kv_read(handle, 0, at + odd, 2, at, at, stream=0))
        attn = dict(layer=0, q=at, q_start=at, kv_len=at, block_table=at, table_stride=4, n_seqs=1, n_tokens=2, max_q=2, o=at, lse=at, q_stride=256,
                    o_stride=256, stream=0)
        for name in ("q_start", "kv_len", "block_table", "lse"):
            misaligned("attention", lambda: ft.ft_kv_attention(handle, **(attn | {name: at + odd})))
        plan = dict(n_new=at, len=at, held=at, block_table=at, table_stride=4, free_pages=at, n_free=at, n_seqs=1, n_tokens=2, q_start=at, kv_len=at,
                    slots=at, len_out=at, held_out=at, n_free_out=at, positions=at, stream=0)
        for name in plan:
            if plan[name] == at:
                misaligned("plan", lambda: ft.ft_kv_plan(handle, **(plan | {name: at + odd})))
        turn = dict(layer=0, q=at, k=at, v=at, slots=at, n=2, q_out=at, positions=at, rope=at, rope_dim=32, n_positions=9, q_stride=256, k_stride=128,
                    v_stride=128, q_out_stride=256, stream=0)
        for name in ("slots", "positions"):
            misaligned("append_rotated", lambda: ft.ft_kv_append_rotated(handle, **(turn | {name: at + odd})))
