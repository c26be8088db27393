"""The paged cache's argument checks, without a GPU: every refusal happens on the host before any device call
(the pointers below are never dereferenced), and the binding refuses tensors that the kernels cannot take."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_ref  # noqa: E402

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    from decoder_only_transformer_gpt_gb300 import binding, build
    build.build()
    return binding.load()


def _store(lib, **k):
    a = dict(qkv=P, pool=P, weight=P, table=P, start=P, count=P, B=2, T=5, H=4, Hkv=2, D=64, pages=9, page=16,
             max_pages=4)
    a.update(k)
    return lib.gptk_paged_store(*a.values(), None)


def _attend(lib, **k):
    a = dict(qkv=P, pool=P, weight=P, table=P, lens=P, y=P, lse2=P, B=2, H=4, Hkv=2, D=64, pages=9, page=16, max_pages=4,
             window=0, sinks=0)
    a.update(k)
    return lib.gptk_paged_attention(*a.values(), None)


def _evict(lib, **k):
    a = dict(pool=P, weight=P, table=P, lens=P, dst_table=P, new_lens=ctypes.c_void_p(0x20000), kept=P, B=2, Hkv=2, D=64,
             pages=9, page=16, max_pages=4, dst_max_pages=2, budget=20, sinks=4, recent=8)
    a.update(k)
    return lib.gptk_paged_evict(*a.values(), None)


CACHE_EINVAL = [dict(pool=None), dict(table=None), dict(B=0), dict(B=8193), dict(Hkv=0), dict(pages=0), dict(page=0),
                dict(page=12), dict(page=4), dict(page=512), dict(max_pages=0), dict(max_pages=1 << 28)]


@pytest.mark.parametrize("call", [_store, _attend, _evict])
def test_cache_arguments(lib, call):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in CACHE_EINVAL:
        assert call(lib, **bad) == binding.GPT_EINVAL, bad
    for bad in (dict(D=48), dict(D=128), dict(pool=ODD)):
        assert call(lib, **bad) == binding.GPT_ECONFIG, bad


def test_store_arguments(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (dict(qkv=None), dict(T=-1), dict(H=0)):
        assert _store(lib, **bad) == binding.GPT_EINVAL, bad
    for bad in (dict(H=3), dict(qkv=ODD)):
        assert _store(lib, **bad) == binding.GPT_ECONFIG, bad
    assert _store(lib, T=0) == binding.GPT_OK                              # nothing to do


def test_attention_arguments(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (dict(qkv=None), dict(lens=None), dict(y=None), dict(H=0), dict(window=-1), dict(sinks=-1)):
        assert _attend(lib, **bad) == binding.GPT_EINVAL, bad
    assert _attend(lib, B=8192, max_pages=1 << 26, page=16) == binding.GPT_EINVAL
    for bad in (dict(H=5), dict(qkv=ODD), dict(y=ODD), dict(H=258)):
        assert _attend(lib, **bad) == binding.GPT_ECONFIG, bad


def test_evict_arguments(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (dict(weight=None), dict(lens=None), dict(dst_table=None), dict(new_lens=None), dict(kept=None),
                dict(new_lens=P), dict(dst_max_pages=0), dict(budget=0), dict(budget=33), dict(sinks=-1), dict(recent=-1),
                dict(sinks=13), dict(sinks=2147483647, recent=2147483647)):
        assert _evict(lib, **bad) == binding.GPT_EINVAL, bad


def test_status_text(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    assert b"page" in lib.gpt_strerror(binding.GPT_EPAGE)


def _cpu_cache(pages=5, Hkv=2, page=8, D=32, B=2, max_pages=2):
    return (torch.zeros(pages, 2, Hkv, page, D, dtype=torch.bfloat16), torch.zeros(B, max_pages, dtype=torch.int32))


@pytest.mark.parametrize("change", ["dtype", "shape", "strides", "device", "table", "weight"])
def test_binding_refuses_tensors(lib, change):
    from decoder_only_transformer_gpt_gb300 import binding
    pool, table = _cpu_cache()
    qkv, lens = torch.zeros(2, 8 * 32, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    y, weight = torch.zeros(2, 4 * 32, dtype=torch.bfloat16), None
    if change == "dtype":
        pool = pool.half()
    elif change == "shape":
        pool = pool[:, :1].contiguous()
    elif change == "strides":
        pool = pool.transpose(2, 3).contiguous().transpose(2, 3)
    elif change == "table":
        table = table.long()
    elif change == "weight":
        weight = torch.zeros(5, 2, 4)
    with pytest.raises(ValueError):
        binding.paged_attention(qkv, pool, table, lens, y, 4, weight=weight)


def test_the_plain_forms_agree_with_a_direct_count():
    # the reference's own window rule at its borders
    assert paged_ref.seen_rows(5, 0, 0) == [0, 1, 2, 3, 4]
    assert paged_ref.seen_rows(5, 1, 0) == [4]
    assert paged_ref.seen_rows(5, 2, 1) == [0, 3, 4]
    assert paged_ref.seen_rows(5, 4, 3) == [0, 1, 2, 3, 4]
    assert paged_ref.seen_rows(1, 3, 0) == [0]
    # an eviction by hand: six rows, two kept by weight between one sink and one recent; a tie goes to the lower row
    pool = np.arange(2 * 2 * 1 * 8 * 32, dtype=float).reshape(2, 2, 1, 8, 32)
    weight = np.zeros((2, 1, 8))
    weight[1, 0, :6] = [0.0, 2.0, 5.0, 2.0, np.nan, 0.0]
    _, w, n, kept = paged_ref.evict(pool, weight, np.array([[1]]), np.array([6]), np.array([[0]]), 4, 1, 1)
    assert n.tolist() == [4] and kept[0, 0].tolist() == [0, 1, 2, 5] and w[0, 0, :4].tolist() == [0.0, 2.0, 5.0, 0.0]


def test_numbers_past_32_bits_are_refused(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    x = torch.zeros(1)
    assert _store(lib, H=2 ** 31 - 2, T=1) == binding.GPT_EINVAL
    for n in (2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5):
        for k in ("window", "sinks"):
            a = dict(window=8, sinks=0)
            a[k] = n
            with pytest.raises(ValueError, match=k):
                binding.attention_window(x, x, 4, 4, **a)
            with pytest.raises(ValueError, match=k):
                binding.attention_window_bwd(x, x, x, x, x, 4, 4, **a)
            with pytest.raises(ValueError, match=k):
                binding.paged_attention(x, x, x, x, x, 4, **a)
        for k in ("budget", "sinks", "recent"):
            a = dict(budget=8, sinks=0, recent=0)
            a[k] = n
            with pytest.raises(ValueError, match=k):
                binding.paged_evict(x, x, x, x, x, x, x, **a)
