"""Sizes next to the end of 32 bits, without a GPU: what the kernels' row numbers would wrap around at is refused on the
host before any device call (the pointers are never dereferenced)."""
import pytest

torch = pytest.importorskip("torch")

from test_paged_host import _attend, _evict, _store, lib  # noqa: E402, F401

MOST = 2 ** 31 - 4096                                        # the header's limit


@pytest.mark.parametrize("call", [_store, _attend, _evict])
@pytest.mark.parametrize("page", [8, 256])
def test_rows_of_a_table(lib, call, page):  # noqa: F811
    # 32 rows of a unit, 2,048 threads of a cluster and 4,096 rows in flight per block step past a list's last row
    from decoder_only_transformer_gpt_gb300 import binding
    for max_pages in ((2 ** 31 - 1) // page, MOST // page + 1):
        assert call(lib, page=page, max_pages=max_pages) == binding.GPT_EINVAL, max_pages
    # at the limit the sizes pass: a refusal of what comes after them is another's
    assert call(lib, page=page, max_pages=MOST // page, D=48) == binding.GPT_ECONFIG


def test_rows_that_an_eviction_keeps(lib):  # noqa: F811
    from decoder_only_transformer_gpt_gb300 import binding
    for budget in (2 ** 31 - 1, 2 ** 31 - 2048, MOST + 1):
        assert _evict(lib, budget=budget, dst_max_pages=2 ** 27, sinks=0, recent=0) == binding.GPT_EINVAL, budget


def test_scratch_is_trimmed_to_a_number_of_bytes(lib):  # noqa: F811
    from decoder_only_transformer_gpt_gb300 import binding
    for keep in (-1, 2 ** 64):
        with pytest.raises(ValueError, match="keep"):
            binding.scratch_trim(keep)
