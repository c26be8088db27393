"""Scratch of the long-context operators: what a large call took can be given back, and wide tables with many heads."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from gpu_util import dev_bf16, dev_i32, rand_bf16  # noqa: E402
from test_gpu_paged import Case  # noqa: E402
from test_gpu_paged_forms import run, widened  # noqa: E402


def _call(B, H, Hkv, rows, lens, weights):
    """A call of paged attention in a table for `rows` rows."""
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(rows)
    D, page, used = 64, 64, max(lens) // 64 + 1
    table = torch.full((B, rows // page), 10 ** 9, dtype=torch.int32, device="cuda")
    table[:, :used] = dev_i32(np.arange(B * used).reshape(B, used))
    pool = dev_bf16(rand_bf16(rng, (B * used, 2, Hkv, page, D)))
    weight = torch.zeros(B * used, Hkv, page, device="cuda") if weights else None
    qkv, d_lens = dev_bf16(rand_bf16(rng, (B, (H + 2 * Hkv) * D))), dev_i32(np.array(lens))
    y = torch.empty(B, H * D, dtype=torch.bfloat16, device="cuda")
    return lambda: binding.paged_attention(qkv, pool, table, d_lens, y, H, weight=weight)


def test_scratch_is_given_back(gpt_lib):
    # weights in a table for 262,144 rows take 4 B H rows bytes: 2 GiB that stay for the next call until they are asked for
    from decoder_only_transformer_gpt_gb300 import binding
    small, big = _call(2, 4, 4, 8192, [30, 5], True), _call(64, 32, 32, 262144, [100] * 64, True)
    small()
    torch.cuda.synchronize()
    binding.scratch_trim()
    before = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        big()
    torch.cuda.synchronize()
    assert before - torch.cuda.mem_get_info()[0] >= 2 ** 31
    binding.scratch_trim(2 ** 30)
    assert before - torch.cuda.mem_get_info()[0] <= 2 ** 30 + 2 ** 26
    binding.scratch_trim()
    binding.scratch_trim()
    assert before - torch.cuda.mem_get_info()[0] <= 2 ** 26
    small()
    binding.status()


@pytest.mark.parametrize("H,Hkv,D", [(48, 48, 64), (64, 4, 32)])
def test_many_heads_in_a_wide_table(gpt_lib, H, Hkv, D):
    # 40 sequences of up to a hundred rows in a table for 32,768: scores lie 32,768 apart, up to 252 MB in all
    rng = np.random.default_rng(H)
    run(widened(Case(H, Hkv, D, 16, rng.integers(-1, 100, 40).tolist(), seed=H), 32768))
