"""The most probable tokens where few threads, or few tokens of a row, have a logit: no floor, or a low one, is left to seek them by.
Tolerances are test_gpu_logprobs'."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_logprobs import BF16, F32, check, logits, run, some_targets  # noqa: E402


def pick(d, rows):
    return {k: None if v is None else v[rows] for k, v in d.items()}


@pytest.mark.parametrize("dtype,V", [(BF16, 2049), (BF16, 2056), (BF16, 2500), (BF16, 3071), (F32, 1025), (F32, 1300), (F32, 1536),
                                     (BF16, 1033), (F32, 700)])
@pytest.mark.parametrize("K", [4, 5, 9, 10, 12, 13, 16, 17, 32])
def test_rows_of_few_chunks(gpt_lib, dtype, V, K):
    # one to three warps of a block have a chunk, of which the last may hold one vector
    from decoder_only_transformer_gpt_gb300 import binding
    for M in (1, 16, 170):
        t = some_targets(M, V, K)
        d, z, _ = run(logits(M, V, V + K), t, K, dtype)
        binding.status()
        keep = sorted({0, 1, M // 2, M - 1} & set(range(M)))
        check(pick(d, keep), z[keep], [t[i] for i in keep], K)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [33, 64, 65, 66, 100, 127, 128, 200, 255, 256, 257, 500])
@pytest.mark.parametrize("K", [15, 17, 32])
def test_rows_of_few_vectors(gpt_lib, dtype, V, K):
    from decoder_only_transformer_gpt_gb300 import binding
    M = 9
    for kind in ("normal", "ties", "rising", "masked"):
        t = some_targets(M, V, K)
        d, z, _ = run(logits(M, V, V + K, kind), t, K, dtype, ld=V + 3, offset=1)
        binding.status()
        check(d, z, t, K)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,V", [(16, 50257), (40, 20011), (200, 9001), (1300, 2500), (300, 2500), (9, 500), (7, 70)])
@pytest.mark.parametrize("K", [3, 10, 16, 17, 32])
def test_rows_of_which_a_mask_leaves_little(gpt_lib, dtype, M, V, K):
    # 1 to 40 tokens, spread or side by side; a NaN among the rest
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(V + K)
    full = logits(M, V, V)
    z = np.full((M, V), -np.inf)
    for i in range(M):
        left = [1, 2, K - 1, K, K + 1, 8, 40][i % 7]
        at = rng.permutation(V)[:left] if i % 2 else (int(rng.integers(0, V - 40)) + np.arange(left))
        z[i, at] = full[i, at]
    if M > 4:
        z[4, rng.integers(0, V)] = np.nan
    t = some_targets(M, V, K)
    d, zd, _ = run(z, t, K, dtype)
    binding.status()
    keep = sorted((set(range(9)) | {M // 2, M - 1}) & set(range(M)))
    check(pick(d, keep), zd[keep], [t[i] for i in keep], K)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,V", [(30, 50257), (60, 50257), (160, 12345), (330, 12345), (1300, 2500)])
def test_equal_rows_give_equal_results(gpt_lib, dtype, M, V):
    # every row of a grid: 8 rows apart they start alike in their 16 bytes, whatever V is
    z = logits(8, V, M)[np.arange(M) % 8]
    d, _, _ = run(z, (np.arange(M) % 8).tolist(), 7, dtype)
    for name, x in d.items():
        for i in range(8, M):
            assert torch.equal(x[i], x[i % 8]), (name, i)
