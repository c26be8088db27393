"""Long-context operators where a rounding or a reference could show: inputs made so that one error stands out.

Tolerances: the terms of tests/test_gpu_paged.py and tests/test_gpu_window.py, which derive them, less those that the
test says the kernel does not have.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_ref  # noqa: E402
from gpu_util import dev_bf16, host  # noqa: E402
from test_gpu_paged import LOG2E, Case  # noqa: E402
from test_gpu_paged_forms import widened  # noqa: E402


@pytest.mark.parametrize("rows", [1024, 4096, 65536])
@pytest.mark.parametrize("H,Hkv,D", [(4, 4, 64), (8, 1, 32), (12, 1, 64), (32, 2, 32)])
def test_decode_rounds_its_output_alone(gpt_lib, rows, H, Hkv, D):
    # small queries: about 100 rows of nearly equal weight, whose values cancel, so that outputs near zero show what
    # the probabilities have lost. They enter the product in two bf16 parts: p - hi - lo is 2^-8 of 2^-8 of p.
    from decoder_only_transformer_gpt_gb300 import binding
    c = widened(Case(H, Hkv, D, 16, [100, 90], seed=H, scale=0.05), rows)
    c.call()
    binding.status()
    c.check()
    y, _, pool, _ = c.expected()
    x, gy = c.qkv.astype(np.float64).reshape(2, H + 2 * Hkv, D), host(c.d_y)
    for b, ln in enumerate(c.lens):
        where = [paged_ref.place(c.table[b], 16, r) for r in range(ln + 1)]
        for h in range(H):
            k, u = (np.stack([pool[p, i, h // (H // Hkv), s] for p, s in where]) for i in (0, 1))
            _, _, a = paged_ref.attend(x[b, h], k, u)
            d = (D + 2) * 2.0 ** -24 * (np.abs(k) @ np.abs(x[b, h])).max() / math.sqrt(D) * (1 + LOG2E) + 2.0 ** -21
            at = slice(h * D, (h + 1) * D)
            tol = (2.0 ** -16 + 2 * d + (ln + 1) * 2.0 ** -24) * (a @ np.abs(u)) + 2.0 ** -8 * np.abs(y[b, at]) * (1 + 2.0 ** -7)
            err = np.abs(gy[b, at] - y[b, at])
            assert np.all(err <= tol), (b, h, err.max(), tol[err.argmax()])
