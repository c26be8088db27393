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
import test_gpu_window as gw  # noqa: E402
from gpu_util import dev_bf16, dev_i32, host  # noqa: E402
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


@pytest.mark.parametrize("D", [32, 64])
@pytest.mark.parametrize("B", [1, 8])
def test_raised_reference_keeps_probabilities(gpt_lib, B, D):
    # Key 64 of every tile of 128 scores 14 to 25 nats above the rest, so the queries behind it raise their reference
    # after the tile's first 64 probabilities were rounded. Each output column reads one of those keys alone, whose value
    # is large: an output is one probability, rounded once, times its value, and is rounded once itself.
    H, T, window = 24, 256, 256
    rng = np.random.default_rng(D + B)
    qkv = np.zeros((B, T, 3, H, D), np.float32)
    qkv[:, :, 0] = rng.standard_normal((B, T, H, D)) * 0.3
    qkv[:, :, 1] = rng.standard_normal((B, T, H, D)) * 0.5
    qkv[:, :, 0, :, 0] = rng.uniform(4, 7, (B, T, H))
    qkv[:, :, 1, :, 0] = 0.0
    qkv[:, 64::128, 1, :, 0] = 3.5 * math.sqrt(D)
    for t in range(T):
        if t % 128 < 64:
            qkv[:, t, 2, :, t % D] = 2.0 ** 20 * rng.uniform(1, 2, (B, H))
    qkv = host(dev_bf16(qkv.reshape(B, T, 3 * H * D))).astype(np.float32)
    y, lse2 = gw._forward(dev_bf16(qkv), H, H, window, 0)
    from decoder_only_transformer_gpt_gb300 import binding
    binding.status()
    gw._check(qkv, np.zeros((B, T, H * D), np.float32), y, lse2, None, H, H, window, 0, only=None if B == 1 else {(7, h) for h in range(H)})


@pytest.mark.parametrize("D", [32, 64])
@pytest.mark.parametrize("B,T,window", [(1, 300, 1), (40, 300, 1), (3, 5, 64), (40, 129, 40)])
def test_a_row_that_sees_one_key_copies_its_value(gpt_lib, B, T, window, D):
    # its probability is 1 in every type, and the sum it is divided by
    H = 4
    qkv, _ = gw._inputs(B, T, H, H, D, seed=T)
    y, lse2 = gw._forward(dev_bf16(qkv), H, H, window, 0)
    n = T if window == 1 else 1
    assert torch.equal(y[:, :n], dev_bf16(qkv)[:, :n, 2 * H * D:])
    x = qkv.astype(np.float64).reshape(B, T, 3, H, D)[:, :n]
    s = np.einsum("bthd,bthd->bht", x[:, :, 0], x[:, :, 1]) / math.sqrt(D) * LOG2E
    tol = 2 * (D + 2) * 2.0 ** -24 * np.einsum("bthd,bthd->bht", abs(x[:, :, 0]), abs(x[:, :, 1])) + 2.0 ** -22 * (1 + abs(s))
    assert np.all(np.abs(host(lse2)[:, :, :n] - s) <= tol)


def test_store_of_counts_far_below_zero(gpt_lib):
    # a count below zero stores nothing, the lowest int32 too: count - 16, for a block's first token, would wrap around
    from decoder_only_transformer_gpt_gb300 import binding
    B, T, H, D, page = 4, 77, 2, 32, 8
    pool = torch.full((B * 10, 2, 1, page, D), 3.0, dtype=torch.bfloat16, device="cuda")
    weight = torch.ones(B * 10, 1, page, device="cuda")
    qkv = torch.ones(B, T, (H + 2) * D, dtype=torch.bfloat16, device="cuda")
    count = dev_i32(np.array([-2 ** 31, -2 ** 31 + 20, -1, -2 ** 31], np.int32))
    binding.paged_store(qkv, pool, dev_i32(np.arange(B * 10).reshape(B, 10)), H, count=count, weight=weight)
    binding.status()
    assert torch.all(pool == 3.0) and torch.all(weight == 1.0)


@pytest.mark.parametrize("rows", [1024, 4096, 65536])
@pytest.mark.parametrize("H,Hkv,length", [(2, 2, 700), (12, 1, 700), (40, 2, 700), (2, 2, 20)])
def test_scores_of_minus_infinity(gpt_lib, rows, H, Hkv, length):
    # products past fp32's range: every score of the first key head's queries is -inf, their softmax 0 / 0
    from decoder_only_transformer_gpt_gb300 import binding
    D, G = 64, H // Hkv
    c = Case(H, Hkv, D, 16, [length, 40], seed=rows)
    x = c.qkv.reshape(2, H + 2 * Hkv, D)
    x[0, :G], x[0, H] = 3e38, -3e38
    for r in range(length):
        p, s = c.table[0, r // 16], r % 16
        c.pool[p, 0, 0, s] = -3e38
    widened(c, rows)
    c.call()
    binding.status()
    y, lse2, w = host(c.d_y).reshape(2, H, D), host(c.d_lse2), host(c.d_weight)
    assert np.isnan(y[0, :G]).all() and np.isfinite(y[0, G:]).all() and np.isfinite(y[1]).all()
    assert np.all(lse2[0, :G] == -np.inf) and np.isfinite(lse2[0, G:]).all() and np.isfinite(lse2[1]).all()
    seen = np.stack([w[c.table[0, r // 16], :, r % 16] for r in range(length + 1)])
    assert np.isnan(seen[:, 0]).all() and np.isfinite(seen[:, 1:]).all()


@pytest.mark.parametrize("B,T", [(1, 700), (12, 700)])
@pytest.mark.parametrize("what", ["sinks high", "sinks low", "first of 32 high", "first of 32 low"])
@pytest.mark.parametrize("D", [32, 64])
def test_derivative_with_scores_far_from_the_rest(gpt_lib, B, T, what, D):
    # the inputs of the forward's test: log-sum-exps of hundreds, from which the derivative makes the probabilities again
    H, window, sinks = 4, 200, 6
    qkv, dy = gw._inputs(B, T, H, H, D, seed=T)
    q, k = qkv[..., :H * D], qkv[..., H * D:2 * H * D]
    q[...] = np.abs(q)
    rows = slice(0, sinks) if what.startswith("sinks") else slice(0, T, 32)
    k[:, rows] = np.abs(k[:, rows]) * (8.0 if what.endswith("high") else -8.0)
    qkv = host(dev_bf16(qkv)).astype(np.float32)
    x = dev_bf16(qkv)
    y, lse2 = gw._forward(x, H, H, window, sinks)
    dqkv = gw._backward(x, y, dev_bf16(dy), lse2, H, H, window, sinks)
    from decoder_only_transformer_gpt_gb300 import binding
    binding.status()
    gw._check(qkv, dy, y, lse2, dqkv, H, H, window, sinks, only={(0, 0), (B - 1, 3)})
