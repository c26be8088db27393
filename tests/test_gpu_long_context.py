"""The long-context operators as they are used together: a prompt through sliding-window attention, its keys and values
into pages, decoding over the pages, an eviction, and decoding on; and training's pair of calls against differences.

Tolerances: tests/test_gpu_paged.py's and tests/test_gpu_window.py's, which derive them.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_ref  # noqa: E402
import window_ref  # noqa: E402
from gpu_util import dev_bf16, dev_f32, dev_i32, host, rand_bf16  # noqa: E402

E8 = 2.0 ** -8


@pytest.mark.parametrize("H,Hkv,D,window,sinks", [(4, 2, 64, 50, 3), (12, 12, 64, 1000, 0), (6, 1, 32, 17, 0)])
def test_decode_continues_a_prompt(gpt_lib, H, Hkv, D, window, sinks):
    """Every decoded token's output is the row that sliding-window attention gives it within the whole sequence."""
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(H)
    B, T, more, page = 3, 150, 20, 16
    prompt = np.array([150, 97, 1], np.int32)                    # real lengths within the padded batch
    qkv = rand_bf16(rng, (B, T + more, (H + 2 * Hkv) * D))
    x = dev_bf16(qkv)
    y = torch.empty(B, T + more, H * D, dtype=torch.bfloat16, device="cuda")
    binding.attention_window(x, y, H, Hkv, window, sinks)
    max_pages = (T + more + page - 1) // page
    table = dev_i32(rng.permutation(B * max_pages).reshape(B, max_pages))
    pool = torch.full((B * max_pages, 2, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lens = dev_i32(prompt)
    binding.paged_store(x, pool, table, H, count=lens)
    out = torch.empty(B, H * D, dtype=torch.bfloat16, device="cuda")
    lse2 = torch.empty(B, H, dtype=torch.float32, device="cuda")
    for step in range(more):
        tok = torch.stack([x[b, int(prompt[b]) + step] for b in range(B)]).contiguous()
        binding.paged_attention(tok, pool, table, lens, out, H, lse2=lse2, window=window, sinks=sinks)
        binding.status()
        whole = torch.stack([y[b, int(prompt[b]) + step] for b in range(B)])
        for b in range(B):
            t = int(prompt[b]) + step
            q, k, u = (qkv[b, :t + 1, c].astype(np.float64) for c in
                       (slice(0, H * D), slice(H * D, (H + Hkv) * D), slice((H + Hkv) * D, None)))
            for h in range(H):
                j = h // (H // Hkv)
                seen = paged_ref.seen_rows(t + 1, window, sinks)
                r, l, a = paged_ref.attend(q[t, h * D:(h + 1) * D], k[seen][:, j * D:(j + 1) * D], u[seen][:, j * D:(j + 1) * D])
                tol = (E8 + 2.0 ** -13) * (a @ np.abs(u[seen][:, j * D:(j + 1) * D])) + E8 * np.abs(r) * (1 + E8)
                for got in (host(out)[b], host(whole)[b]):
                    assert np.all(np.abs(got[h * D:(h + 1) * D] - r) <= tol), (step, b, h)
                assert abs(host(lse2)[b, h] - l) <= 2.0 ** -13 * (1 + abs(l))
        lens += 1


def test_decode_evict_decode(gpt_lib):
    """Steps that sum the weights, an eviction in place by the summed weights, and steps over what is left."""
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(3)
    B, H, Hkv, D, page, budget, sinks, recent = 2, 4, 2, 64, 8, 40, 2, 10
    lens = np.array([70, 33], np.int32)
    max_pages = 12
    table = rng.permutation(B * max_pages + 1)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    pool = dev_bf16(rand_bf16(rng, (B * max_pages + 1, 2, Hkv, page, D)))
    weight = torch.zeros(B * max_pages + 1, Hkv, page, device="cuda")
    y = torch.empty(B, H * D, dtype=torch.bfloat16, device="cuda")
    d_table, d_lens = dev_i32(table), dev_i32(lens)

    def step():
        qkv = rand_bf16(rng, (B, (H + 2 * Hkv) * D), 1.5)
        before = host(pool), host(weight), d_lens.cpu().numpy()
        binding.paged_attention(dev_bf16(qkv), pool, d_table, d_lens, y, H, weight=weight)
        binding.status()
        r, _, p, w = paged_ref.decode(qkv.astype(np.float64), before[0], before[1], table, before[2], H, 0, 0)
        np.testing.assert_array_equal(host(pool), p)
        # |u| is below 6 here: 2^-8 of the probabilities' rounding and of the output's
        assert np.all(np.abs(host(y) - r) <= E8 * 6 + E8 * np.abs(r))
        assert np.all(np.abs(host(weight) - w) <= 2.0 ** -12 * (1 + w))
        d_lens.add_(1)

    for _ in range(8):
        step()
    # every step's weights sum to the number of query heads over each sequence's rows
    total = np.array([[sum(host(weight)[paged_ref.place(table[b], page, r)[0], j, r % page] for r in range(int(d_lens[b])))
                       for j in range(Hkv)] for b in range(B)])
    assert np.all(np.abs(total - 8 * H / Hkv) < 1e-3)
    before = host(pool), weight.cpu().numpy(), d_lens.cpu().numpy()
    new, kept = torch.empty_like(d_lens), torch.empty(B, Hkv, budget, dtype=torch.int32, device="cuda")
    binding.paged_evict(pool, weight, d_table, d_lens, d_table, new, kept, budget, sinks, recent)
    binding.status()
    want = paged_ref.evict(before[0], before[1], table, before[2], table, budget, sinks, recent)
    np.testing.assert_array_equal(host(pool), want[0])
    np.testing.assert_array_equal(weight.cpu().numpy(), want[1])
    np.testing.assert_array_equal(new.cpu().numpy(), want[2])
    np.testing.assert_array_equal(kept.cpu().numpy(), want[3])
    assert new.tolist() == [40, 40]
    d_lens.copy_(new)
    for _ in range(4):
        step()


def test_training_pair_against_differences(gpt_lib):
    """The derivative's direction: along random directions the loss <dy, y> moves as <dqkv, direction> says. The loss is
    the float64 formula's (the kernel's own y is rounded to bf16, too coarse for a difference); the derivative is the
    kernel's, each element off by at most about 2^-7 of the typical gradient, so a sum over n random directions by 2^-7 of
    its spread times a few."""
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(11)
    T, H, Hkv, D, window, sinks = 140, 4, 2, 32, 37, 2
    qkv = rand_bf16(rng, (1, T, (H + 2 * Hkv) * D))
    dy = rand_bf16(rng, (1, T, H * D))
    x, g = dev_bf16(qkv), dev_bf16(dy)
    y = torch.empty(1, T, H * D, dtype=torch.bfloat16, device="cuda")
    lse2 = torch.empty(1, H, T, dtype=torch.float32, device="cuda")
    dqkv = torch.empty_like(x)
    binding.attention_window(x, y, H, Hkv, window, sinks, lse2=lse2)
    binding.attention_window_bwd(x, y, g, lse2, dqkv, H, Hkv, window, sinks)
    binding.status()
    grad = host(dqkv)[0]

    def loss(z):
        z = z.reshape(T, H + 2 * Hkv, D)
        return sum((window_ref.forward(z[:, h], z[:, H + h // (H // Hkv)], z[:, H + Hkv + h // (H // Hkv)], window, sinks)[0]
                    * dy[0].reshape(T, H, D)[:, h]).sum() for h in range(H))

    base = qkv[0].astype(np.float64)
    norm = np.linalg.norm(grad)
    for part in (slice(0, H * D), slice(H * D, (H + Hkv) * D), slice((H + Hkv) * D, None), slice(None)):
        d = np.zeros_like(base)
        d[:, part] = rng.standard_normal(d[:, part].shape)
        h = 1e-5
        slope = (loss(base + h * d) - loss(base - h * d)) / (2 * h)
        assert abs(slope - (grad * d).sum()) <= 2.0 ** -7 * 4 * norm + 1e-6 * abs(slope), (part, slope, (grad * d).sum())
    assert math.isfinite(norm) and norm > 0


def test_many_sequences_take_fewer_warps(gpt_lib):
    # 8,192 sequences: their list leaves room for fewer rings per SM
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(12)
    B, H, D, page = 8192, 2, 64, 8
    lens = rng.integers(-1, 8, B).astype(np.int32)
    pool = rand_bf16(rng, (B, 2, 1, page, D))
    qkv = rand_bf16(rng, (B, (H + 2) * D))
    y = torch.full((B, H * D), 5.0, dtype=torch.bfloat16, device="cuda")
    binding.paged_attention(dev_bf16(qkv), dev_bf16(pool), dev_i32(np.arange(B)[:, None]), dev_i32(lens), y, H)
    binding.status()
    want, _, _, _ = paged_ref.decode(qkv.astype(np.float64), pool.astype(np.float64), None, np.arange(B)[:, None], lens, H, 0, 0)
    got = host(y)
    alive = lens >= 0
    assert np.all(got[~alive] == 5.0)
    u = np.abs(pool[:, 1]).max()
    assert np.all(np.abs(got - want)[alive] <= (E8 + 2.0 ** -12) * max(u, np.abs(qkv).max()) + E8 * np.abs(want[alive]))
