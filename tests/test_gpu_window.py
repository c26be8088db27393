"""Sliding-window attention with sinks and its derivative on the GPU against numpy float64 (tests/window_ref.py).

Inputs are seeded and bf16-exact. Tolerances follow the kernels' arithmetic (half a step: bf16 2^-8, fp32 2^-24):
  * scores in fp32, |ds| <= (D + 2) 2^-24 |q|.|k| / sqrt(D), and ex2.approx of a rounded argument: a probability is off
    by the relative `rel` (2 d for itself and its normaliser, and the fp32 sum over n keys); lse2 by rel log2(e) and its
    own rounding, so the recomputed probabilities of the derivative by 2 rel
  * P is rounded to bf16 for P U: 2^-8 sum A |u|; the output: 2^-8 |y|. Together e_y
  * dS = A (dA - Dsum): rounded to bf16 (2^-8 |dS|); Dsum comes from the bf16 y, off by sum |dy| e_y and 2^-24 D sum
    |dy||y|; dA in fp32 by D 2^-24 |dy|.|u|; A by 2 rel. dQ, dK: these times |k|, |q|, over sqrt(D)
  * dU: P rounded to bf16 and A's own error: (2^-8 + 2 rel) sum A |dy|
  * every gradient is rounded to bf16, and its fp32 sum over n terms adds n 2^-24 of the terms' absolute sum
Products of two such errors are covered by a factor of 1 + 2^-6 on the whole.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import window_ref  # noqa: E402
from gpu_util import dev_bf16, host, rand_bf16  # noqa: E402

LOG2E = 1.0 / math.log(2.0)
E8, E24 = 2.0 ** -8, 2.0 ** -24


def _inputs(B, T, H, Hkv, D, seed=0, scale=1.0):
    rng = np.random.default_rng(seed)
    qkv = rand_bf16(rng, (B, T, (H + 2 * Hkv) * D))
    qkv[..., : (H + Hkv) * D] *= scale
    qkv = host(dev_bf16(qkv)).astype(np.float32)                         # bf16-exact after the factor too
    return qkv, rand_bf16(rng, (B, T, H * D), 0.25)


def _forward(qkv, H, Hkv, window, sinks, **k):
    from decoder_only_transformer_gpt_gb300 import binding
    B, T, row = qkv.shape
    D = row // (H + 2 * Hkv)
    y = torch.full((B, T, H * D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse2 = torch.full((B, H, T), 9.0, dtype=torch.float32, device="cuda")
    binding.attention_window(qkv, y, H, Hkv, window, sinks, lse2=lse2, **k)
    return y, lse2


def _backward(qkv, y, dy, lse2, H, Hkv, window, sinks, **k):
    from decoder_only_transformer_gpt_gb300 import binding
    dqkv = torch.full_like(qkv, 9.0)
    binding.attention_window_bwd(qkv, y, dy, lse2, dqkv, H, Hkv, window, sinks, **k)
    return dqkv


def _within(name, got, want, tol):
    tol = tol * (1 + 2.0 ** -6) + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} off; first at {i}: {got[i]} for {want[i]} (tol {tol[i]})")


def _check(qkv, dy, y, lse2, dqkv, H, Hkv, window, sinks, only=None):
    """Every (sequence, key head), or those in `only`, element by element; dqkv None: the forward alone."""
    B, T, row = qkv.shape
    D, G = row // (H + 2 * Hkv), H // Hkv
    x, g = qkv.astype(np.float64).reshape(B, T, -1, D), dy.astype(np.float64).reshape(B, T, H, D)
    gy, gl = host(y).reshape(B, T, H, D), host(lse2)
    gd = None if dqkv is None else host(dqkv).reshape(B, T, -1, D)
    rd = 1.0 / math.sqrt(D)
    n = np.minimum(np.arange(T) + 1, window + sinks)                     # terms of a row's sums, at most
    for b in range(B):
        for j in range(Hkv):
            if only is not None and (b, j) not in only:
                continue
            k, u = x[b, :, H + j], x[b, :, H + Hkv + j]
            dk, du, tk, tu = (np.zeros((T, D)) for _ in range(4))
            for h in range(j * G, (j + 1) * G):
                q, d = x[b, :, h], g[b, :, h]
                yr, lr, a = window_ref.forward(q, k, u, window, sinks)
                qk = (np.abs(q) @ np.abs(k).T * (a > 0)).max(-1)
                rel = 2 * ((D + 2) * E24 * rd * qk * (1 + LOG2E) + 2.0 ** -21) + n * E24
                ey = (E8 + rel)[:, None] * (a @ np.abs(u)) + E8 * np.abs(yr)
                _within(f"y {b} {h}", gy[b, :, h], yr, ey)
                _within(f"lse2 {b} {h}", gl[b, h], lr, rel * LOG2E + 2.0 ** -22 * (1 + np.abs(lr)))
                if gd is None:
                    continue
                da, dsum = d @ u.T, (d * yr).sum(-1)
                ds = a * (da - dsum[:, None])
                edsum = (np.abs(d) * ey).sum(-1) + D * E24 * (np.abs(d) * np.abs(yr)).sum(-1)
                eds = E8 * np.abs(ds) + a * edsum[:, None] + 2 * rel[:, None] * np.abs(ds) + D * E24 * a * (np.abs(d) @ np.abs(u).T)
                dq = ds @ k * rd
                _within(f"dq {b} {h}", gd[b, :, h], dq,
                        (eds + n[:, None] * E24 * np.abs(ds)) @ np.abs(k) * rd + E8 * np.abs(dq))
                dk += ds.T @ q * rd
                tk += (eds + T * G * E24 * np.abs(ds)).T @ np.abs(q) * rd
                du += a.T @ d
                tu += ((E8 + 2 * rel + T * G * E24)[:, None] * a).T @ np.abs(d)
            if gd is not None:
                _within(f"dk {b} {j}", gd[b, :, H + j], dk, tk + E8 * np.abs(dk))
                _within(f"du {b} {j}", gd[b, :, H + Hkv + j], du, tu + E8 * np.abs(du))


def _case(B, T, H, Hkv, D, window, sinks, seed=0, scale=1.0, only=None):
    from decoder_only_transformer_gpt_gb300 import binding
    qkv, dy = _inputs(B, T, H, Hkv, D, seed, scale)
    x, g = dev_bf16(qkv), dev_bf16(dy)
    y, lse2 = _forward(x, H, Hkv, window, sinks)
    binding.status()
    _check(qkv, dy, y, lse2, None, H, Hkv, window, sinks, only)
    dqkv = _backward(x, y, g, lse2, H, Hkv, window, sinks)
    binding.status()
    _check(qkv, dy, y, lse2, dqkv, H, Hkv, window, sinks, only)


@pytest.mark.parametrize("T", [1, 2, 40, 127, 128, 129, 300, 520])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (128, 0), (129, 130), (1000, 0), (200, 600)])
def test_lengths(gpt_lib, T, window, sinks):
    _case(2, T, 2, 1, 64, window, sinks, seed=T)


@pytest.mark.parametrize("window", [2, 63, 65, 127, 130, 255, 256, 257, 384])
@pytest.mark.parametrize("sinks", [0, 3, 128])
def test_windows(gpt_lib, window, sinks):
    _case(1, 700, 1, 1, 64, window, sinks, seed=window)


@pytest.mark.parametrize("B,H,Hkv,D", [(3, 4, 4, 32), (1, 6, 2, 64), (2, 5, 1, 32), (1, 12, 12, 64), (1, 8, 1, 64)])
def test_heads(gpt_lib, B, H, Hkv, D):
    _case(B, 333, H, Hkv, D, 100, 5, seed=H)


@pytest.mark.parametrize("window,sinks", [(250, 5), (100, 0), (5000, 0)])
def test_many_items(gpt_lib, window, sinks):
    # more pairs of query tiles than SMs: several items per CTA, both softmax groups
    _case(13, 700, 12, 4, 64, window, sinks, seed=window, only={(0, 0), (5, 3), (12, 2)})


def test_long(gpt_lib):
    _case(1, 5000, 4, 1, 64, 700, 4, seed=1)
    _case(1, 4100, 2, 2, 32, 64, 200, seed=2)


def test_peaked_scores(gpt_lib):
    _case(2, 400, 2, 2, 64, 150, 3, seed=3, scale=5.0)


@pytest.mark.parametrize("sinks", [0, 2])
def test_unseen_keys_with_huge_scores(gpt_lib, sinks):
    # keys that leave the window score thousands higher than any seen one: they must not enter a row's reference
    B, T, H, D, window = 1, 600, 2, 64, 90
    qkv, dy = _inputs(B, T, H, H, D, seed=4)
    q, k = qkv[..., :H * D], qkv[..., H * D:2 * H * D]
    q[...] = np.abs(q)
    k[:, 2:200] = 40.0 + np.abs(k[:, 2:200])
    k[:, 200:] *= 0.5
    qkv = host(dev_bf16(qkv)).astype(np.float32)
    x = dev_bf16(qkv)
    y, lse2 = _forward(x, H, H, window, sinks)
    dqkv = _backward(x, y, dev_bf16(dy), lse2, H, H, window, sinks)
    _check(qkv, dy, y, lse2, dqkv, H, H, window, sinks)


def test_a_full_window_is_causal_attention(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    qkv, _ = _inputs(2, 500, 4, 4, 64, seed=5)
    x = dev_bf16(qkv)
    y, _ = _forward(x, 4, 4, 500, 0)
    z = torch.empty_like(y)
    binding.attention(x, z, 4)
    binding.status()
    # two kernels, each within the forward's bound of the exact result
    a = np.abs(qkv[..., 8 * 64:]).max()
    assert np.all(np.abs(host(y) - host(z)) <= 2 * (E8 * a + E8 * np.abs(host(z))) * (1 + 2.0 ** -6))


def test_padding_changes_nothing(gpt_lib):
    # sequences of 300 and 450 real tokens in a batch of 512: the padding's content does not reach them, forward or back
    H, D, window, sinks, ends = 2, 64, 100, 3, (300, 450)
    qkv, dy = _inputs(2, 512, H, H, D, seed=6)
    outs = []
    for fill in (0.0, 50.0):
        x, g = qkv.copy(), dy.copy()
        for b, e in enumerate(ends):
            x[b, e:], g[b, e:] = fill, 0.0
        x, g = dev_bf16(x), dev_bf16(g)
        y, lse2 = _forward(x, H, H, window, sinks)
        dqkv = _backward(x, y, g, lse2, H, H, window, sinks)
        for b, e in enumerate(ends):
            assert torch.all(dqkv[b, e:] == 0)
        outs.append([t for b, e in enumerate(ends) for t in (y[b, :e], lse2[b, :, :e], dqkv[b, :e, H * D:])])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_forward_repeats_bit_for_bit_and_lse_is_optional(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    x = dev_bf16(_inputs(4, 900, 12, 12, 64, seed=7)[0])
    y, lse2 = _forward(x, 12, 12, 256, 4)
    for _ in range(3):
        z = torch.empty_like(y)
        binding.attention_window(x, z, 12, 12, 256, 4)
        assert torch.equal(y, z)


def test_streams_and_graphs(gpt_lib):
    B, T, H, Hkv, D, window, sinks = 2, 600, 4, 2, 64, 130, 4
    qkv, dy = _inputs(B, T, H, Hkv, D, seed=8)
    x, g = dev_bf16(qkv), dev_bf16(dy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y, lse2 = _forward(x, H, Hkv, window, sinks)
        dqkv = _backward(x, y, g, lse2, H, Hkv, window, sinks)
    s.synchronize()
    _check(qkv, dy, y, lse2, dqkv, H, Hkv, window, sinks)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, lse3 = _forward(x, H, Hkv, window, sinks)
        dqkv2 = _backward(x, y2, g, lse3, H, Hkv, window, sinks)
    for seed in (8, 9):                                                  # replayed on other numbers in the same arrays
        qkv, dy = _inputs(B, T, H, Hkv, D, seed=seed)
        x.copy_(dev_bf16(qkv))
        g.copy_(dev_bf16(dy))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        _check(qkv, dy, y2, lse3, dqkv2, H, Hkv, window, sinks)


def test_two_calls_at_once(gpt_lib):
    H, window, sinks = 4, 130, 4
    ins = [_inputs(2, 600, H, H, 64, seed=s) for s in (10, 11)]
    dev = [(dev_bf16(a), dev_bf16(b)) for a, b in ins]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for (x, g), s in zip(dev, streams):
        with torch.cuda.stream(s):
            y, lse2 = _forward(x, H, H, window, sinks)
            outs.append((y, lse2, _backward(x, y, g, lse2, H, H, window, sinks)))
    torch.cuda.synchronize()
    for (qkv, dy), (y, lse2, dqkv) in zip(ins, outs):
        _check(qkv, dy, y, lse2, dqkv, H, H, window, sinks)


@pytest.mark.parametrize("T,H,Hkv,window,sinks", [(3000, 4, 1, 3000, 0), (2500, 3, 1, 100, 300), (4000, 2, 2, 2000, 4)])
def test_shared_key_tiles(gpt_lib, T, H, Hkv, window, sinks):
    # few heads and long windows or sinks: a key tile's query tiles are cut into segments of several CTAs
    _case(1, T, H, Hkv, 64, window, sinks, seed=T)


@pytest.mark.parametrize("window", [31, 32, 33, 127, 128, 129, 256, 300])
@pytest.mark.parametrize("sinks", [0, 1, 15, 16, 17, 31, 129])
def test_borders_in_pairs_of_tiles(gpt_lib, window, sinks):
    # several items per CTA; sinks as one step of 16 keys and as whole tiles; every 32-key part of a tile as a border
    _case(10, 900, 4, 2, 64, window, sinks, seed=window + sinks, only={(0, 0), (9, 1)})
    _case(10, 900, 4, 2, 32, window, sinks, seed=window + sinks, only={(4, 1)})


@pytest.mark.parametrize("B,T", [(1, 700), (12, 700)])
@pytest.mark.parametrize("what", ["sinks high", "sinks low", "first of 32 high", "first of 32 low"])
def test_references_far_from_the_rest(gpt_lib, B, T, what):
    # scores around 0 but for the sinks, or every 32nd key (a warp's reference in its first tile), hundreds above or below
    H, D, window, sinks = 4, 64, 200, 6
    qkv, dy = _inputs(B, T, H, H, D, seed=T)
    q, k = qkv[..., :H * D], qkv[..., H * D:2 * H * D]
    q[...] = np.abs(q)
    rows = slice(0, sinks) if what.startswith("sinks") else slice(0, T, 32)
    k[:, rows] = np.abs(k[:, rows]) * (8.0 if what.endswith("high") else -8.0)
    qkv = host(dev_bf16(qkv)).astype(np.float32)
    y, lse2 = _forward(dev_bf16(qkv), H, H, window, sinks)
    from decoder_only_transformer_gpt_gb300 import binding
    binding.status()
    _check(qkv, dy, y, lse2, None, H, H, window, sinks, only={(0, 0), (B - 1, 3)})
