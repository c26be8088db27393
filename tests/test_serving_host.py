"""Rotation, the 4-bit cache and log probabilities without a GPU: refusals (the pointers below are never dereferenced), the
frequencies in turns, and the references against direct counts, identities and differences."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402
from workloads import round_to_bf16  # noqa: E402

P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
ODDER = ctypes.c_void_p(0x10004)
# pi to 60 digits
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


@pytest.fixture(scope="module")
def lib():
    from decoder_only_transformer_gpt_gb300 import binding, build
    build.build()
    return binding.load()


def _rotary(lib, **k):
    a = dict(qkv=P, out=P, pos=P, turns=P, B=2, T=5, H=4, Hkv=2, D=64, rot=64, interleaved=0, inverse=0)
    a.update(k)
    return lib.gptk_rotary(*a.values(), None)


def _append(lib, **k):
    a = dict(qkv=P, out=P, pool=P, weight=P, table=P, start=P, count=P, pos=P, turns=P, B=2, T=5, H=4, Hkv=2, D=64, rot=64,
             interleaved=0, pages=9, page=16, max_pages=4)
    a.update(k)
    return lib.gptk_paged_append(*a.values(), None)


def _append4(lib, **k):
    a = dict(qkv=P, out=P, pool=P, ranges=P, table=P, start=P, count=P, pos=P, turns=P, B=2, T=5, H=4, Hkv=2, D=64, rot=64,
             interleaved=0, pages=9, page=16, max_pages=4)
    a.update(k)
    return lib.gptk_paged_append4(*a.values(), None)


def _load4(lib, **k):
    a = dict(pool=P, ranges=P, table=P, start=P, count=P, rows=P, B=2, T=5, Hkv=2, D=64, pages=9, page=16, max_pages=4)
    a.update(k)
    return lib.gptk_paged_load4(*a.values(), None)


def _attend4(lib, **k):
    a = dict(qkv=P, pool=P, ranges=P, table=P, lens=P, y=P, lse2=P, B=2, H=4, Hkv=2, D=64, pages=9, page=16, max_pages=4,
             window=0, sinks=0, added=0)
    a.update(k)
    return lib.gptk_paged_attention4(*a.values(), None)


def _logprobs(lib, **k):
    a = dict(logits=P, targets=P, logp=P, entropy=P, stats=P, top_ids=P, top_logp=P, M=3, V=50, ld=50, K=5, dtype=0)
    a.update(k)
    return lib.gptk_logprobs(*a.values(), None)


def _logprobs_bwd(lib, **k):
    a = dict(logits=P, targets=P, stats=P, entropy=P, dlogp=P, dentropy=P, dlogits=P, M=3, V=50, ld=50, dld=50, dtype=0)
    a.update(k)
    return lib.gptk_logprobs_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [_append, _append4, _load4, _attend4])
def test_cache_arguments(lib, call):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (dict(pool=None), dict(table=None), dict(B=0), dict(B=8193), dict(Hkv=0), dict(pages=0), dict(page=0),
                dict(page=12), dict(page=4), dict(page=512), dict(max_pages=0), dict(max_pages=1 << 28)):
        assert call(lib, **bad) == binding.GPT_EINVAL, bad
    for bad in (dict(D=48), dict(D=128), dict(pool=ODD)):
        assert call(lib, **bad) == binding.GPT_ECONFIG, bad
    if call is not _append:
        assert call(lib, ranges=None) == binding.GPT_EINVAL
        assert call(lib, ranges=ODD) == binding.GPT_ECONFIG


@pytest.mark.parametrize("call", [_rotary, _append, _append4])
def test_row_arguments(lib, call):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (dict(qkv=None), dict(T=-1), dict(H=0), dict(Hkv=0), dict(B=0), dict(rot=-16), dict(turns=None), dict(rot=0),
                dict(interleaved=2), dict(B=8192, T=1 << 18), dict(H=1 << 24, Hkv=1 << 24)):
        assert call(lib, **bad) == binding.GPT_EINVAL, bad
    for bad in (dict(H=3), dict(qkv=ODD), dict(out=ODD), dict(rot=8), dict(rot=24), dict(rot=80), dict(turns=ODDER)):
        assert call(lib, **bad) == binding.GPT_ECONFIG, bad
    assert call(lib, T=0) == binding.GPT_OK                                # nothing to do


def test_no_rows_need_no_address(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    for call in (_rotary, _append, _append4):
        assert call(lib, T=0, qkv=None, out=None) == binding.GPT_OK
    assert _load4(lib, T=0, rows=None) == binding.GPT_OK
    assert _rotary(lib, T=0, qkv=None, out=None, turns=None) == binding.GPT_EINVAL


def test_rotary_arguments(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (dict(out=None), dict(turns=None, rot=0), dict(inverse=2)):
        assert _rotary(lib, **bad) == binding.GPT_EINVAL, bad


def test_load_and_attention_arguments(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (dict(rows=None), dict(T=-1), dict(B=8192, T=1 << 18)):
        assert _load4(lib, **bad) == binding.GPT_EINVAL, bad
    assert _load4(lib, rows=ODD) == binding.GPT_ECONFIG
    assert _load4(lib, T=0) == binding.GPT_OK
    for bad in (dict(qkv=None), dict(lens=None), dict(y=None), dict(H=0), dict(window=-1), dict(sinks=-1), dict(added=-1),
                dict(added=65), dict(B=8192, max_pages=1 << 26)):
        assert _attend4(lib, **bad) == binding.GPT_EINVAL, bad
    for bad in (dict(H=5), dict(qkv=ODD), dict(y=ODD), dict(H=258)):
        assert _attend4(lib, **bad) == binding.GPT_ECONFIG, bad


def test_logprobs_arguments(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (dict(logits=None), dict(M=0), dict(V=0), dict(ld=49), dict(dtype=2), dict(dtype=-1), dict(M=1 << 29),
                dict(V=2 ** 31 - 1, ld=2 ** 31), dict(ld=1 << 60)):
        assert _logprobs(lib, **bad) == binding.GPT_EINVAL, bad
        assert _logprobs_bwd(lib, **bad) == binding.GPT_EINVAL, bad
    for bad in (dict(targets=None), dict(logp=None), dict(K=-1), dict(K=33), dict(V=4, ld=4), dict(K=0), dict(top_ids=None),
                dict(top_logp=None), dict(targets=None, logp=None, entropy=None, stats=None, top_ids=None, top_logp=None, K=0)):
        assert _logprobs(lib, **bad) == binding.GPT_EINVAL, bad
    for bad in (dict(logits=ctypes.c_void_p(0x10002)), dict(logits=ctypes.c_void_p(0x10001), dtype=1), dict(stats=ODDER)):
        assert _logprobs(lib, **bad) == binding.GPT_ECONFIG, bad
    for bad in (dict(stats=None), dict(dlogits=None), dict(dld=49), dict(targets=None), dict(dlogp=None), dict(entropy=None),
                dict(dentropy=None), dict(dld=51), dict(targets=None, dlogp=None, entropy=None, dentropy=None)):
        assert _logprobs_bwd(lib, **bad) == binding.GPT_EINVAL, bad
    for bad in (dict(dlogits=ctypes.c_void_p(0x10002)), dict(dlogits=ctypes.c_void_p(0x10001), dtype=1), dict(stats=ODDER)):
        assert _logprobs_bwd(lib, **bad) == binding.GPT_ECONFIG, bad


def test_binding_refuses_what_the_kernels_cannot_take(lib):
    from decoder_only_transformer_gpt_gb300 import binding
    bf, i32 = torch.bfloat16, torch.int32
    qkv, codes = torch.zeros(2, 3, 8 * 64, dtype=bf), torch.zeros(5, 2, 2, 16, 32, dtype=torch.uint8)
    ranges, table = torch.zeros(5, 2, 2, 16, 2, dtype=bf), torch.zeros(2, 2, dtype=i32)
    pool, turns = torch.zeros(5, 2, 2, 16, 64, dtype=bf), torch.zeros(32, dtype=torch.int64)
    for call, word in (
            (lambda: binding.rotary(qkv, qkv, 4, 2, turns), "device"),
            (lambda: binding.rotary(qkv, qkv, 4, 2, turns.float()), "turns"),
            (lambda: binding.rotary(qkv, qkv, 4, 2, turns.view(2, 16)), "turns"),
            (lambda: binding.rotary(qkv[0], qkv, 4, 2, turns), "qkv"),
            (lambda: binding.paged_append(qkv, pool[:, 0], table, 4), "pool"),
            (lambda: binding.paged_append(qkv[:1], pool, table, 4), "device"),
            (lambda: binding.paged_append4(qkv, codes.int(), ranges, table, 4), "codes"),
            (lambda: binding.paged_append4(qkv, codes[0], ranges, table, 4), "codes"),
            (lambda: binding.paged_append4(qkv, codes, ranges, table[0], 4), "table"),
            (lambda: binding.paged_load4(codes, ranges.float(), table, qkv), "device"),
            (lambda: binding.paged_attention4(qkv[:, 0], codes, ranges, table, table[:, 0], qkv, 4, window=1 << 31), "window"),
            (lambda: binding.logprobs(torch.zeros(2, 5, dtype=torch.float16), None, None), "logits"),
            (lambda: binding.logprobs(torch.zeros(5), None, None), "logits"),
            (lambda: binding.logprobs(torch.zeros(2, 5), None, None), "device"),
            (lambda: binding.logprobs_bwd(torch.zeros(2, 5), None, torch.zeros(2, 2), None, torch.zeros(2, 5)), "device")):
        with pytest.raises(ValueError, match=word):
            call()
    for call in (lambda: binding.rotary(None, qkv, 4, 2, turns), lambda: binding.rotary(qkv, qkv, "4", 2, turns),
                 lambda: binding.rotary(qkv, qkv, 4.5, 2, turns), lambda: binding.logprobs(None, None, None)):
        with pytest.raises(TypeError):
            call()
    for H in (2 ** 31, 10 ** 30, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="needs an int32"):
            binding.paged_append(qkv, pool, table, H)
    with pytest.raises(ValueError):
        binding.rotary_turns([[1.0]], device="cpu")
    for bad in (math.nan, math.inf, -2e12):
        with pytest.raises(binding.GptError):
            binding.rotary_turns([bad], device="cpu")


def test_turns_are_the_frequencies_over_a_full_turn(lib):
    # freq / (2 pi) 2^64 modulo 2^64, to the nearest but for the last unit
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(0)
    f = ref.freqs(64) + ref.freqs(32) + [0.0, 1e-30, -1e-18, -0.25, 1e12, -1e12, 2 * math.pi, math.pi] + \
        (rng.standard_normal(200) * 10.0 ** rng.integers(-12, 12, 200)).tolist()
    got = binding.rotary_turns(f, device="cpu").tolist()
    for x, t in zip(f, got):
        want = Fraction(x) / (2 * PI) * 2 ** 64
        off = (t - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 2, (x, t)


def test_rotation_reference():
    # lengths of pairs are kept, the inverse undoes it, a shift of both positions keeps products
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 5, 6, 32))
    for inter in (False, True):
        for rot in (16, 32):
            f = ref.freqs(rot)
            y, _ = ref.rotate(x, 2, 2, f, [3, 100], inter)
            back, _ = ref.rotate(y, 2, 2, f, [3, 100], inter, inverse=True)
            assert np.allclose(back, x, atol=1e-12) and np.array_equal(y[:, :, 4:], x[:, :, 4:])
            assert np.array_equal(y[..., rot:], x[..., rot:])
            assert np.allclose((y[:, :, :4] ** 2).sum(-1), (x[:, :, :4] ** 2).sum(-1))
            z, _ = ref.rotate(x, 2, 2, f, [3 + 7, 100 + 7], inter)
            assert np.allclose(np.einsum("btd,bsd->bts", y[:, :, 0], y[:, :, 2]), np.einsum("btd,bsd->bts", z[:, :, 0], z[:, :, 2]))


def test_rotation_gradient_is_the_inverse():
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((1, 2, 3, 32)), rng.standard_normal((1, 2, 3, 32))
    f = ref.freqs(32)
    dx, _ = ref.rotate(dy, 1, 1, f, [9], True, inverse=True)
    for at in [(0, 0, 0, 3), (0, 1, 1, 30), (0, 1, 2, 5)]:
        d = np.zeros_like(x)
        d[at] = 1e-6
        num = ((ref.rotate(x + d, 1, 1, f, [9], True)[0] - ref.rotate(x - d, 1, 1, f, [9], True)[0]) * dy).sum() / 2e-6
        assert abs(num - dx[at]) < 1e-8


def test_four_bit_reference():
    rng = np.random.default_rng(3)
    x = round_to_bf16((rng.standard_normal((500, 64)) * 10.0 ** rng.integers(-20, 20, (500, 1))).astype(np.float32))
    codes, ranges = ref.quantise(x)
    back = ref.values(codes, ranges)
    # half a scale, and 15 times the scale's own rounding where the largest code is cut
    assert (np.abs(back - x) <= ranges[:, :1].astype(np.float64) * (0.5 + 15 * 2.0 ** -8)).all()
    assert (codes & 15).max() == 15 and (codes >> 4).min() == 0
    flat = np.full((3, 32), 7.5, np.float32)
    flat[1, 3] = np.inf
    flat[2, :2] = (3.3e38, -3.3e38)
    codes, ranges = ref.quantise(flat)
    assert not codes.any() and ranges[0].tolist() == [0.0, 7.5] and np.isnan(ranges[1:]).all()


def test_attention_reference_without_quantisation_error():
    # rows that 4 bits hold exactly: the reference of the 16-bit cache
    import paged_ref
    rng = np.random.default_rng(4)
    n = rng.integers(0, 16, (4, 2, 2, 8, 32))
    n[..., 0], n[..., 1] = 0, 15
    x = (n * 0.25 - 2.0).astype(np.float32)
    codes, ranges = ref.quantise(x)
    assert np.array_equal(ref.values(codes, ranges), x)
    qkv = rng.standard_normal((2, 8 * 32)).astype(np.float32)
    table = np.array([[2, 0], [1, 3]])
    y, lse2, _, _ = ref.attend4(qkv, codes, ranges, table, [11, 4], 4, 5, 2)
    for b, rows in ((0, [0, 1, 6, 7, 8, 9, 10]), (1, [0, 1, 2, 3])):
        for h in range(4):
            k, u = (np.stack([x[table[b, r // 8], w, h // 2, r % 8] for r in rows]).astype(np.float64) for w in (0, 1))
            want = paged_ref.attend(qkv[b].reshape(8, 32)[h].astype(np.float64), k, u)
            assert np.allclose(y[b].reshape(4, 32)[h], want[0]) and abs(lse2[b, h] - want[1]) < 1e-12


def test_logprob_gradient_reference_against_differences():
    rng = np.random.default_rng(5)
    z = rng.standard_normal((3, 11)) * 2
    z[1, 4] = -np.inf
    t, dl, de = [3, 0, -1], rng.standard_normal(3), rng.standard_normal(3)
    _, ent, _, _, p, lp = ref.logprobs(z, t)
    g = ref.logprobs_grad(p, lp, ent, t, dl, de)
    assert g[1, 4] == 0

    def loss(x):
        a, e = ref.logprobs(x, t)[:2]
        return (dl * a).sum() + (de * e).sum()
    for i in range(3):
        for j in range(11):
            if z[i, j] == -np.inf:
                continue
            d = np.zeros_like(z)
            d[i, j] = 1e-5
            assert abs((loss(z + d) - loss(z - d)) / 2e-5 - g[i, j]) < 1e-8


def test_logprob_reference_against_torch():
    rng = np.random.default_rng(6)
    z = rng.standard_normal((4, 300)) * 3
    z[2, 5:90] = -np.inf
    t = [0, 299, 100, 7]
    logp, ent, ids, top, _, _ = ref.logprobs(z, t, 6)
    lp = torch.log_softmax(torch.from_numpy(z), -1)
    assert np.allclose(logp, lp[torch.arange(4), t].numpy(), atol=1e-13)
    assert np.allclose(ent, torch.distributions.Categorical(logits=torch.from_numpy(z)).entropy().numpy(), atol=1e-5)
    v, i = torch.topk(lp, 6)
    assert np.array_equal(ids, i.numpy()) and np.allclose(top, v.numpy(), atol=1e-13)
