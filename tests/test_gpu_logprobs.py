"""Log probabilities, entropy, the most probable tokens and their gradient, against serving_ref.py.

Tolerances, with d = z - m and the sums S = sum e^d, A = sum e^d d in fp32. A term e^d is off by 2^-22 (the exponential), 2^-23 |d|
(d and d log2 e rounded) of itself; a lane adds up V / 256 terms at most one after another where one block has the row, 40 more
steps join the lanes, warps and blocks, each off by 2^-24 of a partial sum: u = 2^-22 + 2^-23 E|d| + 2^-24 (V / 128 + 40) bounds S
relatively, and A with E|d|^2 for E|d| besides. ln S and the last subtractions: 2^-22 (1 + |ln S| + |d_t|).
Gradient: p is off by 2^-22 + 2^-23 |d| + u of itself; then c = g + ge (entropy - ln S) and ge d, three roundings of their size.
A bf16 result is rounded once more (2^-8), an fp32 one 2^-24.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402
from gpu_util import dev_f32, dev_i32, host  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


def logits(M, V, seed, kind="normal"):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((M, V)) * 2.5 - 4.0
    z[np.arange(M), rng.integers(0, V, M)] += 9.0 * rng.random(M)
    if kind == "masked":
        z[:, rng.random(V) < 0.3] = -np.inf
        z[:, rng.integers(0, V)] = 1.0
    if kind == "lowest":
        z[:, rng.random(V) < 0.5] = -3.38953139e38      # the lowest number of bf16
    if kind == "ties":
        z = np.round(z)
    if kind == "rising":
        z = np.sort(z, -1)
    if kind == "far":
        z = z * 100.0 + 5000.0
    return z


def run(z, targets, K, dtype, ld=None, offset=0, want=("entropy", "stats")):
    """(outputs, logits as the device has them in 64 bits, device tensors)."""
    from decoder_only_transformer_gpt_gb300 import binding
    M, V = z.shape
    flat = torch.full((offset + M * (ld or V) + 16,), float("nan"), dtype=dtype, device="cuda")
    dz = flat[offset: offset + M * (ld or V)].view(M, ld or V)[:, :V]
    dz.copy_(torch.from_numpy(z))
    d = {"logp": None if targets is None else torch.full((M,), 7.0, device="cuda"),
         "entropy": torch.full((M,), 7.0, device="cuda") if "entropy" in want else None,
         "stats": torch.full((M, 2), 7.0, device="cuda") if "stats" in want else None,
         "top_ids": torch.full((M, K), 7, dtype=torch.int32, device="cuda") if K else None,
         "top_logp": torch.full((M, K), 7.0, device="cuda") if K else None}
    binding.logprobs(dz, None if targets is None else dev_i32(np.array(targets)), d["logp"], entropy=d["entropy"],
                     stats=d["stats"], top_ids=d["top_ids"], top_logp=d["top_logp"])
    return d, host(dz), dz


def bounds(z, p, lp):
    V = z.shape[1]
    fin = np.where(p > 0, z, 0)
    d = np.where(p > 0, np.abs(fin - z.max(-1, keepdims=True)), 0)
    ed, ed2 = (p * d).sum(-1), (p * d * d).sum(-1)
    steps = 2.0 ** -24 * (V / 128 + 40)
    u = 2.0 ** -22 + 2.0 ** -23 * ed + steps
    ua = (2.0 ** -22 + steps + 2.0 ** -23) * ed + 2.0 ** -23 * ed2
    ln_s = -np.where(p > 0, lp, -np.inf).max(-1)
    return d, ed, u, ua, ln_s


def check(d, z, targets, K):
    M, V = z.shape
    logp, ent, ids, top, p, lp = ref.logprobs(z, targets, K)
    ok = np.isfinite(ent)
    if d["top_ids"] is not None:
        assert np.array_equal(d["top_ids"].cpu().numpy(), ids)
    for name, want in (("logp", logp), ("entropy", ent)):
        if d[name] is not None:
            assert np.isnan(host(d[name])[~ok]).all()
    if d["stats"] is not None:
        assert np.isnan(host(d["stats"])[~ok]).all()
    if d["top_logp"] is not None:
        assert np.isnan(host(d["top_logp"])[~ok]).all()
    if not ok.any():
        return p, lp, ent
    dd, ed, u, ua, ln_s = bounds(z[ok], p[ok], lp[ok])
    if d["logp"] is not None:
        got, t = host(d["logp"])[ok], logp[ok]
        both = np.isfinite(t)
        assert np.array_equal(got[~both], t[~both])
        lim = u + 2.0 ** -22 * (1 + 2 * ln_s + np.abs(np.where(both, t, 0)))
        assert (np.abs(got[both] - t[both]) <= lim[both]).all()
        none = np.array([x == -1 for x in targets])[ok]
        assert (got[none] == 0).all()
    if d["entropy"] is not None:
        assert (np.abs(host(d["entropy"])[ok] - ent[ok]) <= u * (1 + ed) + ua + 2.0 ** -22 * (1 + ln_s + ed)).all()
    if d["stats"] is not None:
        s = host(d["stats"])[ok]
        assert np.array_equal(s[:, 0], z[ok].max(-1))
        want = np.exp(-np.where(p[ok] > 0, lp[ok], -np.inf).max(-1))
        assert (np.abs(s[:, 1] - want) <= u * want * 1.01).all()
    if d["top_logp"] is not None:
        got, t = host(d["top_logp"])[ok], top[ok]
        both = np.isfinite(t)
        assert np.array_equal(got[~both], t[~both])
        lim = u[:, None] + 2.0 ** -22 * (1 + 2 * ln_s[:, None] + np.abs(np.where(both, t, 0)))
        assert (np.abs(got[both] - t[both]) <= lim[both]).all()
    return p, lp, ent


def some_targets(M, V, seed):
    t = np.random.default_rng(seed).integers(0, V, M)
    t[::5] = -1
    t[-1] = V - 1
    if M > 1:
        t[1] = 0
    return t.tolist()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1, 2, 5, 31, 33, 127, 515, 1024, 4099, 9001, 20011])
def test_vocabularies(gpt_lib, dtype, V):
    from decoder_only_transformer_gpt_gb300 import binding
    for M in (1, 7):
        for K in sorted({0, 1, min(V, 5), min(V, 32)}):
            t = some_targets(M, V, V)
            d, z, _ = run(logits(M, V, V + K), t, K, dtype)
            binding.status()
            check(d, z, t, K)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M", [1, 16, 30, 60, 160, 330])
def test_rows_of_a_large_vocabulary(gpt_lib, dtype, M):
    from decoder_only_transformer_gpt_gb300 import binding
    V = 50257 if M < 100 else 12345
    z = logits(8, V, M)[np.arange(M) % 8]
    z = np.where(np.arange(M)[:, None] >= 8, np.roll(z, 17, 1), z)
    t = some_targets(M, V, M)
    d, zd, _ = run(z, t, 5, dtype)
    binding.status()
    keep = sorted(set(range(min(M, 12))) | {M - 1})
    check({k: None if v is None else v[keep] for k, v in d.items()}, zd[keep], [t[i] for i in keep], 5)
    # equal rows give equal results, wherever they are
    for i in range(16, M):
        assert torch.equal(d["entropy"][i], d["entropy"][8 + i % 8]) or M > 100 or V != 50257


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,V", [(3, 50257), (20, 50257), (60, 20011), (130, 9001), (700, 2500), (200, 400)])
@pytest.mark.parametrize("K", [1, 16, 17, 32])
def test_more_equal_logits_than_are_wanted(gpt_lib, dtype, M, V, K):
    # rows all equal; of two values, a few hundred of the larger; the larger ones side by side
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(V + K)
    z = np.full((M, V), -1.5)
    for i in range(1, M, 3):
        z[i, rng.permutation(V)[:300]] = 2.0
    for i in range(2, M, 3):
        at = int(rng.integers(0, V - 200))
        z[i, at: at + 200] = 2.0 + np.arange(200) / 64.0
    t = some_targets(M, V, K)
    d, zd, _ = run(z, t, K, dtype)
    binding.status()
    keep = sorted({0, 1, 2, M // 2, M - 2, M - 1})
    check({k: None if v is None else v[keep] for k, v in d.items()}, zd[keep], [t[i] for i in keep], K)
    for i in range(3, M, 3):                         # equal rows, equal results
        assert torch.equal(d["top_ids"][i], d["top_ids"][0])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,K", [(2049, 1), (3001, 5), (5003, 0), (5003, 32), (5120, 32)])
@pytest.mark.parametrize("M", [1300, 2437])
def test_many_short_rows(gpt_lib, dtype, V, K, M):
    # rows of different shifts of nine, and single ones among them without a distribution or with one token left
    from decoder_only_transformer_gpt_gb300 import binding
    z = logits(9, V, V + K)[np.arange(M) % 9]
    for i in range(9):
        z[i::9] = np.roll(z[i::9], 13 * i, 1)
    bad, alone = [11, 640, M - 2], [12, 641, M - 1]
    z[bad[0], V // 2], z[bad[1], V - 1] = np.nan, np.inf
    z[bad[2]] = -np.inf
    for i in alone:
        z[i] = -np.inf
        z[i, (7 * i) % V] = -3.0
    t = some_targets(M, V, M)
    d, zd, _ = run(z, t, K, dtype, ld=V + 3, offset=1)
    binding.status()
    keep = sorted({0, 1, 7, 8, M // 2, M - 9} | set(bad) | set(alone) | {b - 1 for b in bad} | {a + 1 for a in alone[:2]})
    check({k: None if v is None else v[keep] for k, v in d.items()}, zd[keep], [t[i] for i in keep], K)
    want = np.array([torch.isfinite(d["entropy"][i]).item() for i in range(M)])
    assert (want == ~np.isin(np.arange(M), bad)).all()
    _, ent, _, _, p, lp = ref.logprobs(zd[:9], [0] * 9, 0)
    _, ed, u, ua, ln_s = bounds(zd[:9], p, lp)       # (all rows of a shift have its entropy, to twice the bounds)
    lim = 2.0 * (u * (1 + ed) + ua + 2.0 ** -22 * (1 + ln_s + ed))
    got = host(d["entropy"])
    for i in range(M):
        if i not in bad and i not in alone:
            assert abs(got[i] - ent[i % 9]) <= lim[i % 9]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [65536, 65541, 131075, 300007])
def test_vocabularies_of_several_chunks_a_note(gpt_lib, dtype, V):
    # a thread notes the largest logit of several chunks; the best tokens next to each other, or all equal
    for M in (2, 40):
        z = np.zeros((M, V))
        z[0] = logits(1, V, V)[0]
        z[0, 1000:1040] = 30.0 + np.arange(40) % 7
        z[1, 5:V:3] = -1.0
        t = some_targets(M, V, V)
        d, zd, _ = run(z, t, 32, dtype)
        check({k: None if v is None else v[:2] for k, v in d.items()}, zd[:2], t[:2], 32)
        for i in range(2, M):
            assert d["top_ids"][i].tolist() == list(range(32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["masked", "lowest", "ties", "rising", "far"])
def test_kinds_of_logits(gpt_lib, dtype, kind):
    for M, V in ((3, 700), (2, 9000), (40, 3001)):
        for K in (1, 8, 32):
            t = some_targets(M, V, K)
            d, z, _ = run(logits(M, V, K, kind), t, K, dtype)
            check(d, z, t, K)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_without_a_distribution(gpt_lib, dtype):
    for V in (40, 6000):
        z = logits(9, V, 1)
        z[1] = -np.inf
        z[2, V - 1] = np.nan
        z[3, 0] = np.inf
        z[4] = 2.0
        z[5] = -3.38953139e38
        z[6, 1:] = -np.inf
        z[7, [3, 9]] = (np.inf, np.nan)
        t = [0, 0, 1, 0, V - 1, 2, 0, 3, 5]
        d, zd, _ = run(z, t, 4, dtype)
        check(d, zd, t, 4)
        assert host(d["logp"])[6] == 0 and host(d["entropy"])[6] == 0
        assert d["top_ids"][6].tolist() == [0, 1, 2, 3] and d["top_ids"][5].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_alignment(gpt_lib, dtype):
    for V, ld, offset in ((50, 57, 1), (1000, 1003, 3), (4097, 4100, 5), (4096, 4104, 7), (9, 64, 2)):
        t = some_targets(6, V, V)
        d, z, _ = run(logits(6, V, V), t, 3, dtype, ld=ld, offset=offset)
        check(d, z, t, 3)


def test_a_transposed_or_narrow_tensor_is_refused(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    z, e = torch.zeros(8, 8, device="cuda"), torch.zeros(8, device="cuda")
    for bad in (z.t()[:, :4], z[:, ::2], z[:1, :4].expand(8, 4)):
        with pytest.raises(ValueError, match="strides"):
            binding.logprobs(bad, None, None, entropy=e)


def test_only_what_is_asked_for(gpt_lib):
    z = logits(4, 300, 2)
    t = [5, 6, 7, 8]
    full, zd, _ = run(z, t, 3, F32)
    for targets, K, want in ((t, 0, ()), (None, 0, ("entropy",)), (None, 0, ("stats",)), (None, 3, ())):
        d, _, _ = run(z, targets, K, F32, want=want)
        for k, v in d.items():
            assert v is None or torch.equal(v, full[k])


def test_targets_outside_the_vocabulary(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (300, -2, 2 ** 31 - 1, -2 ** 31):
        t = [5, bad, -1, 8]
        d, z, _ = run(logits(4, 300, 3), t, 2, F32)
        with pytest.raises(binding.GptError) as e:
            binding.status()
        assert e.value.code == binding.GPT_ETOKEN
        binding.status()
        check(d, z, [5, -1, -1, 8], 2)


def grads(z, targets, dtype, dlogp, dentropy, in_place=False, ld=None, offset=0, dld=None, doffset=0):
    from decoder_only_transformer_gpt_gb300 import binding
    d, zd, dz = run(z, targets, 0, dtype, ld=ld, offset=offset)
    M, V = z.shape
    flat = torch.full((doffset + M * (dld or V) + 16,), 99.0, dtype=dtype, device="cuda")
    out = dz if in_place else flat[doffset: doffset + M * (dld or V)].view(M, dld or V)[:, :V]
    binding.logprobs_bwd(dz, None if targets is None else dev_i32(np.array(targets)), d["stats"],
                         None if dlogp is None else dev_f32(dlogp), out,
                         entropy=None if dentropy is None else d["entropy"],
                         dentropy=None if dentropy is None else dev_f32(dentropy))
    binding.status()
    return out, zd, flat


def check_grad(out, z, targets, dtype, dlogp, dentropy):
    M, V = z.shape
    _, ent, _, _, p, lp = ref.logprobs(z, targets)
    want = ref.logprobs_grad(p, lp, ent, targets, dlogp, dentropy)
    got = host(out)
    ok = np.isfinite(ent)
    assert np.isnan(got[~ok]).all()
    if not ok.any():
        return
    z, p, lp, ent, want, got = z[ok], p[ok], lp[ok], ent[ok], want[ok], got[ok]
    d, ed, u, ua, ln_s = bounds(z, p, lp)
    valid = np.array([0 <= t < V for t in targets])[ok] if targets is not None else np.zeros(ok.sum(), bool)
    g = np.abs(np.where(valid, np.asarray(dlogp, np.float64)[ok], 0)) if dlogp is not None else np.zeros(ok.sum())
    ge = np.abs(np.asarray(dentropy, np.float64)[ok]) if dentropy is not None else np.zeros(ok.sum())
    ee = u * (1 + ed) + ua + 2.0 ** -22 * (1 + ln_s + ed)             # the entropy's own error
    size = g[:, None] + ge[:, None] * (ent[:, None] + ln_s[:, None] + d)
    tol = p * ((2.0 ** -22 + 2.0 ** -23 * d + u[:, None]) * size + 3 * 2.0 ** -23 * size + ge[:, None] * (ee + u)[:, None])
    tol = 1.01 * tol + torch.finfo(dtype).eps / 2 * np.abs(want) + 2.0 ** -24 * g[:, None] * (p > 0)
    tol = tol + (2.0 ** -133 if dtype is BF16 else 2.0 ** -149) + 2.0 ** -126 * size   # subnormal results; exponentials below 2^-126 are 0
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [1, 3, 8, 40, 515, 4096, 4099, 9001, 20011])
def test_gradient(gpt_lib, dtype, V):
    rng = np.random.default_rng(V)
    for M, kind in ((1, "normal"), (6, "masked"), (5, "lowest"), (4, "ties")):
        t = some_targets(M, V, V)
        a, b = rng.standard_normal(M).astype(np.float32), (rng.standard_normal(M) * 0.3).astype(np.float32)
        for dl, de, tt in ((a, b, t), (a, None, t), (None, b, None)):
            out, z, _ = grads(logits(M, V, V, kind), tt, dtype, dl, de)
            check_grad(out, z, tt, dtype, dl, de)
        same, _, _ = grads(logits(M, V, V, kind), t, dtype, a, b, in_place=True)
        out, _, _ = grads(logits(M, V, V, kind), t, dtype, a, b)
        assert torch.equal(same, out)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_strides(gpt_lib, dtype):
    rng = np.random.default_rng(1)
    for V, ld, off, dld, doff in ((50, 57, 1, 50, 0), (1000, 1003, 3, 1005, 1), (4097, 4100, 5, 4100, 5), (9, 64, 2, 11, 3)):
        t = some_targets(6, V, V)
        a, b = rng.standard_normal(6).astype(np.float32), rng.standard_normal(6).astype(np.float32)
        out, z, flat = grads(logits(6, V, V), t, dtype, a, b, ld=ld, offset=off, dld=dld, doffset=doff)
        check_grad(out, z, t, dtype, a, b)
        rest = flat[doff: doff + 6 * dld].view(6, dld)[:, V:]
        assert (rest == 99.0).all() and (flat[:doff] == 99.0).all() and (flat[doff + 6 * dld:] == 99.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_of_rows_without_a_distribution(gpt_lib, dtype):
    z = logits(5, 700, 1)
    z[1], z[2, 3], z[3, 699], z[4, 5:] = -np.inf, np.nan, np.inf, -np.inf
    t, a, b = [0, 0, 1, 0, 2], np.ones(5, np.float32), np.ones(5, np.float32)
    out, zd, _ = grads(z, t, dtype, a, b)
    check_grad(out, zd, t, dtype, a, b)


def test_gradient_against_differences(gpt_lib):
    # the forward call's own outputs along a direction: steps of 2^-5, whose error is of the order h^2 = 1e-3 of the slope
    rng = np.random.default_rng(4)
    M, V = 4, 333
    z, u = logits(M, V, 4), rng.standard_normal((M, V))
    t, a, b = [3, 332, 0, 100], rng.standard_normal(M).astype(np.float32), rng.standard_normal(M).astype(np.float32)

    def loss(x):
        d, _, _ = run(x, t, 0, F32)
        return a * host(d["logp"]) + b * host(d["entropy"])
    h = 2.0 ** -5
    slope = (8 * (loss(z + h * u) - loss(z - h * u)) - (loss(z + 2 * h * u) - loss(z - 2 * h * u))) / (12 * h)
    out, _, _ = grads(z, t, F32, a, b)
    # fourth-order differences: h^4 times a fifth derivative of a few units, and fp32 outputs of size 10: 10 2^-23 / h each
    assert (np.abs((host(out) * u).sum(-1) - slope) <= 1e-4 * (np.abs(a) + np.abs(b)) * 10).all()


def test_more_rows_than_a_wave_and_a_graph(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    M, V = 3001, 257
    z = torch.randn(M, V, device="cuda")
    t = torch.randint(0, V, (M,), device="cuda", dtype=torch.int32)
    lp, en, st = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda"), torch.zeros(M, 2, device="cuda")
    ids, top = torch.zeros(M, 3, dtype=torch.int32, device="cuda"), torch.zeros(M, 3, device="cuda")
    g, dl = torch.zeros(M, V, device="cuda"), torch.randn(M, device="cuda")
    graph = torch.cuda.CUDAGraph()
    binding.logprobs(z, t, lp, entropy=en, stats=st, top_ids=ids, top_logp=top)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        binding.logprobs(z, t, lp, entropy=en, stats=st, top_ids=ids, top_logp=top)
        binding.logprobs_bwd(z, t, st, dl, g)
    z.copy_(torch.randn(M, V, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    x = z.double()
    want = torch.log_softmax(x, -1)
    assert torch.allclose(lp.double(), want.gather(1, t.long()[:, None])[:, 0], atol=4e-6, rtol=0)
    assert torch.equal(ids.long(), torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :3])
    one = torch.nn.functional.one_hot(t.long(), V)
    assert torch.allclose(g.double(), dl.double()[:, None] * (one - want.exp()), atol=4e-6, rtol=0)


def test_offsets_past_32_bits(gpt_lib):
    # rows 2.4 GB apart, and one row of 270,000,001 logits
    from decoder_only_transformer_gpt_gb300 import binding
    ld, V = 1_200_000_001, 5000
    flat = torch.empty(2 * ld + V, dtype=BF16, device="cuda")
    z = torch.as_strided(flat, (3, V), (ld, 1))
    z.copy_(torch.from_numpy(logits(3, V, 9)))
    t, lp, st = dev_i32(np.array([0, 77, V - 1])), torch.zeros(3, device="cuda"), torch.zeros(3, 2, device="cuda")
    ids, top = torch.zeros(3, 5, dtype=torch.int32, device="cuda"), torch.zeros(3, 5, device="cuda")
    binding.logprobs(z, t, lp, stats=st, top_ids=ids, top_logp=top)
    a, _, i, v, _, _ = ref.logprobs(host(z), [0, 77, V - 1], 5)
    assert np.array_equal(ids.cpu().numpy(), i) and np.abs(host(lp) - a).max() < 8e-6 and np.abs(host(top) - v).max() < 8e-6
    binding.logprobs_bwd(z, t, st, torch.ones(3, device="cuda"), z)
    p = np.exp(ref.logprobs(host(z), None)[5])
    assert np.isfinite(p).all() and abs(float(z[2, V - 1].float()) - (1 - np.exp(a[2]))) < 2.0 ** -8
    del flat, z
    V = 270_000_001
    z = torch.randn(1, V, device="cuda")
    z[0, [5, V - 1, V // 2]] = torch.tensor([9.0, 9.0, 11.0], device="cuda")
    lp, en = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    ids, top = torch.zeros(1, 3, dtype=torch.int32, device="cuda"), torch.zeros(1, 3, device="cuda")
    binding.logprobs(z, dev_i32(np.array([V - 1])), lp, entropy=en, top_ids=ids, top_logp=top)
    assert ids[0].tolist() == [V // 2, 5, V - 1]
    lse = float(torch.logsumexp(z.double(), -1))
    # V / 2048 sums one after another in a lane of the eight blocks: 2^-24 each
    assert abs(float(lp) - (9.0 - lse)) <= 2.0 ** -24 * V / 1024 and abs(float(top[0, 0]) - (11.0 - lse)) <= 2.0 ** -24 * V / 1024


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,V", [(1, 50257), (16, 50257), (60, 20011), (400, 9001), (1300, 3001), (300, 700)])
def test_one_result_bit_for_bit(gpt_lib, dtype, M, V):
    # whatever order the tokens come in, alone and beside another call
    from decoder_only_transformer_gpt_gb300 import binding
    z = torch.from_numpy(logits(8, V, V)).to(dtype).cuda()[torch.arange(M) % 8].contiguous()
    z[::3, ::11] = 1.5                                  # a few hundred equal ones at most
    t = dev_i32(np.arange(M) % V)
    side = torch.cuda.Stream()
    for K in (1, 5, 16, 32):
        out = []
        for i in range(12):
            d = [torch.empty(M, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, 2, device="cuda"),
                 torch.empty(M, K, dtype=torch.int32, device="cuda"), torch.empty(M, K, device="cuda")]
            torch.cuda.synchronize()
            if i % 2:
                with torch.cuda.stream(side):
                    other = [x.clone() for x in d]
                    binding.logprobs(z, t, other[0], entropy=other[1], stats=other[2], top_ids=other[3], top_logp=other[4])
            binding.logprobs(z, t, d[0], entropy=d[1], stats=d[2], top_ids=d[3], top_logp=d[4])
            torch.cuda.synchronize()
            out.append(d)
            if i % 2:
                out.append(other)
        for d in out[1:]:
            assert all(torch.equal(x, y) for x, y in zip(d, out[0]))
