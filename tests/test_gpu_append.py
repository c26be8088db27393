"""Rotation of fused rows, alone and on the way into the paged caches of 16-bit and 4-bit rows, and 4-bit rows read back,
against the references of serving_ref.py.

Tolerances. A rotated value is a c - b s in fp32: the phase is rounded to fp32 (2^-25 half turns: 9.4e-8 rad), sine and cosine
are off by one unit in the last place (1.2e-7), two roundings (6e-8 each) follow: 4e-7 (|a| + |b|); then one rounding to
bf16, 2^-8 of the value at most. Everything else is copies, or codes whose every rounding the reference repeats: equal.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402
from gpu_util import dev_bf16, dev_f32, dev_i32, host, rand_bf16  # noqa: E402


def close(got, want, mag):
    return (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 4e-7 * mag * (1 + 2.0 ** -8)).all()


class Case:
    def __init__(self, B, T, H, Hkv, D, rot, inter, page=16, seed=0, counts=True, spare=2):
        rng = np.random.default_rng(seed)
        self.B, self.T, self.H, self.Hkv, self.D, self.rot, self.inter, self.page = B, T, H, Hkv, D, rot, inter, page
        self.NH = H + 2 * Hkv
        self.x = rand_bf16(rng, (B, T, self.NH, D))
        self.freq = ref.freqs(rot) if rot else []
        self.pos = rng.integers(-2 ** 31, 2 ** 31 - T, B)
        self.pos[0] = 7
        self.start = rng.integers(0, 3 * page, B)
        self.count = rng.integers(0, T + 1, B) if counts else np.full(B, T)
        self.count[0] = T
        mp = (T + 3 * page + page - 1) // page
        n = B * mp + spare
        self.pages = n
        self.table = rng.permutation(n)[: B * mp].reshape(B, mp).astype(np.int32)

    def device(self):
        from decoder_only_transformer_gpt_gb300 import binding
        self.qkv = dev_bf16(self.x.reshape(self.B, self.T, self.NH * self.D))
        self.turns = binding.rotary_turns(self.freq) if self.rot else None
        self.d = {k: dev_i32(getattr(self, k)) for k in ("pos", "start", "count", "table")}
        return self

    def want(self, pos, inverse=False):
        return ref.rotate(self.x, self.H, self.Hkv, self.freq, pos, self.inter, inverse)

    def rows(self):
        """(sequence, token, page, slot) of every stored token."""
        for b in range(self.B):
            for t in range(self.count[b]):
                r = self.start[b] + t
                yield b, t, self.table[b, r // self.page], r % self.page


SHAPES = [(1, 1, 1, 1, 64, 64, False), (3, 5, 4, 2, 32, 32, True), (2, 33, 12, 12, 64, 64, False), (2, 7, 25, 5, 64, 32, True),
          (4, 1, 7, 7, 32, 16, False), (1, 50, 3, 1, 64, 16, False), (2, 9, 16, 1, 64, 48, True), (5, 3, 9, 3, 32, 32, False),
          (1, 2000, 1, 1, 32, 32, False), (2, 1300, 3, 3, 64, 64, True)]


@pytest.mark.parametrize("shape", SHAPES)
def test_rotary(gpt_lib, shape):
    from decoder_only_transformer_gpt_gb300 import binding
    c = Case(*shape).device()
    for inverse in (False, True):
        for pos in (None, c.d["pos"]):
            out = torch.full_like(c.qkv, 99.0)
            binding.rotary(c.qkv, out, c.H, c.Hkv, c.turns, pos=pos, interleaved=c.inter, inverse=inverse)
            binding.status()
            got = host(out).reshape(c.x.shape)
            want, mag = c.want(np.zeros(c.B) if pos is None else c.pos, inverse)
            assert close(got, want, mag)
            assert np.array_equal(got[:, :, c.H + c.Hkv:], c.x[:, :, c.H + c.Hkv:])
            assert np.array_equal(got[..., c.rot:], c.x[..., c.rot:])
            again = c.qkv.clone()
            binding.rotary(again, again, c.H, c.Hkv, c.turns, pos=pos, interleaved=c.inter, inverse=inverse)
            assert torch.equal(again, out)


def test_far_positions_keep_their_phase(gpt_lib):
    # neighbours at the ends of the 32-bit range: products depend on the distance alone
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(1)
    q, k = rand_bf16(rng, 64), rand_bf16(rng, 64)
    x = np.zeros((1, 2, 3, 64), np.float32)
    x[0, 0, 0], x[0, 1, 1] = q, k
    turns, got = binding.rotary_turns(ref.freqs(64)), []
    for pos in (0, 2 ** 31 - 2, -2 ** 31, 123456789):
        qkv = dev_bf16(x.reshape(1, 2, 192))
        binding.rotary(qkv, qkv, 1, 1, turns, pos=dev_i32(np.array([pos])))
        y = host(qkv).reshape(2, 3, 64)
        got.append(float(y[0, 0] @ y[1, 1]))
    # each factor is off by 2^-8 of itself at most
    assert max(got) - min(got) <= 4 * 2.0 ** -8 * float(np.abs(q) @ np.abs(q) + np.abs(k) @ np.abs(k))
    w, _ = ref.rotate(x, 1, 1, ref.freqs(64), [0], False)
    assert abs(got[0] - w[0, 0, 0] @ w[0, 1, 1]) <= 2 * 2.0 ** -8 * float(np.abs(q) @ np.abs(q) + np.abs(k) @ np.abs(k))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("page", [8, 32])
def test_append(gpt_lib, shape, page):
    from decoder_only_transformer_gpt_gb300 import binding
    c = Case(*shape, page=page, seed=3).device()
    rng = np.random.default_rng(4)
    pool0 = rand_bf16(rng, (c.pages, 2, c.Hkv, page, c.D))
    w0 = rng.random((c.pages, c.Hkv, page)).astype(np.float32)
    for pos in (None, c.d["pos"]):
        pool, weight, out = dev_bf16(pool0), dev_f32(w0), torch.full_like(c.qkv, 99.0)
        binding.paged_append(c.qkv, pool, c.d["table"], c.H, turns=c.turns, start=c.d["start"], count=c.d["count"], pos=pos,
                             weight=weight, out=out, interleaved=c.inter)
        binding.status()
        o, p, w = host(out).reshape(c.x.shape), host(pool), host(weight)
        want, mag = c.want(c.start if pos is None else c.pos)
        seen = np.zeros((c.pages, page), bool)
        for b, t, pg, sl in c.rows():
            assert close(o[b, t], want[b, t], mag[b, t])
            assert np.array_equal(p[pg, 0, :, sl], o[b, t, c.H: c.H + c.Hkv])
            assert np.array_equal(p[pg, 1, :, sl], c.x[b, t, c.H + c.Hkv:])
            assert not w[pg, :, sl].any()
            seen[pg, sl] = True
        keep = ~seen
        assert np.array_equal(p.transpose(0, 3, 1, 2, 4)[keep], pool0.transpose(0, 3, 1, 2, 4)[keep])
        assert np.array_equal(w.transpose(0, 2, 1)[keep], w0.transpose(0, 2, 1)[keep])
        for b in range(c.B):
            assert (o[b, c.count[b]:] == 99.0).all()
        # without the rows, or the weights, or in place: the same cache
        for how in ("no out", "in place"):
            p2, x2 = dev_bf16(pool0), c.qkv.clone()
            binding.paged_append(x2, p2, c.d["table"], c.H, turns=c.turns, start=c.d["start"], count=c.d["count"], pos=pos,
                                 out=x2 if how == "in place" else None, interleaved=c.inter)
            assert torch.equal(p2, pool)
            for b in range(c.B):
                n = c.count[b]
                assert torch.equal(x2[b, :n], (out if how == "in place" else c.qkv)[b, :n]) and torch.equal(x2[b, n:], c.qkv[b, n:])


def test_append_without_rotation_is_a_store(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    c = Case(3, 40, 8, 4, 64, 0, False, seed=5).device()
    pools = [torch.zeros(c.pages, 2, c.Hkv, c.page, c.D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = torch.zeros_like(c.qkv)
    binding.paged_append(c.qkv, pools[0], c.d["table"], c.H, start=c.d["start"], count=c.d["count"], out=out)
    binding.paged_store(c.qkv, pools[1], c.d["table"], c.H, start=c.d["start"], count=c.d["count"])
    assert torch.equal(*pools)
    for b in range(c.B):
        assert torch.equal(out[b, :c.count[b]], c.qkv[b, :c.count[b]])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("page", [8, 64])
def test_append_in_four_bits_and_back(gpt_lib, shape, page):
    from decoder_only_transformer_gpt_gb300 import binding
    c = Case(*shape, page=page, seed=6).device()
    codes = torch.full((c.pages, 2, c.Hkv, page, c.D // 2), 0x5a, dtype=torch.uint8, device="cuda")
    ranges = torch.full((c.pages, 2, c.Hkv, page, 2), 3.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(c.qkv, 99.0)
    binding.paged_append4(c.qkv, codes, ranges, c.d["table"], c.H, turns=c.turns, start=c.d["start"], count=c.d["count"],
                          pos=c.d["pos"], out=out, interleaved=c.inter)
    rows = torch.full((c.B, c.T, 2 * c.Hkv * c.D), 99.0, dtype=torch.bfloat16, device="cuda")
    binding.paged_load4(codes, ranges, c.d["table"], rows, start=c.d["start"], count=c.d["count"])
    binding.status()
    o, rows = host(out).reshape(c.x.shape), host(rows).reshape(c.B, c.T, 2 * c.Hkv, c.D)
    cd, rg = codes.cpu().numpy(), host(ranges)
    want, mag = c.want(c.pos)
    want_codes, want_ranges = ref.quantise(o[:, :, c.H:].astype(np.float32))
    back = ref.values(want_codes, want_ranges).astype(np.float32)
    seen = np.zeros((c.pages, page), bool)
    for b, t, pg, sl in c.rows():
        assert close(o[b, t], want[b, t], mag[b, t])
        for which in (0, 1):
            heads = slice(which * c.Hkv, (which + 1) * c.Hkv)
            assert np.array_equal(cd[pg, which, :, sl], want_codes[b, t, heads])
            assert np.array_equal(rg[pg, which, :, sl], want_ranges[b, t, heads])
        assert np.array_equal(rows[b, t], torch.from_numpy(back[b, t]).bfloat16().double().numpy())
        seen[pg, sl] = True
    assert (cd.transpose(0, 3, 1, 2, 4)[~seen] == 0x5a).all() and (rg.transpose(0, 3, 1, 2, 4)[~seen] == 3.0).all()
    for b in range(c.B):
        assert (rows[b, c.count[b]:] == 99.0).all() and (o[b, c.count[b]:] == 99.0).all()


def test_four_bits_of_odd_rows(gpt_lib):
    # constant rows, subnormal and huge ranges, ties of codes, values that are not finite
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(7)
    D, T = 32, 14
    x = rand_bf16(rng, (1, T, 3, D))
    k = x[0, :, 1]
    k[0] = 2.5
    k[1] = 0.0
    k[2] = np.where(np.arange(D) % 2, 1e-40, 0.0)
    k[3] = np.where(np.arange(D) % 2, 1.5e38, -1.5e38)
    k[4] = np.where(np.arange(D) % 2, 3e38, -3e38)
    k[5, 3] = np.nan
    k[6, 31] = np.inf
    k[7, 0] = -np.inf
    k[8] = np.arange(D) * 0.5 - 3.0                     # half steps: ties
    k[8, 16:] = 4.5
    k[9, :] = -0.0
    k[10] = 1e-37 * rng.random(D)
    k[11, :5] = (np.inf, -np.inf, np.nan, 1, 2)
    k[12] *= 1e30
    k[13] *= 1e-30
    x[0, :, 2] = k[::-1]
    x = torch.from_numpy(x).bfloat16()
    xs = x.float().numpy()
    table = dev_i32(np.array([[1, 0]]))
    codes = torch.zeros(2, 2, 1, 8, D // 2, dtype=torch.uint8, device="cuda")
    ranges = torch.zeros(2, 2, 1, 8, 2, dtype=torch.bfloat16, device="cuda")
    binding.paged_append4(x.view(1, T, 3 * D).cuda(), codes, ranges, table, 1)
    rows = torch.zeros(1, T, 2 * D, dtype=torch.bfloat16, device="cuda")
    binding.paged_load4(codes, ranges, table, rows)
    binding.status()
    want_codes, want_ranges = ref.quantise(xs[0, :, 1:])
    got = host(rows).reshape(T, 2, D)
    for t in range(T):
        pg, sl = (1, t) if t < 8 else (0, t - 8)
        for w in (0, 1):
            assert np.array_equal(codes.cpu().numpy()[pg, w, 0, sl], want_codes[t, w]), (t, w)
            assert np.array_equal(host(ranges)[pg, w, 0, sl], want_ranges[t, w].astype(np.float64), equal_nan=True), (t, w)
            with np.errstate(all="ignore"):
                v = torch.from_numpy(ref.values(want_codes[t, w], want_ranges[t, w]).astype(np.float32)).bfloat16()
            assert np.array_equal(got[t, w], v.double().numpy(), equal_nan=True), (t, w)
    assert np.isnan(got[5, 0]).all() and np.isnan(got[6, 0]).all() and np.isnan(got[4, 0]).all()


def test_no_sequence_and_counts_out_of_range(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    c = Case(4, 6, 4, 2, 64, 64, False, seed=8)
    c.start[1], c.count[:] = -1, (-5, 6, 2 ** 31 - 1, -2 ** 31)
    c.device()
    pool = torch.full((c.pages, 2, c.Hkv, c.page, c.D), 9.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((c.pages, 2, c.Hkv, c.page, c.D // 2), 9, dtype=torch.uint8, device="cuda")
    ranges = torch.full((c.pages, 2, c.Hkv, c.page, 2), 9.0, dtype=torch.bfloat16, device="cuda")
    rows = torch.full((c.B, c.T, 2 * c.Hkv * c.D), 9.0, dtype=torch.bfloat16, device="cuda")
    out, out4 = torch.full_like(c.qkv, 9.0), torch.full_like(c.qkv, 9.0)
    a = dict(turns=c.turns, start=c.d["start"], count=c.d["count"])
    binding.paged_append(c.qkv, pool, c.d["table"], c.H, out=out, **a)
    binding.paged_append4(c.qkv, codes, ranges, c.d["table"], c.H, out=out4, **a)
    binding.paged_load4(codes, ranges, c.d["table"], rows, start=c.d["start"], count=c.d["count"])
    binding.status()
    assert torch.equal(out, out4)
    for t in (out, rows):
        h = host(t)
        assert (h[[0, 1, 3]] == 9.0).all() and not (h[2] == 9.0).all()
    mine = set(c.table[2].tolist())
    for pg in range(c.pages):
        if pg not in mine:
            assert (host(pool)[pg] == 9.0).all() and (codes[pg] == 9).all() and (host(ranges)[pg] == 9.0).all()


def test_bad_pages_and_rows_past_the_table(gpt_lib):
    # neither read nor written, reported; the other sequences are right
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (-1, 10 ** 9, "far"):
        c = Case(3, 20, 4, 2, 64, 64, False, seed=9, counts=False)
        if bad == "far":
            c.start[1] = c.table.shape[1] * c.page - 10
        else:
            c.table[1] = bad
        c.device()
        pool = torch.zeros(c.pages, 2, c.Hkv, c.page, c.D, dtype=torch.bfloat16, device="cuda")
        codes = torch.zeros(c.pages, 2, c.Hkv, c.page, c.D // 2, dtype=torch.uint8, device="cuda")
        ranges = torch.zeros(c.pages, 2, c.Hkv, c.page, 2, dtype=torch.bfloat16, device="cuda")
        rows = torch.zeros(c.B, c.T, 2 * c.Hkv * c.D, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(c.qkv)
        a = dict(turns=c.turns, start=c.d["start"])
        for call in (lambda: binding.paged_append(c.qkv, pool, c.d["table"], c.H, out=out, **a),
                     lambda: binding.paged_append4(c.qkv, codes, ranges, c.d["table"], c.H, **a),
                     lambda: binding.paged_load4(codes, ranges, c.d["table"], rows, start=c.d["start"])):
            call()
            with pytest.raises(binding.GptError) as e:
                binding.status()
            assert e.value.code == binding.GPT_EPAGE
            binding.status()
        o, p, r = host(out).reshape(c.x.shape), host(pool), host(rows).reshape(c.B, c.T, 2 * c.Hkv, c.D)
        cd, rg = ref.quantise(o[:, :, c.H:].astype(np.float32))
        for b in (0, 2):
            for t in range(c.T):
                rr = c.start[b] + t
                pg, sl = c.table[b, rr // c.page], rr % c.page
                assert np.array_equal(p[pg, 0, :, sl], o[b, t, c.H: c.H + c.Hkv])
                assert np.array_equal(r[b, t], torch.from_numpy(ref.values(cd[b, t], rg[b, t]).astype(np.float32)).bfloat16().double().numpy())


def test_captured_and_replayed(gpt_lib):
    # a graph reads what the lengths are when it runs
    from decoder_only_transformer_gpt_gb300 import binding
    c = Case(3, 1, 12, 12, 64, 64, False, seed=10, counts=False).device()
    pool = torch.zeros(c.pages, 2, c.Hkv, c.page, c.D, dtype=torch.bfloat16, device="cuda")
    out, start = torch.zeros_like(c.qkv), torch.zeros(3, dtype=torch.int32, device="cuda")
    args = dict(turns=c.turns, start=start, out=out)
    binding.paged_append(c.qkv, pool, c.d["table"], c.H, **args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.paged_append(c.qkv, pool, c.d["table"], c.H, **args)
        start += 1
    start.zero_()
    for i in range(20):
        g.replay()
    torch.cuda.synchronize()
    binding.status()
    p = host(pool)
    for i in range(20):
        want, mag = c.want(np.full(3, i))
        for b in range(3):
            assert close(p[c.table[b, i // 16], 0, :, i % 16], want[b, 0, c.H: c.H + c.Hkv], mag[b, 0, c.H: c.H + c.Hkv])
