"""The paged key/value cache on the GPU against numpy float64 (tests/paged_ref.py).

Inputs are seeded and bf16-exact. Stores and evictions copy: their results are equal bit for bit, and so is every
place that a call does not own. Tolerances of the attention follow its arithmetic (half a step: bf16 2^-8, fp32 2^-24):
  * a score s = q.k / sqrt(D) in fp32: |ds| <= (D + 2) 2^-24 |q|.|k| / sqrt(D); its exponential in base 2 adds 2^-24 |s|
    log2(e) for the rounded argument and 2^-22 for ex2.approx: relative error of a weight a_r, normaliser included,
    at most twice d = (D + 2) 2^-24 max |q|.|k| / sqrt(D) (1 + log2 e) + 2^-21, plus n 2^-24 for the sums over n rows
  * the probabilities are rounded to bf16 for the product with the values: 2^-8 sum a |u|, and the output: 2^-8 |y|
  * lse2 moves by d log2(e) and the fp32 rounding of its parts, 2^-22 (1 + |lse2|)
  * a row's summed weight: twice d times the sum, and one fp32 addition per query head, 2^-24 of the total each
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged_ref  # noqa: E402
from gpu_util import dev_bf16, dev_f32, dev_i32, host, rand_bf16  # noqa: E402

LOG2E = 1.0 / math.log(2.0)


class Case:
    """A cache whose pages lie shuffled, with NaN wherever no seen row is."""

    def __init__(self, H, Hkv, D, page, lens, window=0, sinks=0, weights=True, seed=0, scale=1.0, spare=2):
        rng = np.random.default_rng(seed)
        self.H, self.Hkv, self.D, self.page, self.window, self.sinks = H, Hkv, D, page, window, sinks
        self.lens = np.array(lens, np.int32)
        B = len(lens)
        max_pages = max(1, (max(lens) + page) // page)
        n = B * max_pages + spare
        self.table = rng.permutation(n)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
        self.qkv = rand_bf16(rng, (B, (H + 2 * Hkv) * D), scale)
        self.pool = np.full((n, 2, Hkv, page, D), np.nan, np.float32)
        self.weight = rng.random((n, Hkv, page)).astype(np.float32) if weights else None
        for b, ln in enumerate(lens):
            for r in paged_ref.seen_rows(ln + 1, window, sinks)[:-1] if ln >= 0 else ():
                p, s = paged_ref.place(self.table[b], page, r)
                self.pool[p, :, :, s] = rand_bf16(rng, (2, Hkv, D))

    def device(self):
        self.d_qkv, self.d_pool, self.d_table, self.d_lens = dev_bf16(self.qkv), dev_bf16(self.pool), \
            dev_i32(self.table), dev_i32(self.lens)
        self.d_weight = None if self.weight is None else dev_f32(self.weight)
        B = len(self.lens)
        self.d_y = torch.full((B, self.H * self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.d_lse2 = torch.full((B, self.H), 7.0, dtype=torch.float32, device="cuda")
        return self

    def call(self, **k):
        from decoder_only_transformer_gpt_gb300 import binding
        binding.paged_attention(self.d_qkv, self.d_pool, self.d_table, self.d_lens, self.d_y, self.H, lse2=self.d_lse2,
                                weight=self.d_weight, window=self.window, sinks=self.sinks, **k)

    def expected(self):
        w = None if self.weight is None else self.weight.astype(np.float64)
        return paged_ref.decode(self.qkv.astype(np.float64), self.pool.astype(np.float64), w, self.table, self.lens, self.H,
                                self.window, self.sinks)

    def check(self, skip=()):
        H, Hkv, D, page, G = self.H, self.Hkv, self.D, self.page, self.H // self.Hkv
        y, lse2, pool, weight = self.expected()
        gy, gl, gp = host(self.d_y), host(self.d_lse2), host(self.d_pool)
        gw = None if weight is None else host(self.d_weight)
        np.testing.assert_array_equal(gp, pool)                          # NaN places included
        wtol = None if weight is None else np.zeros_like(weight)
        rows = self.qkv.astype(np.float64).reshape(len(self.lens), H + 2 * Hkv, D)
        for b, ln in enumerate(self.lens):
            if b in skip:
                continue
            if ln < 0:
                assert np.all(gy[b] == 7.0) and np.all(gl[b] == 7.0), f"row {b} is no sequence"
                continue
            where = [paged_ref.place(self.table[b], page, r) for r in paged_ref.seen_rows(ln + 1, self.window, self.sinks)]
            n = len(where)
            for j in range(Hkv):
                k = np.stack([pool[p, 0, j, s] for p, s in where])
                u = np.stack([pool[p, 1, j, s] for p, s in where])
                for h in range(j * G, (j + 1) * G):
                    q = rows[b, h]
                    _, _, a = paged_ref.attend(q, k, u)
                    d = (D + 2) * 2.0 ** -24 * (np.abs(k) @ np.abs(q)).max() / math.sqrt(D) * (1 + LOG2E) + 2.0 ** -21
                    rel = 2 * d + n * 2.0 ** -24
                    c = slice(h * D, (h + 1) * D)
                    tol = (2.0 ** -8 + rel) * (a @ np.abs(u)) + 2.0 ** -8 * np.abs(y[b, c]) * (1 + 2.0 ** -7)
                    err = np.abs(gy[b, c] - y[b, c])
                    assert np.all(err <= tol), (b, h, err.max(), tol[err.argmax()])
                    tl = rel * LOG2E + 2.0 ** -22 * (1 + abs(lse2[b, h]))
                    assert abs(gl[b, h] - lse2[b, h]) <= tl, (b, h, gl[b, h], lse2[b, h])
                    if wtol is not None:
                        for (p, s), x in zip(where, a):
                            wtol[p, j, s] += rel * x + 2.0 ** -24 * (G + self.weight[p, j, s])
        if weight is not None:
            bad = np.abs(gw - weight) > wtol
            assert not bad.any(), (np.argwhere(bad)[0], np.abs(gw - weight)[bad].max())


HEADS = [(4, 4, 32), (12, 12, 64), (8, 2, 64), (5, 1, 64), (17, 1, 32), (40, 2, 64), (16, 1, 64)]


@pytest.mark.parametrize("H,Hkv,D", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 3)])
def test_attention_lengths(gpt_lib, H, Hkv, D, window, sinks):
    # nothing cached, one row, around a page's and a chunk's end, and longer; one row of the batch is no sequence
    c = Case(H, Hkv, D, 16, [0, 1, 15, 16, -1, 31, 32, 33, 200, 63, 64, 129], window, sinks, seed=H + window).device()
    c.call()
    from decoder_only_transformer_gpt_gb300 import binding
    binding.status()
    c.check()


@pytest.mark.parametrize("page", [8, 32, 64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5), (7, 300), (300, 1000), (1, 1)])
def test_attention_pages(gpt_lib, page, window, sinks):
    c = Case(6, 3, 64, page, [page - 1, page, 3 * page, 777, 5, 300], window, sinks, seed=page + sinks).device()
    c.call()
    c.check()


@pytest.mark.parametrize("D", [32, 64])
def test_attention_without_weights_or_lse(gpt_lib, D):
    from decoder_only_transformer_gpt_gb300 import binding
    c = Case(4, 2, D, 16, [70, 3], weights=False, seed=D).device()
    binding.paged_attention(c.d_qkv, c.d_pool, c.d_table, c.d_lens, c.d_y, 4)
    binding.status()
    assert torch.all(c.d_lse2 == 7.0)
    y = c.d_y.clone()
    c.call()                                                             # the same call again: same place, same result
    c.check()
    assert torch.equal(y, c.d_y)


def test_attention_long_and_ragged(gpt_lib):
    # one long sequence among short ones: its rows are split over many parts and joined
    c = Case(4, 2, 64, 64, [20000, 0, 17, 3000, -1, 900], seed=3).device()
    c.call()
    c.check()


def test_attention_peaked_scores(gpt_lib):
    # scores of several hundred: one row takes nearly all the weight, the rest underflow
    c = Case(4, 4, 64, 16, [500, 40], seed=4, scale=24.0).device()
    c.call()
    c.check()


def test_attention_many_sequences(gpt_lib):
    rng = np.random.default_rng(0)
    c = Case(2, 1, 32, 8, rng.integers(-1, 60, 700).tolist(), seed=5).device()
    c.call()
    c.check()


def test_attention_repeats_bit_for_bit(gpt_lib):
    c = Case(12, 4, 64, 16, [900, 1500, 20, 333], seed=6, weights=False).device()
    c.call()
    y, lse2 = c.d_y.clone(), c.d_lse2.clone()
    for _ in range(3):
        c.d_y.zero_()
        c.call()
        assert torch.equal(y, c.d_y) and torch.equal(lse2, c.d_lse2)


def test_attention_shared_pages(gpt_lib):
    # two sequences with a common start: its pages stand in both tables, and its rows take both sequences' weights
    c = Case(4, 2, 64, 16, [40, 40, 25], seed=7)
    c.table[1, :2] = c.table[0, :2]
    c.device()
    c.call()
    c.check()


def test_attention_beyond_32_bit_offsets(gpt_lib):
    # a pool of more than 2^31 elements, its last pages in use
    from decoder_only_transformer_gpt_gb300 import binding
    c = Case(8, 8, 64, 256, [700, 300], seed=8, spare=0)
    n, far = c.pool.shape[0], 8300
    big = torch.empty(far, 2, 8, 256, 64, dtype=torch.bfloat16, device="cuda")
    bw = torch.zeros(far, 8, 256, dtype=torch.float32, device="cuda")
    assert big.numel() > 2 ** 31
    c.device()
    big[far - n:] = c.d_pool
    bw[far - n:] = c.d_weight
    binding.paged_attention(c.d_qkv, big, c.d_table + (far - n), c.d_lens, c.d_y, 8, lse2=c.d_lse2, weight=bw)
    c.d_pool, c.d_weight = big[far - n:].contiguous(), bw[far - n:].contiguous()
    c.check()
    # and through a store and an eviction
    qkv = dev_bf16(rand_bf16(np.random.default_rng(1), (1, 600, 24 * 64)))
    table = dev_i32(np.array([[far - 1, far - 3, far - 2]]))
    binding.paged_store(qkv, big, table, 8, weight=bw)
    k = torch.cat([big[p, 0] for p in (far - 1, far - 3, far - 2)], 1)[:, :600].permute(1, 0, 2).reshape(600, -1)
    assert torch.equal(k, qkv[0, :, 8 * 64:16 * 64])
    lens, new, kept = dev_i32(np.array([600])), dev_i32(np.array([0])), torch.empty(1, 8, 100, dtype=torch.int32, device="cuda")
    bw[far - 1, :, 11] = 2.0
    binding.paged_evict(big, bw, table, lens, dev_i32(np.array([[far - 4]])), new, kept, 100, 10, 20)
    binding.status()
    want = torch.tensor(list(range(80)) + list(range(580, 600)), dtype=torch.int32, device="cuda")
    assert torch.equal(kept, want.expand(1, 8, 100))
    assert torch.equal(big[far - 4, 0, :, :80], big[far - 1, 0, :, :80])
    assert torch.equal(big[far - 4, 1, :, 80:100], big[far - 2, 1, :, 68:88])


def test_attention_on_another_stream_and_in_a_graph(gpt_lib):
    c = Case(8, 2, 64, 16, [333, 64, 0], seed=9, weights=False).device()
    c.call()
    torch.cuda.synchronize()
    want = c.d_y.clone()
    s = torch.cuda.Stream()
    c.d_y.zero_()
    torch.cuda.synchronize()
    c.call(stream=s)
    s.synchronize()
    assert torch.equal(c.d_y, want)
    # captured; replayed with other lengths and tokens in the same arrays
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.d_y, want)
    d = Case(8, 2, 64, 16, [100, 200, 300], seed=10, weights=False)
    d.table, d.lens = c.table[:, :], np.array([100, 200, 300], np.int32)
    e = Case(8, 2, 64, 16, [333, 333, 333], seed=11, weights=False)      # every row filled
    d.pool, d.table = e.pool, e.table
    c.d_qkv.copy_(dev_bf16(d.qkv))
    c.d_pool.copy_(dev_bf16(d.pool))
    c.d_table.copy_(dev_i32(d.table))
    c.d_lens.copy_(dev_i32(d.lens))
    g.replay()
    torch.cuda.synchronize()
    d.d_y, d.d_lse2, d.d_pool, d.d_weight = c.d_y, c.d_lse2, c.d_pool, None
    d.check()


def test_two_calls_at_once(gpt_lib):
    # two streams, two caches: nothing is shared between calls
    a, b = Case(12, 12, 64, 16, [700] * 8, seed=12).device(), Case(12, 12, 64, 16, [650] * 8, seed=13).device()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(1):
        a.call(stream=s)
        b.call(stream=t)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_bad_pages_and_lengths_are_reported(gpt_lib):
    # a page number past the pool, a negative one and a length past the table: nothing out of bounds is touched, the
    # status says so once, and the sequences without such a page are right
    from decoder_only_transformer_gpt_gb300 import binding
    for what in ("past", "negative", "length"):
        c = Case(4, 2, 64, 16, [100, 50, 60], seed=14, weights=False).device()
        if what == "length":
            c.d_lens[0] = c.table.shape[1] * 16
        else:
            c.d_table[0, 2] = 10 ** 9 if what == "past" else -1
        c.call()
        with pytest.raises(binding.GptError) as e:
            binding.status()
        assert e.value.code == binding.GPT_EPAGE
        binding.status()
        c.d_pool[c.table[0]] = dev_bf16(c.expected()[2])[c.table[0]]
        c.check(skip=(0,))


@pytest.mark.parametrize("B,T,H,Hkv,D,page", [(1, 1, 1, 1, 32, 8), (3, 77, 4, 2, 64, 16), (2, 300, 12, 12, 64, 64),
                                               (5, 33, 6, 1, 32, 256)])
@pytest.mark.parametrize("ragged", [False, True])
def test_store(gpt_lib, B, T, H, Hkv, D, page, ragged):
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(T + page)
    start = rng.integers(0, 2 * page, B).astype(np.int32) if ragged else None
    count = rng.integers(-1, T + 2, B).astype(np.int32) if ragged else None
    max_pages = (T + 2 * page) // page + 1
    n = B * max_pages + 1
    table = rng.permutation(n)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    qkv = rand_bf16(rng, (B, T, (H + 2 * Hkv) * D))
    pool = rand_bf16(rng, (n, 2, Hkv, page, D))
    weight = rng.random((n, Hkv, page)).astype(np.float32)
    d_pool, d_weight = dev_bf16(pool), dev_f32(weight)
    d = [None if x is None else dev_i32(x) for x in (start, count)]
    binding.paged_store(dev_bf16(qkv), d_pool, dev_i32(table), H, start=d[0], count=d[1], weight=d_weight)
    binding.status()
    for b in range(B):
        for t in range(min(T, T if count is None else int(count[b]))):
            p, s = paged_ref.place(table[b], page, t + (0 if start is None else int(start[b])))
            pool[p, 0, :, s] = qkv[b, t, H * D:(H + Hkv) * D].reshape(Hkv, D)
            pool[p, 1, :, s] = qkv[b, t, (H + Hkv) * D:].reshape(Hkv, D)
            weight[p, :, s] = 0.0
    np.testing.assert_array_equal(host(d_pool), pool)
    np.testing.assert_array_equal(host(d_weight), weight)
    d_pool2 = dev_bf16(pool)
    binding.paged_store(dev_bf16(qkv), d_pool2, dev_i32(table), H, start=d[0], count=d[1])      # no weights
    assert torch.equal(d_pool2, d_pool)


def test_store_reports_rows_past_the_table(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    pool = torch.zeros(3, 2, 1, 8, 32, dtype=torch.bfloat16, device="cuda")
    qkv = torch.ones(1, 20, 3 * 32, dtype=torch.bfloat16, device="cuda")
    for start, table in ((0, [[1, 2]]), (-3, [[1, 2]]), (2147483647, [[1, 2]]), (0, [[1, 5]])):
        pool.zero_()
        binding.paged_store(qkv, pool, dev_i32(np.array(table)), 1, start=dev_i32(np.array([start])))
        with pytest.raises(binding.GptError) as e:
            binding.status()
        assert e.value.code == binding.GPT_EPAGE
        assert torch.all(pool[0] == 0)
        rows = {0: 16, -3: 16, 2147483647: 0}[start] if table == [[1, 2]] else 8
        assert int((pool[1:, 0, 0, :, 0] == 1).sum()) == rows


def _evict_case(seed, lens, Hkv, D, page, budget, ties=False, nan=False):
    rng = np.random.default_rng(seed)
    B, max_pages, more = len(lens), (max(max(lens), 1) + page - 1) // page, (budget + page - 1) // page
    n = B * (max_pages + more) + 1
    perm = rng.permutation(n)
    table = perm[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    dst = perm[B * max_pages:B * (max_pages + more)].reshape(B, more).astype(np.int32)
    pool = rand_bf16(rng, (n, 2, Hkv, page, D))
    weight = np.exp(rng.standard_normal((n, Hkv, page)) * 2).astype(np.float32)
    if ties:
        weight = np.floor(weight).astype(np.float32) * np.where(rng.random(weight.shape) < 0.5, -1, 1).astype(np.float32)
    if nan:
        weight[rng.random(weight.shape) < 0.2] = np.nan
        weight[rng.random(weight.shape) < 0.1] = np.inf
        weight[rng.random(weight.shape) < 0.1] = -np.inf
    return pool, weight, table, np.array(lens, np.int32), dst


def _evict_run(pool, weight, table, lens, dst, budget, sinks, recent):
    from decoder_only_transformer_gpt_gb300 import binding
    Hkv = pool.shape[2]
    d_pool, d_weight, d_lens = dev_bf16(pool), dev_f32(weight), dev_i32(lens)
    new = torch.full((len(lens),), 99, dtype=torch.int32, device="cuda")
    kept = torch.full((len(lens), Hkv, budget), 99, dtype=torch.int32, device="cuda")
    binding.paged_evict(d_pool, d_weight, dev_i32(table), d_lens, dev_i32(dst), new, kept, budget, sinks, recent)
    binding.status()
    want = paged_ref.evict(pool.astype(np.float64), weight, table, lens, dst, budget, sinks, recent)
    np.testing.assert_array_equal(host(new), want[2])
    np.testing.assert_array_equal(host(kept), want[3])
    np.testing.assert_array_equal(host(d_weight), want[1])
    np.testing.assert_array_equal(host(d_pool), want[0])


@pytest.mark.parametrize("lens,Hkv,D,page,budget,sinks,recent", [
    ([1], 1, 32, 8, 1, 0, 0), ([2, 3, 9], 2, 64, 8, 2, 0, 1), ([0, -1, 5, 40], 2, 32, 8, 4, 4, 0),
    ([100, 64, 63, 65, 700], 3, 64, 16, 64, 4, 16), ([100, 200], 1, 64, 32, 40, 10, 30), ([513, 1025, 2000], 2, 64, 64, 600, 0, 0),
    ([5000], 1, 32, 256, 4999, 1, 1), ([60000, 100], 1, 32, 256, 700, 4, 64), ([230000], 1, 32, 256, 900, 4, 64), ([3000, 20], 12, 64, 16, 1024, 16, 512)])
@pytest.mark.parametrize("kind", ["plain", "ties", "nan"])
def test_evict(gpt_lib, lens, Hkv, D, page, budget, sinks, recent, kind):
    case = _evict_case(len(lens) + budget, lens, Hkv, D, page, budget, kind == "ties", kind == "nan")
    _evict_run(*case, budget, sinks, recent)                             # into other pages
    pool, weight, table, lens, _ = case
    _evict_run(pool, weight, table, lens, table if table.shape[1] * page >= budget else case[4], budget, sinks, recent)


@pytest.mark.parametrize("budget", [100, 1500])
def test_evict_in_place_into_a_shorter_table(gpt_lib, budget):
    pool, weight, table, lens, _ = _evict_case(3, [3000, 1600, 90], 4, 64, 16, budget)
    _evict_run(pool, weight, table, lens, np.ascontiguousarray(table[:, :(budget + 15) // 16]), budget, 4, 50)


def test_evict_all_equal_and_zero_weights(gpt_lib):
    pool, weight, table, lens, dst = _evict_case(4, [400, 700], 2, 64, 16, 128)
    weight[:] = 0.0
    weight[::2] = -0.0                                                   # equal to +0: the lowest rows stay
    _evict_run(pool, weight, table, lens, dst, 128, 2, 30)


def test_evict_reports_bad_pages(gpt_lib):
    from decoder_only_transformer_gpt_gb300 import binding
    pool, weight, table, lens, dst = _evict_case(5, [100, 100], 2, 64, 16, 32)
    for what in ("src", "dst", "length"):
        d_pool, t, q, ln = dev_bf16(pool), table.copy(), dst.copy(), lens.copy()
        if what == "src":
            t[0, 3] = pool.shape[0]
        elif what == "dst":
            q[0, 1] = -5
        else:
            ln[0] = 16 * table.shape[1] + 1
        new, kept = dev_i32(lens * 0), torch.empty(2, 2, 32, dtype=torch.int32, device="cuda")
        binding.paged_evict(d_pool, dev_f32(weight), dev_i32(t), dev_i32(ln), dev_i32(q), new, kept, 32, 2, 4)
        with pytest.raises(binding.GptError) as e:
            binding.status()
        assert e.value.code == binding.GPT_EPAGE
        want = paged_ref.evict(pool.astype(np.float64), weight, table, lens, dst, 32, 2, 4)
        np.testing.assert_array_equal(host(kept)[1], want[3][1])
        np.testing.assert_array_equal(host(d_pool)[dst[1]], want[0][dst[1]])
