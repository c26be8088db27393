"""Attention over the 4-bit cache where rows differ: in size, in the bits that their weights need, in whether their page exists.
Tolerances: paged4_ref.attend_rows' bounds and one rounding of y to bf16."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import paged4_ref as ref  # noqa: E402
from gpu_util import dev_bf16, dev_i32, host, rand_bf16  # noqa: E402
from paged_ref import seen_rows  # noqa: E402
from serving_ref import quantise, values  # noqa: E402

FORMS = [None, 1024, 4096, 65536]                 # room of the page table, by which the form is chosen
HEADS = [(3, 3, 64), (4, 2, 32), (8, 2, 64), (6, 1, 64), (8, 1, 32), (12, 1, 64), (16, 1, 32), (20, 1, 64)]


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().float().numpy()


class Cache:
    """Sequences whose rows are given: keys and values [B][rows, Hkv, D]."""

    def __init__(self, q, keys, vals, H, page, rows=None, window=0, sinks=0, seed=0):
        B, (n, Hkv, D) = len(keys), keys[0].shape
        rng = np.random.default_rng(seed)
        self.H, self.D, self.window, self.sinks, self.page = H, D, window, sinks, page
        self.lens = np.array([len(k) for k in keys])
        used = -(-int(self.lens.max()) // page)
        self.table = np.full((B, max(used, (rows or 0) // page)), 10 ** 9, np.int32)
        self.table[:, :used] = rng.permutation(B * used).reshape(B, used)
        pool = np.zeros((B * used, 2, Hkv, page, D), np.float32)
        for b in range(B):
            for w, x in enumerate((keys[b], vals[b])):
                for r in range(self.lens[b]):
                    pool[self.table[b, r // page], w, :, r % page] = bf16(x[r])
        self.codes, self.ranges = quantise(pool)
        self.ranges = bf16(self.ranges)
        self.x = np.zeros((B, (H + 2 * Hkv) * D), np.float32)
        self.x[:, : H * D] = bf16(np.asarray(q).reshape(B, H * D))

    def device(self):
        B = len(self.lens)
        self.d = [dev_bf16(self.x), torch.from_numpy(self.codes).cuda(), dev_bf16(self.ranges), dev_i32(self.table),
                  dev_i32(self.lens)]
        self.y = torch.full((B, self.H * self.D), 77.0, dtype=torch.bfloat16, device="cuda")
        self.lse2 = torch.full((B, self.H), 77.0, device="cuda")
        return self

    def call(self):
        from decoder_only_transformer_gpt_gb300 import binding
        binding.paged_attention4(*self.d, self.y, self.H, lse2=self.lse2, window=self.window, sinks=self.sinks)
        return self

    def seen(self, without=()):
        """without: (sequence, page of its table) pairs that are left out."""
        out = []
        for b, n in enumerate(self.lens):
            rows = [r for r in seen_rows(int(n), self.window, self.sinks) if (b, r // self.page) not in without]
            out.append(rows if n >= 0 else None)
        return out

    def check(self, without=()):
        y, lse2, ey, el = ref.attend_rows(self.x, self.codes, self.ranges, self.table, self.seen(without), self.H)
        bad = ref.outside(host(self.y), y, ey)
        assert not bad.any(), (np.abs(host(self.y) - y)[bad].max(), np.abs(y).max())
        assert (np.abs(host(self.lse2) - lse2) <= el).all()


def ordinary(H, Hkv, D, n, seed):
    """Queries that are all positive, and rows of ordinary size."""
    rng = np.random.default_rng(seed)
    return np.abs(rand_bf16(rng, (1, H, D), 0.2)) + 0.05, rand_bf16(rng, (n, Hkv, D)), rand_bf16(rng, (n, Hkv, D))


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("H,Hkv,D", HEADS)
@pytest.mark.parametrize("size", [28, 36, 100])
def test_a_large_row_that_has_no_weight(gpt_lib, rows, H, Hkv, D, size):
    # its score is some thousand below the others': first, in the middle, last
    from decoder_only_transformer_gpt_gb300 import binding
    q, k, u = ordinary(H, Hkv, D, 333, 1)
    for at in (0, 150, 332):
        k1, u1 = k.copy(), u.copy()
        k1[at] = -5000.0
        u1[at] *= 2.0 ** size
        Cache(q, [k1], [u1], H, 16, rows).device().call().check()
    k1, u1 = k.copy(), u.copy()                     # and a third of the rows
    k1[::3], u1[::3] = -5000.0, u[::3] * 2.0 ** size
    Cache(q, [k1], [u1], H, 16, rows).device().call().check()
    binding.status()


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("H,Hkv,D", [(4, 2, 64), (8, 1, 64), (12, 1, 32), (16, 1, 64)])
@pytest.mark.parametrize("size", [20, 60])
def test_a_large_row_that_only_some_heads_see(gpt_lib, rows, H, Hkv, D, size):
    # every other head of a key head has the opposite sign, so that it looks at nothing else
    q, k, u = ordinary(H, Hkv, D, 300, 2)
    q[0, 1::2] *= -1.0
    k[170] = -5000.0
    u[170] *= 2.0 ** size
    Cache(q, [k], [u], H, 16, rows).device().call().check()


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("H,Hkv,D", HEADS)
@pytest.mark.parametrize("down", [False, True])
def test_sizes_that_change_with_the_scores(gpt_lib, rows, H, Hkv, D, down):
    # later rows have larger scores, by 1 in 4 rows and by 40 in the end, and smaller (or larger) values, 2^60 in all
    q, k, u = ordinary(H, Hkv, D, 400, 3)
    r = np.arange(400.0)[:, None, None]
    k = k * 0.01 + (r // 4) * 0.1 + 20.0 * (r > 380)
    u = u * 2.0 ** ((-1 if down else 1) * (r * 60 / 400))
    Cache(q, [k], [u], H, 16, rows).device().call().check()


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("H,Hkv,D", HEADS)
def test_weights_keep_twenty_bits(gpt_lib, rows, H, Hkv, D):
    # few rows with scores of one value of the query, so that scores and sums lose little; some outputs are sums that cancel
    for seed in range(4):
        c = few_rows(H, Hkv, D, rows, seed)
        c.device().call().check()


def few_rows(H, Hkv, D, rows, seed):
    rng = np.random.default_rng(100 + seed)
    q = np.zeros((1, H, D))
    q[0, np.arange(H), rng.integers(0, D, H)] = 0.5
    k, u = rand_bf16(rng, (3, Hkv, D)), rand_bf16(rng, (3, Hkv, D))
    k[:, :, :] = np.clip(k, -1.0, 1.0)
    return Cache(q, [k], [u], H, 8, rows, seed=seed)


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("H,Hkv,D,page", [(3, 3, 64, 16), (8, 2, 32, 8), (12, 1, 64, 64), (4, 2, 64, 128)])
@pytest.mark.parametrize("bad", [-1, -2, 10 ** 9])
def test_rows_of_a_bad_page_are_left_out(gpt_lib, rows, H, Hkv, D, page, bad):
    # reported, and nothing else takes their place: not the rows of another sequence either
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(7)
    lens = [300, 290, 280]
    k, u = ([rand_bf16(rng, (n, Hkv, D)) * 10.0 ** b for b, n in enumerate(lens)] for _ in range(2))
    q = rand_bf16(rng, (3, H, D), 0.3)
    without = {(0, 1), (1, 0), (1, 290 // page), (2, 100 // page)}
    c = Cache(q, k, u, H, page, rows).device()
    c.call()
    for b, i in without:
        c.d[3][b, i] = bad
    out = []
    for _ in range(3):
        c.y.fill_(7.0)
        c.call()
        with pytest.raises(binding.GptError) as e:
            binding.status()
        assert e.value.code == binding.GPT_EPAGE
        c.check(without)
        out.append(c.y.clone())
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("H,Hkv,D,page", [(3, 3, 64, 16), (8, 2, 32, 8), (12, 1, 64, 16), (4, 2, 64, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 0), (50, 3), (200, 20)])
def test_pages_out_of_sight_need_not_exist(gpt_lib, rows, H, Hkv, D, page, window, sinks):
    # a caller that gives pages behind the window back leaves no numbers of them in the table
    from decoder_only_transformer_gpt_gb300 import binding
    rng = np.random.default_rng(8)
    for n in (500, 511, 513, 449):
        k, u = (rand_bf16(rng, (n, Hkv, D)) for _ in range(2))
        c = Cache(rand_bf16(rng, (1, H, D)), [k], [u], H, page, rows, window, sinks).device()
        kept = {r // page for r in c.seen()[0]}
        for i in range(c.table.shape[1]):
            if i not in kept:
                c.d[3][0, i] = -1 if i % 2 else 10 ** 9
        c.call()
        binding.status()
        c.check()


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("H,Hkv,D", HEADS)
def test_a_row_seen_alone_comes_out_as_it_is(gpt_lib, rows, H, Hkv, D):
    # its weight is 1 and nothing is added: the value in fp32, rounded to bf16
    rng = np.random.default_rng(9)
    for n, window in ((1, 0), (200, 1), (65, 1)):
        k, u = (rand_bf16(rng, (n, Hkv, D)) * 2.0 for _ in range(2))
        c = Cache(rand_bf16(rng, (1, H, D)), [k], [u], H, 16, rows, window).device().call()
        pg, slot = c.table[0, (n - 1) // 16], (n - 1) % 16
        held = values(c.codes[pg, 1, :, slot], c.ranges[pg, 1, :, slot]).repeat(H // Hkv, 0)
        assert torch.equal(c.y.cpu().view(H, D), torch.from_numpy(held.astype(np.float32)).bfloat16())
