"""Attention of one token per sequence over the paged cache in 4 bits, against serving_ref.attend4.

Tolerances: attend4's bounds of the arithmetic, and one rounding of y to bf16 (2^-8 of the value at most).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import serving_ref as ref  # noqa: E402
from gpu_util import dev_bf16, dev_f32, dev_i32, host, rand_bf16  # noqa: E402,F401


class Case:
    """A cache of sequences of the given lengths (-1: none) with max_pages pages each, in shuffled order."""

    def __init__(self, H, Hkv, D, page, lens, window=0, sinks=0, seed=0, rows=None, added=0, q_scale=1.5):
        rng = np.random.default_rng(seed)
        self.H, self.Hkv, self.D, self.page, self.window, self.sinks, self.added = H, Hkv, D, page, window, sinks, added
        self.lens = np.array(lens)
        B = len(lens)
        self.x = rand_bf16(rng, (B, (H + 2 * Hkv) * D), q_scale)
        used = max(1, -(-(max(max(lens), 0) + added) // page))
        width = used if rows is None else max(used, rows // page)
        n = B * used + 3
        self.table = np.full((B, width), 10 ** 9, np.int32)     # entries behind the sequences' pages are not used
        self.table[:, :used] = rng.permutation(n)[: B * used].reshape(B, used)
        self.codes, self.ranges = ref.quantise(rand_bf16(rng, (n, 2, Hkv, page, D)) + rand_bf16(rng, (n, 2, Hkv, 1, D)) * 0.5)
        self.ranges = torch.from_numpy(self.ranges).bfloat16().float().numpy()

    def device(self):
        B = len(self.lens)
        self.d_x, self.d_codes, self.d_ranges = dev_bf16(self.x), torch.from_numpy(self.codes).cuda(), dev_bf16(self.ranges)
        self.d_table, self.d_lens = dev_i32(self.table), dev_i32(self.lens)
        self.d_y = torch.full((B, self.H * self.D), 77.0, dtype=torch.bfloat16, device="cuda")
        self.d_lse2 = torch.full((B, self.H), 77.0, dtype=torch.float32, device="cuda")
        return self

    def call(self, lse2=True):
        from decoder_only_transformer_gpt_gb300 import binding
        binding.paged_attention4(self.d_x, self.d_codes, self.d_ranges, self.d_table, self.d_lens, self.d_y, self.H,
                                 lse2=self.d_lse2 if lse2 else None, window=self.window, sinks=self.sinks, added=self.added)

    def check(self, skip=()):
        y, lse2, ey, el = ref.attend4(self.x, self.codes, self.ranges, self.table, self.lens, self.H, self.window, self.sinks,
                                      self.added)
        gy, gl = host(self.d_y), host(self.d_lse2)
        for b in range(len(self.lens)):
            if b in skip:
                continue
            if self.lens[b] < 0:
                assert (gy[b] == 77.0).all() and (gl[b] == 77.0).all()
                continue
            if self.lens[b] + self.added == 0:
                assert (gy[b] == 0.0).all() and (gl[b] == -np.inf).all()
                continue
            assert (np.abs(gy[b] - y[b]) <= 2.0 ** -8 * np.abs(y[b]) + 1.01 * ey[b]).all(), (b, np.abs(gy[b] - y[b]).max())
            assert (np.abs(gl[b] - lse2[b]) <= el[b]).all(), (b, np.abs(gl[b] - lse2[b]).max(), el[b].min())

    def run(self):
        from decoder_only_transformer_gpt_gb300 import binding
        self.device().call()
        binding.status()
        self.check()
        return self


FORMS = [None, 1024, 4096, 16384, 65536]          # room of the page table, by which the form is chosen


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("H,Hkv,D,page", [(4, 4, 64, 16), (8, 1, 32, 8), (12, 1, 64, 64), (16, 1, 32, 16), (9, 3, 64, 128),
                                          (40, 2, 64, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (33, 2), (500, 7)])
def test_lengths_heads_and_windows(gpt_lib, rows, H, Hkv, D, page, window, sinks):
    for lens in ([1], [0], [31, 32, 33, 64], [-1, 255, 256, 257, 0], [600, -1, 2]):
        Case(H, Hkv, D, page, lens, window, sinks, seed=sum(lens), rows=rows).run()


@pytest.mark.parametrize("rows", [2047, 2048, 2049, 4095, 4096, 4097, 9000, 16384, 16385])
def test_full_tables(gpt_lib, rows):
    Case(2, 2, 64, 8, [rows], seed=rows).run()
    Case(4, 2, 32, 64, [rows, 5], seed=rows).run()
    Case(3, 1, 64, 256, [rows - 1, 0], seed=rows, added=1).run()


@pytest.mark.parametrize("B", [1, 30, 200])
@pytest.mark.parametrize("rows", [None, 65536])
def test_batches(gpt_lib, B, rows):
    rng = np.random.default_rng(B)
    Case(2, 2, 32, 8, rng.integers(-1, 300, B).tolist(), seed=B, rows=rows).run()
    Case(12, 3, 64, 16, rng.integers(-1, 90, B).tolist(), seed=B, rows=rows, window=40, sinks=3).run()


def test_more_sequences_than_threads(gpt_lib):
    rng = np.random.default_rng(5)
    Case(1, 1, 32, 8, rng.integers(-1, 20, 1500).tolist(), seed=5, rows=65536 // 8).run()
    Case(1, 1, 64, 8, ([5, -1, 0, 17] * 2048), seed=6).run()


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("scale", [0.0, 30.0])
def test_flat_and_steep_scores(gpt_lib, rows, scale):
    # equal weights for every row; scores hundreds apart
    Case(4, 2, 64, 16, [700, 40], seed=11, rows=rows, q_scale=scale).run()


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_a_nan_in_sight_shows_and_out_of_sight_does_not(gpt_lib, rows, window, sinks):
    from decoder_only_transformer_gpt_gb300 import binding
    for which in (0, 1):
        c = Case(6, 2, 64, 16, [400, 90], window, sinks, seed=3, rows=rows)
        c.ranges[c.table[0, 380 // 16], which, 1, 380 % 16] = np.nan
        c.device().call()
        binding.status()
        y = host(c.d_y).reshape(2, 6, 64)
        assert np.isnan(y[0, 3:]).all() and np.isfinite(y[0, :3]).all() and np.isfinite(y[1]).all()
    # rows behind the last, and between the sinks and the window, hold what they like
    c = Case(6, 2, 64, 16, [391, 90], window, sinks, seed=4, rows=rows)
    c.ranges[c.table[0, 391 // 16], :, :, 391 % 16:] = np.nan
    if window:
        c.ranges[c.table[0, 10], :] = np.inf
    c.device().call()
    binding.status()
    c.check()


@pytest.mark.parametrize("rows", FORMS)
def test_bad_pages_and_lengths(gpt_lib, rows):
    # rows of a page outside the pool are left out and reported; so is a length past the table; the others are right
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (-1, 10 ** 9, "long", "added"):
        c = Case(4, 2, 64, 16, [100, 50], seed=14, rows=rows).device()
        if bad == "long":
            c.d_lens[0] = c.table.shape[1] * 16 + 1
        elif bad == "added":
            c.added = 1
            c.table = c.table[:, : -(-101 // 16)]
            c.d_table = dev_i32(c.table)
            c.d_lens[0] = c.table.shape[1] * 16
        else:
            c.d_table[0, 2] = bad
        c.call()
        with pytest.raises(binding.GptError) as e:
            binding.status()
        assert e.value.code == binding.GPT_EPAGE
        binding.status()
        c.check(skip=(0,))


@pytest.mark.parametrize("rows", FORMS)
def test_one_result_bit_for_bit_without_lse2_and_in_a_graph(gpt_lib, rows):
    c = Case(8, 2, 64, 16, [900, 20, 333], seed=6, rows=rows).device()
    c.call()
    y, lse2 = c.d_y.clone(), c.d_lse2.clone()
    c.device().call(lse2=False)
    assert torch.equal(y, c.d_y) and (c.d_lse2 == 77.0).all()
    c.device()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    for _ in range(3):
        c.d_y.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, c.d_y) and torch.equal(lse2, c.d_lse2)
    # other lengths in the same graph
    c.lens = np.array([5, 640, -1])
    c.table[1, :] = c.table[0, :]                    # (sequences may share pages)
    c.d_table.copy_(dev_i32(c.table))
    c.d_lens.copy_(dev_i32(c.lens))
    c.d_y.fill_(77.0)
    c.d_lse2.fill_(77.0)
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_two_streams_at_once(gpt_lib):
    cases = [Case(12, 4, 64, 16, [3000, 100, 7], seed=s).device() for s in range(2)] + \
        [Case(12, 4, 64, 16, [300, 100, 7], seed=s).device() for s in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                c.call()
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_a_cache_of_more_than_four_gigabytes(gpt_lib):
    # offsets past 32 bits: rows in the last pages of a large pool
    c = Case(2, 2, 64, 256, [700], seed=8)
    pages = (5 << 30) // (2 * 2 * 256 * 32)
    codes = torch.zeros(pages, 2, 2, 256, 32, dtype=torch.uint8, device="cuda")
    ranges = torch.zeros(pages, 2, 2, 256, 2, dtype=torch.bfloat16, device="cuda")
    n = c.codes.shape[0]
    c.device()
    codes[pages - n:] = c.d_codes
    ranges[pages - n:] = c.d_ranges
    c.d_codes, c.d_ranges = codes, ranges
    c.d_table = dev_i32(c.table + (pages - n))
    c.call()
    c.check()


def test_a_large_cache_in_the_joined_form(gpt_lib):
    # the same where the table has room for more rows than a cluster takes
    c = Case(2, 2, 64, 256, [700], seed=8, rows=65536)
    pages = (5 << 30) // (2 * 2 * 256 * 32)
    codes = torch.zeros(pages, 2, 2, 256, 32, dtype=torch.uint8, device="cuda")
    ranges = torch.zeros(pages, 2, 2, 256, 2, dtype=torch.bfloat16, device="cuda")
    n = c.codes.shape[0]
    c.device()
    codes[pages - n:] = c.d_codes
    ranges[pages - n:] = c.d_ranges
    c.d_codes, c.d_ranges = codes, ranges
    c.d_table = dev_i32(c.table + (pages - n))
    c.call()
    c.check()


@pytest.mark.parametrize("H,Hkv,D,page,lens", [
    (2, 1, 64, 64, [170000]),                           # a list of more pieces than a large block joins at once
    (3, 1, 32, 256, [90000, 0, 70001]),
    (24, 2, 64, 16, [6000, 6001, 5, 6200, -1, 3000, 6100]),   # more heads than a large block each takes
    (20, 1, 64, 32, [20000, 333]),                      # two groups of heads on one key head
])
def test_lists_of_many_pieces(gpt_lib, H, Hkv, D, page, lens):
    Case(H, Hkv, D, page, lens, seed=len(lens), rows=65536).run()


@pytest.mark.parametrize("rows", FORMS)
@pytest.mark.parametrize("scale", [1e-30, 1e-3])
def test_small_queries(gpt_lib, rows, scale):
    c = Case(9, 3, 64, 16, [500, 70], seed=12, rows=rows, q_scale=scale)
    c.x[:, ::7] *= 2.0 ** -20                          # beside them much smaller values
    c.x = torch.from_numpy(c.x).bfloat16().float().numpy()
    c.run()
