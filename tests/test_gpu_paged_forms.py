"""The paged operators' forms on the GPU, at the sizes where the choice between them turns.

Attention of one new token: the form for few rows in sight (one launch of clusters, one or two units of 32
rows per warp) and the general one, chosen by the page table's width. Eviction: in one launch, whose choosing blocks
copy as well, or in two, chosen by the lists and the rows that they keep; copies, so equal bit for bit.

The cases, the reference and the tolerances are those of test_gpu_paged.py: both forms take the same roundings, and the
form for few rows one more factor 2^(m - M) per weight, whose 2^-22 the doubled bound of that file covers.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from gpu_util import host  # noqa: E402
from test_gpu_paged import Case, _evict_case, _evict_run  # noqa: E402


def widened(c, rows):
    """A page table for `rows` rows: the entries behind the sequences' pages name no page, and are not used."""
    more = rows // c.page - c.table.shape[1]
    assert more >= 0
    c.table = np.concatenate([c.table, np.full((c.table.shape[0], more), 10 ** 9, np.int32)], axis=1)
    return c.device()


def run(c):
    from decoder_only_transformer_gpt_gb300 import binding
    c.call()
    binding.status()
    c.check()


@pytest.mark.parametrize("rows", [1024, 2048, 4096, 65536])
@pytest.mark.parametrize("H,Hkv,D", [(4, 4, 64), (8, 1, 32), (12, 1, 64), (16, 1, 32), (9, 3, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (33, 2), (500, 7)])
def test_every_form_at_every_length(gpt_lib, rows, H, Hkv, D, window, sinks):
    for lens in ([0], [1], [30, 31, 32], [-1, 255, 256, 257], [600, -1]):
        run(widened(Case(H, Hkv, D, 16, lens, window, sinks, seed=rows + sum(lens)), rows))


@pytest.mark.parametrize("rows", [2047, 2048, 2049, 4095, 4096, 4097])
@pytest.mark.parametrize("weights", [False, True])
def test_full_tables_where_the_form_turns(gpt_lib, rows, weights):
    # the new token's row is the last that the table has room for, or near it
    run(Case(2, 2, 64, 8, [rows - 1], seed=rows, weights=weights).device())
    run(Case(4, 2, 32, 64, [rows - 1, 5], seed=rows, weights=weights).device())


@pytest.mark.parametrize("lists", [12 * 152 - 2, 12 * 152, 12 * 152 + 2])
def test_batches_where_the_form_turns(gpt_lib, lists):
    rng = np.random.default_rng(lists)
    run(Case(2, 2, 32, 8, rng.integers(-1, 255, lists // 2).tolist(), seed=lists).device())


@pytest.mark.parametrize("rows", [1024, 4096, 65536])
@pytest.mark.parametrize("weights", [False, True])
def test_more_query_heads_than_a_tile(gpt_lib, rows, weights):
    run(widened(Case(40, 2, 64, 16, [700, 3, 64], seed=rows, weights=weights), rows))


@pytest.mark.parametrize("rows", [1024, 4096, 65536])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_a_nan_in_sight_shows(gpt_lib, rows, window, sinks):
    # a NaN in a seen key or value makes the outputs of its key head's queries NaN, and no other's
    from decoder_only_transformer_gpt_gb300 import binding
    for which in (0, 1):
        c = Case(6, 2, 64, 16, [400, 90], window, sinks, seed=rows, weights=False)
        p, s = c.table[0, 380 // 16], 380 % 16
        c.pool[p, which, 1, s, 5 if which == 0 else slice(None)] = np.nan
        widened(c, rows)
        c.call()
        binding.status()
        y = host(c.d_y).reshape(2, 6, 64)
        assert np.isnan(y[0, 3:]).all() and np.isfinite(y[0, :3]).all() and np.isfinite(y[1]).all()


@pytest.mark.parametrize("rows", [1024, 4096, 65536])
def test_bad_pages_in_every_form(gpt_lib, rows):
    # rows of a page outside the pool are left out and reported; the other sequences are right
    from decoder_only_transformer_gpt_gb300 import binding
    for bad in (-1, 10 ** 9):
        c = widened(Case(4, 2, 64, 16, [100, 50], seed=14, weights=False), rows)
        c.d_table[0, 2] = bad
        c.call()
        with pytest.raises(binding.GptError) as e:
            binding.status()
        assert e.value.code == binding.GPT_EPAGE
        binding.status()
        c.check(skip=(0,))


def test_one_result_bit_for_bit_in_every_form(gpt_lib):
    for rows in (1024, 4096, 65536):
        c = widened(Case(8, 2, 64, 16, [900, 20, 333], seed=6), rows)
        c.call()
        y, lse2, w0 = c.d_y.clone(), c.d_lse2.clone(), c.d_weight.clone()
        c.device()
        c.call()
        assert torch.equal(y, c.d_y) and torch.equal(lse2, c.d_lse2) and torch.equal(w0, c.d_weight)


@pytest.mark.parametrize("B,Hkv,D,page,rows,budget,sinks,recent", [
    (20, 8, 64, 16, 300, 100, 4, 30), (20, 8, 32, 8, 300, 257, 0, 0), (77, 2, 64, 64, 700, 600, 16, 100),   # 152 lists and more
    (4, 12, 64, 16, 900, 672, 4, 64), (4, 12, 64, 16, 900, 673, 4, 64),          # 48 lists: up to 672 rows in one launch
    (1, 12, 64, 16, 700, 168, 0, 168), (1, 12, 32, 16, 700, 169, 169, 0),        # 12 lists: up to 168; nothing to choose
    (1, 1, 64, 8, 40, 14, 2, 3), (1, 1, 64, 8, 40, 15, 2, 3),
    (80, 2, 32, 64, 4400, 4096, 4, 300), (80, 2, 32, 64, 4400, 4097, 4, 300),    # kept rows past the shared list
    (10, 16, 32, 16, 200, 5000, 0, 0)])                                         # all are kept
def test_evict_in_one_launch_and_in_two(gpt_lib, B, Hkv, D, page, rows, budget, sinks, recent):
    rng = np.random.default_rng(rows)
    lens = rng.integers(-1, rows + 1, B).tolist()
    lens[0] = rows
    for kind in ("plain", "ties", "nan"):
        pool, weight, table, n, dst = _evict_case(budget, lens, Hkv, D, page, budget, kind == "ties", kind == "nan")
        _evict_run(pool, weight, table, n, dst, budget, sinks, recent)
        if table.shape[1] * page >= budget:
            _evict_run(pool, weight, table, n, table, budget, sinks, recent)


def test_evict_in_one_launch_reports_bad_pages(gpt_lib):
    # rows of a page outside the pool are neither read nor written; the other sequences are right
    from decoder_only_transformer_gpt_gb300 import binding
    import paged_ref
    from gpu_util import dev_bf16, dev_f32, dev_i32
    pool, weight, table, lens, dst = _evict_case(9, [300] * 20, 8, 64, 16, 100)
    for bad in (-1, 10 ** 9):
        for where in ("source", "target"):
            t, d = table.copy(), dst.copy()
            (t if where == "source" else d)[0, 3] = bad
            d_pool, d_weight = dev_bf16(pool), dev_f32(weight)
            new = torch.full((20,), 99, dtype=torch.int32, device="cuda")
            kept = torch.full((20, 8, 100), 99, dtype=torch.int32, device="cuda")
            binding.paged_evict(d_pool, d_weight, dev_i32(t), dev_i32(lens), dev_i32(d), new, kept, 100, 4, 30)
            with pytest.raises(binding.GptError) as e:
                binding.status()
            assert e.value.code == binding.GPT_EPAGE
            want = paged_ref.evict(pool.astype(np.float64), weight, table, lens, dst, 100, 4, 30)
            np.testing.assert_array_equal(host(new), want[2])
            np.testing.assert_array_equal(host(kept)[1:], want[3][1:])
            mine = np.concatenate([table[1:].ravel(), dst[1:].ravel()])  # the other sequences' pages
            np.testing.assert_array_equal(host(d_pool)[mine], want[0][mine])
            np.testing.assert_array_equal(host(d_weight)[mine], want[1][mine])


WIDE = 65536                                         # a table this wide takes the general form


@pytest.mark.parametrize("rows", [1024, WIDE])
@pytest.mark.parametrize("weights", [False, True])
def test_two_streams_and_two_graphs_at_once(gpt_lib, rows, weights):
    # two caches: eager calls on two streams, then a graph of each, replayed together
    a = widened(Case(12, 12, 64, 16, [700] * 8, seed=12, weights=weights), rows)
    b = widened(Case(6, 2, 32, 16, [650, 1, -1, 500], 300, 4, seed=13, weights=weights), rows)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a.call(stream=s)
    b.call(stream=t)
    torch.cuda.synchronize()
    a.check()
    b.check()
    graphs = []
    for c in (a, b):
        c.device()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        graphs.append(g)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graphs[0].replay()
    with torch.cuda.stream(t):
        graphs[1].replay()
    torch.cuda.synchronize()
    a.check()
    b.check()


@pytest.mark.parametrize("rows", [1024, WIDE])
def test_a_graph_with_other_lengths(gpt_lib, rows):
    # captured with short sequences, replayed with longer ones and one that has ended
    c = widened(Case(8, 2, 64, 16, [0, 3, 900], seed=9), rows)
    g = torch.cuda.CUDAGraph()
    c.call()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.call()
    d = widened(Case(8, 2, 64, 16, [900, -1, 17], seed=10), rows)
    for x, v in ((c.d_qkv, d.d_qkv), (c.d_pool, d.d_pool), (c.d_table, d.d_table), (c.d_lens, d.d_lens), (c.d_weight, d.d_weight)):
        x.copy_(v)
    c.d_y.fill_(7.0)
    c.d_lse2.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    d.d_y, d.d_lse2, d.d_pool, d.d_weight = c.d_y, c.d_lse2, c.d_pool, c.d_weight
    d.check()


@pytest.mark.parametrize("rows", [1024, WIDE])
def test_sequences_that_share_pages(gpt_lib, rows):
    c = Case(4, 2, 64, 16, [40, 40, 25], seed=7)
    c.table[1, :2] = c.table[0, :2]
    run(widened(c, rows))


@pytest.mark.parametrize("rows", [1024, WIDE])
def test_peaked_scores(gpt_lib, rows):
    # one row takes nearly all the weight, the rest underflow
    run(widened(Case(4, 4, 64, 16, [500, 40], seed=4, scale=24.0), rows))


@pytest.mark.parametrize("budget", [60, 400])
def test_evictions_on_two_streams(gpt_lib, budget):
    # the form with one launch and the one with two, each on two caches at once
    from decoder_only_transformer_gpt_gb300 import binding
    import paged_ref
    from gpu_util import dev_bf16, dev_f32, dev_i32
    runs = []
    for seed in (1, 2):
        pool, weight, table, lens, dst = _evict_case(seed, [500, 450, 480], 2, 64, 16, budget)
        d = [dev_bf16(pool), dev_f32(weight), dev_i32(table), dev_i32(lens), dev_i32(dst),
             torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, 2, budget, dtype=torch.int32, device="cuda")]
        runs.append((torch.cuda.Stream(), d, paged_ref.evict(pool.astype(np.float64), weight, table, lens, dst, budget, 4, 20)))
    torch.cuda.synchronize()
    for s, d, _ in runs:
        binding.paged_evict(*d, budget, 4, 20, stream=s)
    torch.cuda.synchronize()
    binding.status()
    for _, d, want in runs:
        np.testing.assert_array_equal(host(d[5]), want[2])
        np.testing.assert_array_equal(host(d[6]), want[3])
        np.testing.assert_array_equal(host(d[1]), want[1])
        np.testing.assert_array_equal(host(d[0]), want[0])
