"""The reference of attention over given rows of a 4-bit cache, without a GPU: against the one of whole sequences, and its bounds
against calculations that lose more than they allow."""
import numpy as np

import paged4_ref as ref
import serving_ref
from workloads import round_to_bf16


def case(H, Hkv, D, n, seed, q_values=0):
    rng = np.random.default_rng(seed)
    rows = round_to_bf16(rng.standard_normal((n, 2, Hkv, 8, D)).astype(np.float32))
    codes, ranges = serving_ref.quantise(rows)
    x = np.zeros((1, H + 2 * Hkv, D), np.float32)
    if q_values:
        x[0, np.arange(H), rng.integers(0, D, H)] = 0.5
    else:
        x[0] = round_to_bf16(rng.standard_normal((H + 2 * Hkv, D)).astype(np.float32))
    return x.reshape(1, -1), codes, ranges, rng.permutation(n).reshape(1, n)


def test_whole_sequences_and_windows():
    x, codes, ranges, table = case(4, 2, 32, 6, 0)
    for n, window, sinks in ((45, 0, 0), (45, 7, 2), (1, 0, 0), (0, 0, 0)):
        seen = [r for r in range(n) if not window or n - 1 - r < window or r < sinks]
        y, lse2, _, _ = ref.attend_rows(x, codes, ranges, table, [seen], 4)
        y2, lse3, _, _ = serving_ref.attend4(x, codes, ranges, table, [n], 4, window, sinks)
        assert np.array_equal(y, y2) and np.array_equal(lse2, lse3)


def test_the_bounds_hold_for_two_parts_and_not_for_one():
    def two_parts(x):
        x = x * 2.0 ** 8                              # largest near 2^8, as fp16 parts that are cut off
        e = np.floor(np.log2(np.maximum(x, 2.0 ** -14)))
        hi = np.trunc(x / 2.0 ** (e - 10)) * 2.0 ** (e - 10)
        lo = x - hi
        e = np.floor(np.log2(np.maximum(lo, 2.0 ** -14)))
        return (hi + np.trunc(lo / 2.0 ** (e - 10)) * 2.0 ** (e - 10)) * 2.0 ** -8

    def one_part(x):
        return x.astype(np.float16).astype(np.float64)

    off = 0
    for seed in range(4):
        x, codes, ranges, table = case(8, 2, 64, 1, seed, q_values=1)
        y, _, ey, _ = ref.attend_rows(x, codes, ranges, table, [range(3)], 8)
        assert not ref.outside(round_to_bf16(
            ref.attend_rows(x, codes, ranges, table, [range(3)], 8, rounded=two_parts)[0].astype(np.float32)), y, ey).any()
        off += ref.outside(round_to_bf16(
            ref.attend_rows(x, codes, ranges, table, [range(3)], 8, rounded=one_part)[0].astype(np.float32)), y, ey).sum()
    assert off > 10


def test_the_bounds_do_not_hold_where_a_row_without_weight_sets_the_unit():
    x, codes, ranges, table = case(2, 1, 32, 4, 5, q_values=1)
    y, _, ey, _ = ref.attend_rows(x, codes, ranges, table, [range(30)], 2)
    unit = 2.0 ** (36 - 39)                           # of a row 2^36 times larger
    got = ref.attend_rows(x, codes, ranges, table, [range(30)], 2, rounded=lambda v: np.round(v / unit) * unit)[0]
    assert ref.outside(round_to_bf16(got.astype(np.float32)), y, ey).sum() > 10
