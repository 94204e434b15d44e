"""Ends of the ranges of the operators that build, share and cross-read a paged cache, against the plain
implementations (tests/cache_reference.py)."""
import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
from tests.test_gpu_cache import Pool, ints, tables_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
def test_tables_lengths_past_the_last_column(in_place):
    """Lengths and positions count on where the table has no column: step after step, each from the
    lengths that the one before returned."""
    rng = np.random.default_rng(50)
    pool = Pool(rng, [40, 64, 0, 10], 4, 16, 9)
    for n_new in ([30, 1, 3000, 0], [1, 1, 1, 1], [2, 1, 0, 70], [1, 1, -1, 1], [0, 5, 20, 1]):
        tables_step(pool, n_new, sum(max(n, 0) for n in n_new) + 1, in_place)
    assert pool.kv_len.tolist() == [74, 73, 20, 83]


@pytest.mark.parametrize("page", [1, 16, 32768])
def test_tables_lengths_up_to_31_bits(page):
    rng = np.random.default_rng([51, page])
    most = 2 ** 31 - 1
    pool = Pool(rng, [0, 0, 0], 2, page, 9)
    pool.kv_len = np.array([most - 5, 0, 2 ** 30 + 7])
    pool.spans = np.array([[0, 0], [0, 0], [1, 2]])
    tables_step(pool, [5, 1, 2 ** 20], 2 ** 20 + 6)
    assert pool.kv_len.tolist() == [most, 1, 2 ** 30 + 2 ** 20 + 7]
    # beyond: the largest length and position
    got = w4.w4_batch_tables(ints(pool.kv_len), ints([7, 0, 0]), ints(pool.spans), ints(pool.table),
                             page, ints(pool.ring), ints(pool.state), 8)
    assert got[4].tolist() == pool.kv_len.tolist()
    assert got[3].tolist() == [most] * 7 + [-1] and got[1].tolist() == [-1] * 8
