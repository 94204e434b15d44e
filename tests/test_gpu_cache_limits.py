"""Ends of the ranges of the operators that build, share and cross-read a paged cache, against the plain
implementations (tests/cache_reference.py)."""
import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
from tests.test_gpu_cache import Pool, ints, share, tables_step

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


@pytest.mark.parametrize("form", [None, 3])
@pytest.mark.parametrize("H,n_kv,D", [(8, 2, 64), (8, 2, 128), (4, 2, 256)])
def test_idle_sequences_take_no_part_in_their_prefix(H, n_kv, D, form):
    """Sequences without keys (ended, their prefix still named) under a window: the work is cut as if they
    named none, so that the others come out the same, bit for bit."""
    rng = np.random.default_rng([52, D])
    P, idle = 3000, np.arange(24) % 6 != 1
    of = [0] * 24
    lens = [0 if x else P + 20 + 9 * b for b, x in enumerate(idle)]
    nq = None if form is None else [form] * 24
    batch, q, starts, y = share(rng, [P], of, lens, nq, H, n_kv, D, 16, 500, 4)
    _, table, plen = batch.prefixes()
    kw = dict(q_start=starts, window=500, sinks=4, out_dtype=w4.W4_OUT_F32, want_lse=True)
    named = w4.w4_attn_shared(q, *batch.args(), ints(of), table, plen, **kw)
    alone = w4.w4_attn_shared(q, *batch.args(), ints(np.where(idle, -1, 0)), table, plen, **kw)
    assert torch.equal(named[0], alone[0]) and torch.equal(named[1], alone[1])
    rows = torch.from_numpy(np.repeat(idle, form or 1)).cuda()
    assert torch.all(named[0][rows] == 0) and torch.all(torch.isneginf(named[1][rows]))
    assert torch.isfinite(named[1][~rows]).all()
