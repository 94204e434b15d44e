"""Batches past 256 sequences and the precision of the weights in the operators that share and cross-read
a paged cache, against the plain implementations (tests/cache_reference.py)."""
import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
from tests import cache_reference as plain
from tests import layer_reference as ref
from tests.test_gpu_cache import MANY_KEYS, MANY_ROWS, Batch, crossed, ints, seen_slots, share
from tests.test_gpu_layer import bf16, close, f64

pytestmark = pytest.mark.gpu


def many(rng, B, prefix_len):
    """Lengths and prefixes of B sequences: short ones, some without keys, every 50th with thousands."""
    of = rng.integers(-1, len(prefix_len), B)
    own = rng.integers(0, 40, B)
    own[7::50] = rng.integers(1500, 3500, len(own[7::50]))
    lens = np.where(own > 0, own + np.where(of >= 0, np.array(prefix_len)[of], 0), 0)
    return of.tolist(), lens.tolist()


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5), (90, 700)])
@pytest.mark.parametrize("B,H,n_kv,D,page", [(257, 4, 1, 128, 16), (600, 8, 2, 64, 64),
                                             (300, 4, 2, 256, 32), (513, 3, 3, 80, 4)])
def test_shared_past_256_sequences(B, H, n_kv, D, page, window, sinks):
    """Buckets of several sequences: own units in several pieces, narrow and wide; sequences of 128
    stacked rows and more, which read both tables; prefixes that end inside a tile."""
    rng = np.random.default_rng([60, B, window])
    prefix_len = [700, 90, 0, 333]
    of, lens = many(rng, B, prefix_len)
    share(rng, prefix_len, of, lens, None, H, n_kv, D, page, window, sinks)
    nq = rng.integers(0, 4, B)
    G = H // n_kv
    nq[3::100] = 128 // G + rng.integers(0, 40, len(nq[3::100]))
    nq[57::200] = 64 // G
    share(rng, prefix_len, of, lens, nq.tolist(), H, n_kv, D, page, window, sinks, extra=2)


@pytest.mark.parametrize("B,H,n_kv,D,page", [(300, 4, 1, 128, 16), (700, 8, 4, 64, 64),
                                             (257, 2, 1, 256, 32), (400, 5, 5, 40, 4)])
def test_cross_past_256_sequences(B, H, n_kv, D, page):
    """Few rows of each (taken as units), some many, over ragged lengths."""
    rng = np.random.default_rng([61, B])
    lens = rng.integers(0, 300, B)
    lens[7::60] = rng.integers(1500, 4000, len(lens[7::60]))
    G = H // n_kv
    nq = rng.integers(0, 8 // G + 1, B)
    nq[30::120] = 140 // G
    nq[31::120] = 40 // G
    assert nq.sum() * G <= 16 * B
    crossed(rng, lens.tolist(), nq.tolist(), H, n_kv, D, page, extra=1)


@pytest.mark.parametrize("page", [1, 4])
@pytest.mark.parametrize("form,H", [("cross", 34), ("prefill", 34), ("window", 17)])
def test_many_rows_on_small_pages(form, H, page):
    """Workgroups of 64 dims on pages under 8 slots, many enough to run three on a compute unit (with a
    window fewer do), against calls of one sequence, bit for bit."""
    rng = np.random.default_rng([64, page])
    # (448 keys: too few to be split where a sequence is alone)
    lens = [min(max(n, m), 448) for n, m in zip(MANY_KEYS, MANY_ROWS)]
    rows = [min(m, n) for m, n in zip(MANY_ROWS, lens)]
    batch = Batch(rng, [0], [-1] * len(lens), lens, page, H, 64, cols=448 // page)
    starts = np.concatenate([[0], np.cumsum(rows)])
    assert (starts[-1] // 128 + len(lens)) * H > (512 if form == "window" else 1024)
    batch.fill(rng, seen_slots(batch, starts, 0, 0, True))
    q = bf16(2.0 * rng.normal(size=(starts[-1], H * 64))).cuda()
    k, v, table, kv_len = batch.args()

    def call(q, table, kv_len, starts):
        if form == "cross":
            return w4.w4_attn_cross(q, k, v, table, kv_len, ints(starts), out_dtype=w4.W4_OUT_F32)
        return w4.w4_attn_prefill(q, k, v, table, kv_len, ints(starts), out_dtype=w4.W4_OUT_F32,
                                  window=200 if form == "window" else 0)
    y = call(q, table, kv_len, starts)
    assert torch.isfinite(y).all()
    for b, n in enumerate(rows):
        if n:
            one = slice(int(starts[b]), int(starts[b + 1]))
            assert torch.equal(call(q[one], table[b:b + 1], kv_len[b:b + 1], [0, n]), y[one])


# -------------------------------------------------------------------------------------- precision


def check_weights(batch, q, q_start, y, H, scale, cross):
    """y (fp32) held to weights of 16 bits: two bf16 parts, each off by at most 2^-8 of what it rounds."""
    n, D = q.shape[0], batch.D
    wy, _, a, ds, count = plain.attention(f64(q).reshape(n, -1), f64(batch.k), f64(batch.v), batch.at,
                                          batch.lens, q_start, H, float(np.float32(scale)), 0, 0, cross)
    close(y.reshape(n, H, D), wy, ref.attention_bound(a, ds, count, 16), "y")


@pytest.mark.parametrize("H,n_kv,D", [(8, 2, 64), (4, 1, 128), (4, 4, 80), (16, 1, 128), (5, 5, 8)])
def test_shared_weights_of_few_rows(H, n_kv, D):
    """Up to 16 rows over a prefix and of a sequence, up to 128 dims: weights as two bf16 values."""
    rng = np.random.default_rng([62, D])
    G = H // n_kv
    n = 16 // G
    prefix_len = [700, 333]
    of = ([0] * n + [1] * n + [-1])
    lens = [int(x) for x in rng.integers(1, 400, len(of))]
    lens = [x + (prefix_len[g] if g >= 0 else 0) for x, g in zip(lens, of)]
    for nq in (None, [n // 2 + 1] + [0] * (n - 1) + [1] * n + [n]):
        q_start = np.concatenate([[0], np.cumsum([1] * len(of) if nq is None else nq)])
        batch, q, _, y = share(rng, prefix_len, of, lens, nq, H, n_kv, D, 16)
        check_weights(batch, q, q_start, y, H, D ** -0.5, False)


@pytest.mark.parametrize("H,n_kv,D", [(20, 20, 64), (4, 1, 128), (8, 2, 80)])
def test_cross_weights_of_few_rows(H, n_kv, D):
    rng = np.random.default_rng([63, D])
    n = 16 // (H // n_kv)
    nq = [n, 1, 0, n // 2, 2]
    lens = [1500, 33, 70, 900, 1]
    batch, q, _, y = crossed(rng, lens, nq, H, n_kv, D, 16)
    check_weights(batch, q, np.concatenate([[0], np.cumsum(nq)]), y, H, D ** -0.5, True)
