"""Batches past 256 sequences in the operators that share and cross-read a paged cache, against the plain
implementations (tests/cache_reference.py)."""
import numpy as np
import pytest

from tests.test_gpu_cache import crossed, share

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
