"""The operators between a decoder layer's linears at sizes that take other ways through them: more
sequences than lanes of a wave, pages shorter than a tile at every head size, page tables much wider
than any sequence."""
import numpy as np
import pytest

from tests.test_gpu_layer import attend, check_rope

pytestmark = pytest.mark.gpu


def ragged(rng, B, most, around=()):
    """B lengths up to `most`, some zero, zeros on both sides of the multiples of 64."""
    lens = rng.integers(0, most + 1, size=B)
    lens[rng.random(B) < 0.2] = 0
    for b in around:
        if b < B:
            lens[b] = 0
    lens[B - 1] = most
    return [int(n) for n in lens]


@pytest.mark.parametrize("B", [64, 65, 130, 200])
def test_decode_of_many_sequences(B):
    rng = np.random.default_rng([70, B])
    attend(rng, ragged(rng, B, 90, (63, 64, 128)), None, 8, 2, 64, 16)
    # caches that are cut into shares, which the second kernel joins
    attend(rng, ragged(rng, B, 200, (0, 62, 63)), None, 4, 1, 64, 32, cols=400)
    lens = ragged(rng, B, 60, (1, 64, 65))
    lens[66 % B] = lens[3] = 3000
    attend(rng, lens, None, 7, 1, 128, 16)
    attend(rng, lens, None, 4, 2, 80, 16, 700, 40)


@pytest.mark.parametrize("B", [64, 65, 130, 200])
def test_prompts_of_many_sequences(B):
    rng = np.random.default_rng([71, B])
    nq = ragged(rng, B, 40, (63, 64, 128))
    nq[64 % B] = 150
    attend(rng, [n + int(rng.integers(0, 60)) for n in nq], nq, 6, 2, 64, 16)
    attend(rng, [n + 5 for n in nq], nq, 4, 1, 128, 32, 20, 2)


@pytest.mark.parametrize("page", [1, 2, 4, 8])
@pytest.mark.parametrize("H,n_kv,D", [(7, 1, 128), (4, 2, 256), (4, 2, 80), (2, 1, 192)])
def test_short_pages(H, n_kv, D, page):
    rng = np.random.default_rng([72, D, page])
    attend(rng, [5, 130, 0, 77], None, H, n_kv, D, page)
    attend(rng, [2500, 130, 0, 77], None, H, n_kv, D, page, 50 if D > 128 else 0, 3)
    attend(rng, [2500], None, H, n_kv, D, page, order="head", gap=8)
    attend(rng, [150, 0, 77], [150, 0, 10], H, n_kv, D, page)
    attend(rng, [150, 0, 77], [150, 0, 10], H, n_kv, D, page, 50, 3, order="head", gap=8)
    attend(rng, [2500, 600], [3, 40], H, n_kv, D, page)  # the keys split over workgroups


@pytest.mark.parametrize("H,n_kv,D,page", [(7, 1, 128, 16), (4, 2, 256, 32), (8, 8, 64, 64)])
def test_tables_wider_than_any_sequence(H, n_kv, D, page):
    rng = np.random.default_rng([73, D])
    cols = 131072 // page
    attend(rng, [1, 0, 40, 700], None, H, n_kv, D, page, cols=cols)
    attend(rng, [33], None, H, n_kv, D, page, 100, 4, cols=cols)
    attend(rng, [77], [77], H, n_kv, D, page, cols=cols)
    attend(rng, [40, 0, 700], [40, 0, 9], H, n_kv, D, page, cols=cols)
    attend(rng, [40, 0, 700], [40, 0, 9], H, n_kv, D, page, 60, 3, cols=cols)


def test_rope_of_many_sequences():
    rng = np.random.default_rng(74)
    nq = ragged(rng, 130, 9, (63, 64, 128))
    check_rope(rng, [n + 3 for n in nq], nq, 4, 2, 64, 64, 16, 0)
    check_rope(rng, [n + 1 for n in nq], None, 4, 2, 64, 64, 16, 1)
