"""Limits of the operators between a decoder layer's linears, checked on the host before anything is
enqueued (fake device addresses, as in test_layer_abi.py)."""
import numpy as np
import pytest

from tests.test_layer_abi import RANGE, SHAPE, E, cache, lib, rope


def overlap(gap, lda, wa, ldb, wb, T):
    """The definition: do the two sets of elements meet?"""
    a = (np.arange(T)[:, None] * lda + np.arange(wa)).ravel()
    b = (gap + np.arange(T)[:, None] * ldb + np.arange(wb)).ravel()
    return bool(np.intersect1d(a, b).size)


def test_rope_refuses_overlapping_rows():
    """Every offset of q against qkv, row by row: 1 query and 1 key-value head of 8 (24 columns of
    qkv, 8 of q). Only what overlaps is refused with equal row lengths."""
    small = dict(n_kv_heads=1, head_dim=8, page_size=1, n_pages=1, page_stride=8, slot_stride=8,
                 head_stride=8)
    for T, ld in ((1, 24), (1, 64), (3, 24), (3, 32), (3, 40), (2, 64)):
        c = cache(**small, n_seqs=T)
        for gap in range(-(T + 1) * ld, (T + 1) * ld, 8):
            if not overlap(gap, ld, 24, ld, 8, T):
                continue
            got = rope(c, qkv=E, T=T, ld=ld, H=1, rot=8, q=E + 2 * gap, ldq=ld)
            assert got == SHAPE, (T, ld, gap)
    # a q of its own row length that meets qkv
    c = cache(**small, n_seqs=3)
    for gap in range(-8 * 3 + 8, 24 * 3, 8):
        assert rope(c, qkv=E, T=3, ld=24, H=1, rot=8, q=E + 2 * gap, ldq=8) == SHAPE, gap
