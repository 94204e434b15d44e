"""Limits of the operators between a decoder layer's linears, checked on the host before anything is
enqueued (fake device addresses, as in test_layer_abi.py)."""
import numpy as np

import torch

import int4_weight_only_amd as w4
from tests.test_layer_abi import RANGE, SHAPE, E, cache, decode, lib, prefill, rope


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


def one_head(n_seqs, page_size=64, cols=1):
    return cache(n_kv_heads=1, head_dim=8, page_size=page_size, n_pages=1, page_stride=8 * page_size,
                 slot_stride=8, head_stride=8, n_seqs=n_seqs, table_cols=cols, ld_table=cols)


def test_launches_of_too_many_workgroups_are_refused():
    """Before anything is enqueued: 2^24 workgroups of 256 threads are one too many."""
    c = one_head(1 << 24)
    assert decode(c, H=1, ldq=8, ldy=8) == RANGE
    assert lib.w4_attn_decode_work_bytes(1, c, 0, 0) == 0
    c = one_head(1 << 23, cols=40)  # cut caches: the second kernel takes (sequence, head) pairs
    assert decode(c, H=2, ldq=16, ldy=16) == RANGE
    T, c = 1 << 24, one_head(1 << 17)
    assert prefill(c, T=T, H=127, ldq=1024, ldy=1024) == RANGE
    assert lib.w4_attn_prefill_work_bytes(T, 127, c, 0, 0) == 0
    # T * n_heads = 2^31 - 2 rows, which rounded up to tiles pass 31 bits
    assert prefill(one_head(1), T=2099202, H=1023, ldq=8184, ldy=8184) == RANGE


def test_decode_counts_tiles_in_31_bits():
    """255 sequences of 8421503 tiles: their sum fits, rounded up to shares it would not."""
    c = one_head(255, page_size=32, cols=8421503)
    assert decode(c, H=1, ldq=8, ldy=8) == RANGE
    assert lib.w4_attn_decode_work_bytes(1, c, 0, 0) == 0


def test_rope_frequencies_are_host_memory_under_any_default_device():
    want, _ = w4.w4_rope_frequencies(64)
    with torch.device("meta"):
        got, _ = w4.w4_rope_frequencies(64)
    assert got.device.type == "cpu" and torch.equal(got, want)
