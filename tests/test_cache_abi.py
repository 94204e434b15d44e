"""Host-side checks (no GPU) of the operators that build, share and cross-read a paged cache: argument
refusals of the C ABI (fake device addresses that are never dereferenced), size queries, the binding's
refusals."""
import pytest
import torch

import int4_weight_only_amd as w4
from tests.test_layer_abi import (A, B, C, D, E, F, G, ALIGN, CACHE_FAULTS, NULL, RANGE, SHAPE,
                                  UNSUPPORTED, cache, lib)

X, Y, Z = 0x90000, 0xA0000, 0xB0000


def prefixes(**kw):
    a = dict(prefix_of=X, table=Y, len=Z, n_prefixes=3, table_cols=5, ld_table=5)
    a.update(kw)
    return w4._Prefixes(*[a[f[0]] for f in w4._Prefixes._fields_])


def shared(c=None, p=None, **kw):
    a = dict(q=E, T=20, ldq=3584, H=28, qs=C, scale=0.1, window=0, sinks=0, y=F, ldy=3584, dt=0,
             lse=None, work=G, wb=1 << 40)
    a.update(kw)
    return lib.w4_attn_shared(a["q"], a["T"], a["ldq"], a["H"], a["qs"],
                              c if c is not None else cache(), p if p is not None else prefixes(),
                              a["scale"], a["window"], a["sinks"], a["y"], a["ldy"], a["dt"],
                              a["lse"], a["work"], a["wb"], None)


def cross(c=None, **kw):
    a = dict(q=E, T=20, ldq=3584, H=28, qs=C, scale=0.1, y=F, ldy=3584, dt=0, lse=None, work=G,
             wb=1 << 40)
    a.update(kw)
    return lib.w4_attn_cross(a["q"], a["T"], a["ldq"], a["H"], a["qs"],
                             c if c is not None else cache(), a["scale"], a["y"], a["ldy"], a["dt"],
                             a["lse"], a["work"], a["wb"], None)


@pytest.mark.parametrize("kw,status", CACHE_FAULTS)
def test_a_bad_cache_is_refused(kw, status):
    assert shared(cache(**kw)) == status
    assert cross(cache(**kw)) == status
    assert lib.w4_attn_shared_work_bytes(20, 28, cache(**kw), prefixes(), 0, 0) == 0
    assert lib.w4_attn_cross_work_bytes(20, 28, cache(**kw)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(prefix_of=None), NULL), (dict(table=None), NULL), (dict(len=None), NULL),
    (dict(n_prefixes=0), SHAPE), (dict(table_cols=0), SHAPE), (dict(ld_table=4), SHAPE),
    (dict(n_prefixes=257), RANGE), (dict(table_cols=1 << 25, ld_table=1 << 25), RANGE),
    (dict(ld_table=1 << 31), RANGE), (dict(prefix_of=X + 2), ALIGN), (dict(table=Y + 1), ALIGN),
    (dict(len=Z + 3), ALIGN)])
def test_bad_prefixes_are_refused(kw, status):
    assert shared(None, prefixes(**kw)) == status
    assert lib.w4_attn_shared_work_bytes(20, 28, cache(), prefixes(**kw), 0, 0) == 0


@pytest.mark.parametrize("call", [shared, cross])
def test_attention_refusals(call):
    for kw, status in [
            (dict(q=None), NULL), (dict(y=None), NULL), (dict(H=0), SHAPE), (dict(H=30), SHAPE),
            (dict(T=0), SHAPE), (dict(qs=None), SHAPE),  # 20 rows for 3 sequences
            (dict(ldq=3576), SHAPE), (dict(ldy=3583), SHAPE), (dict(ldq=1 << 25), RANGE),
            (dict(T=(1 << 24) + 1), RANGE), (dict(dt=2), UNSUPPORTED),
            (dict(scale=float("nan")), RANGE), (dict(scale=float("inf")), RANGE),
            (dict(scale=-0.1), RANGE), (dict(q=E + 8), ALIGN), (dict(ldq=3588), ALIGN),
            (dict(y=F + 1), ALIGN), (dict(y=F + 2, dt=1), ALIGN), (dict(lse=F + 2), ALIGN),
            (dict(qs=C + 2), ALIGN)]:
        assert call(**kw) == status, kw
    assert call(None, H=1028, ldq=1 << 18, ldy=1 << 18) == RANGE
    # more workgroups than a launch has
    assert call(cache(n_seqs=1 << 24), H=1000, ldq=1 << 17, ldy=1 << 17, T=1 << 24) != 0


def test_shared_limits():
    assert shared(cache(n_seqs=(1 << 16) + 1)) == RANGE
    assert shared(T=(1 << 21) + 1, H=4, ldq=512, ldy=512) == RANGE
    wide = dict(table_cols=1 << 22, ld_table=1 << 22)  # 2^28 positions
    assert shared(cache(**wide)) == RANGE and shared(None, prefixes(**wide)) == RANGE
    # more sequences than that over an encoder's states go the way of prompts
    assert lib.w4_attn_cross_work_bytes(20, 28, cache(n_seqs=(1 << 16) + 1)) == 0


def test_shared_masks():
    assert shared(window=-1) == RANGE and shared(sinks=-1) == RANGE
    assert lib.w4_attn_shared_work_bytes(20, 28, cache(), prefixes(), -1, 0) == 0
    assert lib.w4_attn_shared_work_bytes(0, 28, cache(), prefixes(), 0, 0) == 0
    assert lib.w4_attn_cross_work_bytes(0, 28, cache()) == 0


def test_workspaces_are_checked():
    long = cache(table_cols=4096, ld_table=4096)
    for need, call in ((lib.w4_attn_shared_work_bytes(20, 28, long, prefixes(), 0, 0), shared),
                       (lib.w4_attn_cross_work_bytes(20, 28, long), cross)):
        if need:
            assert call(long, work=None) == NULL
            assert call(long, wb=need - 1) == RANGE
            assert call(long, work=G + 4) == ALIGN


def test_tables_refusals():
    def call(**kw):
        a = dict(kv=A, new=B, spans=C, n=5, table=D, cols=8, ld=8, page=16, ring=E, size=100, state=F,
                 T=10, qs=G, slots=X, seqs=Y, pos=Z, kv_o=A + 256, spans_o=B + 256, state_o=C + 256)
        a.update(kw)
        return lib.w4_batch_tables(*a.values(), None)
    for name in ("kv", "new", "spans", "table", "ring", "state", "qs", "kv_o", "spans_o", "state_o"):
        assert call(**{name: None}) == NULL, name
    for kw, status in [
            (dict(n=0), SHAPE), (dict(cols=0), SHAPE), (dict(ld=7), SHAPE), (dict(page=0), SHAPE),
            (dict(page=-16), SHAPE), (dict(size=0), SHAPE), (dict(T=-1), SHAPE),
            (dict(page=48), UNSUPPORTED), (dict(page=1 << 16), RANGE), (dict(n=(1 << 24) + 1), RANGE),
            (dict(T=(1 << 24) + 1), RANGE), (dict(size=1 << 31), RANGE), (dict(ld=1 << 31), RANGE),
            (dict(cols=1 << 27, ld=1 << 27), RANGE),
            (dict(n=1 << 12, cols=1 << 19, ld=1 << 19, page=1), RANGE),
            (dict(slots=X + 4), ALIGN), (dict(seqs=Y + 2), ALIGN), (dict(pos=Z + 1), ALIGN),
            (dict(kv=A + 2), ALIGN), (dict(new=B + 2), ALIGN), (dict(spans=C + 2), ALIGN),
            (dict(table=D + 2), ALIGN), (dict(ring=E + 2), ALIGN), (dict(state=F + 2), ALIGN),
            (dict(qs=G + 2), ALIGN), (dict(kv_o=A + 2), ALIGN), (dict(spans_o=B + 2), ALIGN),
            (dict(state_o=C + 2), ALIGN)]:
        assert call(**kw) == status, kw


def test_the_binding_refuses_host_tensors():
    q = torch.zeros((1, 64), dtype=torch.bfloat16)
    kv = torch.zeros((1, 16, 1, 64), dtype=torch.bfloat16)
    table, n = torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.w4_attn_shared(q, kv, kv, table, n, n, table, n)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.w4_attn_cross(q, kv, kv, table, n)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.w4_batch_tables(n, n, table, table, 16, n, n, 1)
    with pytest.raises(TypeError):
        w4.w4_batch_tables(n.long(), n, table, table, 16, n, n, 1)
    with pytest.raises(TypeError):
        w4.w4_attn_cross(q.float(), kv, kv, table, n)
