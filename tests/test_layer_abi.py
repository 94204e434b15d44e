"""Host-side checks (no GPU) of the operators between a decoder layer's linears: argument refusals
of the C ABI (fake device addresses that must never be dereferenced: every call below fails a check
first), size queries, the rotary frequencies, and the binding's refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4

OK, NULL, SHAPE, GROUP, ALIGN, RANGE, UNSUPPORTED, HIP = range(8)
A, B, C, D, E, F, G = (0x10000 * i for i in range(1, 8))
lib = w4._lib


def cache(**kw):
    a = dict(k=A, v=B, n_pages=10, page_stride=64 * 4 * 128, slot_stride=4 * 128, head_stride=128,
             page_size=64, n_kv_heads=4, head_dim=128, page_table=C, n_seqs=3, table_cols=5,
             ld_table=5, kv_len=D)
    a.update(kw)
    return w4._KvCache(*[a[f[0]] for f in w4._KvCache._fields_])


def decode(c=None, **kw):
    a = dict(q=E, ldq=3584, H=28, scale=0.1, window=0, sinks=0, y=F, ldy=3584, dt=0, lse=None,
             work=G, wb=1 << 40)
    a.update(kw)
    return lib.w4_attn_decode(a["q"], a["ldq"], a["H"], c if c is not None else cache(),
                              a["scale"], a["window"], a["sinks"], a["y"], a["ldy"], a["dt"],
                              a["lse"], a["work"], a["wb"], None)


def prefill(c=None, **kw):
    a = dict(q=E, T=20, ldq=3584, H=28, qs=C, scale=0.1, window=0, sinks=0, y=F, ldy=3584, dt=0,
             lse=None, work=G, wb=1 << 40)
    a.update(kw)
    return lib.w4_attn_prefill(a["q"], a["T"], a["ldq"], a["H"], a["qs"],
                               c if c is not None else cache(), a["scale"], a["window"],
                               a["sinks"], a["y"], a["ldy"], a["dt"], a["lse"], a["work"],
                               a["wb"], None)


def rope(c=None, **kw):
    a = dict(qkv=E, T=3, ld=4608, H=28, qs=None, f=F, rot=128, layout=0, factor=1.0, q=G, ldq=3584)
    a.update(kw)
    return lib.w4_rope_append(a["qkv"], a["T"], a["ld"], a["H"], a["qs"], a["f"], a["rot"],
                              a["layout"], a["factor"], c if c is not None else cache(), a["q"],
                              a["ldq"], None)


CACHE_FAULTS = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(page_table=None), NULL),
    (dict(kv_len=None), NULL), (dict(n_pages=0), SHAPE), (dict(n_kv_heads=0), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=-16), SHAPE),
    (dict(table_cols=0), SHAPE), (dict(table_cols=6), SHAPE), (dict(n_seqs=0), SHAPE),
    (dict(n_kv_heads=3), SHAPE),  # does not divide the 28 query heads
    (dict(head_stride=120), SHAPE), (dict(slot_stride=64), SHAPE), (dict(page_stride=0), SHAPE),
    (dict(n_pages=1 << 31), RANGE), (dict(page_size=1 << 16), RANGE),
    (dict(table_cols=1 << 26, ld_table=1 << 26), RANGE),  # 2^32 positions
    (dict(slot_stride=1 << 26), RANGE),  # a page of 2^32 elements
    (dict(page_stride=1 << 61), RANGE),
    (dict(page_size=48), UNSUPPORTED), (dict(k=A + 2), ALIGN), (dict(v=B + 8), ALIGN),
    (dict(head_stride=132), ALIGN), (dict(slot_stride=516), ALIGN),
    (dict(page_stride=64 * 512 + 4), ALIGN), (dict(page_table=C + 2), ALIGN),
    (dict(kv_len=D + 1), ALIGN),
]


@pytest.mark.parametrize("kw,status", CACHE_FAULTS)
def test_a_bad_cache_is_refused(kw, status):
    assert decode(cache(**kw)) == status
    assert prefill(cache(**kw)) == status
    assert rope(cache(**kw)) == status
    assert lib.w4_attn_decode_work_bytes(28, cache(**kw), 0, 0) == 0
    assert lib.w4_attn_prefill_work_bytes(20, 28, cache(**kw), 0, 0) == 0


def test_head_dims():
    wide = dict(page_stride=64 * 4 * 264, slot_stride=4 * 264, head_stride=264)
    assert decode(cache(head_dim=264, **wide), ldq=1 << 14, ldy=1 << 14) == RANGE
    assert decode(cache(head_dim=100, **wide)) == UNSUPPORTED
    assert decode(cache(head_dim=4, **wide)) == UNSUPPORTED


@pytest.mark.parametrize("call", [decode, prefill])
def test_attention_refusals(call):
    for kw, status in [
            (dict(q=None), NULL), (dict(y=None), NULL), (dict(H=0), SHAPE), (dict(H=30), SHAPE),
            (dict(ldq=3576), SHAPE), (dict(ldy=3583), SHAPE), (dict(ldq=1 << 25), RANGE),
            (dict(dt=2), UNSUPPORTED), (dict(scale=float("nan")), RANGE),
            (dict(scale=float("inf")), RANGE), (dict(scale=-0.1), RANGE), (dict(window=-1), RANGE),
            (dict(sinks=-1), RANGE), (dict(q=E + 8), ALIGN), (dict(ldq=3588), ALIGN),
            (dict(y=F + 1), ALIGN), (dict(y=F + 2, dt=1), ALIGN), (dict(lse=F + 2), ALIGN)]:
        assert call(**kw) == status, kw
    assert call(None, H=1028, ldq=1 << 18, ldy=1 << 18) == RANGE
    assert lib.w4_attn_decode(E, 3584, 28, None, 0.1, 0, 0, F, 3584, 0, None, G, 0, None) == NULL


def test_prefill_refusals():
    assert prefill(qs=None) == NULL
    assert prefill(qs=C + 2) == ALIGN
    assert prefill(T=0) == SHAPE
    assert prefill(T=(1 << 24) + 1) == RANGE


def test_workspaces_are_checked():
    long = cache(table_cols=4096, ld_table=4096)
    for need, call in ((lib.w4_attn_decode_work_bytes(28, long, 0, 0), decode),
                       (lib.w4_attn_prefill_work_bytes(20, 28, long, 0, 0), prefill)):
        if need:
            assert call(long, work=None) == NULL
            assert call(long, wb=need - 1) == RANGE
            assert call(long, work=G + 4) == ALIGN
    assert lib.w4_attn_decode_work_bytes(28, long, -1, 0) == 0
    assert lib.w4_attn_prefill_work_bytes(0, 28, long, 0, 0) == 0


def test_rope_refusals():
    for kw, status in [
            (dict(qkv=None), NULL), (dict(f=None), NULL), (dict(q=None), NULL),
            (dict(T=0), SHAPE), (dict(T=4), SHAPE),  # without q_start T is the number of sequences
            (dict(ld=4600), SHAPE), (dict(ldq=3576), SHAPE), (dict(rot=0), SHAPE),
            (dict(rot=127), SHAPE), (dict(rot=130), SHAPE), (dict(layout=2), UNSUPPORTED),
            (dict(factor=float("inf")), RANGE), (dict(T=(1 << 24) + 1, qs=C), RANGE),
            (dict(ld=1 << 25), RANGE), (dict(qkv=E + 2), ALIGN), (dict(ld=4612), ALIGN),
            (dict(q=G + 4), ALIGN), (dict(ldq=3588), ALIGN), (dict(f=F + 2), ALIGN),
            (dict(qs=C + 1), ALIGN)]:
        assert rope(**kw) == status, kw


def test_norm_refusals():
    def call(**kw):
        a = dict(x=A, ldx=64, r=B, ldr=64, dt=0, T=2, d=64, wpost=None, wpre=C, off=0.0, gate=None,
                 ldg=0, alpha=1.0, eps=1e-6, ro=D, ldro=64, y=E, ldy=64)
        a.update(kw)
        return lib.w4_residual_norm(a["x"], a["ldx"], a["r"], a["ldr"], a["dt"], a["T"], a["d"],
                                    a["wpost"], a["wpre"], a["off"], a["gate"], a["ldg"],
                                    a["alpha"], a["eps"], a["ro"], a["ldro"], a["y"], a["ldy"],
                                    None)
    nan = float("nan")
    for kw, status in [
            (dict(r=None), NULL), (dict(wpre=None), NULL), (dict(y=None), NULL),
            (dict(ro=None), NULL), (dict(x=None), NULL), (dict(x=None, ro=None, wpost=C), NULL),
            (dict(x=None, ro=None, gate=C), NULL), (dict(T=0), SHAPE), (dict(d=0), SHAPE),
            (dict(ldx=63), SHAPE), (dict(ldr=63), SHAPE), (dict(ldy=63), SHAPE),
            (dict(ldro=63), SHAPE), (dict(gate=F, ldg=63), SHAPE),
            (dict(ro=B, ldro=72), SHAPE),  # in place with another row length
            (dict(d=(1 << 15) + 1, ldx=1 << 16, ldr=1 << 16, ldy=1 << 16, ldro=1 << 16), RANGE),
            (dict(ldx=1 << 25), RANGE), (dict(dt=2), UNSUPPORTED), (dict(eps=-1.0), RANGE),
            (dict(eps=nan), RANGE), (dict(alpha=nan), RANGE), (dict(off=nan), RANGE),
            (dict(x=A + 1), ALIGN), (dict(r=B + 2, dt=1), ALIGN), (dict(ro=D + 1), ALIGN),
            (dict(wpre=C + 1), ALIGN), (dict(wpost=C + 1), ALIGN), (dict(gate=F + 1), ALIGN),
            (dict(y=E + 1), ALIGN)]:
        assert call(**kw) == status, kw


def test_rope_frequencies_by_their_definitions():
    R, base, factor, ctx = 128, 10000.0, 4.0, 4096.0
    i = np.arange(R // 2, dtype=np.float64)
    plain = base ** (-2 * i / R)
    for scaling, want in [
            (w4.W4_ROPE_PLAIN, plain), (w4.W4_ROPE_LINEAR, plain / factor),
            (w4.W4_ROPE_NTK, (base * factor ** (R / (R - 2))) ** (-2 * i / R))]:
        got, amplitude = w4.w4_rope_frequencies(R, scaling, base, factor, ctx)
        assert amplitude == 1.0
        np.testing.assert_allclose(got.numpy(), want, rtol=2.0 ** -23)
    # the stretched base keeps the highest frequency and divides the lowest by the factor
    got, _ = w4.w4_rope_frequencies(R, w4.W4_ROPE_NTK, base, factor)
    assert got[0] == 1.0 and abs(got[-1].item() * factor / plain[-1] - 1) < 1e-6
    got, amplitude = w4.w4_rope_frequencies(R, w4.W4_ROPE_YARN, base, factor, ctx)
    assert abs(amplitude - (0.1 * math.log(factor) + 1)) < 1e-7
    turns = ctx * plain / (2 * math.pi)
    got = got.numpy()
    # outside the two dimensions (rounded outwards by less than one) the rule is exact
    keep, divide = turns > 32 * base ** (2 / R), turns < base ** (-2 / R)
    assert keep.any() and divide.any()
    np.testing.assert_allclose(got[keep], plain[keep], rtol=2.0 ** -23)
    np.testing.assert_allclose(got[divide], plain[divide] / factor, rtol=2.0 ** -23)
    between = ~(keep | divide)
    assert np.all(got[between] <= plain[between] * (1 + 1e-6))
    assert np.all(got[between] >= plain[between] / factor * (1 - 1e-6))
    ratio = got / plain
    assert np.all(np.diff(ratio) <= 1e-6)


def test_rope_frequencies_refusals():
    f = (ctypes.c_float * 128)()

    def call(R=64, s=0, base=1e4, factor=2.0, ctx=4096.0, out=f):
        return lib.w4_rope_frequencies(R, s, base, factor, ctx, out, None)
    assert call() == OK
    assert call(out=None) == NULL
    assert call(R=0) == SHAPE and call(R=63) == SHAPE and call(R=258) == SHAPE
    assert call(R=2, s=2) == SHAPE and call(R=2, s=1) == OK
    assert call(s=4) == UNSUPPORTED and call(s=-1) == UNSUPPORTED
    assert call(base=1.0) == RANGE and call(base=float("inf")) == RANGE
    for s in (1, 2, 3):
        assert call(s=s, factor=0.5) == RANGE and call(s=s, factor=float("nan")) == RANGE
    assert call(s=3, ctx=0.5) == RANGE
    assert call(s=3, ctx=1.0) == OK  # every pair turns less than once
    with pytest.raises(w4.W4Error):
        w4.w4_rope_frequencies(63)


def test_the_binding_refuses_host_tensors():
    q = torch.zeros((1, 64), dtype=torch.bfloat16)
    kv = torch.zeros((1, 16, 1, 64), dtype=torch.bfloat16)
    table, n = torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.w4_attn_decode(q, kv, kv, table, n)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.w4_attn_prefill(q, kv, kv, table, n, torch.tensor([0, 1], dtype=torch.int32))
    with pytest.raises(TypeError):
        w4.w4_attn_prefill(q, kv, kv, table, n, None)
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.w4_rope_append(torch.zeros((1, 192), dtype=torch.bfloat16), 1, kv, kv, table, n,
                          torch.ones(32))
    with pytest.raises(ValueError, match="GPU tensor"):
        w4.w4_residual_norm(q, q, q[0])
    with pytest.raises(TypeError):
        w4.w4_residual_norm(q, q.to(torch.float64), q[0])
