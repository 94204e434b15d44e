"""The operators between a decoder layer's linears against plain implementations in 64 bits
(tests/layer_reference.py), through the public binding.  Bounds come from the arithmetic: half an
ulp of each rounding the definitions name, fp32 sums of the length at hand."""
import contextlib

import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def close(got, want, bound, what):
    got = got if isinstance(got, np.ndarray) else f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: non-finite values"
    over = np.abs(got - want) / bound
    assert over.max(initial=0.0) <= 1.0, \
        f"{what}: {int((over > 1).sum())} of {over.size} outside, worst {over.max():.3g} bounds " \
        f"at {np.unravel_index(over.argmax(), over.shape)}"


class Paged:
    """A cache of NaN, but for the slots written through fill(); page tables of garbage, but for
    the entries in use.  order: "slot" [page][slot][head][D] or "head" [page][head][slot][D]; gap:
    elements between two heads' rows."""

    def __init__(self, rng, lens, page, n_kv, D, order="slot", gap=0, cols=None):
        need = [-(-max(n, 0) // page) for n in lens]
        cols = max(need + [1]) if cols is None else cols
        need = [min(x, cols) for x in need]
        total = sum(need) + 2
        where = rng.permutation(total)
        self.table = rng.choice([-1, -2 ** 31, 2 ** 31 - 1, total], size=(len(lens), cols))
        at = 0
        for b, x in enumerate(need):
            self.table[b, :x] = where[at:at + x]
            at += x
        shape = (total, page, n_kv, D + gap) if order == "slot" else (total, n_kv, page, D + gap)

        def buffer():
            t = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            t = t if order == "slot" else t.permute(0, 2, 1, 3)
            return t[..., :D]
        self.k, self.v = buffer(), buffer()
        self.page, self.n_kv, self.D, self.cols = page, n_kv, D, cols
        self.lens = np.asarray(lens)
        self.d_table = torch.from_numpy(self.table.astype(np.int32)).cuda()
        self.d_len = torch.tensor(lens, dtype=torch.int32).cuda()

    def fill(self, rng, positions, kscale=1.0):
        """Random finite keys and values at the given positions of each sequence."""
        for b, pos in enumerate(positions):
            pos = np.asarray(pos, dtype=np.int64)
            pg = torch.from_numpy(self.table[b][pos // self.page].astype(np.int64)).cuda()
            sl = torch.from_numpy(pos % self.page).cuda()
            for t, s in ((self.k, kscale), (self.v, 1.0)):
                t[pg, sl] = bf16(s * rng.normal(size=(len(pos), self.n_kv, self.D))).cuda()

    def args(self):
        return self.k, self.v, self.d_table, self.d_len

    def host(self):
        return f64(self.k), f64(self.v), self.table


def strided(t, pad):
    """The same values in rows of a wider buffer of NaN."""
    w = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]]


def attend(rng, lens, nq, H, n_kv, D, page, window=0, sinks=0, order="slot", gap=0, kscale=1.0,
           pad=0, scale=None, cols=None):
    """Runs one case in the form that nq asks for (None: one token each) and checks it."""
    cache = Paged(rng, lens, page, n_kv, D, order, gap, cols)
    counts = [1] * len(lens) if nq is None else nq
    q_start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = int(q_start[-1])
    seen = [set() for _ in lens]
    for _, b, pos in ref.rows_of(q_start, lens, cache.cols * page):
        seen[b].update(ref.visible(pos, window, sinks).tolist())
    cache.fill(rng, [sorted(s) for s in seen], kscale)
    q = bf16(2.0 * rng.normal(size=(T, H * D))).cuda()
    q = strided(q, pad) if pad else q
    scale = D ** -0.5 if scale is None else scale

    def call(dt, out=None):
        kw = dict(scale=scale, window=window, sinks=sinks, out_dtype=dt, want_lse=True, out=out)
        if nq is None:
            return w4.w4_attn_decode(q, *cache.args(), **kw)
        return w4.w4_attn_prefill(q, *cache.args(), torch.from_numpy(q_start).cuda(), **kw)
    out = None
    if pad:
        out = torch.full((T, H * D + pad + 1), float("nan"), device="cuda")[:, :H * D]
    y, lse = call(w4.W4_OUT_F32, out)
    y16, lse16 = call(w4.W4_OUT_BF16)
    torch.cuda.synchronize()
    k, v, table = cache.host()
    wy, wl, a, ds, count = ref.attention(f64(q).reshape(T, -1), k, v, table, lens, q_start, H,
                                         float(np.float32(scale)), window, sinks)
    bound = ref.attention_bound(a, ds, count, 16 if nq is None else 8)
    close(y.reshape(T, H, D), wy, bound, "y")
    assert torch.equal(y16, y.to(torch.bfloat16)), "bf16 output is not the rounded fp32 output"
    got = f64(lse)
    empty = np.isinf(wl)
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got - wl)[~empty] <= (2 * ds + 2.0 ** -20 + (count + 4) * ref.F32 * 2
                                               + 2.0 ** -22 * np.abs(wl))[~empty])
    assert torch.equal(lse, lse16)
    if pad:
        assert torch.isnan(out.as_strided((T, pad + 1), (H * D + pad + 1, 1), H * D)).all()
    assert torch.all(y.reshape(T, H, D)[torch.from_numpy(empty).cuda()] == 0)
    return cache, q


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 130, 300]


@pytest.mark.parametrize("H,n_kv,D", [(28, 4, 128), (8, 8, 64), (16, 2, 256), (3, 1, 80),
                                      (32, 1, 128), (5, 5, 8), (9, 3, 192), (64, 4, 24),
                                      (1, 1, 136), (17, 1, 64)])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_lengths_and_heads(H, n_kv, D, page):
    rng = np.random.default_rng([1, H, D, page])
    attend(rng, LENS, None, H, n_kv, D, page)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (32, 0), (33, 4), (64, 64),
                                          (100, 31), (128, 0), (299, 1), (1000, 5), (20, 200),
                                          (20, 10 ** 12), (10 ** 12, 3)])
def test_decode_windows_and_sinks(window, sinks):
    rng = np.random.default_rng([2, window, sinks])
    attend(rng, LENS + [1027], None, 14, 2, 128, 32, window, sinks)
    attend(rng, LENS + [700], None, 4, 4, 80, 16, window, sinks)


@pytest.mark.parametrize("page", [1, 2, 8, 128, 1024])
@pytest.mark.parametrize("order,gap", [("slot", 0), ("head", 0), ("slot", 8), ("head", 24)])
def test_decode_page_sizes_and_layouts(page, order, gap):
    rng = np.random.default_rng([3, page, gap])
    attend(rng, [5, 130, 0, 77], None, 6, 2, 64, page, order=order, gap=gap, pad=8)
    attend(rng, [5, 130, 0, 77], None, 6, 2, 64, page, 50, 3, order=order, gap=gap, pad=16)


def test_decode_long_and_split():
    rng = np.random.default_rng(4)
    attend(rng, [20001], None, 7, 1, 128, 64)
    attend(rng, [9000, 3, 4097], None, 8, 2, 64, 16)
    attend(rng, [8000, 12000], None, 4, 2, 256, 128, 4500, 70)


@pytest.mark.parametrize("form", [None, [3, 1, 40]])
def test_extreme_scores(form):
    rng = np.random.default_rng(5)
    attend(rng, [200, 64, 129], form, 8, 2, 128, 16, kscale=60.0)  # scores of several hundred
    attend(rng, [200, 64, 129], form, 8, 2, 128, 16, scale=0.0)  # all keys alike
    attend(rng, [200, 64, 129], form, 8, 2, 128, 16, scale=1e-30)
    attend(rng, [200, 64, 129], form, 8, 2, 128, 16, kscale=1e18, scale=1e-20)


@pytest.mark.parametrize("form", [None, [4, 30]])
def test_lengths_the_table_cannot_hold(form):
    """kv_len above the table's capacity counts as the capacity, below zero as zero."""
    rng = np.random.default_rng(6)
    attend(rng, [1000, -7], form, 4, 2, 64, 16, cols=5)


@pytest.mark.parametrize("H,n_kv,D", [(28, 4, 128), (8, 8, 64), (16, 2, 256), (3, 1, 80),
                                      (32, 1, 128), (5, 5, 8), (9, 3, 192), (17, 1, 136)])
def test_prefill_lengths_and_heads(H, n_kv, D):
    rng = np.random.default_rng([7, H, D])
    nq = [1, 2, 15, 16, 17, 0, 64, 65, 130, 3]
    attend(rng, [1, 2, 15, 16, 17, 9, 64, 65, 130, 40], nq, H, n_kv, D, 16)
    attend(rng, [90, 2, 170], [33, 2, 65], H, n_kv, D, 64)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (7, 3), (32, 0), (33, 4), (64, 64),
                                          (65, 70), (128, 1), (1000, 5), (20, 200)])
def test_prefill_windows_and_sinks(window, sinks):
    rng = np.random.default_rng([8, window, sinks])
    attend(rng, [300, 40, 513], [300, 7, 200], 14, 2, 128, 32, window, sinks)
    attend(rng, [300, 40, 413], [100, 40, 20], 4, 4, 80, 16, window, sinks)


@pytest.mark.parametrize("page", [1, 4, 128, 512])
@pytest.mark.parametrize("order,gap", [("slot", 0), ("head", 0), ("slot", 8), ("head", 24)])
def test_prefill_page_sizes_and_layouts(page, order, gap):
    rng = np.random.default_rng([9, page, gap])
    attend(rng, [150, 0, 77], [150, 0, 10], 6, 2, 64, page, order=order, gap=gap, pad=8)
    attend(rng, [150, 0, 77], [150, 0, 10], 6, 2, 64, page, 50, 3, order=order, gap=gap, pad=16)


def test_prefill_rows_before_the_cache_begins():
    """More rows than keys: the first rows stand at negative positions and see nothing."""
    rng = np.random.default_rng(10)
    attend(rng, [5, 0, 70], [9, 4, 100], 8, 2, 128, 16)
    attend(rng, [5, 0, 70], [9, 4, 100], 8, 2, 128, 16, 3, 1)


def test_prefill_few_rows_over_a_long_cache():
    rng = np.random.default_rng(11)
    attend(rng, [5000, 33], [3, 2], 8, 2, 128, 64)
    attend(rng, [9000], [17], 7, 1, 64, 16)
    attend(rng, [6000, 4000], [5, 140], 4, 2, 128, 32, 2500, 100)


def test_both_forms_agree_on_one_token():
    rng = np.random.default_rng(12)
    cache, q = attend(rng, [700, 1, 0, 64], None, 28, 4, 128, 16)
    starts = torch.arange(5, dtype=torch.int32).cuda()
    a = w4.w4_attn_decode(q, *cache.args(), out_dtype=w4.W4_OUT_F32)
    b = w4.w4_attn_prefill(q, *cache.args(), starts, out_dtype=w4.W4_OUT_F32)
    assert (a - b).abs().max().item() <= 2.0 ** -7 * 5


@pytest.mark.parametrize("form", [None, [40, 1, 5]])
def test_attention_is_deterministic(form):
    rng = np.random.default_rng(13)
    cache, q = attend(rng, [4500, 1200, 77], form, 8, 2, 128, 16)
    starts = torch.tensor([0, 40, 41, 46], dtype=torch.int32).cuda()

    def run():
        if form is None:
            return w4.w4_attn_decode(q, *cache.args())
        return w4.w4_attn_prefill(q, *cache.args(), starts)
    first = run().clone()
    for _ in range(5):
        assert torch.equal(run(), first)


def test_offsets_past_32_bits():
    """Pages 2^28 elements apart and query rows 2^24 apart: element offsets pass 2^31."""
    rng = np.random.default_rng(14)
    n_kv, D, page, pages, H, T = 2, 64, 16, 12, 4, 140
    stride = 1 << 28

    def buffer():
        flat = torch.empty((pages - 1) * stride + page * n_kv * D, dtype=torch.bfloat16,
                           device="cuda")
        return flat.as_strided((pages, page, n_kv, D), (stride, n_kv * D, D, 1))
    k, v = buffer(), buffer()
    small_k = bf16(rng.normal(size=(pages, page, n_kv, D))).cuda()
    small_v = bf16(rng.normal(size=(pages, page, n_kv, D))).cuda()
    k.copy_(small_k)
    v.copy_(small_v)
    table = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()[None]
    n = torch.tensor([pages * page - 3], dtype=torch.int32).cuda()
    ld = 1 << 24
    flat = torch.empty((T - 1) * ld + H * D, dtype=torch.bfloat16, device="cuda")
    q = flat.as_strided((T, H * D), (ld, 1))
    q.copy_(bf16(rng.normal(size=(T, H * D))).cuda())
    starts = torch.tensor([0, T], dtype=torch.int32).cuda()
    assert torch.equal(w4.w4_attn_prefill(q, k, v, table, n, starts),
                       w4.w4_attn_prefill(q.contiguous(), small_k, small_v, table, n, starts))
    assert torch.equal(w4.w4_attn_decode(q[-1:], k, v, table, n),
                       w4.w4_attn_decode(q[-1:].contiguous(), small_k, small_v, table, n))
    qkv = bf16(rng.normal(size=(1, (H + 2 * n_kv) * D))).cuda()
    f = torch.ones(D // 2, device="cuda")
    a = w4.w4_rope_append(qkv, H, k, v, table, n, f)
    b = w4.w4_rope_append(qkv, H, small_k, small_v, table, n, f)
    assert torch.equal(a, b) and torch.equal(k, small_k) and torch.equal(v, small_v)


# ------------------------------------------------------------------------------- rotary, append


def check_rope(rng, lens, nq, H, n_kv, D, rot, page, layout, factor=1.0, order="slot", gap=0,
               pad=0, cols=None, base=1e6):
    cache = Paged(rng, lens, page, n_kv, D, order, gap, cols)
    counts = [1] * len(lens) if nq is None else nq
    q_start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = int(q_start[-1])
    x = bf16(rng.normal(size=(T, (H + 2 * n_kv) * D))).cuda()
    x = strided(x, pad) if pad else x
    freq = torch.from_numpy((base ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32))
    out = None
    if pad:
        out = torch.full((T, H * D + pad), float("nan"), dtype=torch.bfloat16,
                         device="cuda")[:, :H * D]
    before = cache.k.view(torch.int16).clone(), cache.v.view(torch.int16).clone()
    got = w4.w4_rope_append(
        x, H, *cache.args(), freq.cuda(), layout=layout, factor=factor, out=out,
        q_start=None if nq is None else torch.from_numpy(q_start).cuda())
    torch.cuda.synchronize()
    rows = ref.rows_of(q_start, lens, cache.cols * page)
    pos = np.array([p for _, _, p in rows])
    xs = f64(x).reshape(T, H + 2 * n_kv, D)
    want, size = ref.rope(xs[:, :H + n_kv], pos, freq.numpy(), layout,
                          float(np.float32(factor)))
    # one rounding to bf16, a few fp32 operations on the pair, an angle within 2^-23 of a turn
    bound = 1.01 * ref.BF16 * np.abs(want) + 2e-6 * abs(factor) * size
    bound[..., rot:] = 1e-30  # copied
    close(got.reshape(T, H, D), want[:, :H], bound[:, :H] + 1e-30, "q")
    k, v = f64(cache.k), f64(cache.v)
    touched = np.zeros(before[0].shape[:2], dtype=bool)
    bits = x.reshape(T, H + 2 * n_kv, D).view(torch.int16)
    for t, b, p in rows:
        if p < 0:
            continue
        at = (cache.table[b][p // page], p % page)
        touched[at] = True
        close(k[at], want[t, H:], bound[t, H:] + 1e-30, f"k of row {t}")
        assert torch.equal(cache.v.view(torch.int16)[at], bits[t, H + n_kv:]), f"v of row {t}"
    rest = torch.from_numpy(~touched).cuda()
    for t, was in zip((cache.k, cache.v), before):
        assert torch.equal(t.view(torch.int16)[rest], was[rest]), "a slot changed that is not new"
    if pad:
        assert torch.isnan(out.as_strided((T, pad), (H * D + pad, 1), H * D)).all()


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (80, 40), (256, 64), (8, 8), (8, 2),
                                   (72, 70), (128, 6), (256, 256), (24, 12), (192, 190)])
def test_rope_layouts_and_partial_heads(layout, D, rot):
    rng = np.random.default_rng([20, layout, D, rot])
    check_rope(rng, [1, 5, 130, 64, 17], None, 6, 2, D, rot, 16, layout)
    check_rope(rng, [9, 5, 130, 64], [9, 0, 67, 1], 6, 2, D, rot, 64, layout, factor=1.14)


@pytest.mark.parametrize("page,order,gap,pad", [(1, "slot", 0, 0), (2, "head", 8, 8),
                                                (128, "head", 0, 24), (16, "slot", 16, 8)])
def test_rope_page_sizes_and_layouts(page, order, gap, pad):
    rng = np.random.default_rng([21, page])
    check_rope(rng, [3, 200], [3, 150], 4, 4, 64, 64, page, 0, order=order, gap=gap, pad=pad)
    check_rope(rng, [3, 200], None, 28, 4, 128, 128, page, 1, order=order, gap=gap, pad=pad)


def test_rope_positions_up_to_a_million():
    rng = np.random.default_rng(22)
    check_rope(rng, [1000000, 131073], [37, 5], 2, 1, 64, 64, 32768, 0)
    check_rope(rng, [1000000], None, 2, 1, 8, 8, 32768, 1)


def test_rope_rows_that_are_not_appended():
    """Rows at negative positions and an idle slot leave the cache alone; lengths beyond the table
    are cut to it."""
    rng = np.random.default_rng(23)
    check_rope(rng, [5, 0, 70], [9, 2, 70], 4, 2, 64, 64, 16, 0)
    check_rope(rng, [5, 0, -3], None, 4, 2, 64, 64, 16, 0)
    check_rope(rng, [500, 3], None, 4, 2, 64, 32, 16, 1, cols=4)


def test_rope_drops_appends_to_pages_outside_the_cache():
    x = bf16(np.ones((2, 3 * 64))).cuda()
    k = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[-1], [2]], dtype=torch.int32, device="cuda")
    n = torch.tensor([4, 4], dtype=torch.int32, device="cuda")
    q = w4.w4_rope_append(x, 1, k, v, table, n, torch.ones(32, device="cuda"))
    assert torch.isfinite(q).all() and not k.any() and not v.any()


# ------------------------------------------------------------------------------- residual norm


def check_norm(rng, T, d, f32, post, gate, with_x=True, pad=0, in_place=False, offset=0.0,
               eps=1e-6, alpha=0.7, size=1.0):
    def rows(scale, dtype=torch.bfloat16):
        t = torch.from_numpy((scale * rng.normal(size=(T, d))).astype(np.float32)).to(dtype).cuda()
        return strided(t, pad) if pad else t
    r = rows(3.0 * size, torch.float32 if f32 else torch.bfloat16)
    x = rows(size) if with_x else None
    w_pre = bf16(1 + 0.2 * rng.normal(size=d)).cuda()
    w_post = bf16(1 + 0.2 * rng.normal(size=d)).cuda() if post else None
    g = {None: None, "channel": bf16(rng.normal(size=d)).cuda(), "token": rows(1.0)}[gate]
    r0 = f64(r) if not f32 else r.cpu().numpy().astype(np.float64)
    y, ro = w4.w4_residual_norm(x, r, w_pre, w_post=w_post, gate=g, alpha=alpha, eps=eps,
                                weight_offset=offset,
                                residual_out=r if in_place and with_x else None)
    torch.cuda.synchronize()
    num = [None if t is None else f64(t) for t in (x, w_pre, w_post, g)]
    wy, wr, mag = ref.residual_norm(num[0], r0, num[1], num[2], num[3], float(np.float32(alpha)),
                                    float(np.float32(eps)), float(np.float32(offset)))
    sums = (d + 16) * ref.F32  # an fp32 sum of d terms (its root: half of that), and a few steps
    if with_x:
        close(f64(ro) if not f32 else ro.cpu().numpy().astype(np.float64), wr,
              mag * (2 * sums + (0 if f32 else 1.01 * ref.BF16)) + 1e-30, "r'")
        assert (ro.data_ptr() == r.data_ptr()) == in_place
    scale = np.abs(wy / np.where(wr == 0, 1, wr))
    close(y, wy, np.abs(wy) * (1.01 * ref.BF16 + 2 * sums) + scale * mag * 2 * sums + 1e-30, "y")


@pytest.mark.parametrize("d", [1, 2, 7, 8, 64, 257, 511, 1000, 2048, 3584, 4099, 8192, 16384,
                               20000, 32768])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_widths(d, f32):
    rng = np.random.default_rng([30, d])
    check_norm(rng, 3, d, f32, True, "token")
    check_norm(rng, 1, d, f32, False, None)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("d", [96, 1001])
def test_norm_forms(post, gate, pad, d):
    rng = np.random.default_rng([31, d, pad])
    check_norm(rng, 70, d, pad == 3, post, gate, pad=pad)
    check_norm(rng, 70, d, pad != 3, post, gate, pad=pad, in_place=True, offset=1.0)


def test_norm_without_a_block_output():
    rng = np.random.default_rng(32)
    for d in (5, 3584):
        check_norm(rng, 4, d, False, False, None, with_x=False)
        check_norm(rng, 4, d, True, False, None, with_x=False, pad=8)


def test_norm_eps_and_sizes():
    rng = np.random.default_rng(33)
    check_norm(rng, 2, 256, True, True, None, eps=0.0)
    check_norm(rng, 2, 256, True, True, None, eps=0.5)
    check_norm(rng, 2, 256, False, True, None, size=1e-12)
    check_norm(rng, 2, 256, True, True, "channel", size=1e12)
    z = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")  # a row of zeros stays zero
    y, r = w4.w4_residual_norm(z, z, z[0] + 1, w_post=z[0] + 1)
    assert not y.any() and not r.any()


def test_norm_pointers_off_the_16_byte_grid():
    rng = np.random.default_rng(34)
    T, d = 5, 200
    base = [bf16(rng.normal(size=(T, 256))).cuda() for _ in range(2)]
    w = bf16(rng.normal(size=d)).cuda()
    want = w4.w4_residual_norm(base[0][:, 8:208].contiguous(), base[1][:, 8:208].contiguous(), w)
    for at in (1, 3, 4):
        x, r = (torch.empty((T, 256), dtype=torch.bfloat16, device="cuda")[:, at:at + d]
                for _ in range(2))
        x.copy_(base[0][:, 8:208])
        r.copy_(base[1][:, 8:208])
        got = w4.w4_residual_norm(x, r, w)
        assert torch.equal(got[1], want[1])
        assert (got[0].float() - want[0].float()).abs().max() <= want[0].float().abs().max() / 128


def test_norm_many_rows():
    rng = np.random.default_rng(35)
    check_norm(rng, 3000, 40, False, True, "channel")


# ------------------------------------------------------------------------------- streams, graphs


@contextlib.contextmanager
def other_stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        yield s
    torch.cuda.current_stream().wait_stream(s)


def test_another_stream_and_a_graph():
    """A step (append, then attention, then the norm) runs on the current stream, and in a graph
    whose replays see new lengths and inputs."""
    rng = np.random.default_rng(40)
    H, n_kv, D, page, B = 8, 2, 64, 16, 3
    cache = Paged(rng, [2000, 900, 40], page, n_kv, D)
    cache.fill(rng, [range(2000), range(900), range(40)])
    k0, v0 = cache.k.clone(), cache.v.clone()
    qkv = bf16(rng.normal(size=(B, (H + 2 * n_kv) * D))).cuda()
    res = torch.zeros((B, H * D), dtype=torch.float32, device="cuda")
    w = torch.ones(H * D, dtype=torch.bfloat16, device="cuda")
    f = w4.w4_rope_frequencies(D)[0].cuda()
    need = w4.w4_attn_decode_work_bytes(H, *cache.args())
    work = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def step():
        q = w4.w4_rope_append(qkv, H, *cache.args(), f)
        y = w4.w4_attn_decode(q, *cache.args(), work=work)
        return w4.w4_residual_norm(y, res, w, w_post=w)

    def fresh(lens, seed):
        cache.k.copy_(k0)
        cache.v.copy_(v0)
        cache.d_len.copy_(torch.tensor(lens, dtype=torch.int32))
        qkv.copy_(bf16(np.random.default_rng(seed).normal(size=tuple(qkv.shape))))
        torch.cuda.synchronize()

    fresh([1999, 899, 39], 1)
    want = [t.clone() for t in step()]
    fresh([1999, 899, 39], 1)
    with other_stream():
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i, lens in enumerate([[1999, 899, 39], [1700, 0, 5], [33, 880, 1], [1999, 899, 39]]):
        fresh(lens, i)
        want = [t.clone() for t in step()]
        fresh(lens, i)
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), lens
