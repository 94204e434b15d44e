"""Operators that build, share and cross-read a paged cache against plain implementations
(tests/cache_reference.py), through the public binding.  Attention bounds come from the arithmetic, as
in test_gpu_layer.py: weights rounded to bf16, fp32 sums; whole numbers are equal."""
import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
from tests import cache_reference as plain
from tests import layer_reference as ref
from tests.test_gpu_layer import bf16, close, f64, strided

pytestmark = pytest.mark.gpu

GARBAGE = [-1, -2 ** 31, 2 ** 31 - 1]


def ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype).cuda()


class Batch:
    """Sequences over prefixes in one cache: NaN but for the slots that fill() writes, and garbage in
    every table entry that no position in use needs."""

    def __init__(self, rng, prefix_len, prefix_of, lens, page, n_kv, D, order="slot", gap=0, cols=None,
                 prefix_cols=None):
        self.page, self.n_kv, self.D = page, n_kv, D
        cols = max([-(-n // page) for n in lens] + [1]) if cols is None else cols
        pcols = max([-(-n // page) for n in prefix_len] + [1]) if prefix_cols is None else prefix_cols
        self.lens, self.prefix_len, self.prefix_of = (np.asarray(x, dtype=np.int64) for x in
                                                      (lens, prefix_len, prefix_of))
        cut = [min(max(prefix_len[g], 0), pcols * page) if 0 <= g < len(prefix_len) else 0
               for g in prefix_of]
        own = [range(c // page, min(-(-n // page), cols)) if n > c else range(0)
               for c, n in zip(cut, lens)]
        pre = [range(min(-(-n // page), pcols)) for n in prefix_len]
        total = sum(map(len, own)) + sum(map(len, pre)) + 2
        where = iter(rng.permutation(total))
        self.table = rng.choice(GARBAGE + [total], size=(len(lens), cols))
        self.prefix_table = rng.choice(GARBAGE + [total], size=(len(prefix_len), pcols))
        for table, uses in ((self.table, own), (self.prefix_table, pre)):
            for b, use in enumerate(uses):
                for col in use:
                    table[b, col] = next(where)
        shape = (total, page, n_kv, D + gap) if order == "slot" else (total, n_kv, page, D + gap)

        def buffer():
            t = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            return (t if order == "slot" else t.permute(0, 2, 1, 3))[..., :D]
        self.k, self.v = buffer(), buffer()
        self.at = plain.places(self.table, self.prefix_table, prefix_of, prefix_len, page)

    def fill(self, rng, slots, kscale=1.0):
        slots = torch.from_numpy(np.unique(slots)).cuda()
        for t, s in ((self.k, kscale), (self.v, 1.0)):
            new = bf16(s * rng.normal(size=(len(slots), self.n_kv, self.D))).cuda()
            t[slots // self.page, slots % self.page] = new

    def args(self):
        return (self.k, self.v, ints(self.table), ints(self.lens))

    def prefixes(self):
        return ints(self.prefix_of), ints(self.prefix_table), ints(self.prefix_len)


def seen_slots(batch, q_start, window, sinks, cross=False):
    out = [np.zeros(0, dtype=np.int64)]
    cap = batch.at.shape[1]
    for _, b, pos in ref.rows_of(q_start, batch.lens, cap):
        last = min(max(int(batch.lens[b]), 0), cap) - 1
        out.append(batch.at[b][ref.visible(last if cross else pos, window, sinks)])
    return np.concatenate(out)


def check_rows(call, batch, q, q_start, H, scale, window, sinks, cross, extra=0, pad=0, bits=8):
    """y and lse of a call against the definition; `extra` rows of q behind the last sequence's."""
    T, D = q.shape[0], batch.D
    n = T - extra
    mark = torch.full((T, H * D + pad), 7.0, device="cuda")[:, :H * D]
    y, lse = call(w4.W4_OUT_F32, mark)
    y16, lse16 = call(w4.W4_OUT_BF16, None)
    torch.cuda.synchronize()
    k, v = f64(batch.k), f64(batch.v)
    wy, wl, a, ds, count = plain.attention(f64(q)[:n].reshape(n, -1), k, v, batch.at, batch.lens,
                                           q_start, H, float(np.float32(scale)), window, sinks,
                                           cross)
    close(y[:n].reshape(n, H, D), wy, ref.attention_bound(a, ds, count, bits), "y")
    assert torch.equal(y16[:n], y[:n].to(torch.bfloat16)), "bf16 output is not the rounded fp32 one"
    got, empty = f64(lse)[:n], np.isinf(wl)
    assert np.array_equal(np.isneginf(got), empty)
    with np.errstate(invalid="ignore"):
        assert np.all(np.abs(got - wl)[~empty] <= (2 * ds + 2.0 ** -20 + (count + 4) * ref.F32 * 2
                                                   + 2.0 ** -22 * np.abs(wl))[~empty])
    assert torch.equal(lse[:n], lse16[:n])
    assert torch.all(y[:n].reshape(n, H, D)[torch.from_numpy(empty).cuda()] == 0)
    assert torch.all(y[n:] == 7.0), "a row of no sequence was written"
    return y


def share(rng, prefix_len, prefix_of, lens, nq, H, n_kv, D, page, window=0, sinks=0, kscale=1.0,
          pad=0, scale=None, extra=0, **kw):
    batch = Batch(rng, prefix_len, prefix_of, lens, page, n_kv, D, **kw)
    counts = [1] * len(lens) if nq is None else nq
    q_start = np.concatenate([[0], np.cumsum(counts)])
    batch.fill(rng, seen_slots(batch, q_start, window, sinks), kscale)
    q = bf16(2.0 * rng.normal(size=(q_start[-1] + extra, H * D))).cuda()
    q = strided(q, pad) if pad else q
    scale = D ** -0.5 if scale is None else scale
    starts = None if nq is None else ints(q_start)

    def call(dt, out):
        return w4.w4_attn_shared(q, *batch.args(), *batch.prefixes(), q_start=starts, scale=scale,
                                 window=window, sinks=sinks, out_dtype=dt, out=out, want_lse=True)
    y = check_rows(call, batch, q, q_start, H, scale, window, sinks, False, extra, pad)
    return batch, q, starts, y


# two prefixes in use, one of no key, one that nobody has, sequences without one and without keys;
# own keys from none to more than a tile
PREFIX_LEN = [100, 0, 37, 260]
PREFIX_OF = [0, 3, -1, 0, 3, 1, 0, 7, 3, 3, -1, 0, -2 ** 31, 2 ** 31 - 1, 3]
OWN = [1, 5, 40, 64, 65, 17, 0, 130, 200, 1, 0, 28, 3, 70, 0]
LENS = [n + (PREFIX_LEN[g] if 0 <= g < 4 and n else 0) for g, n in zip(PREFIX_OF, OWN)]
HEADS = [(28, 4, 128), (8, 8, 64), (16, 2, 256), (3, 1, 80), (32, 1, 128), (5, 5, 8), (9, 3, 192),
         (1, 1, 136), (17, 1, 64)]


@pytest.mark.parametrize("H,n_kv,D", HEADS)
@pytest.mark.parametrize("page", [16, 64])
def test_shared_lengths_and_heads(H, n_kv, D, page):
    rng = np.random.default_rng([1, H, D, page])
    share(rng, PREFIX_LEN, PREFIX_OF, LENS, None, H, n_kv, D, page)


@pytest.mark.parametrize("H,n_kv,D", HEADS)
def test_shared_several_tokens(H, n_kv, D):
    rng = np.random.default_rng([2, H, D])
    nq = [1, 5, 2, 33, 0, 9, 0, 4, 130, 1, 0, 7, 1, 16, 3]
    share(rng, PREFIX_LEN, PREFIX_OF, LENS, nq, H, n_kv, D, 16, extra=3)


@pytest.mark.parametrize("nq", [None, [3, 1, 40, 2, 9]])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (7, 3), (33, 4), (64, 64), (65, 70),
                                          (128, 1), (300, 5), (20, 200), (20, 320), (1000, 5),
                                          (20, 10 ** 12), (10 ** 12, 3)])
def test_shared_windows_and_sinks(nq, window, sinks):
    rng = np.random.default_rng([3, window, sinks])
    lens = [310, 250, 300, 90, 513]
    share(rng, [190, 300], [0, 0, 1, -1, 1], lens, nq, 14, 2, 128, 32, window, sinks)
    share(rng, [64, 301], [0, 0, 1, -1, 1], lens, nq, 4, 4, 80, 16, window, sinks)


@pytest.mark.parametrize("nq", [None, [30, 0, 3, 1]])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 128, 1024])
@pytest.mark.parametrize("order,gap", [("slot", 0), ("head", 0), ("slot", 8), ("head", 24)])
def test_shared_page_sizes_and_layouts(nq, page, order, gap):
    rng = np.random.default_rng([4, page, gap])
    for window, sinks, pad in ((0, 0, 8), (50, 3, 16)):
        share(rng, [77, 130], [1, 0, 1, 0], [190, 0, 131, 99], nq, 6, 2, 64, page, window, sinks,
              order=order, gap=gap, pad=pad)


@pytest.mark.parametrize("nq", [None, [5, 70, 3, 100]])
def test_shared_rows_inside_the_prefix(nq):
    """kv_len below, at and just above the prefix' length; rows before the cache begins."""
    rng = np.random.default_rng(5)
    share(rng, [150], [0, 0, 0, 0], [150, 60, 151, 90], nq, 8, 2, 128, 16)
    share(rng, [150], [0, 0, 0, 0], [150, 1, 151, 0], nq, 4, 2, 64, 16, 40, 5)


@pytest.mark.parametrize("nq", [None, [4, 30]])
def test_shared_lengths_the_tables_cannot_hold(nq):
    rng = np.random.default_rng(6)
    share(rng, [1000, -5], [0, 1], [90, 70], nq, 4, 2, 64, 16, prefix_cols=4)
    share(rng, [50], [0, 0], [1000, -7], nq, 4, 2, 64, 16, cols=5)
    share(rng, [500], [0, 0], [1000, 60], nq, 4, 2, 64, 16, cols=5)


@pytest.mark.parametrize("nq", [None, [3, 1, 40]])
def test_shared_extreme_scores(nq):
    rng = np.random.default_rng(7)
    for kscale, scale in ((60.0, None), (1.0, 0.0), (1.0, 1e-30), (1e18, 1e-20)):
        share(rng, [100], [0, 0, -1], [200, 164, 129], nq, 8, 2, 128, 16, kscale=kscale, scale=scale)


def test_shared_long_and_split():
    rng = np.random.default_rng(8)
    share(rng, [9000], [0, 0, 0], [9100, 9001, 12000], None, 7, 1, 128, 64)
    share(rng, [5000, 3000], [0, 1, 0, 1, -1], [5003, 3100, 7000, 3001, 2500], [3, 2, 40, 1, 9], 8, 2,
          64, 16)
    share(rng, [6000], [0] * 4, [8000, 6001, 9000, 6400], None, 4, 2, 256, 128, 4500, 70)


@pytest.mark.parametrize("B,prefixes", [(65, 3), (300, 70), (1500, 1), (1100, 256)])
def test_shared_many_sequences(B, prefixes):
    rng = np.random.default_rng([9, B, prefixes])
    plen = rng.integers(0, 80, prefixes)
    of = rng.integers(-1, prefixes, B)
    lens = rng.integers(0, 30, B)
    lens = [int(n + (plen[g] if g >= 0 and n else 0)) for n, g in zip(lens, of)]
    share(rng, plen.tolist(), of.tolist(), lens, None, 2, 1, 32, 16)
    nq = [int(rng.integers(0, 3)) for _ in lens]
    share(rng, plen.tolist(), of.tolist(), lens, nq, 2, 1, 32, 16, extra=1)


def test_shared_agrees_with_the_other_forms():
    """With the prefix' whole pages in every table row, the forms without sharing say the same."""
    rng = np.random.default_rng(10)
    lens, P, page = [300, 257, 290], 256, 16
    batch, q, _, y = share(rng, [P], [0, 0, 0], lens, None, 28, 4, 128, page)
    table = batch.table.copy()
    table[:, :P // page] = batch.prefix_table[0, :P // page]
    kv = (batch.k, batch.v, ints(table), ints(lens))
    one = w4.w4_attn_decode(q, *kv, out_dtype=w4.W4_OUT_F32)
    assert (y - one).abs().max().item() <= 2.0 ** -7 * 5
    none = w4.w4_attn_shared(q, *kv, ints([-1] * 3), ints(batch.prefix_table), ints([P]),
                             out_dtype=w4.W4_OUT_F32)
    assert (none - one).abs().max().item() <= 2.0 ** -7 * 5


def test_shared_values_that_are_not_finite_reach_only_rows_that_see_them():
    """Values of the prefix and of a sequence's own keys, hidden from some rows by the mask."""
    rng = np.random.default_rng(11)
    nq = [20, 1, 30, 2]
    lens = [110, 201, 290, 77]
    batch, q, starts, y0 = share(rng, [200], [0, 0, 0, -1], lens, nq, 4, 2, 64, 16, 60, 4)

    def run():
        return w4.w4_attn_shared(q, *batch.args(), *batch.prefixes(), q_start=starts, window=60,
                                 sinks=4, out_dtype=w4.W4_OUT_F32).reshape(-1, 4, 64)
    was = run()
    rows = [(t, b, p, set(ref.visible(p, 60, 4).tolist())) for t, b, p in
            ref.rows_of(np.concatenate([[0], np.cumsum(nq)]), lens, batch.at.shape[1])]
    for value in (float("inf"), float("-inf"), float("nan")):
        for b, j in ((0, 100), (0, 3), (0, 95), (2, 230), (3, 70)):
            slot = int(batch.at[b, j])
            keep = batch.v[slot // 16, slot % 16].clone()
            batch.v[slot // 16, slot % 16, 1, 5] = value
            got = run()
            batch.v[slot // 16, slot % 16] = keep
            for t, b1, _, seen in rows:
                sees = any(int(batch.at[b1, i]) == slot for i in seen)
                x = got[t, 2:, 5]
                ok = torch.isnan(x).all() if value != value else (x == value).all()
                assert bool(ok) == sees, (value, b, j, t)
                x[:] = was[t, 2:, 5]
            assert torch.equal(got, was)


@pytest.mark.parametrize("form", [None, [40, 1, 5, 2]])
def test_shared_is_deterministic_and_replays(form):
    """Five calls alike; then a graph whose lengths, tables and prefixes change between replays."""
    rng = np.random.default_rng(12)
    lens = [4500, 2100, 2077, 900]
    batch, q, starts, y = share(rng, [2000, 600], [0, 0, 0, 1], lens, form, 8, 2, 128, 16)
    k, v, table, n = batch.args()
    of, ptable, plen = batch.prefixes()

    def run():
        return w4.w4_attn_shared(q, k, v, table, n, of, ptable, plen, q_start=starts)
    first = run().clone()
    for _ in range(5):
        assert torch.equal(run(), first)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = run()
    torch.cuda.default_stream().wait_stream(side)
    for change in range(4):
        if change == 1:
            n.copy_(ints([4400, 2050, 0, 700]))
        if change == 2:
            plen.copy_(ints([1999, 0]))
            table[:3, 2000 // 16 - 1] = ptable[0, 2000 // 16 - 1]
            table[3] = table[3].where(torch.arange(table.shape[1]).cuda() >= 600 // 16,
                                      ptable[1].new_zeros(1))
            k.nan_to_num_()
            v.nan_to_num_()
        if change == 3:
            of.copy_(ints([-1, 0, 0, 5]))
            table.clamp_(0, k.shape[0] - 1)
        graph.replay()
        want = run()
        assert torch.equal(out, want), change
        assert torch.isfinite(out.float()).all()


def test_shared_work_buffers_and_streams():
    """A workspace of the size asked for, filled with NaN; two calls at once on two streams, each with
    its own."""
    rng = np.random.default_rng(13)
    batch, q, _, y = share(rng, [3000], [0, 0], [3300, 3001], None, 8, 2, 128, 64)
    args = (*batch.args(), *batch.prefixes())
    need = w4.w4_attn_shared_work_bytes(2, 8, *args)
    works = [torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    outs = []
    for s, w in zip(streams, works):
        with torch.cuda.stream(s):
            outs.append([w4.w4_attn_shared(q, *args, out_dtype=w4.W4_OUT_F32, work=w[:need])
                         for _ in range(10)])
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(x, y) for x in got)
    assert all(torch.all(w[need:] == 255) for w in works)
    if need:
        with pytest.raises(w4.W4Error, match="status 5"):
            w4.w4_attn_shared(q, *args, work=works[0][:need - 1])
        with pytest.raises(w4.W4Error, match="status 4"):
            w4.w4_attn_shared(q, *args, work=works[0][4:])


def test_shared_offsets_past_32_bits():
    """Pages 2^28 elements apart: prefix pages beyond element 2^31 of the cache."""
    rng = np.random.default_rng(14)
    n_kv, D, page, pages, H, B = 2, 64, 16, 12, 4, 3
    stride = 1 << 28

    def buffer():
        flat = torch.empty((pages - 1) * stride + page * n_kv * D, dtype=torch.bfloat16,
                           device="cuda")
        return flat.as_strided((pages, page, n_kv, D), (stride, n_kv * D, D, 1))
    small = [bf16(rng.normal(size=(pages, page, n_kv, D))).cuda() for _ in range(2)]
    k, v = buffer(), buffer()
    k.copy_(small[0])
    v.copy_(small[1])
    order = rng.permutation(pages)
    ptable, table = ints(order[None, :6]), ints(np.concatenate([np.zeros((3, 5)),
                                                                order[6:].reshape(3, 2)], 1))
    q = bf16(rng.normal(size=(B, H * D))).cuda()
    rest = (table, ints([111, 100, 90]), ints([0, 0, 0]), ptable, ints([85]))
    assert torch.equal(w4.w4_attn_shared(q, k, v, *rest), w4.w4_attn_shared(q, *small, *rest))
    starts = ints([0, 3])
    cross = (ptable, ints([90]))
    assert torch.equal(w4.w4_attn_cross(q, k, v, *cross, starts),
                       w4.w4_attn_cross(q, *small, *cross, starts))


# -------------------------------------------------------------------------------- cross attention


def crossed(rng, lens, nq, H, n_kv, D, page, kscale=1.0, pad=0, scale=None, extra=0, **kw):
    batch = Batch(rng, [0], [-1] * len(lens), lens, page, n_kv, D, **kw)
    counts = [1] * len(lens) if nq is None else nq
    q_start = np.concatenate([[0], np.cumsum(counts)])
    batch.fill(rng, seen_slots(batch, q_start, 0, 0, True), kscale)
    q = bf16(2.0 * rng.normal(size=(q_start[-1] + extra, H * D))).cuda()
    q = strided(q, pad) if pad else q
    scale = D ** -0.5 if scale is None else scale
    starts = None if nq is None else ints(q_start)

    def call(dt, out):
        return w4.w4_attn_cross(q, *batch.args(), q_start=starts, scale=scale, out_dtype=dt, out=out,
                                want_lse=True)
    y = check_rows(call, batch, q, q_start, H, scale, 0, 0, True, extra, pad)
    return batch, q, starts, y


CROSS_LENS = [1, 2, 15, 17, 0, 64, 65, 130, 300, 40]


@pytest.mark.parametrize("nq", [None, [3, 64, 65, 1, 5, 0, 130, 7, 2, 33]])
@pytest.mark.parametrize("H,n_kv,D", HEADS)
def test_cross_lengths_and_heads(nq, H, n_kv, D):
    rng = np.random.default_rng([20, H, D])
    crossed(rng, CROSS_LENS, nq, H, n_kv, D, 16, extra=0 if nq is None else 2)
    crossed(rng, CROSS_LENS[:4], None if nq is None else nq[:4], H, n_kv, D, 64)


@pytest.mark.parametrize("nq", [None, [150, 0, 10]])
@pytest.mark.parametrize("page", [1, 4, 128, 512])
@pytest.mark.parametrize("order,gap", [("slot", 0), ("head", 0), ("slot", 8), ("head", 24)])
def test_cross_page_sizes_and_layouts(nq, page, order, gap):
    rng = np.random.default_rng([21, page, gap])
    crossed(rng, [150, 0, 77], nq, 6, 2, 64, page, order=order, gap=gap, pad=8)


@pytest.mark.parametrize("nq", [None, [3, 1, 40]])
def test_cross_extremes(nq):
    rng = np.random.default_rng(22)
    for kscale, scale in ((60.0, None), (1.0, 0.0), (1.0, 1e-30), (1e18, 1e-20)):
        crossed(rng, [200, 64, 129], nq, 8, 2, 128, 16, kscale=kscale, scale=scale)
    crossed(rng, [1000, -7, 20], nq, 4, 2, 64, 16, cols=5)


def test_cross_few_rows_over_many_states_and_the_reverse():
    rng = np.random.default_rng(23)
    crossed(rng, [5000, 33], [3, 2], 8, 2, 128, 64)
    crossed(rng, [9000], [17], 7, 1, 64, 16)
    crossed(rng, [3, 1], [700, 300], 8, 2, 128, 16)
    crossed(rng, [6000, 4000], None, 4, 2, 256, 32)
    crossed(rng, [int(x) for x in rng.integers(0, 40, 200)], [int(x) for x in rng.integers(0, 4, 200)],
            2, 1, 32, 16, extra=1)


# sequences whose rows make more workgroups than two for each of 256 compute units, with 16 heads
MANY_ROWS = [500, 300, 0, 431, 17, 640, 129, 128, 350, 700]
MANY_KEYS = [77, 130, 50, 64, 200, 1, 300, 0, 65, 128]


@pytest.mark.parametrize("D,page", [(64, 64), (64, 16), (64, 4), (40, 64), (32, 8)])
def test_cross_of_many_rows_at_small_head_sizes(D, page):
    crossed(np.random.default_rng([24, D, page]), MANY_KEYS, MANY_ROWS, 16, 16, D, page, extra=3)


@pytest.mark.parametrize("page", [64, 16, 4])
@pytest.mark.parametrize("call", [w4.w4_attn_cross, w4.w4_attn_prefill])
@pytest.mark.parametrize("case", ["plain", "far", "inf"])
def test_many_rows_agree_with_each_sequence_alone(call, page, case):
    """A batch of many workgroups at 64 dims against calls of few, bit for bit; with scores far from 0
    and values that are not finite too, which take a second pass."""
    rng = np.random.default_rng([25, page])
    H, D = 16, 64
    lens = [max(n, m) + 20 for n, m in zip(MANY_KEYS, MANY_ROWS)]
    lens = [min(n, 448) for n in lens]
    rows = [min(m, n) for m, n in zip(MANY_ROWS, lens)]
    rows[4] = 400
    lens[4] = 440
    batch = Batch(rng, [0], [-1] * len(lens), lens, page, H, D, cols=448 // page)
    starts = np.concatenate([[0], np.cumsum(rows)])
    assert (starts[-1] // 128 + len(rows)) * H > 512
    batch.fill(rng, seen_slots(batch, starts, 0, 0, True), 1e18 if case == "far" else 1.0)
    if case == "inf":
        for b, pos, value in ((0, 5, float("inf")), (3, 60, float("nan")), (9, 100, -float("inf"))):
            slot = int(batch.at[b][pos])
            batch.v[slot // page, slot % page, 3, 7:40] = value
    q = bf16(2.0 * rng.normal(size=(starts[-1], H * D))).cuda()
    k, v, table, kv_len = batch.args()
    y = call(q, k, v, table, kv_len, ints(starts), out_dtype=w4.W4_OUT_F32)
    for b in range(len(rows)):
        one = slice(int(starts[b]), int(starts[b + 1]))
        if rows[b] == 0:
            continue
        alone = call(q[one], k, v, table[b:b + 1], kv_len[b:b + 1], ints([0, rows[b]]),
                     out_dtype=w4.W4_OUT_F32)
        assert torch.equal(torch.nan_to_num(alone, nan=12345.0), torch.nan_to_num(y[one], nan=12345.0))
        if case == "inf":
            assert torch.isfinite(alone).all() == (b not in (0, 3, 9))


def test_cross_over_a_dense_array_of_states():
    """[B][length][heads][D] seen as pages in order; rows of one sequence are independent beams."""
    rng = np.random.default_rng(24)
    B, L, H, D, beams = 3, 96, 4, 64, 5
    k, v = (bf16(rng.normal(size=(B, L, H, D))).cuda() for _ in range(2))
    q = bf16(rng.normal(size=(B * beams, H * D))).cuda()
    n = [96, 50, 1]
    pages = [x.view(B * L // 32, 32, H, D) for x in (k, v)]
    table = torch.arange(B * L // 32, dtype=torch.int32, device="cuda").view(B, -1)
    y = w4.w4_attn_cross(q, *pages, table, ints(n), ints(np.arange(B + 1) * beams),
                         out_dtype=w4.W4_OUT_F32)
    for b in range(B):
        kk, vv = (x[b, :n[b]].double().transpose(0, 1) for x in (k, v))
        qq = q[b * beams:][:beams].double().view(beams, H, D).transpose(0, 1)
        p = torch.softmax(qq @ kk.transpose(1, 2) * D ** -0.5, -1)
        want = (p @ vv).transpose(0, 1).reshape(beams, -1)
        size = (p @ vv.abs()).transpose(0, 1).reshape(beams, -1)
        got = y[b * beams:][:beams].double()
        assert ((got - want).abs() <= (ref.BF16 + 2.0 ** -14) * size + 1e-30).all()


def test_cross_values_that_are_not_finite():
    rng = np.random.default_rng(25)
    batch, q, starts, _ = crossed(rng, [130, 70], [20, 3], 4, 2, 64, 16)

    def run():
        return w4.w4_attn_cross(q, *batch.args(), starts, out_dtype=w4.W4_OUT_F32).reshape(-1, 4, 64)
    was = run()
    for value in (float("inf"), float("-inf"), float("nan")):
        slot = int(batch.at[0, 129])
        keep = batch.v[slot // 16, slot % 16].clone()
        batch.v[slot // 16, slot % 16, 1, 5] = value
        got = run()
        batch.v[slot // 16, slot % 16] = keep
        x = got[:20, 2:, 5]
        assert bool(torch.isnan(x).all() if value != value else (x == value).all())
        x[:] = was[:20, 2:, 5]
        assert torch.equal(got, was)


def test_cross_replays():
    rng = np.random.default_rng(26)
    batch, q, starts, _ = crossed(rng, [3000, 70, 20], [4, 4, 4], 8, 2, 64, 16)
    k, v, table, n = batch.args()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        w4.w4_attn_cross(q, k, v, table, n, starts)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = w4.w4_attn_cross(q, k, v, table, n, starts)
    torch.cuda.default_stream().wait_stream(side)
    for lens, rows in (([3000, 70, 20], [0, 4, 8, 12]), ([1, 0, 20], [0, 0, 11, 12]),
                       ([2500, 64, 7], [0, 10, 10, 12])):
        n.copy_(ints(lens))
        starts.copy_(ints(rows))
        graph.replay()
        assert torch.equal(out, w4.w4_attn_cross(q, k, v, table, n, starts))


# ------------------------------------------------------------------------------------- the tables


class Pool:
    """A page table with spans, and a ring of the other pages."""

    def __init__(self, rng, held, cols, page, free, ring_size=None, begins=None, head=None):
        B = len(held)
        begins = [0] * B if begins is None else begins
        self.kv_len = np.asarray(held)
        self.spans = np.array([[x, max(x, -(-n // page))] for x, n in zip(begins, held)])
        total = int((self.spans[:, 1] - self.spans[:, 0]).sum()) + free
        order = rng.permutation(total).astype(np.int64)
        self.table = rng.choice(GARBAGE, size=(B, cols))
        at = 0
        for b, (x, y) in enumerate(self.spans):
            self.table[b, x:y] = order[at:at + y - x]
            at += y - x
        R = total if ring_size is None else ring_size
        self.ring = rng.choice(GARBAGE, size=R)
        h = int(rng.integers(R)) if head is None else head
        self.ring[(h + np.arange(free)) % R] = order[at:]
        self.state = np.array([h, free, 5])
        self.page = page


def tables_step(pool, n_new, T, in_place=False, pad=0):
    """One call against the definition; the pool goes on with the library's results."""
    wide = torch.full((pool.table.shape[0], pool.table.shape[1] + pad), 77, dtype=torch.int32,
                      device="cuda")
    table = wide[:, :pool.table.shape[1]]
    table.copy_(ints(pool.table))
    kv, spans, ring, state = ints(pool.kv_len), ints(pool.spans), ints(pool.ring), ints(pool.state)
    before = [x.clone() for x in (kv, spans, state)]
    got = w4.w4_batch_tables(kv, ints(n_new), spans, table, pool.page, ring, state, T, in_place)
    torch.cuda.synchronize()
    want = plain.batch_tables(pool.kv_len, n_new, pool.spans, pool.table, pool.page, pool.ring,
                              pool.state, T)
    names = ("q_start", "slots", "seqs", "positions", "kv_len", "spans", "ring_state")
    for name, x, y in zip(names, got, want):
        assert np.array_equal(x.cpu().numpy(), y), name
    assert np.array_equal(table.cpu().numpy(), pool.table), "page_table"
    assert np.array_equal(ring.cpu().numpy(), pool.ring), "ring"
    assert torch.all(wide[:, pool.table.shape[1]:] == 77)
    for x, was in zip((kv, spans, state), before):
        assert in_place or torch.equal(x, was)
    if in_place:
        assert all(x is y for x, y in zip(got[4:], (kv, spans, state)))
    pool.kv_len, pool.spans, pool.state = (x.cpu().numpy().astype(np.int64) for x in got[4:])
    return got


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [1, 3, 63, 64, 65, 1023, 1024, 1025, 2500])
def test_tables_of_many_sequences(B, in_place):
    rng = np.random.default_rng([30, B])
    page = 16
    pool = Pool(rng, rng.integers(0, 100, B), 12, page, 12 * B)
    for step in range(3):
        n_new = rng.integers(0, 25, B) if step != 1 else np.where(rng.random(B) < 0.3, -1, 1)
        tables_step(pool, n_new, int(np.maximum(n_new, 0).sum()) + step, in_place, pad=step)


@pytest.mark.parametrize("page", [1, 2, 64, 1024, 32768])
def test_tables_page_sizes(page):
    rng = np.random.default_rng([31, page])
    held = [0, 1, page - 1, page, page + 1, 3 * page, 5]
    pool = Pool(rng, held, 9, page, 60)
    tables_step(pool, [1, 0, 1, 1, page, 2 * page + 1, -1], 3 * page + 10)
    tables_step(pool, [page, 2, 1, 0, -1, 1, 1], page + 9, True)


@pytest.mark.parametrize("in_place", [False, True])
def test_tables_of_long_prompts(in_place):
    """Rows and entries of many workgroups."""
    rng = np.random.default_rng(32)
    pool = Pool(rng, [0, 5000, 17, 0, 640], 2000, 16, 4000)
    n_new = [9000, 1, 12345, 0, 20011]
    tables_step(pool, n_new, sum(n_new) + 77, in_place)
    tables_step(pool, [-1, -1, 5, 3, -1], 8, in_place)
    tables_step(pool, [30000, 7, -5, 0, 100], 30107, in_place)


def test_tables_when_pages_run_out():
    """Entries and rows without a page are -1 and counted; pages that come back serve the next call."""
    rng = np.random.default_rng(33)
    pool = Pool(rng, [30, 0, 16, 3], 10, 16, 5)
    got = tables_step(pool, [40, 50, 1, 1], 92)
    assert got[6].tolist()[1:] == [0, 3]  # 3 + 4 + 1 entries, 5 pages
    assert (got[1] == -1).sum().item() == 18 + 1
    rng = np.random.default_rng(34)
    pool = Pool(rng, [30, 20], 10, 16, 0)
    tables_step(pool, [1, 1], 2)  # the last slots of pages they have
    tables_step(pool, [-1, 40], 40)  # pages that come back serve the next call
    tables_step(pool, [0, 1], 1)


def test_tables_of_a_step_made_again():
    """A step that ran out is made again from the lengths, spans and ring that it had: after a call in
    which another sequence gave up its pages, and after pages were put into the ring. No page is lost
    or given out twice."""
    rng = np.random.default_rng(40)
    pool = Pool(rng, [30, 20, 0, 64, 5], 10, 16, 2)
    n_new = [40, -1, 33, 1, 1]  # 3 + 0 + 3 + 1 + 0 pages of 2; 2 come back
    was = [x.copy() for x in (pool.kv_len, pool.spans, pool.state)]
    assert tables_step(pool, n_new, 75)[6].tolist()[1:] == [2, 5]
    pool.kv_len, pool.spans, pool.state = (x.copy() for x in was)
    tables_step(pool, [0, 0, 0, -1, 0], 0)  # 4 pages of sequence 3
    assert pool.state.tolist()[1:] == [6, 0]
    n_new[3] = 0
    was = [x.copy() for x in (pool.kv_len, pool.spans, pool.state)]
    n_new[4] = 28  # two pages more
    assert tables_step(pool, n_new, 101)[6].tolist()[1:] == [2, 2]
    pool.kv_len, pool.spans, pool.state = (x.copy() for x in was)
    extra = len(pool.ring) - int(pool.state[1])
    held = {int(pool.table[b, j]) for b in range(5) for j in range(*pool.spans[b])}
    free = set(pool.ring[(pool.state[0] + np.arange(pool.state[1])) % len(pool.ring)].tolist())
    assert len(free) == 6 and not free & held and extra >= 2
    new = [1000, 1001]
    pool.ring[(pool.state[0] + pool.state[1] + np.arange(2)) % len(pool.ring)] = new
    pool.state[1] += 2
    got = tables_step(pool, n_new, 101)
    assert got[6].tolist()[2] == 0 and (got[1][:int(got[0][-1])] >= 0).all()
    used = [int(pool.table[b, j]) for b in range(5) for j in range(*pool.spans[b])]
    left = pool.ring[(pool.state[0] + np.arange(pool.state[1])) % len(pool.ring)].tolist()
    assert sorted(used + left) == sorted(held | free | set(new))


def test_tables_narrower_than_the_sequences():
    """Tokens past the last column: no page, no entry, slot -1."""
    rng = np.random.default_rng(35)
    pool = Pool(rng, [40, 64, 0], 4, 16, 9)
    got = tables_step(pool, [30, 2, 64], 96)
    assert got[6].tolist()[2] == 0 and (got[1] == -1).sum().item() == 6 + 2


def test_tables_rows_beyond_T():
    """Rows that T does not hold: q_start ends at T."""
    rng = np.random.default_rng(36)
    pool = Pool(rng, [3, 10, 0, 7], 8, 16, 30)
    got = tables_step(pool, [20, 30, 5, 1], 33)
    assert got[0].tolist() == [0, 20, 33, 33, 33]
    pool = Pool(rng, [3, 10], 8, 16, 30)
    tables_step(pool, [0, -1], 0)


def test_tables_after_prefixes():
    """Sequences whose first pages are a prefix': entries below the span are left alone."""
    rng = np.random.default_rng(37)
    pool = Pool(rng, [40, 100, 33], 12, 16, 30, begins=[2, 6, 0])
    pool.spans[0] = [2, 2]  # begins after 40 shared keys: the page they end in is not its own
    tables_step(pool, [1, 30, 2], 33)
    tables_step(pool, [-1, -1, 1], 1)
    assert pool.state[1] == len(pool.ring) - (pool.spans[:, 1] - pool.spans[:, 0]).sum() - 1


def test_tables_ring_wraps_and_overflows():
    rng = np.random.default_rng(38)
    pool = Pool(rng, [100, 50, 0], 12, 16, 9, ring_size=11, head=7)
    tables_step(pool, [30, -1, 20], 50)  # 2 + 2 pages from places 7, 8, 9, 10; 2 of 4 come back
    assert pool.state.tolist() == [0, 7, 0]
    tables_step(pool, [-1, -1, -1], 0)
    assert pool.state[1] == 11


def test_tables_of_nonsense_stay_in_bounds():
    """Lengths, spans and ring states outside their ranges are cut to them; what lies around every
    buffer is left alone."""
    B, cols, R, T, page = 6, 5, 7, 40, 16
    guard = torch.full((1000,), 123, dtype=torch.int32, device="cuda")

    def carve(at, n):
        return guard[at:at + n]
    kv, n_new, spans = carve(10, B), carve(30, B), carve(50, 2 * B).view(B, 2)
    table, ring, state = carve(100, B * cols).view(B, cols), carve(200, R), carve(220, 3)
    table.fill_(3)
    ring.fill_(4)
    for case in range(4):
        kv.copy_(ints([-5, 2 ** 31 - 1, 70, 81, 0, 9]))
        n_new.copy_(ints([2 ** 31 - 1, 5, -2 ** 31, 1, 2 ** 30, 3]))
        spans.copy_(ints([[-7, 2 ** 31 - 1], [9, 2], [-2 ** 31, 99], [4, 3], [0, 0], [-1, -1]]))
        state.copy_(ints([[2 ** 31 - 1, 2 ** 31 - 1, 0], [-1, -1, 0], [6, 7, 0], [3, 2, 9]][case]))
        got = w4.w4_batch_tables(kv, n_new, spans, table, page, ring, state, T, True)
        torch.cuda.synchronize()
        assert got[0].tolist()[0] == 0 and got[0].max().item() <= T
        assert 0 <= state[0].item() < R and 0 <= state[1].item() <= R
        assert (kv >= 0).all() and (spans >= 0).all() and (spans <= cols).all()
        used = torch.zeros(1000, dtype=torch.bool, device="cuda")
        for at, n in ((10, B), (30, B), (50, 2 * B), (100, B * cols), (200, R), (220, 3)):
            used[at:at + n] = True
        assert torch.all(guard[~used] == 123)


def test_tables_replay_as_sequences_begin_grow_and_end():
    """One recorded step in place, replayed with other requests; beside an eager run of the same."""
    rng = np.random.default_rng(39)
    B, page, T = 5, 4, 12
    pool = Pool(rng, [3, 9, 0, 4, 8], 40, page, 100)
    a = [ints(x) for x in (pool.kv_len, pool.spans, pool.table, pool.ring, pool.state)]
    b = [x.clone() for x in a]
    n_new = ints([0] * B)

    def run(x):
        return w4.w4_batch_tables(x[0], n_new, x[1], x[2], page, x[3], x[4], T, True)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        run([x.clone() for x in a])
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = run(a)
    torch.cuda.default_stream().wait_stream(side)
    for want in ([1, 1, 7, 1, 1], [1, -1, 1, 1, 1], [1, 8, 1, -1, 1], [1, 1, 1, 0, 1], [-1] * B):
        n_new.copy_(ints(want))
        graph.replay()
        eager = run(b)
        for x, y in zip((*outs, *a), (*eager, *b)):
            assert torch.equal(x, y)
    assert a[0].tolist() == [0] * B and a[4].tolist()[1:] == [a[3].shape[0], 0]


# --------------------------------------------------------------------------------- used together


def test_a_batch_begins_after_a_prefix_grows_and_ends():
    """Tables made on the GPU, appends by them, attention over the shared prefix: a prompt that two
    samples and a latecomer share (37 tokens, ending inside a page), against each sequence by itself;
    slots agree with where the appends went."""
    rng = np.random.default_rng(40)
    H, n_kv, D, page, P = 4, 2, 64, 16, 37
    width = (H + 2 * n_kv) * D
    freq = w4.w4_rope_frequencies(D)[0].cuda()
    pages = 40
    k, v = (torch.zeros(pages, page, n_kv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    # row 0 holds the prompt, rows 1 .. 3 its samples
    kv, spans, table = ints([0] * 4), ints([[0, 0]] * 4), ints(np.full((4, 8), -1))
    ring, state = ints(rng.permutation(pages)), ints([11, pages, 0])
    tokens = [bf16(rng.normal(size=(n, width))).cuda() for n in (P, 30, 30, 30)]
    done = [0] * 4

    def step(n_new):
        nonlocal kv, spans, state
        T = sum(max(n, 0) for n in n_new)
        starts, slots, seqs, pos, kv, spans, state = w4.w4_batch_tables(
            kv, ints(n_new), spans, table, page, ring, state, T)
        x = torch.cat([t[i:i + max(n, 0)] for t, i, n in zip(tokens, done, n_new)])
        q = w4.w4_rope_append(x, H, k, v, table, kv, freq, starts)
        for i, n in enumerate(n_new):
            done[i] += max(n, 0)
        values = x.view(T, -1, D)[:, H + n_kv:]
        assert torch.equal(v[slots // page, slots % page], values)
        y = w4.w4_attn_shared(q, k, v, table, kv, ints([-1, 0, 0, 0]), table[:1].clone(),
                              ints([P]), q_start=starts, out_dtype=w4.W4_OUT_F32)
        return q, y, starts.tolist()
    step([P, 0, 0, 0])
    spans[1:] = ints([[P // page, P // page]] * 3)
    kv[1:] = ints([P, P, 0])
    got = {1: [], 2: [], 3: []}
    for n_new in ([0, 1, 5, 0], [0, 3, 1, 0], [0, 1, -1, 0], [0, 2, 0, 20], [0, 1, 0, 1]):
        if n_new[3] == 20:
            kv[3:] = ints([P])
        q, y, starts = step(n_new)
        for b in got:
            got[b] += list(zip(q[starts[b]:starts[b + 1]], y[starts[b]:starts[b + 1]]))
    assert state.tolist()[1:] == [pages - 3 - 1 - 2, 0]
    for b, n in ((1, 8), (2, 6), (3, 21)):
        # the same tokens in a cache of their own, and plain attention over it
        x = torch.cat([tokens[0], tokens[b][:n]])
        k1, v1 = (torch.zeros(8, page, n_kv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        own = (k1, v1, torch.arange(8, dtype=torch.int32, device="cuda")[None], ints([P + n]))
        q1 = w4.w4_rope_append(x, H, *own, freq, ints([0, P + n]))[P:]
        assert torch.equal(torch.stack([q for q, _ in got[b]]), q1)
        wy, _, a, ds, count = ref.attention(f64(q1), f64(k1), f64(v1), np.arange(8)[None], [P + n],
                                            [0, n], H, float(np.float32(D ** -0.5)), 0, 0)
        close(torch.stack([y for _, y in got[b]]).view(n, H, D), wy,
              ref.attention_bound(a, ds, count, 8), f"sequence {b}")
