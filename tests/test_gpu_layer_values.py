"""Values at the edges of the number formats in the operators between a decoder layer's linears:
infinities and NaN in keys, values and residuals, scores far from zero.  The plain forms are those of
tests/layer_reference.py or the definition written out; a row that does not see a value that is not
finite keeps every bit of its result."""
import numpy as np
import pytest
import torch

import int4_weight_only_amd as w4
from tests import layer_reference as ref
from tests.test_gpu_layer import Paged, bf16, close, f64

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def run(cache, q, q_start, **kw):
    """(y fp32 [T][H][D], lse); q_start None: one token per sequence."""
    kw = dict(kw, out_dtype=w4.W4_OUT_F32, want_lse=True)
    if q_start is None:
        y, lse = w4.w4_attn_decode(q, *cache.args(), **kw)
    else:
        y, lse = w4.w4_attn_prefill(q, *cache.args(), torch.from_numpy(q_start).cuda(), **kw)
    torch.cuda.synchronize()
    return y.reshape(q.shape[0], -1, cache.D).cpu(), lse.cpu()


def same_classes(got, want, bound, what):
    """NaN where the definition gives NaN, its infinities, and finite values within the bound."""
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf), f"{what}: infinities in other places"
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities of the other sign"
    ok = np.isfinite(want)
    close(np.where(ok, got, 0.0), np.where(ok, want, 0.0), np.where(ok, bound, 1.0), what)


def poisoned(seed, lens, nq, H, n_kv, D, page, spots, window=0, sinks=0):
    """Runs a case before and after values that are not finite enter it at `spots`, (sequence,
    position, key-value head, "k" or "v", dim, value)."""
    rng = np.random.default_rng(seed)
    cache = Paged(rng, lens, page, n_kv, D)
    cache.fill(rng, [range(n) for n in lens])
    counts = [1] * len(lens) if nq is None else nq
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T, G = int(starts[-1]), H // n_kv
    q = bf16(rng.normal(size=(T, H * D))).cuda()
    kw = dict(window=window, sinks=sinks)
    q_start = None if nq is None else starts
    before, lse_before = run(cache, q, q_start, **kw)
    for b, pos, hk, kind, d, value in spots:
        (cache.k if kind == "k" else cache.v)[cache.table[b][pos // page], pos % page, hk, d] = value
    y, lse = run(cache, q, q_start, **kw)
    k, v, table = cache.host()
    with np.errstate(invalid="ignore"):
        wy, wl, a, ds, count = ref.attention(f64(q), k, v, table, lens, starts, H,
                                             float(np.float32(D ** -0.5)), window, sinks)
        bound = ref.attention_bound(a, ds, count, 16 if nq is None else 8)
    same_classes(f64(y), wy, bound, "y")
    assert np.array_equal(np.isnan(f64(lse)), np.isnan(wl)), "lse: NaN in other places"
    ok = np.isfinite(wl)
    assert np.all(np.abs(np.where(ok, f64(lse) - wl, 0))[ok]
                  <= (2 * ds + 2.0 ** -20 + (count + 4) * ref.F32 * 2 + 2.0 ** -22 * np.abs(wl))[ok])
    # rows that see none of the spots: not a bit changes
    seen = np.zeros((T, H), dtype=bool)
    for t, b, pos in ref.rows_of(starts, lens, cache.cols * page):
        vis = set(ref.visible(pos, window, sinks).tolist())
        for sb, spos, hk, *_ in spots:
            if sb == b and spos in vis:
                seen[t, hk * G:(hk + 1) * G] = True
    assert seen.any() and not seen.all()
    assert torch.equal(y[~seen], before[~seen]) and torch.equal(lse[~seen], lse_before[~seen])


@pytest.mark.parametrize("D,page", [(128, 64), (128, 4), (64, 16), (80, 16), (256, 32)])
def test_nan_scores(D, page):
    """y and lse are NaN for the rows that see the key, in both forms, in shares and splits too."""
    spots = [(0, 190, 1, "k", 3, NAN), (1, 69, 0, "k", 0, NAN)]
    poisoned([46, D], [300, 70], [300, 70], 6, 2, D, page, spots)
    poisoned([47, D], [300, 70, 1], None, 6, 2, D, page, spots)
    poisoned([48, D], [9000, 70, 33], None, 6, 2, D, page, spots)
    poisoned([49, D], [5000], [20], 4, 2, D, page, [(0, 4985, 0, "k", 5, NAN)])


PROMPT_SPOTS = [(0, 150, 0, "v", 5, INF), (0, 160, 0, "v", 7, NAN), (0, 171, 1, "v", 0, -INF),
                (0, 180, 1, "v", 0, INF), (0, 190, 1, "k", 3, NAN), (1, 69, 0, "v", 2, -INF)]


@pytest.mark.parametrize("D,page", [(128, 64), (128, 16), (128, 1), (64, 64), (64, 8), (80, 16),
                                    (256, 32), (256, 8), (192, 1), (24, 4)])
def test_prompt_rows_before_a_value_that_is_not_finite(D, page):
    poisoned([50, D, page], [300, 70], [300, 70], 6, 2, D, page, PROMPT_SPOTS)


@pytest.mark.parametrize("D,page", [(128, 64), (80, 16), (256, 32)])
def test_prompt_rows_past_a_value_that_is_not_finite(D, page):
    """The window leaves it behind; sinks stay in sight."""
    poisoned([51, D], [300, 70], [300, 70], 6, 2, D, page, PROMPT_SPOTS, window=21, sinks=3)
    poisoned([52, D], [300, 70], [300, 70], 6, 2, D, page, [(0, 2, 1, "v", 1, INF)], window=21,
             sinks=3)


@pytest.mark.parametrize("D,page", [(128, 64), (128, 16), (64, 64), (256, 32)])
def test_few_rows_over_a_long_cache_with_values_that_are_not_finite(D, page):
    """The keys split over workgroups."""
    spots = [(0, 4990, 0, "v", 5, INF), (0, 4995, 1, "v", 7, NAN), (0, 4993, 1, "v", 1, -INF)]
    poisoned([53, D], [5000], [20], 4, 2, D, page, spots)
    poisoned([55, D], [5000], [20], 4, 2, D, page, [(0, 1990, 0, "v", 5, -INF)], window=3000)


@pytest.mark.parametrize("D,page", [(128, 64), (128, 4), (64, 16), (80, 16), (256, 32), (192, 1)])
@pytest.mark.parametrize("lens", [(300, 70, 1), (9000, 70, 33)])
def test_decode_with_values_that_are_not_finite(D, page, lens):
    """In a share of its own and in one that is joined; the keys that fill up a tile repeat a key."""
    n = lens[0]
    spots = [(0, n - 1, 0, "v", 5, INF), (0, n // 2, 0, "v", 7, -INF), (0, n - 2, 1, "v", 0, NAN),
             (0, 0, 1, "v", 1, INF), (0, 3, 1, "v", 1, -INF), (1, 69, 0, "v", 2, -INF)]
    poisoned([56, D, n], list(lens), None, 6, 2, D, page, spots)
    poisoned([57, D, n], list(lens), None, 6, 2, D, page, [(0, n - 3, 1, "k", 5, NAN),
                                                           (0, 9, 0, "v", 2, -INF)])
    poisoned([58, D, n], list(lens), None, 34, 2, D, page, spots[:2], window=n - 1)


# ------------------------------------------------------------------------------- scores


TOPS = [1e9, 1e12, 1e20, 2.0 ** 110, -1e9, -1e12, -1e29, -1e31, -2.0 ** 126]

def one_dim_scores(form, D, products, scale, seed):
    """Queries and keys along one dim, so that a score is one product of two bf16 values, exact in
    fp32: key j of the sequence has the score scale * products[j][0] * products[j][1]."""
    rng = np.random.default_rng(seed)
    n = len(products)
    cache = Paged(rng, [n], 16, 1, D)
    cache.fill(rng, [range(n)])
    for j, (_, kv) in enumerate(products):
        cache.k[cache.table[0][j // 16], j % 16, 0] = bf16(np.eye(D)[1] * kv).cuda()
    q = bf16(np.tile(np.eye(D)[1] * products[0][0], (1 if form is None else form, 2))).cuda()
    starts = None if form is None else np.array([0, form], dtype=np.int32)
    y, lse = run(cache, q, starts, scale=scale)
    T = q.shape[0]
    k, v, table = cache.host()
    wy, wl, a, _, count = ref.attention(f64(q), k, v, table, [n], np.array([0, T]), 2,
                                        float(np.float32(scale)), 0, 0)
    # scores are exact or their differences so large that no rounding matters
    bound = ref.attention_bound(a, np.zeros(wl.shape), count, 16 if form is None else 8)
    close(f64(y), wy, bound, "y")
    assert np.all(np.abs(f64(lse) - wl) <= 2.0 ** -20 + (count + 4) * ref.F32 * 2
                  + 2.0 ** -22 * np.abs(wl))


@pytest.mark.parametrize("form,top", [(form, top) for form in (None, 1, 40) for top in TOPS])
def test_scores_far_from_zero(form, top):
    """Keys of the largest score share the weight, however far from zero the scores are."""
    rng = np.random.default_rng([60, abs(int(top)) % 1000003])
    top = float(bf16(np.array([top])).item())
    low = 2.0 * top if top < 0 else 0.5 * top
    for D in (64, 128, 256):
        products = [(1.0, top if j < 40 or rng.random() < 0.5 else low) for j in range(150)]
        one_dim_scores(form, D, products, 1.0, [61, D])


@pytest.mark.parametrize("form", [None, 1, 40])
def test_scales_near_the_smallest_number(form):
    big = 2.0 ** 63
    rng = np.random.default_rng(62)
    for scale in (2.0 ** -126, 2.0 ** -127, 0.0):
        products = [(big, big * rng.integers(-4, 5) / 4) for _ in range(150)]
        one_dim_scores(form, 64, products, scale, 63)


# ------------------------------------------------------------------------------- rounding to bf16


def test_nan_residuals_stay_nan():
    """Whatever bits a NaN of the fp32 residual holds, its row of y is NaN, and no other."""
    d = 40
    r = torch.zeros((4, d), dtype=torch.float32) + 1.5
    r.view(torch.int32)[0, 3] = -1  # all bits
    r.view(torch.int32)[1, 9] = 0x7FFFFFFF
    r.view(torch.int32)[2, 0] = 0x7F800001
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((4, d), dtype=torch.bfloat16, device="cuda")
    for args in ((x, r.cuda(), w), (None, r.cuda(), w)):
        y, ro = w4.w4_residual_norm(*args)
        assert torch.isnan(y[:3]).all() and torch.isfinite(y[3]).all()
        assert torch.equal(torch.isnan(ro.cpu()), torch.isnan(r))


def test_residuals_round_to_nearest_even():
    """r' = r + x in bf16, bit for bit: every finite bf16 value plus zero, and sums of values whose
    exponents lie up to 20 apart (ties among them)."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    every = bits.view(torch.bfloat16)
    every = every[torch.isfinite(every)].cuda()
    every = every[:every.numel() // 64 * 64].reshape(-1, 64)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(w4.w4_residual_norm(torch.zeros_like(every), every, w)[1].float(),
                       every.float())
    rng = np.random.default_rng(64)
    r = bf16(rng.integers(-255, 256, size=(4096, 64)) * 2.0 ** rng.integers(-10, 10, (4096, 64)))
    x = bf16(rng.integers(-255, 256, size=(4096, 64)) * 2.0 ** rng.integers(-10, 10, (4096, 64)))
    want = (r.float() + x.float()).bfloat16()
    got = w4.w4_residual_norm(x.cuda(), r.cuda(), w)[1]
    assert torch.equal(got.cpu().float(), want.float())


@pytest.mark.parametrize("form", [None, 3])
def test_nan_rows_with_any_output_stride(form):
    rng = np.random.default_rng(65)
    T = 3 if form is None else 3 * form
    cache = Paged(rng, [50, 60, 70], 16, 1, 64)
    cache.fill(rng, [range(50), range(60), range(70)])
    cache.k[cache.table[1][2], 0, 0, 0] = NAN  # position 32 of sequence 1
    q = bf16(rng.normal(size=(T, 128))).cuda()
    starts = torch.arange(0, T + 1, T // 3, dtype=torch.int32).cuda()
    for pad in (0, 1):
        out = torch.zeros((T, 128 + pad), dtype=torch.bfloat16, device="cuda")
        if form is None:
            w4.w4_attn_decode(q, *cache.args(), out=out)
        else:
            w4.w4_attn_prefill(q, *cache.args(), starts, out=out)
        nan = torch.isnan(out[:, :128]).cpu().reshape(3, -1)
        assert nan[1].all() and not nan[0].any() and not nan[2].any()
