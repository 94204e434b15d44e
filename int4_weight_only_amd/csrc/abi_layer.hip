// abi_layer.hip -- the extern "C" entry points of the operators between a decoder layer's linears
// (rotary positions with the cache append, attention over the paged cache, the residual norm):
// host-side argument validation and dispatch.  The contract of every entry point is stated in
// include/w4.h; nothing here allocates device memory or synchronizes.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/w4.h"
#include "w4_launch.h"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Nothing that the entry points call outside of `guarded` may throw.
static_assert(noexcept(w4::device_cu_count()) && noexcept(w4::hip_fail(hipSuccess)),
              "no exception passes the C boundary");

// Runs a launcher; neither a HIP error nor a C++ exception passes the C boundary.
template <typename F>
int guarded(F &&launch) {
    try {
        const hipError_t err = launch();
        return err == hipSuccess ? W4_OK : w4::hip_fail(err);
    } catch (...) {
        return W4_ERR_HIP;
    }
}

// Do T rows of `wa` elements from a on, `lda` apart, share an element with T rows of `wb` from b on,
// `ldb` apart (ld >= w)? Columns of one buffer (lda == ldb) may interleave; rows of different
// lengths may not.
bool rows_overlap(const uint16_t *a, int64_t lda, int64_t wa, const uint16_t *b, int64_t ldb,
                  int64_t wb, int64_t T) {
    const int64_t gap =  // elements from a's first to b's
        (reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) / 2;
    if (gap >= (T - 1) * lda + wa || -gap >= (T - 1) * ldb + wb) return false;
    if (T == 1 || lda != ldb) return true;
    // row i of b begins in column `col` of row i + rows of a
    const int64_t rows = gap >= 0 ? gap / lda : -((lda - 1 - gap) / lda), col = gap - rows * lda;
    return (col < wa && rows > -T && rows < T) ||
           (col + wb > lda && rows + 1 > -T && rows + 1 < T);
}

int check_cache(const w4_kv_cache *c, int n_heads, w4::KvView *view) {
    if (!c || !c->k || !c->v || !c->page_table || !c->kv_len) return W4_ERR_NULL;
    if (c->n_pages < 1 || c->n_kv_heads < 1 || c->head_dim < 1 || c->page_size < 1 ||
        c->n_seqs < 1 || c->table_cols < 1 || c->ld_table < c->table_cols || n_heads < 1)
        return W4_ERR_SHAPE;
    if (c->n_pages > INT32_MAX || c->n_kv_heads > W4_MAX_HEADS || n_heads > W4_MAX_HEADS ||
        c->head_dim > W4_MAX_HEAD_DIM || c->page_size > 32768 || c->n_seqs > W4_MAX_DIM ||
        c->ld_table > INT32_MAX || c->table_cols > (1 << 30) / c->page_size)
        return W4_ERR_RANGE;
    if (n_heads % c->n_kv_heads != 0) return W4_ERR_SHAPE;
    if (c->head_dim % 8 != 0 || (c->page_size & (c->page_size - 1)) != 0)
        return W4_ERR_UNSUPPORTED;
    // rows do not overlap: a stride that is used holds a row at least
    if ((c->n_pages > 1 && c->page_stride < c->head_dim) ||
        (c->page_size > 1 && c->slot_stride < c->head_dim) ||
        (c->n_kv_heads > 1 && c->head_stride < c->head_dim))
        return W4_ERR_SHAPE;
    if (c->page_stride < 0 || c->slot_stride < 0 || c->head_stride < 0) return W4_ERR_SHAPE;
    if (c->page_stride % 8 != 0 || c->slot_stride % 8 != 0 || c->head_stride % 8 != 0 ||
        !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) ||
        !aligned(c->kv_len, 4))
        return W4_ERR_ALIGN;
    if (c->slot_stride > INT32_MAX || c->head_stride > INT32_MAX) return W4_ERR_RANGE;
    if ((c->page_size - 1) * c->slot_stride + (c->n_kv_heads - 1) * c->head_stride + c->head_dim >
        INT32_MAX)
        return W4_ERR_RANGE;
    if (c->page_stride > INT64_MAX / 4 / c->n_pages) return W4_ERR_RANGE;
    view->k = c->k;
    view->v = c->v;
    view->table = c->page_table;
    view->kv_len = c->kv_len;
    view->page_stride = c->page_stride;
    view->ld_table = c->ld_table;
    view->slot_stride = static_cast<int32_t>(c->slot_stride);
    view->head_stride = static_cast<int32_t>(c->head_stride);
    view->n_pages = static_cast<int32_t>(c->n_pages);
    view->page_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
    view->page_mask = c->page_size - 1;
    view->table_cols = static_cast<int32_t>(c->table_cols);
    view->capacity = static_cast<int32_t>(c->table_cols * c->page_size);
    view->n_kv = c->n_kv_heads;
    view->head_dim = c->head_dim;
    view->n_seqs = static_cast<int32_t>(c->n_seqs);
    return W4_OK;
}

// The window and the sinks as the kernels take them: nothing beyond the cache's capacity.
int check_mask(int64_t window, int64_t sinks, const w4::KvView &c, w4::AttnArgs *a) {
    if (window < 0 || sinks < 0) return W4_ERR_RANGE;
    if (window >= c.capacity) window = 0;
    a->window = static_cast<int>(window);
    a->sinks = window > 0 ? static_cast<int>(sinks < c.capacity ? sinks : c.capacity) : 0;
    return W4_OK;
}

int check_attn(const uint16_t *q, int64_t T, int64_t ldq, int n_heads, const int32_t *q_start,
               const w4_kv_cache *cache, float scale, int64_t window, int64_t sinks, void *y,
               int64_t ldy, int out_dtype, float *lse, void *work, w4::KvView *view,
               w4::AttnArgs *a) {
    if (!q || !y) return W4_ERR_NULL;
    if (int st = check_cache(cache, n_heads, view)) return st;
    const int64_t width = static_cast<int64_t>(n_heads) * view->head_dim;
    if (T < 1 || ldq < width || ldy < width) return W4_ERR_SHAPE;
    if (T > W4_MAX_DIM || ldq > W4_MAX_DIM || ldy > W4_MAX_DIM) return W4_ERR_RANGE;
    // the kernels count (token, head) pairs and workgroups in 31 bits
    if (T * n_heads > INT32_MAX || view->n_seqs * static_cast<int64_t>(n_heads) > INT32_MAX)
        return W4_ERR_RANGE;
    if (out_dtype != W4_OUT_BF16 && out_dtype != W4_OUT_F32) return W4_ERR_UNSUPPORTED;
    if (!std::isfinite(scale) || scale < 0.0f) return W4_ERR_RANGE;
    if (int st = check_mask(window, sinks, *view, a)) return st;
    if (!aligned(q, 16) || ldq % 8 != 0 || !aligned(y, out_dtype == W4_OUT_F32 ? 4 : 2) ||
        (lse && !aligned(lse, 4)) || (q_start && !aligned(q_start, 4)))
        return W4_ERR_ALIGN;
    a->q = q;
    a->T = T;
    a->ldq = ldq;
    a->n_heads = n_heads;
    a->q_start = q_start;
    a->scale = scale;
    a->y = y;
    a->ldy = ldy;
    a->out_f32 = out_dtype == W4_OUT_F32;
    a->lse = lse;
    a->work = work;
    return W4_OK;
}

int check_work(size_t need, const void *work, size_t work_bytes) {
    if (need == 0) return W4_OK;
    if (!work) return W4_ERR_NULL;
    if (work_bytes < need) return W4_ERR_RANGE;
    return aligned(work, 16) ? W4_OK : W4_ERR_ALIGN;
}

}  // namespace

extern "C" {

int w4_rope_frequencies(int rot_dim, int scaling, double base, double factor, double context,
                        float *inv_freq, float *amplitude) {
    if (!inv_freq) return W4_ERR_NULL;
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > W4_MAX_HEAD_DIM) return W4_ERR_SHAPE;
    if (scaling < W4_ROPE_PLAIN || scaling > W4_ROPE_YARN) return W4_ERR_UNSUPPORTED;
    if (!std::isfinite(base) || base <= 1.0) return W4_ERR_RANGE;
    if (scaling != W4_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0)) return W4_ERR_RANGE;
    if (scaling == W4_ROPE_YARN && (!std::isfinite(context) || context < 1.0)) return W4_ERR_RANGE;
    if (scaling == W4_ROPE_NTK && rot_dim < 4) return W4_ERR_SHAPE;
    const double R = rot_dim;
    const double b = scaling == W4_ROPE_NTK ? base * std::pow(factor, R / (R - 2.0)) : base;
    double low = 0.0, high = 0.0;
    if (scaling == W4_ROPE_YARN) {
        // the pair that turns `turns` times over the context: context f_i = 2 pi turns
        const auto pair_of = [&](double turns) {
            return R * std::log(context / (turns * 2.0 * M_PI)) / (2.0 * std::log(base));
        };
        low = std::fmax(std::floor(pair_of(32.0)), 0.0);
        high = std::fmin(std::ceil(pair_of(1.0)), R - 1.0);
        if (high <= low) high = low + 1e-3;  // a step
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(b, -2.0 * i / R);
        if (scaling == W4_ROPE_LINEAR) f /= factor;
        if (scaling == W4_ROPE_YARN) {
            const double g = std::fmin(std::fmax((i - low) / (high - low), 0.0), 1.0);
            f = f * (1.0 - g) + f / factor * g;
        }
        inv_freq[i] = static_cast<float>(f);
    }
    if (amplitude)
        *amplitude = scaling == W4_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0)
                                             : 1.0f;
    return W4_OK;
}

int w4_rope_append(const uint16_t *qkv, int64_t T, int64_t ldqkv, int n_heads,
                   const int32_t *q_start, const float *inv_freq, int rot_dim, int layout,
                   float factor, const w4_kv_cache *cache, uint16_t *q, int64_t ldq,
                   void *stream) {
    if (!qkv || !inv_freq || !q) return W4_ERR_NULL;
    w4::KvView view;
    if (int st = check_cache(cache, n_heads, &view)) return st;
    const int64_t D = view.head_dim;
    if (T < 1 || ldqkv < (n_heads + 2 * static_cast<int64_t>(view.n_kv)) * D || ldq < n_heads * D)
        return W4_ERR_SHAPE;
    if (!q_start && T != view.n_seqs) return W4_ERR_SHAPE;
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > D) return W4_ERR_SHAPE;
    if (T > W4_MAX_DIM || ldqkv > W4_MAX_DIM || ldq > W4_MAX_DIM) return W4_ERR_RANGE;
    if (layout != W4_ROPE_HALF && layout != W4_ROPE_INTERLEAVED) return W4_ERR_UNSUPPORTED;
    if (!std::isfinite(factor)) return W4_ERR_RANGE;
    if (!aligned(qkv, 16) || ldqkv % 8 != 0 || !aligned(q, 16) || ldq % 8 != 0 ||
        !aligned(inv_freq, 4) || (q_start && !aligned(q_start, 4)))
        return W4_ERR_ALIGN;
    if (rows_overlap(qkv, ldqkv, (n_heads + 2 * static_cast<int64_t>(view.n_kv)) * D, q, ldq,
                     n_heads * D, T))
        return W4_ERR_SHAPE;
    return guarded([&] {
        return w4::launch_rope_append(qkv, T, ldqkv, n_heads, q_start, inv_freq, rot_dim,
                                      layout == W4_ROPE_INTERLEAVED, factor, view, q, ldq,
                                      static_cast<hipStream_t>(stream));
    });
}

size_t w4_attn_decode_work_bytes(int n_heads, const w4_kv_cache *cache, int64_t window,
                                 int64_t sinks) {
    w4::KvView view;
    w4::AttnArgs a{};
    if (check_cache(cache, n_heads, &view) || check_mask(window, sinks, view, &a) ||
        !w4::attn_decode_supported(n_heads, view, a.window, a.sinks))
        return 0;
    return w4::attn_decode_work_bytes(n_heads, view, a.window, a.sinks);
}

int w4_attn_decode(const uint16_t *q, int64_t ldq, int n_heads, const w4_kv_cache *cache,
                   float scale, int64_t window, int64_t sinks, void *y, int64_t ldy,
                   int out_dtype, float *lse, void *work, size_t work_bytes, void *stream) {
    w4::KvView view;
    w4::AttnArgs a{};
    if (int st = check_attn(q, cache ? cache->n_seqs : 1, ldq, n_heads, nullptr, cache, scale,
                            window, sinks, y, ldy, out_dtype, lse, work, &view, &a))
        return st;
    if (!w4::attn_decode_supported(n_heads, view, a.window, a.sinks)) return W4_ERR_RANGE;
    if (int st = check_work(w4::attn_decode_work_bytes(n_heads, view, a.window, a.sinks), work,
                            work_bytes))
        return st;
    return guarded(
        [&] { return w4::launch_attn_decode(a, view, static_cast<hipStream_t>(stream)); });
}

size_t w4_attn_prefill_work_bytes(int64_t T, int n_heads, const w4_kv_cache *cache,
                                  int64_t window, int64_t sinks) {
    w4::KvView view;
    w4::AttnArgs a{};
    if (T < 1 || T > W4_MAX_DIM || check_cache(cache, n_heads, &view) ||
        check_mask(window, sinks, view, &a) ||
        !w4::attn_prefill_supported(T, n_heads, view, a.window, a.sinks))
        return 0;
    return w4::attn_prefill_work_bytes(T, n_heads, view, a.window, a.sinks);
}

int w4_attn_prefill(const uint16_t *q, int64_t T, int64_t ldq, int n_heads,
                    const int32_t *q_start, const w4_kv_cache *cache, float scale,
                    int64_t window, int64_t sinks, void *y, int64_t ldy, int out_dtype,
                    float *lse, void *work, size_t work_bytes, void *stream) {
    if (!q_start) return W4_ERR_NULL;
    w4::KvView view;
    w4::AttnArgs a{};
    if (int st = check_attn(q, T, ldq, n_heads, q_start, cache, scale, window, sinks, y, ldy,
                            out_dtype, lse, work, &view, &a))
        return st;
    if (!w4::attn_prefill_supported(T, n_heads, view, a.window, a.sinks)) return W4_ERR_RANGE;
    if (int st = check_work(w4::attn_prefill_work_bytes(T, n_heads, view, a.window, a.sinks),
                            work, work_bytes))
        return st;
    return guarded(
        [&] { return w4::launch_attn_prefill(a, view, static_cast<hipStream_t>(stream)); });
}

int w4_residual_norm(const uint16_t *x, int64_t ldx, const void *r, int64_t ldr, int r_dtype,
                     int64_t T, int64_t d, const uint16_t *w_post, const uint16_t *w_pre,
                     float weight_offset, const uint16_t *gate, int64_t ldg, float alpha,
                     float eps, void *r_out, int64_t ldr_out, uint16_t *y, int64_t ldy,
                     void *stream) {
    if (!r || !w_pre || !y) return W4_ERR_NULL;
    if ((x == nullptr) != (r_out == nullptr) || (!x && (w_post || gate))) return W4_ERR_NULL;
    if (T < 1 || d < 1 || ldr < d || ldy < d) return W4_ERR_SHAPE;
    if (x && (ldx < d || ldr_out < d)) return W4_ERR_SHAPE;
    if (gate && ldg != 0 && ldg < d) return W4_ERR_SHAPE;
    if (d > W4_NORM_MAX_D || T > W4_MAX_DIM || ldr > W4_MAX_DIM || ldy > W4_MAX_DIM ||
        (x && (ldx > W4_MAX_DIM || ldr_out > W4_MAX_DIM)) || (gate && ldg > W4_MAX_DIM))
        return W4_ERR_RANGE;
    if (r_dtype != W4_OUT_BF16 && r_dtype != W4_OUT_F32) return W4_ERR_UNSUPPORTED;
    if (!std::isfinite(weight_offset) || !std::isfinite(alpha) || !std::isfinite(eps) ||
        eps < 0.0f)
        return W4_ERR_RANGE;
    if (r_out == r && r_out && ldr_out != ldr) return W4_ERR_SHAPE;
    const size_t ra = r_dtype == W4_OUT_F32 ? 4 : 2;
    if (!aligned(r, ra) || !aligned(y, 2) || !aligned(w_pre, 2) || (x && !aligned(x, 2)) ||
        (r_out && !aligned(r_out, ra)) || (w_post && !aligned(w_post, 2)) ||
        (gate && !aligned(gate, 2)))
        return W4_ERR_ALIGN;
    w4::NormArgs a{};
    a.x = x;
    a.r = r;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.gate = gate;
    a.r_out = r_out;
    a.y = y;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldg = ldg;
    a.ldr_out = ldr_out;
    a.ldy = ldy;
    a.T = T;
    a.d = static_cast<int>(d);
    a.r_f32 = r_dtype == W4_OUT_F32;
    a.weight_offset = weight_offset;
    a.alpha = alpha;
    a.eps = eps;
    return guarded([&] { return w4::launch_residual_norm(a, static_cast<hipStream_t>(stream)); });
}

}  // extern "C"
