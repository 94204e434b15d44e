// rope.hip -- rotary positions on the fused q/k/v projection, with the append of k and v to the
// paged cache (w4_rope_append).
//
// A pair (a, b) of a head at position p turns by t = p * f: (a cos t - b sin t, a sin t + b cos t).
// The product p * f of a position and an fp32 frequency is exact in fp64 (24 + 31 bits), so the
// reduction modulo one turn is done there: at position 10^5 an fp32 angle would already be off by
// 4e-3, the rounding step of bf16.
#include "w4_device.h"
#include "w4_launch.h"

namespace w4 {

namespace {

__device__ __forceinline__ void turn(int pos, float inv_freq, float factor, float *c, float *s) {
    constexpr double kInv2Pi = 0.15915494309189533577;
    const double turns = static_cast<double>(pos) * static_cast<double>(inv_freq) * kInv2Pi;
    const float t = static_cast<float>(turns - rint(turns));  // [-1/2, 1/2]
    *c = factor * cospif(2.0f * t);
    *s = factor * sinpif(2.0f * t);
}

// One wave per (token, head).
__global__ void __launch_bounds__(64) rope_append_kernel(
    const uint16_t *__restrict__ qkv, int64_t ldqkv, int n_heads,
    const int32_t *__restrict__ q_start, const float *__restrict__ inv_freq, int rot_dim,
    int interleaved, float factor, KvView c, uint16_t *__restrict__ q, int64_t ldq) {
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
    const int D = c.head_dim;
    const uint16_t *src = qkv + t * ldqkv + static_cast<int64_t>(h) * D;
    RowPlace at;
    if (!place_of_row(c, q_start, t, &at)) return;
    const int pos = at.pos;
    uint16_t *dst;
    if (h < n_heads) {
        dst = q + t * ldq + static_cast<int64_t>(h) * D;
    } else {
        if (pos < 0) return;
        const int32_t *row = c.table + at.seq * c.ld_table;
        const int page = row[pos >> c.page_shift];
        if (page < 0 || page >= c.n_pages) return;
        const int hk = h - n_heads;
        dst = (hk < c.n_kv ? c.k : c.v) + kv_offset(c, row, pos, hk < c.n_kv ? hk : hk - c.n_kv);
    }
    const int half = rot_dim / 2;
    if (h < n_heads + c.n_kv) {
        for (int i = lane; i < half; i += 64) {
            const int ia = interleaved ? 2 * i : i, ib = interleaved ? 2 * i + 1 : i + half;
            const float xa = bf16_to_f32(src[ia]), xb = bf16_to_f32(src[ib]);
            float cs, sn;
            turn(pos, inv_freq[i], factor, &cs, &sn);
            dst[ia] = f32_to_bf16(xa * cs - xb * sn);
            dst[ib] = f32_to_bf16(xa * sn + xb * cs);
        }
        for (int i = rot_dim + lane; i < D; i += 64) dst[i] = src[i];
    } else {
        for (int i = lane; i < D; i += 64) dst[i] = src[i];
    }
}

}  // namespace

hipError_t launch_rope_append(const uint16_t *qkv, int64_t T, int64_t ldqkv, int n_heads,
                              const int32_t *q_start, const float *inv_freq, int rot_dim,
                              bool interleaved, float factor, const KvView &cache, uint16_t *q,
                              int64_t ldq, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>(n_heads + 2 * cache.n_kv));
    hipLaunchKernelGGL(rope_append_kernel, grid, dim3(64), 0, stream, qkv, ldqkv, n_heads,
                       q_start, inv_freq, rot_dim, interleaved ? 1 : 0, factor, cache, q, ldq);
    return hipGetLastError();
}

}  // namespace w4
