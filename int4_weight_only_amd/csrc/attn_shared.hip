// attn_shared.hip -- attention of a batch whose sequences share prefixes, and cross attention.
#include "attn_device.h"

namespace w4 {

namespace {

constexpr int kWaves = 4;

// One workgroup for each (token row, query head): its waves take every fourth key, a lane four dims.
template <bool CROSS>
__global__ void __launch_bounds__(kWaves * 64) attn_rows_kernel(AttnArgs a, KvView c, Prefixes x) {
    __shared__ float so[kWaves][256], sm[kWaves], sl[kWaves];
    const int t = blockIdx.x / a.n_heads, h = blockIdx.x % a.n_heads;
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    RowPlace r;
    if (!place_of_row(c, a.q_start, t, &r)) return;
    const int D = c.head_dim, hk = h / (a.n_heads / c.n_kv), pos = CROSS ? r.n_keys - 1 : r.pos;
    const int32_t *own = c.table + r.seq * c.ld_table, *first = own;
    int cut = 0;
    if (!CROSS) cut = prefix_of_seq(x, r.seq, &first);
    const int d = 4 * lane;
    float q[4], o[4] = {0, 0, 0, 0}, M = kNoMax, l = 0.0f;
    for (int i = 0; i < 4; ++i)
        q[i] = d < D ? bf16_to_f32(a.q[t * a.ldq + static_cast<int64_t>(h) * D + d + i]) : 0.0f;
    for (int j = wid; j <= pos; j += kWaves) {
        if (a.window > 0 && j <= pos - a.window && j >= a.sinks) continue;
        const int64_t at = kv_offset(c, j < cut ? first : own, j, hk);
        float s = 0.0f;
        for (int i = 0; i < 4; ++i) s += d < D ? q[i] * bf16_to_f32(c.k[at + d + i]) : 0.0f;
        s = wave_sum(s) * (a.scale * kLog2e);
        const float M2 = fmaxf(M, s), f = exp2f(M - M2), p = exp2f(s - M2);
        M = M2;
        l = l * f + p;
        for (int i = 0; i < 4; ++i) o[i] = o[i] * f + (d < D ? p * bf16_to_f32(c.v[at + d + i]) : 0.0f);
    }
    for (int i = 0; i < 4; ++i) so[wid][d + i] = o[i];
    if (lane == 0) {
        sm[wid] = M;
        sl[wid] = l;
    }
    __syncthreads();
    float m = kNoMax, sum = 0.0f, v = 0.0f;
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sm[w]);
    const int e = threadIdx.x;
    for (int w = 0; w < kWaves; ++w) {
        const float f = exp2f(sm[w] - m);
        sum += f * sl[w];
        v += f * so[w][e];
    }
    if (e < D)
        store_out(a.y, t * a.ldy + static_cast<int64_t>(h) * D + e, v * inverse_sum(sum), a.out_f32);
    if (a.lse && e == 0) a.lse[static_cast<int64_t>(t) * a.n_heads + h] = log_sum(m, sum);
}

}  // namespace

bool attn_shared_supported(int64_t T, int n_heads, const KvView &, const Prefixes &, int, int) {
    return T * n_heads <= static_cast<int64_t>(kMaxThreads) / (kWaves * 64);
}
size_t attn_shared_work_bytes(int64_t, int, const KvView &, const Prefixes &, int, int) { return 0; }
hipError_t launch_attn_shared(const AttnArgs &a, const KvView &c, const Prefixes &x,
                              hipStream_t stream) {
    hipLaunchKernelGGL(attn_rows_kernel<false>, dim3(static_cast<unsigned>(a.T * a.n_heads)),
                       dim3(kWaves * 64), 0, stream, a, c, x);
    return hipGetLastError();
}
}  // namespace w4
