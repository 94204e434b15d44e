// attn_simple.h -- the plainest attention kernel: one wave per (token row, head), one key at a
// time, the running maximum and sum of the softmax beside the weighted sum of the values.
#pragma once

#include "w4_device.h"
#include "w4_launch.h"

namespace w4 {

static __global__ void __launch_bounds__(64) attn_simple_kernel(AttnArgs a, KvView c) {
    const int t = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
    const int D = c.head_dim, hk = h / (a.n_heads / c.n_kv);
    RowPlace r;
    if (!place_of_row(c, a.q_start, t, &r)) return;
    const int pos = r.pos;
    const int32_t *row = c.table + r.seq * c.ld_table;
    float q[4], acc[4];
    for (int i = 0; i < 4; ++i) {
        const int d = lane + 64 * i;
        q[i] = d < D ? bf16_to_f32(a.q[t * a.ldq + h * D + d]) * a.scale : 0.0f;
        acc[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j <= pos; ++j) {
        if (a.window > 0 && j <= pos - a.window && j >= a.sinks) {
            j = pos - a.window;
            continue;
        }
        const int64_t at = kv_offset(c, row, j, hk);
        float s = 0.0f;
        for (int i = 0; i < 4; ++i) {
            const int d = lane + 64 * i;
            if (d < D) s += q[i] * bf16_to_f32(c.k[at + d]);
        }
        s = wave_sum(s);
        const float m2 = fmaxf(m, s);
        const float f = expf(m - m2), p = expf(s - m2);
        m = m2;
        l = l * f + p;
        for (int i = 0; i < 4; ++i) {
            const int d = lane + 64 * i;
            if (d < D) acc[i] = acc[i] * f + p * bf16_to_f32(c.v[at + d]);
        }
    }
    for (int i = 0; i < 4; ++i) {
        const int d = lane + 64 * i;
        if (d < D)
            store_out(a.y, t * a.ldy + h * D + d, l > 0.0f ? acc[i] / l : 0.0f, a.out_f32);
    }
    if (a.lse && lane == 0)
        a.lse[static_cast<int64_t>(t) * a.n_heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace w4
