// norm.hip -- the residual norm (w4_residual_norm): norm after a block, gate, residual scale and
// add, norm before the next block, one workgroup per token.
#include "w4_device.h"
#include "w4_launch.h"

namespace w4 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float *red) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < kThreads / 64; ++w) s += red[w];
    return s;
}

template <bool RF32>
__global__ void __launch_bounds__(kThreads) residual_norm_kernel(NormArgs a) {
    __shared__ float red[kThreads / 64];
    __shared__ float row[1 << 15];
    const int64_t t = blockIdx.x;
    float post = 1.0f;
    if (a.x && a.w_post) {
        float ss = 0.0f;
        for (int i = threadIdx.x; i < a.d; i += kThreads) {
            const float v = bf16_to_f32(a.x[t * a.ldx + i]);
            ss += v * v;
        }
        post = 1.0f / sqrtf(block_sum(ss, red) / a.d + a.eps);
    }
    float ss = 0.0f;
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
        float r = RF32 ? static_cast<const float *>(a.r)[t * a.ldr + i]
                       : bf16_to_f32(static_cast<const uint16_t *>(a.r)[t * a.ldr + i]);
        if (a.x) {
            float n = bf16_to_f32(a.x[t * a.ldx + i]);
            if (a.w_post) n = n * post * (bf16_to_f32(a.w_post[i]) + a.weight_offset);
            if (a.gate) n *= bf16_to_f32(a.gate[t * a.ldg + i]);
            r += a.alpha * n;
            store_out(a.r_out, t * a.ldr_out + i, r, RF32);
        }
        row[i] = r;
        ss += r * r;
    }
    const float pre = 1.0f / sqrtf(block_sum(ss, red) / a.d + a.eps);
    for (int i = threadIdx.x; i < a.d; i += kThreads)
        a.y[t * a.ldy + i] = static_cast<uint16_t>(
            f32_to_bf16(row[i] * pre * (bf16_to_f32(a.w_pre[i]) + a.weight_offset)));
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs &a, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.T));
    if (a.r_f32)
        hipLaunchKernelGGL(residual_norm_kernel<true>, grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(residual_norm_kernel<false>, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace w4
