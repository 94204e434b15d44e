// norm.hip -- the residual norm (w4_residual_norm): norm after a block, gate, residual scale and
// add, norm before the next block.
//
// Memory-bound: each row of x and r is read once, kept in registers (fp32), and r' and y written
// once; the two sums of squares are fp32 sums over the row's threads. A row belongs to one wave
// (no barrier) or, when it is long or the rows are few, to a workgroup.
#include "w4_device.h"
#include "w4_launch.h"

namespace w4 {

namespace {

typedef uint32_t uintx4_t __attribute__((ext_vector_type(4)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));

// Eight consecutive bf16 (n of them inside the row) as fp32, 0 past the row's end. VEC: the
// address is 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ void load8(const uint16_t *p, int n, float *v) {
    if (VEC && n >= 8) {
        const uintx4_t w = *reinterpret_cast<const uintx4_t *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_to_f32(p[i]) : 0.0f;
    }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float *p, int n, float *v) {
    if (VEC && n >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const floatx4_t w = *reinterpret_cast<const floatx4_t *>(p + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * h + i] = w[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(uint16_t *p, int n, const float *v) {
    if (VEC && n >= 8) {
        uintx4_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16(v[2 * i]) | f32_to_bf16(v[2 * i + 1]) << 16;
        *reinterpret_cast<uintx4_t *>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = static_cast<uint16_t>(f32_to_bf16(v[i]));
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *p, int n, const float *v) {
    if (VEC && n >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<floatx4_t *>(p + 4 * h) =
                floatx4_t{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}

// Sum over a row's NT threads; each call has its own slots in LDS.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float *slots) {
    v = wave_sum_dpp(v);
    if (NT == kWave) return v;
    if ((threadIdx.x & (kWave - 1)) == 0) slots[threadIdx.x / kWave] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w) s += slots[w];
    return s;
}

// R: the residual's element type. NT threads a row, each with up to NV chunks of 8 elements.
template <typename R, int NT, int NV, bool VEC>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) residual_norm_kernel(NormArgs a) {
    constexpr int kRowsPerBlock = NT < 256 ? 256 / NT : 1;
    __shared__ float slots[2][NT / kWave];
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock +
                      (NT < 256 ? static_cast<int>(threadIdx.x) / NT : 0);
    if (t >= a.T) return;  // (whole waves; a row's barriers are its own workgroup's)
    const int tid = threadIdx.x % NT;
    const R *r = static_cast<const R *>(a.r) + t * a.ldr;
    const float inv_d = 1.0f / static_cast<float>(a.d);

    float v[NV][8];  // x, then r'
    float res[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = 8 * (tid + j * NT);
        if (e < a.d) {
            load8<VEC>(r + e, a.d - e, res[j]);
            if (a.x) load8<VEC>(a.x + t * a.ldx + e, a.d - e, v[j]);
        }
    }
    if (a.x) {
        float scale = a.alpha;
        if (a.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (8 * (tid + j * NT) < a.d)
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
            scale *= 1.0f / sqrtf(row_sum<NT>(ss, slots[0]) * inv_d + a.eps);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = 8 * (tid + j * NT), n = a.d - e;
            if (n <= 0) continue;
            float w[8];
            if (a.w_post) {
                load8<VEC>(a.w_post + e, n, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] *= w[i] + a.weight_offset;
            }
            if (a.gate) {
                load8<VEC>(a.gate + t * a.ldg + e, n, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] *= w[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) res[j][i] = fmaf(v[j][i], scale, res[j][i]);
            store8<VEC>(static_cast<R *>(a.r_out) + t * a.ldr_out + e, n, res[j]);
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (8 * (tid + j * NT) < a.d)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(res[j][i], res[j][i], ss);
    const float pre = 1.0f / sqrtf(row_sum<NT>(ss, slots[1]) * inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = 8 * (tid + j * NT), n = a.d - e;
        if (n <= 0) continue;
        float w[8];
        load8<VEC>(a.w_pre + e, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = res[j][i] * pre * (w[i] + a.weight_offset);
        store8<VEC>(a.y + t * a.ldy + e, n, w);
    }
}

template <typename R, int NT, int NV>
void launch_nt(const NormArgs &a, bool vec, hipStream_t stream) {
    constexpr int kRowsPerBlock = NT < 256 ? 256 / NT : 1;
    const dim3 grid(static_cast<unsigned>((a.T + kRowsPerBlock - 1) / kRowsPerBlock));
    const dim3 block(NT < 256 ? 256 : NT);
    if (vec)
        hipLaunchKernelGGL((residual_norm_kernel<R, NT, NV, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((residual_norm_kernel<R, NT, NV, false>), grid, block, 0, stream, a);
}

template <typename R>
void launch_r(const NormArgs &a, hipStream_t stream) {
    // 16-byte accesses need every row to start at a 16-byte boundary
    const auto on16 = [](const void *p, int64_t ld, int64_t size) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
    };
    const bool vec = on16(a.x, a.ldx, 2) && on16(a.r, a.ldr, sizeof(R)) &&
                     on16(a.r_out, a.ldr_out, sizeof(R)) && on16(a.y, a.ldy, 2) &&
                     on16(a.gate, a.ldg, 2) && on16(a.w_post, 0, 2) && on16(a.w_pre, 0, 2);
    const int64_t chunks = (a.d + 7) / 8;
    const bool many = a.T >= 4 * device_cu_count();
    if (chunks <= 64)
        launch_nt<R, 64, 1>(a, vec, stream);
    else if (many && chunks <= 512)
        launch_nt<R, 64, 8>(a, vec, stream);
    else if (chunks <= 512)
        launch_nt<R, 256, 2>(a, vec, stream);
    else if (many && chunks <= 1024)
        launch_nt<R, 256, 4>(a, vec, stream);
    else if (many && chunks <= 2048)
        launch_nt<R, 256, 8>(a, vec, stream);
    else
        launch_nt<R, 1024, 4>(a, vec, stream);
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs &a, hipStream_t stream) {
    if (a.r_f32)
        launch_r<float>(a, stream);
    else
        launch_r<uint16_t>(a, stream);
    return hipGetLastError();
}

}  // namespace w4
