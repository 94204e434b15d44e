// norm.hip -- the residual norm (w4_residual_norm): norm after a block, gate, residual scale and
// add, norm before the next block.
//
// Memory-bound: each row of x and r is read once, kept in registers (fp32), and r' and y written
// once; the two sums of squares are fp32 sums over the row's threads. A row of up to 512 elements
// belongs to one wave (no barrier), a longer one to a workgroup. 8192 rows of 3584 with an fp32
// residual stream move 352 MB in 67 us: 5.3 TB/s, a large copy's rate.
#include "bf16_device.h"
#include "w4_device.h"
#include "w4_launch.h"

namespace w4 {

namespace {

// Eight consecutive elements of a row, n of them inside it (the others read as 0 and are not
// written). Rows may start anywhere: the 16-byte accesses need no alignment beyond the element's,
// global memory takes any; only a row's last, partial chunk goes element by element.
typedef uint32_t uint4_t __attribute__((ext_vector_type(4)));
typedef uint32_t uint4_any_t __attribute__((ext_vector_type(4), aligned(2), may_alias));
template <typename E>
__device__ __forceinline__ void read8(const E *p, int n, E *e) {
    if (n >= 8) {
        uint4_t x[sizeof(E) / 2];
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E) / 2); ++i)
            x[i] = reinterpret_cast<const uint4_any_t *>(p)[i];
        __builtin_memcpy(e, x, sizeof(x));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : E(0);
    }
}
template <typename E>
__device__ __forceinline__ void write8(E *p, int n, const E *e) {
    if (n >= 8) {
        uint4_t x[sizeof(E) / 2];
        __builtin_memcpy(x, e, sizeof(x));
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(E) / 2); ++i)
            reinterpret_cast<uint4_any_t *>(p)[i] = x[i];
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) p[i] = e[i];
    }
}
__device__ __forceinline__ void load8(const uint16_t *p, int n, float *v) {
    uint16_t e[8];
    read8(p, n, e);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bf16_to_f32(e[i]);
}
__device__ __forceinline__ void load8(const float *p, int n, float *v) { read8(p, n, v); }
__device__ __forceinline__ void store8(uint16_t *p, int n, const float *v) {
    uint16_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = to_bf16(v[i]);
    write8(p, n, e);
}
__device__ __forceinline__ void store8(float *p, int n, const float *v) { write8(p, n, v); }

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
template <typename R, int NT, int NV>
__global__ void __launch_bounds__(NT == kWave ? 4 * kWave : NT) residual_norm_kernel(NormArgs a) {
    constexpr int kRowsPerBlock = NT == kWave ? 4 : 1;
    __shared__ float slots[2][NT / kWave];
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock +
                      (NT == kWave ? static_cast<int>(threadIdx.x) / kWave : 0);
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
            load8(r + e, a.d - e, res[j]);
            if (a.x) load8(a.x + t * a.ldx + e, a.d - e, v[j]);
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
                load8(a.w_post + e, n, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] *= w[i] + a.weight_offset;
            }
            if (a.gate) {
                load8(a.gate + t * a.ldg + e, n, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] *= w[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) res[j][i] = fmaf(v[j][i], scale, res[j][i]);
            store8(static_cast<R *>(a.r_out) + t * a.ldr_out + e, n, res[j]);
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
        load8(a.w_pre + e, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = res[j][i] * pre * (w[i] + a.weight_offset);
        store8(a.y + t * a.ldy + e, n, w);
    }
}

template <typename R, int NT, int NV>
void launch_nt(const NormArgs &a, hipStream_t stream) {
    constexpr int kRowsPerBlock = NT == kWave ? 4 : 1;
    // A launch has fewer than 2^32 threads: more rows (2^23 of 4096, say) take several.
    constexpr int64_t kMostRows = static_cast<int64_t>(kMaxThreads / (kRowsPerBlock * NT)) *
                                  kRowsPerBlock;
    const auto from = [](auto *p, int64_t elements) { return p ? p + elements : p; };
    for (int64_t t = 0; t < a.T; t += kMostRows) {
        NormArgs part = a;
        part.T = a.T - t < kMostRows ? a.T - t : kMostRows;
        part.x = from(a.x, t * a.ldx);
        part.r = from(static_cast<const R *>(a.r), t * a.ldr);
        part.gate = from(a.gate, t * a.ldg);
        part.r_out = from(static_cast<R *>(a.r_out), t * a.ldr_out);
        part.y = from(a.y, t * a.ldy);
        const dim3 grid(static_cast<unsigned>((part.T + kRowsPerBlock - 1) / kRowsPerBlock));
        hipLaunchKernelGGL((residual_norm_kernel<R, NT, NV>), grid, dim3(kRowsPerBlock * NT), 0,
                           stream, part);
    }
}

// One chunk of 8 elements a thread, as far as 512 threads go: what a thread holds it also waits
// for. (8192 rows of 3584, fp32 residual: 64 threads of 8 chunks 93 us, 128 of 4 83, 256 of 2 73,
// 512 of 1 69; 3000 rows of 8192, bf16: 256 of 4 46, 512 of 2 41, 1024 of 1 43; 1700 of 16384: 256
// of 8 89, 512 of 4 57, 1024 of 2 46.)
template <typename R>
void launch_r(const NormArgs &a, hipStream_t stream) {
    const int64_t chunks = (a.d + 7) / 8;
    if (chunks <= 64)
        launch_nt<R, 64, 1>(a, stream);
    else if (chunks <= 128)
        launch_nt<R, 128, 1>(a, stream);
    else if (chunks <= 256)
        launch_nt<R, 256, 1>(a, stream);
    else if (chunks <= 512)
        launch_nt<R, 512, 1>(a, stream);
    else if (chunks <= 1024)
        launch_nt<R, 512, 2>(a, stream);
    else if (chunks <= 2048)
        launch_nt<R, 1024, 2>(a, stream);
    else
        launch_nt<R, 1024, 4>(a, stream);
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
