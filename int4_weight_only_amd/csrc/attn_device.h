// attn_device.h -- pieces shared by the attention kernels: matrix-core types, transposed LDS
// reads, output stores, sums and maxima over lanes.
#pragma once

#include "bf16_device.h"
#include "w4_device.h"
#include "w4_launch.h"

namespace w4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef float floatx4_t __attribute__((ext_vector_type(4)));
typedef float floatx16_t __attribute__((ext_vector_type(16)));
typedef uint32_t uintx2_t __attribute__((ext_vector_type(2)));
typedef uint32_t uintx4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Running maximum before the first key: the lowest finite number, so that no score lies below it and
// no infinity is subtracted from another.
constexpr float kNoMax = -3.40282347e38f;

// Four bf16 rows of 16 columns, transposed on the way out of LDS: in each group of 16 lanes, lane i
// addresses the 8 bytes at columns 4 (i % 4) of row i / 4 and receives column i of the four rows.
__device__ __forceinline__ uintx2_t lds_read_transposed(const uint16_t *p) {
    typedef __attribute__((address_space(3))) short4_t *lds_t;
    return __builtin_bit_cast(uintx2_t,
                              __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p)));
}

// Eight bf16 values without the ones that are infinite or NaN (0 in their place), and those by kind:
// bf16 1 for infinity, MINUS for minus infinity, NAN_ for NaN (bf16 bit patterns), 0 elsewhere.
template <uint32_t MINUS, uint32_t NAN_>
__device__ __forceinline__ uintx4_t split_values(uintx4_t v, uintx4_t *kind) {
    uintx4_t finite;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t fin = 0, k = 0;
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
            const uint32_t e = v[i] >> h & 0xFFFFu;
            const uint32_t of = e == 0x7F80u ? 0x3F80u : e == 0xFF80u ? MINUS : NAN_;
            const bool odd = (e & 0x7F80u) == 0x7F80u;
            fin |= (odd ? 0u : e) << h;
            k |= (odd ? of : 0u) << h;
        }
        finite[i] = fin;
        (*kind)[i] = k;
    }
    return finite;
}
// Adds n counted values to a sum: infinities in the places of 1, minus infinities in those of MINUS
// (a power of two above the count), NaN from NAN_ on.
template <int MINUS, int NAN_>
__device__ __forceinline__ float add_kinds(float sum, int n) {
    sum = n & (MINUS - 1) ? sum + INFINITY : sum;
    sum = n & (NAN_ - MINUS) ? sum - INFINITY : sum;
    return n >= NAN_ ? __builtin_nanf("") : sum;
}

// Four consecutive elements of an output row, from element idx (a multiple of 4) on. `wide`: the
// output's base and rows allow one store.
__device__ __forceinline__ void store_out4(void *y, int64_t idx, floatx4_t v, bool out_f32,
                                           bool wide) {
    float *y32 = static_cast<float *>(y) + idx;
    uint16_t *y16 = static_cast<uint16_t *>(y) + idx;
    const uintx2_t w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    if (wide) {
        if (out_f32)
            *reinterpret_cast<floatx4_t *>(y32) = v;
        else
            *reinterpret_cast<uintx2_t *>(y16) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (out_f32)
            y32[i] = v[i];
        else
            y16[i] = static_cast<uint16_t>(w[i / 2] >> 16 * (i % 2));
    }
}
__device__ __forceinline__ bool wide_rows(const AttnArgs &a) {
    return (a.ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
}

// What sums weighted by l in all are multiplied with, and ln of l weights of maximum m (log2 units).
// l is 0 where no key is seen; one that is NaN, from a NaN score, stays NaN in both.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Sum over lanes 0 .. own lane (row shifts, then the rows' totals to the rows after them).
__device__ __forceinline__ int wave_scan_dpp(int v) {
    v += dpp_i<0x111, 0xF, true>(v);
    v += dpp_i<0x112, 0xF, true>(v);
    v += dpp_i<0x114, 0xF, true>(v);
    v += dpp_i<0x118, 0xF, true>(v);
    v += dpp_i<0x142, 0xA, false>(v);
    v += dpp_i<0x143, 0xC, false>(v);
    return v;
}

// Largest of 64 values >= 0.
__device__ __forceinline__ int wave_max_dpp(int v) {
    v = max(v, dpp_i<0x111, 0xF, true>(v));
    v = max(v, dpp_i<0x112, 0xF, true>(v));
    v = max(v, dpp_i<0x114, 0xF, true>(v));
    v = max(v, dpp_i<0x118, 0xF, true>(v));
    v = max(v, dpp_i<0x142, 0xA, false>(v));
    v = max(v, dpp_i<0x143, 0xC, false>(v));
    return __builtin_amdgcn_readlane(v, 63);
}

__device__ __forceinline__ float other_half(float v) {  // the value of lane ^ 32
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return __uint_as_float(threadIdx.x & 32 ? r[0] : r[1]);
}
__device__ __forceinline__ float max_of_halves(float v) {  // over lane and lane ^ 32
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

}  // namespace w4
