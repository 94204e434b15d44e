// bf16_device.h -- fp32 to bf16, round to nearest even, by the hardware's conversion: a NaN stays one,
// whatever bits it holds (adding the rounding to its bits can carry an all-ones NaN over to zero).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4 {

// Two values in one dword, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    bf16x2_t r;
    r[0] = static_cast<__bf16>(a);
    r[1] = static_cast<__bf16>(b);
    return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ uint16_t to_bf16(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

}  // namespace w4
