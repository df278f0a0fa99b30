// 8-bit floats (1 sign, 4 exponent, 3 mantissa bits) under a power of two, on the device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ss {

// 16 of them rounded again under a scale that is 2^-by times the old one, by <= 0: a shift
// of the exponent, exact but for what falls below 2^-6. A NaN stays one.
typedef uint32_t kv8x16 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ kv8x16 kv8_shift(kv8x16 w, int by) {
    // 448 shifted by 20 and more rounds to 0, as every shift beyond does
    const float f = __uint_as_float((uint32_t)(127 + max(by, -100)) << 23);
    kv8x16 r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(w[k], true);
        const uint32_t v = __builtin_amdgcn_cvt_pk_fp8_f32(a[0] * f, a[1] * f, 0, false);
        r[k] = __builtin_amdgcn_cvt_pk_fp8_f32(b[0] * f, b[1] * f, v, true);
    }
    return r;
}

}  // namespace ss
