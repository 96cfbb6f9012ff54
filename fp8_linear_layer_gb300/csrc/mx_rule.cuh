// mx_rule.cuh -- the MXFP8 scale rule and scale-byte order, and the packing of
// eight codes, shared by the cast kernels and the norm that casts its output.
// The rule and the order are described at the MXFP8 cast kernels.
#pragma once
#include <cstdint>

#include "cast_rule.cuh"

namespace fp8ll {

// 8 values -> 8 codes packed little-endian in a uint2
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = encode2<FMT>(f[2 * i], f[2 * i + 1], inv);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <int FMT>
__device__ __forceinline__ int mx_exponent(float amax) {
    // FMAX = 1.75 * 2^F; amax = (1 + m) 2^(E - 127) <= 1.75 2^(F + e)
    //   <=> e >= E - 127 - F + (m > 0.75)
    constexpr int F = (FMT == 0) ? 8 : 15;
    const uint32_t b = __float_as_uint(amax);
    if (b == 0u) return 0;
    const int E = static_cast<int>(b >> 23);
    if (E == 0) return -127;  // subnormal amax: far below FMAX 2^-127
    int e = E - 127 - F + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = e < -127 ? -127 : e;
    return e > 127 ? 127 : e;
}

// 2^-e as an fp32 (2^-127 is subnormal)
__device__ __forceinline__ float mx_inverse_scale(int e) {
    return e < 127 ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : __uint_as_float(0x400000u);
}

__device__ __forceinline__ int64_t mx_sf_offset(int64_t kb, int64_t groups, int64_t r, int k) {
    const int64_t rr = r & 127;
    return (kb * groups + (r >> 7)) * 512 + (rr & 31) * 16 + (rr >> 5) * 4 + k;
}

}  // namespace fp8ll
