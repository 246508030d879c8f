// kv_q8.cuh -- what the kernels that append to the 8-bit paged KV cache share: a row's scale
// exponent and its codes (the format stands at the top of kv_q8.cu).
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace bi {

constexpr int kMinExp = -64;  // the smallest scale exponent (a row of zeros has it)

// Largest magnitude of eight bf16 values, as a bf16 bit pattern (magnitudes order as their
// bits; infinities and NaN are the patterns from 0x7f80 on).
__device__ __forceinline__ uint32_t amax_bits(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    return m;
}

// The scale exponent of a row from its largest magnitude (a finite bf16 pattern):
// amax = 1.f * 2^E; 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(uint32_t amax) {
    const int E = int(amax >> 7) - 127;
    return max(kMinExp, E - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0));
}

__device__ __forceinline__ uint2 codes8(const uint4& v, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(w[i] << 16) * inv,
                                                    __uint_as_float(w[i] & 0xffff0000u) * inv),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

}  // namespace bi
