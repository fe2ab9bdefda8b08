// mx_dev.cuh -- MX quantisation arithmetic (OCP Microscaling Formats v1.0)
// shared by the kernels that write MXFP8 rows: E4M3 elements, one E8M0 scale
// 2^(c-127) per 32 consecutive elements.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace moe {

// E4M3 code of x (round to nearest even, saturate to +-448).
__device__ __forceinline__ uint8_t e4m3_rn_sat(float x) {
    return static_cast<uint8_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3));
}

// Block exponent of an MX block from the bits of its max |x| (a non-negative
// float): floor(log2 amax) - 8, clamped to [-127, 127]; -127 for amax = 0.
__device__ __forceinline__ int mx_block_exponent(uint32_t amax_bits) {
    if (amax_bits == 0) return -127;
    const int biased = static_cast<int>(amax_bits >> 23);       // 0 for a subnormal max
    return max(biased - 127 - 8, -127);
}

// 2^-e as an fp32 (normal for every e the exponent rule gives).
__device__ __forceinline__ float mx_inverse_scale(int e) { return __uint_as_float(static_cast<uint32_t>(127 - e) << 23); }

}  // namespace moe
