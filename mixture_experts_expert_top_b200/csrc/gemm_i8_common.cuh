// gemm_i8_common.cuh -- pieces shared by the int8 grouped-GEMM kernels
// (gemm_i8_sm100.cu: few tokens per expert; gemm_i8_pair_sm100.cu: many):
// parameters and the epilogue's arithmetic, which must be the same in both.
#pragma once

#include "gemm_common.cuh"

namespace moe {
namespace gemm {

constexpr int kI8BK = 128;                      // K elements (bytes) per stage and operand row

struct I8Params {
    Params p;
    const float *w_sf;          // [E * w_rows] weight-row scales
    const float *x_sf;          // [token rows] token-row scales
};

inline I8Params make_i8_params(const I8GemmArgs &g, int BN) {
    I8Params ip;
    ip.p = make_params(g.base, BN);
    ip.w_sf = g.w_sf;
    ip.x_sf = g.x_sf;
    return ip;
}

// acc * weight scale * token scale, in this order.
__device__ __forceinline__ float i8_scaled(uint32_t acc, float sw, float sx) {
    return static_cast<float>(static_cast<int>(acc)) * sw * sx;
}

__device__ __forceinline__ uint16_t i8_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

__device__ __forceinline__ uint16_t i8_down(uint32_t acc, float sw, float sx) { return i8_bf16(i8_scaled(acc, sw, sx)); }

// act = bf16(silu(g) * u). The fast exponential and quotient are within 2^-20
// (1 + |g|) of silu's value, below the bf16 rounding's 2^-8; exp(-g) past the
// fp32 range gives a quotient of 0.
__device__ __forceinline__ uint16_t i8_act(float g, float u) {
    return i8_bf16(__fdividef(g, 1.0f + __expf(-g)) * u);
}

}  // namespace gemm
}  // namespace moe
