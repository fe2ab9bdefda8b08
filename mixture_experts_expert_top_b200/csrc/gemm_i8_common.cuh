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

__device__ __forceinline__ uint32_t i8_bf16x2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// silu(g) * u. The fast exponential and quotient are within 2^-20 (1 + |g|) of
// silu's value, below the bf16 rounding's 2^-8; exp(-g) past the fp32 range
// gives a quotient of 0.
__device__ __forceinline__ float i8_act(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// Tensor map of gate/up weights [E, 2I, K] int8 for tiles whose rows alternate
// 16 gate rows and the 16 up rows of the same features: (K, 16, gate/up, I/16,
// E), a box of `groups` such groups. With M rows in this order the 32 TMEM
// lanes of an epilogue warp hold both factors of its 16 features. Feature
// groups past I read zeros.
inline bool make_gate_up_map(CUtensorMap *m, const void *w, uint64_t E, uint64_t I, uint64_t K, uint32_t groups) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[5] = {K, 16, 2, I / 16, E};
    cuuint64_t strides[4] = {K, I * K, 16 * K, 2 * I * K};
    cuuint32_t box[5] = {kI8BK, 16, 2, groups, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(w), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gemm
}  // namespace moe
