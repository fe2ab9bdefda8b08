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

// Waits as a whole warp: one poll and a vote when the phase is complete, the
// bounded wait otherwise. False, for every lane, once the wait gave up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, int *err,
                                          uint32_t max_sleep_ns) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err, max_sleep_ns));
}

// One thread of the (converged) warp: the MMAs of one stage, K = 4 x 32, D (+)=
// A B^T, and the commit that arrives on `bar` once they are done. a and b are
// the low words of the operands' shared-memory descriptors (sw128_kmajor_desc;
// a K step of 32 bytes adds 2), whose high words are equal. One asm block: it
// keeps the issue of a stage near the 45 cycles per MMA that the instruction
// itself takes.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);      // sw128_kmajor_desc's bits 32-63
__device__ __forceinline__ uint32_t desc_low(uint32_t smem_addr) { return ((smem_addr & 0x3FFFFu) >> 4) | (1u << 16); }

__device__ __forceinline__ void umma_i8_stage_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate,
                                                   uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a1, a2, a3, b1, b2, b3;\n\t.reg .b64 x0, x1, x2, x3, y0, y1, y2, y3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.u32 a1, %1, 2;\n\tadd.u32 a2, %1, 4;\n\tadd.u32 a3, %1, 6;\n\t"
        "add.u32 b1, %2, 2;\n\tadd.u32 b2, %2, 4;\n\tadd.u32 b3, %2, 6;\n\t"
        "mov.b64 x0, {%1, %6};\n\tmov.b64 x1, {a1, %6};\n\tmov.b64 x2, {a2, %6};\n\tmov.b64 x3, {a3, %6};\n\t"
        "mov.b64 y0, {%2, %6};\n\tmov.b64 y1, {b1, %6};\n\tmov.b64 y2, {b2, %6};\n\tmov.b64 y3, {b3, %6};\n\t"
        "@e tcgen05.mma.cta_group::2.kind::i8 [%0], x0, y0, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::i8 [%0], x1, y1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::i8 [%0], x2, y2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::i8 [%0], x3, y3, %3, t;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], %7;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(smem_u32(bar)), "r"(kDescHigh), "h"(static_cast<uint16_t>(0x3))
        : "memory");
}

}  // namespace gemm
}  // namespace moe
