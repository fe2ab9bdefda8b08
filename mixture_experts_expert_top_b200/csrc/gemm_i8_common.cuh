// gemm_i8_common.cuh -- pieces shared by the int8 grouped-GEMM kernels
// (gemm_i8_warp_sm100.cu: few tokens per expert; gemm_i8_sm100.cu: middling
// numbers; gemm_i8_pair_sm100.cu: many): parameters and the epilogue's
// arithmetic, which must be the same in all three.
#pragma once

#include "gemm_common.cuh"

namespace moe {

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}\n" : "=r"(r)::"memory");
    return r != 0;
}

// 5-D tiled load by one CTA (coordinates innermost first).
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int c1, int c2,
                                            int c3, int c4, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "l"(policy)
        : "memory");
}

// The same by one CTA of a pair, completing on the barrier at bar_cluster_addr
// (tma_load_2d_pair's).
__device__ __forceinline__ void tma_load_5d_pair(void *dst, const CUtensorMap *map, uint32_t bar_cluster_addr, int x,
                                                 int c1, int c2, int c3, int c4, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(x), "r"(c1), "r"(c2), "r"(c3), "r"(c4),
        "l"(policy)
        : "memory");
}

// 16 lanes x 32 consecutive 32-bit TMEM columns -> 16 registers per thread, in
// the layout of an MMA fragment: thread i holds, for each group g of 8
// columns, columns 8g + 2(i%4) + {0, 1} of lane i/4 in registers 4g, 4g+1 and
// of lane i/4 + 8 in registers 4g+2, 4g+3.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Four 8x8 matrices of 16-bit elements in fragment layout (thread i: row i/4,
// columns 2(i%4) + {0, 1}) to shared memory, transposed: the 16 bytes at the
// address that lane 8m + c gives receive column c of matrix m.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t smem_addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_addr), "r"(a),
                 "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// Instruction descriptor, kind::i8: signed 8-bit A and B (both K-major), int32
// D, shape M x N (M = 128: N = 16 or a multiple of 16 in [32, 256]; M = 256
// across a CTA pair: a multiple of 32 in [32, 256]).
__host__ __device__ __forceinline__ uint32_t idesc_i8_i32(int M, int N) {
    return (2u << 4)                                        // D format: s32
           | (1u << 7)                                      // A format: s8
           | (1u << 10)                                     // B format: s8
           | (static_cast<uint32_t>(N >> 3) << 17)          // N >> 3
           | (static_cast<uint32_t>(M >> 4) << 24);         // M >> 4
}

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

// silu(g) * u = g / (1 + exp(-g)) * u with the approximate exponential and
// reciprocal (2^-22 and 2^-23, and 2^-23 |g| for the exponential's argument):
// within 2^-20 (1 + |g|), below the bf16 rounding's 2^-8. Below g = -87.3, where
// silu(g) is under 2^-119, the reciprocal leaves the normal range and gives 0.
__device__ __forceinline__ float i8_act(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return g * r * u;
}

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

// The tiles of a CTA (or pair) in order, for a converged warp: every 32 tiles
// each lane decodes one of them (a search over the experts and two divisions,
// about 800 cycles), and each tile is then a few shuffles. Tiles have up to
// BLOCK token rows; the instruction's N is their number rounded up to STEP.
template <int BLOCK, int STEP>
struct TileFeed {
    const int *pre, *off;
    int E, MB, tile, step, total, left;
    TileInfo mine;

    __device__ __forceinline__ TileFeed(const int *pre_, const int *off_, int E_, int MB_, int first, int step_)
        : pre(pre_), off(off_), E(E_), MB(MB_), tile(first), step(step_), total(pre_[E_]), left(0) {}

    // False when there is none left.
    __device__ __forceinline__ bool next(TileInfo &t) {
        if (tile >= total) return false;
        if (left == 0) {
            const int lane = threadIdx.x & 31;
            const long long at = tile + static_cast<long long>(lane) * step;
            mine = decode_tile(at < total ? static_cast<int>(at) : tile, pre, off, E, MB, BLOCK);
            left = 32;
        }
        const int src = 32 - left;
        t.e = __shfl_sync(0xffffffffu, mine.e, src);
        t.mb = __shfl_sync(0xffffffffu, mine.mb, src);
        t.row0 = __shfl_sync(0xffffffffu, mine.row0, src);
        t.valid = __shfl_sync(0xffffffffu, mine.valid, src);
        t.n_mma = (t.valid + STEP - 1) & ~(STEP - 1);
        --left;
        tile += step;
        return true;
    }
};

// Weight scales of this thread's accumulator rows in the fragment layout of
// tmem_ld_16x256b_x4: rows lane / 4 + 8 i of the warp's 32 (gate/up: i = 0, 1 gate
// rows, 2, 3 the matching up rows). f0: the warp's first feature.
template <bool SWIGLU>
__device__ __forceinline__ void i8_weight_scales(const I8Params &ip, int e, int f0, float (&sw)[4]) {
    const Params &p = ip.p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int f = f0 + ((threadIdx.x & 31) >> 2) + 8 * (SWIGLU ? i & 1 : i);
        const size_t row = static_cast<size_t>(e) * p.w_rows + f + (SWIGLU && i >= 2 ? p.m_out : 0);
        sw[i] = f < p.m_out ? __ldg(ip.w_sf + row) : 0.f;
    }
}

// Epilogue of 32 tokens by one warp: its 32 accumulator lanes (a: lanes 0-15, b:
// lanes 16-31, tmem_ld_16x256b_x4) scaled, for gate/up combined (lanes 0-15 are
// gate rows, 16-31 the up rows of the same features), rounded to bf16 pairs,
// transposed by stmatrix into rows of tokens in shared memory and stored 16
// bytes at a time.
template <bool SWIGLU>
struct I8RowWriter {
    static constexpr int kFeat = SWIGLU ? 16 : 32;               // features of a warp
    static constexpr int kPieces = kFeat / 8;                    // 16-byte pieces of its token rows
    // 16 bytes of padding keep the eight rows of a stmatrix on different banks
    static constexpr int kRowBytes = 2 * kFeat + 16;
    static constexpr int kBytes = 32 * kRowBytes;                // shared memory per warp
    uint8_t *rows;
    uint32_t st_addr;

    __device__ __forceinline__ explicit I8RowWriter(uint8_t *rows_) : rows(rows_) {
        // this lane's row address of a stmatrix: matrix lane / 8 is 8 features (down) or,
        // gate/up, 8 features of token group lane / 16
        const int lane = threadIdx.x & 31;
        st_addr = smem_u32(rows) + (SWIGLU ? ((lane >> 4) * 8 + (lane & 7)) * kRowBytes + ((lane >> 3) & 1) * 16
                                           : (lane & 7) * kRowBytes + (lane >> 3) * 16);
    }

    // sx: the 32 tokens' scales in shared memory; f0: the warp's first feature;
    // row0: the first token's output row, of which `valid` are the tile's.
    __device__ __forceinline__ void write(const Params &p, const uint32_t (&a)[16], const uint32_t (&b)[16],
                                          const float (&sw)[4], const float *sx, int f0, int row0, int valid) const {
        const int lane = threadIdx.x & 31;
        sx += 2 * (lane & 3);
        uint32_t lo[4], hi[4];                                   // gate/up: features 0-7, 8-15 of each token group
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float2 s = *reinterpret_cast<const float2 *>(sx + 8 * g);
            float v[8];                                          // [row lane / 4 + 8 i][token 0, 1]
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t *r = i < 2 ? a + 4 * g + 2 * i : b + 4 * g + 2 * (i - 2);
                v[2 * i] = i8_scaled(r[0], sw[i], s.x);
                v[2 * i + 1] = i8_scaled(r[1], sw[i], s.y);
            }
            if constexpr (SWIGLU) {
                lo[g] = i8_bf16x2(i8_act(v[0], v[4]), i8_act(v[1], v[5]));
                hi[g] = i8_bf16x2(i8_act(v[2], v[6]), i8_act(v[3], v[7]));
                if (g & 1) stmatrix_x4_trans(st_addr + 8 * (g - 1) * kRowBytes, lo[g - 1], hi[g - 1], lo[g], hi[g]);
            } else {
                stmatrix_x4_trans(st_addr + 8 * g * kRowBytes, i8_bf16x2(v[0], v[1]), i8_bf16x2(v[2], v[3]),
                                  i8_bf16x2(v[4], v[5]), i8_bf16x2(v[6], v[7]));
            }
        }
        __syncwarp();
        const int piece = lane % kPieces;
        if (f0 + 8 * piece < p.m_out) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int t = lane / kPieces + i * (32 / kPieces);
                const uint4 v = *reinterpret_cast<const uint4 *>(rows + t * kRowBytes + 16 * piece);
                if (t < valid)
                    *reinterpret_cast<uint4 *>(p.out + static_cast<size_t>(row0 + t) * p.m_out + f0 + 8 * piece) = v;
            }
        }
        __syncwarp();
    }
};

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

// The same for one CTA; without the commit while another operand A of the stage
// follows.
template <bool COMMIT>
__device__ __forceinline__ void umma_i8_stage(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate,
                                              uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a1, a2, a3, b1, b2, b3;\n\t.reg .b64 x0, x1, x2, x3, y0, y1, y2, y3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.u32 a1, %1, 2;\n\tadd.u32 a2, %1, 4;\n\tadd.u32 a3, %1, 6;\n\t"
        "add.u32 b1, %2, 2;\n\tadd.u32 b2, %2, 4;\n\tadd.u32 b3, %2, 6;\n\t"
        "mov.b64 x0, {%1, %5};\n\tmov.b64 x1, {a1, %5};\n\tmov.b64 x2, {a2, %5};\n\tmov.b64 x3, {a3, %5};\n\t"
        "mov.b64 y0, {%2, %5};\n\tmov.b64 y1, {b1, %5};\n\tmov.b64 y2, {b2, %5};\n\tmov.b64 y3, {b3, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::i8 [%0], x0, y0, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::i8 [%0], x1, y1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::i8 [%0], x2, y2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::i8 [%0], x3, y3, %3, t;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
        : "memory");
    if (COMMIT && elect_one()) umma_commit(bar);
}

}  // namespace gemm
}  // namespace moe
