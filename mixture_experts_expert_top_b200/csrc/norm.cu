// norm.cu -- RMS norm with the residual's addition and the rows that the
// layer's GEMMs take (bf16, MXFP8 or int8), and the int8 quantisation of rows
// on its own.
//
// For a row x of H bf16 values, residual r and weight w:
//   h = x + r                                   (fp32, not rounded)
//   residual_out = bf16(h)
//   y = h / sqrt(sum_i h_i^2 / H + eps) * w     (fp32)
//   bf16 row   bf16(y)
//   MXFP8 row  per 32 elements e = floor(log2 max|y|) - 8, E4M3(y / 2^e)
//   int8 row   scale = max|y| / 127, q = rint(y * 127 / max|y|)
// The norm and both 8-bit forms take the fp32 values, so each output is
// rounded once. A row lives in registers between its one read and its
// writes: the kernel's floor is the bytes of its inputs and outputs.
#include <float.h>

#include "common.cuh"
#include "launch.h"
#include "launch_util.cuh"
#include "mx_dev.cuh"

namespace moe {
namespace {

enum RowOut { kRowNone = 0, kRowMx = 1, kRowI8 = 2 };

// Adding 1.5 * 2^23 rounds a value of at most 2^22 to the nearest integer
// (ties to even), whose two's complement is then in the low bits.
constexpr float kRoundMagic = 12582912.0f;

// Sum over the TPR threads of a row, in a fixed order.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) buf[warp] = v;
        __syncthreads();
        v = buf[0];
#pragma unroll
        for (int i = 1; i < TPR / 32; ++i) v += buf[i];
    }
    return v;
}

// Maximum of non-negative floats by their bits: NaN counts above infinity.
template <int TPR>
__device__ __forceinline__ uint32_t row_max_bits(uint32_t v, uint32_t *buf) {
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) buf[warp] = v;
        __syncthreads();
        v = buf[0];
#pragma unroll
        for (int i = 1; i < TPR / 32; ++i) v = max(v, buf[i]);
    }
    return v;
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = bf16_bits_to_float((w[j >> 1] >> ((j & 1) * 16)) & 0xFFFFu);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t pack_low_bytes(const float *f) {
    const uint32_t lo = __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

struct RowArgs {
    const uint4 *x, *residual, *weight;     // residual: null without one; weight: null without a norm
    float eps;
    int rows, nvec;                         // 8-element vectors per row
    uint4 *residual_out, *y;                // may be null
    uint2 *q;
    void *scales;                           // E8M0 bytes [rows, H/32] or fp32 [rows]
    const int32_t *inv_perm;                // int8 rows written to the `slots` permuted rows of their token
    int slots, pairs;
};

// One row per TPR threads, V vectors of 8 elements per thread.
template <int TPR, int V, int OUT, bool NORM>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
row_kernel(const RowArgs a) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    __shared__ float sum_s[TPR / 32];
    __shared__ uint32_t max_s[TPR / 32];
    __shared__ float again_s[TPR / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x % TPR;
    const int row = blockIdx.x * kRows + threadIdx.x / TPR;
    if (row >= a.rows) return;                                  // a whole row's threads
    const size_t base = static_cast<size_t>(row) * a.nvec;
    float h[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int v = t + TPR * j;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = 0.f;
        if (v < a.nvec) {
            unpack8(a.x[base + v], h[j]);
            if (NORM && a.residual) {
                float r[8];
                unpack8(a.residual[base + v], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] += r[i];
            }
        }
    }
    if constexpr (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
        ss = row_sum<TPR>(ss, sum_s);
        // the outputs may be x or residual themselves: each thread writes the
        // elements that it has read
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = t + TPR * j;
            if (a.residual_out && v < a.nvec) a.residual_out[base + v] = pack8(h[j]);
        }
        const float inv_h = 1.0f / static_cast<float>(a.nvec * 8);
        float eps = a.eps;
        if (!(ss <= FLT_MAX)) {
            // squares past the fp32 range: the row and the root scaled by 2^-70
            eps = a.eps * 0x1p-70f * 0x1p-70f;
            ss = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    h[j][i] *= 0x1p-70f;
                    ss = fmaf(h[j][i], h[j][i], ss);
                }
            ss = row_sum<TPR>(ss, again_s);
        }
        const float rstd = 1.0f / sqrtf(fmaf(ss, inv_h, eps));
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = t + TPR * j;
            if (v < a.nvec) {
                float w[8];
                unpack8(__ldg(a.weight + v), w);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * rstd * w[i];
                if (a.y) a.y[base + v] = pack8(h[j]);
            }
        }
    }
    if constexpr (OUT == kRowMx) {
        // 4 consecutive lanes hold a block of 32 (H % 32 == 0: all or none of them in range)
        uint8_t *scales = static_cast<uint8_t *>(a.scales);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = t + TPR * j;
            uint32_t amax = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(fabsf(h[j][i])));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            if (v < a.nvec) {
                const int e = mx_block_exponent(amax);
                const float inv = mx_inverse_scale(e);
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i >> 2] |= static_cast<uint32_t>(e4m3_rn_sat(__fmul_rn(h[j][i], inv))) << (8 * (i & 3));
                a.q[base + v] = make_uint2(w[0], w[1]);
                if ((v & 3) == 0) scales[(base + v) >> 2] = static_cast<uint8_t>(e + 127);
            }
        }
    }
    if constexpr (OUT == kRowI8) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(fabsf(h[j][i])));
        m = row_max_bits<TPR>(m, max_s);
        float amax = __uint_as_float(m);
        const bool finite = m < 0x7F800000u;
        // a row with an infinity or a NaN: scale NaN, so that every product it enters is NaN
        const float scale = finite ? amax / 127.0f : __uint_as_float(0x7FC00000u);
        if (amax < 0x1p-100f) {                                 // keeps 127 / amax finite
            amax *= 0x1p100f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] *= 0x1p100f;
        }
        const float inv = finite && amax > 0.f ? 127.0f / amax : 0.f;
        uint2 q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (NORM) {
                    r[i] = fmaf(h[j][i], inv, kRoundMagic);
                } else {
                    // Exact for bf16 values: the true quotient 127 x / amax is a
                    // tie n + 1/2 (8 significant bits) or at least 2^-17 (relative)
                    // away from one, and x * inv is within 2^-22 of it. Rounding it
                    // to 18 bits first (Veltkamp's splitting) restores the ties.
                    const float p = __fmul_rn(h[j][i], inv);
                    const float c = __fmul_rn(p, 65.0f);
                    r[i] = __fadd_rn(__fsub_rn(c, __fsub_rn(c, p)), kRoundMagic);
                }
            }
            q[j] = finite ? make_uint2(pack_low_bytes(r), pack_low_bytes(r + 4)) : make_uint2(0u, 0u);
        }
        float *scales = static_cast<float *>(a.scales);
        if (!a.inv_perm) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = t + TPR * j;
                if (v < a.nvec) a.q[base + v] = q[j];
            }
            if (t == 0) scales[row] = scale;
        } else {
            for (int s = 0; s < a.slots; ++s) {
                const int dst = __ldg(a.inv_perm + static_cast<size_t>(row) * a.slots + s);
                if (dst < 0 || dst >= a.pairs) continue;        // a pair that permute dropped (bad expert id)
                const size_t to = static_cast<size_t>(dst) * a.nvec;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int v = t + TPR * j;
                    if (v < a.nvec) a.q[to + v] = q[j];
                }
                if (t == 0) scales[dst] = scale;
            }
        }
    }
}

template <int TPR, int V>
cudaError_t launch_rows(const RowArgs &a, int out, bool norm, cudaStream_t s) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    const dim3 grid((a.rows + kRows - 1) / kRows), block(TPR < 128 ? 128 : TPR);
    if (!norm) return launch_pdl(row_kernel<TPR, V, kRowI8, false>, grid, block, 0, s, a);
    if (out == kRowMx) return launch_pdl(row_kernel<TPR, V, kRowMx, true>, grid, block, 0, s, a);
    if (out == kRowI8) return launch_pdl(row_kernel<TPR, V, kRowI8, true>, grid, block, 0, s, a);
    return launch_pdl(row_kernel<TPR, V, kRowNone, true>, grid, block, 0, s, a);
}

cudaError_t dispatch_rows(const RowArgs &a, int out, bool norm, cudaStream_t s) {
    if (a.rows == 0) return cudaSuccess;
    const int n = a.nvec;
    if (n <= 256) return launch_rows<256, 1>(a, out, norm, s);
    if (n <= 1024) return launch_rows<256, 4>(a, out, norm, s);
    if (n <= 4096) return launch_rows<1024, 4>(a, out, norm, s);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs &n, cudaStream_t s) {
    RowArgs a = {};
    a.x = reinterpret_cast<const uint4 *>(n.x);
    a.residual = reinterpret_cast<const uint4 *>(n.residual);
    a.weight = reinterpret_cast<const uint4 *>(n.weight);
    a.eps = n.eps;
    a.rows = n.rows;
    a.nvec = n.H / 8;
    a.residual_out = reinterpret_cast<uint4 *>(n.residual_out);
    a.y = reinterpret_cast<uint4 *>(n.y);
    a.q = reinterpret_cast<uint2 *>(n.q);
    a.scales = n.scales;
    return dispatch_rows(a, !n.q ? kRowNone : n.int8 ? kRowI8 : kRowMx, true, s);
}

cudaError_t launch_i8_quantize(const uint16_t *x, int rows, int K, int8_t *q, float *scales, const int32_t *inv_perm,
                               int slots, cudaStream_t s) {
    RowArgs a = {};
    a.x = reinterpret_cast<const uint4 *>(x);
    a.rows = rows;
    a.nvec = K / 8;
    a.q = reinterpret_cast<uint2 *>(q);
    a.scales = scales;
    a.inv_perm = inv_perm;
    a.slots = slots;
    a.pairs = inv_perm ? rows * slots : 0;
    return dispatch_rows(a, kRowI8, false, s);
}

}  // namespace moe
