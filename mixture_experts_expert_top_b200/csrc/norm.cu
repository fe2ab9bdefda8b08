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
// rounded once; with MXFP8 rows y is carried past fp32 (scale_to_odd), so that
// an E4M3 code is the formula's own. A row lives in registers between its one read and its
// writes: the kernel's floor is the bytes of its inputs and outputs. Measured
// (B200): norm, residual, bf16 and int8 rows of 8192 x 2048 24.1 us, 6.3 TB/s,
// with MXFP8 rows 25.8 us; int8 rows of 65536 x 768 24.6 us, 6.1 TB/s; 256 rows of
// 7168, bf16 and MXFP8, 4.5 us; one row of 2048 1.5 us, MXFP8 1.9 (latency of the
// load, two reductions and the stores).
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "launch_util.cuh"
#include "mx_dev.cuh"

namespace moe {
namespace {

// Threads of a CTA: at least 8 warps, or one row's.
constexpr int row_threads(int tpr) { return tpr == 32 ? 256 : tpr; }

enum RowOut { kRowNone = 0, kRowMx = 1, kRowI8 = 2 };

// Adding 1.5 * 2^23 rounds a value of at most 2^22 to the nearest integer
// (ties to even), whose two's complement is then in the low bits.
constexpr float kRoundMagic = 12582912.0f;

// Sum over the TPR threads of a row, in a fixed order.
template <int TPR, typename F>
__device__ __forceinline__ F row_sum(F v, F *buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) buf[warp] = v;
        __syncthreads();
        if constexpr (sizeof(F) == 8) {
            // by halves: 64-bit additions take longer
            F part[TPR / 32];
#pragma unroll
            for (int i = 0; i < TPR / 32; ++i) part[i] = buf[i];
#pragma unroll
            for (int n = TPR / 64; n > 0; n >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) part[i] += part[i + n];
            return part[0];
        }
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

// Two floats as the operands of packed arithmetic: half the instructions.
struct Pair {
    float x, y;
};
__device__ __forceinline__ uint64_t bits(Pair p) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(p.x), "f"(p.y));
    return r;
}
__device__ __forceinline__ Pair pair_of(uint64_t b) {
    Pair p;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(p.x), "=f"(p.y) : "l"(b));
    return p;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair_of(r);
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair_of(r);
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair_of(r);
}
__device__ __forceinline__ Pair fma2_rz(Pair a, Pair b, Pair c) {
    uint64_t r;
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair_of(r);
}

// Sum of the squares of a thread's elements times f (a power of two). As a
// float, an fp32 chain. As a double, what the chain's roundings drop is summed
// beside it (two chains, of even and odd elements): with s at least as large as
// the next square, t = fl(s + h^2) is at most 2 s, so s - t is exact and h^2 + (s -
// t) is what is missing. s starts at the largest square, rounded up, for that.
// Each chain's at most 32 squares are kept to 2^-37 of their sum at worst, to
// about 2^-45 as roundings go both ways. MXFP8 rows need it: with fp32 chains 10
// codes of 32 million fell on the other side of a border of E4M3. It takes 0.1
// us of a row of 2048 and of 256 rows of 7168, 0.7 of 8192 x 2048.
template <typename Sum, int V>
__device__ __forceinline__ Sum square_sum(const float (&h)[V][8], float f) {
    if constexpr (sizeof(Sum) == 8) {
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float m[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = fmaxf(fabsf(h[j][2 * i]), fabsf(h[j][2 * i + 1]));
            top = fmaxf(top, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
        }
        top *= f;
        const float first = __fmul_ru(top, top);
        Pair s = {first, first}, lo = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const Pair x = {h[j][i] * f, h[j][i + 1] * f};
                const Pair t = fma2(x, x, s);
                lo = add2(lo, fma2(x, x, fma2(t, {-1.0f, -1.0f}, s)));
                s = t;
            }
        // past the fp32 range, or with a NaN, s says so and lo may be NaN
        const Sum sum = static_cast<Sum>(s.x) + s.y;
        return sum <= 2.0 * FLT_MAX ? sum - 2.0 * first + (lo.x + lo.y) : sum;
    } else {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(h[j][i] * f, h[j][i] * f, s);
        return s;
    }
}

// h <- h (r + r_lo) w, rounded to odd: towards zero, and the last bit set if
// anything was left. Rounded again, to E4M3 or bf16, that gives the product's
// own nearest value; two fp32 products rounded to nearest put one value in 2^21
// on the other side of one of E4M3's borders. fma(h, r, -p) is what p lacks of
// h r. Past the fp32 range y is FLT_MAX: infinity in bf16, saturated in E4M3.
// With square_sum's exact sum 256 rows of 7168 take 4.48 us, 8192 x 2048 25.8
// and a row of 2048 1.92; plain products of fp32 sums 4.08, 24.2 and 1.60. A
// branch for the values that a rounding to nearest puts on a border took longer.
__device__ __forceinline__ void scale_to_odd(float (&h)[8], float r, float r_lo, const float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const Pair x = {h[i], h[i + 1]}, v = {w[i], w[i + 1]};
        const Pair p = mul2(x, {r, r}), minus_p = mul2(x, {-r, -r});
        const Pair t = mul2(fma2(x, {r_lo, r_lo}, fma2(x, {r, r}, minus_p)), v);
        const Pair y = fma2_rz(p, v, t);
        const Pair rest = fma2(t, {-1.0f, -1.0f}, fma2(minus_p, v, y));      // NaN for an infinity or NaN, which stays
        h[i] = __uint_as_float(__float_as_uint(y.x) | (fabsf(rest.x) > 0.f ? 1u : 0u));
        h[i + 1] = __uint_as_float(__float_as_uint(y.y) | (fabsf(rest.y) > 0.f ? 1u : 0u));
    }
}

struct RowArgs {
    const uint4 *x, *residual, *weight;     // residual: null without one; weight: null without a norm
    double inv_h;                           // 1 / row length
    float eps;
    int rows, nvec;                         // 8-element vectors per row
    uint4 *residual_out, *y;                // may be null
    uint2 *q;
    void *scales;                           // E8M0 bytes [rows, H/32] or fp32 [rows]
    const int32_t *inv_perm;                // int8 rows written to the `slots` permuted rows of their token
    int slots, pairs;
};

// One row per TPR threads at a time, V vectors of 8 elements per thread; the
// grid strides over the rows and loads the next row's vectors before it
// computes the current one.
template <int TPR, int V, int OUT, bool NORM>
__global__ void __launch_bounds__(row_threads(TPR))
row_kernel(const RowArgs a) {
    constexpr int kRows = row_threads(TPR) / TPR;
    constexpr int kWarps = TPR / 32;
    constexpr bool kAhead = TPR * V <= 2048;    // longer rows need the registers for themselves
    constexpr bool kHoldWeight = kAhead && V <= 3;
    // written by one row, read until its last reduction, and the next row takes the other half
    using Sum = typename std::conditional<OUT == kRowMx, double, float>::type;
    __shared__ Sum sum_s[2][kWarps], again_s[2][kWarps];
    __shared__ uint32_t max_s[2][kWarps];
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x % TPR;
    const int step = gridDim.x * kRows;
    long long row = blockIdx.x * kRows + threadIdx.x / TPR;
    uint4 wv[V], xv[V], rv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int v = t + TPR * j;
        if (kHoldWeight) wv[j] = NORM && v < a.nvec ? __ldg(a.weight + v) : make_uint4(0, 0, 0, 0);
    }
    auto load = [&](long long r) {
        const size_t at = static_cast<size_t>(r) * a.nvec;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = t + TPR * j;
            const bool in = r < a.rows && v < a.nvec;
            xv[j] = in ? a.x[at + v] : make_uint4(0, 0, 0, 0);
            if (NORM) rv[j] = in && a.residual ? a.residual[at + v] : make_uint4(0, 0, 0, 0);
        }
    };
    if (kAhead) load(row);
    for (int half = 0; row < a.rows; row += step, half ^= 1) {  // the same count for all threads of a row
        const size_t base = static_cast<size_t>(row) * a.nvec;
        if (!kAhead) load(row);
        float h[V][8];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            unpack8(xv[j], h[j]);
            if (NORM) {
                float r[8];
                unpack8(rv[j], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] += r[i];
            }
        }
        if (kAhead) load(row + step);
        if constexpr (NORM) {
            Sum ss = row_sum<TPR>(square_sum<Sum>(h, 1.0f), sum_s[half]);
            // the outputs may be x or residual themselves: each thread writes the
            // elements that it has read
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = t + TPR * j;
                if (a.residual_out && v < a.nvec) a.residual_out[base + v] = pack8(h[j]);
            }
            float eps = a.eps, back = 1.0f;
            if (!(ss <= FLT_MAX)) {
                // squares past the fp32 range: those of h 2^-80, whose sum over a row is at
                // most 2^15 2^96; the root is scaled back in two factors of 2^-40, so that
                // neither h nor 1 / root leaves the normal range
                eps = a.eps * 0x1p-80f * 0x1p-80f;
                back = 0x1p-40f;
                ss = row_sum<TPR>(square_sum<Sum>(h, 0x1p-80f), again_s[half]);
#pragma unroll
                for (int j = 0; j < V; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[j][i] *= 0x1p-40f;
            }
            const Sum mean = fma(ss, static_cast<Sum>(a.inv_h), static_cast<Sum>(eps));
            float rstd = 1.0f / sqrtf(static_cast<float>(mean));
            float rstd_lo = 0.f;                                // MX rows: 1 / sqrt(mean) - rstd, a Newton step
            if constexpr (OUT == kRowMx) {
                if (rstd > 0.f && rstd <= FLT_MAX) {
                    const double r = rstd;
                    rstd_lo = back * static_cast<float>(0.5 * r * fma(-mean * r, r, 1.0));
                }
            }
            rstd *= back;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = t + TPR * j;
                if (v < a.nvec) {
                    float w[8];
                    unpack8(kHoldWeight ? wv[j] : __ldg(a.weight + v), w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if constexpr (OUT != kRowMx) h[j][i] = h[j][i] * rstd * w[i];
                    }
                    if constexpr (OUT == kRowMx) scale_to_odd(h[j], rstd, rstd_lo, w);
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
            m = row_max_bits<TPR>(m, max_s[half]);
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
}

template <int TPR, int V, int OUT, bool NORM>
cudaError_t run_rows(const RowArgs &a, cudaStream_t s) {
    constexpr int kThreads = row_threads(TPR), kRows = kThreads / TPR;
    // A few rounds of resident CTAs, each with its share of the rows: later CTAs
    // even out the SMs. Measured at 8192 x 2048 (norm) 1 round 26.7 us, 2 24.9,
    // 4 24.5, a CTA per row 25.6; at 65536 x 768 (int8 rows alone) 25.3, 25.6,
    // 25.9 and 30.4 us, at 16384 x 2048 20.2, 19.5, 20.1 and 22.6 us.
    constexpr int kRounds = NORM ? 4 : 2;
    static const int resident = [] {
        int per_sm = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, row_kernel<TPR, V, OUT, NORM>, kThreads, 0) !=
            cudaSuccess)
            per_sm = 0;
        return 148 * (per_sm > 0 ? per_sm : 1);
    }();
    const int grid = std::min((a.rows - 1) / kRows + 1, kRounds * resident);
    return launch_pdl(row_kernel<TPR, V, OUT, NORM>, dim3(grid), dim3(kThreads), 0, s, a);
}

template <int TPR, int V>
cudaError_t launch_rows(const RowArgs &a, int out, bool norm, cudaStream_t s) {
    if (!norm) return run_rows<TPR, V, kRowI8, false>(a, s);
    if (out == kRowMx) return run_rows<TPR, V, kRowMx, true>(a, s);
    if (out == kRowI8) return run_rows<TPR, V, kRowI8, true>(a, s);
    return run_rows<TPR, V, kRowNone, true>(a, s);
}

cudaError_t dispatch_rows(const RowArgs &a, int out, bool norm, cudaStream_t s) {
    if (a.rows == 0) return cudaSuccess;
    const int n = a.nvec;
    // The fewest threads per row that keep it in at most 4 vectors each: a warp
    // needs no barrier for its sums, and more vectors in flight per thread beat
    // more threads (65536 x 768: a warp 25.3 us, 128 threads 48.2; 2048 x 7168:
    // 256 threads 22.9 us, 512 25.1, 1024 28.0; one row of 7168: 2.5, 2.5, 2.8).
    if (n <= 32) return launch_rows<32, 1>(a, out, norm, s);
    if (n <= 64) return launch_rows<32, 2>(a, out, norm, s);
    if (n <= 96) return launch_rows<32, 3>(a, out, norm, s);
    if (n <= 128) return launch_rows<32, 4>(a, out, norm, s);
    if (n <= 256) return launch_rows<128, 2>(a, out, norm, s);
    if (n <= 512) return launch_rows<128, 4>(a, out, norm, s);
    if (n <= 1024) return launch_rows<256, 4>(a, out, norm, s);
    if (n <= 2048) return launch_rows<512, 4>(a, out, norm, s);
    if (n <= 4096) return launch_rows<512, 8>(a, out, norm, s);
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
    a.inv_h = 1.0 / n.H;
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
