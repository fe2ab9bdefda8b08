// gemm_i8_warp_sm100.cu -- the int8 grouped products for few rows per expert
// (decode): warp-level MMAs fed straight from global memory. Same results as
// gemm_i8_sm100.cu, bit for bit: int32 sums are exact in any order and the
// epilogue's arithmetic is the same.
//
// Every weight is used by a few rows, so the time is the weights' way from HBM
// plus latency, and a ring of shared-memory stages, tensor maps and TMEM only
// add to the latency. Here a warp takes 16 weight rows of one expert (16 output
// features, or 8 gate rows and their 8 up rows) as the A operand of
// mma.m16n8k32 and 8 token rows per MMA as B. The sum over k may be taken in any
// order, so a lane's 16-byte load of a row (bytes 16t .. 16t+15 of each 64, t =
// lane % 4) serves as it is: its words are the k groups of two MMAs, in A and B
// alike, and nothing is shuffled. With gate rows as A rows 0-7 and up rows as
// 8-15 a lane's accumulators hold both factors of its outputs.
//
// KS warps of a CTA may split K and add their int32 sums through shared
// memory: with few weight rows in all it brings enough warps to the SMs, at
// most the 16 per SM that are resident with 128 registers (1 token of 8 of 128
// experts, 2048 x 768: gate/up 25 MB 6.8 us, down 13 MB 3.9 us; with twice the
// warps, in two rounds, 9.2 and 5.8 us).
#include "gemm_i8_common.cuh"
#include "launch_util.cuh"

namespace moe {
namespace {

using namespace gemm;

constexpr int kWarps = 8;
constexpr int kStepK = 128;                 // K bytes per step: 2 loads of 16 bytes per lane and row

__device__ __forceinline__ uint4 load_weights(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_i8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The idx-th expert with rows: its rows [lo, hi) of the permuted order. False,
// for the whole warp, if there are fewer.
__device__ __forceinline__ bool find_expert(const Params &p, int idx, int &e, int &lo, int &hi) {
    const int lane = threadIdx.x & 31;
    constexpr int kChunks = 4;              // 128 experts' offsets in flight
    for (int base = 0; base < p.E; base += 32 * kChunks) {
        int a[kChunks], b[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int x = base + 32 * c + lane;
            a[c] = x < p.E ? __ldg(p.offsets + x) : 0;
            b[c] = x < p.E ? __ldg(p.offsets + x + 1) : 0;
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            uint32_t mask = __ballot_sync(0xffffffffu, b[c] > a[c]);
            const int n = __popc(mask);
            if (idx < n) {
                for (int i = 0; i < idx; ++i) mask &= mask - 1;
                const int src = __ffs(mask) - 1;
                e = base + 32 * c + src;
                lo = __shfl_sync(0xffffffffu, a[c], src);
                hi = __shfl_sync(0xffffffffu, b[c], src);
                if (kDebugBounds && (lo < 0 || hi > p.P)) {
                    raise_error(p.err, kErrBounds);
                    lo = min(max(lo, 0), p.P);
                    hi = min(max(hi, lo), p.P);
                }
                return true;
            }
            idx -= n;
        }
    }
    return false;
}

// The CTA's shared sums: [warp][register][lane].
struct Sums {
    int *base;
    __device__ __forceinline__ int &at(int warp, int reg) const { return base[(warp * 16 + reg) * 32 + (threadIdx.x & 31)]; }
};

// The barrier of the KS warps that share an item.
__device__ __forceinline__ void item_sync(int KS) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x >> 5) / KS), "r"(32 * KS) : "memory");
}

// Token rows [r0, r0 + 8 NT) (those below hi) against the warp's 16 weight rows,
// whose lane rows lane / 4 and lane / 4 + 8 start at wa and wb; K steps [s0, s1)
// are this warp's. The KS warps of an item come here together; warp ks = 0
// writes.
template <bool SWIGLU, int NT>
__device__ __forceinline__ void rows_times_weights(const I8Params &ip, const uint8_t *wa, const uint8_t *wb, int e, int f0,
                                                   int r0, int hi, int s0, int s1, int ks, int KS, const Sums &sums) {
    const Params &p = ip.p;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // scales of this lane's outputs: weight rows g and g + 8, tokens 2t and 2t + 1 of each tile
    float sw[2], sx[NT][2];
    const int fa = f0 + g, fb = SWIGLU ? fa : f0 + g + 8;
    if (ks == 0) {
        const float *w_sf = ip.w_sf + static_cast<size_t>(e) * p.w_rows;
        sw[0] = __ldg(w_sf + fa);
        sw[1] = __ldg(w_sf + fb + (SWIGLU ? p.m_out : 0));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = r0 + 8 * n + 2 * t + j;
                sx[n][j] = row < hi ? __ldg(ip.x_sf + token_row(p, row)) : 0.f;
            }
    }
    const uint8_t *x[NT];                                        // token row g of each tile (null: none)
    int acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int row = r0 + 8 * n + g;
        x[n] = row < hi ? reinterpret_cast<const uint8_t *>(p.a) + static_cast<size_t>(token_row(p, row)) * p.K : nullptr;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0;
    }
    constexpr int kUnroll = NT == 1 ? 4 : 2;                     // steps whose weights are in flight together
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int s = s0; s < s1; s += kUnroll) {
        uint4 a[kUnroll][2], b[kUnroll][2];
        bool in[kUnroll][2];
#pragma unroll
        for (int q = 0; q < kUnroll; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (s + q) * kStepK + 64 * h + 16 * t;
                in[q][h] = s + q < s1 && k < p.K;
                a[q][h] = in[q][h] ? load_weights(wa + k) : zero;
                b[q][h] = in[q][h] ? load_weights(wb + k) : zero;
            }
#pragma unroll
        for (int q = 0; q < kUnroll; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (s + q) * kStepK + 64 * h + 16 * t;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 v = in[q][h] && x[n] ? __ldg(reinterpret_cast<const uint4 *>(x[n] + k)) : zero;
                    mma_i8(acc[n], a[q][h].x, b[q][h].x, a[q][h].y, b[q][h].y, v.x, v.y);
                    mma_i8(acc[n], a[q][h].z, b[q][h].z, a[q][h].w, b[q][h].w, v.z, v.w);
                }
            }
    }
    if (KS > 1) {
        const int warp = threadIdx.x >> 5;
        if (ks > 0)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sums.at(warp, 4 * n + i) = acc[n][i];
        item_sync(KS);
        if (ks == 0)
            for (int w = 1; w < KS; ++w)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][i] += sums.at(warp + w, 4 * n + i);
        item_sync(KS);
        if (ks > 0) return;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = r0 + 8 * n + 2 * t + j;
            if (row >= hi) continue;
            uint16_t *out = p.out + static_cast<size_t>(row) * p.m_out;
            const float va = i8_scaled(static_cast<uint32_t>(acc[n][j]), sw[0], sx[n][j]);
            const float vb = i8_scaled(static_cast<uint32_t>(acc[n][2 + j]), sw[1], sx[n][j]);
            if (SWIGLU) {
                out[fa] = i8_bf16(i8_act(va, vb));
            } else {
                out[fa] = i8_bf16(va);
                out[fb] = i8_bf16(vb);
            }
        }
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kWarps * 32, 2)
grouped_gemm_i8_warp_kernel(const __grid_constant__ I8Params ip, const uint8_t *__restrict__ weights, int items, int KS) {
    const Params &p = ip.p;
    constexpr int kFeat = SWIGLU ? 8 : 16;                       // features per item; m_out is a multiple of 16
    __shared__ int sums_s[kWarps * 16 * 32];
    const Sums sums = {sums_s};
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ks = warp % KS;
    const int item = blockIdx.x * (kWarps / KS) + warp / KS;
    const int FB = p.m_out / kFeat;
    int e, lo, hi;
    if (item >= items || !find_expert(p, item / FB, e, lo, hi)) return;      // all warps of the item
    const int f0 = (item % FB) * kFeat;
    const int g = lane >> 2;
    const size_t first = static_cast<size_t>(e) * p.w_rows;
    const uint8_t *wa = weights + (first + f0 + g) * p.K;
    const uint8_t *wb = weights + (first + (SWIGLU ? p.m_out + f0 + g : f0 + g + 8)) * p.K;
    const int steps = (p.K + kStepK - 1) / kStepK;
    const int s0 = steps * ks / KS, s1 = steps * (ks + 1) / KS;
    for (int r0 = lo; r0 < hi; r0 += 32) {
        if (hi - r0 <= 8)
            rows_times_weights<SWIGLU, 1>(ip, wa, wb, e, f0, r0, hi, s0, s1, ks, KS, sums);
        else if (hi - r0 <= 16)
            rows_times_weights<SWIGLU, 2>(ip, wa, wb, e, f0, r0, hi, s0, s1, ks, KS, sums);
        else
            rows_times_weights<SWIGLU, 4>(ip, wa, wb, e, f0, r0, hi, s0, s1, ks, KS, sums);
    }
}

template <bool SWIGLU>
cudaError_t run_warp(const I8GemmArgs &g, cudaStream_t s) {
    constexpr int kFeat = SWIGLU ? 8 : 16;
    const long long items = static_cast<long long>(std::min(g.base.E, g.base.P)) * (g.base.m_out / kFeat);
    const int steps = (g.base.K + kStepK - 1) / kStepK;
    int KS = 1;
    while (KS < kWarps && 2 * items * KS <= 148 * 16 && 2 * KS <= steps) KS *= 2;
    const int blocks = static_cast<int>((items * KS + kWarps - 1) / kWarps);
    return launch_pdl(grouped_gemm_i8_warp_kernel<SWIGLU>, dim3(blocks), dim3(kWarps * 32), 0, s, make_i8_params(g, 16),
                      static_cast<const uint8_t *>(g.base.w), static_cast<int>(items), KS);
}

}  // namespace

cudaError_t launch_grouped_gemm_i8_warp(const I8GemmArgs &g, cudaStream_t s) {
    if (g.base.P == 0) return cudaSuccess;
    return g.base.swiglu ? run_warp<true>(g, s) : run_warp<false>(g, s);
}

}  // namespace moe
