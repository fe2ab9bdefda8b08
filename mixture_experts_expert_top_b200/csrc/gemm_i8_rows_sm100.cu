// gemm_i8_rows_sm100.cu -- the int8 grouped products for a few rows in all (a
// decoded token's experts): no tensor cores, no TMA. Same results as
// gemm_i8_sm100.cu, bit for bit: int32 sums are exact in any order and the
// epilogue's arithmetic is the same.
//
// Every weight is used by one or two rows, so the time is the weights' way from
// HBM plus latency, and the latency is what this form saves: a warp takes 8
// weight rows of one expert (8 output features, or 4 gate rows and their 4 up
// rows), its lanes read 16 bytes of each per step straight into registers, and
// dot products of 4 int8 (dp4a) accumulate them against the token rows. There
// is no barrier: each warp finds its expert from the offsets with a few
// ballots. 128 registers, so that 16 warps per SM cover each other's latency:
// down for one token (8 of 128 experts, 2048 x 768, 12.7 MB) takes 3.6 us; with
// 228 registers and two steps unrolled 5.3 us, on the tensor-core kernel 5.9 us.
#include "gemm_i8_common.cuh"
#include "launch_util.cuh"

namespace moe {
namespace {

using namespace gemm;

constexpr int kWarps = 8;
constexpr int kWeightRows = 8;              // per warp
constexpr int kTokenRows = 4;               // token rows that share one read of the weights

__device__ __forceinline__ uint4 load_weights(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ int dot16(const uint4 &w, const uint4 &x, int acc) {
    acc = __dp4a(static_cast<int>(w.x), static_cast<int>(x.x), acc);
    acc = __dp4a(static_cast<int>(w.y), static_cast<int>(x.y), acc);
    acc = __dp4a(static_cast<int>(w.z), static_cast<int>(x.z), acc);
    return __dp4a(static_cast<int>(w.w), static_cast<int>(x.w), acc);
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

// Token rows [r0, r0 + R) (those below hi) against the warp's 8 weight rows.
template <bool SWIGLU, int R>
__device__ __forceinline__ void rows_times_weights(const I8Params &ip, const uint8_t *const (&w)[kWeightRows], int e, int f0,
                                                   int r0, int hi) {
    const Params &p = ip.p;
    const int lane = threadIdx.x & 31;
    constexpr int kFeat = SWIGLU ? kWeightRows / 2 : kWeightRows;
    // lane i + kFeat * r forms feature f0 + i of row r0 + r: its scales are on
    // their way while the weights stream
    const int row = r0 + lane / kFeat, f = f0 + lane % kFeat;
    const bool mine = lane < kFeat * R && row < hi;
    const size_t w_row = static_cast<size_t>(e) * p.w_rows + f;
    const float sg = mine ? __ldg(ip.w_sf + w_row) : 0.f;
    const float su = SWIGLU && mine ? __ldg(ip.w_sf + w_row + p.m_out) : 0.f;
    const float sx = mine ? __ldg(ip.x_sf + token_row(p, row)) : 0.f;
    const uint8_t *x[R];
    int acc[kWeightRows][R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        x[r] = reinterpret_cast<const uint8_t *>(p.a) + static_cast<size_t>(token_row(p, min(r0 + r, hi - 1))) * p.K;
#pragma unroll
        for (int i = 0; i < kWeightRows; ++i) acc[i][r] = 0;
    }
#pragma unroll 1
    for (int k = 16 * lane; k < p.K; k += 512) {
        uint4 wv[kWeightRows], xv[R];
#pragma unroll
        for (int i = 0; i < kWeightRows; ++i) wv[i] = load_weights(w[i] + k);
#pragma unroll
        for (int r = 0; r < R; ++r) xv[r] = __ldg(reinterpret_cast<const uint4 *>(x[r] + k));
#pragma unroll
        for (int i = 0; i < kWeightRows; ++i)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[i][r] = dot16(wv[i], xv[r], acc[i][r]);
    }
#pragma unroll
    for (int i = 0; i < kWeightRows; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[i][r] = __reduce_add_sync(0xffffffffu, acc[i][r]);
    int g = 0, u = 0;
#pragma unroll
    for (int i = 0; i < kFeat; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (lane == i + kFeat * r) {
                g = acc[i][r];
                if (SWIGLU) u = acc[kFeat + i][r];
            }
    if (mine) {
        float v = i8_scaled(static_cast<uint32_t>(g), sg, sx);
        if (SWIGLU) v = i8_act(v, i8_scaled(static_cast<uint32_t>(u), su, sx));
        p.out[static_cast<size_t>(row) * p.m_out + f] = i8_bf16(v);
    }
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kWarps * 32, 2)
grouped_gemm_i8_rows_kernel(const __grid_constant__ I8Params ip, const uint8_t *__restrict__ weights, int items) {
    const Params &p = ip.p;
    constexpr int kFeat = SWIGLU ? kWeightRows / 2 : kWeightRows;
    griddep_launch_dependents();
    griddep_wait();
    const int FB = p.m_out / kFeat;                              // m_out is a multiple of 16
    for (int item = blockIdx.x * kWarps + (threadIdx.x >> 5); item < items; item += gridDim.x * kWarps) {
        int e, lo, hi;
        if (!find_expert(p, item / FB, e, lo, hi)) return;
        const int f0 = (item % FB) * kFeat;
        const uint8_t *w[kWeightRows];
#pragma unroll
        for (int i = 0; i < kWeightRows; ++i) {
            const int row = SWIGLU && i >= kFeat ? p.m_out + f0 + i - kFeat : f0 + i;
            w[i] = weights + (static_cast<size_t>(e) * p.w_rows + row) * p.K;
        }
        if (hi - lo == 1) {
            rows_times_weights<SWIGLU, 1>(ip, w, e, f0, lo, hi);
        } else {
            for (int r0 = lo; r0 < hi; r0 += kTokenRows) rows_times_weights<SWIGLU, kTokenRows>(ip, w, e, f0, r0, hi);
        }
    }
}

template <bool SWIGLU>
cudaError_t run_rows(const I8GemmArgs &g, cudaStream_t s) {
    constexpr int kFeat = SWIGLU ? kWeightRows / 2 : kWeightRows;
    const long long items = static_cast<long long>(std::min(g.base.E, g.base.P)) * (g.base.m_out / kFeat);
    const int blocks = static_cast<int>(std::min<long long>((items + kWarps - 1) / kWarps, 148 * 16));
    return launch_pdl(grouped_gemm_i8_rows_kernel<SWIGLU>, dim3(blocks), dim3(kWarps * 32), 0, s, make_i8_params(g, 16),
                      static_cast<const uint8_t *>(g.base.w), static_cast<int>(items));
}

}  // namespace

cudaError_t launch_grouped_gemm_i8_rows(const I8GemmArgs &g, cudaStream_t s) {
    if (g.base.P == 0) return cudaSuccess;
    return g.base.swiglu ? run_rows<true>(g, s) : run_rows<false>(g, s);
}

}  // namespace moe
