// gemm_i8_sm100.cu -- the MoE layer's grouped GEMMs with int8 weights and int8
// token rows on sm_100a's integer tensor-core MMA (tcgen05.mma kind::i8).
//
// For the rows r of expert e (permuted order) and an output channel n:
//   acc[r, n] = sum_k a[r, k] * w[e, n, k]               int32, exact
//   v[r, n]   = acc * w_scale[e, n] * a_scale[r]         fp32
//   gate/up:  act[r, f] = bf16(silu(v_gate) * v_up),  down: y[r, n] = bf16(v)
// |a w| <= 2^14 and K <= 32768, so an accumulator stays below 2^29 + 1. The
// sum has no rounding at all, so the result does not depend on its order, and
// the three kernels for it (this one; gemm_i8_warp_sm100.cu for few rows per
// expert, gemm_i8_pair_sm100.cu for many) give the same bits.
//
// This kernel, for middling numbers of rows: weights are operand A (M = 128
// rows per tile: 128 output features, or 64 gate rows and their 64 up rows,
// alternating by 16), tokens operand B with N = the tile's rows rounded up to
// 16. A ring stage holds K = 128 bytes (one 128-byte swizzled row per operand
// row). K need only be a multiple of 16: TMA fills the rest of the last stage
// with zeros. Token rows come through perm as gather4 loads, or as boxes.
// Measured (B200): gate/up of 64 tokens x 8 of 128 experts, 2048 x 768, 63.5 us
// (398 MB, 6.3 TB/s), of 256 tokens 66 us; down of 16 tokens 21.9 us (131 MB).
// HBM bounds it; at a few MB of weights the ring's start and end, about 4 us.
#include "gemm_i8_common.cuh"
#include "launch_util.cuh"

namespace moe {
namespace {

using namespace gemm;

constexpr int kI8TileA = kBM * kI8BK;           // 16 KB
constexpr int kEpiWarps = 4;

// Tiles of BN token rows x `features` at most.
inline long long most_tiles(const I8GemmArgs &g, int BN, int features) {
    const long long blocks = (static_cast<long long>(g.base.P) + BN - 1) / BN + std::min(g.base.E, g.base.P);
    return blocks * ((g.base.m_out + features - 1) / features);
}

template <int BN, int STAGES, bool SWIGLU, int NA>
struct I8Cfg {
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    static constexpr int kBox = BN / 2;                          // token rows per TMA box
    static constexpr int kABytes = NA * kI8TileA;
    static constexpr int kStageBytes = kABytes + BN * kI8BK;
    static constexpr int kAccCols = NA * BN;
    static constexpr int kTmemCols = 2 * kAccCols;               // two accumulator sets, a power of two
    static constexpr int kRingBytes = STAGES * kStageBytes;
    static constexpr int kOutBytes = kEpiWarps * I8RowWriter<SWIGLU>::kBytes;
    static constexpr int kScaleBytes = kEpiWarps * BN * 4;       // each epilogue warp's copy of the token scales
    static constexpr int kNumBars = 2 * STAGES + 2 + 2 + 1;
    static constexpr int kSmemBytes =
        1024 + kRingBytes + kOutBytes + kScaleBytes + 8 * kNumBars + 64 + 2 * (kMaxExperts + 1) * 4;
    static_assert(kStageBytes % 1024 == 0, "swizzle atoms");
    static_assert(BN % 32 == 0 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM");
    static_assert(kSmemBytes + 64 <= kSmemLimit, "shared memory");
};

template <int BN, int STAGES, bool SWIGLU, int NA>
__global__ void __launch_bounds__(192, 1)
grouped_gemm_i8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ I8Params ip) {
    using C = I8Cfg<BN, STAGES, SWIGLU, NA>;
    constexpr int kFeatPerA = SWIGLU ? 64 : 128, kFeatPerTile = NA * kFeatPerA;
    const Params &p = ip.p;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = smem;                                    // STAGES x [A | B]
    uint8_t *out_s = ring + C::kRingBytes;                   // per epilogue warp: 32 token rows
    float *scale_s = reinterpret_cast<float *>(out_s + C::kOutBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(out_s + C::kOutBytes + C::kScaleBytes);
    uint64_t *full_bar = bars;
    uint64_t *empty_bar = full_bar + STAGES;
    uint64_t *tfull_bar = empty_bar + STAGES;
    uint64_t *tempty_bar = tfull_bar + 2;
    uint64_t *drain_bar = tempty_bar + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *off_s = reinterpret_cast<int *>(tmem_holder + 16);
    int *pre_s = off_s + (kMaxExperts + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int E = p.E;
    const int MB = (p.m_out + kFeatPerTile - 1) / kFeatPerTile;
    const int KB = (p.K + kI8BK - 1) / kI8BK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, C::kTmemCols);
        tmem_relinquish();
    }
    griddep_wait();
    build_tile_prefix<C::kThreads>(p.offsets, E, MB, BN, off_s, pre_s, p.P, p.err);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    TileFeed<BN, 16> feed(pre_s, off_s, E, MB, blockIdx.x, gridDim.x);
    TileInfo ti;

    if (warp == 0) {
        // ================================ producer ==============================
        // Lane 0 runs the ring and the TMA loads; with perm, lanes i < N/4 issue
        // the token rows as gather4 loads.
        const uint64_t pol_w = p.evict_first_weights ? l2_policy_evict_first() : l2_policy_evict_last();
        const uint64_t pol_x = l2_policy_evict_last();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && feed.next(ti)) {
            const int nbox = (ti.n_mma + C::kBox - 1) / C::kBox;
            const uint32_t tx = C::kABytes + (p.perm ? ti.n_mma : nbox * C::kBox) * kI8BK;
            const bool gather_lane = p.perm && 4 * lane < ti.n_mma;
            int tr[4] = {0, 0, 0, 0};
            if (gather_lane) {
#pragma unroll
                for (int j = 0; j < 4; ++j) tr[j] = token_row(p, ti.row0 + 4 * lane + j);
            }
            for (int kb = 0; kb < KB; ++kb) {
                ok = warp_wait(&empty_bar[stage], phase ^ 1, abort_flag, p.err, 0);
                if (!ok) break;
                uint8_t *st = ring + stage * C::kStageBytes;
                uint8_t *sb = st + C::kABytes;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full_bar[stage], tx);
                    if (SWIGLU)
                        tma_load_5d(st, &tmA, &full_bar[stage], kb * kI8BK, 0, 0, ti.mb * 4 * NA, ti.e, pol_w);
                    else
                        tma_load_2d(st, &tmA, &full_bar[stage], kb * kI8BK, ti.e * p.w_rows + ti.mb * NA * kBM, pol_w);
                    if (!p.perm)
                        for (int b = 0; b < nbox; ++b)
                            tma_load_2d(sb + b * C::kBox * kI8BK, &tmB, &full_bar[stage], kb * kI8BK,
                                        ti.row0 + b * C::kBox, pol_x);
                }
                __syncwarp();
                if (gather_lane)
                    tma_gather4(sb + lane * 4 * kI8BK, &tmB, &full_bar[stage], kb * kI8BK, tr[0], tr[1], tr[2], tr[3],
                                pol_x);
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
        }
    } else if (warp == 1) {
        // ================================ MMA issuer ============================
        const uint32_t ring_lo = desc_low(smem_u32(ring));
        int stage = 0;
        uint32_t phase = 0;
        int buf = 0;
        uint32_t bphase = 0;
        bool ok = true;
        while (ok && feed.next(ti)) {
            const uint32_t idesc = idesc_i8_i32(kBM, ti.n_mma);
            ok = warp_wait(&tempty_bar[buf], bphase ^ 1, abort_flag, p.err, 64);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t d = tmem_base + buf * C::kAccCols;
            for (int kb = 0; kb < KB; ++kb) {
                ok = warp_wait(&full_bar[stage], phase, abort_flag, p.err, 0);
                if (!ok) break;
                const uint32_t a = ring_lo + stage * (C::kStageBytes >> 4);
                const uint32_t b = a + (C::kABytes >> 4);
                if (NA == 2) umma_i8_stage<false>(d, a, b, idesc, kb != 0, nullptr);
                umma_i8_stage<true>(d + (NA - 1) * BN, a + (NA - 1) * (kI8TileA >> 4), b, idesc, kb != 0, &empty_bar[stage]);
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
            if (!ok) break;
            if (elect_one()) umma_commit(&tfull_bar[buf]);
            if (++buf == 2) { buf = 0; bphase ^= 1; }
        }
        if (elect_one()) umma_commit(drain_bar);
        volatile int never = 0;
        mbar_wait(drain_bar, 0, &never, p.err);
    } else {
        // ============================ warps 2-5: epilogue =======================
        const int q = warp & 3;                              // TMEM lane quarter of this warp
        const I8RowWriter<SWIGLU> writer(out_s + (warp - 2) * I8RowWriter<SWIGLU>::kBytes);
        float *sx_s = scale_s + (warp - 2) * BN;
        int buf = 0;
        uint32_t bphase = 0;
        while (feed.next(ti)) {
            const int f0 = ti.mb * kFeatPerTile + (SWIGLU ? 16 : 32) * q;
            const int nch = (ti.valid + 31) >> 5;
            float sw[NA][4];
#pragma unroll
            for (int h = 0; h < NA; ++h) i8_weight_scales<SWIGLU>(ip, ti.e, f0 + h * kFeatPerA, sw[h]);
            for (int c = 0; c < nch; ++c) {
                const int n = 32 * c + lane;
                sx_s[n] = n < ti.valid ? __ldg(ip.x_sf + token_row(p, ti.row0 + n)) : 0.f;
            }
            __syncwarp();
            if (!warp_wait(&tfull_bar[buf], bphase, abort_flag, p.err, 64)) break;
            tc_fence_after_sync();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * C::kAccCols;
            for (int c = 0; c < nch; ++c) {
#pragma unroll
                for (int h = 0; h < NA; ++h) {
                    uint32_t a[16], b[16];
                    tmem_ld_16x256b_x4(tb + h * BN + 32 * c, a);
                    tmem_ld_16x256b_x4(tb + h * BN + (16u << 16) + 32 * c, b);
                    tmem_wait_ld();
                    if (h + 1 == NA && c + 1 == nch) {
                        // the accumulators are read: hand them back before the stores
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tempty_bar[buf]);
                    }
                    writer.write(p, a, b, sw[h], sx_s + 32 * c, f0 + h * kFeatPerA, ti.row0 + 32 * c, ti.valid - 32 * c);
                }
            }
            if (++buf == 2) { buf = 0; bphase ^= 1; }
        }
    }

    griddep_launch_dependents();
    __syncthreads();
    if (*abort_flag) {
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, C::kTmemCols);
    }
}

template <int BN, int STAGES, bool SWIGLU, int NA = 1>
cudaError_t run_i8(const I8GemmArgs &g, cudaStream_t s) {
    using C = I8Cfg<BN, STAGES, SWIGLU, NA>;
    CUtensorMap ta, tb;
    const uint64_t x_rows = g.base.perm ? static_cast<uint64_t>(g.base.T) : static_cast<uint64_t>(g.base.P);
    const uint64_t K = static_cast<uint64_t>(g.base.K);
    const bool map_a = SWIGLU ? make_gate_up_map(&ta, g.base.w, g.base.E, g.base.m_out, K, 4 * NA)
                              : make_map(&ta, g.base.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K,
                                         static_cast<uint64_t>(g.base.E) * g.base.w_rows, kI8BK, NA * kBM,
                                         CU_TENSOR_MAP_SWIZZLE_128B);
    if (!map_a || !make_map(&tb, g.base.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, x_rows, kI8BK,
                            g.base.perm ? 1 : C::kBox, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    auto kern = grouped_gemm_i8_kernel<BN, STAGES, SWIGLU, NA>;
    cudaError_t st = ensure_dynamic_smem(kern, C::kSmemBytes);
    if (st != cudaSuccess) return st;
    const int grid = static_cast<int>(std::min<long long>(num_sms(), most_tiles(g, BN, NA * (SWIGLU ? 64 : 128))));
    if (grid <= 0) return cudaSuccess;
    return launch_pdl(kern, dim3(grid), dim3(C::kThreads), C::kSmemBytes, s, ta, tb, make_i8_params(g, BN));
}

// Gate/up takes two A operands per stage (128 features) against one read of the
// token rows, unless that leaves SMs without a tile: measured with one and with
// two (us): 64 tokens of 128 experts 68.1 / 63.5 (2048 x 768, 1536 and 768
// tiles), 256 tokens 82.5 / 66.1, 16 tokens of 8 experts, 2 each (4096 x 1408,
// 176 and 88 tiles) 25.0 / 18.7, 8 tokens of 8 experts (96 and 48 tiles) 9.0 / 9.5.
constexpr int kTwoOperandTiles = 90;

template <int BN, int STAGES1, int STAGES2, bool SWIGLU>
cudaError_t run_i8_na(const I8GemmArgs &g, cudaStream_t s) {
    if (SWIGLU && most_tiles(g, BN, 128) >= kTwoOperandTiles) return run_i8<BN, STAGES2, SWIGLU, 2>(g, s);
    return run_i8<BN, STAGES1, SWIGLU>(g, s);
}

template <bool SWIGLU>
cudaError_t dispatch(const I8GemmArgs &g, double avg, cudaStream_t s) {
    if (avg <= 24) return run_i8_na<32, 9, 5, SWIGLU>(g, s);
    if (avg <= 48) return run_i8_na<64, 8, 5, SWIGLU>(g, s);
    return run_i8_na<128, 6, 4, SWIGLU>(g, s);
}

// Few rows and few weights: the warp kernel, which starts reading weights
// sooner, if no expert can have more than 64 rows (it takes 32 at a time) and
// the weights are few enough that latency counts more than the last tenth of
// the bandwidth. Measured, the warp kernel and this one (us, gate/up and down):
// 1 token of 128 experts, 8 each (2048 x 768) 6.8 / 9.8 and 3.9 / 5.3, 2 tokens
// 11.9 / 12.3 and 6.0 / 7.3, 4 tokens 22.7 / 21.0 and 12.1 / 11.1; 8 tokens of 8
// experts (25 and 13 MB) 6.7 / 9.0 and 4.0 / 5.0, 16 tokens 8.5 / 9.0 and 4.9 /
// 5.0, 32 tokens 12.7 / 11.0 and 6.5 / 5.0.
bool takes_warp_kernel(const I8GemmArgs &g, double avg) {
    const double bytes = static_cast<double>(std::min(g.base.E, g.base.P)) * g.base.w_rows * g.base.K;
    return g.base.T <= 64 && avg <= 16 && bytes <= (avg <= 1 ? 72e6 : 32e6);
}

}  // namespace

bool gemm_i8_gathers_in_kernel(int P, int E) { return static_cast<double>(P) / E <= 48.0; }

cudaError_t launch_grouped_gemm_i8(const I8GemmArgs &g, cudaStream_t s) {
    if (g.base.P == 0) return cudaSuccess;
    const double avg = static_cast<double>(g.base.P) / g.base.E;
    if (takes_warp_kernel(g, avg)) return launch_grouped_gemm_i8_warp(g, s);
    if (!g.base.perm && avg > 48) return launch_grouped_gemm_i8_pair(g, s);
    return g.base.swiglu ? dispatch<true>(g, avg, s) : dispatch<false>(g, avg, s);
}

}  // namespace moe
