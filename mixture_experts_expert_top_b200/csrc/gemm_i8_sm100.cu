// gemm_i8_sm100.cu -- the MoE layer's grouped GEMMs with int8 weights and int8
// token rows on sm_100a's integer tensor-core MMA (tcgen05.mma kind::i8).
//
// For the rows r of expert e (permuted order) and an output channel n:
//   acc[r, n] = sum_k a[r, k] * w[e, n, k]               int32, exact
//   v[r, n]   = acc * w_scale[e, n] * a_scale[r]         fp32
//   gate/up:  act[r, f] = bf16(silu(v_gate) * v_up),  down: y[r, n] = bf16(v)
// |a w| <= 2^14 and K <= 32768, so an accumulator stays below 2^29 + 1. The
// sum has no rounding at all, so the result does not depend on its order.
//
// GEMM layout as in the MXFP8 kernel (gemm_mxfp8_sm100.cu) without its block
// scales: weights are operand A (M = 128 rows per tile), tokens operand B with
// N = the tile's rows rounded up to 16; gate/up tiles hold the gate and the
// matching up rows and accumulate both. A ring stage holds K = 128 bytes (one
// 128-byte swizzled row per operand row): four MMAs of K = 32 per accumulator.
// K need only be a multiple of 16: TMA fills the rest of the last stage with
// zeros. The scales are applied in the epilogue.
#include "gemm_i8_common.cuh"
#include "launch_util.cuh"

namespace moe {
namespace {

using namespace gemm;

constexpr int kI8TileA = kBM * kI8BK;           // 16 KB

template <int BN, int STAGES, bool SWIGLU>
struct I8Cfg {
    static constexpr int kNumA = SWIGLU ? 2 : 1;
    static constexpr int kThreads = 192;
    static constexpr int kABytes = kNumA * kI8TileA;
    static constexpr int kBBytes = BN * kI8BK;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kAccCols = SWIGLU ? 2 * BN : BN;
    static constexpr int kTmemUsed = 2 * kAccCols;
    static constexpr int kTmemCols = kTmemUsed <= 32 ? 32 : kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128
                                   : kTmemUsed <= 256 ? 256 : 512;
    static constexpr int kRingBytes = STAGES * kStageBytes;
    static constexpr int kNumBars = 2 * STAGES + 2 + 2 + 1;
    static constexpr int kSmemBytes = 1024 + kRingBytes + 8 * kNumBars + 64 + 2 * (kMaxExperts + 1) * 4;
    static_assert(kStageBytes % 1024 == 0, "swizzle atoms");
    static_assert(kTmemUsed <= 512, "TMEM holds 512 32-bit columns");
    static_assert(BN % kBoxN == 0 && BN <= 128, "BN");
    static_assert(kSmemBytes + 64 <= kSmemLimit, "shared memory");
};

template <int BN, int STAGES, bool SWIGLU>
__global__ void __launch_bounds__(192, 1)
grouped_gemm_i8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const I8Params ip) {
    using C = I8Cfg<BN, STAGES, SWIGLU>;
    const Params &p = ip.p;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = smem;                                    // STAGES x [A | A up | B]
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + C::kRingBytes);
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
    const int MB = (p.m_out + kBM - 1) / kBM;
    const int KB = (p.K + kI8BK - 1) / kI8BK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], kEpiThreads);
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
    const int total_tiles = pre_s[E];

    if (warp == 0) {
        // ================================ producer ==============================
        // Lane 0 runs the ring and the TMA loads; with perm, lanes i < N/4 issue
        // the token rows as gather4 loads.
        const uint64_t pol_w = p.evict_first_weights ? l2_policy_evict_first() : l2_policy_evict_last();
        const uint64_t pol_x = l2_policy_evict_last();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < total_tiles && ok; tile += gridDim.x) {
            const TileInfo ti = decode_tile(tile, pre_s, off_s, E, MB, BN);
            const int nbox = ti.n_mma / kBoxN;
            const int a_row = ti.e * p.w_rows + ti.mb * kBM;
            const uint32_t tx = C::kABytes + nbox * kBoxN * kI8BK;
            const bool gather_lane = p.perm && 4 * lane < ti.n_mma;
            int tr[4] = {0, 0, 0, 0};
            if (gather_lane) {
#pragma unroll
                for (int j = 0; j < 4; ++j) tr[j] = token_row(p, ti.row0 + 4 * lane + j);
            }
            for (int kb = 0; kb < KB; ++kb) {
                if (lane == 0) ok = mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag, p.err, 0);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                uint8_t *st = ring + stage * C::kStageBytes;
                uint8_t *sb = st + C::kABytes;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full_bar[stage], tx);
                    tma_load_2d(st, &tmA, &full_bar[stage], kb * kI8BK, a_row, pol_w);
                    if (SWIGLU) tma_load_2d(st + kI8TileA, &tmA, &full_bar[stage], kb * kI8BK, a_row + p.m_out, pol_w);
                    if (!p.perm)
                        for (int b = 0; b < nbox; ++b)
                            tma_load_2d(sb + b * kBoxN * kI8BK, &tmB, &full_bar[stage], kb * kI8BK,
                                        ti.row0 + b * kBoxN, pol_x);
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
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < total_tiles && ok; tile += gridDim.x) {
                const TileInfo ti = decode_tile(tile, pre_s, off_s, E, MB, BN);
                const uint32_t idesc = idesc_i8_i32(kBM, ti.n_mma);
                ok = mbar_wait(&tempty_bar[buf], bphase ^ 1, abort_flag, p.err);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t d0 = tmem_base + buf * C::kAccCols;
                for (int kb = 0; kb < KB; ++kb) {
                    ok = mbar_wait(&full_bar[stage], phase, abort_flag, p.err, 0);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t st = smem_u32(ring + stage * C::kStageBytes);
                    const uint64_t da = sw128_kmajor_desc(st);
                    const uint64_t du = sw128_kmajor_desc(st + kI8TileA);
                    const uint64_t db = sw128_kmajor_desc(st + C::kABytes);
#pragma unroll
                    for (int k = 0; k < kI8BK / 32; ++k) {
                        const uint32_t acc = (kb | k) != 0;
                        // +32 bytes per K step inside the swizzled row: +2 in the >>4 address field
                        umma_i8_ss(d0, da + 2 * k, db + 2 * k, idesc, acc);
                        if (SWIGLU) umma_i8_ss(d0 + BN, du + 2 * k, db + 2 * k, idesc, acc);
                    }
                    umma_commit(&empty_bar[stage]);
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                umma_commit(&tfull_bar[buf]);
                if (++buf == 2) { buf = 0; bphase ^= 1; }
            }
            umma_commit(drain_bar);
            volatile int never = 0;
            mbar_wait(drain_bar, 0, &never, p.err);
        }
    } else {
        // ============================ warps 2-5: epilogue =======================
        const int q = warp & 3;
        int buf = 0;
        uint32_t bphase = 0;
        for (int tile = blockIdx.x; tile < total_tiles; tile += gridDim.x) {
            const TileInfo ti = decode_tile(tile, pre_s, off_s, E, MB, BN);
            const int f = ti.mb * kBM + q * 32 + lane;           // output feature of this thread
            const bool f_ok = f < p.m_out;
            const size_t w_row = static_cast<size_t>(ti.e) * p.w_rows + f;
            const float sg = f_ok ? __ldg(ip.w_sf + w_row) : 0.f;
            const float su = SWIGLU && f_ok ? __ldg(ip.w_sf + w_row + p.m_out) : 0.f;
            if (!__shfl_sync(0xffffffffu, mbar_wait(&tfull_bar[buf], bphase, abort_flag, p.err, 128), 0)) break;
            tc_fence_after_sync();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * C::kAccCols;
            for (int c0 = 0; c0 < ti.n_mma; c0 += 16) {
                uint32_t g[16], u[16];
                tmem_ld_32x32b_x16(tb + c0, g);
                if (SWIGLU) tmem_ld_32x32b_x16(tb + BN + c0, u);
                // the chunk's token scales, one per lane
                const int n_l = c0 + (lane & 15);
                const float sx_l = n_l < ti.valid ? __ldg(ip.x_sf + token_row(p, ti.row0 + n_l)) : 0.f;
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int n = c0 + j;
                    const float sx = __shfl_sync(0xffffffffu, sx_l, j);
                    if (f_ok && n < ti.valid) {
                        p.out[static_cast<size_t>(ti.row0 + n) * p.m_out + f] =
                            i8_bf16(SWIGLU ? i8_act(i8_scaled(g[j], sg, sx), i8_scaled(u[j], su, sx))
                                           : i8_scaled(g[j], sg, sx));
                    }
                }
            }
            tc_fence_before_sync();
            mbar_arrive(&tempty_bar[buf]);
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

template <int BN, int STAGES, bool SWIGLU>
cudaError_t run_i8(const I8GemmArgs &g, cudaStream_t s) {
    using C = I8Cfg<BN, STAGES, SWIGLU>;
    CUtensorMap ta, tb;
    const uint64_t a_rows = static_cast<uint64_t>(g.base.E) * g.base.w_rows;
    const uint64_t x_rows = g.base.perm ? static_cast<uint64_t>(g.base.T) : static_cast<uint64_t>(g.base.P);
    const uint64_t K = static_cast<uint64_t>(g.base.K);
    if (!make_map(&ta, g.base.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, a_rows, kI8BK, kBM,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&tb, g.base.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, x_rows, kI8BK, g.base.perm ? 1 : kBoxN,
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    auto kern = grouped_gemm_i8_kernel<BN, STAGES, SWIGLU>;
    cudaError_t st = ensure_dynamic_smem(kern, C::kSmemBytes);
    if (st != cudaSuccess) return st;
    const int grid = grid_for(g.base, BN);
    if (grid <= 0) return cudaSuccess;
    return launch_pdl(kern, dim3(grid), dim3(C::kThreads), C::kSmemBytes, s, ta, tb, make_i8_params(g, BN));
}

}  // namespace

bool gemm_i8_gathers_in_kernel(int P, int E) { return static_cast<double>(P) / E <= 48.0; }

cudaError_t launch_grouped_gemm_i8(const I8GemmArgs &g, cudaStream_t s) {
    if (g.base.P == 0) return cudaSuccess;
    const double avg = static_cast<double>(g.base.P) / g.base.E;
    // Few rows in all: latency counts, and reading weights into registers starts
    // sooner. Measured against the tensor-core kernel (us, gate/up and down of
    // 2048 x 768, 128 experts): 8 rows 6.0 / 11.7 and 3.6 / 5.9, 32 rows 20.1 /
    // 22.8 and 13.3 / 13.7, 64 rows 33.4 / 31.7 and 21.6 / 19.3. Past 4 rows per
    // expert the weights pass more than once (2 experts, 16 rows: 7.1 / 6.4).
    if (g.base.P <= 32 && avg <= 4) return launch_grouped_gemm_i8_rows(g, s);
    if (!g.base.perm && avg > 48) return launch_grouped_gemm_i8_pair(g, s);
    if (g.base.swiglu) {
        if (avg <= 24) return run_i8<32, 5, true>(g, s);
        if (avg <= 48) return run_i8<64, 5, true>(g, s);
        return run_i8<128, 4, true>(g, s);
    }
    if (avg <= 24) return run_i8<32, 8, false>(g, s);
    if (avg <= 48) return run_i8<64, 8, false>(g, s);
    return run_i8<128, 6, false>(g, s);
}

}  // namespace moe
