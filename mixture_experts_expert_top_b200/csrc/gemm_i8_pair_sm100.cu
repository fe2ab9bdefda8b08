// gemm_i8_pair_sm100.cu -- the int8 grouped GEMMs for many tokens per expert:
// weights on the MMA's M side across a CTA pair, tokens on the N side with the
// instruction N set per tile. Same results as gemm_i8_sm100.cu, bit for bit:
// the int32 sums are exact in any order and the epilogue's arithmetic is the
// same.
//
// The layout is the bf16 pair kernel's (gemm_wm_pair_sm100.cu) with 128 int8
// elements in the 128 bytes of an operand row's stage:
//  - A tile = 256 weight rows, 128 per CTA, one tcgen05.mma.cta_group::2
//    kind::i8 of M = 256 per 32 K.
//  - B tile = up to 256 token rows of one expert; N is the tile's rows rounded
//    up to 32 (kind::i8 across a pair takes multiples of 32). The non-leading
//    CTA loads its rows N/2 into the tile.
//  - gate/up: CTA r holds features fb*128 + 64r + [0, 64), its A rows
//    alternating 16 gate rows and the 16 up rows of the same features (one
//    5-D TMA box), so that a warp's 32 TMEM lanes hold both factors of its 16
//    features and no values pass between warps.
//  - down: CTA r holds output features fb*256 + 128r + [0, 128).
//  - Epilogue per 32 tokens (I8RowWriter): fragment loads, scales, bf16 pairs,
//    stmatrix.trans into rows of tokens, 16-byte stores. A thread per feature
//    with 2-byte stores (each row a partial line) left 60 us of it exposed.
//  - Warp 0 loads (both CTAs), warp 1 issues the MMAs (leading CTA) and owns
//    TMEM, warps 2-9 run the epilogue over a double-buffered 2 x 256-column
//    int32 accumulator.
// Measured (B200): gate/up of 8192 tokens x 8 of 128 experts, 2048 x 768, 172 us
// (2.4 POP/s) in a burst and 209 us at the power limit (1.1 GHz); down of 4096
// tokens x 6 of 64 skewed experts, 4096 x 1408, 108 and 129 us. In a burst the
// operands' way to the SMs bounds both: 32 KB per CTA and stage against 512
// cycles of MMAs, 64 bytes per cycle. The first took 164 us without its
// epilogue, 135 with operands in L2 as well, 108 without loads; a case of 4096
// tokens and 64 experts moves 1.45 GB through L2 in 82.6 us, tensor pipe 65% busy.
// Every mbarrier wait is bounded.
#include "gemm_i8_common.cuh"
#include "launch_util.cuh"

namespace moe {
namespace {

using namespace gemm;

constexpr int kPairM = 256;                          // weight rows per pair tile (MMA M)
constexpr int kTokBlock = 256;                       // token rows per tile at most (MMA N)
constexpr int kBBox = 128;                           // token rows per TMA box: one box per stage
constexpr int kTileA = 128 * kI8BK;                  // 16 KB: this CTA's 128 weight rows
constexpr int kTileB = (kTokBlock / 2) * kI8BK;      // 16 KB: up to 128 token rows of this CTA
constexpr int kStage = kTileA + kTileB;              // 32 KB
constexpr int kAccCols = kTokBlock;                  // int32 accumulator columns per buffer
constexpr int kEpiWarps = 8;
constexpr int kScaleBytes = kEpiWarps * (kTokBlock / 2) * 4;     // token scales of each warp's half tile

template <bool SWIGLU, int STAGES>
struct I8PairCfg {
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    static constexpr int kOutBytes = kEpiWarps * I8RowWriter<SWIGLU>::kBytes;
    static constexpr int kRingBytes = STAGES * kStage;
    static constexpr int kNumBars = 2 * STAGES + 2 + 2 + 1;
    static constexpr int kSmemBytes =
        1024 + kRingBytes + kOutBytes + kScaleBytes + 8 * kNumBars + 64 + 2 * (kMaxExperts + 1) * 4;
    static_assert(kSmemBytes + 64 <= kSmemLimit, "shared memory");
};

template <bool SWIGLU, int STAGES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(320, 1)
grouped_gemm_i8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                            const I8Params ip) {
    using C = I8PairCfg<SWIGLU, STAGES>;
    constexpr int kFeatPerTile = SWIGLU ? 128 : 256;         // output features per pair tile
    const Params &p = ip.p;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = smem;                                    // STAGES x [A own 128 rows | B own rows]
    uint8_t *out_s = ring + C::kRingBytes;                   // per epilogue warp: 32 token rows
    float *scale_s = reinterpret_cast<float *>(out_s + C::kOutBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(out_s + C::kOutBytes + kScaleBytes);
    uint64_t *full_bar = bars;                               // used in the leading CTA: both CTAs' bytes
    uint64_t *empty_bar = full_bar + STAGES;                 // each CTA's own (MMA commit to both)
    uint64_t *tfull_bar = empty_bar + STAGES;                // each CTA's own (MMA commit to both)
    uint64_t *tempty_bar = tfull_bar + 2;                    // used in the leading CTA: 8 warp arrivals per CTA
    uint64_t *drain_bar = tempty_bar + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *off_s = reinterpret_cast<int *>(tmem_holder + 16);
    int *pre_s = off_s + (kMaxExperts + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());   // 0 = leading CTA of the pair
    const int E = p.E;
    const int MB = (p.m_out + kFeatPerTile - 1) / kFeatPerTile;     // feature blocks
    const int KB = (p.K + kI8BK - 1) / kI8BK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull_bar[b], 1);
            mbar_init(&tempty_bar[b], 2 * kEpiWarps);         // every epilogue warp of both CTAs
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
        tmem_alloc_pair(tmem_holder, 2 * kAccCols);
        tmem_relinquish_pair();
    }
    griddep_wait();
    build_tile_prefix<C::kThreads>(p.offsets, E, MB, kTokBlock, off_s, pre_s, p.P, p.err);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();                                          // barriers of both CTAs initialised
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    TileFeed<kTokBlock, 32> feed(pre_s, off_s, E, MB, static_cast<int>(cluster_id_x()), static_cast<int>(cluster_count_x()));
    TileInfo ti;

    if (warp == 0) {
        // ============================ TMA producer (both CTAs) ==================
        const uint64_t pol = l2_policy_evict_last();
        const bool issuer = lane == 0;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && feed.next(ti)) {
            const int b_row = ti.row0 + rank * (ti.n_mma / 2);       // the non-leading CTA's shift
            const int a_row = ti.e * p.w_rows + ti.mb * 256 + 128 * rank;
            for (int kb = 0; kb < KB; ++kb) {
                ok = warp_wait(&empty_bar[stage], phase ^ 1, abort_flag, p.err, 64);
                if (!ok) break;
                if (issuer) {
                    const uint32_t full_leader = cluster_map(smem_u32(&full_bar[stage]), 0);
                    uint8_t *st = ring + stage * kStage;
                    if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2u * kStage);
                    if (SWIGLU)
                        tma_load_5d_pair(st, &tmA, full_leader, kb * kI8BK, 0, 0, ti.mb * 8 + 4 * rank, ti.e, pol);
                    else
                        tma_load_2d_pair(st, &tmA, full_leader, kb * kI8BK, a_row, pol);
                    tma_load_2d_pair(st + kTileA, &tmB, full_leader, kb * kI8BK, b_row, pol);
                }
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
        }
    } else if (warp == 1) {
        // ============================ MMA issuer (leading CTA) ==================
        if (rank == 0) {
            const uint32_t ring_lo = desc_low(smem_u32(ring));
            int stage = 0;
            uint32_t phase = 0;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true;
            while (ok && feed.next(ti)) {
                const uint32_t idesc = idesc_i8_i32(kPairM, ti.n_mma);
                ok = warp_wait(&tempty_bar[buf], bphase ^ 1, abort_flag, p.err, 64);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t d = tmem_base + buf * kAccCols;
                for (int kb = 0; kb < KB; ++kb) {
                    ok = warp_wait(&full_bar[stage], phase, abort_flag, p.err, 0);
                    if (!ok) break;
                    const uint32_t a = ring_lo + stage * (kStage >> 4);
                    umma_i8_stage_pair(d, a, a + (kTileA >> 4), idesc, kb != 0, &empty_bar[stage]);
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                if (elect_one()) umma_commit_pair(&tfull_bar[buf], 0x3);
                if (++buf == 2) { buf = 0; bphase ^= 1; }
            }
            if (elect_one()) umma_commit_pair(drain_bar, 0x1);
            volatile int never = 0;
            mbar_wait(drain_bar, 0, &never, p.err);
        }
    } else {
        // ====================== warps 2-9: epilogue (both CTAs) =================
        const int q = warp & 3;                              // TMEM lane quarter of this warp
        const int h = (warp - 2) >> 2;                       // column half: warps 2-5 first, 6-9 second
        const uint32_t tempty_leader0 = cluster_map(smem_u32(&tempty_bar[0]), 0);
        const uint32_t tempty_leader1 = cluster_map(smem_u32(&tempty_bar[1]), 0);
        const I8RowWriter<SWIGLU> writer(out_s + (warp - 2) * I8RowWriter<SWIGLU>::kBytes);
        float *sx_s = scale_s + (warp - 2) * (kTokBlock / 2);
        int buf = 0;
        uint32_t bphase = 0;
        // TMEM accumulator buffer handed back to the MMA issuer once this
        // warp's last tcgen05.ld of the tile has completed. The arrive orders
        // only those loads, so it is relaxed: a release would first wait for
        // the warp's outstanding global stores.
        auto release = [&]() {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(buf ? tempty_leader1 : tempty_leader0);
        };
        // A tile's scales are loaded while the tile before it is stored: the weight
        // rows' and, one per lane, the tokens' of this half, chunks [c_lo, c_hi) of 32.
        float sw_next[4], sx_next[kTokBlock / 64];
        auto fetch = [&]() {
            const int nch = (ti.valid + 31) >> 5, split = (nch + 1) >> 1;
            const int lo = h ? split : 0, hi = h ? nch : split;
            i8_weight_scales<SWIGLU>(ip, ti.e, ti.mb * kFeatPerTile + (SWIGLU ? 64 * rank + 16 * q : 128 * rank + 32 * q),
                                     sw_next);
#pragma unroll
            for (int c = 0; c < kTokBlock / 64; ++c) {
                const int n = 32 * (lo + c) + lane;
                sx_next[c] = lo + c < hi && n < ti.valid ? __ldg(ip.x_sf + ti.row0 + n) : 0.f;
            }
        };
        bool more = feed.next(ti);
        if (more) fetch();
        while (more) {
            const int nch = (ti.valid + 31) >> 5;
            const int split = (nch + 1) >> 1;
            const int c_lo = h ? split : 0, c_hi = h ? nch : split;
            const int f0 = ti.mb * kFeatPerTile + (SWIGLU ? 64 * rank + 16 * q : 128 * rank + 32 * q);
            const int row0 = ti.row0, valid = ti.valid;
            float sw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sw[i] = sw_next[i];
#pragma unroll
            for (int c = 0; c < kTokBlock / 64; ++c) sx_s[32 * c + lane] = sx_next[c];
            __syncwarp();
            if (!warp_wait(&tfull_bar[buf], bphase, abort_flag, p.err, 128)) break;
            tc_fence_after_sync();
            more = feed.next(ti);
            if (more) fetch();
            if (c_lo >= c_hi) {
                release();
                if (++buf == 2) { buf = 0; bphase ^= 1; }
                continue;
            }
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kAccCols;
            auto load = [&](uint32_t (&a)[16], uint32_t (&b)[16], int c) {
                tmem_ld_16x256b_x4(tb + 32 * c, a);
                tmem_ld_16x256b_x4(tb + (16u << 16) + 32 * c, b);
            };
            auto chunk = [&](const uint32_t (&a)[16], const uint32_t (&b)[16], int c) {
                writer.write(p, a, b, sw, sx_s + 32 * (c - c_lo), f0, row0 + 32 * c, valid - 32 * c);
            };
            // two register sets: the next 32 columns load while this set is stored
            uint32_t a0[16], b0[16], a1[16], b1[16];
            load(a0, b0, c_lo);
            tmem_wait_ld();
            for (int c = c_lo;; c += 2) {
                const bool more_a = c + 1 < c_hi;
                if (more_a) load(a1, b1, c + 1); else release();
                chunk(a0, b0, c);
                if (!more_a) break;
                tmem_wait_ld();
                const bool more_b = c + 2 < c_hi;
                if (more_b) load(a0, b0, c + 2); else release();
                chunk(a1, b1, c + 1);
                if (!more_b) break;
                tmem_wait_ld();
            }
            if (++buf == 2) { buf = 0; bphase ^= 1; }
        }
    }

    // every role is done: the next kernel may start its set-up now
    griddep_launch_dependents();
    __syncthreads();
    if (*abort_flag) {
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
    cluster_sync();                                          // no remote arrival or MMA left in flight
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, 2 * kAccCols);
    }
}

template <bool SWIGLU>
cudaError_t run_i8_pair(const I8GemmArgs &g, cudaStream_t s) {
    constexpr int STAGES = 6;
    using C = I8PairCfg<SWIGLU, STAGES>;
    CUtensorMap ta, tb;
    const uint64_t K = static_cast<uint64_t>(g.base.K);
    const bool map_a = SWIGLU ? make_gate_up_map(&ta, g.base.w, g.base.E, g.base.m_out, K, 4)
                              : make_map(&ta, g.base.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K,
                                         static_cast<uint64_t>(g.base.E) * g.base.w_rows, kI8BK, 128,
                                         CU_TENSOR_MAP_SWIZZLE_128B);
    if (g.base.perm || !map_a ||
        !make_map(&tb, g.base.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, static_cast<uint64_t>(g.base.P), kI8BK, kBBox,
                  CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    auto kern = grouped_gemm_i8_pair_kernel<SWIGLU, STAGES>;
    cudaError_t st = ensure_dynamic_smem(kern, C::kSmemBytes);
    if (st != cudaSuccess) return st;
    constexpr int kFeat = SWIGLU ? 128 : 256;
    const long long MB = (g.base.m_out + kFeat - 1) / kFeat;
    const long long max_tiles =
        ((static_cast<long long>(g.base.P) + kTokBlock - 1) / kTokBlock + std::min(g.base.E, g.base.P)) * MB;
    const int pairs = static_cast<int>(std::min<long long>(num_sms() / 2, max_tiles));
    if (pairs <= 0) return cudaSuccess;
    return launch_pdl(kern, dim3(2 * pairs), dim3(C::kThreads), C::kSmemBytes, s, ta, tb, make_i8_params(g, kTokBlock));
}

}  // namespace

cudaError_t launch_grouped_gemm_i8_pair(const I8GemmArgs &g, cudaStream_t s) {
    if (g.base.P == 0) return cudaSuccess;
    return g.base.swiglu ? run_i8_pair<true>(g, s) : run_i8_pair<false>(g, s);
}

}  // namespace moe
