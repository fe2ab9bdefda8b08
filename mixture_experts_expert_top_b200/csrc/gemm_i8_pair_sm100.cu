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
//  - gate/up: CTA r holds the gate rows of features fb*128 + 64r + [0, 64) in
//    its A rows 0-63 and the up rows of the same features in rows 64-127; the
//    warps of matching gate and up lanes swap halves of each 32-token chunk
//    through shared memory and form act for 16 tokens each.
//  - down: CTA r holds output features fb*256 + 128r + [0, 128).
//  - Warp 0 loads (both CTAs), warp 1 issues the MMAs (leading CTA) and owns
//    TMEM, warps 2-9 run the epilogue over a double-buffered 2 x 256-column
//    int32 accumulator.
// Every mbarrier wait is bounded; the named-barrier hand-off between epilogue
// warps is entered only after a bounded wait succeeded, and both warps of a
// pair take the same number of steps.
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
constexpr int kPairXchgBytes = 2 * 2 * 16 * 32 * 4;  // one warp pair's gate/up hand-off: 2 buffers x 2 x 16 x 32 fp32
constexpr int kScaleBytes = kEpiWarps * 2 * 32 * 4;  // token scales of a chunk: per warp, two buffers

template <bool SWIGLU, int STAGES>
struct I8PairCfg {
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    static constexpr int kXchgBytes = SWIGLU ? 4 * kPairXchgBytes : 0;
    static constexpr int kRingBytes = STAGES * kStage;
    static constexpr int kNumBars = 2 * STAGES + 2 + 2 + 1;
    static constexpr int kSmemBytes =
        1024 + kRingBytes + kXchgBytes + kScaleBytes + 8 * kNumBars + 64 + 2 * (kMaxExperts + 1) * 4;
    static_assert(kSmemBytes + 64 <= kSmemLimit, "shared memory");
};

// Named barriers of the gate/up epilogue (barrier 0 is __syncthreads): per
// warp pair pq (0-3), "go" carries the gate warp's decision for the tile,
// "xchg" separates the writes and reads of one chunk's hand-off buffer.
__device__ __forceinline__ int bar_go(int pq) { return 1 + pq; }
__device__ __forceinline__ int bar_xchg(int pq) { return 5 + pq; }

__device__ __forceinline__ void named_bar_sync(int id, int nthreads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// decode_tile's row count rounded up to 32.
__device__ __forceinline__ TileInfo pair_tile(int tile, const int *pre, const int *off, int E, int MB) {
    TileInfo t = decode_tile(tile, pre, off, E, MB, kTokBlock);
    t.n_mma = (t.valid + 31) & ~31;
    return t;
}

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
    float *xchg = reinterpret_cast<float *>(ring + C::kRingBytes);   // gate/up hand-off buffers
    float *scale_s = reinterpret_cast<float *>(ring + C::kRingBytes + C::kXchgBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + C::kRingBytes + C::kXchgBytes + kScaleBytes);
    uint64_t *full_bar = bars;                               // used in the leading CTA: both CTAs' bytes
    uint64_t *empty_bar = full_bar + STAGES;                 // each CTA's own (MMA commit to both)
    uint64_t *tfull_bar = empty_bar + STAGES;                // each CTA's own (MMA commit to both)
    uint64_t *tempty_bar = tfull_bar + 2;                    // used in the leading CTA: 8 warp arrivals per CTA
    uint64_t *drain_bar = tempty_bar + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    volatile int *go_flag = reinterpret_cast<volatile int *>(tmem_holder + 2);     // [4]
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
    const int total_tiles = pre_s[E];
    const int first_tile = static_cast<int>(cluster_id_x());
    const int tile_step = static_cast<int>(cluster_count_x());

    if (warp == 0) {
        // ============================ TMA producer (both CTAs) ==================
        if (lane == 0) {
            const uint64_t pol = l2_policy_evict_last();
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = first_tile; tile < total_tiles && ok; tile += tile_step) {
                const TileInfo ti = pair_tile(tile, pre_s, off_s, E, MB);
                const int half = ti.n_mma / 2;                       // token rows from each CTA
                const uint32_t tx = 2u * kStage;
                const int b_row = ti.row0 + rank * half;             // the non-leading CTA's shift
                // this CTA's A rows: 64 gate and the matching 64 up rows, or 128 rows
                const int r0 = SWIGLU ? ti.e * p.w_rows + ti.mb * 128 + 64 * rank
                                      : ti.e * p.w_rows + ti.mb * 256 + 128 * rank;
                for (int kb = 0; kb < KB; ++kb) {
                    ok = mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag, p.err, 128);
                    if (!ok) break;
                    const uint32_t full_leader = cluster_map(smem_u32(&full_bar[stage]), 0);
                    uint8_t *st = ring + stage * kStage;
                    if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], tx);
                    tma_load_2d_pair(st, &tmA, full_leader, kb * kI8BK, r0, pol);
                    if (SWIGLU) tma_load_2d_pair(st + kTileA / 2, &tmA, full_leader, kb * kI8BK, r0 + p.m_out, pol);
                    tma_load_2d_pair(st + kTileA, &tmB, full_leader, kb * kI8BK, b_row, pol);
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        // ============================ MMA issuer (leading CTA) ==================
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true;
            for (int tile = first_tile; tile < total_tiles && ok; tile += tile_step) {
                const TileInfo ti = pair_tile(tile, pre_s, off_s, E, MB);
                const uint32_t idesc = idesc_i8_i32(kPairM, ti.n_mma);
                ok = mbar_wait(&tempty_bar[buf], bphase ^ 1, abort_flag, p.err);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t d = tmem_base + buf * kAccCols;
                for (int kb = 0; kb < KB; ++kb) {
                    ok = mbar_wait(&full_bar[stage], phase, abort_flag, p.err, 0);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t st = smem_u32(ring + stage * kStage);
                    const uint64_t da = sw128_kmajor_desc(st);
                    const uint64_t db = sw128_kmajor_desc(st + kTileA);
#pragma unroll
                    for (int k = 0; k < kI8BK / 32; ++k)
                        umma_i8_ss_pair(d, da + 2 * k, db + 2 * k, idesc, (kb | k) != 0);
                    umma_commit_pair(&empty_bar[stage], 0x3);
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                umma_commit_pair(&tfull_bar[buf], 0x3);
                if (++buf == 2) { buf = 0; bphase ^= 1; }
            }
            umma_commit_pair(drain_bar, 0x1);
            volatile int never = 0;
            mbar_wait(drain_bar, 0, &never, p.err);
        }
    } else {
        // ====================== warps 2-9: epilogue (both CTAs) =================
        const int q = warp & 3;                              // TMEM lane quarter of this warp
        const int h = (warp - 2) >> 2;                       // column half: warps 2-5 first, 6-9 second
        const bool gate_warp = q < 2;                        // gate/up: which rows this warp's lanes hold
        const int pq = (q & 1) + 2 * h;                      // gate/up: warp pair index
        const uint32_t tempty_leader0 = cluster_map(smem_u32(&tempty_bar[0]), 0);
        const uint32_t tempty_leader1 = cluster_map(smem_u32(&tempty_bar[1]), 0);
        float *xb = xchg + pq * (kPairXchgBytes / 4);        // [buffer][giver: gate, up][16 tokens][32 lanes]
        float *sx_w = scale_s + (warp - 2) * 64;             // [buffer][32 tokens]
        const int f_in_tile = SWIGLU ? 64 * rank + 32 * (q & 1) + lane : 128 * rank + 32 * q + lane;
        int buf = 0;
        uint32_t bphase = 0, xbuf = 0;
        // TMEM accumulator buffer handed back to the MMA issuer once this
        // warp's last tcgen05.ld of the tile has completed. The arrive orders
        // only those loads, so it is relaxed: a release would first wait for
        // the warp's outstanding global stores.
        auto release = [&]() {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(buf ? tempty_leader1 : tempty_leader0);
        };
        for (int tile = first_tile; tile < total_tiles; tile += tile_step) {
            const TileInfo ti = pair_tile(tile, pre_s, off_s, E, MB);
            const int f = ti.mb * kFeatPerTile + f_in_tile;
            const bool f_ok = f < p.m_out;
            const size_t w_row = static_cast<size_t>(ti.e) * p.w_rows + f;
            // the scale of the accumulator row in this thread's TMEM lane (gate/up:
            // a gate row in a gate warp, the matching up row in an up warp)
            const float sw = f_ok ? __ldg(ip.w_sf + w_row + (SWIGLU && !gate_warp ? p.m_out : 0)) : 0.f;
            if (!SWIGLU || gate_warp) {
                const bool ok =
                    __shfl_sync(0xffffffffu, mbar_wait(&tfull_bar[buf], bphase, abort_flag, p.err, 512), 0);
                if (!SWIGLU && !ok) break;
                // gate/up: one decision for the warp pair (the barriers below are collective)
                if (SWIGLU && lane == 0) go_flag[pq] = ok ? 1 : 0;
            }
            if (SWIGLU) {
                named_bar_sync(bar_go(pq), 64);
                if (!go_flag[pq]) break;
                // the phase has completed (the gate warp saw it): this returns at
                // once and orders this warp's TMEM reads after the MMAs
                if (!gate_warp) mbar_wait(&tfull_bar[buf], bphase, abort_flag, p.err, 512);
            }
            tc_fence_after_sync();
            // this half's columns: chunks [c_lo, c_hi) of 32
            const int nch = (ti.valid + 31) >> 5;
            const int split = (nch + 1) >> 1;
            const int c_lo = h ? split : 0, c_hi = h ? nch : split;
            if (c_lo >= c_hi) {
                release();
                if (++buf == 2) { buf = 0; bphase ^= 1; }
                continue;
            }
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kAccCols;
            uint16_t *col = p.out + static_cast<size_t>(ti.row0) * p.m_out + f;
            // the chunk's token scales, one per lane, into this warp's buffer
            auto scales = [&](int c0) {
                sx_w[xbuf * 32 + lane] = c0 + lane < ti.valid ? __ldg(ip.x_sf + ti.row0 + c0 + lane) : 0.f;
                __syncwarp();
            };
            auto chunk = [&](const uint32_t (&v)[32], int c0) {
                scales(c0);
                const float *sx = sx_w + xbuf * 32;
                if constexpr (!SWIGLU) {
                    if (f_ok) {
                        uint16_t *dst = col + static_cast<size_t>(c0) * p.m_out;
                        const int n = min(32, ti.valid - c0);
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (j < n) *dst = i8_down(v[j], sw, sx[j]);
                            dst += p.m_out;
                        }
                    }
                } else {
                    // this warp's 16 tokens of the chunk: 0-15 (gate warp) or 16-31 (up warp)
                    const int my_half = gate_warp ? 0 : 16;
                    float *give = xb + xbuf * (2 * 16 * 32) + (gate_warp ? 0 : 16 * 32);
                    const float *take = xb + xbuf * (2 * 16 * 32) + (gate_warp ? 16 * 32 : 0);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int o = gate_warp ? 16 + j : j;            // the partner's tokens
                        give[j * 32 + lane] = i8_scaled(gate_warp ? v[16 + j] : v[j], sw, sx[o]);
                    }
                    named_bar_sync(bar_xchg(pq), 64);
                    if (f_ok) {
                        uint16_t *dst = col + static_cast<size_t>(c0 + my_half) * p.m_out;
                        const int n = ti.valid - c0 - my_half;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (j < n) {
                                const float other = take[j * 32 + lane];
                                const float mine = i8_scaled(gate_warp ? v[j] : v[16 + j], sw, sx[my_half + j]);
                                *dst = i8_act(gate_warp ? mine : other, gate_warp ? other : mine);
                            }
                            dst += p.m_out;
                        }
                    }
                }
                xbuf ^= 1;
            };
            // two register sets: the next 32 columns load while this set is stored
            const int c_end = 32 * c_hi;
            uint32_t va[32], vb[32];
            tmem_ld_32x32b_x32(tb + 32 * c_lo, va);
            tmem_wait_ld();
            for (int c0 = 32 * c_lo;; c0 += 64) {
                const bool more_a = c0 + 32 < c_end;
                if (more_a) tmem_ld_32x32b_x32(tb + c0 + 32, vb); else release();
                chunk(va, c0);
                if (!more_a) break;
                tmem_wait_ld();
                const bool more_b = c0 + 64 < c_end;
                if (more_b) tmem_ld_32x32b_x32(tb + c0 + 64, va); else release();
                chunk(vb, c0 + 32);
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
    constexpr int STAGES = SWIGLU ? 5 : 6;
    using C = I8PairCfg<SWIGLU, STAGES>;
    CUtensorMap ta, tb;
    const uint64_t a_rows = static_cast<uint64_t>(g.base.E) * g.base.w_rows;
    const uint64_t K = static_cast<uint64_t>(g.base.K);
    if (g.base.perm ||
        !make_map(&ta, g.base.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, a_rows, kI8BK, SWIGLU ? 64 : 128,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
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
