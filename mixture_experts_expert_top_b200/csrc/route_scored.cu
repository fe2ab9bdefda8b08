// route_scored.cu -- routing by scores: softmax or sigmoid of the router
// logits, a selection bias per expert (load balance), expert groups, top-k and
// weights, one warp per token.
//
// For the logits l of a token (NaN counts as -inf) and the bias b:
//   s_e = exp(l_e - m) / sum_i exp(l_i - m), m = max l      (softmax)
//   s_e = 1 / (1 + exp(-l_e))                               (sigmoid)
//   c_e = s_e + b_e        selection order; without a bias the order of l
//   G_g = sum of the group_top largest c of group g; the topk_group largest
//         groups stay, equal ones by the lower index
//   ids = the top_k largest c of those groups, equal ones by the lower id
//   w_j = scale * s_j / sum_i s_i (renormalised) or scale * s_j
// Both scores rise with the logit, so without a bias the order is that of the
// logits themselves, compared exactly as fp32 keys. With one, two experts may
// differ in the last bits of s + b alone, so the order is that of 64-bit
// values: scores are formed in fp32 with a bound on their error, the selection
// runs on them, and it stands if every gap that decided it (between
// consecutive selected experts, to the first one left out, and between the
// last group kept and the first one dropped) exceeds twice the bound. Where one
// does not (about 1 row in 1000 of 256 experts), the experts down to the next
// such gap are ordered by their 64-bit values, one per lane (refine_64); where
// that does not settle it either (groups that tie, experts that are switched
// off), the whole row is (select_64).
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "launch_util.cuh"
#include "route_dev.cuh"

namespace moe {
namespace {

constexpr int kWarpsPerBlock = 4;
// From this many rows on (20 warps on each of 148 SMs) one warp weighs several
// rows: 16384 x 256 with groups 18.4 -> 16.2 us, 4096 x 128 4.1 -> 3.6 us. With
// fewer the wait for the block's other warps shows (2048 x 128 3.3 -> 3.6 us).
constexpr int kSharedWeighingRows = 20 * 148;

struct RouterArgs {
    const void *logits;
    const float *bias;
    int T, E, k, n_shared;
    int score, n_group, topk_group, group_top, renormalize;
    float scale;
    int32_t *ids;
    float *w;
    int vec;                                // rows and lanes' shares are 16-byte aligned
    int group_shift;                        // log2 of the lanes that hold one group; -1: groups end inside lanes
};

__device__ __forceinline__ float load_logit(const float *p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// The lane's N consecutive values from e0 on (`fill` past E), in 16-byte loads where `vec` allows.
template <int N>
__device__ __forceinline__ void load_lane(const float *row, int e0, int E, bool vec, float fill, float (&x)[N]) {
    if (N % 4 == 0 && vec) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 v = e0 < E ? *reinterpret_cast<const float4 *>(row + e0 + 4 * i) : make_float4(fill, fill, fill, fill);
            x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = e0 + i < E ? row[e0 + i] : fill;
}

template <int N>
__device__ __forceinline__ void load_lane(const __nv_bfloat16 *row, int e0, int E, bool vec, float fill, float (&x)[N]) {
    if (N % 8 == 0 && vec) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            const uint4 v = e0 < E ? *reinterpret_cast<const uint4 *>(row + e0 + 8 * i) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[8 * i + j] = e0 < E ? bf16_bits_to_float((w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu) : fill;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = e0 + i < E ? __bfloat162float(row[e0 + i]) : fill;
}

// The logit as the scores take it: NaN is -inf (logit_key makes -0 equal +0).
__device__ __forceinline__ float clean_logit(float x) { return fmaxf(x, -INFINITY); }

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / x within 2^-23 (relative), 0 for +inf; exp(x) within 2^-22 + 2^-23 |x|.
// Both flush subnormals.
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float fast_exp(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504f));
    return r;
}

__device__ __forceinline__ float warp_min(float v) {
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Order-preserving map of a double onto uint64 (larger value, larger key); NaN
// counts as -inf, -0 as +0. Key 0 is below every value: "not a candidate".
__device__ __forceinline__ uint64_t choice_key(double x) {
    if (x != x) x = -INFINITY;
    if (x == 0.0) x = 0.0;
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x));
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t u = __shfl_xor_sync(0xffffffffu, v, o);
        v = u > v ? u : v;
    }
    return v;
}

// Lane g holds group g's key (g < n_group): the mask of the `keep` largest,
// equal ones by the lower index.
template <typename Key>
__device__ __forceinline__ uint32_t keep_groups(Key mine, int n_group, int keep) {
    const int lane = threadIdx.x & 31;
    int ahead = 0;
    for (int o = 0; o < n_group; ++o) {
        const Key other = __shfl_sync(0xffffffffu, mine, o);
        ahead += (other > mine || (other == mine && o < lane)) ? 1 : 0;
    }
    return __ballot_sync(0xffffffffu, lane < n_group && ahead < keep);
}

// 64-bit scores of the lane's experts (lane l: l*N .. l*N+N-1). The logits are
// read again, so that callers that rarely come here keep theirs in registers.
// No branch between the exponentials: their latencies overlap.
template <int N, typename L>
__device__ __forceinline__ void scores_64(const RouterArgs &a, const L *row, float m, double (&s)[N]) {
    const int e0 = (threadIdx.x & 31) * N;
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = e0 + i < a.E ? clean_logit(load_logit(row + e0 + i)) : -INFINITY;
    if (a.score == MOE_SCORE_SOFTMAX) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s[i] = x[i] == m ? (m == -INFINITY ? 0.0 : 1.0) : exp(static_cast<double>(x[i]) - m);
            sum += s[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (sum > 0.0) s[i] /= sum;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = exp(-static_cast<double>(x[i]));
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = 1.0 / (1.0 + s[i]);
    }
}

// Whether each of the lane's experts is in a kept group, as bits, by 64-bit
// group values: sums of the group_top largest choices (scores without a bias).
template <int N, typename L>
__device__ __noinline__ uint32_t groups_64(const RouterArgs &a, const L *row, float m, double *by_s) {
    const int lane = threadIdx.x & 31;
    const int e0 = lane * N;
    const int size = a.E / a.n_group, gs = a.group_shift;
    double by[N];
    scores_64<N>(a, row, m, by);
    double top1 = -INFINITY, top2 = -INFINITY;
    auto add = [&](double v) {
        if (v > top1) { top2 = top1; top1 = v; }
        else if (v > top2) top2 = v;                             // NaN is never larger: it counts as -inf
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (e0 + i < a.E) {
            if (a.bias) by[i] += static_cast<double>(a.bias[e0 + i]);
            if (gs >= 0) add(by[i]); else by_s[e0 + i] = by[i];
        }
    }
    if (gs >= 0) {
        for (int o = 1; o < (1 << gs); o <<= 1) {
            const double u1 = __shfl_xor_sync(0xffffffffu, top1, o), u2 = __shfl_xor_sync(0xffffffffu, top2, o);
            top2 = fmax(fmin(top1, u1), fmax(top2, u2));
            top1 = fmax(top1, u1);
        }
        top1 = __shfl_sync(0xffffffffu, top1, (lane << gs) & 31);
        top2 = __shfl_sync(0xffffffffu, top2, (lane << gs) & 31);
    } else {
        __syncwarp();
        if (lane < a.n_group)
            for (int i = 0; i < size; ++i) add(by_s[lane * size + i]);
        __syncwarp();
    }
    const uint64_t gk = lane < a.n_group ? choice_key(a.group_top == 2 ? top1 + top2 : top1) : 0;
    const uint32_t kept = keep_groups(gk, a.n_group, a.topk_group);
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (e0 + i < a.E) bits |= ((kept >> ((e0 + i) / size)) & 1u) << i;
    return bits;
}

// The selection in 64 bits among the lane's experts in `bits`. Returns slot j's
// expert in lane j. Only with a bias: without one the logits decide.
template <int N, typename L>
__device__ __noinline__ int select_64(const RouterArgs &a, const L *row, float m, uint32_t bits) {
    const int lane = threadIdx.x & 31;
    const int e0 = lane * N;
    double s[N];
    scores_64<N>(a, row, m, s);
    uint64_t key[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        key[i] = e0 + i < a.E && ((bits >> i) & 1u) ? choice_key(s[i] + static_cast<double>(a.bias[e0 + i])) : 0;
    int my_id = 0;
    for (int j = 0; j < a.k; ++j) {
        uint64_t local = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) local = key[i] > local ? key[i] : local;
        const uint64_t best = warp_max64(local);
        uint32_t cand = 0xffffffffu;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
            if (key[i] == best) cand = static_cast<uint32_t>(e0 + i);
        const int bid = static_cast<int>(__reduce_min_sync(0xffffffffu, cand));
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e0 + i == bid) key[i] = 0;
        if (lane == j) my_id = bid;
    }
    return my_id;
}

// The order of `count` <= 32 candidates (lane j < count: expert id) by their
// 64-bit choices. Returns slot j's expert in lane j. One exponential per lane
// and a rank by comparison with the others: a fraction of select_64's latency,
// which a single row would add to the whole launch.
template <typename L>
__device__ __noinline__ int refine_64(const RouterArgs &a, const L *row, float m, int id, int count) {
    __shared__ int slot_s[kWarpsPerBlock][32];
    const int lane = threadIdx.x & 31;
    const bool soft = a.score == MOE_SCORE_SOFTMAX;
    double sum = 0.0;
    if (soft) {
        for (int e = lane; e < a.E; e += 32) {
            const float x = clean_logit(load_logit(row + e));
            sum += x == m ? 1.0 : exp(static_cast<double>(x) - m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    uint64_t key = 0;
    if (lane < count) {
        const float x = clean_logit(load_logit(row + id));
        double s;
        if (soft)
            s = m == -INFINITY ? 0.0 : (x == m ? 1.0 : exp(static_cast<double>(x) - m)) / sum;
        else
            s = 1.0 / (1.0 + exp(-static_cast<double>(x)));
        key = choice_key(s + static_cast<double>(a.bias[id]));
    }
    int rank = 0;
#pragma unroll 4
    for (int o = 0; o < count; ++o) {
        const uint64_t other = __shfl_sync(0xffffffffu, key, o);
        const int oid = __shfl_sync(0xffffffffu, id, o);
        rank += other > key || (other == key && oid < id) ? 1 : 0;
    }
    int *slots = slot_s[threadIdx.x >> 5];
    if (lane < count) slots[rank] = id;
    __syncwarp();
    const int mine = lane < a.k ? slots[lane] : 0;
    __syncwarp();
    return mine;
}

// fp32 scores s and choices c = s + b of the lane's experts (lane l: l*N ..
// l*N+N-1), their smallest and largest value over the row, and a bound on |c -
// its 64-bit value|. In units of u = 2^-24: the exponential is within (4 + 2
// |x|) u; the reciprocal within 2u; adding b rounds by u |c|. A
// sigmoid passes on (1 - s) of its exponential's error: below 1.6 u, since s (1
// - s) <= 0.25 and s (1 - s) |x| <= 0.23; its sum 1 + e adds one and its
// reciprocal two of s <= 1: 4.6. A softmax term has its argument's rounding,
// u |d|, d = l - m, besides; s |d| <= 0.37 s_max; the sum of the terms adds N + 5
// roundings and its terms' average error (|d| averages below ln E < 7 over a
// softmax). The factor 1.25 covers the products of errors, 1e-37 what the
// exponential or the reciprocal flushes to zero.
template <int N>
__device__ __forceinline__ float scores_32(const RouterArgs &a, const float (&x)[N], float m, float (&s)[N], float (&c)[N],
                                           float &lo, float &hi) {
    const int e0 = (threadIdx.x & 31) * N;
    float err;
    if (a.score == MOE_SCORE_SOFTMAX) {
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s[i] = x[i] == m ? (m == -INFINITY ? 0.f : 1.f) : fast_exp(x[i] - m);
            z += s[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        const float inv = z > 0.f ? 1.0f / z : 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] *= inv;
        err = (N + 45.0f) * inv;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = fast_rcp(1.0f + fast_exp(-x[i]));
        err = 4.6f;
    }
    float b[N];
    if (a.bias) load_lane<N>(a.bias, e0, a.E, a.vec, 0.f, b);
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = a.bias ? fmaxf(s[i] + b[i], -INFINITY) : s[i];    // NaN counts as -inf
    lo = INFINITY;
    hi = -INFINITY;
    // with `vec` a lane's experts are all below E or none is
    if (!a.vec || e0 < a.E) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (a.vec || e0 + i < a.E) {
                lo = fminf(lo, c[i]);
                hi = fmaxf(hi, c[i]);
            }
    }
    lo = warp_min(lo);
    hi = warp_max(hi);
    if (lo == -INFINITY) {                                           // experts that are switched off
        lo = INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e0 + i < a.E && c[i] > -INFINITY) lo = fminf(lo, c[i]);
        lo = warp_min(lo);
    }
    return 0x1p-24f * 1.25f * (err + fmaxf(fabsf(lo), fabsf(hi))) + 1e-37f;
}

// a > b by more than `gap`, for the values of two keys in descending order. A
// missing candidate (key 0) is behind everything; equal keys are never apart.
__device__ __forceinline__ bool apart(uint32_t ka, uint32_t kb, float gap) {
    return kb == 0u || key_logit(ka) - key_logit(kb) > gap;
}

// Lane g holds group g's value as a key (0 from n_group on): the mask of the
// topk_group largest, equal ones by the lower index; the last one kept and the
// first one dropped (0: none).
__device__ __forceinline__ uint32_t pick_groups(const RouterArgs &a, uint32_t gk, uint32_t &last, uint32_t &first) {
    const int lane = threadIdx.x & 31;
    uint32_t kept = 0;
    last = 0;
    for (int j = 0; j < a.topk_group; ++j) {
        last = __reduce_max_sync(0xffffffffu, gk);
        const int win = __ffs(__ballot_sync(0xffffffffu, gk == last && lane < a.n_group && !((kept >> lane) & 1u))) - 1;
        kept |= 1u << win;
        if (lane == win) gk = 0u;
    }
    first = __reduce_max_sync(0xffffffffu, gk);
    return kept;
}

// Whether each of the lane's experts is in a kept group, as bits. by: what
// groups are valued by, within err_by of its 64-bit value.
template <int N>
__device__ __forceinline__ uint32_t kept_experts(const RouterArgs &a, const float (&by)[N], float err_by, float *by_s, bool &sure) {
    const int lane = threadIdx.x & 31;
    const int e0 = lane * N;
    const int size = a.E / a.n_group;
    float top1 = -INFINITY, top2 = -INFINITY;
    auto add = [&](float v) {
        top2 = fmaxf(top2, fminf(top1, v));
        top1 = fmaxf(top1, v);
    };
    uint32_t gk = 0;
    const int gs = a.group_shift;
    if (gs >= 0) {
        // whole lanes per group: each group's two largest by exchanges inside its lanes
#pragma unroll
        for (int i = 0; i < N; ++i) add(e0 + i < a.E ? by[i] : -INFINITY);
        for (int o = 1; o < (1 << gs); o <<= 1) {
            const float u1 = __shfl_xor_sync(0xffffffffu, top1, o), u2 = __shfl_xor_sync(0xffffffffu, top2, o);
            top2 = fmaxf(fminf(top1, u1), fmaxf(top2, u2));
            top1 = fmaxf(top1, u1);
        }
        // group g's value moves to lane g
        const float mine = a.group_top == 2 ? top1 + top2 : top1;
        const float g = __shfl_sync(0xffffffffu, mine, (lane << gs) & 31);
        gk = lane < a.n_group ? logit_key(g) : 0u;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e0 + i < a.E) by_s[e0 + i] = by[i];
        __syncwarp();
        if (lane < a.n_group) {
            for (int i = 0; i < size; ++i) add(by_s[lane * size + i]);
            gk = logit_key(a.group_top == 2 ? top1 + top2 : top1);
        }
        __syncwarp();
    }
    uint32_t last, first, bits = 0;
    const uint32_t kept = pick_groups(a, gk, last, first);
    // a sum of two: twice the error, and its own rounding below it
    if (err_by > 0.f) sure = apart(last, first, (a.group_top == 2 ? 8.0f : 2.0f) * err_by);
    if (gs >= 0) return (kept >> (lane >> gs)) & 1u ? 0xffffffffu : 0u;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (e0 + i < a.E) bits |= ((kept >> ((e0 + i) / size)) & 1u) << i;
    return bits;
}

// The selection by the logits themselves, exact. Returns slot j's expert in lane j.
template <int N>
__device__ __forceinline__ int select_logits(const RouterArgs &a, const float (&x)[N], uint32_t bits) {
    const int lane = threadIdx.x & 31;
    const int e0 = lane * N;
    uint32_t key[N];
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = e0 + i < a.E && ((bits >> i) & 1u) ? logit_key(x[i]) : 0u;
    int my_id = 0;
    for (int j = 0; j < a.k; ++j) {
        uint32_t local = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) local = max(local, key[i]);
        const uint32_t best = __reduce_max_sync(0xffffffffu, local);
        uint32_t cand = 0xffffffffu;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
            if (key[i] == best) cand = static_cast<uint32_t>(e0 + i);
        const uint32_t bid = __reduce_min_sync(0xffffffffu, cand);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (static_cast<uint32_t>(e0 + i) == bid) key[i] = 0u;
        if (lane == j) my_id = static_cast<int>(bid);
    }
    return my_id;
}

// Keys in descending order (odd-even merge sort, every step unrolled).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q && i + j + q < N; ++i)
                    if ((i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t hi = max(key[i + j], key[i + j + q]), lo = min(key[i + j], key[i + j + q]);
                        key[i + j] = hi;
                        key[i + j + q] = lo;
                    }
}

// The selection by c, within err of its 64-bit value. A key holds c on a grid
// from the smallest finite choice lo to the largest, hi, above the inverted
// expert id, so keys differ: each lane sorts its own once (minima and maxima
// only), and a slot takes one reduction over the lanes' largest. Grid value 0
// is an expert that is switched off. Returns slot j's expert in lane j, and in
// `count`: 0 if the 64-bit selection is the same, every gap being beyond the
// errors and the grid; c > 0 if the first c candidates (in lanes 0 .. c-1)
// hold it, but not surely in this order; -1 if it may be anywhere in `bits`,
// the lane's experts in kept groups. Groups that are too near are valued in 64
// bits on the way.
template <int N, typename L>
__device__ __forceinline__ int select_choices(const RouterArgs &a, const L *row, float m, const float (&c)[N], float err,
                                              float lo, float hi, double *by_s, int &count, uint32_t &bits) {
    constexpr int kIdBits = N <= 16 ? 9 : 10;
    constexpr uint32_t kIdMask = (1u << kIdBits) - 1u;
    constexpr float kSteps = static_cast<float>((1u << (32 - kIdBits)) - 4u);
    constexpr float kMagic = 8388608.0f + 1.0f;                  // 2^23: a grid value lands in the low mantissa bits
    const int lane = threadIdx.x & 31;
    const int e0 = lane * N;
    const int gs = a.group_shift;
    bits = 0xffffffffu;
    count = -1;
    const float unit = kSteps / (hi - lo);
    // twice the error and the two keys' rounding, one step each
    const float gap = ceilf(2.0f * err * unit) + 3.0f;
    // one value, an infinity, a span past the fp32 range (unit 0, and c - lo infinite), or a
    // range that the grid does not resolve: not here
    const bool grid_ok = lo < hi && hi - lo < INFINITY && unit < 3e37f && gap < 0.125f * kSteps;
    if (a.n_group > 1 && (gs < 0 || !grid_ok)) {
        bool sure = true;
        bits = kept_experts<N>(a, c, err, reinterpret_cast<float *>(by_s), sure);
        if (!sure) bits = groups_64<N, L>(a, row, m, by_s);
    }
    if (!grid_ok) return 0;
    const uint32_t gap_key = static_cast<uint32_t>(gap);
    uint32_t key[N];
#pragma unroll
    for (int i = 0; i < N; ++i)                                  // -inf gives a zero mantissa: grid value 0
        key[i] = __float_as_uint(fmaf(c[i] - lo, unit, kMagic)) * (1u << kIdBits) + (kIdMask - static_cast<uint32_t>(e0 + i));
    if (a.vec) {
        if (e0 >= a.E)
#pragma unroll
            for (int i = 0; i < N; ++i) key[i] = 0u;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = e0 + i < a.E && ((bits >> i) & 1u) ? key[i] : 0u;
    }
    if (a.vec && bits != 0xffffffffu)
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = (bits >> i) & 1u ? key[i] : 0u;
    sort_keys<N>(key);
    if (a.n_group > 1 && gs >= 0) {
        // groups of whole lanes, valued on the same grid: the two largest by exchanges
        uint32_t top1 = key[0], top2 = N > 1 ? key[N > 1 ? 1 : 0] : 0u;
        for (int o = 1; o < (1 << gs); o <<= 1) {
            const uint32_t u1 = __shfl_xor_sync(0xffffffffu, top1, o), u2 = __shfl_xor_sync(0xffffffffu, top2, o);
            top2 = max(min(top1, u1), max(top2, u2));
            top1 = max(top1, u1);
        }
        top1 >>= kIdBits;
        top2 >>= kIdBits;
        // the sum is -inf (0) where one of two is; below it the inverted group index, so
        // that values differ. Lanes behind the last group are behind every group.
        const uint32_t g = static_cast<uint32_t>(lane) >> gs;
        uint32_t v = a.group_top == 1 ? top1 : top2 == 0u ? 0u : top1 + top2;
        v = g < static_cast<uint32_t>(a.n_group) ? (v << 5) + (31u - g) + 1u : 0u;
        int ahead = 0;
#pragma unroll 4
        for (int o = 1 << gs; o < 32; o += 1 << gs) ahead += __shfl_xor_sync(0xffffffffu, v, o) > v ? 1 : 0;
        const bool kept = ahead < a.topk_group;
        const uint32_t last = __reduce_min_sync(0xffffffffu, kept ? v : 0xffffffffu);
        const uint32_t first = __reduce_max_sync(0xffffffffu, kept ? 0u : v);
        bits = kept ? 0xffffffffu : 0u;
        // a sum of two: twice the error, its own rounding below it, and twice the steps
        if (first != 0u && ((last - 1u) >> 5) - ((first - 1u) >> 5) <= (a.group_top == 2 ? 4u * gap_key : gap_key))
            bits = groups_64<N, L>(a, row, m, by_s);
        if (!bits)
#pragma unroll
            for (int i = 0; i < N; ++i) key[i] = 0u;
    }
    uint32_t my_key = 0;
    auto pop = [&](uint32_t best) {
        const bool mine = key[0] == best;
#pragma unroll
        for (int i = 0; i + 1 < N; ++i) key[i] = mine ? key[i + 1] : key[i];
        key[N - 1] = mine ? 0u : key[N - 1];
    };
#pragma unroll 2
    for (int j = 0; j < a.k; ++j) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
        pop(best);
        if (lane == j) my_key = best;
    }
    // the gap behind each slot, in grid steps (a missing candidate is behind
    // everything); an expert that is switched off (grid value 0) ties exactly
    auto near = [&](uint32_t k0, uint32_t k1) { return k1 != 0u && (k0 >> kIdBits) - (k1 >> kIdBits) <= gap_key; };
    uint32_t next = __reduce_max_sync(0xffffffffu, key[0]);
    const uint32_t after = __shfl_down_sync(0xffffffffu, my_key, 1);
    const uint32_t behind = lane + 1 < a.k ? after : next;
    const bool off = __any_sync(0xffffffffu, lane < a.k && (my_key >> kIdBits) == 0u);
    if (!off && !__any_sync(0xffffffffu, lane < a.k && near(my_key, behind))) {
        count = 0;
    } else if (!off) {
        // candidates down to a gap
        uint32_t last = __shfl_sync(0xffffffffu, my_key, a.k - 1);
        int n = a.k;
        while (n < 32 && near(last, next)) {
            pop(next);
            if (lane == n) my_key = next;
            ++n;
            last = next;
            next = __reduce_max_sync(0xffffffffu, key[0]);
        }
        if (!near(last, next) && (last >> kIdBits) != 0u) count = n;
    }
    return static_cast<int>(kIdMask - (my_key & kIdMask));
}

// The row's experts, that of slot j in lane j (j < k). x: the lane's logits; m:
// softmax, the row's largest logit.
template <int N, typename L>
__device__ __forceinline__ int select_row(const RouterArgs &a, const L *row, double *by_s, float (&x)[N], float &m) {
    const int e0 = (threadIdx.x & 31) * N;
    const bool soft = a.score == MOE_SCORE_SOFTMAX;
    m = -INFINITY;
    load_lane<N>(row, e0, a.E, a.vec, -INFINITY, x);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = clean_logit(x[i]);
        m = fmaxf(m, x[i]);
    }
    if (soft) m = warp_max(m);
    const bool by_logit = a.bias == nullptr;
    int id;
    if (by_logit && a.n_group == 1) {
        id = select_logits<N>(a, x, 0xffffffffu);
    } else if (by_logit && a.group_top == 1) {
        bool sure = true;
        id = select_logits<N>(a, x, kept_experts<N>(a, x, 0.f, reinterpret_cast<float *>(by_s), sure));      // exact
    } else {
        float s[N], c[N], lo, hi;
        const float err = scores_32<N>(a, x, m, s, c, lo, hi);
        if (by_logit) {
            bool sure = true;
            uint32_t bits = kept_experts<N>(a, s, err, reinterpret_cast<float *>(by_s), sure);
            if (!sure) bits = groups_64<N, L>(a, row, m, by_s);
            id = select_logits<N>(a, x, bits);
        } else {
            int count;
            uint32_t bits;
            id = select_choices<N, L>(a, row, m, c, err, lo, hi, by_s, count, bits);
            if (count > 0) id = refine_64<L>(a, row, m, id, count);
            if (count < 0) id = select_64<N, L>(a, row, m, bits);
        }
    }
    return id;
}

// The sum of exp(l - m) over the row in x.
template <int N>
__device__ __forceinline__ float row_sum(const RouterArgs &a, const float (&x)[N], float m) {
    const int e0 = (threadIdx.x & 31) * N;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (e0 + i < a.E) z += x[i] == m ? 1.0f : expf(x[i] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    return z;
}

// The weight of slot j in lane j of the W that hold token t, and the row's
// outputs. Renormalised, only ratios of scores count: softmax takes them
// relative to the largest selected logit, and so does a sigmoid whose selected
// scores are all below e^-60 (there s = exp(l) to fp32), so no sum underflows.
template <int W, typename L, typename Sum>
__device__ __forceinline__ void weigh_row(const RouterArgs &a, const L *row, int t, int id, float m, const Sum &sum_of) {
    const int slot = W == 32 ? threadIdx.x & 31 : threadIdx.x % W;
    const bool soft = a.score == MOE_SCORE_SOFTMAX;
    const bool in = W == 32 || t < a.T;                          // a block's last rows may be behind T
    const bool live = slot < a.k && in;
    float l = -INFINITY;
    bool off = false;
    if (live) {
        l = clean_logit(load_logit(row + id));
        off = a.bias && !(a.bias[id] > -INFINITY);
    }
    float lmax = off ? -INFINITY : l;
    if constexpr (W == 32) {
        lmax = warp_max(lmax);
    } else {
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) lmax = fmaxf(lmax, __shfl_xor_sync(0xffffffffu, lmax, o));
    }
    float s;
    if (soft && !a.renormalize) {
        const float z = sum_of();
        s = (l == m ? 1.0f : expf(l - m)) / z;
    } else if (soft || (a.renormalize && lmax < -60.0f)) {
        s = l == lmax ? 1.0f : expf(l - lmax);
    } else if (a.renormalize) {
        // times 2^100, which the quotient does not see: below -60 s is exp(l) to fp32, as the
        // square of its root, and neither leaves the normal range before the weight does
        const bool low = l < -60.0f;
        const float e = expf(low ? 0.5f * l : -l);
        s = low ? (e * 0x1p50f) * (e * 0x1p50f) : fast_rcp(1.0f + e) * 0x1p100f;
    } else {
        // below -60 s is exp(l) to fp32; from -87.3 on the reciprocal would flush it to 0
        const bool low = l < -60.0f;
        const float e = expf(low ? l : -l);
        s = low ? e : fast_rcp(1.0f + e);
    }
    if (off || l == -INFINITY || !live) s = 0.f;
    float wt = s;
    if (a.renormalize) {
        float sum = 0.f;                                             // slot order; lanes from k on add 0
        for (int j = 0; j < a.k; j += 8)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += __shfl_sync(0xffffffffu, s, j + i, W);
        wt = sum > 0.f ? __fdiv_rn(s, sum) : 0.f;
    }
    wt *= a.scale;
    shared_slot(slot, a.k, a.E, id, wt);
    const int K = a.k + a.n_shared;
    if (slot < K && in) {
        a.ids[static_cast<size_t>(t) * K + slot] = id;
        a.w[static_cast<size_t>(t) * K + slot] = wt;
    }
}

// 32 warps per SM up to 256 experts (64 registers): the row's work is a chain of
// reductions, and other warps fill its latency (16384 x 256 with groups, rows
// weighed one by one: 18.4 us; 75 registers 20.5 us, 48 registers 19.9). A warp
// selects one row. R rows are weighed by one warp, 32 / R lanes each: weights
// take a fifth of a row's instructions, for k of a warp's 32 lanes. Several
// rows selected by one warp in turn would wait longer than that saves (16384 x
// 256: 20.7 us for 2 rows, 21.4 for 4).
template <int N, typename L, int R>
__global__ void __launch_bounds__(kWarpsPerBlock * 32, N <= 8 ? 8 : 1)
route_scored_kernel(const __grid_constant__ RouterArgs a) {
    extern __shared__ double by_all[];                           // [kWarpsPerBlock][E], only with groups
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int t0 = blockIdx.x * kWarpsPerBlock;
    double *by_s = by_all + static_cast<size_t>(warp) * a.E;
    auto row_of = [&](int t) { return static_cast<const L *>(a.logits) + static_cast<size_t>(t) * a.E; };
    float x[N], m;
    if constexpr (R == 1) {
        const int t = t0 + warp;
        if (t >= a.T) return;
        const L *row = row_of(t);
        const int id = select_row<N, L>(a, row, by_s, x, m);
        weigh_row<32, L>(a, row, t, id, m, [&] { return row_sum<N>(a, x, m); });
    } else {
        constexpr int W = 32 / R;
        __shared__ int ids[kWarpsPerBlock * W];
        __shared__ float2 mz[kWarpsPerBlock];
        if (t0 + warp < a.T) {
            const int id = select_row<N, L>(a, row_of(t0 + warp), by_s, x, m);
            if (lane < W) ids[warp * W + lane] = id;
            if (a.score == MOE_SCORE_SOFTMAX && !a.renormalize) {
                const float z = row_sum<N>(a, x, m);
                if (lane == 0) mz[warp] = make_float2(m, z);
            }
        }
        __syncthreads();
        if (warp >= kWarpsPerBlock / R) return;
        const int r = warp * R + lane / W;                       // this lane's row; from T on nothing of it is used
        weigh_row<W, L>(a, row_of(t0 + r), t0 + r, ids[threadIdx.x], mz[r].x, [&] { return mz[r].y; });
    }
}

template <int N, typename L>
cudaError_t launch_n(RouterArgs a, cudaStream_t s) {
    a.vec = a.E % N == 0 && N * sizeof(L) % 16 == 0 && N % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 &&
            reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    const int size = a.E / a.n_group, lanes = size / N;
    a.group_shift = -1;
    if (size % N == 0 && (lanes & (lanes - 1)) == 0)
        for (a.group_shift = 0; (1 << a.group_shift) < lanes;) ++a.group_shift;
    const int blocks = (a.T - 1) / kWarpsPerBlock + 1;           // T up to 2^31 - 1
    const size_t sm = a.n_group > 1 ? static_cast<size_t>(kWarpsPerBlock) * a.E * sizeof(double) : 0;
    auto kernel = route_scored_kernel<N, L, 1>;
    if constexpr (N <= 8) {
        const int slots = a.k + a.n_shared;
        if (a.T >= kSharedWeighingRows && slots <= 16)
            kernel = slots <= 8 ? route_scored_kernel<N, L, 4> : route_scored_kernel<N, L, 2>;
    }
    return launch_pdl(kernel, dim3(blocks), dim3(kWarpsPerBlock * 32), sm, s, a);
}

template <typename L>
cudaError_t launch_l(const RouterArgs &a, cudaStream_t s) {
    const int n = (a.E + 31) / 32;
    if (n <= 1) return launch_n<1, L>(a, s);
    if (n <= 2) return launch_n<2, L>(a, s);
    if (n <= 4) return launch_n<4, L>(a, s);
    if (n <= 8) return launch_n<8, L>(a, s);
    if (n <= 16) return launch_n<16, L>(a, s);
    return launch_n<32, L>(a, s);
}

}  // namespace

cudaError_t launch_route_scored(const void *logits, const float *bias, const moe_router_t &r, int T, int E, int k,
                                int n_shared, int32_t *ids, float *w, cudaStream_t s) {
    if (T == 0) return cudaSuccess;
    RouterArgs a;
    a.logits = logits;
    a.bias = bias;
    a.T = T;
    a.E = E;
    a.k = k;
    a.n_shared = n_shared;
    a.score = r.score;
    a.n_group = r.n_group;
    a.topk_group = r.topk_group;
    a.group_top = r.group_top;
    a.renormalize = r.renormalize;
    a.scale = r.scale;
    a.ids = ids;
    a.w = w;
    return r.logits == MOE_LOGITS_BF16 ? launch_l<__nv_bfloat16>(a, s) : launch_l<float>(a, s);
}

}  // namespace moe
