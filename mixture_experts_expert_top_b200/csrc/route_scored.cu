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
// last group kept and the first one dropped) exceeds twice the bound. The few
// rows where one does not (about 1 in 1000 for 256 experts) are selected again
// from 64-bit scores (select_64).
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "launch_util.cuh"
#include "route_dev.cuh"

namespace moe {
namespace {

constexpr int kWarpsPerBlock = 4;

struct RouterArgs {
    const void *logits;
    const float *bias;
    int T, E, k, n_shared;
    int score, n_group, topk_group, group_top, renormalize;
    float scale;
    int32_t *ids;
    float *w;
};

__device__ __forceinline__ float load_logit(const float *p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// The logit as the scores take it: NaN is -inf, -0 is +0.
__device__ __forceinline__ float clean_logit(float x) {
    if (x != x) return -INFINITY;
    return x == 0.f ? 0.f : x;
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

// The selection in 64 bits. Lane l holds experts l*N .. l*N+N-1 (x: their
// cleaned logits, below E). Returns slot j's expert in lane j.
template <int N>
__device__ __noinline__ int select_64(const RouterArgs &a, const float (&x)[N], float m, double *by_s) {
    const int lane = threadIdx.x & 31;
    const int e0 = lane * N;
    const bool soft = a.score == MOE_SCORE_SOFTMAX;
    const bool by_logit = a.bias == nullptr;                     // experts are ordered by their logits
    const bool groups_by_logit = by_logit && a.group_top == 1;
    double s[N];
    const bool need_scores = !by_logit || (a.n_group > 1 && !groups_by_logit);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = 0.0;
        if (need_scores && e0 + i < a.E) {
            if (soft)
                s[i] = x[i] == m ? (m == -INFINITY ? 0.0 : 1.0) : exp(static_cast<double>(x[i]) - m);
            else
                s[i] = 1.0 / (1.0 + exp(-static_cast<double>(x[i])));
            sum += s[i];
        }
    }
    if (need_scores && soft) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (sum > 0.0) s[i] /= sum;
    }
    uint64_t key[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        key[i] = 0;
        if (e0 + i < a.E) {
            const double c = by_logit ? static_cast<double>(x[i]) : s[i] + static_cast<double>(a.bias[e0 + i]);
            key[i] = choice_key(c);
            if (a.n_group > 1) by_s[e0 + i] = by_logit && !groups_by_logit ? s[i] : c;
        }
    }
    if (a.n_group > 1) {
        __syncwarp();
        const int size = a.E / a.n_group;
        uint64_t gk = 0;
        if (lane < a.n_group) {
            double top1 = -INFINITY, top2 = -INFINITY;
            for (int i = 0; i < size; ++i) {
                double v = by_s[lane * size + i];
                if (v != v) v = -INFINITY;
                if (v > top1) { top2 = top1; top1 = v; }
                else if (v > top2) top2 = v;
            }
            gk = choice_key(a.group_top == 2 ? top1 + top2 : top1);
        }
        const uint32_t kept = keep_groups(gk, a.n_group, a.topk_group);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e0 + i < a.E && !((kept >> ((e0 + i) / size)) & 1u)) key[i] = 0;
    }
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

// fp32 scores of the lane's experts (lane l: l*N .. l*N+N-1) and a bound on
// the error of c = s + b against its 64-bit value, the same in all lanes. In
// units of u = 2^-24: expf is within 2 ulp (4u); a sigmoid adds two roundings;
// a softmax term has its argument's rounding, u |l - m|, besides, the sum of E
// terms at most N + 5 additions and its terms' average error (|l - m| averages
// below ln E < 7 over a softmax), the quotient two. s |l - m| <= 0.37 s_max.
// Adding b rounds by u |c|; infinities are exact.
template <int N>
__device__ __forceinline__ float scores_32(const RouterArgs &a, const float (&x)[N], float m, const float *bias, float (&s)[N],
                                           float (&c)[N]) {
    const int e0 = (threadIdx.x & 31) * N;
    float top = 0.f, big = 0.f;
    if (a.score == MOE_SCORE_SOFTMAX) {
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s[i] = x[i] == m ? (m == -INFINITY ? 0.f : 1.f) : expf(x[i] - m);
            z += s[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        const float inv = z > 0.f ? 1.0f / z : 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] *= inv;
        top = inv;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s[i] = 1.0f / (1.0f + expf(-x[i]));
            top = fmaxf(top, s[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        c[i] = bias && e0 + i < a.E ? s[i] + bias[e0 + i] : s[i];
        if (fabsf(c[i]) < INFINITY) big = fmaxf(big, fabsf(c[i]));
    }
    // both maxima are of non-negative floats: their bits order them
    big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
    if (a.score == MOE_SCORE_SOFTMAX) return 0x1p-24f * 1.25f * ((N + 24.0f) * top + big) + 1e-37f;
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    return 0x1p-24f * 1.25f * (6.0f * top + big) + 1e-37f;
}

// a > b by more than `gap`, for the values of two keys in descending order. A
// missing candidate (key 0) is behind everything; equal keys are never apart.
__device__ __forceinline__ bool apart(uint32_t ka, uint32_t kb, float gap) {
    return kb == 0u || key_logit(ka) - key_logit(kb) > gap;
}

// The selection on fp32 values. by: what groups are valued by; c: what experts
// are ordered by, exact when err is 0. Returns slot j's expert in lane j;
// `sure` (the same in all lanes) says whether the 64-bit selection is the same.
template <int N>
__device__ __forceinline__ int select_32(const RouterArgs &a, const float (&by)[N], const float (&c)[N], float err_by,
                                         float err_c, float *by_s, bool &sure) {
    const int lane = threadIdx.x & 31;
    const int e0 = lane * N;
    sure = true;
    uint32_t key[N];
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = e0 + i < a.E ? logit_key(c[i]) : 0u;
    if (a.n_group > 1) {
        const int size = a.E / a.n_group;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e0 + i < a.E) by_s[e0 + i] = by[i] != by[i] ? -INFINITY : by[i];
        __syncwarp();
        float g = -INFINITY;
        if (lane < a.n_group) {
            float top1 = -INFINITY, top2 = -INFINITY;
            for (int i = 0; i < size; ++i) {
                const float v = by_s[lane * size + i];
                top2 = fmaxf(top2, fminf(top1, v));
                top1 = fmaxf(top1, v);
            }
            g = a.group_top == 2 ? top1 + top2 : top1;
        }
        const uint32_t gk = lane < a.n_group ? logit_key(g) : 0u;
        const uint32_t kept = keep_groups(gk, a.n_group, a.topk_group);
        if (err_by > 0.f && a.topk_group < a.n_group) {
            // a sum of two: twice the error, and its own rounding below it
            const uint32_t last = __reduce_min_sync(0xffffffffu, (kept >> lane) & 1u ? gk : 0xffffffffu);
            const uint32_t first = __reduce_max_sync(0xffffffffu, (kept >> lane) & 1u ? 0u : gk);
            sure = apart(last, first, (a.group_top == 2 ? 8.0f : 2.0f) * err_by);
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e0 + i < a.E && !((kept >> ((e0 + i) / size)) & 1u)) key[i] = 0u;
        __syncwarp();
    }
    int my_id = 0;
    uint32_t before = 0;
    const int rounds = err_c > 0.f ? a.k + 1 : a.k;              // one more to see the gap behind the last
    for (int j = 0; j < rounds; ++j) {
        uint32_t local = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) local = max(local, key[i]);
        const uint32_t best = __reduce_max_sync(0xffffffffu, local);
        if (err_c > 0.f && j > 0) sure = sure && apart(before, best, 2.0f * err_c);
        before = best;
        if (j == a.k) break;
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

template <int N, typename L>
__global__ void __launch_bounds__(kWarpsPerBlock * 32)
route_scored_kernel(const RouterArgs a) {
    extern __shared__ double by_all[];                           // [kWarpsPerBlock][E], only with groups
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kWarpsPerBlock + warp;
    if (t >= a.T) return;
    const L *row = static_cast<const L *>(a.logits) + static_cast<size_t>(t) * a.E;
    const int e0 = lane * N;
    const bool soft = a.score == MOE_SCORE_SOFTMAX;
    float x[N];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = e0 + i < a.E ? clean_logit(load_logit(row + e0 + i)) : -INFINITY;
        m = fmaxf(m, x[i]);
    }
    if (soft) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    double *by_s = by_all + static_cast<size_t>(warp) * a.E;
    const bool by_logit = a.bias == nullptr;
    int id;
    bool sure;
    if (by_logit && (a.n_group == 1 || a.group_top == 1)) {
        id = select_32<N>(a, x, x, 0.f, 0.f, reinterpret_cast<float *>(by_s), sure);      // exact
    } else {
        float s[N], c[N];
        const float err = scores_32<N>(a, x, m, a.bias, s, c);
        if (by_logit)
            id = select_32<N>(a, s, x, err, 0.f, reinterpret_cast<float *>(by_s), sure);
        else
            id = select_32<N>(a, c, c, err, err, reinterpret_cast<float *>(by_s), sure);
        if (!sure) id = select_64<N>(a, x, m, by_s);
    }
    // The weight of slot j, in lane j. Renormalised, only ratios of scores count:
    // softmax takes them relative to the largest selected logit, and so does a
    // sigmoid whose selected scores are all below e^-60 (there s = exp(l) to
    // fp32), so no sum underflows.
    float l = -INFINITY;
    bool off = false;
    if (lane < a.k) {
        l = clean_logit(load_logit(row + id));
        off = a.bias && !(a.bias[id] > -INFINITY);
    }
    float lmax = off ? -INFINITY : l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lmax = fmaxf(lmax, __shfl_xor_sync(0xffffffffu, lmax, o));
    float s;
    if (soft && !a.renormalize) {
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (e0 + i < a.E) z += x[i] == m ? 1.0f : expf(x[i] - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        s = (l == m ? 1.0f : expf(l - m)) / z;
    } else if (soft || (a.renormalize && lmax < -60.0f)) {
        s = l == lmax ? 1.0f : expf(l - lmax);
    } else {
        s = 1.0f / (1.0f + expf(-l));
    }
    if (off || l == -INFINITY || lane >= a.k) s = 0.f;
    float wt = s;
    if (a.renormalize) {
        float sum = 0.f;
        for (int j = 0; j < a.k; ++j) sum += __shfl_sync(0xffffffffu, s, j);      // slot order
        wt = sum > 0.f ? s / sum : 0.f;
    }
    wt *= a.scale;
    int out_id = id;
    shared_slot(lane, a.k, a.E, out_id, wt);
    const int K = a.k + a.n_shared;
    if (lane < K) {
        a.ids[static_cast<size_t>(t) * K + lane] = out_id;
        a.w[static_cast<size_t>(t) * K + lane] = wt;
    }
}

template <int N, typename L>
cudaError_t launch_n(const RouterArgs &a, cudaStream_t s) {
    const int blocks = (a.T + kWarpsPerBlock - 1) / kWarpsPerBlock;
    const size_t sm = a.n_group > 1 ? static_cast<size_t>(kWarpsPerBlock) * a.E * sizeof(double) : 0;
    return launch_pdl(route_scored_kernel<N, L>, dim3(blocks), dim3(kWarpsPerBlock * 32), sm, s, a);
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
