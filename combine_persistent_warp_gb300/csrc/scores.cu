// scores.cu -- the router over sigmoid or softmax scores: a bias for balance, groups of experts, top-k and
// scaled gate weights, and the gradient of the logits.
//
//   s_e = 1/(1 + exp(-l_e)) or exp(l_e)/sum exp(l);  c_e = s_e + b_e (the choice alone sees the bias)
//   a group's score is the sum of its one or two largest c; the best groups stay, and of their experts the k
//   with the largest c are chosen; ties go to the lowest group or expert; -inf is never chosen, NaN counts as the largest
//   w_j = scale * s_j, or scale * s_j / sum_i s_i over the chosen ones (renormalised)
//   gradient, with dot = sum_i w_i dw_i:
//     sigmoid  renormalised w_j (dw_j - dot/scale)(1 - s_j), otherwise w_j dw_j (1 - s_j)
//     softmax  renormalised w_j (dw_j - dot/scale), otherwise p_e (scale [e chosen] dw_e - dot)
//
// The choice is that of c in 64 bits.  Two values of c that 32 bits hold for equal or swap are rare, and
// which expert a token goes to should not hang on a rounding: c is computed in 32 bits with a bound of
// its error, and a token whose choice that bound leaves open is chosen again in 64.
#include <climits>

#include "router_common.cuh"

using namespace cpw;

namespace {

constexpr uint32_t ALL = 0xFFFFFFFFu;
constexpr int MAX_GROUPS = 32;

struct ScoreArgs {
    int T, E, k;
    const void *logits;
    long long ld;
    const float *bias;     // may be null
    const uint8_t *mask;   // nonzero: the token is routed (null: every token)
    int softmax, renorm;
    int groups, kept, pair;   // pair: a group's score is the sum of two
    int per, lanes, shift;    // experts of a group; lanes that look through one, 1 << shift
    uint32_t per_magic;       // e / per = e * per_magic >> 20
    float scale;
    int64_t *idx;
    float *w;
};

__device__ __forceinline__ float warp_max_f(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(ALL, v, o));
    return v;
}
// ------------------------------------------------------------------ the choice ----------
// Where expert e's key lies for the lanes that look through the groups: 4 words further every 32, so that
// the lanes of 8 groups of 16 or 32 read different banks.
__device__ __forceinline__ int spot(int e) { return e + (e >> 5) * 4; }
template <int IPL>
constexpr int SPOTS = IPL * 36;

// Drops the keys of the groups that do not stay.  `least` and `most`: the lowest score that stays and the
// highest that does not (0: none).
template <int IPL, typename K>
__device__ __forceinline__ void keep_groups(const ScoreArgs &a, K (&key)[IPL], K *seen, int lane, K &least, K &most)
{
    __syncwarp();
#pragma unroll
    for (int i = 0; i < IPL; ++i)
        if (i * 32 + lane < a.E)
            seen[spot(i * 32 + lane)] = key[i];
    __syncwarp();
    const int g = lane >> a.shift, part = lane & (a.lanes - 1);
    K first = 0, second = 0;
    if (g < a.groups)
        for (int e = part; e < a.per; e += a.lanes) {
            const K v = seen[spot(g * a.per + e)];
            second = max(second, min(first, v));
            first = max(first, v);
        }
    for (int o = 1; o < a.lanes; o <<= 1) {
        const K f = __shfl_xor_sync(ALL, first, o), s = __shfl_xor_sync(ALL, second, o);
        second = max(max(second, s), min(first, f));
        first = max(first, f);
    }
    K score = first;
    if (a.pair && second != 0)
        score = order_key(key_value(first) + key_value(second));
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
        const K other = __shfl_sync(ALL, score, h << a.shift);
        rank += other > score || (other == score && h < g);
    }
    const bool there = g < a.groups && score != 0, stays = there && rank < a.kept;
    const uint32_t stay = __ballot_sync(ALL, stays);
    // the lowest: the complement of the largest complement
    least = ~warp_max(stays ? static_cast<K>(~score) : static_cast<K>(0));
    most = warp_max(there && !stays ? score : static_cast<K>(0));
#pragma unroll
    for (int i = 0; i < IPL; ++i) {
        const int e = i * 32 + lane, ge = static_cast<int>((static_cast<uint32_t>(e) * a.per_magic) >> 20);
        if (e < a.E && !(stay >> (ge << a.shift) & 1u))
            key[i] = 0;
    }
}

// The k largest keys: lane j gets slot j's expert and key; the one after them (e -1: there is none).
// Returns how many there are.
template <int IPL, typename K>
__device__ __forceinline__ int choose_keys(int k, K (&key)[IPL], int lane, int &my_idx, K &mine, int &next_idx, K &next)
{
    mine = next = 0;
    next_idx = -1;
    for (int j = 0;; ++j) {
        K best = key[0];
#pragma unroll
        for (int i = 1; i < IPL; ++i)
            best = max(best, key[i]);
        const K m = warp_max(best);
        if (m == 0)
            return j;   // only what is never chosen is left
        int at = INT_MAX;
#pragma unroll
        for (int i = IPL - 1; i >= 0; --i)
            at = key[i] == m ? i * 32 + lane : at;
        const int e = __reduce_min_sync(ALL, at);
        if (j == k) {
            next_idx = e;
            next = m;
            return k;
        }
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            key[i] = i * 32 + lane == e ? 0 : key[i];
        my_idx = lane == j ? e : my_idx;
        mine = lane == j ? m : mine;
    }
}

// The choice in 64 bits.
template <typename T, int IPL>
__device__ __noinline__ int choose_exactly(const ScoreArgs &a, const T *l, uint64_t *seen, int lane, int &my_idx)
{
    double c[IPL], top = 0.0, total = 1.0;
#pragma unroll
    for (int i = 0; i < IPL; ++i)
        c[i] = i * 32 + lane < a.E ? static_cast<double>(to_f<T>(l[i * 32 + lane])) : -INFINITY;
    if (a.softmax) {
        float m = -INFINITY;   // (the logits have at most 32 bits)
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            m = fmaxf(m, static_cast<float>(c[i]));
        top = static_cast<double>(warp_max_f(m));
        total = 0.0;
#pragma unroll 1
        for (int i = 0; i < IPL; ++i)
            if (i * 32 + lane < a.E)
                total += exp(c[i] - top);
        total = warp_sum(total);
    }
    uint64_t key[IPL];
#pragma unroll 1
    for (int i = 0; i < IPL; ++i) {
        key[i] = 0;
        if (i * 32 + lane < a.E && c[i] != -INFINITY) {
            const double s = a.softmax ? exp(c[i] - top) / total : 1.0 / (1.0 + exp(-c[i]));
            key[i] = order_key(a.bias ? s + static_cast<double>(a.bias[i * 32 + lane]) : s);
        }
    }
    uint64_t u0, u1, mine;
    int next_idx;
    my_idx = -1;
    if (a.groups > 1)
        keep_groups<IPL>(a, key, seen, lane, u0, u1);
    return choose_keys<IPL>(a.k, key, lane, my_idx, mine, next_idx, u0);
}

template <typename T, int IPL>
__global__ void __launch_bounds__(WARPS * 32) score_kernel(const ScoreArgs a)
{
    __shared__ uint64_t seen[WARPS][SPOTS<IPL>];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * WARPS + warp;
    if (t >= a.T)
        return;
    int my_idx = -1;
    float my_w = 0.0f;
    if (!a.mask || a.mask[t]) {
        const T *l = static_cast<const T *>(a.logits) + static_cast<size_t>(t) * a.ld;
        float f[IPL], top = 0.0f, total = 1.0f;
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            f[i] = i * 32 + lane < a.E ? to_f<T>(l[i * 32 + lane]) : -INFINITY;
        // without a bias scores are in the order of the logits, which are exact
        const bool direct = !a.bias && (a.groups == 1 || !a.pair);
        if (a.softmax && !(direct && a.renorm)) {
            top = f[0];
#pragma unroll
            for (int i = 1; i < IPL; ++i)
                top = fmaxf(top, f[i]);
            top = warp_max_f(top);
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                if (i * 32 + lane < a.E)
                    total += expf(f[i] - top);
            total = warp_sum(total);
        }
        uint32_t key[IPL];
        float open = 0.0f;   // two values this near (and 2^-22 of their size) are open
        if (direct) {
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                key[i] = order_key(f[i]);
        } else {
            // Errors of c in units of 2^-24: sigmoid at most 4 of its exponential, times s (1 - s) <= 1/4, its sum
            // 1/2 and the quotient 1/2; softmax (times 1/total, the largest probability) 8 of the two
            // exponentials and quotients, ln E of the exponents' roundings and 1/2 for each of the sum's IPL + 5
            // additions.  Twice that for two values, and twice again.
            open = a.softmax ? (2.0f * IPL + 72.0f) * 0x1p-24f / total : 0x1p-21f;
#pragma unroll
            for (int i = 0; i < IPL; ++i) {
                const int e = i * 32 + lane;
                key[i] = 0u;
                if (e < a.E && f[i] != -INFINITY) {
                    const float s = a.softmax ? expf(f[i] - top) / total : 1.0f / (1.0f + expf(-f[i]));
                    key[i] = order_key(a.bias ? s + __ldg(a.bias + e) : s);
                }
            }
        }
        bool sure = true;
        if (a.groups > 1) {
            uint32_t least, most;
            keep_groups<IPL>(a, key, reinterpret_cast<uint32_t *>(seen[warp]), lane, least, most);
            if (!direct && most != 0u) {
                const float v = key_value(least);
                sure = v - key_value(most) > 2.0f * open + fabsf(v) * 0x1p-21f;
            }
        }
        uint32_t mine, next;
        int next_idx;
        int found = choose_keys<IPL>(a.k, key, lane, my_idx, mine, next_idx, next);
        float logit = lane < found ? to_f<T>(l[my_idx]) : 0.0f;
        if (!direct) {
            // every slot is above the one after it, or equal to it in what it is computed from
            const float b = a.bias && lane < found ? __ldg(a.bias + my_idx) : 0.0f;
            uint32_t after = __shfl_down_sync(ALL, mine, 1);
            float after_logit = __shfl_down_sync(ALL, logit, 1), after_b = __shfl_down_sync(ALL, b, 1);
            if (lane == a.k - 1) {
                after = next;
                after_logit = next_idx >= 0 ? to_f<T>(l[next_idx]) : 0.0f;
                after_b = next_idx >= 0 && a.bias ? __ldg(a.bias + next_idx) : 0.0f;
            }
            bool ok = true;
            if (lane < found && after != 0u) {
                const float v = key_value(mine);
                ok = v - key_value(after) > open + fabsf(v) * 0x1p-22f || (logit == after_logit && b == after_b);
            }
            sure = __all_sync(ALL, ok && sure);
            if (!sure) {
                found = choose_exactly<T, IPL>(a, l, seen[warp], lane, my_idx);
                logit = lane < found ? to_f<T>(l[my_idx]) : 0.0f;
            }
        }
        float p = 0.0f;
        if (a.softmax) {
            if (a.renorm)
                top = warp_max_f(lane < found ? logit : -INFINITY);
            p = lane < found ? expf(logit - top) : 0.0f;
            if (a.renorm)
                total = warp_sum(p);
        } else {
            // s = exp(l - m) / (1 + exp(l)) * exp(m), m = min(0, largest): all scores may be tiny, their quotients are not
            const float m = a.renorm ? fminf(0.0f, warp_max_f(lane < found ? logit : -INFINITY)) : 0.0f;
            if (lane < found)
                p = (logit >= 0.0f ? 1.0f : expf(logit - m)) / (1.0f + expf(-fabsf(logit)));
            total = a.renorm ? warp_sum(p) : 1.0f;
        }
        if (lane < found)
            my_w = p / total * a.scale;
    }
    if (lane < a.k) {
        a.idx[static_cast<size_t>(t) * a.k + lane] = my_idx;
        a.w[static_cast<size_t>(t) * a.k + lane] = my_w;
    }
}

// ------------------------------------------------------------------ gradient ------------
struct ScoreBwdArgs {
    int T, E, k;
    const float *dw;
    const int64_t *idx;
    const float *w;
    const void *logits;   // not read for renormalised softmax scores
    long long ld;
    int softmax, renorm;
    float scale;
    void *dlogits;        // [T][E]
};

template <typename T, int IPL>
__global__ void __launch_bounds__(WARPS * 32) score_backward_kernel(const ScoreBwdArgs a)
{
    const int t = blockIdx.x * WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= a.T)
        return;
    int e = -1;
    float w = 0.0f, dw = 0.0f;
    if (lane < a.k) {
        const size_t at = static_cast<size_t>(t) * a.k + lane;
        const int64_t id = a.idx[at];
        e = id >= 0 && id < a.E ? static_cast<int>(id) : -1;
        if (e >= 0) {
            w = a.w[at];
            dw = a.dw[at];
        }
    }
    const float dot = warp_sum(w * dw);
    const bool any = __any_sync(ALL, e >= 0);
    const T *l = static_cast<const T *>(a.logits) + static_cast<size_t>(t) * a.ld;
    T *out = static_cast<T *>(a.dlogits) + static_cast<size_t>(t) * a.E;
    const bool dense = a.softmax && !a.renorm && any;
    // what the slot adds: to the expert's logit, or (dense) to what its probability is multiplied by
    float d = dense ? a.scale * dw : a.renorm ? w * (dw - dot / a.scale) : w * dw;
    if (!a.softmax && e >= 0)
        d /= 1.0f + expf(to_f<T>(l[e]));
    // an expert that is in several slots gets their sum, in order
    const uint32_t same = __match_any_sync(ALL, e >= 0 ? e : -1 - lane);
    if (__any_sync(ALL, same & (same - 1u))) {
        float sum = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const float v = __shfl_sync(ALL, d, j);
            sum += same >> j & 1u ? v : 0.0f;
        }
        d = sum;
    }
    float top = 0.0f, inv = 0.0f;
    if (dense) {
        float f[IPL], sum = 0.0f;
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < IPL; ++i) {
            f[i] = i * 32 + lane < a.E ? to_f<T>(l[i * 32 + lane]) : -INFINITY;
            top = fmaxf(top, f[i]);
        }
        top = warp_max_f(top);
#pragma unroll
        for (int i = 0; i < IPL; ++i) {
            f[i] = expf(f[i] - top);   // NaN logits and top = +inf make NaN, as in the forward pass
            if (i * 32 + lane < a.E)
                sum += f[i];
        }
        inv = 1.0f / warp_sum(sum);
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            if (i * 32 + lane < a.E)
                out[i * 32 + lane] = from_f<T>(f[i] * inv * -dot);
    } else {
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            if (i * 32 + lane < a.E)
                out[i * 32 + lane] = from_f<T>(0.0f);
    }
    __syncwarp();   // the chosen ones over what the row's other lanes have written
    if (e >= 0)
        out[e] = from_f<T>(dense ? expf(to_f<T>(l[e]) - top) * inv * (d - dot) : d);
}

// ------------------------------------------------------------------ host side ------------
template <typename T, int IPL>
struct ScoreLaunch {
    static void go(const ScoreArgs &a, cudaStream_t s)
    {
        score_kernel<T, IPL><<<(a.T + WARPS - 1) / WARPS, WARPS * 32, 0, s>>>(a);
    }
};
template <typename T, int IPL>
struct ScoreBwdLaunch {
    static void go(const ScoreBwdArgs &a, cudaStream_t s)
    {
        score_backward_kernel<T, IPL><<<(a.T + WARPS - 1) / WARPS, WARPS * 32, 0, s>>>(a);
    }
};

bool flag(int v) { return v == 0 || v == 1; }
bool scale_ok(float s) { return s - s == 0.0f && s != 0.0f; }   // finite, not zero

}  // namespace

extern "C" {

int moe_route_scores(int T, int E, int topk, const void *logits, int64_t ld, int dtype, int score, const float *bias, int groups,
                     int topk_groups, int group_top, const uint8_t *token_mask, int renormalize, float scale, int64_t *topk_idx,
                     float *topk_w, void *stream)
{
    if (!route_sizes_ok(T, E, topk, dtype) || ld < E || (score != MOE_SCORE_SIGMOID && score != MOE_SCORE_SOFTMAX) ||
        !flag(renormalize) || !scale_ok(scale) || groups < 1 || groups > MAX_GROUPS || E % groups != 0 || topk_groups < 1 ||
        topk_groups > groups || group_top < 1 || group_top > 2 || topk > topk_groups * (E / groups))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    if (!logits || !topk_idx || !topk_w || !op_aligned(logits, dtype_bytes(dtype)) || !op_aligned(bias, 4) ||
        !op_aligned(topk_idx, 8) || !op_aligned(topk_w, 4))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    ScoreArgs a{T, E, topk, logits, ld, bias, token_mask, score == MOE_SCORE_SOFTMAX, renormalize, groups, topk_groups, group_top == 2,
                E / groups, 1, 0, 0, scale, topk_idx, topk_w};
    if (topk_groups == groups)
        a.groups = a.kept = 1;   // all of them stay: no groups
    a.per = E / a.groups;
    while ((a.lanes * 2) * a.groups <= 32) {
        a.lanes *= 2;
        ++a.shift;
    }
    a.per_magic = (1u << 20) / static_cast<uint32_t>(a.per) + 1;   // exact for e, per <= 1024
    by_width<ScoreLaunch>(dtype, E, a, static_cast<cudaStream_t>(stream));
    return launched();
}

int moe_route_scores_backward(int T, int E, int topk, const float *dw, const int64_t *topk_idx, const float *topk_w,
                              const void *logits, int64_t ld, int dtype, int score, int renormalize, float scale, void *dlogits,
                              void *stream)
{
    if (!route_sizes_ok(T, E, topk, dtype) || ld < E || (score != MOE_SCORE_SIGMOID && score != MOE_SCORE_SOFTMAX) ||
        !flag(renormalize) || !scale_ok(scale))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    const bool reads = score == MOE_SCORE_SIGMOID || !renormalize;
    if (!dw || !topk_idx || !topk_w || !dlogits || (reads && !logits) || !op_aligned(dw, 4) || !op_aligned(topk_idx, 8) ||
        !op_aligned(topk_w, 4) || !op_aligned(logits, dtype_bytes(dtype)) || !op_aligned(dlogits, dtype_bytes(dtype)))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    by_width<ScoreBwdLaunch>(dtype, E,
                             ScoreBwdArgs{T, E, topk, dw, topk_idx, topk_w, logits, ld, score == MOE_SCORE_SOFTMAX, renormalize, scale, dlogits},
                             static_cast<cudaStream_t>(stream));
    return launched();
}

}  // extern "C"
