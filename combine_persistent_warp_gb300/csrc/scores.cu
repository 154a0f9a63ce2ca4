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
// its error, and the candidates that this bound leaves open are ranked again in 64.
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
    int group_shift;          // a group is 1 << group_shift lanes (-1: it is not)
    int per, lanes, shift;    // otherwise: experts of a group; lanes that look through one, 1 << shift
    uint32_t per_magic;       // e / per = e * per_magic >> 20
    int vec, bias_vec;        // rows of logits, the bias: in vectors (see load_lane)
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
// Lane l holds experts l * IPL .. l * IPL + IPL - 1 (a group of experts is then a few neighbouring lanes, mostly).
//
// A word is what the choice goes by: the upper bits of c's order key and, below them, the expert (ties to
// the lowest), so that one warp maximum a slot finds both.  The bits that the expert takes from the key make
// more values look equal; what the words leave open is settled by the candidates' exact values.
template <int IPL>
constexpr int BITS = IPL == 1 ? 5 : IPL == 2 ? 6 : IPL == 4 ? 7 : IPL == 8 ? 8 : 10;
template <int IPL>
constexpr uint32_t ID = (1u << BITS<IPL>) - 1u;
template <typename K>   // the key of -inf; words and keys up to it are not there
constexpr K NEVER = sizeof(K) == 4 ? static_cast<K>(0x007FFFFFu) : static_cast<K>(0x000FFFFFFFFFFFFFull);

// Order key of a sum or product (whose NaN is the positive one).
__device__ __forceinline__ uint32_t plain_key(float f)
{
    const uint32_t u = __float_as_uint(f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float plain_value(uint32_t key)
{
    return __uint_as_float(key ^ (static_cast<uint32_t>(static_cast<int32_t>(~key) >> 31) | 0x80000000u));
}
template <int IPL>
__device__ __forceinline__ uint32_t word_of(uint32_t key, int lane, int i)
{
    return (key & ~ID<IPL>) | (ID<IPL> - static_cast<uint32_t>(lane * IPL + i));
}
template <int IPL>
__device__ __forceinline__ int expert_of(uint32_t word) { return static_cast<int>(ID<IPL> - (word & ID<IPL>)); }
// The least and the most that the c of a word can be.
template <int IPL>
__device__ __forceinline__ float least_of(uint32_t word) { return plain_value(word & ~ID<IPL>); }
template <int IPL>
__device__ __forceinline__ float most_of(uint32_t word) { return plain_value(word | ID<IPL>); }

// Whether the lane's group of experts stays, from the group's two largest keys: `least` and `most` are
// the lowest score that stays and the highest that does not (0: none).  Group g is that of the lanes
// g << shift and after.
__device__ __forceinline__ uint32_t key_sum(uint32_t a, uint32_t b) { return plain_key(plain_value(a) + plain_value(b)); }
__device__ __forceinline__ uint64_t key_sum(uint64_t a, uint64_t b) { return order_key(key_value(a) + key_value(b)); }
template <typename K>
__device__ __forceinline__ bool group_stays(const ScoreArgs &a, K first, K second, int lane, int shift, K &least, K &most)
{
    const int g = lane >> shift;
    K score = g < a.groups && first > NEVER<K> ? first : 0;
    if (a.pair && second > NEVER<K>)
        score = key_sum(first, second);
    bool stays = false;
    least = 0;
    for (int j = 0; j < a.kept; ++j) {
        const K m = warp_max(score);
        if (m == 0)
            break;
        least = m;
        const int best = (__ffs(static_cast<int>(__ballot_sync(ALL, score == m))) - 1) >> shift;   // ties: the lowest
        stays = stays || g == best;
        score = g == best ? 0 : score;
    }
    most = warp_max(score);
    return stays;
}
template <typename K>
__device__ __forceinline__ void insert(K v, K &first, K &second)
{
    second = max(second, min(first, v));
    first = max(first, v);
}
template <typename K>
__device__ __forceinline__ void merge_lanes(K &first, K &second, int lanes)
{
    for (int o = 1; o < lanes; o <<= 1) {
        const K f = __shfl_xor_sync(ALL, first, o), s = __shfl_xor_sync(ALL, second, o);
        second = max(max(second, s), min(first, f));
        first = max(first, f);
    }
}
// Where expert e's key lies for the lanes that look through groups that are not whole lanes.
__device__ __forceinline__ int spot(int e) { return e + (e >> 5) * 4; }
template <int IPL>
constexpr int SPOTS = IPL * 36;

// Zeroes the keys of the groups that do not stay.
template <int IPL, typename K>
__device__ __forceinline__ void keep_groups(const ScoreArgs &a, K (&key)[IPL], K *seen, int lane, K &least, K &most)
{
    K first = 0, second = 0;
    if (a.group_shift >= 0) {   // a group is 1 << group_shift lanes
        first = key[0];
#pragma unroll
        for (int i = 1; i < IPL; ++i)
            insert(key[i], first, second);
        merge_lanes(first, second, 1 << a.group_shift);
        const bool stays = group_stays(a, first, second, lane, a.group_shift, least, most);
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            key[i] = stays ? key[i] : 0;
        return;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < IPL; ++i)
        if (lane * IPL + i < a.E)
            seen[spot(lane * IPL + i)] = key[i];
    __syncwarp();
    const int g = lane >> a.shift;
    if (g < a.groups)
        for (int e = lane & (a.lanes - 1); e < a.per; e += a.lanes)
            insert(seen[spot(g * a.per + e)], first, second);
    merge_lanes(first, second, a.lanes);
    const uint32_t stay = __ballot_sync(ALL, group_stays(a, first, second, lane, a.shift, least, most));
#pragma unroll
    for (int i = 0; i < IPL; ++i) {
        const int e = lane * IPL + i, ge = static_cast<int>((static_cast<uint32_t>(e) * a.per_magic) >> 20);
        if (e < a.E && !(stay >> (ge << a.shift) & 1u))
            key[i] = 0;
    }
}

// The choice in 64 bits of all experts.
template <typename T, int IPL>
__device__ __noinline__ int choose_exactly(const ScoreArgs &a, const T *l, uint64_t *seen, int lane, int &my_idx)
{
    constexpr int UNROLL = IPL <= 8 ? IPL : 1;
    double c[IPL], top = 0.0, total = 1.0;
#pragma unroll
    for (int i = 0; i < IPL; ++i)
        c[i] = lane * IPL + i < a.E ? static_cast<double>(to_f<T>(l[lane * IPL + i])) : -INFINITY;
    if (a.softmax) {
        float m = -INFINITY;   // (the logits have at most 32 bits)
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            m = fmaxf(m, static_cast<float>(c[i]));
        top = static_cast<double>(warp_max_f(m));
        total = 0.0;
#pragma unroll UNROLL
        for (int i = 0; i < IPL; ++i)
            if (lane * IPL + i < a.E)
                total += exp(c[i] - top);
        total = warp_sum(total);
    }
    uint64_t key[IPL];
#pragma unroll UNROLL
    for (int i = 0; i < IPL; ++i) {
        key[i] = 0;
        if (lane * IPL + i < a.E && c[i] != -INFINITY) {
            const double s = a.softmax ? exp(c[i] - top) / total : 1.0 / (1.0 + exp(-c[i]));
            key[i] = order_key(a.bias ? s + static_cast<double>(a.bias[lane * IPL + i]) : s);
        }
    }
    if (a.groups > 1) {
        uint64_t least, most;
        keep_groups<IPL>(a, key, seen, lane, least, most);
    }
    my_idx = -1;
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = key[0];
#pragma unroll
        for (int i = 1; i < IPL; ++i)
            best = max(best, key[i]);
        const uint64_t m = warp_max(best);
        if (m == 0)
            return j;   // only what is never chosen is left
        int at = INT_MAX;
#pragma unroll
        for (int i = IPL - 1; i >= 0; --i)
            at = key[i] == m ? lane * IPL + i : at;
        const int e = __reduce_min_sync(ALL, at);
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            key[i] = lane * IPL + i == e ? 0 : key[i];
        my_idx = lane == j ? e : my_idx;
    }
    return a.k;
}

// A lane's words in descending order (a sorting network; words differ), so that a lane's largest is its first;
// more than 8 stay as they are.
template <int IPL>
constexpr bool SORTED = IPL <= 8;
__device__ __forceinline__ void order_two(uint32_t &a, uint32_t &b)
{
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}
template <int IPL>
__device__ __forceinline__ void sort_lane(uint32_t (&w)[IPL])
{
    if constexpr (SORTED<IPL>) {
        // odd-even merges (Batcher)
#pragma unroll
        for (int p = 1; p < IPL; p *= 2)
#pragma unroll
            for (int k = p; k >= 1; k /= 2)
#pragma unroll
                for (int j = k % p; j + k < IPL; j += 2 * k)
#pragma unroll
                    for (int i = 0; i < k; ++i)
                        if (i + j + k < IPL && (i + j) / (2 * p) == (i + j + k) / (2 * p))
                            order_two(w[i + j], w[i + j + k]);
    }
}
// The warp's largest word, taken out.
template <int IPL>
__device__ __forceinline__ uint32_t take_largest(uint32_t (&w)[IPL])
{
    if constexpr (SORTED<IPL>) {
        const uint32_t m = warp_max(w[0]);
        if (w[0] == m) {
#pragma unroll
            for (int i = 0; i + 1 < IPL; ++i)
                w[i] = w[i + 1];
            w[IPL - 1] = 0u;
        }
        return m;
    } else {
        uint32_t best = w[0];
#pragma unroll
        for (int i = 1; i < IPL; ++i)
            best = max(best, w[i]);
        const uint32_t m = warp_max(best);
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            w[i] = w[i] == m ? 0u : w[i];
        return m;
    }
}

// The n candidates in lanes 0 .. n - 1 by their values in 64 bits: lane j gets the j-th.
template <bool DIRECT>
__device__ __noinline__ int rank_exactly(float logit, float bias, bool has_bias, int idx, int n, int lane)
{
    const double l = static_cast<double>(logit), s = DIRECT ? l : 1.0 / (1.0 + exp(-l));
    const uint64_t key = order_key(has_bias ? s + static_cast<double>(bias) : s);
    int rank = 0;
    for (int r = 0; r < n; ++r) {
        const uint64_t other = __shfl_sync(ALL, key, r);
        const int its = __shfl_sync(ALL, idx, r);
        rank += other > key || (other == key && its < idx);
    }
    int got = -1;
    for (int r = 0; r < n; ++r) {
        const int at = __shfl_sync(ALL, rank, r), its = __shfl_sync(ALL, idx, r);
        got = at == lane ? its : got;
    }
    return got;
}

// A lane's IPL neighbouring logits or biases, in accesses of up to 16 bytes where `vec` (the rows allow it);
// -inf past the last expert.
template <typename T, int IPL>
__device__ __forceinline__ void load_lane(float (&f)[IPL], const T *row, int lane, int E, bool vec)
{
    constexpr int BYTES = IPL * static_cast<int>(sizeof(T)), PIECE = BYTES < 16 ? BYTES : 16, N = PIECE / static_cast<int>(sizeof(T));
    if (N > 1 && vec) {   // (whole lanes are in or out)
        struct alignas(PIECE) Piece {
            T v[N];
        };
        Piece q[IPL / N];
        const bool in = lane * IPL < E;
#pragma unroll
        for (int i = 0; i < IPL / N; ++i)
            if (in)
                q[i] = reinterpret_cast<const Piece *>(row + lane * IPL)[i];
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            f[i] = in ? to_f<T>(q[i / N].v[i % N]) : -INFINITY;
    } else {
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            f[i] = lane * IPL + i < E ? to_f<T>(row[lane * IPL + i]) : -INFINITY;
    }
}

// 1/(1 + exp(-l)) by two approximate instructions.
__device__ __forceinline__ float logistic(float l)
{
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
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
        float f[IPL], b[IPL], top = 0.0f, total = 1.0f;
        load_lane<T, IPL>(f, l, lane, a.E, a.vec);
        if (a.bias)
            load_lane<float, IPL>(b, a.bias, lane, a.E, a.bias_vec);
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
                if (lane * IPL + i < a.E)
                    total += expf(f[i] - top);
            total = warp_sum(total);
        }
        uint32_t word[IPL];
        // Two values of c that are this near (and 2^-22 of their size) are open.  Errors in units of 2^-24: the sigmoid's
        // exponential (1.3 |l| + 2.8) times s (1 - s), at most 1, its sum 1/2, the reciprocal 2; softmax (times 1/total, the
        // largest probability) 8 of the two exponentials and quotients, ln E of the exponents' roundings and 1/2
        // for each of the sum's IPL + 5 additions.  Twice that for two values.
        float open = 0.0f;
        if (direct) {
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                word[i] = plain_key(f[i] + 0.0f);   // (-0 as +0)
        } else {
            open = a.softmax ? (2.0f * IPL + 72.0f) * 0x1p-24f / total : 0x1p-21f;
            const float inv = 1.0f / total;
#pragma unroll
            for (int i = 0; i < IPL; ++i) {
                const float s = a.softmax ? expf(f[i] - top) * inv : logistic(f[i]);
                // (the sum is of no account but for a logit of -inf)
                word[i] = plain_key(fminf(a.bias ? s + b[i] : s, f[i] + 3e38f));
            }
        }
        bool sure = true;
        if (a.groups > 1) {
            uint32_t least, most;
            keep_groups<IPL>(a, word, reinterpret_cast<uint32_t *>(seen[warp]), lane, least, most);
            if (!direct && most != 0u) {
                const float v = plain_value(least);
                sure = v - plain_value(most) > 2.0f * open + fabsf(v) * 0x1p-21f;
            }
        }
        int found;
        float logit, e, s = 0.0f;   // of the lane's candidate: its logit, exp(-|logit|), its score
        const auto look = [&](int idx, bool is) {
            logit = is ? to_f<T>(l[idx]) : 0.0f;
            e = expf(-fabsf(logit));
            if (!a.softmax)
                s = __fdividef(logit >= 0.0f ? 1.0f : e, 1.0f + e);
            else if (!direct)
                s = expf(logit - top) / total;
        };
        if (sure) {
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                word[i] = word_of<IPL>(word[i], lane, i);
            sort_lane<IPL>(word);
            // lanes 0 .. n - 1 get the k largest words and the one after them
            uint32_t mine = 0u;
            const int most = min(direct && sizeof(T) == 2 ? a.k : a.k + 1, 32);
            int n = 0;
            bool left = true;   // there are others
            for (; n < most; ++n) {
                const uint32_t m = take_largest<IPL>(word);
                if (m <= NEVER<uint32_t>) {
                    left = false;   // only what is never chosen
                    break;
                }
                mine = lane == n ? m : mine;
            }
            my_idx = lane < n ? expert_of<IPL>(mine) : -1;
            look(my_idx, lane < n);
            found = min(n, a.k);
            if (!direct || sizeof(T) == 4) {
                const bool more = n > a.k || left;   // (with k = 32 the one after them is not in a lane)
                float bias = a.bias && lane < n ? __ldg(a.bias + my_idx) : 0.0f;
                // what the words leave out is below the k-th, and every slot above the one after it, or equal to it in
                // what it is computed from
                const float c = direct ? logit : s + bias;
                const float after = __shfl_down_sync(ALL, c, 1);
                const float near = direct ? 0.0f : 0x1p-22f;
                bool ok = lane + 1 >= n || c - after > open + fabsf(c) * near;
                if (!__all_sync(ALL, ok)) {
                    const float after_logit = __shfl_down_sync(ALL, logit, 1), after_bias = __shfl_down_sync(ALL, bias, 1);
                    const int after_idx = __shfl_down_sync(ALL, my_idx, 1);
                    ok = __all_sync(ALL, ok || (logit == after_logit && bias == after_bias && my_idx < after_idx));
                }
                const uint32_t last = __shfl_sync(ALL, mine, a.k - 1);
                const auto apart = [&](uint32_t word_after) {
                    const float v = least_of<IPL>(last);
                    return v - most_of<IPL>(word_after) > open + fabsf(v) * near;
                };
                bool whole = !more || (n > a.k && apart(__shfl_sync(ALL, mine, a.k & 31)));
                if (!whole || !ok) {
                    while (!whole && n < 32) {
                        const uint32_t m = take_largest<IPL>(word);
                        whole = m <= NEVER<uint32_t>;
                        if (!whole) {
                            mine = lane == n ? m : mine;
                            ++n;
                            whole = apart(m);
                        }
                    }
                    if (!whole || (a.softmax && !direct)) {
                        found = choose_exactly<T, IPL>(a, l, seen[warp], lane, my_idx);
                    } else {
                        my_idx = lane < n ? expert_of<IPL>(mine) : -1;
                        logit = lane < n ? to_f<T>(l[my_idx]) : 0.0f;
                        bias = a.bias && lane < n ? __ldg(a.bias + my_idx) : 0.0f;
                        my_idx = direct ? rank_exactly<true>(logit, 0.0f, false, my_idx, n, lane)
                                        : rank_exactly<false>(logit, bias, a.bias, my_idx, n, lane);
                    }
                    look(my_idx, lane < found);
                }
            }
            my_idx = lane < found ? my_idx : -1;
        } else {
            found = choose_exactly<T, IPL>(a, l, seen[warp], lane, my_idx);
            look(my_idx, lane < found);
        }
        const bool chosen = lane < found;
        float p = 0.0f;
        if (a.softmax) {
            if (a.renorm)
                top = warp_max_f(chosen ? logit : -INFINITY);
            p = chosen ? expf(logit - top) : 0.0f;
            if (a.renorm)
                total = warp_sum(p);
        } else {
            p = chosen ? s : 0.0f;
            // all scores may be tiny, their quotients are not: s = exp(l - m) / (1 + exp(l)) * exp(m) with m the largest
            if (a.renorm && !__any_sync(ALL, chosen && logit >= 0.0f)) {
                const float m = warp_max_f(chosen ? logit : -INFINITY);
                p = chosen ? expf(logit - m) / (1.0f + e) : 0.0f;
            }
            total = a.renorm ? warp_sum(p) : 1.0f;
        }
        if (chosen)
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
    const uint32_t same = __match_any_sync(ALL, e);
    if (__any_sync(ALL, e >= 0 && (same & (same - 1u)) != 0u)) {
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
    ScoreArgs a{};
    a.T = T, a.E = E, a.k = topk;
    a.logits = logits, a.ld = ld, a.bias = bias, a.mask = token_mask;
    a.softmax = score == MOE_SCORE_SOFTMAX, a.renorm = renormalize, a.scale = scale;
    a.idx = topk_idx, a.w = topk_w;
    a.groups = topk_groups == groups ? 1 : groups;   // (if all of them stay there are none)
    a.kept = topk_groups, a.pair = group_top == 2;
    a.per = E / a.groups;
    a.lanes = 1;
    while ((a.lanes * 2) * a.groups <= 32) {
        a.lanes *= 2;
        ++a.shift;
    }
    a.per_magic = (1u << 20) / static_cast<uint32_t>(a.per) + 1;   // exact for e, per <= 1024
    const int ipl = lane_experts(E);
    a.group_shift = -1;
    for (int s = 0; s <= 5; ++s)
        if (a.per == ipl << s)
            a.group_shift = s;
    const auto vectors = [&](const void *p, size_t pitch, size_t size) {
        const size_t piece = ipl * size < 16 ? ipl * size : 16;
        return E % ipl == 0 && op_aligned(p, piece) && pitch * size % piece == 0;
    };
    a.vec = vectors(logits, static_cast<size_t>(ld), dtype_bytes(dtype));
    a.bias_vec = vectors(bias, 0, 4);
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
