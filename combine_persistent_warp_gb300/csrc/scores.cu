// scores.cu -- the router over sigmoid or softmax scores: a bias for balance, groups of experts, top-k and
// scaled gate weights, and the gradient of the logits.
//
//   s_e = 1/(1 + exp(-l_e)) or exp(l_e)/sum exp(l);  c_e = s_e + b_e (the choice alone sees the bias)
//   a group's score is the sum of its one or two largest c (of one where no more can be chosen); the best groups stay, and
//   of their experts the k with the largest c are chosen; ties go to the lowest group or expert; -inf is never chosen, NaN
//   counts as the largest
//   w_j = scale * s_j, or scale * s_j / sum_i s_i over the chosen ones (renormalised)
//   gradient, with dot = sum_i w_i dw_i:
//     sigmoid  renormalised w_j (dw_j - dot/scale)(1 - s_j), otherwise w_j dw_j (1 - s_j)
//     softmax  renormalised w_j (dw_j - dot/scale), otherwise p_e (scale [e chosen] dw_e - dot)
//
// The choice is that of c in 64 bits.  Two values of c that 32 bits hold for equal or swap are rare, and
// which expert a token goes to should not hang on a rounding: c is computed in 32 bits with a bound of
// its error, and the candidates that this bound leaves open are ranked again in 64.
//
// The data is small: the instructions bound it, and how many warps an SM has to hide their latency; for few tokens
// latency alone.  Measured on a GB300 in graphs, bf16, top 8: 16384 x 128 in 8 groups of which 4 stay 11.0 us (a token
// that is ranked in 64 bits adds 1 us, one whose groups are in doubt 2), in one group 8.5, without a bias 6.7; its
// gradient 3.3; x 256 14.6, 9.0, 8.2 and 3.7; 128 x 32 fp32 in 4 groups 2.2 and 1.8.  Slower: tokens whose logits have no
// bias but sums of two (16384 x 128, coarse values whose sums tie) 21; softmax scores with a bias, chosen again with all
// experts where they are open, 19 (in 8 groups 23; x 256 41 and 34); over 256 experts, as lanes hold 32 each, of which 384
// fill 12 lanes and 512 16, unsorted and with ten bits of the word for the expert (x 384 58 in one group, x 512 77 in 8).
#include <climits>

#include "moe_internal.cuh"
#include "ptx.cuh"
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
// A word is what the choice goes by: c in its upper bits and, below them, the expert (ties to the lowest), so that
// one warp maximum a slot finds both.  The bits that the expert takes make a few more values look equal; what
// the words leave open is settled by the candidates' exact values.  c is there as the upper bits of its order
// key or, where it is a sigmoid with a bias between -0.999 and 0.999, as a whole number of 2^-21 (FIXED): near 1 the
// key's 7 bits less would leave 2^-16.
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
// FIXED: 3 * 2^22 + c * 2^21 as a float, whose bits are in order; a c of -1 stands for one that is not there.
constexpr float FIXED_ZERO = 12582912.0f, FIXED_ONE = 2097152.0f;
template <int IPL, bool FIXED>
__device__ __forceinline__ uint32_t word_of(float c, int lane, int i)
{
    const uint32_t id = ID<IPL> - static_cast<uint32_t>(lane * IPL + i);
    if constexpr (FIXED) {
        float t;
        asm("max.NaN.f32 %0, %1, 0fBF800000;" : "=f"(t) : "f"(c));   // (a NaN stays one: the largest)
        t = fmaf(t, FIXED_ONE, FIXED_ZERO);
        return (__float_as_uint(t) << BITS<IPL>) + id;
    } else {
        return (plain_key(c) & ~ID<IPL>) | id;
    }
}
// Words up to this one are not there.
template <int IPL, bool FIXED>
constexpr uint32_t NO_WORD = FIXED ? ((0x4B400000u - 0x200000u) << BITS<IPL>) + ID<IPL> : 0x007FFFFFu;
template <int IPL>
__device__ __forceinline__ int expert_of(uint32_t word) { return static_cast<int>(ID<IPL> - (word & ID<IPL>)); }
// The least (most) that the c of a word can be.
template <int IPL, bool FIXED, bool MOST>
__device__ __forceinline__ float bound_of(uint32_t word)
{
    if constexpr (FIXED) {
        const float t = __uint_as_float(0x4B000000u + (word >> BITS<IPL> & 0xFFFFFFu));
        return (t - FIXED_ZERO) * (1.0f / FIXED_ONE) + (MOST ? 0x1p-22f : -0x1p-22f);
    } else {
        return plain_value(MOST ? word | ID<IPL> : word & ~ID<IPL>);
    }
}

// The sigmoid's c in 64 bits, as a key.  (One copy of this code: what is seldom run is seldom at hand.)
__device__ __noinline__ uint64_t exact_key(float logit, float bias, bool has_bias)
{
    const double s = 1.0 / (1.0 + exp(-static_cast<double>(logit)));
    return logit == -INFINITY ? 0ull : order_key(has_bias ? s + static_cast<double>(bias) : s);
}

// The lanes of a token, of Q side by side.
template <int Q>
constexpr uint32_t SLOTS = Q == 1 ? ALL : (1u << (32 / Q)) - 1u;

// Which groups of experts stay, from the two largest keys of each, of Q tokens side by side: keys of group g are those
// of the lanes g << shift and after.  Lane q * SEG + g gets the score `own` of group g of token q (0: nothing there),
// whether it stays, and the token's lowest score that stays and highest that does not (0: none); with SIZES also half the
// size of what the score is the sum of (half: it is finite).
__device__ __forceinline__ uint32_t key_sum(uint32_t a, uint32_t b) { return plain_key(plain_value(a) + plain_value(b)); }
__device__ __forceinline__ uint64_t key_sum(uint64_t a, uint64_t b) { return order_key(key_value(a) + key_value(b)); }
template <typename K, int Q>
struct Groups {
    K first[Q], second[Q], own, least, most;
    float size;
    bool stays;
};
template <bool SIZES, typename K, int Q>
__device__ __forceinline__ void choose_groups(const ScoreArgs &a, Groups<K, Q> &v, int lane, int shift)
{
    constexpr int SEG = 32 / Q;
    const int seg = lane / SEG, slot = lane % SEG;
    K own = 0;
    float size = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        K score = v.first[q] > NEVER<K> ? v.first[q] : 0;
        const bool two = a.pair && v.second[q] > NEVER<K>;
        if (two)
            score = key_sum(v.first[q], v.second[q]);
        const K its = __shfl_sync(ALL, score, slot << shift & 31);
        own = seg == q ? its : own;
        if constexpr (SIZES) {
            if (a.pair && a.bias) {
                const float first = 0.5f * fabsf(plain_value(v.first[q])), second = two ? 0.5f * fabsf(plain_value(v.second[q])) : 0.0f;
                const float its_size = __shfl_sync(ALL, first + second, slot << shift & 31);
                size = seg == q ? its_size : size;
            }
        }
    }
    own = slot < a.groups ? own : 0;
    if constexpr (SIZES)
        v.size = a.pair && a.bias ? size : 0.5f * fabsf(plain_value(own));
    int rank = 0;   // ties: the lowest first
#pragma unroll 4
    for (int g = 0; g < a.groups; ++g) {
        const K other = __shfl_sync(ALL, own, g, SEG);
        rank += other > own || (other == own && g < slot);
    }
    const uint32_t last = __ballot_sync(ALL, own != 0 && rank == a.kept - 1) >> (seg * SEG) & SLOTS<Q>;
    const uint32_t after = __ballot_sync(ALL, own != 0 && rank == a.kept) >> (seg * SEG) & SLOTS<Q>;
    const K least = __shfl_sync(ALL, own, __ffs(static_cast<int>(last)) - 1, SEG);
    const K most = __shfl_sync(ALL, own, __ffs(static_cast<int>(after)) - 1, SEG);
    v.own = own;
    v.least = last ? least : 0;
    v.most = after ? most : 0;
    v.stays = own != 0 && rank < a.kept;
}
template <typename K>
__device__ __forceinline__ void insert(K v, K &first, K &second)
{
    second = max(second, min(first, v));
    first = max(first, v);
}
template <typename K, int Q>
__device__ __forceinline__ void merge_lanes(Groups<K, Q> &v, int lanes)
{
    for (int o = 1; o < lanes; o <<= 1) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const K f = __shfl_xor_sync(ALL, v.first[q], o), s = __shfl_xor_sync(ALL, v.second[q], o);
            v.second[q] = max(max(v.second[q], s), min(v.first[q], f));
            v.first[q] = max(v.first[q], f);
        }
    }
}
// Where expert e's key lies for the lanes that look through groups that are not whole lanes.
__device__ __forceinline__ int spot(int e) { return e + (e >> 5) * 4; }
template <int IPL>
constexpr int SPOTS = IPL * 36;

// The same of one token, whose scores may be `off` away (lane g: group g): groups that are so far above all that do not stay
// are sure to, and those in doubt are ranked by their scores in 64 bits for the places that are left.  Returns the
// groups that stay.
template <typename T>
__device__ __noinline__ uint32_t groups_exactly(const ScoreArgs &a, const T *l, uint32_t own, bool stays, float off, uint64_t *seen, int lane)
{
    const float v = plain_value(own);
    float low = v - off, high = v + off;   // (a NaN or an infinity: anywhere)
    low = low == low ? low : -INFINITY;
    high = high == high ? high : INFINITY;
    const float least = -warp_max_f(own != 0u && stays ? -low : -INFINITY), most = warp_max_f(own != 0u && !stays ? high : -INFINITY);
    const bool sure = stays && low > most;
    const bool doubt = own != 0u && !sure && (stays || !(high < least));
    const uint32_t in_doubt = __ballot_sync(ALL, doubt);
    const int left = a.kept - __popc(__ballot_sync(ALL, sure)), n = __popc(in_doubt);
    for (int i = lane; i < n * a.per; i += 32) {
        const int nth = static_cast<int>((static_cast<uint32_t>(i) * a.per_magic) >> 20);
        uint32_t after = in_doubt;
        for (int k = 0; k < nth; ++k)
            after &= after - 1u;
        const int e = (__ffs(static_cast<int>(after)) - 1) * a.per + i - nth * a.per;
        seen[i] = exact_key(to_f<T>(l[e]), a.bias ? a.bias[e] : 0.0f, a.bias);
    }
    __syncwarp();
    uint64_t first = 0, second = 0;
    if (lane < n) {
#pragma unroll 4
        for (int i = 0; i < a.per; ++i)
            insert(seen[lane * a.per + i], first, second);
    }
    __syncwarp();
    if (a.pair && second != 0)
        first = key_sum(first, second);
    int rank = 0;
    for (int r = 0; r < n; ++r) {
        const uint64_t other = __shfl_sync(ALL, first, r);
        rank += other > first || (other == first && r < lane);
    }
    const uint32_t chosen = __ballot_sync(ALL, lane < n && rank < left);
    return __ballot_sync(ALL, sure || (doubt && (chosen >> __popc(in_doubt & ((1u << lane) - 1u)) & 1u)));
}

// What a token's softmax is taken with, and how near two values of c are open (beside 2^-22 of their size).
struct Softmax {
    float top, total, open;
};

// -inf in place of the c of the groups that do not stay, of Q tokens from row l on (there: routed[q]).  sure[q] is
// false where scores are softmax and which groups stay is in doubt.
template <typename T, int IPL, int Q, bool FIXED>
__device__ __forceinline__ void keep_groups(const ScoreArgs &a, const T *l, const bool (&routed)[Q], float (&c)[Q][IPL], const Softmax (&sm)[Q],
                                            bool direct, uint64_t *seen, int lane, bool (&sure)[Q])
{
    Groups<uint32_t, Q> v;
    const bool in_lanes = a.group_shift >= 0;   // a group is 1 << group_shift lanes
    const int shift = in_lanes ? a.group_shift : a.shift;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        v.first[q] = v.second[q] = 0u;
        if (in_lanes) {
            v.first[q] = plain_key(c[q][0]);
#pragma unroll
            for (int i = 1; i < IPL; ++i)
                insert(plain_key(c[q][i]), v.first[q], v.second[q]);
        } else {
            uint32_t *keys = reinterpret_cast<uint32_t *>(seen);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                if (lane * IPL + i < a.E)
                    keys[spot(lane * IPL + i)] = plain_key(c[q][i]);
            __syncwarp();
            const int g = lane >> shift;
            if (g < a.groups)
                for (int e = lane & (a.lanes - 1); e < a.per; e += a.lanes)
                    insert(keys[spot(g * a.per + e)], v.first[q], v.second[q]);
            __syncwarp();
        }
    }
    merge_lanes(v, 1 << shift);
    choose_groups<!FIXED>(a, v, lane, shift);
    constexpr int SEG = 32 / Q;
    float open = sm[0].open;
#pragma unroll
    for (int q = 1; q < Q; ++q)
        open = lane / SEG == q ? sm[q].open : open;
    // A score is `off` away at most: its two values as far as two values of c are, 2^-24 of each for their sums with the bias and of
    // their sum's own size, and as much again for the comparison's roundings.  The values' sizes are more than their sum's where
    // their signs differ: by less than 2 with small biases (FIXED, no value below -1), by nothing without one.  Scores that are
    // all on their side of the border by that much are in order.
    const float own = plain_value(v.own), border = 0.5f * plain_value(v.least) + 0.5f * plain_value(v.most);
    const float off = FIXED ? open + 0x1p-23f + fabsf(own) * 0x1p-22f : open + v.size * 0x1p-21f;
    const uint32_t stays = __ballot_sync(ALL, v.stays);
    const uint32_t doubt = __ballot_sync(ALL, !direct && v.most != 0u && v.own != 0u && !(v.stays ? own - off > border : own + off < border));
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        uint32_t stay = stays >> (q * SEG) & SLOTS<Q>;
        if (routed[q] && (doubt >> (q * SEG) & SLOTS<Q>)) {
            if (a.softmax) {
                sure[q] = false;
            } else {
                const int from = q * SEG + lane % SEG;
                const uint32_t its_own = __shfl_sync(ALL, v.own, from);
                const float its_off = __shfl_sync(ALL, off, from);
                stay = groups_exactly<T>(a, l + q * a.ld, lane < SEG ? its_own : 0u, lane < SEG && (stay >> lane & 1u), its_off, seen, lane);
            }
        }
#pragma unroll
        for (int i = 0; i < IPL; ++i) {
            const int e = lane * IPL + i, g = in_lanes ? lane >> shift : static_cast<int>((static_cast<uint32_t>(e) * a.per_magic) >> 20);
            c[q][i] = e < a.E && (stay >> (g & 31) & 1u) ? c[q][i] : -INFINITY;
        }
    }
}

// Without a bias scores are in the order of the logits, which are exact.
__device__ __forceinline__ bool directly(const ScoreArgs &a) { return !a.bias && (a.groups == 1 || !a.pair); }

// The choice in 64 bits of all experts.  Seldom run, so that its code is seldom at hand: short, over keys in shared
// memory.
template <typename T, int IPL>
__device__ __noinline__ int choose_exactly(const ScoreArgs &a, const T *l, uint64_t *seen, int lane, int &my_idx)
{
    const bool direct = directly(a), softmax = a.softmax && !direct;
    double total = 1.0;
    if (softmax) {
        float m = -INFINITY;   // (the logits have at most 32 bits)
        for (int e = lane; e < a.E; e += 32)
            m = fmaxf(m, to_f<T>(l[e]));
        const double top = static_cast<double>(warp_max_f(m));
        double sum = 0.0;
        // (each lane's exponentials wait for the total in the places of its keys)
#pragma unroll 2
        for (int e = lane; e < a.E; e += 32) {
            const double x = exp(static_cast<double>(to_f<T>(l[e])) - top);
            sum += x;
            seen[spot(e)] = static_cast<uint64_t>(__double_as_longlong(x));
        }
        total = warp_sum(sum);
    }
#pragma unroll 2
    for (int e = lane; e < a.E; e += 32) {
        const float f = to_f<T>(l[e]);
        if (direct) {
            seen[spot(e)] = order_key(static_cast<double>(f));
        } else if (a.softmax) {
            const double p = __longlong_as_double(static_cast<long long>(seen[spot(e)])) / total;
            seen[spot(e)] = f == -INFINITY ? 0ull : order_key(a.bias ? p + static_cast<double>(a.bias[e]) : p);
        } else {
            seen[spot(e)] = exact_key(f, a.bias ? a.bias[e] : 0.0f, a.bias);
        }
    }
    __syncwarp();
    if (a.groups > 1) {
        Groups<uint64_t, 1> v;
        uint64_t first = 0, second = 0;
        const int g = lane >> a.shift;
        if (g < a.groups)
#pragma unroll 2
            for (int e = lane & (a.lanes - 1); e < a.per; e += a.lanes)
                insert(seen[spot(g * a.per + e)], first, second);
        v.first[0] = first;
        v.second[0] = second;
        merge_lanes(v, a.lanes);
        choose_groups<false>(a, v, lane, a.shift);
        const uint32_t stay = __ballot_sync(ALL, v.stays);
        for (int e = lane; e < a.E; e += 32)
            if (!(stay >> ((static_cast<uint32_t>(e) * a.per_magic) >> 20) & 1u))
                seen[spot(e)] = 0;
        __syncwarp();
    }
    my_idx = -1;
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = 0;
        int at = INT_MAX;
#pragma unroll 4
        for (int e = lane; e < a.E; e += 32) {
            const uint64_t key = seen[spot(e)];
            at = key > best ? e : at;
            best = max(best, key);
        }
        const uint64_t m = warp_max(best);
        if (m == 0)
            return j;   // only what is never chosen is left
        const int e = __reduce_min_sync(ALL, best == m ? at : INT_MAX);
        if ((e & 31) == lane)
            seen[spot(e)] = 0;
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
    const uint64_t key = DIRECT ? order_key(static_cast<double>(logit)) : exact_key(logit, bias, has_bias);
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

// The same of Q rows from row l on, `there` of which there are, all on their way before the first is looked at.
template <typename T, int IPL>
struct Lane {
    T v[IPL];
};
template <typename T, int IPL, int Q>
__device__ __forceinline__ void load_lanes(Lane<T, IPL> (&f)[Q], const T *l, long long ld, int there, int lane, int E, bool vec)
{
    constexpr int BYTES = IPL * static_cast<int>(sizeof(T)), PIECE = BYTES < 16 ? BYTES : 16, N = PIECE / static_cast<int>(sizeof(T));
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            f[q].v[i] = from_f<T>(0.0f);
    if (N > 1 && vec) {
        struct alignas(PIECE) Piece {
            T v[N];
        };
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < IPL / N; ++i)
                if (q < there && lane * IPL < E) {
                    const Piece p = reinterpret_cast<const Piece *>(l + q * ld + lane * IPL)[i];
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        f[q].v[i * N + k] = p.v[k];
                }
    } else {
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                if (q < there && lane * IPL + i < E)
                    f[q].v[i] = l[q * ld + lane * IPL + i];
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

// The c of Q tokens, from row l on, from their logits and the biases, without those of the groups that do not stay.
// Of tokens that are not routed, or not there, no logit is looked up.
template <typename T, int IPL, int Q, bool FIXED>
__device__ __forceinline__ void make_c(const ScoreArgs &a, const T *l, const bool (&routed)[Q], float (&f)[Q][IPL], const float (&b)[IPL],
                                       bool direct, uint64_t *seen, int lane, Softmax (&sm)[Q], bool (&sure)[Q])
{
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        sm[q] = {0.0f, 1.0f, 0.0f};
        sure[q] = true;
        if (a.softmax && !(direct && a.renorm)) {
            float top = f[q][0], total = 0.0f;
#pragma unroll
            for (int i = 1; i < IPL; ++i)
                top = fmaxf(top, f[q][i]);
            top = warp_max_f(top);
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                if (lane * IPL + i < a.E)
                    total += expf(f[q][i] - top);
            sm[q].top = top;
            sm[q].total = warp_sum(total);
        }
        if (direct) {
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                f[q][i] += 0.0f;   // (-0 as +0)
        } else {
            // Errors of c in units of 2^-24: the sigmoid's exponential (1.3 |l| + 2.8) times s (1 - s), at most 1, its
            // sum 1/2, the reciprocal 2; softmax (times 1/total, the largest probability) 8 of the two exponentials and
            // quotients, ln E of the exponents' roundings and 1/2 for each of the sum's IPL + 5 additions.  Twice that
            // for two values.
            sm[q].open = a.softmax ? (2.0f * IPL + 72.0f) * 0x1p-24f / sm[q].total : 0x1p-21f;
            const float inv = 1.0f / sm[q].total;
#pragma unroll
            for (int i = 0; i < IPL; ++i) {
                const float s = a.softmax ? expf(f[q][i] - sm[q].top) * inv : logistic(f[q][i]);
                // (-inf alone is never chosen: the lowest finite logit has a score of zero like others far below)
                f[q][i] = f[q][i] == -INFINITY ? -INFINITY : a.bias ? s + b[i] : s;
            }
        }
    }
    if (a.groups > 1)
        keep_groups<T, IPL, Q, FIXED>(a, l, routed, f, sm, direct, seen, lane, sure);
}
template <int IPL, bool FIXED>
__device__ __forceinline__ void make_words(uint32_t (&word)[IPL], const float (&c)[IPL], int lane)
{
#pragma unroll
    for (int i = 0; i < IPL; ++i)
        word[i] = word_of<IPL, FIXED>(c[i], lane, i);
    sort_lane<IPL>(word);
}
// Whether what has the word `after` or a lower one is below what has the word `last`.
template <int IPL, bool FIXED>
__device__ __forceinline__ bool apart(uint32_t last, uint32_t after, float open, bool direct)
{
    const float v = bound_of<IPL, FIXED, false>(last);
    return v - bound_of<IPL, FIXED, true>(after) > open + (direct ? 0.0f : fabsf(v) * 0x1p-22f);
}
// The choice of a token whose words leave it open: as many candidates as the words cannot tell from the k-th,
// by their values in 64 bits; failing that, all experts by theirs.  Lane j gets slot j's expert.
template <typename T, int IPL, bool FIXED>
__device__ __noinline__ int choose_again(const ScoreArgs &a, const T *l, uint64_t *seen, int lane, int &my_idx)
{
    const bool direct = directly(a);
    if (!a.softmax || direct) {
        float f[1][IPL], b[IPL];
        load_lane<T, IPL>(f[0], l, lane, a.E, a.vec);
        if (a.bias)
            load_lane<float, IPL>(b, a.bias, lane, a.E, a.bias_vec);
        uint32_t word[IPL], mine = 0u, last = 0u;
        Softmax sm[1];
        bool whole = false, sure[1];
        const bool routed[1] = {true};
        int n = 0;
        make_c<T, IPL, 1, FIXED>(a, l, routed, f, b, direct, seen, lane, sm, sure);
        if (sure[0]) {
            make_words<IPL, FIXED>(word, f[0], lane);
            while (!whole && n < 32) {
                const uint32_t m = take_largest<IPL>(word);
                whole = m <= NO_WORD<IPL, FIXED>;
                if (!whole) {
                    mine = lane == n ? m : mine;
                    last = n == a.k - 1 ? m : last;
                    ++n;
                    whole = n > a.k && apart<IPL, FIXED>(last, m, sm[0].open, direct);
                }
            }
        }
        if (whole) {
            my_idx = lane < n ? expert_of<IPL>(mine) : -1;
            const float logit = lane < n ? to_f<T>(l[my_idx]) : 0.0f;
            const float bias = a.bias && lane < n ? a.bias[my_idx] : 0.0f;
            my_idx = direct ? rank_exactly<true>(logit, 0.0f, false, my_idx, n, lane)
                            : rank_exactly<false>(logit, bias, a.bias, my_idx, n, lane);
            return min(n, a.k);
        }
    }
    return choose_exactly<T, IPL>(a, l, seen, lane, my_idx);
}

// Over the SEG lanes of a token.
template <int SEG>
__device__ __forceinline__ float seg_sum(float v)
{
#pragma unroll
    for (int o = SEG / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(ALL, v, o);
    return v;
}
template <int SEG>
__device__ __forceinline__ float seg_max(float v)
{
#pragma unroll
    for (int o = SEG / 2; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(ALL, v, o));
    return v;
}

// The tokens of the lanes `open`, whose order or last place is in doubt.  What the words leave out, from the one after
// the last slot on, is below the last slot, or is equal to it in what it is computed from and a later
// expert (with all slots in order the last is the lowest: it stays out then), but for one at most: then the slots
// and that one are ranked by their values in 64 bits.  Returns the lanes of the tokens of which more is in doubt.
template <typename T, int IPL, int Q, bool FIXED>
__device__ __forceinline__ uint32_t rank_again(const ScoreArgs &a, const T *l, uint32_t (&word)[Q][IPL], uint32_t last, uint32_t next, bool sure,
                                               bool in_order, float gap, uint32_t open, int found, float logit, float bias, int &my_idx,
                                               int lane)
{
    constexpr int SEG = 32 / Q;
    const int seg = lane / SEG, slot = lane % SEG;
    const bool direct = !FIXED && directly(a);
    if (a.softmax && !direct)
        return open;
    const uint32_t unordered = __ballot_sync(ALL, !in_order) >> (seg * SEG) & SLOTS<Q>;
    const float last_logit = __shfl_sync(ALL, logit, a.k - 1, SEG), last_bias = __shfl_sync(ALL, bias, a.k - 1, SEG);
    const int last_idx = __shfl_sync(ALL, my_idx, a.k - 1, SEG);
    bool mine = (open >> (seg * SEG) & SLOTS<Q>) && sure;
    int x = -1;   // the one more
    float x_logit = 0.0f, x_bias = 0.0f;
    for (;;) {
        const bool more = mine && next > NO_WORD<IPL, FIXED> && !apart<IPL, FIXED>(last, next, gap, direct);
        if (more) {
            const int e = expert_of<IPL>(next);
            const float e_logit = to_f<T>(l[e]), e_bias = a.bias ? a.bias[e] : 0.0f;
            if (unordered || e_logit != last_logit || e_bias != last_bias || e < last_idx) {
                mine = x < 0;
                x = e, x_logit = e_logit, x_bias = e_bias;
            }
        }
        if (!__any_sync(ALL, more && mine))
            break;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const uint32_t m = take_largest<IPL>(word[q]);
            next = seg == q ? m : next;
        }
    }
    x = mine ? x : -1;
    const uint32_t ranked = __ballot_sync(ALL, mine);
    if (__any_sync(ALL, mine && (unordered || x >= 0))) {
        const bool there = mine && slot < found;
        uint64_t key = 0, its_key = 0;
        if (direct) {
            key = order_key(static_cast<double>(logit));
            its_key = order_key(static_cast<double>(x_logit));
        } else {
            key = exact_key(logit, bias, a.bias);
            if (__any_sync(ALL, x >= 0))
                its_key = exact_key(x_logit, x_bias, a.bias);
        }
        int rank = x >= 0 && (its_key > key || (its_key == key && x < my_idx)), its_rank = 0;
        for (int r = 0; r < a.k; ++r) {
            const uint64_t other = __shfl_sync(ALL, key, r, SEG);
            const int its = __shfl_sync(ALL, my_idx, r, SEG);
            rank += its >= 0 && (other > key || (other == key && its < my_idx));
            its_rank += other > its_key || (other == its_key && its < x);
        }
        int got = x >= 0 && its_rank == slot ? x : -1;
        for (int r = 0; r < a.k; ++r) {
            const int at = __shfl_sync(ALL, rank, r, SEG), its = __shfl_sync(ALL, my_idx, r, SEG);
            got = its >= 0 && at == slot ? its : got;
        }
        my_idx = there ? got : my_idx;
    }
    return open & ~ranked;
}

// A warp takes Q tokens: it chooses for each with all lanes, side by side (a token's warp maxima wait for one
// another), and then has the slots of all of them, a lane each (SEG = 32/Q >= k lanes a token), for the
// weights and what is to be checked.
template <typename T, int IPL, int Q, bool FIXED>
__device__ __forceinline__ void score_tokens(const ScoreArgs &a, const Lane<T, IPL> (&its_logits)[Q], bool is_routed, const float (&b)[IPL],
                                             uint64_t *seen, int t0, int lane)
{
    constexpr int SEG = 32 / Q;
    const int seg = lane / SEG, slot = lane % SEG, t = t0 + seg;
    const bool direct = !FIXED && directly(a);
    // token q's row, by all lanes; whether it is there and routed
    const auto row = [&](int q) { return static_cast<const T *>(a.logits) + static_cast<size_t>(t0 + q) * a.ld; };
    const uint32_t lanes = __ballot_sync(ALL, is_routed);
    bool routed[Q];
    float f[Q][IPL];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        routed[q] = lanes >> (q * SEG) & 1u;
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            f[q][i] = lane * IPL + i < a.E ? to_f<T>(its_logits[q].v[i]) : -INFINITY;
    }
    uint32_t word[Q][IPL], largest[Q];
    Softmax its[Q];
    bool its_sure[Q];
    make_c<T, IPL, Q, FIXED>(a, row(0), routed, f, b, direct, seen, lane, its, its_sure);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        make_words<IPL, FIXED>(word[q], f[q], lane);
#pragma unroll
        for (int i = 0; i < IPL; ++i)   // a token that is not routed has none
            word[q][i] = routed[q] ? word[q][i] : 0u;
    }
    // this lane's token: the words of the slot, of the last and of the one after it, how many are found
    uint32_t mine = 0u, next = 0u, last = 0u;
    for (int n = 0; n < a.k; ++n) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            largest[q] = take_largest<IPL>(word[q]);
            mine = lane == q * SEG + n ? largest[q] : mine;
        }
    }
    Softmax sm{0.0f, 1.0f, 0.0f};
    bool sure = true;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const uint32_t after = direct && sizeof(T) == 2 ? 0u : take_largest<IPL>(word[q]);
        if (seg == q) {
            last = largest[q];
            next = after;
            sm = its[q];
            sure = its_sure[q];
        }
    }
    // (what is never chosen comes last)
    int found = __popc(__ballot_sync(ALL, mine > NO_WORD<IPL, FIXED>) >> (seg * SEG) & SLOTS<Q>);
    const T *l = static_cast<const T *>(a.logits) + static_cast<size_t>(t) * a.ld;
    int my_idx = slot < found ? expert_of<IPL>(mine) : -1;
    float logit, e, s;   // of the lane's slot: its logit, exp(-|logit|), its score
    const auto look = [&] {
        logit = slot < found ? to_f<T>(l[my_idx]) : 0.0f;
        if (a.softmax) {
            s = expf(logit - sm.top) / sm.total;
        } else {
            e = expf(-fabsf(logit));
            s = __fdividef(logit >= 0.0f ? 1.0f : e, 1.0f + e);
        }
    };
    look();
    if (!direct || sizeof(T) == 4) {
        // what the words leave out is below the last slot, and every slot above the one after it, or equal to it in what
        // it is computed from
        const float bias = a.bias && slot < found ? a.bias[my_idx] : 0.0f;
        const float c = direct ? logit : s + bias;
        const float after = __shfl_down_sync(ALL, c, 1), after_logit = __shfl_down_sync(ALL, logit, 1);
        const float after_bias = __shfl_down_sync(ALL, bias, 1);
        const int after_idx = __shfl_down_sync(ALL, my_idx, 1);
        const bool edge = next <= NO_WORD<IPL, FIXED> || apart<IPL, FIXED>(last, next, sm.open, direct);
        bool ok = true;
        if (slot + 1 < found)
            ok = c - after > sm.open + (direct ? 0.0f : fabsf(c) * 0x1p-22f) ||
                 (logit == after_logit && bias == after_bias && my_idx < after_idx);
        uint32_t open = __ballot_sync(ALL, !(ok && sure && edge));
        if (open) {
            open = rank_again<T, IPL, Q, FIXED>(a, l, word, last, next, sure, ok, sm.open, open, found, logit, bias, my_idx, lane);
            while (open) {
                const int q = (__ffs(static_cast<int>(open)) - 1) / SEG;
                int idx;
                const int n = choose_again<T, IPL, FIXED>(a, row(q), seen, lane, idx);
                idx = __shfl_sync(ALL, idx, slot);
                if (seg == q) {
                    found = n;
                    my_idx = slot < n ? idx : -1;
                }
                open &= ~(SLOTS<Q> << (q * SEG));
            }
            look();
        }
    }
    const bool chosen = slot < found;
    float p = chosen ? s : 0.0f, total = 1.0f;
    if (a.renorm) {
        // all scores may be tiny, their quotients are not: s = exp(l - m) / (1 + exp(l)) * exp(m) with m the largest
        const float m = seg_max<SEG>(chosen ? logit : -INFINITY);
        if (chosen && a.softmax)
            p = expf(logit - m);
        else if (chosen && m < 0.0f)
            p = expf(logit - m) / (1.0f + e);
        total = seg_sum<SEG>(p);
    }
    if (slot < a.k && t < a.T) {
        const size_t at = static_cast<size_t>(t) * a.k + slot;
        a.idx[at] = my_idx;
        a.w[at] = chosen ? p / total * a.scale : 0.0f;
    }
}

// Seven blocks an SM (at most 72 registers): with the 80 that four tokens would take 6144 x 128 bf16 in 8 groups is 7.8 us
// and not 6.8, 16384 unbiased 7.1 and not 6.6 (in 8 groups 10.4 and 11.1); eight are as slow.
template <typename T, int IPL, int Q>
__global__ void __launch_bounds__(WARPS * 32, IPL <= 4 ? 7 : 1) score_kernel(const ScoreArgs a)
{
    ptx::follow();
    __shared__ uint64_t seen[WARPS][SPOTS<IPL>];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x * WARPS + warp) * Q;
    if (t0 >= a.T)
        return;
    // (what is read is on its way at once: padding too, which is not looked at)
    Lane<T, IPL> l[Q];
    load_lanes<T, IPL, Q>(l, static_cast<const T *>(a.logits) + static_cast<size_t>(t0) * a.ld, a.ld, a.T - t0, lane, a.E, a.vec);
    const int t = t0 + lane / (32 / Q);
    const bool routed = t < a.T && (!a.mask || a.mask[t]);
    float b[IPL];
    bool fixed = false;
    if (a.bias) {
        load_lane<float, IPL>(b, a.bias, lane, a.E, a.bias_vec);
        bool small = true;
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            small = small && (fabsf(b[i]) <= 0.999f || b[i] == -INFINITY);
        fixed = IPL <= 8 && !a.softmax && __all_sync(ALL, small);
    }
    if constexpr (IPL <= 8) {
        if (fixed)
            return score_tokens<T, IPL, Q, true>(a, l, routed, b, seen[warp], t0, lane);
    }
    score_tokens<T, IPL, Q, false>(a, l, routed, b, seen[warp], t0, lane);
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
    int vec;              // the rows that a warp clears start on 16-byte boundaries
};

// Blocks are placed at some 300 cycles each an SM: eight warps a block (65536 x 64 softmax scores as they are 16.9 us with four,
// 12.4 with eight).
constexpr int BWD_WARPS = 8;
// A slot's expert (-1: none), weight and gradient.
struct Slot {
    int e;
    float w, dw;
};
__device__ __forceinline__ Slot load_slot(const ScoreBwdArgs &a, int t, int slot)
{
    Slot s{-1, 0.0f, 0.0f};
    if (slot < a.k && t < a.T) {
        const size_t at = static_cast<size_t>(t) * a.k + slot;
        const int64_t id = a.idx[at];
        if (id >= 0 && id < a.E)
            s = {static_cast<int>(id), a.w[at], a.dw[at]};
    }
    return s;
}
// An expert that is in several slots of its token gets their sum, in order.
template <int Q>
__device__ __forceinline__ float sum_of_slots(float d, int e, int k, int lane)
{
    constexpr int SEG = 32 / Q;
    const uint32_t same = __match_any_sync(ALL, e < 0 ? -1 : e * Q + lane / SEG);
    if (__any_sync(ALL, e >= 0 && (same & (same - 1u)) != 0u)) {
        float sum = 0.0f;
        for (int j = 0; j < k; ++j) {
            const float v = __shfl_sync(ALL, d, j, SEG);
            sum += same >> (lane / SEG * SEG + j) & 1u ? v : 0.0f;
        }
        d = sum;
    }
    return d;
}

// All but softmax scores as they are: a gradient has k values and zeros around them.  A warp takes Q tokens, whose
// rows it clears in one piece, and has the slots of all of them, a lane each.
template <typename T, int Q>
__global__ void __launch_bounds__(BWD_WARPS * 32) score_backward_kernel(const ScoreBwdArgs a)
{
    ptx::follow();
    constexpr int SEG = 32 / Q, N = 16 / static_cast<int>(sizeof(T));
    const int lane = threadIdx.x & 31, t0 = (blockIdx.x * BWD_WARPS + (threadIdx.x >> 5)) * Q, t = t0 + lane / SEG;
    if (t0 >= a.T)
        return;
    const Slot s = load_slot(a, t, lane % SEG);
    T *out = static_cast<T *>(a.dlogits) + static_cast<size_t>(t0) * a.E;
    const int n = min(Q, a.T - t0) * a.E, whole = a.vec ? n / N * N : 0;
    for (int i = lane * N; i < whole; i += 32 * N)
        *reinterpret_cast<uint4 *>(out + i) = make_uint4(0u, 0u, 0u, 0u);
    for (int i = whole + lane; i < n; i += 32)
        out[i] = from_f<T>(0.0f);
    float d = s.w * s.dw;
    const float dot = seg_sum<SEG>(d);
    if (a.renorm)
        d = s.w * (s.dw - dot / a.scale);
    if (!a.softmax && s.e >= 0)
        d /= 1.0f + expf(to_f<T>(static_cast<const T *>(a.logits)[static_cast<size_t>(t) * a.ld + s.e]));
    d = sum_of_slots<Q>(d, s.e, a.k, lane);
    __syncwarp();   // the chosen ones over the zeros that other lanes have written
    if (s.e >= 0)
        out[lane / SEG * a.E + s.e] = from_f<T>(d);
}

// Softmax scores as they are: every logit has a gradient.
template <typename T, int IPL>
__global__ void __launch_bounds__(BWD_WARPS * 32) softmax_backward_kernel(const ScoreBwdArgs a)
{
    ptx::follow();
    const int t = blockIdx.x * BWD_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= a.T)
        return;
    const Slot s = load_slot(a, t, lane);
    const float dot = warp_sum(s.w * s.dw);
    const T *l = static_cast<const T *>(a.logits) + static_cast<size_t>(t) * a.ld;
    T *out = static_cast<T *>(a.dlogits) + static_cast<size_t>(t) * a.E;
    if (!__any_sync(ALL, s.e >= 0)) {
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            if (i * 32 + lane < a.E)
                out[i * 32 + lane] = from_f<T>(0.0f);
        return;
    }
    // what the slots add to that which the expert's probability is multiplied by
    const float d = sum_of_slots<1>(a.scale * s.dw, s.e, a.k, lane);
    float f[IPL], top = -INFINITY, sum = 0.0f;
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
    const float inv = 1.0f / warp_sum(sum);
#pragma unroll
    for (int i = 0; i < IPL; ++i)
        if (i * 32 + lane < a.E)
            out[i * 32 + lane] = from_f<T>(f[i] * inv * -dot);
    __syncwarp();   // the chosen ones over what the row's other lanes have written
    if (s.e >= 0)
        out[s.e] = from_f<T>(expf(to_f<T>(l[s.e]) - top) * inv * (d - dot));
}

// ------------------------------------------------------------------ host side ------------
template <typename T, int IPL, int Q>
void launch_scores(const ScoreArgs &a, cudaStream_t s)
{
    launch_programmatic(score_kernel<T, IPL, Q>, (a.T + WARPS * Q - 1) / (WARPS * Q), WARPS * 32, 0, s, a);
}
// Tokens of a warp: the more there are, the less their slots cost, and the fewer warps there are.  128 experts in 8
// groups, bf16, with 1, 2 and 4 of them: 2048 tokens 5.1, 5.2 and 5.5 us (unbiased, one group: 2.6, 2.8, 3.2), 4096
// 6.5, 6.0, 6.3 (4.0, 3.6, 4.1), 6144 7.8, 7.0, 8.8 (5.6, 4.3, 5.8), 8192 8.3, 6.7, 6.6 (6.4, 4.9, 4.8), 16384 15.6, 12.7, 10.9
// (11.2, 8.1, 6.7), 65536 50, 38, 31 (39, 25, 21).  256 experts: 4096 6.6, 5.5, 5.4 (4.9, 3.7, 3.8), 8192 10.7, 9.9, 10.0 (7.5, 6.1, 5.0),
// 65536 64, 55, 45 (44, 35, 27); 128 in fp32: 4096 6.2, 5.7, 5.6 (4.1, 3.9, 4.3), 8192 8.1, 7.7, 7.4 (7.2, 5.7, 5.8), 65536 48, 37, 31 (39, 26, 21).
constexpr int TWO_TOKENS = 4096, FOUR_TOKENS = 8192;
// Of the gradient, 128 experts, bf16: 1024 tokens 1.8, 2.0, 2.0 us, 2048 2.2, 2.0, 2.1, 4096 2.6, 2.4, 2.2, 16384 4.2, 3.2, 4.0, 32768
// 6.8, 4.8, 4.6, 65536 12.1, 8.1, 7.1; 256 experts: 2048 2.3, 2.1, 2.2, 16384 4.3, 3.7, 4.9, 32768 7.0, 5.7, 5.7, 65536 12.5, 9.6, 9.3.
constexpr int BWD_TWO = 2048, BWD_FOUR = 32768;
template <typename T, int IPL>
struct ScoreLaunch {
    static void go(const ScoreArgs &a, cudaStream_t s)
    {
        if constexpr (IPL <= 8) {
            if (a.k <= 8 && a.groups <= 8 && a.T >= FOUR_TOKENS)
                return launch_scores<T, IPL, 4>(a, s);
            if (a.k <= 16 && a.groups <= 16 && a.T >= TWO_TOKENS)
                return launch_scores<T, IPL, 2>(a, s);
        }
        launch_scores<T, IPL, 1>(a, s);
    }
};
template <typename T, int Q>
void launch_score_backward(ScoreBwdArgs a, cudaStream_t s)
{
    a.vec = op_aligned(a.dlogits, 16) && Q * a.E * static_cast<int>(sizeof(T)) % 16 == 0;
    launch_programmatic(score_backward_kernel<T, Q>, (a.T + BWD_WARPS * Q - 1) / (BWD_WARPS * Q), BWD_WARPS * 32, 0, s, a);
}
template <typename T>
void launch_score_backward(const ScoreBwdArgs &a, cudaStream_t s)
{
    a.k <= 8 && a.T >= BWD_FOUR    ? launch_score_backward<T, 4>(a, s)
    : a.k <= 16 && a.T >= BWD_TWO ? launch_score_backward<T, 2>(a, s)
                                   : launch_score_backward<T, 1>(a, s);
}
template <typename T, int IPL>
struct SoftmaxBwdLaunch {
    static void go(const ScoreBwdArgs &a, cudaStream_t s)
    {
        launch_programmatic(softmax_backward_kernel<T, IPL>, (a.T + BWD_WARPS - 1) / BWD_WARPS, BWD_WARPS * 32, 0, s, a);
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
    const ScoreBwdArgs a{T, E, topk, dw, topk_idx, topk_w, logits, ld, score == MOE_SCORE_SOFTMAX, renormalize, scale, dlogits, 0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.softmax && !renormalize)
        by_width<SoftmaxBwdLaunch>(dtype, E, a, s);
    else
        with_dtype(dtype, [&](auto *t) { launch_score_backward<std::remove_pointer_t<decltype(t)>>(a, s); });
    return launched();
}

}  // extern "C"
