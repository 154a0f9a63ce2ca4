// swiglu.cu -- the experts' activation over rows of gate and up, its gradient, and rows kept in 8 bits
// between the forward and the backward pass.
//
//   s = 1/(1 + exp(-g)):  act = g s u,  dg = da u (s + g s (1 - s)),  du = da g s
//   8 bits: 32 neighbours of a row share X = 2^floor(log2 max|v|) (a byte, its exponent + 127, at least
//   7), and each is n X/64 with the nearest whole n in -127 .. 127, ties to even (an MX block of INT8
//   elements).  X is a power of two, so v 64/X and n X/64 are exact and the rounding to n is the only one.
//
// All of it is elementwise and bound by HBM.  A thread takes E neighbours of gate and of up (32 bytes, or 16 or 8
// where the rows' boundaries allow no more), so 32/E neighbouring lanes hold a group; rows off those boundaries go
// element by element, a group a warp access.  Loads are plain ones, not of the read-only kind: kernels are launched
// before the one that writes what they read is done.
//
// Measured on a GB300 in graphs, floors by bytes at the measured copy bandwidth in brackets (a copy's writes are half of its
// bytes; these kernels' are less): bf16 65536 x 2048 113 us (120), gradient 188 (200), with the checkpoint 153 (162), gradient from it 190
// (202); rows of 32768 x 7168 kept 99 and restored 101 (106); 16-byte accesses and single fp32 operations took 181 for
// the checkpoint and 149 + 122 for the rows.  Rows off the boundaries are bound by issue: 65536 x 1403 104, 169, 177
// and 217 (82, 137, 111, 138), 20000 x 3001 kept 52 and restored 45 (27).
#include <climits>
#include <initializer_list>
#include <type_traits>

#include "moe_internal.cuh"
#include "op_common.cuh"
#include "ptx.cuh"

using namespace cpw;

namespace {

constexpr int THREADS = 256;
constexpr int GROUP = 32;       // values of a scale
constexpr int CHUNK = 256;      // elements of a warp (8 a lane)
constexpr uint32_t ALL = 0xFFFFFFFFu;
__host__ __device__ __forceinline__ int groups_of(int width) { return (width + GROUP - 1) / GROUP; }

// ------------------------------------------------------------------ the activation ------
// 1/(1 + exp(-g)) of a pair.  For 16-bit results two approximate instructions, together 2^-21 off at |g| <= 16 (the
// exponent's rounding grows with |g|); for fp32 the exact functions.  Zero for gates below -88.7, where exp(-g) is past the
// largest number.  The reciprocal flushes what is no normal number, which a bf16 `up` may bring back to an ordinary size (an
// fp16 one does not): there it is taken of a quarter of the sum (65536 x 1403 104 us, 99 without).
template <typename T>
__device__ __forceinline__ float2 logistic2(float2 g)
{
    if constexpr (std::is_same_v<T, float>) {
        return make_float2(1.0f / (1.0f + expf(-g.x)), 1.0f / (1.0f + expf(-g.y)));
    } else {
        constexpr float PART = std::is_same_v<T, __nv_bfloat16> ? 0.25f : 1.0f;
        float2 e = mul2(g, both(-1.44269504f));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
        e = PART == 1.0f ? add2(e, both(1.0f)) : fma2(e, both(PART), both(PART));
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
        return PART == 1.0f ? e : mul2(e, both(PART));
    }
}
// The gradients of a pair of gates and ups (in place; d becomes the activation).
template <typename T>
__device__ __forceinline__ void gradients(float2 &d, float2 &g, float2 &u)
{
    const float2 s = logistic2<T>(g), t = mul2(g, s), part = mul2(d, u);
    u = mul2(t, u);                                                          // the activation
    const float2 du = mul2(d, t);
    g = mul2(part, fma2(t, fma2(s, both(-1.0f), both(1.0f)), s));             // s + t (1 - s)
    d = u;
    u = du;
}

// ------------------------------------------------------------------ 8 bits --------------
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
// The byte of a group whose largest magnitude has these bits (255: a NaN or an infinity among them; the
// whole group is then NaN).
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits)
{
    const uint32_t b = bits >> 23;
    return b < 7u ? 7u : b;
}
// 64/X
__device__ __forceinline__ float steps_per_one(uint32_t byte) { return __uint_as_float((260u - byte) << 23); }
// X/64 of any byte
__device__ __forceinline__ float step_of(uint32_t byte)
{
    const float low = __uint_as_float(0x00010000u << min(byte, 6u));   // (not a normal number)
    const float v = byte > 6u ? __uint_as_float((byte - 6u) << 23) : low;
    return byte == 255u ? __uint_as_float(0x7FC00000u) : v;
}
// n in the low byte: adding 1.5 * 2^23 rounds to the nearest whole number, ties to even.
constexpr float ROUND = 12582912.0f;
__device__ __forceinline__ uint32_t code_of(float v, float per_one)
{
    return __float_as_uint(fmaxf(fminf(fmaf(v, per_one, ROUND), ROUND + 127.0f), ROUND - 127.0f));
}
__device__ __forceinline__ uint32_t four_codes(float2 a, float2 b)
{
    const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
// Codes 2k and 2k + 1 of a word whose bytes are offset by 128: in the last bits of 2^23.
template <int K>
__device__ __forceinline__ float2 two_values(uint32_t offset, float step)
{
    const float2 v = make_float2(__uint_as_float(__byte_perm(offset, 0x4B000000u, 0x7540 | (2 * K))),
                                 __uint_as_float(__byte_perm(offset, 0x4B000000u, 0x7540 | (2 * K + 1))));
    return mul2(add2(v, both(-8388736.0f)), both(step));
}

// ------------------------------------------------------------------ a thread's elements ----
// E neighbours, one access of 32, 16 or 8 bytes, on whose boundaries the rows are.
template <typename T, int E>
struct Elements {
    static constexpr int BYTES = static_cast<int>(sizeof(T)) * E, WORDS = BYTES / 4;
    union {
        T v[E];
        alignas(BYTES < 16 ? BYTES : 16) uint32_t w[WORDS];
    };
    __device__ Elements() {}
};
template <typename T, int E>
__device__ __forceinline__ void load(Elements<T, E> &q, const T *p)
{
    if constexpr (Elements<T, E>::BYTES == 32)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(q.w[0]), "=r"(q.w[1]), "=r"(q.w[2]), "=r"(q.w[3]), "=r"(q.w[4]), "=r"(q.w[5]), "=r"(q.w[6]), "=r"(q.w[7])
                     : "l"(p)
                     : "memory");
    else if constexpr (Elements<T, E>::BYTES == 16)
        *reinterpret_cast<uint4 *>(q.w) = *reinterpret_cast<const uint4 *>(p);
    else
        *reinterpret_cast<uint2 *>(q.w) = *reinterpret_cast<const uint2 *>(p);
}
template <typename T, int E>
__device__ __forceinline__ void store(T *p, const Elements<T, E> &q)
{
    if constexpr (Elements<T, E>::BYTES == 32)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(q.w[0]), "r"(q.w[1]), "r"(q.w[2]), "r"(q.w[3]),
                     "r"(q.w[4]), "r"(q.w[5]), "r"(q.w[6]), "r"(q.w[7])
                     : "memory");
    else if constexpr (Elements<T, E>::BYTES == 16)
        *reinterpret_cast<uint4 *>(p) = make_uint4(q.w[0], q.w[1], q.w[2], q.w[3]);
    else
        *reinterpret_cast<uint2 *>(p) = make_uint2(q.w[0], q.w[1]);
}
template <typename T, int E>
__device__ __forceinline__ void zero(Elements<T, E> &q)
{
#pragma unroll
    for (int i = 0; i < Elements<T, E>::WORDS; ++i)
        q.w[i] = 0u;
}
template <typename T, int E>
__device__ __forceinline__ void to_pairs(float2 (&f)[E / 2], const Elements<T, E> &q)
{
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
        f[i] = pair_of<T>(&q.v[2 * i]);
}
template <typename T, int E>
__device__ __forceinline__ void store_pairs(T *p, const float2 (&f)[E / 2])
{
    Elements<T, E> q;
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
        put_pair<T>(&q.v[2 * i], f[i]);
    store<T, E>(p, q);
}

template <int E>
struct Codes {
    alignas(E) uint32_t w[E / 4];
};
template <int E>
__device__ __forceinline__ void store(int8_t *p, const Codes<E> &c)
{
    if constexpr (E == 16)
        *reinterpret_cast<uint4 *>(p) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
    else if constexpr (E == 8)
        *reinterpret_cast<uint2 *>(p) = make_uint2(c.w[0], c.w[1]);
    else
        *reinterpret_cast<uint32_t *>(p) = c.w[0];
}
template <int E>
__device__ __forceinline__ Codes<E> load_codes(const int8_t *p)
{
    Codes<E> c;
    if constexpr (E == 16)
        *reinterpret_cast<uint4 *>(c.w) = *reinterpret_cast<const uint4 *>(p);
    else if constexpr (E == 8)
        *reinterpret_cast<uint2 *>(c.w) = *reinterpret_cast<const uint2 *>(p);
    else
        c.w[0] = *reinterpret_cast<const uint32_t *>(p);
    return c;
}
template <int E>
__device__ __forceinline__ void values_of(float2 (&f)[E / 2], const Codes<E> &c, float step)
{
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        const uint32_t offset = c.w[i] ^ 0x80808080u;
        f[2 * i] = two_values<0>(offset, step);
        f[2 * i + 1] = two_values<1>(offset, step);
    }
}

// Codes and scale byte of the thread's elements, the same byte in the lanes of a group.  16-bit elements stay
// in pairs as far as they can: the magnitudes (whole numbers order them) and the cut at 127 steps, which
// in units of X is 127/64, a number of either type (of an fp16 group of subnormal numbers no value comes near it).
template <typename T, int E>
__device__ __forceinline__ Codes<E> keep(Elements<T, E> q, uint32_t &byte)
{
    constexpr int LANES = GROUP / E;
    Codes<E> c;
    if constexpr (sizeof(T) == 2) {
        uint32_t m = q.w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < E / 2; ++i)
            m = __vmaxu2(m, q.w[i] & 0x7FFF7FFFu);
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1)
            m = __vmaxu2(m, __shfl_xor_sync(ALL, m, o));
        const uint16_t top = static_cast<uint16_t>(max(m & 0xFFFFu, m >> 16));
        byte = scale_byte(__float_as_uint(to_f<T>(*reinterpret_cast<const T *>(&top))));
        const float per_one = steps_per_one(byte);
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            const __nv_bfloat162 most = __float2bfloat162_rn(__uint_as_float(byte << 23 | 0x7E0000u));
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                __nv_bfloat162 &v = *reinterpret_cast<__nv_bfloat162 *>(&q.w[i]);
                v = __hmax2(__hmin2(v, most), __hneg2(most));
            }
        } else {
            const __half2 most = __float2half2_rn(__uint_as_float(byte << 23 | 0x7E0000u));
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                __half2 &v = *reinterpret_cast<__half2 *>(&q.w[i]);
                v = __hmax2(__hmin2(v, most), __hneg2(most));
            }
        }
        float2 f[E / 2];
        to_pairs(f, q);
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            f[i] = fma2(f[i], both(per_one), both(ROUND));
#pragma unroll
        for (int i = 0; i < E / 4; ++i)
            c.w[i] = four_codes(f[2 * i], f[2 * i + 1]);
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < E; ++i)
            m = max(m, q.w[i] & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1)
            m = max(m, __shfl_xor_sync(ALL, m, o));
        byte = scale_byte(m);
        const float per_one = steps_per_one(byte);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const auto n = [&](int k) { return __uint_as_float(code_of(q.v[4 * i + k], per_one)); };
            c.w[i] = four_codes(make_float2(n(0), n(1)), make_float2(n(2), n(3)));
        }
    }
    return c;
}

// ------------------------------------------------------------------ where a thread works ----
// Units (threads' elements, or warps' chunks) of the rows in a line, `per_row` of them a row.  A block's first
// unit is divided by products' upper halves (exact while units * per_row < 2^64), and its others are at most
// THREADS past it.
struct Units {
    long long count;
    uint64_t magic;      // floor(2^64 / per_row) + 1 (0: one a row)
    uint32_t magic32;    // floor(2^32 / per_row) + 1
    int per_row;
};
Units units(long long rows, int per_row)
{
    const uint64_t d = static_cast<uint64_t>(per_row);
    return {rows * per_row, per_row == 1 ? 0ull : ~0ull / d + 1, static_cast<uint32_t>((1ull << 32) / d + (d > 1)), per_row};
}
// Unit `nth` of the block's `of`: its row, and where in the row it is.
__device__ __forceinline__ long long row_of(const Units &u, int nth, int of, int &within)
{
    const unsigned long long first = static_cast<unsigned long long>(blockIdx.x) * of;
    const unsigned long long row = u.magic ? __umul64hi(first, u.magic) : first;
    const int x = static_cast<int>(first - row * u.per_row) + nth;
    int more;
    if (u.per_row >= THREADS)
        more = x >= u.per_row;
    else
        more = u.per_row == 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), u.magic32));
    within = x - more * u.per_row;
    return static_cast<long long>(row) + more;
}
__device__ __forceinline__ bool there(const Units &u, int nth, int of) { return static_cast<long long>(blockIdx.x) * of + nth < u.count; }

struct ActArgs {
    Units u;
    int I, groups;            // groups of a half's row
    const void *gu, *da;      // either may be null
    long long ldg, ldd;
    int8_t *codes;            // [M][2I]
    uint8_t *scales;          // [M][2 groups]
    void *act, *dgu;          // [M][I], [M][2I]
};

// ------------------------------------------------------------------ packs ---------------
template <typename T, int E, bool KEEP>
__global__ void __launch_bounds__(THREADS) swiglu_pack_kernel(const ActArgs a)
{
    ptx::follow();
    constexpr int LANES = GROUP / E;
    int p;
    const long long row = row_of(a.u, threadIdx.x, THREADS, p);
    const int c = p * E;
    const bool in = there(a.u, threadIdx.x, THREADS) && c < a.I;
    Elements<T, E> qg, qu;
    if (in) {
        const T *src = static_cast<const T *>(a.gu) + row * a.ldg + c;
        load(qg, src);
        load(qu, src + a.I);
    } else {
        zero(qg);
        zero(qu);
    }
    if constexpr (KEEP) {
        uint32_t bg, bu;
        const Codes<E> cg = keep(qg, bg), cu = keep(qu, bu);
        if (in) {
            int8_t *codes = a.codes + row * 2 * a.I + c;
            store(codes, cg);
            store(codes + a.I, cu);
            if (p % LANES == 0) {
                uint8_t *scales = a.scales + row * 2 * a.groups + p / LANES;
                scales[0] = static_cast<uint8_t>(bg);
                scales[a.groups] = static_cast<uint8_t>(bu);
            }
        }
    }
    if (in) {
        float2 g[E / 2], u[E / 2];
        to_pairs(g, qg);
        to_pairs(u, qu);
#pragma unroll
        for (int k = 0; k < E / 2; ++k)
            g[k] = mul2(mul2(g[k], logistic2<T>(g[k])), u[k]);
        store_pairs<T, E>(static_cast<T *>(a.act) + row * a.I + c, g);
    }
}

template <typename T, int E, bool KEPT>
__global__ void __launch_bounds__(THREADS) swiglu_backward_pack_kernel(const ActArgs a)
{
    ptx::follow();
    constexpr int LANES = GROUP / E;
    int p;
    const long long row = row_of(a.u, threadIdx.x, THREADS, p);
    const int c = p * E;
    if (!there(a.u, threadIdx.x, THREADS) || c >= a.I)
        return;
    float2 g[E / 2], u[E / 2], d[E / 2];
    Elements<T, E> qd;
    load(qd, static_cast<const T *>(a.da) + row * a.ldd + c);
    if constexpr (KEPT) {
        const int8_t *codes = a.codes + row * 2 * a.I + c;
        const uint8_t *scales = a.scales + row * 2 * a.groups + p / LANES;
        const Codes<E> cg = load_codes<E>(codes), cu = load_codes<E>(codes + a.I);
        const uint32_t bg = scales[0], bu = scales[a.groups];
        values_of<E>(g, cg, step_of(bg));
        values_of<E>(u, cu, step_of(bu));
    } else {
        Elements<T, E> qg, qu;
        const T *src = static_cast<const T *>(a.gu) + row * a.ldg + c;
        load(qg, src);
        load(qu, src + a.I);
        to_pairs(g, qg);
        to_pairs(u, qu);
    }
    to_pairs(d, qd);
#pragma unroll
    for (int k = 0; k < E / 2; ++k)
        gradients<T>(d[k], g[k], u[k]);
    T *out = static_cast<T *>(a.dgu) + row * 2 * a.I + c;
    store_pairs<T, E>(out, g);
    store_pairs<T, E>(out + a.I, u);
    if (a.act)
        store_pairs<T, E>(static_cast<T *>(a.act) + row * a.I + c, d);
}

struct KeepArgs {
    Units u;
    int H, groups;
    const void *x;
    long long ldx;
    int8_t *codes;     // [M][H]
    uint8_t *scales;   // [M][groups]
    void *out;         // [M][H]
};

template <typename T, int E>
__global__ void __launch_bounds__(THREADS) checkpoint_pack_kernel(const KeepArgs a)
{
    ptx::follow();
    constexpr int LANES = GROUP / E;
    int p;
    const long long row = row_of(a.u, threadIdx.x, THREADS, p);
    const int c = p * E;
    const bool in = there(a.u, threadIdx.x, THREADS) && c < a.H;
    Elements<T, E> q;
    if (in)
        load(q, static_cast<const T *>(a.x) + row * a.ldx + c);
    else
        zero(q);
    uint32_t byte;
    const Codes<E> codes = keep(q, byte);
    if (in) {
        store(a.codes + row * a.H + c, codes);
        if (p % LANES == 0)
            a.scales[row * a.groups + p / LANES] = static_cast<uint8_t>(byte);
    }
}

template <typename T, int E>
__global__ void __launch_bounds__(THREADS) restore_pack_kernel(const KeepArgs a)
{
    ptx::follow();
    constexpr int LANES = GROUP / E;
    int p;
    const long long row = row_of(a.u, threadIdx.x, THREADS, p);
    const int c = p * E;
    if (!there(a.u, threadIdx.x, THREADS) || c >= a.H)
        return;
    float2 v[E / 2];
    const Codes<E> codes = load_codes<E>(a.codes + row * a.H + c);
    values_of<E>(v, codes, step_of(a.scales[row * a.groups + p / LANES]));
    store_pairs<T, E>(static_cast<T *>(a.out) + row * a.H + c, v);
}

// ------------------------------------------------------------------ element by element ----
// A warp's chunk of a row: lane l has its elements l, 32 + l, ..., so every access of the warp is one group
// of 32 neighbours, at any alignment.  WHOLE: the row has all of the chunk, and nothing is asked of the columns.
struct Chunk {
    long long row;
    int c, first;    // this lane's first column, the chunk's
    int lane;
    bool in;         // there is such a chunk
};
__device__ __forceinline__ Chunk chunk_of(const Units &u)
{
    constexpr int WARPS = THREADS / 32;
    const int warp = threadIdx.x >> 5;
    Chunk k;
    int within;
    k.row = row_of(u, warp, WARPS, within);
    k.lane = threadIdx.x & 31;
    k.first = within * CHUNK;
    k.c = k.first + k.lane;
    k.in = there(u, warp, WARPS);
    return k;
}
// (columns past the end: the last one's value, so that no load waits behind a branch, then zeros)
template <bool WHOLE, typename T>
__device__ __forceinline__ void load_spread(float (&f)[8], const T *row, int c, int n)
{
    T v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = row[WHOLE ? c + 32 * j : min(c + 32 * j, n - 1)];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = WHOLE || c + 32 * j < n ? to_f<T>(v[j]) : 0.0f;
}
template <bool WHOLE, typename T>
__device__ __forceinline__ void store_spread(T *row, const float (&f)[8], int c, int n)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (WHOLE || c + 32 * j < n)
            row[c + 32 * j] = from_f<T>(f[j]);
}
template <bool WHOLE>
__device__ __forceinline__ void keep_spread(const float (&f)[8], int8_t *codes, uint8_t *scales, const Chunk &k, int n)
{
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t byte = scale_byte(__reduce_max_sync(ALL, magnitude(f[j])));
        const uint32_t code = code_of(f[j], steps_per_one(byte));
        if (WHOLE || k.c + 32 * j < n)
            codes[k.c + 32 * j] = static_cast<int8_t>(code & 0xFFu);
        mine = k.lane == j ? byte : mine;
    }
    if (k.lane < 8 && (WHOLE || k.first + 32 * k.lane < n))
        scales[(k.first >> 5) + k.lane] = static_cast<uint8_t>(mine);
}
template <bool WHOLE>
__device__ __forceinline__ void restore_spread(float (&f)[8], const int8_t *codes, const uint8_t *scales, const Chunk &k, int n)
{
    // lane j has the step of group j
    const int group = (k.first >> 5) + (k.lane & 7);
    const uint8_t byte = scales[WHOLE ? group : min(group, groups_of(n) - 1)];
    uint8_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = *(reinterpret_cast<const uint8_t *>(codes) + (WHOLE ? k.c + 32 * j : min(k.c + 32 * j, n - 1)));
    const float step = step_of(byte);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float value = (__uint_as_float(0x4B000000u | (v[j] ^ 0x80u)) - 8388736.0f) * __shfl_sync(ALL, step, j);
        f[j] = WHOLE || k.c + 32 * j < n ? value : 0.0f;
    }
}

template <bool WHOLE, typename T, bool KEEP>
__device__ __forceinline__ void swiglu_chunk(const ActArgs &a, const Chunk &k)
{
    float g[8], u[8];
    const T *src = static_cast<const T *>(a.gu) + k.row * a.ldg;
    load_spread<WHOLE>(g, src, k.c, a.I);
    load_spread<WHOLE>(u, src + a.I, k.c, a.I);
    if constexpr (KEEP) {
        int8_t *codes = a.codes + k.row * 2 * a.I;
        uint8_t *scales = a.scales + k.row * 2 * a.groups;
        keep_spread<WHOLE>(g, codes, scales, k, a.I);
        keep_spread<WHOLE>(u, codes + a.I, scales + a.groups, k, a.I);
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 v = make_float2(g[j], g[j + 1]);
        const float2 r = mul2(mul2(v, logistic2<T>(v)), make_float2(u[j], u[j + 1]));
        g[j] = r.x, g[j + 1] = r.y;
    }
    store_spread<WHOLE>(static_cast<T *>(a.act) + k.row * a.I, g, k.c, a.I);
}
template <typename T, bool KEEP>
__global__ void __launch_bounds__(THREADS) swiglu_kernel(const ActArgs a)
{
    ptx::follow();
    const Chunk k = chunk_of(a.u);
    if (!k.in)
        return;
    if (k.first + CHUNK <= a.I)
        swiglu_chunk<true, T, KEEP>(a, k);
    else
        swiglu_chunk<false, T, KEEP>(a, k);
}

template <bool WHOLE, typename T, bool KEPT>
__device__ __forceinline__ void swiglu_backward_chunk(const ActArgs &a, const Chunk &k)
{
    float g[8], u[8], d[8];
    load_spread<WHOLE>(d, static_cast<const T *>(a.da) + k.row * a.ldd, k.c, a.I);
    if constexpr (KEPT) {
        const int8_t *codes = a.codes + k.row * 2 * a.I;
        const uint8_t *scales = a.scales + k.row * 2 * a.groups;
        restore_spread<WHOLE>(g, codes, scales, k, a.I);
        restore_spread<WHOLE>(u, codes + a.I, scales + a.groups, k, a.I);
    } else {
        const T *src = static_cast<const T *>(a.gu) + k.row * a.ldg;
        load_spread<WHOLE>(g, src, k.c, a.I);
        load_spread<WHOLE>(u, src + a.I, k.c, a.I);
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float2 d2 = make_float2(d[j], d[j + 1]), g2 = make_float2(g[j], g[j + 1]), u2 = make_float2(u[j], u[j + 1]);
        gradients<T>(d2, g2, u2);
        d[j] = d2.x, d[j + 1] = d2.y;
        g[j] = g2.x, g[j + 1] = g2.y;
        u[j] = u2.x, u[j + 1] = u2.y;
    }
    T *out = static_cast<T *>(a.dgu) + k.row * 2 * a.I;
    store_spread<WHOLE>(out, g, k.c, a.I);
    store_spread<WHOLE>(out + a.I, u, k.c, a.I);
    if (a.act)
        store_spread<WHOLE>(static_cast<T *>(a.act) + k.row * a.I, d, k.c, a.I);
}
template <typename T, bool KEPT>
__global__ void __launch_bounds__(THREADS) swiglu_backward_kernel(const ActArgs a)
{
    ptx::follow();
    const Chunk k = chunk_of(a.u);
    if (!k.in)
        return;
    if (k.first + CHUNK <= a.I)
        swiglu_backward_chunk<true, T, KEPT>(a, k);
    else
        swiglu_backward_chunk<false, T, KEPT>(a, k);
}

template <typename T>
__global__ void __launch_bounds__(THREADS) checkpoint_kernel(const KeepArgs a)
{
    ptx::follow();
    const Chunk k = chunk_of(a.u);
    if (!k.in)
        return;
    const auto go = [&](auto whole) {
        float v[8];
        load_spread<decltype(whole)::value>(v, static_cast<const T *>(a.x) + k.row * a.ldx, k.c, a.H);
        keep_spread<decltype(whole)::value>(v, a.codes + k.row * a.H, a.scales + k.row * a.groups, k, a.H);
    };
    if (k.first + CHUNK <= a.H)
        go(std::true_type());
    else
        go(std::false_type());
}

template <typename T>
__global__ void __launch_bounds__(THREADS) restore_kernel(const KeepArgs a)
{
    ptx::follow();
    const Chunk k = chunk_of(a.u);
    if (!k.in)
        return;
    const auto go = [&](auto whole) {
        float v[8];
        restore_spread<decltype(whole)::value>(v, a.codes + k.row * a.H, a.scales + k.row * a.groups, k, a.H);
        store_spread<decltype(whole)::value>(static_cast<T *>(a.out) + k.row * a.H, v, k.c, a.H);
    };
    if (k.first + CHUNK <= a.H)
        go(std::true_type());
    else
        go(std::false_type());
}

// ------------------------------------------------------------------ host side ------------
constexpr int MAX_WIDTH = 1 << 20;

bool sizes_ok(long long M, int width, int dtype) { return M >= 0 && M <= MAX_ROWS && width >= 1 && width <= MAX_WIDTH && dtype_ok(dtype); }
// How rows move: element by element (0), or the elements of a thread, for which every tensor (null: not there)
// starts, row by row, on their boundaries.
struct Rows {
    const void *p;
    long long ld;   // elements
    size_t size;    // of an element
};
int elements_of(int width, int dtype, std::initializer_list<Rows> tensors)
{
    const auto fits = [&](int e) {
        if (width % e != 0)
            return false;
        for (const Rows &r : tensors)
            if (r.p && (!op_aligned(r.p, e * r.size) || r.ld % e != 0))
                return false;
        return true;
    };
    if (dtype != MOE_F32 && fits(16))
        return 16;
    return fits(8) ? 8 : fits(4) ? 4 : 0;
}
// E: the elements of a thread, the last group's included where it is not whole; chunks of warps if 0.
Units units_of(long long M, int width, int e)
{
    return e ? units(M, GROUP / e * groups_of(width)) : units(M, (width + CHUNK - 1) / CHUNK);
}
// Blocks of THREADS threads, or -1: more than a grid has (2^39 threads, which no memory holds).
long long blocks_of(const Units &u, int e)
{
    const long long b = ((e ? u.count : 32 * u.count) + THREADS - 1) / THREADS;
    return b <= INT_MAX ? b : -1;
}
// Calls f with a null pointer of the element type and the elements of a thread.
template <typename F>
void with_elements(int dtype, int e, F f)
{
    with_dtype(dtype, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        if constexpr (sizeof(T) == 2) {
            if (e == 16)
                return f(t, std::integral_constant<int, 16>());
        }
        if (e == 8)
            return f(t, std::integral_constant<int, 8>());
        e ? f(t, std::integral_constant<int, 4>()) : f(t, std::integral_constant<int, 0>());
    });
}

}  // namespace

extern "C" {

int moe_swiglu(int64_t M, int I, const void *gu, int64_t ldg, int dtype, void *act, int8_t *codes, uint8_t *scales, void *stream)
{
    if (!sizes_ok(M, I, dtype) || ldg < 2ll * I || !codes != !scales)
        return MOE_ERR_INVALID_ARG;
    if (M == 0)
        return MOE_OK;
    const size_t b = dtype_bytes(dtype);
    if (!gu || !act || !op_aligned(gu, b) || !op_aligned(act, b))
        return MOE_ERR_INVALID_ARG;
    const int e = elements_of(I, dtype, {{gu, ldg, b}, {act, I, b}, {codes, 2ll * I, 1}});
    ActArgs a{};
    a.u = units_of(M, I, e);
    const long long blocks = blocks_of(a.u, e);
    if (blocks < 0)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    a.I = I;
    a.groups = groups_of(I);
    a.gu = gu;
    a.ldg = ldg;
    a.codes = codes;
    a.scales = scales;
    a.act = act;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int grid = static_cast<int>(blocks);
    with_elements(dtype, e, [&](auto *t, auto elements) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int E = decltype(elements)::value;
        if constexpr (E > 0)
            codes ? launch_programmatic(swiglu_pack_kernel<T, E, true>, grid, THREADS, 0, s, a) : launch_programmatic(swiglu_pack_kernel<T, E, false>, grid, THREADS, 0, s, a);
        else
            codes ? launch_programmatic(swiglu_kernel<T, true>, grid, THREADS, 0, s, a) : launch_programmatic(swiglu_kernel<T, false>, grid, THREADS, 0, s, a);
    });
    return launched();
}

int moe_swiglu_backward(int64_t M, int I, const void *dact, int64_t ldd, const void *gu, int64_t ldg, const int8_t *codes,
                        const uint8_t *scales, int dtype, void *dgu, void *act, void *stream)
{
    if (!sizes_ok(M, I, dtype) || ldd < I || (gu && ldg < 2ll * I) || !codes != !scales)
        return MOE_ERR_INVALID_ARG;
    if (M == 0)
        return MOE_OK;
    const size_t b = dtype_bytes(dtype);
    if (!dact || !dgu || !gu == !codes || !op_aligned(dact, b) || !op_aligned(gu, b) || !op_aligned(dgu, b) || !op_aligned(act, b))
        return MOE_ERR_INVALID_ARG;
    const int e = elements_of(I, dtype, {{dact, ldd, b}, {gu, ldg, b}, {dgu, 2ll * I, b}, {act, I, b}, {codes, 2ll * I, 1}});
    ActArgs a{};
    a.u = units_of(M, I, e);
    const long long blocks = blocks_of(a.u, e);
    if (blocks < 0)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    a.I = I;
    a.groups = groups_of(I);
    a.gu = gu;
    a.ldg = ldg;
    a.da = dact;
    a.ldd = ldd;
    a.codes = const_cast<int8_t *>(codes);
    a.scales = const_cast<uint8_t *>(scales);
    a.act = act;
    a.dgu = dgu;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int grid = static_cast<int>(blocks);
    with_elements(dtype, e, [&](auto *t, auto elements) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int E = decltype(elements)::value;
        if constexpr (E > 0)
            codes ? launch_programmatic(swiglu_backward_pack_kernel<T, E, true>, grid, THREADS, 0, s, a)
                  : launch_programmatic(swiglu_backward_pack_kernel<T, E, false>, grid, THREADS, 0, s, a);
        else
            codes ? launch_programmatic(swiglu_backward_kernel<T, true>, grid, THREADS, 0, s, a) : launch_programmatic(swiglu_backward_kernel<T, false>, grid, THREADS, 0, s, a);
    });
    return launched();
}

int moe_checkpoint_rows(int64_t M, int H, const void *x, int64_t ldx, int dtype, int8_t *codes, uint8_t *scales, void *stream)
{
    if (!sizes_ok(M, H, dtype) || ldx < H)
        return MOE_ERR_INVALID_ARG;
    if (M == 0)
        return MOE_OK;
    if (!x || !codes || !scales || !op_aligned(x, dtype_bytes(dtype)))
        return MOE_ERR_INVALID_ARG;
    const int e = elements_of(H, dtype, {{x, ldx, dtype_bytes(dtype)}, {codes, H, 1}});
    const Units u = units_of(M, H, e);
    const long long blocks = blocks_of(u, e);
    if (blocks < 0)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const KeepArgs a{u, H, groups_of(H), x, ldx, codes, scales, nullptr};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int grid = static_cast<int>(blocks);
    with_elements(dtype, e, [&](auto *t, auto elements) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int E = decltype(elements)::value;
        if constexpr (E > 0)
            launch_programmatic(checkpoint_pack_kernel<T, E>, grid, THREADS, 0, s, a);
        else
            launch_programmatic(checkpoint_kernel<T>, grid, THREADS, 0, s, a);
    });
    return launched();
}

int moe_restore_rows(int64_t M, int H, const int8_t *codes, const uint8_t *scales, int dtype, void *x, void *stream)
{
    if (!sizes_ok(M, H, dtype))
        return MOE_ERR_INVALID_ARG;
    if (M == 0)
        return MOE_OK;
    if (!x || !codes || !scales || !op_aligned(x, dtype_bytes(dtype)))
        return MOE_ERR_INVALID_ARG;
    const int e = elements_of(H, dtype, {{x, H, dtype_bytes(dtype)}, {codes, H, 1}});
    const Units u = units_of(M, H, e);
    const long long blocks = blocks_of(u, e);
    if (blocks < 0)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const KeepArgs a{u, H, groups_of(H), nullptr, 0, const_cast<int8_t *>(codes), const_cast<uint8_t *>(scales), x};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int grid = static_cast<int>(blocks);
    with_elements(dtype, e, [&](auto *t, auto elements) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int E = decltype(elements)::value;
        if constexpr (E > 0)
            launch_programmatic(restore_pack_kernel<T, E>, grid, THREADS, 0, s, a);
        else
            launch_programmatic(restore_kernel<T>, grid, THREADS, 0, s, a);
    });
    return launched();
}

}  // extern "C"
