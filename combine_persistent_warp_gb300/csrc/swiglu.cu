// swiglu.cu -- the experts' activation over rows of gate and up, its gradient, and rows kept in 8 bits
// between the forward and the backward pass.
//
//   s = 1/(1 + exp(-g)):  act = g s u,  dg = da u (s + g s (1 - s)),  du = da g s
//   8 bits: 32 neighbours of a row share X = 2^floor(log2 max|v|) (a byte, its exponent + 127, at least
//   7), and each is n X/64 with the nearest whole n in -127 .. 127, ties to even (an MX block of INT8
//   elements).  X is a power of two, so v 64/X and n X/64 are exact and the rounding to n is the only one.
//
// All of it is elementwise and bound by HBM.  A thread takes a pack of 8 neighbours of gate and of up, so
// four neighbouring lanes hold a group of 32; rows that are not whole packs on 16-byte boundaries go
// element by element, a group a warp access.
#include <climits>
#include <type_traits>

#include "op_common.cuh"

using namespace cpw;

namespace {

constexpr int THREADS = 256;
constexpr int GROUP = 32;       // values of a scale
constexpr int CHUNK = 256;      // elements of a warp (8 a lane)
constexpr uint32_t ALL = 0xFFFFFFFFu;

// ------------------------------------------------------------------ the activation ------
// 1/(1 + exp(-g)).  For 16-bit results two approximate instructions, together 2^-21 off at |g| <= 16 (the
// exponent's rounding grows with |g|), below 2^-126 zero; for fp32 the exact functions.
template <typename T>
__device__ __forceinline__ float logistic(float g)
{
    if constexpr (std::is_same_v<T, float>) {
        return 1.0f / (1.0f + expf(-g));
    } else {
        float e, s;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
        return s;
    }
}
struct Grads {
    float dg, du, act;
};
template <typename T>
__device__ __forceinline__ Grads gradients(float da, float g, float u)
{
    const float s = logistic<T>(g), t = g * s, du = da * t;
    // s + t (1 - s)
    return {da * u * fmaf(t, 1.0f - s, s), du, t * u};
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
    if (byte == 255u)
        return __uint_as_float(0x7FC00000u);
    return __uint_as_float(byte > 6u ? (byte - 6u) << 23 : 1u << (byte + 16u));
}
// n in the low byte: adding 1.5 * 2^23 rounds to the nearest whole number, ties to even.
__device__ __forceinline__ uint32_t code_of(float v, float per_one)
{
    constexpr float BIG = 12582912.0f;
    return __float_as_uint(fmaxf(fminf(fmaf(v, per_one, BIG), BIG + 127.0f), BIG - 127.0f));
}
__device__ __forceinline__ uint32_t four_codes(const float *v, float per_one)
{
    const uint32_t lo = __byte_perm(code_of(v[0], per_one), code_of(v[1], per_one), 0x0040);
    const uint32_t hi = __byte_perm(code_of(v[2], per_one), code_of(v[3], per_one), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
// Code k of a word: its byte, offset by 128, in the last bits of 2^23.
template <int K>
__device__ __forceinline__ float value_of(uint32_t offset, float step)
{
    return (__uint_as_float(__byte_perm(offset, 0x4B000000u, 0x7540 | K)) - 8388736.0f) * step;
}
__device__ __forceinline__ void eight_values(float (&v)[8], uint2 codes, float step)
{
    const uint32_t lo = codes.x ^ 0x80808080u, hi = codes.y ^ 0x80808080u;
    v[0] = value_of<0>(lo, step);
    v[1] = value_of<1>(lo, step);
    v[2] = value_of<2>(lo, step);
    v[3] = value_of<3>(lo, step);
    v[4] = value_of<0>(hi, step);
    v[5] = value_of<1>(hi, step);
    v[6] = value_of<2>(hi, step);
    v[7] = value_of<3>(hi, step);
}

// A thread's eight elements, packed: the group's four lanes agree on its byte; its codes.
__device__ __forceinline__ uint2 keep_pack(const float (&v)[8], uint32_t &byte)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, magnitude(v[i]));
    m = max(m, __shfl_xor_sync(ALL, m, 1));
    m = max(m, __shfl_xor_sync(ALL, m, 2));
    byte = scale_byte(m);
    const float per_one = steps_per_one(byte);
    return make_uint2(four_codes(v, per_one), four_codes(v + 4, per_one));
}

template <typename T>
__device__ __forceinline__ void unpack8(float (&f)[8], const Pack<T, 8> &q)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = to_f<T>(q.v[i]);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8])
{
    Pack<T, 8> q;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q.v[i] = from_f<T>(f[i]);
    store_pack<T, 8>(p, q);
}

// ------------------------------------------------------------------ where a thread works ----
// Units (packs, or warps' chunks) of the rows in a line, `per_row` of them a row: a row's index is a
// product's upper half (magic = floor(2^64 / per_row) + 1, exact while units * per_row < 2^64).
struct Units {
    long long count;
    uint64_t magic;
    int per_row;
};
Units units(long long rows, int per_row)
{
    return {rows * per_row, per_row == 1 ? 0ull : ~0ull / static_cast<uint64_t>(per_row) + 1, per_row};
}
__device__ __forceinline__ long long row_of(const Units &u, long long i, int &within)
{
    const long long row = u.magic ? static_cast<long long>(__umul64hi(static_cast<uint64_t>(i), u.magic)) : i;
    within = static_cast<int>(i - row * u.per_row);
    return row;
}

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
template <typename T, bool KEEP>
__global__ void __launch_bounds__(THREADS) swiglu_pack_kernel(const ActArgs a)
{
    const long long i = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
    int p;
    const long long row = row_of(a.u, i, p);
    const int c = p * 8;
    const bool in = i < a.u.count && c < a.I;
    float g[8], u[8];
    if (in) {
        const T *src = static_cast<const T *>(a.gu) + row * a.ldg + c;
        const Pack<T, 8> qg = load_pack<T, 8>(src), qu = load_pack<T, 8>(src + a.I);
        unpack8(g, qg);
        unpack8(u, qu);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            g[k] = u[k] = 0.0f;
    }
    if constexpr (KEEP) {
        uint32_t bg, bu;
        const uint2 cg = keep_pack(g, bg), cu = keep_pack(u, bu);
        if (in) {
            int8_t *codes = a.codes + row * 2 * a.I + c;
            *reinterpret_cast<uint2 *>(codes) = cg;
            *reinterpret_cast<uint2 *>(codes + a.I) = cu;
            if ((p & 3) == 0) {
                uint8_t *scales = a.scales + row * 2 * a.groups + (p >> 2);
                scales[0] = static_cast<uint8_t>(bg);
                scales[a.groups] = static_cast<uint8_t>(bu);
            }
        }
    }
    if (in) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            g[k] = g[k] * logistic<T>(g[k]) * u[k];
        store8(static_cast<T *>(a.act) + row * a.I + c, g);
    }
}

template <typename T, bool KEPT>
__global__ void __launch_bounds__(THREADS) swiglu_backward_pack_kernel(const ActArgs a)
{
    const long long i = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
    int p;
    const long long row = row_of(a.u, i, p);
    const int c = p * 8;
    if (i >= a.u.count || c >= a.I)
        return;
    float g[8], u[8], d[8];
    const Pack<T, 8> qd = load_pack<T, 8>(static_cast<const T *>(a.da) + row * a.ldd + c);
    if constexpr (KEPT) {
        const int8_t *codes = a.codes + row * 2 * a.I + c;
        const uint8_t *scales = a.scales + row * 2 * a.groups + (p >> 2);
        const uint2 cg = __ldg(reinterpret_cast<const uint2 *>(codes)), cu = __ldg(reinterpret_cast<const uint2 *>(codes + a.I));
        const uint32_t bg = __ldg(scales), bu = __ldg(scales + a.groups);
        eight_values(g, cg, step_of(bg));
        eight_values(u, cu, step_of(bu));
    } else {
        const T *src = static_cast<const T *>(a.gu) + row * a.ldg + c;
        const Pack<T, 8> qg = load_pack<T, 8>(src), qu = load_pack<T, 8>(src + a.I);
        unpack8(g, qg);
        unpack8(u, qu);
    }
    unpack8(d, qd);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const Grads r = gradients<T>(d[k], g[k], u[k]);
        g[k] = r.dg;
        u[k] = r.du;
        d[k] = r.act;
    }
    T *out = static_cast<T *>(a.dgu) + row * 2 * a.I + c;
    store8(out, g);
    store8(out + a.I, u);
    if (a.act)
        store8(static_cast<T *>(a.act) + row * a.I + c, d);
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

template <typename T>
__global__ void __launch_bounds__(THREADS) checkpoint_pack_kernel(const KeepArgs a)
{
    const long long i = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
    int p;
    const long long row = row_of(a.u, i, p);
    const int c = p * 8;
    const bool in = i < a.u.count && c < a.H;
    float v[8];
    if (in) {
        unpack8(v, load_pack<T, 8>(static_cast<const T *>(a.x) + row * a.ldx + c));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = 0.0f;
    }
    uint32_t byte;
    const uint2 codes = keep_pack(v, byte);
    if (in) {
        *reinterpret_cast<uint2 *>(a.codes + row * a.H + c) = codes;
        if ((p & 3) == 0)
            a.scales[row * a.groups + (p >> 2)] = static_cast<uint8_t>(byte);
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS) restore_pack_kernel(const KeepArgs a)
{
    const long long i = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
    int p;
    const long long row = row_of(a.u, i, p);
    const int c = p * 8;
    if (i >= a.u.count || c >= a.H)
        return;
    float v[8];
    const uint2 codes = __ldg(reinterpret_cast<const uint2 *>(a.codes + row * a.H + c));
    eight_values(v, codes, step_of(__ldg(a.scales + row * a.groups + (p >> 2))));
    store8(static_cast<T *>(a.out) + row * a.H + c, v);
}

// ------------------------------------------------------------------ element by element ----
// A warp's chunk of a row: lane l has its elements l, 32 + l, ..., so every access of the warp is one group
// of 32 neighbours, at any alignment.
struct Chunk {
    long long row;
    int c, first;    // this lane's first column, the chunk's
    int lane;
    bool in;         // there is such a chunk
};
__device__ __forceinline__ Chunk chunk_of(const Units &u)
{
    const long long w = (static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x) >> 5;
    Chunk k;
    int within;
    k.row = row_of(u, w, within);
    k.lane = threadIdx.x & 31;
    k.first = within * CHUNK;
    k.c = k.first + k.lane;
    k.in = w < u.count;
    return k;
}
template <typename T>
__device__ __forceinline__ void load_spread(float (&f)[8], const T *row, int c, int n)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = c + 32 * j < n ? to_f<T>(__ldg(row + c + 32 * j)) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store_spread(T *row, const float (&f)[8], int c, int n)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + 32 * j < n)
            row[c + 32 * j] = from_f<T>(f[j]);
}
__device__ __forceinline__ void keep_spread(const float (&f)[8], int8_t *codes, uint8_t *scales, const Chunk &k, int n)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (k.first + 32 * j >= n)
            break;
        const uint32_t byte = scale_byte(__reduce_max_sync(ALL, magnitude(f[j])));
        if (k.c + 32 * j < n)
            codes[k.c + 32 * j] = static_cast<int8_t>(code_of(f[j], steps_per_one(byte)) & 0xFFu);
        if (k.lane == 0)
            scales[(k.first >> 5) + j] = static_cast<uint8_t>(byte);
    }
}
__device__ __forceinline__ void restore_spread(float (&f)[8], const int8_t *codes, const uint8_t *scales, const Chunk &k, int n)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = k.c + 32 * j < n ? static_cast<float>(__ldg(codes + k.c + 32 * j)) * step_of(__ldg(scales + (k.first >> 5) + j)) : 0.0f;
}

template <typename T, bool KEEP>
__global__ void __launch_bounds__(THREADS) swiglu_kernel(const ActArgs a)
{
    const Chunk k = chunk_of(a.u);
    if (!k.in)
        return;
    float g[8], u[8];
    const T *src = static_cast<const T *>(a.gu) + k.row * a.ldg;
    load_spread(g, src, k.c, a.I);
    load_spread(u, src + a.I, k.c, a.I);
    if constexpr (KEEP) {
        int8_t *codes = a.codes + k.row * 2 * a.I;
        uint8_t *scales = a.scales + k.row * 2 * a.groups;
        keep_spread(g, codes, scales, k, a.I);
        keep_spread(u, codes + a.I, scales + a.groups, k, a.I);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        g[j] = g[j] * logistic<T>(g[j]) * u[j];
    store_spread(static_cast<T *>(a.act) + k.row * a.I, g, k.c, a.I);
}

template <typename T, bool KEPT>
__global__ void __launch_bounds__(THREADS) swiglu_backward_kernel(const ActArgs a)
{
    const Chunk k = chunk_of(a.u);
    if (!k.in)
        return;
    float g[8], u[8], d[8];
    load_spread(d, static_cast<const T *>(a.da) + k.row * a.ldd, k.c, a.I);
    if constexpr (KEPT) {
        const int8_t *codes = a.codes + k.row * 2 * a.I;
        const uint8_t *scales = a.scales + k.row * 2 * a.groups;
        restore_spread(g, codes, scales, k, a.I);
        restore_spread(u, codes + a.I, scales + a.groups, k, a.I);
    } else {
        const T *src = static_cast<const T *>(a.gu) + k.row * a.ldg;
        load_spread(g, src, k.c, a.I);
        load_spread(u, src + a.I, k.c, a.I);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const Grads r = gradients<T>(d[j], g[j], u[j]);
        g[j] = r.dg;
        u[j] = r.du;
        d[j] = r.act;
    }
    T *out = static_cast<T *>(a.dgu) + k.row * 2 * a.I;
    store_spread(out, g, k.c, a.I);
    store_spread(out + a.I, u, k.c, a.I);
    if (a.act)
        store_spread(static_cast<T *>(a.act) + k.row * a.I, d, k.c, a.I);
}

template <typename T>
__global__ void __launch_bounds__(THREADS) checkpoint_kernel(const KeepArgs a)
{
    const Chunk k = chunk_of(a.u);
    if (!k.in)
        return;
    float v[8];
    load_spread(v, static_cast<const T *>(a.x) + k.row * a.ldx, k.c, a.H);
    keep_spread(v, a.codes + k.row * a.H, a.scales + k.row * a.groups, k, a.H);
}

template <typename T>
__global__ void __launch_bounds__(THREADS) restore_kernel(const KeepArgs a)
{
    const Chunk k = chunk_of(a.u);
    if (!k.in)
        return;
    float v[8];
    restore_spread(v, a.codes + k.row * a.H, a.scales + k.row * a.groups, k, a.H);
    store_spread(static_cast<T *>(a.out) + k.row * a.H, v, k.c, a.H);
}

// ------------------------------------------------------------------ host side ------------
constexpr int MAX_WIDTH = 1 << 20;

int groups_of(int width) { return (width + GROUP - 1) / GROUP; }
bool sizes_ok(long long M, int width, int dtype) { return M >= 0 && M <= MAX_ROWS && width >= 1 && width <= MAX_WIDTH && dtype_ok(dtype); }
// Rows of whole packs on 16-byte boundaries (null: not there).
bool packed(const void *p, long long ld, int dtype) { return op_aligned(p, 16) && (p == nullptr || ld * dtype_bytes(dtype) % 16 == 0); }

// Blocks of THREADS threads, or -1: more than a grid has (2^39 threads, which no memory holds).
long long blocks_of(long long threads)
{
    const long long b = (threads + THREADS - 1) / THREADS;
    return b <= INT_MAX ? b : -1;
}
// Packs: four lanes a group, the last group's included where it is not whole.
Units pack_units(long long M, int width) { return units(M, 4 * groups_of(width)); }
Units chunk_units(long long M, int width) { return units(M, (width + CHUNK - 1) / CHUNK); }

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
    const bool packs = I % 8 == 0 && packed(gu, ldg, dtype) && packed(act, I, dtype) && op_aligned(codes, 8);
    ActArgs a{};
    a.u = packs ? pack_units(M, I) : chunk_units(M, I);
    const long long blocks = blocks_of(packs ? a.u.count : 32 * a.u.count);
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
    const dim3 grid(static_cast<unsigned>(blocks));
    with_dtype(dtype, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        if (packs && codes)
            swiglu_pack_kernel<T, true><<<grid, THREADS, 0, s>>>(a);
        else if (packs)
            swiglu_pack_kernel<T, false><<<grid, THREADS, 0, s>>>(a);
        else if (codes)
            swiglu_kernel<T, true><<<grid, THREADS, 0, s>>>(a);
        else
            swiglu_kernel<T, false><<<grid, THREADS, 0, s>>>(a);
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
    const bool packs = I % 8 == 0 && packed(dact, ldd, dtype) && packed(gu, ldg, dtype) && packed(dgu, 2ll * I, dtype) &&
                       packed(act, I, dtype) && op_aligned(codes, 8);
    ActArgs a{};
    a.u = packs ? pack_units(M, I) : chunk_units(M, I);
    const long long blocks = blocks_of(packs ? a.u.count : 32 * a.u.count);
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
    const dim3 grid(static_cast<unsigned>(blocks));
    with_dtype(dtype, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        if (packs && codes)
            swiglu_backward_pack_kernel<T, true><<<grid, THREADS, 0, s>>>(a);
        else if (packs)
            swiglu_backward_pack_kernel<T, false><<<grid, THREADS, 0, s>>>(a);
        else if (codes)
            swiglu_backward_kernel<T, true><<<grid, THREADS, 0, s>>>(a);
        else
            swiglu_backward_kernel<T, false><<<grid, THREADS, 0, s>>>(a);
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
    const bool packs = H % 8 == 0 && packed(x, ldx, dtype) && op_aligned(codes, 8);
    const Units u = packs ? pack_units(M, H) : chunk_units(M, H);
    const long long blocks = blocks_of(packs ? u.count : 32 * u.count);
    if (blocks < 0)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const KeepArgs a{u, H, groups_of(H), x, ldx, codes, scales, nullptr};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(blocks));
    with_dtype(dtype, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        if (packs)
            checkpoint_pack_kernel<T><<<grid, THREADS, 0, s>>>(a);
        else
            checkpoint_kernel<T><<<grid, THREADS, 0, s>>>(a);
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
    const bool packs = H % 8 == 0 && packed(x, H, dtype) && op_aligned(codes, 8);
    const Units u = packs ? pack_units(M, H) : chunk_units(M, H);
    const long long blocks = blocks_of(packs ? u.count : 32 * u.count);
    if (blocks < 0)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const KeepArgs a{u, H, groups_of(H), nullptr, 0, const_cast<int8_t *>(codes), const_cast<uint8_t *>(scales), x};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(blocks));
    with_dtype(dtype, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        if (packs)
            restore_pack_kernel<T><<<grid, THREADS, 0, s>>>(a);
        else
            restore_kernel<T><<<grid, THREADS, 0, s>>>(a);
    });
    return launched();
}

}  // extern "C"
