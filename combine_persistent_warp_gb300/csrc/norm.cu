// norm.cu -- layer norm over the hidden dimension: forward, the FP8 form that the expert layer
// reads, and backward with the sums of the weight's and the bias's gradients.
//
//   mean = sum(x)/H, rstd = 1/sqrt(sum((x-mean)^2)/H + eps), xh = (x-mean)*rstd, y = xh*g + b
//   a = dy*g:  dx = rstd*(a - mean(a) - xh*mean(a*xh)),  dg = sum_t dy*xh,  db = sum_t dy
//
// All of it is bound by HBM: a row is read once into registers, where both passes of the
// statistics run (the centred second pass keeps the variance free of cancellation), and every
// statistic and sum is held in fp32.
//
// Measured on a GB300, bf16: 16384 x 4096 forward 45 us, backward 72 us (HBM floors 40 and 60 us
// at the measured copy bandwidth), FP8 form 48 us (floor 30: its group maxima and conversions
// take issue slots); 128 x 7168 FP8 form 2.9 us in a graph; 4099 x 1001 fp32 9 and 13 us; 8939 x 2895
// fp16, rows off 16-byte boundaries, 29 and 45 (2896: 20 and 39; floors 16 and 23).  fp32: 16384 x 4096
// 90 and 153 us (floors 80 and 121).  Over 8192 columns the backward pass holds more than its registers
// and spills 320 to 700 bytes a thread: 4096 x 12288 bf16 44 and 103 us (floors 30 and 45), off the
// boundaries (12287) 92 and 352; 4096 x 16384 fp32 140 and 221 (80 and 121).
//
// Long batches run in persistent blocks that keep the next rows on their way: every thread
// copies the packs of the rows ahead that it will itself use into its own slots of shared memory
// (cp.async), so the copies need no barrier, and a block waits only for the sums of a row.
#include <type_traits>

#include "moe_internal.cuh"
#include "op_common.cuh"
#include "ptx.cuh"

using namespace cpw;

namespace {

constexpr int MAX_H = 16384;   // as moe_create: a row fits one block's registers

// ------------------------------------------------------------------ elements in pairs ----
// Two fp32 values an instruction: these kernels would otherwise be bound by issue, not by HBM.
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
    return reinterpret_cast<float2 &>(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)));
    return reinterpret_cast<float2 &>(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(reinterpret_cast<unsigned long long &>(a)), "l"(reinterpret_cast<unsigned long long &>(b)),
          "l"(reinterpret_cast<unsigned long long &>(c)));
    return reinterpret_cast<float2 &>(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// ------------------------------------------------------------------ a thread's part of a row ----
// VPT packs of V elements (V = 8: 16-byte accesses; V = 1: any alignment), pack j at position
// t + j * step of the row for thread t of the `step` threads that share it; held as pairs.
template <int V, int VPT>
constexpr int PAIRS = V * VPT / 2;

template <typename T>
__device__ __forceinline__ float2 pair_of(const T *q)
{
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const uint32_t u = *reinterpret_cast<const uint32_t *>(q);
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    } else {
        return make_float2(to_f<T>(q[0]), to_f<T>(q[1]));
    }
}

template <typename T, int V, int VPT>
__device__ __forceinline__ void unpack(float2 (&f)[PAIRS<V, VPT>], const Pack<T, V> (&q)[VPT])
{
#pragma unroll
    for (int i = 0; i < PAIRS<V, VPT>; ++i) {
        if constexpr (V == 1)
            f[i] = make_float2(to_f<T>(q[2 * i].v[0]), to_f<T>(q[2 * i + 1].v[0]));
        else
            f[i] = pair_of<T>(&q[2 * i / V].v[2 * i % V]);
    }
}

// LEAD: rows that start `lead` elements past a 16-byte boundary.  Pack p holds elements p * V - lead ...
// of the row, so that packs are aligned; the first and the last may hold bytes of the neighbouring rows
// (clip() drops them, put() leaves them alone).
template <int V, bool LEAD>
__device__ __forceinline__ int packs_of(int H, int lead)
{
    return LEAD ? (lead + H + V - 1) / V : H / V;
}

// Packs past the row's end are zeros.
template <typename T, int V, int VPT>
__device__ __forceinline__ void fetch(Pack<T, V> (&q)[VPT], const T *row, int t, int step, int packs)
{
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int p = t + j * step;
        if (p < packs) {
            q[j] = load_pack<T, V>(row + static_cast<size_t>(p) * V);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                q[j].v[i] = from_f<T>(0.0f);
        }
    }
}

template <typename T, int V, int VPT, bool LEAD = false>
__device__ __forceinline__ void put(T *row, const float2 (&f)[PAIRS<V, VPT>], int t, int step, int packs, int lead = 0, int H = 0)
{
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int p = t + j * step, e = p * V - lead;
        if (p < packs) {
            Pack<T, V> q;
            if constexpr (V == 1) {
                q.v[0] = from_f<T>((j & 1) ? f[j / 2].y : f[j / 2].x);
            } else {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float2 u = f[j * (V / 2) + i];
                    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                        *reinterpret_cast<__nv_bfloat162 *>(&q.v[2 * i]) = __float22bfloat162_rn(u);
                    } else {
                        q.v[2 * i] = from_f<T>(u.x);
                        q.v[2 * i + 1] = from_f<T>(u.y);
                    }
                }
            }
            if (!LEAD || (e >= 0 && e + V <= H)) {
                store_pack<T, V>(row + e, q);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e + i >= 0 && e + i < H)
                        row[e + i] = q.v[i];
            }
        }
    }
}
// One of the thread's packs lies partly outside the row.
template <int V, int VPT>
__device__ __forceinline__ bool cut_packs(int t, int step, int lead, int H)
{
    bool cut = false;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int e = (t + j * step) * V - lead;
        cut = cut || (e < 0 && e + V > 0) || (e < H && e + V > H);
    }
    return cut;
}
// Zeroes the pairs (or halves of pairs) past the row's end and, in threads with cut packs, outside the row:
// those are in two warps of a row, and the others step over it.
template <int V, int VPT>
__device__ __forceinline__ void clip(float2 (&f)[PAIRS<V, VPT>], int t, int step, int packs, bool cut = false, int lead = 0, int H = 0)
{
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const bool in = t + j * step < packs;
        if constexpr (V == 1) {
            if (j & 1)
                f[j / 2].y = in ? f[j / 2].y : 0.0f;
            else
                f[j / 2].x = in ? f[j / 2].x : 0.0f;
        } else if (!in) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                f[j * (V / 2) + i] = both(0.0f);
        }
    }
    if (V > 1 && cut) {
#pragma unroll
        for (int i = 0; i < PAIRS<V, VPT>; ++i) {
            const int c = (t + 2 * i / V * step) * V - lead + 2 * i % V;
            f[i] = make_float2(c >= 0 && c < H ? f[i].x : 0.0f, c + 1 >= 0 && c + 1 < H ? f[i].y : 0.0f);
        }
    }
}

// A weight's or bias's columns (`none` where there is no such vector).
template <typename W, int V, int VPT, bool LEAD>
__device__ __forceinline__ void fetch_columns(float2 (&f)[PAIRS<V, VPT>], const W *p, int t, int step, int packs, int lead, int H)
{
    Pack<W, V> q[VPT];
    if constexpr (LEAD) {
        // of any alignment: 16 bytes are shifted out of two aligned vectors, all of them asked for before
        // the first is waited for; where those would leave the vector, element by element
        constexpr int N = VEC<W>, M = V / N;
        Halves h[VPT * M];
#pragma unroll
        for (int j = 0; j < VPT * M; ++j) {
            const int c = (t + j / M * step) * V - lead + j % M * N;
            h[j] = load_halves(p + c, c >= N - 1 && c + 2 * N <= H);
        }
#pragma unroll
        for (int j = 0; j < VPT * M; ++j) {
            const int c = (t + j / M * step) * V - lead + j % M * N;
            Pack<W, N> u = shifted(h[j], p + c);
            if (!(c >= N - 1 && c + 2 * N <= H) && c + N > 0 && c < H) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    u.v[i] = c + i >= 0 && c + i < H ? __ldg(p + c + i) : from_f<W>(0.0f);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                q[j / M].v[j % M * N + i] = u.v[i];
        }
    } else {
        fetch<W, V, VPT>(q, p, t, step, packs);
    }
    unpack<W, V, VPT>(f, q);
}
template <typename T, int V, int VPT, bool LEAD = false>
__device__ __forceinline__ void load_columns(float2 (&f)[PAIRS<V, VPT>], const void *p, int w32, float none, int t, int step, int packs,
                                             int lead = 0, int H = 0)
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < PAIRS<V, VPT>; ++i)
            f[i] = both(none);
    } else if (w32) {
        fetch_columns<float, V, VPT, LEAD>(f, static_cast<const float *>(p), t, step, packs, lead, H);
    } else {
        fetch_columns<T, V, VPT, LEAD>(f, static_cast<const T *>(p), t, step, packs, lead, H);
    }
}

// Sum of v over the block, the same in every thread and in a fixed order.  `slot` alternates
// between calls, so one barrier a call is enough: a thread that is a call ahead writes the other
// half of `red`.  Up to eight warps' sums are read by every thread (zeros in place of absent
// warps, see clear_sums), more by a lane each.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *red, int slot)
{
    const int warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = warp_sum(v[i]);
    if (warps == 1)
        return;
    float *r = red + slot * 32 * N;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            r[i * 32 + (threadIdx.x >> 5)] = v[i];
    }
    __syncthreads();
    if (warps <= 8) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float4 q = *reinterpret_cast<const float4 *>(r + i * 32);
            v[i] = (q.x + q.y) + (q.z + q.w);
            if (warps > 4) {
                const float4 u = *reinterpret_cast<const float4 *>(r + i * 32 + 4);
                v[i] += (u.x + u.y) + (u.z + u.w);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = warp_sum(r[i * 32 + (threadIdx.x & 31)]);
    }
}

// The sums of warps that a block does not have: zeros, before the first block_sum's barrier.
template <int N>
__device__ __forceinline__ void clear_sums(float *red)
{
    const int warps = blockDim.x >> 5;
    for (int i = threadIdx.x; i < 2 * N * 32; i += blockDim.x)
        if ((i & 31) >= warps)
            red[i] = 0.0f;
}

// The same over the threads that share a row: a warp or the block.
template <bool WARP, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float *red, int slot)
{
    if constexpr (WARP) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = warp_sum(v[i]);
    } else {
        block_sum(v, red, slot);
    }
}

struct NormArgs {
    int T, H;
    const void *x;
    long long ldx;
    const void *weight, *bias;   // either may be null
    int w32;                     // weight and bias are fp32 (else x's type)
    float eps;
    void *y;
    float *mean, *rstd;          // either may be null
    uint8_t *q;                  // FP8 form
    float *sf;
    int pow2;
};

// ------------------------------------------------------------------ copies ahead --------
// A thread's slots: pack j of ring stage g at slot (g * VPT + j) * blockDim + thread, so a
// warp's accesses are contiguous.
// CUT: only the first `bytes` of the pack (which may be none) are there; zeros in place of the others.
template <typename T, int V, bool CUT>
__device__ __forceinline__ void copy_ahead(Pack<T, V> *slot, const T *src, int bytes)
{
    constexpr int BYTES = static_cast<int>(sizeof(Pack<T, V>));
    const uint32_t dst = ptx::smem_u32(slot);
    static_assert(BYTES % 16 == 0, "copies of 16 bytes");
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
        const uint64_t from = reinterpret_cast<uint64_t>(src) + 16 * i;
        if constexpr (CUT) {
            const int n = max(0, min(16, bytes - 16 * i));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * i), "l"(n ? from : from - 16 * i), "r"(n) : "memory");
        } else {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * i), "l"(from) : "memory");
        }
    }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Row r's packs of this thread into ring stage g (nothing past the last row).
template <typename T, int V, int VPT, bool LEAD>
__device__ __forceinline__ void fetch_ahead(Pack<T, V> *ring, int g, const void *base, long long ld, int r, int T_, int H, int packs, int lead)
{
    if (r < T_) {
        const int left = r == T_ - 1 ? H : H + V;   // elements that may be read
        const T *x = static_cast<const T *>(base) + static_cast<size_t>(r) * ld;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int p = threadIdx.x + j * blockDim.x, e = p * V - lead;
            if (p < packs)
                copy_ahead<T, V, LEAD>(ring + (g * VPT + j) * blockDim.x + threadIdx.x, x + e, (left - e) * static_cast<int>(sizeof(T)));
        }
    }
}
// (slots past the row's end were never copied to: clip() the pairs)
template <typename T, int V, int VPT>
__device__ __forceinline__ void from_ring(float2 (&f)[PAIRS<V, VPT>], const Pack<T, V> *ring, int g)
{
    Pack<T, V> q[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        q[j] = ring[(g * VPT + j) * blockDim.x + threadIdx.x];
    unpack<T, V, VPT>(f, q);
}

// ------------------------------------------------------------------ unaligned rows ahead ----
// Rows of any alignment, copied by the whole block in the 16-byte vectors that cover them: the
// row lies in its stage at the byte phase that it has in memory, so both sides are aligned, and
// a thread then reads single elements.  The vectors may hold neighbouring bytes of the matrix,
// but none outside [begin, end): the last ones are cut short (cp.async fills with zeros), and
// the elements of one that starts before the matrix are moved one by one.
struct ByteRows {
    const char *begin, *end;   // of the matrix
    long long pitch;           // bytes
    int bytes;                 // of a row
};
template <typename T>
ByteRows byte_rows(const void *p, long long ld, int T_, int H)
{
    const char *b = static_cast<const char *>(p);
    const long long pitch = ld * static_cast<long long>(sizeof(T));
    return {b, b + pitch * (T_ - 1) + static_cast<long long>(H) * sizeof(T), pitch, static_cast<int>(H * sizeof(T))};
}
__host__ __device__ __forceinline__ int stage_bytes(int row_bytes) { return (row_bytes + 15 + 15) / 16 * 16; }
template <typename T>
__device__ __forceinline__ void fetch_bytes(uint8_t *stage, const ByteRows &m, int row)
{
    const char *a = m.begin + m.pitch * row;
    const int phase = static_cast<int>(reinterpret_cast<uint64_t>(a) & 15);
    const char *a0 = a - phase;
    const int vectors = (phase + m.bytes + 15) >> 4;
    for (int v = threadIdx.x; v < vectors; v += blockDim.x) {
        const char *src = a0 + 16 * static_cast<long long>(v);
        if (src < m.begin) {
            const int stop = min(16, phase + m.bytes);
            for (int i = phase; i < stop; i += static_cast<int>(sizeof(T)))
                *reinterpret_cast<T *>(stage + i) = *reinterpret_cast<const T *>(a0 + i);
        } else {
            const long long left = m.end - src;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(stage + 16 * v)),
                         "l"(reinterpret_cast<uint64_t>(src)), "r"(static_cast<int>(left < 16 ? left : 16))
                         : "memory");
        }
    }
}
// Elements t, t + step, ... of a row in its stage (zeros past its end).
template <typename T, int VPT>
__device__ __forceinline__ void from_bytes(float2 (&f)[PAIRS<1, VPT>], const uint8_t *stage, const ByteRows &m, int row, int H)
{
    const T *e = reinterpret_cast<const T *>(stage + (reinterpret_cast<uint64_t>(m.begin + m.pitch * row) & 15));
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = threadIdx.x + j * blockDim.x;
        const float v = c < H ? to_f<T>(e[c]) : 0.0f;
        if (j & 1)
            f[j / 2].y = v;
        else
            f[j / 2].x = v;
    }
}

// ------------------------------------------------------------------ FP8 scales ----------
__device__ __forceinline__ float fp8_scale(float m, int pow2)
{
    const float sf = fmaxf(m, 1e-4f) / 448.0f;
    if (!pow2)
        return sf;
    // the smallest power of two >= sf (sf is a normal number)
    return __uint_as_float((__float_as_uint(sf) + 0x7FFFFFu) & 0xFF800000u);
}
// Scales of the groups that the half-warp's packs j make up, from the lanes' maxima m[j]: stored, and one
// reciprocal r[j] a group, not a quotient an element: the product is within a few fp32 roundings of
// the quotient, so a code whose quotient lies that near to the middle between two may be its neighbour
// (with power-of-two scales the reciprocal is exact, and so is every code).  Of four groups every lane reduces one (lane
// bits 3 and 2 name it): 9 shuffles and one division, where four apart take 16 and 4 (16384 x 4096 bf16 54
// us so).
template <int VPT>
__device__ __forceinline__ void fp8_scales(const float (&m)[VPT], float (&r)[VPT], float *sf, int t, int step, int packs, int pow2)
{
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    float k;
    if constexpr (VPT == 4) {
        const bool b8 = lane & 8, b4 = lane & 4;
        const float k0 = fmaxf(b8 ? m[2] : m[0], __shfl_xor_sync(ALL, b8 ? m[0] : m[2], 8));
        const float k1 = fmaxf(b8 ? m[3] : m[1], __shfl_xor_sync(ALL, b8 ? m[1] : m[3], 8));
        k = fmaxf(b4 ? k1 : k0, __shfl_xor_sync(ALL, b4 ? k0 : k1, 4));
    } else {
        static_assert(VPT == 1, "one group a half-warp, or four");
        k = fmaxf(m[0], __shfl_xor_sync(ALL, m[0], 8));
        k = fmaxf(k, __shfl_xor_sync(ALL, k, 4));
    }
    k = fmaxf(k, __shfl_xor_sync(ALL, k, 2));
    k = fmaxf(k, __shfl_xor_sync(ALL, k, 1));
    const float scale = fp8_scale(k, pow2), inverse = __fdividef(1.0f, scale);
    const int p = t + (VPT == 4 ? (lane >> 2 & 3) * step : 0);
    if ((lane & (VPT == 4 ? 3 : 15)) == 0 && p < packs)
        sf[p >> 4] = scale;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        r[j] = VPT == 4 ? __shfl_sync(ALL, inverse, (lane & 16) | j << 2) : inverse;
}

// ------------------------------------------------------------------ forward -------------
// The row held in f (zeros past its end), its statistics and outputs; w and b: the thread's
// columns of weight and bias.  FP8: e4m3 codes and 1x128 scales instead of y (V = 8: 16 lanes
// hold one group of 128).  `after_read` runs once every thread has its row in registers.
template <typename T, int V, int VPT, bool FP8, bool WARP, bool LEAD, typename F>
__device__ __forceinline__ void norm_row(const NormArgs &a, int row, int lead, bool cut, float2 (&f)[PAIRS<V, VPT>], const float2 (&w)[PAIRS<V, VPT>],
                                         const float2 (&b)[PAIRS<V, VPT>], float *red, F after_read)
{
    constexpr int P = PAIRS<V, VPT>;
    const int packs = packs_of<V, LEAD>(a.H, lead), t = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
    const float inv = 1.0f / static_cast<float>(a.H);
    float2 acc = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i)
        acc = add2(acc, f[i]);
    float s[1] = {acc.x + acc.y};
    row_sum<WARP>(s, red, 0);
    after_read();
    const float mean = s[0] * inv;
#pragma unroll
    for (int i = 0; i < P; ++i)
        f[i] = add2(f[i], both(-mean));
    clip<V, VPT>(f, t, step, packs, LEAD && cut, lead, a.H);
    acc = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i)
        acc = fma2(f[i], f[i], acc);
    s[0] = acc.x + acc.y;
    row_sum<WARP>(s, red, 1);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    if (t == 0) {
        if (a.mean)
            a.mean[row] = mean;
        if (a.rstd)
            a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
        f[i] = fma2(mul2(f[i], both(rstd)), w[i], b[i]);
    if constexpr (FP8) {
        // packs of a group of 128 lie in one half-warp; whole groups are in or out
        float m[VPT], r[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            m[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 y = f[j * (V / 2) + i];
                m[j] = fmaxf(m[j], fmaxf(fabsf(y.x), fabsf(y.y)));
            }
        }
        float *sf = a.sf + static_cast<size_t>(row) * (a.H / 128);
        fp8_scales(m, r, sf, t, step, packs, a.pow2);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const float2 *y = f + j * (V / 2);
            const int p = t + j * step;
            if (p < packs) {
                uint32_t code[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 lo = mul2(y[2 * h], both(r[j])), hi = mul2(y[2 * h + 1], both(r[j]));
                    code[h] = ptx::cvt_e4m3x2(lo.x, lo.y) | (ptx::cvt_e4m3x2(hi.x, hi.y) << 16);
                }
                *reinterpret_cast<uint2 *>(a.q + static_cast<size_t>(row) * a.H + static_cast<size_t>(p) * V) = make_uint2(code[0], code[1]);
            }
        }
    } else {
        put<T, V, VPT, LEAD>(static_cast<T *>(a.y) + static_cast<size_t>(row) * a.H, f, t, step, packs, lead, a.H);
    }
}

// One row a block; or (WARP, rows of at most 1024 elements) one row a warp at a time, the next
// one on its way.  The weight and bias are loaded beside the first row, ahead of its sums.
constexpr int ROW_WARPS = 4;
template <typename T, int V, int VPT, bool FP8, bool WARP>
__global__ void __launch_bounds__(WARP ? ROW_WARPS * 32 : V * VPT == 32 ? 512 : 1024) norm_kernel(const NormArgs a)
{
    constexpr int P = PAIRS<V, VPT>;
    __shared__ __align__(16) float red[WARP ? 4 : 64];
    const int packs = a.H / V, t = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
    if constexpr (!WARP)
        clear_sums<1>(red);
    const T *x = static_cast<const T *>(a.x);
    int row = WARP ? blockIdx.x * ROW_WARPS + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.T)
        return;
    Pack<T, V> q[VPT];
    fetch<T, V, VPT>(q, x + static_cast<size_t>(row) * a.ldx, t, step, packs);
    float2 f[P], w[P], b[P];
    load_columns<T, V, VPT>(w, a.weight, a.w32, 1.0f, t, step, packs);
    load_columns<T, V, VPT>(b, a.bias, a.w32, 0.0f, t, step, packs);
    if constexpr (WARP) {
        for (;;) {
            unpack<T, V, VPT>(f, q);
            const int next = row + gridDim.x * ROW_WARPS;
            if (next < a.T)
                fetch<T, V, VPT>(q, x + static_cast<size_t>(next) * a.ldx, t, step, packs);
            norm_row<T, V, VPT, FP8, true, false>(a, row, 0, false, f, w, b, red, [] {});
            if (next >= a.T)
                return;
            row = next;
        }
    } else {
        unpack<T, V, VPT>(f, q);
        norm_row<T, V, VPT, FP8, false, false>(a, row, 0, false, f, w, b, red, [] {});
    }
}

// Persistent blocks: rows copied AHEAD rows before their use, weight and bias kept in registers.
template <typename T, int V, int VPT, bool FP8, int AHEAD, bool LEAD>
__global__ void __launch_bounds__(512) norm_ring_kernel(const NormArgs a)
{
    constexpr int P = PAIRS<V, VPT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[64];
    Pack<T, V> *ring = reinterpret_cast<Pack<T, V> *>(smem);
    const int lead = LEAD ? lead_of(static_cast<const T *>(a.x) + static_cast<size_t>(blockIdx.x) * a.ldx) : 0;
    const int packs = packs_of<V, LEAD>(a.H, lead);
    const bool cut = LEAD && cut_packs<V, VPT>(threadIdx.x, blockDim.x, lead, a.H);
#pragma unroll
    for (int g = 0; g < AHEAD; ++g) {
        fetch_ahead<T, V, VPT, LEAD>(ring, g, a.x, a.ldx, blockIdx.x + g * gridDim.x, a.T, a.H, packs, lead);
        copies_commit();
    }
    clear_sums<1>(red);
    float2 w[P], b[P];
    load_columns<T, V, VPT, LEAD>(w, a.weight, a.w32, 1.0f, threadIdx.x, blockDim.x, packs, lead, a.H);
    load_columns<T, V, VPT, LEAD>(b, a.bias, a.w32, 0.0f, threadIdx.x, blockDim.x, packs, lead, a.H);
    int g = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x) {
        copies_wait<AHEAD - 1>();
        float2 f[P];
        from_ring<T, V, VPT>(f, ring, g);
        clip<V, VPT>(f, threadIdx.x, blockDim.x, packs, LEAD && cut, lead, a.H);
        norm_row<T, V, VPT, FP8, false, LEAD>(a, row, lead, cut, f, w, b, red, [&] {
            fetch_ahead<T, V, VPT, LEAD>(ring, g, a.x, a.ldx, row + AHEAD * gridDim.x, a.T, a.H, packs, lead);
            copies_commit();
        });
        g = g == AHEAD - 1 ? 0 : g + 1;
    }
}

// Persistent blocks over rows of any alignment (more than 1024 elements).
template <typename T, int VPT, int AHEAD>
__global__ void __launch_bounds__(512) norm_bytes_kernel(const NormArgs a, const ByteRows m)
{
    constexpr int P = PAIRS<1, VPT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[64];
    const int size = stage_bytes(m.bytes);
#pragma unroll
    for (int g = 0; g < AHEAD; ++g) {
        const int row = blockIdx.x + g * gridDim.x;
        if (row < a.T)
            fetch_bytes<T>(smem + g * size, m, row);
        copies_commit();
    }
    clear_sums<1>(red);
    float2 w[P], b[P];
    load_columns<T, 1, VPT>(w, a.weight, a.w32, 1.0f, threadIdx.x, blockDim.x, a.H);
    load_columns<T, 1, VPT>(b, a.bias, a.w32, 0.0f, threadIdx.x, blockDim.x, a.H);
    int g = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x) {
        copies_wait<AHEAD - 1>();
        __syncthreads();   // the other threads' copies
        float2 f[P];
        from_bytes<T, VPT>(f, smem + g * size, m, row, a.H);
        norm_row<T, 1, VPT, false, false, false>(a, row, 0, false, f, w, b, red, [&] {
            const int next = row + AHEAD * gridDim.x;
            if (next < a.T)
                fetch_bytes<T>(smem + g * size, m, next);
            copies_commit();
        });
        g = g == AHEAD - 1 ? 0 : g + 1;
    }
}

// ------------------------------------------------------------------ backward ------------
struct NormBwdArgs {
    int T, H;
    const void *dy, *x;
    long long lddy, ldx;
    const void *weight;
    int w32;
    const float *mean, *rstd;
    void *dx;
    float *part;   // [2][blocks][pitch] sums of dy*xh and of dy over each block's rows (LEAD: from their lead on)
    int pitch;
};

// xh and a = dy*g of one row, its two sums, and the columns' sums so far.
template <int P>
__device__ __forceinline__ void backward_sums(float2 (&xh)[P], const float2 (&d)[P], const float2 (&w)[P], float2 (&dg)[P], float2 (&db)[P],
                                              float mean, float rstd, float (&s)[2])
{
    float2 s0 = both(0.0f), s1 = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        xh[i] = mul2(add2(xh[i], both(-mean)), both(rstd));
        dg[i] = fma2(d[i], xh[i], dg[i]);
        db[i] = add2(db[i], d[i]);
        const float2 g = mul2(d[i], w[i]);
        s0 = add2(s0, g);
        s1 = fma2(g, xh[i], s1);
    }
    s[0] = s0.x + s0.y;
    s[1] = s1.x + s1.y;
}
template <int P>
__device__ __forceinline__ void backward_out(float2 (&o)[P], const float2 (&xh)[P], const float2 (&d)[P], const float2 (&w)[P], float inv,
                                             float rstd, const float (&s)[2])
{
    const float2 ma = both(-s[0] * inv), mb = both(-s[1] * inv);
#pragma unroll
    for (int i = 0; i < P; ++i)
        o[i] = mul2(fma2(xh[i], mb, fma2(d[i], w[i], ma)), both(rstd));
}

// Rows b, b + blocks, ... of block b: a thread keeps its columns' two sums in registers over all
// of them, so dy and x are read once from HBM.  AHEAD > 0: rows of x and dy copied that many rows
// before use, and read from shared memory twice (for the sums, then for dx) instead of held in
// registers between.
template <typename T, int V, int VPT, int AHEAD, bool LEAD>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormBwdArgs a)
{
    constexpr int P = PAIRS<V, VPT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[128];
    const int t = threadIdx.x, step = blockDim.x;
    const int lead = LEAD ? lead_of(static_cast<const T *>(a.x) + static_cast<size_t>(blockIdx.x) * a.ldx) : 0;
    const int packs = packs_of<V, LEAD>(a.H, lead);
    const bool cut = LEAD && cut_packs<V, VPT>(t, step, lead, a.H);
    const float inv = 1.0f / static_cast<float>(a.H);
    Pack<T, V> *ring_x = reinterpret_cast<Pack<T, V> *>(smem), *ring_d = ring_x + AHEAD * VPT * blockDim.x;
    if constexpr (AHEAD > 0) {
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) {
            fetch_ahead<T, V, VPT, LEAD>(ring_x, g, a.x, a.ldx, blockIdx.x + g * gridDim.x, a.T, a.H, packs, lead);
            fetch_ahead<T, V, VPT, LEAD>(ring_d, g, a.dy, a.lddy, blockIdx.x + g * gridDim.x, a.T, a.H, packs, lead);
            copies_commit();
        }
    }
    clear_sums<2>(red);
    float2 w[P], dg[P], db[P];
    load_columns<T, V, VPT, LEAD>(w, a.weight, a.w32, 1.0f, t, step, packs, lead, a.H);
#pragma unroll
    for (int i = 0; i < P; ++i)
        dg[i] = db[i] = both(0.0f);
    int slot = 0, stage = 0;
    float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];   // (no more blocks than rows)
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, slot ^= 1) {
        const int next = row + gridDim.x;
        const float mean1 = next < a.T ? a.mean[next] : 0.0f, rstd1 = next < a.T ? a.rstd[next] : 0.0f;
        float2 xh[P], d[P];
        if constexpr (AHEAD > 0) {
            copies_wait<AHEAD - 1>();
            from_ring<T, V, VPT>(xh, ring_x, stage);
            from_ring<T, V, VPT>(d, ring_d, stage);
        } else {
            Pack<T, V> q[VPT];
            fetch<T, V, VPT>(q, static_cast<const T *>(a.x) + static_cast<size_t>(row) * a.ldx, t, step, packs);
            unpack<T, V, VPT>(xh, q);
            fetch<T, V, VPT>(q, static_cast<const T *>(a.dy) + static_cast<size_t>(row) * a.lddy, t, step, packs);
            unpack<T, V, VPT>(d, q);
        }
        if constexpr (AHEAD > 0) {   // what lies outside the row is not there: no products with it
            clip<V, VPT>(xh, t, step, packs, LEAD && cut, lead, a.H);
            clip<V, VPT>(d, t, step, packs, LEAD && cut, lead, a.H);
        }
        float s[2];
        backward_sums<P>(xh, d, w, dg, db, mean, rstd, s);
        block_sum(s, red, slot);
        float2 o[P];
        if constexpr (AHEAD > 0) {
            from_ring<T, V, VPT>(xh, ring_x, stage);
            from_ring<T, V, VPT>(d, ring_d, stage);
#pragma unroll
            for (int i = 0; i < P; ++i)
                xh[i] = mul2(add2(xh[i], both(-mean)), both(rstd));
        }
        backward_out<P>(o, xh, d, w, inv, rstd, s);
        put<T, V, VPT, LEAD>(static_cast<T *>(a.dx) + static_cast<size_t>(row) * a.H, o, t, step, packs, lead, a.H);
        if constexpr (AHEAD > 0) {   // (every value read above has been used by now)
            fetch_ahead<T, V, VPT, LEAD>(ring_x, stage, a.x, a.ldx, row + AHEAD * gridDim.x, a.T, a.H, packs, lead);
            fetch_ahead<T, V, VPT, LEAD>(ring_d, stage, a.dy, a.lddy, row + AHEAD * gridDim.x, a.T, a.H, packs, lead);
            copies_commit();
            stage = stage == AHEAD - 1 ? 0 : stage + 1;
        }
        mean = mean1;
        rstd = rstd1;
    }
    if (a.part) {
        float *p = a.part + static_cast<size_t>(blockIdx.x) * a.pitch;
        put<float, V, VPT>(p, dg, t, step, packs);
        put<float, V, VPT>(p + static_cast<size_t>(gridDim.x) * a.pitch, db, t, step, packs);
    }
    ptx::launch_dependents();
}

// Rows of any alignment (more than 1024 elements).
template <typename T, int VPT, int AHEAD>
__global__ void __launch_bounds__(512) norm_backward_bytes_kernel(const NormBwdArgs a, const ByteRows mx, const ByteRows md)
{
    constexpr int P = PAIRS<1, VPT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[128];
    const int t = threadIdx.x, step = blockDim.x, size = stage_bytes(mx.bytes);
    const float inv = 1.0f / static_cast<float>(a.H);
    uint8_t *ring_d = smem + AHEAD * size;
#pragma unroll
    for (int g = 0; g < AHEAD; ++g) {
        const int row = blockIdx.x + g * gridDim.x;
        if (row < a.T) {
            fetch_bytes<T>(smem + g * size, mx, row);
            fetch_bytes<T>(ring_d + g * size, md, row);
        }
        copies_commit();
    }
    clear_sums<2>(red);
    float2 w[P], dg[P], db[P];
    load_columns<T, 1, VPT>(w, a.weight, a.w32, 1.0f, t, step, a.H);
#pragma unroll
    for (int i = 0; i < P; ++i)
        dg[i] = db[i] = both(0.0f);
    int slot = 0, g = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, slot ^= 1) {
        const float mean = a.mean[row], rstd = a.rstd[row];
        copies_wait<AHEAD - 1>();
        __syncthreads();   // the other threads' copies
        float2 xh[P], d[P], o[P];
        from_bytes<T, VPT>(xh, smem + g * size, mx, row, a.H);
        from_bytes<T, VPT>(d, ring_d + g * size, md, row, a.H);
        float s[2];
        backward_sums<P>(xh, d, w, dg, db, mean, rstd, s);
        block_sum(s, red, slot);
        const int next = row + AHEAD * gridDim.x;   // every thread has read the stage
        if (next < a.T) {
            fetch_bytes<T>(smem + g * size, mx, next);
            fetch_bytes<T>(ring_d + g * size, md, next);
        }
        copies_commit();
        g = g == AHEAD - 1 ? 0 : g + 1;
        backward_out<P>(o, xh, d, w, inv, rstd, s);
        put<T, 1, VPT>(static_cast<T *>(a.dx) + static_cast<size_t>(row) * a.H, o, t, step, a.H);
    }
    if (a.part) {
        float *p = a.part + static_cast<size_t>(blockIdx.x) * a.pitch;
        put<float, 1, VPT>(p, dg, t, step, a.H);
        put<float, 1, VPT>(p + static_cast<size_t>(gridDim.x) * a.pitch, db, t, step, a.H);
    }
    ptx::launch_dependents();
}

// Rows of at most 1024 elements: one row a warp at a time, the next one on its way; the block's
// warps add their columns' sums at the end, in order.
template <typename T, int V, int VPT>
__global__ void __launch_bounds__(ROW_WARPS * 32) norm_backward_warp_kernel(const NormBwdArgs a)
{
    constexpr int P = PAIRS<V, VPT>;
    struct alignas(16) Sums {
        float v[32 * V * VPT];
    };
    static_assert(alignof(Sums) >= alignof(Pack<float, V>), "put() stores whole packs into them");
    __shared__ Sums sums[2][ROW_WARPS];
    const int packs = a.H / V, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float inv = 1.0f / static_cast<float>(a.H);
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    float2 w[P], dg[P], db[P];
    load_columns<T, V, VPT>(w, a.weight, a.w32, 1.0f, lane, 32, packs);
#pragma unroll
    for (int i = 0; i < P; ++i)
        dg[i] = db[i] = both(0.0f);
    int row = blockIdx.x * ROW_WARPS + warp;
    if (row < a.T) {
        Pack<T, V> qx[VPT], qd[VPT];
        fetch<T, V, VPT>(qx, x + static_cast<size_t>(row) * a.ldx, lane, 32, packs);
        fetch<T, V, VPT>(qd, dy + static_cast<size_t>(row) * a.lddy, lane, 32, packs);
        float mean = a.mean[row], rstd = a.rstd[row];
        for (;;) {
            float2 xh[P], d[P], o[P];
            unpack<T, V, VPT>(xh, qx);
            unpack<T, V, VPT>(d, qd);
            const int next = row + gridDim.x * ROW_WARPS;
            const float m = mean, r = rstd;
            if (next < a.T) {
                fetch<T, V, VPT>(qx, x + static_cast<size_t>(next) * a.ldx, lane, 32, packs);
                fetch<T, V, VPT>(qd, dy + static_cast<size_t>(next) * a.lddy, lane, 32, packs);
                mean = a.mean[next];
                rstd = a.rstd[next];
            }
            float s[2];
            backward_sums<P>(xh, d, w, dg, db, m, r, s);
            row_sum<true>(s, nullptr, 0);
            backward_out<P>(o, xh, d, w, inv, r, s);
            put<T, V, VPT>(static_cast<T *>(a.dx) + static_cast<size_t>(row) * a.H, o, lane, 32, packs);
            if (next >= a.T)
                break;
            row = next;
        }
    }
    if (a.part) {
        put<float, V, VPT>(sums[0][warp].v, dg, lane, 32, 32 * VPT);
        put<float, V, VPT>(sums[1][warp].v, db, lane, 32, 32 * VPT);
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.H; i += ROW_WARPS * 32) {
            const int which = i >= a.H, c = i - which * a.H;
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < ROW_WARPS; ++k)
                v += sums[which][k].v[c];
            a.part[(static_cast<size_t>(which) * gridDim.x + blockIdx.x) * a.pitch + c] = v;
        }
    }
    ptx::launch_dependents();
}

// Column sums of the partial sums, in a fixed order: a block of 32 columns x 32 row lanes.  Row b of them
// starts at b * step elements past a boundary of `boundary`.
struct PartRows {
    const float *part;
    int blocks, pitch, step, boundary;
};
template <typename TW>
__global__ void norm_reduce_kernel(const PartRows p, int H, TW *dweight, TW *dbias)
{
    __shared__ float tile[32][33];
    ptx::grid_dependency_wait();
    const float *src = p.part + static_cast<size_t>(blockIdx.y) * p.blocks * p.pitch;
    TW *dst = blockIdx.y == 0 ? dweight : dbias;
    if (!dst)
        return;
    const int col = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (col < H) {
#pragma unroll 4
        for (int b = threadIdx.y; b < p.blocks; b += 32)
            s += src[static_cast<size_t>(b) * p.pitch + col + ((b * p.step) & (p.boundary - 1))];
    }
    tile[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = warp_sum(tile[threadIdx.x][threadIdx.y]);
    const int out = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && out < H)
        dst[out] = from_f<TW>(s);
}

// Started while the last rows are still worked on; it waits for them before it reads.
template <typename TW>
cudaError_t launch_reduce(const PartRows &p, int H, TW *dweight, TW *dbias, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((H + 31) / 32, 2);
    cfg.blockDim = dim3(32, 32);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_reduce_kernel<TW>, p, H, dweight, dbias);
}

int round32(int v) { return (v + 31) / 32 * 32; }

// How rows move.  PACKED: every row starts on a 16-byte boundary and has whole packs of 8 elements.
// PHASED: packs too, where rows start off the boundaries (or end inside a pack) but the same row of
// every tensor at the same place past one: rows a multiple of 8 apart then have one lead, so with such
// a stride a block's columns stay and only its packs' ends differ.  ANY: element by element
// (neighbouring lanes on neighbouring elements).
enum Rows { PACKED, PHASED, ANY };
Rows rows_of(int H, int dtype, const void *p, long long ld)
{
    const size_t b = dtype_bytes(dtype);
    if (!op_aligned(p, 16) || static_cast<size_t>(ld - H) * b % 16 != 0 || H < 8)
        return ANY;
    return H % 8 == 0 ? PACKED : PHASED;
}
Rows worst(Rows a, Rows b) { return a > b ? a : b; }
// weight or bias
Rows affine_of(const void *p) { return p == nullptr || op_aligned(p, 16) ? PACKED : PHASED; }
// Packs of a row, at most.
template <typename T>
int most_packs(int H, Rows rows)
{
    return rows == PACKED ? H / 8 : (H + 16 / static_cast<int>(sizeof(T)) - 1 + 7) / 8;
}
// Rows in packs with a lead, in the persistent kernels (forward and backward in us, element by element in
// brackets): 16384 x 5001 bf16 74 and 133 (155 and 218), 5000 x 2001 12.8 and 20 (14.8 and 24), fp32 16384 x
// 3001 backward 117 (142).  Not where they are no faster: rows of a warp, 16384 x 1001 bf16 21 and 33 (21
// and 31); single rows of a block, whose columns' shifts come once a row, 3000 x 1501 bf16 12 and 16 (9.1
// and 16); 2000 x 8191 bf16, whose packs take four a thread, 27 and 54 (28 and 41); and fp32's
// forward, 8192 x 7001 114 (106).
template <typename T>
bool phased(int H, Rows rows)
{
    return rows == PHASED && H > 1024 && most_packs<T>(H, rows) <= 1024;
}

bool norm_args_ok(int T, int H, int dtype, int w_dtype, const void *weight, const void *bias)
{
    if (T < 0 || T > MAX_ROWS || H < 1 || H > MAX_H || !dtype_ok(dtype))
        return false;
    if ((weight || bias) && w_dtype != dtype && w_dtype != MOE_F32)
        return false;
    const size_t wb = dtype_bytes(w_dtype);
    return op_aligned(weight, wb) && op_aligned(bias, wb);
}

template <typename K>
bool allow_smem(K kern, size_t bytes)
{
    // (without the attribute a block's static and dynamic shared memory together stay within 48 KB)
    return bytes <= 40 * 1024 ||
           ensure_max_dynamic_smem(reinterpret_cast<const void *>(kern), static_cast<int>(bytes)) == cudaSuccess;
}

// Persistent blocks an SM of `threads` threads, AHEAD stages and `tensors` tensors in the ring:
// about 512 threads, within the SM's shared memory.
template <typename T, int V, int VPT>
int ring_blocks(int threads, int ahead, int tensors, size_t &smem)
{
    smem = static_cast<size_t>(ahead) * VPT * threads * sizeof(Pack<T, V>) * tensors;
    const size_t fit = smem ? 200 * 1024 / smem : 0;
    const size_t want = threads >= 512 ? 1 : 512 / threads;
    return static_cast<int>(fit < want ? fit : want);
}

// Leads repeat after at most 8 rows: with a stride of whole eights a block's rows have one lead.
int ring_grid(int per_sm, int num_sms) { return per_sm * num_sms / 8 * 8; }

template <typename T, bool FP8, int AHEAD, bool LEAD>
bool try_norm_ring(const NormArgs &a, int packs, int num_sms, cudaStream_t s)
{
    const int threads = round32((packs + 3) / 4);
    size_t smem;
    const int per_sm = ring_blocks<T, 8, 4>(threads, AHEAD, 1, smem);
    // long batches only: every block has rows to copy ahead of
    if (per_sm < 1 || a.T < AHEAD * per_sm * num_sms)
        return false;
    const auto kern = norm_ring_kernel<T, 8, 4, FP8, AHEAD, LEAD>;
    if (!allow_smem(kern, smem))
        return false;
    kern<<<ring_grid(per_sm, num_sms), threads, smem, s>>>(a);
    return true;
}

// Blocks of one-row-a-warp kernels: a warp for each row up to `per_sm` blocks an SM.
int warp_blocks(int T, int per_sm, int num_sms)
{
    const int need = (T + ROW_WARPS - 1) / ROW_WARPS, most = per_sm * num_sms;
    return need < most ? need : most;
}

// Blocks an SM (about 512 threads), stages and shared memory of the kernels for rows of any
// alignment, `tensors` rows a stage.
struct BytesPlan {
    int threads, per_sm, ahead;
    size_t smem;
};
BytesPlan bytes_plan(int H, size_t elem, int tensors)
{
    BytesPlan p{};
    p.threads = round32(H <= 8192 ? (H + 15) / 16 : (H + 31) / 32);
    const size_t stage = static_cast<size_t>(stage_bytes(static_cast<int>(H * elem))) * tensors;
    p.ahead = 3 * stage <= 200 * 1024 ? 3 : 1;
    p.smem = p.ahead * stage;
    const size_t fit = 200 * 1024 / p.smem, want = 512 / p.threads;
    p.per_sm = static_cast<int>(fit < want ? fit : want);
    return p;
}

template <typename T, int VPT, int AHEAD>
bool launch_norm_bytes(const NormArgs &a, const BytesPlan &p, int num_sms, cudaStream_t s)
{
    const auto kern = norm_bytes_kernel<T, VPT, AHEAD>;
    if (!allow_smem(kern, p.smem))
        return false;
    const int most = p.per_sm * num_sms;
    kern<<<a.T < most ? a.T : most, p.threads, p.smem, s>>>(a, byte_rows<T>(a.x, a.ldx, a.T, a.H));
    return true;
}

template <typename T, int VPT, int AHEAD>
bool launch_backward_bytes(const NormBwdArgs &a, const BytesPlan &p, int blocks, cudaStream_t s)
{
    const auto kern = norm_backward_bytes_kernel<T, VPT, AHEAD>;
    if (!allow_smem(kern, p.smem))
        return false;
    kern<<<blocks, p.threads, p.smem, s>>>(a, byte_rows<T>(a.x, a.ldx, a.T, a.H), byte_rows<T>(a.dy, a.lddy, a.T, a.H));
    return true;
}

template <typename T, int V, int VPT, bool FP8>
void launch_norm_warps(const NormArgs &a, int num_sms, cudaStream_t s)
{
    norm_kernel<T, V, VPT, FP8, true><<<warp_blocks(a.T, 8, num_sms), ROW_WARPS * 32, 0, s>>>(a);
}

template <typename T, bool FP8>
void launch_norm_packs(const NormArgs &a, int num_sms, cudaStream_t s)
{
    // few rows: as many threads a row as it has packs, for latency (128 x 7168 bf16 2.6 us, four packs a
    // thread 2.8; 600 x 4096 4.5 and 3.4)
    const bool few = a.T <= 2 * num_sms;
    const int packs = a.H / 8;
    if (packs <= 32)
        launch_norm_warps<T, 8, 1, FP8>(a, num_sms, s);
    else if (packs <= 128 && !few)
        launch_norm_warps<T, 8, 4, FP8>(a, num_sms, s);
    else if (few && packs <= 1024)
        norm_kernel<T, 8, 1, FP8, false><<<a.T, round32(packs), 0, s>>>(a);
    else if (!try_norm_ring<T, FP8, 4, false>(a, packs, num_sms, s))
        norm_kernel<T, 8, 4, FP8, false><<<a.T, round32((packs + 3) / 4), 0, s>>>(a);
}

template <typename T>
bool launch_norm(const NormArgs &a, Rows rows, int num_sms, cudaStream_t s)
{
    if (rows == PACKED) {
        launch_norm_packs<T, false>(a, num_sms, s);
        return true;
    }
    if constexpr (sizeof(T) == 2)   // (see phased)
        if (phased<T>(a.H, rows) && try_norm_ring<T, false, 4, true>(a, most_packs<T>(a.H, rows), num_sms, s))
            return true;
    if (a.H <= 256)
        launch_norm_warps<T, 1, 8, false>(a, num_sms, s);
    else if (a.H <= 576)
        launch_norm_warps<T, 1, 18, false>(a, num_sms, s);
    else if (a.H <= 1024)
        launch_norm_warps<T, 1, 32, false>(a, num_sms, s);
    else {
        const BytesPlan p = bytes_plan(a.H, sizeof(T), 1);
        return a.H > 8192    ? (p.ahead == 3 ? launch_norm_bytes<T, 32, 3>(a, p, num_sms, s) : launch_norm_bytes<T, 32, 1>(a, p, num_sms, s))
               : p.ahead == 3 ? launch_norm_bytes<T, 16, 3>(a, p, num_sms, s)
                              : launch_norm_bytes<T, 16, 1>(a, p, num_sms, s);
    }
    return true;
}

// The backward pass: kernel, blocks (each keeps a row of partial sums) and how they are found.
enum Plan { WARPS_1, WARPS_4, RING, DIRECT, BYTES };
template <typename T>
Plan backward_plan(int T_, int H, Rows rows, int num_sms, int &blocks)
{
    if (H <= 256 || (H <= 1024 && (rows != PACKED || T_ > 2 * num_sms))) {
        blocks = warp_blocks(T_, 3, num_sms);
        return H <= 256 ? WARPS_1 : WARPS_4;
    }
    if (rows == PACKED || phased<T>(H, rows)) {
        size_t smem;
        const int packs = most_packs<T>(H, rows);
        const int per_sm = packs <= 1024 ? ring_blocks<T, 8, 2>(round32((packs + 1) / 2), packs <= 512 ? 4 : 3, 2, smem)
                                         : ring_blocks<T, 8, 4>(round32((packs + 3) / 4), 2, 2, smem);
        if (per_sm >= 1 && T_ >= 4 * per_sm * num_sms) {
            blocks = ring_grid(per_sm, num_sms);
            return RING;
        }
    }
    blocks = rows == PACKED ? (H >= 4096 ? 1 : 2) * num_sms : bytes_plan(H, sizeof(T), 2).per_sm * num_sms;
    blocks = T_ < blocks ? T_ : blocks;
    return rows == PACKED ? DIRECT : BYTES;
}
// (the workspace covers every alignment)
template <typename T>
int most_backward_blocks(int T_, int H, int num_sms)
{
    int most = 0;
    for (const Rows rows : {PACKED, PHASED, ANY}) {
        int b;
        backward_plan<T>(T_, H, rows, num_sms, b);
        most = b > most ? b : most;
    }
    return most;
}

// Floats of a row of partial sums: whole packs after any lead.
int part_pitch(int H) { return (H + 7 + 7) / 8 * 8; }

template <typename T, int VPT, int AHEAD, bool LEAD>
bool launch_backward_ring(const NormBwdArgs &a, int packs, int blocks, cudaStream_t s)
{
    const int threads = round32((packs + VPT - 1) / VPT);
    size_t smem;
    ring_blocks<T, 8, VPT>(threads, AHEAD, 2, smem);
    const auto kern = norm_backward_kernel<T, 8, VPT, AHEAD, LEAD>;
    if (!allow_smem(kern, smem))
        return false;
    kern<<<blocks, threads, smem, s>>>(a);
    return true;
}

template <typename T>
bool launch_backward(const NormBwdArgs &a, Rows rows, int num_sms, PartRows &part, cudaStream_t s)
{
    int blocks;
    const Plan plan = backward_plan<T>(a.T, a.H, rows, num_sms, blocks);
    const bool packed = rows == PACKED;
    const int packs = most_packs<T>(a.H, rows);
    constexpr int boundary = VEC<T>;
    part = {a.part, blocks, a.pitch, plan == RING && !packed ? a.H % boundary : 0, boundary};
    if (plan == RING && !packed)
        return packs <= 512 ? launch_backward_ring<T, 2, 4, true>(a, packs, blocks, s) : launch_backward_ring<T, 2, 3, true>(a, packs, blocks, s);
    if (plan == RING)
        return packs <= 512    ? launch_backward_ring<T, 2, 4, false>(a, packs, blocks, s)
               : packs <= 1024 ? launch_backward_ring<T, 2, 3, false>(a, packs, blocks, s)
                               : launch_backward_ring<T, 4, 2, false>(a, packs, blocks, s);
    if (plan == WARPS_1 && packed)
        norm_backward_warp_kernel<T, 8, 1><<<blocks, ROW_WARPS * 32, 0, s>>>(a);
    else if (plan == WARPS_4 && packed)
        norm_backward_warp_kernel<T, 8, 4><<<blocks, ROW_WARPS * 32, 0, s>>>(a);
    else if (plan == DIRECT && packs <= 1024)
        norm_backward_kernel<T, 8, 2, 0, false><<<blocks, round32((packs + 1) / 2), 0, s>>>(a);
    else if (plan == DIRECT)
        norm_backward_kernel<T, 8, 4, 0, false><<<blocks, round32((packs + 3) / 4), 0, s>>>(a);
    else if (plan == WARPS_1)
        norm_backward_warp_kernel<T, 1, 8><<<blocks, ROW_WARPS * 32, 0, s>>>(a);
    else if (plan == WARPS_4 && a.H <= 576)
        norm_backward_warp_kernel<T, 1, 18><<<blocks, ROW_WARPS * 32, 0, s>>>(a);
    else if (plan == WARPS_4)
        norm_backward_warp_kernel<T, 1, 32><<<blocks, ROW_WARPS * 32, 0, s>>>(a);
    else {
        const BytesPlan p = bytes_plan(a.H, sizeof(T), 2);
        return a.H > 8192     ? (p.ahead == 3 ? launch_backward_bytes<T, 32, 3>(a, p, blocks, s) : launch_backward_bytes<T, 32, 1>(a, p, blocks, s))
               : p.ahead == 3 ? launch_backward_bytes<T, 16, 3>(a, p, blocks, s)
                              : launch_backward_bytes<T, 16, 1>(a, p, blocks, s);
    }
    return true;
}

}  // namespace

extern "C" {

int moe_layer_norm(int T, int H, const void *x, int64_t ldx, int dtype, const void *weight, const void *bias,
                   int w_dtype, float eps, void *y, float *mean, float *rstd, void *stream)
{
    if (!norm_args_ok(T, H, dtype, w_dtype, weight, bias) || ldx < H || !(eps >= 0.0f))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    const size_t b = dtype_bytes(dtype);
    if (!x || !y || !op_aligned(x, b) || !op_aligned(y, b) || !op_aligned(mean, 4) || !op_aligned(rstd, 4))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const NormArgs a{T, H, x, ldx, weight, bias, w_dtype == MOE_F32 && dtype != MOE_F32, eps, y, mean, rstd, nullptr, nullptr, 0};
    const Rows rows = worst(worst(rows_of(H, dtype, x, ldx), rows_of(H, dtype, y, H)), worst(affine_of(weight), affine_of(bias)));
    const bool ok = with_dtype(dtype, [&](auto *t) {
        return launch_norm<std::remove_pointer_t<decltype(t)>>(a, rows, sms, static_cast<cudaStream_t>(stream));
    });
    return ok ? launched() : MOE_ERR_CUDA;
}

int moe_layer_norm_fp8(int T, int H, const void *x, int64_t ldx, int dtype, const void *weight, const void *bias,
                       int w_dtype, float eps, int pow2_scales, uint8_t *q, float *sf, void *stream)
{
    if (!norm_args_ok(T, H, dtype, w_dtype, weight, bias) || ldx < H || !(eps >= 0.0f) || H % 128 != 0 ||
        pow2_scales < 0 || pow2_scales > 1)
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    if (!x || !q || !sf || rows_of(H, dtype, x, ldx) != PACKED || !op_aligned(q, 16) || !op_aligned(sf, 4) ||
        affine_of(weight) != PACKED || affine_of(bias) != PACKED)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const NormArgs a{T, H, x, ldx, weight, bias, w_dtype == MOE_F32 && dtype != MOE_F32, eps, nullptr, nullptr, nullptr, q, sf, pow2_scales};
    with_dtype(dtype, [&](auto *t) {
        launch_norm_packs<std::remove_pointer_t<decltype(t)>, true>(a, sms, static_cast<cudaStream_t>(stream));
    });
    return launched();
}

int moe_layer_norm_backward_workspace(int T, int H, uint64_t *bytes)
{
    if (T < 0 || T > MAX_ROWS || H < 1 || H > MAX_H || !bytes)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    // enough for every element type
    const int a = most_backward_blocks<float>(T, H, sms), b = most_backward_blocks<__nv_bfloat16>(T, H, sms);
    *bytes = 2ull * (a > b ? a : b) * static_cast<uint64_t>(part_pitch(H)) * sizeof(float);
    return MOE_OK;
}

int moe_layer_norm_backward(int T, int H, const void *dy, int64_t lddy, const void *x, int64_t ldx, int dtype,
                            const void *weight, int w_dtype, const float *mean, const float *rstd, void *dx,
                            void *dweight, void *dbias, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (!norm_args_ok(T, H, dtype, w_dtype, weight, nullptr) || ldx < H || lddy < H)
        return MOE_ERR_INVALID_ARG;
    if ((dweight || dbias) && ((w_dtype != dtype && w_dtype != MOE_F32) || !op_aligned(dweight, dtype_bytes(w_dtype)) ||
                               !op_aligned(dbias, dtype_bytes(w_dtype))))
        return MOE_ERR_INVALID_ARG;
    const size_t b = dtype_bytes(dtype);
    if (T > 0 && (!dy || !x || !mean || !rstd || !dx || !op_aligned(dy, b) || !op_aligned(x, b) || !op_aligned(dx, b) ||
                  !op_aligned(mean, 4) || !op_aligned(rstd, 4)))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool sums = dweight || dbias;
    uint64_t need = 0;
    if (sums && T > 0 &&
        (!workspace || !op_aligned(workspace, 16) || moe_layer_norm_backward_workspace(T, H, &need) != MOE_OK || workspace_bytes < need))
        return MOE_ERR_INVALID_ARG;
    PartRows part{};
    if (T > 0) {
        const NormBwdArgs a{T, H, dy, x, lddy, ldx, weight, w_dtype == MOE_F32 && dtype != MOE_F32, mean, rstd, dx,
                            sums ? static_cast<float *>(workspace) : nullptr, part_pitch(H)};
        const Rows rows = worst(worst(rows_of(H, dtype, x, ldx), rows_of(H, dtype, dy, lddy)),
                                worst(rows_of(H, dtype, dx, H), affine_of(weight)));
        const bool ok = with_dtype(dtype, [&](auto *t) {
            return launch_backward<std::remove_pointer_t<decltype(t)>>(a, rows, sms, part, s);
        });
        if (!ok || launched() != MOE_OK)
            return MOE_ERR_CUDA;
    }
    if (sums) {
        // T == 0: no partial rows, the sums are zero
        const cudaError_t e = with_dtype(w_dtype, [&](auto *t) {
            using E = std::remove_pointer_t<decltype(t)>;
            return launch_reduce<E>(part, H, static_cast<E *>(dweight), static_cast<E *>(dbias), s);
        });
        return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // extern "C"
