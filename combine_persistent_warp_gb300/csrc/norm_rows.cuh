// norm_rows.cuh -- what the norms over the hidden dimension (norm.cu, rms_norm.cu) share: rows held
// in registers as pairs, copied ahead, summed over a warp or a block; FP8 scales; column sums.
#pragma once

#include <type_traits>

#include "moe_internal.cuh"
#include "op_common.cuh"
#include "ptx.cuh"

namespace cpw {

constexpr int MAX_H = 16384;   // as moe_create: a row fits one block's registers
constexpr int ROW_WARPS = 4;   // rows of a block in the kernels of one row a warp

// ------------------------------------------------------------------ a thread's part of a row ----
// VPT packs of V elements (V = 8: 16-byte accesses; V = 1: any alignment), pack j at position
// t + j * step of the row for thread t of the `step` threads that share it; held as pairs.
template <int V, int VPT>
constexpr int PAIRS = V * VPT / 2;

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

// What is past the row's ends is zeros.
template <typename T, int V, int VPT, bool LEAD = false>
__device__ __forceinline__ void fetch(Pack<T, V> (&q)[VPT], const T *row, int t, int step, int packs, int lead = 0, int H = 0)
{
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int p = t + j * step;
        const long long e = static_cast<long long>(p) * V - lead;
        if (p < packs && (!LEAD || (e >= 0 && e + V <= H))) {
            q[j] = load_pack<T, V, false>(row + e);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                q[j].v[i] = LEAD && p < packs && e + i >= 0 && e + i < H ? row[e + i] : from_f<T>(0.0f);
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
            h[j] = load_halves<false>(p + c, c >= N - 1 && c + 2 * N <= H);
        }
#pragma unroll
        for (int j = 0; j < VPT * M; ++j) {
            const int c = (t + j / M * step) * V - lead + j % M * N;
            Pack<W, N> u = shifted(h[j], p + c);
            if (!(c >= N - 1 && c + 2 * N <= H) && c + N > 0 && c < H) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    u.v[i] = c + i >= 0 && c + i < H ? p[c + i] : from_f<W>(0.0f);
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

// A row's e4m3 codes and 1x128 scales from the thread's elements of it.
template <int V, int VPT>
__device__ __forceinline__ void put_fp8(uint8_t *q, float *sf, const float2 (&f)[PAIRS<V, VPT>], int t, int step, int packs, int pow2)
{
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
    fp8_scales(m, r, sf, t, step, packs, pow2);
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
            *reinterpret_cast<uint2 *>(q + static_cast<size_t>(p) * V) = make_uint2(code[0], code[1]);
        }
    }
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
        int b = threadIdx.y;
        const auto add = [&](auto count) {   // so many loads at a time
            constexpr int N = decltype(count)::value;
            for (; b + 32 * (N - 1) < p.blocks; b += 32 * N) {
                float v[N];
#pragma unroll
                for (int i = 0; i < N; ++i)
                    v[i] = src[static_cast<size_t>(b + 32 * i) * p.pitch + col + (((b + 32 * i) * p.step) & (p.boundary - 1))];
#pragma unroll
                for (int i = 0; i < N; ++i)
                    s += v[i];
            }
        };
        add(std::integral_constant<int, 8>());
        add(std::integral_constant<int, 4>());
        add(std::integral_constant<int, 1>());
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
    cfg.gridDim = dim3((H + 31) / 32, dbias ? 2 : 1);
    cfg.blockDim = dim3(32, 32);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_reduce_kernel<TW>, p, H, dweight, dbias);
}

inline int round32(int v) { return (v + 31) / 32 * 32; }

// How rows move.  PACKED: every row starts on a 16-byte boundary and has whole packs of 8 elements.
// PHASED: packs too, where rows start off the boundaries (or end inside a pack) but the same row of
// every tensor at the same place past one: rows a multiple of 8 apart then have one lead, so with such
// a stride a block's columns stay and only its packs' ends differ.  ANY: element by element
// (neighbouring lanes on neighbouring elements).
enum Rows { PACKED, PHASED, ANY };
inline Rows rows_of(int H, int dtype, const void *p, long long ld)
{
    const size_t b = dtype_bytes(dtype);
    if (!op_aligned(p, 16) || static_cast<size_t>(ld - H) * b % 16 != 0 || H < 8)
        return ANY;
    return H % 8 == 0 ? PACKED : PHASED;
}
inline Rows worst(Rows a, Rows b) { return a > b ? a : b; }
// weight or bias
inline Rows affine_of(const void *p) { return p == nullptr || op_aligned(p, 16) ? PACKED : PHASED; }
// Packs of a row, at most.
template <typename T>
int most_packs(int H, Rows rows)
{
    return rows == PACKED ? H / 8 : (H + 16 / static_cast<int>(sizeof(T)) - 1 + 7) / 8;
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
inline int ring_grid(int per_sm, int num_sms) { return per_sm * num_sms / 8 * 8; }

// Blocks of one-row-a-warp kernels: a warp for each row up to `per_sm` blocks an SM.
inline int warp_blocks(int T, int per_sm, int num_sms)
{
    const int need = (T + ROW_WARPS - 1) / ROW_WARPS, most = per_sm * num_sms;
    return need < most ? need : most;
}

// Floats of a row of partial sums: whole packs after any lead.
inline int part_pitch(int H) { return (H + 7 + 7) / 8 * 8; }

}  // namespace cpw
