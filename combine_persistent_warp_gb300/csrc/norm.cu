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

// V elements as V / 2 pairs (V = 1: one pair whose second value is not used).
template <int V>
constexpr int PAIRS = V == 1 ? 1 : V / 2;

template <typename T, int V>
__device__ __forceinline__ void unpack(float2 (&f)[PAIRS<V>], const Pack<T, V> &q)
{
    if constexpr (V == 1) {
        f[0] = make_float2(to_f<T>(q.v[0]), 0.0f);
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const uint32_t *u = reinterpret_cast<const uint32_t *>(&q);
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            f[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            f[i] = make_float2(to_f<T>(q.v[2 * i]), to_f<T>(q.v[2 * i + 1]));
    }
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float2 (&f)[PAIRS<V>])
{
    Pack<T, V> q;
    if constexpr (V == 1) {
        q.v[0] = from_f<T>(f[0].x);
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            *reinterpret_cast<__nv_bfloat162 *>(&q.v[2 * i]) = __float22bfloat162_rn(f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            q.v[2 * i] = from_f<T>(f[i].x);
            q.v[2 * i + 1] = from_f<T>(f[i].y);
        }
    }
    return q;
}

// A weight's or bias's V values (`none` where there is no such vector).
template <typename T, int V>
__device__ __forceinline__ void load_affine(float2 (&f)[PAIRS<V>], const void *p, int w32, size_t at, float none)
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < PAIRS<V>; ++i)
            f[i] = both(none);
    } else if (w32) {
        unpack<float, V>(f, load_pack<float, V>(static_cast<const float *>(p) + at));
    } else {
        unpack<T, V>(f, load_pack<T, V>(static_cast<const T *>(p) + at));
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
template <typename T, int V>
__device__ __forceinline__ void copy_ahead(Pack<T, V> *slot, const T *src)
{
    constexpr int BYTES = static_cast<int>(sizeof(Pack<T, V>));
    const uint32_t dst = ptx::smem_u32(slot);
    if constexpr (BYTES >= 16) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * i),
                         "l"(reinterpret_cast<uint64_t>(src) + 16 * i)
                         : "memory");
    } else {
        static_assert(BYTES == 4, "copies of 4 or 16 bytes");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
    }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
constexpr int AHEAD = 4;   // ring stages

// Row r's packs of this thread into ring stage g (nothing past the last row).
template <typename T, int V, int VPT>
__device__ __forceinline__ void fetch_row(Pack<T, V> *ring, int g, const void *base, long long ld, int r, int T_, int packs)
{
    if (r < T_) {
        const T *x = static_cast<const T *>(base) + static_cast<size_t>(r) * ld;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int p = threadIdx.x + j * blockDim.x;
            if (p < packs)
                copy_ahead<T, V>(ring + (g * VPT + j) * blockDim.x + threadIdx.x, x + static_cast<size_t>(p) * V);
        }
    }
}

// ------------------------------------------------------------------ forward -------------
// The row held in f (zeros in packs past its end), its statistics and outputs; w and b: the
// thread's columns of weight and bias.  FP8: e4m3 codes and 1x128 scales instead of y (V = 8: 16
// lanes hold one group of 128).  `after_read` runs once every thread has its row in registers.
template <typename T, int V, int VPT, bool FP8, typename F>
__device__ __forceinline__ void norm_row(const NormArgs &a, int row, float2 (&f)[VPT][PAIRS<V>], const float2 (&w)[VPT][PAIRS<V>],
                                         const float2 (&b)[VPT][PAIRS<V>], float *red, F after_read)
{
    constexpr int P = PAIRS<V>;
    const int packs = a.H / V;
    const float inv = 1.0f / static_cast<float>(a.H);
    float2 acc = both(0.0f);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i)
            acc = add2(acc, f[j][i]);
    float s[1] = {acc.x + acc.y};
    block_sum(s, red, 0);
    after_read();
    const float mean = s[0] * inv;
    acc = both(0.0f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (static_cast<int>(threadIdx.x + j * blockDim.x) < packs) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                f[j][i] = add2(f[j][i], make_float2(-mean, V == 1 ? 0.0f : -mean));
                acc = fma2(f[j][i], f[j][i], acc);
            }
        }
    }
    s[0] = acc.x + acc.y;
    block_sum(s, red, 1);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean)
            a.mean[row] = mean;
        if (a.rstd)
            a.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int p = threadIdx.x + j * blockDim.x;
        const bool in = p < packs;
        float2 y[P];
#pragma unroll
        for (int i = 0; i < P; ++i)
            y[i] = fma2(mul2(f[j][i], both(rstd)), w[j][i], b[j][i]);
        if constexpr (FP8) {
            // packs of a group of 128 lie in one half-warp; whole groups are in or out
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i)
                m = fmaxf(m, fmaxf(fabsf(y[i].x), fabsf(y[i].y)));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            float sf = fmaxf(m, 1e-4f) / 448.0f;
            if (a.pow2) {   // the smallest power of two >= sf (sf is a normal number)
                const uint32_t u = __float_as_uint(sf);
                sf = __uint_as_float((u + 0x7FFFFFu) & 0xFF800000u);
            }
            if (in) {
                uint32_t code[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    code[h] = ptx::cvt_e4m3x2(y[2 * h].x / sf, y[2 * h].y / sf) |
                              (ptx::cvt_e4m3x2(y[2 * h + 1].x / sf, y[2 * h + 1].y / sf) << 16);
                *reinterpret_cast<uint2 *>(a.q + static_cast<size_t>(row) * a.H + static_cast<size_t>(p) * V) =
                    make_uint2(code[0], code[1]);
                if ((p & 15) == 0)
                    a.sf[static_cast<size_t>(row) * (a.H / 128) + (p >> 4)] = sf;
            }
        } else if (in) {
            store_pack<T, V>(static_cast<T *>(a.y) + static_cast<size_t>(row) * a.H + static_cast<size_t>(p) * V, pack<T, V>(y));
        }
    }
}

template <typename T, int V, int VPT>
__device__ __forceinline__ void load_columns(float2 (&w)[VPT][PAIRS<V>], const void *p, int w32, int packs, float none)
{
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int at = threadIdx.x + j * blockDim.x;
        load_affine<T, V>(w[j], at < packs ? p : nullptr, w32, static_cast<size_t>(at) * V, none);
    }
}

// One block a row.  The weight and bias are loaded beside the row, ahead of its sums.
template <typename T, int V, int VPT, bool FP8>
__global__ void __launch_bounds__(V * VPT == 32 || V * VPT == 8 && V == 1 ? 512 : 1024) norm_kernel(const NormArgs a)
{
    __shared__ __align__(16) float red[64];
    const int packs = a.H / V;
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(blockIdx.x) * a.ldx;
    clear_sums<1>(red);
    float2 f[VPT][PAIRS<V>], w[VPT][PAIRS<V>], b[VPT][PAIRS<V>];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int p = threadIdx.x + j * blockDim.x;
        if (p < packs) {
            unpack<T, V>(f[j], load_pack<T, V>(x + static_cast<size_t>(p) * V));
        } else {
#pragma unroll
            for (int i = 0; i < PAIRS<V>; ++i)
                f[j][i] = both(0.0f);
        }
    }
    load_columns<T, V, VPT>(w, a.weight, a.w32, packs, 1.0f);
    load_columns<T, V, VPT>(b, a.bias, a.w32, packs, 0.0f);
    norm_row<T, V, VPT, FP8>(a, blockIdx.x, f, w, b, red, [] {});
}

// Persistent blocks: rows copied AHEAD rows before their use, weight and bias kept in registers.
template <typename T, int V, int VPT, bool FP8>
__global__ void __launch_bounds__(512) norm_ring_kernel(const NormArgs a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[64];
    Pack<T, V> *ring = reinterpret_cast<Pack<T, V> *>(smem);
    const int packs = a.H / V;
#pragma unroll
    for (int g = 0; g < AHEAD; ++g) {
        fetch_row<T, V, VPT>(ring, g, a.x, a.ldx, blockIdx.x + g * gridDim.x, a.T, packs);
        copies_commit();
    }
    clear_sums<1>(red);
    float2 w[VPT][PAIRS<V>], b[VPT][PAIRS<V>];
    load_columns<T, V, VPT>(w, a.weight, a.w32, packs, 1.0f);
    load_columns<T, V, VPT>(b, a.bias, a.w32, packs, 0.0f);
    int g = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x) {
        copies_wait<AHEAD - 1>();
        float2 f[VPT][PAIRS<V>];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (static_cast<int>(threadIdx.x + j * blockDim.x) < packs) {
                unpack<T, V>(f[j], ring[(g * VPT + j) * blockDim.x + threadIdx.x]);
            } else {
#pragma unroll
                for (int i = 0; i < PAIRS<V>; ++i)
                    f[j][i] = both(0.0f);
            }
        }
        norm_row<T, V, VPT, FP8>(a, row, f, w, b, red, [&] {
            fetch_row<T, V, VPT>(ring, g, a.x, a.ldx, row + AHEAD * gridDim.x, a.T, packs);
            copies_commit();
        });
        g = g == AHEAD - 1 ? 0 : g + 1;
    }
}

struct NormBwdArgs {
    int T, H;
    const void *dy, *x;
    long long lddy, ldx;
    const void *weight;
    int w32;
    const float *mean, *rstd;
    void *dx;
    float *part;   // [2][blocks][H] sums of dy*xh and of dy over each block's rows
};

// Block b takes rows b, b + blocks, ...: a thread keeps its columns' two sums in registers over
// all of them, so dy and x are read once.  RING: rows of x and dy copied AHEAD rows before use.
template <typename T, int V, int VPT, bool RING>
__global__ void __launch_bounds__(V == 1 && VPT == 16 ? 1024 : 512) norm_backward_kernel(const NormBwdArgs a)
{
    constexpr int P = PAIRS<V>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[128];
    const int packs = a.H / V;
    const float inv = 1.0f / static_cast<float>(a.H);
    Pack<T, V> *ring_x = reinterpret_cast<Pack<T, V> *>(smem), *ring_d = ring_x + AHEAD * VPT * blockDim.x;
    if constexpr (RING) {
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) {
            fetch_row<T, V, VPT>(ring_x, g, a.x, a.ldx, blockIdx.x + g * gridDim.x, a.T, packs);
            fetch_row<T, V, VPT>(ring_d, g, a.dy, a.lddy, blockIdx.x + g * gridDim.x, a.T, packs);
            copies_commit();
        }
    }
    clear_sums<2>(red);
    float2 w[VPT][P], dg[VPT][P], db[VPT][P];
    load_columns<T, V, VPT>(w, a.weight, a.w32, packs, 1.0f);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i)
            dg[j][i] = db[j][i] = both(0.0f);
    int slot = 0, stage = 0;
    float mean = 0.0f, rstd = 0.0f;
    if (static_cast<int>(blockIdx.x) < a.T) {
        mean = a.mean[blockIdx.x];
        rstd = a.rstd[blockIdx.x];
    }
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, slot ^= 1) {
        const int next = row + gridDim.x;
        const float mean1 = next < a.T ? a.mean[next] : 0.0f, rstd1 = next < a.T ? a.rstd[next] : 0.0f;
        if constexpr (RING)
            copies_wait<AHEAD - 1>();
        float2 xh[VPT][P], g[VPT][P];
        float2 s0 = both(0.0f), s1 = both(0.0f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int p = threadIdx.x + j * blockDim.x;
            if (p < packs) {
                float2 d[P];
                if constexpr (RING) {
                    unpack<T, V>(xh[j], ring_x[(stage * VPT + j) * blockDim.x + threadIdx.x]);
                    unpack<T, V>(d, ring_d[(stage * VPT + j) * blockDim.x + threadIdx.x]);
                } else {
                    unpack<T, V>(xh[j], load_pack<T, V>(static_cast<const T *>(a.x) + static_cast<size_t>(row) * a.ldx + static_cast<size_t>(p) * V));
                    unpack<T, V>(d, load_pack<T, V>(static_cast<const T *>(a.dy) + static_cast<size_t>(row) * a.lddy + static_cast<size_t>(p) * V));
                }
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    xh[j][i] = mul2(add2(xh[j][i], both(-mean)), both(rstd));
                    dg[j][i] = fma2(d[i], xh[j][i], dg[j][i]);
                    db[j][i] = add2(db[j][i], d[i]);
                    g[j][i] = mul2(d[i], w[j][i]);
                    s0 = add2(s0, g[j][i]);
                    s1 = fma2(g[j][i], xh[j][i], s1);
                }
            }
        }
        // (V = 1: the second values of d are zeros, and so are all products with them)
        float s[2] = {s0.x + s0.y, s1.x + s1.y};
        block_sum(s, red, slot);
        if constexpr (RING) {   // every value read above has been used in the sums
            fetch_row<T, V, VPT>(ring_x, stage, a.x, a.ldx, row + AHEAD * gridDim.x, a.T, packs);
            fetch_row<T, V, VPT>(ring_d, stage, a.dy, a.lddy, row + AHEAD * gridDim.x, a.T, packs);
            copies_commit();
            stage = stage == AHEAD - 1 ? 0 : stage + 1;
        }
        const float2 ma = both(-s[0] * inv), mb = both(-s[1] * inv);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int p = threadIdx.x + j * blockDim.x;
            if (p < packs) {
                float2 o[P];
#pragma unroll
                for (int i = 0; i < P; ++i)
                    o[i] = mul2(fma2(xh[j][i], mb, add2(g[j][i], ma)), both(rstd));
                store_pack<T, V>(static_cast<T *>(a.dx) + static_cast<size_t>(row) * a.H + static_cast<size_t>(p) * V, pack<T, V>(o));
            }
        }
        mean = mean1;
        rstd = rstd1;
    }
    if (!a.part)
        return;
    float *pg = a.part + static_cast<size_t>(blockIdx.x) * a.H;
    float *pb = pg + static_cast<size_t>(gridDim.x) * a.H;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int p = threadIdx.x + j * blockDim.x;
        if (p < packs) {
            if constexpr (V == 1) {
                pg[p] = dg[j][0].x;
                pb[p] = db[j][0].x;
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    *reinterpret_cast<float2 *>(pg + static_cast<size_t>(p) * V + 2 * i) = dg[j][i];
                    *reinterpret_cast<float2 *>(pb + static_cast<size_t>(p) * V + 2 * i) = db[j][i];
                }
            }
        }
    }
}

// Column sums of the partial sums, in a fixed order: a block of 32 columns x 32 row lanes.
template <typename TW>
__global__ void norm_reduce_kernel(const float *part, int blocks, int H, TW *dweight, TW *dbias)
{
    __shared__ float tile[32][33];
    const float *src = part + static_cast<size_t>(blockIdx.y) * blocks * H;
    TW *dst = blockIdx.y == 0 ? dweight : dbias;
    if (!dst)
        return;
    const int col = blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (col < H) {
#pragma unroll 4
        for (int b = threadIdx.y; b < blocks; b += 32)
            s += src[static_cast<size_t>(b) * H + col];
    }
    tile[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = warp_sum(tile[threadIdx.x][threadIdx.y]);
    const int out = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && out < H)
        dst[out] = from_f<TW>(s);
}

int round32(int v) { return (v + 31) / 32 * 32; }

// Rows whose H elements and addresses allow 16-byte accesses move as packs of 8 elements, others
// an element at a time (neighbouring lanes on neighbouring elements).
bool packed_rows(int H, int dtype, const void *p, long long ld)
{
    const size_t b = dtype_bytes(dtype);
    return H % 8 == 0 && op_aligned(p, 16) && static_cast<size_t>(ld) * b % 16 == 0;
}
bool packed_affine(const void *p) { return p == nullptr || op_aligned(p, 16); }

bool norm_args_ok(int T, int H, int dtype, int w_dtype, const void *weight, const void *bias)
{
    if (T < 0 || H < 1 || H > MAX_H || !dtype_ok(dtype))
        return false;
    if ((weight || bias) && w_dtype != dtype && w_dtype != MOE_F32)
        return false;
    const size_t wb = dtype_bytes(w_dtype);
    return op_aligned(weight, wb) && op_aligned(bias, wb);
}

// Persistent blocks an SM: about 512 threads, each with rows on their way.
int ring_blocks_per_sm(int threads)
{
    const int n = 512 / threads;
    return n < 1 ? 1 : n > 8 ? 8 : n;
}

// Shared memory of a block's ring, and whether its blocks fit an SM.
size_t ring_bytes(int threads, int vpt, size_t pack_bytes, int tensors)
{
    return static_cast<size_t>(AHEAD) * vpt * threads * pack_bytes * tensors;
}
bool ring_fits(size_t bytes, int per_sm) { return bytes * per_sm <= 200 * 1024; }

template <typename K>
bool allow_smem(K kern, size_t bytes)
{
    return bytes <= 48 * 1024 ||
           ensure_max_dynamic_smem(reinterpret_cast<const void *>(kern), static_cast<int>(bytes)) == cudaSuccess;
}

template <typename T, int V, int VPT, bool FP8>
bool try_norm_ring(const NormArgs &a, int num_sms, cudaStream_t s)
{
    const int threads = round32((a.H / V + VPT - 1) / VPT);
    if (threads > 512)
        return false;
    const int per_sm = ring_blocks_per_sm(threads);
    const size_t smem = ring_bytes(threads, VPT, sizeof(Pack<T, V>), 1);
    // long batches only: every block has rows to copy ahead of
    if (a.T < AHEAD * per_sm * num_sms || !ring_fits(smem, per_sm))
        return false;
    const auto kern = norm_ring_kernel<T, V, VPT, FP8>;
    if (!allow_smem(kern, smem))
        return false;
    kern<<<per_sm * num_sms, threads, smem, s>>>(a);
    return true;
}

template <typename T, bool FP8>
void launch_norm(const NormArgs &a, bool packed, int num_sms, cudaStream_t s)
{
    if (packed) {
        const int packs = a.H / 8;
        if (try_norm_ring<T, 8, 4, FP8>(a, num_sms, s))
            return;
        // few rows: as many threads as a row has packs (latency); else four packs a thread
        if (a.T <= 4 * num_sms && packs <= 1024)
            norm_kernel<T, 8, 1, FP8><<<a.T, round32(packs), 0, s>>>(a);
        else
            norm_kernel<T, 8, 4, FP8><<<a.T, round32((packs + 3) / 4), 0, s>>>(a);
    } else if constexpr (!FP8) {
        if constexpr (sizeof(T) == 4)
            if (try_norm_ring<T, 1, 8, false>(a, num_sms, s))
                return;
        if (a.H <= 4096)
            norm_kernel<T, 1, 8, false><<<a.T, round32((a.H + 7) / 8), 0, s>>>(a);
        else
            norm_kernel<T, 1, 16, false><<<a.T, round32((a.H + 15) / 16), 0, s>>>(a);
    }
}

// Blocks of the backward kernel: each keeps one row of partial sums.
int backward_blocks(int T, int H, int num_sms)
{
    const int most = ring_blocks_per_sm(H >= 8192 ? 512 : H >= 1024 ? 256 : 128) * num_sms;
    return T < most ? T : most;
}

template <typename T, int V, int VPT>
void launch_backward(const NormBwdArgs &a, int blocks, cudaStream_t s)
{
    const int threads = round32((a.H / V + VPT - 1) / VPT);
    if constexpr (sizeof(Pack<T, V>) >= 4) {
        const size_t smem = ring_bytes(threads, VPT, sizeof(Pack<T, V>), 2);
        const auto kern = norm_backward_kernel<T, V, VPT, true>;
        if (a.T >= AHEAD * blocks && smem <= 100 * 1024 && allow_smem(kern, smem)) {
            kern<<<blocks, threads, smem, s>>>(a);
            return;
        }
    }
    norm_backward_kernel<T, V, VPT, false><<<blocks, threads, 0, s>>>(a);
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
    const bool packed = packed_rows(H, dtype, x, ldx) && op_aligned(y, 16) && packed_affine(weight) && packed_affine(bias);
    with_dtype(dtype, [&](auto *t) {
        launch_norm<std::remove_pointer_t<decltype(t)>, false>(a, packed, sms, static_cast<cudaStream_t>(stream));
    });
    return launched();
}

int moe_layer_norm_fp8(int T, int H, const void *x, int64_t ldx, int dtype, const void *weight, const void *bias,
                       int w_dtype, float eps, int pow2_scales, uint8_t *q, float *sf, void *stream)
{
    if (!norm_args_ok(T, H, dtype, w_dtype, weight, bias) || ldx < H || !(eps >= 0.0f) || H % 128 != 0 ||
        pow2_scales < 0 || pow2_scales > 1)
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    if (!x || !q || !sf || !packed_rows(H, dtype, x, ldx) || !op_aligned(q, 16) || !op_aligned(sf, 4) ||
        !packed_affine(weight) || !packed_affine(bias))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const NormArgs a{T, H, x, ldx, weight, bias, w_dtype == MOE_F32 && dtype != MOE_F32, eps, nullptr, nullptr, nullptr, q, sf, pow2_scales};
    with_dtype(dtype, [&](auto *t) {
        launch_norm<std::remove_pointer_t<decltype(t)>, true>(a, true, sms, static_cast<cudaStream_t>(stream));
    });
    return launched();
}

int moe_layer_norm_backward_workspace(int T, int H, uint64_t *bytes)
{
    if (T < 0 || H < 1 || H > MAX_H || !bytes)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    *bytes = 2ull * backward_blocks(T, H, sms) * static_cast<uint64_t>(H) * sizeof(float);
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
    const int blocks = backward_blocks(T, H, sms);
    const bool sums = dweight || dbias;
    if (sums && T > 0 &&
        (!workspace || !op_aligned(workspace, 16) || workspace_bytes < 2ull * blocks * static_cast<uint64_t>(H) * sizeof(float)))
        return MOE_ERR_INVALID_ARG;
    if (T > 0) {
        const NormBwdArgs a{T, H, dy, x, lddy, ldx, weight, w_dtype == MOE_F32 && dtype != MOE_F32, mean, rstd, dx,
                            sums ? static_cast<float *>(workspace) : nullptr};
        const bool packed = packed_rows(H, dtype, x, ldx) && packed_rows(H, dtype, dy, lddy) && op_aligned(dx, 16) &&
                            packed_affine(weight);
        with_dtype(dtype, [&](auto *t) {
            using E = std::remove_pointer_t<decltype(t)>;
            if (packed && H <= 8192)
                launch_backward<E, 8, 2>(a, blocks, s);
            else if (packed)
                launch_backward<E, 8, 4>(a, blocks, s);
            else if (H <= 4096)
                launch_backward<E, 1, 8>(a, blocks, s);
            else
                launch_backward<E, 1, 16>(a, blocks, s);
        });
        const int rc = launched();
        if (rc != MOE_OK)
            return rc;
    }
    if (sums) {
        // T == 0: no partial rows, the sums are zero
        with_dtype(w_dtype, [&](auto *t) {
            using E = std::remove_pointer_t<decltype(t)>;
            norm_reduce_kernel<E><<<dim3((H + 31) / 32, 2), dim3(32, 32), 0, s>>>(
                static_cast<const float *>(workspace), blocks, H, static_cast<E *>(dweight), static_cast<E *>(dbias));
        });
        return launched();
    }
    return MOE_OK;
}

}  // extern "C"
