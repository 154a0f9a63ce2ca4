// norm.cu -- layer norm over the hidden dimension: forward, the FP8 form that the expert layer
// reads, and backward with the sums of the weight's and the bias's gradients.
//
//   mean = sum(x)/H, rstd = 1/sqrt(sum((x-mean)^2)/H + eps), xh = (x-mean)*rstd, y = xh*g + b
//   a = dy*g:  dx = rstd*(a - mean(a) - xh*mean(a*xh)),  dg = sum_t dy*xh,  db = sum_t dy
//
// All of it is bound by HBM: a row is read once into registers, where both passes of the
// statistics run (the centred second pass keeps the variance free of cancellation), and every
// statistic and sum is held in fp32.
#include <type_traits>

#include "op_common.cuh"
#include "ptx.cuh"

using namespace cpw;

namespace {

constexpr int MAX_H = 16384;   // as moe_create: a row fits one block's registers

// Sum of v over the block, the same in every thread.  `slot` alternates between calls, so one
// barrier a call is enough: a thread that is a call ahead writes the other half of `red`.
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
            r[(threadIdx.x >> 5) * N + i] = v[i];
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = warp_sum(lane < warps ? r[lane * N + i] : 0.0f);
}

template <typename T, int V>
__device__ __forceinline__ void load_affine(float (&f)[V], const void *p, int w32, size_t at)
{
    if (w32) {
        const Pack<float, V> q = load_pack<float, V>(static_cast<const float *>(p) + at);
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] = q.v[i];
    } else {
        const Pack<T, V> q = load_pack<T, V>(static_cast<const T *>(p) + at);
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] = to_f<T>(q.v[i]);
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

// One block a row, VPT packs of V elements a thread; FP8: e4m3 codes and 1x128 scales instead
// of y (V = 8: 16 lanes hold one group of 128).
template <typename T, int V, int VPT, bool FP8>
__global__ void __launch_bounds__(V * VPT == 32 ? 512 : 1024) norm_kernel(const NormArgs a)
{
    __shared__ float red[64];
    const int row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(row) * a.ldx;
    const int packs = a.H / V;
    float f[VPT][V];
    float s[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int p = threadIdx.x + j * blockDim.x;
        if (p < packs) {
            const Pack<T, V> q = load_pack<T, V>(x + static_cast<size_t>(p) * V);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[j][i] = to_f<T>(q.v[i]);
                s[0] += f[j][i];
            }
        }
    }
    block_sum(s, red, 0);
    const float mean = s[0] / static_cast<float>(a.H);
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (static_cast<int>(threadIdx.x + j * blockDim.x) < packs) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[j][i] -= mean;
                s[0] = fmaf(f[j][i], f[j][i], s[0]);
            }
        }
    }
    block_sum(s, red, 1);
    const float rstd = 1.0f / sqrtf(s[0] / static_cast<float>(a.H) + a.eps);
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
        float y[V];
        if (in) {
            float w[V], b[V];
            if (a.weight)
                load_affine<T, V>(w, a.weight, a.w32, static_cast<size_t>(p) * V);
            if (a.bias)
                load_affine<T, V>(b, a.bias, a.w32, static_cast<size_t>(p) * V);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                y[i] = f[j][i] * rstd;
                if (a.weight)
                    y[i] *= w[i];
                if (a.bias)
                    y[i] += b[i];
            }
        }
        if constexpr (FP8) {
            // packs of a group of 128 lie in one half-warp; whole groups are in or out
            float m = 0.0f;
            if (in) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    m = fmaxf(m, fabsf(y[i]));
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            float sf = fmaxf(m, 1e-4f) / 448.0f;
            if (a.pow2) {   // the smallest power of two >= sf (sf is a normal number)
                const uint32_t u = __float_as_uint(sf);
                sf = __uint_as_float((u + 0x7FFFFFu) & 0xFF800000u);
            }
            if (in) {
                uint32_t w01[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t lo = ptx::cvt_e4m3x2(y[4 * h] / sf, y[4 * h + 1] / sf);
                    const uint32_t hi = ptx::cvt_e4m3x2(y[4 * h + 2] / sf, y[4 * h + 3] / sf);
                    w01[h] = lo | (hi << 16);
                }
                *reinterpret_cast<uint2 *>(a.q + static_cast<size_t>(row) * a.H + static_cast<size_t>(p) * V) =
                    make_uint2(w01[0], w01[1]);
                if ((p & 15) == 0)
                    a.sf[static_cast<size_t>(row) * (a.H / 128) + (p >> 4)] = sf;
            }
        } else if (in) {
            Pack<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i)
                o.v[i] = from_f<T>(y[i]);
            store_pack<T, V>(static_cast<T *>(a.y) + static_cast<size_t>(row) * a.H + static_cast<size_t>(p) * V, o);
        }
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
// all of them, so dy and x are read once.
template <typename T, int V, int VPT>
__global__ void __launch_bounds__(V == 1 ? 1024 : VPT == 1 ? 256 : 512) norm_backward_kernel(const NormBwdArgs a)
{
    __shared__ float red[128];
    const int packs = a.H / V;
    float dg[VPT][V], db[VPT][V];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i)
            dg[j][i] = db[j][i] = 0.0f;
    int slot = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, slot ^= 1) {
        const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(row) * a.ldx;
        const T *dy = static_cast<const T *>(a.dy) + static_cast<size_t>(row) * a.lddy;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float xh[VPT][V], g[VPT][V];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int p = threadIdx.x + j * blockDim.x;
            if (p < packs) {
                const Pack<T, V> qx = load_pack<T, V>(x + static_cast<size_t>(p) * V);
                const Pack<T, V> qd = load_pack<T, V>(dy + static_cast<size_t>(p) * V);
                float w[V];
                if (a.weight)
                    load_affine<T, V>(w, a.weight, a.w32, static_cast<size_t>(p) * V);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xh[j][i] = (to_f<T>(qx.v[i]) - mean) * rstd;
                    const float d = to_f<T>(qd.v[i]);
                    dg[j][i] = fmaf(d, xh[j][i], dg[j][i]);
                    db[j][i] += d;
                    g[j][i] = a.weight ? d * w[i] : d;
                    s[0] += g[j][i];
                    s[1] = fmaf(g[j][i], xh[j][i], s[1]);
                }
            }
        }
        block_sum(s, red, slot);
        const float ma = s[0] / static_cast<float>(a.H), mb = s[1] / static_cast<float>(a.H);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int p = threadIdx.x + j * blockDim.x;
            if (p < packs) {
                Pack<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o.v[i] = from_f<T>((g[j][i] - ma - xh[j][i] * mb) * rstd);
                store_pack<T, V>(static_cast<T *>(a.dx) + static_cast<size_t>(row) * a.H + static_cast<size_t>(p) * V, o);
            }
        }
    }
    if (!a.part)
        return;
    float *pg = a.part + static_cast<size_t>(blockIdx.x) * a.H;
    float *pb = pg + static_cast<size_t>(gridDim.x) * a.H;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int p = threadIdx.x + j * blockDim.x;
        if (p < packs) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                pg[static_cast<size_t>(p) * V + i] = dg[j][i];
                pb[static_cast<size_t>(p) * V + i] = db[j][i];
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

template <typename T, bool FP8>
void launch_norm(const NormArgs &a, bool packed, int num_sms, cudaStream_t s)
{
    if (packed) {
        const int packs = a.H / 8;
        // few rows: as many threads as a row has packs (latency); many rows: four packs a thread
        // so that each keeps 64 bytes of loads in flight (bandwidth)
        if (a.T <= 4 * num_sms && packs <= 1024)
            norm_kernel<T, 8, 1, FP8><<<a.T, round32(packs), 0, s>>>(a);
        else
            norm_kernel<T, 8, 4, FP8><<<a.T, round32((packs + 3) / 4), 0, s>>>(a);
    } else if constexpr (!FP8) {
        if (a.H <= 4096)
            norm_kernel<T, 1, 4, false><<<a.T, round32((a.H + 3) / 4), 0, s>>>(a);
        else
            norm_kernel<T, 1, 16, false><<<a.T, round32((a.H + 15) / 16), 0, s>>>(a);
    }
}

// Blocks of the backward kernel: each keeps one row of partial sums.
int backward_blocks(int T, int num_sms)
{
    const int most = 2 * num_sms;
    return T < most ? T : most;
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
    *bytes = 2ull * backward_blocks(T, sms) * static_cast<uint64_t>(H) * sizeof(float);
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
    const int blocks = backward_blocks(T, sms);
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
            if (packed) {
                const int packs = H / 8;
                if (packs <= 256)
                    norm_backward_kernel<E, 8, 1><<<blocks, round32(packs), 0, s>>>(a);
                else if (packs <= 1024)
                    norm_backward_kernel<E, 8, 2><<<blocks, round32((packs + 1) / 2), 0, s>>>(a);
                else
                    norm_backward_kernel<E, 8, 4><<<blocks, round32((packs + 3) / 4), 0, s>>>(a);
            } else if (H <= 4096) {
                norm_backward_kernel<E, 1, 4><<<blocks, round32((H + 3) / 4), 0, s>>>(a);
            } else {
                norm_backward_kernel<E, 1, 16><<<blocks, round32((H + 15) / 16), 0, s>>>(a);
            }
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
