// rms_norm.cu -- RMS norm over the hidden dimension with the residual's addition: forward, the FP8 form
// that the expert layer reads, and backward with the sums of the weight's gradient.
//
//   h = x + r (rounded to their type: it is the residual stream), rstd = 1/sqrt(sum(h^2)/H + eps), y = h rstd g
//   a = dy g, xh = h rstd:  dx = dh + rstd (a - xh mean(a xh))  (of x and of r alike),  dg = sum_t dy xh
//
// Bound by HBM: every row is read once into registers and its sum of squares held in fp32.
#include "norm_rows.cuh"

using namespace cpw;

namespace {

struct RmsArgs {
    int T, H;
    const void *x, *r;   // r: null without a residual
    long long ldx, ldr;
    const void *weight;  // may be null
    int w32;             // weight is fp32 (else x's type)
    float eps;
    void *h;             // [T][H] the sum (with a residual)
    void *y;
    float *rstd;         // may be null
    uint8_t *q;          // FP8 form
    float *sf;
    int pow2;
};

// ------------------------------------------------------------------ forward -------------
// The row held in f (zeros past its end): its statistic and outputs; w: the thread's columns of the weight.
template <typename T, int V, int VPT, bool FP8, bool WARP>
__device__ __forceinline__ void rms_row(const RmsArgs &a, int row, float2 (&f)[PAIRS<V, VPT>], const float2 (&w)[PAIRS<V, VPT>], float *red)
{
    constexpr int P = PAIRS<V, VPT>;
    const int packs = a.H / V, t = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
    float2 acc = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i)
        acc = fma2(f[i], f[i], acc);
    float s[1] = {acc.x + acc.y};
    row_sum<WARP>(s, red, 0);
    const float rstd = 1.0f / sqrtf(s[0] / static_cast<float>(a.H) + a.eps);
    if (t == 0 && a.rstd)
        a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < P; ++i)
        f[i] = mul2(mul2(f[i], both(rstd)), w[i]);
    if constexpr (FP8)
        put_fp8<V, VPT>(a.q + static_cast<size_t>(row) * a.H, a.sf + static_cast<size_t>(row) * (a.H / 128), f, t, step, packs, a.pow2);
    else
        put<T, V, VPT>(static_cast<T *>(a.y) + static_cast<size_t>(row) * a.H, f, t, step, packs);
}

// x + r in x's type, as the stream keeps it.
template <typename T, int V, int VPT>
__device__ __forceinline__ void add_residual(float2 (&f)[PAIRS<V, VPT>], const Pack<T, V> (&q)[VPT])
{
    float2 r[PAIRS<V, VPT>];
    unpack<T, V, VPT>(r, q);
#pragma unroll
    for (int i = 0; i < PAIRS<V, VPT>; ++i) {
        const float2 v = add2(f[i], r[i]);
        f[i] = make_float2(to_f<T>(from_f<T>(v.x)), to_f<T>(from_f<T>(v.y)));
    }
}

// One row a block; or (WARP, rows of at most 1024 elements) one row a warp.
template <typename T, int V, int VPT, bool FP8, bool WARP>
__global__ void __launch_bounds__(WARP ? ROW_WARPS * 32 : V * VPT == 32 ? 512 : 1024) rms_kernel(const RmsArgs a)
{
    constexpr int P = PAIRS<V, VPT>;
    __shared__ __align__(16) float red[WARP ? 4 : 64];
    const int packs = a.H / V, t = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
    if constexpr (!WARP)
        clear_sums<1>(red);
    const int row = WARP ? blockIdx.x * ROW_WARPS + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.T)
        return;
    Pack<T, V> q[VPT];
    float2 f[P], w[P];
    fetch<T, V, VPT>(q, static_cast<const T *>(a.x) + static_cast<size_t>(row) * a.ldx, t, step, packs);
    unpack<T, V, VPT>(f, q);
    if (a.r) {
        fetch<T, V, VPT>(q, static_cast<const T *>(a.r) + static_cast<size_t>(row) * a.ldr, t, step, packs);
        add_residual<T, V, VPT>(f, q);
        put<T, V, VPT>(static_cast<T *>(a.h) + static_cast<size_t>(row) * a.H, f, t, step, packs);
    }
    load_columns<T, V, VPT>(w, a.weight, a.w32, 1.0f, t, step, packs);
    rms_row<T, V, VPT, FP8, WARP>(a, row, f, w, red);
}

// ------------------------------------------------------------------ backward ------------
struct RmsBwdArgs {
    int T, H;
    const void *dy, *h, *dh;   // dh may be null
    long long lddy, ldh, lddh;
    const void *weight;
    int w32;
    const float *rstd;
    void *dx;
    float *part;   // [blocks][pitch] sums of dy*xh over each block's rows (null: not wanted)
    int pitch;
};

// Rows b, b + blocks, ... of block b: a thread keeps its columns' sums in registers over all of them.
template <typename T, int V, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 : 512) rms_backward_kernel(const RmsBwdArgs a)
{
    constexpr int P = PAIRS<V, VPT>;
    __shared__ __align__(16) float red[64];
    const int t = threadIdx.x, step = blockDim.x, packs = a.H / V;
    const float inv = 1.0f / static_cast<float>(a.H);
    clear_sums<1>(red);
    float2 w[P], dg[P];
    load_columns<T, V, VPT>(w, a.weight, a.w32, 1.0f, t, step, packs);
#pragma unroll
    for (int i = 0; i < P; ++i)
        dg[i] = both(0.0f);
    int slot = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, slot ^= 1) {
        const float rstd = a.rstd[row];
        Pack<T, V> q[VPT];
        float2 xh[P], d[P];
        fetch<T, V, VPT>(q, static_cast<const T *>(a.h) + static_cast<size_t>(row) * a.ldh, t, step, packs);
        unpack<T, V, VPT>(xh, q);
        fetch<T, V, VPT>(q, static_cast<const T *>(a.dy) + static_cast<size_t>(row) * a.lddy, t, step, packs);
        unpack<T, V, VPT>(d, q);
        float2 acc = both(0.0f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            xh[i] = mul2(xh[i], both(rstd));
            dg[i] = fma2(d[i], xh[i], dg[i]);
            d[i] = mul2(d[i], w[i]);
            acc = fma2(d[i], xh[i], acc);
        }
        float s[1] = {acc.x + acc.y};
        row_sum<WARP>(s, red, slot);
        const float2 m = both(-s[0] * inv);
#pragma unroll
        for (int i = 0; i < P; ++i)
            d[i] = mul2(fma2(xh[i], m, d[i]), both(rstd));
        if (a.dh) {
            fetch<T, V, VPT>(q, static_cast<const T *>(a.dh) + static_cast<size_t>(row) * a.lddh, t, step, packs);
            unpack<T, V, VPT>(xh, q);
#pragma unroll
            for (int i = 0; i < P; ++i)
                d[i] = add2(d[i], xh[i]);
        }
        put<T, V, VPT>(static_cast<T *>(a.dx) + static_cast<size_t>(row) * a.H, d, t, step, packs);
    }
    if (a.part)
        put<float, V, VPT>(a.part + static_cast<size_t>(blockIdx.x) * a.pitch, dg, t, step, packs);
    ptx::launch_dependents();
}

// ------------------------------------------------------------------ host side ------------
template <typename T, bool FP8>
void launch_rms(const RmsArgs &a, Rows rows, cudaStream_t s)
{
    const int packs = a.H / 8, warps = (a.T + ROW_WARPS - 1) / ROW_WARPS;
    if (rows == PACKED) {
        if (packs <= 128)
            rms_kernel<T, 8, 4, FP8, true><<<warps, ROW_WARPS * 32, 0, s>>>(a);
        else
            rms_kernel<T, 8, 4, FP8, false><<<a.T, round32((packs + 3) / 4), 0, s>>>(a);
        return;
    }
    if constexpr (!FP8) {
        if (a.H <= 1024)
            rms_kernel<T, 1, 32, false, true><<<warps, ROW_WARPS * 32, 0, s>>>(a);
        else
            rms_kernel<T, 1, 32, false, false><<<a.T, round32((a.H + 31) / 32), 0, s>>>(a);
    }
}

int backward_blocks(int T, int num_sms) { return T < 2 * num_sms ? T : 2 * num_sms; }

template <typename T>
void launch_rms_backward(const RmsBwdArgs &a, Rows rows, int blocks, cudaStream_t s)
{
    const int packs = a.H / 8;
    if (rows == PACKED)
        rms_backward_kernel<T, 8, 4, false><<<blocks, round32((packs + 3) / 4), 0, s>>>(a);
    else
        rms_backward_kernel<T, 1, 32, false><<<blocks, round32((a.H + 31) / 32), 0, s>>>(a);
}

bool sizes_ok(int T, int H, int dtype, int w_dtype, const void *weight)
{
    return T >= 0 && T <= MAX_ROWS && H >= 1 && H <= MAX_H && dtype_ok(dtype) && (!weight || w_dtype == dtype || w_dtype == MOE_F32) &&
           op_aligned(weight, dtype_bytes(w_dtype));
}
// The forward calls' x, residual and sum.
bool stream_ok(int H, const void *x, int64_t ldx, const void *r, int64_t ldr, const void *h, int dtype)
{
    const size_t b = dtype_bytes(dtype);
    return x && op_aligned(x, b) && op_aligned(r, b) && op_aligned(h, b) && (!r || h) && ldx >= H && (!r || ldr >= H);
}
Rows rows_or_absent(int H, int dtype, const void *p, long long ld) { return p ? rows_of(H, dtype, p, ld) : PACKED; }

}  // namespace

extern "C" {

int moe_rms_norm(int T, int H, const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, const void *weight,
                 int w_dtype, float eps, void *h, void *y, float *rstd, void *stream)
{
    if (!sizes_ok(T, H, dtype, w_dtype, weight) || !(eps >= 0.0f))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    if (!stream_ok(H, x, ldx, residual, ldr, h, dtype) || !y || !op_aligned(y, dtype_bytes(dtype)) || !op_aligned(rstd, 4))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const RmsArgs a{T, H, x, residual, ldx, ldr, weight, w_dtype == MOE_F32 && dtype != MOE_F32, eps, h, y, rstd, nullptr, nullptr, 0};
    const Rows rows = worst(worst(worst(rows_of(H, dtype, x, ldx), rows_or_absent(H, dtype, residual, ldr)),
                                  residual ? rows_of(H, dtype, h, H) : PACKED),
                            worst(rows_of(H, dtype, y, H), affine_of(weight)));
    with_dtype(dtype, [&](auto *t) {
        launch_rms<std::remove_pointer_t<decltype(t)>, false>(a, rows, static_cast<cudaStream_t>(stream));
    });
    return launched();
}

int moe_rms_norm_fp8(int T, int H, const void *x, int64_t ldx, const void *residual, int64_t ldr, int dtype, const void *weight,
                     int w_dtype, float eps, int pow2_scales, void *h, uint8_t *q, float *sf, void *stream)
{
    if (!sizes_ok(T, H, dtype, w_dtype, weight) || !(eps >= 0.0f) || H % 128 != 0 || pow2_scales < 0 || pow2_scales > 1)
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    if (!stream_ok(H, x, ldx, residual, ldr, h, dtype) || !q || !sf || !op_aligned(q, 16) || !op_aligned(sf, 4) ||
        rows_of(H, dtype, x, ldx) != PACKED || rows_or_absent(H, dtype, residual, ldr) != PACKED ||
        (residual && rows_of(H, dtype, h, H) != PACKED) || affine_of(weight) != PACKED)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const RmsArgs a{T, H, x, residual, ldx, ldr, weight, w_dtype == MOE_F32 && dtype != MOE_F32, eps, h, nullptr, nullptr, q, sf, pow2_scales};
    with_dtype(dtype, [&](auto *t) {
        launch_rms<std::remove_pointer_t<decltype(t)>, true>(a, PACKED, static_cast<cudaStream_t>(stream));
    });
    return launched();
}

int moe_rms_norm_backward_workspace(int T, int H, uint64_t *bytes)
{
    if (T < 0 || T > MAX_ROWS || H < 1 || H > MAX_H || !bytes)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    *bytes = static_cast<uint64_t>(backward_blocks(T, sms)) * static_cast<uint64_t>(part_pitch(H)) * sizeof(float);
    return MOE_OK;
}

int moe_rms_norm_backward(int T, int H, const void *dy, int64_t lddy, const void *h, int64_t ldh, const void *dh, int64_t lddh,
                          int dtype, const void *weight, int w_dtype, const float *rstd, void *dx, void *dweight, void *workspace,
                          uint64_t workspace_bytes, void *stream)
{
    if (!sizes_ok(T, H, dtype, w_dtype, weight) || ldh < H || lddy < H || (dh && lddh < H))
        return MOE_ERR_INVALID_ARG;
    if (dweight && ((w_dtype != dtype && w_dtype != MOE_F32) || !op_aligned(dweight, dtype_bytes(w_dtype))))
        return MOE_ERR_INVALID_ARG;
    const size_t b = dtype_bytes(dtype);
    if (T > 0 && (!dy || !h || !rstd || !dx || !op_aligned(dy, b) || !op_aligned(h, b) || !op_aligned(dh, b) || !op_aligned(dx, b) ||
                  !op_aligned(rstd, 4)))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint64_t need = 0;
    if (dweight && T > 0 &&
        (!workspace || !op_aligned(workspace, 16) || moe_rms_norm_backward_workspace(T, H, &need) != MOE_OK || workspace_bytes < need))
        return MOE_ERR_INVALID_ARG;
    PartRows part{};
    if (T > 0) {
        const int blocks = backward_blocks(T, sms);
        const RmsBwdArgs a{T, H, dy, h, dh, lddy, ldh, lddh, weight, w_dtype == MOE_F32 && dtype != MOE_F32, rstd, dx,
                           dweight ? static_cast<float *>(workspace) : nullptr, part_pitch(H)};
        part = {a.part, blocks, a.pitch, 0, 8};
        const Rows rows = worst(worst(worst(rows_of(H, dtype, h, ldh), rows_of(H, dtype, dy, lddy)), rows_or_absent(H, dtype, dh, lddh)),
                                worst(rows_of(H, dtype, dx, H), affine_of(weight)));
        with_dtype(dtype, [&](auto *t) { launch_rms_backward<std::remove_pointer_t<decltype(t)>>(a, rows, blocks, s); });
        if (launched() != MOE_OK)
            return MOE_ERR_CUDA;
    }
    if (dweight) {
        // T == 0: no partial rows, the sums are zero
        const cudaError_t e = with_dtype(w_dtype, [&](auto *t) {
            using E = std::remove_pointer_t<decltype(t)>;
            return launch_reduce<E>(part, H, static_cast<E *>(dweight), static_cast<E *>(nullptr), s);
        });
        return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // extern "C"
