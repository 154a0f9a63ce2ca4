// rms_norm.cu -- RMS norm over the hidden dimension with the residual's addition: forward, the FP8 form
// that the expert layer reads, and backward with the sums of the weight's gradient.
//
//   h = x + r (rounded to their type: it is the residual stream), rstd = 1/sqrt(sum(h^2)/H + eps), y = h rstd g
//   a = dy g, xh = h rstd:  dx = dh + rstd (a - xh mean(a xh))  (of x and of r alike),  dg = sum_t dy xh
//
// Bound by HBM: every row is read once into registers and its sum of squares held in fp32.  Long batches run in
// persistent blocks that copy the rows ahead into shared memory, as the layer norm's do; short rows go one a warp,
// and rows off 16-byte boundaries in aligned packs whose lead a block's rows share.
//
// Measured on a GB300 in graphs, floors by bytes at the measured copy bandwidth in brackets: bf16 16384 x 4096 with the
// residual forward 88 us (80), backward with dh 84 (80), FP8 form 82 (70); without either 47 and 70 (40, 60); fp16 6001
// x 2003 15.7 and 22 (14.4 and 14.4; x 2008 15.6 and 20.9), of which the columns' sums are 4; 128 x 7168 FP8 form 3.2.  From 1025
// packs on (H over 8192, off the boundaries over 8185) a ring's block has 288 threads and more, and an SM one of them, where 1024 packs
// have two of 256 forward and one of 512 backward: 2000 x 8192 bf16 10 and 19 us without and with the residual, backward 22 and
// 28 without and with dh (floors 10, 20, 15, 20), x 8200 17, 25, 33 and 40, x 8191 18, 30, 35 and 43.  Of short batches there (300 x 12288 14 and 17,
// floors 3.3 and 4.4) the blocks without a ring spill up to 800 bytes a thread.
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
// x + r in x's type, as the stream keeps it.
template <typename T, int P>
__device__ __forceinline__ void add_residual(float2 (&f)[P], const float2 (&r)[P])
{
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float2 v = add2(f[i], r[i]);
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            const __nv_bfloat162 h = __float22bfloat162_rn(v);
            f[i] = pair_of<T>(&h.x);
        } else {
            f[i] = make_float2(to_f<T>(from_f<T>(v.x)), to_f<T>(from_f<T>(v.y)));
        }
    }
}

// The row held in f (zeros past its end): its statistic and outputs; w: the thread's columns of the weight.
// `after_read` runs once every thread has its row in registers.
template <typename T, int V, int VPT, bool FP8, bool WARP, bool LEAD, typename F>
__device__ __forceinline__ void rms_row(const RmsArgs &a, int row, int lead, float2 (&f)[PAIRS<V, VPT>], const float2 (&w)[PAIRS<V, VPT>],
                                        float *red, int slot, F after_read)
{
    constexpr int P = PAIRS<V, VPT>;
    const int packs = packs_of<V, LEAD>(a.H, lead), t = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
    float2 acc = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i)
        acc = fma2(f[i], f[i], acc);
    float s[1] = {acc.x + acc.y};
    row_sum<WARP>(s, red, slot);
    after_read();
    const float rstd = 1.0f / sqrtf(s[0] / static_cast<float>(a.H) + a.eps);
    if (t == 0 && a.rstd)
        a.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < P; ++i)
        f[i] = mul2(mul2(f[i], both(rstd)), w[i]);
    if constexpr (FP8)
        put_fp8<V, VPT>(a.q + static_cast<size_t>(row) * a.H, a.sf + static_cast<size_t>(row) * (a.H / 128), f, t, step, packs, a.pow2);
    else
        put<T, V, VPT, LEAD>(static_cast<T *>(a.y) + static_cast<size_t>(row) * a.H, f, t, step, packs, lead, a.H);
}

// One row a block; or (WARP, rows of at most 1024 elements) one row a warp at a time, the next one on its
// way.  The weight is loaded beside the first row, ahead of its sum.
template <typename T, int V, int VPT, bool FP8, bool WARP, bool LEAD, bool RES>
__global__ void __launch_bounds__(WARP ? ROW_WARPS * 32 : V * VPT == 32 ? 512 : 1024) rms_kernel(const RmsArgs a)
{
    ptx::follow();
    constexpr int P = PAIRS<V, VPT>;
    __shared__ __align__(16) float red[WARP ? 4 : 64];
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
    if constexpr (!WARP)
        clear_sums<1>(red);
    const T *x = static_cast<const T *>(a.x), *r = static_cast<const T *>(a.r);
    int row = WARP ? blockIdx.x * ROW_WARPS + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.T)
        return;
    const int lead = LEAD ? lead_of(x + static_cast<size_t>(row) * a.ldx) : 0, packs = packs_of<V, LEAD>(a.H, lead);
    Pack<T, V> q[VPT], qr[RES ? VPT : 1];
    fetch<T, V, VPT, LEAD>(q, x + static_cast<size_t>(row) * a.ldx, t, step, packs, lead, a.H);
    if constexpr (RES)
        fetch<T, V, VPT, LEAD>(qr, r + static_cast<size_t>(row) * a.ldr, t, step, packs, lead, a.H);
    float2 f[P], w[P];
    load_columns<T, V, VPT, LEAD>(w, a.weight, a.w32, 1.0f, t, step, packs, lead, a.H);
    for (;;) {
        unpack<T, V, VPT>(f, q);
        if constexpr (RES) {
            float2 g[P];
            unpack<T, V, VPT>(g, qr);
            add_residual<T>(f, g);
            put<T, V, VPT, LEAD>(static_cast<T *>(a.h) + static_cast<size_t>(row) * a.H, f, t, step, packs, lead, a.H);
        }
        const int next = WARP ? row + gridDim.x * ROW_WARPS : a.T;
        if (WARP && next < a.T) {
            fetch<T, V, VPT, LEAD>(q, x + static_cast<size_t>(next) * a.ldx, t, step, packs, lead, a.H);
            if constexpr (RES)
                fetch<T, V, VPT, LEAD>(qr, r + static_cast<size_t>(next) * a.ldr, t, step, packs, lead, a.H);
        }
        rms_row<T, V, VPT, FP8, WARP, LEAD>(a, row, lead, f, w, red, 0, [] {});
        if (next >= a.T)
            return;
        row = next;
    }
}

// Persistent blocks: rows copied AHEAD rows before their use, the weight kept in registers.
template <typename T, int VPT, bool FP8, int AHEAD, bool LEAD, bool RES>
__global__ void __launch_bounds__(512) rms_ring_kernel(const RmsArgs a)
{
    ptx::follow();
    constexpr int V = 8, P = PAIRS<V, VPT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[64];
    Pack<T, V> *ring_x = reinterpret_cast<Pack<T, V> *>(smem), *ring_r = ring_x + AHEAD * VPT * blockDim.x;
    const int lead = LEAD ? lead_of(static_cast<const T *>(a.x) + static_cast<size_t>(blockIdx.x) * a.ldx) : 0;
    const int packs = packs_of<V, LEAD>(a.H, lead);
    const bool cut = LEAD && cut_packs<V, VPT>(threadIdx.x, blockDim.x, lead, a.H);
    const auto ahead = [&](int g, int row) {
        fetch_ahead<T, V, VPT, LEAD>(ring_x, g, a.x, a.ldx, row, a.T, a.H, packs, lead);
        if constexpr (RES)
            fetch_ahead<T, V, VPT, LEAD>(ring_r, g, a.r, a.ldr, row, a.T, a.H, packs, lead);
        copies_commit();
    };
#pragma unroll
    for (int g = 0; g < AHEAD; ++g)
        ahead(g, blockIdx.x + g * gridDim.x);
    clear_sums<1>(red);
    float2 w[P];
    load_columns<T, V, VPT, LEAD>(w, a.weight, a.w32, 1.0f, threadIdx.x, blockDim.x, packs, lead, a.H);
    int g = 0, slot = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, slot ^= 1) {
        copies_wait<AHEAD - 1>();
        float2 f[P];
        from_ring<T, V, VPT>(f, ring_x, g);
        if constexpr (RES) {
            float2 r[P];
            from_ring<T, V, VPT>(r, ring_r, g);
            add_residual<T>(f, r);
        }
        clip<V, VPT>(f, threadIdx.x, blockDim.x, packs, LEAD && cut, lead, a.H);
        if constexpr (RES)
            put<T, V, VPT, LEAD>(static_cast<T *>(a.h) + static_cast<size_t>(row) * a.H, f, threadIdx.x, blockDim.x, packs, lead, a.H);
        rms_row<T, V, VPT, FP8, false, LEAD>(a, row, lead, f, w, red, slot, [&] { ahead(g, row + AHEAD * gridDim.x); });
        g = g == AHEAD - 1 ? 0 : g + 1;
    }
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
    float *part;   // [blocks][pitch] sums of dy*xh over each block's rows (null: not wanted; LEAD: from their lead on)
    int pitch;
};

// xh and a = dy*g of one row, their sum, and the columns' sums so far.
template <int P>
__device__ __forceinline__ float backward_sum(float2 (&xh)[P], float2 (&d)[P], const float2 (&w)[P], float2 (&dg)[P], float rstd)
{
    float2 acc = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        xh[i] = mul2(xh[i], both(rstd));
        dg[i] = fma2(d[i], xh[i], dg[i]);
        d[i] = mul2(d[i], w[i]);
        acc = fma2(d[i], xh[i], acc);
    }
    return acc.x + acc.y;
}
template <int P>
__device__ __forceinline__ void backward_out(float2 (&d)[P], const float2 (&xh)[P], float mean, float rstd)
{
#pragma unroll
    for (int i = 0; i < P; ++i)
        d[i] = mul2(fma2(xh[i], both(-mean), d[i]), both(rstd));
}
template <int P>
__device__ __forceinline__ void add_all(float2 (&d)[P], const float2 (&v)[P])
{
#pragma unroll
    for (int i = 0; i < P; ++i)
        d[i] = add2(d[i], v[i]);
}

// Rows b, b + blocks, ... of block b: a thread keeps its columns' sums in registers over all of them, so
// every tensor is read once from HBM.  AHEAD > 0: rows copied that many rows before use, and h and dy read from
// shared memory twice (for the sum, then for dx) instead of held in registers between.
template <typename T, int V, int VPT, int AHEAD, bool LEAD, bool DH>
__global__ void __launch_bounds__(512) rms_backward_kernel(const RmsBwdArgs a)
{
    ptx::grid_dependency_wait();
    constexpr int P = PAIRS<V, VPT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[64];
    const int t = threadIdx.x, step = blockDim.x;
    const int lead = LEAD ? lead_of(static_cast<const T *>(a.h) + static_cast<size_t>(blockIdx.x) * a.ldh) : 0;
    const int packs = packs_of<V, LEAD>(a.H, lead);
    const bool cut = LEAD && cut_packs<V, VPT>(t, step, lead, a.H);
    const float inv = 1.0f / static_cast<float>(a.H);
    Pack<T, V> *ring_h = reinterpret_cast<Pack<T, V> *>(smem), *ring_d = ring_h + AHEAD * VPT * step, *ring_u = ring_d + AHEAD * VPT * step;
    const auto ahead = [&](int g, int row) {
        if constexpr (AHEAD > 0) {
            fetch_ahead<T, V, VPT, LEAD>(ring_h, g, a.h, a.ldh, row, a.T, a.H, packs, lead);
            fetch_ahead<T, V, VPT, LEAD>(ring_d, g, a.dy, a.lddy, row, a.T, a.H, packs, lead);
            if constexpr (DH)
                fetch_ahead<T, V, VPT, LEAD>(ring_u, g, a.dh, a.lddh, row, a.T, a.H, packs, lead);
            copies_commit();
        }
    };
#pragma unroll
    for (int g = 0; g < AHEAD; ++g)
        ahead(g, blockIdx.x + g * gridDim.x);
    clear_sums<1>(red);
    float2 w[P], dg[P];
    load_columns<T, V, VPT, LEAD>(w, a.weight, a.w32, 1.0f, t, step, packs, lead, a.H);
#pragma unroll
    for (int i = 0; i < P; ++i)
        dg[i] = both(0.0f);
    int slot = 0, stage = 0;
    float rstd = a.rstd[blockIdx.x];   // (no more blocks than rows)
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, slot ^= 1) {
        const int next = row + gridDim.x;
        const float rstd1 = next < a.T ? a.rstd[next] : 0.0f;
        float2 xh[P], d[P];
        Pack<T, V> q[VPT];
        if constexpr (AHEAD > 0) {
            copies_wait<AHEAD - 1>();
            from_ring<T, V, VPT>(xh, ring_h, stage);
            from_ring<T, V, VPT>(d, ring_d, stage);
            // what lies outside the row is not there: no products with it
            clip<V, VPT>(xh, t, step, packs, LEAD && cut, lead, a.H);
            clip<V, VPT>(d, t, step, packs, LEAD && cut, lead, a.H);
        } else {
            fetch<T, V, VPT, LEAD>(q, static_cast<const T *>(a.h) + static_cast<size_t>(row) * a.ldh, t, step, packs, lead, a.H);
            unpack<T, V, VPT>(xh, q);
            fetch<T, V, VPT, LEAD>(q, static_cast<const T *>(a.dy) + static_cast<size_t>(row) * a.lddy, t, step, packs, lead, a.H);
            unpack<T, V, VPT>(d, q);
            if constexpr (DH)
                fetch<T, V, VPT, LEAD>(q, static_cast<const T *>(a.dh) + static_cast<size_t>(row) * a.lddh, t, step, packs, lead, a.H);
        }
        float s[1] = {backward_sum(xh, d, w, dg, rstd)};
        block_sum(s, red, slot);
        if constexpr (AHEAD > 0) {
            from_ring<T, V, VPT>(xh, ring_h, stage);
            from_ring<T, V, VPT>(d, ring_d, stage);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                xh[i] = mul2(xh[i], both(rstd));
                d[i] = mul2(d[i], w[i]);
            }
        }
        backward_out(d, xh, s[0] * inv, rstd);
        if constexpr (DH) {
            if constexpr (AHEAD > 0)
                from_ring<T, V, VPT>(xh, ring_u, stage);
            else
                unpack<T, V, VPT>(xh, q);
            add_all(d, xh);
        }
        put<T, V, VPT, LEAD>(static_cast<T *>(a.dx) + static_cast<size_t>(row) * a.H, d, t, step, packs, lead, a.H);
        if constexpr (AHEAD > 0) {   // (every value read above has been used by now)
            ahead(stage, row + AHEAD * gridDim.x);
            stage = stage == AHEAD - 1 ? 0 : stage + 1;
        }
        rstd = rstd1;
    }
    if (a.part)
        put<float, V, VPT>(a.part + static_cast<size_t>(blockIdx.x) * a.pitch, dg, t, step, packs);
    ptx::launch_dependents();
}

// Rows of at most 1024 elements: one row a warp at a time, the next one on its way; the block's warps add
// their columns' sums at the end, in order.
template <typename T, int V, int VPT, bool DH>
__global__ void __launch_bounds__(ROW_WARPS * 32) rms_backward_warp_kernel(const RmsBwdArgs a)
{
    ptx::grid_dependency_wait();
    constexpr int P = PAIRS<V, VPT>;
    struct alignas(16) Sums {
        float v[32 * V * VPT];
    };
    static_assert(alignof(Sums) >= alignof(Pack<float, V>), "put() stores whole packs into them");
    __shared__ Sums sums[ROW_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int packs = a.H / V;
    const float inv = 1.0f / static_cast<float>(a.H);
    const T *h = static_cast<const T *>(a.h), *dy = static_cast<const T *>(a.dy), *dh = static_cast<const T *>(a.dh);
    float2 w[P], dg[P];
    load_columns<T, V, VPT>(w, a.weight, a.w32, 1.0f, lane, 32, packs);
#pragma unroll
    for (int i = 0; i < P; ++i)
        dg[i] = both(0.0f);
    int row = blockIdx.x * ROW_WARPS + warp;
    if (row < a.T) {
        Pack<T, V> qh[VPT], qd[VPT], qu[DH ? VPT : 1];
        const auto load = [&](int r) {
            fetch<T, V, VPT>(qh, h + static_cast<size_t>(r) * a.ldh, lane, 32, packs);
            fetch<T, V, VPT>(qd, dy + static_cast<size_t>(r) * a.lddy, lane, 32, packs);
            if constexpr (DH)
                fetch<T, V, VPT>(qu, dh + static_cast<size_t>(r) * a.lddh, lane, 32, packs);
        };
        load(row);
        float rstd = a.rstd[row];
        for (;;) {
            float2 xh[P], d[P], u[DH ? P : 1];
            unpack<T, V, VPT>(xh, qh);
            unpack<T, V, VPT>(d, qd);
            if constexpr (DH)
                unpack<T, V, VPT>(u, qu);
            const int next = row + gridDim.x * ROW_WARPS;
            const float rs = rstd;
            if (next < a.T) {
                load(next);
                rstd = a.rstd[next];
            }
            const float s = warp_sum(backward_sum(xh, d, w, dg, rs));
            backward_out(d, xh, s * inv, rs);
            if constexpr (DH)
                add_all(d, u);
            put<T, V, VPT>(static_cast<T *>(a.dx) + static_cast<size_t>(row) * a.H, d, lane, 32, packs);
            if (next >= a.T)
                break;
            row = next;
        }
    }
    if (a.part) {
        put<float, V, VPT>(sums[warp].v, dg, lane, 32, 32 * VPT);
        __syncthreads();
        for (int c = threadIdx.x; c < a.H; c += ROW_WARPS * 32) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < ROW_WARPS; ++k)
                v += sums[k].v[c];
            a.part[static_cast<size_t>(blockIdx.x) * a.pitch + c] = v;
        }
    }
    ptx::launch_dependents();
}

// ------------------------------------------------------------------ host side ------------
// Rows in packs, without a lead or with one; others go element by element.  Not rows of at most 1024 elements with
// a lead, whose ends are much of what a warp does then (16384 x 1001 bf16, with the residual and its gradient, 53 and 74 us in
// packs).
template <typename T>
bool in_packs(int H, Rows rows)
{
    return rows == PACKED || (rows == PHASED && H > 1024 && most_packs<T>(H, rows) <= 2048);
}
// A ring's blocks, `per_sm` to an SM.  Launched ahead of the kernel before they are placed as its blocks leave, and
// where an SM has room for many more, they crowd on the SMs that are left first (16384 x 4096 bf16 backward, room for
// three: 81 us, and 70 launched after it); else it saves the launch (6001 x 2003 fp16 forward and backward
// 47 -> 44).
template <typename A>
bool launch_ring(void (*kern)(A), int blocks, int threads, size_t smem, int per_sm, cudaStream_t s, const A &a)
{
    if (!allow_smem(kern, smem))
        return false;
    const int room = static_cast<int>(228 * 1024 / (smem + 1024));
    if (8 * room <= 9 * per_sm)
        launch_programmatic(kern, blocks, threads, static_cast<int>(smem), s, a);
    else
        kern<<<blocks, threads, smem, s>>>(a);
    return true;
}

template <typename T, bool FP8, int AHEAD, bool LEAD, bool RES>
bool try_rms_ring(const RmsArgs &a, int packs, int num_sms, cudaStream_t s)
{
    const int threads = round32((packs + 3) / 4);
    size_t smem;
    const int per_sm = ring_blocks<T, 8, 4>(threads, AHEAD, RES ? 2 : 1, smem);
    // long batches only: every block has rows to copy ahead of
    if (per_sm < 1 || a.T < AHEAD * per_sm * num_sms)
        return false;
    return launch_ring(rms_ring_kernel<T, 4, FP8, AHEAD, LEAD, RES>, ring_grid(per_sm, num_sms), threads, smem, per_sm, s, a);
}

template <typename T, int V, int VPT, bool FP8, bool RES>
void launch_rms_warps(const RmsArgs &a, int num_sms, cudaStream_t s)
{
    launch_programmatic(rms_kernel<T, V, VPT, FP8, true, false, RES>, warp_blocks(a.T, 8, num_sms), ROW_WARPS * 32, 0, s, a);
}

template <typename T, bool FP8, bool LEAD, bool RES>
void launch_rms_packs(const RmsArgs &a, int packs, int num_sms, cudaStream_t s)
{
    // few rows: as many threads a row as it has packs, for latency
    const bool few = a.T <= 2 * num_sms;
    if (packs <= 32 && !LEAD)
        launch_rms_warps<T, 8, 1, FP8, RES>(a, num_sms, s);
    else if (packs <= 128 && !few && !LEAD)
        launch_rms_warps<T, 8, 4, FP8, RES>(a, num_sms, s);
    else if (few && packs <= 1024)
        launch_programmatic(rms_kernel<T, 8, 1, FP8, false, LEAD, RES>, a.T, round32(packs), 0, s, a);
    else if (packs > 2048 || !try_rms_ring<T, FP8, RES ? 3 : 4, LEAD, RES>(a, packs, num_sms, s))
        launch_programmatic(rms_kernel<T, 8, 4, FP8, false, LEAD, RES>, a.T, round32((packs + 3) / 4), 0, s, a);
}

template <typename T, bool FP8, bool RES>
void launch_rms(const RmsArgs &a, Rows rows, int num_sms, cudaStream_t s)
{
    const int packs = most_packs<T>(a.H, rows);
    if (rows == PACKED)
        return launch_rms_packs<T, FP8, false, RES>(a, packs, num_sms, s);
    if constexpr (!FP8) {
        if (in_packs<T>(a.H, rows))
            return launch_rms_packs<T, false, true, RES>(a, packs, num_sms, s);
        if (a.H <= 256)
            launch_rms_warps<T, 1, 8, false, RES>(a, num_sms, s);
        else if (a.H <= 576 && a.T > 2 * num_sms)
            launch_rms_warps<T, 1, 18, false, RES>(a, num_sms, s);
        else if (a.H <= 1024 && a.T > 2 * num_sms)
            launch_rms_warps<T, 1, 32, false, RES>(a, num_sms, s);
        else if (a.H <= 8192)
            launch_programmatic(rms_kernel<T, 1, 8, false, false, false, RES>, a.T, round32((a.H + 7) / 8), 0, s, a);
        else
            launch_programmatic(rms_kernel<T, 1, 16, false, false, false, RES>, a.T, round32((a.H + 15) / 16), 0, s, a);
    }
}

// The backward pass: kernel, blocks (each keeps a row of partial sums) and how they are found.
enum Plan { WARPS, RING, DIRECT, ELEMENT_WARPS, ELEMENTS };
// Rows of a warp are held in registers, with dh many of them, so that with dh longer rows go through rings (bf16, 16384 x
// 1024 30.6 us by warps and 28.7 in rings, without dh 22.5 and 21.4, but x 768 15.5 and 19.1; off the boundaries, x 1001
// 63 and 32, x 701 47 and 30, and without dh 26 and 28, 19 and 28).
template <typename T>
Plan backward_plan(int T_, int H, Rows rows, bool dh, int num_sms, int &blocks)
{
    const int packs = most_packs<T>(H, rows);
    const bool in_rings = rows == PHASED && dh && H > 576 && H <= 1024;
    if (in_packs<T>(H, rows) || in_rings) {
        size_t smem;
        const int per_sm = packs <= 1024 ? ring_blocks<T, 8, 2>(round32((packs + 1) / 2), packs <= 512 ? 4 : 2, 3, smem)
                                         : ring_blocks<T, 8, 4>(round32((packs + 3) / 4), 2, 3, smem);
        const bool ring = per_sm >= 1 && T_ >= 4 * per_sm * num_sms;
        if (rows == PACKED && (packs <= 32 || (packs <= 128 && T_ > 2 * num_sms && !(ring && dh && packs > 64)))) {
            blocks = warp_blocks(T_, 3, num_sms);
            return WARPS;
        }
        if (ring) {
            blocks = ring_grid(per_sm, num_sms);
            return RING;
        }
        if (!in_rings) {
            const int most = ring_grid(2, num_sms);
            blocks = T_ < most ? T_ : most;
            return DIRECT;
        }
    }
    if (H <= 256 || (H <= 1024 && T_ > 2 * num_sms)) {
        blocks = warp_blocks(T_, 3, num_sms);
        return ELEMENT_WARPS;
    }
    blocks = T_ < 2 * num_sms ? T_ : 2 * num_sms;
    return ELEMENTS;
}
// (the workspace covers every alignment)
template <typename T>
int most_backward_blocks(int T_, int H, int num_sms)
{
    int most = 0;
    for (const Rows rows : {PACKED, PHASED, ANY})
        for (const bool dh : {false, true}) {
            int b;
            backward_plan<T>(T_, H, rows, dh, num_sms, b);
            most = b > most ? b : most;
        }
    return most;
}

template <typename T, int VPT, int AHEAD, bool LEAD, bool DH>
bool launch_backward_ring(const RmsBwdArgs &a, int packs, int blocks, int num_sms, cudaStream_t s)
{
    const int threads = round32((packs + VPT - 1) / VPT);
    size_t smem;
    ring_blocks<T, 8, VPT>(threads, AHEAD, DH ? 3 : 2, smem);
    return launch_ring(rms_backward_kernel<T, 8, VPT, AHEAD, LEAD, DH>, blocks, threads, smem, (blocks + num_sms - 1) / num_sms, s, a);
}

template <typename T, bool LEAD, bool DH>
bool launch_backward_packs(const RmsBwdArgs &a, Plan plan, int packs, int blocks, int num_sms, cudaStream_t s)
{
    if (plan == RING)
        return packs <= 512    ? launch_backward_ring<T, 2, 4, LEAD, DH>(a, packs, blocks, num_sms, s)
               : packs <= 1024 ? launch_backward_ring<T, 2, 2, LEAD, DH>(a, packs, blocks, num_sms, s)
                               : launch_backward_ring<T, 4, 2, LEAD, DH>(a, packs, blocks, num_sms, s);
    if (packs <= 1024)
        launch_programmatic(rms_backward_kernel<T, 8, 2, 0, LEAD, DH>, blocks, round32((packs + 1) / 2), 0, s, a);
    else
        launch_programmatic(rms_backward_kernel<T, 8, 4, 0, LEAD, DH>, blocks, round32((packs + 3) / 4), 0, s, a);
    return true;
}

template <typename T, int V, int VPT, bool DH>
void launch_backward_warps(const RmsBwdArgs &a, int blocks, cudaStream_t s)
{
    launch_programmatic(rms_backward_warp_kernel<T, V, VPT, DH>, blocks, ROW_WARPS * 32, 0, s, a);
}

template <typename T, bool DH>
bool launch_rms_backward(const RmsBwdArgs &a, Rows rows, int num_sms, PartRows &part, cudaStream_t s)
{
    int blocks;
    const Plan plan = backward_plan<T>(a.T, a.H, rows, DH, num_sms, blocks);
    const int packs = most_packs<T>(a.H, rows);
    constexpr int boundary = VEC<T>;
    // (a block's row of sums starts at its rows' lead)
    part = {a.part, blocks, a.pitch, rows == PHASED && (plan == RING || plan == DIRECT) ? a.H % boundary : 0, boundary};
    if (plan == WARPS)
        packs <= 32 ? launch_backward_warps<T, 8, 1, DH>(a, blocks, s) : launch_backward_warps<T, 8, 4, DH>(a, blocks, s);
    else if (plan == ELEMENT_WARPS)
        a.H <= 256   ? launch_backward_warps<T, 1, 8, DH>(a, blocks, s)
        : a.H <= 576 ? launch_backward_warps<T, 1, 18, DH>(a, blocks, s)
                     : launch_backward_warps<T, 1, 32, DH>(a, blocks, s);
    else if (plan == ELEMENTS && a.H <= 8192)
        launch_programmatic(rms_backward_kernel<T, 1, 16, 0, false, DH>, blocks, round32((a.H + 15) / 16), 0, s, a);
    else if (plan == ELEMENTS)
        launch_programmatic(rms_backward_kernel<T, 1, 32, 0, false, DH>, blocks, round32((a.H + 31) / 32), 0, s, a);
    else
        return rows == PACKED ? launch_backward_packs<T, false, DH>(a, plan, packs, blocks, num_sms, s)
                              : launch_backward_packs<T, true, DH>(a, plan, packs, blocks, num_sms, s);
    return true;
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
        using E = std::remove_pointer_t<decltype(t)>;
        residual ? launch_rms<E, false, true>(a, rows, sms, static_cast<cudaStream_t>(stream))
                 : launch_rms<E, false, false>(a, rows, sms, static_cast<cudaStream_t>(stream));
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
        using E = std::remove_pointer_t<decltype(t)>;
        residual ? launch_rms<E, true, true>(a, PACKED, sms, static_cast<cudaStream_t>(stream))
                 : launch_rms<E, true, false>(a, PACKED, sms, static_cast<cudaStream_t>(stream));
    });
    return launched();
}

int moe_rms_norm_backward_workspace(int T, int H, uint64_t *bytes)
{
    if (T < 0 || T > MAX_ROWS || H < 1 || H > MAX_H || !bytes)
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    // enough for every element type
    const int a = most_backward_blocks<float>(T, H, sms), b = most_backward_blocks<__nv_bfloat16>(T, H, sms);
    *bytes = static_cast<uint64_t>(a > b ? a : b) * static_cast<uint64_t>(part_pitch(H)) * sizeof(float);
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
        const RmsBwdArgs a{T, H, dy, h, dh, lddy, ldh, lddh, weight, w_dtype == MOE_F32 && dtype != MOE_F32, rstd, dx,
                           dweight ? static_cast<float *>(workspace) : nullptr, part_pitch(H)};
        const Rows rows = worst(worst(worst(rows_of(H, dtype, h, ldh), rows_of(H, dtype, dy, lddy)), rows_or_absent(H, dtype, dh, lddh)),
                                worst(rows_of(H, dtype, dx, H), affine_of(weight)));
        const bool ok = with_dtype(dtype, [&](auto *t) {
            using E = std::remove_pointer_t<decltype(t)>;
            return dh ? launch_rms_backward<E, true>(a, rows, sms, part, s) : launch_rms_backward<E, false>(a, rows, sms, part, s);
        });
        if (!ok || launched() != MOE_OK)
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
