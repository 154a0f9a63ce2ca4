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
#include "norm_rows.cuh"

using namespace cpw;

namespace {

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
        put_fp8<V, VPT>(a.q + static_cast<size_t>(row) * a.H, a.sf + static_cast<size_t>(row) * (a.H / 128), f, t, step, packs, a.pow2);
    } else {
        put<T, V, VPT, LEAD>(static_cast<T *>(a.y) + static_cast<size_t>(row) * a.H, f, t, step, packs, lead, a.H);
    }
}

// One row a block; or (WARP, rows of at most 1024 elements) one row a warp at a time, the next
// one on its way.  The weight and bias are loaded beside the first row, ahead of its sums.
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
