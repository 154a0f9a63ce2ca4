// rows.cu -- rows moved from token order into expert-major order and weighted back out of it,
// with both directions' gradients.  rows[t][j] is the row of slot j of token t (-1: none).
//
//   gather    out[rows[t][j]] = x[t]
//   combine   out[t] = sum_j w[t][j] * y[rows[t][j]]      (fp32, j ascending, rounded once)
//   its gradients   dy[rows[t][j]] = w[t][j] * dout[t],   dw[t][j] = sum_h dout[t][h] * y[rows[t][j]][h]
//
// Measured on a GB300, bf16: gather of 16384 x 8 x 4096 189 us (floor 181), combine of 8192 x 8 x
// 7168 180 us and its gradients 282 us with 5% of the slots skipped (both 462 us, floor 444), combine
// of 128 x 8 x 7168 4.4 us.
//
// The gradient of gather is combine with w = 1.  All three are bound by HBM: a thread handles a
// piece of a token for all of its slots, so the token's row is read (or written) once however
// many slots it has, and every row in expert order once.
#include <type_traits>

#include "op_common.cuh"

using namespace cpw;

namespace {

constexpr int MAX_K = 32;
constexpr int SLOTS = 8;   // slots of a token handled together
constexpr int COMBINE_BLOCK = 128;
// packs of a row up to which a block of 128 threads takes several tokens (combine of 16384 x 8 x 256:
// 15.5 us, 28.7 with a block a token; 768 columns: 56.6 and 58.7)
constexpr int NARROW = 96;
constexpr int BWD_BLOCK = 128;   // 8192 x 8 x 7168 bf16: 493 us for both passes (64: 497, 256: 507, 448: 550)

struct RowArgs {
    int T, k, H;
    int M;                   // rows in expert order
    const void *x;           // [T][H]: gather's input, combine's gradient
    long long ldx;
    const void *y;           // [M][H]
    const int32_t *rows;     // [T][k]
    const float *w;          // [T][k] or null (1)
    const int32_t *total;    // rows that are named: rows from there on are zeroed
    void *out;               // gather [M][H], combine [T][H]
    void *dy;                // [M][H]
    float *dw;               // [T][k]
};

// Rows and weights of a token's slots j0 .. j0 + SLOTS - 1 (-1 and 0 where there is none): one
// load a lane (fetch_slot), then shuffles (spread_slots), so that a warp has all of them after
// one memory latency, and can ask for the next token's ahead of time.
struct Slot {
    int row;
    float w;
};
__device__ __forceinline__ Slot fetch_slot(const RowArgs &a, int t, int j0)
{
    const int lane = threadIdx.x & 31, j = j0 + lane;
    Slot s{-1, 0.0f};
    if (lane < SLOTS && j < a.k && t < a.T) {
        const size_t at = static_cast<size_t>(t) * a.k + j;
        s.row = a.rows[at];
        s.w = a.w ? a.w[at] : 1.0f;
    }
    return s;
}
__device__ __forceinline__ void spread_slots(const RowArgs &a, const Slot &s, int (&r)[SLOTS], float (&w)[SLOTS])
{
    const bool in = s.row >= 0 && s.row < a.M;
    const int row = in ? s.row : -1;
    const float weight = in ? s.w : 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
        r[i] = __shfl_sync(0xFFFFFFFFu, row, i);
        w[i] = __shfl_sync(0xFFFFFFFFu, weight, i);
    }
}
__device__ __forceinline__ void load_slots(const RowArgs &a, int t, int j0, int (&r)[SLOTS], float (&w)[SLOTS])
{
    spread_slots(a, fetch_slot(a, t, j0), r, w);
}

// Zeroes the rows that no slot names; block b of `blocks`.
template <typename T, int V>
__device__ __forceinline__ void zero_rest(const RowArgs &a, void *out, int b, int blocks)
{
    const int packs = a.H / V;
    int first = *a.total;
    first = first < 0 ? 0 : first;
    Pack<T, V> z;
#pragma unroll
    for (int i = 0; i < V; ++i)
        z.v[i] = from_f<T>(0.0f);
    for (int r = first + b; r < a.M; r += blocks)
        for (int p = threadIdx.x; p < packs; p += blockDim.x)
            store_pack<T, V>(static_cast<T *>(out) + static_cast<size_t>(r) * a.H + static_cast<size_t>(p) * V, z);
}

// Packs of a thread: a block covers a like number of bytes of a row whatever its packs' size.
template <typename T, int V>
constexpr int PACKS = sizeof(T) * V >= 16 ? 1 : V == 2 ? 2 : 4;

template <typename T, int V>
__global__ void __launch_bounds__(1024) gather_kernel(const RowArgs a)
{
    if (static_cast<int>(blockIdx.x) >= a.T) {
        zero_rest<T, V>(a, a.out, blockIdx.x - a.T, gridDim.x - a.T);
        return;
    }
    const int t = blockIdx.x, packs = a.H / V;
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(t) * a.ldx;
    T *out = static_cast<T *>(a.out);
    for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
        int r[SLOTS];
        float w[SLOTS];
        load_slots(a, t, j0, r, w);
        constexpr int N = PACKS<T, V>;
        for (int p = threadIdx.x; p < packs; p += N * blockDim.x) {
            Pack<T, V> v[N];
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (p + n * static_cast<int>(blockDim.x) < packs)
                    v[n] = load_pack<T, V>(x + static_cast<size_t>(p + n * blockDim.x) * V);
#pragma unroll
            for (int i = 0; i < SLOTS; ++i)
#pragma unroll
                for (int n = 0; n < N; ++n)
                    if (r[i] >= 0 && p + n * static_cast<int>(blockDim.x) < packs)
                        store_pack<T, V>(out + static_cast<size_t>(r[i]) * a.H + static_cast<size_t>(p + n * blockDim.x) * V, v[n]);
        }
    }
}

// A block takes a run of columns of `tokens` tokens, one after the other: the loads of all slots
// of a token are in flight together, those of the next token's slots beside them, and many
// small blocks share an SM.
template <typename T, int V>
__global__ void __launch_bounds__(COMBINE_BLOCK) combine_rows_kernel(const RowArgs a, int tokens)
{
    constexpr int N = PACKS<T, V>;
    const int packs = a.H / V, p0 = blockIdx.x * (COMBINE_BLOCK * N) + threadIdx.x;
    const T *y = static_cast<const T *>(a.y);
    int t = (blockIdx.y + blockIdx.z * gridDim.y) * tokens;
    const int end = min(a.T, t + tokens);
    if (t >= end)
        return;
    Slot ahead = fetch_slot(a, t, 0);
    for (; t < end; ++t) {
        float acc[N][V];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < V; ++i)
                acc[n][i] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
            int r[SLOTS];
            float w[SLOTS];
            spread_slots(a, ahead, r, w);
            Pack<T, V> v[N][SLOTS];
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < SLOTS; ++i)
                    if (r[i] >= 0 && p0 + n * COMBINE_BLOCK < packs)
                        v[n][i] = load_pack<T, V>(y + static_cast<size_t>(r[i]) * a.H + static_cast<size_t>(p0 + n * COMBINE_BLOCK) * V);
            ahead = j0 + SLOTS < a.k ? fetch_slot(a, t, j0 + SLOTS) : fetch_slot(a, t + 1, 0);
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < SLOTS; ++i)
                    if (r[i] >= 0 && p0 + n * COMBINE_BLOCK < packs) {
#pragma unroll
                        for (int c = 0; c < V; ++c)
                            acc[n][c] = fmaf(w[i], to_f<T>(v[n][i].v[c]), acc[n][c]);
                    }
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (p0 + n * COMBINE_BLOCK < packs) {
                Pack<T, V> o;
#pragma unroll
                for (int c = 0; c < V; ++c)
                    o.v[c] = from_f<T>(acc[n][c]);
                store_pack<T, V>(static_cast<T *>(a.out) + static_cast<size_t>(t) * a.H + static_cast<size_t>(p0 + n * COMBINE_BLOCK) * V, o);
            }
    }
}

// One pack of a token's gradient: its part of the slots' sums, and the rows' gradients.
template <typename T, int V>
__device__ __forceinline__ void backward_pack(const RowArgs &a, const T *d, const T *y, T *dy, int p, const int (&r)[SLOTS],
                                              const float (&w)[SLOTS], float (&dot)[SLOTS])
{
                const Pack<T, V> q = load_pack<T, V>(d + static_cast<size_t>(p) * V);
                Pack<T, V> v[SLOTS];
#pragma unroll
                for (int i = 0; i < SLOTS; ++i)
                    if (r[i] >= 0)
                        v[i] = load_pack<T, V>(y + static_cast<size_t>(r[i]) * a.H + static_cast<size_t>(p) * V);
#pragma unroll
                for (int i = 0; i < SLOTS; ++i)
                    if (r[i] >= 0) {
                        Pack<T, V> o;
#pragma unroll
                        for (int c = 0; c < V; ++c) {
                            const float g = to_f<T>(q.v[c]);
                            dot[i] = fmaf(g, to_f<T>(v[i].v[c]), dot[i]);
                            o.v[c] = from_f<T>(w[i] * g);
                        }
                        store_pack<T, V>(dy + static_cast<size_t>(r[i]) * a.H + static_cast<size_t>(p) * V, o);
                    }
}

// Short rows (at most NARROW packs): a thread a (token, pack), so that a warp is not left with
// lanes past the row's end.
__device__ __forceinline__ void slot_of(const RowArgs &a, int t, int j, int &r, float &w)
{
    r = -1;
    w = 0.0f;
    if (j < a.k) {
        const size_t at = static_cast<size_t>(t) * a.k + j;
        const int v = a.rows[at];
        if (v >= 0 && v < a.M) {
            r = v;
            w = a.w ? a.w[at] : 1.0f;
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(COMBINE_BLOCK) gather_narrow_kernel(const RowArgs a, int blocks)
{
    if (static_cast<int>(blockIdx.x) >= blocks) {
        zero_rest<T, V>(a, a.out, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
    const int packs = a.H / V;
    const long long i = static_cast<long long>(blockIdx.x) * COMBINE_BLOCK + threadIdx.x;
    const int t = static_cast<int>(i / packs), p = static_cast<int>(i - static_cast<long long>(t) * packs);
    if (t >= a.T)
        return;
    const Pack<T, V> v = load_pack<T, V>(static_cast<const T *>(a.x) + static_cast<size_t>(t) * a.ldx + static_cast<size_t>(p) * V);
    for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
        int r[SLOTS];
        float w[SLOTS];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            slot_of(a, t, j0 + s, r[s], w[s]);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (r[s] >= 0)
                store_pack<T, V>(static_cast<T *>(a.out) + static_cast<size_t>(r[s]) * a.H + static_cast<size_t>(p) * V, v);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(COMBINE_BLOCK) combine_narrow_kernel(const RowArgs a)
{
    const int packs = a.H / V;
    const long long i = static_cast<long long>(blockIdx.x) * COMBINE_BLOCK + threadIdx.x;
    const int t = static_cast<int>(i / packs), p = static_cast<int>(i - static_cast<long long>(t) * packs);
    if (t >= a.T)
        return;
    const T *y = static_cast<const T *>(a.y) + static_cast<size_t>(p) * V;
    float acc[V];
#pragma unroll
    for (int c = 0; c < V; ++c)
        acc[c] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
        int r[SLOTS];
        float w[SLOTS];
        Pack<T, V> v[SLOTS];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            slot_of(a, t, j0 + s, r[s], w[s]);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (r[s] >= 0)
                v[s] = load_pack<T, V>(y + static_cast<size_t>(r[s]) * a.H);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (r[s] >= 0) {
#pragma unroll
                for (int c = 0; c < V; ++c)
                    acc[c] = fmaf(w[s], to_f<T>(v[s].v[c]), acc[c]);
            }
    }
    Pack<T, V> o;
#pragma unroll
    for (int c = 0; c < V; ++c)
        o.v[c] = from_f<T>(acc[c]);
    store_pack<T, V>(static_cast<T *>(a.out) + static_cast<size_t>(t) * a.H + static_cast<size_t>(p) * V, o);
}

// A warp a token: its sums over the columns need no other warp.
template <typename T, int V>
__global__ void __launch_bounds__(COMBINE_BLOCK) combine_narrow_backward_kernel(const RowArgs a, int blocks)
{
    if (static_cast<int>(blockIdx.x) >= blocks) {
        zero_rest<T, V>(a, a.dy, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
    const int t = blockIdx.x * (COMBINE_BLOCK / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31, packs = a.H / V;
    if (t >= a.T)
        return;
    const T *d = static_cast<const T *>(a.x) + static_cast<size_t>(t) * a.ldx;
    const T *y = static_cast<const T *>(a.y);
    T *dy = static_cast<T *>(a.dy);
    for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
        int r[SLOTS];
        float w[SLOTS], dot[SLOTS];
        load_slots(a, t, j0, r, w);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            dot[s] = 0.0f;
        for (int p = lane; p < packs; p += 32)
            backward_pack<T, V>(a, d, y, dy, p, r, w, dot);
        float mine = 0.0f;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const float v = warp_sum(dot[s]);
            mine = lane == s ? v : mine;
        }
        if (a.dw && lane < SLOTS && j0 + lane < a.k)
            a.dw[static_cast<size_t>(t) * a.k + j0 + lane] = mine;
    }
}

// A block takes a whole token, for the sums over its columns.
template <typename T, int V>
__global__ void __launch_bounds__(512) combine_rows_backward_kernel(const RowArgs a)
{
    if (static_cast<int>(blockIdx.x) >= a.T) {
        zero_rest<T, V>(a, a.dy, blockIdx.x - a.T, gridDim.x - a.T);
        return;
    }
    __shared__ float red[16][SLOTS];
    const int t = blockIdx.x, packs = a.H / V;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const T *d = static_cast<const T *>(a.x) + static_cast<size_t>(t) * a.ldx;
    const T *y = static_cast<const T *>(a.y);
    T *dy = static_cast<T *>(a.dy);
    for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
        int r[SLOTS];
        float w[SLOTS], dot[SLOTS];
        load_slots(a, t, j0, r, w);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            dot[i] = 0.0f;
        for (int p = threadIdx.x; p < packs; p += blockDim.x)
            backward_pack<T, V>(a, d, y, dy, p, r, w, dot);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            dot[i] = warp_sum(dot[i]);
        __syncthreads();
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < SLOTS; ++i)
                red[warp][i] = dot[i];
        }
        __syncthreads();
        if (a.dw && threadIdx.x < SLOTS && j0 + static_cast<int>(threadIdx.x) < a.k) {
            float s = 0.0f;
            for (int wi = 0; wi < warps; ++wi)
                s += red[wi][threadIdx.x];
            // a slot without a row: its dot stayed zero
            a.dw[static_cast<size_t>(t) * a.k + j0 + threadIdx.x] = s;
        }
    }
}

int rows_threads(int packs)
{
    const int t = (packs + 31) / 32 * 32;
    return t < 32 ? 32 : t > 512 ? 512 : t;
}

// The sums' kernel: small blocks, of which many share an SM, unless there are few tokens (128 x 8 x
// 7168: 5.1 us, 6.3 with small blocks; 500 tokens: 25.7 and 19.7).
int backward_threads(int packs, int T, int sms)
{
    const int most = rows_threads(packs);
    return T > sms && most > BWD_BLOCK ? BWD_BLOCK : most;
}

bool rows_sizes_ok(int T, int k, int H, long long M, int dtype)
{
    return T >= 0 && T <= MAX_ROWS && k >= 1 && k <= MAX_K && H >= 1 && M >= 0 && M <= MAX_ROWS && dtype_ok(dtype);
}

// 16-byte packs where every row starts on a 16-byte boundary, pairs of 16-bit elements where it
// does on a 4-byte one, single elements otherwise.
template <typename F>
int by_rows(int dtype, int H, long long ldx, const void *p0, const void *p1, const void *p2, F f)
{
    const size_t b = dtype_bytes(dtype);
    const auto all = [&](size_t n) {
        return H * b % n == 0 && static_cast<size_t>(ldx) * b % n == 0 && op_aligned(p0, n) && op_aligned(p1, n) && op_aligned(p2, n);
    };
    with_dtype(dtype, [&](auto *t) {
        using E = std::remove_pointer_t<decltype(t)>;
        if (all(16)) {
            f(t, std::integral_constant<int, 16 / static_cast<int>(sizeof(E))>{});
            return;
        }
        if constexpr (sizeof(E) == 2)
            if (all(4)) {
                f(t, std::integral_constant<int, 2>{});
                return;
            }
        f(t, std::integral_constant<int, 1>{});
    });
    return launched();
}

}  // namespace

extern "C" {

int moe_gather_rows(int T, int topk, int H, int E, int64_t M, const void *x, int64_t ldx, int dtype,
                    const int32_t *rows, const int32_t *offsets, void *out, void *stream)
{
    if (!rows_sizes_ok(T, topk, H, M, dtype) || E < 1 || ldx < H)
        return MOE_ERR_INVALID_ARG;
    if (M == 0)
        return MOE_OK;
    const size_t b = dtype_bytes(dtype);
    if (!out || !offsets || !op_aligned(out, b) || !op_aligned(offsets, 4) ||
        (T > 0 && (!x || !rows || !op_aligned(x, b) || !op_aligned(rows, 4))))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const RowArgs a{T, topk, H, static_cast<int>(M), x, ldx, nullptr, rows, nullptr, offsets + E, out, nullptr, nullptr};
    return by_rows(dtype, H, ldx, x, out, nullptr, [&](auto *t, auto v) {
        using Ty = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value;
        if (H / V <= NARROW) {
            const int blocks = static_cast<int>((static_cast<long long>(T) * (H / V) + COMBINE_BLOCK - 1) / COMBINE_BLOCK);
            gather_narrow_kernel<Ty, V><<<blocks + sms, COMBINE_BLOCK, 0, static_cast<cudaStream_t>(stream)>>>(a, blocks);
            return;
        }
        gather_kernel<Ty, V><<<T + sms, rows_threads(H / V), 0, static_cast<cudaStream_t>(stream)>>>(a);
    });
}

int moe_combine_rows(int T, int topk, int H, int64_t M, const void *y, int dtype, const int32_t *rows, const float *w,
                     void *out, void *stream)
{
    if (!rows_sizes_ok(T, topk, H, M, dtype))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    const size_t b = dtype_bytes(dtype);
    if (!out || !rows || (M > 0 && !y) || !op_aligned(out, b) || !op_aligned(y, b) || !op_aligned(rows, 4) || !op_aligned(w, 4))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const RowArgs a{T, topk, H, static_cast<int>(M), nullptr, H, y, rows, w, nullptr, out, nullptr, nullptr};
    return by_rows(dtype, H, H, y, out, nullptr, [&](auto *t, auto v) {
        using Ty = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value;
        if (H / V <= NARROW) {
            const int blocks = static_cast<int>((static_cast<long long>(T) * (H / V) + COMBINE_BLOCK - 1) / COMBINE_BLOCK);
            combine_narrow_kernel<Ty, V><<<blocks, COMBINE_BLOCK, 0, static_cast<cudaStream_t>(stream)>>>(a);
            return;
        }
        constexpr int RUN = COMBINE_BLOCK * PACKS<Ty, V>;
        const int runs = (H / V + RUN - 1) / RUN;
        // tokens a block: as many as leave about eight blocks an SM, up to eight
        const long long each = static_cast<long long>(T) * runs / (8 * sms);
        const int tokens = each < 1 ? 1 : each > 8 ? 8 : static_cast<int>(each);
        const int groups = (T + tokens - 1) / tokens, gy = groups < 32768 ? groups : 32768;
        combine_rows_kernel<Ty, V><<<dim3(runs, gy, (groups + gy - 1) / gy), COMBINE_BLOCK, 0, static_cast<cudaStream_t>(stream)>>>(a, tokens);
    });
}

int moe_combine_rows_backward(int T, int topk, int H, int E, int64_t M, const void *dout, int64_t lddout, const void *y,
                              int dtype, const int32_t *rows, const float *w, const int32_t *offsets, void *dy,
                              float *dw, void *stream)
{
    if (!rows_sizes_ok(T, topk, H, M, dtype) || E < 1 || lddout < H)
        return MOE_ERR_INVALID_ARG;
    if (T == 0 && M == 0)
        return MOE_OK;
    const size_t b = dtype_bytes(dtype);
    if (!offsets || !op_aligned(offsets, 4) || (M > 0 && (!y || !dy)) || !op_aligned(y, b) || !op_aligned(dy, b) ||
        (T > 0 && (!dout || !rows || !op_aligned(dout, b) || !op_aligned(rows, 4))) || !op_aligned(w, 4) || !op_aligned(dw, 4))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    const RowArgs a{T, topk, H, static_cast<int>(M), dout, lddout, y, rows, w, offsets + E, nullptr, dy, dw};
    return by_rows(dtype, H, lddout, dout, y, dy, [&](auto *t, auto v) {
        using Ty = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value;
        if (H / V <= NARROW) {
            const int blocks = (T + COMBINE_BLOCK / 32 - 1) / (COMBINE_BLOCK / 32);
            combine_narrow_backward_kernel<Ty, V><<<blocks + sms, COMBINE_BLOCK, 0, static_cast<cudaStream_t>(stream)>>>(a, blocks);
            return;
        }
        combine_rows_backward_kernel<Ty, V><<<T + sms, backward_threads(H / V, T, sms), 0, static_cast<cudaStream_t>(stream)>>>(a);
    });
}

}  // extern "C"
