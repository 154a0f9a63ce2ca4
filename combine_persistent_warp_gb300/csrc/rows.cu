// rows.cu -- rows moved from token order into expert-major order and weighted back out of it,
// with both directions' gradients.  rows[t][j] is the row of slot j of token t (-1: none).
//
//   gather    out[rows[t][j]] = x[t]
//   combine   out[t] = sum_j w[t][j] * y[rows[t][j]]      (fp32, j ascending, rounded once)
//   its gradients   dy[rows[t][j]] = w[t][j] * dout[t],   dw[t][j] = sum_h dout[t][h] * y[rows[t][j]][h]
//
// The gradient of gather is combine with w = 1.  All three are bound by HBM: a thread handles 16 bytes
// of a token for all of its slots, so the token's row is read (or written) once however many
// slots it has, and every row in expert order once.  Gather and combine take the vectors of all
// tokens in a line, so that no lane is left over whatever a row's length.
//
// Measured on a GB300, bf16: gather of 16384 x 8 x 4096 180 us (floor 181); combine of 8192 x 8 x 7168
// 174 us (158) and with its gradients, 5% of the slots skipped, 457 us (444); combine of 128 x 8 x
// 7168 3.7 us; 8000 x 4 x 3000 gather 38 us, combine 45, gradients 68 (36, 36, 65), and with 3001
// columns, off 16-byte boundaries, 43, 58 and 78.
#include <type_traits>

#include "op_common.cuh"
#include "rows_index.h"

using namespace cpw;

namespace {

constexpr int MAX_K = 32;
// Slots of a token whose loads are in flight together.  Four need few enough registers for twice the
// warps, and a call of up to four slots a token has no others (gradients of 8000 x 4 x 3000: 68 us,
// 83 with eight; 16384 x 2 x 4096: 110 and 154); with more, eight (8192 x 8 x 7168: 292 us, 310 with
// four at a time).
constexpr int SLOTS = 8, FEW_SLOTS = 4;
constexpr int BLOCK = 128;
// Gradients: packs (or vectors) of a row up to which a warp takes a token instead of a block: it has no
// barrier to wait at (16384 x 8 x 400: 45 us, 51 with blocks), and twice as many where there are
// tokens enough to fill the GPU with warps (16384 x 8 x 1024: 89 and 107; 1000 tokens of 777 columns:
// 15.6 and 12.3).
constexpr int NARROW = 96;
// The same for rows off 16-byte boundaries: elements up to which a warp moves them one by one; the
// shifted vectors' ends cost more (16384 x 8 x 289: 64 us, 78 shifted; 777: 41 and 36).
constexpr int NARROW_ELEMENTS = 512;
// And for gather (16384 x 8 x 33: 6.2 us, 14.0 shifted; 8000 x 2 x 95: 6.6 and 4.2).
constexpr int SHORT = 64;
// Gradients with a block a token: its threads (8192 x 8 x 7168 bf16, both passes: 493 us; 64: 497, 256:
// 507, 448: 550).
constexpr int BWD_BLOCK = 128;

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
    int rim;                 // see amid()
};

// Row and weight of slot j of token t (-1 and 0 where there is none).
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
// Slots j0 .. j0 + S - 1 of a warp's token: one load a lane, then shuffles.
template <int S>
__device__ __forceinline__ void load_slots(const RowArgs &a, int t, int j0, int (&r)[S], float (&w)[S])
{
    const int lane = threadIdx.x & 31;
    int row = -1;
    float weight = 0.0f;
    if (lane < S)
        slot_of(a, t, j0 + lane, row, weight);
#pragma unroll
    for (int i = 0; i < S; ++i) {
        r[i] = __shfl_sync(0xFFFFFFFFu, row, i);
        w[i] = __shfl_sync(0xFFFFFFFFu, weight, i);
    }
}

// Zeroes the rows that no slot names; block b of `blocks`.
template <typename T, int V>
__device__ __forceinline__ void zero_rest(const RowArgs &a, void *out, int b, int blocks)
{
    const int packs = a.H / V;
    const int first = rest_begin(*a.total, a.M);
    Pack<T, V> z;
#pragma unroll
    for (int i = 0; i < V; ++i)
        z.v[i] = from_f<T>(0.0f);
    for (int r = first + b; r < a.M; r += blocks)
        for (int p = threadIdx.x; p < packs; p += blockDim.x)
            store_pack<T, V>(static_cast<T *>(out) + static_cast<size_t>(r) * a.H + static_cast<size_t>(p) * V, z);
}

// One pack of a token's gradient: its part of the slots' sums, and the rows' gradients.
template <typename T, int V, int S>
struct PackBackward {
    static constexpr int AT_ONCE = S, BLOCKS = S == SLOTS ? 1 : 2;
    int count;   // packs of a row
    __device__ __forceinline__ void operator()(const RowArgs &a, int, const T *d, const T *y, T *dy, int p, const int (&r)[S],
                                               const float (&w)[S], float (&dot)[S]) const
    {
        const Pack<T, V> q = load_pack<T, V>(d + static_cast<size_t>(p) * V);
        Pack<T, V> v[S];
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (r[i] >= 0)
                v[i] = load_pack<T, V>(y + static_cast<size_t>(r[i]) * a.H + static_cast<size_t>(p) * V);
#pragma unroll
        for (int i = 0; i < S; ++i)
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
    __device__ __forceinline__ void zero(const RowArgs &a, int b, int blocks) const { zero_rest<T, V>(a, a.dy, b, blocks); }
};

// Vectors (or elements) of all tokens in a line; a thread takes `run` of them, a block's width apart.
struct Line {
    int t, g;
};
__device__ __forceinline__ Line line_start(int vectors, int run)
{
    const long long i = static_cast<long long>(blockIdx.x) * BLOCK * run + threadIdx.x;
    const int t = static_cast<int>(i / vectors);
    return {t, static_cast<int>(i - static_cast<long long>(t) * vectors)};
}
__device__ __forceinline__ void line_step(Line &l, int vectors)
{
    for (l.g += BLOCK; l.g >= vectors; l.g -= vectors)
        ++l.t;
}

template <typename T, int V>
__global__ void __launch_bounds__(BLOCK) gather_kernel(const RowArgs a, int vectors, int blocks)
{
    if (static_cast<int>(blockIdx.x) >= blocks) {
        zero_rest<T, V>(a, a.out, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
    const Line l = line_start(vectors, 1);
    if (l.t >= a.T)
        return;
    const Pack<T, V> v = load_pack<T, V>(static_cast<const T *>(a.x) + static_cast<size_t>(l.t) * a.ldx + static_cast<size_t>(l.g) * V);
    for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
        int r[SLOTS];
        float w[SLOTS];
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            slot_of(a, l.t, j0 + i, r[i], w[i]);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            if (r[i] >= 0)
                store_pack<T, V>(static_cast<T *>(a.out) + static_cast<size_t>(r[i]) * a.H + static_cast<size_t>(l.g) * V, v);
    }
}

// S slots' loads in flight together.
template <typename T, int S>
__global__ void __launch_bounds__(BLOCK) combine_kernel(const RowArgs a, int vectors, int run)
{
    constexpr int V = VEC<T>;
    Line l = line_start(vectors, run);
    for (int n = 0; n < run && l.t < a.T; ++n, line_step(l, vectors)) {
        const T *y = static_cast<const T *>(a.y) + static_cast<size_t>(l.g) * V;
        float acc[V];
#pragma unroll
        for (int c = 0; c < V; ++c)
            acc[c] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += S) {
            int r[S];
            float w[S];
            uint4 q[S];
#pragma unroll
            for (int i = 0; i < S; ++i)
                slot_of(a, l.t, j0 + i, r[i], w[i]);
#pragma unroll
            for (int i = 0; i < S; ++i)
                q[i] = load_aligned(y + static_cast<long long>(r[i]) * a.H, r[i] >= 0);
#pragma unroll
            for (int i = 0; i < S; ++i) {   // (an absent slot adds 0 * 0)
                const Pack<T, V> v = reinterpret_cast<const Pack<T, V> &>(q[i]);
#pragma unroll
                for (int c = 0; c < V; ++c)
                    acc[c] = fmaf(w[i], to_f<T>(v.v[c]), acc[c]);
            }
        }
        Pack<T, V> o;
#pragma unroll
        for (int c = 0; c < V; ++c)
            o.v[c] = from_f<T>(acc[c]);
        store_pack<T, V>(static_cast<T *>(a.out) + static_cast<size_t>(l.t) * a.H + static_cast<size_t>(l.g) * V, o);
    }
}

// ------------------------------------------------------------------ rows of any alignment ----
// Where rows do not all start on 16-byte boundaries, a row is written in the aligned 16-byte
// vectors of its own place: vector g starts at element g * V - lead_of(row).  Its bytes come from the
// two aligned vectors of the source that cover them, shifted (the lanes' second vectors are their
// neighbours' first, so they come from L1).  Those may hold bytes of the neighbouring rows, which
// are not used, but none outside the matrix: a vector whose sources might leave it is moved by
// elements.  Nothing outside a row is written.

// Elements e .. e + V - 1 of a row one by one, zeros outside it.
template <typename T>
__device__ __forceinline__ Pack<T, VEC<T>> load_elements(const T *row, int e, int H)
{
    Pack<T, VEC<T>> v;
#pragma unroll
    for (int c = 0; c < VEC<T>; ++c)
        v.v[c] = e + c >= 0 && e + c < H ? __ldg(row + e + c) : from_f<T>(0.0f);
    return v;
}
// Elements e .. e + V - 1 of a row, where e is a multiple of V from its first vector.
template <typename T>
__device__ __forceinline__ void store_vector(T *row, int e, int H, const Pack<T, VEC<T>> &v)
{
    if (e >= 0 && e + VEC<T> <= H) {
        store_pack<T, VEC<T>>(row + e, v);
    } else {
#pragma unroll
        for (int c = 0; c < VEC<T>; ++c)
            if (e + c >= 0 && e + c < H)
                row[e + c] = v.v[c];
    }
}

template <typename T>
__device__ __forceinline__ void zero_rest_shifted(const RowArgs &a, void *out, int vectors, int b, int blocks)
{
    constexpr int V = VEC<T>;
    const int first = rest_begin(*a.total, a.M);
    Pack<T, V> z;
#pragma unroll
    for (int i = 0; i < V; ++i)
        z.v[i] = from_f<T>(0.0f);
    for (int r = first + b; r < a.M; r += blocks) {
        T *o = static_cast<T *>(out) + static_cast<size_t>(r) * a.H;
        for (int g = threadIdx.x; g < vectors; g += blockDim.x)
            store_vector<T>(o, g * V - lead_of(o), a.H, z);
    }
}

template <typename T>
__global__ void __launch_bounds__(BLOCK) gather_shifted_kernel(const RowArgs a, int vectors, int blocks)
{
    constexpr int V = VEC<T>;
    if (static_cast<int>(blockIdx.x) >= blocks) {
        zero_rest_shifted<T>(a, a.out, vectors, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
    const Line l = line_start(vectors, 1);
    if (l.t >= a.T)
        return;
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(l.t) * a.ldx;
    const bool in = inside(l.g, a.H, VEC<T>) || amid(l.t, a.T, a.rim);
    for (int j0 = 0; j0 < a.k; j0 += FEW_SLOTS) {
        int r[FEW_SLOTS];
        float w[FEW_SLOTS];
#pragma unroll
        for (int i = 0; i < FEW_SLOTS; ++i)
            slot_of(a, l.t, j0 + i, r[i], w[i]);
#pragma unroll
        for (int i = 0; i < FEW_SLOTS; ++i)
            if (r[i] >= 0) {
                T *o = static_cast<T *>(a.out) + static_cast<size_t>(r[i]) * a.H;
                const int e = l.g * V - lead_of(o);
                store_vector<T>(o, e, a.H, in ? shifted(load_halves(x + e), x + e) : load_elements(x, e, a.H));
            }
    }
}

template <typename T>
__global__ void __launch_bounds__(BLOCK) combine_shifted_kernel(const RowArgs a, int vectors, int run)
{
    constexpr int V = VEC<T>;
    const T *y = static_cast<const T *>(a.y);
    Line l = line_start(vectors, run);
    for (int n = 0; n < run && l.t < a.T; ++n, line_step(l, vectors)) {
        T *out = static_cast<T *>(a.out) + static_cast<size_t>(l.t) * a.H;
        const int e = l.g * V - lead_of(out);
        int r[FEW_SLOTS];
        float w[FEW_SLOTS];
        float acc[V];
#pragma unroll
        for (int c = 0; c < V; ++c)
            acc[c] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += FEW_SLOTS) {
            bool in = true;
#pragma unroll
            for (int i = 0; i < FEW_SLOTS; ++i) {
                slot_of(a, l.t, j0 + i, r[i], w[i]);
                in = in && (r[i] < 0 || amid(r[i], a.M, a.rim));
            }
            if (in || inside(l.g, a.H, VEC<T>)) {
                Halves h[FEW_SLOTS];
#pragma unroll
                for (int i = 0; i < FEW_SLOTS; ++i)
                    h[i] = load_halves(y + static_cast<long long>(r[i]) * a.H + e, r[i] >= 0);
#pragma unroll
                for (int i = 0; i < FEW_SLOTS; ++i) {
                    if (r[i] < 0)
                        continue;
                    const Pack<T, V> v = shifted(h[i], y + static_cast<long long>(r[i]) * a.H + e);
#pragma unroll
                    for (int c = 0; c < V; ++c)
                        acc[c] = fmaf(w[i], to_f<T>(v.v[c]), acc[c]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < FEW_SLOTS; ++i) {
                    if (r[i] < 0)
                        continue;
                    const Pack<T, V> v = load_elements(y + static_cast<long long>(r[i]) * a.H, e, a.H);
#pragma unroll
                    for (int c = 0; c < V; ++c)
                        acc[c] = fmaf(w[i], to_f<T>(v.v[c]), acc[c]);
                }
            }
        }
        Pack<T, V> o;
#pragma unroll
        for (int c = 0; c < V; ++c)
            o.v[c] = from_f<T>(acc[c]);
        store_vector<T>(out, e, a.H, o);
    }
}

// Vector g of a token's gradient.  (Each slot's row has vectors of its own: their columns differ
// between the slots, and the token's sums take every column of each once.)
// SAME: rows of y and dy start alike, so that those of y need no shift.
template <typename T, bool SAME>
struct ShiftedBackward {
    static constexpr int AT_ONCE = FEW_SLOTS, BLOCKS = 2;
    int count;
    __device__ __forceinline__ void operator()(const RowArgs &a, int t, const T *d, const T *y, T *dy, int g, const int (&r)[FEW_SLOTS],
                                               const float (&w)[FEW_SLOTS], float (&dot)[FEW_SLOTS]) const
    {
        constexpr int V = VEC<T>;
        const bool whole = g >= 1 && (g + 1) * V <= a.H;   // for any lead
        bool in = amid(t, a.T, a.rim);
        int e[FEW_SLOTS];
#pragma unroll
        for (int i = 0; i < FEW_SLOTS; ++i) {
            e[i] = g * V - lead_of(dy + static_cast<long long>(r[i]) * a.H);
            in = in && (r[i] < 0 || amid(r[i], a.M, a.rim));
        }
        if (in || inside(g, a.H, VEC<T>)) {
            uint4 lo[FEW_SLOTS], hi[SAME ? 1 : FEW_SLOTS];
#pragma unroll
            for (int i = 0; i < FEW_SLOTS; ++i) {
                const T *at = y + static_cast<long long>(r[i]) * a.H + e[i];
                lo[i] = load_aligned(at, r[i] >= 0);
                if constexpr (!SAME)
                    hi[i] = load_aligned(at, r[i] >= 0, 1);
            }
#pragma unroll
            for (int i = 0; i < FEW_SLOTS; ++i) {
                if (r[i] < 0)
                    continue;
                const long long at = static_cast<long long>(r[i]) * a.H;
                Pack<T, V> v;
                if constexpr (SAME)
                    v = reinterpret_cast<const Pack<T, V> &>(lo[i]);
                else
                    v = shifted(Halves{lo[i], hi[i]}, y + at + e[i]);
                const Pack<T, V> q = shifted(load_halves(d + e[i]), d + e[i]);
                Pack<T, V> o;
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    const float f = to_f<T>(q.v[c]);
                    o.v[c] = from_f<T>(w[i] * f);
                    dot[i] = whole || (e[i] + c >= 0 && e[i] + c < a.H) ? fmaf(f, to_f<T>(v.v[c]), dot[i]) : dot[i];
                }
                if (whole)
                    store_pack<T, V>(dy + at + e[i], o);
                else
                    store_vector<T>(dy + at, e[i], a.H, o);
            }
        } else {
#pragma unroll
            for (int i = 0; i < FEW_SLOTS; ++i) {
                if (r[i] < 0)
                    continue;
                const long long at = static_cast<long long>(r[i]) * a.H;
                const Pack<T, V> v = load_elements(y + at, e[i], a.H), q = load_elements(d, e[i], a.H);
                Pack<T, V> o;
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    const float f = to_f<T>(q.v[c]);
                    dot[i] = fmaf(f, to_f<T>(v.v[c]), dot[i]);
                    o.v[c] = from_f<T>(w[i] * f);
                }
                store_vector<T>(dy + at, e[i], a.H, o);
            }
        }
    }
    __device__ __forceinline__ void zero(const RowArgs &a, int b, int blocks) const { zero_rest_shifted<T>(a, a.dy, count, b, blocks); }
};

// ------------------------------------------------------------------ gradients of combine ----
// A warp a token: its sums over the columns need no other warp.
template <typename T, typename PART>
__global__ void __launch_bounds__(BLOCK) combine_backward_warp_kernel(const RowArgs a, const PART part, int blocks)
{
    if (static_cast<int>(blockIdx.x) >= blocks) {
        part.zero(a, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
    const int t = blockIdx.x * (BLOCK / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= a.T)
        return;
    const T *d = static_cast<const T *>(a.x) + static_cast<size_t>(t) * a.ldx;
    const T *y = static_cast<const T *>(a.y);
    T *dy = static_cast<T *>(a.dy);
    for (int j0 = 0; j0 < a.k; j0 += PART::AT_ONCE) {
        int r[PART::AT_ONCE];
        float w[PART::AT_ONCE], dot[PART::AT_ONCE];
        load_slots(a, t, j0, r, w);
#pragma unroll
        for (int s = 0; s < PART::AT_ONCE; ++s)
            dot[s] = 0.0f;
        for (int p = lane; p < part.count; p += 32)
            part(a, t, d, y, dy, p, r, w, dot);
        float mine = 0.0f;
#pragma unroll
        for (int s = 0; s < PART::AT_ONCE; ++s) {
            const float v = warp_sum(dot[s]);
            mine = lane == s ? v : mine;
        }
        if (a.dw && lane < PART::AT_ONCE && j0 + lane < a.k)
            a.dw[static_cast<size_t>(t) * a.k + j0 + lane] = mine;
    }
}

// A block takes a whole token, for the sums over its columns.
template <typename T, typename PART>
__global__ void __launch_bounds__(512, PART::BLOCKS) combine_backward_kernel(const RowArgs a, const PART part)
{
    if (static_cast<int>(blockIdx.x) >= a.T) {
        part.zero(a, blockIdx.x - a.T, gridDim.x - a.T);
        return;
    }
    __shared__ float red[16][PART::AT_ONCE];
    const int t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const T *d = static_cast<const T *>(a.x) + static_cast<size_t>(t) * a.ldx;
    const T *y = static_cast<const T *>(a.y);
    T *dy = static_cast<T *>(a.dy);
    for (int j0 = 0; j0 < a.k; j0 += PART::AT_ONCE) {
        int r[PART::AT_ONCE];
        float w[PART::AT_ONCE], dot[PART::AT_ONCE];
        load_slots(a, t, j0, r, w);
#pragma unroll
        for (int i = 0; i < PART::AT_ONCE; ++i)
            dot[i] = 0.0f;
        for (int p = threadIdx.x; p < part.count; p += blockDim.x)
            part(a, t, d, y, dy, p, r, w, dot);
#pragma unroll
        for (int i = 0; i < PART::AT_ONCE; ++i)
            dot[i] = warp_sum(dot[i]);
        __syncthreads();
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < PART::AT_ONCE; ++i)
                red[warp][i] = dot[i];
        }
        __syncthreads();
        if (a.dw && threadIdx.x < PART::AT_ONCE && j0 + static_cast<int>(threadIdx.x) < a.k) {
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

// Small blocks, of which many share an SM, unless there are few tokens (128 x 8 x 7168: 5.1 us, 6.3 with
// small blocks; 500 tokens: 25.7 and 19.7).
int backward_threads(int packs, int T, int sms)
{
    const int most = rows_threads(packs);
    return T > sms && most > BWD_BLOCK ? BWD_BLOCK : most;
}

bool rows_sizes_ok(int T, int k, int H, long long M, int dtype)
{
    return T >= 0 && T <= MAX_ROWS && k >= 1 && k <= MAX_K && H >= 1 && H <= MAX_ROWS && M >= 0 && M <= MAX_ROWS && dtype_ok(dtype);
}

// Calls `aligned` where every row starts on a 16-byte boundary, `shifted` otherwise.
template <typename F, typename G>
int by_rows(int dtype, int H, long long ldx, const void *p0, const void *p1, const void *p2, F aligned, G shifted)
{
    const size_t b = dtype_bytes(dtype);
    const bool all = H * b % 16 == 0 && static_cast<size_t>(ldx) * b % 16 == 0 && op_aligned(p0, 16) && op_aligned(p1, 16) &&
                     op_aligned(p2, 16);
    with_dtype(dtype, [&](auto *t) {
        if (all)
            aligned(t);
        else
            shifted(t);
    });
    return launched();
}

// Vectors of combine that a thread takes: up to four, as long as a block stays within a token and there
// are about sixteen blocks an SM (8192 x 8 x 7168: 174 us, 184 with one; 16384 x 8 x 1024: 62 with
// four, 57 with one).
int run_of(long long T, int vectors, int sms)
{
    const long long blocks = T * vectors / (16ll * BLOCK * sms), token = vectors / BLOCK;
    const long long run = blocks < token ? blocks : token;
    return run < 1 ? 1 : run > 4 ? 4 : static_cast<int>(run);
}
int blocks_of(long long T, int vectors, int run)
{
    return static_cast<int>((T * vectors + BLOCK * run - 1) / (BLOCK * run));
}

template <typename T, typename PART>
void launch_warps(const RowArgs &a, const PART &part, int sms, cudaStream_t stream)
{
    const int blocks = (a.T + BLOCK / 32 - 1) / (BLOCK / 32);
    combine_backward_warp_kernel<T, PART><<<blocks + sms, BLOCK, 0, stream>>>(a, part, blocks);
}
template <typename T, typename PART>
void launch_backward(const RowArgs &a, const PART &part, int sms, cudaStream_t stream)
{
    if (part.count <= (a.T > 16 * sms ? 2 * NARROW : NARROW))
        launch_warps<T>(a, part, sms, stream);
    else
        combine_backward_kernel<T, PART><<<a.T + sms, backward_threads(part.count, a.T, sms), 0, stream>>>(a, part);
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
    RowArgs a{T, topk, H, static_cast<int>(M), x, ldx, nullptr, rows, nullptr, offsets + E, out, nullptr, nullptr, 0};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return by_rows(dtype, H, ldx, x, out, nullptr, [&](auto *t) {
        using Ty = std::remove_pointer_t<decltype(t)>;
        const int vectors = H / VEC<Ty>, blocks = blocks_of(T, vectors, 1);
        gather_kernel<Ty, VEC<Ty>><<<blocks + sms, BLOCK, 0, st>>>(a, vectors, blocks);
    }, [&](auto *t) {
        using Ty = std::remove_pointer_t<decltype(t)>;
        if (H <= SHORT) {
            const int blocks = blocks_of(T, H, 1);
            gather_kernel<Ty, 1><<<blocks + sms, BLOCK, 0, st>>>(a, H, blocks);
            return;
        }
        a.rim = rim_of(H, VEC<Ty>);
        const int vectors = vectors_of(H, VEC<Ty>), blocks = blocks_of(T, vectors, 1);
        gather_shifted_kernel<Ty><<<blocks + sms, BLOCK, 0, st>>>(a, vectors, blocks);
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
    RowArgs a{T, topk, H, static_cast<int>(M), nullptr, H, y, rows, w, nullptr, out, nullptr, nullptr, 0};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return by_rows(dtype, H, H, y, out, nullptr, [&](auto *t) {
        using Ty = std::remove_pointer_t<decltype(t)>;
        const int vectors = H / VEC<Ty>, run = run_of(T, vectors, sms), blocks = blocks_of(T, vectors, run);
        if (topk <= FEW_SLOTS)
            combine_kernel<Ty, FEW_SLOTS><<<blocks, BLOCK, 0, st>>>(a, vectors, run);
        else
            combine_kernel<Ty, SLOTS><<<blocks, BLOCK, 0, st>>>(a, vectors, run);
    }, [&](auto *t) {
        using Ty = std::remove_pointer_t<decltype(t)>;
        a.rim = rim_of(H, VEC<Ty>);
        const int vectors = vectors_of(H, VEC<Ty>), run = run_of(T, vectors, sms);
        combine_shifted_kernel<Ty><<<blocks_of(T, vectors, run), BLOCK, 0, st>>>(a, vectors, run);
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
    RowArgs a{T, topk, H, static_cast<int>(M), dout, lddout, y, rows, w, offsets + E, nullptr, dy, dw, 0};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return by_rows(dtype, H, lddout, dout, y, dy, [&](auto *t) {
        using Ty = std::remove_pointer_t<decltype(t)>;
        if (topk <= FEW_SLOTS)
            launch_backward<Ty>(a, PackBackward<Ty, VEC<Ty>, FEW_SLOTS>{H / VEC<Ty>}, sms, st);
        else
            launch_backward<Ty>(a, PackBackward<Ty, VEC<Ty>, SLOTS>{H / VEC<Ty>}, sms, st);
    }, [&](auto *t) {
        using Ty = std::remove_pointer_t<decltype(t)>;
        a.rim = rim_of(H, VEC<Ty>);
        if (H <= NARROW_ELEMENTS && topk <= FEW_SLOTS)
            launch_warps<Ty>(a, PackBackward<Ty, 1, FEW_SLOTS>{H}, sms, st);
        else if (H <= NARROW_ELEMENTS)
            launch_warps<Ty>(a, PackBackward<Ty, 1, SLOTS>{H}, sms, st);
        else if (op_aligned(reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(y) - reinterpret_cast<uintptr_t>(dy)), 16))
            launch_backward<Ty>(a, ShiftedBackward<Ty, true>{vectors_of(H, VEC<Ty>)}, sms, st);
        else
            launch_backward<Ty>(a, ShiftedBackward<Ty, false>{vectors_of(H, VEC<Ty>)}, sms, st);
    });
}

}  // extern "C"
