// router.cu -- the router of an expert layer: top-k experts of each token with their gate
// weights, the gradient of the logits, and the expert-major order of the chosen slots.
//
//   chosen: the k largest logits of a token, ties to the lowest index; a NaN counts as the
//   largest value, a logit of -inf is never chosen, a masked token chooses nothing (-1, 0)
//   renormalised gate weights  w_j = exp(l_j - m) / sum_i exp(l_i - m) over the chosen ones
//   otherwise                  w_j = exp(l_j - m) / sum_e exp(l_e - m) over all experts
//   gradient, renormalised     dl_j = w_j (dw_j - sum_i w_i dw_i), zero elsewhere
//   otherwise                  dl_e = p_e ([e chosen] dw_e - sum_i w_i dw_i)
//
// A warp takes a token and holds its logits in registers.  The data is small (a few MB at 16384
// tokens), so issue and latency bound these kernels, not bandwidth.  Measured on a GB300 in a graph:
// 16384 x 128 bf16, top 8: choice 8.9 us, order 7.4 us, gradient 5.0 to 5.4 us (softmax over
// all experts: choice 9.6, gradient 7.1); 128 x 32 fp32: 2.0, 3.1 and 1.6 to 1.9 us.
#include <climits>
#include <type_traits>

#include "op_common.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"
#include "router_common.cuh"

using namespace cpw;

namespace {

struct RouteArgs {
    int T, E, k;
    const void *logits;
    long long ld;
    const uint8_t *mask;   // nonzero: the token is routed (null: every token)
    int renorm;
    int64_t *idx;
    float *w;
};

// The k largest of a token's logits, IPL a lane (lane l holds experts l, l + 32, ...): one warp
// maximum and one warp minimum a slot.  Returns how many there are; lane j gets slot j's expert and
// logit, every lane the largest logit.
template <int IPL>
__device__ __forceinline__ int choose(int k, const float (&f)[IPL], int lane, int &my_idx, float &mine, float &top)
{
    uint32_t key[IPL], kept = 0u, first = 0u;
#pragma unroll
    for (int i = 0; i < IPL; ++i)
        key[i] = order_key(f[i]);
    int j = 0;
    for (; j < k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < IPL; ++i)
            best = max(best, key[i]);
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
        if (m == 0)
            break;   // only logits of -inf are left
        int at = INT_MAX;
#pragma unroll
        for (int i = IPL - 1; i >= 0; --i)
            at = key[i] == m ? i * 32 + lane : at;
        const int e = __reduce_min_sync(0xFFFFFFFFu, at);
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            key[i] = i * 32 + lane == e ? 0u : key[i];
        my_idx = lane == j ? e : my_idx;
        kept = lane == j ? m : kept;
        first = j == 0 ? m : first;
    }
    mine = key_value(kept);
    top = key_value(first);
    return j;
}

// 16-bit logits: the key (its upper 19 bits: the fp32 image of a 16-bit float has a sign, 8 bits
// of exponent and at most 10 of fraction) and the expert (10 bits, ties to the lowest) fit one
// word, so one warp maximum a slot finds both.
constexpr uint32_t KEY16 = 0xFFFFE000u;
__device__ __forceinline__ float key16_value(uint32_t word)
{
    // the low bits of a positive value's key are zeros, of a negative one's are ones
    const uint32_t up = word & KEY16;
    return up == KEY16 ? __uint_as_float(0x7FC00000u) : key_value((up & 0x80000000u) ? up : up | ~KEY16);
}
template <int IPL>
__device__ __forceinline__ int choose16(int k, const float (&f)[IPL], int lane, int &my_idx, float &mine, float &top)
{
    uint32_t key[IPL], kept = 0u, first = 0u;
#pragma unroll
    for (int i = 0; i < IPL; ++i) {
        const uint32_t v = order_key(f[i]);
        key[i] = v == 0u ? 0u : (v & KEY16) | static_cast<uint32_t>(1023 - (i * 32 + lane));
    }
    int j = 0;
    for (; j < k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < IPL; ++i)
            best = max(best, key[i]);
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
        if (m == 0)
            break;
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            key[i] = key[i] == m ? 0u : key[i];
        kept = lane == j ? m : kept;
        first = j == 0 ? m : first;
    }
    if (lane < j)
        my_idx = 1023 - static_cast<int>(kept & ~KEY16);
    mine = key16_value(kept);
    top = key16_value(first);
    return j;
}

template <typename T, int IPL>
__global__ void __launch_bounds__(WARPS * 32) route_kernel(const RouteArgs a)
{
    const int t = blockIdx.x * WARPS + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= a.T)
        return;
    int my_idx = -1;
    float my_w = 0.0f;
    if (!a.mask || a.mask[t]) {
        const T *l = static_cast<const T *>(a.logits) + static_cast<size_t>(t) * a.ld;
        float f[IPL];
#pragma unroll
        for (int i = 0; i < IPL; ++i) {
            const int e = i * 32 + lane;
            f[i] = e < a.E ? to_f<T>(l[e]) : -INFINITY;
        }
        float top = 0.0f, mine = 0.0f;
        int found;
        if constexpr (sizeof(T) == 2)
            found = choose16<IPL>(a.k, f, lane, my_idx, mine, top);
        else
            found = choose<IPL>(a.k, f, lane, my_idx, mine, top);
        const float p = lane < found ? expf(mine - top) : 0.0f;
        float sum = p;
        if (!a.renorm) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                if (i * 32 + lane < a.E)
                    sum += expf(f[i] - top);
        }
        sum = warp_sum(sum);
        if (lane < found)
            my_w = p / sum;
    }
    if (lane < a.k) {
        a.idx[static_cast<size_t>(t) * a.k + lane] = my_idx;
        a.w[static_cast<size_t>(t) * a.k + lane] = my_w;
    }
}

struct RouteBwdArgs {
    int T, E, k;
    const float *dw;
    const int64_t *idx;
    const float *w;
    const void *logits;   // read only where not renormalised
    long long ld;
    int renorm;
    void *dlogits;        // [T][E]
};

template <typename T, int IPL>
__global__ void __launch_bounds__(WARPS * 32) route_backward_kernel(const RouteBwdArgs a)
{
    const int t = blockIdx.x * WARPS + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= a.T)
        return;
    int e = -1;
    float w = 0.0f, dw = 0.0f;
    if (lane < a.k) {
        const size_t at = static_cast<size_t>(t) * a.k + lane;
        const int64_t id = a.idx[at];
        e = id >= 0 && id < a.E ? static_cast<int>(id) : -1;
        if (e >= 0) {
            w = a.w[at];
            dw = a.dw[at];
        }
    }
    const float dot = warp_sum(w * dw);
    const bool any = __any_sync(0xFFFFFFFFu, e >= 0);
    float d[IPL];
    if (a.renorm || !any) {
        const float mine = w * (dw - dot);
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            d[i] = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int ej = __shfl_sync(0xFFFFFFFFu, e, j);
            const float v = __shfl_sync(0xFFFFFFFFu, mine, j);
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                d[i] += ej == i * 32 + lane ? v : 0.0f;
        }
    } else {
        const T *l = static_cast<const T *>(a.logits) + static_cast<size_t>(t) * a.ld;
        float f[IPL], m = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < IPL; ++i) {
            const int ei = i * 32 + lane;
            f[i] = ei < a.E ? to_f<T>(l[ei]) : -INFINITY;
            m = fmaxf(m, f[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
#pragma unroll
        for (int i = 0; i < IPL; ++i) {
            f[i] = expf(f[i] - m);   // NaN logits and m = +inf make NaN, as in the forward pass
            if (i * 32 + lane < a.E)
                sum += f[i];
        }
        const float inv = 1.0f / warp_sum(sum);
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            d[i] = -dot;
        for (int j = 0; j < a.k; ++j) {
            const int ej = __shfl_sync(0xFFFFFFFFu, e, j);
            const float v = __shfl_sync(0xFFFFFFFFu, dw, j);
#pragma unroll
            for (int i = 0; i < IPL; ++i)
                d[i] += ej == i * 32 + lane ? v : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < IPL; ++i)
            d[i] *= f[i] * inv;
    }
    T *out = static_cast<T *>(a.dlogits) + static_cast<size_t>(t) * a.E;
#pragma unroll
    for (int i = 0; i < IPL; ++i) {
        const int ei = i * 32 + lane;
        if (ei < a.E)
            out[ei] = from_f<T>(d[i]);
    }
}

// ------------------------------------------------------------------ expert-major order ----
// A stable counting sort of the n = T*k slots by expert.  Each block has a run of `chunk`
// slots, each of its warps an equal part of it; counts per (warp, expert) in shared memory give
// every slot its row without atomics on shared results, so equal inputs give equal rows.  More
// than one block: a first kernel counts each block's slots, and every block of the second sums
// the counts of all blocks for itself.
constexpr int ORDER_THREADS = 512;
constexpr int ORDER_WARPS = ORDER_THREADS / 32;
constexpr int ORDER_CHUNK = 2048;
constexpr int ORDER_SLOTS = ORDER_CHUNK / ORDER_THREADS;   // slots of a lane in a run of ORDER_CHUNK

struct OrderArgs {
    int n, E, chunk;
    const int64_t *idx;
    int32_t *offsets;   // [E+1]
    int32_t *rows;      // [n]
    int32_t *status;
    int32_t *hist;      // [blocks][E] (more than one block)
};

__device__ __forceinline__ int slot_expert(const OrderArgs &a, int i, bool &bad)
{
    const int64_t v = a.idx[i];
    if (v >= 0 && v < a.E)
        return static_cast<int>(v);
    bad = bad || v != -1;
    return -1;
}

__global__ void __launch_bounds__(ORDER_THREADS) order_count_kernel(const OrderArgs a)
{
    extern __shared__ int32_t cnt[];   // [E]
    ptx::launch_dependents();
    for (int e = threadIdx.x; e < a.E; e += ORDER_THREADS)
        cnt[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *a.status = MOE_OK;   // before the placing kernel, whose blocks record bad ids
    __syncthreads();
    const int lo = blockIdx.x * a.chunk, hi = min(a.n, lo + a.chunk);
    bool bad = false;
#pragma unroll 4
    for (int i = lo + threadIdx.x; i < hi; i += ORDER_THREADS) {
        const int e = slot_expert(a, i, bad);
        if (e >= 0)
            atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += ORDER_THREADS)
        a.hist[static_cast<size_t>(blockIdx.x) * a.E + e] = cnt[e];
}

// Rows of the slots i0 .. i0 + 31 of a warp whose counters (the next row of each expert within the
// block's run) are `mine`.
__device__ __forceinline__ void place_slots(const OrderArgs &a, int i, int hi, int ex, const int32_t *start, int32_t *mine, int lane)
{
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, ex);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int at = -1;
    if (ex >= 0)
        at = start[ex] + mine[ex] + rank;
    __syncwarp();
    if (ex >= 0 && rank == 0)
        mine[ex] += __popc(same);
    __syncwarp();
    if (i < hi)
        a.rows[i] = at;
}

__global__ void __launch_bounds__(ORDER_THREADS) order_place_kernel(const OrderArgs a)
{
    extern __shared__ int32_t smem[];
    int32_t *cnt = smem;                        // [ORDER_WARPS][E]
    int32_t *start = smem + ORDER_WARPS * a.E;  // [E]: rows of the blocks before this one, then first rows
    int32_t *all = start + a.E;                 // [E]: rows of all blocks
    __shared__ int32_t wsum[ORDER_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < (ORDER_WARPS + 2) * a.E; i += ORDER_THREADS)
        smem[i] = 0;
    // this warp's run; a run of the usual length is held in registers
    const int lo = min(a.n, blockIdx.x * a.chunk), hi = min(a.n, lo + a.chunk);
    const int per = a.chunk / ORDER_WARPS;
    const int wlo = min(hi, lo + warp * per), whi = min(hi, wlo + per);
    const bool held = a.chunk == ORDER_CHUNK;
    int ex[ORDER_SLOTS];
    bool bad = false;
    if (held) {
#pragma unroll
        for (int s = 0; s < ORDER_SLOTS; ++s) {
            const int i = wlo + s * 32 + lane;
            ex[s] = i < whi ? slot_expert(a, i, bad) : -2;
        }
    }
    __syncthreads();
    int32_t *mine = cnt + warp * a.E;
    if (held) {
#pragma unroll
        for (int s = 0; s < ORDER_SLOTS; ++s)
            if (ex[s] >= 0)
                atomicAdd(&mine[ex[s]], 1);
    } else {
        for (int i = wlo + lane; i < whi; i += 32) {
            const int e = slot_expert(a, i, bad);
            if (e >= 0)
                atomicAdd(&mine[e], 1);
        }
    }
    if (gridDim.x > 1) {
        ptx::grid_dependency_wait();   // the counting kernel
        // counts of all blocks and of those before this one: groups of E (rounded up to a warp)
        // threads take every groups-th block
        const int wide = min(ORDER_THREADS, (a.E + 31) / 32 * 32), groups = ORDER_THREADS / wide;
        const int g = threadIdx.x / wide;
        for (int e = threadIdx.x % wide; e < a.E && g < groups; e += wide) {
            int total = 0, before = 0;
#pragma unroll 8
            for (int b = g; b < static_cast<int>(gridDim.x); b += groups) {
                const int c = a.hist[static_cast<size_t>(b) * a.E + e];
                total += c;
                before += b < static_cast<int>(blockIdx.x) ? c : 0;
            }
            atomicAdd(&all[e], total);      // sums of integers: any order gives the same
            atomicAdd(&start[e], before);
        }
    }
    __syncthreads();
    // per expert: the warps' starts, then an exclusive sum of the rows over the experts
    int carry = 0;
    for (int e0 = 0; e0 < a.E; e0 += ORDER_THREADS) {
        const int e = e0 + threadIdx.x;
        int total = 0;
        if (e < a.E) {
#pragma unroll
            for (int w = 0; w < ORDER_WARPS; ++w) {
                const int c = cnt[w * a.E + e];
                cnt[w * a.E + e] = total;
                total += c;
            }
            if (gridDim.x > 1)
                total = all[e];
        }
        int incl = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            incl += lane >= o ? v : 0;
        }
        __syncthreads();
        if (lane == 31)
            wsum[warp] = incl;
        __syncthreads();
        const int base = carry + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? wsum[lane] : 0);
        carry += __reduce_add_sync(0xFFFFFFFFu, lane < ORDER_WARPS ? wsum[lane] : 0);
        if (e < a.E) {
            start[e] += base + incl - total;
            if (blockIdx.x == 0) {
                a.offsets[e] = base + incl - total;
                if (e == a.E - 1)
                    a.offsets[a.E] = base + incl;
            }
        }
    }
    __syncthreads();
    if (held) {
#pragma unroll
        for (int s = 0; s < ORDER_SLOTS; ++s)
            place_slots(a, wlo + s * 32 + lane, whi, ex[s], start, mine, lane);
    } else {
        for (int i0 = wlo; i0 < whi; i0 += 32) {
            const int i = i0 + lane;
            place_slots(a, i, whi, i < whi ? slot_expert(a, i, bad) : -2, start, mine, lane);
        }
    }
    if (gridDim.x == 1) {
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0)
            *a.status = bad ? MOE_ERR_BAD_INDEX : MOE_OK;
    } else if (bad) {
        atomicExch(a.status, static_cast<int32_t>(MOE_ERR_BAD_INDEX));
    }
}

// Blocks and slots a block: a block for each run of ORDER_CHUNK slots (one block is one launch; 4096
// slots take 4.9 us in two blocks, 6.7 in one), and longer runs where the blocks' counts, which
// every block reads, would pass 32768 words.
void order_shape(long long n, int E, int &blocks, int &chunk)
{
    const long long most = 32768 / E < 32 ? 32 : 32768 / E > 256 ? 256 : 32768 / E;
    long long c = ORDER_CHUNK;
    if (n > c * most)
        c = (n + most - 1) / most;
    c = (c + ORDER_THREADS - 1) / ORDER_THREADS * ORDER_THREADS;
    chunk = static_cast<int>(c);
    blocks = static_cast<int>(n <= 0 ? 1 : (n + c - 1) / c);
}

template <typename T, int IPL>
struct RouteLaunch {
    static void go(const RouteArgs &a, cudaStream_t s)
    {
        route_kernel<T, IPL><<<(a.T + WARPS - 1) / WARPS, WARPS * 32, 0, s>>>(a);
    }
};
template <typename T, int IPL>
struct RouteBwdLaunch {
    static void go(const RouteBwdArgs &a, cudaStream_t s)
    {
        route_backward_kernel<T, IPL><<<(a.T + WARPS - 1) / WARPS, WARPS * 32, 0, s>>>(a);
    }
};

}  // namespace

extern "C" {

int moe_route_topk(int T, int E, int topk, const void *logits, int64_t ld, int dtype, const uint8_t *token_mask,
                   int renormalize, int64_t *topk_idx, float *topk_w, void *stream)
{
    if (!route_sizes_ok(T, E, topk, dtype) || ld < E || renormalize < 0 || renormalize > 1)
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    if (!logits || !topk_idx || !topk_w || !op_aligned(logits, dtype_bytes(dtype)) || !op_aligned(topk_idx, 8) ||
        !op_aligned(topk_w, 4))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    by_width<RouteLaunch>(dtype, E, RouteArgs{T, E, topk, logits, ld, token_mask, renormalize, topk_idx, topk_w},
                          static_cast<cudaStream_t>(stream));
    return launched();
}

int moe_route_topk_backward(int T, int E, int topk, const float *dw, const int64_t *topk_idx, const float *topk_w,
                            const void *logits, int64_t ld, int dtype, int renormalize, void *dlogits, void *stream)
{
    if (!route_sizes_ok(T, E, topk, dtype) || ld < E || renormalize < 0 || renormalize > 1)
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    if (!dw || !topk_idx || !topk_w || !dlogits || (!renormalize && !logits) || !op_aligned(dw, 4) ||
        !op_aligned(topk_idx, 8) || !op_aligned(topk_w, 4) || !op_aligned(logits, dtype_bytes(dtype)) ||
        !op_aligned(dlogits, dtype_bytes(dtype)))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    by_width<RouteBwdLaunch>(dtype, E, RouteBwdArgs{T, E, topk, dw, topk_idx, topk_w, logits, ld, renormalize, dlogits},
                             static_cast<cudaStream_t>(stream));
    return launched();
}

int moe_expert_order_workspace(int T, int topk, int E, uint64_t *bytes)
{
    const long long n = static_cast<long long>(T) * topk;
    if (T < 0 || topk < 1 || topk > 32 || E < 1 || E > 1024 || n > MAX_ROWS || !bytes)
        return MOE_ERR_INVALID_ARG;
    int blocks, chunk;
    order_shape(n, E, blocks, chunk);
    *bytes = blocks > 1 ? static_cast<uint64_t>(blocks) * E * sizeof(int32_t) : 0;
    return MOE_OK;
}

int moe_expert_order(int T, int topk, int E, const int64_t *topk_idx, int32_t *offsets, int32_t *rows,
                     int32_t *status, void *workspace, uint64_t workspace_bytes, void *stream)
{
    uint64_t need = 0;
    if (moe_expert_order_workspace(T, topk, E, &need) != MOE_OK)
        return MOE_ERR_INVALID_ARG;
    const long long n = static_cast<long long>(T) * topk;
    if (!offsets || !status || !op_aligned(offsets, 4) || !op_aligned(status, 4) ||
        (n > 0 && (!topk_idx || !rows || !op_aligned(topk_idx, 8) || !op_aligned(rows, 4))) ||
        (need > 0 && (!workspace || !op_aligned(workspace, 4) || workspace_bytes < need)))
        return MOE_ERR_INVALID_ARG;
    OP_DEVICE(sms);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int blocks, chunk;
    order_shape(n, E, blocks, chunk);
    const OrderArgs a{static_cast<int>(n), E, chunk, topk_idx, offsets, rows, status, static_cast<int32_t *>(workspace)};
    if (blocks > 1) {
        order_count_kernel<<<blocks, ORDER_THREADS, E * sizeof(int32_t), s>>>(a);
        if (launched() != MOE_OK)
            return MOE_ERR_CUDA;
    }
    const int smem = (ORDER_WARPS + 2) * E * static_cast<int>(sizeof(int32_t));
    if (smem > 40 * 1024 &&   // (static shared memory counts towards the 48 KB that need no attribute)
        ensure_max_dynamic_smem(reinterpret_cast<const void *>(&order_place_kernel), smem) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (blocks > 1)
        return launch_programmatic(order_place_kernel, blocks, ORDER_THREADS, smem, s, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    order_place_kernel<<<blocks, ORDER_THREADS, smem, s>>>(a);
    return launched();
}

}  // extern "C"
