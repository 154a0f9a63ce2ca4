// router_common.cuh -- what the routers (router.cu, scores.cu) share: the order of values as keys, and kernels by
// how many experts a lane of the warp that takes a token holds.  Which they are is each file's: l, l + 32, ... in lane l in
// router.cu and in the gradient of softmax scores as they are, neighbours in the choice by scores.
#pragma once

#include <type_traits>

#include "op_common.cuh"

namespace cpw {

constexpr int WARPS = 4;   // of a block (a token each, or in scores.cu up to four)

// Order-preserving 32-bit key of a logit: 0 for -inf (never chosen), the largest for NaN, the
// same for both zeros.
__device__ __forceinline__ uint32_t order_key(float f)
{
    if (f != f)
        return 0xFFFFFFFFu;
    if (f == -INFINITY)
        return 0u;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return k == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// 64-bit twins of order_key and key_value.
__device__ __forceinline__ uint64_t order_key(double f)
{
    if (f != f)
        return ~0ull;
    if (f == -INFINITY)
        return 0ull;
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(f + 0.0));
    return (u >> 63) ? ~u : (u | 1ull << 63);
}
__device__ __forceinline__ double key_value(uint64_t k)
{
    if (k == ~0ull)
        return __longlong_as_double(0x7FF8000000000000ll);
    return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xFFFFFFFFu, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Experts of a lane.
inline int lane_experts(int E)
{
    const int n = (E + 31) / 32;
    return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : n <= 8 ? 8 : 32;
}
template <template <typename, int> class Launch, typename A>
void by_width(int dtype, int E, const A &a, cudaStream_t s)
{
    with_dtype(dtype, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const int ipl = lane_experts(E);
        if (ipl == 1)
            Launch<T, 1>::go(a, s);
        else if (ipl == 2)
            Launch<T, 2>::go(a, s);
        else if (ipl == 4)
            Launch<T, 4>::go(a, s);
        else if (ipl == 8)
            Launch<T, 8>::go(a, s);
        else
            Launch<T, 32>::go(a, s);
    });
}

inline bool route_sizes_ok(int T, int E, int topk, int dtype)
{
    return T >= 0 && T <= MAX_ROWS && E >= 1 && E <= 1024 && topk >= 1 && topk <= 32 && topk <= E && dtype_ok(dtype);
}

}  // namespace cpw
