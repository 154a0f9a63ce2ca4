// op_common.cuh -- what the translation units of the operators around the expert layer
// (norm.cu, router.cu, rows.cu, grouped_mm.cu) share: element types, vector loads and stores,
// block sums, argument checks.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/cpw_moe.h"

namespace cpw {

// ------------------------------------------------------------------ element types ------
template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// N consecutive elements moved by as few accesses of at most 16 bytes as they fill; the address
// is aligned to the access.
template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack {
    T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T *p)
{
    if constexpr (N == 1) {
        Pack<T, 1> r;
        r.v[0] = __ldg(p);
        return r;
    } else {
        static_assert(sizeof(T) * N % 16 == 0, "whole accesses");
        union {
            Pack<T, N> pack;
            uint4 q[sizeof(T) * N / 16];
        } u;
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) * N / 16); ++i)
            u.q[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        return u.pack;
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, N> &v)
{
    if constexpr (N == 1) {
        *p = v.v[0];
    } else {
        static_assert(sizeof(T) * N % 16 == 0, "whole accesses");
        union {
            Pack<T, N> pack;
            uint4 q[sizeof(T) * N / 16];
        } u;
        u.pack = v;
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) * N / 16); ++i)
            reinterpret_cast<uint4 *>(p)[i] = u.q[i];
    }
}

// ------------------------------------------------------------------ rows of any alignment ----
template <typename T>
constexpr int VEC = 16 / static_cast<int>(sizeof(T));

// Elements that a row starts past a 16-byte boundary.
template <typename T>
__device__ __forceinline__ int lead_of(const T *row)
{
    return static_cast<int>(reinterpret_cast<uint64_t>(row) & 15) / static_cast<int>(sizeof(T));
}
// The aligned vector that holds p (zeros where `is` is false).  Written out, so that the loads of
// all slots are issued without a branch between them.
template <typename T>
__device__ __forceinline__ uint4 load_aligned(const T *p, bool is, int ahead = 0)
{
    uint4 q;
    asm volatile("{\n\t"
                 ".reg .pred p;\n\t"
                 "setp.ne.s32 p, %5, 0;\n\t"
                 "mov.b32 %0, 0;\n\t"
                 "mov.b32 %1, 0;\n\t"
                 "mov.b32 %2, 0;\n\t"
                 "mov.b32 %3, 0;\n\t"
                 "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t"
                 "}"
                 : "=&r"(q.x), "=&r"(q.y), "=&r"(q.z), "=&r"(q.w)
                 : "l"((reinterpret_cast<uint64_t>(p) & ~15ull) + 16 * ahead), "r"(static_cast<int>(is)));
    return q;
}
// 16 bytes at any element: the two aligned vectors that cover them, shifted.
struct Halves {
    uint4 lo, hi;
};
template <typename T>
__device__ __forceinline__ Halves load_halves(const T *p, bool is = true)
{
    return {load_aligned(p, is), load_aligned(p, is, 1)};
}
// The 16 bytes from p on.
template <typename T>
__device__ __forceinline__ Pack<T, VEC<T>> shifted(const Halves &h, const T *p)
{
    const uint32_t s = static_cast<uint32_t>(reinterpret_cast<uint64_t>(p));
    const uint32_t u[8] = {h.lo.x, h.lo.y, h.lo.z, h.lo.w, h.hi.x, h.hi.y, h.hi.z, h.hi.w};
    uint32_t v[6], x[5];
#pragma unroll
    for (int i = 0; i < 6; ++i)
        v[i] = s & 8 ? u[i + 2] : u[i];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        x[i] = s & 4 ? v[i + 1] : v[i];
    union {
        Pack<T, VEC<T>> pack;
        uint32_t word[4];
    } o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o.word[i] = sizeof(T) == 4 ? x[i] : __funnelshift_r(x[i], x[i + 1], 8 * (s & 2));
    return o.pack;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// ------------------------------------------------------------------ host side ----------
inline bool op_aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline size_t dtype_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
// Most tokens, slots or rows of a call: row indices plus a grid's strides stay in 31 bits.
constexpr long long MAX_ROWS = 1ll << 30;
inline bool dtype_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }

// Number of SMs of the current device; 0 if a CUDA call failed, -1 if it is not an sm_103 GPU.
// The answer of a device is looked up once.
inline int op_num_sms()
{
    constexpr int MAX_DEV = 64;
    static int cache[MAX_DEV];   // written with the one value that every thread would write
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEV)
        return 0;
    const int c = __atomic_load_n(&cache[dev], __ATOMIC_RELAXED);
    if (c)
        return c;
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    const int got = major == 10 && minor == 3 ? sms : -1;
    __atomic_store_n(&cache[dev], got, __ATOMIC_RELAXED);
    return got;
}

#define OP_DEVICE(sms)                                                       \
    const int sms = cpw::op_num_sms();                                       \
    do {                                                                     \
        if (sms <= 0)                                                        \
            return sms == 0 ? MOE_ERR_CUDA : MOE_ERR_UNSUPPORTED_DEVICE;     \
    } while (0)

// Calls f with a null pointer of the element type that `dtype` names.
template <typename F>
inline auto with_dtype(int dtype, F f)
{
    if (dtype == MOE_F32)
        return f(static_cast<float *>(nullptr));
    if (dtype == MOE_BF16)
        return f(static_cast<__nv_bfloat16 *>(nullptr));
    return f(static_cast<__half *>(nullptr));
}

inline int launched() { return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace cpw
