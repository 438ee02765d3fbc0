// What the kernels that verify and draw tokens share: values as they lie, weights of logits, and what CTAs of a cluster tell each other.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <climits>
#include <type_traits>

#include "cluster.cuh"
#include "kv8_device.cuh"
#include "serve.h"
#include "tc_ptx.cuh"

namespace tq {
namespace serve {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMostCtas = 8, kParts = kWarps * kMostCtas;   // CTAs of a cluster at most, and their warps
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLn2 = 0.69314718f;
constexpr float kUsual = 8192.0f;   // exponents below which one product makes a weight (see Seen::take)

__device__ __forceinline__ float number(float x) { return x; }
__device__ __forceinline__ float number(__half x) { return __half2float(x); }
__device__ __forceinline__ float number(__nv_bfloat16 x) { return __bfloat162float(x); }

// The values of 16 bytes, in pairs.
__device__ __forceinline__ void numbers(const uint4& u, float2* x, float) {
    x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y)), x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ void numbers(const uint4& u, float2* x, __nv_bfloat16) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void numbers(const uint4& u, float2* x, __half) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
}
// 8 values at a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) numbers(__ldg(reinterpret_cast<const uint4*>(p) + i), x + i * 8 / sizeof(T), T());
}

using kv8::ex2;
using kv8::rcp;

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The largest of three numbers, NaN if one of them is.
__device__ __forceinline__ float largest(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A logit as it counts: +inf the largest number, NaN -inf.
__device__ __forceinline__ float logit(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }

// log2(e) / T as c + lo, both positive, so that what is masked (-inf) stays -inf in either product: log2(e) = 1.442695 (rounded down)
// + 1.9259630e-8; c is below the quotient, lo what it leaves. To 2^-40.
struct Scale {
    float c, lo, near;   // near: c + lo in one number, off by 2^-24 of itself at most
    __device__ __forceinline__ explicit Scale(float T) {
        constexpr float hi = 0x1.715476p+0f, rest = 1.9259630e-8f;
        const float r = rcp(T);
        c = hi * r * (1.0f - 0x1p-21f);   // (the reciprocal is off by 2^-23, the products by 2^-24)
        lo = (fmaf(-c, T, hi) + rest) * r;
        near = c + lo;
    }
    __device__ __forceinline__ float weight(float d) const { return ex2(fmaf(d, c, d * lo)); }   // d <= 0
    // The same with the exponent's rounding put back: to 2^-21, and d's own. NaN of a masked value.
    __device__ __forceinline__ float weight_near(float d) const {
        const float t = d * c, w = ex2(t);
        return fmaf(w, fmaf(d, lo, fmaf(d, c, -t)) * kLn2, w);
    }
    __device__ __forceinline__ float log(float d) const {   // d / T
        const float t = d * c;
        return fmaf(t, kLn2, fmaf(d, lo, fmaf(d, c, -t)) * kLn2 + t * -1.9046543e-9f);   // (ln 2 less kLn2)
    }
};

// Values [i0, i1) of a row on their way into the L2 cache (one thread; whole units).
template <typename T>
__device__ __forceinline__ void ahead(const T* row, int i0, int i1) {
    const uintptr_t a = (reinterpret_cast<uintptr_t>(row + i0) + 15) & ~static_cast<uintptr_t>(15), e = reinterpret_cast<uintptr_t>(row + i1) & ~static_cast<uintptr_t>(15);
    if (i0 < i1 && a < e) tc::bulk_prefetch_l2(reinterpret_cast<const void*>(a), static_cast<unsigned>(e - a));
}

// The largest of the warp's numbers (no NaN), as integers that are ordered as they are.
__device__ __forceinline__ float warp_max(float x) {
    const int i = __float_as_int(x), k = __reduce_max_sync(kAll, i ^ (i >> 31 & 0x7FFFFFFF));
    return __int_as_float(k ^ (k >> 31 & 0x7FFFFFFF));
}

// A token and its score, a positive number (0: none).
struct __align__(8) Best {
    float v;
    int i;
    __device__ __forceinline__ void meet(float w, int j) {   // the larger, the lower index of equals
        if (w > v || (w == v && j < i)) v = w, i = j;
    }
    __device__ __forceinline__ void join() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) meet(__shfl_xor_sync(kAll, v, o), __shfl_xor_sync(kAll, i, o));
    }
};

// 2^log_ctas CTAs of a cluster for each sequence.
inline cudaError_t launch_cluster(void (*kernel)(VerifyArgs, int), const VerifyArgs& a, int log_ctas, int smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.batch) << log_ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << log_ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, log_ctas);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return e;
}

}  // namespace serve
}  // namespace tq
