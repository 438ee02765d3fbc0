// Device helpers shared by the 8-bit cache's kernels: rows of heads, the
// position rotation, code conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "kv8.h"

namespace tq {
namespace kv8 {

// Let `kernel` (this one instance of it) have `smem` bytes of dynamic shared
// memory, once on each device.
template <typename K>
cudaError_t allow_smem(K kernel, int smem, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// ------------------------------------------------------------------ inputs

// 8 consecutive elements (16-byte aligned) as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <typename T>
__device__ __forceinline__ uint32_t pack_out(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack_out<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack_out<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------------------ rotation

// f / (2 pi) modulo 1 in units of 2^-64: the 53-bit significand of f times
// 2^66 / (2 pi) (rounded to an integer), shifted to f's exponent. For
// |f| < 1024 the error is below 2^-52 of the value and 2^-64 of a turn, so p
// times the result, modulo 2^64, is the fraction of a turn at position p to
// within p (2^-64 + |f| 2^-54). Integer arithmetic: the fp64 pipe is slow here.
__device__ __forceinline__ uint64_t turns_of(double f) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(f));
    const int ex = static_cast<int>((u >> 52) & 0x7FF);
    if (ex == 0) return 0;   // zero, and subnormals
    const uint64_t m = (u & 0xFFFFFFFFFFFFFull) | (1ull << 52);
    const uint64_t kC = 0xA2F9836E4E44152Aull;   // 2^66 / (2 pi)
    const uint64_t hi = __umul64hi(m, kC), lo = m * kC;
    const int sh = 54 - (ex - 1023);   // value = (hi:lo) >> sh
    uint64_t t;
    if (sh >= 128) t = 0;
    else if (sh >= 64) t = hi >> (sh - 64);
    else if (sh > 0) t = (lo >> sh) | (hi << (64 - sh));
    else t = 0;   // |f| >= 2^54: no angle
    return (u >> 63) ? 0 - t : t;
}

// cos and sin of the angle `t` / 2^64 of a turn: to the nearest quarter turn
// (exact), then the Taylor series in the remainder y, |y| <= pi/4 (the first
// terms left out are y^11/11! and y^12/12!, below 2e-9 and 2e-10), with what
// fp32 leaves out of y added to first order: within about 2^-24.
__device__ __forceinline__ void turn_cos_sin(uint64_t t, float& co, float& si) {
    constexpr float kHi = 1.462918120e-09f, kLo = -4.070940433e-17f;   // 2 pi / 2^32
    const uint32_t h = static_cast<uint32_t>(t >> 32);
    const uint32_t quad = (h + 0x20000000u) >> 30;
    const int32_t r = static_cast<int32_t>(h - (quad << 30));   // [-2^29, 2^29] / 2^32 of a turn
    const float rf = static_cast<float>(r), rl = static_cast<float>(r - static_cast<int32_t>(rf));
    const float y = rf * kHi;
    const float dy = fmaf(rl, kHi, fmaf(rf, kLo, fmaf(rf, kHi, -y)));
    const float z = y * y;
    float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    s = fmaf(z, s, 8.3333333e-3f);
    s = fmaf(z, s, -1.6666667e-1f);
    float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    c = fmaf(z, c, -1.3888889e-3f);
    c = fmaf(z, c, 4.1666667e-2f);
    c = fmaf(z, c, -0.5f);
    const float c1 = fmaf(z, c, 1.0f);
    s = fmaf(y * z, s, dy * c1);
    c = fmaf(z, c, -dy * y);
    s += y;
    c += 1.0f;
    const float a = (quad & 1) ? s : c, b = (quad & 1) ? c : s;
    co = ((quad + 1) & 2) ? -a : a;
    si = (quad & 2) ? -b : b;
}

// A head's coordinates in two chunks of 8 that hold whole rotation pairs:
// chunk pair j < D / 16 is coordinates a..a+7 and b..b+7.
__device__ __forceinline__ void chunk_pair(int j, int rot, int inter, int& a, int& b) {
    if (!inter && 16 * j < rot) {
        a = 8 * j;
        b = rot / 2 + 8 * j;
    } else {
        a = 16 * j;
        b = 16 * j + 8;
    }
}

// Rotate chunk pair j by `angle(i)`, cos and sin of its pair i < 8.
template <typename F>
__device__ __forceinline__ void rotate_by(float (&xa)[8], float (&xb)[8], int inter, F&& angle) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 cs = angle(i);
        float* u;
        float* w;
        if (inter) {
            u = i < 4 ? &xa[(2 * i) & 7] : &xb[(2 * i) & 7];
            w = i < 4 ? &xa[(2 * i + 1) & 7] : &xb[(2 * i + 1) & 7];
        } else {
            u = &xa[i];
            w = &xb[i];
        }
        const float x = *u, y = *w;
        *u = fmaf(x, cs.x, -(y * cs.y));
        *w = fmaf(y, cs.x, x * cs.y);
    }
}

// cos and sin (times the rotation's scale) of frequency `turns` at position p.
__device__ __forceinline__ float2 angle_at(const Rope& r, uint64_t turns, int p) {
    float co, si;
    turn_cos_sin(static_cast<uint64_t>(static_cast<int64_t>(p)) * turns, co, si);
    return make_float2(co * r.scale, si * r.scale);
}

// Rotate chunk pair j of a vector at position p; `turns`: the frequencies (shared memory).
__device__ __forceinline__ void rotate_pair(float (&xa)[8], float (&xb)[8], int j, const Rope& r, const uint64_t* turns,
                                            int p) {
    if (16 * j >= r.rot) return;
    rotate_by(xa, xb, r.inter, [&](int i) { return angle_at(r, turns[8 * j + i], p); });
}

// ------------------------------------------------------------------ codes

// Two e4m3 codes (low 16 bits) as fp16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16_hi(uint32_t w) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(r) : "r"(w));
    return r;
}

// Four codes of a word as two fp16 pairs (bytes 0, 1 and 2, 3), exactly. An
// integer code c is the byte u = c + 128 (its top bit flipped) in the low byte
// of 1024 + u, less 1152.
template <bool I8>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (I8) {
        const uint32_t x = w ^ 0x80808080u;
        const __half2 off = __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
        const __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), off), hb = __hsub2(*reinterpret_cast<__half2*>(&b), off);
        lo = *reinterpret_cast<const uint32_t*>(&ha);
        hi = *reinterpret_cast<const uint32_t*>(&hb);
    } else {
        lo = e4m3x2_f16(w);
        hi = e4m3x2_f16_hi(w);
    }
}

// Codes of four values (scale divided out), rounded to nearest even. kAny: they may
// be out of range (kept in range) or NaN (0); else they are in range.
template <bool I8, bool kAny = true>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (kAny) a = a == a ? a : 0.0f, b = b == b ? b : 0.0f, c = c == c ? c : 0.0f, d = d == d ? d : 0.0f;
    if constexpr (I8) {
        auto one = [](float x) {
            if constexpr (kAny) x = fminf(fmaxf(x, -127.0f), 127.0f);
            int r;
            asm("cvt.rni.s32.f32 %0, %1;\n" : "=r"(r) : "f"(x));
            return static_cast<uint32_t>(r);
        };
        return __byte_perm(__byte_perm(one(a), one(b), 0x0040), __byte_perm(one(c), one(d), 0x0040), 0x5410);
    } else {
        uint32_t r;
        asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
            " mov.b32 %0, {lo, hi};\n}\n"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
        return r;
    }
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

// ------------------------------------------------------------------ scores

// cap2 tanh(x), cap2 = log2(e) cap, x = score / cap, as 1 - 2 / (1 + e^2x): within 2^-22 of the cap, so within 2^-16 for
// the caps that models use.
constexpr float kUsualCap = 64.0f;
__device__ __forceinline__ float capped(float x, float cap2) { return fmaf(-2.0f * cap2, rcp(1.0f + ex2(x * 2.8853900818f)), cap2); }

// The same for larger caps, to 2^-19 of itself: for small x, where the form above cancels, the odd series
// x - x^3/3 + 2 x^5/15 - 17 x^7/315, whose next term is below 2^-21 of x. (For every cap it would cost a short
// prompt at head_dim 256 33.8 us for 30.4.)
__device__ __forceinline__ float capped_wide(float x, float cap2) {
    const float z = x * x;
    const float near = cap2 * fmaf(x * z, fmaf(z, fmaf(z, -5.3968254e-2f, 1.3333333e-1f), -3.3333333e-1f), x);
    return fabsf(x) < 0.25f ? near : capped(x, cap2);
}

// ------------------------------------------------------------------ what a query sees

// The visible keys of one query: [lo, p] and [0, prefix), below the sequence's end.
struct Sight {
    int p, lo, prefix;
    __device__ __forceinline__ bool sees(int t) const { return (t <= p && t >= lo) || t < prefix; }
};

}  // namespace kv8
}  // namespace tq
