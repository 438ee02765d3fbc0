// Position rotation of queries and keys.
//
// A pair (x1, x2) of a row at position p becomes scale (x1 cos a - x2 sin a, x2 cos a +
// x1 sin a), a = p inv_freq: three operations a value against one read and one write of it, so
// memory bounds it, but for the angles, which cost some 60 instructions a pair. All heads of a token
// turn by the same ones: a CTA takes a few tokens, computes cos and sin of each (token, pair) once, in
// shared memory, and a thread then keeps the eight of its place in a head in registers over all the heads it takes.
//
// A thread has two chunks of 8 coordinates that hold whole pairs; the lanes of a warp lie beside each other
// in a row, then in neighbouring tokens, so that a warp reads and writes runs of 64 bytes at least whatever the order of the axes.
// The first heads' chunks are on their way while the angles are computed.
//
// Measured: 8192 tokens, 64 + 8 heads of 128, bf16, out of a fused projection into contiguous heads: 51 us (5.9 TB/s); 6 x 1999 tokens, 12
// heads of 256, f32: 47 us (6.2). Two heads ahead (one in fp32) at five CTAs an SM: with four and three CTAs 57 and 51, with one
// and six 54 and 55.
#include <algorithm>
#include <type_traits>

#include "kv8_device.cuh"
#include "serve.h"

namespace tq {
namespace serve {
namespace {

constexpr int kThreads = 256;
constexpr int kPlaces = 64;   // tokens of a CTA x chunk pairs of a head: head_dim / 16 at most, or about a warp

// 8 coordinates as they lie. (Loads that other writes of the kernel may not pass: an output may be its input.)
template <typename T>
struct Chunk {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                         : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                         : "l"(reinterpret_cast<const uint4*>(p) + i)
                         : "memory");
    }
    __device__ __forceinline__ void store(T* p, bool stream) const {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
            if (stream) __stcs(reinterpret_cast<uint4*>(p) + i, v[i]);
            else reinterpret_cast<uint4*>(p)[i] = v[i];
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(w[i]);
            } else if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i / 2]));
                x[i] = i % 2 ? f.y : f.x;
            } else {
                x[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
            }
        }
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll
        for (int i = 0; i < static_cast<int>(2 * sizeof(T)); ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
            else w[i] = kv8::pack_out<T>(x[2 * i], x[2 * i + 1]);
        }
    }
};

// `tokens` of a CTA, `slots` of heads side by side: threads (slot, token, chunk pair). Grid: tokens, then parts of the heads.
template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads, 5) rope_kernel(const __grid_constant__ RopeArgs A, int tokens, int slots) {
    __shared__ float2 s_angles[8 * kPlaces];   // [pair of the chunk pair][token][chunk pair]
    constexpr int kAhead = sizeof(T) == 4 ? 1 : 2;
    const int J = A.D / 16, j = threadIdx.x % J, tok = threadIdx.x / J % tokens, slot = threadIdx.x / (J * tokens);
    const int rot = A.rope.rot;
    const unsigned all = A.batch * A.n, g = blockIdx.x * tokens + tok;
    bool here = g < all;
    const int b = here ? g / A.n : 0, i = here ? g % A.n : 0;
    if (here && A.news) {
        const int n = A.news[b];
        if ((n < 0 || n > A.n) && i == 0 && j == 0 && slot == 0 && blockIdx.y == 0) atomicOr(A.err, TQ_DEVERR_SEQLEN);
        here = i < n;
    }
    int ca, cb;
    kv8::chunk_pair(j, rot, kInter, ca, cb);
    const int heads = A.heads[0] + A.heads[1], part = (heads + gridDim.y - 1) / gridDim.y;
    const int h_end = here ? min(heads, static_cast<int>(blockIdx.y + 1) * part) : 0;
    const bool turns = 16 * j < rot;
    auto at = [&](const kv8::Rows (&rows)[2], int h) {
        const bool k = h >= A.heads[0];
        const kv8::Rows& r = k ? rows[1] : rows[0];
        return static_cast<T*>(r.data) + b * r.sb + (k ? h - A.heads[0] : h) * r.sh + i * r.st;
    };
    // chunks that pass in place are left alone
    auto takes = [&](int h) { return h < h_end && (turns || A.in[h >= A.heads[0]].data != A.out[h >= A.heads[0]].data); };
    Chunk<T> xa[kAhead], xb[kAhead];
    auto fetch = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = h0 + u * slots;
            if (takes(h)) {
                const T* p = at(A.in, h);
                xa[u].load(p + ca);
                xb[u].load(p + cb);
            }
        }
    };
    int h0 = blockIdx.y * part + slot;
    fetch(h0);
    const int pairs = rot / 2;
    for (int x = threadIdx.x; x < tokens * pairs; x += blockDim.x) {
        const int q = x % pairs, t = x / pairs;
        const unsigned gg = min(blockIdx.x * tokens + t, all - 1);
        const int64_t p = A.rope.positions ? A.rope.positions[gg] : (A.starts ? A.starts[gg / A.n] : 0) + static_cast<int64_t>(gg % A.n);
        float co, si;
        kv8::turn_cos_sin(static_cast<uint64_t>(p) * kv8::turns_of(A.rope.inv_freq[q]), co, si);
        s_angles[(q % 8 * tokens + t) * J + q / 8] = make_float2(co * A.rope.scale, (A.back ? -si : si) * A.rope.scale);
    }
    __syncthreads();
    float2 cs[8];
    if (turns) {
#pragma unroll
        for (int u = 0; u < 8; ++u) cs[u] = s_angles[(u * tokens + tok) * J + j];
    }
    while (h0 < h_end) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = h0 + u * slots;
            if (takes(h)) {
                T* p = at(A.out, h);
                if (turns) {
                    float ya[8], yb[8];
                    xa[u].get(ya);
                    xb[u].get(yb);
                    kv8::rotate_by(ya, yb, kInter, [&](int v) { return cs[v]; });
                    xa[u].put(ya);
                    xb[u].put(yb);
                }
                xa[u].store(p + ca, A.stream);
                xb[u].store(p + cb, A.stream);
            }
        }
        h0 += kAhead * slots;
        fetch(h0);
    }
}

template <typename T>
cudaError_t launch(RopeArgs a, int sms, cudaStream_t s) {
    // outputs that the L2 cache (129 MB, inputs in it too) will not hold go past it: 6 x 1999 tokens of 12 heads of 256 in fp32 47 us, 50 without (the call alone)
    a.stream = static_cast<int64_t>(a.batch) * a.n * (a.heads[0] + a.heads[1]) * a.D * static_cast<int64_t>(sizeof(T)) > (64 << 20);
    const int J = a.D / 16, all = a.batch * a.n, heads = a.heads[0] + a.heads[1];
    const int tokens = std::min(all, std::max(1, 32 / J)), slots = std::max(1, std::min(heads, kThreads / (J * tokens)));
    const int tiles = (all - 1) / tokens + 1;   // (all up to 2^31 - 1)
    // the heads in parts, as long as there are fewer CTAs than SMs
    const int parts = std::max(1, std::min((heads + slots - 1) / slots, sms / tiles));
    auto kernel = a.rope.inter ? rope_kernel<T, true> : rope_kernel<T, false>;
    kernel<<<dim3(tiles, parts), J * tokens * slots, 0, s>>>(a, tokens, slots);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, int sms, cudaStream_t s) {
    if (dtype == TQ_F32) return launch<float>(a, sms, s);
    if (dtype == TQ_F16) return launch<__half>(a, sms, s);
    return launch<__nv_bfloat16>(a, sms, s);
}

}  // namespace serve
}  // namespace tq
