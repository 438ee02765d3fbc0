// Appending keys and values to the 8-bit cache, the keys rotated on the way.
//
// The unit is one block's new tokens of one KV head, keys or values, because that
// is what has a scale: a CTA reads them once, rotates them (fp32), reduces the
// largest magnitude to the block's power-of-two scale, and writes the codes at
// that scale. Nothing is shared between CTAs, no atomics, one launch. A block that
// already held tokens keeps its scale unless the new tokens need a larger one;
// then its earlier codes are rounded to the new one by the same CTA.
//
// A CTA takes several heads of its block, as long as there are two CTAs for every
// SM. The heads turn by the same angles, so cos and sin of each (token, pair) are
// computed once, in shared memory: they are what a rotation costs. Nothing else is
// held: the codes come from a second look at the input, which is still in the L1
// cache, or at worst in the L2. (With the block in registers instead, the few CTAs
// that fit an SM left it waiting: 28 us for the first case below, 49 with more heads.)
//
// Bound: memory (2 or 4 bytes read and 1 written a value), but for rotated keys
// instructions. Measured: 8192 tokens of 8 heads of 128, bf16, blocks of 64: 25 us (2.0
// TB/s; 15 unrotated); 6 x 4096 tokens of 4 heads of 256, f32, blocks of 128: 80 us (3.1).
#include "kv8_device.cuh"

namespace tq {
namespace kv8 {
namespace {

// max(m, |a|, |b|); NaN if one of them is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

// The smallest e in [-63, 63] with top / 2^e <= the largest code (448 = 1.75 x
// 2^8, 127 = 1.984375 x 2^6), from top's exponent and significand.
template <bool I8>
__device__ __forceinline__ int scale_exponent(float top) {
    const uint32_t u = __float_as_uint(top);
    const int e = static_cast<int>(u >> 23) - 127 - (I8 ? 6 : 8) + ((u & 0x7FFFFFu) > (I8 ? 0x7E0000u : 0x600000u) ? 1 : 0);
    return min(max(e, -63), 63);
}

// Four codes times 2^-down (down > 0), rounded to the format again.
template <bool I8>
__device__ __forceinline__ uint32_t recode(uint32_t w, float down) {
    uint32_t lo, hi;
    codes_f16<I8>(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo)), b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return encode4<I8>(a.x * down, a.y * down, b.x * down, b.y * down);
}

// kMost threads at most.
template <typename T, int D, bool I8, int kMost>
__global__ void __launch_bounds__(kMost, 1024 / kMost) append_kernel(const __grid_constant__ AppendArgs A, int heads) {
    extern __shared__ float2 s_angles[];   // [token of the block][pair], if the launch gave it room
    __shared__ uint64_t s_turns[D / 2];
    __shared__ uint32_t s_top[2][kMost / 32];
    const bool is_v = blockIdx.x & 1;
    const int j = blockIdx.x >> 1, b = blockIdx.z, tid = threadIdx.x, threads = blockDim.x;
    const Pool& P = A.pool;
    const int64_t start = A.seq[b];
    int n = A.news ? A.news[b] : A.n_new;
    const bool first_cta = tid == 0 && j == 0 && blockIdx.y == 0;
    if (start < 0 || n < 0 || n > A.n_new) {
        if (first_cta) atomicOr(A.err, TQ_DEVERR_SEQLEN);
        return;
    }
    const int64_t cap = static_cast<int64_t>(P.max_blocks) << P.bt_shift;
    if (start + n > cap) {
        if (first_cta) atomicOr(A.err, TQ_DEVERR_CAPACITY);
        n = static_cast<int>(start < cap ? cap - start : 0);
    }
    const int64_t lb = (start >> P.bt_shift) + j;          // logical block
    const int64_t t0 = lb << P.bt_shift;                   // its first position
    if (n == 0 || t0 >= start + n) return;
    const int64_t id = P.table ? P.table[b * static_cast<int64_t>(P.max_blocks) + lb] : b * static_cast<int64_t>(P.max_blocks) + lb;
    if (id < 0 || id >= P.num_blocks) {
        if (tid == 0) atomicOr(A.err, TQ_DEVERR_BLOCK);
        return;
    }
    const int first = static_cast<int>(start > t0 ? start - t0 : 0);                 // first new slot of the block
    const int count = static_cast<int>((start + n < t0 + P.BT ? start + n - t0 : P.BT)) - first;
    const int i0 = static_cast<int>(t0 + first - start);   // its index among the new tokens
    const Rows& R = is_v ? A.v : A.k;
    const bool turn = !is_v && A.rope.rot > 0;
    const int rot = turn ? A.rope.rot : 0, inter = A.rope.inter, pairs = rot / 2;
    const int32_t* pos = A.rope.positions ? A.rope.positions + b * static_cast<int64_t>(A.n_new) + i0 : nullptr;
    auto position = [&](int tok) { return pos ? pos[tok] : static_cast<int>(t0) + first + tok; };
    const bool shared = turn && A.angle_smem > 0;
    if (turn) {
        for (int i = tid; i < pairs; i += threads) s_turns[i] = turns_of(A.rope.inv_freq[i]);
        __syncthreads();
    }
    // angle of token tok and pair 8 jj + i: neighbouring lanes (jj, then tok) on neighbouring banks
    constexpr int J = D / 16, kPerToken = D / 2 + 8;
    // a thread has chunk pair jj of tokens tok0, tok0 + step, ..
    const int jj = tid % J, tok0 = tid / J, step = threads / J;
    int ca, cc;
    chunk_pair(jj, rot, inter, ca, cc);
    const bool turns_here = 16 * jj < rot;
    const int h_begin = blockIdx.y * heads, h_end = min(P.H, h_begin + heads);
    if (shared) {
        // the inputs on their way to the L2 cache meanwhile
        for (int h = h_begin; h < h_end; ++h)
            for (int tok = tok0; tok < count; tok += step)
                asm volatile("prefetch.global.L2 [%0];\n" ::"l"(static_cast<const T*>(R.data) + b * R.sb + h * R.sh + (i0 + tok) * R.st + ca));
        // a thread has one pair, of every few tokens
        const int q = tid % pairs, rows = threads / pairs;
        if (rows == 0) {   // more pairs than threads
            for (int e = tid; e < count * pairs; e += threads)
                s_angles[e / pairs * kPerToken + e % pairs % 8 * J + e % pairs / 8] = angle_at(A.rope, s_turns[e % pairs], position(e / pairs));
        } else if (tid < rows * pairs) {
            const uint64_t turns = s_turns[q];
            for (int tok = tid / pairs; tok < count; tok += rows)
                s_angles[tok * kPerToken + q % 8 * J + q / 8] = angle_at(A.rope, turns, position(tok));
        }
        __syncthreads();
    }
    for (int h = h_begin; h < h_end; ++h) {
        const T* src = static_cast<const T*>(R.data) + b * R.sb + h * R.sh + i0 * R.st;
        const int64_t unit = id * P.H + h;
        uint8_t* sx = (is_v ? P.vx : P.kx) + unit;
        const int e_old = first > 0 ? min(max(static_cast<int>(*sx) - 127, -126), 126) : -63;
        // f(token, its two chunks) for each of the thread's tokens
        auto each = [&](auto&& f) {
            const T* pa = src + tok0 * R.st + ca;
            const int to_c = cc - ca;
            const int64_t stride = step * R.st;
            const float2* cs = s_angles + tok0 * kPerToken + jj;
#pragma unroll 2
            for (int tok = tok0; tok < count; tok += step) {
                float xa[8], xb[8];
                load8(pa, xa);
                load8(pa + to_c, xb);
                pa += stride;
                if (turns_here) {
                    if (shared) rotate_by(xa, xb, inter, [&](int i) { return cs[i * J]; });
                    else rotate_pair(xa, xb, jj, A.rope, s_turns, position(tok));
                }
                cs += step * kPerToken;
                f(tok, xa, xb);
            }
        };
        float peak = 0.0f;   // a NaN stays one
        each([&](int, const float (&xa)[8], const float (&xb)[8]) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                peak = max_abs(peak, xa[i], xa[i + 1]);
                peak = max_abs(peak, xb[i], xb[i + 1]);
            }
        });
        // (two sets, in turn: one barrier a head; as bits, infinities and NaNs come out on top)
        auto over_block = [&](uint32_t x) {
            x = __reduce_max_sync(0xffffffffu, x);
            if ((tid & 31) == 0) s_top[h & 1][tid >> 5] = x;
            __syncthreads();
            return __reduce_max_sync(0xffffffffu, (tid & 31) < threads / 32 ? s_top[h & 1][tid & 31] : 0u);
        };
        uint32_t top = over_block(__float_as_uint(peak) & 0x7FFFFFFFu);
        const bool odd = top > 0x7F7FFFFFu;
        if (odd) {   // again, without them
            if (tid == 0) atomicOr(A.err, TQ_DEVERR_NONFINITE);
            top = 0;
            each([&](int, const float (&xa)[8], const float (&xb)[8]) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t u = __float_as_uint(i < 8 ? xa[i & 7] : xb[i & 7]) & 0x7FFFFFFFu;
                    if (u <= 0x7F7FFFFFu) top = max(top, u);
                }
            });
            __syncthreads();
            top = over_block(top);
            __syncthreads();
        }
        const int e_new = scale_exponent<I8>(__uint_as_float(top)), e = max(e_old, e_new);
        const bool any = odd || e_new == 63;   // some value may be out of range
        const float inv = exp2i(-e);
        uint8_t* dst = (is_v ? P.vc : P.kc) + unit * (static_cast<int64_t>(P.BT) * D);
        each([&](int tok, const float (&xa)[8], const float (&xb)[8]) {
            uint8_t* d = dst + (first + tok) * D;
            auto code = [&](const float (&y)[8]) {
                return any ? make_uint2(encode4<I8>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv), encode4<I8>(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv))
                           : make_uint2(encode4<I8, false>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                        encode4<I8, false>(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
            };
            const uint2 wa = code(xa), wb = code(xb);
            if (cc == ca + 8) {
                *reinterpret_cast<uint4*>(d + ca) = make_uint4(wa.x, wa.y, wb.x, wb.y);
            } else {
                *reinterpret_cast<uint2*>(d + ca) = wa;
                *reinterpret_cast<uint2*>(d + cc) = wb;
            }
        });
        if (first > 0 && e > e_old) {   // the earlier tokens' codes at the larger scale
            const float down = exp2i(max(e_old - e, -126));
            for (int c = tid; c < first * (D / 16); c += threads) {
                uint4* p = reinterpret_cast<uint4*>(dst) + c;
                uint4 w = *p;
                w.x = recode<I8>(w.x, down), w.y = recode<I8>(w.y, down), w.z = recode<I8>(w.z, down), w.w = recode<I8>(w.w, down);
                *p = w;
            }
        }
        if (tid == 0) *sx = static_cast<uint8_t>(e + 127);
    }
}

template <typename T, int D, bool I8>
cudaError_t launch_append_f(const AppendArgs& args, int sms, cudaStream_t s) {
    AppendArgs a = args;
    const int blocks = a.n_new == 1 ? 1 : (a.n_new - 1) / a.pool.BT + 2;   // a run of n_new slots touches at most these
    const int tokens = std::min(a.n_new, a.pool.BT);
    // heads of a CTA: the most that leave two CTAs for every SM
    int heads = 1;
    while (heads < a.pool.H && static_cast<int64_t>(2) * blocks * a.batch * ((a.pool.H + 2 * heads - 1) / (2 * heads)) >= 2 * sms) heads *= 2;
    // the angles in shared memory, but for the largest blocks and rotations; the more they take, the fewer
    // CTAs an SM holds, and the more threads each has
    constexpr int kMostSmem = 192 * 1024;
    const int angles = a.rope.rot > 0 ? tokens * (D / 2 + 8) * 8 : 0;
    a.angle_smem = angles <= kMostSmem ? angles : 0;
    const int most = angles > 100 * 1024 ? 1024 : angles > 50 * 1024 ? 512 : 256;
    const int threads = std::max(32, std::min(most, (tokens * (D / 16) + 31) / 32 * 32));
    const int k = most == 1024 ? 2 : most == 512 ? 1 : 0;
    auto kernel = k == 2 ? append_kernel<T, D, I8, 1024> : k == 1 ? append_kernel<T, D, I8, 512> : append_kernel<T, D, I8, 256>;
    if (a.angle_smem > 40 * 1024) {   // (a launch's first 48 KB hold the static arrays too, 1.3 KB at most)
        static std::atomic<uint64_t> allowed[3] = {};
        const cudaError_t e = allow_smem(kernel, kMostSmem, allowed[k]);
        if (e != cudaSuccess) return e;
    }
    kernel<<<dim3(2 * blocks, (a.pool.H + heads - 1) / heads, a.batch), threads, a.angle_smem, s>>>(a, heads);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_append_t(const AppendArgs& a, int format, int sms, cudaStream_t s) {
    return format == TQ_KV8_INT8 ? launch_append_f<T, D, true>(a, sms, s) : launch_append_f<T, D, false>(a, sms, s);
}

template <typename T>
cudaError_t launch_append_d(const AppendArgs& a, int D, int format, int sms, cudaStream_t s) {
    return D == 64 ? launch_append_t<T, 64>(a, format, sms, s)
                   : D == 128 ? launch_append_t<T, 128>(a, format, sms, s) : launch_append_t<T, 256>(a, format, sms, s);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int D, int format, int dtype, int sms, cudaStream_t s) {
    if (dtype == TQ_F32) return launch_append_d<float>(a, D, format, sms, s);
    if (dtype == TQ_F16) return launch_append_d<__half>(a, D, format, sms, s);
    return launch_append_d<__nv_bfloat16>(a, D, format, sms, s);
}

}  // namespace kv8
}  // namespace tq
