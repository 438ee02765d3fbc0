// Appending keys and values to the 8-bit cache, the keys rotated on the way.
//
// One CTA owns the new tokens of one block for one KV head, keys or values: it
// reads them once, rotates them (fp32), reduces the largest magnitude to the
// block's power-of-two scale, and writes the codes at that scale. The block is
// the unit because its scale is: nothing is shared between CTAs, no atomics, one
// launch. A block that already held tokens keeps its scale unless the new
// tokens need a larger one; then its earlier codes are rounded to the new one
// by the same CTA.
//
// Bound: memory (2 or 4 bytes read and 1 written a value).
#include "kv8_device.cuh"

namespace tq {
namespace kv8 {
namespace {

constexpr int kHeld = 4;   // items (16 coordinates of one token) that a thread keeps in registers

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

template <typename T, int D, bool I8>
__global__ void __launch_bounds__(256) append_kernel(AppendArgs A) {
    __shared__ uint64_t s_turns[128];
    __shared__ float s_top[8];
    __shared__ int s_id;
    const bool is_v = blockIdx.x & 1;
    const int j = blockIdx.x >> 1, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const Pool& P = A.pool;
    const int64_t start = A.seq[b];
    int n = A.news ? A.news[b] : A.n_new;
    if (start < 0 || n < 0 || n > A.n_new) {
        if (tid == 0 && j == 0 && h == 0) atomicOr(A.err, TQ_DEVERR_SEQLEN);
        return;
    }
    const int64_t cap = static_cast<int64_t>(P.max_blocks) << P.bt_shift;
    if (start + n > cap) {
        if (tid == 0 && j == 0 && h == 0) atomicOr(A.err, TQ_DEVERR_CAPACITY);
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
    const T* src = static_cast<const T*>(R.data) + b * R.sb + h * R.sh + i0 * R.st;
    const bool turn = !is_v && A.rope.rot > 0;
    if (turn) {
        for (int i = tid; i < A.rope.rot / 2; i += blockDim.x) s_turns[i] = turns_of(A.rope.inv_freq[i]);
        __syncthreads();
    }
    const int32_t* pos = A.rope.positions ? A.rope.positions + b * static_cast<int64_t>(A.n_new) + i0 : nullptr;

    // item = token * (D / 16) + chunk pair
    constexpr int J = D / 16;
    const int items = count * J;
    const int rot = turn ? A.rope.rot : 0, inter = A.rope.inter;
    auto fetch = [&](int it, float (&xa)[8], float (&xb)[8]) {
        const int tok = it / J, jj = it % J;
        int a, c;
        chunk_pair(jj, rot, inter, a, c);
        load8(src + tok * R.st + a, xa);
        load8(src + tok * R.st + c, xb);
        if (turn) rotate_pair(xa, xb, jj, A.rope, s_turns, pos ? pos[tok] : static_cast<int>(t0) + first + tok);
    };
    float top = 0.0f;
    bool odd = false;
    auto look = [&](const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float m = fabsf(x[i]);
            const bool fine = m <= FLT_MAX;
            odd |= !fine;
            top = fmaxf(top, fine ? m : 0.0f);
        }
    };
    float xa[kHeld][8], xb[kHeld][8];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        const int it = tid + k * blockDim.x;
        if (it < items) {
            fetch(it, xa[k], xb[k]);
            look(xa[k]);
            look(xb[k]);
        }
    }
    for (int it = tid + kHeld * blockDim.x; it < items; it += blockDim.x) {
        float ya[8], yb[8];
        fetch(it, ya, yb);
        look(ya);
        look(yb);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
    if (odd) atomicOr(A.err, TQ_DEVERR_NONFINITE);
    const int64_t unit = id * P.H + h;
    uint8_t* sx = (is_v ? P.vx : P.kx) + unit;
    if (tid == 0) s_id = first > 0 ? min(max(static_cast<int>(*sx) - 127, -126), 126) : -63;
    __syncthreads();
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) top = fmaxf(top, s_top[w]);
    const int e_old = s_id;
    const int e = max(e_old, scale_exponent<I8>(top));
    const float inv = exp2i(-e);
    uint8_t* dst = (is_v ? P.vc : P.kc) + unit * (static_cast<int64_t>(P.BT) * D);
    auto store = [&](int it, const float (&ya)[8], const float (&yb)[8]) {
        const int tok = it / J, jj = it % J;
        int a, c;
        chunk_pair(jj, rot, inter, a, c);
        uint8_t* d = dst + (first + tok) * D;
        *reinterpret_cast<uint2*>(d + a) = make_uint2(encode4<I8>(ya[0] * inv, ya[1] * inv, ya[2] * inv, ya[3] * inv),
                                                     encode4<I8>(ya[4] * inv, ya[5] * inv, ya[6] * inv, ya[7] * inv));
        *reinterpret_cast<uint2*>(d + c) = make_uint2(encode4<I8>(yb[0] * inv, yb[1] * inv, yb[2] * inv, yb[3] * inv),
                                                     encode4<I8>(yb[4] * inv, yb[5] * inv, yb[6] * inv, yb[7] * inv));
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        const int it = tid + k * blockDim.x;
        if (it < items) store(it, xa[k], xb[k]);
    }
    for (int it = tid + kHeld * blockDim.x; it < items; it += blockDim.x) {
        float ya[8], yb[8];
        fetch(it, ya, yb);
        store(it, ya, yb);
    }
    if (first > 0 && e > e_old) {   // the earlier tokens' codes at the larger scale
        const float down = exp2i(max(e_old - e, -126));
        for (int c = tid; c < first * (D / 16); c += blockDim.x) {
            uint4* p = reinterpret_cast<uint4*>(dst) + c;
            uint4 w = *p;
            w.x = recode<I8>(w.x, down), w.y = recode<I8>(w.y, down), w.z = recode<I8>(w.z, down), w.w = recode<I8>(w.w, down);
            *p = w;
        }
    }
    if (tid == 0) *sx = static_cast<uint8_t>(e + 127);
}

template <typename T, int D>
cudaError_t launch_append_t(const AppendArgs& a, int format, cudaStream_t s) {
    const int blocks = (a.n_new - 1) / a.pool.BT + 2;   // a run of n_new slots touches at most these
    const int items = std::min(a.n_new, a.pool.BT) * (D / 16);
    const int threads = std::min(256, (items + 31) / 32 * 32);
    const dim3 grid(2 * (a.n_new == 1 ? 1 : blocks), a.pool.H, a.batch);
    if (format == TQ_KV8_INT8) append_kernel<T, D, true><<<grid, threads, 0, s>>>(a);
    else append_kernel<T, D, false><<<grid, threads, 0, s>>>(a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_append_d(const AppendArgs& a, int D, int format, cudaStream_t s) {
    return D == 64 ? launch_append_t<T, 64>(a, format, s)
                   : D == 128 ? launch_append_t<T, 128>(a, format, s) : launch_append_t<T, 256>(a, format, s);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int D, int format, int dtype, cudaStream_t s) {
    if (dtype == TQ_F32) return launch_append_d<float>(a, D, format, s);
    if (dtype == TQ_F16) return launch_append_d<__half>(a, D, format, s);
    return launch_append_d<__nv_bfloat16>(a, D, format, s);
}

}  // namespace kv8
}  // namespace tq
