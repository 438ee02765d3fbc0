// Verification of drafted tokens against the target's rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "serve.h"

namespace tq {
namespace serve {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMostRows = 65;

__device__ __forceinline__ float value(const void* p, int64_t i, int dtype) {
    if (dtype == TQ_F32) return static_cast<const float*>(p)[i];
    if (dtype == TQ_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// A logit as it counts: +inf the largest number, NaN -inf.
__device__ __forceinline__ float logit(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }

// The larger value, the lower index of equals.
__device__ __forceinline__ void larger(float& v, int& i, float w, int j) {
    if (w > v || (w == v && j < i)) v = w, i = j;
}

struct Shared {
    float v[kWarps];
    int i[kWarps];
    float s[kWarps];
    float top[kMostRows], sum[kMostRows];   // of a row: its largest logit, the sum of exp((x - top) / T)
    int at[kMostRows];                      // where the largest is
    int kept;
};

template <typename F>
__device__ void best_of(Shared& S, float v, int i, F&& done) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        const int j = __shfl_xor_sync(0xffffffffu, i, o);
        larger(v, i, w, j);
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) S.v[threadIdx.x / 32] = v, S.i[threadIdx.x / 32] = i;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWarps; ++w) larger(v, i, S.v[w], S.i[w]);
        done(v, i);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyArgs A) {
    __shared__ Shared S;
    const int b = blockIdx.x, tid = threadIdx.x, V = A.V, K = A.K;
    const tq_drafts& D = A.d;
    int k = D.draft_lens ? D.draft_lens[b] : K;
    if (k < 0 || k > K) {
        if (tid == 0) atomicOr(A.err, TQ_DEVERR_SEQLEN);
        k = min(max(k, 0), K);
    }
    const float T = !D.noise ? 0.0f : D.temperatures ? D.temperatures[b] : 1.0f;
    const bool greedy = !(T > 0.0f);
    const double inv_t = greedy ? 1.0 : 1.0 / static_cast<double>(fminf(fmaxf(T, 0x1p-120f), 0x1p100f));
    const int64_t target = b * D.target_stride_batch, draft = b * D.draft_stride_batch;
    // log2(e) / T as c + c_lo, both positive: a masked token's -inf stays -inf in either product
    const double c64 = inv_t * 1.4426950408889634;
    float c = __double2float_rd(c64);
    if (static_cast<double>(c) == c64) c = __uint_as_float(__float_as_uint(c) - 1);
    const float c_lo = static_cast<float>(c64 - static_cast<double>(c));
    // ---- each row's largest value, where it is, and its sum
    for (int i = 0; i <= k; ++i) {
        if (D.target_probs && !greedy) break;   // as they are
        const int64_t row = target + i * D.target_stride_row;
        float v = -INFINITY;
        int at = V;
        bool odd = false;
        for (int t = tid; t < V; t += kThreads) {
            const float raw = value(D.target, row + t, D.target_dtype), x = logit(raw);
            odd |= !(raw < INFINITY);
            if (x > v) v = x, at = t;
        }
        if (odd) atomicOr(A.err, TQ_DEVERR_NONFINITE);
        best_of(S, v, at, [&](float v, int at) { S.top[i] = v, S.at[i] = at; });
        const float top = S.top[i];
        float s = 0.0f;
        if (top > -INFINITY && !D.target_probs)
            for (int t = tid; t < V; t += kThreads) {
                const float x = logit(value(D.target, row + t, D.target_dtype)) - top;
                s += exp2f(fmaf(x, c, x * c_lo));
            }
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid % 32 == 0) S.s[tid / 32] = s;
        __syncthreads();
        if (tid == 0) {
            s = 0.0f;
            for (int w = 0; w < kWarps; ++w) s += S.s[w];
            S.sum[i] = s;
        }
        __syncthreads();
    }
    const float nothing = D.target_probs ? 0.0f : -INFINITY;   // the largest value of a row in which nothing can be
    // what one token hangs on, in 64 bits
    auto chance = [&](int i, int t) {
        const float x = value(D.target, target + i * D.target_stride_row + t, D.target_dtype);
        if (D.target_probs) return static_cast<double>(x);
        return exp((static_cast<double>(logit(x)) - S.top[i]) * inv_t) / S.sum[i];
    };
    auto log_chance = [&](int i, int t) {
        const float x = value(D.target, target + i * D.target_stride_row + t, D.target_dtype);
        if (D.target_probs) return static_cast<float>(log(static_cast<double>(x)));
        return static_cast<float>((static_cast<double>(logit(x)) - S.top[i]) * inv_t - log(static_cast<double>(S.sum[i])));
    };
    if (tid == 0) {
        int n = 0;
        for (; n < k; ++n) {
            const int d = D.draft_tokens[static_cast<int64_t>(b) * K + n];
            if (d < 0 || d >= V) break;
            if (greedy) {
                if (d != S.at[n] || !(S.top[n] > nothing)) break;
            } else {
                const double q = D.draft ? value(D.draft, draft + n * D.draft_stride_row + d, D.draft_dtype) : 1.0f;
                if (!(D.uniforms[static_cast<int64_t>(b) * K + n] * q < chance(n, d))) break;
            }
        }
        S.kept = n;
    }
    __syncthreads();
    const int n = S.kept;
    auto finish = [&](int next) {   // one thread
        int32_t* tokens = A.tokens + static_cast<int64_t>(b) * (K + 1);
        float* logs = A.logprobs ? A.logprobs + static_cast<int64_t>(b) * (K + 1) : nullptr;
        for (int i = 0; i <= K; ++i) {
            const int t = i < n ? D.draft_tokens[static_cast<int64_t>(b) * K + i] : i == n ? next : -1;
            tokens[i] = t;
            if (logs) logs[i] = t >= 0 ? log_chance(i, t) : 0.0f;
        }
        A.accepted[b] = n;
        if (A.keep) A.keep[b] = D.seq_lens[b] + n + 1;
        if (next < 0) atomicOr(A.err, TQ_DEVERR_NONFINITE);
    };
    if (greedy) {
        if (tid == 0) finish(S.top[n] > nothing ? S.at[n] : -1);
        return;
    }
    // ---- the next token
    const int64_t row = target + n * D.target_stride_row;
    const int own = n < k && !D.draft ? D.draft_tokens[static_cast<int64_t>(b) * K + n] : -1;
    const float* noise = D.noise + b * D.noise_stride;
    const float top = D.target_probs ? 0.0f : S.top[n], inv = D.target_probs ? 1.0f : 1.0f / S.sum[n];
    float vr = -1.0f, vp = -1.0f;
    int tr = V, tp = V;
    for (int t = tid; t < V; t += kThreads) {
        float p = value(D.target, row + t, D.target_dtype);
        if (!D.target_probs) {
            const float x = logit(p) - top;
            p = exp2f(fmaf(x, c, x * c_lo)) * inv;
        }
        const float e = fmaxf(noise[t], 0x1p-100f);
        const float q = n == k ? 0.0f : D.draft ? value(D.draft, draft + n * D.draft_stride_row + t, D.draft_dtype) : t == own ? 1.0f : 0.0f;
        const float r = p - q;
        if (r > 0.0f && r / e > vr) vr = r / e, tr = t;
        if (p > 0.0f && p / e > vp) vp = p / e, tp = t;
    }
    best_of(S, vr, tr, [&](float, int t) { S.i[0] = t; });
    tr = S.i[0];
    best_of(S, vp, tp, [&](float, int t) { S.i[0] = t; });
    tp = S.i[0];
    if (tid == 0) finish(tr < V ? tr : tp < V ? tp : -1);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
    verify_kernel<<<a.batch, kThreads, 0, s>>>(a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

}  // namespace serve
}  // namespace tq
