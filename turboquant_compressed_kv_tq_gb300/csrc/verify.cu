// Verification of drafted tokens against the target's rows.
//
// Of each row of logits the largest value and the sum of weights 2^((x - top) log2(e) / T) are needed to tell whether its draft
// stands (u q(d) < p(d)); of the first row whose draft does not (or the last one), the token with the largest max(p - q, 0) / noise.
// So every logit is read once, and one row of the drafts' probabilities, of the noise and, out of the L2 cache, of the logits
// again: memory bounds it where there is much to read, the chain of steps where there is little.
//
// A cluster of CTAs has a sequence: each CTA a part of the vocabulary, of all its rows in a run without a barrier between them. The
// parts' (largest, where, sum) go into every CTA of the cluster, which all find the same number of kept drafts, and take the
// next token's row, again in parts. One launch, no workspace, nothing that two calls share; no order of arrival changes a result.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <climits>

#include "serve.h"

namespace cg = cooperative_groups;

namespace tq {
namespace serve {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMostRows = 65, kMostCtas = 8;
constexpr int kAhead = 4;   // chunks of 8 logits that a thread has on their way
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float number(float x) { return x; }
__device__ __forceinline__ float number(__half x) { return __half2float(x); }
__device__ __forceinline__ float number(__nv_bfloat16 x) { return __bfloat162float(x); }

// 8 values at a 16-byte boundary.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ void load8(const __half* p, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}

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

// Pairs of fp32 numbers in one register pair.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// A logit as it counts: +inf the largest number, NaN -inf.
__device__ __forceinline__ float logit(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }

// log2(e) / T as c + lo, both positive, so that what is masked (-inf) stays -inf in either product.
struct Scale {
    float c, lo;
    __device__ explicit Scale(double inv_t) {
        const double c64 = inv_t * 1.4426950408889634;
        c = __double2float_rd(c64);
        if (static_cast<double>(c) == c64) c = __uint_as_float(__float_as_uint(c) - 1);
        lo = static_cast<float>(c64 - static_cast<double>(c));
    }
    __device__ __forceinline__ float weight(float d) const { return ex2(fmaf(d, c, d * lo)); }   // d <= 0
};

// A row as a CTA's share of it: aligned chunks of 8, the values before them (first CTA) and behind them (last CTA).
struct Share {
    int head, v0, v1, tail;   // values before the chunks; the CTA's chunks; the first value behind them
    __device__ Share(const void* row, int size, int V, int rank, int ctas) {
        head = min(V, static_cast<int>((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / size));
        const int chunks = (V - head) / 8;
        tail = head + chunks * 8;
        const int each = (chunks + ctas - 1) / ctas;
        v0 = min(chunks, rank * each);
        v1 = min(chunks, v0 + each);
    }
};

// What a thread knows of a row: the largest value, the sum of weights relative to it, and where it is.
struct Seen {
    float top, sum;   // (nothing but masked values: sum 0)
    int at;
    template <int N, typename F>
    __device__ __forceinline__ void take(const float (&x)[N], const Scale& S, bool where, F&& index) {
        float t = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) t = fmaxf(t, x[i]);
        if (t > top || (where && at == INT_MAX && t == top)) {
            sum *= S.weight(top - t);
            top = t;
            if (where) {
#pragma unroll
                for (int i = N - 1; i >= 0; --i)
                    if (x[i] == t) at = index(i);
            }
        }
        if constexpr (N == 1) {
            sum += S.weight(x[0] - top);
        } else {
            const uint64_t off = pair(-top, -top), c = pair(S.c, S.c), lo = pair(S.lo, S.lo);
            uint64_t s = 0;
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const uint64_t d = add2(pair(x[i], x[i + 1]), off);
                float a, b;
                split(fma2(d, c, mul2(d, lo)), a, b);
                s = add2(s, pair(ex2(a), ex2(b)));
            }
            float a, b;
            split(s, a, b);
            sum += a + b;
        }
    }
};

// A thread's part of a row. kClean: some of its values are +inf or NaN.
template <bool kClean, typename T>
__device__ __forceinline__ Seen see(const T* row, int V, const Share& part, int rank, int ctas, const Scale& S, bool where) {
    Seen seen{-FLT_MAX, 0.0f, INT_MAX};
    const int tid = threadIdx.x;
    auto single = [&](int i) {
        const float x[1] = {kClean ? logit(number(row[i])) : number(row[i])};
        seen.take(x, S, where, [&](int) { return i; });
    };
    if (rank == 0 && tid < part.head) single(tid);
    for (int v = part.v0 + tid; v < part.v1; v += kAhead * kThreads) {
        float x[kAhead * 8];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            float y[8];
            if (v + u * kThreads < part.v1) {
                load8(row + part.head + static_cast<int64_t>(v + u * kThreads) * 8, y);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u * 8 + i] = kClean ? logit(y[i]) : y[i];
        }
        seen.take(x, S, where, [&](int i) { return part.head + (v + i / 8 * kThreads) * 8 + i % 8; });
    }
    if (rank == ctas - 1 && part.tail + tid < V) single(part.tail + tid);
    return seen;
}

// The larger value, the lower index of equals.
__device__ __forceinline__ void larger(float& v, int& i, float w, int j) {
    if (w > v || (w == v && j < i)) v = w, i = j;
}

struct Best {
    float v;
    int i;
};
constexpr Best kNone{-1.0f, INT_MAX};   // scores are not negative

struct Shared {
    Seen warp[kMostRows][kWarps];
    Seen part[kMostCtas][kMostRows];   // written by each CTA of the cluster
    Best best_warp[kWarps];
    Best best[2][kMostCtas];           // written by each CTA of the cluster
    float top[kMostRows];
    double sum[kMostRows];
    int at[kMostRows];
    int kept;
};

template <typename T, typename Q>
__global__ void __launch_bounds__(kThreads, 3) verify_kernel(const __grid_constant__ VerifyArgs A) {
    __shared__ Shared S;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int b = blockIdx.x / ctas, tid = threadIdx.x, lane = tid % 32, V = A.V, K = A.K;
    const tq_drafts& D = A.d;
    cluster.barrier_arrive();   // (waited for before the first write into another CTA)
    int k = D.draft_lens ? D.draft_lens[b] : K;
    if (k < 0 || k > K) {
        if (rank == 0 && tid == 0) atomicOr(A.err, TQ_DEVERR_SEQLEN);
        k = min(max(k, 0), K);
    }
    const float T_ = !D.noise ? 0.0f : D.temperatures ? D.temperatures[b] : 1.0f;
    const bool greedy = !(T_ > 0.0f), probs = D.target_probs != 0;
    const double inv_t = greedy ? 1.0 : 1.0 / static_cast<double>(fminf(fmaxf(T_, 0x1p-120f), 0x1p100f));
    const Scale scale(inv_t);
    const T* target = static_cast<const T*>(D.target) + b * D.target_stride_batch;
    const Q* draft = static_cast<const Q*>(D.draft) + (D.draft ? b * D.draft_stride_batch : 0);
    // thread i: draft i, on its way meanwhile
    int d = -1;
    float x_d = 0.0f, q_d = 1.0f, u_d = 0.0f;
    if (tid < k) {
        d = D.draft_tokens[static_cast<int64_t>(b) * K + tid];
        if (d >= 0 && d < V) {
            x_d = number(target[tid * D.target_stride_row + d]);
            if (D.draft && !greedy) q_d = number(draft[tid * D.draft_stride_row + d]);
        }
        if (!greedy) u_d = D.uniforms[static_cast<int64_t>(b) * K + tid];
    }
    // ---- each row's largest value, where it is, and its sum (probabilities are as they are)
    const bool stats = !probs || greedy;
    if (stats) {
        for (int i = 0; i <= k; ++i) {
            const T* row = target + i * D.target_stride_row;
            const Share part(row, sizeof(T), V, rank, ctas);
            Seen s = see<false>(row, V, part, rank, ctas, scale, greedy);
            if (!(s.sum < INFINITY)) {   // a NaN, or +inf (inf - inf)
                atomicOr(A.err, TQ_DEVERR_NONFINITE);
                s = see<true>(row, V, part, rank, ctas, scale, greedy);
            }
            float top = s.top;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
            s.sum *= scale.weight(s.top - top);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s.sum += __shfl_xor_sync(kAll, s.sum, o);
            s.at = static_cast<int>(__reduce_min_sync(kAll, s.top == top ? static_cast<unsigned>(s.at) : static_cast<unsigned>(INT_MAX)));
            s.top = top;
            if (lane == 0) S.warp[i][tid / 32] = s;
        }
    }
    if (tid == 0) S.kept = k;
    __syncthreads();
    cluster.barrier_wait();
    if (stats) {
        auto merge = [&](const Seen* s, int n, int stride, Seen& all, double& sum) {
            all = s[0];
            for (int w = 1; w < n; ++w) larger(all.top, all.at, s[w * stride].top, s[w * stride].at);
            sum = 0.0;
            for (int w = 0; w < n; ++w) sum += static_cast<double>(s[w * stride].sum * scale.weight(s[w * stride].top - all.top));
        };
        Seen all;
        double sum;
        if (tid <= k) {
            merge(S.warp[tid], kWarps, 1, all, sum);
            all.sum = static_cast<float>(sum);
            for (int r = 0; r < ctas; ++r) cluster.map_shared_rank(&S, r)->part[rank][tid] = all;
        }
        cluster.sync();
        if (tid <= k) {
            merge(&S.part[0][tid], ctas, kMostRows, all, sum);
            S.top[tid] = all.top;
            S.at[tid] = all.at;
            S.sum[tid] = sum;
        }
        __syncthreads();
    }
    // ---- how many drafts stand; what one token hangs on, in 64 bits
    if (tid < k) {
        bool stands = d >= 0 && d < V;
        if (greedy) {
            stands = stands && d == S.at[tid] && (probs ? S.top[tid] > 0.0f : S.sum[tid] > 0.0);
        } else if (stands) {
            const double p = probs ? static_cast<double>(x_d) : exp((static_cast<double>(logit(x_d)) - S.top[tid]) * inv_t) / S.sum[tid];
            stands = static_cast<double>(u_d) * static_cast<double>(q_d) < p;
        }
        if (!stands) atomicMin(&S.kept, tid);
    }
    __syncthreads();
    const int n = S.kept;
    const T* row = target + n * D.target_stride_row;
    int next = -1;
    if (greedy) {
        if (probs ? S.top[n] > 0.0f : S.sum[n] > 0.0) next = S.at[n];
    } else {
        // ---- the next token: in the second round, only where the first finds nothing, without the drafts' probabilities
        const float* noise = D.noise + b * D.noise_stride;
        const float top = probs ? 0.0f : S.top[n], inv = probs ? 1.0f : static_cast<float>(1.0 / S.sum[n]);
        for (int round = 0; round < 2 && next < 0; ++round) {
            const bool minus = round == 0 && n < k;
            if (round == 1 && n == k) break;
            const Q* q = minus && D.draft ? draft + n * D.draft_stride_row : nullptr;
            const int own = minus && !D.draft ? D.draft_tokens[static_cast<int64_t>(b) * K + n] : -1;
            Best best = kNone;
            auto race = [&](float x, float y, float e, int i) {
                float p = x;
                if (!probs) {
                    // the exponent's rounding goes back into the weight
                    const float z = logit(x) - top, t = z * scale.c;
                    const float r = fmaf(z, scale.c, -t) + z * scale.lo;
                    const float w = ex2(t);
                    p = (t > -126.0f ? fmaf(w, r * 0.69314718f, w) : 0.0f) * inv;
                }
                p -= i == own ? 1.0f : y;
                const float s = p * rcp(fmaxf(e, 0x1p-100f));
                if (p > 0.0f && s > best.v) best.v = s, best.i = i;
            };
            Share part(row, sizeof(T), V, rank, ctas);
            const bool whole = reinterpret_cast<uintptr_t>(noise + part.head) % 16 == 0 && (!q || reinterpret_cast<uintptr_t>(q + part.head) % 16 == 0);
            if (whole) {
                auto single = [&](int i) { race(number(row[i]), q ? number(q[i]) : 0.0f, noise[i], i); };
                if (rank == 0 && tid < part.head) single(tid);
                for (int v = part.v0 + tid; v < part.v1; v += kThreads) {
                    const int64_t i0 = part.head + static_cast<int64_t>(v) * 8;
                    float x[8], y[8] = {}, e[8];
                    load8(row + i0, x);
                    load8(noise + i0, e);
                    if (q) load8(q + i0, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) race(x[i], y[i], e[i], static_cast<int>(i0) + i);
                }
                if (rank == ctas - 1 && part.tail + tid < V) single(part.tail + tid);
            } else {   // rows that do not lie alike: one value at a time
                const int each = (V + ctas - 1) / ctas, i1 = min(V, (rank + 1) * each);
#pragma unroll 4
                for (int i = rank * each + tid; i < i1; i += kThreads) race(number(row[i]), q ? number(q[i]) : 0.0f, noise[i], i);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float w = __shfl_xor_sync(kAll, best.v, o);
                const int j = __shfl_xor_sync(kAll, best.i, o);
                larger(best.v, best.i, w, j);
            }
            if (lane == 0) S.best_warp[tid / 32] = best;
            __syncthreads();
            if (tid < ctas) {
                best = S.best_warp[0];
                for (int w = 1; w < kWarps; ++w) larger(best.v, best.i, S.best_warp[w].v, S.best_warp[w].i);
                cluster.map_shared_rank(&S, tid)->best[round][rank] = best;
            }
            cluster.sync();
            best = kNone;
            for (int r = 0; r < ctas; ++r) larger(best.v, best.i, S.best[round][r].v, S.best[round][r].i);
            next = best.i < V ? best.i : -1;
        }
    }
    if (rank != 0) return;
    if (next < 0 && tid == 0) atomicOr(A.err, TQ_DEVERR_NONFINITE);
    if (tid <= K) {
        const int t = tid < n ? d : tid == n ? next : -1;
        A.tokens[static_cast<int64_t>(b) * (K + 1) + tid] = t;
        if (A.logprobs) {
            float l = 0.0f;
            if (t >= 0) {
                const double x = tid < n ? x_d : number(row[t]);
                l = probs ? static_cast<float>(log(x)) : static_cast<float>((static_cast<double>(logit(static_cast<float>(x))) - S.top[tid]) * inv_t - log(S.sum[tid]));
            }
            A.logprobs[static_cast<int64_t>(b) * (K + 1) + tid] = l;
        }
    }
    if (tid == 0) {
        A.accepted[b] = n;
        if (A.keep) A.keep[b] = D.seq_lens[b] + n + 1;
    }
}

template <typename T, typename Q>
cudaError_t launch(const VerifyArgs& a, cudaStream_t s) {
    // CTAs of a cluster: a chunk for each thread, at most
    int ctas = 1;
    while (ctas < kMostCtas && static_cast<int64_t>(ctas) * kThreads * 8 < a.V) ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<T, Q>, a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return e;
}

template <typename T>
cudaError_t launch_q(const VerifyArgs& a, cudaStream_t s) {
    if (!a.d.draft || a.d.draft_dtype == TQ_F32) return launch<T, float>(a, s);
    if (a.d.draft_dtype == TQ_F16) return launch<T, __half>(a, s);
    return launch<T, __nv_bfloat16>(a, s);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
    if (a.d.target_dtype == TQ_F32) return launch_q<float>(a, s);
    if (a.d.target_dtype == TQ_F16) return launch_q<__half>(a, s);
    return launch_q<__nv_bfloat16>(a, s);
}

}  // namespace serve
}  // namespace tq
