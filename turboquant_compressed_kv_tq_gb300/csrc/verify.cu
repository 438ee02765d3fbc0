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

#include "kv8_device.cuh"
#include "serve.h"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace tq {
namespace serve {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMostCtas = 8;
constexpr int kUnits = 128, kStages = 3;   // a warp's pieces of a row: units of 16 bytes, and how many are on their way
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLn2 = 0.69314718f;

__device__ __forceinline__ float number(float x) { return x; }
__device__ __forceinline__ float number(__half x) { return __half2float(x); }
__device__ __forceinline__ float number(__nv_bfloat16 x) { return __bfloat162float(x); }

// The values of 16 bytes.
__device__ __forceinline__ void numbers(const uint4& u, float* x, float) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void numbers(const uint4& u, float* x, __nv_bfloat16) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ void numbers(const uint4& u, float* x, __half) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}
// 8 values at a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) numbers(__ldg(reinterpret_cast<const uint4*>(p) + i), x + i * 16 / sizeof(T), T());
}

using kv8::ex2;
using kv8::rcp;

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

// log2(e) / T as c + lo, both positive, so that what is masked (-inf) stays -inf in either product: log2(e) = 1.442695 (rounded down)
// + 1.9259630e-8, the quotient rounded down, and what the division leaves. To 2^-44.
struct Scale {
    float c, lo;
    __device__ __forceinline__ explicit Scale(float T) {
        constexpr float hi = 0x1.715476p+0f, rest = 1.9259630e-8f;
        c = __fdiv_rd(hi, T);
        lo = __fdividef(fmaf(-c, T, hi) + rest, T);
    }
    __device__ __forceinline__ float weight(float d) const { return ex2(fmaf(d, c, d * lo)); }   // d <= 0
    // The same with the exponent's rounding put back: to 2^-22. NaN of a masked value.
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

// A row as units of 16 bytes: the values before the first whole one, a CTA's units [u0, u1), the first value behind the last one.
struct Units {
    int head, u0, u1, tail;
};
template <typename T>
__device__ __forceinline__ Units units(const T* row, int V, int each, int rank) {
    constexpr int kIn = 16 / sizeof(T);
    Units r;
    r.head = min(V, static_cast<int>((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(T)));
    const int n = (V - r.head) / kIn;
    r.tail = r.head + n * kIn;
    r.u0 = min(n, rank * each);
    r.u1 = min(n, r.u0 + each);
    return r;
}

// What is known of a row, or a part of it: the largest value, the sum of weights relative to it, and where it is.
struct Seen {
    float top, sum;   // (nothing but masked values: sum 0)
    int at;
    template <int N, typename F>
    __device__ __forceinline__ void take(const float (&x)[N], const Scale& S, bool where, F&& index) {
        float t = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) t = fmaxf(t, x[i]);
        if (t > top) {
            sum *= S.weight(top - t);
            top = t;
            at = INT_MAX;
        }
        if (where && t == top) {
#pragma unroll
            for (int i = N - 1; i >= 0; --i)
                if (x[i] == t) at = min(at, index(i));
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
    // With what the lanes o apart know, for all of them.
    __device__ __forceinline__ void join(const Scale& S, int lanes) {
        float t = top;
        for (int o = lanes / 2; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(kAll, t, o));
        sum *= S.weight(top - t);
        if (top < t) at = INT_MAX;
        top = t;
        for (int o = lanes / 2; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(kAll, sum, o);
            at = min(at, __shfl_xor_sync(kAll, at, o));
        }
    }
};
__device__ __forceinline__ Seen nothing() { return Seen{-FLT_MAX, 0.0f, INT_MAX}; }

struct Best {
    float v;   // a positive score
    int i;
    __device__ __forceinline__ void meet(float w, int j) {   // the larger, the lower index of equals
        if (w > v || (w == v && j < i)) v = w, i = j;
    }
};
__device__ __forceinline__ Best nobody() { return Best{0.0f, INT_MAX}; }

struct Shared {
    uint64_t bars[kWarps][kStages];
    Best best_warp[kWarps];
    Best best[2][kMostCtas];   // written by each CTA of the cluster
    int kept, odd;             // odd: a value of this CTA's part of some row is +inf or NaN
};

// Shared memory behind `Shared`: of each row what the warps saw, what the CTAs saw (written by each of the cluster), and all of it;
// then the warps' pieces.
__host__ __device__ constexpr int seen_bytes(int rows) { return (rows * (kWarps + kMostCtas + 1) * static_cast<int>(sizeof(Seen)) + 127) / 128 * 128; }
constexpr int kRing = kWarps * kStages * kUnits * 16;

template <typename T, typename Q>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const __grid_constant__ VerifyArgs A) {
    constexpr int kIn = 16 / sizeof(T), kPer = kUnits / 32;   // values of a unit, units of a lane in a piece
    __shared__ Shared S;
    extern __shared__ __align__(128) unsigned char s_dynamic[];
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int b = blockIdx.x / ctas, tid = threadIdx.x, lane = tid % 32, warp = tid / 32, V = A.V, K = A.K;
    const tq_drafts& D = A.d;
    Seen* const seen_warp = reinterpret_cast<Seen*>(s_dynamic);    // [row][warp]
    Seen* const seen_part = seen_warp + (K + 1) * kWarps;           // [row][CTA]
    Seen* const seen = seen_part + (K + 1) * kMostCtas;             // [row]
    uint4* const ring = reinterpret_cast<uint4*>(s_dynamic + seen_bytes(K + 1)) + warp * kStages * kUnits;
    cluster.barrier_arrive();   // (waited for before the first write into another CTA)
    const bool probs = D.target_probs != 0;
    const T* target = static_cast<const T*>(D.target) + b * D.target_stride_batch;
    const Q* draft = static_cast<const Q*>(D.draft) + (D.draft ? b * D.draft_stride_batch : 0);
    const int each = (static_cast<int>(V / kIn) + ctas - 1) / ctas;
    if (tid == 0) S.kept = K, S.odd = 0;
    if (lane < kStages) tc::mbar_init(&S.bars[warp][lane], 1);
    tc::mbar_fence_init();
    __syncwarp();
    // ---- a warp's pieces of the rows, one row behind the other (lane 0 asks for them)
    int issued = 0, done = 0, last_row = probs ? -1 : 0, ask_row = 0;   // the first row is needed whatever k is
    Units ask = units(target, V, each, rank);
    int ask_u = ask.u0 + warp * kUnits;
    auto fill = [&]() {
        while (issued - done < kStages && last_row >= 0) {
            if (ask_u < ask.u1) {
                const T* from = target + ask_row * D.target_stride_row + ask.head + static_cast<int64_t>(ask_u) * kIn;
                const unsigned bytes = min(kUnits, ask.u1 - ask_u) * 16;
                uint64_t* bar = &S.bars[warp][issued % kStages];
                tc::mbar_expect_tx(bar, bytes);
                tc::bulk_g2s(ring + issued % kStages * kUnits, from, bytes, bar);
                ++issued;
                ask_u += kWarps * kUnits;
            } else if (ask_row < last_row) {
                ++ask_row;
                ask = units(target + ask_row * D.target_stride_row, V, each, rank);
                ask_u = ask.u0 + warp * kUnits;
            } else {
                break;
            }
        }
    };
    if (lane == 0) fill();
    int k = D.draft_lens ? D.draft_lens[b] : K;
    const float T_ = !D.noise ? 0.0f : D.temperatures ? D.temperatures[b] : 1.0f;
    if (k < 0 || k > K) {
        if (rank == 0 && tid == 0) atomicOr(A.err, TQ_DEVERR_SEQLEN);
        k = min(max(k, 0), K);
    }
    const bool greedy = !(T_ > 0.0f), stats = !probs || greedy;   // (probabilities are as they are)
    const Scale scale(greedy ? 1.0f : fminf(fmaxf(T_, 0x1p-120f), 0x1p100f));
    last_row = stats ? k : -1;
    if (lane == 0) fill();
    // draft i is lane i / 8 of warp i % 8's
    const int mine = warp + kWarps * lane;
    int d = -1;
    float x_d = 0.0f, q_d = 1.0f, u_d = 0.0f;
    if (lane < 8 && mine < k) {
        d = D.draft_tokens[static_cast<int64_t>(b) * K + mine];
        if (!greedy) u_d = D.uniforms[static_cast<int64_t>(b) * K + mine];
    }
    const int share = (V + ctas - 1) / ctas, i_begin = min(V, rank * share), i_end = min(V, i_begin + share);
    if (tid == 32 && !greedy) ahead(D.noise + b * D.noise_stride, i_begin, i_end);
    // ---- each row's largest value, where it is, and its sum
    if (stats) {
        for (int i = 0; i <= k; ++i) {
            const T* row = target + i * D.target_stride_row;
            const Units part = units(row, V, each, rank);
            // what lies outside whole units: before them the first CTA's, behind them the last one's
            int edge = -1;
            if (warp == 0) {
                if (rank == 0 && lane < part.head) edge = lane;
                if (rank == ctas - 1 && lane >= 16 && part.tail + lane - 16 < V) edge = part.tail + lane - 16;
            }
            Seen s = nothing();
            auto where = [&](int u, int e) { return part.head + (u + e / kIn * 32 + lane) * kIn + e % kIn; };
            for (int u = part.u0 + warp * kUnits; u < part.u1; u += kWarps * kUnits) {
                const int st = done % kStages;
                if (!tc::mbar_wait(&S.bars[warp][st], done / kStages & 1)) {
                    if (lane == 0) atomicOr(A.err, TQ_DEVERR_TIMEOUT);
                    tc::mbar_wait(&S.bars[warp][st], done / kStages & 1);
                }
                float x[kPer * kIn];
#pragma unroll
                for (int v = 0; v < kPer; ++v) {
                    if (u + v * 32 + lane < part.u1) {
                        numbers(ring[st * kUnits + v * 32 + lane], x + v * kIn, T());
                    } else {
#pragma unroll
                        for (int e = 0; e < kIn; ++e) x[v * kIn + e] = -INFINITY;
                    }
                }
                __syncwarp();
                ++done;
                if (lane == 0) fill();
                s.take(x, scale, greedy, [&](int e) { return where(u, e); });
            }
            if (edge >= 0) {
                const float x[1] = {number(row[edge])};
                s.take(x, scale, greedy, [&](int) { return edge; });
            }
            if (!(s.sum < INFINITY)) {   // a NaN, or +inf (inf - inf): once more, as they count
                S.odd = 1;
                atomicOr(A.err, TQ_DEVERR_NONFINITE);
                s = nothing();
                auto one = [&](int at) {
                    const float x[1] = {logit(number(row[at]))};
                    s.take(x, scale, greedy, [&](int) { return at; });
                };
                for (int u = part.u0 + warp * kUnits; u < part.u1; u += kWarps * kUnits)
                    for (int e = 0; e < kPer * kIn; ++e)
                        if (u + e / kIn * 32 + lane < part.u1) one(where(u, e));
                if (edge >= 0) one(edge);
            }
            s.join(scale, 32);
            if (lane == 0) seen_warp[i * kWarps + warp] = s;
        }
    }
    if (lane < 8 && mine < k && d >= 0 && d < V) {
        x_d = number(target[mine * D.target_stride_row + d]);
        if (D.draft && !greedy) q_d = number(draft[mine * D.draft_stride_row + d]);
    }
    __syncthreads();
    cluster.barrier_wait();
    if (stats) {   // row i is warp i % 8's, here and below
        for (int i = warp; i <= k; i += kWarps) {
            Seen s = lane < kWarps ? seen_warp[i * kWarps + lane] : nothing();
            s.join(scale, kWarps);
            if (lane < ctas) cluster.map_shared_rank(seen_part, lane)[i * kMostCtas + rank] = s;
        }
        cluster.sync();
    }
    // ---- how many drafts stand
    for (int i = warp; i <= k; i += kWarps) {
        Seen s = nothing();
        if (stats) {
            if (lane < ctas) s = seen_part[i * kMostCtas + lane];
            s.join(scale, kMostCtas);
            s.top = __shfl_sync(kAll, s.top, 0), s.sum = __shfl_sync(kAll, s.sum, 0), s.at = __shfl_sync(kAll, s.at, 0);
            if (lane == 0) seen[i] = s;
        }
        if (lane == i / kWarps && i < k) {
            bool stands = d >= 0 && d < V;
            if (greedy) {
                stands = stands && d == s.at && (probs ? s.top > 0.0f : s.sum > 0.0f);
            } else if (stands) {   // u q < p, times the sum
                const float p = probs ? x_d : scale.weight_near(logit(x_d) - s.top);
                stands = static_cast<double>(u_d) * q_d * (probs ? 1.0f : s.sum) < p;
            }
            if (!stands) atomicMin(&S.kept, i);
        }
    }
    if (tid == 0) atomicMin(&S.kept, k);
    __syncthreads();
    const int n = S.kept;
    const T* row = target + n * D.target_stride_row;
    int next = -1;
    if (greedy) {
        if (probs ? seen[n].top > 0.0f : seen[n].sum > 0.0f) next = seen[n].at;
    } else {
        // ---- the next token, by scores times the sum: in the second round, only where the first finds nothing, without the
        // drafts' probabilities
        const float* noise = D.noise + b * D.noise_stride;
        const float top = probs ? 0.0f : seen[n].top, sum = probs ? 1.0f : seen[n].sum;
        const bool odd = S.odd != 0;
        const uint64_t off = pair(-top, -top), c = pair(scale.c, scale.c), nc = pair(-scale.c, -scale.c), nlo = pair(-scale.lo, -scale.lo),
                       nln2 = pair(-kLn2, -kLn2), nsum = pair(-sum, -sum);
        for (int round = 0; round < 2 && next < 0; ++round) {
            const bool minus = round == 0 && n < k;
            if (round == 1 && n == k) break;
            const Q* q = minus && D.draft ? draft + n * D.draft_stride_row : nullptr;
            const int own = minus && !D.draft ? D.draft_tokens[static_cast<int64_t>(b) * K + n] : -1;
            if (tid == 0 && q) ahead(q, i_begin, i_end);
            Best best = nobody();
            // 8 values, those that are none -inf (0 of probabilities)
            auto race = [&](float (&x)[8], float (&y)[8], const float (&e)[8], auto&& index) {
                if (odd && !probs) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = logit(x[i]);
                }
                if (own >= 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (index(i) == own) y[i] = 1.0f;
                }
                float s[8];
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    uint64_t w = pair(x[i], x[i + 1]);
                    if (!probs) {   // the exponent's rounding goes back into the weight (NaN of a masked value, which wins nothing)
                        const uint64_t z = add2(w, off), t = mul2(z, c), r = fma2(z, nlo, fma2(z, nc, t));
                        float t0, t1;
                        split(t, t0, t1);
                        w = pair(ex2(t0), ex2(t1));
                        w = fma2(mul2(w, nln2), r, w);
                    }
                    if (minus) w = fma2(pair(y[i], y[i + 1]), nsum, w);
                    const float e0 = fminf(fmaxf(e[i], 0x1p-100f), 0x1p24f), e1 = fminf(fmaxf(e[i + 1], 0x1p-100f), 0x1p24f);
                    split(mul2(w, pair(rcp(e0), rcp(e1))), s[i], s[i + 1]);
                }
                float m = s[0];
#pragma unroll
                for (int i = 1; i < 8; ++i) m = fmaxf(m, s[i]);
                if (m > best.v) {
                    best.v = m;
#pragma unroll
                    for (int i = 7; i >= 0; --i)
                        if (s[i] == m) best.i = index(i);
                }
            };
            const float none = probs ? 0.0f : -INFINITY;
            auto scattered = [&](int first, int step, int end) {
                for (int i0 = first; i0 < end; i0 += 8 * step) {
                    float x[8], y[8], e[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int at = i0 + i * step;
                        x[i] = none, y[i] = 0.0f, e[i] = 1.0f;
                        if (at < end) {
                            x[i] = number(row[at]), e[i] = noise[at];
                            if (q) y[i] = number(q[at]);
                        }
                    }
                    race(x, y, e, [&](int i) { return i0 + i * step; });
                }
            };
            const int head = units(row, V, each, rank).head;
            if (reinterpret_cast<uintptr_t>(noise + head) % 16 == 0 && (!q || reinterpret_cast<uintptr_t>(q + head) % 16 == 0)) {
                const int chunks = (V - head) / 8, per = (chunks + ctas - 1) / ctas, end = min(chunks, (rank + 1) * per);
#pragma unroll 2
                for (int v = rank * per + tid; v < end; v += kThreads) {
                    const int i0 = head + v * 8;
                    float x[8], y[8] = {}, e[8];
                    load8(row + i0, x);
                    load8(noise + i0, e);
                    if (q) load8(q + i0, y);
                    race(x, y, e, [&](int i) { return i0 + i; });
                }
                if (rank == 0) scattered(tid, kThreads, head);
                if (rank == ctas - 1) scattered(head + chunks * 8 + tid, kThreads, V);
            } else {   // rows that do not lie alike: one value at a time
                scattered(i_begin + tid, kThreads, i_end);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) best.meet(__shfl_xor_sync(kAll, best.v, o), __shfl_xor_sync(kAll, best.i, o));
            if (lane == 0) S.best_warp[warp] = best;
            __syncthreads();
            if (tid < ctas) {
                best = S.best_warp[0];
                for (int w = 1; w < kWarps; ++w) best.meet(S.best_warp[w].v, S.best_warp[w].i);
                cluster.map_shared_rank(&S, tid)->best[round][rank] = best;
            }
            cluster.sync();
            best = nobody();
            for (int r = 0; r < ctas; ++r) best.meet(S.best[round][r].v, S.best[round][r].i);
            next = best.i < V ? best.i : -1;
        }
    }
    if (rank != 0) return;
    if (next < 0 && tid == 0) atomicOr(A.err, TQ_DEVERR_NONFINITE);
    if (lane <= 8 && mine <= K) {
        const int64_t at = static_cast<int64_t>(b) * (K + 1) + mine;
        const int t = mine < n ? d : mine == n ? next : -1;
        A.tokens[at] = t;
        if (A.logprobs) {
            float l = 0.0f;
            if (t >= 0) {
                const float x = mine < n ? x_d : number(row[t]);
                l = probs ? logf(x) : scale.log(logit(x) - seen[mine].top) - logf(seen[mine].sum);
            }
            A.logprobs[at] = l;
        }
    }
    if (tid == 0) {
        A.accepted[b] = n;
        if (A.keep) A.keep[b] = D.seq_lens[b] + n + 1;
    }
}

template <typename T, typename Q>
cudaError_t launch(const VerifyArgs& a, cudaStream_t s) {
    // CTAs of a cluster: a piece for each warp, at most
    int ctas = 1;
    while (ctas < kMostCtas && static_cast<int64_t>(ctas) * kWarps * kUnits * 16 / static_cast<int>(sizeof(T)) < a.V) ctas *= 2;
    const int smem = seen_bytes(a.K + 1) + kRing;
    if (smem > 40 * 1024) {
        static std::atomic<uint64_t> allowed{0};
        const cudaError_t e = kv8::allow_smem(verify_kernel<T, Q>, seen_bytes(65) + kRing, allowed);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
