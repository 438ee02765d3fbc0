// Verification of drafted tokens against the target's rows.
//
// Of each row of logits the largest value and the sum of weights 2^((x - top) log2(e) / T) are needed to tell whether its draft
// stands (u q(d) < p(d)); of the first row whose draft does not (or the last one), the token with the largest max(p - q, 0) / noise.
// So every logit is read once, and one row of the drafts' probabilities, of the noise and of the logits again (which the L2 cache holds
// in part: 177 MB are read for 151): memory bounds it where there is much to read, the chain of steps where there is little.
//
// A cluster of CTAs has a sequence: each CTA a part of the vocabulary, of all its rows in a run. Each warp has a ring of bulk copies of its own
// (2 KB a piece) and goes through its pieces without waiting for other warps; what it saw of a row goes into every CTA of the cluster as soon
// as the row is through. All find the same number of kept drafts then, and take the next token's row, again in parts.
// One launch, no workspace, nothing that two calls share; no order of arrival changes a result.
//
// Measured: 64 sequences of 4 drafts, 131,072 tokens, bf16: 37.5 us (151 MB, 4.0 TB/s; the largest values alone, 84 MB, 24 us); one
// sequence of a draft, 32,000 tokens: 8.4 us. Pieces of 2 KB, two on their way: with three or four, three CTAs fit an SM, and 43 to 56 us.
#include <algorithm>

#include "verify_device.cuh"

namespace tq {
namespace serve {
namespace {

constexpr int kUnits = 128, kStages = 2;   // a warp's pieces of a row: units of 16 bytes, and how many are on their way

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
struct __align__(16) Seen {
    float top, sum;   // (nothing but masked values: sum 0)
    int at;
    int piece;        // of a lane while it goes through a row: the piece (its first unit) in which the largest stood first, or -1;
                      // of what is joined: 1 where a value is +inf or NaN

    __device__ __forceinline__ void rise(float t, const Scale& S, int from_piece) {
        if (t > top) {
            sum *= S.weight(top - t);
            top = t;
            at = INT_MAX;
            piece = from_piece;
        }
    }
    __device__ __forceinline__ void take(float x, const Scale& S, int i) {
        rise(x, S, -1);
        if (x == top) at = min(at, i);
        sum += S.weight(x - top);
    }
    // A lane's units of a piece, every 32nd from `from`. Usually the weights are
    // 2^(x c - m), m = top c rounded, so that each takes one product, and their sum is brought from m to the exact top c (a factor
    // 1 - delta ln 2, |delta| < 2^-11) once; c's own error, 2^-24 of itself, is common to sum and weights but for what it does to
    // (x - top) / T: with the exponent's rounding, weights 2^-d are off by 2^-22 + d 2^-23. Where m is large (temperatures near 0, rows of the lowest numbers) differences come first.
    template <typename T>
    __device__ __forceinline__ void take(const uint4* from, const Scale& S, int from_piece) {
        constexpr int kIn = 16 / sizeof(T), kPer = kUnits / 32, N = kPer * kIn / 2;
        float2 x[N];
#pragma unroll
        for (int v = 0; v < kPer; ++v) numbers(from[v * 32], x + v * kIn / 2, T());
        float t = largest(x[0].x, x[0].x, x[0].y);   // NaN if one is among them: top stays, and the sum becomes NaN
#pragma unroll
        for (int i = 1; i < N; ++i) t = largest(t, x[i].x, x[i].y);
        rise(t, S, from_piece);
        if (t == top && piece < 0) piece = from_piece;   // (a largest value of -FLT_MAX)
        const float m = top * S.near;
        if (fabsf(m) < kUsual) {
            const float2 c = both(S.near), off = both(-m);
            float2 s = both(0.0f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float2 e = __ffma2_rn(x[i], c, off);
                s = __fadd2_rn(s, make_float2(ex2(e.x), ex2(e.y)));
            }
            sum = fmaf(s.x + s.y, fmaf(fmaf(top, S.near, -m), -kLn2, 1.0f), sum);
        } else if (t > -INFINITY) {   // seldom: one value after the other
#pragma unroll 1
            for (int e = 0; e < kPer * kIn; ++e) sum += S.weight(number(reinterpret_cast<const T*>(from + e / kIn * 32)[e % kIn]) - top);
        } else if (t != t) {   // among masked tokens only
            sum = t;
        }
    }
    // Where the largest value is, by another look at the piece (`row`: its first whole unit, of `end` units; value 0 of it is value
    // `head`): only lanes that have the warp's largest look.
    template <typename T>
    __device__ __forceinline__ void find(const T* row, int end, int head) {
        constexpr int kIn = 16 / sizeof(T);
        const float t = warp_max(top);
        if (top == t && piece >= 0) {
#pragma unroll 1
            for (int v = kUnits / 32 - 1; v >= 0; --v) {
                const int u = piece + v * 32 + threadIdx.x % 32;
                if (u >= end) continue;
                float2 x[kIn / 2];
                numbers(__ldg(reinterpret_cast<const uint4*>(row) + u), x, T());
#pragma unroll
                for (int i = kIn / 2 - 1; i >= 0; --i) {
                    if (x[i].y == t) at = min(at, head + u * kIn + 2 * i + 1);
                    if (x[i].x == t) at = min(at, head + u * kIn + 2 * i);
                }
            }
        }
    }
    // With what the warp's other lanes know, for all of them.
    __device__ __forceinline__ void join(const Scale& S) {
        const float t = warp_max(top);
        sum *= S.weight(top - t);
        at = static_cast<int>(__reduce_min_sync(kAll, static_cast<unsigned>(top < t ? INT_MAX : at)));
        top = t;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
};
__device__ __forceinline__ Seen nothing() { return Seen{-FLT_MAX, 0.0f, INT_MAX, -1}; }

struct Shared {
    uint64_t bars[kWarps][kStages];
    Best best[2][kParts];      // written by every warp of the cluster
    int kept;
};

// Shared memory behind `Shared`: of each row what the cluster's warps saw (written by them) and all of it; then the warps' pieces.
__host__ __device__ constexpr int seen_bytes(int rows) { return rows * (kParts + 1) * static_cast<int>(sizeof(Seen)); }
constexpr int kRing = kWarps * kStages * kUnits * 16;

template <typename T, typename Q>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const __grid_constant__ VerifyArgs A, int log_ctas) {
    constexpr int kIn = 16 / sizeof(T), kPer = kUnits / 32;   // values of a unit, units of a lane in a piece
    __shared__ Shared S;
    extern __shared__ __align__(128) unsigned char s_dynamic[];
    const int ctas = 1 << log_ctas, rank = cluster_rank();
    const int b = blockIdx.x >> log_ctas, tid = threadIdx.x, lane = tid % 32, warp = tid / 32, V = A.V, K = A.K;
    const tq_drafts& D = A.d;
    int k = D.draft_lens ? D.draft_lens[b] : K;
    const float asked_T = !D.noise ? 0.0f : D.temperatures ? D.temperatures[b] : 1.0f;
    Seen* const seen = reinterpret_cast<Seen*>(s_dynamic);     // [row]
    Seen* const seen_part = seen + K + 1;                       // [row][CTA][warp]
    uint4* const ring = reinterpret_cast<uint4*>(s_dynamic + seen_bytes(K + 1)) + warp * kStages * kUnits;
    const bool probs = D.target_probs != 0;
    const T* target = static_cast<const T*>(D.target) + b * D.target_stride_batch;
    const Q* draft = static_cast<const Q*>(D.draft) + (D.draft ? b * D.draft_stride_batch : 0);
    const int each = (V / kIn + ctas - 1) >> log_ctas, pieces = max(1, (each + kUnits - 1) / kUnits);   // of this CTA's part of a row
    if (lane < kStages) tc::mbar_init(&S.bars[warp][lane], 1);
    if (tid == 0) S.kept = K;
    tc::mbar_fence_init();
    __syncwarp();
    cluster_arrive();   // (waited for before the first word to another CTA)
    if (k < 0 || k > K) {
        if (rank == 0 && tid == 0) atomicOr(A.err, TQ_DEVERR_SEQLEN);
        k = min(max(k, 0), K);
    }
    const bool greedy = !(asked_T > 0.0f), stats = !probs || greedy;   // (probabilities are as they are)
    // ---- all rows' pieces, one row behind the other, are dealt to the warps in eight runs, so that a warp has few rows (lane 0 asks for
    // them, each as another has been taken)
    const int all = stats ? (k + 1) * pieces : 0;
    auto run = [&](int w) { return all * w / kWarps; };   // where warp w's begins
    const int g0 = run(warp), g1 = run(warp + 1);
    int ask_g = g0, ask_row = g0 / pieces, ask_piece = g0 % pieces, ask_u0 = 0, ask_end = 0, ask_st = 0;
    const T* ask_from = nullptr;   // of unit 0
    auto ask = [&]() {
        while (ask_g < g1) {
            if (ask_piece == 0 || !ask_from) {
                const T* r = target + ask_row * D.target_stride_row;
                const Units part = units(r, V, each, rank);
                ask_from = r + part.head;
                ask_u0 = part.u0;
                ask_end = part.u1;
            }
            const int u = ask_u0 + ask_piece * kUnits;
            ++ask_g;
            if (++ask_piece == pieces) ask_piece = 0, ++ask_row;
            if (u >= ask_end) continue;   // (rows that begin elsewhere may have a unit less)
            const unsigned bytes = min(kUnits, ask_end - u) * 16;
            uint64_t* bar = &S.bars[warp][ask_st];
            tc::mbar_expect_tx(bar, bytes);
            tc::bulk_g2s(ring + ask_st * kUnits, ask_from + static_cast<int64_t>(u) * kIn, bytes, bar);
            ask_st = ask_st + 1 < kStages ? ask_st + 1 : 0;
            return;
        }
    };
    if (lane == 0) {
#pragma unroll 1
        for (int i = 0; i < kStages; ++i) ask();
    }
    // draft i is lane i / 8 of warp i % 8's
    const int mine = warp + kWarps * lane;
    int d = -1;
    float x_d = 0.0f, q_d = 1.0f, u_d = 0.0f;
    if (lane < 8 && mine < k) {
        d = D.draft_tokens[static_cast<int64_t>(b) * K + mine];
        if (!greedy) u_d = D.uniforms[static_cast<int64_t>(b) * K + mine];
    }
    const Scale scale(greedy ? 1.0f : fminf(fmaxf(asked_T, 0x1p-120f), 0x1p100f));
    const int share = (V + ctas - 1) >> log_ctas, i_begin = min(V, rank * share), i_end = min(V, i_begin + share);
    if (tid == 32 && !greedy) ahead(D.noise + b * D.noise_stride, i_begin, i_end);
    // ---- each row's largest value, where it is, and its sum
    bool begun = false;   // every CTA of the cluster has
    if (g0 < g1) {
        int st = 0, phase = 0;
#pragma unroll 1
        for (int i = g0 / pieces; i * pieces < g1; ++i) {
            const T* row = target + i * D.target_stride_row;
            const Units part = units(row, V, each, rank);
            const int first = part.u0 + max(0, g0 - i * pieces) * kUnits, last = min(part.u1, part.u0 + (g1 - i * pieces) * kUnits);   // of this warp
            // what lies outside whole units: before them the first CTA's, behind them the last one's
            int edge = -1;
            float x_edge = 0.0f;
            if (g0 <= i * pieces) {   // (the warp that has its first piece)
                if (rank == 0 && lane < part.head) edge = lane;
                if (rank == ctas - 1 && lane >= 16 && part.tail + lane - 16 < V) edge = part.tail + lane - 16;
                if (edge >= 0) x_edge = number(row[edge]);
            }
            Seen s = nothing();
            auto where = [&](int u, int e) { return part.head + (u + e / kIn * 32 + lane) * kIn + e % kIn; };
#pragma unroll 1
            for (int u = first; u < last; u += kUnits) {
                if (!tc::mbar_wait(&S.bars[warp][st], phase)) {   // once more, so that no copy is on its way when the kernel ends
                    if (lane == 0) atomicOr(A.err, TQ_DEVERR_TIMEOUT);
                    tc::mbar_wait(&S.bars[warp][st], phase);
                }
                uint4* from = ring + st * kUnits + lane;
                if (u + kUnits > part.u1) {   // behind the last unit nothing can be
                    const uint32_t none = sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
#pragma unroll 1
                    for (int v = 0; v < kPer; ++v)
                        if (u + v * 32 + lane >= part.u1) from[v * 32] = make_uint4(none, none, none, none);
                    tc::fence_proxy_async_smem();
                }
                s.template take<T>(from, scale, u);
                __syncwarp();
                if (lane == 0) ask();
                if (++st == kStages) st = 0, phase ^= 1;
            }
            if (edge >= 0) s.take(x_edge, scale, edge);
            const bool odd = __any_sync(kAll, !(s.sum < INFINITY));
            if (!(s.sum < INFINITY)) {   // a NaN, or +inf (inf - inf): once more, as they count
                if (!probs) atomicOr(A.err, TQ_DEVERR_NONFINITE);
                s = nothing();
#pragma unroll 1
                for (int u = first; u < last; u += kUnits)
#pragma unroll 1
                    for (int e = 0; e < kPer * kIn; ++e)
                        if (u + e / kIn * 32 + lane < part.u1) s.take(logit(number(row[where(u, e)])), scale, where(u, e));
                if (edge >= 0) s.take(logit(x_edge), scale, edge);
            }
            if (__any_sync(kAll, s.sum > 0.0f)) {
                if (greedy) s.find(row + part.head, part.u1, part.head);
                s.join(scale);
            }
            if (!begun) cluster_wait();
            begun = true;
            if (lane < ctas)
                send(remote(&seen_part[(i * kMostCtas + rank) * kWarps + warp], lane), __float_as_uint(s.top), __float_as_uint(s.sum), static_cast<uint32_t>(s.at), odd ? 1u : 0u);
        }
    }
    if (lane < 8 && mine < k && d >= 0 && d < V) {
        x_d = number(target[mine * D.target_stride_row + d]);
        if (D.draft && !greedy) q_d = number(draft[mine * D.draft_stride_row + d]);
    }
    if (!begun) cluster_wait();
    if (stats) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // ---- how many drafts stand: row i is warp i % 8's
#pragma unroll 1
    for (int i = warp; i <= k; i += kWarps) {
        Seen s = nothing();
        if (stats) {
            // (of each CTA the warps that have pieces of the row)
            const Seen* p = seen_part + i * kParts;
            const int w = lane % kWarps;
            const bool theirs = max(run(w), i * pieces) < min(run(w + 1), (i + 1) * pieces);
            if (theirs && lane < ctas * kWarps) s = p[lane];
            Seen more = theirs && lane + 32 < ctas * kWarps ? p[lane + 32] : nothing();
            const bool odd = __any_sync(kAll, s.piece > 0 || more.piece > 0);
            if (more.top > s.top) { const Seen x = s; s = more; more = x; }
            s.sum += more.sum * scale.weight(more.top - s.top);
            if (more.top == s.top) s.at = min(s.at, more.at);
            s.join(scale);
            s.piece = odd;
            if (lane == 0) seen[i] = s;
        }
        if (lane == i / kWarps && i < k) {
            bool stands = d >= 0 && d < V;
            if (greedy) {
                stands = stands && d == s.at && (probs ? s.top > 0.0f : s.sum > 0.0f);
            } else if (stands) {   // u q < p, times the sum
                stands = u_d * q_d * (probs ? 1.0f : s.sum) < (probs ? x_d : scale.weight_near(logit(x_d) - s.top));
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
        const bool odd = stats && seen[n].piece > 0;
        const float m = top * scale.near;
        const bool usual = fabsf(m) < kUsual;   // as in Seen::take: the weights are then relative to m, and so is their sum
        const float whole = usual && !probs ? fmaf(sum, fmaf(top, scale.near, -m) * kLn2, sum) : sum;
        const int head = units(row, V, each, rank).head, chunks = (V - head) / 8;
#pragma unroll 1
        for (int round = 0; round < 2 && next < 0; ++round) {
            const bool minus = round == 0 && n < k;
            if (round == 1 && n == k) break;
            const Q* q = minus && D.draft ? draft + n * D.draft_stride_row : nullptr;
            const int own = minus && !D.draft ? D.draft_tokens[static_cast<int64_t>(b) * K + n] : -1;
            if (tid == 0 && q) ahead(q, i_begin, i_end);
            Best best{0.0f, INT_MAX};
            // 8 values, those that are none -inf (0 of probabilities)
            auto race = [&](float2 (&x)[4], float2 (&y)[4], const float2 (&e)[4], auto&& index) {
                if (!probs) {
                    if (odd) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = make_float2(logit(x[i].x), logit(x[i].y));
                    }
                    if (usual) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 t = __ffma2_rn(x[i], both(scale.near), both(-m));
                            x[i] = make_float2(ex2(t.x), ex2(t.y));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = make_float2(scale.weight(x[i].x - top), scale.weight(x[i].y - top));
                    }
                }
                if (own >= 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (index(2 * i) == own) y[i].x = 1.0f;
                        if (index(2 * i + 1) == own) y[i].y = 1.0f;
                    }
                }
                float2 s[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 w = minus ? __ffma2_rn(y[i], both(-whole), x[i]) : x[i];
                    s[i] = __fmul2_rn(w, make_float2(rcp(fmaxf(e[i].x, 0x1p-100f)), rcp(fmaxf(e[i].y, 0x1p-100f))));
                }
                const float here = fmaxf(fmaxf(fmaxf(s[0].x, s[0].y), fmaxf(s[1].x, s[1].y)), fmaxf(fmaxf(s[2].x, s[2].y), fmaxf(s[3].x, s[3].y)));
                if (here >= best.v && here > 0.0f) {
                    int at = 0;
#pragma unroll
                    for (int i = 3; i >= 0; --i) {
                        if (s[i].y == here) at = index(2 * i + 1);
                        if (s[i].x == here) at = index(2 * i);
                    }
                    best.meet(here, at);
                }
            };
            // rows that lie alike in chunks of 8, and what lies outside those (the first CTA's) one value at a time; others all so
            const bool alike = reinterpret_cast<uintptr_t>(noise + head) % 16 == 0 && (!q || reinterpret_cast<uintptr_t>(q + head) % 16 == 0);
            const int per = (chunks + ctas - 1) >> log_ctas;
#pragma unroll 1
            for (int job = 0; job < (alike && rank == 0 ? 3 : 1); ++job) {
                const bool eight = alike && job == 0;
                const int step = eight ? 1 : kThreads;   // between a thread's 8 values
                const int begin = !alike ? i_begin : job == 0 ? head + rank * per * 8 : job == 1 ? 0 : head + chunks * 8;
                const int end = !alike ? i_end : job == 0 ? head + min(chunks, (rank + 1) * per) * 8 : job == 1 ? head : V;
#pragma unroll 1
                for (int i0 = begin + (eight ? tid * 8 : tid); i0 < end; i0 += 8 * kThreads) {
                    float2 x[4], y[4] = {}, e[4];
                    if (eight) {
                        load8(row + i0, x);
                        load8(noise + i0, e);
                        if (q) load8(q + i0, y);
                    } else {
                        const float none = probs ? 0.0f : -INFINITY;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float &xi = i % 2 ? x[i / 2].y : x[i / 2].x, &yi = i % 2 ? y[i / 2].y : y[i / 2].x, &ei = i % 2 ? e[i / 2].y : e[i / 2].x;
                            const int at = i0 + i * kThreads;
                            xi = none, ei = 1.0f;
                            if (at < end) {
                                xi = number(row[at]), ei = noise[at];
                                if (q) yi = number(q[at]);
                            }
                        }
                    }
                    race(x, y, e, [&](int i) { return i0 + i * step; });
                }
            }
            best.join();
            if (lane < ctas) send(remote(&S.best[round][rank * kWarps + warp], lane), __float_as_uint(best.v), static_cast<uint32_t>(best.i));
            cluster_arrive();
            cluster_wait();
            best = Best{0.0f, INT_MAX};
            if (lane < ctas * kWarps) best = S.best[round][lane];
            if (lane + 32 < ctas * kWarps) best.meet(S.best[round][lane + 32].v, S.best[round][lane + 32].i);
            best.join();
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
cudaError_t launch(const VerifyArgs& a, int sms, cudaStream_t s) {
    // CTAs of a cluster: as many as fill the SMs once (four on each), and a piece for each warp, at most
    int log_ctas = 0;
    while ((1 << log_ctas) < kMostCtas && (static_cast<int64_t>(kWarps * kUnits * 16 / sizeof(T)) << log_ctas) < a.V &&
           (static_cast<int64_t>(a.batch) << (log_ctas + 1)) <= 4 * sms)
        ++log_ctas;
    const int smem = seen_bytes(a.K + 1) + kRing;
    if (smem > 40 * 1024) {   // (a launch's first 48 KB hold `Shared` too)
        static std::atomic<uint64_t> allowed{0};
        const cudaError_t e = kv8::allow_smem(verify_kernel<T, Q>, seen_bytes(65) + kRing, allowed);
        if (e != cudaSuccess) return e;
    }
    return launch_cluster(verify_kernel<T, Q>, a, log_ctas, smem, s);
}

template <typename T>
cudaError_t launch_q(const VerifyArgs& a, int sms, cudaStream_t s) {
    if (!a.d.draft || a.d.draft_dtype == TQ_F32) return launch<T, float>(a, sms, s);
    if (a.d.draft_dtype == TQ_F16) return launch<T, __half>(a, sms, s);
    return launch<T, __nv_bfloat16>(a, sms, s);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int sms, cudaStream_t s) {
    if (a.K == 0 && a.d.noise) return launch_draw(a, sms, s);   // (the likeliest tokens of 1000 rows of 131072, bf16: 53 us here, 90 there)
    if (a.d.target_dtype == TQ_F32) return launch_q<float>(a, sms, s);
    if (a.d.target_dtype == TQ_F16) return launch_q<__half>(a, sms, s);
    return launch_q<__nv_bfloat16>(a, sms, s);
}

}  // namespace serve
}  // namespace tq
