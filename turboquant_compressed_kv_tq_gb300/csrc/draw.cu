// The next token of each sequence where nothing was drafted: verification's form for single tokens.
//
// The token with the largest p / noise, p = softmax(x / T), is the one with the largest weight 2^((x - top) log2(e) / T) / noise, whatever the
// sum of weights: one pass over logits and noise finds it, the largest logit and the sum (for the logprob) together. A thread's weights are
// relative to the largest logit that it has seen so far; its best token is kept with its logit and noise, and scored once more
// against the row's largest at the end, so that equals are equal wherever in the row they stand.
//
// A cluster of CTAs has a sequence, as many as fill the SMs once: a cluster's last steps (two barriers, its last threads' loads) are as
// long for a short share of a row as for a long one. Each warp has a ring of bulk copies of its own, as in verify.cu.
//
// Measured: 200 rows of 131,072, f32, a third of them greedy (whose noise is not read: 175 MB): 36 us (4.8 TB/s); 42 with the values loaded to
// registers, 47 in two passes. Three CTAs an SM and two pieces a ring: two and three 41 us, four and one 38.
#include <algorithm>

#include "verify_device.cuh"

namespace tq {
namespace serve {
namespace {

constexpr int kResident = 3;                   // CTAs on an SM
constexpr int kValues = 16;                    // of a thread at a time
constexpr int kPiece = 32 * kValues, kStages = 2;   // values of a warp's piece, and how many pieces are on their way

struct DrawShared {
    uint64_t bars[kWarps][kStages];
    float2 seen[2][kParts];   // (largest, sum) of the cluster's warps, of either round
    Best best[kParts];
};
template <typename T>
constexpr int kStageBytes = kPiece * (sizeof(T) + 4);   // logits, then noise

template <typename T>
__global__ void __launch_bounds__(kThreads, kResident) draw_kernel(const __grid_constant__ VerifyArgs A, int log_ctas) {
    constexpr int kGroup = 16 / sizeof(T);   // values of a thread that lie together
    __shared__ __align__(16) DrawShared S;
    extern __shared__ __align__(128) unsigned char s_ring[];
    const int ctas = 1 << log_ctas, rank = cluster_rank();
    const int b = blockIdx.x >> log_ctas, tid = threadIdx.x, lane = tid % 32, warp = tid / 32, V = A.V;
    const tq_drafts& D = A.d;
    const float asked_T = D.temperatures ? D.temperatures[b] : 1.0f;
    if (tid == 0 && rank == 0 && D.draft_lens && D.draft_lens[b] != 0) atomicOr(A.err, TQ_DEVERR_SEQLEN);   // (of no drafts)
    if (lane < kStages) tc::mbar_init(&S.bars[warp][lane], 1);
    tc::mbar_fence_init();
    __syncwarp();
    cluster_arrive();   // (waited for before the first word to another CTA)
    const T* row = static_cast<const T*>(D.target) + b * D.target_stride_batch;
    const float* noise = D.noise + b * D.noise_stride;   // (without noise all rows are the other kernel's)
    const bool probs = D.target_probs != 0, greedy = !(asked_T > 0.0f);
    const Scale scale(greedy ? 1.0f : fminf(fmaxf(asked_T, 0x1p-120f), 0x1p100f));
    // A CTA's values: whole chunks of 8 through its warps' rings, where logits and noise lie alike, and what lies outside those (the
    // first CTA's) one value at a time; else all so.
    const int head = min(V, static_cast<int>((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(T))), chunks = (V - head) / 8;
    const bool alike = greedy || reinterpret_cast<uintptr_t>(noise + head) % 16 == 0;
    const int per = alike ? ((chunks + ctas - 1) >> log_ctas) * 8 : (V + ctas - 1) >> log_ctas;
    const int main_end = alike ? head + chunks * 8 : V, main_begin = min(main_end, (alike ? head : 0) + rank * per), my_end = min(main_end, main_begin + per);
    unsigned char* const ring = s_ring + warp * kStages * kStageBytes<T>;
    int asked = 0;   // by lane 0: the first value of the next piece
    auto ask = [&](int st) {
        const int at = asked, n = min(kPiece, my_end - at);
        if (n <= 0) return;
        asked = at + kWarps * kPiece;
        uint64_t* bar = &S.bars[warp][st];
        tc::mbar_expect_tx(bar, n * (greedy ? static_cast<int>(sizeof(T)) : static_cast<int>(sizeof(T)) + 4));
        tc::bulk_g2s(ring + st * kStageBytes<T>, row + at, n * static_cast<int>(sizeof(T)), bar);
        if (!greedy) tc::bulk_g2s(ring + st * kStageBytes<T> + kPiece * sizeof(T), noise + at, n * 4, bar);
    };
    int st = 0, phase = 0;

    float top, sum;
    Best best;
#pragma unroll 1
    for (int round = 0;; ++round) {   // in the second, only where there are some, +inf and NaN as they count
        const bool clean = round > 0;
        top = -FLT_MAX, sum = 0.0f;
        best = Best{0.0f, INT_MAX};       // relative to `top`
        float best_x = 0.0f, best_e = 1.0f;
        int piece = -1, piece_step = 1;   // where the largest stood first
        if (alike && lane == 0) {
            asked = main_begin + warp * kPiece;
#pragma unroll 1
            for (int i = 0; i < kStages; ++i) ask((st + i) % kStages);
        }
#pragma unroll 1
        for (int job = alike && rank == 0 ? 0 : 1; job < (alike && rank == 0 ? 3 : 2); ++job) {   // (in the order of their values)
            const bool piped = alike && job == 1;
            const int begin = job == 0 ? 0 : job == 1 ? main_begin : main_end, end = job == 0 ? head : job == 1 ? my_end : V;
            const int step = piped ? 1 : kThreads, far = piped ? 32 * kGroup : kGroup * kThreads;   // between values of a group, and groups
#pragma unroll 1
            for (int i0 = begin + (piped ? warp * kPiece : tid); i0 < end; i0 += piped ? kWarps * kPiece : kValues * kThreads) {
                float2 x[kValues / 2], e[kValues / 2];
                const float none = probs ? 0.0f : -INFINITY;
                const int mine = piped ? i0 + lane * kGroup : i0;   // the thread's first
                if (piped) {
                    if (!tc::mbar_wait(&S.bars[warp][st], phase)) {   // once more, so that no copy is on its way when the kernel ends
                        if (lane == 0) atomicOr(A.err, TQ_DEVERR_TIMEOUT);
                        tc::mbar_wait(&S.bars[warp][st], phase);
                    }
                    const uint4* xs = reinterpret_cast<const uint4*>(ring + st * kStageBytes<T>);
                    const float4* es = reinterpret_cast<const float4*>(ring + st * kStageBytes<T> + kPiece * sizeof(T));
#pragma unroll
                    for (int g = 0; g < kValues / kGroup; ++g) {
                        if (mine + g * far < end) {
                            numbers(xs[g * 32 + lane], x + g * kGroup / 2, T());
                            if (!greedy) {
#pragma unroll
                                for (int i = 0; i < kGroup / 4; ++i) {
                                    const float4 v = es[(g * 32 + lane) * (kGroup / 4) + i];
                                    e[g * kGroup / 2 + 2 * i] = make_float2(v.x, v.y), e[g * kGroup / 2 + 2 * i + 1] = make_float2(v.z, v.w);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < kGroup / 2; ++i) x[g * kGroup / 2 + i] = both(none), e[g * kGroup / 2 + i] = both(1.0f);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) ask(st);
                    if (++st == kStages) st = 0, phase ^= 1;
                } else {
#pragma unroll
                    for (int i = 0; i < kValues; ++i) {
                        float &xi = i % 2 ? x[i / 2].y : x[i / 2].x, &ei = i % 2 ? e[i / 2].y : e[i / 2].x;
                        const int at = i0 + i * kThreads;
                        xi = none, ei = 1.0f;
                        if (at < end) {
                            xi = number(row[at]);
                            if (!greedy) ei = noise[at];
                        }
                    }
                }
                auto index = [&](int i) { return mine + i / kGroup * far + i % kGroup * step; };
                if (clean) {
                    bool odd = false;
#pragma unroll
                    for (int i = 0; i < kValues / 2; ++i) {
                        odd |= !(x[i].x < INFINITY) || !(x[i].y < INFINITY);
                        x[i] = make_float2(logit(x[i].x), logit(x[i].y));
                    }
                    if (odd) atomicOr(A.err, TQ_DEVERR_NONFINITE);
                }
                float t = fmaxf(x[0].x, x[0].y);
#pragma unroll
                for (int i = 1; i < kValues / 2; ++i) t = fmaxf(fmaxf(t, x[i].x), x[i].y);
                if (t > top) {
                    const float f = scale.weight(top - t);
                    sum *= f;
                    best.v = probs ? best.v : best.v * f;
                    top = t;
                    piece = mine, piece_step = step;
                } else if (t == top && piece < 0) {   // (-FLT_MAX)
                    piece = mine, piece_step = step;
                }
                // weights as in Seen::take: relative to m, and a factor `exact` from m to the exact top
                const float m = top * scale.near;
                const bool usual = fabsf(m) < kUsual;
                const float exact = usual && !probs ? fmaf(fmaf(top, scale.near, -m), -kLn2, 1.0f) : 1.0f;
                auto weight = [&](float v) { return usual ? ex2(fmaf(v, scale.near, -m)) : scale.weight(v - top); };
                float2 w[kValues / 2];
                if (probs) {
#pragma unroll
                    for (int i = 0; i < kValues / 2; ++i) w[i] = x[i];
                } else if (usual) {
                    float2 s = both(0.0f);
#pragma unroll
                    for (int i = 0; i < kValues / 2; ++i) {
                        const float2 a = __ffma2_rn(x[i], both(scale.near), both(-m));
                        w[i] = make_float2(ex2(a.x), ex2(a.y));
                        s = __fadd2_rn(s, w[i]);
                    }
                    sum = fmaf(s.x + s.y, exact, sum);
                } else {
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < kValues / 2; ++i) {
                        w[i] = make_float2(scale.weight(x[i].x - top), scale.weight(x[i].y - top));
                        s += w[i].x + w[i].y;
                    }
                    sum += s;
                }
                if (greedy) continue;
#pragma unroll
                for (int i = 0; i < kValues / 2; ++i) w[i] = __fmul2_rn(w[i], make_float2(rcp(fmaxf(e[i].x, 0x1p-100f)), rcp(fmaxf(e[i].y, 0x1p-100f))));
                float here = fmaxf(w[0].x, w[0].y);
#pragma unroll
                for (int i = 1; i < kValues / 2; ++i) here = fmaxf(fmaxf(here, w[i].x), w[i].y);
                const float score = here * exact;
                if (here > 0.0f && score >= best.v * (1.0f - 0x1p-20f)) {
                    int at = 0;
                    float at_x = 0.0f, at_e = 1.0f;
#pragma unroll
                    for (int i = kValues - 1; i >= 0; --i)
                        if ((i % 2 ? w[i / 2].y : w[i / 2].x) == here)
                            at = index(i), at_x = i % 2 ? x[i / 2].y : x[i / 2].x, at_e = i % 2 ? e[i / 2].y : e[i / 2].x;
                    // scores nearer to each other than what a change of `top` rounds: once more, against one top
                    const float was = (probs ? best_x : weight(best_x)) * rcp(fmaxf(best_e, 0x1p-100f));
                    if (best.i == INT_MAX || here > was || (here == was && at < best.i)) {
                        best = Best{score, at};
                        best_x = at_x, best_e = at_e;
                    }
                }
            }
        }
        // ---- the row's largest and its sum, from what all warps of the cluster saw
        float t = warp_max(top), s = sum * scale.weight(top - t);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        if (round == 0) cluster_wait();
        if (lane < ctas) send(remote(&S.seen[round][rank * kWarps + warp], lane), __float_as_uint(t), __float_as_uint(s));
        cluster_arrive();
        cluster_wait();
        const float2 none = make_float2(-FLT_MAX, 0.0f), u = lane < ctas * kWarps ? S.seen[round][lane] : none, v = lane + 32 < ctas * kWarps ? S.seen[round][lane + 32] : none;
        t = warp_max(fmaxf(u.x, v.x));
        s = u.y * scale.weight(u.x - t) + v.y * scale.weight(v.x - t);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        if (!probs && round == 0 && !(s < INFINITY)) continue;   // a NaN, or +inf (inf - inf)
        // ---- the thread's token against that
        if (greedy) {
            best = Best{0.0f, INT_MAX};
            if (top == t && piece >= 0 && (probs ? t > 0.0f : s > 0.0f)) {
#pragma unroll 1
                for (int i = 0; i < kValues; ++i) {
                    const int at = piece + i / kGroup * (piece_step == 1 ? 32 * kGroup : kGroup * kThreads) + i % kGroup * piece_step;
                    // (behind a share's end lies another's, or the row's: what is as large there is no lower)
                    if (at < V && (clean ? logit(number(row[at])) : number(row[at])) == t) {
                        best = Best{1.0f, at};
                        break;
                    }
                }
            }
        } else if (best.i != INT_MAX) {
            const float m = t * scale.near;
            best.v = (probs ? best_x : fabsf(m) < kUsual ? ex2(fmaf(best_x, scale.near, -m)) : scale.weight(best_x - t)) * rcp(fmaxf(best_e, 0x1p-100f));
            if (!(best.v > 0.0f)) best = Best{0.0f, INT_MAX};   // (likely only beside what this thread saw)
        }
        top = t, sum = s;
        break;
    }
    best.join();
    if (lane == 0) send(remote(&S.best[rank * kWarps + warp], 0), __float_as_uint(best.v), static_cast<uint32_t>(best.i));
    cluster_arrive();
    cluster_wait();
    if (rank != 0 || warp != 0) return;
    best = Best{0.0f, INT_MAX};
    if (lane < ctas * kWarps) best = S.best[lane];
    if (lane + 32 < ctas * kWarps) best.meet(S.best[lane + 32].v, S.best[lane + 32].i);
    best.join();
    if (lane != 0) return;
    const int next = best.i < V ? best.i : -1;
    if (next < 0) atomicOr(A.err, TQ_DEVERR_NONFINITE);
    A.accepted[b] = 0;
    A.tokens[b] = next;
    if (A.logprobs) {
        const float x = next < 0 ? 0.0f : number(row[next]);
        A.logprobs[b] = next < 0 ? 0.0f : probs ? logf(x) : scale.log(logit(x) - top) - logf(sum);
    }
    if (A.keep) A.keep[b] = D.seq_lens[b] + 1;
}

template <typename T>
cudaError_t launch(const VerifyArgs& a, int sms, cudaStream_t s) {
    int log_ctas = 0;
    while ((1 << log_ctas) < kMostCtas && (kWarps * kPiece << log_ctas) < a.V && (static_cast<int64_t>(a.batch) << (log_ctas + 1)) <= kResident * sms) ++log_ctas;
    constexpr int smem = kWarps * kStages * kStageBytes<T>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = kv8::allow_smem(draw_kernel<T>, smem, allowed);
    return e != cudaSuccess ? e : launch_cluster(draw_kernel<T>, a, log_ctas, smem, s);
}

}  // namespace

cudaError_t launch_draw(const VerifyArgs& a, int sms, cudaStream_t s) {
    if (a.d.target_dtype == TQ_F32) return launch<float>(a, sms, s);
    if (a.d.target_dtype == TQ_F16) return launch<__half>(a, sms, s);
    return launch<__nv_bfloat16>(a, sms, s);
}

}  // namespace serve
}  // namespace tq
