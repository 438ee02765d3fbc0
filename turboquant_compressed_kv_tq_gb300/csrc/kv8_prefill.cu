// Attention over the 8-bit cache for many query rows (chunks of a prompt), on
// the 5th-generation tensor cores.
//
// A CTA owns kHalves x 128 query rows of one KV head (row r = l G + g: query l,
// head g of the group, so that neighbouring rows see nearly the same keys) and
// walks tiles of kT tokens (flash attention: one pass, running reference M and
// sum l per row). Sixteen warps:
//   convert  4 for keys, 3 for values: codes from global memory (cp.async into a place of each
//            lane's own, a tile ahead) to fp16, to the operands in shared memory: both as
//            [8 tokens x 8 coordinates] core matrices, which are K-major for S = Q K^T and
//            MN-major for O += P V, so nothing is transposed
//   mma      1 thread: S = Q K^T (operands in shared memory, S in TMEM), O += P V (P in TMEM)
//   softmax  4 a half, one row a thread: S from TMEM, masks, p = 2^(u - M) to TMEM as fp16,
//            64 columns at a time so that P V begins on the first, the row's sum; O is rescaled
//            in TMEM only when a score passes the reference by 8 (log2 units)
// With two halves one's softmax runs while the tensor cores work for the other;
// with one (head_dim 256, whose O fills half of TMEM) the scores of the next tile
// are computed ahead into a second buffer.
//
// Block scales are powers of two. Within a tile the codes are brought to the
// tile's largest scale in fp16; that one scale is a factor of the row's scores, and
// for values moves the softmax's reference: u = log2(e) score + log2(scale),
// p = 2^(u - M), l += p / scale. Where the tile's scales lie too far apart for that
// (keys: 2^15 for e4m3, 2^24 for integers, to be exact; values: 2^6; blocks of zeros,
// other documents), the codes stay as they are and the softmax warps take each group of 8 tokens at
// its own scales: the keys' a factor of its scores, the values' a part of its u, and
// l from u without it (2^63 a key of zeros, next to values whose M is 2^63).
//
// Bound: next to the tensor cores' 4 D flops per row and key, shared memory (both
// operands of S and one of P V come from it, and the converters pass through it)
// and the softmax's latency. Measured: 4096 queries x 32 heads over 12,288 tokens,
// 8 KV heads of 128: 677 us, 1.01 PFLOP/s, 54 % of what a plain bf16 product reaches.
#include <climits>
#include <type_traits>

#include "kv8_device.cuh"
#include "tc_ptx.cuh"
#include "tc_tmem_wide.cuh"

namespace tq {
namespace kv8 {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -FLT_MAX;   // below every score
constexpr float kGap = 8.0f;
constexpr int kKWarp = 8, kVWarp = 12, kMmaWarp = 15, kThreads = 32 * (kMmaWarp + 1);

// kFine: the queries in two fp16 parts (head_dim 64).
template <int D, bool kFine>
struct Shape {
    static constexpr int kHalves = D == 256 ? 1 : 2;
    static constexpr int kRows = 128 * kHalves;
    static constexpr int kT = D == 256 ? 64 : 128;         // tokens of a tile
    static constexpr int kOperand = kT * D * 2;            // bytes of a tile's keys or values as fp16
    static constexpr int kVOff = 0, kKOff = 2 * kOperand, kQOff = 4 * kOperand;
    static constexpr int kQ = kRows * D * 2;               // bytes of the queries (of each part)
    static constexpr int kRawOff = kQOff + kQ * (kFine ? 2 : 1), kRaw = kT * D;   // a tile's codes, keys then values
    static constexpr int kSmem = kRawOff + 2 * kRaw;
    // TMEM columns: O, S and P of half (or tile parity) x
    static constexpr int kO = 0, kS = kHalves * D, kSStep = kT;
    // P over the scores it comes from where TMEM is full (D 128), else apart
    static constexpr bool kPOver = D == 128;
    static constexpr int kP = kPOver ? kS : kS + 2 * kSStep, kPStep = kPOver ? kSStep : kT / 2;
    static_assert((kPOver ? kS + 2 * kSStep : kP + 2 * kPStep) <= 512, "TMEM columns");
    static constexpr int kGroups = kT / 8;                 // groups of 8 tokens
};

// Wait for the phase with this parity; false after about a second.
__device__ __forceinline__ bool arrived(uint64_t* bar, unsigned parity) {
    const uint32_t a = tc::smem_addr(bar);
    for (unsigned it = 0; it < (1u << 18); ++it) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(a), "r"(parity)
            : "memory");
        if (done) return true;
    }
    return false;
}

// The same by a whole warp, with one answer for all its lanes: what follows, waited for or given up, is warp-wide
// (tensor memory, shuffles), and must not find a part of the warp gone.
__device__ __forceinline__ bool arrived_warp(uint64_t* bar, unsigned parity) { return __all_sync(0xffffffffu, arrived(bar, parity)); }

// Byte offset of (row, d) in an operand of core matrices: 8 rows x 16 bytes.
template <int D>
__device__ __forceinline__ int core(int row, int d) {
    return ((row >> 3) * (D / 8) + (d >> 3)) * 128 + (row & 7) * 16;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return r;
}

// 16 bytes to shared memory, not by way of the L1 cache: next to 200 KB of shared
// memory it has too few lines for what is on its way.
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int K>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(K) : "memory"); }

struct Tiles {
    int n1, first, n2;
    __device__ __forceinline__ int at(int i) const { return i < n1 ? i : first + (i - n1); }
    __device__ __forceinline__ int count() const { return n1 + n2; }
};

// What the converters say about a tile.
constexpr int kWide = 1 << 12;
struct TileInfo {
    int kref, vref;    // its scales' exponents; kref + kWide where they are too far apart for one scale in fp16, or too small: see s_below
    unsigned gone;     // groups of 8 tokens that belong to no block
};

// A row's softmax over a wide tile (or one of large scores), in 8 columns at a time: a group's scores have its own key scale, its u its own value
// scale. (Rare, and a function of its own: the usual tile's code and registers stay as they are without it; in the
// usual tile's code: 695 us for 669. With every tile wide the prompt above takes 1637.)
struct WideTile {
    uint32_t t_s, t_p, t_o;    // S, P and O of this thread's rows
    bool some;                 // O holds something
    const uint16_t* below;     // s_below, or null: all of them at the tile's scales
    int kref, vref;            // the tile's largest exponents
    float fac, cap, slope;     // of the scores, but for the key scale
    Sight sight;
    int t0;
    unsigned gone;
    float m, l;
};

template <int D, int kT, bool MOD>
__device__ __noinline__ float2 wide_tile(const WideTile w) {
    const float cap2 = w.cap * kLog2e, cap_in = w.cap > 0.0f ? 1.0f / w.cap : 0.0f;
    float m = w.m, l = w.l, top = -INFINITY;
#pragma unroll 1
    for (int g = 0; g < kT / 8; ++g) {   // u, masked, back to where the scores were
        const int below = w.below ? w.below[g] : 0;
        const float kg = w.fac * exp2i(max(w.kref - (below & 0xFF), -126)), lv = static_cast<float>(w.vref - (below >> 8));
        float x[8];
        tc::tmem_ld8(w.t_s + 8 * g, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int t = w.t0 + 8 * g + e;
            x[e] *= kg;
            x[e] = MOD && w.cap > 0.0f ? capped_wide(x[e] * cap_in, cap2) : x[e] * kLog2e;
            if (MOD) x[e] = fmaf(-w.slope, fabsf(static_cast<float>(t - w.sight.p)), x[e]);
            x[e] = w.sight.sees(t) && !((w.gone >> g) & 1u) ? x[e] + lv : -INFINITY;
            top = fmaxf(top, x[e]);
        }
        tc::tmem_st8(w.t_s + 8 * g, x);
    }
    if (__any_sync(0xffffffffu, top > m + kGap)) {
        const float x = fmaxf(top, m);
        const float half = ex2(0.5f * (m - x)), alpha = half * half;   // (l may be 2^63 a key, of zeros, or 2^-63)
        m = x;
        l = l * half * half;
        if (w.some) {
#pragma unroll 1
            for (int c = 0; c < D / 8; ++c) {
                float v[8];
                tc::tmem_ld8(w.t_o + 8 * c, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= alpha;
                tc::tmem_st8(w.t_o + 8 * c, v);
            }
        }
    }
#pragma unroll 1
    for (int n = 0; n < kT / 32; ++n) {   // p, 32 columns at a time (over scores that were read, where P lies over S)
        uint32_t pr[16];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float lv = static_cast<float>(w.vref - (w.below ? w.below[4 * n + g] >> 8 : 0));
            float x[8];
            tc::tmem_ld8(w.t_s + 32 * n + 8 * g, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] -= m;
                l += ex2(x[e] - lv);
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) pr[4 * g + e / 2] = pack_out<__half>(ex2(x[e]), ex2(x[e + 1]));
        }
        tc::tmem_st16u(w.t_p + 16 * n, pr);
    }
    return make_float2(m, l);
}

template <typename T, int D, bool I8, bool MOD, bool kFine>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ AttendArgs A) {
    using S = Shape<D, kFine>;
    constexpr int kT = S::kT, kH = S::kHalves;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ uint64_t s_turns[D / 2];
    __shared__ __align__(8) uint64_t s_bar[18];
    __shared__ float s_fac[S::kRows];
    __shared__ TileInfo s_info[4];
    __shared__ uint16_t s_below[4][S::kGroups];   // of a wide tile's groups: how far their exponents are below kref and (high byte) vref
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
    uint64_t *k_full = s_bar, *k_free = s_bar + 2, *v_full = s_bar + 4, *v_free = s_bar + 6;
    uint64_t *s_ready = s_bar + 8, *p_ready = s_bar + 10, *o_done = s_bar + 12, *drained = s_bar + 14, *p_second = s_bar + 15, *q_ready = s_bar + 17;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Pool& P = A.pool;
    // the longest rows first: the last wave then holds short ones
    const int grp = A.groups - 1 - blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int rows = min(A.G * A.L - grp * S::kRows, S::kRows);

    int N = A.seq[b], nq = A.qlens ? A.qlens[b] : A.L;
    const bool bad_n = N < 0 || N > A.max_seq || (N + P.BT - 1) >> P.bt_shift > P.max_blocks, bad_q = nq < 0 || nq > A.L;
    if (bad_n) N = 0;
    if (bad_q) nq = nq < 0 ? 0 : A.L;
    if ((bad_n || bad_q) && tid == 0 && blockIdx.x == 0 && h == 0) atomicOr(A.err, TQ_DEVERR_SEQLEN);
    const int l_first = grp * S::kRows / A.G, l_last = min((grp * S::kRows + rows - 1) / A.G, nq - 1);
    if (l_first >= nq) return;   // only rows behind the sequence's queries

    const int pre = A.prefix ? min(max(A.prefix[b], 0), N) : 0;
    auto sight_of = [&](int l) {
        Sight s;
        s.p = N - nq + l;
        s.lo = 0;
        if (A.window > 0) s.lo = max(s.lo, s.p - A.window + 1);
        if (A.docs) s.lo = max(s.lo, A.docs[static_cast<int64_t>(b) * A.L + l]);
        s.prefix = pre;
        return s;
    };
    // the smallest first key of any row (each warp for itself)
    int lo_min = INT_MAX;
    if (A.docs) {
        for (int l = l_first + lane; l <= l_last; l += 32) lo_min = min(lo_min, sight_of(l).lo);
        lo_min = __reduce_min_sync(0xffffffffu, lo_min);
    } else {
        lo_min = sight_of(l_first).lo;
    }
    const int p_max = N - nq + l_last;
    Tiles tiles;
    tiles.n1 = (pre + kT - 1) / kT;
    tiles.first = max(tiles.n1, lo_min / kT);
    tiles.n2 = p_max < 0 || lo_min > p_max ? 0 : max(0, p_max / kT + 1 - tiles.first);
    const int n_tiles = tiles.count();

    const bool two = kH == 2 && rows > 128;   // the second half has rows

    // ---------------- set up: TMEM, barriers, the queries (rotated, scaled by a power of two, fp16)
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&s_tmem, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&k_full[s], kVWarp - kKWarp);
            tc::mbar_init(&v_full[s], kMmaWarp - kVWarp);
            tc::mbar_init(&k_free[s], 1);
            tc::mbar_init(&v_free[s], 1);
            tc::mbar_init(&s_ready[s], 1);
            tc::mbar_init(&p_ready[s], 4);
            tc::mbar_init(&p_second[s], 4);
            tc::mbar_init(&o_done[s], 1);
        }
        tc::mbar_init(drained, 1);
        tc::mbar_init(q_ready, 8);
        tc::mbar_fence_init();
        s_fail = 0;
    }
    if (A.rope.rot > 0)
        for (int i = tid; i < A.rope.rot / 2; i += kThreads) s_turns[i] = turns_of(A.rope.inv_freq[i]);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem;
    if (warp < 8) {
        // ================================================= the queries: rotated, scaled by a power of two, fp16
        if (n_tiles > 0) {
            // The heads of a query turn by the same angles: cos and sin of each (query, pair) once, in the operands'
            // second stages (values, then keys), which the converters enter when the queries are done. With one head
            // to a group (or so many pairs that they do not fit) each row computes its own.
            constexpr int kHalf = S::kOperand / 8;
            const int pairs = A.rope.rot / 2, angles = (l_last - l_first + 1) * pairs;
            const bool shared = angles > 0 && angles <= 2 * kHalf && A.G > 1;
            auto position = [&](int l) { return A.rope.positions ? A.rope.positions[static_cast<int64_t>(b) * A.L + l] : N - nq + l; };
            auto place = [&](int e) {
                return reinterpret_cast<float2*>(smem + (e < kHalf ? S::kVOff : S::kKOff - S::kOperand) + S::kOperand) + e;
            };
            if (shared) {
                for (int e = tid; e < angles; e += 256) *place(e) = angle_at(A.rope, s_turns[e % pairs], position(l_first + e / pairs));
                asm volatile("bar.sync 2, 256;\n" ::: "memory");
            }
            constexpr int J = D / 16;   // chunk pairs of a row: J consecutive lanes
            const float sign = A.scale < 0.0f ? -1.0f : 1.0f;
            for (int it = tid; it < S::kRows * J; it += 256) {
                const int r = it / J, j = it % J;
                const int rr = grp * S::kRows + r, l = rr / A.G;
                float xa[8] = {}, xb[8] = {};
                int a0, b0;
                chunk_pair(j, A.rope.rot, A.rope.inter, a0, b0);
                if (r < rows && l < nq) {
                    const T* q = static_cast<const T*>(A.q.data) + b * A.q.sb + static_cast<int64_t>(h * A.G + rr % A.G) * A.q.sh + l * A.q.st;
                    load8(q + a0, xa);
                    load8(q + b0, xb);
                    if (shared) {
                        const int e = (l - l_first) * pairs + 8 * j;
                        if (16 * j < A.rope.rot) rotate_by(xa, xb, A.rope.inter, [&](int i) { return *place(e + i); });
                    } else if (A.rope.rot > 0) {
                        rotate_pair(xa, xb, j, A.rope, s_turns, position(l));
                    }
                }
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(fabsf(xa[i]), fabsf(xb[i])));
#pragma unroll
                for (int o = J / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -126), 126);
                const float f = sign * exp2i(-e);
                auto put = [&](const float (&x)[8], int d) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __half2 w = __floats2half2_rn(x[2 * i] * f, x[2 * i + 1] * f);
                        const float2 back = __half22float2(w);
                        hi[i] = *reinterpret_cast<const uint32_t*>(&w);
                        lo[i] = pack_out<__half>(x[2 * i] * f - back.x, x[2 * i + 1] * f - back.y);
                    }
                    unsigned char* at = smem + S::kQOff + core<D>(r, d);
                    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if constexpr (kFine) *reinterpret_cast<uint4*>(at + S::kQ) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                };
                put(xa, a0);
                put(xb, b0);
                if (j == 0) s_fac[r] = fabsf(A.scale) * exp2i(e);
            }
            tc::fence_proxy_async_smem();
            asm volatile("bar.sync 2, 256;\n" ::: "memory");   // s_fac, for the softmax
            if (lane == 0) tc::mbar_arrive(q_ready);
        }
        // ================================================= softmax
        const int half = warp >> 2;
        const int row = 128 * half + 32 * (warp & 3) + lane;
        const bool mine = kH == 1 ? half == 0 : (half == 0 || two);
        const uint32_t t_row = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t t_o = t_row + S::kO + (kH == 2 ? half * D : 0);
        float m = kNone, l_sum = 0.0f;
        bool ok = true;
        const int rr = grp * S::kRows + min(row, rows - 1);
        const int l_row = min(rr / A.G, nq - 1);
        if (mine && n_tiles > 0) {
            const Sight sight = sight_of(l_row);
            const int p_min = __reduce_min_sync(0xffffffffu, sight.p), lo_max = __reduce_max_sync(0xffffffffu, sight.lo);
            const float fac = s_fac[min(row, S::kRows - 1)];
            const float cap2 = A.cap * kLog2e, cap_in = A.cap > 0.0f ? 1.0f / A.cap : 0.0f;
            const float slope = MOD && A.slopes ? A.slopes[h * A.G + rr % A.G] * kLog2e : 0.0f;
            // u less its reference, in one rounding, leaves the row's largest within what the reference was rounded by: up to 1
            // for scores below 2^24 (kref at most k_most by what queries in [1, 2) and the largest codes allow, and the bias).
            // Larger ones go the way of wide tiles, where u is rounded first and the largest gets exactly 2^0
            constexpr int kCodes = (I8 ? 8 : 10) + (D == 64 ? 6 : D == 128 ? 7 : 8);   // log2 (rounded down) of the largest code times log2(e), 2, D
            const int k_most = __reduce_min_sync(0xffffffffu, fabsf(slope) * static_cast<float>(N) > 0x1p23f
                                                                  ? -256 : 23 - kCodes - (static_cast<int>(__float_as_uint(fac) >> 23) - 126));
            for (int i = 0;;) {
                for (; i < n_tiles; ++i) {
                    const int t0 = tiles.at(i) * kT;
                    const int sb = kH == 2 ? half : i & 1;                    // buffer of S and P
                    ok = arrived_warp(&s_ready[sb], kH == 2 ? i & 1 : (i >> 1) & 1);
                    if (!ok) break;
                    tc::tc_fence_after();
                    const TileInfo info = s_info[i & 3];
                    if (info.kref > k_most) break;
                    const float kf = fac * exp2i(info.kref), lv = static_cast<float>(info.vref);
                    const float f = MOD ? 1.0f : fmaxf(kf * kLog2e, FLT_MIN);
                    const bool open = info.gone == 0 && ((t0 + kT - 1 <= p_min && t0 >= lo_max) || t0 + kT <= pre);
                    // 64 columns of the row's scores, k a multiple of 64: cap and bias applied, unseen ones -inf
                    auto finish = [&](uint32_t (&sr)[64], int k) {
                        if constexpr (MOD) {
                            if (A.cap > 0.0f) {
                                const float k2 = kf * cap_in;
                                if (A.cap <= kUsualCap) {
#pragma unroll
                                    for (int e = 0; e < 64; ++e) sr[e] = __float_as_uint(capped(__uint_as_float(sr[e]) * k2, cap2));
                                } else {
#pragma unroll
                                    for (int e = 0; e < 64; ++e) sr[e] = __float_as_uint(capped_wide(__uint_as_float(sr[e]) * k2, cap2));
                                }
                            } else {
                                const float k2 = kf * kLog2e;
#pragma unroll
                                for (int e = 0; e < 64; ++e) sr[e] = __float_as_uint(__uint_as_float(sr[e]) * k2);
                            }
                            if (A.slopes) {
                                const float from = static_cast<float>(t0 + k - sight.p);
#pragma unroll
                                for (int e = 0; e < 64; ++e)
                                    sr[e] = __float_as_uint(fmaf(-slope, fabsf(from + static_cast<float>(e)), __uint_as_float(sr[e])));
                            }
                        }
                        if (!open) {
                            // the seen columns as bits, 32 at a time
                            auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
#pragma unroll
                            for (int n = 0; n < 64; n += 32) {
                                const int at = t0 + k + n;
                                uint32_t see = (below(sight.p - at + 1) & ~below(sight.lo - at)) | below(sight.prefix - at);
                                if (info.gone) {
#pragma unroll
                                    for (int g = 0; g < 4; ++g)
                                        if ((info.gone >> ((k + n) / 8 + g)) & 1u) see &= ~(0xFFu << (8 * g));
                                }
#pragma unroll
                                for (int e = 0; e < 32; ++e) sr[n + e] = (see >> e) & 1u ? sr[n + e] : 0xFF800000u;
                            }
                        }
                    };
                    auto largest = [&](const uint32_t (&sr)[64]) {
                        float x[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            x[q] = max3(sr[16 * q], sr[16 * q + 1], sr[16 * q + 2]);
#pragma unroll
                            for (int e = 3; e < 15; e += 2) x[q] = max3(__float_as_uint(x[q]), sr[16 * q + e], sr[16 * q + e + 1]);
                        }
                        x[0] = max3(__float_as_uint(x[0]), sr[15], sr[31]);
                        x[1] = max3(__float_as_uint(x[1]), sr[47], sr[63]);
                        return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                    };
                    // a row at once would be 128 registers: the upper 64 scores are looked at
                    // for the maximum, and read again once the lower are done
                    const uint32_t t_s = t_row + S::kS + sb * S::kSStep;
                    uint32_t sr[64];
                    float top = -INFINITY;
#pragma unroll 1   // (unrolled, the two halves' registers would live side by side)
                    for (int k = kT - 64; k >= 0; k -= 64) {
                        tc::tmem_ld(t_s + k, sr);
                        finish(sr, k);
                        if (k > 0 && (MOD || !open)) tc::tmem_st(t_s + k, sr);
                        top = fmaxf(top, largest(sr));
                    }
                    top = fmaf(top, f, lv);
                    const bool pass = top > m + kGap;
                    if (kH == 1 && i > 0) {   // every phase in its turn: a wait by parity tells neighbouring phases apart, no others
                        ok = arrived_warp(&o_done[0], (i - 1) & 1);
                        if (!ok) break;
                        tc::tc_fence_after();
                    }
                    if (__any_sync(0xffffffffu, pass)) {
                        const float x = fmaxf(top, m);
                        const float half = ex2(0.5f * (m - x)), alpha = half * half;
                        m = x;
                        l_sum = l_sum * half * half;
                        if (i > 0) {
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                float v[16];
                                tc::tmem_ld16(t_o + 16 * c, v);
#pragma unroll
                                for (int e = 0; e < 16; ++e) v[e] *= alpha;
                                tc::tmem_st16(t_o + 16 * c, v);
                            }
                        }
                    }
                    const uint64_t f2 = pack2(f, f), o2 = pack2(lv - m, lv - m);
                    uint64_t sum0 = 0, sum1 = 0;
#pragma unroll 1
                    for (int k = 0; k < kT / 64; ++k) {
                        if (k == 1) tc::tmem_ld(t_s + 64, sr);
#pragma unroll
                        for (int n = 0; n < 64; n += 32) {
                            uint32_t pr[16];
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                float a, c, d, g;
                                unpack2(fma2(pack2(__uint_as_float(sr[n + e]), __uint_as_float(sr[n + e + 1])), f2, o2), a, c);
                                unpack2(fma2(pack2(__uint_as_float(sr[n + e + 2]), __uint_as_float(sr[n + e + 3])), f2, o2), d, g);
                                a = ex2(a), c = ex2(c), d = ex2(d), g = ex2(g);
                                sum0 = add2(sum0, pack2(a, c));
                                sum1 = add2(sum1, pack2(d, g));
                                pr[e / 2] = pack_out<__half>(a, c);
                                pr[e / 2 + 1] = pack_out<__half>(d, g);
                            }
                            tc::tmem_st16u(t_row + S::kP + sb * S::kPStep + (64 * k + n) / 2, pr);
                        }
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(k == 0 ? &p_ready[sb] : &p_second[sb]);
                    }
                    float a, c, d, g;
                    unpack2(sum0, a, c);
                    unpack2(sum1, d, g);
                    l_sum = fmaf((a + c) + (d + g), exp2i(-info.vref), l_sum);
                }
                if (!ok || i == n_tiles) break;
                // a wide one, or of large scores, which are there
                const int t0 = tiles.at(i) * kT, sb = kH == 2 ? half : i & 1;
                const TileInfo info = s_info[i & 3];
                if (kH == 1 && i > 0) {
                    ok = arrived_warp(&o_done[0], (i - 1) & 1);
                    if (!ok) break;
                    tc::tc_fence_after();
                }
                const float2 ml = wide_tile<D, kT, MOD>(WideTile{
                    t_row + S::kS + sb * S::kSStep, t_row + S::kP + sb * S::kPStep, t_o, i > 0, info.kref >= kWide / 2 ? s_below[i & 3] : nullptr, info.kref >= kWide / 2 ? info.kref - kWide : info.kref,
                    info.vref, fac, A.cap, slope, sight, t0, info.gone, m, l_sum});
                m = ml.x;
                l_sum = ml.y;
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&p_ready[sb]);
                    if (kT == 128) tc::mbar_arrive(&p_second[sb]);
                }
                ++i;
            }
            if (ok) ok = arrived_warp(&o_done[kH == 2 ? half : 0], kH == 2 ? 0 : (n_tiles - 1) & 1);
            if (!ok) {
                s_fail = 1;
                atomicOr(A.err, TQ_DEVERR_TIMEOUT);
            }
            tc::tc_fence_after();
        }
        // ---------------- the rows out, once every copy of s_fail is in
        asm volatile("bar.sync 1, 256;\n" ::: "memory");
        const bool failed = *const_cast<volatile int*>(&s_fail) != 0;
        if (mine) {
            // by way of the rows' own place among the queries (nothing reads it any more), so that a row's bytes
            // are stored together; 16-byte chunks trade places by their row, free of bank conflicts
            const bool some = !failed && l_sum != 0.0f;   // (a NaN among the scores makes the row NaN)
            const float inv = some ? 1.0f / l_sum : 0.0f;
            constexpr int kChunks = D / 8;
            unsigned char* stage = smem + S::kQOff + (128 * half + 32 * (warp & 3)) * D * 2;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float v[32];
                if (n_tiles > 0) tc::tmem_ld32(t_o + 32 * c, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (some) {
                        w.x = pack_out<T>(v[8 * e] * inv, v[8 * e + 1] * inv), w.y = pack_out<T>(v[8 * e + 2] * inv, v[8 * e + 3] * inv);
                        w.z = pack_out<T>(v[8 * e + 4] * inv, v[8 * e + 5] * inv), w.w = pack_out<T>(v[8 * e + 6] * inv, v[8 * e + 7] * inv);
                    }
                    *reinterpret_cast<uint4*>(stage + lane * D * 2 + (((4 * c + e) ^ (lane & 7)) * 16)) = w;
                }
            }
            __syncwarp();
#pragma unroll 4
            for (int k = lane; k < 32 * kChunks; k += 32) {
                const int r = k / kChunks, c = k % kChunks;
                const int at = 128 * half + 32 * (warp & 3) + r, ro = grp * S::kRows + at, l = ro / A.G;
                if (at < rows && l < nq) {
                    T* dst = static_cast<T*>(A.out.data) + b * A.out.sb + static_cast<int64_t>(h * A.G + ro % A.G) * A.out.sh + l * A.out.st;
                    *reinterpret_cast<uint4*>(dst + 8 * c) = *reinterpret_cast<const uint4*>(stage + r * D * 2 + ((c ^ (r & 7)) * 16));
                }
            }
        }
    } else if (warp < kMmaWarp) {
        // ================================================= convert
        const bool is_v = warp >= kVWarp;
        const int w = warp - (is_v ? kVWarp : kKWarp), nw = is_v ? kMmaWarp - kVWarp : kVWarp - kKWarp;
        uint64_t *full = is_v ? v_full : k_full, *free = is_v ? v_free : k_free;
        const uint8_t* codes = is_v ? P.vc : P.kc;
        unsigned char* operand = smem + (is_v ? S::kVOff : S::kKOff);
        constexpr int CQ = D / 64;               // quarters of 64 coordinates: a unit is a lane's 16 bytes of one
        constexpr int TG = (S::kGroups + 2) / 3;   // token groups of a warp, at most: w, w + nw, ..
        const int64_t unit_bytes = static_cast<int64_t>(P.BT) * D;
        const int tok = lane & 7, ch = lane >> 3;
        // a batch of kPer tiles: lane kGroups j + g holds the block and scale bytes of tile j's group g. Looked up in
        // two steps, each a batch before what needs it: the block table's entry, then the scales
        constexpr int kPer = 32 / S::kGroups;
        constexpr int kDeep = -24;               // value exponents below it: p may be too small for fp32 where its share of l is not
        constexpr int kExact = I8 ? 24 : 15;     // keys: 2^-kExact of the smallest code (1; 2^-9) is fp16's smallest
        // values: a token's weight goes by the tile's largest scale, which may be that of a block its row does not see, and
        // takes as much from the fp16 range that other tiles' weights have below it: 2^6 of 2^14
        constexpr int kClose = 6;
        const int my_tile = lane / S::kGroups, my_group = lane % S::kGroups;
        struct Found {
            int id, kx, vx;
        };
        auto seen = [&](int i) {
            if (i >= n_tiles) return false;
            const int t = tiles.at(i) * kT + 8 * my_group, first = t & ~(P.BT - 1);
            return t < N && (t <= p_max || t < pre) && (first + P.BT > lo_min || first < pre);
        };
        auto entry = [&](int batch) {
            const int i = kPer * batch + my_tile;
            const int lb = seen(i) ? (tiles.at(i) * kT + 8 * my_group) >> P.bt_shift : 0;
            const int64_t at = b * static_cast<int64_t>(P.max_blocks) + lb;
            return P.table ? P.table[at] : static_cast<int>(at);
        };
        auto look_up = [&](int batch, int e) {
            Found f{-1, 0, 0};
            if (seen(kPer * batch + my_tile)) {
                if (e >= 0 && e < P.num_blocks) {
                    f.id = e;
                    f.kx = P.kx[static_cast<int64_t>(e) * P.H + h];
                    f.vx = P.vx[static_cast<int64_t>(e) * P.H + h];
                } else {
                    atomicOr(A.err, TQ_DEVERR_BLOCK);
                }
            }
            return f;
        };
        // a unit: bytes 64 c + 16 ch of token tok of a group (of the block's own memory behind the sequence's end, and of
        // block 0 where there is no block: zeroed below)
        unsigned char* raw = smem + S::kRawOff + (is_v ? S::kRaw : 0) + 16 * lane;   // this lane's units, 512 bytes apart
        auto load = [&](int i, int id) {
            const int t0 = tiles.at(i) * kT, from = i % kPer * S::kGroups;
            const uint32_t dst = tc::smem_addr(raw);
#pragma unroll
            for (int q = 0; q < TG; ++q) {
                const int g = w + nw * q;
                if (g >= S::kGroups) break;
                const int gid = max(__shfl_sync(0xffffffffu, id, from + g), 0);
                const uint8_t* p = codes + (static_cast<int64_t>(gid) * P.H + h) * unit_bytes + ((t0 + 8 * g + tok) & (P.BT - 1)) * D + 16 * ch;
#pragma unroll
                for (int c = 0; c < CQ; ++c) copy_async(dst + (g * CQ + c) * 512, p + 64 * c);
            }
            copies_close();
        };
        // the codes times 2^-below (their group's exponent under the tile's), as fp16 (`left`: tokens that the sequence
        // still has from the tile's first on; `id`: the groups' blocks)
        auto convert_as = [&](auto plain, int below, int id, int from, int left, unsigned char* dst) {
            constexpr bool kPlain = decltype(plain)::value;   // every token there, at the tile's scale
#pragma unroll
            for (int q = 0; q < TG; ++q) {
                const int g = w + nw * q;
                if (g >= S::kGroups) break;
                bool here = true;
                __half2 mul2{};
                if constexpr (!kPlain) {
                    here = __shfl_sync(0xffffffffu, id, from + g) >= 0 && 8 * g + tok < left;
                    const __half mul = __float2half_rn(exp2i(-__shfl_sync(0xffffffffu, below, from + g)));
                    mul2 = __half2(mul, mul);
                }
#pragma unroll
                for (int c = 0; c < CQ; ++c) {
                    uint4 x = *reinterpret_cast<const uint4*>(raw + (g * CQ + c) * 512);
                    if (!kPlain && !here) x = make_uint4(0, 0, 0, 0);
                    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        codes_f16<I8>(in[e], y[2 * e], y[2 * e + 1]);
                        if constexpr (!kPlain) {
                            const __half2 a = __hmul2(*reinterpret_cast<__half2*>(&y[2 * e]), mul2), d = __hmul2(*reinterpret_cast<__half2*>(&y[2 * e + 1]), mul2);
                            y[2 * e] = *reinterpret_cast<const uint32_t*>(&a);
                            y[2 * e + 1] = *reinterpret_cast<const uint32_t*>(&d);
                        }
                    }
                    unsigned char* o = dst + core<D>(8 * g + tok, 64 * c + 16 * ch);
                    *reinterpret_cast<uint4*>(o) = make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4*>(o + 128) = make_uint4(y[4], y[5], y[6], y[7]);
                }
            }
        };
        // (a tile all there at one scale, the usual one, needs no multiplication: the prompt above, unrotated: 666 us, and 722
        // with scales 2^4 apart in turn)
        auto convert = [&](int below, int id, int from, int left, unsigned char* dst) {
            const bool plain = left >= kT && __all_sync(0xffffffffu, lane - from < 0 || lane - from >= S::kGroups || (id >= 0 && below == 0));
            if (plain) convert_as(std::true_type{}, below, id, from, left, dst);
            else convert_as(std::false_type{}, below, id, from, left, dst);
        };
        bool ok = true;
        if (n_tiles > 0) {
            const int e0 = entry(0), e1 = entry(1);
            int e_next = entry(2);
            Found now = look_up(0, e0), next = look_up(1, e1);
            load(0, now.id);
            for (int i = 0; i < n_tiles; ++i) {
                const int st = i & 1, t0 = tiles.at(i) * kT, from = i % kPer * S::kGroups;
                const bool mine = lane >= from && lane < from + S::kGroups;
                const bool there = mine && now.id >= 0;
                const int kx = now.kx - 127, vx = now.vx - 127;
                const int kref = __reduce_max_sync(0xffffffffu, there ? kx : -64), vref = __reduce_max_sync(0xffffffffu, there ? vx : -64);
                const int k_below = there ? kref - kx : 0, v_below = there ? vref - vx : 0;
                const bool k_wide = __any_sync(0xffffffffu, k_below > kExact), v_wide = __any_sync(0xffffffffu, v_below > kClose || (there && vx < kDeep));
                // groups of no block among those that have tokens
                const unsigned gone = __ballot_sync(0xffffffffu, mine && now.id < 0 && t0 + 8 * my_group < N) >> from;
                copies_wait<0>();
                // (a lane whose wait ran out waits no more, but goes on with its warp: the prompt above: 676 us; with a vote here 688)
                if (i > 0 && ok) ok = i >= 2 ? arrived(&free[st], ((i >> 1) - 1) & 1) : arrived(q_ready, 0);   // whose angles are in the second stages
                if (warp == kKWarp) {
                    if ((k_wide || v_wide) && mine) s_below[i & 3][my_group] = static_cast<uint16_t>((k_wide ? k_below : 0) | (v_wide ? v_below : 0) << 8);
                    if (lane == 0) s_info[i & 3] = TileInfo{kref + (k_wide || v_wide ? kWide : 0), vref, gone};
                }
                convert((is_v ? v_wide : k_wide) ? 0 : is_v ? v_below : k_below, now.id, from, N - t0, operand + st * S::kOperand);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&full[st]);
                if ((i + 1) % kPer == 0) {
                    now = next;
                    const int batch = (i + 1) / kPer;
                    next = look_up(batch + 1, e_next);
                    e_next = entry(batch + 2);
                }
                if (i + 1 < n_tiles) load(i + 1, now.id);
            }
            copies_wait<0>();
            if (!ok) {
                s_fail = 1;
                atomicOr(A.err, TQ_DEVERR_TIMEOUT);
            }
        }
    } else {
        // ================================================= mma
        if (lane == 0 && n_tiles > 0) {
            constexpr uint32_t id_s = tc::idesc_f16_f32(128, kT);
            constexpr uint32_t id_o = tc::idesc_f16_f32(128, D) | (1u << 16);   // B is MN-major: coordinates contiguous
            constexpr uint32_t kRowStep = (D / 8) * 128;                        // bytes between groups of 8 rows
            const uint32_t base = tc::smem_addr(smem);
            const uint64_t dq = tc::smem_desc(base + S::kQOff, 128, kRowStep);
            const uint64_t dk = tc::smem_desc(base + S::kKOff, 128, kRowStep);
            const uint64_t dv = tc::smem_desc(base + S::kVOff, kRowStep, 128);
            auto scores = [&](int x, int buf, int st) {   // half x's rows with stage st's keys into buffer buf
                const uint64_t q = dq + static_cast<uint64_t>(x * 128 * D * 2 >> 4), k = dk + static_cast<uint64_t>(st * S::kOperand >> 4);
#pragma unroll
                for (int s = 0; s < D / 16; ++s) tc::mma_f16(tmem + S::kS + buf * S::kSStep, q + 16 * s, k + 16 * s, id_s, s > 0);
                if constexpr (kFine)
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        tc::mma_f16(tmem + S::kS + buf * S::kSStep, q + static_cast<uint64_t>(S::kQ >> 4) + 16 * s, k + 16 * s, id_s, 1);
                tc::mma_commit(&s_ready[buf]);
            };
            // O += P V of 64 tokens, from step `from` on
            auto values = [&](int x, int buf, int st, int from, bool first) {
                const uint64_t v = dv + static_cast<uint64_t>(st * S::kOperand >> 4);
                const uint32_t lo = static_cast<uint32_t>(v), hi = static_cast<uint32_t>(v >> 32);
                const uint32_t o = tmem + S::kO + x * D, p = tmem + S::kP + buf * S::kPStep;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if (s == 0 && first) tc::mma_f16_ta_w<false>(o, p, lo, hi, id_o);
                    else tc::mma_f16_ta_w<true>(o, p + 8 * (from + s), lo + (from + s) * (2 * kRowStep >> 4), hi, id_o);
                }
            };
            bool ok = arrived(q_ready, 0) && arrived(&k_full[0], 0);
            tc::tc_fence_after();
            if constexpr (kH == 2) {
                const int nh = two ? 2 : 1;
                if (ok) {
                    for (int x = 0; x < nh; ++x) scores(x, x, 0);
                    tc::mma_commit(&k_free[0]);
                }
                for (int i = 0; i < n_tiles && ok; ++i) {
                    const int st = i & 1, sn = st ^ 1;
                    for (int x = 0; x < nh && ok; ++x) {
                        ok = (x > 0 || arrived(&v_full[st], (i >> 1) & 1)) && arrived(&p_ready[x], i & 1);
                        if (!ok) break;
                        tc::tc_fence_after();
                        values(x, x, st, 0, i == 0);
                        ok = arrived(&p_second[x], i & 1);
                        if (!ok) break;
                        tc::tc_fence_after();
                        values(x, x, st, 4, false);
                        if (x == nh - 1) tc::mma_commit(&v_free[st]);
                        if (i + 1 == n_tiles) {
                            tc::mma_commit(&o_done[x]);
                        } else {
                            ok = x > 0 || arrived(&k_full[sn], ((i + 1) >> 1) & 1);
                            if (!ok) break;
                            tc::tc_fence_after();
                            scores(x, x, sn);
                            if (x == nh - 1) tc::mma_commit(&k_free[sn]);
                        }
                    }
                }
            } else {
                if (ok) {
                    scores(0, 0, 0);
                    tc::mma_commit(&k_free[0]);
                }
                for (int i = 0; i < n_tiles && ok; ++i) {
                    const int st = i & 1, sn = st ^ 1;
                    if (i + 1 < n_tiles) {
                        ok = arrived(&k_full[sn], ((i + 1) >> 1) & 1);
                        if (!ok) break;
                        tc::tc_fence_after();
                        scores(0, sn, sn);
                        tc::mma_commit(&k_free[sn]);
                    }
                    // (one barrier a buffer: the next tile's P may be there too)
                    ok = arrived(&v_full[st], (i >> 1) & 1) && arrived(&p_ready[st], (i >> 1) & 1);
                    if (!ok) break;
                    tc::tc_fence_after();
                    values(0, st, st, 0, i == 0);
                    tc::mma_commit(&v_free[st]);
                    tc::mma_commit(&o_done[0]);
                }
            }
            if (!ok) {
                s_fail = 1;
                atomicOr(A.err, TQ_DEVERR_TIMEOUT);
            }
            // nothing is in flight when the CTA ends
            tc::mma_commit(drained);
            (void)arrived(drained, 0);
        }
        __syncwarp();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
    if (tid == 0)
        for (int s = 0; s < 18; ++s) tc::mbar_inval(&s_bar[s]);
}

template <typename T, int D, bool I8, bool MOD, bool kFine>
cudaError_t launch_f(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
    using S = Shape<D, kFine>;
    static_assert(S::kSmem <= 227 * 1024 - 2560, "shared memory");
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(prefill_kernel<T, D, I8, MOD, kFine>, S::kSmem, allowed);
    if (e != cudaSuccess) return e;
    prefill_kernel<T, D, I8, MOD, kFine><<<dim3(p.groups, a.pool.H, a.batch), kThreads, S::kSmem, s>>>(a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

template <typename T, int D, bool I8, bool MOD>
cudaError_t launch_m(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
    // fp16 queries that are rotated here lose as much by one rounding as the output by its own (error 4.2e-4, and 2.5e-4
    // with a second part, where the output's rounding alone is 2.1e-4; bf16 outputs do not notice). At head_dim 64 a
    // second part costs 10 %; at 128 it would leave room for tiles of 64 tokens only (1211 us for 725), at 256 for none.
    if constexpr (!std::is_same<T, __nv_bfloat16>::value && D == 64)
        if (a.rope.rot > 0) return launch_f<T, D, I8, MOD, true>(a, p, s);
    return launch_f<T, D, I8, MOD, false>(a, p, s);
}

template <typename T, int D>
cudaError_t launch_d(const AttendArgs& a, const AttendPlan& p, int format, cudaStream_t s) {
    const bool mod = a.cap > 0.0f || a.slopes;
    if (format == TQ_KV8_INT8) return mod ? launch_m<T, D, true, true>(a, p, s) : launch_m<T, D, true, false>(a, p, s);
    return mod ? launch_m<T, D, false, true>(a, p, s) : launch_m<T, D, false, false>(a, p, s);
}

template <typename T>
cudaError_t launch_dtype(const AttendArgs& a, const AttendPlan& p, int D, int format, cudaStream_t s) {
    return D == 64 ? launch_d<T, 64>(a, p, format, s) : D == 128 ? launch_d<T, 128>(a, p, format, s) : launch_d<T, 256>(a, p, format, s);
}

}  // namespace

cudaError_t launch_prefill(const AttendArgs& a, const AttendPlan& p, int D, int format, int dtype, cudaStream_t s) {
    return dtype == TQ_F16 ? launch_dtype<__half>(a, p, D, format, s) : launch_dtype<__nv_bfloat16>(a, p, D, format, s);
}

}  // namespace kv8
}  // namespace tq
