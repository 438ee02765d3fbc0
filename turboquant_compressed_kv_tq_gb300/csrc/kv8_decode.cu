// Attention over the 8-bit cache for few query rows: single tokens, a few
// speculative ones.
//
// The rows of one KV head (r = l G + g: query l, head g of the group) are taken
// kRows = 8 NT at a time; such a group of rows is a unit, and its keys come in
// tiles of 16 tokens. One CTA to an SM; the tiles of all units, one
// after another, are dealt out to them in equal shares, by lengths that only the
// device knows: sequences of any lengths keep every SM busy to the end. A unit
// that lies in one share is finished there; of the others each share leaves a
// state (at most two a CTA), which a second kernel joins. Within a share each
// warp walks tiles of its own. Per tile (mma.sync m16n8k16, fp16 in, fp32
// out; tokens and coordinates on M, query rows on N, so that 8 rows waste
// nothing):
//   S^T = K Q^T      A = the tile's key codes, B = the queries (registers)
//   u   = log2(e) score + log2(value scale)   masks, cap and bias on the way
//   p   = 2^(u - M)  M: the row's reference, moved only when u passes it by 8
//   l  += p / value scale
//   O^T += V^T P     A = the tile's value codes, B = p (two 8x8 transposes)
// Codes become fp16 exactly; block scales are powers of two and stay out of the
// operands: the keys' is a factor of the scores, the values' moves the softmax's
// reference (p <= 2^8 whatever the scales are) and is divided out of the sum. So l
// runs from 2^-63 to 2^63 a key: it is rescaled by the square root of alpha, twice,
// and takes tiles of very small values (zeros), whose p may be below fp32's
// smallest, by way of 2^64 p.
//
// Layout. The coordinates (and for values the token pairs) that an MMA operand
// wants in one lane are whatever order both operands share, so each lane takes
// 16 consecutive bytes: of keys, lane (g, c) reads tokens g and g + 8 at bytes
// 64 i + 16 c; of values, tokens 2c, 2c + 1, 2c + 8, 2c + 9 at bytes 128 i + 16 g.
// A tile's keys and values are 16 D contiguous bytes each: one bulk copy into the
// warp's own queue of stages in shared memory.
//
// Bound: memory, 2 D bytes a token. Measured: 32 sequences of 4096 to 32,768 tokens,
// 8 KV heads of 128, 4 rows each: 213 us, 5.8 TB/s (86 % of a plain copy); 16 rows
// over 262,144 tokens: 109 us, 4.9 TB/s (instructions that wait on one another).
#include <climits>
#include <type_traits>

#include "kv8_device.cuh"
#include "tc_ptx.cuh"

namespace tq {
namespace kv8 {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -FLT_MAX;  // reference of a row that has seen nothing: below every score
constexpr float kGap = 8.0f;       // how far scores may pass the reference (log2 units)
constexpr int kDeep = -24;         // tiles of value exponents below it: p may be too small for fp32 where its share of l is not,
constexpr float kLift = 64.0f;     // so l takes p 2^kLift (without a branch: one cost 215 us for 212 in the batch measured above)

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
    return r;
}

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

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&w)[W], const unsigned char* p) {
    if constexpr (W == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x, w[1] = u.y;
    }
}

template <int D, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    // warps by the registers that a warp needs, one CTA to an SM (16 rows at head_dim 128 with the query fragments in
    // registers: 8 warps, 119 us for the long case; from shared memory, 12 warps: 111)
    static constexpr bool kQShared = D == 128 && NT == 2;   // the query fragments stay in shared memory
    static constexpr int kWarps = kQShared ? 12 : D * NT >= 256 ? 8 : D * NT == 128 ? 12 : 16;
    static constexpr int kU = D == 256 ? 1 : 2;        // tiles taken together: two chains of dependent instructions
    static constexpr int kKL = D / 64;                 // key loads per token
    static constexpr int kVW = D >= 128 ? 4 : 2;       // words of a value load
    static constexpr int kVL = D / (32 * kVW);         // value loads per token
    static constexpr int kMT = D / 16;                 // value MMAs
    static constexpr int kTileBytes = 32 * D;          // keys and values of 16 tokens
    static constexpr int kStages = 192 * 1024 / (kWarps * kTileBytes * kU);   // of kU tiles
    static constexpr int kRing = kStages * kWarps * kTileBytes * kU;
    static constexpr int kOut = kWarps * kRows * D * 4;          // the warps' outputs, over the queues
    static constexpr int kSmem = kRing > kOut ? kRing : kOut;    // and the queries, at the end
    static_assert(kStages >= 2, "a stage to use and one on its way");
};

// A sequence's lengths, checked.
struct Seq {
    int N, nq, pre;
    bool bad;
    __device__ __forceinline__ Seq(const AttendArgs& A, int b) {
        N = A.seq[b];
        nq = A.qlens ? A.qlens[b] : A.L;
        const bool bad_n = N < 0 || N > A.max_seq || (N + A.pool.BT - 1) >> A.pool.bt_shift > A.pool.max_blocks, bad_q = nq < 0 || nq > A.L;
        if (bad_n) N = 0;
        if (bad_q) nq = nq < 0 ? 0 : A.L;
        bad = bad_n || bad_q;
        pre = A.prefix ? min(max(A.prefix[b], 0), N) : 0;
    }
};

__device__ __forceinline__ Sight sight_of(const AttendArgs& A, const Seq& q, int b, int l) {
    Sight s;
    s.p = q.N - q.nq + l;
    s.lo = 0;
    if (A.window > 0) s.lo = max(s.lo, s.p - A.window + 1);
    if (A.docs) s.lo = max(s.lo, A.docs[static_cast<int64_t>(b) * A.L + l]);
    s.prefix = q.pre;
    return s;
}

// What the rows of a group see, as tiles: [0, n1) and then [first, first + n2).
struct Tiles {
    int l_first, l_last, rows;     // the group's queries and rows
    int lo_max;                    // the largest first key of a row
    int n1, first, n2;
    __device__ __forceinline__ Tiles(const AttendArgs& A, const Seq& q, int b, int grp, int group_rows) {
        rows = min(A.G * A.L - grp * group_rows, group_rows);
        l_first = grp * group_rows / A.G;
        l_last = min((grp * group_rows + rows - 1) / A.G, q.nq - 1);
        int lo_min = INT_MAX;
        lo_max = 0;
        for (int l = l_first; l <= l_last; ++l) {
            const int lo = sight_of(A, q, b, l).lo;
            lo_min = min(lo_min, lo);
            lo_max = max(lo_max, lo);
        }
        const int p_max = q.N - q.nq + l_last;
        n1 = (q.pre + 15) >> 4;
        first = max(n1, lo_min >> 4);
        n2 = p_max < 0 || lo_min > p_max ? 0 : max(0, (p_max >> 4) + 1 - first);
    }
    __device__ __forceinline__ bool none() const { return l_last < l_first; }   // only rows behind the sequence's queries
    __device__ __forceinline__ int at(int i) const { return i < n1 ? i : first + (i - n1); }
    // a unit that sees nothing counts as one tile: its rows are written too
    __device__ __forceinline__ int count() const { return none() ? 0 : max(1, n1 + n2); }
    // its place in the shares
    __device__ __forceinline__ int room(const AttendArgs& A) const { return none() ? 0 : count() + A.pad; }
};

template <typename T, int D, int NT, bool I8>
__global__ void __launch_bounds__(32 * Shape<D, NT>::kWarps, 1) decode_kernel(const __grid_constant__ AttendArgs A) {
    using S = Shape<D, NT>;
    constexpr int kRows = S::kRows, kThreads = 32 * S::kWarps;
    extern __shared__ __align__(16) unsigned char smem[];
    // the queries as operand fragments, one uint2 (4 coordinates) a lane: coordinates 16 (kKL c + i) + 4 s .. of
    // row 8 nt + g at step 4 i + s, lane 4 g + c; with fp16 queries a second set holds what the first rounded off
    constexpr bool kFine = sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value;
    auto s_frag = [&](int part, int r, int d) {
        const int ks = 4 * ((d >> 4) % S::kKL) + ((d >> 2) & 3), ln = 4 * (r & 7) + (d >> 4) / S::kKL;
        return reinterpret_cast<uint2*>(smem + S::kSmem) + ((part * NT + (r >> 3)) * (D / 16) + ks) * 32 + ln;
    };
    auto split = [](float x0, float x1, float x2, float x3, uint2& lo) {
        const __half2 a = __floats2half2_rn(x0, x1), d = __floats2half2_rn(x2, x3);
        const float2 fa = __half22float2(a), fd = __half22float2(d);
        lo = make_uint2(pack_out<__half>(x0 - fa.x, x1 - fa.y), pack_out<__half>(x2 - fd.x, x3 - fd.y));
        return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&d));
    };
    __shared__ uint64_t s_turns[D / 2];
    __shared__ float s_fac[kRows], s_m[S::kWarps][kRows], s_l[S::kWarps][kRows];
    __shared__ Sight s_sight[kRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const Pool& P = A.pool;

    // ---------------- this CTA's share of the tiles of all units. A pair (sequence, row group) has the
    // tiles of its P.H units, one head after another
    __shared__ long long s_scan[S::kWarps], s_at;
    __shared__ __align__(8) uint64_t s_bar[S::kWarps * S::kStages];
    if (lane == 0) {
        for (int k = 0; k < S::kStages; ++k) tc::mbar_init(&s_bar[warp * S::kStages + k], 1);
        tc::mbar_fence_init();
    }
    __shared__ int s_pair;
    const int pairs = A.batch * A.groups, each = (pairs + kThreads - 1) / kThreads;
    long long sum = 0;
    for (int p = tid * each; p < min((tid + 1) * each, pairs); ++p) {
        const int b = p / A.groups;
        const Seq q(A, b);
        if (q.bad && blockIdx.x == 0) atomicOr(A.err, TQ_DEVERR_SEQLEN);
        sum += static_cast<long long>(Tiles(A, q, b, p % A.groups, kRows).room(A)) * P.H;
    }
    long long upto = sum;   // inclusive over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < S::kWarps; ++w) {
        if (w < warp) upto += s_scan[w];
        total += s_scan[w];
    }
    // equal shares, but at least a tile for each warp, and no cut through sequences that are all short
    const long long even = total < (1ll << 31) ? static_cast<long long>((static_cast<unsigned>(total) + gridDim.x - 1) / gridDim.x)
                                               : (total + gridDim.x - 1) / gridDim.x;
    const int longest = ((A.max_seq + 15) >> 4) + A.pad;
    const long long share = max(static_cast<long long>(longest <= 2 * S::kWarps ? max(longest, 1) : S::kWarps), even);
    const long long begin = blockIdx.x * share, end = min(begin + share, total);
    if (begin >= end) return;
    if (upto - sum <= begin && begin < upto) {
        long long at = upto - sum;
        for (int p = tid * each;; ++p) {
            const int b = p / A.groups;
            const long long n = static_cast<long long>(Tiles(A, Seq(A, b), b, p % A.groups, kRows).room(A)) * P.H;
            if (begin < at + n) {
                s_pair = p;
                s_at = at;
                break;
            }
            at += n;
        }
    }
    if (A.rope.rot > 0)
        for (int i = tid; i < A.rope.rot / 2; i += kThreads) s_turns[i] = turns_of(A.rope.inv_freq[i]);
    __syncthreads();

    uint64_t* bars = s_bar + warp * S::kStages;
    unsigned puts = 0, gets = 0;   // of the warp's stages, over all its segments
    bool dead = false;             // a copy did not come: nothing more is started
    int pair = s_pair;
    long long pair_at = s_at;
    for (long long from = begin; from < end;) {
        const int b = pair / A.groups, grp = pair % A.groups;
        const Seq seq(A, b);
        const Tiles tiles(A, seq, b, grp, kRows);
        const int N = seq.N, nq = seq.nq, rows = tiles.rows, lo_max = tiles.lo_max, p_min = N - nq + tiles.l_first;
        const int unit_tiles = tiles.count(), unit_room = tiles.room(A);
        if (unit_room == 0) {
            ++pair;
            continue;
        }
        const long long in_pair = from - pair_at;
        const int h = static_cast<int>(in_pair < (1ll << 31) ? static_cast<long long>(static_cast<unsigned>(in_pair) / static_cast<unsigned>(unit_room))
                                                             : in_pair / unit_room);
        const int i_begin = static_cast<int>(in_pair - static_cast<long long>(h) * unit_room);
        const int i_room = static_cast<int>(min(static_cast<long long>(unit_room - i_begin), end - from));
        auto next_segment = [&]() {
            from += i_room;
            if (from == pair_at + static_cast<long long>(unit_room) * P.H) {
                pair_at = from;
                ++pair;
            }
        };
        if (i_begin >= unit_tiles) {   // only what is counted behind a unit's tiles
            next_segment();
            continue;
        }
        const int i_all = min(i_room, unit_tiles - i_begin);                                               // tiles of this segment
        const int i_end = min(i_begin + i_all, tiles.n1 + tiles.n2);                                        // without the one that is none
        const int per = (max(i_end - i_begin, 0) + S::kWarps - 1) / S::kWarps;   // tiles of a warp, consecutive
        const int w_begin = min(i_begin + warp * per, i_end), w_end = min(w_begin + per, i_end);
        const int64_t unit = static_cast<int64_t>(pair) * P.H + h;
        if (tid == 0 && i_begin == 0 && gridDim.x > 1)   // the shares that the unit lies in
            *reinterpret_cast<int2*>(A.unit_shares + 2 * unit) =
                make_int2(blockIdx.x, static_cast<int>((pair_at + static_cast<long long>(h) * unit_room + unit_tiles - 1) / share));

        // ---------------- the copies of the first tiles, on their way while the queries are prepared
        const bool busy = w_begin < w_end && !dead;
        const int64_t unit_bytes = static_cast<int64_t>(P.BT) * D;

        // lane k holds the block and scales of the warp's tile base + k, and of the 32 after those
        int base = w_begin;
        int64_t id = -1, id_next = -1;
        uint32_t meta = 0, meta_next = 0;   // scale bytes, and whether there is a block
        auto look_up = [&](int from, int64_t& x, uint32_t& sc) {
            x = -1;
            sc = 0;
            const int i = from + lane;
            if (i < w_end) {
                const int lb = (tiles.at(i) << 4) >> P.bt_shift;
                const int64_t at = P.table ? P.table[b * static_cast<int64_t>(P.max_blocks) + lb] : b * static_cast<int64_t>(P.max_blocks) + lb;
                if (at >= 0 && at < P.num_blocks) {
                    x = at * P.H + h;
                    sc = P.kx[x] | (P.vx[x] << 8) | 0x10000u;
                } else {
                    atomicOr(A.err, TQ_DEVERR_BLOCK);
                }
            }
        };
        constexpr int kStep = S::kTileBytes * S::kU, kU = S::kU;
        unsigned char* ring = smem + warp * S::kStages * kStep;
        uint32_t ahead[S::kStages - 1][kU];   // meta of the tiles on their way
        // start the copies of the kU tiles from i (none behind the warp's last tile); their metas
        auto fetch = [&](int i, uint32_t (&mt)[kU]) {
            const unsigned st = puts % S::kStages;
            if (i < w_end) {
                if (lane == 0) tc::mbar_expect_tx(&bars[st], i + kU <= w_end ? kStep : S::kTileBytes);
                ++puts;
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                mt[u] = 0;
                if (i + u >= w_end) continue;
                if (i + u - base == 32) {
                    base = i + u;
                    id = id_next;
                    meta = meta_next;
                    look_up(base + 32, id_next, meta_next);
                }
                const int64_t x = __shfl_sync(0xffffffffu, id, i + u - base);
                mt[u] = __shfl_sync(0xffffffffu, meta, i + u - base);
                if (lane == 0) {   // where there is no block: any block, which nobody sees
                    const int64_t off = (x < 0 ? 0 : x) * unit_bytes + static_cast<int64_t>((tiles.at(i + u) << 4) & (P.BT - 1)) * D;
                    unsigned char* dst = ring + st * kStep + u * S::kTileBytes;
                    tc::bulk_g2s(dst, P.kc + off, 16 * D, &bars[st]);
                    tc::bulk_g2s(dst + 16 * D, P.vc + off, 16 * D, &bars[st]);
                }
            }
        };
        if (busy) {
            look_up(base, id, meta);
            look_up(base + 32, id_next, meta_next);
#pragma unroll
            for (int k = 0; k < S::kStages - 1; ++k) fetch(w_begin + k * kU, ahead[k]);
        }

        // ---------------- the queries: rotated, scaled by a power of two, fp16
        if (i_begin < i_end) {
            constexpr int J = D / 16;   // chunk pairs of a row: J consecutive lanes
            for (int it = tid; it < kRows * J; it += kThreads) {
                const int r = it / J, j = it % J;
                const int rr = grp * kRows + r, l = rr / A.G;
                float xa[8] = {}, xb[8] = {};
                int a0, b0;
                chunk_pair(j, A.rope.rot, A.rope.inter, a0, b0);
                if (r < rows && l < nq) {
                    const T* q = static_cast<const T*>(A.q.data) + b * A.q.sb + static_cast<int64_t>(h * A.G + rr % A.G) * A.q.sh + l * A.q.st;
                    load8(q + a0, xa);
                    load8(q + b0, xb);
                    if (A.rope.rot > 0)
                        rotate_pair(xa, xb, j, A.rope, s_turns, A.rope.positions ? A.rope.positions[static_cast<int64_t>(b) * A.L + l] : N - nq + l);
                }
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(fabsf(xa[i]), fabsf(xb[i])));
#pragma unroll
                for (int o = J / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                // to [1, 2): fp16 then keeps 11 bits down to 2^-14 of the row's largest
                const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -126), 126);
                const float f = exp2i(-e);
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    uint2 lo;
                    *s_frag(0, r, a0 + i) = split(xa[i] * f, xa[i + 1] * f, xa[i + 2] * f, xa[i + 3] * f, lo);
                    if constexpr (kFine) *s_frag(1, r, a0 + i) = lo;
                    *s_frag(0, r, b0 + i) = split(xb[i] * f, xb[i + 1] * f, xb[i + 2] * f, xb[i + 3] * f, lo);
                    if constexpr (kFine) *s_frag(1, r, b0 + i) = lo;
                }
                if (j == 0) s_fac[r] = A.scale * exp2i(e);
            }
        }
        if (tid < kRows) s_sight[tid] = sight_of(A, seq, b, min((grp * kRows + tid) / A.G, tiles.l_last));
        __syncthreads();

        float acc[NT][S::kMT][4];
        float m[NT][2], l_sum[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < S::kMT; ++j) acc[nt][j][0] = acc[nt][j][1] = acc[nt][j][2] = acc[nt][j][3] = 0.0f;
            m[nt][0] = m[nt][1] = kNone;
            l_sum[nt][0] = l_sum[nt][1] = 0.0f;
        }
        if (busy) {
            uint32_t qf[NT][D / 16][2];
            float fac[NT][2], slope[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int ks = 0; ks < (S::kQShared ? 0 : D / 16); ++ks) {
                    const uint2 f = reinterpret_cast<const uint2*>(smem + S::kSmem)[(nt * (D / 16) + ks) * 32 + lane];
                    qf[nt][ks][0] = f.x;
                    qf[nt][ks][1] = f.y;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * nt + 2 * c + e;
                    fac[nt][e] = s_fac[r];
                    const int rr = grp * kRows + r;
                    slope[nt][e] = A.slopes && r < rows ? A.slopes[h * A.G + rr % A.G] * kLog2e : 0.0f;
                }
            }
            const bool plain = A.cap <= 0.0f && !A.slopes;
            const float cap2 = A.cap * kLog2e, cap_in = A.cap > 0.0f ? 1.0f / A.cap : 0.0f;
            for (int i = w_begin; i < w_end; i += kU) {
                uint32_t mt[kU];
                int t0[kU];   // a tile behind the warp's last one: behind the sequence's end
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    mt[u] = ahead[0][u];
                    t0[u] = i + u < w_end ? tiles.at(i + u) << 4 : N;
#pragma unroll
                    for (int k = 0; k < S::kStages - 2; ++k) ahead[k][u] = ahead[k + 1][u];
                }
                __syncwarp();   // every lane has read the stage that is filled now
                fetch(i + (S::kStages - 1) * kU, ahead[S::kStages - 2]);
                const unsigned st = gets % S::kStages;
                dead = !arrived(&bars[st], (gets / S::kStages) & 1);
                if (__any_sync(0xffffffffu, dead)) {
                    dead = true;
                    break;
                }
                ++gets;
                const unsigned char* src = ring + st * kStep;
                // ---------------- scores
                float sc[kU][NT][4];
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) sc[u][nt][0] = sc[u][nt][1] = sc[u][nt][2] = sc[u][nt][3] = 0.0f;
#pragma unroll
                for (int k = 0; k < S::kKL; ++k) {
                    uint32_t w0[kU][4], w1[kU][4];
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        load_words(w0[u], src + u * S::kTileBytes + g * D + 16 * (S::kKL * c + k));
                        load_words(w1[u], src + u * S::kTileBytes + (g + 8) * D + 16 * (S::kKL * c + k));
                    }
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint2 fine[NT], now[NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            now[nt] = S::kQShared ? reinterpret_cast<const uint2*>(smem + S::kSmem)[(nt * (D / 16) + 4 * k + w) * 32 + lane]
                                                  : make_uint2(qf[nt][4 * k + w][0], qf[nt][4 * k + w][1]);
                        if constexpr (kFine)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                fine[nt] = reinterpret_cast<const uint2*>(smem + S::kSmem)[((NT + nt) * (D / 16) + 4 * k + w) * 32 + lane];
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            uint32_t a0, a1, a2, a3;
                            codes_f16<I8>(w0[u][w], a0, a2);
                            codes_f16<I8>(w1[u][w], a1, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816(sc[u][nt], a0, a1, a2, a3, now[nt].x, now[nt].y);
                                if constexpr (kFine) mma16816(sc[u][nt], a0, a1, a2, a3, fine[nt].x, fine[nt].y);
                            }
                        }
                    }
                }
                // ---------------- u = log2(e) score + log2(value scale), masked
                float lg[kU][NT][4];
                bool pass = false;
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int kx = mt[u] & 0xFF, vx = (mt[u] >> 8) & 0xFF;
                    const bool here = mt[u] >> 16;
                    const float ks2 = exp2i(kx == 0 ? -126 : kx - 127), lv = static_cast<float>(vx - 127);
                    // e: token g + 8 (e >> 1), row 2c + (e & 1)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[u][nt][e] *= fac[nt][e & 1] * ks2;
                    if (plain) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) lg[u][nt][e] = fmaf(sc[u][nt][e], kLog2e, lv);
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) lg[u][nt][e] = sc[u][nt][e] * kLog2e;
                        if (A.cap > kUsualCap) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) lg[u][nt][e] = capped_wide(sc[u][nt][e] * cap_in, cap2);
                        } else if (A.cap > 0.0f) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) lg[u][nt][e] = capped(sc[u][nt][e] * cap_in, cap2);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (A.slopes) {
                                    const int p = s_sight[8 * nt + 2 * c + (e & 1)].p;
                                    lg[u][nt][e] -= slope[nt][e & 1] * fabsf(static_cast<float>(p - (t0[u] + g + 8 * (e >> 1))));
                                }
                                lg[u][nt][e] += lv;
                            }
                    }
                    if (!(here && t0[u] + 15 <= p_min && t0[u] >= lo_max)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int t = t0[u] + g + 8 * (e >> 1);
                                if (!(here && t < N && s_sight[8 * nt + 2 * c + (e & 1)].sees(t))) lg[u][nt][e] = -INFINITY;
                            }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) pass |= lg[u][nt][e] > m[nt][e & 1] + kGap;
                }
                // ---------------- the reference moves only when a score passes it by the gap
                if (__any_sync(0xffffffffu, pass)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = fmaxf(lg[0][nt][e], lg[0][nt][e + 2]);
                            if constexpr (kU == 2) x = fmaxf(x, fmaxf(lg[1][nt][e], lg[1][nt][e + 2]));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                            x = fmaxf(x, m[nt][e]);
                            const float half = ex2(0.5f * (m[nt][e] - x)), alpha = half * half;
                            m[nt][e] = x;
                            l_sum[nt][e] = l_sum[nt][e] * half * half;
#pragma unroll
                            for (int j = 0; j < S::kMT; ++j) {
                                acc[nt][j][e] *= alpha;
                                acc[nt][j][e + 2] *= alpha;
                            }
                        }
                }
                // ---------------- p, its sum, and p as the second operand (rows on N)
                uint32_t pb[kU][NT][2];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int vx = (mt[u] >> 8) & 0xFF;
                    const float lift = vx < 127 + kDeep ? kLift : 0.0f, drop = vx < 127 + kDeep ? exp2i(-static_cast<int>(kLift)) : 1.0f;
                    const float iv = exp2i(127 - vx < -126 ? -126 : min(127 - vx, 126)) * drop;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            p[e] = ex2((lg[u][nt][e] - m[nt][e & 1]) + lift);
                            l_sum[nt][e & 1] = fmaf(p[e], iv, l_sum[nt][e & 1]);
                        }
                        pb[u][nt][0] = transpose8x8(pack_out<__half>(p[0] * drop, p[1] * drop));
                        pb[u][nt][1] = transpose8x8(pack_out<__half>(p[2] * drop, p[3] * drop));
                    }
                }
                // ---------------- O^T += V^T P
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int k = 0; k < S::kVL; ++k) {
                        const unsigned char* from_v = src + u * S::kTileBytes + 16 * D + 32 * S::kVW * k + 4 * S::kVW * g;
                        uint32_t vw[4][S::kVW];
#pragma unroll
                        for (int t = 0; t < 4; ++t) load_words(vw[t], from_v + (2 * c + (t & 1) + 8 * (t >> 1)) * D);
                        // codes behind the sequence's end, or of no block, may be anything: their weight is 0, so they have to be finite
                        if (t0[u] + 16 > N || !(mt[u] >> 16)) {
#pragma unroll
                            for (int t = 0; t < 4; ++t)
                                if (t0[u] + 2 * c + (t & 1) + 8 * (t >> 1) >= N || !(mt[u] >> 16))
#pragma unroll
                                    for (int w = 0; w < S::kVW; ++w) vw[t][w] = 0;
                        }
#pragma unroll
                        for (int w = 0; w < S::kVW; ++w) {
                            uint32_t x[2][4];   // [token pair][coordinate]: fp16 pairs of two tokens
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                const uint32_t a = vw[2 * t][w], d = vw[2 * t + 1][w];
                                codes_f16<I8>(__byte_perm(a, d, 0x5140), x[t][0], x[t][1]);
                                codes_f16<I8>(__byte_perm(a, d, 0x7362), x[t][2], x[t][3]);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816(acc[nt][(k * S::kVW + w) * 2], x[0][0], x[0][1], x[1][0], x[1][1], pb[u][nt][0], pb[u][nt][1]);
                                mma16816(acc[nt][(k * S::kVW + w) * 2 + 1], x[0][2], x[0][3], x[1][2], x[1][3], pb[u][nt][0], pb[u][nt][1]);
                            }
                        }
                    }
            }
        }

        if (dead) {   // what is in flight ends (or is given up) before its shared memory is used for anything else
            if (lane == 0) atomicOr(A.err, TQ_DEVERR_TIMEOUT);
            for (; gets < puts; ++gets) (void)arrived(&bars[gets % S::kStages], (gets / S::kStages) & 1);
        }
        // ---------------- the CTA's state of each row: the states of the warps that had tiles, at their largest reference
        const int had = per > 0 ? (i_end - i_begin + per - 1) / per : 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l_sum[nt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0) {
                    s_m[warp][8 * nt + 2 * c + e] = m[nt][e];
                    s_l[warp][8 * nt + 2 * c + e] = x;
                }
            }
        __syncthreads();   // and the queries in shared memory are done with
        float* s_o = reinterpret_cast<float*>(smem);   // [warps][kRows][D]
        if (warp < had)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * nt + 2 * c + e;
                float top = s_m[0][r];
                for (int w = 1; w < had; ++w) top = fmaxf(top, s_m[w][r]);
                const float f = ex2(m[nt][e] - top);
                float* o = s_o + (warp * kRows + r) * D;
#pragma unroll
                for (int k = 0; k < S::kVL; ++k)
#pragma unroll
                    for (int w = 0; w < S::kVW; ++w) {
                        const int j = (k * S::kVW + w) * 2;
                        const int d = 32 * S::kVW * k + 4 * S::kVW * g + 4 * w;
                        *reinterpret_cast<float4*>(o + d) =
                            make_float4(acc[nt][j][e] * f, acc[nt][j][e + 2] * f, acc[nt][j + 1][e] * f, acc[nt][j + 1][e + 2] * f);
                    }
            }
        __syncthreads();
        for (int it = tid; it < rows * (D / 4); it += kThreads) {
            const int r = it / (D / 4), d = 4 * (it % (D / 4));
            const int rr = grp * kRows + r, l = rr / A.G;
            if (l >= nq) continue;
            float top = s_m[0][r];
            for (int w = 1; w < had; ++w) top = fmaxf(top, s_m[w][r]);
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float sum = 0.0f;
            for (int w = 0; w < had; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(s_o + (w * kRows + r) * D + d);
                o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
                const float half = ex2(0.5f * (s_m[w][r] - top));
                sum = fmaf(s_l[w][r] * half, half, sum);
            }
            if (i_all == unit_tiles) {
                const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
                T* dst = static_cast<T*>(A.out.data) + b * A.out.sb + static_cast<int64_t>(h * A.G + rr % A.G) * A.out.sh + l * A.out.st + d;
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack_out<T>(o.x * inv, o.y * inv), pack_out<T>(o.z * inv, o.w * inv));
            } else {
                // the unit goes on behind this share (state 1 of the CTA), or began before it (state 0)
                const int64_t at = (2 * static_cast<int64_t>(blockIdx.x) + (i_begin == 0 ? 1 : 0)) * kRows + r;
                *reinterpret_cast<float4*>(A.part_o + at * D + d) = o;
                if (d == 0) *reinterpret_cast<float2*>(A.part_ml + 2 * at) = make_float2(top, sum);
            }
        }
        next_segment();
        tc::fence_proxy_async_smem();
        __syncthreads();   // before the next segment's queries and copies
    }
    tc::grid_release_dependents();
}

// Joins the states of the units that lie in several shares:
// out = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) l_i. One warp a row.
template <typename T, int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttendArgs A, int group_rows) {
    tc::grid_wait_prior();
    constexpr int kLanes = D / 4 < 32 ? D / 4 : 32, kV = D / 128 > 0 ? D / 128 : 1;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);   // over batch, row groups, H, rows of a group
    const int lane = threadIdx.x & 31, H = A.pool.H;
    const int64_t unit = row / group_rows;
    const int r = static_cast<int>(row % group_rows);
    if (unit >= static_cast<int64_t>(A.batch) * A.groups * H) return;
    const int h = static_cast<int>(unit % H), grp = static_cast<int>(unit / H % A.groups), b = static_cast<int>(unit / H / A.groups);
    const int rr = grp * group_rows + r, l = rr / A.G;
    const int nq = A.qlens ? min(A.qlens[b], A.L) : A.L;
    if (rr >= A.G * A.L || l >= nq || grp * group_rows / A.G >= nq) return;
    const int2 sh = *reinterpret_cast<const int2*>(A.unit_shares + 2 * unit);
    if (sh.x == sh.y) return;   // finished by its CTA
    auto state = [&](int i) { return (2 * static_cast<int64_t>(i) + (i == sh.x ? 1 : 0)) * group_rows + r; };
    float top = kNone;
    for (int i = sh.x + lane; i <= sh.y; i += 32) top = fmaxf(top, A.part_ml[2 * state(i)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.0f;
    float4 o[kV] = {};
#pragma unroll 4
    for (int i = sh.x; i <= sh.y; ++i) {
        const int64_t a = state(i);
        const float2 ml = *reinterpret_cast<const float2*>(A.part_ml + 2 * a);
        const float half = ex2(0.5f * (ml.x - top)), f = half * half;
        sum = fmaf(ml.y * half, half, sum);
        if (lane < kLanes)
#pragma unroll
            for (int k = 0; k < kV; ++k) {
                const float4 x = *reinterpret_cast<const float4*>(A.part_o + a * D + 128 * k + 4 * lane);
                o[k].x = fmaf(x.x, f, o[k].x), o[k].y = fmaf(x.y, f, o[k].y), o[k].z = fmaf(x.z, f, o[k].z), o[k].w = fmaf(x.w, f, o[k].w);
            }
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    T* dst = static_cast<T*>(A.out.data) + b * A.out.sb + static_cast<int64_t>(h * A.G + rr % A.G) * A.out.sh + l * A.out.st;
    if (lane < kLanes)
#pragma unroll
        for (int k = 0; k < kV; ++k)
            *reinterpret_cast<uint2*>(dst + 128 * k + 4 * lane) =
                make_uint2(pack_out<T>(o[k].x * inv, o[k].y * inv), pack_out<T>(o[k].z * inv, o[k].w * inv));
}

template <typename T, int D, int NT, bool I8>
cudaError_t launch_t(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
    using S = Shape<D, NT>;
    constexpr bool kFine = !std::is_same<T, __nv_bfloat16>::value;
    const int smem = S::kSmem + S::kRows * D * 2 * (kFine ? 2 : 1);
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(decode_kernel<T, D, NT, I8>, smem, allowed);
    if (e != cudaSuccess) return e;
    decode_kernel<T, D, NT, I8><<<p.ctas, 32 * S::kWarps, smem, s>>>(a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.ctas == 1) return e;
    const int64_t rows = static_cast<int64_t>(a.batch) * a.groups * a.pool.H * p.group_rows;
    e = launch_overlapped(join_kernel<T, D>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, s, a, p.group_rows);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return e;
}

template <typename T, int D>
cudaError_t launch_d(const AttendArgs& a, const AttendPlan& p, int format, cudaStream_t s) {
    if (format == TQ_KV8_INT8) return p.group_rows == 8 ? launch_t<T, D, 1, true>(a, p, s) : launch_t<T, D, 2, true>(a, p, s);
    return p.group_rows == 8 ? launch_t<T, D, 1, false>(a, p, s) : launch_t<T, D, 2, false>(a, p, s);
}

template <typename T>
cudaError_t launch_dtype(const AttendArgs& a, const AttendPlan& p, int D, int format, cudaStream_t s) {
    return D == 64 ? launch_d<T, 64>(a, p, format, s) : D == 128 ? launch_d<T, 128>(a, p, format, s) : launch_d<T, 256>(a, p, format, s);
}

}  // namespace

cudaError_t launch_decode(const AttendArgs& a, const AttendPlan& p, int D, int format, int dtype, cudaStream_t s) {
    return dtype == TQ_F16 ? launch_dtype<__half>(a, p, D, format, s) : launch_dtype<__nv_bfloat16>(a, p, D, format, s);
}

}  // namespace kv8
}  // namespace tq
