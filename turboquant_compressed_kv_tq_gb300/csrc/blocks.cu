// Block tables and slot maps from request lengths.
//
// What a row takes from the free list, and gives back, lies behind what the rows before it do: sums over all rows stand between
// looking at the entries and writing them. A cluster of CTAs has the table, a thread for each row; rows of many blocks go to
// warps, a lane for each entry. The CTAs tell each other their sums (two barriers of the cluster a call), so that one launch is
// enough, without a workspace, and no atomics decide an order. Nothing here is large: the chain of dependent loads (length, entry, free
// block, entry) and the launches bound it. Maps of few tokens are written by the same launch, those of many by a second one over all SMs,
// where what is written (16 bytes a token) counts.
//
// Measured: places and maps of a token for each of 32 rows 3.6 us; of up to 5 tokens for each of 300 rows, and a release, 9.7 us together; of
// 512 prompts up to 4096 tokens (17 MB of maps) 15.3 us.
#include <algorithm>

#include "cluster.cuh"
#include "serve.h"

namespace tq {
namespace serve {
namespace {

constexpr int kRows = 1024;       // threads of a CTA at most: rows that it takes at once
constexpr int kFewest = 128;      // threads of a CTA at least
constexpr int kFew = 4;           // entries that a thread looks at by itself
constexpr int kGroups = 4;        // groups of 32 entries that a warp looks up at once
constexpr int kMostCtas = 8;
constexpr int kFusedTokens = 16384;   // maps of up to so many tokens are written by the rows' own launch (a second one costs 2 us and more)
constexpr unsigned kAll = 0xffffffffu;

struct Shared {
    int64_t warp[32];
    int64_t totals[2][2][kMostCtas];   // of the cluster's CTAs: [chunk of rows, by turns][sum]
    int64_t start[kRows];              // of each row: its blocks' place among all that move, then its first packed token
    int value[kRows];                  // of each row: blocks, then tokens
    int longs[kRows], n_longs;         // rows of many blocks
    int first[kRows], end[kRows];      // the entries of those
    int64_t len[kRows];                // lengths of those
};

// Exclusive sum of v over the CTA's threads; `total`: of all.
template <typename N>
__device__ N scan(N v, N* s_warp, N& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    N x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const N y = __shfl_up_sync(kAll, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    N w = lane < blockDim.x >> 5 ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const N y = __shfl_up_sync(kAll, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(kAll, w, 31);
    const N before = __shfl_sync(kAll, w, (warp + 31) & 31);
    return x - v + (warp > 0 ? before : 0);
}

// The same over the cluster's CTAs, in the order of their ranks: one barrier. `mine`: of this CTA.
template <typename N>
__device__ N scan_cluster(N v, Shared& S, int64_t (&slot)[kMostCtas], int ctas, int rank, N& total, N& mine) {
    const N before = scan(v, reinterpret_cast<N*>(S.warp), mine);
    if (ctas == 1) {
        total = mine;
        return before;
    }
    if (threadIdx.x < ctas) send(remote(&slot[rank], threadIdx.x), static_cast<uint32_t>(mine), static_cast<uint32_t>(static_cast<int64_t>(mine) >> 32));
    cluster_arrive();
    cluster_wait();
    N ahead = 0;
    total = 0;
    for (int r = 0; r < ctas; ++r) {
        const N x = static_cast<N>(slot[r]);
        if (r < rank) ahead += x;
        total += x;
    }
    return before + ahead;
}

// Rows of a call: chunks of ctas x `rows` of them, `rows` to a CTA.
struct Rows {
    int ctas, rank, rows, batch;
    __device__ __forceinline__ Rows(int log_ctas, int n) : ctas(1 << log_ctas), rank(log_ctas ? static_cast<int>(cluster_rank()) : 0), batch(n) {
        rows = min(static_cast<int>(blockDim.x), (n + ctas - 1) >> log_ctas);
    }
    __device__ __forceinline__ int row(int chunk, int i) const {   // -1: none
        const int64_t b = (static_cast<int64_t>(chunk) * ctas + rank) * rows + i;
        return i < rows && b < batch ? static_cast<int>(b) : -1;
    }
    __device__ __forceinline__ int chunks() const { return rows ? (batch + ctas * rows - 1) / (ctas * rows) : 0; }
};

__device__ __forceinline__ void write_maps(const BlocksArgs& A, int64_t i, int b, int pos) {
    if (A.places.seq_ids) A.places.seq_ids[i] = b;
    if (A.places.positions) A.places.positions[i] = pos;
    if (A.places.slots) {
        int64_t slot = -1;
        if (b >= 0) {
            const int id = A.table[static_cast<int64_t>(b) * A.max_blocks + (pos >> A.bt_shift)];
            if (id >= 0 && id < A.num_blocks) slot = (static_cast<int64_t>(id) << A.bt_shift) + (pos & ((1 << A.bt_shift) - 1));
        }
        A.places.slots[i] = slot;
    }
}

__global__ void __launch_bounds__(kRows) reserve_kernel(const __grid_constant__ BlocksArgs A, int log_ctas, int fused) {
    __shared__ Shared S;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t cap = static_cast<int64_t>(A.max_blocks) << A.bt_shift;
    if (!fused && A.places.max_tokens > 0) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");   // the maps' launch, which waits for this one's end
    const Rows R(log_ctas, A.batch);
    if (R.ctas > 1) cluster_arrive();   // (waited for before the first word to another CTA)
    const int was_used = *A.n_used;
    int taken = 0, tokens = 0;   // of the chunks before (blocks and tokens of a call are below 2^31)
    for (int chunk = 0; chunk < R.chunks(); ++chunk) {
        const int b = R.row(chunk, tid);
        int64_t len = 0;
        int n = 0, first = 0, end = 0;
        if (tid == 0) S.n_longs = 0;
        __syncthreads();
        int32_t* row = A.table + static_cast<int64_t>(b) * A.max_blocks;
        int ids[kFew];
        int need = 0;
        if (b >= 0) {   // where its new tokens lie: entries [first, end)
            len = A.seq[b];
            n = A.news ? A.news[b] : A.n_new;
            if (n < 0 || n > A.n_new) {
                atomicOr(A.err, TQ_DEVERR_SEQLEN);
                n = min(max(n, 0), A.n_new);
            }
            if (len < 0 || len > cap) {
                atomicOr(A.err, TQ_DEVERR_SEQLEN);
                len = 0;
                n = 0;
            }
            if (len + n > cap) {
                atomicOr(A.err, TQ_DEVERR_CAPACITY);
                n = static_cast<int>(cap - len);
            }
            first = static_cast<int>(len >> A.bt_shift);
            end = n > 0 ? static_cast<int>((len + n + (1 << A.bt_shift) - 1) >> A.bt_shift) : first;
            if (end - first > kFew) {
                S.longs[atomicAdd(&S.n_longs, 1)] = tid;   // (in any order: each writes its own row's)
                S.first[tid] = first;
                S.end[tid] = end;
                S.len[tid] = len;
            } else {
#pragma unroll
                for (int e = 0; e < kFew; ++e)
                    if (first + e < end) ids[e] = row[first + e];
#pragma unroll
                for (int e = 0; e < kFew; ++e)
                    if (first + e < end) need += ids[e] < 0;
            }
        }
        __syncthreads();
        for (int l = warp; l < S.n_longs; l += blockDim.x >> 5) {
            const int i = S.longs[l];
            const int32_t* entries = A.table + static_cast<int64_t>(R.row(chunk, i)) * A.max_blocks;
            int count = 0;
            const int last = S.end[i];
            for (int lb = S.first[i] + lane; lb < last; lb += 32 * kGroups) {
                int id[kGroups];
#pragma unroll
                for (int g = 0; g < kGroups; ++g) id[g] = lb + g * 32 < last ? entries[lb + g * 32] : 0;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) count += id[g] < 0;
            }
            count = __reduce_add_sync(kAll, count);
            if (lane == 0) S.value[i] = count;
        }
        __syncthreads();
        const bool few = end - first <= kFew;
        if (b >= 0 && !few) need = S.value[tid];
        if (chunk == 0 && R.ctas > 1) cluster_wait();
        int total, mine;
        const int rank0 = taken + scan_cluster(need, S, S.totals[chunk & 1][0], R.ctas, R.rank, total, mine);
        taken += total;
        const bool good = was_used >= 0 && was_used <= A.n_free;
        const int used = good ? was_used : A.n_free, left = A.n_free - used;
        // the rows' entries; n: tokens before the first place without a block
        if (b >= 0 && few) {
            int rank = rank0;
            bool out = false;
#pragma unroll
            for (int e = 0; e < kFew; ++e) {
                const int lb = first + e;
                if (lb >= end || out) continue;
                if (ids[e] < 0) {
                    if (rank >= left) {
                        atomicOr(A.err, TQ_DEVERR_CAPACITY);
                        n = static_cast<int>(max((static_cast<int64_t>(lb) << A.bt_shift) - len, static_cast<int64_t>(0)));
                        out = true;
                        continue;
                    }
                    ids[e] = A.free_blocks[used + rank++];
                    row[lb] = ids[e];
                }
                if (ids[e] < 0 || ids[e] >= A.num_blocks) atomicOr(A.err, TQ_DEVERR_BLOCK);
            }
        }
        S.start[tid] = rank0;
        S.value[tid] = n;
        __syncthreads();
        for (int l = warp; l < S.n_longs; l += blockDim.x >> 5) {
            const int i = S.longs[l];
            int32_t* entries = A.table + static_cast<int64_t>(R.row(chunk, i)) * A.max_blocks;
            int rank = static_cast<int>(S.start[i]);
            const int last = S.end[i];
            bool out = false;
            for (int lb0 = S.first[i]; lb0 < last && !out; lb0 += 32 * kGroups) {
                int id[kGroups];
#pragma unroll
                for (int g = 0; g < kGroups; ++g) id[g] = lb0 + g * 32 + lane < last ? entries[lb0 + g * 32 + lane] : 0;
                unsigned lacking[kGroups];
                int mine[kGroups];
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    lacking[g] = __ballot_sync(kAll, id[g] < 0);
                    mine[g] = rank + __popc(lacking[g] & ((1u << lane) - 1));
                    rank += __popc(lacking[g]);
                }
                // the first place without a block, and the blocks of those before it: all looked up at once
                int stop = last;
#pragma unroll
                for (int g = kGroups - 1; g >= 0; --g) {
                    const unsigned gone = __ballot_sync(kAll, id[g] < 0 && mine[g] >= left);
                    if (gone) stop = lb0 + g * 32 + __ffs(gone) - 1;
                }
#pragma unroll
                for (int g = 0; g < kGroups; ++g) lacking[g] = lb0 + g * 32 + lane < stop && id[g] < 0;
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
                    if (lacking[g]) id[g] = A.free_blocks[used + mine[g]];
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int lb = lb0 + g * 32 + lane;
                    if (lacking[g]) entries[lb] = id[g];
                    if (lb < stop && (id[g] < 0 || id[g] >= A.num_blocks)) atomicOr(A.err, TQ_DEVERR_BLOCK);
                }
                if (stop < last) {
                    out = true;
                    if (lane == 0) {
                        atomicOr(A.err, TQ_DEVERR_CAPACITY);
                        S.value[i] = static_cast<int>(max((static_cast<int64_t>(stop) << A.bt_shift) - S.len[i], static_cast<int64_t>(0)));
                    }
                }
            }
        }
        __syncthreads();
        n = b >= 0 ? S.value[tid] : 0;
        if (b >= 0 && A.places.granted) A.places.granted[b] = n;
        const int start = tokens + scan_cluster(n, S, S.totals[chunk & 1][1], R.ctas, R.rank, total, mine);
        if (b >= 0 && A.places.starts) A.places.starts[b] = start;
        tokens += total;
        if (fused) {
            S.start[tid] = start;
            S.value[tid] = static_cast<int>(len);
            __syncthreads();
            // this CTA's rows' tokens, a thread for each: its row by bisection
            const int rows = min(R.rows, max(0, R.batch - (chunk * R.ctas + R.rank) * R.rows));
            const int i0 = static_cast<int>(S.start[0]), i1 = static_cast<int>(min(static_cast<int64_t>(i0) + mine, static_cast<int64_t>(A.places.max_tokens)));
            for (int i = i0 + tid; rows > 0 && i < i1; i += blockDim.x) {
                int lo = 0, hi = rows;   // start[lo] <= i < start[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (S.start[mid] <= i) lo = mid;
                    else hi = mid;
                }
                write_maps(A, i, R.row(chunk, lo), S.value[lo] + static_cast<int>(i - S.start[lo]));
            }
            __syncthreads();
        }
    }
    if (R.rank != 0) return;
    // (behind the last barrier: every thread has read n_used)
    if (tid == 0) {
        const bool good = was_used >= 0 && was_used <= A.n_free;
        if (!good) atomicOr(A.err, TQ_DEVERR_CAPACITY);
        if (A.places.starts) A.places.starts[A.batch] = tokens;
        if (A.places.max_tokens > 0 && tokens > A.places.max_tokens) atomicOr(A.err, TQ_DEVERR_CAPACITY);
        *A.n_used = good ? was_used + min(taken, A.n_free - was_used) : A.n_free;
    }
    if (fused)
        for (int i = tokens + tid; i < A.places.max_tokens; i += blockDim.x) write_maps(A, i, -1, 0);
}

constexpr int kMapThreads = 256, kMapTokens = 4096;   // of a CTA

// Grid: pieces of each row's new tokens (parts of a row side by side), then the maps' ends. Four neighbouring tokens to a thread, in
// stores of 16 bytes, where the maps lie for it.
__global__ void __launch_bounds__(kMapThreads) maps_kernel(const __grid_constant__ BlocksArgs A, int parts) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");   // for the rows' launch
    const int64_t piece = blockIdx.x, rows = static_cast<int64_t>(A.batch) * parts;
    const tq_places& P = A.places;
    if (piece >= rows) {
        const int64_t total = P.starts[A.batch], i0 = (piece - rows) * kMapTokens, end = min(i0 + kMapTokens, static_cast<int64_t>(P.max_tokens));
        for (int64_t i = max(i0, total) + threadIdx.x; i < end; i += kMapThreads) write_maps(A, i, -1, 0);
        return;
    }
    const int b = static_cast<int>(piece / parts), j0 = static_cast<int>(piece % parts) * kMapTokens;
    const int64_t start = P.starts[b], i0 = start + j0;
    const int64_t i1 = min(min(static_cast<int64_t>(P.starts[b + 1]), static_cast<int64_t>(P.max_tokens)), i0 + kMapTokens);
    if (i0 >= i1) return;
    const int ahead = A.seq[b] - static_cast<int>(start);   // position less packed place
    const bool wide = ((reinterpret_cast<uintptr_t>(P.seq_ids) | reinterpret_cast<uintptr_t>(P.positions) | reinterpret_cast<uintptr_t>(P.slots)) & 15) == 0;
    const int64_t a0 = wide ? min(i1, (i0 + 3) & ~static_cast<int64_t>(3)) : i1, a1 = wide ? max(a0, i1 & ~static_cast<int64_t>(3)) : i1;   // whole fours
    for (int64_t i = i0 + threadIdx.x; i < a0; i += kMapThreads) write_maps(A, i, b, ahead + static_cast<int>(i));
    for (int64_t i = a1 + threadIdx.x; i < i1; i += kMapThreads) write_maps(A, i, b, ahead + static_cast<int>(i));
    const int32_t* row = A.table + static_cast<int64_t>(b) * A.max_blocks;
    const int mask = (1 << A.bt_shift) - 1;
#pragma unroll 2
    for (int64_t i = a0 + 4 * threadIdx.x; i < a1; i += 4 * kMapThreads) {
        const int pos = ahead + static_cast<int>(i);
        if (P.seq_ids) *reinterpret_cast<int4*>(P.seq_ids + i) = make_int4(b, b, b, b);
        if (P.positions) *reinterpret_cast<int4*>(P.positions + i) = make_int4(pos, pos + 1, pos + 2, pos + 3);
        if (P.slots) {
            const int lb = pos >> A.bt_shift, lb3 = (pos + 3) >> A.bt_shift, id = row[lb], id3 = row[lb3];
            longlong2 v[2];
            long long* slot = reinterpret_cast<long long*>(v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int mine = (pos + k) >> A.bt_shift == lb ? id : id3;
                slot[k] = mine >= 0 && mine < A.num_blocks ? (static_cast<long long>(mine) << A.bt_shift) + ((pos + k) & mask) : -1;
            }
            reinterpret_cast<longlong2*>(P.slots + i)[0] = v[0];
            reinterpret_cast<longlong2*>(P.slots + i)[1] = v[1];
        }
    }
}

__global__ void __launch_bounds__(kRows) release_kernel(const __grid_constant__ BlocksArgs A, int log_ctas) {
    __shared__ Shared S;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Rows R(log_ctas, A.batch);
    if (R.ctas > 1) cluster_arrive();   // (waited for before the first word to another CTA)
    int used = *A.n_used;
    if (used < 0 || used > A.n_free) {
        if (tid == 0 && R.rank == 0) atomicOr(A.err, TQ_DEVERR_CAPACITY);
        used = min(max(used, 0), A.n_free);
    }
    if (R.ctas > 1) cluster_wait();
    // how many come back, then where each goes: the last one lies just before the blocks that are left
    int64_t all = 0;
    int turn = 0;
    for (int pass = R.chunks() > 1 ? 0 : 1; pass < 2; ++pass) {   // (one chunk: its own sum is all)
        int64_t before = 0;
        for (int chunk = 0; chunk < R.chunks(); ++chunk, ++turn) {
            const int b = R.row(chunk, tid);
            if (tid == 0) S.n_longs = 0;
            __syncthreads();
            int32_t* row = A.table + static_cast<int64_t>(b) * A.max_blocks;
            int ids[kFew], held = 0, first = A.max_blocks;
            bool few = true;
            if (b >= 0) {
                const int keep = A.seq[b];
                if (keep < 0 && (pass == 0 || R.chunks() == 1)) atomicOr(A.err, TQ_DEVERR_SEQLEN);
                if (keep >= 0) first = static_cast<int>(min(static_cast<int64_t>(A.max_blocks), (static_cast<int64_t>(keep) + (1 << A.bt_shift) - 1) >> A.bt_shift));
#pragma unroll
                for (int e = 0; e < kFew; ++e) ids[e] = first + e < A.max_blocks ? row[first + e] : -1;
                while (held < kFew && (held == 0 ? ids[0] : held == 1 ? ids[1] : held == 2 ? ids[2] : ids[3]) >= 0) ++held;
                if (held == kFew) {
                    few = false;
                    S.longs[atomicAdd(&S.n_longs, 1)] = tid;
                    S.first[tid] = first;
                }
            }
            int count = 0;
#pragma unroll
            for (int e = 0; e < kFew; ++e) count += e < held && ids[e] < A.num_blocks;
            __syncthreads();
            // f(entry, id) of a long row's entries up to the first negative one, a lane for each; kGroups x 32 looked up at once
            auto each = [&](int i, auto&& f) {
                const int32_t* entries = A.table + static_cast<int64_t>(R.row(chunk, i)) * A.max_blocks;
                for (int lb0 = S.first[i]; lb0 < A.max_blocks; lb0 += 32 * kGroups) {
                    int id[kGroups];
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) id[g] = lb0 + g * 32 + lane < A.max_blocks ? entries[lb0 + g * 32 + lane] : -1;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const unsigned gone = __ballot_sync(kAll, id[g] < 0);
                        const int n = gone ? __ffs(gone) - 1 : 32;
                        f(lb0 + g * 32 + lane, id[g], lane < n);
                        if (gone) return;
                    }
                }
            };
            for (int l = warp; l < S.n_longs; l += blockDim.x >> 5) {
                int n = 0;
                each(S.longs[l], [&](int, int id, bool there) { n += there && id < A.num_blocks; });
                n = __reduce_add_sync(kAll, n);
                if (lane == 0) S.value[S.longs[l]] = n;
            }
            __syncthreads();
            if (!few) count = S.value[tid];
            int64_t total, mine;
            const int64_t rank0 = before + scan_cluster<int64_t>(b >= 0 ? count : 0, S, S.totals[turn & 1][0], R.ctas, R.rank, total, mine);
            before += total;
            if (R.chunks() == 1) all = total;
            if (pass == 1) {
                auto give = [&](int64_t rank, int id) {
                    const int64_t at = used - all + rank;
                    if (at >= 0) A.free_blocks[at] = id;
                };
                if (few) {
                    int64_t rank = rank0;
#pragma unroll
                    for (int e = 0; e < kFew; ++e) {
                        if (e < held) {
                            row[first + e] = -1;
                            if (ids[e] < A.num_blocks) give(rank++, ids[e]);
                            else atomicOr(A.err, TQ_DEVERR_BLOCK);
                        }
                    }
                }
                S.start[tid] = rank0;
                __syncthreads();
                for (int l = warp; l < S.n_longs; l += blockDim.x >> 5) {
                    const int i = S.longs[l];
                    int32_t* entries = A.table + static_cast<int64_t>(R.row(chunk, i)) * A.max_blocks;
                    int64_t rank = S.start[i];
                    each(i, [&](int lb, int id, bool there) {
                        const bool good = there && id < A.num_blocks;
                        const unsigned them = __ballot_sync(kAll, good);
                        if (good) give(rank + __popc(them & ((1u << lane) - 1)), id);
                        if (there) {
                            entries[lb] = -1;
                            if (!good) atomicOr(A.err, TQ_DEVERR_BLOCK);
                        }
                        rank += __popc(them);
                    });
                }
                __syncthreads();
            }
        }
        if (pass == 0) all = before;
    }
    if (tid == 0 && R.rank == 0) {   // (behind the last cluster barrier: every CTA has read n_used)
        if (all > used) atomicOr(A.err, TQ_DEVERR_CAPACITY);
        *A.n_used = static_cast<int>(max(used - all, static_cast<int64_t>(0)));
    }
}

template <typename... Params, typename... Args>
cudaError_t launch_rows(void (*kernel)(Params...), int log_ctas, int threads, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1u << log_ctas);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << log_ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = log_ctas ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return e;
}

}  // namespace

cudaError_t launch_reserve(const BlocksArgs& a, cudaStream_t s) {
    // one CTA where each row is a thread's; eight where rows may be warps', or there are more than a CTA's threads
    const int log_ctas = a.batch > kRows || (a.batch > 32 && (a.n_new >> a.bt_shift) + 2 > kFew) ? 3 : 0;
    const bool fused = a.places.max_tokens > 0 && a.places.max_tokens <= kFusedTokens;
    // threads of a CTA: one for a row, one for every other packed token
    const int threads = log_ctas ? kRows : std::min(kRows, std::max(kFewest, (std::max(a.batch, fused ? a.places.max_tokens / 2 : 0) + 31) / 32 * 32));
    const cudaError_t e = launch_rows(reserve_kernel, log_ctas, threads, s, a, log_ctas, fused ? 1 : 0);
    if (e != cudaSuccess || a.places.max_tokens == 0 || fused) return e;
    const int64_t most = std::min<int64_t>(a.n_new, static_cast<int64_t>(a.max_blocks) << a.bt_shift);
    const int parts = static_cast<int>(std::max<int64_t>(1, (most + kMapTokens - 1) / kMapTokens));
    const int64_t grid = static_cast<int64_t>(a.batch) * parts + (a.places.max_tokens + kMapTokens - 1) / kMapTokens;
    const cudaError_t f = launch_overlapped(maps_kernel, dim3(static_cast<unsigned>(grid)), dim3(kMapThreads), 0, s, a, parts);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return f;
}

cudaError_t launch_release(const BlocksArgs& a, cudaStream_t s) {
    // (how many blocks come back is not known here: rows of many are warps')
    // Measured, one CTA of a thread for each row, eight of 256 and of 1024: 300 rows, a block or none from each: 5.0, 5.2, 6.7 us;
    // 1000 rows of 64 blocks, all of them (and taken before): 61, 32, 24; 64 rows of 2048: 94, 40, 41.
    const int log_ctas = a.batch > 32 ? 3 : 0;
    const int threads = !log_ctas ? 512 : a.batch > 2048 ? kRows : 256;
    return launch_rows(release_kernel, log_ctas, threads, s, a, log_ctas);
}

}  // namespace serve
}  // namespace tq
