// Block tables and slot maps from request lengths.
#include "serve.h"

namespace tq {
namespace serve {
namespace {

constexpr int kRows = 1024;   // rows that a CTA takes at once, a thread each

// Exclusive sum of v over the CTA's kRows threads; `total`: of all.
__device__ int64_t scan(int64_t v, int64_t* s_warp, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int64_t w = lane < kRows / 32 ? s_warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return x - v + (warp > 0 ? before : 0);
}

__global__ void __launch_bounds__(kRows) reserve_kernel(const __grid_constant__ BlocksArgs A) {
    __shared__ int64_t s_warp[32];
    const int64_t cap = static_cast<int64_t>(A.max_blocks) << A.bt_shift;
    int used = *A.n_used;
    if (used < 0 || used > A.n_free) {
        if (threadIdx.x == 0) atomicOr(A.err, TQ_DEVERR_CAPACITY);
        used = A.n_free;
    }
    const int left = A.n_free - used;
    int64_t taken = 0, tokens = 0;   // of the rows before
    for (int row0 = 0; row0 < A.batch; row0 += kRows) {
        const int b = row0 + threadIdx.x;
        int64_t len = 0;
        int n = 0;
        int32_t* row = A.table + static_cast<int64_t>(b) * A.max_blocks;
        int first = 0, end = 0, need = 0;
        if (b < A.batch) {
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
            for (int lb = first; lb < end; ++lb) need += row[lb] < 0;
        }
        int64_t total;
        int64_t rank = taken + scan(need, s_warp, total);
        taken += total;
        if (b < A.batch) {
            for (int lb = first; lb < end; ++lb) {
                int id = row[lb];
                if (id < 0) {
                    if (rank >= left) {   // the first place without a block
                        atomicOr(A.err, TQ_DEVERR_CAPACITY);
                        n = static_cast<int>(max((static_cast<int64_t>(lb) << A.bt_shift) - len, static_cast<int64_t>(0)));
                        break;
                    }
                    id = A.free_blocks[used + rank++];
                    row[lb] = id;
                }
                if (id < 0 || id >= A.num_blocks) atomicOr(A.err, TQ_DEVERR_BLOCK);
            }
            if (A.places.granted) A.places.granted[b] = n;
        }
        const int64_t start = tokens + scan(n, s_warp, total);
        if (b < A.batch && A.places.starts) A.places.starts[b] = static_cast<int32_t>(start);
        tokens += total;
    }
    if (threadIdx.x == 0) {
        if (A.places.starts) A.places.starts[A.batch] = static_cast<int32_t>(tokens);
        if ((A.places.seq_ids || A.places.positions || A.places.slots) && tokens > A.places.max_tokens) atomicOr(A.err, TQ_DEVERR_CAPACITY);
    }
    __syncthreads();
    if (threadIdx.x == 0) *A.n_used = used + static_cast<int>(min(taken, static_cast<int64_t>(left)));
}

// A thread for each packed token: its row by bisection of the starts.
__global__ void __launch_bounds__(256) maps_kernel(const __grid_constant__ BlocksArgs A) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= A.places.max_tokens) return;
    const int32_t* starts = A.places.starts;
    int b = -1, pos = 0;
    int64_t slot = -1;
    if (i < starts[A.batch]) {
        int lo = 0, hi = A.batch;   // starts[lo] <= i < starts[hi]
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (starts[mid] <= i) lo = mid;
            else hi = mid;
        }
        b = lo;
        pos = A.seq[b] + (i - starts[b]);
        const int id = A.table[static_cast<int64_t>(b) * A.max_blocks + (pos >> A.bt_shift)];
        if (id >= 0 && id < A.num_blocks) slot = (static_cast<int64_t>(id) << A.bt_shift) + (pos & ((1 << A.bt_shift) - 1));
    }
    if (A.places.seq_ids) A.places.seq_ids[i] = b;
    if (A.places.positions) A.places.positions[i] = pos;
    if (A.places.slots) A.places.slots[i] = slot;
}

__global__ void __launch_bounds__(kRows) release_kernel(const __grid_constant__ BlocksArgs A) {
    __shared__ int64_t s_warp[32];
    int used = *A.n_used;
    if (used < 0 || used > A.n_free) {
        if (threadIdx.x == 0) atomicOr(A.err, TQ_DEVERR_CAPACITY);
        used = min(max(used, 0), A.n_free);
    }
    // how many come back, then where each goes: the last one lies just before the blocks that are left
    int64_t all = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int64_t before = 0;
        for (int row0 = 0; row0 < A.batch; row0 += kRows) {
            const int b = row0 + threadIdx.x;
            int32_t* row = A.table + static_cast<int64_t>(b) * A.max_blocks;
            int first = A.max_blocks, count = 0;
            if (b < A.batch) {
                const int keep = A.seq[b];
                if (keep < 0) {
                    if (pass == 0) atomicOr(A.err, TQ_DEVERR_SEQLEN);
                } else {
                    first = static_cast<int>((static_cast<int64_t>(keep) + (1 << A.bt_shift) - 1) >> A.bt_shift);
                }
                for (int lb = first; lb < A.max_blocks && row[lb] >= 0; ++lb) count += row[lb] < A.num_blocks;
            }
            int64_t total;
            int64_t rank = before + scan(count, s_warp, total);
            before += total;
            if (pass == 1) {
                for (int lb = first; lb < A.max_blocks && row[lb] >= 0; ++lb) {
                    const int id = row[lb];
                    row[lb] = -1;
                    if (id >= A.num_blocks) {
                        atomicOr(A.err, TQ_DEVERR_BLOCK);
                        continue;
                    }
                    const int64_t at = used - all + rank++;
                    if (at >= 0) A.free_blocks[at] = id;
                }
            }
        }
        all = before;
    }
    if (threadIdx.x == 0) {
        if (all > used) atomicOr(A.err, TQ_DEVERR_CAPACITY);
        *A.n_used = static_cast<int>(max(used - all, static_cast<int64_t>(0)));
    }
}

}  // namespace

cudaError_t launch_reserve(const BlocksArgs& a, cudaStream_t s) {
    reserve_kernel<<<1, kRows, 0, s>>>(a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.places.max_tokens == 0) return e;
    maps_kernel<<<(a.places.max_tokens + 255) / 256, 256, 0, s>>>(a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

cudaError_t launch_release(const BlocksArgs& a, cudaStream_t s) {
    release_kernel<<<1, kRows, 0, s>>>(a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

}  // namespace serve
}  // namespace tq
