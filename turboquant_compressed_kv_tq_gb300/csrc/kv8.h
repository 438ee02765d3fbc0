// Internal declarations of the 8-bit cache's kernels (kv8_api.cu checks the
// arguments and launches; kv8_append.cu, kv8_decode.cu and kv8_prefill.cu hold
// the kernels).
#pragma once

#include "tq_internal.h"

namespace tq {

// The current device's error word and its number of SMs (either may be null): api.cu.
tq_status device_state(unsigned** err, int* num_sms);

namespace kv8 {

// One layer of an 8-bit cache and the block table over it.
struct Pool {
    uint8_t *kc, *vc;   // codes [block][head][token][dim]
    uint8_t *kx, *vx;   // scale bytes [block][head]
    const int32_t* table;
    int max_blocks, num_blocks, H, BT, bt_shift;
};

struct Rows {
    void* data;
    int64_t sb, sh, st;   // strides in elements
};

struct Rope {
    const double* inv_freq;
    int rot, inter;
    float scale;
    const int32_t* positions;   // [batch][n] or null
};

struct AppendArgs {
    Pool pool;
    Rows k, v;
    Rope rope;
    int batch, n_new;
    const int32_t *seq, *news;
    int angle_smem;   // bytes for the angles of a block's tokens, or 0 (set by the launch)
    unsigned* err;
};

struct AttendArgs {
    Pool pool;
    Rows q, out;
    Rope rope;
    int batch, G, L;
    const int32_t *seq, *qlens;
    int max_seq;
    float scale, cap;
    const float* slopes;
    int window;
    const int32_t *prefix, *docs;
    int groups;                // row groups per (sequence, KV head)
    // few rows: states of units that lie in several CTAs' shares, [CTA][2][rows of a group] x (reference, sum)
    // and x D, and the first and last such CTA of each unit [batch][groups][H]
    float *part_ml, *part_o;
    int* unit_shares;
    int pad;                   // what a unit costs besides its tiles, in tiles: counted behind them when shares are dealt out
    unsigned* err;
};

// The launch shape of an attention call, shared by workspace sizing and the launch.
struct AttendPlan {
    int chunk;         // 1: the tensor-memory kernel (many rows), 0: the split kernel (few rows)
    int group_rows;    // query rows of a group
    int groups;        // ceil(G q_len / group_rows)
    int ctas, pad;     // of the split kernel
    size_t ml_bytes, unit_bytes, total;
};

AttendPlan attend_plan(int D, int batch, int H, int G, int L, int max_seq, int num_sms);

#ifdef __CUDACC__
cudaError_t launch_append(const AppendArgs& a, int D, int format, int dtype, int sms, cudaStream_t s);
cudaError_t launch_decode(const AttendArgs& a, const AttendPlan& p, int D, int format, int dtype, cudaStream_t s);
cudaError_t launch_prefill(const AttendArgs& a, const AttendPlan& p, int D, int format, int dtype, cudaStream_t s);
#endif

}  // namespace kv8
}  // namespace tq
