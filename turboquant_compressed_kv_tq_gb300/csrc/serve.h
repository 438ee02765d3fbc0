// Internal declarations of the calls around the caches': block tables, position
// rotation, drafted tokens (serve_api.cu checks the arguments; blocks.cu, rope.cu
// and verify.cu hold the kernels).
#pragma once

#include "kv8.h"

namespace tq {
namespace serve {

struct BlocksArgs {
    int32_t* table;
    int32_t* free_blocks;
    int32_t* n_used;
    int n_free, max_blocks, bt_shift, num_blocks;
    int batch, n_new;
    const int32_t *seq, *news;   // release: seq is the lengths to keep
    tq_places places;
    unsigned* err;
};

struct RopeArgs {
    kv8::Rows in[2], out[2];   // queries, keys
    int heads[2];
    kv8::Rope rope;            // rot 0: nothing turns
    int back;                  // the opposite angle
    int stream;                // outputs past the L2 cache (set by the launch)
    int batch, n, D;
    const int32_t *starts, *news;
    unsigned* err;
};

struct VerifyArgs {
    tq_drafts d;
    int batch, K, V;
    int32_t *accepted, *tokens, *keep;
    float* logprobs;
    unsigned* err;
};

#ifdef __CUDACC__
cudaError_t launch_reserve(const BlocksArgs& a, cudaStream_t s);
cudaError_t launch_release(const BlocksArgs& a, cudaStream_t s);
cudaError_t launch_rope(const RopeArgs& a, int dtype, int sms, cudaStream_t s);
cudaError_t launch_verify(const VerifyArgs& a, int sms, cudaStream_t s);
cudaError_t launch_draw(const VerifyArgs& a, int sms, cudaStream_t s);   // no drafts: verification's form for single tokens
#endif

}  // namespace serve
}  // namespace tq
