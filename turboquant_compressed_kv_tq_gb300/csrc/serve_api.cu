// C ABI of the calls around the caches': argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "rows.h"
#include "serve.h"

namespace tq {
namespace serve {
namespace {

constexpr int64_t kMost = 2147483647;

tq_status check_blocks(const tq_blocks* b, int batch) {
    if (!b || !b->table || !b->n_used || b->n_free < 0 || (b->n_free > 0 && !b->free_blocks) || b->max_blocks <= 0 || b->num_blocks <= 0 || batch < 0 || batch > (1 << 24))
        return TQ_ERR_INVALID_ARG;
    if (b->block_tokens < 16 || (b->block_tokens & (b->block_tokens - 1)) != 0) return TQ_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(b->max_blocks) * b->block_tokens > kMost) return TQ_ERR_INVALID_ARG;
    return TQ_OK;
}

tq_status blocks_args(const tq_blocks* b, int batch, BlocksArgs* a) {
    if (device_state(&a->err, nullptr) != TQ_OK) return TQ_ERR_CUDA;
    a->table = b->table;
    a->free_blocks = b->free_blocks;
    a->n_used = b->n_used;
    a->n_free = b->n_free;
    a->max_blocks = b->max_blocks;
    while ((1 << a->bt_shift) < b->block_tokens) ++a->bt_shift;
    a->num_blocks = b->num_blocks;
    a->batch = batch;
    return TQ_OK;
}

kv8::Rows rows_of(const tq_rows* r) { return kv8::Rows{r->data, r->stride_batch, r->stride_head, r->stride_token}; }

}  // namespace
}  // namespace serve
}  // namespace tq

using namespace tq;
using namespace tq::serve;

extern "C" {

tq_status tq_blocks_reserve(const tq_blocks* blocks, int batch, const int32_t* seq_lens, const int32_t* new_lens, int n_new,
                            const tq_places* places, tq_stream_t stream) {
    tq_status st = check_blocks(blocks, batch);
    if (st != TQ_OK) return st;
    if (n_new < 0 || (batch > 0 && !seq_lens) || (places && places->max_tokens < 0)) return TQ_ERR_INVALID_ARG;
    // a row is given at most its capacity: packed places are counted in 32 bits
    if (static_cast<int64_t>(batch) * std::min<int64_t>(n_new, static_cast<int64_t>(blocks->max_blocks) * blocks->block_tokens) > kMost) return TQ_ERR_INVALID_ARG;
    BlocksArgs a{};
    if (places) a.places = *places;
    const bool maps = a.places.seq_ids || a.places.positions || a.places.slots;
    if (!maps) a.places.max_tokens = 0;
    if (maps && a.places.max_tokens > 0 && !a.places.starts) return TQ_ERR_INVALID_ARG;
    if (batch == 0 && !a.places.starts) return TQ_OK;
    {
        // (the maps' launch looks lengths and entries up once more, behind the counts)
        const tq_places& p = a.places;
        const Span written[] = {{blocks->table, 4 * int64_t(batch) * blocks->max_blocks}, {blocks->free_blocks, 4 * int64_t(blocks->n_free)}, {blocks->n_used, 4},
                                {p.granted, 4 * int64_t(batch)}, {p.starts, 4 * (int64_t(batch) + 1)}, {p.seq_ids, 4 * int64_t(p.max_tokens)},
                                {p.positions, 4 * int64_t(p.max_tokens)}, {p.slots, 8 * int64_t(p.max_tokens)}};
        const Span read[] = {{seq_lens, 4 * int64_t(batch)}, {new_lens == p.granted ? nullptr : new_lens, 4 * int64_t(batch)}};
        if (spans_meet(written, read)) return TQ_ERR_INVALID_ARG;
    }
    if ((st = blocks_args(blocks, batch, &a)) != TQ_OK) return st;
    a.seq = seq_lens;
    a.news = new_lens;
    a.n_new = n_new;
    return launch_reserve(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

tq_status tq_blocks_release(const tq_blocks* blocks, int batch, const int32_t* keep_lens, tq_stream_t stream) {
    tq_status st = check_blocks(blocks, batch);
    if (st != TQ_OK) return st;
    if (batch == 0) return TQ_OK;
    if (!keep_lens) return TQ_ERR_INVALID_ARG;
    const Span written[] = {{blocks->table, 4 * int64_t(batch) * blocks->max_blocks}, {blocks->free_blocks, 4 * int64_t(blocks->n_free)}, {blocks->n_used, 4}};
    const Span read[] = {{keep_lens, 4 * int64_t(batch)}};
    if (spans_meet(written, read)) return TQ_ERR_INVALID_ARG;
    BlocksArgs a{};
    if ((st = blocks_args(blocks, batch, &a)) != TQ_OK) return st;
    a.seq = keep_lens;
    return launch_release(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

tq_status tq_rope_apply(const tq_rope* rope, int transposed, tq_dtype dtype, int head_dim, int batch, int n,
                        const tq_rows* q, int q_heads, const tq_rows* q_out, const tq_rows* k, int k_heads,
                        const tq_rows* k_out, const int32_t* starts, const int32_t* new_lens, const int32_t* positions,
                        tq_stream_t stream) {
    if (!rope) return TQ_ERR_INVALID_ARG;
    if (head_dim <= 0 || head_dim > 1024 || head_dim % 16 != 0) return TQ_ERR_UNSUPPORTED;
    if (rope->rot_dim < 0 || rope->rot_dim > head_dim || rope->rot_dim % 16 != 0) return TQ_ERR_UNSUPPORTED;
    if ((rope->rot_dim > 0 && !rope->inv_freq) || !std::isfinite(rope->scale)) return TQ_ERR_INVALID_ARG;
    if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16) return TQ_ERR_INVALID_ARG;
    if (batch < 0 || n < 0 || static_cast<int64_t>(batch) * n > kMost || q_heads <= 0 || q_heads > 65535 || (k && (k_heads <= 0 || k_heads > 65535)))
        return TQ_ERR_INVALID_ARG;
    if (batch == 0 || n == 0) return TQ_OK;
    const int elem = dtype == TQ_F32 ? 4 : 2, sets = k ? 2 : 1;
    const tq_rows *in[2] = {q, k}, *out[2] = {q_out, k_out};
    const int heads[2] = {q_heads, k ? k_heads : 0};
    RopeArgs a{};
    for (int i = 0; i < sets; ++i) {
        tq_status st = check_rows(in[i], elem);
        if (st == TQ_OK) st = check_rows(out[i], elem);
        if (st != TQ_OK) return st;
        a.in[i] = rows_of(in[i]);
        a.out[i] = rows_of(out[i]);
        a.heads[i] = heads[i];
    }
    for (int i = 0; i < sets; ++i) {
        if (Axes(out[i], batch, heads[i], n).meets_itself(head_dim)) return TQ_ERR_INVALID_ARG;
        if (i == 1 && rows_meet(out[0], heads[0], out[1], heads[1], batch, n, head_dim, elem)) return TQ_ERR_INVALID_ARG;
        for (int j = 0; j < sets; ++j) {
            if (i == j && in[i]->data == out[i]->data && same_layout(in[i], out[i], batch, heads[i], n)) continue;
            if (rows_meet(in[j], heads[j], out[i], heads[i], batch, n, head_dim, elem)) return TQ_ERR_INVALID_ARG;
        }
    }
    int sms = 0;
    if (device_state(&a.err, &sms) != TQ_OK) return TQ_ERR_CUDA;
    a.rope = kv8::Rope{rope->inv_freq, rope->rot_dim, rope->interleaved != 0, rope->scale == 0.0f ? 1.0f : rope->scale, positions};
    a.back = transposed != 0;
    a.batch = batch;
    a.n = n;
    a.D = head_dim;
    a.starts = starts;
    a.news = new_lens;
    return launch_rope(a, dtype, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

tq_status tq_verify_drafts(const tq_drafts* drafts, int batch, int num_drafts, int vocab, int32_t* accepted, int32_t* tokens,
                           float* logprobs, int32_t* keep_lens, tq_stream_t stream) {
    if (!drafts || batch < 0 || batch > (1 << 24) || num_drafts < 0 || vocab <= 0 || vocab > (1 << 28)) return TQ_ERR_INVALID_ARG;
    if (num_drafts > 64) return TQ_ERR_UNSUPPORTED;
    auto known = [](int t) { return t == TQ_F32 || t == TQ_BF16 || t == TQ_F16; };
    if (!known(drafts->target_dtype) || (drafts->draft && !known(drafts->draft_dtype))) return TQ_ERR_INVALID_ARG;
    if (batch == 0) return TQ_OK;
    if (!drafts->target || !accepted || !tokens || (num_drafts > 0 && !drafts->draft_tokens) ||
        (num_drafts > 0 && drafts->noise && !drafts->uniforms) || (keep_lens && !drafts->seq_lens))
        return TQ_ERR_INVALID_ARG;
    auto off = [](const void* p, int t) { return !aligned(p, t == TQ_F32 ? 4 : 2); };
    if (off(drafts->target, drafts->target_dtype) || (drafts->draft && off(drafts->draft, drafts->draft_dtype))) return TQ_ERR_INVALID_ARG;
    const int64_t rows = num_drafts + 1, B = batch;
    {
        // an output in an input could change what the cluster's other CTAs have still to read
        const bool drawn = drafts->noise != nullptr;
        const Span written[] = {{accepted, 4 * B}, {tokens, 4 * B * rows}, {logprobs, 4 * B * rows}, {keep_lens, 4 * B}};
        const Span read[] = {{drafts->draft_tokens, 4 * B * num_drafts}, {drafts->draft_lens, 4 * B}, {drawn ? drafts->temperatures : nullptr, 4 * B},
                             {drawn ? drafts->uniforms : nullptr, 4 * B * num_drafts}, {keep_lens == drafts->seq_lens ? nullptr : drafts->seq_lens, keep_lens ? 4 * B : 0}};
        if (spans_meet(written, read)) return TQ_ERR_INVALID_ARG;
        const int size = drafts->target_dtype == TQ_F32 ? 4 : 2, q_size = drafts->draft_dtype == TQ_F32 ? 4 : 2;
        for (const Span& w : written)
            if (w.meets_rows(drafts->target, drafts->target_stride_batch * size, B, drafts->target_stride_row * size, rows, static_cast<int64_t>(vocab) * size) ||
                w.meets_rows(drawn ? drafts->draft : nullptr, drafts->draft_stride_batch * q_size, B, drafts->draft_stride_row * q_size, num_drafts, static_cast<int64_t>(vocab) * q_size) ||
                w.meets_rows(drafts->noise, drafts->noise_stride * 4, B, 0, 1, static_cast<int64_t>(vocab) * 4))
                return TQ_ERR_INVALID_ARG;
    }
    VerifyArgs a{};
    int sms = 0;
    if (device_state(&a.err, &sms) != TQ_OK) return TQ_ERR_CUDA;
    a.d = *drafts;
    a.batch = batch;
    a.K = num_drafts;
    a.V = vocab;
    a.accepted = accepted;
    a.tokens = tokens;
    a.logprobs = logprobs;
    a.keep = keep_lens;
    return launch_verify(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
