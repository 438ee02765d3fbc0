// C ABI of the 8-bit cache: argument checks, launch plans and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "kv8.h"
#include "rows.h"

namespace tq {
namespace kv8 {
namespace {

constexpr int kMaxTokens = 1 << 30;   // positions, with room for sums in 32 bits

tq_status check_cache(const tq_kv8_cache* c) {
    if (!c) return TQ_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return TQ_ERR_UNSUPPORTED;
    if (c->block_tokens < 16 || c->block_tokens > 256 || (c->block_tokens & (c->block_tokens - 1)) != 0)
        return TQ_ERR_UNSUPPORTED;
    if (c->format != TQ_KV8_E4M3 && c->format != TQ_KV8_INT8) return TQ_ERR_UNSUPPORTED;
    if (c->num_layers <= 0 || c->num_blocks <= 0 || c->num_kv_heads <= 0 || c->num_kv_heads > 65535)
        return TQ_ERR_INVALID_ARG;
    return TQ_OK;
}

tq_status check_pool(const tq_kv8_cache* c, int layer) {
    if (layer < 0 || layer >= c->num_layers) return TQ_ERR_INVALID_ARG;
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return TQ_ERR_INVALID_ARG;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16)) return TQ_ERR_INVALID_ARG;
    const int64_t units = static_cast<int64_t>(c->num_blocks) * c->num_kv_heads;
    if (c->num_layers > 1 && (c->code_layer_stride % 16 != 0 || c->code_layer_stride < units * c->block_tokens * c->head_dim ||
                              c->scale_layer_stride < units))
        return TQ_ERR_INVALID_ARG;
    return TQ_OK;
}

tq_status check_table(const tq_kv8_cache* c, int batch, const int32_t* table, int max_blocks) {
    if (batch < 0 || batch > 32767 || max_blocks <= 0 || max_blocks > kMaxTokens / c->block_tokens) return TQ_ERR_INVALID_ARG;
    if (!table && static_cast<int64_t>(batch) * max_blocks > c->num_blocks) return TQ_ERR_CAPACITY;
    return TQ_OK;
}

// Whether rows of out share memory with each other, or with q's rows where those lie as out's do.
bool out_overlaps(const tq_rows* q, const tq_rows* out, int64_t nb, int64_t nh, int64_t nt, int D) {
    const Axes o(out, nb, nh, nt);
    if (o.meets_itself(D) || q->data == out->data) return true;
    if (!same_layout(q, out, nb, nh, nt)) return false;
    const int64_t apart = (reinterpret_cast<intptr_t>(out->data) - reinterpret_cast<intptr_t>(q->data)) / 2;
    return o.meet(apart, D);
}

tq_status make_rope(const tq_rope* r, int D, const int32_t* positions, Rope* out) {
    *out = Rope{};
    if (!r || r->rot_dim == 0) return TQ_OK;
    if (r->rot_dim < 0 || r->rot_dim > D || r->rot_dim % 16 != 0) return TQ_ERR_UNSUPPORTED;
    if (!r->inv_freq || !std::isfinite(r->scale)) return TQ_ERR_INVALID_ARG;
    *out = Rope{r->inv_freq, r->rot_dim, r->interleaved != 0, r->scale == 0.0f ? 1.0f : r->scale, positions};
    return TQ_OK;
}

Pool make_pool(const tq_kv8_cache* c, int layer, const int32_t* table, int max_blocks) {
    Pool p{};
    const int64_t co = layer * c->code_layer_stride, so = layer * c->scale_layer_stride;
    p.kc = static_cast<uint8_t*>(c->k_codes) + co;
    p.vc = static_cast<uint8_t*>(c->v_codes) + co;
    p.kx = static_cast<uint8_t*>(c->k_scales) + so;
    p.vx = static_cast<uint8_t*>(c->v_scales) + so;
    p.table = table;
    p.max_blocks = max_blocks;
    p.num_blocks = c->num_blocks;
    p.H = c->num_kv_heads;
    p.BT = c->block_tokens;
    while ((1 << p.bt_shift) < p.BT) ++p.bt_shift;
    return p;
}

Rows make_rows(const tq_rows* r) { return Rows{r->data, r->stride_batch, r->stride_head, r->stride_token}; }

tq_status check_sizes(const tq_kv8_cache* c, int batch, int Hq, int L, int max_seq) {
    if (batch < 0 || batch > 32767 || L < 0 || L > kMaxTokens || max_seq < 0 || max_seq > kMaxTokens) return TQ_ERR_INVALID_ARG;
    if (Hq <= 0 || Hq % c->num_kv_heads != 0) return TQ_ERR_INVALID_ARG;
    const int64_t rows = static_cast<int64_t>(Hq / c->num_kv_heads) * L;
    if (rows > kMaxTokens) return TQ_ERR_INVALID_ARG;
    return TQ_OK;
}

}  // namespace

AttendPlan attend_plan(int D, int batch, int H, int G, int L, int max_seq, int num_sms) {
    AttendPlan p{};
    const int rows = G * L;
    // Which kernel, for more than 16 rows a KV head (by lengths alone: what a window or documents hide is not counted, and
    // costs both less). The split kernel reads the cache once for each 16 rows, at about
    // 4.8 TB/s (4 at head_dim 64), behind some 18 us of set-up and 4 us for each unit that an SM takes; the chunk kernel
    // reads it once for 256 (128), but walks a sequence on one SM, at 1.5 / 2.1 / 1.9 us a tile of 128 / 128 / 64 tokens.
    // Measured, split and chunk, us: 4 heads x 16 queries over 32768 tokens, 8 KV heads, head_dim 128: 68, 531; 64 queries
    // over 4096: 45, 82; 512 over 4096: 245, 83; 8 sequences x 32 over 1024: 67, 26; head_dim 256, 200 queries x 8 heads
    // over 8192, 2 KV heads: 170, 235; 333 x 4 over 500: 61, 31; head_dim 64, 4 sequences, 16 x 8 over 8192: 81, 104.
    const double kv_bytes = 2.0 * D * max_seq, sets = static_cast<double>(batch) * H;
    const double split_units = sets * ((rows + 15) / 16), chunk_rows = D == 256 ? 128 : 256;
    const double split_us = 18 + 4 * split_units / num_sms + split_units * kv_bytes / (D == 64 ? 4.0e6 : 4.8e6);
    const double waves = std::ceil(sets * std::ceil(rows / chunk_rows) / num_sms);
    const double chunk_us = 12 + waves * std::ceil(max_seq / (D == 256 ? 64.0 : 128.0)) * (D == 64 ? 1.5 : D == 128 ? 2.1 : 1.85);
    if (rows > 16 && chunk_us < split_us) {
        p.chunk = 1;
        p.group_rows = D == 256 ? 128 : 256;
        p.groups = (rows + p.group_rows - 1) / p.group_rows;
        return p;
    }
    p.group_rows = rows <= 8 ? 8 : 16;
    p.groups = (rows + p.group_rows - 1) / p.group_rows;
    // one share of the tiles for each SM, at least a tile for each of its CTA's warps (eight or more)
    const int64_t units = static_cast<int64_t>(batch) * H * p.groups;
    const int64_t tiles = units * std::max(1, (max_seq + 15) / 16);
    p.ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(num_sms, (tiles + 7) / 8)));
    // taking up a unit costs an SM about 4 us, some 32 tiles' time: counted where SMs take several, so that prompts' first
    // rows, whose units have a tile or two, do not pile up on a few (512 x 4 rows over 512 tokens: 484 us without)
    p.pad = units > num_sms ? 32 : 0;
    if (p.ctas > 1) {
        const size_t n = static_cast<size_t>(2) * p.ctas * p.group_rows;
        p.ml_bytes = (n * 8 + 255) / 256 * 256;
        p.unit_bytes = (static_cast<size_t>(units) * 8 + 255) / 256 * 256;
        p.total = p.ml_bytes + p.unit_bytes + n * D * 4;
    }
    return p;
}

}  // namespace kv8
}  // namespace tq

using namespace tq;
using namespace tq::kv8;

extern "C" {

tq_status tq_kv8_append(const tq_kv8_cache* cache, int layer, const tq_rows* k, const tq_rows* v, tq_dtype dtype,
                        int batch, int n_new, const int32_t* seq_lens, const int32_t* new_lens,
                        const int32_t* block_table, int max_blocks, const tq_rope* rope, const int32_t* positions,
                        tq_stream_t stream) {
    tq_status st = check_cache(cache);
    if (st == TQ_OK) st = check_pool(cache, layer);
    if (st == TQ_OK) st = check_table(cache, batch, block_table, max_blocks);
    if (st != TQ_OK) return st;
    if (dtype != TQ_F32 && dtype != TQ_BF16 && dtype != TQ_F16) return TQ_ERR_INVALID_ARG;
    if (n_new < 0) return TQ_ERR_INVALID_ARG;
    if (static_cast<int64_t>(n_new) > static_cast<int64_t>(max_blocks) * cache->block_tokens) return TQ_ERR_CAPACITY;
    AppendArgs a{};
    if ((st = make_rope(rope, cache->head_dim, positions, &a.rope)) != TQ_OK) return st;
    if (batch == 0 || n_new == 0) return TQ_OK;
    const int elem = dtype == TQ_F32 ? 4 : 2;
    if ((st = check_rows(k, elem)) != TQ_OK || (st = check_rows(v, elem)) != TQ_OK) return st;
    if (!seq_lens) return TQ_ERR_INVALID_ARG;
    int sms = 0;
    if (device_state(&a.err, &sms) != TQ_OK) return TQ_ERR_CUDA;
    a.pool = make_pool(cache, layer, block_table, max_blocks);
    a.k = make_rows(k);
    a.v = make_rows(v);
    a.batch = batch;
    a.n_new = n_new;
    a.seq = seq_lens;
    a.news = new_lens;
    return launch_append(a, cache->head_dim, cache->format, dtype, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? TQ_OK
               : TQ_ERR_CUDA;
}

tq_status tq_kv8_workspace_bytes(const tq_kv8_cache* cache, int batch, int num_q_heads, int q_len, int max_seq_len,
                                 size_t* bytes) {
    if (!bytes) return TQ_ERR_INVALID_ARG;
    *bytes = 0;
    tq_status st = check_cache(cache);
    if (st == TQ_OK) st = check_sizes(cache, batch, num_q_heads, q_len, max_seq_len);
    if (st != TQ_OK || batch == 0 || q_len == 0) return st;
    int sms = 0;
    if (device_state(nullptr, &sms) != TQ_OK) return TQ_ERR_CUDA;
    *bytes = attend_plan(cache->head_dim, batch, cache->num_kv_heads, num_q_heads / cache->num_kv_heads, q_len, max_seq_len, sms).total;
    return TQ_OK;
}

tq_status tq_kv8_attention(const tq_kv8_cache* cache, int layer, const tq_rows* q, tq_dtype dtype, int batch,
                           int num_q_heads, int q_len, const int32_t* seq_lens, const int32_t* q_lens,
                           const int32_t* block_table, int max_blocks, int max_seq_len, const tq_kv8_scores* scores,
                           const tq_rows* out, void* workspace, size_t workspace_bytes, tq_stream_t stream) {
    tq_status st = check_cache(cache);
    if (st == TQ_OK) st = check_pool(cache, layer);
    if (st == TQ_OK) st = check_table(cache, batch, block_table, max_blocks);
    if (st == TQ_OK) st = check_sizes(cache, batch, num_q_heads, q_len, max_seq_len);
    if (st != TQ_OK) return st;
    if (dtype == TQ_F32) return TQ_ERR_UNSUPPORTED;
    if (dtype != TQ_BF16 && dtype != TQ_F16) return TQ_ERR_INVALID_ARG;
    AttendArgs a{};
    const tq_kv8_scores none{};
    const tq_kv8_scores& sc = scores ? *scores : none;
    if (!std::isfinite(sc.scale) || !std::isfinite(sc.softcap) || sc.softcap < 0.0f || sc.window < 0) return TQ_ERR_INVALID_ARG;
    if ((st = make_rope(sc.rope, cache->head_dim, sc.positions, &a.rope)) != TQ_OK) return st;
    if (batch == 0 || q_len == 0) return TQ_OK;
    if ((st = check_rows(q, 2)) != TQ_OK || (st = check_rows(out, 2)) != TQ_OK) return st;
    // (with q_lens, rows behind a sequence's queries are neither read nor written: only a row's own heads are known to be)
    if (!seq_lens || out_overlaps(q, out, q_lens ? 1 : batch, num_q_heads, q_lens ? 1 : q_len, cache->head_dim)) return TQ_ERR_INVALID_ARG;
    int sms = 0;
    if (device_state(&a.err, &sms) != TQ_OK) return TQ_ERR_CUDA;
    const AttendPlan p = attend_plan(cache->head_dim, batch, cache->num_kv_heads, num_q_heads / cache->num_kv_heads, q_len, max_seq_len, sms);
    if (p.total > 0) {
        if (!workspace || !aligned(workspace, 256)) return TQ_ERR_INVALID_ARG;
        if (workspace_bytes < p.total) return TQ_ERR_CAPACITY;
    }
    a.pool = make_pool(cache, layer, block_table, max_blocks);
    a.q = make_rows(q);
    a.out = make_rows(out);
    a.batch = batch;
    a.G = num_q_heads / cache->num_kv_heads;
    a.L = q_len;
    a.seq = seq_lens;
    a.qlens = q_lens;
    a.max_seq = max_seq_len;
    a.scale = sc.scale == 0.0f ? 1.0f / std::sqrt(static_cast<float>(cache->head_dim)) : sc.scale;
    a.cap = sc.softcap > 0.0f ? std::min(std::max(sc.softcap, 1e-20f), 0x1p120f) : 0.0f;   // beyond: all scores alike, or none capped
    a.slopes = sc.slopes;
    a.window = std::min(sc.window, kMaxTokens);   // wider than any sequence: none, and positions less it stay in 32 bits
    a.prefix = sc.prefix_lens;
    a.docs = sc.doc_starts;
    char* ws = static_cast<char*>(workspace);
    a.part_ml = reinterpret_cast<float*>(ws);
    a.unit_shares = reinterpret_cast<int*>(ws + p.ml_bytes);
    a.part_o = reinterpret_cast<float*>(ws + p.ml_bytes + p.unit_bytes);
    a.groups = p.groups;
    a.pad = p.pad;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = p.chunk ? launch_prefill(a, p, cache->head_dim, cache->format, dtype, s)
                                  : launch_decode(a, p, cache->head_dim, cache->format, dtype, s);
    return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
