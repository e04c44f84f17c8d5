// kq_step_api.cpp -- the C ABI between two products of a layer: the paged
// cache, the attention over it and the log probabilities.  As in kq_api.cpp
// every argument check comes before the first HIP call, so invalid calls return
// a status without touching the runtime.
#include "../../include/kq.h"

#include <atomic>
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "kq_step.hpp"
#include "kq_step_check.hpp"

namespace {

using namespace kq;

// Sizes of kq_attn_tree and its workspace query (pointers aside)
int check_attn(const kq_cache *c, const kq_batch *s, int64_t q_heads, int64_t max_tokens, int64_t max_len) {
    int rc = check_cache(c);
    if (rc != KQ_OK) return rc;
    rc = check_batch(s);
    if (rc < 0) return rc;
    if (q_heads < 1 || q_heads > kMaxHeads || q_heads % c->heads) return KQ_ERR_SHAPE;
    if (max_tokens < 0 || max_len < 0 || max_len > kMaxLen) return KQ_ERR_SHAPE;
    if (max_tokens > KQ_ATTN_MAX_TOKENS) return KQ_ERR_UNSUPPORTED;
    if (rc == KQ_OK) return KQ_OK;
    if (s->n_tokens * q_heads >= ((int64_t)1 << 31) / c->dim) return KQ_ERR_UNSUPPORTED;
    if (max_tokens == 0 || max_len == 0) return KQ_ERR_SHAPE;  // rows to compute, none allowed
    if (s->n_tokens > s->n_seqs * max_tokens) return KQ_ERR_SHAPE;  // some sequence has more
    // the kernels count units in int32: at most a row block to every 16 rows
    const int64_t blocks = (max_tokens * (q_heads / c->heads) + 15) / 16;
    if (s->n_seqs > kMaxInt / (c->heads * ((max_len + ATTN_UNIT - 1) / ATTN_UNIT) * blocks)) return KQ_ERR_UNSUPPORTED;
    return 1;
}

// Successful calls by variant, as kq.h numbers them.
enum StepVariant { V_ROPE_APPEND, V_ATTN_FEW, V_ATTN_ROWS, V_CACHE_KEEP, V_LOGPROBS_ROW, V_LOGPROBS_PARTS, V_COUNT };
const char *const kNames[V_COUNT] = {"rope_append", "attn_few", "attn_rows", "cache_keep", "logprobs_row", "logprobs_parts"};
std::atomic<uint64_t> g_count[V_COUNT];
void count_step(int variant) { g_count[variant].fetch_add(1); }

}  // namespace

namespace kq {

AttnPlan attn_plan(const kq_cache &cache, int64_t n_seqs, int64_t q_heads, int64_t max_tokens, int64_t max_len) {
    AttnPlan p;
    const int64_t heads = cache.heads, group = q_heads / heads, dim = cache.dim;
    // Waves of 32 rows, at dim 256 of 16 (whose sums and operands fit the
    // registers); 8 of them where there are rows for more than 4 (96 rows: 103 us
    // with 4, 124 with 8), and at dim 256.
    const int64_t rows = max_tokens * group;
    const int rows_wave = dim == 256 ? 16 : 32;
    p.waves = rows <= 16 ? 0 : rows <= 4 * rows_wave && dim < 256 ? 4 : 8;
    p.rows_wg = p.waves ? p.waves * rows_wave : 16;
    p.row_blocks = (int)((rows + p.rows_wg - 1) / p.rows_wg);
    p.slot_rows = (int)std::min<int64_t>(rows, p.rows_wg);
    // Workgroups: as many as stay on 256 compute units together (8 waves each),
    // or the units there can be.
    p.unit_shift = ATTN_UNIT_SHIFT;
    // Few rows of short sequences, no more of them than compute units: a workgroup
    // of 8 waves takes a head's keys whole, and no second kernel is launched.  In
    // parts / whole, 8 heads, us of a call from Python and (of the kernels alone):
    //                       250 slots               500                     1000
    //   bf16, 64:   1 seq  13.7/10.0 (10.0/ 6.4)   13.8/ 9.8 (10.0/ 7.2)   13.5/ 9.8 ( 9.9/ 8.8)
    //               8      13.5/ 9.7 (10.2/ 6.4)   13.6/ 9.7 (10.1/ 7.3)   13.3/10.0 (11.7/ 9.9)
    //              32      13.2/ 9.6 (12.1/ 6.6)   13.4/ 9.5 (13.2/ 8.5)   19.4/14.7 (19.6/15.0)
    //   bf16, 128:  1      13.3/ 9.6 ( 9.7/ 8.0)   13.6/ 9.7 ( 9.8/ 9.5)   13.5/12.2 ( 9.8/12.1)
    //               8      13.6/ 9.7 (10.0/ 8.0)   13.3/11.0 (10.1/11.0)   13.3/16.1 (12.5/16.1)
    //              32      13.5/ 9.5 (13.3/ 9.2)   19.6/15.8 (19.7/16.0)   28.7/24.9 (28.7/25.1)
    //   f8, 64:     1      13.2/ 9.6 ( 9.2/ 5.4)   13.6/ 9.8 ( 9.2/ 6.1)   13.7/ 9.7 ( 9.1/ 7.4)
    //              32      13.3/ 9.8 (11.1/ 5.5)   13.3/ 9.5 (11.3/ 6.6)   13.5/ 9.5 (13.3/ 8.5)
    //   f8, 128:    1      13.5/ 9.7 ( 9.9/ 7.2)   13.6/ 9.7 (10.0/ 8.1)   13.5/10.5 (10.1/10.3)
    //              32      13.2/ 9.5 (12.9/ 7.5)   13.9/ 9.5 (13.9/ 9.4)   20.1/15.9 (20.2/16.1)
    // It loses towards 1000 slots of 16-bit heads of 128 in few sequences (the rate of
    // one compute unit), in a captured step from 500 on; 2000 slots of one sequence
    // 15.6 / 20.1; more than 256 heads: 200 sequences of 500 62 / 76.  (At dim 256 8
    // waves' sums do not fit the registers.)
    if (p.waves == 0 && max_len > ATTN_UNIT && max_len <= ATTN_WHOLE && n_seqs * heads <= 256 && dim < 256)
        p.unit_shift = ATTN_WHOLE_SHIFT;
    const int unit = 1 << p.unit_shift;
    const int64_t units = n_seqs * heads * p.row_blocks * ((max_len + unit - 1) / unit);
    p.grid = (int)std::min<int64_t>(units, p.waves == 8 ? 256 : 512);
    const int64_t slots = max_len > unit ? 2 * (int64_t)p.grid * p.slot_rows : 0;
    p.o_bytes = slots * dim * 4;
    p.ml_end = p.o_bytes + (slots + (slots & 1)) * 8;
    p.bytes = slots ? p.ml_end + n_seqs * 16 : 0;
    return p;
}

LogprobsPlan logprobs_plan(int64_t M, int64_t V, int64_t n_top) {
    LogprobsPlan p;
    // 4096 values (a batch to each wave of a workgroup) at least, and no more
    // parts than give each compute unit a few workgroups
    const int64_t want = std::max<int64_t>(1, 1024 / std::max<int64_t>(1, M));
    int64_t part = (V + want - 1) / want;
    part = std::max<int64_t>(4096, (part + 4095) / 4096 * 4096);
    p.part = (int)std::min<int64_t>(part, kMaxInt / 2 + 1);
    p.parts = (int)std::max<int64_t>(1, (V + p.part - 1) / p.part);
    p.bytes = p.parts > 1 ? (M * p.parts * 12 + 7) / 8 * 8 + M * p.parts * 8 * n_top : 0;
    return p;
}

}  // namespace kq

extern "C" {

int kq_num_step_variants(void) { return V_COUNT; }
const char *kq_step_variant_name(int variant) {
    return variant >= 0 && variant < V_COUNT ? kNames[variant] : nullptr;
}
uint64_t kq_step_count(int variant) { return variant >= 0 && variant < V_COUNT ? g_count[variant].load() : 0; }
void kq_step_count_reset(void) {
    for (auto &c : g_count) c.store(0);
}

int kq_rope_append(const kq_cache *cache, const kq_batch *batch, const float *x, int64_t ldx, int64_t q_heads,
                   const float *q_norm, const float *k_norm, float eps, const float *rope, int64_t n_pos,
                   int64_t rot_dim, int pairs, const int32_t *positions, int q_type, void *q, hipStream_t stream) {
    int rc = check_cache(cache);
    if (rc != KQ_OK) return rc;
    if (!type16(q_type) || (cache->type != KQ_T_F8 && cache->type != q_type)) return KQ_ERR_FMT;
    const int work = check_batch(batch);
    if (work < 0) return work;
    if (q_heads < 1 || q_heads > kMaxHeads) return KQ_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim > cache->dim || rot_dim % 8 || n_pos < 0 || n_pos > kMaxInt) return KQ_ERR_SHAPE;
    if (rot_dim && n_pos == 0 && work == 1) return KQ_ERR_SHAPE;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return KQ_ERR_SHAPE;
    const float k_inv = 1.0f / cache->k_scale, v_inv = 1.0f / cache->v_scale;
    if (!std::isfinite(k_inv) || !std::isfinite(v_inv)) return KQ_ERR_SHAPE;  // (0 times infinity were NaN)
    if (ldx % 4 || ldx < (q_heads + 2 * (int64_t)cache->heads) * cache->dim || ldx > kMaxLen) return KQ_ERR_SHAPE;
    if (work == KQ_OK) return KQ_OK;
    rc = check_step(cache, batch);
    if (rc != KQ_OK) return rc;
    if (!x || !q || (rot_dim && !rope)) return KQ_ERR_NULL;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(rope, 16) || !aligned(q_norm, 16) || !aligned(k_norm, 16) ||
        !aligned(positions, 4))
        return KQ_ERR_ALIGN;
    // waves are counted in int32: at most one to a head and row
    if (batch->n_tokens > kMaxInt / (q_heads + 2 * cache->heads) ||
        rope_plan(batch->n_tokens, q_heads, cache->heads, cache->dim).blocks > MAX_GROUPS)
        return KQ_ERR_UNSUPPORTED;
    RopeArgs a;
    a.cache = cache_args(cache);
    a.batch = batch_args(batch);
    a.x = x;
    a.ldx = ldx;
    a.q_heads = (int)q_heads;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    a.k_inv = k_inv;
    a.v_inv = v_inv;
    a.rope = rope;
    a.n_pos = (int)n_pos;
    a.rot = (int)rot_dim;
    a.pairs = pairs != 0;
    a.positions = positions;
    a.q = static_cast<char *>(q);
    if (launch_rope_append(a, cache->type, cache->dim, q_type, stream) != hipSuccess) return KQ_ERR_HIP;
    count_step(V_ROPE_APPEND);
    return KQ_OK;
}

size_t kq_attn_tree_workspace(const kq_cache *cache, const kq_batch *batch, int64_t q_heads, int64_t max_tokens,
                              int64_t max_len) {
    if (check_attn(cache, batch, q_heads, max_tokens, max_len) <= 0) return 0;
    return (size_t)attn_plan(*cache, batch->n_seqs, q_heads, max_tokens, max_len).bytes;
}

int kq_attn_tree(const kq_cache *cache, const kq_batch *batch, int q_type, const void *q, int64_t q_heads,
                 const uint64_t *mask, float scale, int64_t max_tokens, int64_t max_len, int out_type, void *out,
                 void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int rc = check_cache(cache);
    if (rc != KQ_OK) return rc;
    if (!type16(q_type) || (cache->type != KQ_T_F8 && cache->type != q_type)) return KQ_ERR_FMT;
    if (out_type != q_type && out_type != KQ_T_F32) return KQ_ERR_FMT;
    const double to_log2 = (double)scale * cache->k_scale * 1.44269504088896340736;
    if (!(std::fabs(to_log2) <= FLT_MAX)) return KQ_ERR_SHAPE;
    const float c = (float)to_log2;
    rc = check_attn(cache, batch, q_heads, max_tokens, max_len);
    if (rc <= 0) return rc;
    rc = check_step(cache, batch);
    if (rc != KQ_OK) return rc;
    const AttnPlan p = attn_plan(*cache, batch->n_seqs, q_heads, max_tokens, max_len);
    if (p.bytes && batch->n_tokens > MAX_GROUPS) return KQ_ERR_UNSUPPORTED;  // a workgroup to a row joins the parts
    if (!q || !out || (p.bytes && !workspace)) return KQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(mask, 8) || !aligned(workspace, 16)) return KQ_ERR_ALIGN;
    if (workspace_bytes < (size_t)p.bytes) return KQ_ERR_SHAPE;
    AttnArgs a;
    a.cache = cache_args(cache);
    a.batch = batch_args(batch);
    a.q = static_cast<const char *>(q);
    a.group = (int)(q_heads / cache->heads);
    a.mask = mask;
    a.q_keep = c == 0.f ? 0u : ~0u;
    a.q_flip = c < 0.f ? 0x80008000u : 0u;
    a.score_scale = c == 0.f ? 1.f : std::fabs(c);
    a.v_scale = cache->v_scale;
    a.max_tokens = (int)max_tokens;
    a.max_len = (int)max_len;
    a.out_f32 = out_type == KQ_T_F32;
    a.out = static_cast<char *>(out);
    a.ws_o = static_cast<float *>(workspace);
    a.ws_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.o_bytes);
    a.ws_seq = p.bytes ? reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + p.ml_end) : nullptr;
    a.rows_wg = p.rows_wg;
    a.slot_rows = p.slot_rows;
    a.grid = p.grid;
    a.unit_shift = p.unit_shift;
    if (launch_attn(a, p, cache->type, cache->dim, q_type, stream) != hipSuccess) return KQ_ERR_HIP;
    count_step(p.waves == 0 ? V_ATTN_FEW : V_ATTN_ROWS);
    return KQ_OK;
}

int kq_cache_keep(const kq_cache *caches, int64_t n_caches, const kq_batch *batch, const int32_t *path,
                  const int32_t *counts, hipStream_t stream) {
    if (n_caches < 0 || n_caches > kMaxInt) return KQ_ERR_SHAPE;
    if (n_caches && !caches) return KQ_ERR_NULL;
    for (int64_t i = 0; i < n_caches; ++i) {
        const int rc = check_cache(caches + i);
        if (rc != KQ_OK) return rc;
        const kq_cache &c = caches[i], &d = caches[0];
        if (c.type != d.type || c.heads != d.heads || c.dim != d.dim || c.page != d.page || c.n_pages != d.n_pages)
            return KQ_ERR_SHAPE;
    }
    int rc = check_batch(batch);
    if (rc <= 0) return rc;
    if (n_caches == 0) return KQ_OK;
    if (batch->n_seqs > MAX_GROUPS) return KQ_ERR_UNSUPPORTED;  // a workgroup to a sequence (and head and cache)
    for (int64_t i = 0; i < n_caches; ++i) {
        rc = check_step(caches + i, batch);
        if (rc != KQ_OK) return rc;
    }
    if (!path || !counts) return KQ_ERR_NULL;
    if (!aligned(path, 4) || !aligned(counts, 4)) return KQ_ERR_ALIGN;
    KeepArgs a;
    a.cache = cache_args(caches);
    a.batch = batch_args(batch);
    a.path = path;
    a.counts = counts;
    for (int64_t i = 0; i < n_caches; i += KEEP_CACHES) {
        const int n = (int)std::min<int64_t>(KEEP_CACHES, n_caches - i);
        for (int j = 0; j < KEEP_CACHES; ++j) {
            a.k[j] = static_cast<char *>(caches[i + (j < n ? j : 0)].k);
            a.v[j] = static_cast<char *>(caches[i + (j < n ? j : 0)].v);
        }
        if (launch_keep(a, n, caches->type == KQ_T_F8 ? 1 : 2, caches->dim, stream) != hipSuccess) return KQ_ERR_HIP;
        count_step(V_CACHE_KEEP);
    }
    return KQ_OK;
}

size_t kq_logprobs_workspace(int64_t M, int64_t V, int64_t n_top) {
    if (M < 1 || V < 1 || M > kMaxInt || V > kMaxLen || n_top < 0 || n_top > KQ_LOGPROBS_MAX_TOP || n_top > V) return 0;
    return (size_t)logprobs_plan(M, V, n_top).bytes;
}

int kq_logprobs(int type, const void *logits, int64_t M, int64_t V, int64_t ldx, const int32_t *tokens,
                int64_t n_given, int64_t n_top, float *logprob, float *entropy, int32_t *top_ids, float *top_logprobs,
                void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (type != KQ_T_F32 && type != KQ_T_BF16 && type != KQ_T_F16) return KQ_ERR_FMT;
    if (M < 0 || V < 0 || n_given < 0 || n_top < 0 || M > kMaxInt || V > kMaxLen || n_given > kMaxInt) return KQ_ERR_SHAPE;
    if (ldx < V || ldx > ((int64_t)1 << 40)) return KQ_ERR_SHAPE;
    if (M == 0) return KQ_OK;
    if (V == 0 || n_top > V) return KQ_ERR_SHAPE;
    if (n_top > KQ_LOGPROBS_MAX_TOP) return KQ_ERR_UNSUPPORTED;
    const LogprobsPlan p = logprobs_plan(M, V, n_top);
    if (M > MAX_GROUPS / p.parts) return KQ_ERR_UNSUPPORTED;  // a workgroup to a part
    if (!logits || (n_given && (!tokens || !logprob)) || (n_top && (!top_ids || !top_logprobs)) ||
        (p.bytes && !workspace))
        return KQ_ERR_NULL;
    if (!aligned(logits, type == KQ_T_F32 ? 4 : 2) || !aligned(tokens, 4) || !aligned(logprob, 4) ||
        !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4) || !aligned(workspace, 16))
        return KQ_ERR_ALIGN;
    if (workspace_bytes < (size_t)p.bytes) return KQ_ERR_SHAPE;
    LogprobsArgs a;
    a.x = static_cast<const char *>(logits);
    a.ldx = ldx;
    a.V = (int)V;
    a.part = p.part;
    a.parts = p.parts;
    a.tokens = tokens;
    a.n_given = (int)n_given;
    a.n_top = (int)n_top;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.ws = static_cast<char *>(workspace);
    if (launch_logprobs(a, type, M, stream) != hipSuccess) return KQ_ERR_HIP;
    count_step(p.parts == 1 ? V_LOGPROBS_ROW : V_LOGPROBS_PARTS);
    return KQ_OK;
}

}  // extern "C"
