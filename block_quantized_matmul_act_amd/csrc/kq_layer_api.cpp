// kq_layer_api.cpp -- the C ABI of the operators around the products of a layer
// that serves many requests: norm and quantization, attention of chunks, adapters.
// As in kq_api.cpp every argument check comes before the first HIP call, so
// invalid calls return a status without touching the runtime.
#include "../../include/kq.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "kq_act_layout.hpp"
#include "kq_layer.hpp"
#include "kq_step_check.hpp"

namespace {

using namespace kq;

constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool type_of_row(int t) { return t == KQ_T_F32 || type16(t); }

// Sizes of kq_attn_chunk and its workspace query (pointers aside)
int check_chunk(const kq_cache *c, const kq_batch *s, int64_t q_heads, int64_t window, int64_t sinks,
                int64_t max_tokens, int64_t max_len) {
    int rc = check_cache(c);
    if (rc != KQ_OK) return rc;
    rc = check_batch(s);
    if (rc < 0) return rc;
    if (q_heads < 1 || q_heads > kMaxHeads || q_heads % c->heads) return KQ_ERR_SHAPE;
    if (window < 0 || window > kMaxLen || sinks < 0 || sinks > kMaxLen) return KQ_ERR_SHAPE;
    if (max_tokens < 0 || max_tokens > kMaxLen || max_len < 0 || max_len > kMaxLen) return KQ_ERR_SHAPE;
    if (rc == KQ_OK) return KQ_OK;
    if (s->n_tokens * q_heads >= ((int64_t)1 << 31) / c->dim) return KQ_ERR_UNSUPPORTED;
    if (max_tokens == 0 || max_len == 0) return KQ_ERR_SHAPE;  // rows to compute, none expected
    const ChunkPlan p = chunk_plan(*c, *s, q_heads, window, sinks, max_tokens, max_len);
    if (p.grid > MAX_GROUPS / 2) return KQ_ERR_UNSUPPORTED;  // workgroups of up to 512 threads
    return 1;
}

int check_lora(int type, int64_t rank, int64_t n_adapters, int act_fmt, int64_t M, int64_t N, int64_t K) {
    if (!type16(type) || !bs_of(act_fmt)) return KQ_ERR_FMT;
    ActLayout L;
    if (!act_layout(act_fmt, M, K, &L)) return KQ_ERR_SHAPE;
    if (N < 0 || N > kMaxDim || n_adapters < 0 || n_adapters > kMaxDim || rank < 1) return KQ_ERR_SHAPE;
    if (rank != 8 && rank != 16 && rank != 32 && rank != 64 && rank != 128) return KQ_ERR_UNSUPPORTED;
    if (n_adapters && std::max(N, K) > kMaxBytes / rank / n_adapters) return KQ_ERR_SHAPE;
    if (M == 0 || N == 0) return KQ_OK;
    // 32 rows or more to a workgroup along a grid's second dimension; columns are counted
    // in 32 bits, outputs up to 255 past the last, inputs (in steps of up to 4096) a step
    if (M > (int64_t)65535 * 32 || N > kMaxDim - 256 || K > kMaxDim - 4096) return KQ_ERR_UNSUPPORTED;
    return 1;
}

// Successful calls by variant, as kq.h numbers them.
enum LayerVariant { V_NORM_QUANTIZE, V_CHUNK_FEW, V_CHUNK_ROWS, V_LORA_FEW, V_LORA_TILE, V_COUNT };
const char *const kNames[V_COUNT] = {"norm_quantize", "chunk_few", "chunk_rows", "lora_few", "lora_tile"};
std::atomic<uint64_t> g_count[V_COUNT];
void count_layer(int variant) { g_count[variant].fetch_add(1); }

}  // namespace

namespace kq {

ChunkPlan chunk_plan(const kq_cache &cache, const kq_batch &batch, int64_t q_heads, int64_t window, int64_t sinks,
                     int64_t max_tokens, int64_t max_len) {
    ChunkPlan p;
    const int64_t heads = cache.heads, group = q_heads / heads, dim = cache.dim;
    max_tokens = std::min(max_tokens, batch.n_tokens);
    const int64_t rows = max_tokens * group;
    // the units of a block whose sequence has `slots` slots, at most
    const auto units_of = [&](int64_t slots, int rows_shift) {
        if (window) slots = std::min(slots, window + sinks + ((int64_t)1 << rows_shift) / group + 1);
        return (slots + CHUNK_UNIT - 1) / CHUNK_UNIT + 2;
    };
    // Which blocks?  Larger ones read a tile for more rows, smaller ones spread over more of the
    // chip and cost less to begin and end.  Heads of 128, 4 waves for 128 rows or 8 for 256, us:
    // 16 prompts of 512 57/68, 8 pieces of 300 over 600 37/54, a window of 1024 over 2 pieces of 512
    // 41/50, a prompt of 1024 33/37, of 2048 59/62, 4 of them 118/110, of 4096 166/140.  Heads of
    // 256, 8 waves for 128 rows or 256: a prompt of 1024 45/63, of 2500 144/136, of 4096 318/264, 8
    // pieces of 300 over 600 73/85, 16 of 40 over 3000 121/104; in 8 bits a piece of 512 over
    // 2000 79/70.
    const bool few_among_many = 4 * batch.n_tokens < batch.n_seqs * max_tokens;
    if (rows <= 16) {
        p.waves = 0;
        p.rows_shift = 4;
    } else if (dim == 64 || (dim == 128 && (rows <= 128 || (!few_among_many && units_of(max_len, 7) <= 32)))) {
        p.waves = 4;
        p.rows_shift = 7;
    } else {
        p.waves = 8;
        p.rows_shift = 8;
        if (dim == 256) {
            const bool f8 = cache.type == KQ_T_F8;
            const bool large = batch.n_seqs * (((rows - 1) >> 8) + 1) * heads > 320 || units_of(max_len, 8) >= (f8 ? 40 : 48);
            // (16 bits: the few have no way of their own there)
            if (rows <= 128 || !large || (few_among_many && !f8)) p.rows_shift = 7;
        }
    }
    p.blocks = ((batch.n_tokens * group) >> p.rows_shift) + batch.n_seqs;
    const int64_t units = units_of(max_len, p.rows_shift), groups = p.blocks * heads;
    // Places for workgroups on the chip.  (Heads of 64 have 1024, but runs are shorter then: a prompt 90
    // -> 107 us.  The kernel for few rows has 256 to 1280, by type and head; of 8 bits and heads of 128,
    // which have 768, runs over 768 take what they take over 512, 79 us, over 1024 99.)
    const int64_t chip = p.waves == 8 ? 256 : p.waves == 4 && dim == 64 ? 768 : 512;
    // Whole blocks or runs?  Few rows: runs where blocks are fewer than places for them on the
    // chip, or long (their lengths then differ by much).  More: runs where some sequences bring far
    // fewer rows than others, or are long, or by what either way takes in units: as many turns of
    // the longest block as there are blocks to a place, against an equal share of all
    // and what the cuts and the second kernel take (some 20 units).  Whole / in runs, us: 4096
    // tokens, 8 heads of 128 139/157, 2048 61/66, 1024 37/37, 16 prompts of 512 68/81; 8 pieces
    // of 512 over 4000 slots 310/316; 2 over 32k 1067/704; one among 23 single tokens 201/123.
    const int64_t each = ((rows - 1) >> p.rows_shift) + 1;  // blocks of a sequence of max_tokens
    const int64_t there = std::min(groups, batch.n_seqs * each * heads);
    if (p.waves == 0) {
        p.runs = there < chip || units >= 64;
    } else if (few_among_many) {
        p.runs = there < 16 * chip;
    } else if (units >= 256) {
        p.runs = true;
    } else {
        // (a prompt's blocks have half the longest one's units, and long and short ones pair)
        const bool prompt = max_len < 2 * max_tokens && !window;
        const int64_t share = there * ((prompt ? units / 2 : units) + CHUNK_BEGIN) / chip;
        const int64_t turns = prompt ? std::max(units + CHUNK_BEGIN, share) : (there + chip - 1) / chip * (units + CHUNK_BEGIN);
        p.runs = there < 4 * chip && turns > share + 20;
    }
    p.runs = p.runs && units > 4;
    // (units are counted in int32, whatever the lengths; 512 threads or fewer join a block, 256 a token)
    if (p.blocks > CHUNK_RUN_BLOCKS || batch.n_tokens > MAX_GROUPS || groups > MAX_GROUPS / 2 || units_of(batch.max_pages * cache.page, p.rows_shift) + CHUNK_BEGIN > kMaxInt / groups)
        p.runs = false;
    p.grid = p.runs ? std::min(chip, groups * units / 2) : groups;
    const int64_t slot_rows = p.runs ? 2 * p.grid << p.rows_shift : 0;
    p.o_bytes = slot_rows * dim * 4;
    p.ml_end = p.o_bytes + slot_rows * 8;
    p.bytes = p.runs ? p.ml_end + (p.blocks + 1) * 4 : 0;
    return p;
}

}  // namespace kq

extern "C" {

int kq_num_layer_variants(void) { return V_COUNT; }
const char *kq_layer_variant_name(int variant) {
    return variant >= 0 && variant < V_COUNT ? kNames[variant] : nullptr;
}
uint64_t kq_layer_count(int variant) { return variant >= 0 && variant < V_COUNT ? g_count[variant].load() : 0; }
void kq_layer_count_reset(void) {
    for (auto &c : g_count) c.store(0);
}

int kq_norm_quantize(int act_fmt, int x_type, const void *x, int64_t ldx, int r_type, const void *residual,
                     int64_t ldr, void *sum, int64_t lds, const float *weight, float eps, int64_t M, int64_t K,
                     void *a_q8, hipStream_t stream) {
    const int bs = bs_of(act_fmt);
    if (!bs || !type_of_row(x_type) || ((residual || sum) && !type_of_row(r_type))) return KQ_ERR_FMT;
    ActLayout L;
    if (!act_layout(act_fmt, M, K, &L)) return KQ_ERR_SHAPE;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return KQ_ERR_SHAPE;
    // rows start 16-byte aligned: strides of 4 fp32 or 8 16-bit elements
    const auto bad_stride = [&](int type, int64_t ld) { return ld < K || ld > kMaxStride || ld % (type == KQ_T_F32 ? 4 : 8); };
    if (bad_stride(x_type, ldx) || (residual && bad_stride(r_type, ldr)) || (sum && bad_stride(r_type, lds))) return KQ_ERR_SHAPE;
    if (residual && sum == residual && lds != ldr) return KQ_ERR_SHAPE;
    if (M == 0 || K == 0) return KQ_OK;
    if (K > NORM_MAX_K) return KQ_ERR_UNSUPPORTED;
    if (!x || !a_q8) return KQ_ERR_NULL;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(sum) || !aligned16(weight) || !aligned16(a_q8)) return KQ_ERR_ALIGN;
    char *to = static_cast<char *>(a_q8);
    NormArgs a;
    a.x = static_cast<const char *>(x);
    a.residual = static_cast<const char *>(residual);
    a.sum = static_cast<char *>(sum);
    a.weight = weight;
    a.ldx = ldx;
    a.ldr = ldr;
    a.lds = lds;
    a.eps = eps;
    a.M = M;
    a.K = (int)K;
    a.qs = reinterpret_cast<int8_t *>(to);
    a.d = reinterpret_cast<float *>(to + L.d);
    a.bsums = L.bsums >= 0 ? reinterpret_cast<int16_t *>(to + L.bsums) : nullptr;
    a.alpha = L.alpha >= 0 ? reinterpret_cast<uint16_t *>(to + L.alpha) : nullptr;
    // (neither a residual nor a sum: its type is never looked at)
    if (launch_norm_quantize(a, bs, x_type, residual || sum ? r_type : KQ_T_F32, stream) != hipSuccess) return KQ_ERR_HIP;
    count_layer(V_NORM_QUANTIZE);
    return KQ_OK;
}

size_t kq_attn_chunk_workspace(const kq_cache *cache, const kq_batch *batch, int64_t q_heads, int64_t window,
                               int64_t sinks, int64_t max_tokens, int64_t max_len) {
    if (check_chunk(cache, batch, q_heads, window, sinks, max_tokens, max_len) <= 0) return 0;
    return (size_t)chunk_plan(*cache, *batch, q_heads, window, sinks, max_tokens, max_len).bytes;
}

int kq_attn_chunk(const kq_cache *cache, const kq_batch *batch, int q_type, const void *q, int64_t q_heads,
                  int64_t window, int64_t sinks, float scale, int64_t max_tokens, int64_t max_len, int out_type,
                  void *out, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int rc = check_cache(cache);
    if (rc != KQ_OK) return rc;
    if (!type16(q_type) || (cache->type != KQ_T_F8 && cache->type != q_type)) return KQ_ERR_FMT;
    if (out_type != q_type && out_type != KQ_T_F32) return KQ_ERR_FMT;
    const double to_log2 = (double)scale * cache->k_scale * 1.44269504088896340736;
    if (!(std::fabs(to_log2) <= FLT_MAX)) return KQ_ERR_SHAPE;
    rc = check_chunk(cache, batch, q_heads, window, sinks, max_tokens, max_len);
    if (rc <= 0) return rc;
    rc = check_step(cache, batch);
    if (rc != KQ_OK) return rc;
    const ChunkPlan p = chunk_plan(*cache, *batch, q_heads, window, sinks, max_tokens, max_len);
    if (!q || !out || (p.bytes && !workspace)) return KQ_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return KQ_ERR_ALIGN;
    if (workspace_bytes < (size_t)p.bytes) return KQ_ERR_SHAPE;
    const float c = (float)to_log2;
    ChunkArgs k = {};
    AttnArgs &a = k.a;
    a.cache = cache_args(cache);
    a.batch = batch_args(batch);
    a.q = static_cast<const char *>(q);
    a.group = (int)(q_heads / cache->heads);
    a.q_keep = c == 0.f ? 0u : ~0u;
    a.q_flip = c < 0.f ? 0x80008000u : 0u;
    a.score_scale = c == 0.f ? 1.f : std::fabs(c);
    a.v_scale = cache->v_scale;
    a.out_f32 = out_type == KQ_T_F32;
    a.out = static_cast<char *>(out);
    a.ws_o = static_cast<float *>(workspace);
    a.ws_ml = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.o_bytes);
    k.window = window ? (int)window : INT32_MAX;
    k.sinks = window ? (int)sinks : 0;
    a.ws_seq = p.runs ? reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + p.ml_end) : nullptr;
    a.grid = (int)p.grid;
    k.rows_shift = p.rows_shift;
    k.blocks = (int)p.blocks;
    k.runs = p.runs;
    k.begin = p.waves ? CHUNK_BEGIN : 0;
    if (launch_chunk(k, p, cache->type, cache->dim, q_type, stream) != hipSuccess) return KQ_ERR_HIP;
    count_layer(p.waves == 0 ? V_CHUNK_FEW : V_CHUNK_ROWS);
    return KQ_OK;
}

size_t kq_lora_workspace(int64_t rank, int64_t M) {
    if (M < 1 || M > kMaxDim || rank < 1 || rank > 128) return 0;
    return (size_t)(M * rank * 4);
}

int kq_lora(int type, int64_t rank, const void *A, const void *B, const float *scale, int64_t n_adapters, int act_fmt,
            const void *a_q8, int64_t M, int64_t N, int64_t K, const int32_t *ids, const float *base, int64_t ldb,
            float *out, int64_t ldo, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const int rc = check_lora(type, rank, n_adapters, act_fmt, M, N, K);
    if (rc < 0) return rc;
    if (ldo < N || ldo > kMaxStride || (base && (ldb < N || ldb > kMaxStride))) return KQ_ERR_SHAPE;
    if (base && base == out && ldb != ldo) return KQ_ERR_SHAPE;
    if (rc == KQ_OK) return KQ_OK;
    if (!a_q8 || !ids || !out || !workspace || (n_adapters && (!A || !B))) return KQ_ERR_NULL;
    if (!aligned16(A) || !aligned16(B) || !aligned16(a_q8) || !aligned16(workspace) || !aligned(scale, 4) ||
        !aligned(ids, 4) || !aligned(base, 4) || !aligned(out, 4))
        return KQ_ERR_ALIGN;
    if (workspace_bytes < kq_lora_workspace(rank, M)) return KQ_ERR_SHAPE;
    ActLayout L;
    act_layout(act_fmt, M, K, &L);
    LoraArgs a;
    a.A = static_cast<const char *>(A);
    a.B = static_cast<const char *>(B);
    a.scale = scale;
    a.n_adapters = (int)n_adapters;
    a.rank = (int)rank;
    a.qs = static_cast<const int8_t *>(a_q8);
    a.d = reinterpret_cast<const float *>(static_cast<const char *>(a_q8) + L.d);
    a.bs = bs_of(act_fmt);
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.ids = ids;
    a.base = base;
    a.ldb = ldb;
    a.out = out;
    a.ldo = ldo;
    a.t = static_cast<float *>(workspace);
    if (launch_lora(a, type, stream) != hipSuccess) return KQ_ERR_HIP;
    count_layer(lora_few(M, rank) ? V_LORA_FEW : V_LORA_TILE);
    return KQ_OK;
}

}  // extern "C"
