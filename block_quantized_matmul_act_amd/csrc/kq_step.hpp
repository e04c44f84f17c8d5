// kq_step.hpp -- launchers of the kernels between two products of a layer
// (paged cache, attention over it, log probabilities), and the rules that cut
// their work, shared by the launchers and the workspace queries.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/kq.h"

namespace kq {

// The device arrays and sizes of a cache and a step, as kernels take them.
struct CacheArgs {
    char *k, *v;
    int64_t n_pages;
    int heads, page_shift;  // page = 1 << page_shift tokens
};
struct BatchArgs {
    const int32_t *offsets, *lens, *pages;
    int n_seqs, n_tokens, max_pages;
};

// Slots of a sequence: with as many rows of a step still an int.
constexpr int MAX_LEN = 1 << 30;

// A launch counts its threads along a dimension in 32 bits, and workgroups here
// have at least this many.
constexpr int64_t MAX_GROUPS = UINT32_MAX / 256;

struct RopeArgs {
    CacheArgs cache;
    BatchArgs batch;
    const float *x;
    int64_t ldx;
    int q_heads;
    const float *q_norm, *k_norm;
    float eps, k_inv, v_inv;  // 1 / scale
    const float *rope;
    int n_pos, rot, pairs;
    const int32_t *positions;
    char *q;
};
// How many rows of values a workgroup takes and how many groups of 512 / dim heads a
// wave.  Fewer values: as many waves and tiles as there can be.  More: tiles of 64
// rows, of which all but the ends are whole runs, and two groups of heads to a wave
// (1k rows of 48 heads of 128: 11 us and 14; 2k of 40: 18 and 16; 12k of 40: 105 and 93).
struct RopePlan {
    int tile, groups;
    int64_t value_blocks, blocks;  // workgroups of values, and all
};
inline RopePlan rope_plan(int64_t n_tokens, int64_t q_heads, int64_t heads, int dim) {
    RopePlan p;
    const bool few = n_tokens * (q_heads + heads) * dim < (1 << 23);
    p.tile = few ? 16 : 64;
    p.groups = few ? 1 : 2;
    const int64_t wave_heads = 512 / dim * p.groups, waves = (q_heads + heads + wave_heads - 1) / wave_heads;
    p.value_blocks = (n_tokens + p.tile - 1) / p.tile * heads;
    p.blocks = p.value_blocks + (waves * n_tokens + 3) / 4;
    return p;
}
// type / q_type: KQ_T_*; dim: 64, 128 or 256 (checked by the caller)
hipError_t launch_rope_append(const RopeArgs &a, int type, int dim, int q_type, hipStream_t stream);

// How attention over the cache is shared out: `waves` waves (0: the kernel for
// up to 16 rows) hold rows_wg query rows, `grid` workgroups take equal runs of
// units of 2^unit_shift slots and leave at most two cut blocks each (slot_rows rows
// of the workspace to a block).
constexpr int ATTN_UNIT_SHIFT = 7, ATTN_UNIT = 1 << ATTN_UNIT_SHIFT;
constexpr int ATTN_WHOLE_SHIFT = 10, ATTN_WHOLE = 1 << ATTN_WHOLE_SHIFT;  // short sequences that are not cut
struct AttnPlan {
    int waves, rows_wg, row_blocks, slot_rows, grid, unit_shift;
    // workspace: sums, their maxima and weights (to ml_end), 16 bytes to a sequence
    int64_t o_bytes, ml_end, bytes;
};
AttnPlan attn_plan(const kq_cache &cache, int64_t n_seqs, int64_t q_heads, int64_t max_tokens, int64_t max_len);

struct AttnArgs {
    CacheArgs cache;
    BatchArgs batch;
    const char *q;
    int group;
    const uint64_t *mask;
    // scores are (q & q_keep ^ q_flip) . k * score_scale in log2 units, score_scale
    // > 0: a negative scale flips the signs of q, a zero one clears q
    uint32_t q_keep, q_flip;
    float score_scale, v_scale;
    int max_tokens, max_len;
    int out_f32;
    char *out;
    float *ws_o, *ws_ml;
    int32_t *ws_seq;
    int rows_wg, slot_rows, grid, unit_shift;
};
hipError_t launch_attn(const AttnArgs &a, const AttnPlan &p, int type, int dim, int q_type, hipStream_t stream);

constexpr int KEEP_CACHES = 64;  // caches to a launch (their pointers are kernel arguments)
struct KeepArgs {
    char *k[KEEP_CACHES], *v[KEEP_CACHES];
    CacheArgs cache;
    BatchArgs batch;
    const int32_t *path, *counts;
};
hipError_t launch_keep(const KeepArgs &a, int n_caches, int elem_bytes, int dim, hipStream_t stream);

// Rows of logits cut into parts of `part` values (parts = 1: one workgroup to
// a row and no second kernel).
struct LogprobsPlan {
    int part, parts;
    int64_t bytes;
};
LogprobsPlan logprobs_plan(int64_t M, int64_t V, int64_t n_top);

struct LogprobsArgs {
    const char *x;
    int64_t ldx;
    int V, part, parts;
    const int32_t *tokens;
    int n_given, n_top;
    float *logprob, *entropy;
    int32_t *top_ids;
    float *top_logprobs;
    char *ws;
};
hipError_t launch_logprobs(const LogprobsArgs &a, int type, int64_t M, hipStream_t stream);

}  // namespace kq
