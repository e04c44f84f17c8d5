// kq_layer.hpp -- launchers of the operators around the products of a layer that
// serves many requests (norm and quantization, attention of chunks, adapters), and
// the rules that cut their work, shared by the launchers and the workspace queries.
#pragma once

#include "kq_step.hpp"

namespace kq {

struct NormArgs {
    const char *x;
    const char *residual;  // or NULL
    char *sum;             // or NULL
    const float *weight;   // or NULL
    int64_t ldx, ldr, lds;  // in elements
    float eps;
    int64_t M;
    int K;
    int8_t *qs;
    float *d;
    int16_t *bsums;
    uint16_t *alpha;
};
constexpr int64_t NORM_MAX_K = 65536;  // a row is held in the registers of one workgroup
// bs: values to a scale; x_type / r_type: KQ_T_*
hipError_t launch_norm_quantize(const NormArgs &a, int bs, int x_type, int r_type, hipStream_t stream);

// How attention of chunks is shared out: blocks of 1 << rows_shift query rows of a
// key head, numbered so that a block's sequence can be found from the offsets
// alone (some numbers stay unused); a block's keys, in units of CHUNK_UNIT slots, are
// cut into at most `parts` parts of `part_units` units or more.
constexpr int CHUNK_UNIT_SHIFT = 6, CHUNK_UNIT = 1 << CHUNK_UNIT_SHIFT;
struct ChunkPlan {
    int waves;  // 0: the kernel for up to 16 rows
    int rows_shift, parts, part_units;
    int64_t blocks;                 // numbers, for one key head
    int64_t o_bytes, bytes;         // workspace: sums, then their maxima and weights
};
ChunkPlan chunk_plan(const kq_cache &cache, int64_t n_seqs, int64_t n_tokens, int64_t q_heads, int64_t window,
                     int64_t sinks, int64_t max_tokens, int64_t max_len);
struct ChunkArgs {
    AttnArgs a;
    int window, sinks;  // window: INT32_MAX where there is none
    int rows_shift, blocks, parts, part_units;
};
hipError_t launch_chunk(const ChunkArgs &a, const ChunkPlan &p, int type, int dim, int q_type, hipStream_t stream);

struct LoraArgs {
    const char *A, *B;
    const float *scale;  // or NULL
    int n_adapters, rank;
    const int8_t *qs;
    const float *d;
    int bs;  // values to a scale
    int M, N, K;
    const int32_t *ids;
    const float *base;  // or NULL
    int64_t ldb;
    float *out;
    int64_t ldo;
    float *t;  // [M][rank]
};
bool lora_few(int64_t M);
hipError_t launch_lora(const LoraArgs &a, int type, hipStream_t stream);

}  // namespace kq
