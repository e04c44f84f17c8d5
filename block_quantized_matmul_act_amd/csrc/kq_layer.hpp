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
// alone (some numbers stay unused).  A workgroup takes a block, or (runs) `grid`
// workgroups take equal runs of units of CHUNK_UNIT slots (or 2) of all the blocks and leave at
// most two cut blocks each, a slot of the workspace to either.
constexpr int CHUNK_UNIT_SHIFT = 6, CHUNK_UNIT = 1 << CHUNK_UNIT_SHIFT;
constexpr int CHUNK_BEGIN = 6;  // what the begin and end of a block of many rows take, in units
constexpr int CHUNK_RUN_BLOCKS = 1024;  // block numbers of a key head in a call of runs (2048 take a workgroup of 4 waves its place)
struct ChunkPlan {
    int waves;  // 0: the kernel for up to 16 rows
    int rows_shift;
    bool runs;
    int64_t blocks;  // numbers, for one key head
    int64_t grid;    // workgroups
    // workspace: sums, their maxima and weights (to ml_end), the units before each block
    int64_t o_bytes, ml_end, bytes;
};
ChunkPlan chunk_plan(const kq_cache &cache, const kq_batch &batch, int64_t q_heads, int64_t window, int64_t sinks,
                     int64_t max_tokens, int64_t max_len);
struct ChunkArgs {
    AttnArgs a;
    int window, sinks;  // window: INT32_MAX where there is none
    int rows_shift, blocks, runs;
    int begin;      // units that the begin and end of a block count for
    int few_shift;  // units of a block of 16 rows or fewer: 1 << few_shift slots (set by the launcher)
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
// Few rows: a wave to a value of t and to 64 outputs of a row, whatever adapters the rows
// have.  More: tiles of rows, an adapter of a tile after another.  The ids lie on the device, so
// the bound counts on prompts: past it rows of one adapter gain up to 16 us, and rows with
// one each lose 20 to 57.  rows x outputs of 4096 inputs, us of a call, few / tiles (13.4: the
// call on the host), every row with an adapter of its own, and all with one:
//   rank 16:  256 x 14336  18.8/44.5 17.8/13.5   256 x 4096  13.4/40.0 13.6/13.5
//             512 x 14336  30.7/56.7 29.6/15.9   512 x 4096  15.9/40.5 15.5/13.8
//   rank 64:   96 x 14336  37.1/94.5 18.4/15.4    96 x 4096  16.5/65.0 13.6/13.9
//             256 x 14336  77.7/109  34.0/18.5   256 x 4096  22.1/64.9 17.6/14.4
inline bool lora_few(int64_t M, int64_t rank) { return M * rank <= 4096; }
hipError_t launch_lora(const LoraArgs &a, int type, hipStream_t stream);

}  // namespace kq
