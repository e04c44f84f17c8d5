// Host-side driver of the argument handling of the operators around the products of
// a layer (kq_layer_api.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_layer_abi.py.  The launchers are stubs
// that hold what they get to what the kernels assume, so every entry point runs on
// extreme sizes (a signed overflow in a size computation is reported).  The numbers
// that attention of chunks gives to blocks are checked over random batches.  Prints
// "ok" and exits 0 when every expectation holds.
#include "../../include/kq.h"

#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "../../block_quantized_matmul_act_amd/csrc/kq_layer.hpp"

namespace {
int failures = 0, norms = 0, chunks = 0, loras = 0;
#define EXPECT(c)                                                        \
    do {                                                                 \
        if (!(c)) {                                                      \
            std::fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c); \
            ++failures;                                                  \
        }                                                                \
    } while (0)
char *const P = reinterpret_cast<char *>((uintptr_t)1 << 20);
constexpr int64_t THREADS = UINT32_MAX;
kq::NormArgs norm;
kq::ChunkPlan plan;
}  // namespace

namespace kq {
hipError_t launch_norm_quantize(const NormArgs &a, int bs, int, int, hipStream_t) {
    ++norms;
    norm = a;
    EXPECT(a.M > 0 && a.K > 0 && a.K <= NORM_MAX_K && a.K % bs == 0);
    EXPECT((a.bsums != nullptr) == (bs == 256) && (a.alpha != nullptr) == (bs == 256));
    return hipSuccess;
}
hipError_t launch_chunk(const ChunkArgs &c, const ChunkPlan &p, int, int dim, int, hipStream_t) {
    ++chunks;
    plan = p;
    const int64_t heads = c.a.cache.heads;
    EXPECT(p.grid >= 1 && p.grid * (p.waves == 8 ? 512 : 256) <= THREADS);
    EXPECT(p.runs == (p.bytes != 0) && p.runs == (c.runs != 0) && c.window >= 1);
    if (p.runs) {
        // units of every length that the pages hold fit an int, block numbers the kernels' arrays
        const int64_t slots = ((int64_t)c.a.batch.max_pages << c.a.cache.page_shift);
        const int64_t most = slots < (int64_t)c.window + c.sinks + 300 ? slots : (int64_t)c.window + c.sinks + 300;
        EXPECT(p.blocks <= CHUNK_RUN_BLOCKS && p.grid <= 768);
        EXPECT(p.blocks * heads * (most / CHUNK_UNIT) <= INT32_MAX);
        EXPECT(p.blocks * heads * 512 <= THREADS && c.a.batch.n_tokens * (int64_t)256 <= THREADS);
        EXPECT(p.o_bytes == (2 * p.grid << p.rows_shift) * dim * 4 && p.ml_end == p.o_bytes + (2 * p.grid << p.rows_shift) * 8);
        EXPECT(p.bytes == p.ml_end + (p.blocks + 1) * 4 && p.ml_end % 16 == 0);
    } else {
        EXPECT(p.grid == p.blocks * heads);
    }
    EXPECT(p.rows_shift == (p.waves == 0 ? 4 : p.waves == 4 ? 7 : 8) || (p.waves == 8 && dim == 256 && p.rows_shift == 7));
    EXPECT(!(p.waves == 4 && dim == 256));
    return hipSuccess;
}
hipError_t launch_lora(const LoraArgs &a, int, hipStream_t) {
    ++loras;
    EXPECT(a.M > 0 && a.N > 0 && a.N <= INT32_MAX - 256);
    EXPECT((a.M + 31) / 32 <= 65535);
    EXPECT(((int64_t)a.N + 127) / 128 * 256 <= THREADS);
    EXPECT(((int64_t)a.M + 15) / 16 * 512 <= THREADS);
    return hipSuccess;
}
}  // namespace kq

int main() {
    const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 7, 128, 256, 512, 4096, 65536, 65792, INT32_MAX - 1, INT32_MAX,
                             (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX};
    const float *F = reinterpret_cast<const float *>(P);
    float *W = reinterpret_cast<float *>(P);
    const int32_t *I = reinterpret_cast<const int32_t *>(P);
    for (int64_t M : sizes)
        for (int64_t K : sizes)
            for (int64_t ld : sizes) {
                kq_norm_quantize(KQ_ACT_Q8_K, KQ_T_F32, P, ld, KQ_T_BF16, P, ld, P, ld, F, 0.f, M, K, P, nullptr);
                kq_norm_quantize(KQ_ACT_Q8_128, KQ_T_F16, P, ld, KQ_T_F32, nullptr, ld, P, K, nullptr, 1.f, M, K, P, nullptr);
                for (int64_t n : sizes) {
                    kq_lora(KQ_T_F16, 8, P, P, F, n, KQ_ACT_Q8_K, P, M, ld, K, I, F, ld, W, ld, P, SIZE_MAX, nullptr);
                    kq_lora(KQ_T_BF16, 128, P, P, F, 3, KQ_ACT_Q8_128, P, M, n, K, I, nullptr, 0, W, ld, P, SIZE_MAX, nullptr);
                }
                kq_lora_workspace(M, K);
                kq_cache c = {P, P, 100, KQ_T_BF16, 8, 128, 64, 1.f, 1.f};
                kq_batch s = {I, I, I, M, K, 100};
                for (int64_t w : sizes) {
                    kq_attn_chunk(&c, &s, KQ_T_BF16, P, 32, w, ld, 1.f, ld, w, KQ_T_F32, P, P, SIZE_MAX, nullptr);
                    kq_attn_chunk(&c, &s, KQ_T_BF16, P, 8, ld, 4, 1.f, w, 4096, KQ_T_F32, P, P, SIZE_MAX, nullptr);
                    kq_attn_chunk_workspace(&c, &s, w, 0, 0, ld, 4096);
                }
            }
    EXPECT(norms > 50 && chunks > 50 && loras > 50);

    // sections as an activation buffer has them
    EXPECT(kq_norm_quantize(KQ_ACT_Q8_K, KQ_T_F32, P, 512, KQ_T_F32, P, 512, P, 512, F, 0.f, 3, 512, P, nullptr) == KQ_OK);
    EXPECT(reinterpret_cast<char *>(norm.qs) == P && reinterpret_cast<char *>(norm.d) == P + 1536);
    EXPECT(reinterpret_cast<char *>(norm.bsums) == P + 1536 + 256 && reinterpret_cast<char *>(norm.alpha) == P + 1536 + 256 + 256);

    // grids at sizes around what a launch can count
    for (int shift = 14; shift <= 30; ++shift)
        for (int64_t off = -1; off <= 1; ++off)
            for (int dim : {64, 128, 256})
                for (int heads : {1, 3, 64})
                    for (int group : {1, 5, 16})
                        for (int64_t tokens : {1, 20, 1000}) {
                            const int64_t n = ((int64_t)1 << shift) + off;
                            if (n > INT32_MAX / 2) continue;
                            kq_cache c = {P, P, 100, KQ_T_F16, heads, dim, 64, 1.f, 1.f};
                            for (int64_t seqs : {n, n / tokens + 1, (int64_t)1}) {
                                kq_batch s = {I, I, I, seqs, n, dim == 64 ? 10 : 1 << 20};
                                const int rc = kq_attn_chunk(&c, &s, KQ_T_F16, P, heads * group, 0, 0, 1.f, tokens, 4096, KQ_T_F32, P, P, SIZE_MAX, nullptr);
                                EXPECT(rc == KQ_OK || rc == KQ_ERR_UNSUPPORTED);
                            }
                        }

    // the first block of sequence b is number (offsets[b] * group >> shift) + b: every
    // block of b comes before the first of b + 1, and all before `blocks`
    std::mt19937 gen(1);
    for (int round = 0; round < 2000; ++round) {
        const int seqs = 1 + gen() % 40, group = 1 + gen() % 17, most = 1 + (1 << gen() % 10);
        std::vector<int64_t> at(1, 0);
        for (int b = 0; b < seqs; ++b) at.push_back(at.back() + gen() % (most + 1));
        if (!at.back()) continue;
        kq_cache c = {P, P, 100, KQ_T_F16, 1, 128, 64, 1.f, 1.f};
        kq_batch s = {I, I, I, seqs, at.back(), 100};
        const kq::ChunkPlan p = kq::chunk_plan(c, s, group, 0, 0, 1 + gen() % 600, 1 + gen() % 5000);
        int64_t next = 0;
        for (int b = 0; b < seqs; ++b) {
            const int64_t first = (at[b] * group >> p.rows_shift) + b;
            const int64_t rows = (at[b + 1] - at[b]) * group, blocks = (rows + (1 << p.rows_shift) - 1) >> p.rows_shift;
            EXPECT(first >= next);
            next = first + (blocks ? blocks : 1);
        }
        EXPECT(next <= p.blocks);
    }
    if (failures) return 1;
    std::puts("ok");
    return 0;
}
