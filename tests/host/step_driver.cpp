// Host-side driver of the step operators' argument handling
// (kq_step_api.cpp), built with AddressSanitizer and UndefinedBehaviorSanitizer
// by tests/test_step_abi.py.  The launchers are stubs that record what they
// get, so every entry point runs on extreme sizes (a signed overflow in a size
// computation is reported) and the plans can be held to what the kernels
// assume.  Prints "ok" and exits 0 when every expectation holds.
#include "../../include/kq.h"

#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../block_quantized_matmul_act_amd/csrc/kq_step.hpp"

namespace {
int failures = 0;
#define EXPECT(c)                                                        \
    do {                                                                 \
        if (!(c)) {                                                      \
            std::fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c); \
            ++failures;                                                  \
        }                                                                \
    } while (0)

int ropes = 0, attns = 0, keeps = 0, logs = 0;
kq::AttnArgs attn;
kq::AttnPlan plan;
kq::KeepArgs keep;
int keep_n = 0;
kq::LogprobsArgs lp;
}  // namespace

namespace kq {
hipError_t launch_rope_append(const RopeArgs &, int, int, int, hipStream_t) {
    ++ropes;
    return hipSuccess;
}
hipError_t launch_attn(const AttnArgs &a, const AttnPlan &p, int, int, int, hipStream_t) {
    ++attns;
    attn = a;
    plan = p;
    return hipSuccess;
}
hipError_t launch_keep(const KeepArgs &a, int n, int, int, hipStream_t) {
    ++keeps;
    keep = a;
    keep_n = n;
    return hipSuccess;
}
hipError_t launch_logprobs(const LogprobsArgs &a, int, int64_t, hipStream_t) {
    ++logs;
    lp = a;
    return hipSuccess;
}
}  // namespace kq

// calls counted under a variant's name
int counted(const char *name) {
    for (int v = 0; v < kq_num_step_variants(); ++v)
        if (!std::strcmp(kq_step_variant_name(v), name)) return (int)kq_step_count(v);
    return -1;
}

int main() {
    char *const A = reinterpret_cast<char *>((uintptr_t)1 << 20);
    float *const F = reinterpret_cast<float *>(A);
    int32_t *const I = reinterpret_cast<int32_t *>(A);
    const int64_t ext[] = {INT64_MIN, -1, 0, 1, 5, 64, 65, 129, 8191, 65535, 65536, INT32_MAX, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX};
    const int dims[] = {64, 128, 256}, pages[] = {16, 32, 64, 128, 256};

    // extreme sizes through every entry point
    for (int64_t n : ext)
        for (int64_t m : ext)
            for (int64_t q : ext) {
                kq_cache c = {A, A, n > 0 ? n : 1, KQ_T_BF16, (int32_t)(q & 0xFFFFFFFF), 128, 64, 1.f, 1.f};
                kq_batch s = {I, I, I, n, m, q};
                kq_rope_append(&c, &s, F, m, q, F, F, 0.f, F, n, 64, 0, I, KQ_T_BF16, A, nullptr);
                for (int64_t x : ext) {
                    kq_attn_tree_workspace(&c, &s, q, x, m);
                    kq_attn_tree(&c, &s, KQ_T_BF16, A, q, nullptr, 1.f, x, m, KQ_T_F32, A, A, SIZE_MAX, nullptr);
                    kq_logprobs_workspace(n, m, x);
                    kq_logprobs(KQ_T_F32, A, n, m, x, I, q, 3, F, F, I, F, A, SIZE_MAX, nullptr);
                }
                kq_cache_keep(&c, n < 2 ? n : 1, &s, I, I, nullptr);
            }

    // plans: rows covered by the blocks, no more workgroups than units, and a
    // workspace of two blocks' rows of sums, maximum and weight to each workgroup
    // where a block can be cut
    for (int dim : dims)
        for (int page : pages)
            for (int64_t seqs : {1, 3, 64, 4096})
                for (int64_t T : {1, 2, 17, 64})
                    for (int64_t G : {1, 5, 16, 64})
                        for (int64_t len : {1, 127, 128, 129, 1024, 1025, 5000, 131075, 1 << 30}) {
                            kq_cache c = {A, A, 100, KQ_T_F16, 2, dim, page, 1.f, 1.f};
                            kq_batch s = {I, I, I, seqs, seqs, 10};
                            const int before = attns;
                            const size_t bytes = kq_attn_tree_workspace(&c, &s, 2 * G, T, len);
                            const int rc = kq_attn_tree(&c, &s, KQ_T_F16, A, 2 * G, nullptr, 1.f, T, len, KQ_T_F16, A, A, bytes, nullptr);
                            if (rc == KQ_ERR_UNSUPPORTED) continue;
                            EXPECT(rc == KQ_OK && attns == before + 1);
                            const int wave = dim == 256 ? 16 : 32;
                            EXPECT(plan.waves == (T * G <= 16 ? 0 : T * G <= 4 * wave && dim < 256 ? 4 : 8));
                            EXPECT(plan.rows_wg == (plan.waves ? plan.waves * wave : 16));
                            EXPECT((int64_t)plan.rows_wg * plan.row_blocks >= T * G);
                            EXPECT((int64_t)plan.rows_wg * (plan.row_blocks - 1) < T * G);
                            EXPECT(plan.slot_rows == (T * G < plan.rows_wg ? T * G : plan.rows_wg));
                            const int unit = plan.waves == 0 && len > 128 && len <= 1024 && seqs * 2 <= 256 && dim < 256 ? 1024 : 128;
                            EXPECT(1 << plan.unit_shift == unit && attn.unit_shift == plan.unit_shift);
                            const int64_t units = seqs * 2 * plan.row_blocks * ((len + unit - 1) / unit);
                            EXPECT(units <= INT32_MAX && plan.grid >= 1 && plan.grid <= units && plan.grid <= 512);
                            const int64_t rows = len > unit ? 2 * (int64_t)plan.grid * plan.slot_rows : 0;
                            EXPECT((int64_t)bytes == (rows ? rows * (dim * 4 + 8) + (rows & 1) * 8 + seqs * 16 : 0));
                            EXPECT(plan.o_bytes == rows * dim * 4);
                            EXPECT((char *)attn.ws_seq == (bytes ? A + bytes - seqs * 16 : nullptr) && plan.ml_end % 16 == 0);
                            EXPECT((char *)attn.ws_ml == A + plan.o_bytes && (char *)attn.ws_o == A);
                            EXPECT(1 << attn.cache.page_shift == page && attn.group == G && attn.grid == plan.grid);
                            EXPECT(attn.rows_wg == plan.rows_wg && attn.slot_rows == plan.slot_rows && attn.max_len == len);
                            if (bytes) EXPECT(kq_attn_tree(&c, &s, KQ_T_F16, A, 2 * G, nullptr, 1.f, T, len, KQ_T_F16, A, A, bytes - 1, nullptr) == KQ_ERR_SHAPE);
                        }

    // caches in groups of kernel arguments
    static kq_cache many[150];
    for (int i = 0; i < 150; ++i) many[i] = kq_cache{A + 4096 * i, A + 4096 * i + 2048, 10, KQ_T_F8, 4, 64, 32, 1.f, 1.f};
    kq_batch s = {I, I, I, 3, 9, 4};
    const int before = keeps;
    EXPECT(kq_cache_keep(many, 150, &s, I, I, nullptr) == KQ_OK);
    EXPECT(keeps == before + 3 && keep_n == 150 - 2 * kq::KEEP_CACHES);
    EXPECT(keep.k[0] == A + 4096 * 128 && keep.v[keep_n - 1] == A + 4096 * 149 + 2048 && keep.cache.page_shift == 5);

    // rows of logits: parts cover the row, none is empty
    for (int64_t M : {1, 2, 63, 1000, 5000})
        for (int64_t V : {1, 4095, 4096, 4097, 128256, 1 << 20}) {
            const size_t bytes = kq_logprobs_workspace(M, V, V < 7 ? 1 : 7);
            EXPECT(kq_logprobs(KQ_T_BF16, A, M, V, V, I, 2, V < 7 ? 1 : 7, F, nullptr, I, F, A, bytes, nullptr) == KQ_OK);
            EXPECT((int64_t)lp.part * lp.parts >= V && (int64_t)lp.part * (lp.parts - 1) < V);
            EXPECT(bytes == (lp.parts > 1 ? (size_t)((M * lp.parts * 12 + 7) / 8 * 8 + M * lp.parts * 8 * 7) : 0));
            if (bytes) EXPECT(kq_logprobs(KQ_T_BF16, A, M, V, V, I, 2, 7, F, nullptr, I, F, A, bytes - 1, nullptr) == KQ_ERR_SHAPE);
        }
    EXPECT(ropes == counted("rope_append"));
    EXPECT(attns == counted("attn_few") + counted("attn_rows"));
    EXPECT(logs == counted("logprobs_row") + counted("logprobs_parts") && keeps == counted("cache_keep"));
    EXPECT(!kq_step_variant_name(-1) && !kq_step_variant_name(kq_num_step_variants()));
    kq_step_count_reset();
    EXPECT(counted("rope_append") == 0 && kq_step_count(-1) == 0);
    if (failures) return 1;
    std::puts("ok");
    return 0;
}
