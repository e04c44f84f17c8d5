// The grids of the step operators' launches, at sizes around what a launch can
// count (2^32 - 1 threads along a dimension).  kq_step_api.cpp is linked with
// stubs in place of the launchers, which work out the workgroups of the launch.
// Prints "ok" and exits 0 when every launch that is let through fits, and sizes on
// both sides of the limit were met.
#include "../../include/kq.h"

#include <cstdint>
#include <cstdio>

#include "../../block_quantized_matmul_act_amd/csrc/kq_step.hpp"

namespace {
int failures = 0, launches = 0;
void fits(const char *what, int64_t groups, int64_t threads = 256) {
    ++launches;
    if (groups >= 1 && groups * threads <= (int64_t)UINT32_MAX) return;
    std::fprintf(stderr, "%s: %lld workgroups of %lld threads\n", what, (long long)groups, (long long)threads);
    ++failures;
}
}  // namespace

namespace kq {
hipError_t launch_rope_append(const RopeArgs &a, int, int dim, int, hipStream_t) {
    fits("rope_append", rope_plan(a.batch.n_tokens, a.q_heads, a.cache.heads, dim).blocks);
    return hipSuccess;
}
hipError_t launch_attn(const AttnArgs &a, const AttnPlan &p, int, int, int, hipStream_t) {
    fits("attn_tree", p.grid, 512);
    if (p.bytes) fits("attn_tree's join", a.batch.n_tokens);
    return hipSuccess;
}
hipError_t launch_keep(const KeepArgs &a, int, int, int, hipStream_t) {
    fits("cache_keep", a.batch.n_seqs);
    return hipSuccess;
}
hipError_t launch_logprobs(const LogprobsArgs &a, int, int64_t M, hipStream_t) {
    fits("logprobs", M * a.parts);
    return hipSuccess;
}
}  // namespace kq

int main() {
    char *const A = reinterpret_cast<char *>((uintptr_t)1 << 20);
    float *const F = reinterpret_cast<float *>(A);
    int32_t *const I = reinterpret_cast<int32_t *>(A);
    int refused = 0;
    auto met = [&](int rc) {
        if (rc == KQ_ERR_UNSUPPORTED)
            ++refused;
        else if (rc != KQ_OK)
            ++failures, std::fprintf(stderr, "status %d\n", rc);
    };
    for (int shift = 18; shift <= 30; ++shift)
        for (int64_t off = -1; off <= 1; ++off) {
            const int64_t n = ((int64_t)1 << shift) + off;
            if (n > INT32_MAX / 2) continue;
            for (int dim : {64, 128, 256})
                for (int heads : {1, 3, 8})
                    for (int group : {1, 5}) {
                        kq_cache c = {A, A, 100, KQ_T_BF16, heads, dim, 64, 1.f, 1.f};
                        kq_batch s = {I, I, I, n, n, 10};
                        const int64_t ldx = (int64_t)(group + 2) * heads * dim;
                        met(kq_rope_append(&c, &s, F, ldx, group * heads, F, F, 0.f, F, 100, dim, 0, I, KQ_T_BF16, A, nullptr));
                        for (int len : {1, 129, 5000})
                            met(kq_attn_tree(&c, &s, KQ_T_BF16, A, group * heads, nullptr, 1.f, 1, len, KQ_T_F32, A, A, SIZE_MAX, nullptr));
                        met(kq_cache_keep(&c, 1, &s, I, I, nullptr));
                    }
            for (int64_t V : {1, 64, 5000, 1 << 20}) met(kq_logprobs(KQ_T_F32, A, n, V, V, I, 1, 1, F, F, I, F, A, SIZE_MAX, nullptr));
        }
    for (int64_t M = 1; M <= 2048; ++M) met(kq_logprobs(KQ_T_F32, A, M, 1 << 30, 1 << 30, I, 1, 1, F, F, I, F, A, SIZE_MAX, nullptr));
    if (failures || refused < 100 || launches < 100) return 1;
    std::puts("ok");
    return 0;
}
