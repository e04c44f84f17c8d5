// kq_variants.hpp -- the kernel variants that the dispatch counters tell apart.
#pragma once

namespace kq {

enum Variant {
    V_QUANT_Q8K = 0,
    V_QUANT_Q8_128,
    V_GEMM_Q4K_128x128,
    V_GEMM_Q4K_MATVEC,
    V_GEMM_Q6K_128x128,
    V_GEMM_Q6K_MATVEC,
    V_GEMM_TQ_128x128,
    V_GEMM_TQ_MATVEC,
    V_SUBSUMS_Q4K,
    V_SUBSUMS_Q6K,
    V_SUBSUMS_TQ,
    V_GEMM_TQ2_128x128,
    V_SUBSUMS_TQ2,
    V_GEMM_ID_128x128,
    V_GEMM_Q4K_64x128,
    V_GEMM_ID_Q4K_64x128,
    V_GEMM_Q4K_64x128_K2,
    V_GEMM_Q4K_M16,
    V_GEMM_TQ_128x128_REG,
    V_GEMM_Q4K_M64_RING,
    V_GEMM_Q6K_RING,
    V_GEMM_TQ2_RING,
    V_GEMM_TQ_RING,
    V_GEMM_Q4K_RING_KP,
    V_GEMM_TQ2_MATVEC,
    V_GEMM_Q6K_128x128_K2,
    V_GEMM_TQ_128x128_K2,
    V_GEMM_TQ2_128x128_K2,
    V_ROPE_APPEND,
    V_ATTN_FEW,
    V_ATTN_ROWS,
    V_CACHE_KEEP,
    V_LOGPROBS_ROW,
    V_LOGPROBS_PARTS,
    V_COUNT
};

// One more successful launch of a variant (the counters live in kq_api.cpp).
void count_dispatch(int variant);

}  // namespace kq
