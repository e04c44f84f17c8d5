// kq_quant_device.hpp -- quantization of a row's blocks in registers, shared by
// the kernels that write activation buffers (gfx950 only).
//
// A lane owns 16 consecutive values, so a block is 16 lanes (Q8_K) or 8 lanes
// (Q8_128) and a per-16 sum is lane-local.
#pragma once

#include "kq_device.hpp"

namespace kq {

// DPP controls: quad permutes (lane ^ 1, lane ^ 2 within a quad) and the
// half-row (lane i <- 7 - i in each 8) and row (lane i <- 15 - i in each 16)
// mirrors
constexpr int DPP_QUAD_XOR1 = 0xB1, DPP_QUAD_XOR2 = 0x4E;
constexpr int DPP_ROW_HALF_MIRROR = 0x141, DPP_ROW_MIRROR = 0x140;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// The sections of an activation buffer (bsums and alpha: Q8_K only).
struct ActSections {
    int8_t *qs;
    float *d;
    int16_t *bsums;
    uint16_t *alpha;
};

// The largest |value| of this lane's block of BS values (every lane of the block
// takes part): exact and order-free, |x| compared as bit patterns.
template <int BS>
__device__ __forceinline__ float block_amax(const v4f (&v)[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, __builtin_bit_cast(uint32_t, fabsf(v[i][e])));
    m = max(m, dpp<DPP_QUAD_XOR1>(m));
    m = max(m, dpp<DPP_QUAD_XOR2>(m));
    m = max(m, dpp<DPP_ROW_HALF_MIRROR>(m));
    if constexpr (BS == 256) m = max(m, dpp<DPP_ROW_MIRROR>(m));
    return __builtin_bit_cast(float, m);
}

// The lane's 16 values as int8 under the block's amax, their sum and the scale:
// d = amax / 127, q = clamp(rint(x * 127 / amax), +-127), all zero where amax is
// 0 or 127 / amax is not finite.
struct Quantized {
    v4i qs;
    int sum;
    float d;
};
__device__ __forceinline__ Quantized quantize16(const v4f (&v)[4], float amax) {
    const float s = 127.0f / amax;
    const bool zero = !(amax > 0.0f) || !isfinite(s);
    Quantized r;
    r.qs = v4i{0, 0, 0, 0};
    r.sum = 0;
    if (!zero) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int q = (int)fminf(fmaxf(rintf(v[i][e] * s), -127.f), 127.f);
                r.sum += q;
                w |= (uint32_t)(q & 0xFF) << (8 * e);
            }
            r.qs[i] = (int)w;
        }
    }
    r.d = zero ? 0.0f : amax / 127.0f;
    return r;
}

// The lane's 16 values to the buffer: values [col, col + 16) of row `row` of M rows of
// K, lane gl of the lanes of block sblk.  Every lane of a wave takes part (the Q8_K
// sums of 32 are formed across lanes); only valid ones store.
template <int BS, bool BSUMS>
__device__ __forceinline__ void put16(const ActSections &a, const Quantized &q, bool valid, int64_t row, int64_t M,
                                      int64_t K, int64_t col, int sblk, int gl) {
    if (valid) {
        *reinterpret_cast<v4i *>(a.qs + row * K + col) = q.qs;
        if (gl == 0) a.d[sblk * M + row] = q.d;
    }
    if constexpr (BSUMS) {
        // this lane's 16 values are one bsums group
        if (valid) a.bsums[row * (K / 16) + col / 16] = (int16_t)q.sum;
        // 32 values = lanes 2j, 2j+1: B_j = sum32 (|B_j| <= 4064), parts
        // 64 * floor(B_j / 64) (a 7-bit integer times 64) and B_j mod 64, both
        // exact in bf16
        const int sum32 = q.sum + (int)dpp<DPP_QUAD_XOR1>((uint32_t)q.sum);
        const __bf16 p0 = (__bf16)(float)(sum32 & ~63);
        const __bf16 p1 = (__bf16)(float)(sum32 & 63);
        if (valid && (gl & 1) == 0) {
            const int j = gl >> 1;
            a.alpha[((sblk * 2 + 0) * M + row) * 8 + j] = __builtin_bit_cast(uint16_t, p0);
            a.alpha[((sblk * 2 + 1) * M + row) * 8 + j] = __builtin_bit_cast(uint16_t, p1);
        }
    }
}

}  // namespace kq
