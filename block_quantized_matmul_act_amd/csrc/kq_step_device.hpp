// kq_step_device.hpp -- device helpers of the paged-cache and log-probability
// kernels (gfx950 only).
#pragma once

#include "kq_device.hpp"
#include "kq_step.hpp"

namespace kq {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));

// Two fp32 rounded (to nearest even) to a packed pair of 16-bit values.
template <class E>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__bf16>(float a, float b) {
    const v2bf r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}
template <>
__device__ __forceinline__ uint32_t pack2<_Float16>(float a, float b) {
    const v2h r = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, r);
}

// Four fp32 to four e4m3 bytes, clamped to the largest finite value (NaN stays
// NaN: the comparisons are false for it).
__device__ __forceinline__ float clamp_f8(float x) { return x > 448.f ? 448.f : x < -448.f ? -448.f : x; }
__device__ __forceinline__ uint32_t pack4_f8(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_f8(a), clamp_f8(b), 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_f8(c), clamp_f8(d), r, true);
    return (uint32_t)r;
}

// The rows of sequence b in this step, held inside the step whatever the
// arrays say: first row and count.
__device__ __forceinline__ void batch_rows(const BatchArgs &s, int b, int &first, int &count) {
    first = min(max(s.offsets[b], 0), s.n_tokens);
    count = min(max(s.offsets[b + 1], first), s.n_tokens) - first;
}

// The tokens of sequence b in the cache, held where a row's slot does not overflow.
__device__ __forceinline__ int batch_len(const BatchArgs &s, int b) { return min(max(s.lens[b], 0), MAX_LEN); }

// The page of slot `slot` of sequence b: its entry in the table, held inside the
// cache; a page outside the cache or a slot past the table gives a wrong page,
// never one outside the cache.
// The arrays of a step are read as constants: where b and slot are the same for
// a wave, the load is a scalar one.
typedef const int32_t __attribute__((address_space(4))) *const_ints;
__device__ __forceinline__ int slot_entry(const CacheArgs &c, const BatchArgs &s, int b, int slot) {
    const int col = min(max(slot, 0) >> c.page_shift, s.max_pages - 1);
    return ((const_ints)s.pages)[(int64_t)b * s.max_pages + col];
}
__device__ __forceinline__ int page_inside(const CacheArgs &c, int entry) {
    return (int)min((int64_t)max(entry, 0), c.n_pages - 1);
}
__device__ __forceinline__ int slot_page(const CacheArgs &c, const BatchArgs &s, int b, int slot) {
    return page_inside(c, slot_entry(c, s, b, slot));
}

// The sequence of token row `row`, found by a whole wave together: the last b
// with offsets[b] <= row (sequences without rows are passed over).
__device__ __forceinline__ int batch_seq(const BatchArgs &s, int row) {
    const int lane = __lane_id();
    int lo = 0, n = s.n_seqs;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const int at = lo + lane * step;
        const bool le = at < lo + n && s.offsets[at] <= row;
        const int k = __popcll(__ballot(le));
        const int from = lo + max(k - 1, 0) * step;
        n = min(step, lo + n - from);
        lo = from;
    }
    return lo;
}

}  // namespace kq
