// kq_act_layout.hpp -- where the sections of an activation buffer lie, shared by
// the entry points that write and read them (host code).
#pragma once

#include <cstdint>

#include "../../include/kq.h"

namespace kq {

constexpr int64_t kMaxDim = INT32_MAX;  // kernels index rows and columns with int
constexpr int64_t kMaxBytes = (int64_t)1 << 46;

inline int bs_of(int act_fmt) {
    return act_fmt == KQ_ACT_Q8_K ? 256 : act_fmt == KQ_ACT_Q8_128 ? 128 : 0;
}
inline int64_t align256(int64_t v) { return (v + 255) & ~(int64_t)255; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Section offsets of an activation buffer; false when invalid.
struct ActLayout {
    int64_t d, bsums, alpha, total;  // byte offsets; -1 for absent sections
};
inline bool act_layout(int act_fmt, int64_t M, int64_t K, ActLayout *L) {
    const int bs = bs_of(act_fmt);
    if (!bs || M < 0 || K < 0 || K % bs || M > kMaxDim || K > kMaxDim) return false;
    if (M != 0 && K > kMaxBytes / M) return false;
    const int64_t qs_bytes = align256(M * K);
    const int64_t d_bytes = align256(M * (K / bs) * 4);
    L->d = qs_bytes;
    if (act_fmt == KQ_ACT_Q8_K) {
        L->bsums = qs_bytes + d_bytes;
        L->alpha = L->bsums + align256(M * (K / 16) * 2);
        L->total = L->alpha + align256((K / 256) * 2 * M * 8 * 2);
    } else {
        L->bsums = -1;
        L->alpha = -1;
        L->total = qs_bytes + d_bytes;
    }
    return true;
}

}  // namespace kq
