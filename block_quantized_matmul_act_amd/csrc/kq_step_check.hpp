// kq_step_check.hpp -- checks of the paged cache and of a step's sequences,
// shared by the entry points that take them (host code).
#pragma once

#include <cmath>
#include <cstdint>

#include "kq_step.hpp"

namespace kq {

constexpr int64_t kMaxInt = INT32_MAX;
constexpr int64_t kMaxLen = MAX_LEN;
constexpr int64_t kMaxPages = (int64_t)1 << 31;
constexpr int64_t kMaxHeads = 65535;           // a grid's second dimension

inline bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// KQ_OK, or the error of a cache descriptor
inline int check_cache(const kq_cache *c) {
    if (!c) return KQ_ERR_NULL;
    if (c->type != KQ_T_BF16 && c->type != KQ_T_F16 && c->type != KQ_T_F8) return KQ_ERR_FMT;
    if (c->n_pages < 0 || c->n_pages >= kMaxPages || c->heads < 1 || c->heads > kMaxHeads) return KQ_ERR_SHAPE;
    if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || !std::isfinite(c->k_scale) || !std::isfinite(c->v_scale))
        return KQ_ERR_SHAPE;
    if (c->dim != 64 && c->dim != 128 && c->dim != 256) return KQ_ERR_UNSUPPORTED;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256) return KQ_ERR_UNSUPPORTED;
    return KQ_OK;
}
// 1: work to do; KQ_OK: no rows; an error otherwise
inline int check_batch(const kq_batch *s) {
    if (!s) return KQ_ERR_NULL;
    if (s->n_seqs < 0 || s->n_tokens < 0 || s->max_pages < 0) return KQ_ERR_SHAPE;
    if (s->n_seqs > kMaxInt || s->n_tokens > kMaxInt / 2 || s->max_pages > kMaxInt) return KQ_ERR_SHAPE;
    return s->n_tokens == 0 || s->n_seqs == 0 ? KQ_OK : 1;
}
// pointers and sizes that a call with rows needs
inline int check_step(const kq_cache *c, const kq_batch *s) {
    if (c->n_pages == 0 || s->max_pages == 0) return KQ_ERR_SHAPE;
    if (!c->k || !c->v || !s->offsets || !s->lens || !s->pages) return KQ_ERR_NULL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(s->offsets, 4) || !aligned(s->lens, 4) ||
        !aligned(s->pages, 4))
        return KQ_ERR_ALIGN;
    return KQ_OK;
}
inline CacheArgs cache_args(const kq_cache *c) {
    int shift = 4;
    while ((1 << shift) < c->page) ++shift;
    return CacheArgs{static_cast<char *>(c->k), static_cast<char *>(c->v), c->n_pages, c->heads, shift};
}
inline BatchArgs batch_args(const kq_batch *s) {
    return BatchArgs{s->offsets, s->lens, s->pages, (int)s->n_seqs, (int)s->n_tokens, (int)s->max_pages};
}
inline bool type16(int t) { return t == KQ_T_BF16 || t == KQ_T_F16; }

}  // namespace kq
