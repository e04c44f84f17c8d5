// kq_attn_device.hpp -- pieces of attention over a paged cache, shared by the
// kernels of kq_attn.hip (a token or a tree of drafts) and kq_chunk.hip (chunks of
// a text): operands, tiles in LDS, the softmax sums of a wave's rows (gfx950 only).
// How they fit together is at the head of kq_attn.hip.
#pragma once

#include "kq_step_device.hpp"

namespace kq {

namespace {

constexpr float M_START = -3.402823466e38f;  // no finite score is below it; finite: exp2(-inf - m) is 0, not NaN
// m: how far below a row's maximum it is set, and how far a score may pass it
template <class E>
constexpr float M_BELOW = std::is_same_v<E, _Float16> ? 7.f : -20.f;
template <class E>
constexpr float M_SLACK = M_BELOW<E> + 8.f;
// From here on the rounding of score * scale (half of 2^-23 of it) is felt in exp2 of
// its distance from m, and further out passes every type: see far.
constexpr float M_FAR = 1048576.f;

typedef float v2f __attribute__((ext_vector_type(2)));

// A lane's value and that of the lane 32 (16) away, in both, in no order.
__device__ __forceinline__ v2f across32(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return v2f{__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}
__device__ __forceinline__ v2f across16(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return v2f{__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}
// Over the lane groups of RW lanes: the largest, the sum.
template <int RW>
__device__ __forceinline__ float groups_max(float x) {
    v2f r = across32(x);
    x = fmaxf(r[0], r[1]);
    if constexpr (RW == 16) {
        r = across16(x);
        x = fmaxf(r[0], r[1]);
    }
    return x;
}
template <int RW>
__device__ __forceinline__ float groups_sum(float x) {
    v2f r = across32(x);
    x = r[0] + r[1];
    if constexpr (RW == 16) {
        r = across16(x);
        x = r[0] + r[1];
    }
    return x;
}
// A constant that stays where it is used (hoisted out of a path that is hardly
// ever taken, it would cost the loops a register).
__device__ __forceinline__ uint32_t here(uint32_t c) {
    uint32_t r;
    asm volatile("v_mov_b32 %0, %1" : "=v"(r) : "i"(c));
    return r;
}

// 4 neighbouring sums: finished ones to the output, a part's to the workspace.
template <class E>
__device__ __forceinline__ void put4(const AttnArgs &a, bool whole, v4f x, int64_t out, int64_t slot) {
    if (!whole)
        *reinterpret_cast<v4f *>(a.ws_o + slot) = x;
    else if (a.out_f32)
        *reinterpret_cast<v4f *>(reinterpret_cast<float *>(a.out) + out) = x;
    else
        *reinterpret_cast<v2u *>(a.out + out * 2) = v2u{pack2<E>(x[0], x[1]), pack2<E>(x[2], x[3])};
}

template <class E, int RW>
struct Mfma;
template <>
struct Mfma<__bf16, 16> {
    typedef v8bf op;
    typedef v4f acc;
    static __device__ __forceinline__ acc mul(op a, op b, acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mfma<_Float16, 16> {
    typedef v8h op;
    typedef v4f acc;
    static __device__ __forceinline__ acc mul(op a, op b, acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mfma<__bf16, 32> {
    typedef v8bf op;
    typedef v16f acc;
    static __device__ __forceinline__ acc mul(op a, op b, acc c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mfma<_Float16, 32> {
    typedef v8h op;
    typedef v16f acc;
    static __device__ __forceinline__ acc mul(op a, op b, acc c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

__device__ __forceinline__ uint64_t first_bits(int n) { return n ? (2ull << (n - 1)) - 1ull : 0ull; }  // n <= 64

// Which of 8 keys a row sees (bit e: the e-th), the first being node `node` of
// the drafted tokens (below 0: that many cached ones come first).  sees: the
// row's mask, cut to the sequence's rows.
__device__ __forceinline__ uint32_t seen8(uint64_t sees, int node) {
    const uint32_t drafted = node > 63 ? 0u : (uint32_t)(sees >> (node & 63));
    const int cached = min(max(-node, 0), 8);
    const uint32_t both = (uint32_t)sees << cached | ((1u << cached) - 1u);
    return node >= 0 ? drafted : both;
}

// Marks of infinite and NaN values: 1, 128 and 16384, whole numbers that both
// 16-bit types hold, set so far apart that sums of 32 do not run into the next.
template <class E>
struct Marks {
    uint32_t pos, neg, nan;
    __device__ __forceinline__ Marks() {
        constexpr bool bf = std::is_same_v<E, __bf16>;
        pos = here(bf ? 0x3F80u : 0x3C00u);
        neg = here(bf ? 0x4300u : 0x5800u);
        nan = here(bf ? 0x4680u : 0x7400u);
    }
};

// Eight cached values as they lie in memory, and as an operand.
template <class E, bool F8>
struct Frag;
template <class E>
struct Frag<E, false> {
    typedef v4u raw;
    static constexpr int BYTES = 2;
    // keep the first n (0 .. 8) values, zeros after them
    static __device__ __forceinline__ void first(raw &r, int n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = n - 2 * j;
            r[j] &= k >= 2 ? 0xFFFFFFFFu : k == 1 ? 0xFFFFu : 0u;
        }
    }
    // infinite and NaN values become zeros; whether there were any
    static __device__ __forceinline__ bool drop_odd(raw &r) {
        constexpr uint32_t e = std::is_same_v<E, __bf16> ? 0x7F80u : 0x7C00u;
        bool any = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool lo = (r[j] & e) == e, hi = (r[j] & (e << 16)) == e << 16;
            r[j] &= (lo ? 0xFFFF0000u : ~0u) & (hi ? 0xFFFFu : ~0u);
            any = any || lo || hi;
        }
        return any;
    }
    // value i's mark: see add_odd
    static __device__ __forceinline__ uint32_t mark(raw r, int i, const Marks<E> &m) {
        constexpr uint32_t e = std::is_same_v<E, __bf16> ? 0x7F80u : 0x7C00u;
        const uint32_t x = r[i >> 1] >> (16 * (i & 1)) & 0xFFFFu;
        return (x & 0x7FFFu) < e ? 0u : (x & 0x7FFFu) > e ? m.nan : x >> 15 ? m.neg : m.pos;
    }
    template <class OP>
    static __device__ __forceinline__ OP op(raw r) {
        return __builtin_bit_cast(OP, r);
    }
};
template <class E>
struct Frag<E, true> {
    typedef v2u raw;
    static constexpr int BYTES = 1;
    static __device__ __forceinline__ void first(raw &r, int n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = min(max(n - 4 * j, 0), 4);
            r[j] &= k == 4 ? ~0u : (1u << (8 * k)) - 1u;
        }
    }
    static __device__ __forceinline__ bool drop_odd(raw &r) {
        uint32_t any = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            // bit 7 of a byte: its low 7 bits are all ones (the NaN of either sign)
            const uint32_t x = ((r[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            r[j] &= ~((x >> 7) * 0xFFu);
            any |= x;
        }
        return any != 0;
    }
    static __device__ __forceinline__ uint32_t mark(raw r, int i, const Marks<E> &m) {
        return ((r[i >> 2] >> (8 * (i & 3))) & 0x7Fu) == 0x7Fu ? m.nan : 0u;
    }
    static __device__ __forceinline__ uint32_t pair(uint32_t r, bool hi) {
        if constexpr (std::is_same_v<E, __bf16>)
            return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r, 1.f, true))
                      : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r, 1.f, false));
        else
            return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r, 1.f, true))
                      : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r, 1.f, false));
    }
    template <class OP>
    static __device__ __forceinline__ OP op(raw r) {  // e4m3 values are exact in both 16-bit types
        const v4u w = {pair(r[0], false), pair(r[0], true), pair(r[1], false), pair(r[1], true)};
        return __builtin_bit_cast(OP, w);
    }
};

// A sequence as the kernels see it: rows and slots held inside the step and the
// bounds of the call.
struct Seq {
    int first, rows, T, len, total;  // T of the rows are computed
};
__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int b) {
    Seq q;
    batch_rows(a.batch, b, q.first, q.rows);
    q.T = min(q.rows, a.max_tokens);
    q.len = min(batch_len(a.batch, b), a.max_len);
    q.total = min(q.len + q.T, a.max_len);
    return q;
}

// Equal runs of `units` for `groups` workgroups (at least as many units as groups):
// the first `more` have one unit more than the others.
struct Runs {
    int size, more;
    __device__ __forceinline__ Runs(int units, int groups) {
        size = units / groups;
        more = units - size * groups;
    }
    __device__ __forceinline__ int begin(int w) const { return w * size + min(w, more); }
    __device__ __forceinline__ int holder(int u) const {  // the workgroup that has unit u
        const int longer = more * (size + 1);
        return u < longer ? u / (size + 1) : more + (u - longer) / size;
    }
};

// Where a sequence's values lie, for what add_odd reads again.
struct ValueRows {
    const CacheArgs &cache;
    const BatchArgs &batch;
    int b, h, total;
};

// An infinity or NaN among the values of drafted tokens belongs to the rows that
// see its token and to no other, but a product with P would spoil them all (0 *
// inf).  Such values are zeros in the product; here they are added for one step
// of it (512 / RW keys from key0): marks of them times a 0 / 1 matrix of who
// sees what count the infinities and NaNs that reach each sum.  sees(k): which of the 8
// keys from k this lane's row sees.
template <class E, bool F8, int D, int RW, class SEES>
__device__ __forceinline__ void add_odd(const ValueRows &va, int key0, int lane, SEES sees,
                                        typename Mfma<E, RW>::acc (&o)[D / RW]) {
    typedef Mfma<E, RW> MM;
    typedef Frag<E, F8> FR;
    constexpr int ES = FR::BYTES;
    const int n = lane & (RW - 1), g = lane / RW;
    const int key = key0 + 8 * g;  // the first of this lane's 8
    const Marks<E> marks;
    const float inf = __builtin_bit_cast(float, here(0x7F800000u));
    const uint32_t on = sees(key);
    v4u w = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 1] |= (on >> e & 1u) * (marks.pos << (16 * (e & 1)));
    const typename MM::op seen = __builtin_bit_cast(typename MM::op, w);
    const int shift = va.cache.page_shift;
    const int slot = min(key & ~15, (va.total - 1) & ~15);
    const char *p = va.cache.v +
                    (((int64_t)slot_page(va.cache, va.batch, va.b, slot) * va.cache.heads + va.h) * D << shift) * ES +
                    ((slot & ((1 << shift) - 1)) + (key & 8)) * ES;
#pragma unroll
    for (int d = 0; d < D / RW; ++d) {
        typename FR::raw r = *reinterpret_cast<const typename FR::raw *>(p + ((d * RW + n) << shift) * ES);
        FR::first(r, min(max(va.total - key, 0), 8));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = FR::mark(r, 2 * j, marks) | FR::mark(r, 2 * j + 1, marks) << 16;
        const typename MM::acc count =
            MM::mul(__builtin_bit_cast(typename MM::op, w), seen, typename MM::acc{});
#pragma unroll
        for (int i = 0; i < RW * RW / 64; ++i) {
            const int c = (int)count[i];
            float x = (c & 127) ? inf : 0.f;
            x = c & (127 << 7) ? x - inf : x;
            o[d][i] += c >> 14 ? inf - inf : x;
        }
        __builtin_amdgcn_sched_barrier(0);  // one at a time: this path must not cost the others registers
    }
}

// ---------------------------------------------------------------- tiles

// A tile of KEYS keys and values in LDS, staged by THREADS threads through
// registers.  MFMA operands straight from memory would make the 16 lanes of a
// quarter wave read 16 different rows, one cache access each (measured: 63
// accesses to an 8-byte load of a wave, and 4 TB/s); staged, the lanes of a load
// read whole runs of rows.
// ONCE: the keys are read by this workgroup alone, and pass the caches by, which
// leaves these to the values, whose lines (one feature of a page) several waves
// share: 257 -> 234 us for 1.4 GB; the values too: up to 291 us.
// LDS holds 16-byte pieces; a row's pieces are permuted by an XOR with bits of
// the row, so that the lanes of a read, which want one piece of many rows, meet
// different banks.
template <class E, bool F8, int D, int KEYS, int RW, int THREADS, bool ONCE>
struct Tile {
    typedef Frag<E, F8> FR;
    typedef typename FR::raw raw_t;
    static constexpr int ES = FR::BYTES;
    static constexpr int KB = D * ES, VB = KEYS * ES;  // bytes of a key row and of a feature row
    static constexpr int KP = KB / 16, VP = VB / 16;   // their 16-byte pieces
    static constexpr int PIECES = KEYS * KP;           // of the keys, and as many of the values
    static constexpr int N = (PIECES + THREADS - 1) / THREADS;  // loads of a thread for each
    static constexpr int KSTEP = THREADS / KP, VSTEP = THREADS / VP;  // rows between a thread's loads
    static constexpr int K_BYTES = KEYS * KB, BYTES = 2 * K_BYTES;

    // The 16 lanes that a read serves together are 0-3, 12-15, 20-23 and 24-27 of a
    // half wave, or the others; the XORs give them 16 different places of 256 bytes.
    // They take bits of the row, so the place of row x | y is that of x with a
    // constant XORed and one added.
    static __device__ __forceinline__ constexpr int k_xor(int key) {
        return KP >= 16  ? (RW == 32 ? key & 15 : (key & 3) | ((key >> 1) & 12))
               : KP == 8 ? (RW == 32 ? (key >> 1) & 7 : ((key >> 1) & 1) | ((key >> 2) & 6))
                         : (key >> 3) & 3;
    }
    static __device__ __forceinline__ constexpr int v_xor(int d) {
        return VP >= 8 ? (d >> 1) & 7 : VP == 4 ? -(d >> 2) & 3 : (d >> 3) & 1;
    }
    static __device__ __forceinline__ int k_pos(int key, int piece) { return key * KB + (piece ^ k_xor(key)) * 16; }
    static __device__ __forceinline__ int v_pos(int d, int piece) { return d * VB + (piece ^ v_xor(d)) * 16; }

    // A thread's part: piece t (+ i * THREADS) of the keys and of the values
    const AttnArgs &a;
    int t, k_row, k_piece, v_row, v_piece;
    int k_to, v_to;  // places in a tile
    bool stages;
    int page_shift, page_mask;
    // the sequence and head
    int b, h, len, total, last;  // last: a slot of the sequence's last run
    v4u stage[2 * N];

    __device__ __forceinline__ Tile(const AttnArgs &a_, int t_) : a(a_), t(t_) {
        k_row = t / KP;
        k_piece = t % KP;
        v_row = t / VP;
        v_piece = t % VP;
        k_to = k_pos(k_row, k_piece);
        v_to = v_pos(v_row, v_piece);
        stages = PIECES >= THREADS || t < PIECES;
        page_shift = a.cache.page_shift;
        page_mask = (1 << page_shift) - 1;
    }
    __device__ __forceinline__ void aim(int b_, int h_, const Seq &q) {
        b = b_;
        h = h_;
        len = q.len;
        total = q.total;
        last = (total - 1) & ~15;
    }
    // Where a tile lies: the pages of its runs of 16 slots, looked up a turn before
    // the load needs them.  16 consecutive slots from a multiple of 16 lie in one
    // page, often the tile does.  A run past the sequence's end is taken to be its
    // last one (masked later).
    struct Place {
        int key, entries[KEYS / 16];  // of the page table as they are: nothing waits for them here
    };
    __device__ __forceinline__ Place find(int key0) const {
        Place p;
        p.key = key0;
        p.entries[0] = slot_entry(a.cache, a.batch, b, min(key0, last));
        if ((1 << page_shift) < KEYS) {
#pragma unroll
            for (int r = 1; r < KEYS / 16; ++r) p.entries[r] = slot_entry(a.cache, a.batch, b, min(key0 + 16 * r, last));
        }
        return p;
    }
    __device__ __forceinline__ int64_t page_at(int entry) const {
        return ((int64_t)page_inside(a.cache, entry) * a.cache.heads + h) * ((int64_t)D * ES << page_shift);
    }
    // Its keys to the registers.  A wave's load lies in one run.
    __device__ __forceinline__ void load_k(const Place &pl) {
        if (!stages) return;
        if ((1 << page_shift) >= KEYS) {
            // (pages are whole in memory, past the sequence's end too)
            const char *p = a.cache.k + page_at(pl.entries[0]) + (min(pl.key, last & -KEYS) & page_mask) * KB + t * 16;
#pragma unroll
            for (int i = 0; i < N; ++i) get(stage[i], p + i * (THREADS * 16));
            return;
        }
        int64_t run[KEYS / 16];
#pragma unroll
        for (int r = 0; r < KEYS / 16; ++r) run[r] = page_at(pl.entries[r]) + (min(pl.key + 16 * r, last) & page_mask) * KB;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int mine = __builtin_amdgcn_readfirstlane(k_row + i * KSTEP) >> 4;
            int64_t at = run[0];
#pragma unroll
            for (int r = 1; r < KEYS / 16; ++r) at = r == mine ? run[r] : at;
            get(stage[i], a.cache.k + at + (((k_row + i * KSTEP) & 15) * KB + k_piece * 16));
        }
    }
    // Its values.
    __device__ __forceinline__ void load_v(const Place &pl) {
        if (!stages) return;
        const char *p = a.cache.v + (v_row << page_shift) * ES;
        if ((1 << page_shift) >= KEYS) {
            p += page_at(pl.entries[0]) + (min(pl.key, last & -KEYS) & page_mask) * ES + v_piece * 16;
        } else {
            int64_t at = 0;
#pragma unroll
            for (int r = 0; r < KEYS / 16; ++r) {
                const int64_t o = page_at(pl.entries[r]) + (min(pl.key + 16 * r, last) & page_mask) * ES;
                at = r == v_piece * (16 / ES) >> 4 ? o : at;
            }
            p += at + (v_piece * 16 & (16 * ES - 1));
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            stage[N + i] = *reinterpret_cast<const v4u *>(p);
            p += VSTEP * ES << page_shift;
        }
    }
    static __device__ __forceinline__ void get(v4u &r, const char *p) {
        if constexpr (ONCE)
            r = __builtin_nontemporal_load(reinterpret_cast<const v4u *>(p));
        else
            r = *reinterpret_cast<const v4u *>(p);
    }
    // The keys to LDS (the tile at byte `buf`, a multiple of 1024).
    __device__ __forceinline__ void store_k(char *lds, int buf) const {
        if (!stages) return;
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<v4u *>(lds + ((k_to + buf) ^ (k_xor(i * KSTEP) * 16)) + i * KSTEP * KB) = stage[i];
    }
    // The values to LDS.  In a tile that some row does not see whole (one that reaches past
    // the cached slots, or `edge` if not DRAFTS): zeros for slots past the end, which may hold
    // anything, and for infinite and NaN values; whether this thread met any of those.
    template <bool DRAFTS = true>
    __device__ __forceinline__ bool store_v(char *lds, int buf, int key0, bool edge = false) {
        bool found = false;
        if (!stages) return false;
        if (DRAFTS ? key0 + KEYS > len : edge) {
            const int left = total - (key0 + v_piece * (16 / ES));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v4u &r = stage[N + i];
                if constexpr (F8) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        raw_t half = {r[2 * j], r[2 * j + 1]};
                        FR::first(half, min(max(left - 8 * j, 0), 8));
                        found |= FR::drop_odd(half);
                        r[2 * j] = half[0];
                        r[2 * j + 1] = half[1];
                    }
                } else {
                    FR::first(r, min(max(left, 0), 8));
                    found |= FR::drop_odd(r);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<v4u *>(lds + ((v_to + buf) ^ (v_xor(i * VSTEP) * 16)) + i * VSTEP * VB) = stage[N + i];
        return found;
    }
};

// The softmax sums of RW rows of a wave over tiles of KEYS keys.
// RUNS: values lie in LDS by runs of 16 slots, [run][feature][16], not by feature; in 16
// bits the halves of features 16 .. 31 of each 32 are swapped where a wave reads 32 features at
// once, which makes the reads conflict-free.
template <class E, bool F8, int D, int KEYS, int RW, bool RUNS = false>
struct Attend {
    typedef Mfma<E, RW> MM;
    typedef typename MM::op op_t;
    typedef typename MM::acc acc_t;
    typedef Frag<E, F8> FR;
    typedef typename FR::raw raw_t;
    typedef Tile<E, F8, D, KEYS, RW, 64, true> TL;  // (for the places in LDS alone)
    static constexpr int NG = 64 / RW;             // lane groups: 8 of a step's keys, 8 of a step's features to each
    static constexpr int NK = D / (8 * NG), ND = D / RW;         // steps of the first product, results of the second
    static constexpr int NT = KEYS / RW, NS = KEYS / (8 * NG);   // results of the first, steps of the second
    static constexpr int NR = RW * RW / 64;
    static constexpr int RUN_BYTES = D * 16 * FR::BYTES;  // values of 16 slots

    const AttnArgs &a;
    int lane, n, g;
    int k_from, v_from;  // places in a tile
    bool used;
    int64_t q_row;  // of q and out
    uint64_t sees;
    op_t qf[NK];
    acc_t o[ND];
    float m, l;
    // Some row's m is beyond M_FAR: the scores are then scaled first and m is taken
    // from them after (in one fma m is rounded and the product it came from is not).
    // The same for the whole wave; set where m is.
    bool far;

    __device__ __forceinline__ Attend(const AttnArgs &a_) : Attend(a_, threadIdx.x) {}
    __device__ __forceinline__ Attend(const AttnArgs &a_, unsigned thread) : a(a_) {
        lane = thread & 63;
        n = lane & (RW - 1);
        g = lane / RW;
        // this lane's row of the first product's results: see the head of the file
        const int krow = RW == 16 ? 8 * (n >> 2) + (n & 3) : 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);
        k_from = TL::k_pos(krow, F8 ? g >> 1 : g) + (F8 ? 8 * (g & 1) : 0);
        if constexpr (RUNS)
            v_from = (g >> 1) * RUN_BYTES + n * 16 * FR::BYTES + ((g & 1) ^ (!F8 && RW == 32 ? n >> 4 : 0)) * 8 * FR::BYTES;
        else
            v_from = TL::v_pos(n, F8 ? g >> 1 : g) + (F8 ? 8 * (g & 1) : 0);
    }
    // 8 values of this lane: row t (and step kk) of the keys, row d (step s) of the values
    __device__ __forceinline__ raw_t k_frag(const char *lds, int at, int t, int kk) const {
        const int row = RW == 16 ? 32 * (t >> 1) + 4 * (t & 1) : 32 * t;
        return *reinterpret_cast<const raw_t *>(lds + (at ^ (kk * NG * 8 * FR::BYTES)) + row * TL::KB);
    }
    __device__ __forceinline__ raw_t v_frag(const char *lds, int at, int d, int s) const {
        if constexpr (RUNS)
            return *reinterpret_cast<const raw_t *>(lds + at + s * (NG / 2 * RUN_BYTES) + RW * d * 16 * FR::BYTES);
        return *reinterpret_cast<const raw_t *>(lds + (at ^ (s * NG * 8 * FR::BYTES)) + RW * d * TL::VB);
    }
    // begin rows row0 .. of key head h (DRAFTS: and what they see of the drafted tokens); this
    // lane's token
    template <bool DRAFTS = true>
    __device__ __forceinline__ int begin(const Seq &sq, int h, int row0) {
        const int G = a.group, row = row0 + n;
        used = row < sq.T * G;
        const int tok = used ? row / G : 0;
        q_row = (int64_t)(sq.first + tok) * ((int64_t)a.cache.heads * G) + h * G + (used ? row % G : 0);
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
            v4u w = {0u, 0u, 0u, 0u};
            if (used) w = (*reinterpret_cast<const v4u *>(a.q + (q_row * D + 8 * (NG * kk + g)) * 2) & a.q_keep) ^ a.q_flip;
            qf[kk] = __builtin_bit_cast(op_t, w);
        }
        if constexpr (DRAFTS) {
            sees = 0;
            if (used) sees = (a.mask ? a.mask[sq.first + tok] : (2ull << tok) - 1ull) & first_bits(sq.total - sq.len);
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] = acc_t{};
        m = M_START;
        l = 0.f;
        far = false;
        return tok;
    }
    // Matrix products of one stream: with VALUES the probabilities pf times the values
    // at byte v of the LDS are added to the sums, with SCORES p gets the scores of
    // the keys at byte k; p[r]: key key0 + 8 NG (r / 8) + 8 g + r % 8 of this lane's
    // row.  The operands are read AHEAD products before they are used (left to itself
    // the compiler reads each right before its product, and waits for it).
    template <bool VALUES, bool SCORES, int AHEAD>
    __device__ __forceinline__ void products(const char *lds, int v, const op_t (&pf)[NS], int k, float (&p)[NT * NR]) {
        constexpr int NV = VALUES ? NS * ND : 0, ALL = NV + (SCORES ? NT * NK : 0), RING = AHEAD + 2;
        const int from_v = v_from + v, from_k = k_from + k;
        raw_t ring[RING];
        acc_t sc[NT];
        auto read = [&](auto X) {
            constexpr int x = decltype(X)::value;
            if constexpr (x < NV)
                ring[x % RING] = v_frag(lds, from_v, x % ND, x / ND);
            else if constexpr (x < ALL)
                ring[x % RING] = k_frag(lds, from_k, (x - NV) % NT, (x - NV) / NT);
        };
        if constexpr (SCORES) {
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[t] = acc_t{};
        }
        static_for<0, AHEAD>(read);
        static_for<0, ALL / 2>([&](auto X) {
            constexpr int x = 2 * decltype(X)::value;
            read(IC<x + AHEAD>{});
            read(IC<x + AHEAD + 1>{});
            __builtin_amdgcn_sched_barrier(0);
            static_for<x, x + 2>([&](auto Y) {
                constexpr int y = decltype(Y)::value;
                const op_t w = FR::template op<op_t>(ring[y % RING]);
                if constexpr (y < NV)
                    o[y % ND] = MM::mul(w, pf[y / ND], o[y % ND]);
                else
                    sc[(y - NV) % NT] = MM::mul(w, qf[(y - NV) / NT], sc[(y - NV) % NT]);
            });
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (SCORES) {
#pragma unroll
            for (int r = 0; r < NT * NR; ++r) p[r] = sc[r / NR][r % NR];
        }
    }
    // Masks the scores, and raises m and rescales the sums where it must.
    __device__ __forceinline__ void raise(int key0, int len, float (&p)[NT * NR]) {
        if (key0 + KEYS > len) {
            int k0 = key0;
            asm volatile("" : "+s"(k0));  // (the masks are not worked out ahead of this branch)
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const uint32_t on = seen8(sees, k0 + 8 * NG * s + 8 * g - len);
#pragma unroll
                for (int r = 0; r < 8; ++r) p[8 * s + r] = on >> r & 1u ? p[8 * s + r] : -__builtin_inff();
            }
        }
        lift(p);
    }
    // top: this lane's largest score
    __device__ __forceinline__ void raise_to(float top) {
        top = groups_max<RW>(top);
        const float up = fmaxf(m, top - M_BELOW<E>);
        const float f = __builtin_amdgcn_exp2f(m - up);
        m = up;
        l *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] *= f;
        far = __any(fabsf(m) >= M_FAR && m > M_START);  // (M_START: a row that has seen nothing)
    }
    // Raises m and rescales the sums where it must.
    __device__ __forceinline__ void lift(float (&p)[NT * NR]) {
        float top = p[0];
#pragma unroll
        for (int r = 1; r < NT * NR; ++r) top = fmaxf(top, p[r]);
        top *= a.score_scale;
        if (__any(top - m > M_SLACK<E>)) raise_to(top);  // (exact where it is near; P past the slack could be infinite)
        if (far) {
#pragma unroll
            for (int r = 0; r < NT * NR; ++r) p[r] *= a.score_scale;
        }
    }
    // The probabilities of step s of the second product, their sum to `sum` (a tile's,
    // which then goes to l at once: one by one, small ones would be lost beside it).
    __device__ __forceinline__ op_t probabilities(const float (&p)[NT * NR], int s, float &sum) {
        v4u w;
        const float by = far ? 1.f : a.score_scale;  // (far: scaled already)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p0 = __builtin_amdgcn_exp2f(fmaf(p[8 * s + 2 * j], by, -m));
            const float p1 = __builtin_amdgcn_exp2f(fmaf(p[8 * s + 2 * j + 1], by, -m));
            sum += p0 + p1;
            w[j] = pack2<E>(p0, p1);
        }
        return __builtin_bit_cast(op_t, w);
    }
    __device__ __forceinline__ void tile(const char *lds, int buf, int key0, int len) {
        float p[NT * NR];
        op_t pf[NS];
        products<false, true, 4>(lds, 0, pf, buf, p);
        raise(key0, len, p);
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < NS; ++s) pf[s] = probabilities(p, s, sum);
        l += sum;
        products<true, false, 4>(lds, buf + TL::K_BYTES, pf, 0, p);
    }
    // What infinite and NaN values of drafted tokens among keys [from, to) add; at a
    // piece's end, where the loop's registers are free.
    __device__ __forceinline__ void odd_values(int b, int h, const Seq &sq, int from, int to) {
#pragma nounroll
        for (int key = max(from, sq.len & -KEYS); key < to; key += 8 * NG)
            add_odd<E, F8, D, RW>(ValueRows{a.cache, a.batch, b, h, sq.total}, key, lane, [&](int k) { return seen8(sees, k - sq.len); }, o);
    }
    // the whole rows' weights (the lane groups hold parts of them)
    __device__ __forceinline__ void end() {
        l = groups_sum<RW>(l);
    }
    // end, and the rows to the output or to the workspace from row slot_row
    __device__ __forceinline__ void put(bool whole, int64_t slot_row) {
        end();
        if (!used) return;
        slot_row += n;
        const float norm = whole ? (l == 0.f ? 0.f : a.v_scale / l) : 1.f;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < NR; r += 4) {
                const int dim = RW * d + 2 * r + 4 * g;
                put4<E>(a, whole, v4f{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]} * norm, q_row * D + dim,
                        slot_row * D + dim);
            }
        if (!whole && g == 0) *reinterpret_cast<v2f *>(a.ws_ml + 2 * slot_row) = v2f{m, l};
    }
};

}  // namespace

}  // namespace kq
