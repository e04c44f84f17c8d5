// kq_attn.hip -- attention of a step's new rows (one token, or a tree of
// drafts) over a paged cache (gfx950).
//
// For each sequence and key head the T * group query rows that share the head
// are the columns of two matrix products, so that no operand and no result ever
// moves between lanes:
//   S^T [keys][rows]  = K [keys][dim] x Q^T [dim][rows]
//   O^T [dim][rows]  += V^T [dim][keys] x P^T [keys][rows],  P = exp2(S^T - m).
// A matrix-core result holds, for one column, rows 4g .. 4g + 3 (and + 8j) in
// lane group g; the operand of the next product wants 8 consecutive k of its
// column in lane group g.  Which key is row r of the first product is free, so
// the keys are dealt such that the scores a lane gets ARE the 8 consecutive
// keys it must supply.  K rows and (the cache keeps values transposed) V rows
// are then operands as they lie in memory: 16 bytes of a lane, straight into
// registers.
//
// One pass over the keys with the running maximum m and sum l of a softmax in
// fp32.  m is raised only when a score passes it by more than 8 (in log2
// units): until then exp2(S - m) stays within 2^8 of what it began at, and neither
// a cross-lane maximum nor a rescaling of O is needed.
//
// P enters the second product in q's type, since the matrix cores take two 16-bit
// operands (fp32 ones run at a sixteenth of the rate, P in two halves would double
// the products): each probability is off by up to 2^-8 (bfloat16) or 2^-11
// (float16) of it, where the output's own rounding is as much of the whole.  float16 has no
// normal numbers below 2^-14, and many small probabilities beside a dominant one can
// weigh more than a rounding, so there m is kept 7 below the maximum it is raised
// to: P begins at 2^7, stays within 2^15, and loses bits from 2^-21 of the dominant
// one down (131071 keys 25 below one: 1.9e-3 off without, 7e-5 with).  bfloat16 has
// fp32's range: there m is 20 above the maximum, so that sums of P times values stay
// in fp32 where their mean does (P from 2^-20 to 2^-12).
//
// A wave holds the sums of RW query rows (16 or 32).
//
// How the work is shared: a unit is 128 (short sequences: 1024) slots of one (sequence, key head, block
// of rows).  The lengths are known to the device alone, so every workgroup of a
// grid that just fills the chip adds up the units itself and takes an equal run
// of them, whatever the mix of lengths.  A run covers parts of at most two
// blocks and any number of whole ones; whole ones are finished where they are,
// a part leaves its sums (unnormalised, with m and l) in the workspace, and a
// second kernel joins the parts.
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

// ---------------------------------------------------------------- sharing

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

// What one wave knows of 64 sequences (lane i: sequence 64 chunk + i): their units
// for one key head and how many come before.
struct Share {
    int chunk, before, incl, all, tiles, blocks;
    bool more;  // the sequence has more rows than the call allows
};
__device__ __forceinline__ void share_chunk(const AttnArgs &a, Share &s, int chunk) {
    const int lane = threadIdx.x & 63, b = chunk * 64 + lane;
    int tiles = 0, blocks = 0;
    s.more = false;
    if (b < a.batch.n_seqs) {
        const Seq q = seq_of(a, b);
        s.more = q.rows > q.T;
        tiles = q.T ? (q.total + (1 << a.unit_shift) - 1) >> a.unit_shift : 0;
        blocks = (q.T * a.group + a.rows_wg - 1) / a.rows_wg;
    }
    int incl = tiles * blocks;
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x111, 0xF, 0xF, false);  // in rows of 16: from 1, 2, 4, 8 to the left
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x112, 0xF, 0xF, false);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x114, 0xF, 0xF, false);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x118, 0xF, 0xF, false);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x142, 0xA, 0xF, false);  // lane 15 of rows 0 and 2 to rows 1 and 3
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x143, 0xC, 0xF, false);  // lane 31 to the upper half
    s.chunk = chunk;
    s.incl = incl;
    s.tiles = tiles;
    s.blocks = blocks;
}
__device__ __forceinline__ int last_lane(int v) { return __builtin_amdgcn_readlane(v, 63); }
// The output of rows past the bound of the call: NaN, by the whole grid together.
__device__ __forceinline__ void put_past(const AttnArgs &a, const Share &s, int dim) {
    uint64_t more = __ballot(s.more);
    if (!more) return;
    const int pieces = a.cache.heads * a.group * dim / (a.out_f32 ? 4 : 8);  // of 16 bytes, to a row
    const v4u nan = {0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu};    // of every type
    for (; more; more &= more - 1) {
        const Seq q = seq_of(a, s.chunk * 64 + __ffsll((unsigned long long)more) - 1);
        v4u *out = reinterpret_cast<v4u *>(a.out) + (int64_t)(q.first + q.T) * pieces;
        const int64_t n = (int64_t)(q.rows - q.T) * pieces;
        for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
            out[i] = nan;
    }
}
// all the units of one key head, and the first chunk; one wave of the grid notes
// them for the kernel that joins the parts
__device__ __forceinline__ Share share_of(const AttnArgs &a, int dim) {
    Share s;
    share_chunk(a, s, 0);
    put_past(a, s, dim);
    s.before = 0;
    s.all = last_lane(s.incl);
    if (a.batch.n_seqs > 64) {
        Share t;
        for (int c = 1; c * 64 < a.batch.n_seqs; ++c) {
            share_chunk(a, t, c);
            put_past(a, t, dim);
            s.all += last_lane(t.incl);
        }
    }
    if (blockIdx.x == 0 && threadIdx.x < 64 && a.ws_seq) {
        Share t = s;
        for (int c = 0; c * 64 < a.batch.n_seqs; ++c) {
            if (c) {
                t.before += last_lane(t.incl);
                share_chunk(a, t, c);
            }
            const int b = c * 64 + threadIdx.x;
            if (b < a.batch.n_seqs)
                reinterpret_cast<v4i *>(a.ws_seq)[b] = v4i{t.before + t.incl - t.tiles * t.blocks, t.tiles, t.blocks, s.all};
        }
    }
    return s;
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

// One block's share of a run: keys [from, to) of a row block of a head; `whole`
// if that is all of its keys, else the workspace slot of its sums.
struct Piece {
    int b, h, rb, from, to, units;
    bool whole;
};
// the piece that unit u (of all heads) begins or continues; s moves on with u
__device__ __forceinline__ Piece piece_at(const AttnArgs &a, Share &s, int u, int end) {
    const int heads = a.cache.heads;
    const int x = u / heads;
    while (x >= s.before + last_lane(s.incl)) {
        const int before = s.before + last_lane(s.incl);
        share_chunk(a, s, s.chunk + 1);
        s.before = before;
    }
    const int lane = __ffsll((unsigned long long)__ballot(s.before + s.incl > x)) - 1;
    const int tiles = __builtin_amdgcn_readlane(s.tiles, lane), blocks = __builtin_amdgcn_readlane(s.blocks, lane);
    const int mine = tiles * blocks;
    const int in_seq = u - heads * (s.before + __builtin_amdgcn_readlane(s.incl, lane) - mine);
    Piece p;
    p.b = s.chunk * 64 + lane;
    p.h = in_seq / mine;
    const int in_head = in_seq - p.h * mine;
    p.rb = in_head / tiles;
    const int tile = in_head - p.rb * tiles;
    p.units = min(tiles - tile, end - u);
    p.from = tile << a.unit_shift;
    p.to = (tile + p.units) << a.unit_shift;  // (past the sequence's end in its last unit)
    p.whole = p.units == tiles;
    return p;
}

// Where a sequence's values lie, for what add_odd reads again.
struct ValueRows {
    const CacheArgs &cache;
    const BatchArgs &batch;
    int b, h, len, total;
};

// An infinity or NaN among the values of drafted tokens belongs to the rows that
// see its token and to no other, but a product with P would spoil them all (0 *
// inf).  Such values are zeros in the product; here they are added for one step
// of it (512 / RW keys from key0): marks of them times a 0 / 1 matrix of who
// sees what count the infinities and NaNs that reach each sum.
template <class E, bool F8, int D, int RW>
__device__ __forceinline__ void add_odd(const ValueRows &va, int key0, int lane, uint64_t sees,
                                        typename Mfma<E, RW>::acc (&o)[D / RW]) {
    typedef Mfma<E, RW> MM;
    typedef Frag<E, F8> FR;
    constexpr int ES = FR::BYTES;
    const int n = lane & (RW - 1), g = lane / RW;
    const int key = key0 + 8 * g;  // the first of this lane's 8
    const Marks<E> marks;
    const float inf = __builtin_bit_cast(float, here(0x7F800000u));
    const uint32_t on = seen8(sees, key - va.len);
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
    // The values to LDS.  In a tile that reaches past the cached slots: zeros for
    // slots past the end, which may hold anything, and for infinite and NaN values
    // of drafted tokens; whether this thread met any of those.
    __device__ __forceinline__ bool store_v(char *lds, int buf, int key0) {
        bool found = false;
        if (!stages) return false;
        if (key0 + KEYS > len) {
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
template <class E, bool F8, int D, int KEYS, int RW>
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

    __device__ __forceinline__ Attend(const AttnArgs &a_) : a(a_) {
        lane = threadIdx.x & 63;
        n = lane & (RW - 1);
        g = lane / RW;
        // this lane's row of the first product's results: see the head of the file
        const int krow = RW == 16 ? 8 * (n >> 2) + (n & 3) : 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);
        k_from = TL::k_pos(krow, F8 ? g >> 1 : g) + (F8 ? 8 * (g & 1) : 0);
        v_from = TL::v_pos(n, F8 ? g >> 1 : g) + (F8 ? 8 * (g & 1) : 0);
    }
    // 8 values of this lane: row t (and step kk) of the keys, row d (step s) of the values
    __device__ __forceinline__ raw_t k_frag(const char *lds, int at, int t, int kk) const {
        const int row = RW == 16 ? 32 * (t >> 1) + 4 * (t & 1) : 32 * t;
        return *reinterpret_cast<const raw_t *>(lds + (at ^ (kk * NG * 8 * FR::BYTES)) + row * TL::KB);
    }
    __device__ __forceinline__ raw_t v_frag(const char *lds, int at, int d, int s) const {
        return *reinterpret_cast<const raw_t *>(lds + (at ^ (s * NG * 8 * FR::BYTES)) + RW * d * TL::VB);
    }
    // begin rows row0 .. of key head h
    __device__ __forceinline__ void begin(const Seq &sq, int h, int row0) {
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
        sees = 0;
        if (used) sees = (a.mask ? a.mask[sq.first + tok] : (2ull << tok) - 1ull) & first_bits(sq.total - sq.len);
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] = acc_t{};
        m = M_START;
        l = 0.f;
        far = false;
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
        float top = p[0];
#pragma unroll
        for (int r = 1; r < NT * NR; ++r) top = fmaxf(top, p[r]);
        top *= a.score_scale;
        if (__any(top - m > M_SLACK<E>)) {  // (exact where it is near; P past the slack could be infinite)
            top = groups_max<RW>(top);
            const float up = fmaxf(m, top - M_BELOW<E>);
            const float f = __builtin_amdgcn_exp2f(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] *= f;
            far = __any(fabsf(m) >= M_FAR && m > M_START);  // (M_START: a row that has seen nothing)
        }
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
            add_odd<E, F8, D, RW>(ValueRows{a.cache, a.batch, b, h, sq.len, sq.total}, key, lane, sees, o);
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

// Bound: HBM bandwidth.  64 sequences of up to 8191 slots, 4 rows to a key head of 128,
// bfloat16: 218 us for 1.39 GB, 6.4 TB/s; two of 131k slots in 8 bits, 8 rows: 79 us
// for 473 MB, 6.0 TB/s.
// Up to 16 rows: one wave's worth, so the waves of a workgroup take tiles in
// turn, each its own in LDS without a barrier, and their sums are joined in LDS.
template <class E, bool F8, int D, int WAVES>
__global__ __launch_bounds__(WAVES * 64, D == 256 || WAVES == 8 ? 1 : 2) void attn_few_kernel(const AttnArgs a) {
    constexpr int RW = 16;
    constexpr int KEYS = D * (F8 ? 1 : 2) >= 256 ? 32 : 64;
    typedef Tile<E, F8, D, KEYS, RW, 64, true> TL;
    typedef Attend<E, F8, D, KEYS, RW> AT;
    constexpr int O_FLOATS = RW * (D + 4);
    constexpr int WAVE_BYTES = TL::BYTES > O_FLOATS * 4 ? TL::BYTES : (O_FLOATS * 4 + 1023) / 1024 * 1024;

    __shared__ __align__(1024) char lds[WAVES * WAVE_BYTES];  // a wave's tile, then its sums [row][dim]
    __shared__ float lm[WAVES * RW], ll[WAVES * RW];

    Share share = share_of(a, D);
    const int heads = a.cache.heads, units = share.all * heads, groups = min((int)gridDim.x, units);
    if ((int)blockIdx.x >= groups) return;
    const Runs runs(units, groups);
    const int begin = runs.begin(blockIdx.x), end = runs.begin(blockIdx.x + 1);

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mine = wave * WAVE_BYTES;
    TL tl(a, threadIdx.x & 63);
    AT at(a);

    for (int u = begin; u < end;) {
        const Piece pc = piece_at(a, share, u, end);
        const Seq sq = seq_of(a, pc.b);
        const int R = sq.T * a.group, to = min(pc.to, sq.total);
        tl.aim(pc.b, pc.h, sq);
        int key0 = pc.from + KEYS * wave;
        typename TL::Place next = tl.find(key0);
        tl.load_k(next);
        tl.load_v(next);
        next = tl.find(key0 + WAVES * KEYS);
        at.begin(sq, pc.h, 0);
        if (u != begin) __syncthreads();  // the piece before has been joined
        bool odd = false;
        for (; key0 < to; key0 += WAVES * KEYS) {
            tl.store_k(lds, mine);
            odd |= tl.store_v(lds, mine + TL::K_BYTES, key0);
            if (key0 + WAVES * KEYS < to) {
                tl.load_k(next);
                tl.load_v(next);
                next = tl.find(key0 + 2 * WAVES * KEYS);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            at.tile(lds, mine, key0, sq.len);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        if (__any(odd)) {
            for (key0 = pc.from + KEYS * wave; key0 < to; key0 += WAVES * KEYS)
                at.odd_values(pc.b, pc.h, sq, key0, min(key0 + KEYS, to));
        }
        at.end();

        // Join the waves.
        float *lo = reinterpret_cast<float *>(lds + mine);
#pragma unroll
        for (int d = 0; d < AT::ND; ++d) *reinterpret_cast<v4f *>(lo + at.n * (D + 4) + d * RW + 4 * at.g) = at.o[d];
        if (at.g == 0) {
            lm[wave * RW + at.n] = at.m;
            ll[wave * RW + at.n] = at.l;
        }
        __syncthreads();
        const int row = threadIdx.x >> 4, jt = threadIdx.x & 15;  // 16 threads to a row
        if (row < R) {
            float mm = M_START;
#pragma unroll
            for (int k = 0; k < WAVES; ++k) mm = fmaxf(mm, lm[row + k * RW]);
            float f[WAVES], sum = 0.f;
#pragma unroll
            for (int k = 0; k < WAVES; ++k) {
                f[k] = __builtin_amdgcn_exp2f(lm[row + k * RW] - mm);
                sum += f[k] * ll[row + k * RW];
            }
            const int64_t slot_row = (2 * (int64_t)blockIdx.x + (u != begin)) * a.slot_rows + row;
            const float norm = pc.whole ? (sum == 0.f ? 0.f : a.v_scale / sum) : 1.f;
            const int64_t o_row =
                (int64_t)(sq.first + row / a.group) * ((int64_t)heads * a.group) + pc.h * a.group + row % a.group;
#pragma unroll
            for (int v = 0; v < D; v += 64) {
                const int dim = v + jt * 4;
                v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < WAVES; ++k)
                    acc += f[k] * *reinterpret_cast<const v4f *>(lds + k * WAVE_BYTES + (row * (D + 4) + dim) * 4);
                put4<E>(a, pc.whole, acc * norm, o_row * D + dim, slot_row * D + dim);
            }
            if (!pc.whole && jt == 0) *reinterpret_cast<v2f *>(a.ws_ml + 2 * slot_row) = v2f{mm, sum};
        }
        u += pc.units;
    }
}

// More rows, up to 4 waves' worth: the waves share the tiles (two in LDS: one in
// use, one being written; the registers hold the one after), so memory is read
// once for all the rows.  24 trees of up to 24 tokens, 4 rows to a token, heads of 64,
// up to 4100 slots: 30 us for 65 MB, bound by the begin and end of runs of 4 units.
template <class E, bool F8, int D>
__global__ __launch_bounds__(256, 2) void attn_tile_kernel(const AttnArgs a) {
    constexpr int RW = 32, KEYS = D == 128 ? 32 : 64;  // (64 at dim 128 would not fit the registers)
    typedef Tile<E, F8, D, KEYS, RW, 256, true> TL;
    typedef Attend<E, F8, D, KEYS, RW> AT;

    __shared__ __align__(1024) char lds[2 * TL::BYTES];
    __shared__ int odd;  // whether drafted tokens staged so far have infinite or NaN values

    Share share = share_of(a, D);
    const int heads = a.cache.heads, units = share.all * heads, groups = min((int)gridDim.x, units);
    if ((int)blockIdx.x >= groups) return;
    const Runs runs(units, groups);
    const int begin = runs.begin(blockIdx.x), end = runs.begin(blockIdx.x + 1);

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    TL tl(a, threadIdx.x);
    AT at(a);
    if (threadIdx.x == 0) odd = 0;

    for (int u = begin; u < end;) {
        const Piece pc = piece_at(a, share, u, end);
        const Seq sq = seq_of(a, pc.b);
        const int to = min(pc.to, sq.total);
        tl.aim(pc.b, pc.h, sq);
        typename TL::Place next = tl.find(pc.from);
        tl.load_k(next);
        tl.load_v(next);
        next = tl.find(pc.from + KEYS);
        const int row0 = pc.rb * a.rows_wg + wave * RW;
        // (a wave without rows only stages: trees of 5 tokens by 4 heads over 16k slots 77 -> 65 us)
        const bool rows = row0 < sq.T * a.group;
        at.begin(sq, pc.h, row0);
        __syncthreads();  // the piece before has been read
        tl.store_k(lds, 0);
        if (tl.store_v(lds, TL::K_BYTES, pc.from)) odd = 1;
        tl.load_k(next);
        tl.load_v(next);
        next = tl.find(pc.from + 2 * KEYS);
        int buf = 0;
        for (int key0 = pc.from; key0 < to; key0 += KEYS) {
            __syncthreads();
            if (rows) at.tile(lds, buf, key0, sq.len);
            buf = TL::BYTES - buf;
            if (key0 + KEYS < to) {
                tl.store_k(lds, buf);
                if (tl.store_v(lds, buf + TL::K_BYTES, key0 + KEYS)) odd = 1;
                tl.load_k(next);
                tl.load_v(next);
                next = tl.find(key0 + 3 * KEYS);
            }
        }
        if (odd) at.odd_values(pc.b, pc.h, sq, pc.from, to);
        at.put(pc.whole, (2 * (int64_t)blockIdx.x + (u != begin)) * a.slot_rows + wave * RW);
        u += pc.units;
    }
}

// Still more rows: 8 waves, two to a SIMD, share the tiles, and the second four
// run half a turn behind the first.  A turn has a half of matrix products (the
// values of the tile before, the scores of this one) and a half of vector work
// (softmax, staging), as long as each other, so that one wave of a SIMD keeps its
// matrix unit busy while the other has its vector unit; a barrier ends every half
// (the later waves meet one more at the begin, the earlier ones at the end).
// Times in halves: the early waves multiply tile i at 2 i, the late ones at 2 i + 1.
// Each wave stages its share of keys i + 2 and values i + 1 after scores i, so
// early or late they are in LDS by 2 i + 3, before anyone's products at 2 i + 4; what
// they overwrite, keys i - 1 and values i - 2 (three of each in LDS), was last read at
// 2 i - 1.
// Bound: matrix products and softmax on one SIMD.  512 rows to a key head of 128: 860
// TFLOP/s at even load (8 trees of 64 over 16384 slots each, 320 us with the join),
// 168 - 216 us for 1.2e11 operations on 8 ragged trees.
template <class E, bool F8, int D>
__global__ __launch_bounds__(512, 2) void attn_wide_kernel(const AttnArgs a) {
    constexpr int RW = D == 256 ? 16 : 32, KEYS = D == 256 ? 32 : 64;
    typedef Tile<E, F8, D, KEYS, RW, 512, false> TL;
    typedef Attend<E, F8, D, KEYS, RW> AT;

    __shared__ __align__(1024) char lds[3 * TL::BYTES];  // keys and values by turns
    __shared__ int odd;  // whether drafted tokens staged so far have infinite or NaN values

    Share share = share_of(a, D);
    const int heads = a.cache.heads, units = share.all * heads, groups = min((int)gridDim.x, units);
    if ((int)blockIdx.x >= groups) return;
    const Runs runs(units, groups);
    const int begin = runs.begin(blockIdx.x), end = runs.begin(blockIdx.x + 1);

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool late = wave >= 4;
    TL tl(a, threadIdx.x);
    AT at(a);
    if (threadIdx.x == 0) odd = 0;

    for (int u = begin; u < end;) {
        const Piece pc = piece_at(a, share, u, end);
        const Seq sq = seq_of(a, pc.b);
        const int to = min(pc.to, sq.total), tiles = (to - pc.from + KEYS - 1) / KEYS;
        tl.aim(pc.b, pc.h, sq);
        // keys 0, 1 and values 0 to LDS; keys 2 and values 1 on their way
        typename TL::Place p0 = tl.find(pc.from), p1 = tl.find(pc.from + KEYS), p2 = tl.find(pc.from + 2 * KEYS);
        tl.load_k(p0);
        tl.load_v(p0);
        at.begin(sq, pc.h, pc.rb * a.rows_wg + wave * RW);
        __syncthreads();  // the piece before has been read
        tl.store_k(lds, 0);
        if (tl.store_v(lds, TL::K_BYTES, pc.from)) odd = 1;
        tl.load_k(p1);
        tl.store_k(lds, TL::BYTES);
        tl.load_v(p1);
        tl.load_k(p2);
        p1 = p2;
        p2 = tl.find(pc.from + 3 * KEYS);
        float p[AT::NT * AT::NR];
        typename AT::op_t pf[AT::NS];
        int key0 = pc.from, buf = 0;  // buf: where tile i is (i % 3)
        __syncthreads();
        if (late) __syncthreads();
        auto vector_half = [&](int i, int before, int after) {
            at.raise(key0, sq.len, p);
            float sum = 0.f;
#pragma unroll
            for (int s = 0; s < AT::NS; ++s) {
                v4u w = __builtin_bit_cast(v4u, at.probabilities(p, s, sum));
                asm volatile("" : "+v"(w));  // (now, while the loads for the staging below arrive)
                pf[s] = __builtin_bit_cast(typename AT::op_t, w);
            }
            at.l += sum;
            if (i + 1 < tiles) {
                tl.store_k(lds, before);  // keys i + 2
                if (tl.store_v(lds, after + TL::K_BYTES, key0 + KEYS)) odd = 1;
                tl.load_v(p1);
                tl.load_k(p2);
                p1 = p2;
                p2 = tl.find(key0 + 4 * KEYS);
            }
        };
        at.template products<false, true, 6>(lds, 0, pf, 0, p);
        __syncthreads();
        vector_half(0, 2 * TL::BYTES, TL::BYTES);
        __syncthreads();
        for (int i = 1; i < tiles; ++i) {
            key0 += KEYS;
            const int before = buf;
            buf = buf == 2 * TL::BYTES ? 0 : buf + TL::BYTES;
            at.template products<true, true, 6>(lds, before + TL::K_BYTES, pf, buf, p);
            __syncthreads();
            vector_half(i, before, buf == 2 * TL::BYTES ? 0 : buf + TL::BYTES);
            __syncthreads();
        }
        at.template products<true, false, 6>(lds, buf + TL::K_BYTES, pf, 0, p);
        __syncthreads();
        if (!late) __syncthreads();
        if (odd) at.odd_values(pc.b, pc.h, sq, pc.from, to);
        at.put(pc.whole, (2 * (int64_t)blockIdx.x + (u != begin)) * a.slot_rows + wave * RW);
        u += pc.units;
    }
}

// out = sum over the parts of a cut block, each weighted by exp2(its maximum -
// the largest).  A workgroup has `rows` (1 or group) rows of a token's heads; D / 4
// threads read a part's sums, and the 256 / (D / 4) such sets share out the rows
// and, where there are more sets than rows, the parts.
template <class E, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a, int rows) {
    constexpr int TPP = D / 4, SETS = 256 / TPP;
    __shared__ v4f so[256];
    __shared__ v2f sml[SETS];
    const int heads = a.cache.heads, G = a.group;
    const int tok = blockIdx.x, head0 = blockIdx.y * rows, h = head0 / G;
    const int b = batch_seq(a.batch, tok);
    const Seq sq = seq_of(a, b);
    const int i = tok - sq.first;
    if (i < 0 || i >= sq.T) return;
    const v4i sh = reinterpret_cast<const v4i *>(a.ws_seq)[b];  // units before, tiles, blocks, all units
    const int units = sh[3] * heads, tiles = sh[1];
    const Runs runs(units, min(a.grid, units));
    int sets = 1;  // sets of threads to a row
    while (2 * sets * rows <= SETS) sets *= 2;
    const int lane = threadIdx.x % TPP, set = threadIdx.x / TPP, sub = set % sets;
    for (int j = set / sets; j < rows + SETS; j += SETS / sets) {  // (the same number of turns for all)
        if (j - set / sets >= rows) break;
        const int row = i * G + head0 % G + min(j, rows - 1), rb = row / a.rows_wg;
        const int from = heads * sh[0] + h * tiles * sh[2] + rb * tiles;
        // the workgroups that hold the block's first and last unit
        const int w0 = runs.holder(from), w1 = runs.holder(from + tiles - 1);
        float m = M_START, l = 0.f;
        v4f o = {0.f, 0.f, 0.f, 0.f};
        for (int w = w0 == w1 ? w1 + 1 : w0 + sub; w <= w1; w += sets) {  // (one workgroup: finished there)
            // a workgroup's first piece lies in its first slot
            const int second = runs.begin(w) < from;
            const int64_t r = (2 * (int64_t)w + second) * a.slot_rows + (row - rb * a.rows_wg);
            const v2f ml = *reinterpret_cast<const v2f *>(a.ws_ml + 2 * r);
            const v4f po = *reinterpret_cast<const v4f *>(a.ws_o + r * D + 4 * lane);
            const float up = fmaxf(m, ml[0]);
            const float f = __builtin_amdgcn_exp2f(m - up), pf = __builtin_amdgcn_exp2f(ml[0] - up);
            m = up;
            l = l * f + ml[1] * pf;
            o = o * f + po * pf;
        }
        if (sets > 1) {
            __syncthreads();
            so[threadIdx.x] = o;
            if (lane == 0) sml[set] = v2f{m, l};
            __syncthreads();
            if (sub == 0) {
                for (int k = 1; k < sets; ++k) {
                    const v2f ml = sml[set + k];
                    const float up = fmaxf(m, ml[0]);
                    const float f = __builtin_amdgcn_exp2f(m - up), pf = __builtin_amdgcn_exp2f(ml[0] - up);
                    m = up;
                    l = l * f + ml[1] * pf;
                    o = o * f + so[threadIdx.x + k * TPP] * pf;
                }
            }
        }
        if (sub == 0 && j < rows && w0 != w1) {
            const float norm = l == 0.f ? 0.f : a.v_scale / l;
            put4<E>(a, true, o * norm, ((int64_t)tok * ((int64_t)heads * G) + head0 + j) * D + 4 * lane, 0);
        }
    }
}

template <class E, bool F8, int D>
hipError_t launch_dim(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    const dim3 grid((unsigned)p.grid);
    if constexpr (D < 256) {
        if (p.waves == 0 && p.unit_shift != ATTN_UNIT_SHIFT) {
            hipLaunchKernelGGL((attn_few_kernel<E, F8, D, 8>), grid, dim3(512), 0, stream, a);
            return hipGetLastError();
        }
    }
    if (p.waves == 0)
        hipLaunchKernelGGL((attn_few_kernel<E, F8, D, 4>), grid, dim3(256), 0, stream, a);
    else if (p.waves == 8)
        hipLaunchKernelGGL((attn_wide_kernel<E, F8, D>), grid, dim3(512), 0, stream, a);
    else if constexpr (D < 256)
        hipLaunchKernelGGL((attn_tile_kernel<E, F8, D>), grid, dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.bytes == 0) return e;  // no workspace: nothing is cut
    // many rows: the heads of a group together, which find their parts once
    const int heads = a.cache.heads * a.group;
    const int rows = (int64_t)a.batch.n_tokens * heads > 2048 ? a.group : 1;
    hipLaunchKernelGGL((attn_join_kernel<E, D>), dim3((unsigned)a.batch.n_tokens, (unsigned)(heads / rows)), dim3(256), 0,
                       stream, a, rows);
    return hipGetLastError();
}

template <class E, bool F8>
hipError_t launch_type(const AttnArgs &a, const AttnPlan &p, int dim, hipStream_t stream) {
    switch (dim) {
        case 64: return launch_dim<E, F8, 64>(a, p, stream);
        case 128: return launch_dim<E, F8, 128>(a, p, stream);
        default: return launch_dim<E, F8, 256>(a, p, stream);
    }
}

}  // namespace

hipError_t launch_attn(const AttnArgs &a, const AttnPlan &p, int type, int dim, int q_type, hipStream_t stream) {
    if (q_type == KQ_T_BF16)
        return type == KQ_T_F8 ? launch_type<__bf16, true>(a, p, dim, stream)
                               : launch_type<__bf16, false>(a, p, dim, stream);
    return type == KQ_T_F8 ? launch_type<_Float16, true>(a, p, dim, stream)
                           : launch_type<_Float16, false>(a, p, dim, stream);
}

}  // namespace kq
