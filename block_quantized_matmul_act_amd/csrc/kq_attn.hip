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
// units): until then exp2(S - m) stays within 2^8, far inside every type, and
// neither a cross-lane maximum nor a rescaling of O is needed.
//
// A wave holds the sums of RW query rows (16 or 32).  A sequence's slots are cut
// into parts so that few long sequences fill the chip; a second kernel joins
// the parts.
#include "kq_step_device.hpp"

namespace kq {

namespace {

constexpr float M_START = -1e30f;  // below every score, and finite: exp2(-inf - m) is 0, not NaN
constexpr float M_SLACK = 8.f;

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

// Which of 8 keys a row sees (bit e: the e-th), the first being node `node` of
// the drafted tokens (below 0: that many cached ones come first).  sees: the
// row's mask, cut to the sequence's rows.
__device__ __forceinline__ uint32_t seen8(uint64_t sees, int node) {
    const uint32_t drafted = node > 63 ? 0u : (uint32_t)(sees >> (node & 63));
    const int cached = min(max(-node, 0), 8);
    const uint32_t both = (uint32_t)sees << cached | ((1u << cached) - 1u);
    return node >= 0 ? drafted : both;
}

// Marks of infinite and NaN values: whole numbers that both 16-bit types hold,
// set so far apart that sums of 32 do not run into the next.
constexpr float MARK_POS = 1.f, MARK_NEG = 128.f, MARK_NAN = 16384.f;

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
    // a value's mark: see add_odd
    static __device__ __forceinline__ float mark(raw r, int i) {
        constexpr uint32_t e = std::is_same_v<E, __bf16> ? 0x7F80u : 0x7C00u;
        const uint32_t x = r[i >> 1] >> (16 * (i & 1)) & 0xFFFFu;
        return (x & 0x7FFFu) < e ? 0.f : (x & 0x7FFFu) > e ? MARK_NAN : x >> 15 ? MARK_NEG : MARK_POS;
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
    static __device__ __forceinline__ float mark(raw r, int i) {
        return ((r[i >> 2] >> (8 * (i & 3))) & 0x7Fu) == 0x7Fu ? MARK_NAN : 0.f;
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
    const uint32_t on = seen8(sees, key - va.len);
    v4u w = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 1] |= (on >> e & 1u) * (pack2<E>(1.f, 0.f) << (16 * (e & 1)));
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
        for (int j = 0; j < 4; ++j) w[j] = pack2<E>(FR::mark(r, 2 * j), FR::mark(r, 2 * j + 1));
        const typename MM::acc count =
            MM::mul(__builtin_bit_cast(typename MM::op, w), seen, typename MM::acc{});
#pragma unroll
        for (int i = 0; i < RW * RW / 64; ++i) {
            const int c = (int)count[i];
            float x = (c & 127) ? __builtin_inff() : 0.f;
            x = c & (127 << 7) ? x - __builtin_inff() : x;
            o[d][i] += c >> 14 ? __builtin_nanf("") : x;
        }
        __builtin_amdgcn_sched_barrier(0);  // one at a time: this path must not cost the others registers
    }
}

// Up to 16 rows: one wave's worth, so the 4 waves of a workgroup cut the keys
// (32 at a time in turn) and their sums are joined in LDS.
template <class E, bool F8, int D>
__global__ __launch_bounds__(256, D == 64 ? 4 : D == 128 ? 3 : 2) void attn_few_kernel(const AttnArgs a) {
    constexpr int RW = 16;
    typedef Mfma<E, RW> MM;
    typedef typename MM::op op_t;
    typedef typename MM::acc acc_t;
    typedef Frag<E, F8> FR;
    typedef typename FR::raw raw_t;
    constexpr int NK = D / 32;  // steps of the first product
    constexpr int ND = D / RW;  // results of the second product
    constexpr int ES = FR::BYTES;

    __shared__ float lo[4 * RW * (D + 4)];  // sums of the waves: [wave][row][dim]
    __shared__ float lm[4 * RW], ll[4 * RW];

    // part c of key head h of sequence b
    const int64_t item = blockIdx.x;
    const int c = (int)(item % a.parts);
    const int h = (int)(item / a.parts % a.cache.heads);
    const int b = (int)(item / a.parts / a.cache.heads);
    int first, T;
    batch_rows(a.batch, b, first, T);
    T = min(T, a.max_tokens);
    const int G = a.group, R = T * G;
    const int len = max(a.batch.lens[b], 0);
    const int total = min(len, INT32_MAX - 64) + T;
    const int from = c * a.part;
    if (R == 0 || from >= total) return;
    const int to = min(from + a.part, total);

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const bool used = n < R;
    const int tok = used ? n / G : 0;
    const int head = h * G + (used ? n % G : 0);
    const int64_t q_row = (int64_t)(first + tok) * ((int64_t)a.cache.heads * G) + head;

    op_t qf[NK];
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
        v4u w = {0u, 0u, 0u, 0u};
        if (used) w = *reinterpret_cast<const v4u *>(a.q + (q_row * D + 32 * kk + 8 * g) * 2);
        qf[kk] = __builtin_bit_cast(op_t, w);
    }
    uint64_t sees = 0;
    if (used) sees = (a.mask ? a.mask[first + tok] : (2ull << tok) - 1ull) & ((2ull << (T - 1)) - 1ull);

    // Key of this lane's row of the first product's two results (of 16 keys each):
    // see the head of the file.
    const int krow[2] = {8 * (n >> 2) + (n & 3), 8 * (n >> 2) + 4 + (n & 3)};
    // Addresses: 16 consecutive slots from a multiple of 16 lie in one page, so a
    // tile of 32 has two runs whose addresses are the same for the whole wave
    // (scalar registers); a lane adds its place in its run, which never changes.
    const int page_shift = a.cache.page_shift;
    const int page_mask = (1 << page_shift) - 1;
    const int64_t head_bytes = (int64_t)D * ES << page_shift;
    const int heads = a.cache.heads;
    const int last_run = (total - 1) & ~15;
    struct Runs {
        int64_t page[2];  // offset of the head's page
        int slot[2];      // place in it
    };
    auto runs = [&](int key) {
        Runs r;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int slot = min(key + 16 * i, last_run);  // (a run past the end: the last one again, masked)
            r.page[i] = ((int64_t)slot_page(a.cache, a.batch, b, slot) * heads + h) * head_bytes;
            r.slot[i] = slot & page_mask;
        }
        return r;
    };
    // (both of a lane's keys lie in the same run)
    auto load_k = [&](const Runs &ru, raw_t(&kf)[2][NK]) {
        const int64_t at = n >> 3 ? ru.page[1] + ru.slot[1] * (D * ES) : ru.page[0] + ru.slot[0] * (D * ES);
        const char *p = a.cache.k + at + ((krow[0] & 15) * (D * ES) + 8 * g * ES);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) kf[t][kk] = *reinterpret_cast<const raw_t *>(p + (4 * t * D + 32 * kk) * ES);
    };
    auto load_v = [&](const Runs &ru, raw_t(&vf)[ND]) {
        const int64_t at = g >> 1 ? ru.page[1] + ru.slot[1] * ES : ru.page[0] + ru.slot[0] * ES;
        const char *p = a.cache.v + at + ((n << page_shift) + 8 * (g & 1)) * ES;
        const int step = (RW * ES) << page_shift;
#pragma unroll
        for (int d = 0; d < ND; ++d) vf[d] = *reinterpret_cast<const raw_t *>(p + d * step);
    };

    acc_t o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = acc_t{};
    float m = M_START, l = 0.f;

    int key0 = from + 32 * wave;
    Runs ru = runs(key0);
    // Keys are loaded a turn ahead, values at the turn's begin, where the
    // registers hold both (512 bytes of a lane at dim 256 they do not: there
    // each is loaded when the other is done with).
    constexpr bool AHEAD = D * ES <= 256;
    raw_t kf[2][NK];
    if (AHEAD && key0 < to) load_k(ru, kf);
    for (; key0 < to; key0 += 128) {
        raw_t vf[ND];
        const int next = key0 + 128;
        if constexpr (AHEAD) {
            load_v(ru, vf);
            ru = runs(next);
        } else {
            load_k(ru, kf);
        }

        acc_t sc[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            sc[t] = acc_t{};
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) sc[t] = MM::mul(FR::template op<op_t>(kf[t][kk]), qf[kk], sc[t]);
        }
        if constexpr (AHEAD) {
            if (next < to) load_k(ru, kf);
        } else {
            load_v(ru, vf);
            ru = runs(next);
        }

        // p[e]: key key0 + 8 g + e of this lane's row
        float p[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) p[r] = sc[r >> 2][r & 3] * a.score_scale;
        const bool ragged = key0 + 32 > len;
        if (ragged) {
            const uint32_t on = seen8(sees, key0 + 8 * g - len);
#pragma unroll
            for (int r = 0; r < 8; ++r) p[r] = on >> r & 1u ? p[r] : -__builtin_inff();
        }
        float top = p[0];
#pragma unroll
        for (int r = 1; r < 8; ++r) top = fmaxf(top, p[r]);
        if (__any(top > m + M_SLACK)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float up = fmaxf(m, top);
            const float f = __builtin_amdgcn_exp2f(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] *= f;
        }
        v4u w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p0 = __builtin_amdgcn_exp2f(p[2 * j] - m), p1 = __builtin_amdgcn_exp2f(p[2 * j + 1] - m);
            l += p0 + p1;
            w[j] = pack2<E>(p0, p1);
        }
        const op_t pf = __builtin_bit_cast(op_t, w);
        bool odd = false;
        if (ragged) {
            // slots past the end hold anything: zeros
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                FR::first(vf[d], min(max(total - (key0 + 8 * g), 0), 8));
                odd |= FR::drop_odd(vf[d]);
            }
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d] = MM::mul(FR::template op<op_t>(vf[d]), pf, o[d]);
        if (__any(odd)) add_odd<E, F8, D, RW>(ValueRows{a.cache, a.batch, b, h, len, total}, key0, lane, sees, o);
    }

    // Join the waves.
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
#pragma unroll
    for (int d = 0; d < ND; ++d) *reinterpret_cast<v4f *>(lo + (wave * RW + n) * (D + 4) + d * RW + 4 * g) = o[d];
    if (g == 0) {
        lm[wave * RW + n] = m;
        ll[wave * RW + n] = l;
    }
    __syncthreads();
    const int out_row = threadIdx.x >> 4, jt = threadIdx.x & 15;  // 16 threads to a row
    if (out_row >= R) return;
    float mm = M_START;
#pragma unroll
    for (int k = 0; k < 4; ++k) mm = fmaxf(mm, lm[out_row + k * RW]);
    float f[4], sum = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[k] = __builtin_amdgcn_exp2f(lm[out_row + k * RW] - mm);
        sum += f[k] * ll[out_row + k * RW];
    }
    const int64_t part_row = (((int64_t)b * heads + h) * a.parts + c) * ((int64_t)a.max_tokens * G) + out_row;
    const bool whole = a.parts == 1;
    const float norm = whole ? (sum == 0.f ? 0.f : a.v_scale / sum) : 1.f;
    const int64_t o_row = ((int64_t)(first + out_row / G) * ((int64_t)heads * G) + h * G + out_row % G) * D;
#pragma unroll
    for (int v = 0; v < D; v += 64) {
        const int dim = v + jt * 4;
        v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 4; ++k) acc += f[k] * *reinterpret_cast<const v4f *>(lo + (out_row + k * RW) * (D + 4) + dim);
        acc *= norm;
        if (!whole)
            *reinterpret_cast<v4f *>(a.ws_o + part_row * D + dim) = acc;
        else if (a.out_f32)
            *reinterpret_cast<v4f *>(reinterpret_cast<float *>(a.out) + o_row + dim) = acc;
        else
            *reinterpret_cast<v2u *>(a.out + (o_row + dim) * 2) = v2u{pack2<E>(acc[0], acc[1]), pack2<E>(acc[2], acc[3])};
    }
    if (!whole && jt == 0) {
        a.ws_ml[2 * part_row] = mm;
        a.ws_ml[2 * part_row + 1] = sum;
    }
}

// The same sums for sequences that bring more than a wave's rows: 4 waves of 32
// rows share tiles of KEYS keys staged in LDS (two tiles: one in use, one being
// written; the registers hold the one after).  Read from memory a line at a
// time, a tile is read once for 128 rows instead of once for each wave.
// LDS holds 16-byte pieces; a row's pieces are permuted by an XOR with bits of
// the row, so that the lanes of a read, which want one piece of many rows, meet
// different banks.
template <class E, bool F8, int D>
struct Tile {
    static constexpr int ES = F8 ? 1 : 2;
    static constexpr int KEYS = D == 256 ? 32 : 64;
    static constexpr int KB = D * ES, VB = KEYS * ES;          // bytes of a key row and of a feature row
    static constexpr int KP = KB / 16, VP = VB / 16;           // their 16-byte pieces
    static constexpr int KROWS = KEYS / 4, VROWS = D / 4;      // rows that one wave stages
    static constexpr int KN = KROWS * KB / 1024, VN = VROWS * VB / 1024;  // loads of a lane
    static constexpr int K_BYTES = KEYS * KB, BYTES = K_BYTES + D * VB;

    static __device__ __forceinline__ int k_pos(int key, int piece) {
        const int f = KP >= 8 ? (key & 3) | ((key >> 1) & 4) : (key >> 1) & (KP - 1);
        return key * KB + (piece ^ f) * 16;
    }
    static __device__ __forceinline__ int v_pos(int d, int piece) {
        const int f = VP == 8 ? d & 7 : VP == 4 ? (d >> 1) & 3 : (d >> 2) & 1;
        return K_BYTES + d * VB + (piece ^ f) * 16;
    }
};

template <class E, bool F8, int D>
__global__ __launch_bounds__(256, 2) void attn_tile_kernel(const AttnArgs a) {
    constexpr int RW = D == 256 ? 16 : 32;
    typedef Mfma<E, RW> MM;
    typedef typename MM::op op_t;
    typedef typename MM::acc acc_t;
    typedef Frag<E, F8> FR;
    typedef typename FR::raw raw_t;
    typedef Tile<E, F8, D> TL;
    constexpr int ES = TL::ES, KEYS = TL::KEYS;
    constexpr int NG = 64 / RW;                    // lane groups: 8 of a step's keys, 8 of a step's features to each
    constexpr int NK = D / (8 * NG), ND = D / RW;  // steps of the first product, results of the second
    constexpr int NT = KEYS / RW, NS = KEYS / (8 * NG);  // results of the first, steps of the second
    constexpr int NR = RW * RW / 64;

    __shared__ __align__(16) char tile[2 * TL::BYTES];
    __shared__ int odd;  // whether drafted tokens staged so far have infinite or NaN values

    const int id = blockIdx.x;
    const int rb = (id >> 3) % a.row_blocks;
    const int64_t item = (int64_t)((id >> 3) / a.row_blocks) * 8 + (id & 7);
    const int c = (int)(item % a.parts);
    const int h = (int)(item / a.parts % a.cache.heads);
    const int64_t b64 = item / a.parts / a.cache.heads;
    if (b64 >= a.batch.n_seqs) return;
    const int b = (int)b64;
    int first, T;
    batch_rows(a.batch, b, first, T);
    T = min(T, a.max_tokens);
    const int G = a.group, R = T * G;
    const int len = max(a.batch.lens[b], 0);
    const int total = min(len, INT32_MAX - 64) + T;
    const int from = c * a.part;
    if (rb * a.rows_wg >= R || from >= total) return;
    const int to = min(from + a.part, total);

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & (RW - 1), g = lane / RW;
    const int row = rb * a.rows_wg + wave * RW + n;
    const bool used = row < R;
    const int tok = used ? row / G : 0;
    const int head = h * G + (used ? row % G : 0);
    const int heads = a.cache.heads;
    const int64_t q_row = (int64_t)(first + tok) * ((int64_t)heads * G) + head;

    op_t qf[NK];
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
        v4u w = {0u, 0u, 0u, 0u};
        if (used) w = *reinterpret_cast<const v4u *>(a.q + (q_row * D + 8 * (NG * kk + g)) * 2);
        qf[kk] = __builtin_bit_cast(op_t, w);
    }
    uint64_t sees = 0;
    if (used) sees = (a.mask ? a.mask[first + tok] : (2ull << tok) - 1ull) & ((2ull << (T - 1)) - 1ull);

    // staging: this lane's rows and pieces
    const int page_shift = a.cache.page_shift, page_mask = (1 << page_shift) - 1;
    const int64_t head_bytes = (int64_t)D * ES << page_shift;
    const int last_run = (total - 1) & ~15;
    const int k_row = wave * TL::KROWS + lane / TL::KP, k_piece = lane % TL::KP;  // + i * 64 / KP
    const int v_row = wave * TL::VROWS + lane / TL::VP, v_piece = lane % TL::VP;
    const int v_run = v_piece * (16 / ES) >> 4;
    const int v_off = (v_row << page_shift) * ES + (v_piece * 16 & (16 * ES - 1));
    v4u stage[TL::KN + TL::VN];
    auto head_page = [&](int slot) { return ((int64_t)slot_page(a.cache, a.batch, b, slot) * heads + h) * head_bytes; };
    auto load = [&](int key0) {
        const int k_slot = min(key0 + (wave * TL::KROWS & ~15), last_run);  // one run to a wave
        const char *kp = a.cache.k + head_page(k_slot) + (k_slot & page_mask) * TL::KB;
        const int k_off = (k_row & 15) * TL::KB + k_piece * 16;
#pragma unroll
        for (int i = 0; i < TL::KN; ++i) stage[i] = *reinterpret_cast<const v4u *>(kp + k_off + i * 1024);
        const char *vp = a.cache.v;
        int64_t at = 0;
#pragma unroll
        for (int r = 0; r < KEYS / 16; ++r) {
            const int slot = min(key0 + 16 * r, last_run);
            const int64_t o = head_page(slot) + (slot & page_mask) * ES;
            at = r == v_run ? o : at;
        }
        vp += at + v_off;
#pragma unroll
        for (int i = 0; i < TL::VN; ++i)
            stage[TL::KN + i] = *reinterpret_cast<const v4u *>(vp + ((int64_t)(i * (64 / TL::VP)) << page_shift) * ES);
    };
    auto store = [&](char *to_lds, int key0) {
        if (key0 + KEYS > len) {
            // slots past the end hold anything: zeros; infinite and NaN values of
            // drafted tokens: zeros here, and noted
            const int left = total - (key0 + v_piece * (16 / ES));
            bool found = false;
#pragma unroll
            for (int i = 0; i < TL::VN; ++i) {
                v4u &r = stage[TL::KN + i];
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
            if (found) odd = 1;
        }
#pragma unroll
        for (int i = 0; i < TL::KN; ++i)
            *reinterpret_cast<v4u *>(to_lds + TL::k_pos(k_row + i * (64 / TL::KP), k_piece)) = stage[i];
#pragma unroll
        for (int i = 0; i < TL::VN; ++i)
            *reinterpret_cast<v4u *>(to_lds + TL::v_pos(v_row + i * (64 / TL::VP), v_piece)) = stage[TL::KN + i];
    };
    // where this lane reads: 8 values of a key (or feature) from an even or odd half piece
    const int krow = RW == 16 ? 8 * (n >> 2) + (n & 3) : 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);
    auto k_frag = [&](const char *at, int t, int kk) {
        const int key = RW == 16 ? krow + 32 * (t >> 1) + 4 * (t & 1) : krow + 32 * t;
        const int half = NG * kk + g;  // in units of 8 values
        return *reinterpret_cast<const raw_t *>(at + TL::k_pos(key, F8 ? half >> 1 : half) + (F8 ? 8 * (half & 1) : 0));
    };
    auto v_frag = [&](const char *at, int d, int s) {
        const int half = NG * s + g;
        return *reinterpret_cast<const raw_t *>(at + TL::v_pos(RW * d + n, F8 ? half >> 1 : half) + (F8 ? 8 * (half & 1) : 0));
    };

    acc_t o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = acc_t{};
    float m = M_START, l = 0.f;

    load(from);
    if (threadIdx.x == 0) odd = 0;
    __syncthreads();
    store(tile, from);
    load(from + KEYS);  // (past the end: the last run again)
    int odd_tile = 0;
    for (int key0 = from; key0 < to; key0 += KEYS) {
        __syncthreads();
        const char *at = tile + odd_tile * TL::BYTES;
        acc_t sc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            sc[t] = acc_t{};
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) sc[t] = MM::mul(FR::template op<op_t>(k_frag(at, t, kk)), qf[kk], sc[t]);
        }
        // p[r]: key key0 + 8 NG (r / 8) + 8 g + r % 8 of this lane's row
        float p[NT * NR];
#pragma unroll
        for (int r = 0; r < NT * NR; ++r) p[r] = sc[r / NR][r % NR] * a.score_scale;
        const bool ragged = key0 + KEYS > len;
        if (ragged) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const uint32_t on = seen8(sees, key0 + 8 * NG * s + 8 * g - len);
#pragma unroll
                for (int r = 0; r < 8; ++r) p[8 * s + r] = on >> r & 1u ? p[8 * s + r] : -__builtin_inff();
            }
        }
        float top = p[0];
#pragma unroll
        for (int r = 1; r < NT * NR; ++r) top = fmaxf(top, p[r]);
        if (__any(top > m + M_SLACK)) {
#pragma unroll
            for (int x = RW; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
            const float up = fmaxf(m, top);
            const float f = __builtin_amdgcn_exp2f(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] *= f;
        }
        op_t pf[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            v4u w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p0 = __builtin_amdgcn_exp2f(p[8 * s + 2 * j] - m);
                const float p1 = __builtin_amdgcn_exp2f(p[8 * s + 2 * j + 1] - m);
                l += p0 + p1;
                w[j] = pack2<E>(p0, p1);
            }
            pf[s] = __builtin_bit_cast(op_t, w);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] = MM::mul(FR::template op<op_t>(v_frag(at, d, s)), pf[s], o[d]);
        if (ragged && odd) {
            const ValueRows va = {a.cache, a.batch, b, h, len, total};
#pragma nounroll
            for (int s = 0; s < NS; ++s) add_odd<E, F8, D, RW>(va, key0 + 8 * NG * s, lane, sees, o);
        }
        odd_tile ^= 1;
        if (key0 + KEYS < to) {
            store(tile + odd_tile * TL::BYTES, key0 + KEYS);
            load(key0 + 2 * KEYS);
        }
    }

#pragma unroll
    for (int x = RW; x < 64; x <<= 1) l += __shfl_xor(l, x);
    if (!used) return;
    const bool whole = a.parts == 1;
    const float norm = whole ? (l == 0.f ? 0.f : a.v_scale / l) : 1.f;
    const int64_t part_row = (((int64_t)b * heads + h) * a.parts + c) * ((int64_t)a.max_tokens * G) + row;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < NR; r += 4) {
            const int dim = RW * d + 2 * r + 4 * g;
            const v4f acc = v4f{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]} * norm;
            if (!whole)
                *reinterpret_cast<v4f *>(a.ws_o + part_row * D + dim) = acc;
            else if (a.out_f32)
                *reinterpret_cast<v4f *>(reinterpret_cast<float *>(a.out) + q_row * D + dim) = acc;
            else
                *reinterpret_cast<v2u *>(a.out + (q_row * D + dim) * 2) = v2u{pack2<E>(acc[0], acc[1]), pack2<E>(acc[2], acc[3])};
        }
    if (!whole && g == 0) {
        a.ws_ml[2 * part_row] = m;
        a.ws_ml[2 * part_row + 1] = l;
    }
}

// out = sum over the parts, each weighted by exp2(its maximum - the largest).
// One workgroup to a (token, head): the waves cut the parts, lanes the dim.
template <class E, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a) {
    constexpr int VPL = D / 64;
    __shared__ float so[4][D];
    __shared__ float sm[4], sl[4];
    const int heads = a.cache.heads, G = a.group;
    const int tok = blockIdx.x, head = blockIdx.y;
    const int b = batch_seq(a.batch, tok);
    int first, T;
    batch_rows(a.batch, b, first, T);
    T = min(T, a.max_tokens);
    const int i = tok - first;
    if (i < 0 || i >= T) return;
    const int total = min(max(a.batch.lens[b], 0), INT32_MAX - 64) + T;
    const int parts = min((int)(((int64_t)total + a.part - 1) / a.part), a.parts);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t stride = (int64_t)a.max_tokens * G;
    const int64_t row0 = (((int64_t)b * heads + head / G) * a.parts) * stride + (int64_t)i * G + head % G;
    float m = M_START, l = 0.f, o[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) o[v] = 0.f;
    for (int c = wave; c < parts; c += 4) {
        const int64_t r = row0 + c * stride;
        const float pm = a.ws_ml[2 * r], pl = a.ws_ml[2 * r + 1];
        float po[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) po[v] = a.ws_o[r * D + lane * VPL + v];
        const float up = fmaxf(m, pm);
        const float f = __builtin_amdgcn_exp2f(m - up), pf = __builtin_amdgcn_exp2f(pm - up);
        m = up;
        l = l * f + pl * pf;
#pragma unroll
        for (int v = 0; v < VPL; ++v) o[v] = o[v] * f + po[v] * pf;
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) so[wave][lane * VPL + v] = o[v];
    if (lane == 0) {
        sm[wave] = m;
        sl[wave] = l;
    }
    __syncthreads();
    if (wave) return;
    float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float sum = 0.f, acc[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) acc[v] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(sm[w] - mm);
        sum += f * sl[w];
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] += f * so[w][lane * VPL + v];
    }
    const float norm = sum == 0.f ? 0.f : a.v_scale / sum;
    const int64_t at = ((int64_t)tok * ((int64_t)heads * G) + head) * D + lane * VPL;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        if (a.out_f32)
            reinterpret_cast<float *>(a.out)[at + v] = acc[v] * norm;
        else
            reinterpret_cast<E *>(a.out)[at + v] = (E)(acc[v] * norm);
    }
}

template <class E, bool F8, int D>
hipError_t launch_dim(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    const int64_t items = (int64_t)a.batch.n_seqs * a.cache.heads * a.parts;
    if (p.rows_wg == 16)
        hipLaunchKernelGGL((attn_few_kernel<E, F8, D>), dim3((unsigned)items), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((attn_tile_kernel<E, F8, D>), dim3((unsigned)((items + 7) / 8 * 8 * a.row_blocks)), dim3(256),
                           0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    hipLaunchKernelGGL((attn_join_kernel<E, D>), dim3((unsigned)a.batch.n_tokens, (unsigned)(a.cache.heads * a.group)),
                       dim3(256), 0, stream, a);
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
