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
// registers, no LDS.
//
// One pass over the keys with the running maximum m and sum l of a softmax in
// fp32.  m is raised only when a score passes it by more than 8 (in log2
// units): until then exp2(S - m) stays within 2^8, far inside every type, and
// neither a cross-lane maximum nor a rescaling of O is needed.
//
// A wave takes 32 keys at a time for RW query rows: 16 where a sequence brings
// no more, or where dim is 256 (a wave of 32 would need 320 registers for its
// sums and operands alone), else 32.  The waves of a workgroup share the
// rows (WR of them side by side) and cut the keys; their sums are joined in
// LDS.  A sequence's slots are cut into parts so that few long sequences fill
// the chip; a second kernel joins the parts.
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
    // the values that are infinite or NaN, zeros in place of the others
    static __device__ __forceinline__ raw odd(raw r) {
        constexpr uint32_t e = std::is_same_v<E, __bf16> ? 0x7F80u : 0x7C00u;
        raw x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool lo = (r[j] & e) == e, hi = (r[j] & (e << 16)) == e << 16;
            x[j] = r[j] & ((lo ? 0xFFFFu : 0u) | (hi ? 0xFFFF0000u : 0u));
        }
        return x;
    }
    static __device__ __forceinline__ bool any(raw r) { return (r[0] | r[1] | r[2] | r[3]) != 0; }
    // value e alone (none for e < 0)
    static __device__ __forceinline__ raw only(raw r, int e) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] &= e >> 1 == j ? (e & 1 ? 0xFFFF0000u : 0xFFFFu) : 0u;
        return r;
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
    static __device__ __forceinline__ raw odd(raw r) {
        raw x;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            // bit 7 of a byte of n: its low 7 bits are all ones (the one NaN of either sign)
            const uint32_t n = ((r[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            x[j] = r[j] & ((n >> 7) * 0xFFu);
        }
        return x;
    }
    static __device__ __forceinline__ bool any(raw r) { return (r[0] | r[1]) != 0; }
    static __device__ __forceinline__ raw only(raw r, int e) {
#pragma unroll
        for (int j = 0; j < 2; ++j) r[j] &= e >> 2 == j ? 0xFFu << (8 * (e & 3)) : 0u;
        return r;
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

template <int D, int RW, int WR>
constexpr int attn_lds_floats() {
    constexpr int o = 4 * RW * (D + 4) + 8 * RW;
    return o;
}

// Workgroup: 4 waves, WR side by side over the rows, 4 / WR over the keys.
template <class E, bool F8, int D, int RW, int WR>
__global__ __launch_bounds__(256) void attn_kernel(const AttnArgs a) {
    typedef Mfma<E, RW> MM;
    typedef typename MM::op op_t;
    typedef typename MM::acc acc_t;
    typedef Frag<E, F8> FR;
    typedef typename FR::raw raw_t;
    constexpr int NG = 64 / RW;         // lane groups
    constexpr int KT = RW == 16 ? 2 : 1;  // results of the first product over 32 keys
    constexpr int KS = RW == 16 ? 1 : 2;  // steps of the second product over 32 keys
    constexpr int NK = D / (8 * NG);    // steps of the first product
    constexpr int ND = D / RW;          // results of the second product
    constexpr int NR = RW * RW / 64;    // result registers
    constexpr int WK = 4 / WR;
    constexpr int ES = FR::BYTES;

    extern __shared__ float lds[];

    // part c of key head h of sequence b, row block rb: the row blocks of one
    // part run on one XCD (workgroups are dealt round robin to the 8), which
    // then reads the part once
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
    const int wr = wave / WK, wk = wave % WK;
    const int row = rb * a.rows_wg + wr * RW + n;
    const bool used = row < R;
    const int tok = used ? row / G : 0;
    const int head = h * G + (used ? row % G : 0);
    const int64_t q_row = (int64_t)(first + tok) * ((int64_t)a.cache.heads * G) + head;

    op_t qf[NK];
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) {
        v4u w = {0u, 0u, 0u, 0u};
        if (used) w = *reinterpret_cast<const v4u *>(a.q + (q_row * D + 8 * (kk * NG + g)) * 2);
        qf[kk] = __builtin_bit_cast(op_t, w);
    }
    uint64_t sees = 0;
    if (used) sees = a.mask ? a.mask[first + tok] : (2ull << tok) - 1ull;

    // Key of row m of the first product's result t: see the head of the file.
    int krow[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        const int j = n >> 2, i = n & 3;
        if constexpr (RW == 16)
            krow[t] = 8 * j + 4 * t + i;
        else
            krow[t] = 16 * (j >> 2) + 8 * (j & 1) + 4 * ((j >> 1) & 1) + i;
    }
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
    auto load_k = [&](const Runs &ru, raw_t(&kf)[KT][NK]) {
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const int i = krow[t] >> 4;
            const int64_t at = i ? ru.page[1] + ru.slot[1] * (D * ES) : ru.page[0] + ru.slot[0] * (D * ES);
            const char *p = a.cache.k + at + ((krow[t] & 15) * (D * ES) + 8 * g * ES);
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) kf[t][kk] = *reinterpret_cast<const raw_t *>(p + kk * NG * 8 * ES);
        }
    };
    auto load_v = [&](const Runs &ru, raw_t(&vf)[ND][KS]) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int i = RW == 32 ? s : g >> 1;
            const int64_t at = i ? ru.page[1] + ru.slot[1] * ES : ru.page[0] + ru.slot[0] * ES;
            const char *p = a.cache.v + at + ((n << page_shift) + 8 * (g & 1)) * ES;
            const int step = (RW * ES) << page_shift;
#pragma unroll
            for (int d = 0; d < ND; ++d) vf[d][s] = *reinterpret_cast<const raw_t *>(p + d * step);
        }
    };

    acc_t o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] = acc_t{};
    float m = M_START, l = 0.f;

    int key0 = from + 32 * wk;
    Runs ru = runs(key0);
    raw_t kf[KT][NK];
    if (key0 < to) load_k(ru, kf);
    for (; key0 < to; key0 += 32 * WK) {
        raw_t vf[ND][KS];
        load_v(ru, vf);
        const int next = key0 + 32 * WK;
        ru = runs(next);

        acc_t sc[KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            sc[t] = acc_t{};
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) sc[t] = MM::mul(FR::template op<op_t>(kf[t][kk]), qf[kk], sc[t]);
        }
        if (next < to) load_k(ru, kf);

        // p[8 s + e]: key key0 + 16 s + 8 g + e of this lane's row
        float p[8 * KS];
#pragma unroll
        for (int r = 0; r < 8 * KS; ++r) p[r] = sc[r / NR][r % NR] * a.score_scale;
        const bool ragged = key0 + 32 > len;
        if (ragged) {
#pragma unroll
            for (int r = 0; r < 8 * KS; ++r) {
                const int key = key0 + 16 * (r >> 3) + 8 * g + (r & 7);
                const bool on = key < len || (key < total && ((sees >> (key - len)) & 1ull));
                p[r] = on ? p[r] : -__builtin_inff();
            }
        }
        float top = p[0];
#pragma unroll
        for (int r = 1; r < 8 * KS; ++r) top = fmaxf(top, p[r]);
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
#pragma unroll
        for (int r = 0; r < 8 * KS; ++r) {
            p[r] = __builtin_amdgcn_exp2f(p[r] - m);
            l += p[r];
        }
        op_t pf[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            v4u w;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack2<E>(p[8 * s + 2 * j], p[8 * s + 2 * j + 1]);
            pf[s] = __builtin_bit_cast(op_t, w);
        }
        if (ragged) {
            // Slots past the end hold anything: zeros. An infinity or NaN of a
            // slot that some rows do not see would spoil those rows too (0 *
            // inf), so such values leave the product below and are added here,
            // one key at a time, to the rows (columns, so lanes) that see it.
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    FR::first(vf[d][s], min(max(total - (key0 + 16 * s + 8 * g), 0), 8));
                    const raw_t odd = FR::odd(vf[d][s]);
                    if (__any(FR::any(odd))) {
#pragma nounroll
                        for (int kx = 0; kx < 8 * NG; ++kx) {
                            const int key = key0 + 16 * s + kx;
                            const bool on = key < len || (key < total && ((sees >> ((key - len) & 63)) & 1ull));
                            const int e = kx >> 3 == g ? kx & 7 : -1;
                            const op_t pk = __builtin_bit_cast(
                                op_t, Frag<E, false>::only(__builtin_bit_cast(v4u, pf[s]), e));
                            const acc_t sum = MM::mul(FR::template op<op_t>(FR::only(odd, e)), pk, o[d]);
#pragma unroll
                            for (int r = 0; r < NR; ++r) o[d][r] = on ? sum[r] : o[d][r];
                        }
                        vf[d][s] ^= odd;
                    }
                }
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int d = 0; d < ND; ++d) o[d] = MM::mul(FR::template op<op_t>(vf[d][s]), pf[s], o[d]);
    }

    // Join the waves: o to LDS as [wave][row][dim], weights beside it.
#pragma unroll
    for (int x = RW; x < 64; x <<= 1) l += __shfl_xor(l, x);
    float *lo = lds, *lm = lds + 4 * RW * (D + 4), *ll = lm + 4 * RW;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < NR; r += 4) {
            const int dim = d * RW + 8 * (r >> 2) + 4 * g;
            *reinterpret_cast<v4f *>(lo + (wave * RW + n) * (D + 4) + dim) =
                v4f{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]};
        }
    if (g == 0) {
        lm[wave * RW + n] = m;
        ll[wave * RW + n] = l;
    }
    __syncthreads();
    constexpr int TPR = 256 / (RW * WR);  // threads to a row
    constexpr int VPT = D / TPR;          // values to a thread: 4 at a time, TPR * 4 apart
    const int jr = threadIdx.x / TPR, jt = threadIdx.x % TPR;
    const int out_row = rb * a.rows_wg + jr;
    if (out_row >= R) return;
    const int jn = (jr / RW) * WK * RW + jr % RW;  // [wave][row] index of the row's first key wave
    float mm = M_START;
#pragma unroll
    for (int k = 0; k < WK; ++k) mm = fmaxf(mm, lm[jn + k * RW]);
    float f[WK], sum = 0.f;
#pragma unroll
    for (int k = 0; k < WK; ++k) {
        f[k] = __builtin_amdgcn_exp2f(lm[jn + k * RW] - mm);
        sum += f[k] * ll[jn + k * RW];
    }
    const int64_t part_row = (((int64_t)b * heads + h) * a.parts + c) * ((int64_t)a.max_tokens * G) + out_row;
    const bool whole = a.parts == 1;
    const float norm = whole ? (sum == 0.f ? 0.f : a.v_scale / sum) : 1.f;
    const int64_t o_row = ((int64_t)(first + out_row / G) * ((int64_t)heads * G) + h * G + out_row % G) * D;
#pragma unroll
    for (int v = 0; v < VPT; v += 4) {
        const int dim = v * TPR + jt * 4;
        v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < WK; ++k) acc += f[k] * *reinterpret_cast<const v4f *>(lo + (jn + k * RW) * (D + 4) + dim);
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

template <class E, bool F8, int D, int RW, int WR>
hipError_t launch(const AttnArgs &a, int64_t items, hipStream_t stream) {
    const size_t lds = attn_lds_floats<D, RW, WR>() * sizeof(float);
    auto *kernel = attn_kernel<E, F8, D, RW, WR>;
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    const unsigned grid = (unsigned)((items + 7) / 8 * 8 * a.row_blocks);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), lds, stream, a);
    return hipGetLastError();
}

template <class E, bool F8, int D>
hipError_t launch_dim(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    const int64_t items = (int64_t)a.batch.n_seqs * a.cache.heads * a.parts;
    hipError_t e;
    if (p.rows_wave == 16 && p.rows_wg == 16)
        e = launch<E, F8, D, 16, 1>(a, items, stream);
    else if constexpr (D == 256)
        e = p.rows_wg == 32 ? launch<E, F8, D, 16, 2>(a, items, stream) : launch<E, F8, D, 16, 4>(a, items, stream);
    else
        e = p.rows_wg == 32   ? launch<E, F8, D, 32, 1>(a, items, stream)
            : p.rows_wg == 64 ? launch<E, F8, D, 32, 2>(a, items, stream)
                              : launch<E, F8, D, 32, 4>(a, items, stream);
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
