// kq_rope.hip -- from the fp32 product of a layer to its queries and a paged
// cache of keys and values, in one pass (gfx950): norm of each query and key
// head, rotation by position, rounding, and the stores to the rows' slots.
//
//   y = x * w / sqrt(mean x^2 + eps),   (a, b) -> (a c - b s, b c + a s)
//
// Eight features of a head to a lane (4i .. 4i + 3 and dim/2 + 4i ..): the two
// halves of a full rotation meet in one lane, the mean is a reduction over
// dim/8 lanes.  Queries and keys leave with 8-byte stores.  Values lie
// transposed in their page, so a workgroup stages a tile of rows in LDS and
// stores, feature by feature, 8 consecutive slots at once where 8 rows of the
// tile are an aligned run of one page; rows outside such runs (the ends of a
// sequence, single tokens) go value by value.  x is read once, past the caches.
//
// Bound: HBM bandwidth (4 bytes read, 2 or 1 written per value): 12k rows of 32 + 16
// heads of 128 in 91 us, 5.4 TB/s.  A call of few rows is bound by its launch and
// two dependent loads (row -> sequence -> page): one row 3.2 us, 1k rows of 40 + 16
// heads into 8 bits 11.7 us for 42 MB.
#include "kq_step_device.hpp"

namespace kq {

namespace {

// E: the type of q; C: how the cache holds its values (0: as q, 1: e4m3).
template <class E, bool F8, int D>
struct Rope {
    static constexpr int LPH = D / 8;     // lanes to a head
    static constexpr int HPW = 64 / LPH;  // heads to a wave
    static constexpr int ES = F8 ? 1 : 2;

    static __device__ __forceinline__ v4f at(const float *p) { return *reinterpret_cast<const v4f *>(p); }

    // 4 consecutive features of a head -> 4 stored values
    static __device__ __forceinline__ void store4(char *p, v4f y) {
        if constexpr (F8)
            *reinterpret_cast<uint32_t *>(p) = pack4_f8(y[0], y[1], y[2], y[3]);
        else
            *reinterpret_cast<v2u *>(p) = v2u{pack2<E>(y[0], y[1]), pack2<E>(y[2], y[3])};
    }

    // Features f .. f + 3 of a head whose scaled values are y; xp / w: the head
    // and its norm weights in memory, rs: the factor of its norm.
    static __device__ __forceinline__ v4f rotate(const RopeArgs &a, v4f y, int f, const float *xp, const float *w,
                                                 float rs, const float *cs) {
        const int rot = a.rot, half = rot >> 1;
        if (f >= rot) return y;
        if (a.pairs) {
            const int j = f >> 1;
            const float c0 = cs[j], c1 = cs[j + 1], s0 = cs[half + j], s1 = cs[half + j + 1];
            return v4f{fmaf(y[0], c0, -y[1] * s0), fmaf(y[1], c0, y[0] * s0), fmaf(y[2], c1, -y[3] * s1),
                       fmaf(y[3], c1, y[2] * s1)};
        }
        const bool low = f < half;
        const int j = low ? f : f - half;
        const v4f c = at(cs + j), s = at(cs + half + j);
        v4f z = at(xp + (low ? f + half : f - half));  // the other of each pair, still in the L1
        z *= rs;
        if (w) z *= at(w + (low ? f + half : f - half));
        v4f r;
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = fmaf(y[e], c[e], (low ? -z[e] : z[e]) * s[e]);
        return r;
    }

    // One wave: GROUPS times HPW consecutive query / key heads of one row, from
    // `head0`.  The row's place and its cosines are found once.
    template <int GROUPS>
    static __device__ __forceinline__ void heads(const RopeArgs &a, int row, int head0) {
        const int lane = threadIdx.x & 63;
        const int i = lane % LPH, hd0 = head0 + lane / LPH;
        const int kv = a.cache.heads, n_heads = a.q_heads + kv;
        const float *xr = a.x + (int64_t)row * a.ldx;
        v4f lo[GROUPS], hi[GROUPS];
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) {
            const int hd = min(hd0 + j * HPW, n_heads - 1);
            lo[j] = __builtin_nontemporal_load(reinterpret_cast<const v4f *>(xr + hd * D + 4 * i));
            hi[j] = __builtin_nontemporal_load(reinterpret_cast<const v4f *>(xr + hd * D + D / 2 + 4 * i));
        }
        // the slot is needed by keys and by positions that follow it
        int slot = 0, page = 0;
        if (head0 + GROUPS * HPW > a.q_heads || !a.positions) {
            const int b = batch_seq(a.batch, row);
            int first, count;
            batch_rows(a.batch, b, first, count);
            slot = batch_len(a.batch, b) + (row - first);
            page = slot_page(a.cache, a.batch, b, slot);
        }
        const float *cs = a.rope;
        v4f c = {0.f, 0.f, 0.f, 0.f}, s = c;
        const bool whole = a.rot == D && !a.pairs;  // the halves that lo and hi are
        if (a.rot) {
            cs += (int64_t)min(max(a.positions ? a.positions[row] : slot, 0), a.n_pos - 1) * a.rot;
            if (whole) {
                c = at(cs + 4 * i);
                s = at(cs + D / 2 + 4 * i);
            }
        }
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) {
            const int hd = hd0 + j * HPW;
            const bool is_q = hd < a.q_heads;
            const float *w = is_q ? a.q_norm : a.k_norm;
            float rs = 1.f;
            if (a.q_norm || a.k_norm) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) ss = fmaf(lo[j][e], lo[j][e], fmaf(hi[j][e], hi[j][e], ss));
#pragma unroll
                for (int x = 1; x < LPH; x <<= 1) ss += __shfl_xor(ss, x);
                if (w) rs = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
            }
            v4f ylo = lo[j] * rs, yhi = hi[j] * rs;
            if (w) {
                ylo *= at(w + 4 * i);
                yhi *= at(w + D / 2 + 4 * i);
            }
            if (whole) {
                v4f z;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[e] = fmaf(ylo[e], c[e], -yhi[e] * s[e]);
                    yhi[e] = fmaf(yhi[e], c[e], ylo[e] * s[e]);
                }
                ylo = z;
            } else if (a.rot) {
                const float *xp = xr + min(hd, n_heads - 1) * D;
                ylo = rotate(a, ylo, 4 * i, xp, w, rs, cs);
                yhi = rotate(a, yhi, D / 2 + 4 * i, xp, w, rs, cs);
            }
            if (is_q) {
                char *p = a.q + (((int64_t)row * a.q_heads + hd) * D + 4 * i) * 2;
                *reinterpret_cast<v2u *>(p) = v2u{pack2<E>(ylo[0], ylo[1]), pack2<E>(ylo[2], ylo[3])};
                *reinterpret_cast<v2u *>(p + D) = v2u{pack2<E>(yhi[0], yhi[1]), pack2<E>(yhi[2], yhi[3])};
            } else if (hd < n_heads) {
                const int shift = a.cache.page_shift;
                char *p = a.cache.k + 4 * i * ES +
                          ((((int64_t)page * kv + (hd - a.q_heads)) << shift) + (slot & ((1 << shift) - 1))) * (D * ES);
                store4(p, ylo * a.k_inv);
                store4(p + D / 2 * ES, yhi * a.k_inv);
            }
        }
    }

    // One workgroup: rows [row0, row0 + TT) of value head h.
    template <int TT>
    static __device__ __forceinline__ void values(const RopeArgs &a, int row0, int h) {
        constexpr int PITCH = D * ES + 4;  // 4 bytes past a row: feature-wise reads of 8 rows miss no bank twice
        __shared__ __align__(16) char tile[TT * PITCH];
        __shared__ int64_t where[TT];      // byte offset of the row's slot in v for feature 0
        __shared__ int runs[TT], ones[TT];  // rows that lead 8 of a page, rows that go alone
        __shared__ int n_runs, n_ones;
        const int rows = min(TT, a.batch.n_tokens - row0);
        const int shift = a.cache.page_shift, kv = a.cache.heads;
        const int lane = threadIdx.x & 63;
        if (threadIdx.x < 64) {
            // a lane to a row: its sequence (the first row's, and those that begin
            // up to it), its slot, its place
            const int b0 = batch_seq(a.batch, row0);
            const int next = b0 + 1 + lane;
            const int begins = next < a.batch.n_seqs ? a.batch.offsets[next] : INT32_MAX;
            int b = b0;
            for (int r = 0; r < rows; ++r) {
                const int more = __popcll(__ballot(begins <= row0 + r));
                if (lane == r) b = b0 + more;
            }
            if (__any(b == b0 + 64)) {  // (more than 64 sequences in the tile: some have no rows)
                for (int r = 0; r < rows; ++r) {
                    const int each = batch_seq(a.batch, row0 + r);
                    if (lane == r) b = each;
                }
            }
            const bool row = lane < rows;
            int64_t at = -1;
            int in = 1;
            if (row) {
                int first, count;
                batch_rows(a.batch, b, first, count);
                const int slot = batch_len(a.batch, b) + (row0 + lane - first);
                in = slot & ((1 << shift) - 1);
                at = ((((int64_t)slot_page(a.cache, a.batch, b, slot) * kv + h) * D << shift) + in) * ES;
                where[lane] = at;
            }
            // A row leads a run if its place is a multiple of 8 and it and the 7 after
            // it lie one after another; it then stores for all 8.
            const int64_t then = __shfl_down(at, 1);
            const uint64_t joined = __ballot(lane + 1 < rows && then == at + ES);
            const uint64_t leads = __ballot(row && (in & 7) == 0 && ((joined >> lane) & 127ull) == 127ull);
            uint64_t led = leads;
            led |= led << 1;
            led |= led << 2;
            led |= led << 4;
            const uint64_t alone = __ballot(row) & ~led;
            const uint64_t below = (1ull << lane) - 1ull;
            if (leads >> lane & 1ull) runs[__popcll(leads & below)] = lane;
            if (alone >> lane & 1ull) ones[__popcll(alone & below)] = lane;
            if (lane == 0) {
                n_runs = __popcll(leads);
                n_ones = __popcll(alone);
            }
        }
        constexpr int RPP = 256 / LPH;  // rows to a pass
        const int i = threadIdx.x % LPH;
        for (int r = threadIdx.x / LPH; r < rows; r += RPP) {
            const float *xp = a.x + (int64_t)(row0 + r) * a.ldx + (int64_t)(a.q_heads + kv + h) * D + 4 * i;
            const v4f lo = __builtin_nontemporal_load(reinterpret_cast<const v4f *>(xp)) * a.v_inv;
            const v4f hi = __builtin_nontemporal_load(reinterpret_cast<const v4f *>(xp + D / 2)) * a.v_inv;
            char *p = tile + r * PITCH + 4 * i * ES;
            if constexpr (F8) {
                *reinterpret_cast<uint32_t *>(p) = pack4_f8(lo[0], lo[1], lo[2], lo[3]);
                *reinterpret_cast<uint32_t *>(p + D / 2) = pack4_f8(hi[0], hi[1], hi[2], hi[3]);
            } else {
                uint32_t *q = reinterpret_cast<uint32_t *>(p), *u = reinterpret_cast<uint32_t *>(p + D);
                q[0] = pack2<E>(lo[0], lo[1]);
                q[1] = pack2<E>(lo[2], lo[3]);
                u[0] = pack2<E>(hi[0], hi[1]);
                u[1] = pack2<E>(hi[2], hi[3]);
            }
        }
        __syncthreads();
        char *v = a.cache.v;
        constexpr int RUNS = TT / 8;  // at most: the runs of a feature to neighbouring lanes, whose stores adjoin
        const int n = n_runs, alone = n_ones;
        if ((int)threadIdx.x % RUNS < n) {
            const int r = runs[threadIdx.x % RUNS];
            const char *s = tile + r * PITCH;
            char *p = v + where[r];
            for (int d = threadIdx.x / RUNS; d < D; d += 256 / RUNS) {
                char *to = p + ((int64_t)d << shift) * ES;
                if constexpr (F8) {
                    v2u w = {0u, 0u};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j >> 2] |= (uint32_t) * reinterpret_cast<const uint8_t *>(s + d + j * PITCH) << (8 * (j & 3));
                    *reinterpret_cast<v2u *>(to) = w;
                } else {
                    v4u w = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j >> 1] |= (uint32_t) * reinterpret_cast<const uint16_t *>(s + d * 2 + j * PITCH) << (16 * (j & 1));
                    *reinterpret_cast<v4u *>(to) = w;
                }
            }
        }
        for (int t = threadIdx.x; t < alone * D; t += 256) {
            const int r = ones[t / D], d = t % D;
            const char *s = tile + r * PITCH + d * ES;
            char *p = v + where[r] + ((int64_t)d << shift) * ES;
            if constexpr (F8)
                *p = *s;
            else
                *reinterpret_cast<uint16_t *>(p) = *reinterpret_cast<const uint16_t *>(s);
        }
    }
};

// Blocks [0, value_blocks): tiles of value rows; then 4 waves of heads each.
template <class E, bool F8, int D, int TT, int GROUPS>
__global__ __launch_bounds__(256) void rope_append_kernel(const RopeArgs a, int value_blocks) {
    typedef Rope<E, F8, D> RO;
    const int kv = a.cache.heads;
    if ((int)blockIdx.x < value_blocks) {
        RO::template values<TT>(a, (int)(blockIdx.x / kv) * TT, blockIdx.x % kv);
        return;
    }
    constexpr int HEADS = RO::HPW * GROUPS;
    const int waves = (a.q_heads + kv + HEADS - 1) / HEADS;  // to a row
    const int item = (blockIdx.x - value_blocks) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = item / waves;
    if (row < a.batch.n_tokens) RO::template heads<GROUPS>(a, row, (item - row * waves) * HEADS);
}

template <class E, bool F8, int D>
hipError_t launch(const RopeArgs &a, hipStream_t stream) {
    const RopePlan p = rope_plan(a.batch.n_tokens, a.q_heads, a.cache.heads, D);
    const dim3 grid((unsigned)p.blocks);
    if (p.tile == 16)
        hipLaunchKernelGGL((rope_append_kernel<E, F8, D, 16, 1>), grid, dim3(256), 0, stream, a, (int)p.value_blocks);
    else
        hipLaunchKernelGGL((rope_append_kernel<E, F8, D, 64, 2>), grid, dim3(256), 0, stream, a, (int)p.value_blocks);
    return hipGetLastError();
}

template <class E, bool F8>
hipError_t launch_dim(const RopeArgs &a, int dim, hipStream_t stream) {
    switch (dim) {
        case 64: return launch<E, F8, 64>(a, stream);
        case 128: return launch<E, F8, 128>(a, stream);
        default: return launch<E, F8, 256>(a, stream);
    }
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs &a, int type, int dim, int q_type, hipStream_t stream) {
    if (q_type == KQ_T_BF16)
        return type == KQ_T_F8 ? launch_dim<__bf16, true>(a, dim, stream) : launch_dim<__bf16, false>(a, dim, stream);
    return type == KQ_T_F8 ? launch_dim<_Float16, true>(a, dim, stream) : launch_dim<_Float16, false>(a, dim, stream);
}

}  // namespace kq
