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
#include "kq_attn_device.hpp"

namespace kq {

namespace {

// ---------------------------------------------------------------- sharing

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
