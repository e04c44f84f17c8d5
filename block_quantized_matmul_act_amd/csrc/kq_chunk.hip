// kq_chunk.hip -- attention of chunks of new tokens over a paged cache (gfx950):
// any number of rows of a sequence, each over the slots up to its own, and of
// those under a window only the last `window` and the first `sinks`.
//
// The arithmetic is that of kq_attn.hip (see there): scores and sums with the keys
// dealt so that nothing moves between lanes, one pass with the running maximum and
// sum of a softmax.  What differs is the shape of the work.  The rows of a sequence
// that share a key head (tokens * group) are cut into blocks of 16, 128 or 256, and a
// block reads the slots that one of its rows sees: a run from the window's start
// of its first token to the slot of its last, and before that the sinks.  Tiles that
// every row sees whole are not masked.
//
// Block numbers are offsets[b] * group / rows + b for the first block of sequence b
// and follow each other from there.  That leaves room for every block of b before the
// number of b + 1, grows with b, and needs no sum over the sequences: a
// workgroup finds its block by one search of the offsets.  A few numbers have no
// block, and their workgroups end at once.
//
// Many blocks: a workgroup to a block, those late in a text, which have the most keys,
// first.  Few (or long ones among them): a grid that just fills the chip adds up the
// units of all blocks and every workgroup takes an equal run of them.  A run covers
// parts of at most two blocks and any number of whole ones; a part leaves its sums in
// the workspace and a second kernel joins the parts, in a fixed order.
#include "kq_attn_device.hpp"
#include "kq_copy.hpp"
#include "kq_layer.hpp"

namespace kq {

namespace {

// A block's share of the work: units [from, to), first those of the sinks, then those of
// the window.
struct Block {
    int b, h, rb;
    Seq sq;
    int pos0, pos1;  // slots of its first and last token
    int shift;       // a unit is 1 << shift slots
    int sink_units, window_unit, units;
    int from, to;
    bool whole;
};

// The first block number of sequence b.
__device__ __forceinline__ int64_t first_block(const ChunkArgs &c, int b) {
    const int64_t row = (int64_t)min(max(c.a.batch.offsets[b], 0), c.a.batch.n_tokens) * c.a.group;
    return (row >> c.rows_shift) + b;
}
// The sequence that has block number j of a key head: the last one whose first
// number is not above it; found by a whole wave together.
__device__ __forceinline__ int block_seq(const ChunkArgs &c, int j) {
    const int lane = __lane_id();
    int lo = 0, n = c.a.batch.n_seqs;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const int at = lo + lane * step;
        const bool le = at < lo + n && first_block(c, at) <= j;
        const int k = __popcll(__ballot(le));
        const int from = lo + max(k - 1, 0) * step;
        n = min(step, lo + n - from);
        lo = from;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}
// The same for one lane by itself.
__device__ __forceinline__ int lane_seq(const ChunkArgs &c, int j) {
    int lo = 0, hi = c.a.batch.n_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_block(c, mid) <= j)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Block j as one of sequence b; false if there is none.
__device__ __forceinline__ bool block_of(const ChunkArgs &c, int b, int j, Block &k) {
    k.b = b;
    k.rb = j - (int)first_block(c, b);
    Seq &q = k.sq;
    batch_rows(c.a.batch, b, q.first, q.rows);
    q.T = q.rows;
    q.len = batch_len(c.a.batch, b);
    // slots past the sequence's row of the page table are not there
    const int64_t table = (int64_t)c.a.batch.max_pages << c.a.cache.page_shift;
    q.total = (int)min((int64_t)q.len + q.T, table);
    const int64_t row0 = (int64_t)k.rb << c.rows_shift, rows = (int64_t)q.T * c.a.group;
    k.units = 0;
    if (k.rb < 0 || row0 >= rows) return false;
    const int64_t row1 = min(row0 + (1 << c.rows_shift), rows);
    k.pos0 = q.len + (int)((uint32_t)row0 / (uint32_t)c.a.group);
    k.pos1 = q.len + (int)((uint32_t)(row1 - 1) / (uint32_t)c.a.group);
    const int end = min(k.pos1 + 1, q.total);
    const int begin = min(max(k.pos0 - (c.window - 1), 0), end);
    k.shift = rows <= 16 ? c.few_shift : CHUNK_UNIT_SHIFT;
    const int64_t up = (1 << k.shift) - 1;
    k.window_unit = begin >> k.shift;
    const int end_unit = (int)((end + up) >> k.shift);
    const int sinks = (int)((min(c.sinks, end) + up) >> k.shift);
    k.sink_units = min(sinks, k.window_unit);
    k.units = k.sink_units + max(end_unit - k.window_unit, 1);
    return true;
}

// The units of all blocks of a key head, c.begin more to each (what its begin and end
// take), added up by the whole workgroup: before[j] (in LDS) is what comes before block j,
// before[blocks] all.
template <int THREADS>
__device__ __forceinline__ void add_up(const ChunkArgs &c, int *before, int *waves) {
    int base = 0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j0 = 0; j0 < c.blocks; j0 += THREADS) {
        const int j = j0 + threadIdx.x;
        Block k;
        k.units = 0;
        if (j < c.blocks && block_of(c, lane_seq(c, j), j, k)) k.units += c.begin;
        int incl = k.units;
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x111, 0xF, 0xF, false);  // in rows of 16: from 1, 2, 4, 8 to the left
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x112, 0xF, 0xF, false);
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x114, 0xF, 0xF, false);
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x118, 0xF, 0xF, false);
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x142, 0xA, 0xF, false);  // lane 15 of rows 0 and 2 to rows 1 and 3
        incl += __builtin_amdgcn_update_dpp(0, incl, 0x143, 0xC, 0xF, false);  // lane 31 to the upper half
        if (lane == 63) waves[wave] = incl;
        __syncthreads();
        int all = 0, mine = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) {
            mine = w < wave ? mine + waves[w] : mine;
            all += waves[w];
        }
        if (j < c.blocks) before[j] = base + mine + incl - k.units;
        base += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) before[c.blocks] = base;
    __syncthreads();
}

// What a workgroup does, piece by piece.
template <int THREADS>
struct Work {
    const ChunkArgs &c;
    int *before;
    int u, end, begin, group, all;
    // lds: CHUNK_RUN_BLOCKS + 1 and a wave's number of ints
    __device__ __forceinline__ Work(const ChunkArgs &c_, int *lds, int *waves) : c(c_), before(lds) {
        u = begin = 0;
        end = 1;
        group = blockIdx.x;
        if (!c.runs) return;
        add_up<THREADS>(c, before, waves);
        all = before[c.blocks];
        const int units = all * c.a.cache.heads, groups = min((int)gridDim.x, units);
        // workgroups go round the chip's 8 dies: neighbouring runs, which mostly share a
        // head's keys, to the same one
        const int per = (int)gridDim.x >> 3;
        if (((int)gridDim.x & 7) == 0) group = (group & 7) * per + (group >> 3);
        if (blockIdx.x == 0)
            for (int j = threadIdx.x; j <= c.blocks; j += THREADS) c.a.ws_seq[j] = before[j];
        if (group >= groups) {
            end = 0;
            return;
        }
        const Runs runs(units, groups);
        u = begin = runs.begin(group);
        end = runs.begin(group + 1);
    }
    // The next piece and, where it is a part, its slot; false at the end.
    __device__ __forceinline__ bool next(Block &k, int64_t &slot) {
        const int heads = c.a.cache.heads;
        slot = 0;
        if (!c.runs) {
            if (u >= end) return false;
            u = end;
            const unsigned w = blockIdx.x, back = w / heads;
            const int j = c.blocks - 1 - (int)back;
            k.h = (int)(w - back * heads);
            if (!block_of(c, block_seq(c, j), j, k)) return false;
            k.from = 0;
            k.to = k.units;
            k.whole = true;
            return true;
        }
        while (u < end) {
            k.h = u / all;
            const int x = u - k.h * all;
            // the last block with before[j] <= x (those without units share their number with it)
            const int lane = __lane_id();
            int lo = 0, n = c.blocks;
            while (n > 1) {
                const int step = (n + 63) >> 6, at = lo + lane * step;
                const int few = __popcll(__ballot(at < lo + n && before[at] <= x));
                const int from = lo + max(few - 1, 0) * step;
                n = min(step, lo + n - from);
                lo = from;
            }
            const int j = __builtin_amdgcn_readfirstlane(lo);
            block_of(c, block_seq(c, j), j, k);
            // the run's share [x, x + some) of the block's c.begin + units, as they were added up (with
            // offsets that fall, the search can find another sequence than add_up did)
            const int in = x - __builtin_amdgcn_readfirstlane(before[j]);
            const int some = min(__builtin_amdgcn_readfirstlane(before[j + 1]) - x, end - u);
            slot = 2 * (int64_t)group + (u != begin);
            u += some;
            k.from = max(in - c.begin, 0);
            k.to = min(max(in + some - c.begin, 0), k.units);
            k.whole = k.to - k.from == k.units;
            if (k.to > k.from) return true;
        }
        return false;
    }
};

// The tiles of a part, counted from the block's first, and who sees what of them.
template <int KEYS>
struct Tiles {
    const ChunkArgs &c;
    int sink_tiles, start;  // tiles of the sinks; the slot of the first tile after them
    int from, to;
    // Tiles that some row between two slots does not see whole: [low0, low1), where sinks
    // or the window end, and from `high` on, where the rows' own slots are.
    struct Edges {
        int low0, low1, high;
        __device__ __forceinline__ bool low(int t) const { return t >= low0 && t < low1; }
        __device__ __forceinline__ bool at(int t) const { return low(t) || t >= high; }
    };
    Edges block;
    __device__ __forceinline__ Edges edges(int pos0, int pos1) const {
        Edges e;
        e.low0 = min(sink_tiles, c.sinks / KEYS);
        // (the slots not below start: their differences fit 32 bits)
        e.low1 = sink_tiles + max(pos1 - (c.window - 1) - start + KEYS - 1, 0) / KEYS;
        e.high = sink_tiles + max(pos0 + 1 - start, 0) / KEYS;
        return e;
    }
    __device__ __forceinline__ Tiles(const ChunkArgs &c_, const Block &k) : c(c_) {
        const int f = (1 << k.shift) / KEYS;
        sink_tiles = k.sink_units * f;
        start = k.window_unit << k.shift;
        from = k.from * f;
        to = k.to * f;
        while (to - 1 > from && key(to - 1) > k.pos1) --to;  // (tiles of the last unit that lie past the end)
        block = edges(k.pos0, k.pos1);
    }
    __device__ __forceinline__ int key(int t) const { return t < sink_tiles ? t * KEYS : start + (t - sink_tiles) * KEYS; }
    // which of the 8 keys from k the row of slot pos sees
    __device__ __forceinline__ uint32_t on(int k, int pos) const {
        const int back = max(pos - k, -1);  // (below 0 for all the same: the sums stay in 32 bits)
        const int upto = min(back + 1, 8), out = min(max(back - (c.window - 1), 0), 8);
        const int sink = min(max(c.sinks - k, 0), 8);
        return ((1u << upto) - 1u) & (~((1u << out) - 1u) | ((1u << sink) - 1u));
    }
};

// The thread's number, worked out anew for each piece: what follows from it is not kept
// in registers across the pieces (the ways of few and of many rows together have too many).
__device__ __forceinline__ unsigned this_thread() {
    unsigned t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// Two 16-bit values, whose sum is added to an fp32 one (exactly, but for one rounding; float16's
// smallest values count).
__device__ __forceinline__ float add2(uint32_t w, float sum, __bf16) {
    constexpr uint32_t one = 0x3F803F80u;
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, w), __builtin_bit_cast(v2bf, one), sum, false);
}
__device__ __forceinline__ float add2(uint32_t w, float sum, _Float16) {
    constexpr uint32_t one = 0x3C003C00u;
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(v2h, w), __builtin_bit_cast(v2h, one), sum, false);
}

// One wave's rows over the tiles.
template <class E, bool F8, int D, int KEYS, int RW, bool RUNS>
struct Rows {
    typedef Attend<E, F8, D, KEYS, RW, RUNS> AT;
    AT at;
    const Tiles<KEYS> &tiles;
    int pos;  // slot of this lane's row
    typename Tiles<KEYS>::Edges edge;
    __device__ __forceinline__ Rows(const AttnArgs &a, const Tiles<KEYS> &t, unsigned thread) : at(a, thread), tiles(t) {}
    __device__ __forceinline__ void begin(const Block &k, int row0) {
        const int G = at.a.group;
        pos = k.sq.len + at.template begin<false>(k.sq, k.h, row0);
        const int pos0 = __builtin_amdgcn_readfirstlane(min(k.sq.len + row0 / G, k.pos1));
        const int pos1 = __builtin_amdgcn_readfirstlane(min(k.sq.len + (row0 + RW - 1) / G, k.pos1));
        if (!at.used) pos = pos1;
        edge = tiles.edges(pos0, pos1);
    }
    // Masks the scores of tile t, the one at key0.  p[r] is key key0 + 8 NG (r / 8) + 8 g + r % 8.
    __device__ __forceinline__ void mask(int t, int key0, float (&p)[AT::NT * AT::NR]) {
        if (edge.at(t)) {
            int k0 = key0;
            asm volatile("" : "+s"(k0));  // (the masks are not worked out ahead of this branch)
            const int back = pos - (k0 + 8 * at.g);  // the last key that is not after the row
            if (t >= edge.high) {
#pragma unroll
                for (int r = 0; r < AT::NT * AT::NR; ++r) p[r] = 8 * AT::NG * (r / 8) + r % 8 <= back ? p[r] : -__builtin_inff();
            }
            if (edge.low(t)) {
                const int out = max(back, -1) - tiles.c.window, sink = tiles.c.sinks - (k0 + 8 * at.g);
#pragma unroll
                for (int r = 0; r < AT::NT * AT::NR; ++r) {
                    const float s = 8 * AT::NG * (r / 8) + r % 8 < sink ? p[r] : -__builtin_inff();
                    p[r] = 8 * AT::NG * (r / 8) + r % 8 > out ? p[r] : s;
                }
            }
        }
    }
    // The probabilities of a tile's scores, as operands of the second product; their sum is added
    // to the rows' weights.  It is taken after their rounding: the weights of a row then
    // add up to 1, and what rounding does to a large one is taken back by the division.
    // m is not compared with every score: a score too far above it shows in the sum,
    // which is as large as the largest, and then the tile is weighed again under a new m
    // (a maximum of 32 scores would be a tenth of the vector work of a tile at dim 64).
    __device__ __forceinline__ void weigh(float (&p)[AT::NT * AT::NR], typename AT::op_t (&pf)[AT::NS]) {
        constexpr float MOST = M_SLACK<E> > 0 ? (float)(1u << (int)(M_SLACK<E> > 0 ? M_SLACK<E> : 0))
                                              : 1.f / (float)(1u << (int)(M_SLACK<E> > 0 ? 0 : -M_SLACK<E>));
        bool scaled = at.far, raised = false;
        float sum[2];
        if (scaled) scale(p);
        while (true) {
            const float by = scaled ? 1.f : at.a.score_scale;
            sum[0] = sum[1] = 0.f;
#pragma unroll
            for (int s = 0; s < AT::NS; ++s) {
                v4u w;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p0 = __builtin_amdgcn_exp2f(fmaf(p[8 * s + 2 * j], by, -at.m));
                    const float p1 = __builtin_amdgcn_exp2f(fmaf(p[8 * s + 2 * j + 1], by, -at.m));
                    w[j] = pack2<E>(p0, p1);
                    sum[j & 1] = add2(w[j], sum[j & 1], E{});
                }
                pf[s] = __builtin_bit_cast(typename AT::op_t, w);
            }
            if (raised || !__any(sum[0] + sum[1] > MOST)) break;
            float top = p[0];
#pragma unroll
            for (int r = 1; r < AT::NT * AT::NR; ++r) top = fmaxf(top, p[r]);
            at.raise_to(top * by);
            raised = true;
            if (at.far && !scaled) {
                scale(p);
                scaled = true;
            }
        }
        at.l += sum[0] + sum[1];
    }
    __device__ __forceinline__ void scale(float (&p)[AT::NT * AT::NR]) {
#pragma unroll
        for (int r = 0; r < AT::NT * AT::NR; ++r) p[r] *= at.a.score_scale;
    }
    __device__ __forceinline__ void tile(const char *lds, int buf, int t, int key0) {
        float p[AT::NT * AT::NR];
        typename AT::op_t pf[AT::NS];
        at.template products<false, true, 4>(lds, 0, pf, buf, p);
        mask(t, key0, p);
        weigh(p, pf);
        at.template products<true, false, 4>(lds, buf + AT::TL::K_BYTES, pf, 0, p);
    }
    // The wave's rows to the output or, a part, to the workspace as they lie in the lanes.
    __device__ __forceinline__ void put(const Block &k, int64_t slot, int wave) {
        if (k.whole) {
            at.put(true, 0);
            return;
        }
        at.end();
        const int64_t wave_rows = (slot << tiles.c.rows_shift) + wave * RW;
        v4f *o = reinterpret_cast<v4f *>(at.a.ws_o + wave_rows * D) + at.lane;
#pragma unroll
        for (int d = 0; d < AT::ND; ++d)
#pragma unroll
            for (int r = 0; r < AT::NR; r += 4)
                o[(d * AT::NR + r) * 16] = v4f{at.o[d][r], at.o[d][r + 1], at.o[d][r + 2], at.o[d][r + 3]};
        if (at.g == 0) *reinterpret_cast<v2f *>(at.a.ws_ml + 2 * (wave_rows + at.n)) = v2f{at.m, at.l};
    }
    // What infinite and NaN values in tiles that some row does not see whole add.
    __device__ __forceinline__ void odd_values(const Block &k, int from, int step) {
#pragma nounroll
        for (int t = from; t < tiles.to; t += step) {
            if (!tiles.block.at(t)) continue;
            const int key0 = tiles.key(t);
#pragma nounroll
            for (int key = key0; key < key0 + KEYS; key += 8 * AT::NG)
                add_odd<E, F8, D, RW>(ValueRows{at.a.cache, at.a.batch, k.b, k.h, k.sq.total}, key, at.lane,
                                      [&](int k8) { return tiles.on(k8, pos); }, at.o);
        }
    }
};

// Up to 16 rows: the waves take tiles in turn, each its own in LDS without a barrier,
// and their sums are joined in LDS.  What bounds them is memory, and what keeps it busy the waves
// on a compute unit: tiles of 32 keys leave room for 3 workgroups (8 bits, dim 128; 96 sequences
// under a window of 2048, 64 query and 8 key heads: 79 us, 5.1 TB/s; tiles of 64 keys 87).
template <class E, bool F8, int D>
struct Few {
    static constexpr int RW = 16, KEYS = 32;
    typedef Tile<E, F8, D, KEYS, RW, 64, true> TL;
    typedef Rows<E, F8, D, KEYS, RW, false> RS;
    static constexpr int O_FLOATS = RW * (D + 4);
    static constexpr int WAVE_BYTES = TL::BYTES > O_FLOATS * 4 ? TL::BYTES : (O_FLOATS * 4 + 1023) / 1024 * 1024;
};
// The waves that take few rows in the kernel of many: 8, or none (dim 256 in 16 bits) where
// neither LDS nor registers hold them.
template <class E, bool F8, int D>
constexpr int FEW_IN_WIDE = 8 * Few<E, F8, D>::WAVE_BYTES <= 147456 ? 8 : 0;
// lds: WAVES * WAVE_BYTES, a wave's tile and then its sums [row][dim]; lm, ll: WAVES * 16
template <class E, bool F8, int D, int WAVES>
__device__ __forceinline__ void few_rows(const ChunkArgs &c, const Block &k, int64_t slot, char *lds, float *lm, float *ll) {
    typedef Few<E, F8, D> FW;
    typedef typename FW::TL TL;
    typedef typename FW::RS RS;
    constexpr int RW = FW::RW, KEYS = FW::KEYS, WAVE_BYTES = FW::WAVE_BYTES;
    const AttnArgs &a = c.a;
    const Tiles<KEYS> tiles(c, k);
    const unsigned thread = this_thread();
    const int wave = __builtin_amdgcn_readfirstlane(thread >> 6);
    const int mine = wave * WAVE_BYTES;
    TL tl(a, thread & 63);
    RS rs(a, tiles, thread);
    typename RS::AT &at = rs.at;
    tl.aim(k.b, k.h, k.sq);
    int t = tiles.from + wave;
    typename TL::Place next = tl.find(tiles.key(t));
    tl.load_k(next);
    tl.load_v(next);
    next = tl.find(tiles.key(t + WAVES));
    const int row0 = k.rb << c.rows_shift;
    rs.begin(k, row0);
    bool odd = false;
    for (; t < tiles.to; t += WAVES) {
        const int key0 = tiles.key(t);
        tl.store_k(lds, mine);
        odd |= tl.template store_v<false>(lds, mine + TL::K_BYTES, key0, tiles.block.at(t));
        if (t + WAVES < tiles.to) {
            tl.load_k(next);
            tl.load_v(next);
            next = tl.find(tiles.key(t + 2 * WAVES));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        rs.tile(lds, mine, t, key0);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    if (__any(odd)) rs.odd_values(k, tiles.from + wave, WAVES);
    at.end();

    // Join the waves.
    float *lo = reinterpret_cast<float *>(lds + mine);
#pragma unroll
    for (int d = 0; d < RS::AT::ND; ++d) *reinterpret_cast<v4f *>(lo + at.n * (D + 4) + d * RW + 4 * at.g) = at.o[d];
    if (at.g == 0) {
        lm[wave * RW + at.n] = at.m;
        ll[wave * RW + at.n] = at.l;
    }
    __syncthreads();
    const int row = thread >> 4, jt = thread & 15;  // 16 threads to a row
    if (row >= RW || row0 + row >= k.sq.T * a.group) return;  // (no barrier follows here)
    const bool all = k.whole;
    const int64_t slot_row = slot << c.rows_shift;
    float mm = M_START;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) mm = fmaxf(mm, lm[row + w * RW]);
    float f[WAVES], sum = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        f[w] = __builtin_amdgcn_exp2f(lm[row + w * RW] - mm);
        sum += f[w] * ll[row + w * RW];
    }
    const float norm = all ? (sum == 0.f ? 0.f : a.v_scale / sum) : 1.f;
    const int tok = (row0 + row) / a.group;
    const int64_t o_row =
        (int64_t)(k.sq.first + tok) * ((int64_t)a.cache.heads * a.group) + k.h * a.group + (row0 + row - tok * a.group);
#pragma unroll
    for (int v = 0; v < D; v += 64) {
        const int dim = v + jt * 4;
        v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            acc += f[w] * *reinterpret_cast<const v4f *>(lds + w * WAVE_BYTES + (row * (D + 4) + dim) * 4);
        put4<E>(a, all, acc * norm, o_row * D + dim, (slot_row + row) * D + dim);
    }
    if (!all && jt == 0) *reinterpret_cast<v2f *>(a.ws_ml + 2 * (slot_row + row)) = v2f{mm, sum};
}
template <class E, bool F8, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void chunk_few_kernel(const ChunkArgs c) {
    constexpr int WAVES = 4;
    __shared__ __align__(1024) char lds[WAVES * Few<E, F8, D>::WAVE_BYTES];
    __shared__ float lm[WAVES * 16], ll[WAVES * 16];
    __shared__ int before[CHUNK_RUN_BLOCKS + 1], waves[WAVES];
    Work<256> work(c, before, waves);
    Block k;
    int64_t slot;
    while (work.next(k, slot)) {
        few_rows<E, F8, D, WAVES>(c, k, slot, lds, lm, ll);
        __syncthreads();  // (the sums in LDS have been read)
    }
}

// A wave's share of the copies of tiles into LDS.  A copy fills 1 KB of LDS in the order of
// the lanes, so the places in LDS (Tile::k_pos, and values by runs of 16 slots: see
// Attend) are met by what each lane reads: the piece that belongs where it writes.  A
// wave's keys lie in one page and so do its values: their addresses are scalar, looked up a
// turn before they are needed, and a lane adds an offset that never changes.  (With values by
// features in LDS, every lane of a tile of small pages chose its page: ragged prompts under a
// window, heads of 64, took 108 us with pages of 16 and 99 with 64, and take 94 now with both.)
template <class E, bool F8, int D, int KEYS, int RW, int WAVES>
struct Stage {
    typedef Tile<E, F8, D, KEYS, RW, 64, true> PL;  // (for the places of keys alone)
    typedef Frag<E, F8> FR;
    static constexpr int ES = FR::BYTES, KB = PL::KB;
    static constexpr int COPIES = KEYS * KB / 1024;             // of a tile's keys, and of its values
    static constexpr int N = COPIES / WAVES;                    // a wave's of each
    static constexpr int TURN = 2 * N;                          // a wave's of a tile
    static constexpr int K_ROWS = N * 1024 / KB;                // keys of a wave, in one run of 16
    static constexpr int RUN_BYTES = D * 16 * ES;               // values of 16 slots
    static_assert(16 % K_ROWS == 0 && COPIES % WAVES == 0 && RUN_BYTES % (N * 1024) == 0, "a wave's keys share a page, and its values");

    const_ints pages;     // the sequence's row of the table
    const char *k_head, *v_head;  // the head's place in page 0
    uint64_t page_bytes;  // from page to page
    int last_page, shift;
    int wave, lane, total;
    uint32_t k_off[N], v_off[N];  // of this lane's pieces from the first key's row / the run's first value
    uint32_t lds;

    __device__ __forceinline__ Stage(const AttnArgs &a, const Block &k, char *lds_, int wave_, int lane_) : wave(wave_), lane(lane_) {
        shift = a.cache.page_shift;
        total = k.sq.total;
        pages = (const_ints)a.batch.pages + (int64_t)k.b * a.batch.max_pages;
        last_page = (int)(a.cache.n_pages - 1);
        page_bytes = (uint64_t)a.cache.heads * (D * ES) << shift;
        const int64_t head = (int64_t)k.h * (D * ES) << shift;
        k_head = a.cache.k + head;
        v_head = a.cache.v + head;
        lds = lds_offset(lds_);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k_at = copy(i) * 1024 + lane * 16;  // in the tile
            const int row = k_at / KB, piece = (k_at % KB / 16) ^ PL::k_xor(row);
            k_off[i] = (row - k_row()) * KB + piece * 16;
            const int v_at = k_at - v_run() * RUN_BYTES;  // in the run
            v_off[i] = ((uint32_t)(v_at / (16 * ES)) << shift) * ES + v_half(i) * 16;
        }
    }
    __device__ __forceinline__ int copy(int i) const { return N * wave + i; }
    __device__ __forceinline__ int k_row() const { return copy(0) * 1024 / KB; }
    __device__ __forceinline__ int v_run() const { return copy(0) * 1024 / RUN_BYTES; }
    // Which 16 bytes of a feature's run this lane copies.
    __device__ __forceinline__ int v_half(int i) const {
        const int d = (copy(i) * 64 + lane) / ES % D;
        return F8 ? 0 : (lane & 1) ^ (RW == 32 ? d >> 4 & 1 : 0);
    }

    // A slot past the sequence's end is taken to lie in its last run (masked later).
    __device__ __forceinline__ int k_slot(int key0) const { return min(key0 + k_row(), (total - 1) & -K_ROWS); }
    __device__ __forceinline__ int v_slot(int key0) const { return min(key0 + 16 * v_run(), (total - 1) & ~15); }
    __device__ __forceinline__ uint64_t page_at(int e) const { return (uint64_t)(uint32_t)min(max(e, 0), last_page) * page_bytes; }
    // The page entries of a tile's copies.
    __device__ __forceinline__ int k_entry(int key0) const { return pages[k_slot(key0) >> shift]; }
    __device__ __forceinline__ int v_entry(int key0) const { return pages[v_slot(key0) >> shift]; }
    __device__ __forceinline__ void copy_k(int buf, int key0, int e) const {
        const char *p = k_head + page_at(e) + (uint32_t)((k_slot(key0) & ((1 << shift) - 1)) * KB);
#pragma unroll
        for (int i = 0; i < N; ++i) copy16(lds + buf + copy(i) * 1024, p, k_off[i]);
    }
    __device__ __forceinline__ void copy_v(int buf, int key0, int e) const {
        const char *p = v_head + page_at(e) + (uint32_t)((v_slot(key0) & ((1 << shift) - 1)) * ES);
#pragma unroll
        for (int i = 0; i < N; ++i) copy16(lds + buf + copy(i) * 1024, p, v_off[i]);
    }
    // In a tile that some row does not see whole, after this wave's copies of it have arrived:
    // zeros for values past the end, which may be anything, and for infinite and NaN ones;
    // whether this lane met any of those.
    __device__ __forceinline__ bool clean_v(char *at, int buf, int key0) const {
        bool found = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v4u *p = reinterpret_cast<v4u *>(at + buf + copy(i) * 1024 + lane * 16);
            v4u w = *p;
            const int left = total - (key0 + 16 * v_run() + 8 * v_half(i));
            if constexpr (F8) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    typename FR::raw r = {w[2 * j], w[2 * j + 1]};
                    FR::first(r, min(max(left - 8 * j, 0), 8));
                    found |= FR::drop_odd(r);
                    w[2 * j] = r[0];
                    w[2 * j + 1] = r[1];
                }
            } else {
                FR::first(w, min(max(left, 0), 8));
                found |= FR::drop_odd(w);
            }
            *p = w;
        }
        return found;
    }
};

// Up to 128 rows, short texts with heads of 128, and all of heads of 64: 4 waves of 32 rows share the tiles; one is in use and
// AHEAD are on their way.  Copies of tile i + AHEAD start when all waves are done with tile i - 1.
// Heads of 64 leave room for four workgroups on a compute unit if only one tile is on its
// way (98 -> 95 us against three workgroups with two).  Ragged prompts under a window of 1024,
// 24 + 8 heads of 64: 95 us, 600 TFLOP/s.  The vector unit works in 51% of the cycles (some 200
// instructions to a tile of 64 keys and a wave, half of them the softmax's), the matrix unit in
// 28%, both at once in 11%; waves wait 40% of their time for their turn to issue and 28% for
// copies and barriers.  Neither unit is full: what bounds it is how the two take turns.
template <class E, bool F8, int D>
__global__ __launch_bounds__(256, D == 64 ? 4 : 2) void chunk_tile_kernel(const ChunkArgs c) {
    constexpr int RW = 32, KEYS = D == 128 ? 32 : 64;  // (64 at dim 128 would not fit the registers)
    constexpr int AHEAD = D == 64 ? 1 : 2, BUFS = AHEAD + 1;  // tiles on their way
    typedef Stage<E, F8, D, KEYS, RW, 4> ST;
    typedef Rows<E, F8, D, KEYS, RW, true> RS;
    constexpr int BYTES = RS::AT::TL::BYTES, K_BYTES = RS::AT::TL::K_BYTES;

    __shared__ __align__(1024) char lds[BUFS * BYTES];
    __shared__ int odd;  // whether masked tiles copied so far have infinite or NaN values
    __shared__ int before[CHUNK_RUN_BLOCKS + 1], waves[4];

    Work<256> work(c, before, waves);
    Block k;
    int64_t slot;
    const AttnArgs &a = c.a;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (threadIdx.x == 0) odd = 0;
    while (work.next(k, slot)) {
        __syncthreads();  // the piece before has been read
        const Tiles<KEYS> ts(c, k);
        const unsigned thread = this_thread();
        const ST st(a, k, lds, wave, thread & 63);
        RS rs(a, ts, thread);
        const int first = ts.from, n = ts.to - ts.from;
        int key[BUFS];  // the first slots of this tile and those after it
#pragma unroll
        for (int i = 0; i < BUFS; ++i) key[i] = ts.key(first + i);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            st.copy_v(i * BYTES + K_BYTES, key[i], st.v_entry(key[i]));
            st.copy_k(i * BYTES, key[i], st.k_entry(key[i]));
        }
        int ke = st.k_entry(key[AHEAD]);  // of the tile to be copied next
        int ve = st.v_entry(key[AHEAD]);
        const int row0 = (k.rb << c.rows_shift) + wave * RW;
        const bool rows = row0 < k.sq.T * a.group;  // (a wave without rows only copies)
        rs.begin(k, row0);
        int buf = 0;
        for (int i = 0; i < n; ++i) {
            const int t = first + i;
            // (where q's loads are among the newest, this waits for more than it has to)
            arrived<(AHEAD - 1) * ST::TURN>();
            if (ts.block.at(t) && st.clean_v(lds, buf + K_BYTES, key[0])) odd = 1;
            __syncthreads();
            const int next = buf == 0 ? AHEAD * BYTES : buf - BYTES;  // of tile i + AHEAD
            st.copy_v(next + K_BYTES, key[AHEAD], ve);
            st.copy_k(next, key[AHEAD], ke);
            const int then = ts.key(t + BUFS);
            ke = st.k_entry(then);
            ve = st.v_entry(then);
            if (rows) rs.tile(lds, buf, t, key[0]);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) key[j] = key[j + 1];
            key[AHEAD] = then;
            buf = buf == AHEAD * BYTES ? 0 : buf + BYTES;
        }
        arrived<0>();  // (copies of tiles past the last)
        __syncthreads();
        if (odd) rs.odd_values(k, ts.from, 1);
        rs.put(k, slot, wave);
    }
}

// More rows: 8 waves, two to a SIMD, share the tiles, and the second four run half a turn
// behind the first.  A turn has a half of matrix products (the values of the tile before,
// the scores of this one) and a half of vector work (softmax, copies), so that one wave
// of a SIMD keeps its matrix unit busy while the other has its vector unit; a barrier ends
// every half.  Times in halves: the early waves multiply tile i at 2 i, the late ones at
// 2 i + 1.  There are three buffers each for keys and values.  In its vector half i an
// early wave (at 2 i + 1) starts its copies of keys i + 2 and values i + 1: keys i - 1 and
// values i - 2 before them were last read at 2 i - 1, by the late waves.  A late wave (at 2 i
// + 2) starts those of keys i + 3 and values i + 2: keys i and values i - 1 were last read
// at 2 i + 1.  Both wait for them at the end of their next vector half, at 2 i + 4 at
// the latest, and they are first read (keys i + 2 and values i + 1 by the early waves, at
// 2 i + 4; keys i + 3 at 2 i + 6) after the barrier that follows.
// A sequence that brings only a few rows among others that bring many takes the way of
// the few.
// What bounds it is the chip's clock under products, and the waits of a turn: their loop alone
// runs at 1440 TFLOP/s, with copies and softmax at 1000 to 1020 (a prompt of 4096, 32 query and 8
// key heads of 128, 137 to 142 us; 2 pieces of 512 over 32768, 64 query heads, 691 us; a
// library's product of two matrices of 8192: 1310).  The clock, 2.4 GHz at most, is 2.05 in the
// first and 1.6 in the second, where the matrix unit works in 41% and 53% of the cycles and the
// vector unit in 35% and 39%.  All waves in step: 160 and 800 us.  Staged through registers
// instead of copied: 148 and 864.
// RW: rows of a wave, 32, or 16 for less work at dim 256.
template <class E, bool F8, int D, int RW>
__global__ __launch_bounds__(512, 2) void chunk_wide_kernel(const ChunkArgs c) {
    constexpr int KEYS = D == 256 ? 32 : 64;
    // operands read ahead (6 do not fit the registers beside 32 rows of 256: 363 us for 268)
    constexpr int AHEAD = D == 256 && RW == 32 && !F8 ? 2 : 6;
    typedef Stage<E, F8, D, KEYS, RW, 8> ST;
    typedef Rows<E, F8, D, KEYS, RW, true> RS;
    typedef typename RS::AT AT;
    constexpr int BYTES = AT::TL::BYTES, K_BYTES = AT::TL::K_BYTES, FEW_BYTES = Few<E, F8, D>::WAVE_BYTES;
    constexpr int FEW_WAVES = FEW_IN_WIDE<E, F8, D>;
    constexpr int LDS = 3 * BYTES > FEW_WAVES * FEW_BYTES ? 3 * BYTES : FEW_WAVES * FEW_BYTES;

    __shared__ __align__(1024) char lds[LDS];  // keys and values by turns
    __shared__ float lm[FEW_WAVES * 16 + 1], ll[FEW_WAVES * 16 + 1];
    __shared__ int odd;
    __shared__ int before_j[CHUNK_RUN_BLOCKS + 1], waves[8];

    Work<512> work(c, before_j, waves);
    Block k;
    int64_t slot;
    const AttnArgs &a = c.a;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool late = wave >= 4;
    if (threadIdx.x == 0) odd = 0;
    while (work.next(k, slot)) {
        __syncthreads();  // the piece before has been read
        if constexpr (FEW_WAVES > 0) {
            if (k.sq.T * a.group <= 16) {
                few_rows<E, F8, D, FEW_WAVES>(c, k, slot, lds, lm, ll);
                continue;
            }
        }
        const Tiles<KEYS> ts(c, k);
        const unsigned thread = this_thread();
        const ST st(a, k, lds, wave, thread & 63);
        RS rs(a, ts, thread);
        AT &at = rs.at;
        // tiles first .. first + n - 1
        const int first = ts.from, n = ts.to - ts.from;
        const int ahead = late ? 1 : 0;  // the copies of a vector half: keys i + 2 + ahead, values i + 1 + ahead
        for (int i = 0; i < 2 + ahead; ++i) {
            const int key = ts.key(first + i);
            st.copy_k(i * BYTES, key, st.k_entry(key));
            if (i < 1 + ahead) st.copy_v(i * BYTES + K_BYTES, key, st.v_entry(key));
        }
        int kn = ts.key(first + 2 + ahead), vn = ts.key(first + 1 + ahead);  // the slots of the next
        int ke = st.k_entry(kn);
        int ve = st.v_entry(vn);
        int kb = late ? 0 : 2 * BYTES, vb = late ? 2 * BYTES : BYTES;  // and their buffers
        rs.begin(k, (k.rb << c.rows_shift) + wave * RW);
        float p[AT::NT * AT::NR];
        typename AT::op_t pf[AT::NS];
        int key0 = ts.key(first), buf = 0;  // where the turn's tile is
        arrived<0>();
        for (int i = 0; i < 1 + ahead; ++i)
            if (ts.block.at(first + i) && st.clean_v(lds, i * BYTES + K_BYTES, ts.key(first + i))) odd = 1;
        __syncthreads();
        if (late) __syncthreads();
        auto vector_half = [&](int i) {
            const int t = first + i;
            const int clean = t + ahead;  // the tile whose values' copies, started a turn ago, are waited for here
            const bool more = i + 1 < n;
            const int old = vb == 0 ? 2 * BYTES : vb - BYTES;
            if (more) {
                const int kn2 = ts.key(t + 3 + ahead), ke2 = st.k_entry(kn2);
                const int ve2 = st.v_entry(kn);
                st.copy_v(vb + K_BYTES, vn, ve);
                st.copy_k(kb, kn, ke);
                vn = kn;
                kn = kn2;
                ke = ke2;
                ve = ve2;
                kb = kb == 2 * BYTES ? 0 : kb + BYTES;
                vb = vb == 2 * BYTES ? 0 : vb + BYTES;
            }
            rs.mask(t, key0, p);
            rs.weigh(p, pf);
#pragma unroll
            for (int s = 0; s < AT::NS; ++s) {
                v4u w = __builtin_bit_cast(v4u, pf[s]);
                asm volatile("" : "+v"(w));  // (here, and not among the products)
                pf[s] = __builtin_bit_cast(typename AT::op_t, w);
            }
            key0 = ts.key(t + 1);
            if (more)
                arrived<ST::TURN>();
            else
                arrived<0>();
            if (i && clean < ts.to && ts.block.at(clean) && st.clean_v(lds, old + K_BYTES, ts.key(clean))) odd = 1;
        };
        at.template products<false, true, AHEAD>(lds, 0, pf, 0, p);
        __syncthreads();
        vector_half(0);
        __syncthreads();
        for (int i = 1; i < n; ++i) {
            const int before = buf;
            buf = buf == 2 * BYTES ? 0 : buf + BYTES;
            at.template products<true, true, AHEAD>(lds, before + K_BYTES, pf, buf, p);
            __syncthreads();
            vector_half(i);
            __syncthreads();
        }
        at.template products<true, false, AHEAD>(lds, buf + K_BYTES, pf, 0, p);
        __syncthreads();
        if (!late) __syncthreads();
        if (odd) rs.odd_values(k, ts.from, 1);
        rs.put(k, slot, wave);
    }
}

// Where the parts of block j of head h lie: workgroups w0 .. w1 have one each.
struct Parts {
    int from, w0, w1;
    Runs runs;
    // all: the units of a key head (1, with nothing to be found, where offsets that fall leave none)
    __device__ __forceinline__ Parts(const ChunkArgs &c, int j, int h, int all)
        : runs(all * c.a.cache.heads, min(c.a.grid, all * c.a.cache.heads)) {
        from = h * all + c.a.ws_seq[j];
        const int to = h * all + c.a.ws_seq[j + 1];  // (blocks' units follow each other)
        w0 = runs.holder(min(from + c.begin, max(to - 1, 0)));
        w1 = runs.holder(max(to - 1, 0));
    }
    // a workgroup's first piece lies in its first slot
    __device__ __forceinline__ int64_t slot(int w) const { return 2 * (int64_t)w + (runs.begin(w) < from); }
};
// Adds a part (maximum and weight ml, sums po) to the sums o, weight l under maximum m.
template <int N>
__device__ __forceinline__ void join(v4f (&o)[N], float &m, float &l, v2f ml, const v4f (&po)[N]) {
    const float up = fmaxf(m, ml[0]);
    const float f = __builtin_amdgcn_exp2f(m - up), pf = __builtin_amdgcn_exp2f(ml[0] - up);
    m = up;
    l = l * f + ml[1] * pf;
#pragma unroll
    for (int q = 0; q < N; ++q) o[q] = o[q] * f + po[q] * pf;
}
// A row of a cut block that few_rows left: D / 4 threads to a row, `sets` sets of them, which
// share out its parts.  Threads of a set without a row (used) only meet the barrier.
template <class E, int D>
__device__ __forceinline__ void join_few(const ChunkArgs &c, const Parts &parts, int row_in_block, int64_t out_row, bool used,
                                         int sets, v4f *so, v2f *sml) {
    constexpr int TPP = D / 4;
    const int lane = threadIdx.x % TPP, set = threadIdx.x / TPP, sub = set % sets;
    float m = M_START, l = 0.f;
    v4f o[1] = {v4f{0.f, 0.f, 0.f, 0.f}};
    if (used) {
        for (int w = parts.w0 + sub; w <= parts.w1; w += sets) {
            const int64_t r = (parts.slot(w) << c.rows_shift) + row_in_block;
            const v4f po[1] = {*reinterpret_cast<const v4f *>(c.a.ws_o + r * D + 4 * lane)};
            join<1>(o, m, l, *reinterpret_cast<const v2f *>(c.a.ws_ml + 2 * r), po);
        }
    }
    if (sets > 1) {
        so[threadIdx.x] = o[0];
        if (lane == 0) sml[set] = v2f{m, l};
        __syncthreads();
        if (sub) return;
        for (int s = 1; s < sets; ++s) {
            const v4f po[1] = {so[threadIdx.x + s * TPP]};
            join<1>(o, m, l, sml[set + s], po);
        }
    }
    if (used) put4<E>(c.a, true, o[0] * (l == 0.f ? 0.f : c.a.v_scale / l), out_row * D + 4 * lane, 0);
}
// out = sum over the parts of a cut block, each weighted by exp2(its maximum - the
// largest).  Blocks of 16 rows: a workgroup to `rows` heads of a token (a divisor of the
// group, as many sets of threads to each as there are).
template <class E, int D>
__global__ __launch_bounds__(256) void chunk_join_few_kernel(const ChunkArgs c, int rows) {
    constexpr int SETS = 1024 / D;
    __shared__ v4f so[256];
    __shared__ v2f sml[SETS];
    const int G = c.a.group, q_heads = c.a.cache.heads * G;
    const int tok = blockIdx.x, head0 = blockIdx.y * rows, h = head0 / G;
    const int b = __builtin_amdgcn_readfirstlane(batch_seq(c.a.batch, tok));
    int first, count;
    batch_rows(c.a.batch, b, first, count);
    const int i = tok - first;
    if (i < 0 || i >= count) return;  // (a row of no sequence)
    const int all = max(c.a.ws_seq[c.blocks], 1);
    const int sets = SETS / rows, set = threadIdx.x / (D / 4);
    const int row = i * G + head0 % G + min(set / sets, rows - 1);
    const int j = (int)first_block(c, b) + (row >> c.rows_shift);
    const Parts parts(c, j, h, all);
    const bool used = set / sets < rows && parts.w0 != parts.w1;  // (one workgroup: finished there)
    join_few<E, D>(c, parts, row & ((1 << c.rows_shift) - 1), (int64_t)tok * q_heads + head0 + set / sets, used, sets, so, sml);
}
// More rows: a workgroup (its number along y) to the rows that one wave left, a quarter of their
// features to each of its waves; the next part is on its way while one is added.  (A workgroup
// to a block is too few where blocks are few and cut into many parts: 2 pieces of 16 tokens over
// 32768, 64 query and 8 key heads of 128, 90 -> 74 us, of 64, 83 -> 59.)
template <class E, int D, int RW, bool FEW>
__global__ __launch_bounds__(256) void chunk_join_kernel(const ChunkArgs c) {
    constexpr int QUADS = RW * D / 1024;
    const int G = c.a.group, j = (int)(blockIdx.x / (unsigned)c.a.cache.heads), h = (int)(blockIdx.x - (unsigned)j * c.a.cache.heads);
    const Parts parts(c, j, h, max(c.a.ws_seq[c.blocks], 1));
    if (parts.w0 == parts.w1) return;  // finished there, or no block
    const int b = block_seq(c, j);
    int first, count;
    batch_rows(c.a.batch, b, first, count);
    const int64_t rows = (int64_t)count * G;
    const int row0 = (j - (int)first_block(c, b)) << c.rows_shift;
    if (row0 < 0) return;  // (offsets that fall)
    // the output's row of the sequence's row r
    const auto out_row = [&](int r) { return (int64_t)(first + r / G) * ((int64_t)c.a.cache.heads * G) + h * G + r % G; };
    if (FEW && rows <= 16) {
        constexpr int TPP = D / 4, SETS = 256 / TPP;
        for (int r = blockIdx.y * SETS + threadIdx.x / TPP; r < rows; r += SETS * gridDim.y) join_few<E, D>(c, parts, r, out_row(r), true, 1, nullptr, nullptr);
        return;
    }
    const int wave = blockIdx.y, lane = threadIdx.x & 63, n = lane & (RW - 1), g = lane / RW, row = wave * RW + n;
    if (row0 + wave * RW >= rows) return;
    const int q0 = (threadIdx.x >> 6) * QUADS;
    float m = M_START, l = 0.f;
    v4f o[QUADS], next[QUADS];
    v2f next_ml;
#pragma unroll
    for (int q = 0; q < QUADS; ++q) o[q] = v4f{0.f, 0.f, 0.f, 0.f};
    const auto load = [&](int w) {
        const int64_t wave_rows = (parts.slot(w) << c.rows_shift) + wave * RW;
        const v4f *from = reinterpret_cast<const v4f *>(c.a.ws_o + wave_rows * D) + lane;
        next_ml = *reinterpret_cast<const v2f *>(c.a.ws_ml + 2 * (wave_rows + n));
#pragma unroll
        for (int q = 0; q < QUADS; ++q) next[q] = from[(q0 + q) * 64];
    };
    load(parts.w0);
    for (int w = parts.w0; w <= parts.w1; ++w) {
        v4f po[QUADS];
#pragma unroll
        for (int q = 0; q < QUADS; ++q) po[q] = next[q];
        const v2f ml = next_ml;
        if (w < parts.w1) load(w + 1);
        join<QUADS>(o, m, l, ml, po);
    }
    if (row0 + row >= rows) return;
    const float norm = l == 0.f ? 0.f : c.a.v_scale / l;
    const int64_t to = out_row(row0 + row) * D;
    constexpr int NR = RW * RW / 64;
#pragma unroll
    for (int q = 0; q < QUADS; ++q) {
        const int d = (q0 + q) / (NR / 4), r = (q0 + q) % (NR / 4) * 4;
        put4<E>(c.a, true, o[q] * norm, to + RW * d + 2 * r + 4 * g, 0);
    }
}

template <class E, bool F8, int D, int RW>
hipError_t launch_wide(const ChunkArgs &c, const ChunkPlan &p, hipStream_t stream) {
    hipLaunchKernelGGL((chunk_wide_kernel<E, F8, D, RW>), dim3((unsigned)p.grid), dim3(512), 0, stream, c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.runs) return e;
    hipLaunchKernelGGL((chunk_join_kernel<E, D, RW, FEW_IN_WIDE<E, F8, D> != 0>), dim3((unsigned)(p.blocks * c.a.cache.heads), 8), dim3(256),
                       0, stream, c);
    return hipGetLastError();
}

template <class E, bool F8, int D>
hipError_t launch_dim(const ChunkArgs &args, const ChunkPlan &p, hipStream_t stream) {
    ChunkArgs c = args;
    // Among many rows, few count by their bytes: 64 KB of keys and values are read about while 64
    // slots are multiplied by 256 rows (a piece of 512 rows and 23 single tokens over 6000
    // slots of 8 heads of 128, us: 32 KB 136, 64 KB 107, 128 KB 129; in 8 bits 16 KB 153, 64 KB 101,
    // 128 KB 95; 59 tokens and a piece of 300, 8 bits: 64 KB 127, 128 KB 128).
    c.few_shift = CHUNK_UNIT_SHIFT;
    if (p.waves == 8 && FEW_IN_WIDE<E, F8, D>) c.few_shift = D * (F8 ? 1 : 2) == 128 ? 8 : 7;
    const dim3 grid((unsigned)p.grid);
    const unsigned blocks = (unsigned)(p.blocks * c.a.cache.heads);
    if (p.waves == 0) {
        hipLaunchKernelGGL((chunk_few_kernel<E, F8, D>), grid, dim3(256), 0, stream, c);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || !p.runs) return e;
        // many rows: the heads of a group together, as far as there are threads, which find their parts once
        const int heads = c.a.cache.heads * c.a.group;
        int rows = 1;
        if ((int64_t)c.a.batch.n_tokens * heads > 2048)
            while (2 * rows <= 1024 / D && c.a.group % (2 * rows) == 0) rows *= 2;
        hipLaunchKernelGGL((chunk_join_few_kernel<E, D>), dim3((unsigned)c.a.batch.n_tokens, (unsigned)(heads / rows)), dim3(256), 0, stream, c, rows);
        return hipGetLastError();
    }
    if constexpr (D < 256) {
        if (p.waves == 4) {
            hipLaunchKernelGGL((chunk_tile_kernel<E, F8, D>), grid, dim3(256), 0, stream, c);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess || !p.runs) return e;
            hipLaunchKernelGGL((chunk_join_kernel<E, D, 32, false>), dim3(blocks, 4), dim3(256), 0, stream, c);
            return hipGetLastError();
        }
    }
    if constexpr (D == 256) {
        if (p.rows_shift == 7) return launch_wide<E, F8, D, 16>(c, p, stream);
    }
    if constexpr (D > 64) return launch_wide<E, F8, D, 32>(c, p, stream);
    return hipGetLastError();
}

template <class E, bool F8>
hipError_t launch_type(const ChunkArgs &c, const ChunkPlan &p, int dim, hipStream_t stream) {
    switch (dim) {
        case 64: return launch_dim<E, F8, 64>(c, p, stream);
        case 128: return launch_dim<E, F8, 128>(c, p, stream);
        default: return launch_dim<E, F8, 256>(c, p, stream);
    }
}

}  // namespace

hipError_t launch_chunk(const ChunkArgs &c, const ChunkPlan &p, int type, int dim, int q_type, hipStream_t stream) {
    if (q_type == KQ_T_BF16)
        return type == KQ_T_F8 ? launch_type<__bf16, true>(c, p, dim, stream)
                               : launch_type<__bf16, false>(c, p, dim, stream);
    return type == KQ_T_F8 ? launch_type<_Float16, true>(c, p, dim, stream)
                           : launch_type<_Float16, false>(c, p, dim, stream);
}

}  // namespace kq
