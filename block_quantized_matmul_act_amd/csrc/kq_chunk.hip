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
// Where the blocks do not fill the chip their keys are cut into equal parts, which
// leave their sums in the workspace for a second kernel to join, in a fixed order.
// Blocks late in a text have the most keys, and go first.
#include "kq_attn_device.hpp"
#include "kq_layer.hpp"

namespace kq {

namespace {

// A block's share of the work: tiles [from, to) of KEYS slots.  Slots are counted in
// units of 64: first the units of the sinks, then those of the window.
struct Block {
    int b, h, rb;
    Seq sq;
    int pos0, pos1;  // slots of its first and last token
    int sink_units, window_unit;
    int from, to;    // units
    int part, parts;
};

// The sequence that has block number j of a key head: the last one whose first
// number is not above it.
__device__ __forceinline__ int64_t first_block(const ChunkArgs &c, int b) {
    const int64_t row = (int64_t)min(max(c.a.batch.offsets[b], 0), c.a.batch.n_tokens) * c.a.group;
    return (row >> c.rows_shift) + b;
}
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
    return lo;
}

// Block j of head h; false if there is none, or no such part of it.
__device__ __forceinline__ bool block_at(const ChunkArgs &c, int j, int h, int part, Block &k) {
    const int b = __builtin_amdgcn_readfirstlane(block_seq(c, j));
    k.b = b;
    k.h = h;
    k.rb = j - (int)first_block(c, b);
    Seq &q = k.sq;
    batch_rows(c.a.batch, b, q.first, q.rows);
    q.T = q.rows;
    q.len = batch_len(c.a.batch, b);
    // slots past the sequence's row of the page table are not there
    const int64_t table = (int64_t)c.a.batch.max_pages << c.a.cache.page_shift;
    q.total = (int)min((int64_t)q.len + q.T, table);
    const int64_t row0 = (int64_t)k.rb << c.rows_shift, rows = (int64_t)q.T * c.a.group;
    if (k.rb < 0 || row0 >= rows) return false;
    const int64_t row1 = min(row0 + (1 << c.rows_shift), rows);
    k.pos0 = q.len + (int)(row0 / c.a.group);
    k.pos1 = q.len + (int)((row1 - 1) / c.a.group);
    const int end = min(k.pos1 + 1, q.total);
    const int begin = min(max(k.pos0 - (c.window - 1), 0), end);
    k.window_unit = begin >> CHUNK_UNIT_SHIFT;
    const int end_unit = (int)(((int64_t)end + CHUNK_UNIT - 1) >> CHUNK_UNIT_SHIFT);
    const int sinks = (min(c.sinks, end) + CHUNK_UNIT - 1) >> CHUNK_UNIT_SHIFT;
    k.sink_units = min(sinks, k.window_unit);
    const int units = k.sink_units + end_unit - k.window_unit;
    const int size = max(c.part_units, (units + c.parts - 1) / c.parts);
    k.parts = max(1, (units + size - 1) / size);
    k.part = part;
    k.from = min(part * size, units);
    k.to = min(k.from + size, units);
    return part < k.parts;
}

// What a workgroup does of the grid.
__device__ __forceinline__ bool my_block(const ChunkArgs &c, Block &k, int64_t &slot_row) {
    const int heads = c.a.cache.heads;
    const unsigned w = blockIdx.x, rest = w / heads;
    const int h = (int)(w - rest * heads), part = (int)(rest % c.parts), j = c.blocks - 1 - (int)(rest / c.parts);
    slot_row = (((int64_t)j * heads + h) * c.parts + part) << c.rows_shift;
    return block_at(c, j, h, part, k);
}

// The tiles of a part, and who sees what of them.
template <int KEYS>
struct Tiles {
    static constexpr int F = CHUNK_UNIT / KEYS;
    const ChunkArgs &c;
    int sink_units, window_unit, from, to;  // tiles
    int pos0, pos1;
    __device__ __forceinline__ Tiles(const ChunkArgs &c_, const Block &k) : c(c_) {
        sink_units = k.sink_units;
        window_unit = k.window_unit;
        from = k.from * F;
        to = k.to * F;
        pos0 = k.pos0;
        pos1 = k.pos1;
        if (F > 1 && to > from && key(to - 1) > pos1) --to;  // half a unit past the end
    }
    __device__ __forceinline__ int key(int t) const {
        const int u = t / F;
        return ((u < sink_units ? u : u - sink_units + window_unit) << CHUNK_UNIT_SHIFT) + t % F * KEYS;
    }
    // whether rows from slot p0 to slot p1 all see the whole tile at key0
    __device__ __forceinline__ bool whole(int key0, int p0, int p1) const {
        return key0 + KEYS - 1 <= p0 && (key0 > p1 - c.window || key0 + KEYS <= c.sinks);
    }
    __device__ __forceinline__ bool edge(int key0) const { return !whole(key0, pos0, pos1); }
    // which of the 8 keys from k the row of slot pos sees
    __device__ __forceinline__ uint32_t on(int k, int pos) const {
        const int back = max(pos - k, -1);  // (below 0 for all the same: the sums stay in 32 bits)
        const int upto = min(back + 1, 8), out = min(max(back - (c.window - 1), 0), 8);
        const int sink = min(max(c.sinks - k, 0), 8);
        return ((1u << upto) - 1u) & (~((1u << out) - 1u) | ((1u << sink) - 1u));
    }
};

// One wave's rows over the tiles.
template <class E, bool F8, int D, int KEYS, int RW>
struct Rows {
    typedef Attend<E, F8, D, KEYS, RW> AT;
    AT at;
    const Tiles<KEYS> &tiles;
    int pos, pos0, pos1;  // slot of this lane's row, of the wave's first and last
    __device__ __forceinline__ Rows(const AttnArgs &a, const Tiles<KEYS> &t) : at(a), tiles(t) {}
    __device__ __forceinline__ void begin(const Block &k, int row0) {
        const int G = at.a.group;
        pos = k.sq.len + at.begin_rows(k.sq, k.h, row0);
        pos0 = __builtin_amdgcn_readfirstlane(min(k.sq.len + row0 / G, k.pos1));
        pos1 = __builtin_amdgcn_readfirstlane(min(k.sq.len + (row0 + RW - 1) / G, k.pos1));
        if (!at.used) pos = pos1;
    }
    __device__ __forceinline__ void mask(int key0, float (&p)[AT::NT * AT::NR]) {
        if (!tiles.whole(key0, pos0, pos1)) {
            int k0 = key0;
            asm volatile("" : "+s"(k0));  // (the masks are not worked out ahead of this branch)
            at.hide(p, [&](int s) { return tiles.on(k0 + 8 * AT::NG * s + 8 * at.g, pos); });
        }
        at.lift(p);
    }
    __device__ __forceinline__ void tile(const char *lds, int buf, int key0) {
        float p[AT::NT * AT::NR];
        typename AT::op_t pf[AT::NS];
        at.template products<false, true, 4>(lds, 0, pf, buf, p);
        mask(key0, p);
        at.add_values(lds, buf, p, pf);
    }
    // What infinite and NaN values in tiles that some row does not see whole add.
    __device__ __forceinline__ void odd_values(const Block &k, int from, int step) {
#pragma nounroll
        for (int t = from; t < tiles.to; t += step) {
            const int key0 = tiles.key(t);
            if (!tiles.edge(key0)) continue;
#pragma nounroll
            for (int key = key0; key < key0 + KEYS; key += 8 * AT::NG)
                add_odd<E, F8, D, RW>(ValueRows{at.a.cache, at.a.batch, k.b, k.h, k.sq.total}, key, at.lane,
                                      tiles.on(key + 8 * at.g, pos), at.o);
        }
    }
};

// Up to 16 rows: the waves take tiles in turn, each its own in LDS without a barrier,
// and their sums are joined in LDS.
template <class E, bool F8, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void chunk_few_kernel(const ChunkArgs c) {
    constexpr int RW = 16, WAVES = 4;
    constexpr int KEYS = D * (F8 ? 1 : 2) >= 256 ? 32 : 64;
    typedef Tile<E, F8, D, KEYS, RW, 64, true> TL;
    typedef Rows<E, F8, D, KEYS, RW> RS;
    constexpr int O_FLOATS = RW * (D + 4);
    constexpr int WAVE_BYTES = TL::BYTES > O_FLOATS * 4 ? TL::BYTES : (O_FLOATS * 4 + 1023) / 1024 * 1024;

    __shared__ __align__(1024) char lds[WAVES * WAVE_BYTES];  // a wave's tile, then its sums [row][dim]
    __shared__ float lm[WAVES * RW], ll[WAVES * RW];

    Block k;
    int64_t slot_row;
    if (!my_block(c, k, slot_row)) return;
    const AttnArgs &a = c.a;
    const Tiles<KEYS> tiles(c, k);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mine = wave * WAVE_BYTES;
    TL tl(a, threadIdx.x & 63);
    RS rs(a, tiles);
    typename RS::AT &at = rs.at;
    tl.aim(k.b, k.h, k.sq);
    int t = tiles.from + wave;
    typename TL::Place next = tl.find(tiles.key(t));
    tl.load_k(next);
    tl.load_v(next);
    next = tl.find(tiles.key(t + WAVES));
    const int row0 = k.rb * RW;
    rs.begin(k, row0);
    bool odd = false;
    for (; t < tiles.to; t += WAVES) {
        const int key0 = tiles.key(t);
        tl.store_k(lds, mine);
        odd |= tl.store_v(lds, mine + TL::K_BYTES, key0, tiles.edge(key0));
        if (t + WAVES < tiles.to) {
            tl.load_k(next);
            tl.load_v(next);
            next = tl.find(tiles.key(t + 2 * WAVES));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        rs.tile(lds, mine, key0);
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
    const int row = threadIdx.x >> 4, jt = threadIdx.x & 15;  // 16 threads to a row
    if (row0 + row >= k.sq.T * a.group) return;
    const bool all = k.parts == 1;
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

// Up to 128 rows: 4 waves of 32 share the tiles, two in LDS.
template <class E, bool F8, int D>
__global__ __launch_bounds__(256, 2) void chunk_tile_kernel(const ChunkArgs c) {
    constexpr int RW = 32, KEYS = D == 128 ? 32 : 64;
    typedef Tile<E, F8, D, KEYS, RW, 256, false> TL;
    typedef Rows<E, F8, D, KEYS, RW> RS;

    __shared__ __align__(1024) char lds[2 * TL::BYTES];
    __shared__ int odd;  // whether masked tiles staged so far have infinite or NaN values

    Block k;
    int64_t slot_row;
    if (!my_block(c, k, slot_row)) return;
    const AttnArgs &a = c.a;
    const Tiles<KEYS> tiles(c, k);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    TL tl(a, threadIdx.x);
    RS rs(a, tiles);
    if (threadIdx.x == 0) odd = 0;
    tl.aim(k.b, k.h, k.sq);
    const int first = tiles.from;
    typename TL::Place next = tl.find(tiles.key(first));
    tl.load_k(next);
    tl.load_v(next);
    next = tl.find(tiles.key(first + 1));
    const int row0 = (k.rb << c.rows_shift) + wave * RW;
    const bool rows = row0 < k.sq.T * a.group;  // (a wave without rows only stages)
    rs.begin(k, row0);
    __syncthreads();
    tl.store_k(lds, 0);
    if (tl.store_v(lds, TL::K_BYTES, tiles.key(first), tiles.edge(tiles.key(first)))) odd = 1;
    tl.load_k(next);
    tl.load_v(next);
    next = tl.find(tiles.key(first + 2));
    int buf = 0;
    for (int t = first; t < tiles.to; ++t) {
        __syncthreads();
        if (rows) rs.tile(lds, buf, tiles.key(t));
        buf = TL::BYTES - buf;
        if (t + 1 < tiles.to) {
            const int key1 = tiles.key(t + 1);
            tl.store_k(lds, buf);
            if (tl.store_v(lds, buf + TL::K_BYTES, key1, tiles.edge(key1))) odd = 1;
            tl.load_k(next);
            tl.load_v(next);
            next = tl.find(tiles.key(t + 3));
        }
    }
    __syncthreads();
    if (odd) rs.odd_values(k, tiles.from, 1);
    rs.at.put(k.parts == 1, slot_row + wave * RW);
}

// More rows: 8 waves, two to a SIMD, the second four half a turn behind the first
// (kq_attn.hip, attn_wide_kernel: the same turns).
template <class E, bool F8, int D>
__global__ __launch_bounds__(512, 2) void chunk_wide_kernel(const ChunkArgs c) {
    constexpr int RW = D == 256 ? 16 : 32, KEYS = D == 256 ? 32 : 64;
    typedef Tile<E, F8, D, KEYS, RW, 512, false> TL;
    typedef Rows<E, F8, D, KEYS, RW> RS;
    typedef typename RS::AT AT;

    __shared__ __align__(1024) char lds[3 * TL::BYTES];  // keys and values by turns
    __shared__ int odd;

    Block k;
    int64_t slot_row;
    if (!my_block(c, k, slot_row)) return;
    const AttnArgs &a = c.a;
    const Tiles<KEYS> ts(c, k);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool late = wave >= 4;
    TL tl(a, threadIdx.x);
    RS rs(a, ts);
    AT &at = rs.at;
    if (threadIdx.x == 0) odd = 0;
    const int first = ts.from, tiles = ts.to - ts.from;
    tl.aim(k.b, k.h, k.sq);
    // keys 0, 1 and values 0 to LDS; keys 2 and values 1 on their way
    typename TL::Place p0 = tl.find(ts.key(first)), p1 = tl.find(ts.key(first + 1)), p2 = tl.find(ts.key(first + 2));
    tl.load_k(p0);
    tl.load_v(p0);
    rs.begin(k, (k.rb << c.rows_shift) + wave * RW);
    __syncthreads();
    tl.store_k(lds, 0);
    if (tl.store_v(lds, TL::K_BYTES, ts.key(first), ts.edge(ts.key(first)))) odd = 1;
    tl.load_k(p1);
    tl.store_k(lds, TL::BYTES);
    tl.load_v(p1);
    tl.load_k(p2);
    p1 = p2;
    p2 = tl.find(ts.key(first + 3));
    float p[AT::NT * AT::NR];
    typename AT::op_t pf[AT::NS];
    int key0 = ts.key(first), buf = 0;  // buf: where tile i is (i % 3)
    __syncthreads();
    if (late) __syncthreads();
    auto vector_half = [&](int i, int before, int after) {
        rs.mask(key0, p);
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < AT::NS; ++s) {
            v4u w = __builtin_bit_cast(v4u, at.probabilities(p, s, sum));
            asm volatile("" : "+v"(w));  // (now, while the loads for the staging below arrive)
            pf[s] = __builtin_bit_cast(typename AT::op_t, w);
        }
        at.l += sum;
        if (i + 1 < tiles) {
            const int key1 = ts.key(first + i + 1);
            tl.store_k(lds, before);  // keys i + 2
            if (tl.store_v(lds, after + TL::K_BYTES, key1, ts.edge(key1))) odd = 1;
            tl.load_v(p1);
            tl.load_k(p2);
            p1 = p2;
            p2 = tl.find(ts.key(first + i + 4));
        }
    };
    at.template products<false, true, 6>(lds, 0, pf, 0, p);
    __syncthreads();
    vector_half(0, 2 * TL::BYTES, TL::BYTES);
    __syncthreads();
    for (int i = 1; i < tiles; ++i) {
        key0 = ts.key(first + i);
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
    if (odd) rs.odd_values(k, ts.from, 1);
    at.put(k.parts == 1, slot_row + wave * RW);
}

// out = sum over the parts of a cut block, each weighted by exp2(its maximum - the
// largest).  D / 4 threads read a part's sums of a row; a workgroup has 256 / (D / 4)
// such sets, `sets` of them to a row, which share out its parts.
template <class E, int D>
__global__ __launch_bounds__(256) void chunk_join_kernel(const ChunkArgs c, int sets) {
    constexpr int TPP = D / 4, SETS = 256 / TPP;
    __shared__ v4f so[256];
    __shared__ v2f sml[SETS];
    const AttnArgs &a = c.a;
    const int heads = a.cache.heads, rows_wg = SETS / sets;
    const unsigned turns = (1u << c.rows_shift) / rows_wg;  // workgroups of a block
    const unsigned jh = blockIdx.x / turns;
    const int j = (int)(jh / heads), h = (int)(jh % heads);
    Block k;
    if (!block_at(c, j, h, 0, k) || k.parts == 1) return;
    const int lane = threadIdx.x % TPP, set = threadIdx.x / TPP, sub = set % sets;
    const int row = (int)(blockIdx.x % turns) * rows_wg + set / sets;
    const int64_t in_seq = ((int64_t)k.rb << c.rows_shift) + row;
    const bool used = in_seq < (int64_t)k.sq.T * a.group;
    const int64_t slot0 = (((int64_t)j * heads + h) * c.parts << c.rows_shift) + row;
    float m = M_START, l = 0.f;
    v4f o = {0.f, 0.f, 0.f, 0.f};
    if (used) {
        for (int p = sub; p < k.parts; p += sets) {
            const int64_t r = slot0 + ((int64_t)p << c.rows_shift);
            const v2f ml = *reinterpret_cast<const v2f *>(a.ws_ml + 2 * r);
            const v4f po = *reinterpret_cast<const v4f *>(a.ws_o + r * D + 4 * lane);
            const float up = fmaxf(m, ml[0]);
            const float f = __builtin_amdgcn_exp2f(m - up), pf = __builtin_amdgcn_exp2f(ml[0] - up);
            m = up;
            l = l * f + ml[1] * pf;
            o = o * f + po * pf;
        }
    }
    if (sets > 1) {
        so[threadIdx.x] = o;
        if (lane == 0) sml[set] = v2f{m, l};
        __syncthreads();
        if (sub) return;
        for (int s = 1; s < sets; ++s) {
            const v2f ml = sml[set + s];
            const float up = fmaxf(m, ml[0]);
            const float f = __builtin_amdgcn_exp2f(m - up), pf = __builtin_amdgcn_exp2f(ml[0] - up);
            m = up;
            l = l * f + ml[1] * pf;
            o = o * f + so[threadIdx.x + s * TPP] * pf;
        }
    }
    if (!used) return;
    const float norm = l == 0.f ? 0.f : a.v_scale / l;
    const int tok = (int)(in_seq / a.group);
    const int64_t row_out = (int64_t)(k.sq.first + tok) * ((int64_t)heads * a.group) + h * a.group + (in_seq - (int64_t)tok * a.group);
    put4<E>(a, true, o * norm, row_out * D + 4 * lane, 0);
}

template <class E, bool F8, int D>
hipError_t launch_dim(const ChunkArgs &c, const ChunkPlan &p, hipStream_t stream) {
    const int64_t heads = c.a.cache.heads;
    const dim3 grid((unsigned)(p.blocks * heads * p.parts));
    if (p.waves == 0)
        hipLaunchKernelGGL((chunk_few_kernel<E, F8, D>), grid, dim3(256), 0, stream, c);
    else if (p.waves == 8)
        hipLaunchKernelGGL((chunk_wide_kernel<E, F8, D>), grid, dim3(512), 0, stream, c);
    else if constexpr (D < 256)
        hipLaunchKernelGGL((chunk_tile_kernel<E, F8, D>), grid, dim3(256), 0, stream, c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.bytes == 0) return e;
    constexpr int SETS = 1024 / D;
    const int sets = p.waves == 0 ? SETS : 1;
    hipLaunchKernelGGL((chunk_join_kernel<E, D>), dim3((unsigned)(p.blocks * heads * ((1 << p.rows_shift) * sets / SETS))),
                       dim3(256), 0, stream, c, sets);
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
