// kq_logprobs.hip -- log probabilities of given tokens, entropy and the n
// largest of each row of logits, in one pass over the logits (gfx950).
//
//   m = max x,  s = sum e^(x - m),  t = sum e^(x - m) (x - m)
//   logprob = (x - m) - log s,  entropy = log s - t / s
//
// Every lane keeps its own (m, s, t) in fp32 over 16 values at a time: when m
// rises by u, s and t become s e^-u and (t - u s) e^-u.
//
// The largest values live sorted in the lanes of each wave (lane i: the i-th), as
// 64-bit keys: the value's bits in an order of whole numbers, then the
// complement of its index, so that ties go to the lower index, the order is total
// and the result does not depend on how the row is cut.  A value is a candidate if
// it beats the n-th of them; candidates gather in LDS, and up to 64 at a time
// are sorted by a network over the lanes and merged (the larger of list i and
// candidate 63 - i are the 64 largest of both, in an order that 6 steps sort).
// Before the first values the n-th largest of the lanes' largest bounds the n-th
// from below, so even they bring few candidates; later a candidate is rare, and
// the search costs one comparison per 16 values.
//
// A row is cut into parts where there are too few rows to fill the chip; each
// part leaves (m, s, t) and its n largest, and a second kernel joins them.
// Bound: HBM bandwidth (each logit is read once): 1537 rows of 100277 fp32 logits with 8
// alternatives in 109 us, 5.6 TB/s (a batch loaded a turn ahead: 118 us without).  One
// row of 128256 with 20 alternatives: 8 - 9 us and 7 for the join, bound by latency.  In
// between the selection's fixed cost counts (a sort, candidates and joins in turn for
// every part of a row): 300 x 128256 47 us, 2.2 times the read; and 16-bit logits take
// hardly less time than fp32 ones (1537 x 100277: 107 us), bound by the work on each value.
#include "kq_step_device.hpp"

namespace kq {

namespace {

// finite, so that x - m is never inf - inf for x = -inf, and above no finite x
constexpr float M_START = -3.402823466e38f;
constexpr int BATCH = 1024;        // values of one step of a wave: 16 to a lane
constexpr int WG = 256;

struct Stat {
    float m, s, t;
};
constexpr Stat STAT_0 = {M_START, 0.f, 0.f};
__device__ __forceinline__ float exp_of(float z) { return __builtin_amdgcn_exp2f(z * 1.44269504088896340736f); }

__device__ __forceinline__ void rise(Stat &a, float m) {
    // (-1000 is as good as any u below it, and s = 0 times it is 0 where -inf were NaN)
    const float u = fmaxf(a.m - m, -1000.f), f = exp_of(u);
    a.t = (a.t + u * a.s) * f;
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ void join(Stat &a, Stat b) {
    const float m = fmaxf(a.m, b.m);
    rise(a, m);
    rise(b, m);
    a.s += b.s;
    a.t += b.t;
}

// v of lane (this ^ D)
template <int D>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
    auto dpp = [](uint32_t x, auto C) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(C)::value, 0xF, 0xF, false);
    };
    const int lane = threadIdx.x & 63;
    if constexpr (D == 1) return dpp(v, IC<0xB1>{});
    if constexpr (D == 2) return dpp(v, IC<0x4E>{});
    if constexpr (D == 4) return dpp(dpp(v, IC<0x141>{}), IC<0x1B>{});  // ^ 7, ^ 3
    if constexpr (D == 8) return dpp(v, IC<0x128>{});
    if constexpr (D == 15) return dpp(v, IC<0x140>{});
    if constexpr (D == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return lane & 16 ? r[0] : r[1];
    }
    if constexpr (D == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return lane & 32 ? r[0] : r[1];
    }
}
typedef uint64_t Key;
template <int D>
__device__ __forceinline__ Key key_xor(Key k) {
    return (Key)lane_xor<D>((uint32_t)(k >> 32)) << 32 | lane_xor<D>((uint32_t)k);
}
// One step of a sorting network: the larger key to the lane with bit D clear, or
// in lanes with bit UP set the other way round.
template <int D, int UP>
__device__ __forceinline__ void order(Key &k) {
    const int lane = threadIdx.x & 63;
    const Key o = key_xor<D>(k);
    const bool larger = ((lane & D) == 0) != ((lane & UP) != 0);
    k = (k > o) == larger ? k : o;
}
// a bitonic sequence of 64 keys to a falling one
__device__ __forceinline__ void merge64(Key &k) {
    order<32, 0>(k);
    order<16, 0>(k);
    order<8, 0>(k);
    order<4, 0>(k);
    order<2, 0>(k);
    order<1, 0>(k);
}
__device__ __forceinline__ void sort64(Key &k) {
    order<1, 2>(k);
    order<2, 4>(k), order<1, 4>(k);
    order<4, 8>(k), order<2, 8>(k), order<1, 8>(k);
    order<8, 16>(k), order<4, 16>(k), order<2, 16>(k), order<1, 16>(k);
    order<16, 32>(k), order<8, 32>(k), order<4, 32>(k), order<2, 32>(k), order<1, 32>(k);
    merge64(k);
}
// the 64 largest of two falling sequences, falling
__device__ __forceinline__ Key join64(Key a, Key b) {
    b = key_xor<15>(key_xor<16>(key_xor<32>(b)));  // reversed
    a = a > b ? a : b;
    merge64(a);
    return a;
}

// -inf < ... < -0 = 0 < ... < inf as whole numbers, and back.
__device__ __forceinline__ uint32_t rank_of(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.f);  // (-0 becomes 0)
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t r) {
    return __builtin_bit_cast(float, r ^ ((int)r < 0 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ Key key_of(float v, int i) { return (Key)rank_of(v) << 32 | ~(uint32_t)i; }
__device__ __forceinline__ uint32_t lane_u(uint32_t v, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// The largest keys a wave has seen (0: none), and what candidates must beat: the
// n-th of them, or a bound below it.
struct Top {
    Key list = 0, last = 0;
    float last_v = -__builtin_inff();  // last's value (its rank 0 is below all)
    int held = 0;                      // candidates in LDS
    __device__ __forceinline__ void bound(Key k) {
        last = k;
        last_v = k ? value_of((uint32_t)(k >> 32)) : -__builtin_inff();
    }
    __device__ __forceinline__ void add(Key falling, int n) {
        list = join64(list, falling);
        const Key k = (Key)lane_u((uint32_t)(list >> 32), n - 1) << 32 | lane_u((uint32_t)list, n - 1);
        if (k > last) bound(k);
    }
    __device__ __forceinline__ void flush(const Key *mine, int n) {
        const int lane = threadIdx.x & 63;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        Key k = lane < held ? mine[lane] : 0;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        sort64(k);
        add(k, n);
        held = 0;
    }
    // each lane's (v, i), where `on`
    __device__ __forceinline__ void offer(Key *mine, float v, int i, bool on, int n) {
        const Key k = key_of(v, i);
        uint64_t better = __ballot(on && k > last);
        if (!better) return;
        if (held + __popcll(better) > 64) {
            flush(mine, n);
            better = __ballot(on && k > last);
        }
        if (on && k > last) {
            const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(better >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)better, 0));
            mine[held + before] = k;
        }
        held += __popcll(better);
    }
};

// 16 consecutive-by-pieces values of the row for one lane; rows need only the
// alignment of their type.
template <class T>
struct Load {
    typedef v4u raw;
    static constexpr int PIECE = 16 / sizeof(T);
    static __device__ __forceinline__ raw get(const T *p) {
        typedef v4u __attribute__((aligned(4))) at4;
        typedef v4u __attribute__((aligned(2))) at2;
        if constexpr (sizeof(T) == 4)
            return __builtin_nontemporal_load(reinterpret_cast<const at4 *>(p));
        else
            return __builtin_nontemporal_load(reinterpret_cast<const at2 *>(p));
    }
    static __device__ __forceinline__ void open(raw w, float *x) {
#pragma unroll
        for (int e = 0; e < PIECE; ++e) {
            // the element as a value first: a bit cast of the element itself reads element 0
            const unsigned word = w[sizeof(T) == 4 ? e : e >> 1];
            if constexpr (sizeof(T) == 4)
                x[e] = __builtin_bit_cast(float, word);
            else
                x[e] = (float)__builtin_bit_cast(T, (unsigned short)(word >> (16 * (e & 1))));
        }
    }
};

__device__ __forceinline__ Stat wave_join(Stat a) {
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
        Stat b;
        b.m = __shfl_xor(a.m, x);
        b.s = __shfl_xor(a.s, x);
        b.t = __shfl_xor(a.t, x);
        join(a, b);
    }
    return a;
}

// The workgroup's waves -> one Stat (in every thread of wave 0) and the largest
// keys (in wave 0's list).  keys: LDS, 64 for each wave.
template <bool TOP>
__device__ __forceinline__ void workgroup_join(Stat &st, Top &top, Key *keys, int n) {
    __shared__ Stat stats[WG / 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    st = wave_join(st);
    if (lane == 0) stats[wave] = st;
    if constexpr (TOP) {
        if (top.held) top.flush(keys + wave * 64, n);
        keys[wave * 64 + lane] = top.list;
    }
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int w = 1; w < WG / 64; ++w) {
        join(st, stats[w]);
        if constexpr (TOP) top.list = join64(top.list, keys[w * 64 + lane]);
    }
}

// The row's results, by wave 0.
template <class T, bool TOP>
__device__ __forceinline__ void finish(const LogprobsArgs &a, int64_t row, const T *x, Stat st, const Top &top) {
    const int lane = threadIdx.x & 63;
    const float log_s = logf(st.s);
    for (int i = lane; i < a.n_given; i += 64) {
        const int t = a.tokens[row * a.n_given + i];
        a.logprob[row * a.n_given + i] = t >= 0 && t < a.V ? ((float)x[t] - st.m) - log_s : -__builtin_inff();
    }
    if (a.entropy && lane == 0) a.entropy[row] = log_s - st.t / st.s;
    if constexpr (TOP) {
        if (lane < a.n_top) {
            // (a row with NaNs may have found fewer: any index will do)
            a.top_ids[row * a.n_top + lane] = min(max((int)~(uint32_t)top.list, 0), a.V - 1);
            a.top_logprobs[row * a.n_top + lane] = (value_of((uint32_t)(top.list >> 32)) - st.m) - log_s;
        }
    }
}

template <class T, bool TOP>
__global__ __launch_bounds__(WG) void logprobs_kernel(const LogprobsArgs a) {
    constexpr int PIECE = Load<T>::PIECE, PIECES = 16 / PIECE;
    const int64_t row = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts;
    const int from = part * a.part, to = min(from + a.part, a.V);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const T *x = reinterpret_cast<const T *>(a.x) + row * a.ldx;
    const int n = a.n_top;
    __shared__ Key keys[TOP ? WG : 1];
    Key *mine = keys + (TOP ? wave * 64 : 0);
    Stat st = STAT_0;
    Top top;
    // whole batches are loaded a turn ahead
    constexpr int STEP = WG / 64 * BATCH;
    typename Load<T>::raw next[PIECES];
    auto load = [&](int at) {
#pragma unroll
        for (int p = 0; p < PIECES; ++p) next[p] = Load<T>::get(x + at + (p * 64 + lane) * PIECE);
    };
    int at = from + wave * BATCH;
    if (at + BATCH <= to) load(at);
    for (; at < to; at += STEP) {
        float v[16];
        if (at + BATCH <= to) {
#pragma unroll
            for (int p = 0; p < PIECES; ++p) Load<T>::open(next[p], v + p * PIECE);
            if (at + STEP + BATCH <= to) load(at + STEP);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int i = at + (j / PIECE * 64 + lane) * PIECE + j % PIECE;
                v[j] = i < to ? (float)x[i] : -__builtin_inff();
            }
        }
        float best = v[0];
#pragma unroll
        for (int j = 1; j < 16; ++j) best = fmaxf(best, v[j]);
        if (best > st.m) rise(st, best);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float z = v[j] - st.m, e = exp_of(z);
            st.s += e;
            st.t = fmaf(e, fmaxf(z, -1000.f), st.t);  // (e = 0 where z is below: never 0 * -inf)
        }
        if constexpr (TOP) {
            if (at == from + wave * BATCH) {
                // the n-th largest of the lanes' largest: at least n values reach it
                // (of a lane past the end: none, so the bound is none, too)
                Key k = at + lane * PIECE < to ? key_of(best, INT32_MAX) : 0;
                sort64(k);
                const uint32_t r = lane_u((uint32_t)(k >> 32), n - 1);
                if (r) top.bound((Key)r << 32);
            }
            const int i0 = at + lane * PIECE;  // the lowest index of this lane's values
            if (__any(best > top.last_v || (best == top.last_v && ~(uint32_t)i0 > (uint32_t)top.last))) {
#pragma nounroll
                for (int p = 0; p < PIECES; ++p)
#pragma unroll
                    for (int e = 0; e < PIECE; ++e) {
                        float w = v[e];
#pragma unroll
                        for (int q = 1; q < PIECES; ++q) w = p == q ? v[q * PIECE + e] : w;
                        const int i = at + (p * 64 + lane) * PIECE + e;
                        top.offer(mine, w, i, i < to, n);
                    }
                if (top.held >= 16) top.flush(mine, n);
            }
        }
    }
    workgroup_join<TOP>(st, top, keys, n);
    if (wave) return;
    if (a.parts == 1) {
        finish<T, TOP>(a, row, x, st, top);
        return;
    }
    Stat *stats = reinterpret_cast<Stat *>(a.ws);
    if (lane == 0) stats[blockIdx.x] = st;
    if constexpr (TOP) {
        Key *lists = reinterpret_cast<Key *>(a.ws + (12 * (int64_t)gridDim.x + 7) / 8 * 8);
        if (lane < n) lists[(int64_t)blockIdx.x * n + lane] = top.list;
    }
}

// One workgroup to a row joins its parts.
template <class T, bool TOP>
__global__ __launch_bounds__(WG) void logprobs_join_kernel(const LogprobsArgs a) {
    const int64_t row = blockIdx.x, items = (int64_t)gridDim.x * a.parts;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Stat *stats = reinterpret_cast<const Stat *>(a.ws);
    Stat st = STAT_0;
    Top top;
    for (int p = threadIdx.x; p < a.parts; p += WG) join(st, stats[row * a.parts + p]);
    __shared__ Key keys[TOP ? WG : 1];
    if constexpr (TOP) {
        const int n = a.n_top;
        const Key *lists = reinterpret_cast<const Key *>(a.ws + (12 * items + 7) / 8 * 8) + row * a.parts * n;
        Key next = wave < a.parts && lane < n ? lists[wave * n + lane] : 0;
        for (int p = wave; p < a.parts; p += WG / 64) {
            const Key now = next;
            next = p + WG / 64 < a.parts && lane < n ? lists[(p + WG / 64) * n + lane] : 0;
            top.list = join64(top.list, now);
        }
    }
    workgroup_join<TOP>(st, top, keys, a.n_top);
    if (wave == 0)
        finish<T, TOP>(a, row, reinterpret_cast<const T *>(a.x) + row * a.ldx, st, top);
}

template <class T, bool TOP>
hipError_t launch(const LogprobsArgs &a, int64_t M, hipStream_t stream) {
    hipLaunchKernelGGL((logprobs_kernel<T, TOP>), dim3((unsigned)(M * a.parts)), dim3(WG), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    hipLaunchKernelGGL((logprobs_join_kernel<T, TOP>), dim3((unsigned)M), dim3(WG), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const LogprobsArgs &a, int type, int64_t M, hipStream_t stream) {
    switch (type) {
        case KQ_T_F32: return a.n_top ? launch<float, true>(a, M, stream) : launch<float, false>(a, M, stream);
        case KQ_T_BF16: return a.n_top ? launch<__bf16, true>(a, M, stream) : launch<__bf16, false>(a, M, stream);
        default: return a.n_top ? launch<_Float16, true>(a, M, stream) : launch<_Float16, false>(a, M, stream);
    }
}

}  // namespace kq
