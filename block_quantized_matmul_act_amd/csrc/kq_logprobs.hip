// kq_logprobs.hip -- log probabilities of given tokens, entropy and the n
// largest of each row of logits, in one pass over the logits (gfx950).
//
//   m = max x,  s = sum e^(x - m),  t = sum e^(x - m) (x - m)
//   lse = m + log s,  logprob = x - lse,  entropy = log s - t / s
//
// Every lane keeps its own (m, s, t) in fp32 over 16 values at a time: when m
// rises by u, s and t become s e^-u and (t - u s) e^-u.  The n largest live
// sorted in the lanes of each wave (lane i: the i-th); a value enters only if
// it beats the last of them, which after the first 1024 values of a wave is
// rare, so the search costs one comparison per 16 values.  Ties go to the
// lower index, so the order is total and the result does not depend on how
// the row is cut.
//
// A row is cut into parts where there are too few rows to fill the chip; each
// part leaves (m, s, t) and its n largest, and a second kernel joins them.
// Bound: HBM bandwidth (each logit is read once).
#include "kq_step_device.hpp"

namespace kq {

namespace {

constexpr float M_START = -3e38f;  // finite, so that x - m is never inf - inf for x = -inf
constexpr int BATCH = 1024;        // values of one step of a wave: 16 to a lane
constexpr int WG = 256;

struct Stat {
    float m, s, t;
};
constexpr Stat STAT_0 = {M_START, 0.f, 0.f};
__device__ __forceinline__ float exp_of(float z) { return __builtin_amdgcn_exp2f(z * 1.44269504088896340736f); }

__device__ __forceinline__ void rise(Stat &a, float m) {
    const float u = a.m - m, f = exp_of(u);
    a.t = (a.t + u * a.s) * f;
    // (s = 0 and u = -inf where a row holds +inf: the NaN is the result wanted)
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

// The n largest (value, index) seen by a wave, lane i holding the i-th;
// last_v / last_i (uniform): the n-th.
struct Top {
    float v = -__builtin_inff();
    int i = INT32_MAX;
    float last_v = -__builtin_inff();
    int last_i = INT32_MAX;
};
__device__ __forceinline__ bool beats(float v, int i, float v2, int i2) { return v > v2 || (v == v2 && i < i2); }
__device__ __forceinline__ float lane_f(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// every lane's (v, i) that beats the n-th enters; a lane without a value passes on = false
__device__ __forceinline__ void enter(Top &top, float v, int i, bool on, int n) {
    const int lane = threadIdx.x & 63;
    uint64_t todo = __ballot(on && beats(v, i, top.last_v, top.last_i));
    while (todo) {
        const int src = __ffsll((unsigned long long)todo) - 1;
        todo &= todo - 1;
        const float nv = lane_f(v, src);
        const int ni = __builtin_amdgcn_readlane(i, src);
        if (!beats(nv, ni, top.last_v, top.last_i)) continue;
        const int at = __popcll(__ballot(beats(top.v, top.i, nv, ni)));
        const float pv = __shfl_up(top.v, 1);
        const int pi = __shfl_up(top.i, 1);
        if (lane > at) {
            top.v = pv;
            top.i = pi;
        } else if (lane == at) {
            top.v = nv;
            top.i = ni;
        }
        top.last_v = lane_f(top.v, n - 1);
        top.last_i = __builtin_amdgcn_readlane(top.i, n - 1);
    }
}

// 16 consecutive-by-pieces values of the row for one lane; rows need only the
// alignment of their type.
template <class T>
struct Load;
template <>
struct Load<float> {
    static constexpr int PIECE = 4;
    static __device__ __forceinline__ void get(const float *p, float *x) {
        typedef v4f __attribute__((aligned(4))) u4;
        const v4f w = *reinterpret_cast<const u4 *>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = w[e];
    }
};
template <class T>
struct Load {
    static constexpr int PIECE = 8;
    static __device__ __forceinline__ void get(const T *p, float *x) {
        typedef v4u __attribute__((aligned(2))) u4;
        const v4u w = *reinterpret_cast<const u4 *>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)__builtin_bit_cast(T, (unsigned short)(w[e >> 1] >> (16 * (e & 1))));
    }
};

// What a part leaves in the workspace: [M][parts] Stat, then [M][parts][n] pairs.
struct Pair {
    float v;
    int i;
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

// The workgroup's waves -> one Stat (in every thread of wave 0) and the n
// largest (in wave 0's Top).
template <bool TOP>
__device__ __forceinline__ void workgroup_join(Stat &st, Top &top, int n) {
    __shared__ Stat stats[WG / 64];
    __shared__ Pair pairs[WG / 64][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    st = wave_join(st);
    if (lane == 0) stats[wave] = st;
    if constexpr (TOP) {
        if (lane < n) pairs[wave][lane] = Pair{top.v, top.i};
    }
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int w = 1; w < WG / 64; ++w) {
        join(st, stats[w]);
        if constexpr (TOP) {
            const Pair p = lane < n ? pairs[w][lane] : Pair{0.f, 0};
            enter(top, p.v, p.i, lane < n && p.i != INT32_MAX, n);
        }
    }
}

// The row's results, by wave 0.
template <class T, bool TOP>
__device__ __forceinline__ void finish(const LogprobsArgs &a, int64_t row, const T *x, Stat st, const Top &top) {
    const int lane = threadIdx.x & 63;
    const float log_s = logf(st.s), lse = st.m + log_s;
    for (int i = lane; i < a.n_given; i += 64) {
        const int t = a.tokens[row * a.n_given + i];
        a.logprob[row * a.n_given + i] = t >= 0 && t < a.V ? (float)x[t] - lse : -__builtin_inff();
    }
    if (a.entropy && lane == 0) a.entropy[row] = log_s - st.t / st.s;
    if constexpr (TOP) {
        if (lane < a.n_top) {
            // (a row with NaNs may have found fewer: any index will do)
            a.top_ids[row * a.n_top + lane] = min(max(top.i, 0), a.V - 1);
            a.top_logprobs[row * a.n_top + lane] = top.v - lse;
        }
    }
}

template <class T, bool TOP>
__global__ __launch_bounds__(WG) void logprobs_kernel(const LogprobsArgs a) {
    constexpr int PIECE = Load<T>::PIECE, PIECES = 16 / PIECE;
    const int64_t row = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts;
    const int from = part * a.part, to = min(from + a.part, a.V);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const T *x = reinterpret_cast<const T *>(a.x) + row * a.ldx;
    const int n = a.n_top;
    Stat st = STAT_0;
    Top top;
    for (int at = from + wave * BATCH; at < to; at += WG / 64 * BATCH) {
        float v[16];
        if (at + BATCH <= to) {
#pragma unroll
            for (int p = 0; p < PIECES; ++p) Load<T>::get(x + at + (p * 64 + lane) * PIECE, v + p * PIECE);
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
            const int i0 = at + lane * PIECE;  // the lowest index of this lane's values
            if (__any(best > top.last_v || (best == top.last_v && i0 < top.last_i))) {
#pragma nounroll
                for (int p = 0; p < PIECES; ++p)
#pragma unroll
                    for (int e = 0; e < PIECE; ++e) {
                        float w = v[e];
#pragma unroll
                        for (int q = 1; q < PIECES; ++q) w = p == q ? v[q * PIECE + e] : w;
                        const int i = at + (p * 64 + lane) * PIECE + e;
                        enter(top, w, i, i < to, n);
                    }
            }
        }
    }
    workgroup_join<TOP>(st, top, n);
    if (wave) return;
    if (a.parts == 1) {
        finish<T, TOP>(a, row, x, st, top);
        return;
    }
    Stat *stats = reinterpret_cast<Stat *>(a.ws);
    if (lane == 0) stats[blockIdx.x] = st;
    if constexpr (TOP) {
        Pair *pairs = reinterpret_cast<Pair *>(stats + (int64_t)gridDim.x);
        if (lane < n) pairs[(int64_t)blockIdx.x * n + lane] = Pair{top.v, top.i};
    }
}

// One workgroup to a row joins its parts.
template <class T, bool TOP>
__global__ __launch_bounds__(WG) void logprobs_join_kernel(const LogprobsArgs a) {
    const int64_t row = blockIdx.x, items = (int64_t)gridDim.x * a.parts;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Stat *stats = reinterpret_cast<const Stat *>(a.ws);
    Stat st = STAT_0;
    Top top;
    for (int p = threadIdx.x; p < a.parts; p += WG) join(st, stats[row * a.parts + p]);
    if constexpr (TOP) {
        const Pair *pairs = reinterpret_cast<const Pair *>(stats + items) + row * a.parts * a.n_top;
        const int all = a.parts * a.n_top;
        for (int p0 = wave * 64; p0 < all; p0 += WG) {
            const bool on = p0 + lane < all;
            const Pair p = on ? pairs[p0 + lane] : Pair{0.f, 0};
            enter(top, p.v, p.i, on && p.i != INT32_MAX, a.n_top);
        }
    }
    workgroup_join<TOP>(st, top, a.n_top);
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
