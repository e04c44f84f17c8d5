// kq_norm.hip -- the input of a product from a layer's running sum (gfx950):
//   s = x + residual,   y = s * w / sqrt(mean s^2 + eps),   a_q8 = quantize(y).
//
// A workgroup holds a row in registers between the two passes over it, so x and
// the residual are read once and s, the int8 blocks and what goes with them are
// written once.  A lane owns runs of 16 consecutive values, as the quantization
// wants them (kq_quant_device.hpp); the mean is the only sum over the row.
// Everything is fp32; s is rounded once to the residual's type, y is formed from
// the unrounded s.
//
// What bounds it is memory: 4096 rows of 4096, fp32, take 49 us, 4.5 TB/s of what is read and
// written, where a copy of 4 GB runs at 4.8 to 5.1.  Tried and slower: lanes that own 4
// neighbouring values, whose loads are whole runs, with the blocks' maxima over more lanes
// (62 us; rows of 14336 54 -> 96), stores or loads past the caches (62 to 78).  One row is
// latency, 3.7 us.
//
// Sums of squares that leave fp32's range (a row's values past 2^60 or so, or so
// small that the squares vanish beside an eps as small) are formed again in 64 bits.
// A row with an infinity or a NaN has no norm: its scales are NaN and its values 0,
// so every product with it is NaN.
#include "kq_layer.hpp"
#include "kq_quant_device.hpp"

#include <algorithm>

namespace kq {

namespace {

// 16 consecutive values of a row as fp32.
template <class T>
struct Run16;
template <>
struct Run16<float> {
    v4f r[4];
    __device__ __forceinline__ void load(const char *p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = reinterpret_cast<const v4f *>(p)[i];
    }
    __device__ __forceinline__ v4f get(int i) const { return r[i]; }
    static __device__ __forceinline__ void store(char *p, const v4f (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) reinterpret_cast<v4f *>(p)[i] = v[i];
    }
};
template <class T>
struct Run16 {
    typedef T v8 __attribute__((ext_vector_type(8)));
    v8 r[2];
    __device__ __forceinline__ void load(const char *p) {
#pragma unroll
        for (int i = 0; i < 2; ++i) r[i] = reinterpret_cast<const v8 *>(p)[i];
    }
    __device__ __forceinline__ v4f get(int i) const {
        const v8 w = r[i >> 1];
        v4f f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = (float)w[4 * (i & 1) + e];
        return f;
    }
    static __device__ __forceinline__ void store(char *p, const v4f (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v8 w;
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = (T)v[2 * i + (e >> 2)][e & 3];
            reinterpret_cast<v8 *>(p)[i] = w;
        }
    }
};

template <class S>
__device__ __forceinline__ S wave_sum(S x) {
#pragma unroll
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

// The sum of x over the WAVES waves of a row, to all its threads.
template <class S, int WAVES>
__device__ __forceinline__ S row_sum(S x, S *lds) {
    x = wave_sum(x);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
        __syncthreads();
        x = lds[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) x += lds[w];
        __syncthreads();  // (the array is used again)
    }
    return x;
}

constexpr int NORM_WIDE = 4;  // rows to a workgroup where a wave takes a whole row

// XT, RT: types of x and of the residual; a row of up to 1024 * WAVES * C values.
template <class XT, class RT, int BS, int WAVES, int C>
__global__ __launch_bounds__((WAVES == 1 ? NORM_WIDE : WAVES) * 64) void norm_kernel(const NormArgs a) {
    constexpr int G = BS / 16, NT = WAVES * 64;
    __shared__ double wide[WAVES];
    float *narrow = reinterpret_cast<float *>(wide);
    const int rows_wg = WAVES == 1 ? NORM_WIDE : 1;
    const int t = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
    const ActSections act = {a.qs, a.d, a.bsums, a.alpha};
    // Workgroups go round the chip's 8 dies, each with a cache of its own.  A die takes 8
    // neighbouring rows of 64, whose scales and sums share lines of the buffer, so that
    // they leave one cache together (16-bit rows 30.4 -> 27.3 us, 1024 rows of 14336 53.6 -> 50.5;
    // all of a die's rows in one run, 48.6 -> 52.9).
    for (int64_t b = blockIdx.x; b < (((a.M + rows_wg - 1) / rows_wg + 63) & ~(int64_t)63); b += gridDim.x) {
        const int64_t row = ((b & ~(int64_t)63) + (b & 7) * 8 + ((b >> 3) & 7)) * rows_wg + (WAVES == 1 ? threadIdx.x >> 6 : 0);
        if (row >= a.M) continue;  // (the same for all threads of the row)
        v4f v[C][4];
        Run16<XT> x[C];
        Run16<RT> r[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = 16 * (t + NT * c);
            if (col < a.K) {
                x[c].load(a.x + (row * a.ldx + col) * sizeof(XT));
                if (a.residual) r[c].load(a.residual + (row * a.ldr + col) * sizeof(RT));
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = 16 * (t + NT * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[c][i] = v4f{0.f, 0.f, 0.f, 0.f};
            if (col < a.K) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[c][i] = x[c].get(i);
                    if (a.residual) v[c][i] += r[c].get(i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) ss = fmaf(v[c][i][e], v[c][i][e], ss);
                }
                if (a.sum) Run16<RT>::store(a.sum + (row * a.lds + col) * sizeof(RT), v[c]);
            }
        }
        ss = row_sum<float, WAVES>(ss, narrow);
        float inv = 1.0f / sqrtf(ss / (float)a.K + a.eps);
        bool odd = false;
        double inv64 = 0.0;
        // (in sum: the squares neither pass fp32 nor, where eps does not cover it, lose bits at its low end)
        const bool far = !(ss < 0x1p120f) || (ss < 0x1p-80f && a.eps < 0x1p-60f);
        if (far) {
            double s64 = 0.0;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s64 += (double)v[c][i][e] * (double)v[c][i][e];
            s64 = row_sum<double, WAVES>(s64, wide);
            odd = !(s64 < __builtin_inf());
            const double mean = s64 / a.K + (double)a.eps;
            inv64 = mean > 0.0 ? 1.0 / sqrt(mean) : 0.0;  // a row of zeros stays one
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = 16 * (t + NT * c);
            const bool valid = col < a.K;
            if (NT * c * 16 >= a.K) break;
            const float *w = a.weight ? a.weight + col : nullptr;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v4f wi = {1.f, 1.f, 1.f, 1.f};
                if (w && valid) wi = *reinterpret_cast<const v4f *>(w + 4 * i);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float s = v[c][i][e];
                    v[c][i][e] = (far ? (float)((double)s * inv64) : s * inv) * wi[e];
                }
            }
            const float amax = block_amax<BS>(v[c]);
            const bool lost = odd || !(amax <= 3.402823466e38f);
            Quantized q = quantize16(v[c], lost ? 0.f : amax);
            if (lost) q.d = __builtin_nanf("");
            put16<BS, BS == 256>(act, q, valid, row, a.M, a.K, col, col / BS, (col / 16) & (G - 1));
        }
    }
}

template <class XT, class RT, int BS>
hipError_t launch_types(const NormArgs &a, hipStream_t stream) {
    const int need = (a.K + 1023) / 1024;  // waves with a run to each lane
    constexpr int64_t MOST = 1 << 20;      // workgroups to a launch: they go on to further rows
    const auto groups = [&](int waves) { return waves == 1 ? (a.M + NORM_WIDE - 1) / NORM_WIDE : a.M; };
#define KQ_NORM(W, C)                                                                                     \
    hipLaunchKernelGGL((norm_kernel<XT, RT, BS, W, C>),                                                   \
                       dim3((unsigned)std::min<int64_t>(MOST, (groups(W) + 63) / 64 * 64)),                      \
                       dim3((W == 1 ? NORM_WIDE : W) * 64), 0, stream, a)
    if (need <= 1)
        KQ_NORM(1, 1);
    else if (need <= 2)
        KQ_NORM(2, 1);
    else if (need <= 4)
        KQ_NORM(4, 1);
    else if (need <= 8)
        KQ_NORM(8, 1);
    else if (need <= 16)
        KQ_NORM(16, 1);
    else if (need <= 32)
        KQ_NORM(16, 2);
    else
        KQ_NORM(16, 4);
#undef KQ_NORM
    return hipGetLastError();
}

template <class XT, class RT>
hipError_t launch_block(const NormArgs &a, int bs, hipStream_t stream) {
    return bs == 256 ? launch_types<XT, RT, 256>(a, stream) : launch_types<XT, RT, 128>(a, stream);
}
template <class XT>
hipError_t launch_residual(const NormArgs &a, int bs, int r_type, hipStream_t stream) {
    switch (r_type) {
        case KQ_T_BF16: return launch_block<XT, __bf16>(a, bs, stream);
        case KQ_T_F16: return launch_block<XT, _Float16>(a, bs, stream);
        default: return launch_block<XT, float>(a, bs, stream);
    }
}

}  // namespace

hipError_t launch_norm_quantize(const NormArgs &a, int bs, int x_type, int r_type, hipStream_t stream) {
    switch (x_type) {
        case KQ_T_BF16: return launch_residual<__bf16>(a, bs, r_type, stream);
        case KQ_T_F16: return launch_residual<_Float16>(a, bs, r_type, stream);
        default: return launch_residual<float>(a, bs, r_type, stream);
    }
}

}  // namespace kq
