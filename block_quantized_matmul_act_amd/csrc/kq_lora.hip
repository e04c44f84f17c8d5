// kq_lora.hip -- low-rank adapters of many requests beside a shared product
// (gfx950):  out[m] = base[m] + scale_i B_i (A_i a^[m]),  i = ids[m].
//
// Two kernels: the first writes t = scale_i A_i a^ ([M][rank], fp32, in the
// workspace), the second adds B_i t.  a^ are the quantized activations that the shared
// product reads, d * qs: int8 values are exact in both 16-bit types, so the first
// product runs on the 16-bit matrix cores without a rounding of its own, block by
// block, and the blocks' scales are applied to its fp32 sums.  t stays in fp32 and the
// second product is formed in fp32 (rounded to 16 bits, t would leave the result off
// by 2^-9 of the adapters' part): in vector operations where there are few rows, on the
// fp32 matrix cores where there are many.
#include "kq_device.hpp"
#include "kq_layer.hpp"

#include <algorithm>

namespace kq {

namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));

template <class E>
struct Vec8;
template <>
struct Vec8<__bf16> {
    typedef v8bf type;
    static __device__ __forceinline__ v4f mul(type a, type b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Vec8<_Float16> {
    typedef v8h type;
    static __device__ __forceinline__ v4f mul(type a, type b, v4f c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

__device__ __forceinline__ float int8_of(uint32_t w, int e) { return (float)(int8_t)(w >> (8 * e)); }

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

// ------------------------------------------------------------------- few rows

// t of RR of the rank rows of one token: a wave to them, its lanes along K.
template <class E, int RR>
__global__ __launch_bounds__(256) void shrink_few_kernel(const LoraArgs a) {
    typedef typename Vec8<E>::type v8;
    const int lane = threadIdx.x & 63;
    const int per = a.rank / RR;  // waves of a token
    const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int m = (int)(at / per), r0 = (int)(at % per) * RR;
    if (m >= a.M) return;
    const int id = __builtin_amdgcn_readfirstlane(a.ids[m]);
    if (id < 0 || id >= a.n_adapters) return;
    const E *w = reinterpret_cast<const E *>(a.A) + ((int64_t)id * a.rank + r0) * a.K;
    const int8_t *q = a.qs + (int64_t)m * a.K;
    const int shift = a.bs == 256 ? 8 : 7;
    float sum[RR];
#pragma unroll
    for (int r = 0; r < RR; ++r) sum[r] = 0.f;
#pragma unroll 2
    for (int k = lane * 8; k < a.K; k += 512) {
        const v2u x = *reinterpret_cast<const v2u *>(q + k);
        const float d = a.d[(int64_t)(k >> shift) * a.M + m];
        v8 wr[RR];
#pragma unroll
        for (int r = 0; r < RR; ++r) wr[r] = *reinterpret_cast<const v8 *>(w + (int64_t)r * a.K + k);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = int8_of(x[e >> 2], e & 3);
#pragma unroll
        for (int r = 0; r < RR; ++r) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(f[e], (float)wr[r][e], s);
            sum[r] = fmaf(s, d, sum[r]);
        }
    }
    const float by = a.scale ? a.scale[id] : 1.f;
#pragma unroll
    for (int r = 0; r < RR; ++r) {
        const float s = wave_sum(sum[r]);
        if (lane == r) a.t[(int64_t)m * a.rank + r0 + r] = s * by;
    }
}

// 64 outputs of a token to a wave.  L = rank / 8 lanes share a row of B, 16 bytes each,
// so a load of the wave is one run of 1 KB; after L loads every lane has one output.
template <class E, int L>
__global__ __launch_bounds__(256) void expand_few_kernel(const LoraArgs a) {
    typedef typename Vec8<E>::type v8;
    const int lane = threadIdx.x & 63, c = lane & (L - 1), row = lane / L;
    const int m = blockIdx.y;
    const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 64;
    if (n0 >= a.N) return;
    const int id = __builtin_amdgcn_readfirstlane(a.ids[m]);
    const int mine = n0 + c * (64 / L) + row;  // this lane's output
    float *out = a.out + (int64_t)m * a.ldo + mine;
    const float *base = a.base ? a.base + (int64_t)m * a.ldb + mine : nullptr;
    const float b = base && mine < a.N ? *base : 0.f;
    if (id < 0 || id >= a.n_adapters) {
        if (mine < a.N && base != out) *out = b;
        return;
    }
    const v4f *t = reinterpret_cast<const v4f *>(a.t + (int64_t)m * a.rank + 8 * c);
    const E *w = reinterpret_cast<const E *>(a.B) + (int64_t)id * a.N * (8 * L) + 8 * c;
    v8 wr[L];
#pragma unroll
    for (int j = 0; j < L; ++j)
        wr[j] = *reinterpret_cast<const v8 *>(w + (int64_t)min(n0 + j * (64 / L) + row, a.N - 1) * (8 * L));
    const v4f t0 = t[0], t1 = t[1];
    float mine_sum = 0.f;
#pragma unroll
    for (int j = 0; j < L; ++j) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf((float)wr[j][e], e < 4 ? t0[e & 3] : t1[e & 3], s);
#pragma unroll
        for (int o = 1; o < L; o <<= 1) s += __shfl_xor(s, o);
        mine_sum = c == j ? s : mine_sum;
    }
    if (mine < a.N) *out = b + mine_sum;
}

// ------------------------------------------------------------------ many rows

// The tokens of a wave's lanes by their adapters, one adapter after another:
// f(id, which lanes).  Lanes past the end hold an id below 0.
template <class F>
__device__ __forceinline__ void each_adapter(int id, int n_adapters, F f) {
    uint64_t left = __ballot(id >= 0 && id < n_adapters);
    while (left) {
        const int one = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
        const uint64_t same = __ballot(id == one);
        left &= ~same;
        f(one, same);
    }
}

// t of 16 tokens: the adapter's rows are the rows of the product and the tokens its
// columns; the 8 waves share out the blocks of K, and their sums are joined in LDS.
template <class E>
__global__ __launch_bounds__(512) void shrink_tile_kernel(const LoraArgs a) {
    typedef typename Vec8<E>::type v8;
    __shared__ v4f part[8][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    const int m0 = blockIdx.x * 16, m = min(m0 + n, a.M - 1);
    const int id = m0 + n < a.M ? a.ids[m] : -1;
    const int8_t *q = a.qs + (int64_t)m * a.K;
    const int steps = a.bs / 32, blocks = a.K / a.bs;
    each_adapter(id, a.n_adapters, [&](int one, uint64_t same) {
        const E *w0 = reinterpret_cast<const E *>(a.A) + (int64_t)one * a.rank * a.K;
        for (int r0 = 0; r0 < a.rank; r0 += 16) {
            // (rank 8: rows 8 .. 15 repeat, and are not stored)
            const E *w = w0 + (int64_t)min(r0 + n, a.rank - 1) * a.K;
            v4f sum = {0.f, 0.f, 0.f, 0.f};
            for (int b = wave; b < blocks; b += 8) {
                const float d = a.d[(int64_t)b * a.M + m];
                v4f s = {0.f, 0.f, 0.f, 0.f};
                const int k0 = b * a.bs + 8 * g;
#pragma unroll 4
                for (int i = 0; i < steps; ++i) {
                    const v8 wr = *reinterpret_cast<const v8 *>(w + k0 + 32 * i);
                    const v2u x = *reinterpret_cast<const v2u *>(q + k0 + 32 * i);
                    v8 f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = (E)int8_of(x[e >> 2], e & 3);
                    s = Vec8<E>::mul(wr, f, s);
                }
                sum += s * d;
            }
            part[wave][lane] = sum;
            __syncthreads();
            if (wave == 0) {
#pragma unroll
                for (int k = 1; k < 8; ++k) sum += part[k][lane];
                const float by = a.scale ? a.scale[one] : 1.f;
                if ((same >> n & 1) && r0 + 4 * g < a.rank)
                    *reinterpret_cast<v4f *>(a.t + (int64_t)m * a.rank + r0 + 4 * g) = sum * by;
            }
            __syncthreads();
        }
    });
}

// 64 tokens by 128 outputs: a wave has 32 of the outputs.  The product's rows are tokens
// and its columns outputs, so that a register of the result is 128 neighbouring bytes
// of two rows.  P: rank indices that a lane supplies to one run of products (the two
// lane groups take runs of P).
template <class E, int P>
__global__ __launch_bounds__(256) void expand_tile_kernel(const LoraArgs a) {
    typedef E run __attribute__((ext_vector_type(P)));
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 31, g = lane >> 5;
    const int m0 = blockIdx.y * 64, col = blockIdx.x * 128 + wave * 32 + n;
    const int id = m0 + lane < a.M ? a.ids[m0 + lane] : -1;
    const uint64_t inside = __ballot(m0 + lane < a.M);
    const uint64_t none = inside & ~__ballot(id >= 0 && id < a.n_adapters);
    auto each_row = [&](uint64_t rows, auto f) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = 32 * h + mfma32_row(i, lane);
                if ((rows >> r & 1) && col < a.N) f(h, i, (int64_t)(m0 + r));
            }
    };
    if (none && a.base != a.out)
        each_row(none, [&](int, int, int64_t m) { a.out[m * a.ldo + col] = a.base ? a.base[m * a.ldb + col] : 0.f; });
    each_adapter(id, a.n_adapters, [&](int one, uint64_t same) {
        const E *w = reinterpret_cast<const E *>(a.B) + ((int64_t)one * a.N + min(col, a.N - 1)) * a.rank + P * g;
        const float *t0 = a.t + (int64_t)min(m0 + n, a.M - 1) * a.rank + P * g;
        const float *t1 = a.t + (int64_t)min(m0 + 32 + n, a.M - 1) * a.rank + P * g;
        v16f acc[2];
        acc[0] = acc[1] = v16f{};
        for (int r = 0; r < a.rank; r += 2 * P) {
            const run wr = *reinterpret_cast<const run *>(w + r);
#pragma unroll
            for (int j = 0; j < P; j += 4) {
                const v4f x0 = *reinterpret_cast<const v4f *>(t0 + r + j), x1 = *reinterpret_cast<const v4f *>(t1 + r + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y = (float)wr[j + e];
                    acc[0] = __builtin_amdgcn_mfma_f32_32x32x2f32(x0[e], y, acc[0], 0, 0, 0);
                    acc[1] = __builtin_amdgcn_mfma_f32_32x32x2f32(x1[e], y, acc[1], 0, 0, 0);
                }
            }
        }
        each_row(same, [&](int h, int i, int64_t m) {
            a.out[m * a.ldo + col] = (a.base ? a.base[m * a.ldb + col] : 0.f) + acc[h][i];
        });
    });
}

template <class E>
hipError_t launch_type(const LoraArgs &a, hipStream_t stream) {
    if (lora_few(a.M)) {
        const int64_t waves = (int64_t)a.M * a.rank;
        if (waves <= 4096)
            hipLaunchKernelGGL((shrink_few_kernel<E, 1>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((shrink_few_kernel<E, 4>), dim3((unsigned)((waves / 4 + 3) / 4)), dim3(256), 0, stream, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const dim3 grid((unsigned)((a.N + 255) / 256), (unsigned)a.M);
        switch (a.rank) {
            case 8: hipLaunchKernelGGL((expand_few_kernel<E, 1>), grid, dim3(256), 0, stream, a); break;
            case 16: hipLaunchKernelGGL((expand_few_kernel<E, 2>), grid, dim3(256), 0, stream, a); break;
            case 32: hipLaunchKernelGGL((expand_few_kernel<E, 4>), grid, dim3(256), 0, stream, a); break;
            case 64: hipLaunchKernelGGL((expand_few_kernel<E, 8>), grid, dim3(256), 0, stream, a); break;
            default: hipLaunchKernelGGL((expand_few_kernel<E, 16>), grid, dim3(256), 0, stream, a); break;
        }
        return hipGetLastError();
    }
    hipLaunchKernelGGL((shrink_tile_kernel<E>), dim3((unsigned)((a.M + 15) / 16)), dim3(512), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((a.N + 127) / 128), (unsigned)((a.M + 63) / 64));
    switch (a.rank) {
        case 8: hipLaunchKernelGGL((expand_tile_kernel<E, 4>), grid, dim3(256), 0, stream, a); break;
        case 16: hipLaunchKernelGGL((expand_tile_kernel<E, 8>), grid, dim3(256), 0, stream, a); break;
        default: hipLaunchKernelGGL((expand_tile_kernel<E, 16>), grid, dim3(256), 0, stream, a); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraArgs &a, int type, hipStream_t stream) {
    return type == KQ_T_BF16 ? launch_type<__bf16>(a, stream) : launch_type<_Float16>(a, stream);
}

}  // namespace kq
