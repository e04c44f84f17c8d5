// kq_lora.hip -- low-rank adapters of many requests beside a shared product
// (gfx950):  out[m] = base[m] + scale_i B_i (A_i a^[m]),  i = ids[m].
//
// Two kernels: the first writes t = scale_i A_i a^ ([M][rank], fp32, in the
// workspace), the second adds B_i t.  a^ are the quantized activations that the shared
// product reads, d * qs: int8 values are exact in both 16-bit types, so the first
// product runs on the 16-bit matrix cores without a rounding of its own, block by
// block, and the blocks' scales are applied to its fp32 sums.  t stays in fp32, and so
// does the second product (rounded to 16 bits, t would leave the result off by 2^-9 of the
// adapters' part): in vector operations where there are few rows, with t in parts of 16
// bits where there are many.
//
// What bounds them is memory: 2048 rows, 4096 inputs, 14336 outputs, rank 64: 12 and 55 to 60
// us, of which base and out (235 MB) take 47 at the rate of a large copy.  One row of rank 16:
// 3.4 and 2.9 us, two launches' latency; 64 rows with an adapter each 7.4 and 6.7.  Of rank 128
// the second kernel does not fit its registers (three workgroups to a compute unit leave 168; 41
// to 44 are kept in memory): the call takes 158 (bfloat16) and 166 us (float16).
#include "kq_copy.hpp"
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

// One value of t to a wave, its lanes along K.
template <class E>
__global__ __launch_bounds__(256) void shrink_few_kernel(const LoraArgs a) {
    typedef typename Vec8<E>::type v8;
    const int lane = threadIdx.x & 63;
    const int at = blockIdx.x * 4 + (threadIdx.x >> 6), m = at / a.rank, r = at - m * a.rank;
    if (m >= a.M) return;
    const int id = __builtin_amdgcn_readfirstlane(a.ids[m]);
    if (id < 0 || id >= a.n_adapters) return;
    const E *w = reinterpret_cast<const E *>(a.A) + ((int64_t)id * a.rank + r) * a.K;
    const int8_t *q = a.qs + (int64_t)m * a.K;
    const int shift = a.bs == 256 ? 8 : 7;
    float sum = 0.f;
#pragma unroll 4
    for (int k = lane * 8; k < a.K; k += 512) {
        const v2u x = *reinterpret_cast<const v2u *>(q + k);
        const v8 wr = *reinterpret_cast<const v8 *>(w + k);
        const float d = a.d[(int64_t)(k >> shift) * a.M + m];
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(int8_of(x[e >> 2], e & 3), (float)wr[e], s);
        sum = fmaf(s, d, sum);
    }
    sum = wave_sum(sum);
    if (lane == 0) a.t[(int64_t)m * a.rank + r] = sum * (a.scale ? a.scale[id] : 1.f);
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
// f(which one, id, which lanes).  Lanes past the end hold an id below 0.
template <class F>
__device__ __forceinline__ void each_adapter(int id, int n_adapters, F f) {
    uint64_t left = __ballot(id >= 0 && id < n_adapters);
    for (int i = 0; left; ++i) {
        const int one = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
        const uint64_t same = __ballot(id == one);
        left &= ~same;
        f(i, one, same);
    }
}

// t of 16 tokens: the adapter's rows are the rows of the product and the tokens its
// columns; the waves share out K, and their sums are joined in LDS.  RB: the rank in 16s
// (rank 8: rows 8 .. 15 repeat, and are not stored).  BS: values to a scale.
// A wave brings KS columns of the adapter's rows to LDS, whole runs of a row at a time: as
// operands straight from memory, 16 neighbouring lanes would read 16 rows, a cache access
// each (2048 rows of 4096, rank 64: 65 us so).
template <class E, int RB, int BS>
struct Shrink {
    static constexpr int WAVES = RB >= 8 ? 8 : 16;
    static constexpr int KS = RB >= 4 ? 64 : RB == 2 || BS == 128 ? 128 : 256;
    static constexpr int ROW = KS * 2, PIECES = ROW / 16;  // bytes and 16-byte pieces of a row
    static constexpr int BYTES = RB * 16 * ROW, COPIES = BYTES / 1024;
    static_assert(BS % KS == 0 && WAVES * BYTES <= 131072, "");
    // a row's pieces are permuted by an XOR with bits of the row: the rows that a read
    // serves together lie in different banks
    static __device__ __forceinline__ int xored(int row, int piece) { return ((piece ^ row) & 7) | (piece & ~7); }
    static __device__ __forceinline__ int place(int row, int piece) { return row * ROW + xored(row, piece) * 16; }
};
// The adapters of a tile (where requests meet, or rows come in any order) are shared out over
// this many workgroups; most tiles have one.
constexpr int SHRINK_SHARE = 4;
template <class E, int RB, int BS>
__global__ __launch_bounds__((Shrink<E, RB, BS>::WAVES * 64)) void shrink_tile_kernel(const LoraArgs a) {
    typedef typename Vec8<E>::type v8;
    typedef Shrink<E, RB, BS> SH;
    constexpr int KS = SH::KS, WAVES = SH::WAVES;
    __shared__ __align__(1024) char lds[WAVES * SH::BYTES];
    __shared__ v4f part[WAVES][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int m0 = blockIdx.x * 16, m = min(m0 + n, a.M - 1);
    const int id = m0 + n < a.M ? a.ids[m] : -1;
    const int8_t *q = a.qs + (int64_t)m * a.K + 16 * g;
    char *mine = lds + wave * SH::BYTES;
    const uint32_t to = lds_offset(mine);
    each_adapter(id, a.n_adapters, [&](int i, int one, uint64_t same) {
        if (i % SHRINK_SHARE != (int)blockIdx.y) return;
        const char *w = a.A + (int64_t)one * a.rank * a.K * 2;
        v4f sum[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) sum[r] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int k0 = wave * KS; k0 < a.K; k0 += WAVES * KS) {
            reads_done();
#pragma unroll
            for (int i = 0; i < SH::COPIES; ++i) {
                const int at = i * 1024 + lane * 16, row = at / SH::ROW, p = at % SH::ROW / 16;
                const int piece = SH::xored(row, p);
                copy16(to + i * 1024, w + ((int64_t)min(row, a.rank - 1) * a.K + k0 + piece * 8) * 2);
            }
            v4i x[KS / 64];
#pragma unroll
            for (int i = 0; i < KS / 64; ++i) x[i] = *reinterpret_cast<const v4i *>(q + k0 + 64 * i);
            const float d = a.d[(int64_t)(k0 / BS) * a.M + m];
            arrived<0>();
            v4f s[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) s[r] = v4f{0.f, 0.f, 0.f, 0.f};
            // of 64 columns lane group g has 16 g .. 16 g + 15, half of them in each product
#pragma unroll
            for (int i = 0; i < KS / 32; ++i) {
                v8 f;
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = (E)int8_of(x[i >> 1][2 * (i & 1) + (e >> 2)], e & 3);
                const int piece = 8 * (i >> 1) + 2 * g + (i & 1);
#pragma unroll
                for (int r = 0; r < RB; ++r)
                    s[r] = Vec8<E>::mul(*reinterpret_cast<const v8 *>(mine + SH::place(16 * r + n, piece)), f, s[r]);
            }
#pragma unroll
            for (int r = 0; r < RB; ++r) sum[r] += s[r] * d;
        }
        const float by = a.scale ? a.scale[one] : 1.f;
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            part[wave][lane] = sum[r];
            __syncthreads();
            if (wave == r % WAVES) {
                v4f t = part[0][lane];
#pragma unroll
                for (int k = 1; k < WAVES; ++k) t += part[k][lane];
                if ((same >> n & 1) && 16 * r + 4 * g < a.rank)
                    *reinterpret_cast<v4f *>(a.t + (int64_t)m * a.rank + 16 * r + 4 * g) = t * by;
            }
            __syncthreads();
        }
    });
}

// 16-bit parts of fp32 values, on the matrix cores: t in three bfloat16 parts of 8 bits each is
// exact (below 2^-110 to 2^-133, the smallest bfloat16), an adapter's bfloat16 is one part and its float16 two.  The products of parts
// below 2^-24 of the whole are left out; the rest, added in fp32, is as near to fp32
// products as their sum is.  (fp32 matrix products take 5 times as long: 77 us for
// the 48 of memory at 2048 x 14336, rank 64.)
template <class E>
struct Parts;
template <>
struct Parts<__bf16> {
    static constexpr int N = 1;
    static __device__ __forceinline__ void split(v8bf x, v8bf (&p)[1]) { p[0] = x; }
};
template <>
struct Parts<_Float16> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void split(v8h x, v8bf (&p)[2]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float f = (float)x[e];
            p[0][e] = (__bf16)f;
            p[1][e] = (__bf16)(f - (float)p[0][e]);
        }
    }
};

// 32 tokens by 128 outputs (64 tokens: 73 us where these take 64, and 77 where these take 40 if
// all have adapters of their own); a wave has 32 of the outputs.  The product's rows are tokens and
// its columns outputs.  The parts of t are read from LDS, and the result goes through
// LDS, so that base and out are read and written in whole runs of a row; base is on its
// way while the products run.  R: the rank; WIDE: rows of base and out are 16-byte aligned.
template <class E, int R, bool WIDE>
__global__ __launch_bounds__(256, 3) void expand_tile_kernel(const LoraArgs a) {
    typedef typename Vec8<E>::type v8;
    typedef Parts<E> PT;
    constexpr int TM = 32, TN = 128, LD = TN + 4;
    constexpr int K = R < 16 ? 16 : R, LT = K + 8;  // (rank 8: zeros follow)
    __shared__ __align__(16) float tile[TM * LD];
    __shared__ __align__(16) __bf16 t[3][TM * LT];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 31, g = lane >> 5;
    const int m0 = blockIdx.y * TM, n0 = blockIdx.x * TN;
    const int id = lane < TM && m0 + lane < a.M ? a.ids[m0 + lane] : -1;
    // this thread's part of the result: 4 neighbouring columns of some rows, or one of more
    constexpr int W = WIDE ? 4 : 1, PER = TN / W, STEP = 256 / PER, ROWS = TM / STEP;
    typedef std::conditional_t<WIDE, v4f, float> vw;
    const int row0 = threadIdx.x / PER, c = threadIdx.x % PER * W;
    const int col = min(n0 + c, a.N - W), last = a.M - 1 - m0;  // (past the ends: read again, not written)
    vw base[ROWS];
    if (a.base) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            base[i] = __builtin_nontemporal_load(
                reinterpret_cast<const vw *>(a.base + (int64_t)(m0 + min(row0 + STEP * i, last)) * a.ldb + col));
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) base[i] = vw{};
    }
    const uint64_t some = __ballot(id >= 0 && id < a.n_adapters);
    if (some) {  // (rows without an adapter hold anything, and lead to nothing)
#pragma unroll
        for (int at = threadIdx.x * 4; at < TM * K; at += 1024) {
            const int row = at / K, k = at % K;
            v4f x = {0.f, 0.f, 0.f, 0.f};
            if (k < R) x = *reinterpret_cast<const v4f *>(a.t + (int64_t)(m0 + min(row, last)) * R + k);
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                // (cut off: three times 8 bits are all 24; rounded, the largest would become infinite)
                typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
                v4bf y;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float whole = x[e];  // (a bit cast of an element itself takes the first)
                    const uint32_t top = __builtin_bit_cast(uint32_t, whole) & 0xFFFF0000u;
                    y[e] = __builtin_bit_cast(__bf16, (uint16_t)(top >> 16));
                    x[e] = whole - __builtin_bit_cast(float, top);
                }
                *reinterpret_cast<v4bf *>(&t[p][row * LT + k]) = y;
            }
        }
    }
    __syncthreads();
    // the adapters of the tile one after another, the next one's rows on their way
    const E *w = reinterpret_cast<const E *>(a.B) + (int64_t)min(n0 + wave * 32 + n, a.N - 1) * R + 8 * g;
    const auto rows_of = [&](uint64_t left, v8 (&b)[K / 16]) {
        const int one = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
#pragma unroll
        for (int k = 0; k < K; k += 16) {
            b[k / 16] = v8{};
            if (k + 8 * g < R) b[k / 16] = *reinterpret_cast<const v8 *>(w + (int64_t)one * a.N * R + k);
        }
        return left & ~__ballot(id == one);
    };
    v8 b[K / 16];
    uint64_t left = some, after = 0;
    if (left) after = rows_of(left, b);
    while (left) {
        const uint64_t same = left & ~after;
        v8 next[K / 16];
        uint64_t after_next = 0;
        if (after) after_next = rows_of(after, next);
        v16f acc = {};
#pragma unroll
        for (int k = 0; k < K; k += 16) {
            v8bf bp[PT::N];
            PT::split(b[k / 16], bp);
#pragma unroll
            for (int p = 2; p >= 0; --p) {  // (the small ones first)
                const v8bf x = *reinterpret_cast<const v8bf *>(&t[p][n * LT + k + 8 * g]);
#pragma unroll
                for (int j = PT::N - 1; j >= 0; --j)
                    if (p + j < 3) acc = mfma_bf16_32x32x16(x, bp[j], acc);
            }
        }
        // register i: row 8 (i / 4) + 4 g + i % 4
        float *to = tile + 4 * g * LD + wave * 32 + n;
        const uint32_t rows = (uint32_t)(same >> (4 * g));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int row = 8 * (i >> 2) + (i & 3);
            if (rows >> row & 1u) to[row * LD] = acc[i];
        }
#pragma unroll
        for (int k = 0; k < K / 16; ++k) b[k] = next[k];
        left = after;
        after = after_next;
    }
    __syncthreads();
    const bool in_place = a.base == a.out;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = row0 + STEP * i;
        const bool has = some >> row & 1;
        const vw sum = base[i] + *reinterpret_cast<const vw *>(tile + row * LD + c);
        // (a row without an adapter takes base's bits; what its place of the tile holds is not looked at)
        if (n0 + c < a.N && row <= last && (has || !in_place))
            __builtin_nontemporal_store(has ? sum : base[i], reinterpret_cast<vw *>(a.out + (int64_t)(m0 + row) * a.ldo + n0 + c));
    }
}

template <class E>
hipError_t launch_shrink_tile(const LoraArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.M + 15) / 16), SHRINK_SHARE);
#define KQ_SHRINK(RB)                                                                                       \
    if (a.bs == 256)                                                                                        \
        hipLaunchKernelGGL((shrink_tile_kernel<E, RB, 256>), grid, dim3(Shrink<E, RB, 256>::WAVES * 64), 0, stream, a); \
    else                                                                                                    \
        hipLaunchKernelGGL((shrink_tile_kernel<E, RB, 128>), grid, dim3(Shrink<E, RB, 128>::WAVES * 64), 0, stream, a)
    switch (a.rank) {
        case 8:
        case 16: KQ_SHRINK(1); break;
        case 32: KQ_SHRINK(2); break;
        case 64: KQ_SHRINK(4); break;
        default: KQ_SHRINK(8); break;
    }
#undef KQ_SHRINK
    return hipGetLastError();
}

template <class E, bool WIDE>
hipError_t launch_expand_tile(const LoraArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.N + 127) / 128), (unsigned)((a.M + 31) / 32));
    switch (a.rank) {
        case 8: hipLaunchKernelGGL((expand_tile_kernel<E, 8, WIDE>), grid, dim3(256), 0, stream, a); break;
        case 16: hipLaunchKernelGGL((expand_tile_kernel<E, 16, WIDE>), grid, dim3(256), 0, stream, a); break;
        case 32: hipLaunchKernelGGL((expand_tile_kernel<E, 32, WIDE>), grid, dim3(256), 0, stream, a); break;
        case 64: hipLaunchKernelGGL((expand_tile_kernel<E, 64, WIDE>), grid, dim3(256), 0, stream, a); break;
        default: hipLaunchKernelGGL((expand_tile_kernel<E, 128, WIDE>), grid, dim3(256), 0, stream, a); break;
    }
    return hipGetLastError();
}

template <class E>
hipError_t launch_type(const LoraArgs &a, hipStream_t stream) {
    if (lora_few(a.M, a.rank)) {
        hipLaunchKernelGGL((shrink_few_kernel<E>), dim3((unsigned)((a.M * a.rank + 3) / 4)), dim3(256), 0, stream, a);
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
    const hipError_t e = launch_shrink_tile<E>(a, stream);
    if (e != hipSuccess) return e;
    const bool wide = a.N % 4 == 0 && a.ldo % 4 == 0 && (uintptr_t)a.out % 16 == 0 &&
                      (!a.base || (a.ldb % 4 == 0 && (uintptr_t)a.base % 16 == 0));
    return wide ? launch_expand_tile<E, true>(a, stream) : launch_expand_tile<E, false>(a, stream);
}

}  // namespace

hipError_t launch_lora(const LoraArgs &a, int type, hipStream_t stream) {
    return type == KQ_T_BF16 ? launch_type<__bf16>(a, stream) : launch_type<_Float16>(a, stream);
}

}  // namespace kq
