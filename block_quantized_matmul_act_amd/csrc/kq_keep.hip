// kq_keep.hip -- keep an accepted branch: in every cache, slot len + j of a
// sequence takes what slot len + path[j] held (gfx950).
//
// One workgroup to a (sequence, key head, cache) reads all its sources into
// registers before it writes one, so sources and destinations may overlap in any
// way.  The work is small (a few slots); what bounds it is the launch and the
// chain of dependent loads (rows, count, path, page, source), and for many layers
// the lines of the transposed values (a slot's value is 2 bytes of one line for
// each feature, so a move reads and writes 64 times what it moves).  So all
// layers go in one launch, nothing but the places of the slots is in LDS, and
// eight workgroups to a compute unit have their chains under way together: 16
// layers x 32 sequences x 8 heads of 128 in 22 us (27 with the slots in LDS, where
// four workgroups fit).
#include "kq_step_device.hpp"

namespace kq {

namespace {

constexpr int MAX = KQ_KEEP_MAX_TOKENS;
struct Places {
    int page[2][MAX], in[2][MAX];  // of the sources, of the destinations
};

// n <= N slots of one head, N threads side by side
template <class T, int D, int N>
__device__ __forceinline__ void move(const Places &pl, char *k, char *v, int n, int heads, int h, int shift) {
    constexpr int ES = sizeof(T), KV = D * ES / 16;  // 16-byte pieces of a key
    constexpr int KN = (N * KV + 255) / 256, DN = D * N / 256;
    const int t = threadIdx.x, j = t % N;
    auto key = [&](int which, int piece) {
        const int s = piece / KV;
        return reinterpret_cast<v4u *>(k + ((((int64_t)pl.page[which][s] * heads + h) << shift) + pl.in[which][s]) * (D * ES)) +
               piece % KV;
    };
    auto value = [&](int which) {  // feature t / N of slot j
        return reinterpret_cast<T *>(v) + ((((int64_t)pl.page[which][j] * heads + h) * D + t / N) << shift) + pl.in[which][j];
    };
    v4u ks[KN];
    T vs[DN];
#pragma unroll
    for (int i = 0; i < KN; ++i)
        if (t + 256 * i < n * KV) ks[i] = *key(0, t + 256 * i);
    if (j < n) {
        const T *p = value(0);
#pragma unroll
        for (int i = 0; i < DN; ++i) vs[i] = p[(int64_t)(i * (256 / N)) << shift];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KN; ++i)
        if (t + 256 * i < n * KV) *key(1, t + 256 * i) = ks[i];
    if (j < n) {
        T *p = value(1);
#pragma unroll
        for (int i = 0; i < DN; ++i) p[(int64_t)(i * (256 / N)) << shift] = vs[i];
    }
}

template <class T, int D>
__global__ __launch_bounds__(256) void keep_kernel(const KeepArgs a) {
    __shared__ Places pl;
    const int b = blockIdx.x, h = blockIdx.y, layer = blockIdx.z;
    int first, rows;
    batch_rows(a.batch, b, first, rows);
    const int n = min(min(max(a.counts[b], 0), rows), MAX);
    if (n == 0) return;
    const int len = batch_len(a.batch, b);
    const int shift = a.cache.page_shift;
    if (threadIdx.x < 2 * MAX) {
        const int which = threadIdx.x / MAX, j = threadIdx.x % MAX;
        if (j < n) {
            const int at = which ? j : min(max(a.path[first + j], 0), rows - 1);
            pl.page[which][j] = slot_page(a.cache, a.batch, b, len + at);
            pl.in[which][j] = (len + at) & ((1 << shift) - 1);
        }
    }
    __syncthreads();
    if (n <= 16)
        move<T, D, 16>(pl, a.k[layer], a.v[layer], n, a.cache.heads, h, shift);
    else
        move<T, D, 64>(pl, a.k[layer], a.v[layer], n, a.cache.heads, h, shift);
}

template <class T>
hipError_t launch(const KeepArgs &a, int n_caches, int dim, hipStream_t stream) {
    const dim3 grid((unsigned)a.batch.n_seqs, (unsigned)a.cache.heads, (unsigned)n_caches);
    switch (dim) {
        case 64: hipLaunchKernelGGL((keep_kernel<T, 64>), grid, dim3(256), 0, stream, a); break;
        case 128: hipLaunchKernelGGL((keep_kernel<T, 128>), grid, dim3(256), 0, stream, a); break;
        default: hipLaunchKernelGGL((keep_kernel<T, 256>), grid, dim3(256), 0, stream, a); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_keep(const KeepArgs &a, int n_caches, int elem_bytes, int dim, hipStream_t stream) {
    return elem_bytes == 1 ? launch<uint8_t>(a, n_caches, dim, stream) : launch<uint16_t>(a, n_caches, dim, stream);
}

}  // namespace kq
