// kq_keep.hip -- keep an accepted branch: in every cache, slot len + j of a
// sequence takes what slot len + path[j] held (gfx950).
//
// One workgroup to a (cache, key head, sequence) reads all its slots into LDS
// before it writes one, so sources and destinations may overlap in any way.
// The work is small (a few slots); what bounds it is the launch and three
// dependent loads (count, path, page), so all layers go in one launch.
#include "kq_step_device.hpp"

namespace kq {

namespace {

template <class T, int D>
__global__ __launch_bounds__(256) void keep_kernel(const KeepArgs a) {
    constexpr int ES = sizeof(T);
    constexpr int KV = D * ES / 16;  // 16-byte pieces of a key
    constexpr int MAX = KQ_KEEP_MAX_TOKENS;
    __shared__ __align__(16) v4u ks[MAX * KV];
    __shared__ T vs[MAX * D];
    __shared__ int page[2][MAX], place[2][MAX];  // source and destination
    const int b = blockIdx.x, h = blockIdx.y, layer = blockIdx.z;
    int first, T_;
    batch_rows(a.batch, b, first, T_);
    const int n = min(min(max(a.counts[b], 0), T_), MAX);
    if (n == 0) return;
    const int len = max(a.batch.lens[b], 0);
    const int shift = a.cache.page_shift, heads = a.cache.heads;
    if (threadIdx.x < 2 * n) {
        const int which = threadIdx.x / n, j = threadIdx.x % n;
        const int at = which ? j : min(max(a.path[first + j], 0), T_ - 1);
        page[which][j] = slot_page(a.cache, a.batch, b, len + at);
        place[which][j] = (len + at) & ((1 << shift) - 1);
    }
    __syncthreads();
    char *k = a.k[layer], *v = a.v[layer];
    auto key = [&](int which, int j) {
        return reinterpret_cast<v4u *>(k + ((((int64_t)page[which][j] * heads + h) << shift) + place[which][j]) * (D * ES));
    };
    auto value = [&](int which, int j, int d) {
        return reinterpret_cast<T *>(v) + (((int64_t)page[which][j] * heads + h) * D << shift) + ((int64_t)d << shift) +
               place[which][j];
    };
    for (int t = threadIdx.x; t < n * KV; t += 256) ks[t] = key(0, t / KV)[t % KV];
    for (int t = threadIdx.x; t < n * D; t += 256) vs[t] = *value(0, t % n, t / n);
    __syncthreads();
    for (int t = threadIdx.x; t < n * KV; t += 256) key(1, t / KV)[t % KV] = ks[t];
    for (int t = threadIdx.x; t < n * D; t += 256) *value(1, t % n, t / n) = vs[t];
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
