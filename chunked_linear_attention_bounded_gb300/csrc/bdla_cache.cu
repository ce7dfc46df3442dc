// The paged cache: writing rows into its pages, and attention of a sequence's
// newest tokens over it.
#include "bdla_attn_internal.h"
#include "bdla_sm100.cuh"

namespace bdla {

namespace {

// Row of position t of a sequence in the cache's [n_pages * page] rows, or -1
// where the table or the page does not reach.
__device__ __forceinline__ int64_t cache_row(const bdla_cache &c, const int32_t *table, int t)
{
    const int e = t / c.page;
    if (t < 0 || e >= c.max_pages)
        return -1;
    const int pg = table[e];
    if (pg < 0 || pg >= c.n_pages)
        return -1;
    return (int64_t)pg * c.page + (t - e * c.page);
}

constexpr int kAppendThreads = 256;

// One warp writes one row of keys and values: Hk * d features, read and
// written once, 16 bytes a lane, four loads of each in flight.
__global__ void __launch_bounds__(kAppendThreads)
cache_append_kernel(const uint4 *__restrict__ k, const uint4 *__restrict__ v, const __grid_constant__ bdla_cache c,
                    const int32_t *__restrict__ rows, const int32_t *__restrict__ counts, int T, int64_t total,
                    int width, DeviceStatus *st)
{
    const int64_t item = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (item >= total)
        return;
    const int b = (int)(item / T), j = (int)(item - (int64_t)b * T);
    int n = T;
    if (counts != nullptr) {
        n = counts[b];
        if (n < 0 || n > T) {
            if (lane == 0)
                set_status(st, BDLA_ERR_DEVICE, (unsigned)b);
            n = n < 0 ? 0 : T;
        }
    }
    if (j >= n)
        return;
    const int src = rows != nullptr ? rows[item] : j;
    const int len = c.lens[b];
    const int64_t row = len < 0 || len > INT32_MAX - T ? -1 : cache_row(c, c.pages + (int64_t)b * c.max_pages, len + j);
    if (row < 0 || src < 0 || src >= T) {
        if (lane == 0)
            set_status(st, BDLA_ERR_DEVICE, (unsigned)b);
        return;
    }
    const uint4 *sk = k + ((int64_t)b * T + src) * width, *sv = v + ((int64_t)b * T + src) * width;
    uint4 *dk = static_cast<uint4 *>(c.k) + row * width, *dv = static_cast<uint4 *>(c.v) + row * width;
    for (int i0 = lane; i0 < width; i0 += 128) {
        uint4 a[4], e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i0 + 32 * u < width) {
                a[u] = sk[i0 + 32 * u];
                e[u] = sv[i0 + 32 * u];
            }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i0 + 32 * u < width) {
                dk[i0 + 32 * u] = a[u];
                dv[i0 + 32 * u] = e[u];
            }
    }
}

// One warp per (sequence, new token, query head), each lane d/32 features.
template <int D>
__global__ void __launch_bounds__(128)
attn_cached_kernel(const __nv_bfloat16 *__restrict__ q, const __grid_constant__ bdla_cache c,
                   const uint64_t *__restrict__ tree, float scale, __nv_bfloat16 *__restrict__ o,
                   float *__restrict__ lse, int T, int Hq, int Hk, int64_t total, DeviceStatus *st)
{
    constexpr int E = D / 32;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (item >= total)
        return;
    const int h = (int)(item % Hq), i = (int)(item / Hq % T), b = (int)(item / Hq / T);
    const int kh = h / (Hq / Hk);
    const int32_t *table = c.pages + (int64_t)b * c.max_pages;
    int len = c.lens[b];
    const int64_t cap = (int64_t)c.max_pages * c.page;
    if (len < 0 || len + (int64_t)T > cap) {
        if (lane == 0)
            set_status(st, BDLA_ERR_DEVICE, (unsigned)b);
    }
    uint64_t see = tree != nullptr ? tree[(int64_t)b * T + i] : (i >= 63 ? ~0ull : (2ull << i) - 1);
    if (T < 64)
        see &= (1ull << T) - 1;
    int end = (int)(len + (int64_t)T < cap ? len + (int64_t)T : cap);
    if (len < 0)
        end = 0;
    float x[E], acc[E], m = -INFINITY, z = 0.0f;
    for (int e = 0; e < E; ++e) {
        x[e] = bf2f(q[item * D + lane * E + e]) * scale;
        acc[e] = 0.0f;
    }
    for (int t = 0; t < end; ++t) {
        if (t >= len && !((see >> (t - len)) & 1))
            continue;
        const int64_t row = cache_row(c, table, t);
        if (row < 0) {
            if (lane == 0)
                set_status(st, BDLA_ERR_DEVICE, (unsigned)b);
            continue;
        }
        const int64_t off = (row * Hk + kh) * D + lane * E;
        float s = 0.0f;
        for (int e = 0; e < E; ++e)
            s = fmaf(x[e], bf2f(static_cast<const __nv_bfloat16 *>(c.k)[off + e]), s);
        for (int w = 16; w > 0; w >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, w);
        const float mn = fmaxf(m, s);
        const float a = m == -INFINITY ? 0.0f : expf(m - mn), p = mn == -INFINITY ? 0.0f : expf(s - mn);
        z = z * a + p;
        for (int e = 0; e < E; ++e)
            acc[e] = acc[e] * a + p * bf2f(static_cast<const __nv_bfloat16 *>(c.v)[off + e]);
        m = mn;
    }
    const float inv = z > 0.0f ? 1.0f / z : (z == 0.0f ? 0.0f : z);
    for (int e = 0; e < E; ++e)
        o[item * D + lane * E + e] = __float2bfloat16_rn(acc[e] * inv);
    if (lane == 0)
        lse[item] = z == 0.0f ? -INFINITY : m + logf(z);
}

}  // namespace

cudaError_t launch_cache_append(const __nv_bfloat16 *k, const __nv_bfloat16 *v, const bdla_cache &c,
                                const int32_t *rows, const int32_t *counts, const bdla_attn_dims &d,
                                DeviceStatus *st, cudaStream_t stream)
{
    const int64_t total = (int64_t)d.B * d.T;
    if (total == 0)
        return cudaSuccess;
    const int per = kAppendThreads / 32;
    cache_append_kernel<<<(unsigned)((total + per - 1) / per), kAppendThreads, 0, stream>>>(
        reinterpret_cast<const uint4 *>(k), reinterpret_cast<const uint4 *>(v), c, rows, counts, d.T, total,
        d.Hk * d.d / 8, st);
    return cudaGetLastError();
}

int cached_splits(const bdla_attn_dims &, int64_t) { return 1; }
size_t cached_partial_bytes(const bdla_attn_dims &, int) { return 0; }

cudaError_t launch_attn_cached(const __nv_bfloat16 *q, const bdla_cache &c, const uint64_t *tree, float scale,
                               __nv_bfloat16 *o, float *lse, const bdla_attn_dims &d, int, void *,
                               DeviceStatus *st, cudaStream_t stream)
{
    const int64_t total = (int64_t)d.B * d.T * d.Hq;
    const unsigned grid = (unsigned)((total + 3) / 4);
    if (d.d == 64)
        attn_cached_kernel<64><<<grid, 128, 0, stream>>>(q, c, tree, scale, o, lse, d.T, d.Hq, d.Hk, total, st);
    else
        attn_cached_kernel<128><<<grid, 128, 0, stream>>>(q, c, tree, scale, o, lse, d.T, d.Hq, d.Hk, total, st);
    return cudaGetLastError();
}

}  // namespace bdla
