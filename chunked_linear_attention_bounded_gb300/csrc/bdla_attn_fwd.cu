// Causal softmax attention over whole documents, forward.
#include "bdla_attn_internal.h"

namespace bdla {

namespace {

// One warp per (token, query head), each lane d/32 features.
template <int D>
__global__ void __launch_bounds__(128)
attn_fwd_kernel(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ k,
                const __nv_bfloat16 *__restrict__ v, const int32_t *__restrict__ cu, int n_docs, int T, int64_t tokens,
                int Hq, int Hk, float scale, __nv_bfloat16 *__restrict__ o, float *__restrict__ lse)
{
    constexpr int E = D / 32;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (item >= tokens * Hq)
        return;
    const int64_t t = item / Hq;
    const int h = (int)(item % Hq), kh = h / (Hq / Hk);
    int64_t start = t / (T > 0 ? T : 1) * T;
    if (cu != nullptr) {
        start = -1;
        for (int n = 0; n < n_docs; ++n) {
            const DocSpan s = doc_span(cu, n, T);
            if (doc_valid(s, tokens) && t >= s.start && t < s.start + s.len)
                start = s.start;
        }
        if (start < 0)
            return;
    }
    float x[E], acc[E], m = -INFINITY, z = 0.0f;
    for (int e = 0; e < E; ++e) {
        x[e] = bf2f(q[item * D + lane * E + e]) * scale;
        acc[e] = 0.0f;
    }
    for (int64_t j = start; j <= t; ++j) {
        const int64_t off = (j * Hk + kh) * D + lane * E;
        float s = 0.0f;
        for (int e = 0; e < E; ++e)
            s = fmaf(x[e], bf2f(k[off + e]), s);
        for (int w = 16; w > 0; w >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, w);
        const float mn = fmaxf(m, s);
        const float a = m == -INFINITY ? 0.0f : expf(m - mn), p = mn == -INFINITY ? 0.0f : expf(s - mn);
        z = z * a + p;
        for (int e = 0; e < E; ++e)
            acc[e] = acc[e] * a + p * bf2f(v[off + e]);
        m = mn;
    }
    for (int e = 0; e < E; ++e)
        o[item * D + lane * E + e] = __float2bfloat16_rn(z == 0.0f ? 0.0f : acc[e] / z);
    if (lane == 0)
        lse[h * tokens + t] = z == 0.0f ? -INFINITY : m + logf(z);
}

__global__ void doc_report_kernel(const int32_t *cu, int n_docs, int64_t tokens, DeviceStatus *st)
{
    for (int n = threadIdx.x; n < n_docs; n += blockDim.x)
        if (cu[n + 1] < cu[n] || (n == 0 && cu[0] != 0) || (n == n_docs - 1 && cu[n_docs] != tokens))
            set_status(st, BDLA_ERR_DEVICE, (unsigned)n);
}

}  // namespace

cudaError_t launch_doc_report(const AttnProblem &p)
{
    if (p.cu != nullptr)
        doc_report_kernel<<<1, 256, 0, p.stream>>>(p.cu, p.n_docs, p.tokens, p.st);
    return cudaGetLastError();
}

cudaError_t launch_attn_fwd(const AttnProblem &p, const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                            const __nv_bfloat16 *v, __nv_bfloat16 *o, float *lse)
{
    const cudaError_t err = launch_doc_report(p);
    if (err != cudaSuccess || p.tokens == 0)
        return err;
    const unsigned grid = (unsigned)((p.tokens * p.Hq + 3) / 4);
    if (p.d == 64)
        attn_fwd_kernel<64><<<grid, 128, 0, p.stream>>>(q, k, v, p.cu, p.n_docs, p.T, p.tokens, p.Hq, p.Hk, p.scale, o, lse);
    else
        attn_fwd_kernel<128><<<grid, 128, 0, p.stream>>>(q, k, v, p.cu, p.n_docs, p.T, p.tokens, p.Hq, p.Hk, p.scale, o, lse);
    return cudaGetLastError();
}

}  // namespace bdla
