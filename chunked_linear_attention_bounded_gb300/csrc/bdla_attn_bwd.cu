// Causal softmax attention over whole documents, gradient.
#include "bdla_attn_internal.h"

namespace bdla {

namespace {

struct Span2 {
    int64_t start, end;
};

__device__ Span2 document_of(const int32_t *cu, int n_docs, int T, int64_t tokens, int64_t t)
{
    if (cu == nullptr)
        return {t / T * T, t / T * T + T};
    Span2 r = {-1, -1};
    for (int n = 0; n < n_docs; ++n) {
        const DocSpan s = doc_span(cu, n, T);
        if (doc_valid(s, tokens) && t >= s.start && t < s.start + s.len)
            r = {s.start, s.start + s.len};
    }
    return r;
}

__device__ __forceinline__ float warp_sum(float s)
{
    for (int w = 16; w > 0; w >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, w);
    return s;
}

// One warp per (token, query head): delta = dO . o, then dq.
template <int D>
__global__ void __launch_bounds__(128)
attn_dq_kernel(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ k,
               const __nv_bfloat16 *__restrict__ v, const __nv_bfloat16 *__restrict__ o, const float *__restrict__ lse,
               const __nv_bfloat16 *__restrict__ dO, const int32_t *__restrict__ cu, int n_docs, int T, int64_t tokens,
               int Hq, int Hk, float scale, __nv_bfloat16 *__restrict__ dq, float *__restrict__ delta)
{
    constexpr int E = D / 32;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (item >= tokens * Hq)
        return;
    const int64_t t = item / Hq;
    const int h = (int)(item % Hq), kh = h / (Hq / Hk);
    const Span2 doc = document_of(cu, n_docs, T, tokens, t);
    if (doc.start < 0)
        return;
    float x[E], g[E], acc[E], dl = 0.0f;
    for (int e = 0; e < E; ++e) {
        const int64_t off = item * D + lane * E + e;
        x[e] = bf2f(q[off]) * scale;
        g[e] = bf2f(dO[off]);
        dl = fmaf(g[e], bf2f(o[off]), dl);
        acc[e] = 0.0f;
    }
    dl = warp_sum(dl);
    const float l = lse[h * tokens + t];
    for (int64_t j = doc.start; j <= t; ++j) {
        const int64_t off = (j * Hk + kh) * D + lane * E;
        float s = 0.0f, dp = 0.0f;
        for (int e = 0; e < E; ++e) {
            s = fmaf(x[e], bf2f(k[off + e]), s);
            dp = fmaf(g[e], bf2f(v[off + e]), dp);
        }
        const float ds = expf(warp_sum(s) - l) * (warp_sum(dp) - dl) * scale;
        for (int e = 0; e < E; ++e)
            acc[e] = fmaf(ds, bf2f(k[off + e]), acc[e]);
    }
    for (int e = 0; e < E; ++e)
        dq[item * D + lane * E + e] = __float2bfloat16_rn(acc[e]);
    if (lane == 0)
        delta[h * tokens + t] = dl;
}

// One warp per (token, key head).
template <int D>
__global__ void __launch_bounds__(128)
attn_dkv_kernel(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ k,
                const __nv_bfloat16 *__restrict__ v, const float *__restrict__ lse,
                const __nv_bfloat16 *__restrict__ dO, const float *__restrict__ delta, const int32_t *__restrict__ cu,
                int n_docs, int T, int64_t tokens, int Hq, int Hk, float scale, __nv_bfloat16 *__restrict__ dk,
                __nv_bfloat16 *__restrict__ dv)
{
    constexpr int E = D / 32;
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (item >= tokens * Hk)
        return;
    const int64_t t = item / Hk;
    const int kh = (int)(item % Hk), G = Hq / Hk;
    const Span2 doc = document_of(cu, n_docs, T, tokens, t);
    if (doc.start < 0)
        return;
    float x[E], y[E], ak[E], av[E];
    for (int e = 0; e < E; ++e) {
        x[e] = bf2f(k[item * D + lane * E + e]) * scale;
        y[e] = bf2f(v[item * D + lane * E + e]);
        ak[e] = av[e] = 0.0f;
    }
    for (int h = kh * G; h < (kh + 1) * G; ++h)
        for (int64_t i = t; i < doc.end; ++i) {
            const int64_t off = (i * Hq + h) * D + lane * E;
            float s = 0.0f, dp = 0.0f;
            for (int e = 0; e < E; ++e) {
                s = fmaf(x[e], bf2f(q[off + e]), s);
                dp = fmaf(y[e], bf2f(dO[off + e]), dp);
            }
            const float p = expf(warp_sum(s) - lse[h * tokens + i]);
            const float ds = p * (warp_sum(dp) - delta[h * tokens + i]) * scale;
            for (int e = 0; e < E; ++e) {
                ak[e] = fmaf(ds, bf2f(q[off + e]), ak[e]);
                av[e] = fmaf(p, bf2f(dO[off + e]), av[e]);
            }
        }
    for (int e = 0; e < E; ++e) {
        dk[item * D + lane * E + e] = __float2bfloat16_rn(ak[e]);
        dv[item * D + lane * E + e] = __float2bfloat16_rn(av[e]);
    }
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnProblem &p, const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                            const __nv_bfloat16 *v, const __nv_bfloat16 *o, const float *lse,
                            const __nv_bfloat16 *dO, __nv_bfloat16 *dq, __nv_bfloat16 *dk, __nv_bfloat16 *dv,
                            float *delta)
{
    const cudaError_t err = launch_doc_report(p);
    if (err != cudaSuccess || p.tokens == 0)
        return err;
    const unsigned gq = (unsigned)((p.tokens * p.Hq + 3) / 4), gk = (unsigned)((p.tokens * p.Hk + 3) / 4);
#define BDLA_GO(D_)                                                                                                  \
    do {                                                                                                             \
        attn_dq_kernel<D_><<<gq, 128, 0, p.stream>>>(q, k, v, o, lse, dO, p.cu, p.n_docs, p.T, p.tokens, p.Hq, p.Hk, \
                                                     p.scale, dq, delta);                                            \
        attn_dkv_kernel<D_><<<gk, 128, 0, p.stream>>>(q, k, v, lse, dO, delta, p.cu, p.n_docs, p.T, p.tokens, p.Hq,  \
                                                      p.Hk, p.scale, dk, dv);                                        \
    } while (0)
    if (p.d == 64)
        BDLA_GO(64);
    else
        BDLA_GO(128);
#undef BDLA_GO
    return cudaGetLastError();
}

}  // namespace bdla
