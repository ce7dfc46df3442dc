// RMS norm of queries and keys per head with the position rotation in the
// same pass, and its gradient.
//
//   n = x r,  r = 1 / sqrt(mean(x^2) + eps),  y = n o w,  pairs of y rotated
//   dy' = the rotation's transpose on dy,  h = dy' o w
//   dx = r (h - n mean(h o n)),   dw = sum over tokens and heads of dy' o n
//
// Both directions are one pass over the tensors (4 bytes an element forward,
// 6 backward) and bound by HBM.  A head of 64 or 128 features is 8 or 16
// lanes of 16 bytes, so one head is one coalesced 128- or 256-byte access and
// its mean a 3- or 4-step shuffle.  Such a group of lanes keeps one token and
// walks a chunk of its heads, because the sines and cosines (8 per lane)
// belong to the token: they are formed once per chunk, and four heads' loads
// are in flight at a time.
//
// Angles.  pos * f with f = base^(-2i/rotary) loses its fraction of a turn in
// fp32 for far positions.  f / (2 pi) is therefore kept as a 64-bit binary
// fraction of a turn; the product with the position modulo 2^64 drops whole
// turns exactly, and its top 32 bits go to sincospif.
#include <math.h>

#include "bdla_attn_internal.h"
#include "bdla_sm100.cuh"

namespace bdla {

namespace {

using sm100::bf16_hi;
using sm100::bf16_lo;
using sm100::pack_bf16;

constexpr int kThreads = 256;
constexpr int kBatch = 4;   // heads in flight per group of lanes

struct Turns {
    uint64_t f[64];   // turns per position of each pair, times 2^64
};

struct NormParams {
    const __nv_bfloat16 *x[2];      // q, k
    int64_t token[2], head[2];      // element strides
    const float *w[2];
    const int32_t *positions, *cu;
    int n_docs, T, tokens, Hq, Hk, rotary, chunk, n_chunks;
    float eps;
};

// Position of a token: given, or its index in its document.  The search stays
// inside cu[0 .. n_docs] whatever the offsets hold.
__device__ __forceinline__ int token_position(const NormParams &p, int t)
{
    if (p.positions != nullptr)
        return p.positions[t];
    if (p.cu == nullptr)
        return t % p.T;
    int lo = 0, hi = p.n_docs - 1;   // last document that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return t - p.cu[lo];
}

// Sines and cosines of a lane's eight features.  Pairs at a distance: feature
// e rotates with pair e mod rotary/2, and `sn` carries the sign of its role
// (first of the pair: a cos - b sin).  Interleaved: entry 2m holds pair m of
// the lane.  Features past `rotary` get (1, 0).
template <bool INTER>
__device__ __forceinline__ void lane_angles(const Turns &tu, int rotary, int e0, int pos, float (&cs)[8],
                                            float (&sn)[8])
{
    const bool live = e0 < rotary;
    const int half = rotary >> 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        cs[j] = 1.0f;
        sn[j] = 0.0f;
        if (!live || (INTER && (j & 1)))
            continue;
        const int i = INTER ? (e0 + j) >> 1 : (e0 < half ? e0 + j : e0 - half + j);
        const uint64_t turns = (uint64_t)(int64_t)pos * tu.f[i];
        sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f, &sn[j], &cs[j]);   // 2^-31: half turns
        if (!INTER && e0 < half)
            sn[j] = -sn[j];
    }
}

// y -> rotated y (or, with `back`, the transpose).  All lanes of the warp
// take part; `partner` is the lane that holds the other halves of the pairs.
template <bool INTER>
__device__ __forceinline__ void rotate(float (&y)[8], const float (&cs)[8], const float (&sn)[8], int partner,
                                       bool back)
{
    if (INTER) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float s = back ? -sn[j] : sn[j];
            const float a = y[j], b = y[j + 1];
            y[j] = a * cs[j] - b * s;
            y[j + 1] = b * cs[j] + a * s;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float o = __shfl_sync(0xffffffffu, y[j], partner);
            y[j] = y[j] * cs[j] + (back ? -sn[j] : sn[j]) * o;
        }
    }
}

template <int LANES> __device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// What a group of lanes works on: item -> (token, first head of its chunk).
template <int D> struct Group {
    static constexpr int kLanes = D / 8;
    static constexpr int kPerBlock = kThreads / kLanes;
    int lane, e0, partner;
    __device__ __forceinline__ explicit Group(int rotary)
    {
        lane = threadIdx.x % kLanes;
        e0 = 8 * lane;
        const int step = rotary / 16;   // lanes between the two halves of a pair
        const int other = e0 < rotary / 2 ? lane + step : (e0 < rotary ? lane - step : lane);
        partner = (int)(threadIdx.x & 31) - lane + other;
    }
};

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads)
qk_norm_kernel(const __grid_constant__ NormParams p, const __grid_constant__ Turns tu, __nv_bfloat16 *__restrict__ qn,
               __nv_bfloat16 *__restrict__ kn)
{
    using G = Group<D>;
    const G g(p.rotary);
    const int64_t item = (int64_t)blockIdx.x * G::kPerBlock + threadIdx.x / G::kLanes;
    // a group past the end follows along (shuffles need whole warps) and loads and stores nothing
    const bool any = item < (int64_t)p.tokens * p.n_chunks;
    const int t = any ? (int)(item / p.n_chunks) : 0;
    const int h0 = any ? (int)(item % p.n_chunks) * p.chunk : 0;
    const int heads = p.Hq + p.Hk;
    const int h1 = any ? min(h0 + p.chunk, heads) : 0;
    float w[2][8];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[s][j] = p.w[s][g.e0 + j];
    float cs[8], sn[8];
    lane_angles<INTER>(tu, p.rotary, g.e0, any ? token_position(p, t) : 0, cs, sn);
    for (int b = 0; b < p.chunk; b += kBatch) {
        uint4 in[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = h0 + b + u;
            if (b + u < p.chunk && h < h1) {
                const int s = h >= p.Hq;
                in[u] = *reinterpret_cast<const uint4 *>(p.x[s] + t * p.token[s] + (s ? h - p.Hq : h) * p.head[s] + g.e0);
            } else {
                in[u] = make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = h0 + b + u;
            const bool key = h >= p.Hq;
            float x[8];
            unpack8(in[u], x);
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ss = fmaf(x[j], x[j], ss);
            const float r = rsqrtf(group_sum<G::kLanes>(ss) * (1.0f / D) + p.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = x[j] * r * (key ? w[1][j] : w[0][j]);
            if (p.rotary > 0)
                rotate<INTER>(x, cs, sn, g.partner, false);
            if (b + u < p.chunk && h < h1) {
                __nv_bfloat16 *dst = key ? kn + ((int64_t)t * p.Hk + h - p.Hq) * D : qn + ((int64_t)t * p.Hq + h) * D;
                *reinterpret_cast<uint4 *>(dst + g.e0) = pack8(x);
            }
        }
    }
}

template <bool GF32>
__device__ __forceinline__ void load_grad(const void *base, int64_t off, float (&x)[8])
{
    if (GF32) {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + off);
        const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + off + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + off), x);
    }
}

template <int D, bool INTER, bool GF32>
__global__ void __launch_bounds__(kThreads)
qk_norm_bwd_kernel(const __grid_constant__ NormParams p, const __grid_constant__ Turns tu,
                   const void *__restrict__ dqn, const void *__restrict__ dkn, __nv_bfloat16 *__restrict__ dq,
                   __nv_bfloat16 *__restrict__ dk, float *__restrict__ part)
{
    using G = Group<D>;
    constexpr int kB = 2;   // heads in flight: two tensors are read
    __shared__ float red[G::kPerBlock][2 * D];
    const G g(p.rotary);
    const int gi = threadIdx.x / G::kLanes;
    float w[2][8], dw[2][8];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[s][j] = p.w[s][g.e0 + j];
            dw[s][j] = 0.0f;
        }
    const int heads = p.Hq + p.Hk;
    const int64_t items = (int64_t)p.tokens * p.n_chunks;
    const int64_t stride = (int64_t)gridDim.x * G::kPerBlock;
    // the block's groups stay together, so that whole warps reach the shuffles
    for (int64_t base = (int64_t)blockIdx.x * G::kPerBlock; base < items; base += stride) {
        const int64_t item = base + gi;
        const bool any = item < items;
        const int t = any ? (int)(item / p.n_chunks) : 0;
        const int h0 = any ? (int)(item % p.n_chunks) * p.chunk : 0;
        const int h1 = any ? min(h0 + p.chunk, heads) : 0;
        float cs[8], sn[8];
        lane_angles<INTER>(tu, p.rotary, g.e0, any ? token_position(p, t) : 0, cs, sn);
        for (int b = 0; b < p.chunk; b += kB) {
            float x[kB][8], y[kB][8];
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                const int h = h0 + b + u;
                if (b + u < p.chunk && h < h1) {
                    const int s = h >= p.Hq;
                    const int hh = s ? h - p.Hq : h;
                    unpack8(*reinterpret_cast<const uint4 *>(p.x[s] + t * p.token[s] + hh * p.head[s] + g.e0), x[u]);
                    load_grad<GF32>(s ? dkn : dqn, ((int64_t)t * (s ? p.Hk : p.Hq) + hh) * D + g.e0, y[u]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[u][j] = y[u][j] = 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                const int h = h0 + b + u;
                const bool live = b + u < p.chunk && h < h1;
                const bool key = h >= p.Hq;
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    ss = fmaf(x[u][j], x[u][j], ss);
                const float r = live ? rsqrtf(group_sum<G::kLanes>(ss) * (1.0f / D) + p.eps)
                                     : (group_sum<G::kLanes>(ss), 0.0f);
                if (p.rotary > 0)
                    rotate<INTER>(y[u], cs, sn, g.partner, true);
                float hn = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[u][j] *= r;   // n
                    const float d = y[u][j] * x[u][j];
                    if (live) {
                        dw[0][j] += key ? 0.0f : d;
                        dw[1][j] += key ? d : 0.0f;
                    }
                    y[u][j] *= key ? w[1][j] : w[0][j];   // h
                    hn = fmaf(y[u][j], x[u][j], hn);
                }
                const float m = group_sum<G::kLanes>(hn) * (1.0f / D);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[u][j] = r * (y[u][j] - x[u][j] * m);
                if (live) {
                    __nv_bfloat16 *dst = key ? dk + ((int64_t)t * p.Hk + h - p.Hq) * D : dq + ((int64_t)t * p.Hq + h) * D;
                    *reinterpret_cast<uint4 *>(dst + g.e0) = pack8(y[u]);
                }
            }
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            red[gi][s * D + g.e0 + j] = dw[s][j];
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
        float v = 0.0f;
        for (int i = 0; i < G::kPerBlock; ++i)
            v += red[i][c];
        part[(size_t)blockIdx.x * 2 * D + c] = v;
    }
}

// Sums the blocks' partial weight gradients, 32 columns a CTA, in the order of
// the blocks: the same sizes give the same bits.
__global__ void __launch_bounds__(256)
norm_dw_kernel(const float *__restrict__ part, int n_part, int D, float *__restrict__ dwq, float *__restrict__ dwk)
{
    __shared__ float red[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    float v = 0.0f;
    for (int i = y; i < n_part; i += 8)
        v += part[(size_t)i * 2 * D + c];
    red[y][threadIdx.x & 31] = v;
    __syncthreads();
    if (y == 0) {
        float s = 0.0f;
        for (int i = 0; i < 8; ++i)
            s += red[i][threadIdx.x];
        (c < D ? dwq : dwk)[c < D ? c : c - D] = s;
    }
}

// Heads per group of lanes: as few as keep the GPU's lanes busy when tokens
// are few, up to 16 when the angles' cost is worth sharing.
int head_chunk(const bdla_attn_dims &d)
{
    const int64_t vecs = (int64_t)d.B * d.T * (d.Hq + d.Hk);
    const int64_t want = vecs / ((int64_t)sm_count() * 256);
    const int c = want < 1 ? 1 : (want > 16 ? 16 : (int)want);
    return c > d.Hq + d.Hk ? d.Hq + d.Hk : c;
}

NormParams norm_params(const bdla_qk_norm_args &a, const bdla_attn_dims &d)
{
    NormParams p;
    p.x[0] = static_cast<const __nv_bfloat16 *>(a.q);
    p.x[1] = static_cast<const __nv_bfloat16 *>(a.k);
    p.token[0] = a.q_token;
    p.token[1] = a.k_token;
    p.head[0] = a.q_head;
    p.head[1] = a.k_head;
    p.w[0] = a.wq;
    p.w[1] = a.wk;
    p.positions = a.positions;
    p.cu = a.cu_seqlens;
    p.n_docs = a.n_docs;
    p.T = d.T;
    p.tokens = d.B * d.T;
    p.Hq = d.Hq;
    p.Hk = d.Hk;
    p.rotary = a.rotary;
    p.chunk = head_chunk(d);
    p.n_chunks = (d.Hq + d.Hk + p.chunk - 1) / p.chunk;
    p.eps = a.eps;
    return p;
}

Turns turns_of(const bdla_qk_norm_args &a)
{
    Turns t;
    for (int i = 0; i < 64; ++i) {
        t.f[i] = 0;
        if (2 * i < a.rotary) {
            // turns per position, at most 1 / (2 pi); scaled by 2^64 without passing 2^63
            const double f = pow(a.base, -2.0 * i / a.rotary) / (2.0 * 3.14159265358979323846);
            t.f[i] = (uint64_t)ldexp(f, 64);
        }
    }
    return t;
}

}  // namespace

cudaError_t launch_qk_norm(const bdla_qk_norm_args &a, __nv_bfloat16 *qn, __nv_bfloat16 *kn,
                           const bdla_attn_dims &d, cudaStream_t stream)
{
    if (d.T == 0)
        return cudaSuccess;
    const NormParams p = norm_params(a, d);
    const Turns tu = turns_of(a);
    const int64_t items = (int64_t)p.tokens * p.n_chunks;
    const int per = kThreads / (d.d / 8);
    const unsigned grid = (unsigned)((items + per - 1) / per);
    if (d.d == 64) {
        if (a.interleaved)
            qk_norm_kernel<64, true><<<grid, kThreads, 0, stream>>>(p, tu, qn, kn);
        else
            qk_norm_kernel<64, false><<<grid, kThreads, 0, stream>>>(p, tu, qn, kn);
    } else {
        if (a.interleaved)
            qk_norm_kernel<128, true><<<grid, kThreads, 0, stream>>>(p, tu, qn, kn);
        else
            qk_norm_kernel<128, false><<<grid, kThreads, 0, stream>>>(p, tu, qn, kn);
    }
    return cudaGetLastError();
}

int norm_bwd_blocks(const bdla_attn_dims &d)
{
    const int chunk = head_chunk(d);
    const int64_t items = (int64_t)d.B * d.T * ((d.Hq + d.Hk + chunk - 1) / chunk);
    const int per = kThreads / (d.d / 8);
    const int64_t need = (items + per - 1) / per, most = (int64_t)sm_count() * 4;
    return (int)(need < most ? need : most);
}

cudaError_t launch_qk_norm_bwd(const bdla_qk_norm_args &a, const void *dqn, const void *dkn, int g_f32,
                               __nv_bfloat16 *dq, __nv_bfloat16 *dk, float *dwq, float *dwk, float *part,
                               const bdla_attn_dims &d, cudaStream_t stream)
{
    const int blocks = norm_bwd_blocks(d);
    if (blocks > 0) {
        const NormParams p = norm_params(a, d);
        const Turns tu = turns_of(a);
#define BDLA_NORM_GO(D_, I_, G_)                                                                                    \
    qk_norm_bwd_kernel<D_, I_, G_><<<blocks, kThreads, 0, stream>>>(p, tu, dqn, dkn, dq, dk, part)
#define BDLA_NORM_D(D_)                                                                                             \
    do {                                                                                                            \
        if (a.interleaved) {                                                                                        \
            if (g_f32)                                                                                              \
                BDLA_NORM_GO(D_, true, true);                                                                       \
            else                                                                                                    \
                BDLA_NORM_GO(D_, true, false);                                                                      \
        } else {                                                                                                    \
            if (g_f32)                                                                                              \
                BDLA_NORM_GO(D_, false, true);                                                                      \
            else                                                                                                    \
                BDLA_NORM_GO(D_, false, false);                                                                     \
        }                                                                                                           \
    } while (0)
        if (d.d == 64)
            BDLA_NORM_D(64);
        else
            BDLA_NORM_D(128);
#undef BDLA_NORM_D
#undef BDLA_NORM_GO
        const cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess)
            return err;
    }
    norm_dw_kernel<<<2 * d.d / 32, 256, 0, stream>>>(part, blocks, d.d, dwq, dwk);
    return cudaGetLastError();
}

}  // namespace bdla
