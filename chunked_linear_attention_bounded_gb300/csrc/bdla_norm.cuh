// What the kernels that norm and rotate heads share: how lanes divide a head,
// positions, angles, and a lane's arithmetic.
//
// Angles.  pos * f with f = base^(-2i/rotary) loses its fraction of a turn in
// fp32 for far positions.  f / (2 pi) is therefore kept as a 64-bit binary
// fraction of a turn; the product with the position modulo 2^64 drops whole
// turns exactly.  Its top 32 bits, to the nearest quarter turn and the rest (at
// most an eighth), give sine and cosine from their Taylor series to x^9 and
// x^10 (remainders (pi/4)^11 / 11! = 2e-9 and (pi/4)^12 / 12! = 1e-10, below
// half a step of fp32): with sincospif the angles were a third of the gradient's
// instructions, which bound it.
#pragma once

#include <math.h>

#include "bdla_attn_sm100.cuh"

namespace bdla {
namespace norm {

using attn::add2;
using attn::fma2;
using attn::mul2;
using attn::pair;
using attn::unpair;
using sm100::bf16_hi;
using sm100::bf16_lo;
using sm100::pack_bf16;

constexpr int kThreads = 256;
constexpr int kBatch = 8;   // heads in flight per group of lanes (64K packed tokens from cold: 258 us with 4, 213 with 8)

struct Turns {
    uint64_t f[64];   // turns per position of each pair, times 2^64
};

struct NormParams {
    const __nv_bfloat16 *x[2];      // q, k
    int64_t token[2], head[2];      // element strides
    const float *w[2];
    const int32_t *positions, *cu;
    int n_docs, T, tokens, heads[2], rotary, chunk, q_chunks, n_chunks;
    float eps;
};

// Last document that starts at or before token t.  The search stays inside
// cu[0 .. n_docs - 1] whatever the offsets hold.
__device__ __forceinline__ int document_of(const NormParams &p, int t)
{
    int lo = 0, hi = p.n_docs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Position of a token: given, or its index in its document.
__device__ __forceinline__ int token_position(const NormParams &p, int t)
{
    if (p.positions != nullptr)
        return p.positions[t];
    if (p.cu == nullptr)
        return t % p.T;
    return t - p.cu[document_of(p, t)];
}

// Cosine and sine of h / 2^32 turns.
__device__ __forceinline__ void turn(uint32_t h, float &c, float &s)
{
    const uint32_t q = (h + 0x20000000u) >> 30;   // nearest quarter, 0 .. 3 (4 wraps to 0)
    const float x = (float)(int32_t)(h - (q << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
    const float z = x * x;
    const float a = x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), 1.0f);
    const float b =
        fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const float sa = q & 1 ? b : a, ca = q & 1 ? a : b;
    s = __uint_as_float(__float_as_uint(sa) ^ ((q & 2) << 30));
    c = __uint_as_float(__float_as_uint(ca) ^ (((q + 1) & 2) << 30));
}

// What a group of lanes works on: one token and a chunk of its query (s = 0)
// or key (s = 1) heads.  The lane's sixteen features are f0 .. f0 + 7 and
// f1 .. f1 + 7.  Pairs at a distance: feature f0 + j turns with f1 + j, and
// lanes past the rotated features hold sixteen in a row.  Interleaved: sixteen
// in a row, features 2m and 2m + 1 turn together.
constexpr int kPairs = 8, kFeat = 2 * kPairs;   // of a lane
template <int D, bool INTER> struct Group {
    static constexpr int kLanes = D / kFeat;
    static constexpr int kPerBlock = kThreads / kLanes;
    int f0, f1, t, s, h0, h1;
    bool turns;
    __device__ __forceinline__ explicit Group(const NormParams &p)
    {
        const int lane = threadIdx.x % kLanes;
        turns = kFeat * lane < p.rotary;
        f0 = turns && !INTER ? kPairs * lane : kFeat * lane;
        f1 = turns && !INTER ? (p.rotary >> 1) + kPairs * lane : kFeat * lane + kPairs;
    }
    // A group past the end has no heads, and follows along: shuffles need whole warps.
    __device__ __forceinline__ void take(const NormParams &p, int64_t item)
    {
        const bool any = item < (int64_t)p.tokens * p.n_chunks;
        t = any ? (int)(item / p.n_chunks) : 0;
        const int c = any ? (int)(item - (int64_t)t * p.n_chunks) : 0;
        s = c >= p.q_chunks;
        h0 = (s ? c - p.q_chunks : c) * p.chunk;
        h1 = any ? min(h0 + p.chunk, p.heads[s]) : h0;
    }
    // The same over the chunks of queries or of keys alone.
    __device__ __forceinline__ void take_of(const NormParams &p, int which, int64_t item)
    {
        const int n = which ? p.n_chunks - p.q_chunks : p.q_chunks;
        const bool any = item < (int64_t)p.tokens * n;
        t = any ? (int)(item / n) : 0;
        s = which;
        h0 = any ? (int)(item - (int64_t)t * n) * p.chunk : 0;
        h1 = any ? min(h0 + p.chunk, p.heads[s]) : h0;
    }
    // Cosine and sine of the lane's pairs.
    __device__ __forceinline__ void angles(const NormParams &p, const Turns &tu, float (&cs)[kPairs], float (&sn)[kPairs]) const
    {
        angles_at(turns ? token_position(p, t) : 0, tu, cs, sn);
    }
    __device__ __forceinline__ void angles_at(int pos, const Turns &tu, float (&cs)[kPairs], float (&sn)[kPairs]) const
    {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const uint64_t u = turns ? (uint64_t)(int64_t)pos * tu.f[(INTER ? f0 >> 1 : f0) + j] : 0;
            turn(static_cast<uint32_t>(u >> 32), cs[j], sn[j]);
        }
    }
};

template <int LANES> __device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A lane's sixteen features as eight pairs of neighbours.
struct Pairs {
    uint64_t v[kPairs];
    __device__ __forceinline__ void unpack(const uint4 &a, const uint4 &b)
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            v[i] = pair(bf16_lo(w[i]), bf16_hi(w[i]));
    }
    __device__ __forceinline__ float sum_of_products(const Pairs &o) const
    {
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            s = fma2(v[i], o.v[i], s);
        float a, b;
        unpair(s, a, b);
        return a + b;
    }
    __device__ __forceinline__ void scale(uint64_t f)
    {
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            v[i] = mul2(v[i], f);
    }
};

// What a feature is multiplied by: itself (own) and the other of its pair.
// rotated = own o x + other o partner(x), the partner being the pair at a
// distance, or the neighbour (INTER).
template <bool INTER> __device__ __forceinline__ uint64_t partner(const Pairs &x, int i)
{
    if (!INTER)
        return x.v[i ^ 4];
    float a, b;
    unpair(x.v[i], a, b);
    return pair(b, a);
}
template <bool INTER>
__device__ __forceinline__ void rotation(const float (&cs)[kPairs], const float (&sn)[kPairs], bool back, Pairs &own, Pairs &other)
{
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        // the first of a pair takes -sin of the second, the second +sin of the first; the transpose the other way
        const int m = INTER ? i : 2 * (i & 3), n = INTER ? i : m + 1;
        const float f = INTER ? -1.0f : (i < 4 ? -1.0f : 1.0f), g = INTER ? 1.0f : f, d = back ? -1.0f : 1.0f;
        own.v[i] = pair(cs[m], cs[n]);
        other.v[i] = pair(d * f * sn[m], d * g * sn[n]);
    }
}

__device__ __forceinline__ uint4 load8(const __nv_bfloat16 *p) { return __ldcs(reinterpret_cast<const uint4 *>(p)); }

__device__ __forceinline__ void store16(__nv_bfloat16 *row, int f0, int f1, const Pairs &x)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        float a, b;
        unpair(x.v[i], a, b);
        w[i] = pack_bf16(a, b);
    }
    __stcs(reinterpret_cast<uint4 *>(row + f0), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(reinterpret_cast<uint4 *>(row + f1), make_uint4(w[4], w[5], w[6], w[7]));
}

__device__ __forceinline__ Pairs load_weights(const float *w, int f0, int f1)
{
    Pairs x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 a = *reinterpret_cast<const float4 *>(w + (i < 2 ? f0 : f1) + 4 * (i & 1));
        x.v[2 * i] = pair(a.x, a.y);
        x.v[2 * i + 1] = pair(a.z, a.w);
    }
    return x;
}

// The weights' products with cosines and signed sines.
template <bool INTER>
__device__ __forceinline__ void weighted_rotation(const Pairs &w, const float (&cs)[kPairs], const float (&sn)[kPairs],
                                                  Pairs &own, Pairs &other)
{
    rotation<INTER>(cs, sn, false, own, other);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        own.v[i] = mul2(own.v[i], w.v[i]);
        other.v[i] = mul2(other.v[i], partner<INTER>(w, i));
    }
}

// A head's features, normed and turned; run by whole warps.
template <int D, bool INTER>
__device__ __forceinline__ Pairs normed(const uint4 &a, const uint4 &b, float eps, const Pairs &own, const Pairs &other)
{
    Pairs x, y;
    x.unpack(a, b);
    const float r = rsqrtf(group_sum<D / kFeat>(x.sum_of_products(x)) * (1.0f / D) + eps);
    x.scale(pair(r, r));
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
        y.v[i] = fma2(partner<INTER>(x, i), other.v[i], mul2(x.v[i], own.v[i]));
    return y;
}

// Heads per group of lanes: as few as keep the GPU's lanes busy when tokens
// are few, up to 8 when the angles' cost is worth sharing.
inline int head_chunk(const bdla_attn_dims &d, int heads)
{
    const int64_t vecs = (int64_t)d.B * d.T * heads;
    const int64_t want = vecs / ((int64_t)sm_count() * 256);
    const int c = want < 1 ? 1 : (want > 8 ? 8 : (int)want);
    return c > d.Hq ? d.Hq : c;
}

inline NormParams norm_params(const bdla_qk_norm_args &a, const bdla_attn_dims &d, int chunk)
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
    p.heads[0] = d.Hq;
    p.heads[1] = d.Hk;
    p.rotary = a.rotary;
    p.chunk = chunk;
    p.q_chunks = (d.Hq + p.chunk - 1) / p.chunk;
    p.n_chunks = p.q_chunks + (d.Hk + p.chunk - 1) / p.chunk;
    p.eps = a.eps;
    return p;
}

// The pairs' frequencies, formed once per thread and (base, rotary): 64 calls
// of pow are as long as the kernel of a decode step.
inline const Turns &turns_of(const bdla_qk_norm_args &a)
{
    thread_local Turns t{};
    thread_local double base = 0.0;   // no valid base
    thread_local int rotary = -1;
    if (base != a.base || rotary != a.rotary) {
        for (int i = 0; i < 64; ++i) {
            t.f[i] = 0;
            if (2 * i < a.rotary) {
                // turns per position, at most 1 / (2 pi); scaled by 2^64 without passing 2^63
                const double f = pow(a.base, -2.0 * i / a.rotary) / (2.0 * 3.14159265358979323846);
                t.f[i] = (uint64_t)ldexp(f, 64);
            }
        }
        base = a.base;
        rotary = a.rotary;
    }
    return t;
}

}  // namespace norm
}  // namespace bdla
