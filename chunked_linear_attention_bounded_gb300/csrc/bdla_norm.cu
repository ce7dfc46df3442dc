// RMS norm of queries and keys per head with the position rotation in the
// same pass, and its gradient.
//
//   n = x r,  r = 1 / sqrt(mean(x^2) + eps),  y = n o w,  pairs of y rotated
//   dy' = the rotation's transpose on dy,  h = dy' o w
//   dx = r (h - n mean(h o n)),   dw = sum over tokens and heads of dy' o n
//
// Both directions are one pass over the tensors (4 bytes an element forward,
// 6 backward) and bound by HBM.  A head of 64 or 128 features belongs to 4 or 8
// lanes, each with two groups of eight features that hold both halves of its
// pairs, so the rotation stays in the lane, the mean is a 2- or 3-step shuffle
// and the accesses of the lanes together cover whole lines.  Such a group of
// lanes keeps one token and walks a chunk of its query or key heads: the eight
// angles of a lane belong to the token, and the products of weights and sines
// are formed once per chunk; several heads' loads are in flight at a time.
// Measured for 65536 tokens, 32 + 8 heads of 128: forward 203 us (6.6 TB/s),
// gradient 305 us (6.6 TB/s; loads through registers, two heads at a time, 364),
// from fp32 gradients, 8 bytes an element, 393 us (6.8 TB/s).  Registers end at
// the 128 of two CTAs an SM: the forward and two forms of the gradient spill 12 to
// 16 bytes.
#include "bdla_cache.cuh"
#include "bdla_norm.cuh"

namespace bdla {

namespace {

using namespace norm;

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2)
qk_norm_kernel(const __grid_constant__ NormParams p, const __grid_constant__ Turns tu, __nv_bfloat16 *__restrict__ qn,
               __nv_bfloat16 *__restrict__ kn)
{
    using G = Group<D, INTER>;
    G g(p);
    g.take(p, (int64_t)blockIdx.x * G::kPerBlock + threadIdx.x / G::kLanes);
    const __nv_bfloat16 *src = p.x[g.s] + g.t * p.token[g.s];
    const int64_t step = p.head[g.s];
    __nv_bfloat16 *dst = (g.s ? kn : qn) + (int64_t)g.t * p.heads[g.s] * D;
    Pairs own, other;
    {
        float cs[kPairs], sn[kPairs];
        const Pairs w = load_weights(p.w[g.s], g.f0, g.f1);
        g.angles(p, tu, cs, sn);
        weighted_rotation<INTER>(w, cs, sn, own, other);
    }
    for (int b = 0; b < p.chunk; b += kBatch) {
        uint4 in[kBatch][2];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = g.h0 + b + u;
            in[u][0] = in[u][1] = make_uint4(0, 0, 0, 0);
            if (h < g.h1) {
                in[u][0] = load8(src + h * step + g.f0);
                in[u][1] = load8(src + h * step + g.f1);
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = g.h0 + b + u;
            const Pairs y = normed<D, INTER>(in[u][0], in[u][1], p.eps, own, other);
            if (h < g.h1)
                store16(dst + h * D, g.f0, g.f1, y);
        }
    }
}

// The gradient's ring of heads in shared memory: rows of x and of the incoming
// gradient, kB heads a turn, 16 bytes a piece.  A group's lanes fetch a row's
// pieces in order (a sector that two instructions touch would come twice) and
// read those of their features, so that a warp's barrier is all that stands
// between.  Loads of the next kTurns - 1 turns are in flight while one is worked
// on; two CTAs' rings fit into an SM.
template <int D, bool GF32> struct Ring {
    static constexpr int kLanes = D / kFeat;
    static constexpr int kB = 2, kTurns = GF32 ? 2 : 3, kGrad = GF32 ? 4 : 2, kPieces = 2 + kGrad;
    static constexpr int kBytes = kTurns * kB * kPieces * kThreads * 16;
    uint4 *own;   // this thread's slots
    int x[2], g[kGrad];   // the lane's pieces, from its own slots
    __device__ __forceinline__ Ring(unsigned char *smem, int f0, int f1)
        : own(reinterpret_cast<uint4 *>(smem) + threadIdx.x)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            x[i] = place((i ? f1 : f0) >> 3);
#pragma unroll
        for (int i = 0; i < kGrad; ++i)
            g[i] = 2 * kThreads + (GF32 ? place(((i < 2 ? f0 : f1) >> 2) + (i & 1)) : x[i & 1]);
    }
    // Piece n of the row: lane n of the group fetched it, in its n / kLanes-th turn.
    __device__ __forceinline__ static int place(int n)
    {
        return n / kLanes * kThreads + n % kLanes - (int)threadIdx.x % kLanes;
    }
    __device__ __forceinline__ uint4 *slot(int turn, int u) const { return own + (turn * kB + u) * kPieces * kThreads; }
    // A head that is not there (live false) is not read, and is zero.
    __device__ __forceinline__ void fetch(int turn, int u, const __nv_bfloat16 *row, const void *grad, int64_t off,
                                          bool live) const
    {
        const uint32_t dst = (uint32_t)__cvta_generic_to_shared(slot(turn, u));
        const int lane = threadIdx.x % kLanes;
        const char *gr = static_cast<const char *>(grad) + off * (GF32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            cache::cp16(dst + i * kThreads * 16, row + (i * kLanes + lane) * 8, live);
#pragma unroll
        for (int i = 0; i < kGrad; ++i)
            cache::cp16(dst + (2 + i) * kThreads * 16, gr + (i * kLanes + lane) * 16, live);
    }
    __device__ __forceinline__ void get(int turn, int u, Pairs &v, Pairs &grad) const
    {
        const uint4 *p = slot(turn, u);
        v.unpack(p[x[0]], p[x[1]]);
        if constexpr (GF32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = *reinterpret_cast<const float4 *>(p + g[i]);
                grad.v[2 * i] = pair(f.x, f.y);
                grad.v[2 * i + 1] = pair(f.z, f.w);
            }
        } else {
            grad.unpack(p[g[0]], p[g[1]]);
        }
    }
};

// The first q_blocks CTAs take the query heads, the others the key heads, so
// that a thread sums one weight gradient; CTA i leaves its sums in part[i].
template <int D, bool INTER, bool GF32>
__global__ void __launch_bounds__(kThreads, 2)
qk_norm_bwd_kernel(const __grid_constant__ NormParams p, const __grid_constant__ Turns tu, int q_blocks,
                   const void *__restrict__ dqn, const void *__restrict__ dkn, __nv_bfloat16 *__restrict__ dq,
                   __nv_bfloat16 *__restrict__ dk, float *__restrict__ part)
{
    using G = Group<D, INTER>;
    using R = Ring<D, GF32>;
    constexpr int kB = R::kB;
    extern __shared__ __align__(16) unsigned char ring_smem[];
    __shared__ __align__(8) float red[G::kPerBlock][D];
    G g(p), ahead(p);
    const R ring(ring_smem, g.f0, g.f1);
    attn::next_may_start();
    const int gi = threadIdx.x / G::kLanes;
    const int s = (int)blockIdx.x >= q_blocks;
    const int block = (int)blockIdx.x - (s ? q_blocks : 0), blocks = s ? (int)gridDim.x - q_blocks : q_blocks;
    const Pairs w = load_weights(p.w[s], g.f0, g.f1);
    Pairs dw;
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
        dw.v[i] = 0;
    const int64_t items = (int64_t)p.tokens * (s ? p.n_chunks - p.q_chunks : p.q_chunks);
    const int64_t stride = (int64_t)blocks * G::kPerBlock, step = p.head[s];
    const void *grad = s ? dkn : dqn;

    // the loads' own way through the block's heads
    int64_t next = (int64_t)block * G::kPerBlock;
    int done = 0, into = 0;   // heads of the item at `next` that are fetched; turn to fetch into
    ahead.take_of(p, s, next + gi);
    auto fetch = [&] {
        if (next < items) {
            const __nv_bfloat16 *src = p.x[s] + ahead.t * p.token[s];
            const int64_t row = (int64_t)ahead.t * p.heads[s] * D;
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                const int h = ahead.h0 + done + u;
                ring.fetch(into, u, src + h * step, grad, row + (int64_t)h * D, h < ahead.h1);
            }
            if ((done += kB) >= p.chunk) {
                done = 0;
                next += stride;
                ahead.take_of(p, s, next + gi);
            }
        }
        into = into + 1 < R::kTurns ? into + 1 : 0;
        cache::cp_commit();
    };
#pragma unroll
    for (int i = 1; i < R::kTurns; ++i)
        fetch();

    int turn = 0;
    // the block's groups stay together, so that whole warps reach the shuffles
    for (int64_t base = (int64_t)block * G::kPerBlock; base < items; base += stride) {
        g.take_of(p, s, base + gi);
        __nv_bfloat16 *dst = (s ? dk : dq) + (int64_t)g.t * p.heads[s] * D;
        Pairs own, other;
        {
            float cs[kPairs], sn[kPairs];
            g.angles(p, tu, cs, sn);
            rotation<INTER>(cs, sn, true, own, other);
        }
        for (int h = g.h0; h < g.h0 + p.chunk; h += kB) {
            __syncwarp();
            fetch();   // over the turn before this one, whose values are used up
            cache::cp_wait<R::kTurns - 1>();
            __syncwarp();
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                Pairs x, y, z;
                ring.get(turn, u, x, z);
                const float sum = group_sum<G::kLanes>(x.sum_of_products(x));
                const float r = h + u < g.h1 ? rsqrtf(sum * (1.0f / D) + p.eps) : 0.0f;   // no head: 0, not 0 / 0
                x.scale(pair(r, r));   // n
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    y.v[i] = fma2(partner<INTER>(z, i), other.v[i], mul2(z.v[i], own.v[i]));
                    dw.v[i] = fma2(y.v[i], x.v[i], dw.v[i]);
                    y.v[i] = mul2(y.v[i], w.v[i]);   // h
                }
                const float m = group_sum<G::kLanes>(y.sum_of_products(x)) * (1.0f / D);
#pragma unroll
                for (int i = 0; i < kPairs; ++i)
                    y.v[i] = fma2(x.v[i], pair(-m, -m), y.v[i]);
                y.scale(pair(r, r));
                if (h + u < g.h1)
                    store16(dst + (h + u) * D, g.f0, g.f1, y);
            }
            turn = turn + 1 < R::kTurns ? turn + 1 : 0;
        }
    }
    cache::cp_wait<0>();
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        float a, b;
        unpair(dw.v[i], a, b);
        *reinterpret_cast<float2 *>(&red[gi][i < 4 ? g.f0 + 2 * i : g.f1 + 2 * i - 8]) = make_float2(a, b);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < G::kPerBlock; ++i)
            v += red[i][c];
        part[(size_t)blockIdx.x * D + c] = v;
    }
}

// Sums the CTAs' partial weight gradients, 8 columns a CTA, each of 128
// threads a column every 128th partial, then the threads in order: the same
// sizes give the same bits.
__global__ void __launch_bounds__(1024)
norm_dw_kernel(const float *part, int q_blocks, int blocks, int D, float *__restrict__ dwq,
               float *__restrict__ dwk)
{
    __shared__ float red[128][9];
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3, per = D / 8;
    const int s = (int)blockIdx.x >= per, c = ((int)blockIdx.x - s * per) * 8 + x;
    const int first = s ? q_blocks : 0, last = s ? blocks : q_blocks;
    float v = 0.0f;
    attn::wait_for_previous();
#pragma unroll 4
    for (int i = first + y; i < last; i += 128)
        v += part[(size_t)i * D + c];
    red[y][x] = v;
    __syncthreads();
    for (int w = 64; w > 0; w >>= 1) {
        if (y < w)
            red[y][x] += red[y + w][x];
        __syncthreads();
    }
    if (y == 0)
        (s ? dwk : dwq)[c] = red[0][x];
}

}  // namespace

cudaError_t launch_qk_norm(const bdla_qk_norm_args &a, __nv_bfloat16 *qn, __nv_bfloat16 *kn,
                           const bdla_attn_dims &d, cudaStream_t stream)
{
    if (d.T == 0)
        return cudaSuccess;
    const NormParams p = norm_params(a, d, head_chunk(d, d.Hq + d.Hk));
    const Turns &tu = turns_of(a);
    const int64_t items = (int64_t)p.tokens * p.n_chunks;
    const int per = kThreads / (d.d / kFeat);
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

// CTAs for the query and for the key heads, in proportion to their work.
static int norm_q_blocks(const bdla_attn_dims &d, int *total)
{
    const int chunk = head_chunk(d, d.Hq + d.Hk), per = kThreads / (d.d / kFeat);
    // the last CTAs' unequal ends: 65536 tokens 346 us with 4 CTAs an SM, 311 with 8, 301 with 24
    const int64_t most = (int64_t)sm_count() * 24, tokens = (int64_t)d.B * d.T;
    int64_t n[2];
    for (int s = 0; s < 2; ++s) {
        const int heads = s ? d.Hk : d.Hq;
        const int64_t items = tokens * ((heads + chunk - 1) / chunk), need = (items + per - 1) / per;
        int64_t share = most * d.Hk / (d.Hq + d.Hk);
        share = share < 1 ? 1 : share;
        share = s ? share : most - share;
        n[s] = need < share ? need : share;
    }
    *total = (int)(n[0] + n[1]);
    return (int)n[0];
}

int norm_bwd_blocks(const bdla_attn_dims &d)
{
    int total;
    norm_q_blocks(d, &total);
    return total;
}

cudaError_t launch_qk_norm_bwd(const bdla_qk_norm_args &a, const void *dqn, const void *dkn, int g_f32,
                               __nv_bfloat16 *dq, __nv_bfloat16 *dk, float *dwq, float *dwk, float *part,
                               const bdla_attn_dims &d, cudaStream_t stream)
{
    int blocks;
    const int q_blocks = norm_q_blocks(d, &blocks);
    if (blocks > 0) {
        const NormParams p = norm_params(a, d, head_chunk(d, d.Hq + d.Hk));
        const Turns &tu = turns_of(a);
        cudaError_t err = cudaSuccess;
#define BDLA_NORM_GO(D_, I_, G_)                                                                                    \
    do {                                                                                                            \
        err = cudaFuncSetAttribute(qk_norm_bwd_kernel<D_, I_, G_>, cudaFuncAttributeMaxDynamicSharedMemorySize,     \
                                   Ring<D_, G_>::kBytes);                                                               \
        if (err == cudaSuccess)                                                                                     \
            qk_norm_bwd_kernel<D_, I_, G_><<<blocks, kThreads, Ring<D_, G_>::kBytes, stream>>>(p, tu, q_blocks, dqn,    \
                                                                                           dkn, dq, dk, part);      \
    } while (0)
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
        if (err == cudaSuccess)
            err = cudaGetLastError();
        if (err != cudaSuccess)
            return err;
    }
    return attn::launch_second(norm_dw_kernel, 2 * d.d / 8, 1024, 0, stream, part, q_blocks, blocks, d.d, dwq, dwk);
}

}  // namespace bdla
