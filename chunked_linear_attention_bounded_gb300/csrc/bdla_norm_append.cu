// New tokens into a paged cache in one launch: queries and keys normed and
// rotated as in bdla_norm.cu, keys and values written to their rows of the
// cache.  Saves the keys' way through memory (4 bytes an element) and a launch
// against bdla_qk_norm followed by bdla_cache_append, whose bits it gives.
//
// A group of lanes takes one token and a chunk of its query, key or value heads,
// and a warp the same chunk of four or eight tokens, so that values are copied by
// whole warps without the norm's arithmetic.  The first heads are asked for before
// the token's place is looked up (length, page), so that the two chains overlap.
//
// Bound by HBM: 65536 packed tokens of 8 sequences, 32 + 8 + 8 heads of 128, in 250
// us (6.4 TB/s; 304 where a warp's groups took different kinds of heads).  Few
// tokens are bound by the chain of length, page and first line, and take as few
// heads a warp as put all warps on the SMs at once: 256 single tokens 4.7 to 5.1 us
// (9.4 with eight heads a warp), one token 3.9 to 4.5 (5.2), 91 x 61 chosen rows
// 13.0 (15.6).  The 128 registers of two CTAs an SM hold the eight heads in flight,
// angles and weights but for 24 to 40 bytes, which cost 36 to 220 bytes of reloads a
// thread and nothing that HBM's rate shows.
#include "bdla_cache.cuh"
#include "bdla_norm.cuh"

namespace bdla {

namespace {

using namespace norm;

struct AppendParams {
    const __nv_bfloat16 *v;
    int64_t v_token, v_head;   // element strides
    bdla_cache c;
    const int32_t *rows, *counts;
    int kv_chunks;             // chunks of the key heads, and of the value heads
    DeviceStatus *st;
};

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2)
norm_append_kernel(const __grid_constant__ NormParams p, const __grid_constant__ Turns tu,
                   const __grid_constant__ AppendParams a, __nv_bfloat16 *__restrict__ qn)
{
    using G = Group<D, INTER>;
    if (blockIdx.x == 0 && p.cu != nullptr)
        attn::check_offsets(p.cu, p.n_docs, p.tokens, a.st);
    G g(p);
    // a warp takes one chunk (of queries, keys or values) of kTokens tokens
    constexpr int kTokens = 32 / G::kLanes;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), block = unit / p.n_chunks;
    int c = (int)(unit - block * p.n_chunks);
    const int64_t token = block * kTokens + (threadIdx.x & 31) / G::kLanes;
    const bool any = token < p.tokens;
    if (block * kTokens >= p.tokens)
        return;   // the whole warp
    const int t = any ? (int)token : 0;
    const int kind = c < p.q_chunks ? 0 : c < p.q_chunks + a.kv_chunks ? 1 : 2;   // queries, keys, values
    c -= kind == 0 ? 0 : kind == 1 ? p.q_chunks : p.q_chunks + a.kv_chunks;
    const int s = kind > 0, h0 = c * p.chunk;
    int h1 = any ? min(h0 + p.chunk, p.heads[s]) : h0;

    // the token's sequence, and its number among the sequence's new ones
    int b, j;
    bool good = true;
    if (p.cu != nullptr) {
        b = document_of(p, t);
        j = t - p.cu[b];
        good = j >= 0 && t < p.cu[b + 1];
    } else {
        b = t / p.T;
        j = t - b * p.T;
    }
    // place j of the sequence is filled from this token
    int src = t;
    if (s && a.rows != nullptr) {
        const int r = a.rows[t];
        good &= r >= 0 && r < p.T;
        src = b * p.T + (good ? r : 0);
    }
    const __nv_bfloat16 *x = kind == 2 ? a.v + src * a.v_token : p.x[s] + src * p.token[s];
    const int64_t step = kind == 2 ? a.v_head : p.head[s];
    uint4 in[kBatch][2];
    const auto fetch = [&](int first) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = first + u;
            in[u][0] = in[u][1] = make_uint4(0, 0, 0, 0);
            if (h < h1) {
                in[u][0] = load8(x + h * step + g.f0);
                in[u][1] = load8(x + h * step + g.f1);
            }
        }
    };
    fetch(h0);

    const int len = a.c.lens[b];
    __nv_bfloat16 *dst = qn + (int64_t)t * p.heads[0] * D;
    if (s) {
        int n = p.T;
        if (a.counts != nullptr) {
            n = a.counts[b];
            if (n < 0 || n > p.T) {
                if (any)
                    set_status(a.st, BDLA_ERR_DEVICE, (unsigned)b);
                n = n < 0 ? 0 : p.T;
            }
        }
        const int64_t at = (int64_t)len + j;
        const int64_t row = good && len >= 0 && at <= INT32_MAX ? cache::cache_row(a.c, a.c.pages + (int64_t)b * a.c.max_pages, (int)at) : -1;
        if (j >= n) {
            h1 = h0;
        } else if (row < 0) {
            if (any)
                set_status(a.st, BDLA_ERR_DEVICE, (unsigned)b);
            h1 = h0;
        }
        dst = static_cast<__nv_bfloat16 *>(kind == 1 ? a.c.k : a.c.v) + (row < 0 ? 0 : row) * p.heads[1] * D;
    }
    if (kind == 2) {   // copied
        for (int first = h0; first < h0 + p.chunk; first += kBatch) {
            if (first > h0)
                fetch(first);
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (first + u < h1) {
                    __stcs(reinterpret_cast<uint4 *>(dst + (first + u) * D + g.f0), in[u][0]);
                    __stcs(reinterpret_cast<uint4 *>(dst + (first + u) * D + g.f1), in[u][1]);
                }
        }
        return;
    }
    Pairs own, other;
    {
        float cs[kPairs], sn[kPairs];
        const Pairs w = load_weights(p.w[s], g.f0, g.f1);
        const int pos = p.positions != nullptr ? p.positions[src] : (int)((uint32_t)len + (uint32_t)j);
        g.angles_at(g.turns ? pos : 0, tu, cs, sn);
        weighted_rotation<INTER>(w, cs, sn, own, other);
    }
    for (int first = h0; first < h0 + p.chunk; first += kBatch) {
        if (first > h0)
            fetch(first);
        const auto one = [&](int u) {
            const Pairs y = normed<D, INTER>(in[u][0], in[u][1], p.eps, own, other);
            if (first + u < h1)
                store16(dst + (first + u) * D, g.f0, g.f1, y);
        };
        if (first + kBatch <= h0 + p.chunk) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                one(u);
        } else {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (first + u < h0 + p.chunk)   // (all lanes: a few tokens' few heads skip the arithmetic of the others)
                    one(u);
        }
    }
}

}  // namespace

cudaError_t launch_qk_norm_append(const bdla_qk_norm_args &a, const __nv_bfloat16 *v, int64_t v_token, int64_t v_head,
                                  const bdla_cache &c, const int32_t *rows, const int32_t *counts, __nv_bfloat16 *qn,
                                  const bdla_attn_dims &d, DeviceStatus *st, cudaStream_t stream)
{
    const int q_heads = a.q != nullptr ? d.Hq : 0;
    // heads of a warp: as few as put all warps onto the SMs at once (16 each), up to 8, which share the angles' cost
    const int per = 32 / (d.d / kFeat);   // tokens of a warp
    const int64_t blocks = ((int64_t)d.B * d.T + per - 1) / per, held = (int64_t)sm_count() * (kThreads / 32) * 2;
    const int64_t even = (blocks * (q_heads + 2 * d.Hk) + held - 1) / held, widest = q_heads > d.Hk ? q_heads : d.Hk;
    const int64_t chunk = even < 8 ? even : 8;
    NormParams p = norm_params(a, d, (int)(chunk < widest ? chunk : widest));
    AppendParams ap = {v, v_token, v_head, c, rows, counts, (d.Hk + p.chunk - 1) / p.chunk, st};
    p.heads[0] = q_heads;
    p.q_chunks = (q_heads + p.chunk - 1) / p.chunk;
    p.n_chunks = p.q_chunks + 2 * ap.kv_chunks;
    const Turns &tu = turns_of(a);
    const int64_t warps = blocks * p.n_chunks, grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    auto *kern = d.d == 64 ? (a.interleaved ? norm_append_kernel<64, true> : norm_append_kernel<64, false>)
                           : (a.interleaved ? norm_append_kernel<128, true> : norm_append_kernel<128, false>);
    kern<<<(unsigned)grid, kThreads, 0, stream>>>(p, tu, ap, qn);
    return cudaGetLastError();
}

}  // namespace bdla
