// What the kernels over the paged cache share: how a sequence's positions are
// cut into pieces, and what a new token sees.
#pragma once

#include "bdla_attn_internal.h"

namespace bdla {
namespace cache {

// The pieces of a call: at most `ns` a sequence, of at least `least` positions,
// a multiple of `unit`.
struct Pieces {
    int ns, least, unit;
};

// How one sequence is cut.
struct Cut {
    int len, end;     // committed positions; all positions inside the table
    int size, used;   // positions a piece, pieces
};
__device__ __forceinline__ Cut cut_of(const bdla_cache &c, int b, int T, const Pieces &p)
{
    Cut k;
    k.len = c.lens[b];
    const int64_t cap = (int64_t)c.max_pages * c.page, all = (int64_t)k.len + T;
    k.end = k.len < 0 ? 0 : (int)(all < cap ? all : cap);
    const int even = (int)(((int64_t)k.end + p.ns - 1) / p.ns);
    k.size = even < p.least ? p.least : (even + p.unit - 1) / p.unit * p.unit;
    k.used = k.end > 0 ? (k.end + k.size - 1) / k.size : 1;
    return k;
}

__device__ __forceinline__ bool cut_is_short(const bdla_cache &c, const Cut &k, int T)
{
    return k.len < 0 || (int64_t)k.len + T > (int64_t)c.max_pages * c.page;
}

// New tokens that token i sees (bit j: token j).
__device__ __forceinline__ uint64_t sees(const uint64_t *tree, int64_t b, int T, int i)
{
    const uint64_t m = tree != nullptr ? tree[b * T + i] : (i >= 63 ? ~0ull : (2ull << i) - 1);
    return T < 64 ? m & ((1ull << T) - 1) : m;
}

// New tokens that any of the sequence's sees (a whole warp).
__device__ __forceinline__ uint64_t sees_any(const uint64_t *tree, int64_t b, int T, int lane)
{
    uint64_t m = 0;
    for (int i = lane; i < T; i += 32)
        m |= sees(tree, b, T, i);
    for (int w = 16; w > 0; w >>= 1)
        m |= __shfl_xor_sync(0xffffffffu, m, w);
    return m;
}

// Division of positions (31 bits) by the page without a division: with
// s = ceil(log2 page) and mul = ceil(2^(31 + s) / page), which has 32 bits at
// most, mul page exceeds 2^(31 + s) by less than 2^s, so t mul / 2^(31 + s)
// exceeds t / page by less than 1 / page for t < 2^31.
struct PageDiv {
    uint32_t mul;
    int shift, page;
    static PageDiv of(int page)
    {
        int s = 0;
        while ((1 << s) < page)
            ++s;
        return {(uint32_t)((((uint64_t)1 << (31 + s)) + page - 1) / page), 31 + s, page};
    }
    __device__ __forceinline__ int entry(int t) const { return (int)(((uint64_t)(uint32_t)t * mul) >> shift); }
    __device__ __forceinline__ int offset(int t) const { return t - entry(t) * page; }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

struct Call {
    const __nv_bfloat16 *q;
    bdla_cache c;
    const uint64_t *tree;
    float scale;
    __nv_bfloat16 *o;
    float *lse;
    float *part_o, *part_ml;   // [B][Hk][ns][T * G] rows of D, and of (maximum, sum)
    int T, Hq, Hk;
    PageDiv div;
    Pieces pieces;
    DeviceStatus *st;
};

}  // namespace cache

// More than 32 rows a key head: tensor-memory MMAs (bdla_cache_wide.cu).
constexpr int kWideRows = 256;
cudaError_t launch_cached_wide(const cache::Call &call, const bdla_attn_dims &d, cudaStream_t stream);

}  // namespace bdla
