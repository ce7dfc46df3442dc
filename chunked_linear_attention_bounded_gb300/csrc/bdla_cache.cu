// The paged cache: writing rows into its pages, and attention of a sequence's
// newest tokens over it.
#include "bdla_attn_sm100.cuh"
#include "bdla_cache.cuh"

namespace bdla {

namespace {

using namespace cache;

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
// written once, 16 bytes a lane, four loads of each in flight.  Bound by HBM:
// the accepted of 5 x 4093 rows of 8 heads of 128, 20 us (5.0 TB/s).
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

// ---------------------------------------------------------------- attention over the cache
//
//   s = scale q . k over the visible positions,  o = (sum_t e^{s_t - m} v_t) / sum_t e^{s_t - m}
//
// A key head's cache is read once for all rows that use it: the new tokens of a
// sequence times the query heads of the group.  With up to 32 rows the pass is
// bound by HBM: their products cost nothing beside 512 bytes of keys and values
// a position, so they run as warp MMAs (m16n8k16, 16 or 32 rows) straight from
// the tiles that cp.async brings in.  Keys and values of 64 positions have two
// buffers each, and a buffer is filled again as soon as its own product is done:
// 64 KB a CTA, three CTAs an SM.  256 ragged sequences, 676 us (6.3 TB/s; three
// whole tiles a CTA, two CTAs an SM: 736); one of 262144 positions, with the
// join, 170 us (6.3 TB/s).  With 32 rows 12 to 16 bytes of registers are spilled.
// Pieces are counted from the table's width, so a table for 262144 positions over
// sequences of up to 8192 launches CTAs that find nothing to do: 856 us for 688 (both
// from cold).  A CTA's four warps split the rows first and the
// positions of the tile with what is left, and join through shared memory at the
// end.  Warp MMAs run at an
// eighth of the tensor cores' rate here: with 64 rows they took longer than the
// keys' way from HBM (244 rows a key head: 100 us for 96 MB), so more rows go to
// the tensor-memory kernel of bdla_cache_wide.cu.
//
// The long axis is split: every sequence into at most `ns` pieces of equal
// length, as the lengths on the device say.  A sequence of one piece is
// finished by its CTA; the others leave an fp32 sum per row and piece, which
// combine_kernel joins in the order of the pieces.
//
// Positions are looked up in the page table two tiles ahead of their load, by
// 64 threads into shared memory, so any page size works and no tile has to end
// with a page.  A position that nobody may see is not loaded: its rows are
// zeros.
constexpr int kKeys = 64;         // positions of a tile
constexpr int kCStages = 2;       // of keys, and of values
constexpr int kCThreads = 128;

template <int D> struct CachedSmem {
    alignas(128) unsigned char kv[kCStages][2][kKeys * D * 2];
    int row[4][kKeys];            // cache row of a tile's positions, -1: not seen
    uint32_t valid[4][2];
};

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
using attn::ex2;

template <int D, int WR>
__global__ void __launch_bounds__(kCThreads, D == 128 ? 3 : 4)
cached_kernel(const __grid_constant__ Call a, int row_blocks)
{
    constexpr int WK = 4 / WR;          // warps along the positions
    constexpr int KW = kKeys / WK;      // positions of a warp
    constexpr int MR = 16 * WR;         // rows of the CTA
    constexpr int kChunks = D / 8;      // 16-byte chunks of a row
    extern __shared__ __align__(128) unsigned char smem_raw[];
    CachedSmem<D> &sm = *reinterpret_cast<CachedSmem<D> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wr = warp % WR, wk = warp / WR;
    const bdla_cache &c = a.c;
    const int T = a.T, Hq = a.Hq, Hk = a.Hk, ns = a.pieces.ns;
    // heads of one position lie next to each other in the cache: keep them together in time
    int idx = blockIdx.x;
    const int rb = idx % row_blocks;
    idx /= row_blocks;
    const int kh = idx % Hk;
    idx /= Hk;
    const int piece = idx % ns, b = idx / ns;
    attn::next_may_start();
    const Cut cut = cut_of(c, b, T, a.pieces);
    if (piece >= cut.used)
        return;
    if (piece == 0 && kh == 0 && rb == 0 && tid == 0 && cut_is_short(c, cut, T))
        set_status(a.st, BDLA_ERR_DEVICE, (unsigned)b);
    const int G = Hq / Hk, R = T * G;
    const int k0 = piece * cut.size, k1 = min(cut.end, k0 + cut.size);
    const int nt = (k1 - k0 + kKeys - 1) / kKeys;
    const int32_t *table = c.pages + (int64_t)b * c.max_pages;
    const bool drafts = k1 > cut.len;   // the piece holds new tokens
    const uint64_t seen = drafts ? sees_any(a.tree, b, T, lane) : 0;

    // page table entry of position t (a tile's 64 positions, by the first 64 threads)
    auto lookup = [&](int t) { return t < k1 ? table[a.div.entry(t)] : -1; };
    auto place = [&](int n, int t, int pg) {
        bool live = t < k1 && (t < cut.len || ((seen >> (t - cut.len)) & 1));
        if (live && (pg < 0 || pg >= c.n_pages)) {
            set_status(a.st, BDLA_ERR_DEVICE, (unsigned)b);
            live = false;
        }
        sm.row[n & 3][tid] = live ? pg * c.page + a.div.offset(t) : -1;
        const uint32_t m = __ballot_sync(0xffffffffu, live);
        if (lane == 0)
            sm.valid[n & 3][tid >> 5] = m;
    };
    // tile n of the keys (v = 0) or of the values (v = 1), one cp.async group
    auto load = [&](int n, int v) {
        if (n < nt) {
            const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(sm.kv[n % kCStages][v]));
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(v ? c.v : c.k) + (int64_t)kh * D;
#pragma unroll
            for (int u = 0; u < kKeys * kChunks / kCThreads; ++u) {
                const int e = tid + u * kCThreads, r = e / kChunks, ch = e % kChunks;
                const int row = sm.row[n & 3][r];
                cp16(dst + (r * kChunks + (ch ^ (r & 7))) * 16, src + (int64_t)max(row, 0) * Hk * D + 8 * ch, row >= 0);
            }
        }
        cp_commit();
    };
    if (tid < kKeys)
        for (int n = 0; n < 3; ++n) {
            const int t = k0 + n * kKeys + tid;
            place(n, t, lookup(t));
        }
    __syncthreads();
    load(0, 0);
    load(0, 1);
    load(1, 0);
    load(1, 1);

    // query fragments: rows lane/4 and lane/4 + 8 of the warp's 16
    const int r0 = rb * MR + 16 * wr + (lane >> 2), r1 = r0 + 8;
    const int i0 = min(r0, R - 1) / G, i1 = min(r1, R - 1) / G;
    const __nv_bfloat16 *qa = a.q + (((int64_t)b * T + i0) * Hq + kh * G + min(r0, R - 1) % G) * D + 2 * (lane & 3);
    const __nv_bfloat16 *qb = a.q + (((int64_t)b * T + i1) * Hq + kh * G + min(r1, R - 1) % G) * D + 2 * (lane & 3);
    uint32_t fq[D / 16][4];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        fq[ks][0] = *reinterpret_cast<const uint32_t *>(qa + 16 * ks);
        fq[ks][1] = *reinterpret_cast<const uint32_t *>(qb + 16 * ks);
        fq[ks][2] = *reinterpret_cast<const uint32_t *>(qa + 16 * ks + 8);
        fq[ks][3] = *reinterpret_cast<const uint32_t *>(qb + 16 * ks + 8);
    }
    const uint64_t see0 = drafts ? sees(a.tree, b, T, i0) : 0, see1 = drafts ? sees(a.tree, b, T, i1) : 0;
    const float cs = a.scale * 1.4426950408889634f;
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
        acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;

    for (int n = 0; n < nt; ++n) {
        // in flight: V n, K n + 1, V n + 1 at most; one barrier says that K n is here and V n - 1 is done with
        if (n == 0)
            cp_wait<3>();
        else
            cp_wait<2>();
        __syncthreads();
        if (n > 0)
            load(n + 1, 1);
        const int t3 = k0 + (n + 3) * kKeys + tid;
        const int pg3 = tid < kKeys ? lookup(t3) : -1;
        const uint32_t sk = static_cast<uint32_t>(__cvta_generic_to_shared(sm.kv[n % kCStages][0]));
        const uint32_t sv = sk + kKeys * D * 2;
        float s[KW / 8][4];
#pragma unroll
        for (int i = 0; i < KW / 8; ++i)
            s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int nb = 0; nb < KW / 16; ++nb) {
                const int row = wk * KW + nb * 16 + (lane & 7) + ((lane >> 4) << 3), ch = 2 * ks + ((lane >> 3) & 1);
                uint32_t f[4];
                ldm4(f, sk + (row * kChunks + (ch ^ (row & 7))) * 16);
                mma16816(s[2 * nb], fq[ks], f[0], f[1]);
                mma16816(s[2 * nb + 1], fq[ks], f[2], f[3]);
            }
        // the same for V n and K n
        cp_wait<2>();
        __syncthreads();
        load(n + 2, 0);
        const uint64_t ok = (uint64_t)sm.valid[n & 3][0] | ((uint64_t)sm.valid[n & 3][1] << 32);
        const int t0 = k0 + n * kKeys;
        if (ok != ~0ull || t0 + kKeys > cut.len) {
#pragma unroll
            for (int i = 0; i < KW / 8; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int kk = wk * KW + 8 * i + 2 * (lane & 3) + u, j = t0 + kk - cut.len;
                    const bool live = (ok >> kk) & 1;
                    if (!(live && (j < 0 || ((see0 >> j) & 1))))
                        s[i][u] = -INFINITY;
                    if (!(live && (j < 0 || ((see1 >> j) & 1))))
                        s[i][2 + u] = -INFINITY;
                }
        }
        float x0 = s[0][0], x1 = s[0][2];
#pragma unroll
        for (int i = 0; i < KW / 8; ++i) {
            x0 = fmaxf(x0, fmaxf(s[i][0], s[i][1]));
            x1 = fmaxf(x1, fmaxf(s[i][2], s[i][3]));
        }
#pragma unroll
        for (int w = 1; w < 4; w <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, w));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, w));
        }
        if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
            const float a0 = n0 == m0 ? 1.0f : ex2((m0 - n0) * cs), a1 = n1 == m1 ? 1.0f : ex2((m1 - n1) * cs);
            m0 = n0;
            m1 = n1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                acc[i][0] *= a0;
                acc[i][1] *= a0;
                acc[i][2] *= a1;
                acc[i][3] *= a1;
            }
        }
        // rows that have seen nothing yet: every weight is e^(-inf)
        const float b0 = m0 == -INFINITY ? 0.0f : m0 * cs, b1 = m1 == -INFINITY ? 0.0f : m1 * cs;
#pragma unroll
        for (int nb = 0; nb < KW / 16; ++nb) {
            uint32_t fp[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float *x = s[2 * nb + u];
                const float p0 = ex2(fmaf(x[0], cs, -b0)), p1 = ex2(fmaf(x[1], cs, -b0));
                const float p2 = ex2(fmaf(x[2], cs, -b1)), p3 = ex2(fmaf(x[3], cs, -b1));
                l0 += p0 + p1;
                l1 += p2 + p3;
                fp[2 * u] = sm100::pack_bf16(p0, p1);
                fp[2 * u + 1] = sm100::pack_bf16(p2, p3);
            }
            const int row = wk * KW + nb * 16 + (lane & 15);
#pragma unroll
            for (int dn = 0; dn < D / 16; ++dn) {
                const int ch = 2 * dn + (lane >> 4);
                uint32_t f[4];
                ldm4t(f, sv + (row * kChunks + (ch ^ (row & 7))) * 16);
                mma16816(acc[2 * dn], fp, f[0], f[1]);
                mma16816(acc[2 * dn + 1], fp, f[2], f[3]);
            }
        }
        if (tid < kKeys)
            place(n + 3, t3, pg3);
    }
    cp_wait<0>();
    __syncthreads();   // the tiles' memory is free for the join

    float *jo = reinterpret_cast<float *>(sm.kv[0][0]);          // [WK][MR][D]
    float *jm = jo + WK * MR * D;                                // [WK][MR][2]
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, w);
        l1 += __shfl_xor_sync(0xffffffffu, l1, w);
    }
    {
        const int ra = 16 * wr + (lane >> 2);
        float *x = jo + (wk * MR + ra) * D + 2 * (lane & 3), *y = x + 8 * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            *reinterpret_cast<float2 *>(x + 8 * i) = make_float2(acc[i][0], acc[i][1]);
            *reinterpret_cast<float2 *>(y + 8 * i) = make_float2(acc[i][2], acc[i][3]);
        }
        if ((lane & 3) == 0) {
            *reinterpret_cast<float2 *>(jm + 2 * (wk * MR + ra)) = make_float2(m0, l0);
            *reinterpret_cast<float2 *>(jm + 2 * (wk * MR + ra + 8)) = make_float2(m1, l1);
        }
    }
    __syncthreads();
    for (int e = tid; e < MR * (D / 4); e += kCThreads) {
        const int r = e / (D / 4), d4 = 4 * (e % (D / 4)), row = rb * MR + r;
        if (row >= R)
            break;
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < WK; ++w)
            m = fmaxf(m, jm[2 * (w * MR + r)]);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            const float2 ml = *reinterpret_cast<const float2 *>(jm + 2 * (w * MR + r));
            const float f = ml.x == m ? 1.0f : ex2((ml.x - m) * cs);
            const float4 y = *reinterpret_cast<const float4 *>(jo + (w * MR + r) * D + d4);
            l = fmaf(ml.y, f, l);
            v.x = fmaf(y.x, f, v.x);
            v.y = fmaf(y.y, f, v.y);
            v.z = fmaf(y.z, f, v.z);
            v.w = fmaf(y.w, f, v.w);
        }
        if (cut.used > 1) {
            const int64_t at = (((int64_t)b * Hk + kh) * ns + piece) * R + row;
            *reinterpret_cast<float4 *>(a.part_o + at * D + d4) = v;
            if (d4 == 0)
                *reinterpret_cast<float2 *>(a.part_ml + 2 * at) = make_float2(m, l);
        } else {
            const int64_t at = ((int64_t)b * T + row / G) * Hq + kh * G + row % G;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            *reinterpret_cast<uint2 *>(a.o + at * D + d4) =
                make_uint2(sm100::pack_bf16(v.x * inv, v.y * inv), sm100::pack_bf16(v.z * inv, v.w * inv));
            if (d4 == 0)
                a.lse[at] = l == 0.0f ? -INFINITY : fmaf(m, a.scale, logf(l));
        }
    }
}

// Joins the pieces of a row, W warps a row: each sums every W-th piece, and the
// warps' sums are added in order.  W follows the most pieces of a sequence: one
// warp for up to 16, so that a CTA joins four rows, 16 beyond.
template <int D, int W>
__global__ void __launch_bounds__(W < 4 ? 128 : 32 * W)
combine_kernel(const __grid_constant__ Call a, int64_t rows)
{
    constexpr int E = D / 32, kRows = W < 4 ? 4 / W : 1;
    __shared__ float red_l[kRows][W], red_m[kRows][W];
    __shared__ __align__(16) float red_o[kRows][W][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp / W, w = warp % W;
    const int64_t at = (int64_t)blockIdx.x * kRows + mine;
    const int T = a.T, Hq = a.Hq, G = Hq / a.Hk;
    const bool any = at < rows;
    const int h = any ? (int)(at % Hq) : 0, i = any ? (int)(at / Hq % T) : 0, b = any ? (int)(at / Hq / T) : 0;
    Cut cut = cut_of(a.c, b, T, a.pieces);
    attn::wait_for_previous();
    const bool live = any && cut.used > 1;   // one piece: finished by its own CTA
    if (W > 1 && !live)
        return;   // the whole CTA
    if (!live)
        cut.used = 0;
    const int64_t first = ((int64_t)b * a.Hk + h / G) * a.pieces.ns;
    const int R = T * G, row = i * G + h % G;
    const float cs = a.scale * 1.4426950408889634f;
    float m = -INFINITY;
    for (int s = w * 32 + lane; s < cut.used; s += 32 * W)
        m = fmaxf(m, a.part_ml[2 * ((first + s) * R + row)]);
    for (int x = 16; x > 0; x >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    if (W > 1) {
        if (lane == 0)
            red_m[mine][w] = m;
        __syncthreads();
        for (int x = 0; x < W; ++x)
            m = fmaxf(m, red_m[mine][x]);
    }
    float l = 0.0f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        v[e] = 0.0f;
#pragma unroll 8
    for (int s = w; s < cut.used; s += W) {
        const int64_t p = (first + s) * R + row;
        const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + 2 * p);
        const float f = ml.x == m ? 1.0f : ex2((ml.x - m) * cs);
        l = fmaf(ml.y, f, l);
        const float *y = a.part_o + p * D + E * lane;
        if (E == 4) {
            const float4 z = *reinterpret_cast<const float4 *>(y);
            v[0] = fmaf(z.x, f, v[0]);
            v[1] = fmaf(z.y, f, v[1]);
            v[E - 2] = fmaf(z.z, f, v[E - 2]);
            v[E - 1] = fmaf(z.w, f, v[E - 1]);
        } else {
            const float2 z = *reinterpret_cast<const float2 *>(y);
            v[0] = fmaf(z.x, f, v[0]);
            v[1] = fmaf(z.y, f, v[1]);
        }
    }
    if (W > 1) {
        if (lane == 0)
            red_l[mine][w] = l;
#pragma unroll
        for (int e = 0; e < E; ++e)
            red_o[mine][w][E * lane + e] = v[e];
        __syncthreads();
        if (w != 0)
            return;
        for (int x = 1; x < W; ++x) {
            l += red_l[mine][x];
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[e] += red_o[mine][x][E * lane + e];
        }
    }
    if (!live)
        return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t *>(a.o + at * D + E * lane + e) = sm100::pack_bf16(v[e] * inv, v[e + 1] * inv);
    if (lane == 0)
        a.lse[at] = l == 0.0f ? -INFINITY : fmaf(m, a.scale, logf(l));
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

// Rows of a CTA: the smallest block that holds a key head's rows.
static int cached_rows(const bdla_attn_dims &d)
{
    const int R = d.T * (d.Hq / d.Hk);
    return R <= 16 ? 16 : R <= 32 ? 32 : kWideRows;
}

// Pieces of a sequence.  Few sequences: as many pieces as fill the SMs once, or
// two or three times where they stay over 1024 positions (one sequence of
// 262144 positions: 176 us in 3 rounds, 180 in 2.7), of at least 128.  Many:
// pieces of about 2048 positions, so that long and short sequences end together,
// and of at least 1024, so that a CTA's start-up (length, page table, first tile)
// stays small beside its keys.  The wide kernel holds an SM alone: as many pieces as fill the SMs a whole number
// of times, with at most 8192 positions (160 CTAs for 152 SMs cost a second
// round: 4 x 65536 positions, 186 us).  No more than 256 MB of partial sums, or
// a grid of 2^17 CTAs (more only where the sequences alone are more).
static Pieces cached_pieces(const bdla_attn_dims &d, int64_t max_keys)
{
    const int mr = cached_rows(d), R = d.T * (d.Hq / d.Hk);
    const bool wide = mr == kWideRows;
    const int64_t units = (int64_t)d.B * d.Hk * ((R + mr - 1) / mr), sms = sm_count();
    Pieces p;
    p.unit = wide ? 128 : kKeys;
    p.least = units >= 4 * sms ? 1024 : units >= sms ? 512 : units >= sms / 4 ? 256 : 128;
    int64_t ns;
    if (wide) {
        const int64_t rounds = (max_keys * units + 8192 * sms - 1) / (8192 * sms);
        ns = (rounds < 1 ? 1 : rounds) * sms / units;
    } else {
        const int64_t even = (max_keys + 2047) / 2048;
        const int64_t held = sms * (d.d == 128 ? 3 : 4);   // CTAs at a time
        int64_t rounds = 3;
        while (rounds > 1 && max_keys * units < 1024 * rounds * held)
            --rounds;
        ns = rounds * held / units;
        ns = ns > even ? ns : even;
    }
    const int64_t most[3] = {(max_keys + p.least - 1) / p.least,
                             ((int64_t)256 << 20) / ((int64_t)d.B * d.T * d.Hq * (d.d + 2) * 4), (1 << 17) / units};
    for (int i = 0; i < 3; ++i)
        ns = ns < most[i] ? ns : most[i];
    p.ns = ns < 1 ? 1 : (int)ns;
    return p;
}

int cached_splits(const bdla_attn_dims &d, int64_t max_keys) { return cached_pieces(d, max_keys).ns; }

size_t cached_partial_bytes(const bdla_attn_dims &d, int splits)
{
    return splits > 1 ? (size_t)splits * d.B * d.T * d.Hq * (d.d + 2) * 4 : 0;
}

template <int D, int WR>
static cudaError_t cached_go(const Call &a, const bdla_attn_dims &d, cudaStream_t stream)
{
    const int R = d.T * (d.Hq / d.Hk), row_blocks = (R + 16 * WR - 1) / (16 * WR);
    const int64_t grid = (int64_t)d.B * d.Hk * row_blocks * a.pieces.ns;
    const size_t smem = sizeof(CachedSmem<D>);
    const cudaError_t err = cudaFuncSetAttribute(cached_kernel<D, WR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess)
        return err;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    cached_kernel<D, WR><<<(unsigned)grid, kCThreads, smem, stream>>>(a, row_blocks);
    return cudaGetLastError();
}

template <int D> static cudaError_t combine_go(const Call &a, int64_t rows, cudaStream_t stream)
{
    return a.pieces.ns > 16 ? attn::launch_second(combine_kernel<D, 16>, (unsigned)rows, 512, 0, stream, a, rows)
                            : attn::launch_second(combine_kernel<D, 1>, (unsigned)((rows + 3) / 4), 128, 0, stream, a, rows);
}

cudaError_t launch_attn_cached(const __nv_bfloat16 *q, const bdla_cache &c, const uint64_t *tree, float scale,
                               __nv_bfloat16 *o, float *lse, const bdla_attn_dims &d, int64_t max_keys, void *partials,
                               DeviceStatus *st, cudaStream_t stream)
{
    const int mr = cached_rows(d);
    const int64_t rows = (int64_t)d.B * d.T * d.Hq;
    Call a;
    a.q = q;
    a.c = c;
    if ((int64_t)c.n_pages * c.page == 0)   // no rows: nothing is read, from an address that exists all the same
        a.c.k = a.c.v = const_cast<__nv_bfloat16 *>(q);
    a.tree = tree;
    a.scale = scale;
    a.o = o;
    a.lse = lse;
    a.T = d.T;
    a.Hq = d.Hq;
    a.Hk = d.Hk;
    a.pieces = cached_pieces(d, max_keys);
    a.div = PageDiv::of(c.page);
    a.st = st;
    a.part_o = static_cast<float *>(partials);
    a.part_ml = a.part_o + (size_t)a.pieces.ns * rows * d.d;
    KernelMark mark_(BDLA_KERNEL_ATTN_CACHED, stream);
    cudaError_t err;
    if (mr == kWideRows)
        err = launch_cached_wide(a, d, stream);
    else if (d.d == 64)
        err = mr == 16 ? cached_go<64, 1>(a, d, stream) : cached_go<64, 2>(a, d, stream);
    else
        err = mr == 16 ? cached_go<128, 1>(a, d, stream) : cached_go<128, 2>(a, d, stream);
    if (err != cudaSuccess || a.pieces.ns == 1)
        return err;
    return d.d == 64 ? combine_go<64>(a, rows, stream) : combine_go<128>(a, rows, stream);
}

}  // namespace bdla
