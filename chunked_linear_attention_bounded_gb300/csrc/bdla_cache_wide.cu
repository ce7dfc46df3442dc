// Attention over the paged cache for many rows a key head (a tree of drafts
// times the query heads of a group), on the sm_100-family tensor cores.
//
// The mathematics and the pieces are those of bdla_cache.cu; the pipeline is
// that of the whole-prompt forward (bdla_attn_fwd.cu): up to 256 rows as two
// tiles of 128 that take turns between the tensor cores and their softmax
// warps, scores and outputs in tensor memory, weights read from there by the
// P V product, a reference maximum that moves only when a score passes it by
// 2^8.  What differs is where the keys come from: positions are looked up in
// the page table, so three warps fetch tiles of 128 positions row by row with
// cp.async into the swizzled layout that the MMAs read, two or three tiles
// ahead.  256 rows need 1024 tensor cycles for 64 KB of keys and values, which
// take 2800 cycles of an SM's share of HBM: the pass is bound by the latter.
//
// Warp 0 issues the MMAs, warps 1-3 fetch, warps 4-7 and 8-11 are the softmax
// of the two tiles, one thread a row.
#include "bdla_attn_sm100.cuh"
#include "bdla_cache.cuh"

namespace bdla {

namespace {

using namespace sm100;
using namespace attn;
using namespace cache;

constexpr int kFetch = 96;                  // fetching threads
constexpr int kThreads = 32 + kFetch + 256;
constexpr int kAhead = 3;                   // tiles in flight per thread

template <int D> struct WideSmem {
    static constexpr int kPanels = D / 64;
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int kStages = D == 128 ? 5 : 8;
    // A tile's slot is written again once the fetching warps are kStages tiles further: by then its softmax is done.
    static constexpr int kSlots = D == 128 ? 4 : 8;
    alignas(1024) unsigned char q[2][kTile];
    alignas(1024) unsigned char ring[kStages][kTile];   // K_0 V_0 K_1 V_1 ...
    int row[kSlots][BT];     // cache row of a tile's positions, -1: not seen
    uint32_t valid[kSlots][4];
    uint64_t q_ready, full[kStages], empty[kStages], s_full[2], o_done[2], drain;
    uint64_t p_ready[2][2];   // weights of the first and of the last 64 positions of a tile
    uint64_t wait_ns;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(WideSmem<128>) <= kMaxSmem && sizeof(WideSmem<64>) <= kMaxSmem, "shared memory of a CTA");

__device__ __forceinline__ void fetch_sync() { asm volatile("bar.sync 1, 96;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cached_wide_kernel(const __grid_constant__ Call a, int row_blocks, uint64_t wait_ns)
{
    using Smem = WideSmem<D>;
    constexpr int NS = Smem::kStages, SL = Smem::kSlots, kChunks = D / 8;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bdla_cache &c = a.c;
    const int T = a.T, Hq = a.Hq, Hk = a.Hk, ns = a.pieces.ns, G = Hq / Hk, R = T * G;
    int idx = blockIdx.x;
    const int rb = idx % row_blocks;
    idx /= row_blocks;
    const int kh = idx % Hk;
    idx /= Hk;
    const int piece = idx % ns, b = idx / ns;
    const Cut cut = cut_of(c, b, T, a.pieces);
    if (piece >= cut.used)
        return;
    if (piece == 0 && kh == 0 && rb == 0 && tid == 0 && cut_is_short(c, cut, T))
        set_status(a.st, BDLA_ERR_DEVICE, (unsigned)b);
    if ((smem_u32(smem_raw) & 1023u) != 0u) {
        if (tid == 0)
            set_status(a.st, BDLA_ERR_DEVICE, 0xA11u);
        return;
    }
    const int k0 = piece * cut.size, k1 = min(cut.end, k0 + cut.size);
    const int nt = (k1 - k0 + BT - 1) / BT;
    const int tiles = R - rb * kWideRows > BT ? 2 : 1;   // row tiles of this CTA

    if (warp == 0) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    if (tid == 32) {
        mbar_init(&sm.q_ready, 256);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sm.full[s], kFetch);
            mbar_init(&sm.empty[s], 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&sm.s_full[w], 1);
            mbar_init(&sm.p_ready[w][0], BT);
            mbar_init(&sm.p_ready[w][1], BT);
            mbar_init(&sm.o_done[w], 1);
        }
        mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
        sm.wait_ns = wait_ns;
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    volatile int *abort_flag = &sm.abort_flag;

    if (warp == 0) {
        // ---------------------------------------------------------------- MMA issuer
        const uint64_t q[2] = {rows_desc(smem_u32(sm.q[0])), rows_desc(smem_u32(sm.q[1]))};
        bool ok = warp_wait(&sm.q_ready, 0, &sm.wait_ns, abort_flag);
        auto issue_qk = [&](int w, int j) {
            const int it = 2 * j;
            if (!warp_wait(&sm.full[it % NS], (it / NS) & 1, &sm.wait_ns, abort_flag))
                return false;
            tc_fence_after();
            const uint64_t k = rows_desc(smem_u32(sm.ring[it % NS]));
            if (elect_one()) {
                mma_rows<D>(tmem + BT * w, q[w], k);
                umma_commit(&sm.s_full[w]);
                if (w == tiles - 1)   // the last reader of this key tile
                    umma_commit(&sm.empty[it % NS]);
            }
            __syncwarp();
            return true;
        };
        for (int w = 0; ok && nt > 0 && w < tiles; ++w)
            ok = issue_qk(w, 0);
        for (int j = 0; ok && j < nt; ++j) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (!ok || w >= tiles)
                    continue;
                const int it = 2 * j + 1;
                ok = warp_wait(&sm.full[it % NS], (it / NS) & 1, &sm.wait_ns, abort_flag) &&
                     warp_wait(&sm.p_ready[w][0], (uint32_t)(j & 1), &sm.wait_ns, abort_flag);
                if (!ok)
                    continue;
                tc_fence_after();
                const uint64_t v = sum_desc(smem_u32(sm.ring[it % NS]));
                const uint32_t acc = tmem + 2 * BT + BT * w, wt = tmem + BT * w;
                if (elect_one())
                    mma_sum<D, 32, 0, BT / 32>(acc, wt, v, j > 0);
                __syncwarp();
                ok = warp_wait(&sm.p_ready[w][1], (uint32_t)(j & 1), &sm.wait_ns, abort_flag);
                if (!ok)
                    continue;
                tc_fence_after();
                if (elect_one()) {
                    mma_sum<D, 32, BT / 32, BT / 16>(acc, wt, v, true);
                    if (w == tiles - 1)
                        umma_commit(&sm.empty[it % NS]);
                    if (j + 1 == nt)
                        umma_commit(&sm.o_done[w]);
                }
                __syncwarp();
                if (j + 1 < nt)
                    ok = issue_qk(w, j + 1);
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(a.st, BDLA_ERR_TIMEOUT, 0x30u);
        }
        // every MMA issued above has completed before TMEM is released
        if (elect_one())
            umma_commit(&sm.drain);
        __syncwarp();
        mbar_wait(&sm.drain, 0, kDrainNs);
    } else if (warp < 4) {
        // ---------------------------------------------------------------- fetching
        const int ft = tid - 32, fw = warp - 1;
        const int32_t *table = c.pages + (int64_t)b * c.max_pages;
        const uint64_t seen = k1 > cut.len ? sees_any(a.tree, b, T, lane) : 0;
        // the page of this lane's positions of a tile (groups of 32: fw and, for the first warp, 3)
        auto lookup = [&](int j, int g) {
            const int t = k0 + j * BT + 32 * g + lane;
            return t < k1 ? table[t / c.page] : -1;
        };
        auto place = [&](int j, int g, int pg) {
            const int t = k0 + j * BT + 32 * g + lane;
            bool live = t < k1 && (t < cut.len || ((seen >> (t - cut.len)) & 1));
            if (live && (pg < 0 || pg >= c.n_pages)) {
                set_status(a.st, BDLA_ERR_DEVICE, (unsigned)b);
                live = false;
            }
            sm.row[j % SL][32 * g + lane] = live ? pg * c.page + t % c.page : -1;
            const uint32_t m = __ballot_sync(0xffffffffu, live);
            if (lane == 0)
                sm.valid[j % SL][g] = m;
        };
        auto arrive = [&](int it) {
            fence_proxy_async_smem();
            mbar_arrive(&sm.full[it % NS]);
        };
        // this thread's 16-byte chunk of every kRowStep-th row
        constexpr int kRowStep = kFetch / kChunks, kRows = (BT + kRowStep - 1) / kRowStep;
        const int ch = ft % kChunks, r0 = ft / kChunks;
        int pg0 = nt > 0 ? lookup(0, fw) : -1, pg3 = nt > 0 && fw == 0 ? lookup(0, 3) : -1;
        bool ok = true;
        int done = 0;   // tiles handed over
        for (int j = 0; j < nt; ++j) {
            place(j, fw, pg0);
            if (fw == 0)
                place(j, 3, pg3);
            if (j + 1 < nt) {
                pg0 = lookup(j + 1, fw);
                if (fw == 0)
                    pg3 = lookup(j + 1, 3);
            }
            fetch_sync();
            // the rows' offsets serve keys and values
            int64_t off[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int r = r0 + u * kRowStep;
                const int row = r < BT ? sm.row[j % SL][r] : -1;
                off[u] = row < 0 ? -1 : ((int64_t)row * Hk + kh) * D + 8 * ch;
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int it = 2 * j + v;
                // a wait that ran out: the tile is not fetched, and the consumers' waits run out as well
                if (ok && it >= NS)
                    ok = lane_wait(&sm.empty[it % NS], (uint32_t)((it / NS - 1) & 1), &sm.wait_ns, abort_flag);
                if (ok) {
                    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(v ? c.v : c.k);
                    const uint32_t dst = smem_u32(sm.ring[it % NS]) + (ch >> 3) * kPanel;
#pragma unroll
                    for (int u = 0; u < kRows; ++u) {
                        const int r = r0 + u * kRowStep;
                        if (r < BT)
                            cp16(dst + sw128_offset(r, ch & 7), src + (off[u] < 0 ? 0 : off[u]), off[u] >= 0);
                    }
                }
                cp_commit();
                if (it >= kAhead - 1) {
                    cp_wait<kAhead - 1>();
                    if (ok)
                        arrive(done);
                    ++done;
                }
            }
        }
        cp_wait<0>();
        if (ok) {
            for (; done < 2 * nt; ++done)
                arrive(done);
        } else {
            *abort_flag = 1;
            if (lane == 0)
                set_status(a.st, BDLA_ERR_TIMEOUT, 0x31u);
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const int w = (warp - 4) >> 2, q4 = warp & 3, r = 32 * q4 + lane;
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const uint32_t t_s = tmem + BT * w + lane_off, t_o = tmem + 2 * BT + BT * w + lane_off;
        const int rr = rb * kWideRows + w * BT + r;   // row of the key head
        const bool live_row = rr < R;
        const int i = live_row ? rr / G : 0, h = kh * G + (live_row ? rr - i * G : 0);
        const int64_t at = ((int64_t)b * T + i) * Hq + h;   // row of q, o, lse
        {
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + at * D);
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch)
                *reinterpret_cast<uint4 *>(sm.q[w] + (ch >> 3) * kPanel + sw128_offset(r, ch & 7)) =
                    live_row ? src[ch] : make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            mbar_arrive(&sm.q_ready);
        }
        const uint64_t see = k1 > cut.len ? sees(a.tree, b, T, i) : 0;
        const float cs = a.scale * kLog2e;
        RowSoftmax row;
        bool ok = true;
        const int n = w < tiles ? nt : 0;
        for (int j = 0; j < n; ++j) {
            ok = warp_wait(&sm.s_full[w], (uint32_t)(j & 1), &sm.wait_ns, abort_flag);
            if (!ok)
                break;
            tc_fence_after();
            uint32_t x[4][32];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                tmem_ld32(t_s + 32 * k, x[k]);
            tmem_ld_wait();
            const int t0 = k0 + j * BT;
            uint32_t all = 0xffffffffu;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                all &= sm.valid[j % SL][k];
            if (all != 0xffffffffu || t0 + BT > cut.len) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // what this row sees of the 32 positions: the context, and its bits of the new tokens
                    const int j0 = t0 + 32 * k - cut.len;   // first of them as a new token
                    uint32_t mask = j0 <= -32 ? 0xffffffffu
                                              : j0 < 0 ? ((1u << -j0) - 1) | (uint32_t)(see << -j0)
                                                       : j0 < 64 ? (uint32_t)(see >> j0) : 0u;
                    mask &= sm.valid[j % SL][k];
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        x[k][e] = (mask >> e) & 1 ? x[k][e] : 0xff800000u;
                }
            }
            row_weights<D>(x, cs, t_s, t_o, j == 0, row, [&](int half) { mbar_arrive(&sm.p_ready[w][half]); });
        }
        if (ok && n > 0)
            ok = warp_wait(&sm.o_done[w], 0, &sm.wait_ns, abort_flag);
        if (ok && w < tiles) {
            tc_fence_after();
            const bool part = cut.used > 1;
            const int64_t pt = (((int64_t)b * Hk + kh) * ns + piece) * R + rr;
            const float inv = row.l == 0.0f ? 0.0f : 1.0f / row.l;
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
                uint32_t y[32];
                if (n > 0) {
                    tmem_ld32(t_o + 32 * k, y);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        y[e] = 0u;
                }
                if (!live_row)
                    continue;
                if (part) {
                    uint4 *dst = reinterpret_cast<uint4 *>(a.part_o + pt * D + 32 * k);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(a.o + at * D + 32 * k);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t v[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            v[u] = pack_bf16(__uint_as_float(y[8 * e + 2 * u]) * inv, __uint_as_float(y[8 * e + 2 * u + 1]) * inv);
                        dst[e] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            if (live_row && part)
                *reinterpret_cast<float2 *>(a.part_ml + 2 * pt) = make_float2(row.m, row.l);
            else if (live_row)
                a.lse[at] = row.l == 0.0f ? -INFINITY : fmaf(row.m, a.scale, logf(row.l));
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(a.st, BDLA_ERR_TIMEOUT, 0x32u);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tmem, 512);
}

template <int D> cudaError_t go(const Call &a, const bdla_attn_dims &d, cudaStream_t stream)
{
    const int R = d.T * (d.Hq / d.Hk), row_blocks = (R + kWideRows - 1) / kWideRows;
    const int64_t grid = (int64_t)d.B * d.Hk * row_blocks * a.pieces.ns;
    const size_t smem = sizeof(WideSmem<D>);
    const cudaError_t err = cudaFuncSetAttribute(cached_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess)
        return err;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    cached_wide_kernel<D><<<(unsigned)grid, kThreads, smem, stream>>>(a, row_blocks, g_wait_ns.load());
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cached_wide(const cache::Call &a, const bdla_attn_dims &d, cudaStream_t stream)
{
    return d.d == 64 ? go<64>(a, d, stream) : go<128>(a, d, stream);
}

}  // namespace bdla
