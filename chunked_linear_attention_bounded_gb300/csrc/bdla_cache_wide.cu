// Attention over the paged cache for many rows a key head (a tree of drafts
// times the query heads of a group), on the sm_100-family tensor cores.
//
// The mathematics and the pieces are those of bdla_cache.cu; the pipeline is
// that of the whole-prompt forward (bdla_attn_fwd.cu): up to 256 rows as two
// tiles of 128 that take turns between the tensor cores and their softmax
// warps, scores and outputs in tensor memory, weights read from there by the
// P V product, a reference maximum that moves only when a score passes it by
// 2^8.  What differs is where the keys come from: three warps take the tiles of
// 128 positions in turn, look the positions up in the page table (two tiles of
// the other warps pass between a lookup and its use) and fetch.  Where 16 or
// more consecutive positions always share a page, a tile that is wholly visible
// comes by TMA, one box for each such run, and only a tile with something to
// leave out (the last of a sequence, a bad page) row by row with cp.async, which
// writes zeros for a row.  Other page sizes take cp.async throughout.
//
// Warp 0 issues the MMAs, warps 1-3 fetch, warps 4-7 and 8-11 are the softmax
// of the two tiles, one thread a row.
//
// Between HBM and the tensor cores (61% and 59% of their peaks): 4 sequences of
// 65536 positions, 61 drafts, 16 heads on 4, d = 128: 113 us (4.8 TB/s), from cold
// and with the join 123; at a few thousand positions the start-up, a CTA's first
// tiles and the join weigh more.  168 registers a thread, 20 bytes spilled.
#include <cudaTypedefs.h>

#include "bdla_attn_sm100.cuh"
#include "bdla_cache.cuh"

namespace bdla {

namespace {

using namespace sm100;
using namespace attn;
using namespace cache;

constexpr int kFetchWarps = 3;
constexpr int kThreads = 32 + 32 * kFetchWarps + 256;

template <int D> struct WideSmem {
    static constexpr int kPanels = D / 64;
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int kStages = D == 128 ? 5 : 8;
    // `valid` of a tile is written again by the tile eight later, which is looked up when at most six tiles (the ring
    // and the warps' own) lie between it and the softmax.
    static constexpr int kSlots = 8;
    alignas(1024) unsigned char q[2][kTile];
    alignas(1024) unsigned char ring[kStages][kTile];   // K_0 V_0 K_1 V_1 ...
    int row[kFetchWarps][BT];    // cache row of the positions of a warp's tile, -1: not seen
    uint32_t valid[kSlots][4];   // positions of a tile that may be seen
    uint64_t full[kStages], empty[kStages], s_full[2], o_done[2], drain, never;
    uint64_t p_ready[2][2];   // weights of the first and of the last 64 positions of a tile
    uint64_t wait_ns;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(WideSmem<128>) <= kMaxSmem && sizeof(WideSmem<64>) <= kMaxSmem, "shared memory of a CTA");

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}

// `run`: consecutive positions that always share a page (a power of two, 16 ..
// 128; the maps' boxes have that many rows), or 0: no TMA.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cached_wide_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, int run,
                   const __grid_constant__ Call a, int row_blocks, uint64_t wait_ns, int stall)
{
    using Smem = WideSmem<D>;
    constexpr int NS = Smem::kStages, SL = Smem::kSlots, NP = Smem::kPanels, kChunks = D / 8;
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
    next_may_start();
    // softmax threads: tile, row of the tile, row of the key head, row of q, o and lse; their queries are asked for
    // before the lengths, which the rest waits for
    const int w = warp >= 8, q4 = warp & 3, r = 32 * q4 + lane;
    const int rr = rb * kWideRows + w * BT + r;
    const bool live_row = warp >= 4 && rr < R;
    const int i = live_row ? rr / G : 0;
    const int64_t at = ((int64_t)b * T + i) * Hq + kh * G + (live_row ? rr - i * G : 0);
    uint4 qrow[kChunks];
#pragma unroll
    for (int ch = 0; ch < kChunks; ++ch)
        qrow[ch] = live_row ? reinterpret_cast<const uint4 *>(a.q + at * D)[ch] : make_uint4(0, 0, 0, 0);
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

    // fetching warps: pages of the lane's four positions of a tile
    const int fw = warp - 1;
    const int32_t *table = c.pages + (int64_t)b * c.max_pages;
    auto lookup = [&](int j, int (&pg)[4]) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = k0 + j * BT + 4 * lane + u;
            pg[u] = j < nt && t < k1 ? table[a.div.entry(t)] : -1;
        }
    };
    int pg[4];
    uint64_t seen = 0;
    if (warp == 0) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    } else if (warp < 4) {
        lookup(fw, pg);
        if (tid == 32) {
            for (int s = 0; s < NS; ++s) {
                mbar_init(&sm.full[s], 32);
                mbar_init(&sm.empty[s], 1);
            }
            for (int x = 0; x < 2; ++x) {
                mbar_init(&sm.s_full[x], 1);
                mbar_init(&sm.p_ready[x][0], BT);
                mbar_init(&sm.p_ready[x][1], BT);
                mbar_init(&sm.o_done[x], 1);
            }
            mbar_init(&sm.drain, 1);
            mbar_init(&sm.never, 1);
            sm.abort_flag = 0;
            sm.wait_ns = wait_ns;
            mbar_fence_init();
        }
        if (k1 > cut.len)
            seen = sees_any(a.tree, b, T, lane);
        asm volatile("bar.sync 2, 96;" ::: "memory");   // the barriers are there: fetching starts
    } else {
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch)
            *reinterpret_cast<uint4 *>(sm.q[w] + (ch >> 3) * kPanel + sw128_offset(r, ch & 7)) = qrow[ch];
        fence_proxy_async_smem();
    }
    tc_fence_before();
    if (warp >= 1 && warp < 4)
        asm volatile("bar.arrive 1, 384;" ::: "memory");
    else
        asm volatile("bar.sync 1, 384;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem = warp >= 1 && warp < 4 ? 0 : sm.tmem_base;   // (the fetching warps do not wait for it)
    volatile int *abort_flag = &sm.abort_flag;
    const int stall_at = nt > 1 ? 1 : 0;   // test hook: the tile at which a role stalls

    if (warp == 0) {
        // ---------------------------------------------------------------- MMA issuer
        const uint64_t q[2] = {rows_desc(smem_u32(sm.q[0])), rows_desc(smem_u32(sm.q[1]))};
        bool ok = true;
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
                const bool hook = stall == BDLA_STALL_MMA && j == stall_at;
                ok = warp_wait(&sm.full[it % NS], (it / NS) & 1, &sm.wait_ns, abort_flag) &&
                     warp_wait(hook ? &sm.never : &sm.p_ready[w][0], hook ? 0u : (uint32_t)(j & 1), &sm.wait_ns, abort_flag);
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
        bool ok = true;
        int issued = -1;   // this warp's last tile asked of TMA
        for (int j = fw; ok && j < nt; j += kFetchWarps) {
            int row[4];
            uint32_t bits = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int t = k0 + j * BT + 4 * lane + u;
                bool live = t < k1 && (t < cut.len || ((seen >> (t - cut.len)) & 1));
                if (live && (pg[u] < 0 || pg[u] >= c.n_pages)) {
                    set_status(a.st, BDLA_ERR_DEVICE, (unsigned)b);
                    live = false;
                }
                row[u] = live ? pg[u] * c.page + a.div.offset(t) : -1;
                bits |= (live ? 1u : 0u) << u;
            }
            const bool whole = run > 0 && __all_sync(0xffffffffu, bits == 15u);
            bits <<= 4 * (lane & 7);
#pragma unroll
            for (int x = 1; x < 8; x <<= 1)
                bits |= __shfl_xor_sync(0xffffffffu, bits, x);
            if ((lane & 7) == 0)
                sm.valid[j % SL][lane >> 3] = bits;
            if (!whole) {
                *reinterpret_cast<int4 *>(&sm.row[fw][4 * lane]) = make_int4(row[0], row[1], row[2], row[3]);
                __syncwarp();
            }
            lookup(j + kFetchWarps, pg);
#pragma unroll 1
            for (int v = 0; ok && v < 2; ++v) {
                const int it = 2 * j + v, s = it % NS;
                const bool hook = stall == BDLA_STALL_PRODUCER && it == 2 * stall_at;
                if (it >= NS || hook)
                    ok = warp_wait(hook ? &sm.never : &sm.empty[s], hook ? 0u : (uint32_t)((it / NS - 1) & 1), &sm.wait_ns,
                                   abort_flag);
                if (!ok)
                    break;
                if (whole) {
                    if (elect_one())
                        mbar_arrive_expect_tx(&sm.full[s], (uint32_t)Smem::kTile);
                    else
                        mbar_arrive(&sm.full[s]);
                    __syncwarp();
                    for (int x = 0; x < BT; x += run) {
                        const int first = __shfl_sync(0xffffffffu, row[0], x >> 2);
                        if (elect_one()) {
#pragma unroll
                            for (int p = 0; p < NP; ++p)
                                tma_load_2d(sm.ring[s] + p * kPanel + x * 128, v ? &tv : &tk, &sm.full[s], kh * D + 64 * p,
                                            first);
                        }
                        __syncwarp();
                    }
                    issued = it;
                } else {
                    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(v ? c.v : c.k) + (int64_t)kh * D;
                    const int ch = lane % kChunks;
                    const uint32_t dst = smem_u32(sm.ring[s]) + (ch >> 3) * kPanel;
#pragma unroll 8
                    for (int x = lane / kChunks; x < BT; x += 32 / kChunks) {
                        const int at_row = sm.row[fw][x];
                        cp16(dst + sw128_offset(x, ch & 7), src + (int64_t)max(at_row, 0) * Hk * D + 8 * ch, at_row >= 0);
                    }
                    cp_commit();
                    if (v == 1) {   // keys first, while the values are on their way
                        cp_wait<1>();
                        fence_proxy_async_smem();
                        mbar_arrive(&sm.full[(it - 1) % NS]);
                        cp_wait<0>();
                        fence_proxy_async_smem();
                        mbar_arrive(&sm.full[s]);
                    }
                }
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(a.st, BDLA_ERR_TIMEOUT, 0x31u);
            // this warp's copies in flight land before the CTA exits
            cp_wait<0>();
            for (int it = max(issued - NS + 1, 0); it <= issued; ++it)
                if ((it >> 1) % kFetchWarps == fw)
                    mbar_wait(&sm.full[it % NS], (it / NS) & 1, kDrainNs);
        }
    } else {
        // ---------------------------------------------------------------- softmax
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const uint32_t t_s = tmem + BT * w + lane_off, t_o = tmem + 2 * BT + BT * w + lane_off;
        const uint64_t see = k1 > cut.len ? sees(a.tree, b, T, i) : 0;
        const float cs = a.scale * kLog2e;
        RowSoftmax row;
        bool ok = true;
        const int n = w < tiles ? nt : 0;
        for (int j = 0; j < n; ++j) {
            const bool hook = stall == BDLA_STALL_EPILOGUE && j == stall_at;
            ok = warp_wait(hook ? &sm.never : &sm.s_full[w], hook ? 0u : (uint32_t)(j & 1), &sm.wait_ns, abort_flag);
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
            // 32 rows of 128 bytes at a time through the warp's own part of its query tile (read by now), so that whole
            // lines leave: 32 fp32 columns of a piece, or 64 bf16 columns of an output
            uint4 *stage = reinterpret_cast<uint4 *>(sm.q[w] + q4 * 4096);
#pragma unroll 1
            for (int k = 0; k < D / 32; k += part ? 1 : 2) {
                uint32_t y[32];
                for (int u = 0; u < (part ? 1 : 2); ++u) {
                    if (n > 0) {
                        tmem_ld32(t_o + 32 * (k + u), y);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            y[e] = 0u;
                    }
                    if (part) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            stage[lane * 8 + (e ^ (lane & 7))] = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t z[4];
#pragma unroll
                            for (int f = 0; f < 4; ++f)
                                z[f] = pack_bf16(__uint_as_float(y[8 * e + 2 * f]) * inv, __uint_as_float(y[8 * e + 2 * f + 1]) * inv);
                            stage[lane * 8 + ((4 * u + e) ^ (lane & 7))] = make_uint4(z[0], z[1], z[2], z[3]);
                        }
                    }
                }
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int x = 4 * u + (lane >> 3), row_x = rr - lane + x;   // row of the warp, of the key head
                    const uint4 z = stage[x * 8 + ((lane & 7) ^ (x & 7))];
                    if (row_x >= R)
                        continue;
                    if (part) {
                        *reinterpret_cast<uint4 *>(a.part_o + (pt - lane + x) * D + 32 * k + 4 * (lane & 7)) = z;
                    } else {
                        const int i_x = row_x / G;
                        *reinterpret_cast<uint4 *>(a.o + (((int64_t)b * T + i_x) * Hq + kh * G + row_x - i_x * G) * D + 32 * k +
                                                   8 * (lane & 7)) = z;
                    }
                }
                __syncwarp();
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

// 2-D map over the cache's rows [n_pages * page][Hk * d]: box = 64 features x
// `run` rows, 128-byte swizzle.
bool make_rows_map(CUtensorMap *map, const void *ptr, int64_t width, int64_t rows, int run)
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (fn == nullptr)
        return false;
    cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)width * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)run};
    cuuint32_t es[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D> cudaError_t go(const Call &a, const bdla_attn_dims &d, cudaStream_t stream)
{
    const int R = d.T * (d.Hq / d.Hk), row_blocks = (R + kWideRows - 1) / kWideRows;
    const int64_t grid = (int64_t)d.B * d.Hk * row_blocks * a.pieces.ns;
    const size_t smem = sizeof(WideSmem<D>);
    const cudaError_t err = cudaFuncSetAttribute(cached_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess)
        return err;
    int run = a.c.page & -a.c.page;   // the largest power of two in the page
    run = run > BT ? BT : run;
    CUtensorMap tk{}, tv{};
    const int64_t rows = (int64_t)a.c.n_pages * a.c.page, width = (int64_t)d.Hk * D;
    if (run < 16 || rows == 0)
        run = 0;
    else if (!make_rows_map(&tk, a.c.k, width, rows, run) || !make_rows_map(&tv, a.c.v, width, rows, run))
        return cudaErrorInvalidValue;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    cached_wide_kernel<D><<<(unsigned)grid, kThreads, smem, stream>>>(tk, tv, run, a, row_blocks, g_wait_ns.load(),
                                                              g_test_stall[BDLA_KERNEL_ATTN_CACHED].load());
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cached_wide(const cache::Call &a, const bdla_attn_dims &d, cudaStream_t stream)
{
    return d.d == 64 ? go<64>(a, d, stream) : go<128>(a, d, stream);
}

}  // namespace bdla
