// Causal softmax attention over whole documents, forward, on the sm_100-family
// tensor cores.
//
//   s_ij = scale q_i . k_j (j <= i),  p_ij = e^{s_ij - m_i},  o_i = (sum_j p_ij v_j) / l_i,
//   l_i = sum_j p_ij,  lse_i = m_i + log l_i
// in one pass over the keys with a reference m_i that follows the running
// maximum.
//
// One CTA takes 256 consecutive queries of one document and head as two tiles
// of 128, and walks the keys in tiles of 128 up to the diagonal.  The two query
// tiles share every key and value tile and run in turn: while the tensor cores
// multiply for one, the four warps of the other turn scores into weights, so
// that neither pipe waits for a whole tile of the other.  Warp 0 loads (TMA,
// a ring of key and value tiles), warp 1 issues the MMAs, warps 2-5 and 6-9
// are the softmax of tile 0 and 1, one thread a query row.
//
// Tensor memory: scores of either tile (128 columns each), outputs (D columns
// each).  A thread reads its 128 scores, and writes the bf16 weights over them,
// from where the P V product takes its A operand.  m_i moves only when a score
// exceeds it by more than a factor 2^8 (kSlack): weights then stay below 2^8,
// far from overflow, sums lose nothing in fp32, and the output is rescaled in
// tensor memory in the first tiles only instead of in every one.  The order of
// the MMAs makes that safe without a barrier of its own: Q K of tile j is
// issued after P V of tile j - 1, so the scores' arrival says that the output
// is at rest.
//
// Rounding: scores, maxima, sums and outputs are fp32; the weights enter the
// P V product as bf16 (half a step, 2^-8 of each), as the tensor cores take
// them; the sum adds them before that rounding.
//
// Rows past a document's end hold the next document.  Their scores are masked
// by selection, and the values of the last tile's rows past the end are
// cleared in shared memory, so that 0 times another document's infinity or NaN
// never enters a sum.
//
// Bound by the tensor cores' turns (69% of the cycles), then by the chain from a
// tile's scores to its weights.  Measured, d = 128: 65536 tokens in 8 documents,
// 32 heads on 8, 4.32 ms (1.46 PFLOP/s, under the power cap); one document of
// 16384, 16 on 4, 0.68 ms (1.61 PFLOP/s, the GEMM's own rate being 1.91).  168
// registers a thread, 24 to 28 bytes of them spilled.
#include <cudaTypedefs.h>

#include "bdla_attn_sm100.cuh"

namespace bdla {

namespace {

using namespace sm100;
using namespace attn;

constexpr int kPairBlocks = 2;                   // query tiles of a CTA
constexpr int kThreads = 64 + kPairBlocks * BT;  // loader, MMA issuer, softmax

template <int D> struct FwdSmem {
    static constexpr int kPanels = D / 64;
    static constexpr int kTile = kPanels * kPanel;
    static constexpr int kStages = D == 128 ? 5 : 8;
    alignas(1024) unsigned char q[kPairBlocks][kTile];   // queries, then the output's staging
    alignas(1024) unsigned char ring[kStages][kTile];    // K_0 V_0 K_1 V_1 ...
    uint64_t full_q, full[kStages], empty[kStages], s_full[kPairBlocks], o_done[kPairBlocks];
    uint64_t p_ready[kPairBlocks][2];   // weights of the first and of the last 64 keys of a tile
    uint64_t drain, never;
    uint64_t wait_ns;
    uint32_t tmem_base;
    int abort_flag;
};

static_assert(sizeof(FwdSmem<128>) <= kMaxSmem && sizeof(FwdSmem<64>) <= kMaxSmem, "shared memory of a CTA");

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                const __grid_constant__ CUtensorMap tv, const int32_t *__restrict__ cu, int n_docs, int T,
                int64_t tokens, int Hq, int group, int n_slots, float scale, __nv_bfloat16 *__restrict__ o,
                float *__restrict__ lse, DeviceStatus *st, uint64_t wait_ns, int stall)
{
    using Smem = FwdSmem<D>;
    constexpr int NS = Smem::kStages, NP = Smem::kPanels;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && cu != nullptr)
        check_offsets(cu, n_docs, tokens, st);
    // heads fastest, so that the CTAs in flight share keys; late (long) query
    // blocks first, so that the short ones fill the end
    const int h = blockIdx.x % Hq;
    const SegSpan span = seg_span(cu, T, tokens, n_docs, n_slots - 1 - (int)(blockIdx.x / Hq), kPairBlocks);
    if (!span.valid || span.len <= 0)
        return;
    if ((smem_u32(smem_raw) & 1023u) != 0u) {
        if (tid == 0)
            set_status(st, BDLA_ERR_DEVICE, 0xA11u);
        return;
    }
    const int kh = h / group;
    // key tiles of each query tile: up to and with its own (0: no such tile)
    const int n_kv[2] = {span.blk_base + 1, span.len > BT ? span.blk_base + 2 : 0};
    const int n_max = n_kv[1] ? n_kv[1] : n_kv[0];
    const int64_t doc_start = span.doc_start;

    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        mbar_init(&sm.full_q, 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int w = 0; w < kPairBlocks; ++w) {
            mbar_init(&sm.s_full[w], 1);
            mbar_init(&sm.p_ready[w][0], BT);
            mbar_init(&sm.p_ready[w][1], BT);
            mbar_init(&sm.o_done[w], 1);
        }
        mbar_init(&sm.drain, 1);
        mbar_init(&sm.never, 1);
        sm.abort_flag = 0;
        sm.wait_ns = wait_ns;
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    volatile int *abort_flag = &sm.abort_flag;
    const int stall_at = n_max > 1 ? 1 : 0;   // test hook: the key tile at which a role stalls

    if (warp == 0) {
        // ---------------------------------------------------------------- loader
        if (lane == 0) {
            tma_prefetch_desc(&tq);
            tma_prefetch_desc(&tk);
            tma_prefetch_desc(&tv);
            const int tiles_q = n_kv[1] ? 2 : 1;
            mbar_arrive_expect_tx(&sm.full_q, (uint32_t)(tiles_q * Smem::kTile));
            for (int w = 0; w < tiles_q; ++w)
                for (int p = 0; p < NP; ++p)
                    tma_load_3d(sm.q[w] + p * kPanel, &tq, &sm.full_q, p * 64, h, (int)(span.start + w * BT));
            int issued = 0;
            bool ok = true;
            for (int it = 0; it < 2 * n_max; ++it) {
                const int s = it % NS;
                const bool hook = stall == BDLA_STALL_PRODUCER && it == 2 * stall_at;
                if ((it >= NS || hook) && !lane_wait(hook ? &sm.never : &sm.empty[s],
                                                     hook ? 0u : (uint32_t)((it / NS - 1) & 1), &sm.wait_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&sm.full[s], (uint32_t)Smem::kTile);
                for (int p = 0; p < NP; ++p)
                    tma_load_3d(sm.ring[s] + p * kPanel, (it & 1) ? &tv : &tk, &sm.full[s], p * 64, kh,
                                (int)(doc_start + (int64_t)(it >> 1) * BT));
                issued = it + 1;
            }
            if (!ok) {
                *abort_flag = 1;
                set_status(st, BDLA_ERR_TIMEOUT, 0x10u);
                // the copies this thread started land before the CTA exits
                mbar_wait(&sm.full_q, 0, kDrainNs);
                for (int it = issued > NS ? issued - NS : 0; it < issued; ++it)
                    mbar_wait(&sm.full[it % NS], (it / NS) & 1, kDrainNs);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        const uint64_t q[2] = {rows_desc(smem_u32(sm.q[0])), rows_desc(smem_u32(sm.q[1]))};
        bool ok = warp_wait(&sm.full_q, 0, &sm.wait_ns, abort_flag);
        // S_w = Q_w K_j^T over the scores (and weights) of tile j - 1
        auto issue_qk = [&](int w, int j) {
            const int it = 2 * j;
            if (!warp_wait(&sm.full[it % NS], (it / NS) & 1, &sm.wait_ns, abort_flag))
                return false;
            tc_fence_after();
            const uint64_t k = rows_desc(smem_u32(sm.ring[it % NS]));
            if (elect_one()) {
                mma_rows<D>(tmem + BT * w, q[w], k);
                umma_commit(&sm.s_full[w]);
                if (w == 1 || j >= n_kv[1])   // the last reader of this key tile
                    umma_commit(&sm.empty[it % NS]);
            }
            __syncwarp();
            return true;
        };
        for (int w = 0; ok && w < 2; ++w)
            if (n_kv[w] > 0)
                ok = issue_qk(w, 0);
        for (int j = 0; ok && j < n_max; ++j) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (!ok || j >= n_kv[w])
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
                    if (w == 1 || j >= n_kv[1])
                        umma_commit(&sm.empty[it % NS]);
                    if (j + 1 >= n_kv[w])
                        umma_commit(&sm.o_done[w]);
                }
                __syncwarp();
                if (j + 1 < n_kv[w])
                    ok = issue_qk(w, j + 1);
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(st, BDLA_ERR_TIMEOUT, 0x11u);
        }
        // every MMA issued above has completed before TMEM is released
        if (elect_one())
            umma_commit(&sm.drain);
        __syncwarp();
        mbar_wait(&sm.drain, 0, kDrainNs);
    } else {
        // ---------------------------------------------------------------- softmax
        const int w = (warp - 2) >> 2;
        const int q4 = warp & 3;
        const int r = 32 * q4 + lane;   // row of the tile, TMEM lane
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const uint32_t t_s = tmem + BT * w + lane_off, t_o = tmem + 2 * BT + BT * w + lane_off;
        const int n = n_kv[w];
        const int valid = (int)(span.len - w * BT);   // rows of the tile inside the document (may exceed 128)
        const float c = scale * kLog2e;
        RowSoftmax row;
        bool ok = true;
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
            if (j == n - 1) {   // the diagonal tile: keys past the query (and with them all past the end)
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[k][i] = 32 * k + i > r ? 0xff800000u : x[k][i];
            }
            if (j == n - 1 && valid < BT) {
                // this tile alone reads the document's last values: clear the rows past the end
                const int it = 2 * j + 1;
                ok = warp_wait(&sm.full[it % NS], (it / NS) & 1, &sm.wait_ns, abort_flag);
                if (!ok)
                    break;
                clear_rows(sm.ring[it % NS], NP, valid, r, BT);
                fence_proxy_async_smem();
            }
            row_weights<D>(x, c, t_s, t_o, j == 0, row, [&](int half) { mbar_arrive(&sm.p_ready[w][half]); });
        }
        if (ok && n > 0)
            ok = warp_wait(&sm.o_done[w], 0, &sm.wait_ns, abort_flag);
        if (ok && n > 0) {
            tc_fence_after();
            const int64_t t0 = span.start + w * BT;
            if (r < valid)
                lse[(int64_t)h * tokens + t0 + r] = (row.mc + log2f(row.l)) * kLn2;
            const float inv = 1.0f / row.l;
            // the tile's queries have been read: a warp stages its own 32 rows of 128 bytes there
#pragma unroll
            for (int p = 0; p < NP; ++p)
                store_rows64(t_o + 64 * p, inv, sm.q[w] + q4 * 4096, o + ((size_t)(t0 + 32 * q4) * Hq + h) * D + p * 64,
                             (size_t)Hq * D, valid - 32 * q4, lane);
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(st, BDLA_ERR_TIMEOUT, 0x12u);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem, 512);
}

// The check of a packed call that has no tokens (and so no attention CTA).
__global__ void doc_report_kernel(const int32_t *cu, int n_docs, int64_t tokens, DeviceStatus *st)
{
    check_offsets(cu, n_docs, tokens, st);
}

template <int D>
cudaError_t go(const AttnProblem &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
               __nv_bfloat16 *o, float *lse)
{
    auto kern = attn_fwd_kernel<D>;
    const size_t smem = sizeof(FwdSmem<D>);
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess)
        return err;
    const int64_t rows = kPairBlocks * BT;
    const int64_t n_slots = (p.tokens + rows - 1) / rows + p.n_docs;
    if (n_slots * p.Hq > INT32_MAX)
        return cudaErrorInvalidValue;
    kern<<<(unsigned)(n_slots * p.Hq), kThreads, smem, p.stream>>>(
        mq, mk, mv, p.cu, p.n_docs, p.T, p.tokens, p.Hq, p.Hq / p.Hk, (int)n_slots, p.scale, o, lse, p.st,
        g_wait_ns.load(), g_test_stall[BDLA_KERNEL_ATTN_FWD].load());
    return cudaGetLastError();
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
    KernelMark mark_(BDLA_KERNEL_ATTN_FWD, p.stream);
    if (p.tokens == 0)
        return launch_doc_report(p);
    CUtensorMap mq, mk, mv;
    if (!make_token_map(&mq, q, p.d, p.Hq, p.tokens) || !make_token_map(&mk, k, p.d, p.Hk, p.tokens) ||
        !make_token_map(&mv, v, p.d, p.Hk, p.tokens))
        return cudaErrorInvalidValue;
    return p.d == 64 ? go<64>(p, mq, mk, mv, o, lse) : go<128>(p, mq, mk, mv, o, lse);
}

}  // namespace bdla
