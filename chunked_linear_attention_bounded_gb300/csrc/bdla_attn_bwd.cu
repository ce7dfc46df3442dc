// Causal softmax attention over whole documents, gradient, on the sm_100-family
// tensor cores.
//
//   p_ij = e^{s_ij - lse_i},  delta_i = dO_i . o_i,  dp_ij = dO_i . v_j,  ds_ij = p_ij (dp_ij - delta_i)
//   dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i,   dv_j = sum_i p_ij dO_i
//   (dk, dv also summed over the query heads of the key head)
//
// Two kernels, each of which owns what it sums into: one per tile of queries
// that walks its keys (dq, and delta for the second), one per tile of keys that
// walks the queries of all heads of its group (dk, dv).  Scores and dp are
// formed in both, seven products of the pairs instead of five, and in return
// nothing is added through memory: no fp32 copy of dq (four bytes an element
// written and read again for every key tile), no atomics, and the same bits
// from the same inputs.
//
// Both kernels: warp 0 loads (TMA, a ring of tiles), warp 1 issues the MMAs,
// warps 2-9 form the weights, two warps for every 32 rows, 64 columns each.
// The rows of the accumulators are the rows of what is summed into (queries, or
// keys: the scores are then formed transposed), so that p and ds go back to
// tensor memory as the A operand of the next product and never pass through
// shared memory.  They are written over the scores (or dp) that they were
// formed from, each warp inside its own 64 columns.
//
// Rounding: scores, dp, delta and the accumulators are fp32; p and ds enter
// their products as bf16 (half a step, 2^-8 of each); ds is formed from the
// fp32 p.  delta is dO . o with the o that the forward rounded to bf16 for dq,
// which needs it before it has seen every key; the same kernel sums p o dp in
// fp32 on its way, and the second takes that delta, free of o's rounding (dk's
// error against 64 bits 2.8e-3 -> 2.4e-3 of its norm at 1537 tokens).  A tile of
// queries with one tile of keys, the first of every document, has all of its
// weights at hand: it normalises them by their own sum and takes delta from them
// before ds, so that short rows, where o's rounding weighs most, are as exact as
// their weights, and a document's first token, whose ds is 0, gets 0.
//
// All of that stands in for the formula only while it cannot be told from it: the
// sum of p o dp for dO . o within the rounding of o's entries, 2^-8 sum |dO o|, and
// the weights over their sum for the weights where that sum is 1 within 2^-8, the
// rounding of ds.  o and lse that were joined with other keys' (a sink, another
// set of keys) are outside, and p = e^{s - lse} and delta = dO . o are then taken
// as they are.
//
// Rows past a document's end hold the next document.  Their p and ds are
// zeroed by selection, and where such rows are the summed side of a product
// their operand rows are cleared in shared memory, so that another document's
// infinity or NaN never enters a sum.
//
// Bound by the tensor cores' turns (62 and 69% of the cycles of the two) and the
// chain from scores to weights between them.  Measured, d = 128: 4 documents of
// 8192, 16 heads on 4, 2.78 ms, 0.99 PFLOP/s of the five products that a gradient
// needs, 1.39 of the seven; one of 16384, 16 on 4, 2.54 ms, 1.08 and 1.51.  Up to
// 168 registers a thread; the first kernel spills 4 to 8 bytes.
#include <cudaTypedefs.h>

#include "bdla_attn_sm100.cuh"

namespace bdla {

namespace {

using namespace sm100;
using namespace attn;

constexpr int kEpi = 256;              // weight threads
constexpr int kThreads = 64 + kEpi;    // + loader and MMA issuer
constexpr float kHalfStep = 0x1p-8f;   // of bf16, relative

template <int D> struct BwdSmem {
    static constexpr int kPanels = D / 64;
    static constexpr int kTile = kPanels * kPanel;
    // Tiles of K and V (of Q and dO) in a ring each.  K (Q) is held from the scores to the last product of its tile,
    // V (dO) for less long, so K's ring is the longer: in one ring of five, V waited for K, and a load's latency stood
    // in every tile's time.
    static constexpr int kA = D == 128 ? 3 : 4, kB = D == 128 ? 2 : 4, kStages = kA + kB;
    alignas(1024) unsigned char own[2][kTile];          // Q, dO of the query tile, or K, V of the key tile
    alignas(1024) unsigned char ring[kStages][kTile];   // kA tiles of K (Q), kB of V (dO)
    static __host__ __device__ constexpr int slot(int it) { return it & 1 ? kA + (it >> 1) % kB : (it >> 1) % kA; }
    static __host__ __device__ constexpr int turn(int it) { return it & 1 ? (it >> 1) / kB : (it >> 1) / kA; }
    float col[2][2][BT];   // key tiles: -lse * log2 e and -delta of a query tile; query tiles: halves of dO . o, of sum |dO o|
    uint64_t full_own, full[kStages], empty[kStages], s_full[2], dp_full, dp_free, done;
    uint64_t ready[2][2];   // [tile, or p and ds][part]: weights whose first, last 32 columns of each warp's 64 are there
    uint64_t drain, never;
    uint64_t wait_ns;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(BwdSmem<128>) <= kMaxSmem && sizeof(BwdSmem<64>) <= kMaxSmem, "shared memory of a CTA");

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The same barrier, which also says whether every thread still runs.
__device__ __forceinline__ bool epi_all(bool v)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// Tensor memory: both kernels hold two 128-column tiles of scores or dp and
// their accumulators.
template <typename Smem>
__device__ __forceinline__ void setup(Smem &sm, int tid, uint64_t wait_ns)
{
    if ((tid >> 5) == 1) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        mbar_init(&sm.full_own, 1);
        for (int s = 0; s < Smem::kStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.s_full[b], 1);
            mbar_init(&sm.ready[b][0], kEpi);
            mbar_init(&sm.ready[b][1], kEpi);
        }
        mbar_init(&sm.dp_full, 1);
        mbar_init(&sm.dp_free, kEpi);
        mbar_init(&sm.done, 1);
        mbar_init(&sm.drain, 1);
        mbar_init(&sm.never, 1);
        sm.abort_flag = 0;
        sm.wait_ns = wait_ns;
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

// The loader's rings: `n` tiles, K_0 V_0 K_1 V_1 ..., tile `it` fetched by
// load(it, slot).  Lets its copies land before it returns from a wait that ran
// out.
template <typename Smem, typename Load>
__device__ __forceinline__ void run_loader(Smem &sm, int n, int stall_it, DeviceStatus *st, Load load)
{
    volatile int *abort_flag = &sm.abort_flag;
    int issued = 0;
    bool ok = true;
    for (int it = 0; it < n; ++it) {
        const int s = Smem::slot(it), turn = Smem::turn(it);
        const bool hook = it == stall_it;
        if ((turn > 0 || hook) && !lane_wait(hook ? &sm.never : &sm.empty[s], hook ? 0u : (uint32_t)((turn - 1) & 1),
                                             &sm.wait_ns, abort_flag)) {
            ok = false;
            break;
        }
        mbar_arrive_expect_tx(&sm.full[s], (uint32_t)Smem::kTile);
        load(it, s);
        issued = it + 1;
    }
    if (!ok) {
        *abort_flag = 1;
        set_status(st, BDLA_ERR_TIMEOUT, 0x20u);
        mbar_wait(&sm.full_own, 0, kDrainNs);
        // the last tile of every slot
        for (int it = issued > 2 * Smem::kStages ? issued - 2 * Smem::kStages : 0; it < issued; ++it)
            if (it + 2 * (it & 1 ? Smem::kB : Smem::kA) >= issued)
                mbar_wait(&sm.full[Smem::slot(it)], Smem::turn(it) & 1, kDrainNs);
    }
}

// ---------------------------------------------------------------- dq
// Tensor memory: scores of even and odd key tiles (ds over them), dp, dq.  While
// the weights of tile j are formed, the tensor cores run S of j + 1, dp of j + 1
// (dp is free once it is in registers) and dq of j - 1.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_dq_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
               const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
               const __nv_bfloat16 *__restrict__ o, const __nv_bfloat16 *__restrict__ dO, const float *__restrict__ lse,
               const int32_t *__restrict__ cu, int n_docs, int T, int64_t tokens, int Hq, int group, int n_slots,
               float scale, __nv_bfloat16 *__restrict__ dq, float *__restrict__ delta, DeviceStatus *st,
               uint64_t wait_ns, int stall)
{
    using Smem = BwdSmem<D>;
    constexpr int NP = Smem::kPanels;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    next_may_start();
    if (blockIdx.x == 0 && cu != nullptr)
        check_offsets(cu, n_docs, tokens, st);
    // late (long) query tiles first
    const int h = blockIdx.x % Hq;
    const SegSpan span = seg_span(cu, T, tokens, n_docs, n_slots - 1 - (int)(blockIdx.x / Hq), 1);
    if (!span.valid || span.len <= 0)
        return;
    if ((smem_u32(smem_raw) & 1023u) != 0u) {
        if (tid == 0)
            set_status(st, BDLA_ERR_DEVICE, 0xA11u);
        return;
    }
    const int kh = h / group;
    const int n = span.blk_base + 1;       // key tiles up to the diagonal
    const int valid = (int)span.len;       // rows of the tile (and keys of the diagonal one) inside the document
    const int stall_at = n > 1 ? 1 : 0;
    setup(sm, tid, wait_ns);
    const uint32_t tmem = sm.tmem_base, t_dp = tmem + 2 * BT, t_dq = tmem + 3 * BT;
    volatile int *abort_flag = &sm.abort_flag;

    if (warp == 0) {
        if (lane == 0) {
            mbar_arrive_expect_tx(&sm.full_own, 2u * Smem::kTile);
            for (int p = 0; p < NP; ++p) {
                tma_load_3d(sm.own[0] + p * kPanel, &tq, &sm.full_own, p * 64, h, (int)span.start);
                tma_load_3d(sm.own[1] + p * kPanel, &tdo, &sm.full_own, p * 64, h, (int)span.start);
            }
            run_loader(sm, 2 * n, stall == BDLA_STALL_PRODUCER ? 2 * stall_at : -1, st, [&](int it, int s) {
                for (int p = 0; p < NP; ++p)
                    tma_load_3d(sm.ring[s] + p * kPanel, (it & 1) ? &tv : &tk, &sm.full[s], p * 64, kh,
                                (int)(span.doc_start + (int64_t)(it >> 1) * BT));
            });
        }
    } else if (warp == 1) {
        const uint64_t q = rows_desc(smem_u32(sm.own[0])), g = rows_desc(smem_u32(sm.own[1]));
        auto tile = [&](int it) { return smem_u32(sm.ring[Smem::slot(it)]); };
        auto landed = [&](int it) { return warp_wait(&sm.full[Smem::slot(it)], Smem::turn(it) & 1, &sm.wait_ns, abort_flag); };
        auto issue_s = [&](int j) {
            if (!landed(2 * j))
                return false;
            tc_fence_after();
            if (elect_one()) {
                mma_rows<D>(tmem + BT * (j & 1), q, rows_desc(tile(2 * j)));
                umma_commit(&sm.s_full[j & 1]);
            }
            __syncwarp();
            return true;
        };
        auto issue_dp = [&](int j) {
            if (!landed(2 * j + 1))
                return false;
            tc_fence_after();
            if (elect_one()) {
                mma_rows<D>(t_dp, g, rows_desc(tile(2 * j + 1)));
                umma_commit(&sm.dp_full);
                umma_commit(&sm.empty[Smem::slot(2 * j + 1)]);
            }
            __syncwarp();
            return true;
        };
        bool ok = warp_wait(&sm.full_own, 0, &sm.wait_ns, abort_flag) && issue_s(0) && issue_dp(0);
        for (int j = 0; ok && j < n; ++j) {
            const bool hook = stall == BDLA_STALL_MMA && j == stall_at;
            if (j + 1 < n)
                ok = issue_s(j + 1) && warp_wait(&sm.dp_free, j & 1, &sm.wait_ns, abort_flag) && issue_dp(j + 1);
            const uint32_t turn = (uint32_t)((j >> 1) & 1);
            ok = ok && warp_wait(hook ? &sm.never : &sm.ready[j & 1][0], hook ? 0u : turn, &sm.wait_ns, abort_flag);
            if (!ok)
                break;
            tc_fence_after();
            const uint64_t k = sum_desc(tile(2 * j));
            if (elect_one())
                mma_sum_part<D, 0>(t_dq, tmem + BT * (j & 1), k, j > 0);
            __syncwarp();
            if (!(ok = warp_wait(&sm.ready[j & 1][1], turn, &sm.wait_ns, abort_flag)))
                break;
            tc_fence_after();
            if (elect_one()) {
                mma_sum_part<D, 1>(t_dq, tmem + BT * (j & 1), k, true);
                umma_commit(&sm.empty[Smem::slot(2 * j)]);
                if (j == n - 1)
                    umma_commit(&sm.done);
            }
            __syncwarp();
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(st, BDLA_ERR_TIMEOUT, 0x21u);
        }
        if (elect_one())
            umma_commit(&sm.drain);
        __syncwarp();
        mbar_wait(&sm.drain, 0, kDrainNs);
    } else {
        const int half = (warp - 2) >> 2, q4 = warp & 3, r = 32 * q4 + lane, e = 128 * half + r;
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const int64_t t = span.start + r;
        // delta of the row, and how far o's rounding may have moved it, half the features each
        float dl = 0.0f, dev = 0.0f, l2 = 0.0f;
        if (r < valid) {
            const size_t off = ((size_t)t * Hq + h) * D + half * (D / 2);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const uint4 a = *reinterpret_cast<const uint4 *>(o + off + 8 * i);
                const uint4 b = *reinterpret_cast<const uint4 *>(dO + off + 8 * i);
                const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float f = bf16_lo(x[u]) * bf16_lo(y[u]), g = bf16_hi(x[u]) * bf16_hi(y[u]);   // exact
                    dl = g + (f + dl);
                    dev += fabsf(f) + fabsf(g);
                }
            }
            l2 = lse[(int64_t)h * tokens + t] * kLog2e;
        }
        sm.col[0][half][r] = dl;
        sm.col[1][half][r] = dev;
        epi_sync();
        dl = sm.col[0][0][r] + sm.col[0][1][r];
        // The row's own delta in dO . o's place, if o's rounding covers the difference.
        auto chosen = [&](float own) {
            const float given = sm.col[0][0][r] + sm.col[0][1][r];
            return fabsf(own - given) <= kHalfStep * (sm.col[1][0][r] + sm.col[1][1][r]) ? own : given;
        };
        // The two halves' sums of a row, over dO's tile: written after the last dp has come from it.
        float (*sums)[2][BT] = reinterpret_cast<float (*)[2][BT]>(sm.own[1]);
        const float c = scale * kLog2e;
        const uint64_t c2 = pair(c, c), nl2 = pair(-l2, -l2), nd2 = pair(-dl, -dl);
        uint64_t sum2 = 0;   // of p dp, the row's own delta
        bool ok = true;
        if (n == 1) {
            // Both barriers are for every warp, whether its waits ran out or not.
            const uint32_t t_s = tmem + lane_off + 64 * half;
            ok = warp_wait(stall == BDLA_STALL_EPILOGUE ? &sm.never : &sm.s_full[0], 0u, &sm.wait_ns, abort_flag) &&
                 warp_wait(&sm.dp_full, 0u, &sm.wait_ns, abort_flag);
            uint32_t x[2][32], y[2][32];
            float sum = 0.0f;
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    tmem_ld32(t_s + 32 * k, x[k]);
                    tmem_ld32(t_dp + lane_off + 64 * half + 32 * k, y[k]);
                }
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int m = 0; m < 32; ++m) {
                        const bool out = 64 * half + 32 * k + m > r;
                        const float p = out ? 0.0f : ex2(fmaf(__uint_as_float(x[k][m]), c, -l2));
                        x[k][m] = __float_as_uint(p);
                        y[k][m] = out ? 0u : y[k][m];
                        sum += p;
                    }
                sums[0][half][r] = sum;
                if (valid < BT) {
                    clear_rows(sm.ring[Smem::slot(0)], NP, valid, e, kEpi);
                    fence_proxy_async_smem();
                }
            }
            ok = epi_all(ok);
            float own = 0.0f;
            if (ok) {
                sum = sums[0][0][r] + sums[0][1][r];
                const bool whole = fabsf(sum - 1.0f) <= kHalfStep;   // these keys are all that lse has seen
                const float inv = whole ? 1.0f / sum : 1.0f;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int m = 0; m < 32; ++m) {
                        const float w = __uint_as_float(x[k][m]);
                        const float p = whole && w == sum ? 1.0f : w * inv;   // exactly 1 for a lone key
                        x[k][m] = __float_as_uint(p);
                        own = fmaf(p, __uint_as_float(y[k][m]), own);
                    }
                sums[1][half][r] = own;
            }
            ok = epi_all(ok);
            if (ok) {
                own = chosen(sums[1][0][r] + sums[1][1][r]);
                if (half == 0 && r < valid)
                    delta[(int64_t)h * tokens + t] = own;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t u[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float a = __uint_as_float(x[k][2 * i]) * (__uint_as_float(y[k][2 * i]) - own);
                        const float b = __uint_as_float(x[k][2 * i + 1]) * (__uint_as_float(y[k][2 * i + 1]) - own);
                        u[i] = pack_bf16(64 * half + 32 * k + 2 * i > r ? 0.0f : a,
                                         64 * half + 32 * k + 2 * i + 1 > r ? 0.0f : b);
                    }
                    tmem_st16(t_s + 16 * k, u);
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&sm.ready[0][k]);
                }
            }
        }
        for (int j = 0; j < n && n > 1; ++j) {
            const bool hook = stall == BDLA_STALL_EPILOGUE && j == stall_at;
            const uint32_t t_s = tmem + BT * (j & 1) + lane_off + 64 * half;
            ok = warp_wait(hook ? &sm.never : &sm.s_full[j & 1], hook ? 0u : (uint32_t)((j >> 1) & 1), &sm.wait_ns, abort_flag);
            if (!ok)
                break;
            tc_fence_after();
            uint32_t x[2][32], y[2][32];
            tmem_ld32(t_s, x[0]);
            tmem_ld32(t_s + 32, x[1]);
            ok = warp_wait(&sm.dp_full, j & 1, &sm.wait_ns, abort_flag);
            if (!ok)
                break;
            tc_fence_after();
            tmem_ld32(t_dp + lane_off + 64 * half, y[0]);
            tmem_ld32(t_dp + lane_off + 64 * half + 32, y[1]);
            tmem_ld_wait();
            tc_fence_before();
            mbar_arrive(&sm.dp_free);
            const bool diag = j == n - 1;
            if (diag && valid < BT) {
                // dq sums over the diagonal tile's keys: clear those past the end (S has read them)
                clear_rows(sm.ring[Smem::slot(2 * j)], NP, valid, e, kEpi);
                fence_proxy_async_smem();
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int m = 0; m < 32; m += 2) {
                    float a, b;
                    unpair(fma2(pair(__uint_as_float(x[k][m]), __uint_as_float(x[k][m + 1])), c2, nl2), a, b);
                    x[k][m] = __float_as_uint(ex2(a));
                    x[k][m + 1] = __float_as_uint(ex2(b));
                }
                if (diag) {   // p to 0, and dp as well: 0 times another document's NaN
#pragma unroll
                    for (int m = 0; m < 32; ++m) {
                        const bool out = 64 * half + 32 * k + m > r;
                        x[k][m] = out ? 0u : x[k][m];
                        y[k][m] = out ? 0u : y[k][m];
                    }
                }
#pragma unroll
                for (int m = 0; m < 32; m += 2) {
                    const uint64_t p2 = pair(__uint_as_float(x[k][m]), __uint_as_float(x[k][m + 1]));
                    const uint64_t d2 = pair(__uint_as_float(y[k][m]), __uint_as_float(y[k][m + 1]));
                    float a, b;
                    sum2 = fma2(p2, d2, sum2);
                    unpair(mul2(p2, add2(d2, nd2)), a, b);
                    y[k][m] = __float_as_uint(a);
                    y[k][m + 1] = __float_as_uint(b);
                }
                uint32_t u[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    u[i] = pack_bf16(__uint_as_float(y[k][2 * i]), __uint_as_float(y[k][2 * i + 1]));
                tmem_st16(t_s + 16 * k, u);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&sm.ready[j & 1][k]);
            }
        }
        if (n > 1) {
            float a, b;
            unpair(sum2, a, b);
            if (ok)
                sums[1][half][r] = a + b;
            // every warp comes here, after its last tile or a wait that ran out
            if (epi_all(ok) && half == 0 && r < valid)
                delta[(int64_t)h * tokens + t] = chosen(sums[1][0][r] + sums[1][1][r]);
        }
        if (ok)
            ok = warp_wait(&sm.done, 0, &sm.wait_ns, abort_flag);
        if (ok && half < NP) {
            tc_fence_after();
            // 64 features a half, staged in the query tile (read by now)
            store_rows64(t_dq + lane_off + 64 * half, scale, sm.own[0] + half * kPanel + q4 * 4096,
                         dq + ((size_t)(span.start + 32 * q4) * Hq + h) * D + 64 * half, (size_t)Hq * D, valid - 32 * q4,
                         lane);
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(st, BDLA_ERR_TIMEOUT, 0x22u);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- dk, dv
// Tensor memory: S^T (p over it), dp^T (ds over it), dv, dk.  The two halves of
// a tile's work alternate with the tensor cores: dv of t and S^T of t + 1 run
// while ds of t is formed, dk of t and dp^T of t + 1 while p of t + 1 is.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_dkv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                const float *lse, const float *delta, const int32_t *__restrict__ cu,
                int n_docs, int T, int64_t tokens, int Hk, int group, float scale, __nv_bfloat16 *__restrict__ dk,
                __nv_bfloat16 *__restrict__ dv, float *__restrict__ part, DeviceStatus *st, uint64_t wait_ns, int stall)
{
    using Smem = BwdSmem<D>;
    constexpr int NP = Smem::kPanels;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Early key tiles, which the most queries see, first.  With `part` a CTA takes one query head of the group alone.
    const int units = part != nullptr ? Hk * group : Hk, unit = blockIdx.x % units;
    const int kh = part != nullptr ? unit / group : unit, h0 = part != nullptr ? unit : kh * group;
    const SegSpan span = seg_span(cu, T, tokens, n_docs, (int)(blockIdx.x / units), 1);
    const bool aligned = (smem_u32(smem_raw) & 1023u) == 0u;
    next_may_start();
    if (!span.valid || span.len <= 0 || !aligned) {
        wait_for_previous();
        if (tid == 0 && !aligned)
            set_status(st, BDLA_ERR_DEVICE, 0xA11u);
        return;
    }
    const int64_t doc_len = doc_span(cu, span.n, T).len;
    const int nq = (int)((doc_len + BT - 1) / BT) - span.blk_base;   // query tiles from the diagonal on
    const int n = part != nullptr ? nq : nq * group;                 // of every head of the group in turn
    const int stall_at = n > 1 ? 1 : 0;
    setup(sm, tid, wait_ns);
    wait_for_previous();   // delta; ahead of every bounded wait, none of which is to count the first kernel's time
    const uint32_t tmem = sm.tmem_base, t_dp = tmem + BT, t_dv = tmem + 2 * BT, t_dk = tmem + 3 * BT;
    volatile int *abort_flag = &sm.abort_flag;

    if (warp == 0) {
        if (lane == 0) {
            mbar_arrive_expect_tx(&sm.full_own, 2u * Smem::kTile);
            for (int p = 0; p < NP; ++p) {
                tma_load_3d(sm.own[0] + p * kPanel, &tk, &sm.full_own, p * 64, kh, (int)span.start);
                tma_load_3d(sm.own[1] + p * kPanel, &tv, &sm.full_own, p * 64, kh, (int)span.start);
            }
            run_loader(sm, 2 * n, stall == BDLA_STALL_PRODUCER ? 2 * stall_at : -1, st, [&](int it, int s) {
                const int g = (it >> 1) / nq, i = (it >> 1) % nq;
                for (int p = 0; p < NP; ++p)
                    tma_load_3d(sm.ring[s] + p * kPanel, (it & 1) ? &tdo : &tq, &sm.full[s], p * 64, h0 + g,
                                (int)(span.start + (int64_t)i * BT));
            });
        }
    } else if (warp == 1) {
        const uint64_t k = rows_desc(smem_u32(sm.own[0])), v = rows_desc(smem_u32(sm.own[1]));
        auto tile = [&](int it) { return smem_u32(sm.ring[Smem::slot(it)]); };
        auto landed = [&](int it) { return warp_wait(&sm.full[Smem::slot(it)], Smem::turn(it) & 1, &sm.wait_ns, abort_flag); };
        auto issue_s = [&](int t) {
            if (!landed(2 * t))
                return false;
            tc_fence_after();
            if (elect_one()) {
                mma_rows<D>(tmem, k, rows_desc(tile(2 * t)));
                umma_commit(&sm.s_full[0]);
            }
            __syncwarp();
            return true;
        };
        auto issue_dp = [&](int t) {
            if (!landed(2 * t + 1))
                return false;
            tc_fence_after();
            if (elect_one()) {
                mma_rows<D>(t_dp, v, rows_desc(tile(2 * t + 1)));
                umma_commit(&sm.dp_full);
            }
            __syncwarp();
            return true;
        };
        bool ok = warp_wait(&sm.full_own, 0, &sm.wait_ns, abort_flag) && issue_s(0) && issue_dp(0);
        for (int t = 0; ok && t < n; ++t) {
            const bool hook = stall == BDLA_STALL_MMA && t == stall_at;
            ok = warp_wait(hook ? &sm.never : &sm.ready[0][0], hook ? 0u : (uint32_t)(t & 1), &sm.wait_ns, abort_flag);
            if (!ok)
                break;
            tc_fence_after();
            const uint64_t g = sum_desc(tile(2 * t + 1)), q = sum_desc(tile(2 * t));
            if (elect_one())
                mma_sum_part<D, 0>(t_dv, tmem, g, t > 0);
            __syncwarp();
            if (!(ok = warp_wait(&sm.ready[0][1], t & 1, &sm.wait_ns, abort_flag)))
                break;
            tc_fence_after();
            if (elect_one()) {
                mma_sum_part<D, 1>(t_dv, tmem, g, true);
                umma_commit(&sm.empty[Smem::slot(2 * t + 1)]);
            }
            __syncwarp();
            if (t + 1 < n && !(ok = issue_s(t + 1)))
                break;
            if (!(ok = warp_wait(&sm.ready[1][0], t & 1, &sm.wait_ns, abort_flag)))
                break;
            tc_fence_after();
            if (elect_one())
                mma_sum_part<D, 0>(t_dk, t_dp, q, t > 0);
            __syncwarp();
            if (!(ok = warp_wait(&sm.ready[1][1], t & 1, &sm.wait_ns, abort_flag)))
                break;
            tc_fence_after();
            if (elect_one()) {
                mma_sum_part<D, 1>(t_dk, t_dp, q, true);
                umma_commit(&sm.empty[Smem::slot(2 * t)]);
                if (t == n - 1)
                    umma_commit(&sm.done);
            }
            __syncwarp();
            if (t + 1 < n)
                ok = issue_dp(t + 1);
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(st, BDLA_ERR_TIMEOUT, 0x23u);
        }
        if (elect_one())
            umma_commit(&sm.drain);
        __syncwarp();
        mbar_wait(&sm.drain, 0, kDrainNs);
    } else {
        const int half = (warp - 2) >> 2, q4 = warp & 3, r = 32 * q4 + lane, e = 128 * half + r;
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const uint32_t t_s = tmem + lane_off + 64 * half, t_d = t_dp + lane_off + 64 * half;
        const float c = scale * kLog2e;
        const uint64_t c2 = pair(c, c);
        // this thread's entry of a query tile's lse (half 0) or delta (half 1), fetched one tile ahead
        const float *src = half ? delta : lse;
        auto fetch = [&](int t) {
            const int g = t / nq, i = t % nq;
            const int64_t row = (int64_t)(span.blk_base + i) * BT + r;
            if (row >= doc_len)
                return 0.0f;
            const float x = src[(int64_t)(h0 + g) * tokens + span.doc_start + row];
            return half ? -x : x * -kLog2e;
        };
        float next = fetch(0);
        bool ok = true;
        for (int t = 0; t < n; ++t) {
            const bool hook = stall == BDLA_STALL_EPILOGUE && t == stall_at;
            const int i_tile = t % nq;
            // queries of the tile inside the document
            const int valid = (int)(doc_len - (int64_t)(span.blk_base + i_tile) * BT);
            sm.col[t & 1][half][r] = next;
            // Every thread is done with the entries of two tiles before.  A warp whose wait ran out skips the
            // rest of its tile and leaves with all the others here.
            if (!(ok = epi_all(ok)))
                break;
            if (t + 1 < n)
                next = fetch(t + 1);
            ok = warp_wait(hook ? &sm.never : &sm.s_full[0], hook ? 0u : (uint32_t)(t & 1), &sm.wait_ns, abort_flag);
            if (ok && valid < BT) {
                // dv and dk sum over this tile's queries: clear those past the end once S and dp have read them
                ok = warp_wait(&sm.dp_full, t & 1, &sm.wait_ns, abort_flag);
                if (ok) {
                    clear_rows(sm.ring[Smem::slot(2 * t)], NP, valid, e, kEpi);
                    clear_rows(sm.ring[Smem::slot(2 * t + 1)], NP, valid, e, kEpi);
                    fence_proxy_async_smem();
                }
            }
            const bool mask = i_tile == 0 || valid < BT;   // the diagonal, or queries past the end
            float p[64];
            if (ok) {
                tc_fence_after();
                uint32_t x[2][32];
                tmem_ld32(t_s, x[0]);
                tmem_ld32(t_s + 32, x[1]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int m = 0; m < 32; m += 4) {
                        const ulonglong2 l4 = *reinterpret_cast<const ulonglong2 *>(&sm.col[t & 1][0][64 * half + 32 * k + m]);
                        float a, b;
                        unpair(fma2(pair(__uint_as_float(x[k][m]), __uint_as_float(x[k][m + 1])), c2, l4.x), a, b);
                        p[32 * k + m] = ex2(a);
                        p[32 * k + m + 1] = ex2(b);
                        unpair(fma2(pair(__uint_as_float(x[k][m + 2]), __uint_as_float(x[k][m + 3])), c2, l4.y), a, b);
                        p[32 * k + m + 2] = ex2(a);
                        p[32 * k + m + 3] = ex2(b);
                    }
                    if (mask) {
#pragma unroll
                        for (int m = 32 * k; m < 32 * k + 32; ++m) {
                            const int q = 64 * half + m;
                            p[m] = (i_tile == 0 && q < r) || q >= valid ? 0.0f : p[m];
                        }
                    }
                    uint32_t u[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        u[i] = pack_bf16(p[32 * k + 2 * i], p[32 * k + 2 * i + 1]);
                    tmem_st16(t_s + 16 * k, u);
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&sm.ready[0][k]);
                }
            }
            if (ok)
                ok = warp_wait(&sm.dp_full, t & 1, &sm.wait_ns, abort_flag);
            if (!ok) {
                *abort_flag = 1;
                continue;
            }
            tc_fence_after();
            uint32_t y[2][32];
            tmem_ld32(t_d, y[0]);
            tmem_ld32(t_d + 32, y[1]);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int m = 0; m < 32; m += 4) {
                    const ulonglong2 d4 = *reinterpret_cast<const ulonglong2 *>(&sm.col[t & 1][1][64 * half + 32 * k + m]);
                    float a, b;
                    unpair(mul2(pair(p[32 * k + m], p[32 * k + m + 1]),
                                add2(pair(__uint_as_float(y[k][m]), __uint_as_float(y[k][m + 1])), d4.x)), a, b);
                    y[k][m] = __float_as_uint(a);
                    y[k][m + 1] = __float_as_uint(b);
                    unpair(mul2(pair(p[32 * k + m + 2], p[32 * k + m + 3]),
                                add2(pair(__uint_as_float(y[k][m + 2]), __uint_as_float(y[k][m + 3])), d4.y)), a, b);
                    y[k][m + 2] = __float_as_uint(a);
                    y[k][m + 3] = __float_as_uint(b);
                }
                if (mask) {   // 0 times another document's NaN
#pragma unroll
                    for (int m = 0; m < 32; ++m) {
                        const int q = 64 * half + 32 * k + m;
                        y[k][m] = (i_tile == 0 && q < r) || q >= valid ? 0u : y[k][m];
                    }
                }
                uint32_t u[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    u[i] = pack_bf16(__uint_as_float(y[k][2 * i]), __uint_as_float(y[k][2 * i + 1]));
                tmem_st16(t_d + 16 * k, u);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&sm.ready[1][k]);
            }
        }
        if (ok)
            ok = warp_wait(&sm.done, 0, &sm.wait_ns, abort_flag);
        if (ok) {
            tc_fence_after();
            const int rows = (int)span.len - 32 * q4;
            const size_t row0 = ((size_t)(span.start + 32 * q4) * Hk + kh) * D;
            unsigned char *stage = sm.own[half] + q4 * 4096;   // K and V have been read
            // 128 features: each half takes 64 of both; 64 features: one tensor each
            const int f = NP == 2 ? 64 * half : 0;
            if (part != nullptr) {   // fp32 rows [2][tokens][Hq][D]: dv, then dk
                const size_t rowp = ((size_t)(span.start + 32 * q4) * units + unit) * D + f, all = (size_t)tokens * units * D;
                if (NP == 2 || half == 0)
                    store_rows64_f32(t_dv + lane_off + f, stage, part + rowp, (size_t)units * D, rows, lane);
                if (NP == 2 || half == 1)
                    store_rows64_f32(t_dk + lane_off + f, stage, part + all + rowp, (size_t)units * D, rows, lane);
            } else {
                if (NP == 2 || half == 0)
                    store_rows64(t_dv + lane_off + f, 1.0f, stage, dv + row0 + f, (size_t)Hk * D, rows, lane);
                if (NP == 2 || half == 1)
                    store_rows64(t_dk + lane_off + f, scale, stage, dk + row0 + f, (size_t)Hk * D, rows, lane);
            }
        }
        if (!ok) {
            *abort_flag = 1;
            if (lane == 0)
                set_status(st, BDLA_ERR_TIMEOUT, 0x24u);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem, 512);
}

// dv and dk of a key head from the fp32 sums of its query heads, in their order;
// four features a thread.
__global__ void __launch_bounds__(256)
dkv_join_kernel(const float *part, int64_t n4, int d4, int group, float scale, __nv_bfloat16 *__restrict__ dv,
                __nv_bfloat16 *__restrict__ dk)
{
    wait_for_previous();
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;   // float4 of [tokens][Hk][d]
    if (e >= n4)
        return;
    const int64_t row = e / d4;   // token and key head
    const float4 *src = reinterpret_cast<const float4 *>(part) + (blockIdx.y ? n4 * group : 0) + row * group * d4 + e % d4;
    float4 s = src[0];
    for (int g = 1; g < group; ++g) {
        const float4 x = src[(int64_t)g * d4];
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
    }
    const float f = blockIdx.y ? scale : 1.0f;
    *reinterpret_cast<uint2 *>((blockIdx.y ? dk : dv) + 4 * e) = make_uint2(pack_bf16(s.x * f, s.y * f), pack_bf16(s.z * f, s.w * f));
}

template <int D>
cudaError_t go(const AttnProblem &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
               const CUtensorMap &mdo, const __nv_bfloat16 *o, const __nv_bfloat16 *dO, const float *lse,
               __nv_bfloat16 *dq, __nv_bfloat16 *dk, __nv_bfloat16 *dv, float *delta, float *part)
{
    const size_t smem = sizeof(BwdSmem<D>);
    cudaError_t err = cudaFuncSetAttribute(attn_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(attn_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess)
        return err;
    const int64_t n_slots = (p.tokens + BT - 1) / BT + p.n_docs;
    if (n_slots * p.Hq > INT32_MAX)
        return cudaErrorInvalidValue;
    const uint64_t ns = g_wait_ns.load();
    const int stall = g_test_stall[BDLA_KERNEL_ATTN_BWD].load(), group = p.Hq / p.Hk;
    attn_dq_kernel<D><<<(unsigned)(n_slots * p.Hq), kThreads, smem, p.stream>>>(
        mq, mk, mv, mdo, o, dO, lse, p.cu, p.n_docs, p.T, p.tokens, p.Hq, group, (int)n_slots, p.scale, dq, delta, p.st,
        ns, stall);
    err = cudaGetLastError();
    if (err != cudaSuccess)
        return err;
    err = launch_second(attn_dkv_kernel<D>, (unsigned)(n_slots * (part ? p.Hq : p.Hk)), kThreads, smem, p.stream, mq, mk, mv,
                        mdo, lse, delta, p.cu, p.n_docs, p.T, p.tokens, p.Hk, group, p.scale, dk, dv, part, p.st, ns, stall);
    if (err != cudaSuccess || part == nullptr)
        return err;
    const int64_t n4 = p.tokens * p.Hk * D / 4;
    return launch_second(dkv_join_kernel, dim3((unsigned)((n4 + 255) / 256), 2), 256, 0, p.stream, part, n4, D / 4, group,
                         p.scale, dv, dk);
}

}  // namespace

// Key tiles of all heads that leave SMs idle while each walks the queries of a
// whole group: one CTA a query head then, and fp32 sums to join (1537 tokens, 3
// heads to a key head: 43 us without).
size_t attn_bwd_part_floats(const bdla_attn_dims &d, int n_docs)
{
    const int64_t tokens = (int64_t)d.B * d.T, tiles = tokens / BT + n_docs;
    return d.Hq > d.Hk && tiles * d.Hk < sm_count() ? (size_t)tokens * d.Hq * d.d * 2 : 0;
}

cudaError_t launch_attn_bwd(const AttnProblem &p, const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                            const __nv_bfloat16 *v, const __nv_bfloat16 *o, const float *lse,
                            const __nv_bfloat16 *dO, __nv_bfloat16 *dq, __nv_bfloat16 *dk, __nv_bfloat16 *dv,
                            float *delta, float *part)
{
    KernelMark mark_(BDLA_KERNEL_ATTN_BWD, p.stream);
    if (p.tokens == 0)
        return launch_doc_report(p);
    CUtensorMap mq, mk, mv, mdo;
    if (!make_token_map(&mq, q, p.d, p.Hq, p.tokens) || !make_token_map(&mk, k, p.d, p.Hk, p.tokens) ||
        !make_token_map(&mv, v, p.d, p.Hk, p.tokens) || !make_token_map(&mdo, dO, p.d, p.Hq, p.tokens))
        return cudaErrorInvalidValue;
    return p.d == 64 ? go<64>(p, mq, mk, mv, mdo, o, dO, lse, dq, dk, dv, delta, part)
                     : go<128>(p, mq, mk, mv, mdo, o, dO, lse, dq, dk, dv, delta, part);
}

}  // namespace bdla
