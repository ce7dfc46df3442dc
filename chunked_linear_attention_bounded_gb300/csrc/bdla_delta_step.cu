// Recurrent steps of the gated delta rule from resident states: the serving
// side of the rule that bdla_delta.cu evaluates chunk by chunk.  For each
// sequence and head, token by token,
//     r = S^T k,  e = v - g r,  S <- g S + beta k e^T,  o = S^T q
// with g = e^lambda.  Both sums over the rows of S are taken from the state as
// it was: o = g (S^T q) + beta (k . q) e, so a token is one pass over S.
//
// A column of S depends on no other, so a warp takes 16 columns of one head (32
// where the state has 64 rows) and holds them in registers for all tokens of the
// call, 16 rows and 4 columns a lane: the state is read once and written once,
// whatever the number of tokens.  The sums over the rows end in two or three
// shuffle steps; a warp shares its k and q through shared memory and nothing with
// other warps, so a CTA is one warp and there is no barrier.
//
// One token: bound by HBM, 256 sequences of 32 heads of 128 x 128 in 164 us (6.5
// TB/s); one sequence 2.5 us (CTAs of four warps with 32 columns each: 4.2).  Many
// tokens: bound by fp32 arithmetic (8 paired operations a row, token and four
// columns; 48 x 33 tokens of 16 heads of 128 x 64: 65 us in two rounds of warps).
// 128 registers a thread are what 16 warps an SM allow; 96 spill in the token
// loop (95 us), and 32 rows a lane with 168 registers spill as well (62, but 3.1 for
// one sequence and 10.0 for 37 x 5 tokens, where 16 rows take 7.9).
#include "bdla_attn_sm100.cuh"
#include "bdla_cache.cuh"

namespace bdla {

namespace {

using attn::fma2;
using attn::mul2;
using attn::pair;
using attn::unpair;
using sm100::bf16_hi;
using sm100::bf16_lo;

constexpr int kRun = 8;    // consecutive rows of a lane: 16 bytes of k and q
constexpr int kHeld = 16;  // rows of a lane

// How a warp divides its columns of a state with DK rows.
template <int DK> struct Split {
    static constexpr int kRowGroups = DK / kHeld;        // 8 or 4
    static constexpr int kColLanes = 32 / kRowGroups;    // four columns each
    static constexpr int kCols = 4 * kColLanes;
};

struct StepParams {
    const __nv_bfloat16 *q, *k, *v;
    const float *a, *beta;
    float b;
    int mode;
    float *state;
    const int32_t *slots, *counts;
    int n_slots;
    void *o;
    int o_f32;
    int B, T, H;
    DeviceStatus *st;
};

// Sum over the row groups of a warp.
template <int DK> __device__ __forceinline__ float over_rows(float x)
{
#pragma unroll
    for (int w = Split<DK>::kColLanes; w < 32; w <<= 1)
        x += __shfl_xor_sync(0xffffffffu, x, w);
    return x;
}

__device__ __forceinline__ void store_out(const StepParams &p, int64_t at, float x0, float x1, float x2, float x3)
{
    if (p.o_f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at) = make_float4(x0, x1, x2, x3);
    else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + at) =
            make_uint2(sm100::pack_bf16(x0, x1), sm100::pack_bf16(x2, x3));
}

template <int DK, int DV>
__global__ void __launch_bounds__(32, 16)
delta_step_kernel(const __grid_constant__ StepParams p)
{
    constexpr int R = kHeld, kRowGroups = Split<DK>::kRowGroups, kColLanes = Split<DK>::kColLanes, kCols = Split<DK>::kCols;
    __shared__ __align__(16) __nv_bfloat16 rows[2][2][DK];   // k and q of a token, and of the next
    const int lane = threadIdx.x;
    constexpr int kSlices = DV / kCols;
    const int64_t item = blockIdx.x, unit = item / kSlices;
    const int b = (int)(unit / p.H), h = (int)(unit - (int64_t)b * p.H);
    const int rg = lane / kColLanes, j = (int)(item - unit * kSlices) * kCols + 4 * (lane % kColLanes);
    // token t of this sequence and head: element t * H + head of the tensors
    const int64_t head = (int64_t)b * p.T * p.H + h;

    int slot = p.slots != nullptr ? p.slots[b] : b;
    int count = p.counts != nullptr ? p.counts[b] : p.T;
    if (slot < -1 || (p.slots != nullptr && slot >= p.n_slots)) {
        if (lane == 0)
            set_status(p.st, BDLA_ERR_DEVICE, (unsigned)b);
        slot = -1;
    }
    // the lane's rows, from its first: runs of eight, the row groups' runs in turn
    const auto row = [](int i) { return i / kRun * (kRun * kRowGroups) + i % kRun; };
    float *S = p.state + (int64_t)(slot < 0 ? 0 : slot) * p.H * DK * DV + (int64_t)h * DK * DV + kRun * rg * DV + j;
    uint64_t s[R][2];
    if (slot >= 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const ulonglong2 x = __ldcs(reinterpret_cast<const ulonglong2 *>(S + row(i) * DV));
            s[i][0] = x.x;
            s[i][1] = x.y;
        }
        // a state that two places of the batch name belongs to the first
        if (p.slots != nullptr) {
            bool taken = false;
            for (int i = lane; i < b; i += 32)
                taken |= p.slots[i] == slot;
            if (__any_sync(0xffffffffu, taken)) {
                if (lane == 0)
                    set_status(p.st, BDLA_ERR_DEVICE, (unsigned)b);
                slot = -1;
            }
        }
    }
    if (count < 0 || count > p.T) {
        if (lane == 0)
            set_status(p.st, BDLA_ERR_DEVICE, (unsigned)b);
        count = 0;
    }
    if (slot < 0) {   // an unused place of the batch, or one that was refused
        if (rg == 0)
            for (int t = 0; t < p.T; ++t)
                store_out(p, (head + (int64_t)t * p.H) * DV + j, 0.0f, 0.0f, 0.0f, 0.0f);
        return;
    }
    const auto store_state = [&] {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            __stcs(reinterpret_cast<ulonglong2 *>(S + row(i) * DV), make_ulonglong2(s[i][0], s[i][1]));
        }
    };

    // A token's inputs are asked for a token ahead: k and q into shared memory, the lane's values, the logit and the
    // strength into registers.
    const auto fetch = [&](int t) {
        if (t < p.T) {
            const int64_t at = (head + (int64_t)t * p.H) * DK;
            constexpr int kPieces = DK / 8;   // 16 bytes each
            const int which = lane / kPieces, x = lane % kPieces * 8;
            if (lane < 2 * kPieces)
                cache::cp16((uint32_t)__cvta_generic_to_shared(&rows[t & 1][which][x]), (which ? p.q : p.k) + at + x, true);
        }
        cache::cp_commit();
    };
    struct Token {
        uint2 v;
        float a, beta;
    };
    const auto load = [&](int t) {
        const int64_t at = head + (int64_t)t * p.H;
        return Token{*reinterpret_cast<const uint2 *>(p.v + at * DV + j), p.a[at], p.beta[at]};
    };
    fetch(0);
    Token next = load(0);
#pragma unroll 1
    for (int t = 0; t < p.T; ++t) {
        const Token tok = next;
        fetch(t + 1);
        if (t + 1 < p.T)
            next = load(t + 1);
        cache::cp_wait<1>();
        __syncwarp();
        const __nv_bfloat16 *ks = rows[t & 1][0], *qs = rows[t & 1][1];
        const float g = expf(log_decay(tok.a, p.b, p.mode));
        uint64_t r2[2] = {0, 0}, o2[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < R / kRun; ++c) {
            const uint4 kr = *reinterpret_cast<const uint4 *>(ks + (c * kRowGroups + rg) * kRun);
            const uint4 qr = *reinterpret_cast<const uint4 *>(qs + (c * kRowGroups + rg) * kRun);
            const uint32_t kw[4] = {kr.x, kr.y, kr.z, kr.w}, qw[4] = {qr.x, qr.y, qr.z, qr.w};
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                const float kf = e & 1 ? bf16_hi(kw[e >> 1]) : bf16_lo(kw[e >> 1]);
                const float qf = e & 1 ? bf16_hi(qw[e >> 1]) : bf16_lo(qw[e >> 1]);
                const uint64_t k2 = pair(kf, kf), q2 = pair(qf, qf);
                const int i = c * kRun + e;
                r2[0] = fma2(k2, s[i][0], r2[0]);
                r2[1] = fma2(k2, s[i][1], r2[1]);
                o2[0] = fma2(q2, s[i][0], o2[0]);
                o2[1] = fma2(q2, s[i][1], o2[1]);
            }
            asm volatile("" ::: "memory");   // the next rows are not read ahead: their registers are the state's
        }
        float r[4], o[4];
        unpair(r2[0], r[0], r[1]);
        unpair(r2[1], r[2], r[3]);
        unpair(o2[0], o[0], o[1]);
        unpair(o2[1], o[2], o[3]);
        // k . q, 2 or 4 features a lane
        float kq = 0.0f;
        {
            const uint32_t *kd = reinterpret_cast<const uint32_t *>(ks), *qd = reinterpret_cast<const uint32_t *>(qs);
#pragma unroll
            for (int i = 0; i < DK / 2; i += 32)
                kq = fmaf(bf16_lo(kd[i + lane]), bf16_lo(qd[i + lane]), fmaf(bf16_hi(kd[i + lane]), bf16_hi(qd[i + lane]), kq));
#pragma unroll
            for (int x = 1; x < 32; x <<= 1)
                kq += __shfl_xor_sync(0xffffffffu, kq, x);
        }
        const float v[4] = {bf16_lo(tok.v.x), bf16_hi(tok.v.x), bf16_lo(tok.v.y), bf16_hi(tok.v.y)};
        float w[4];   // beta e
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = tok.beta * fmaf(-g, over_rows<DK>(r[e]), v[e]);
            o[e] = fmaf(g, over_rows<DK>(o[e]), kq * w[e]);
        }
        if (rg == 0)
            store_out(p, (head + (int64_t)t * p.H) * DV + j, o[0], o[1], o[2], o[3]);
        const uint64_t g2 = pair(g, g), w2[2] = {pair(w[0], w[1]), pair(w[2], w[3])};
        if (t == count && count > 0)
            store_state();
#pragma unroll
        for (int c = 0; c < R / kRun; ++c) {
            const uint4 kr = *reinterpret_cast<const uint4 *>(ks + (c * kRowGroups + rg) * kRun);
            const uint32_t kw[4] = {kr.x, kr.y, kr.z, kr.w};
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                const float kf = e & 1 ? bf16_hi(kw[e >> 1]) : bf16_lo(kw[e >> 1]);
                const uint64_t k2 = pair(kf, kf);
                const int i = c * kRun + e;
                s[i][0] = fma2(g2, s[i][0], mul2(k2, w2[0]));
                s[i][1] = fma2(g2, s[i][1], mul2(k2, w2[1]));
            }
            asm volatile("" ::: "memory");
        }
        __syncwarp();   // k and q have been read: those of the token after the next may take their place
    }
    if (count == p.T)
        store_state();
}

}  // namespace

int64_t delta_step_ctas(const bdla_dims &d)
{
    return (int64_t)d.B * d.H * (d.dv / (d.dk == 64 ? Split<64>::kCols : Split<128>::kCols));
}

cudaError_t launch_delta_step(const bdla_dims &d, const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                              const __nv_bfloat16 *v, const float *a, const float *beta, float b, int mode, float *state,
                              const int32_t *slots, int n_slots, const int32_t *counts, void *o, int o_f32,
                              DeviceStatus *st, cudaStream_t stream)
{
    const StepParams p = {q, k, v, a, beta, b, mode, state, slots, counts, n_slots, o, o_f32, d.B, d.T, d.H, st};
    auto *kern = d.dk == 64 ? (d.dv == 64 ? delta_step_kernel<64, 64> : delta_step_kernel<64, 128>)
                            : (d.dv == 64 ? delta_step_kernel<128, 64> : delta_step_kernel<128, 128>);
    kern<<<(unsigned)delta_step_ctas(d), 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace bdla
