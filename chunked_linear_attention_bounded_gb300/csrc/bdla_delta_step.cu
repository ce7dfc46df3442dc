// Recurrent steps of the gated delta rule from resident states: the serving
// side of the rule that bdla_delta.cu evaluates chunk by chunk.  For each
// sequence and head, token by token,
//     r = S^T k,  e = v - g r,  S <- g S + beta k e^T,  o = S^T q
// with g = e^lambda.  Both sums over the rows of S are taken from the state as
// it was: o = g (S^T q) + beta (k . q) e, so a token is one pass over S.
//
// A column of S depends on no other, so a warp takes 32 columns of one head and
// holds them in registers for all tokens of the call: the state is read once
// and written once, whatever the number of tokens.  Lane (row group, four
// columns): the loads of a warp cover whole 128-byte lines, the sums over the
// rows end in two shuffle steps, and there is no shared memory and no barrier.
#include "bdla_attn_sm100.cuh"

namespace bdla {

namespace {

using attn::fma2;
using attn::mul2;
using attn::pair;
using attn::unpair;
using sm100::bf16_hi;
using sm100::bf16_lo;

constexpr int kWarps = 4;
constexpr int kCols = 32;                    // columns of a warp
constexpr int kColLanes = kCols / 4;
constexpr int kRowGroups = 32 / kColLanes;   // 4
constexpr int kRun = 8;                      // consecutive rows of a lane: 16 bytes of k and q

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
    int B, T, H, dv;
    DeviceStatus *st;
};

// Sum over the row groups of a warp.
__device__ __forceinline__ float over_rows(float x)
{
#pragma unroll
    for (int w = kColLanes; w < 32; w <<= 1)
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

template <int DK>
__global__ void __launch_bounds__(32 * kWarps)
delta_step_kernel(const __grid_constant__ StepParams p)
{
    constexpr int R = DK / kRowGroups;   // rows of a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slices = p.dv / kCols;
    const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
    if (item >= (int64_t)p.B * p.H * slices)
        return;
    const int64_t unit = item / slices;
    const int b = (int)(unit / p.H), h = (int)(unit - (int64_t)b * p.H);
    const int rg = lane / kColLanes, j = (int)(item - unit * slices) * kCols + 4 * (lane % kColLanes);
    // token t of this sequence and head: element t * H + head of the tensors
    const int64_t head = (int64_t)b * p.T * p.H + h;

    int slot = p.slots != nullptr ? p.slots[b] : b;
    int count = p.counts != nullptr ? p.counts[b] : p.T;
    if (slot < -1 || (p.slots != nullptr && slot >= p.n_slots)) {
        if (lane == 0)
            set_status(p.st, BDLA_ERR_DEVICE, (unsigned)b);
        slot = -1;
    }
    // the lane's rows: runs of eight, the row groups' runs in turn
    const auto row = [&](int i) { return i / kRun * (kRun * kRowGroups) + rg * kRun + i % kRun; };
    float *S = p.state + (int64_t)(slot < 0 ? 0 : slot) * p.H * DK * p.dv + (int64_t)h * DK * p.dv + j;
    uint64_t s[R][2];
    if (slot >= 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float4 x = __ldcs(reinterpret_cast<const float4 *>(S + (int64_t)row(i) * p.dv));
            s[i][0] = pair(x.x, x.y);
            s[i][1] = pair(x.z, x.w);
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
                store_out(p, (head + (int64_t)t * p.H) * p.dv + j, 0.0f, 0.0f, 0.0f, 0.0f);
        return;
    }
    const auto store_state = [&] {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float4 x;
            unpair(s[i][0], x.x, x.y);
            unpair(s[i][1], x.z, x.w);
            __stcs(reinterpret_cast<float4 *>(S + (int64_t)row(i) * p.dv), x);
        }
    };

    for (int t = 0; t < p.T; ++t) {
        const int64_t at = head + (int64_t)t * p.H;
        uint4 kr[R / kRun], qr[R / kRun];
#pragma unroll
        for (int c = 0; c < R / kRun; ++c) {
            kr[c] = *reinterpret_cast<const uint4 *>(p.k + at * DK + row(c * kRun));
            qr[c] = *reinterpret_cast<const uint4 *>(p.q + at * DK + row(c * kRun));
        }
        const uint2 vr = *reinterpret_cast<const uint2 *>(p.v + at * p.dv + j);
        const float g = expf(log_decay(p.a[at], p.b, p.mode)), beta = p.beta[at];
        uint64_t r2[2] = {0, 0}, o2[2] = {0, 0};
        float kq = 0.0f;
#pragma unroll
        for (int c = 0; c < R / kRun; ++c) {
            const uint32_t kw[4] = {kr[c].x, kr[c].y, kr[c].z, kr[c].w}, qw[4] = {qr[c].x, qr[c].y, qr[c].z, qr[c].w};
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                const float kf = e & 1 ? bf16_hi(kw[e >> 1]) : bf16_lo(kw[e >> 1]);
                const float qf = e & 1 ? bf16_hi(qw[e >> 1]) : bf16_lo(qw[e >> 1]);
                kq = fmaf(kf, qf, kq);
                const uint64_t k2 = pair(kf, kf), q2 = pair(qf, qf);
                const int i = c * kRun + e;
                r2[0] = fma2(k2, s[i][0], r2[0]);
                r2[1] = fma2(k2, s[i][1], r2[1]);
                o2[0] = fma2(q2, s[i][0], o2[0]);
                o2[1] = fma2(q2, s[i][1], o2[1]);
            }
        }
        float r[4], o[4];
        unpair(r2[0], r[0], r[1]);
        unpair(r2[1], r[2], r[3]);
        unpair(o2[0], o[0], o[1]);
        unpair(o2[1], o[2], o[3]);
        kq = over_rows(kq);
        const float v[4] = {bf16_lo(vr.x), bf16_hi(vr.x), bf16_lo(vr.y), bf16_hi(vr.y)};
        float w[4];   // beta e
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = beta * fmaf(-g, over_rows(r[e]), v[e]);
            o[e] = fmaf(g, over_rows(o[e]), kq * w[e]);
        }
        if (rg == 0)
            store_out(p, at * p.dv + j, o[0], o[1], o[2], o[3]);
        const uint64_t g2 = pair(g, g), w2[2] = {pair(w[0], w[1]), pair(w[2], w[3])};
        if (t == count && count > 0)
            store_state();
#pragma unroll
        for (int c = 0; c < R / kRun; ++c) {
            const uint32_t kw[4] = {kr[c].x, kr[c].y, kr[c].z, kr[c].w};
#pragma unroll
            for (int e = 0; e < kRun; ++e) {
                const float kf = e & 1 ? bf16_hi(kw[e >> 1]) : bf16_lo(kw[e >> 1]);
                const uint64_t k2 = pair(kf, kf);
                const int i = c * kRun + e;
                s[i][0] = fma2(g2, s[i][0], mul2(k2, w2[0]));
                s[i][1] = fma2(g2, s[i][1], mul2(k2, w2[1]));
            }
        }
    }
    if (count == p.T)
        store_state();
}

}  // namespace

cudaError_t launch_delta_step(const bdla_dims &d, const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                              const __nv_bfloat16 *v, const float *a, const float *beta, float b, int mode, float *state,
                              const int32_t *slots, int n_slots, const int32_t *counts, void *o, int o_f32,
                              DeviceStatus *st, cudaStream_t stream)
{
    const StepParams p = {q, k, v, a, beta, b, mode, state, slots, counts, n_slots, o, o_f32, d.B, d.T, d.H, d.dv, st};
    const int64_t items = (int64_t)d.B * d.H * (d.dv / kCols), grid = (items + kWarps - 1) / kWarps;
    if (grid > INT32_MAX)
        return cudaErrorInvalidValue;
    if (d.dk == 64)
        delta_step_kernel<64><<<(unsigned)grid, 32 * kWarps, 0, stream>>>(p);
    else
        delta_step_kernel<128><<<(unsigned)grid, 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace bdla
