// What the softmax attention kernels share: tile sizes, the base-2
// exponential, the check of packed offsets, and the store of 32 rows.
#pragma once

#include "bdla_attn_internal.h"
#include "bdla_sm100.cuh"

namespace bdla {

bool make_token_map(CUtensorMap *map, const void *ptr, int d, int H, int64_t tokens);

namespace attn {

constexpr int BT = 128;              // rows of a tile
constexpr uint32_t kPanel = 16384;   // 128 rows x 128 swizzled bytes (64 features)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// drains of a CTA's own copies and MMAs before it exits keep the full limit
constexpr uint64_t kDrainNs = kDefaultWaitNs;
constexpr size_t kMaxSmem = 232448;   // 227 KB opt-in shared memory per CTA

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Packed offsets: cu[0] = 0, non-decreasing, cu[n_docs] = tokens; the first
// bad document is recorded.  Run by the threads of one CTA.
__device__ __forceinline__ void check_offsets(const int32_t *cu, int n_docs, int64_t tokens, DeviceStatus *st)
{
    for (int n = threadIdx.x; n < n_docs; n += blockDim.x)
        if (cu[n + 1] < cu[n] || (n == 0 && cu[0] != 0) || (n == n_docs - 1 && cu[n_docs] != tokens))
            set_status(st, BDLA_ERR_DEVICE, (unsigned)n);
}

// All lanes' waits, as one answer for the warp (the tensor-memory accesses
// that follow need whole warps).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const uint64_t *limit, volatile int *abort_flag)
{
    const bool ok = sm100::mbar_wait_lim(bar, parity, limit) && !*abort_flag;
    return __all_sync(0xffffffffu, ok);
}

// Zeroes rows [first, 128) of a tile of `panels` panels; `i` of `n` threads.
// Whole rows, so the swizzle does not matter.
__device__ __forceinline__ void clear_rows(unsigned char *tile, int panels, int first, int i, int n)
{
    const int per = (BT - first) * 8;
    for (int e = i; e < per * panels; e += n) {
        const int p = e / per, f = e % per;
        *reinterpret_cast<uint4 *>(tile + p * kPanel + (first + (f >> 3)) * 128 + (f & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// One warp: 64 columns of its 32 accumulator rows (TMEM address `t`), times
// `f`, as bf16 through `stage` (4096 bytes of the warp's own) to rows of
// `stride` elements at dst; only the first n_valid rows are written.
__device__ __forceinline__ void store_rows64(uint32_t t, float f, unsigned char *stage, __nv_bfloat16 *dst, size_t stride,
                                             int n_valid, int lane)
{
    uint4 *s4 = reinterpret_cast<uint4 *>(stage);
    uint32_t y[2][32];
    sm100::tmem_ld32(t, y[0]);
    sm100::tmem_ld32(t + 32, y[1]);
    sm100::tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = sm100::pack_bf16(__uint_as_float(y[k >> 2][8 * (k & 3) + 2 * i]) * f,
                                    __uint_as_float(y[k >> 2][8 * (k & 3) + 2 * i + 1]) * f);
        s4[lane * 8 + (k ^ (lane & 7))] = make_uint4(v[0], v[1], v[2], v[3]);
    }
    __syncwarp();
#pragma unroll
    for (int it = 0; it < 8; ++it) {
        const int row = 4 * it + (lane >> 3), c8 = lane & 7;
        const uint4 v = s4[row * 8 + (c8 ^ (row & 7))];
        if (row < n_valid)
            *reinterpret_cast<uint4 *>(dst + (size_t)row * stride + 8 * c8) = v;
    }
    __syncwarp();
}

}  // namespace attn
}  // namespace bdla
