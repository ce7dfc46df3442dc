// What the softmax attention kernels share: tile sizes, paired fp32 arithmetic
// and the base-2 exponential, one row's softmax in tensor memory, the check of
// packed offsets, the launch of a call's second kernel, products of 128-row
// tiles, bounded waits of warps, and the stores of 32 rows.
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

// Two fp32 values in one 64-bit register, and the operations that take both at
// the cost of one.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Softmax of one row in one pass: reference m, the reference times the factor
// c of the scores in base 2 (0 until something has been seen), and the sum of
// the weights e^{(s - m)} so far.
struct RowSoftmax {
    float m = -INFINITY, mc = 0.0f, l = 0.0f;
};

constexpr float kSlack = 8.0f;   // log2 of how far weights may exceed 1

// One thread's 128 scores x (masked ones -inf) into bf16 weights over them in
// tensor memory (t_s), 64 at a time, each half handed over by half_done(0 / 1).
// The reference moves only when a score exceeds it by more than kSlack; the
// output so far (t_o, D columns, none if `first`) is then rescaled there.
template <int D, typename Half>
__device__ __forceinline__ void row_weights(uint32_t (&x)[4][32], float c, uint32_t t_s, uint32_t t_o, bool first,
                                            RowSoftmax &s, Half half_done)
{
    float mx[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        mx[k] = fmaxf(__uint_as_float(x[k][0]), __uint_as_float(x[k][1]));
#pragma unroll
        for (int i = 2; i < 32; i += 2)
            mx[k] = max3(mx[k], __uint_as_float(x[k][i]), __uint_as_float(x[k][i + 1]));
    }
    const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
    const bool move = (top - s.m) * c > kSlack;
    if (__any_sync(0xffffffffu, move)) {
        const float f = !move ? 1.0f : s.m == -INFINITY ? 0.0f : ex2(s.mc - top * c);
        if (move) {
            s.m = top;
            s.mc = top * c;
        }
        s.l *= f;
        if (!first) {
#pragma unroll 1
            for (int k = 0; k < D / 16; ++k) {
                uint32_t y[16];
                sm100::tmem_ld16(t_o + 16 * k, y);
                sm100::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                sm100::tmem_st16(t_o + 16 * k, y);
            }
        }
    }
    const uint64_t c2 = pair(c, c), b2 = pair(-s.mc, -s.mc);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float a, b;
            unpair(fma2(pair(__uint_as_float(x[k][2 * i]), __uint_as_float(x[k][2 * i + 1])), c2, b2), a, b);
            a = ex2(a);
            b = ex2(b);
            sum[i & 1] = add2(sum[i & 1], pair(a, b));
            u[i] = sm100::pack_bf16(a, b);
        }
        sm100::tmem_st16(t_s + 16 * k, u);
        if (k & 1) {
            sm100::tmem_st_wait();
            sm100::tc_fence_before();
            half_done(k >> 1);
        }
    }
    float a, b;
    unpair(add2(sum[0], sum[1]), a, b);
    s.l += a + b;
}

// Packed offsets: cu[0] = 0, non-decreasing, cu[n_docs] = tokens; the first
// bad document is recorded.  Run by the threads of one CTA.
__device__ __forceinline__ void check_offsets(const int32_t *cu, int n_docs, int64_t tokens, DeviceStatus *st)
{
    for (int n = threadIdx.x; n < n_docs; n += blockDim.x)
        if (cu[n + 1] < cu[n] || (n == 0 && cu[0] != 0) || (n == n_docs - 1 && cu[n_docs] != tokens))
            set_status(st, BDLA_ERR_DEVICE, (unsigned)n);
}

// Two kernels of one call, the second of which reads what the first wrote: the
// first says at its start that the second's CTAs may take the places that its own
// last ones leave, and the second waits, before it reads and before any CTA ends,
// until the first is done and its writes are there.  That takes the launch, and
// the second's set-up, out of the time between them (a kernel boundary otherwise
// costs 3 to 4 us).  What the second reads of the first is not `__restrict__`:
// such loads could move above the wait.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_second(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A... args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// One lane of a whole warp, the same one each time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// Products of two 128-row tiles.  A K step of 16 takes the tensor cores 64
// cycles, so issuing it must take less: the whole warp walks the tiles, so that
// descriptors are warp-uniform values, and one elected lane issues a product's
// steps (one lane of a diverged warp took 85 to 120 cycles a step, which left
// the tensor cores at half of their time).  A step's descriptors are a constant
// added to the tile's (the address field holds all of shared memory: no carry
// leaves it).
__device__ __forceinline__ uint64_t rows_desc(uint32_t tile) { return sm100::sdesc_sw128(tile, 16, 1024); }
__device__ __forceinline__ uint64_t sum_desc(uint32_t tile) { return sm100::sdesc_sw128(tile, kPanel, 1024); }

// D[acc] = A B^T: rows of both tiles are the operands' rows, features summed.
template <int D> __device__ __forceinline__ void mma_rows(uint32_t acc, uint64_t a, uint64_t b)
{
    constexpr uint32_t id = sm100::idesc_bf16_f32(BT, BT, false, false);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = ((ks >> 2) * kPanel + (ks & 3) * 32) >> 4;
        sm100::umma_bf16(acc, a + off, b + off, id, ks > 0);
    }
}

// D[acc] (+)= A B: K steps [First, Last) of A, bf16 [128 x 128] in tensor memory
// with its 64 left columns' pairs at `a` and the others at `a + Right`, and B a
// tile whose rows are summed over.
template <int D, int Right, int First = 0, int Last = BT / 16>
__device__ __forceinline__ void mma_sum(uint32_t acc, uint32_t a, uint64_t b, bool accumulate)
{
    constexpr uint32_t id = sm100::idesc_bf16_f32(BT, D, false, true);
#pragma unroll
    for (int ks = First; ks < Last; ++ks)
        sm100::umma_bf16_ts(acc, a + (ks >> 2) * Right + (ks & 3) * 8, b + ks * (2048 >> 4), id, accumulate || ks > 0);
}

// The same in two parts with the weights laid out by two warps a row, 64 columns
// each: Part 0 takes the first 32 of either's columns, Part 1 the others.
template <int D, int Part> __device__ __forceinline__ void mma_sum_part(uint32_t acc, uint32_t a, uint64_t b, bool accumulate)
{
    constexpr uint32_t id = sm100::idesc_bf16_f32(BT, D, false, true);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ks = (i >> 1) * 4 + 2 * Part + (i & 1);
        sm100::umma_bf16_ts(acc, a + (ks >> 2) * 64 + (ks & 3) * 8, b + ks * (2048 >> 4), id, accumulate || Part > 0 || i > 0);
    }
}

// All lanes' waits, as one answer for the warp (the tensor-memory accesses
// that follow need whole warps).  The abort flag is read only after a wait that
// was not over at once: the read cost the MMA warp a few hundred cycles each
// time, a quarter of the forward's time.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const uint64_t *limit, volatile int *abort_flag)
{
    if (__all_sync(0xffffffffu, sm100::mbar_try_wait(bar, parity)))
        return true;
    const bool ok = sm100::mbar_wait_lim(bar, parity, limit) && !*abort_flag;
    return __all_sync(0xffffffffu, ok);
}

// The same for threads on their own.
__device__ __forceinline__ bool lane_wait(uint64_t *bar, uint32_t parity, const uint64_t *limit, volatile int *abort_flag)
{
    return sm100::mbar_try_wait(bar, parity) || (sm100::mbar_wait_lim(bar, parity, limit) && !*abort_flag);
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

// The same in fp32 without a factor, 32 columns (128 bytes a row) at a time.
__device__ __forceinline__ void store_rows64_f32(uint32_t t, unsigned char *stage, float *dst, size_t stride, int n_valid, int lane)
{
    uint4 *s4 = reinterpret_cast<uint4 *>(stage);
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
        uint32_t y[32];
        sm100::tmem_ld32(t + 32 * c, y);
        sm100::tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s4[lane * 8 + (k ^ (lane & 7))] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int row = 4 * it + (lane >> 3), c8 = lane & 7;
            const uint4 v = s4[row * 8 + (c8 ^ (row & 7))];
            if (row < n_valid)
                *reinterpret_cast<uint4 *>(dst + (size_t)row * stride + 32 * c + 4 * c8) = v;
        }
        __syncwarp();
    }
}

}  // namespace attn
}  // namespace bdla
