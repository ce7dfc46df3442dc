// Host-side launcher interface between the softmax-layer entry points
// (bdla_attn_api.cu) and their kernels.
#pragma once

#include "../../include/bdla_attn.h"
#include "bdla_internal.h"

namespace bdla {

struct AttnProblem {
    const int32_t *cu;   // device cu_seqlens or nullptr (fixed-length)
    int n_docs;          // documents (B for fixed-length calls)
    int T;               // per-document length (fixed) or total tokens (packed)
    int64_t tokens;
    int Hq, Hk, d;
    float scale;
    DeviceStatus *st;
    cudaStream_t stream;
};

int sm_count();   // of the current device

// Norm and rotation.  `tokens` = B * T; T > 0 gives fixed-length rows when cu is null.
cudaError_t launch_qk_norm(const bdla_qk_norm_args &a, __nv_bfloat16 *qn, __nv_bfloat16 *kn,
                           const bdla_attn_dims &d, cudaStream_t stream);
// `part`: norm_bwd_blocks() partial sums of d floats.
int norm_bwd_blocks(const bdla_attn_dims &d);
cudaError_t launch_qk_norm_bwd(const bdla_qk_norm_args &a, const void *dqn, const void *dkn, int g_f32,
                               __nv_bfloat16 *dq, __nv_bfloat16 *dk, float *dwq, float *dwk, float *part,
                               const bdla_attn_dims &d, cudaStream_t stream);

// Packed calls: records a malformed cu_seqlens as BDLA_ERR_DEVICE.
cudaError_t launch_doc_report(const AttnProblem &p);
cudaError_t launch_attn_fwd(const AttnProblem &p, const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                            const __nv_bfloat16 *v, __nv_bfloat16 *o, float *lse);
// `delta`: [Hq][tokens] fp32 scratch.  `part`: attn_bwd_part_floats() floats, or null where that is 0.
size_t attn_bwd_part_floats(const bdla_attn_dims &d, int n_docs);
cudaError_t launch_attn_bwd(const AttnProblem &p, const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                            const __nv_bfloat16 *v, const __nv_bfloat16 *o, const float *lse,
                            const __nv_bfloat16 *dO, __nv_bfloat16 *dq, __nv_bfloat16 *dk, __nv_bfloat16 *dv,
                            float *delta, float *part);

cudaError_t launch_cache_append(const __nv_bfloat16 *k, const __nv_bfloat16 *v, const bdla_cache &c,
                                const int32_t *rows, const int32_t *counts, const bdla_attn_dims &d,
                                DeviceStatus *st, cudaStream_t stream);
// Key splits of one call and the bytes of their partial results.
int cached_splits(const bdla_attn_dims &d, int64_t max_keys);
size_t cached_partial_bytes(const bdla_attn_dims &d, int splits);
cudaError_t launch_attn_cached(const __nv_bfloat16 *q, const bdla_cache &c, const uint64_t *tree, float scale,
                               __nv_bfloat16 *o, float *lse, const bdla_attn_dims &d, int64_t max_keys, void *partials,
                               DeviceStatus *st, cudaStream_t stream);

}  // namespace bdla
