// C entry points of the softmax layer (include/bdla_attn.h): argument checks,
// workspace carving and launches.
#include <math.h>

#include "bdla_attn_internal.h"

using namespace bdla;

namespace bdla {

int sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return 152;   // a GB300, for sizing without a device
    return n;
}

}  // namespace bdla

namespace {

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Sizes common to every call.  Tokens are 32-bit coordinates in the kernels.
bdla_status check_attn_dims(const bdla_attn_dims &d, bool packed, int n_docs)
{
    if (d.B < 1 || d.T < 0 || d.Hq < 1 || d.Hk < 1 || d.Hq % d.Hk != 0)
        return BDLA_ERR_SHAPE;
    if (packed && (d.B != 1 || n_docs < 1))
        return BDLA_ERR_SHAPE;
    if ((packed ? n_docs : d.B) > 65535 || d.Hq > 65535 || (d.d != 64 && d.d != 128))
        return BDLA_ERR_UNSUPPORTED;
    // one token row of heads, and all tokens, stay within 32-bit coordinates
    if ((int64_t)d.B * d.T > INT32_MAX - 65536 || (int64_t)d.Hq * d.d > (1 << 24))
        return BDLA_ERR_TOO_LARGE;
    return BDLA_OK;
}

bdla_status check_ws(const void *ws, size_t ws_bytes, size_t need)
{
    if (ws == nullptr || ws_bytes < need || !aligned16(ws))
        return BDLA_ERR_WORKSPACE;
    return BDLA_OK;
}

bdla_status check_norm(const bdla_qk_norm_args &a, const bdla_attn_dims &d)
{
    if (d.T > 0 && (!a.q || !a.k || !a.wq || !a.wk))
        return BDLA_ERR_NULL;
    if (a.rotary < 0 || a.rotary > d.d || a.rotary % 16 != 0)
        return BDLA_ERR_SHAPE;
    if (a.q_token % 8 != 0 || a.q_head % 8 != 0 || a.k_token % 8 != 0 || a.k_head % 8 != 0)
        return BDLA_ERR_ALIGN;
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.wq) || !aligned16(a.wk))
        return BDLA_ERR_ALIGN;
    if (!isfinite(a.eps) || a.eps < 0.0f || (a.rotary > 0 && !(isfinite(a.base) && a.base >= 1.0)))
        return BDLA_ERR_RANGE;
    return BDLA_OK;
}

// Whole documents: a CTA for every (128 tokens of a document, head) is a grid extent.
bdla_status check_grid(const bdla_attn_dims &d, int n_docs)
{
    const int64_t tiles = (int64_t)d.B * d.T / 128 + 1 + n_docs;
    return tiles * d.Hq <= INT32_MAX ? BDLA_OK : BDLA_ERR_TOO_LARGE;
}

bdla_status check_scale(float s) { return isfinite(s) && s > 0.0f ? BDLA_OK : BDLA_ERR_RANGE; }

bdla_status check_cache(const bdla_cache &c)
{
    if (c.n_pages < 0 || c.max_pages < 0 || c.page < 1)
        return BDLA_ERR_SHAPE;
    if (c.page > 65536)
        return BDLA_ERR_UNSUPPORTED;
    // positions and rows of the cache are 32-bit (2^31 rows are more than the GPU's memory holds)
    if ((int64_t)c.max_pages * c.page > INT32_MAX - 65536 || (int64_t)c.n_pages * c.page > INT32_MAX)
        return BDLA_ERR_TOO_LARGE;
    if (!c.lens || (c.max_pages > 0 && !c.pages) || (c.n_pages > 0 && (!c.k || !c.v)))
        return BDLA_ERR_NULL;
    if (!aligned16(c.k) || !aligned16(c.v))
        return BDLA_ERR_ALIGN;
    return BDLA_OK;
}

AttnProblem make_attn(const bdla_attn_dims &d, const int32_t *cu, int n_docs, float scale, void *ws, void *stream)
{
    AttnProblem p;
    p.cu = cu;
    p.n_docs = cu ? n_docs : d.B;
    p.T = d.T;
    p.tokens = (int64_t)d.B * d.T;
    p.Hq = d.Hq;
    p.Hk = d.Hk;
    p.d = d.d;
    p.scale = scale;
    p.st = static_cast<DeviceStatus *>(ws);
    p.stream = static_cast<cudaStream_t>(stream);
    return p;
}

#define BDLA_TRY(expr)                                                                             \
    do {                                                                                           \
        bdla_status s_ = (expr);                                                                   \
        if (s_ != BDLA_OK)                                                                         \
            return s_;                                                                             \
    } while (0)
#define BDLA_CUDA(expr)                                                                            \
    do {                                                                                           \
        if ((expr) != cudaSuccess)                                                                 \
            return BDLA_ERR_CUDA;                                                                  \
    } while (0)

template <typename T> const __nv_bfloat16 *cb(const T *p) { return static_cast<const __nv_bfloat16 *>(p); }
__nv_bfloat16 *mb(void *p) { return static_cast<__nv_bfloat16 *>(p); }

}  // namespace

extern "C" {

size_t bdla_workspace_bytes_attn(int op, bdla_attn_dims d, int n_docs, int64_t max_keys)
{
    if (check_attn_dims(d, n_docs > 0, n_docs) != BDLA_OK)
        return 0;
    const size_t head = round_up(kStatusBytes);
    switch (op) {
    case BDLA_ATTN_FWD:
    case BDLA_ATTN_APPEND:
        return head;
    case BDLA_ATTN_BWD:
        return head + round_up((size_t)d.B * d.T * d.Hq * sizeof(float)) +
               round_up(attn_bwd_part_floats(d, n_docs > 0 ? n_docs : d.B) * sizeof(float));
    case BDLA_ATTN_NORM_BWD:
        return head + round_up((size_t)norm_bwd_blocks(d) * d.d * sizeof(float));
    case BDLA_ATTN_CACHED:
        if (max_keys < 0 || d.T < 1 || d.T > 64)   // the sizes bdla_attn_cached refuses: no rows to cut pieces for
            return 0;
        return head + round_up(cached_partial_bytes(d, cached_splits(d, max_keys)));
    }
    return 0;
}

bdla_status bdla_qk_norm(bdla_qk_norm_args a, void *qn, void *kn, bdla_attn_dims d, void *stream)
{
    const bool packed = a.cu_seqlens != nullptr;
    BDLA_TRY(check_attn_dims(d, packed, a.n_docs));
    BDLA_TRY(check_norm(a, d));
    if (d.T > 0 && (!qn || !kn))
        return BDLA_ERR_NULL;
    if (!aligned16(qn) || !aligned16(kn))
        return BDLA_ERR_ALIGN;
    BDLA_CUDA(launch_qk_norm(a, mb(qn), mb(kn), d, static_cast<cudaStream_t>(stream)));
    return BDLA_OK;
}

bdla_status bdla_qk_norm_bwd(bdla_qk_norm_args a, const void *dqn, const void *dkn, bdla_dtype g_dtype, void *dq,
                             void *dk, float *dwq, float *dwk, bdla_attn_dims d, void *ws, size_t ws_bytes,
                             void *stream)
{
    const bool packed = a.cu_seqlens != nullptr;
    BDLA_TRY(check_attn_dims(d, packed, a.n_docs));
    BDLA_TRY(check_norm(a, d));
    if ((d.T > 0 && (!dqn || !dkn || !dq || !dk)) || !dwq || !dwk)
        return BDLA_ERR_NULL;
    if (!aligned16(dqn) || !aligned16(dkn) || !aligned16(dq) || !aligned16(dk) || !aligned16(dwq) || !aligned16(dwk))
        return BDLA_ERR_ALIGN;
    if (g_dtype != BDLA_BF16 && g_dtype != BDLA_F32)
        return BDLA_ERR_DTYPE;
    BDLA_TRY(check_ws(ws, ws_bytes, bdla_workspace_bytes_attn(BDLA_ATTN_NORM_BWD, d, packed ? a.n_docs : 0, 0)));
    float *part = reinterpret_cast<float *>(static_cast<char *>(ws) + round_up(kStatusBytes));
    BDLA_CUDA(launch_qk_norm_bwd(a, dqn, dkn, g_dtype == BDLA_F32, mb(dq), mb(dk), dwq, dwk, part, d,
                                 static_cast<cudaStream_t>(stream)));
    return BDLA_OK;
}

bdla_status bdla_attn_fwd(const void *q, const void *k, const void *v, const int32_t *cu_seqlens, int n_docs,
                          float scale, void *o, float *lse, bdla_attn_dims d, void *ws, size_t ws_bytes,
                          void *stream)
{
    const bool packed = cu_seqlens != nullptr;
    BDLA_TRY(check_attn_dims(d, packed, n_docs));
    BDLA_TRY(check_grid(d, packed ? n_docs : d.B));
    BDLA_TRY(check_scale(scale));
    if (d.T > 0 && (!q || !k || !v || !o || !lse))
        return BDLA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return BDLA_ERR_ALIGN;
    BDLA_TRY(check_ws(ws, ws_bytes, bdla_workspace_bytes_attn(BDLA_ATTN_FWD, d, packed ? n_docs : 0, 0)));
    const AttnProblem p = make_attn(d, cu_seqlens, n_docs, scale, ws, stream);
    BDLA_CUDA(launch_attn_fwd(p, cb(q), cb(k), cb(v), mb(o), lse));
    return BDLA_OK;
}

bdla_status bdla_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                          const void *dO, const int32_t *cu_seqlens, int n_docs, float scale, void *dq, void *dk,
                          void *dv, bdla_attn_dims d, void *ws, size_t ws_bytes, void *stream)
{
    const bool packed = cu_seqlens != nullptr;
    BDLA_TRY(check_attn_dims(d, packed, n_docs));
    BDLA_TRY(check_grid(d, packed ? n_docs : d.B));
    BDLA_TRY(check_scale(scale));
    if (d.T > 0 && (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv))
        return BDLA_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dO) ||
        !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return BDLA_ERR_ALIGN;
    BDLA_TRY(check_ws(ws, ws_bytes, bdla_workspace_bytes_attn(BDLA_ATTN_BWD, d, packed ? n_docs : 0, 0)));
    const AttnProblem p = make_attn(d, cu_seqlens, n_docs, scale, ws, stream);
    float *delta = reinterpret_cast<float *>(static_cast<char *>(ws) + round_up(kStatusBytes));
    float *part = nullptr;
    if (attn_bwd_part_floats(d, p.n_docs) != 0)
        part = reinterpret_cast<float *>(reinterpret_cast<char *>(delta) + round_up((size_t)d.B * d.T * d.Hq * sizeof(float)));
    BDLA_CUDA(launch_attn_bwd(p, cb(q), cb(k), cb(v), cb(o), lse, cb(dO), mb(dq), mb(dk), mb(dv), delta, part));
    return BDLA_OK;
}

bdla_status bdla_cache_append(const void *k, const void *v, bdla_cache c, const int32_t *rows,
                              const int32_t *counts, bdla_attn_dims d, void *ws, size_t ws_bytes, void *stream)
{
    BDLA_TRY(check_attn_dims(d, false, 0));
    BDLA_TRY(check_cache(c));
    if (d.T > 0 && (!k || !v))
        return BDLA_ERR_NULL;
    if (!aligned16(k) || !aligned16(v))
        return BDLA_ERR_ALIGN;
    BDLA_TRY(check_ws(ws, ws_bytes, bdla_workspace_bytes_attn(BDLA_ATTN_APPEND, d, 0, 0)));
    BDLA_CUDA(launch_cache_append(cb(k), cb(v), c, rows, counts, d, static_cast<DeviceStatus *>(ws),
                                  static_cast<cudaStream_t>(stream)));
    return BDLA_OK;
}

bdla_status bdla_attn_cached(const void *q, bdla_cache c, const uint64_t *tree, float scale, void *o, float *lse,
                             bdla_attn_dims d, void *ws, size_t ws_bytes, void *stream)
{
    BDLA_TRY(check_attn_dims(d, false, 0));
    if (d.T < 1)
        return BDLA_ERR_SHAPE;
    if (d.T > 64)
        return BDLA_ERR_UNSUPPORTED;
    if ((int64_t)d.B * d.T * d.Hq > INT32_MAX)   // rows are a grid extent
        return BDLA_ERR_TOO_LARGE;
    BDLA_TRY(check_scale(scale));
    BDLA_TRY(check_cache(c));
    if (!q || !o || !lse)
        return BDLA_ERR_NULL;
    if (!aligned16(q) || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(tree) & 7u) != 0)
        return BDLA_ERR_ALIGN;
    const int64_t max_keys = (int64_t)c.max_pages * c.page;
    BDLA_TRY(check_ws(ws, ws_bytes, bdla_workspace_bytes_attn(BDLA_ATTN_CACHED, d, 0, max_keys)));
    BDLA_CUDA(launch_attn_cached(cb(q), c, tree, scale, mb(o), lse, d, max_keys,
                                 static_cast<char *>(ws) + round_up(kStatusBytes), static_cast<DeviceStatus *>(ws),
                                 static_cast<cudaStream_t>(stream)));
    return BDLA_OK;
}

}  // extern "C"
