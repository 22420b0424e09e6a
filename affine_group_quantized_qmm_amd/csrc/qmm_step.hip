// C ABI of the operators between the products of a decode step: argument
// checks and launches. Declarations and the full contract are in
// include/qmm.h.
#include "qmm.h"
#include "qmm_kernels.hpp"
#include "qmm_step.hpp"

#include <math.h>
#include <stdint.h>

namespace {

bool aligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool output_type(int type) { return type == QMM_F16 || type == QMM_BF16; }
bool any_type(int type) { return output_type(type) || type == QMM_F32; }

// The paged cache's sizes, common to both operators that touch it.
int check_cache(int num_pages, int page_size, int Hkv)
{
    if (num_pages < 1 || page_size < 1 || Hkv < 1)
        return QMM_ERR_SHAPE;
    // slots are 32-bit numbers, rows of the cache (slot, head) unsigned ones
    if ((int64_t)num_pages * page_size > INT32_MAX || (uint64_t)num_pages * page_size >= UINT32_MAX / (uint64_t)Hkv)
        return QMM_ERR_SHAPE;
    return QMM_OK;
}

int check_attention_sizes(int T, int B, int Hq, int Hkv, int D, int max_rows, int max_context, int window, int sinks)
{
    if (T < 1 || B < 1 || Hq < 1 || Hkv < 1 || max_rows < 1 || max_context < 0 || window < 0 || sinks < 0)
        return QMM_ERR_SHAPE;
    if (T >= (1 << 28) || B > 65535 || Hq > 65535 || max_rows > T)
        return QMM_ERR_SHAPE;
    if (Hq % Hkv != 0 || !qmm::attn_head_dim_supported(D))
        return QMM_ERR_HEAD;
    if ((int64_t)max_rows * Hq >= (1 << 30))
        return QMM_ERR_SHAPE;
    return QMM_OK;
}

constexpr int kFar = 1 << 30;  // positions minus the window stay in 32 bits

qmm::AttnPlan plan_of(int B, int Hq, int Hkv, int D, int max_rows, int max_context, int window, int sinks,
                      int page_size, int max_pages)
{
    return qmm::attn_plan(B, Hq, Hkv, D, max_rows, max_context, window < kFar ? window : 0, sinks, page_size,
                          max_pages);
}

}  // namespace

extern "C" {

int qmm_qk_norm_rope(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                     int in_type, const float *q_weight, const float *k_weight, float eps, float weight_offset,
                     const int32_t *positions, const float *inv_freq, int R, int interleaved, const int32_t *slots,
                     void *q_out, void *k_cache, void *v_cache, int out_type, int M, int Hq, int Hkv, int D,
                     int num_pages, int page_size, hipStream_t stream)
{
    if (!q || !k || !v || !q_weight || !k_weight || !positions || !slots || !q_out || !k_cache || !v_cache ||
        (R > 0 && !inv_freq))
        return QMM_ERR_NULL;
    if (!any_type(in_type) || !output_type(out_type))
        return QMM_ERR_TYPE;
    // a workgroup of 256 threads for each row: the runtime counts a launch's threads in 32 bits
    if (M < 1 || Hq < 1 || M > (int)(UINT32_MAX / 256) || Hq > 65535 || Hkv > 65535)
        return QMM_ERR_SHAPE;
    const int rc = check_cache(num_pages, page_size, Hkv);
    if (rc != QMM_OK)
        return rc;
    if (D < 8 || D > 256 || D % 8 != 0 || R < 0 || R > D || R % 8 != 0)
        return QMM_ERR_HEAD;
    if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D)
        return QMM_ERR_SHAPE;
    if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(q, 16) || !aligned(k, 16) ||
        !aligned(v, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(inv_freq, 16) ||
        !aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(positions, 4) ||
        !aligned(slots, 4))
        return QMM_ERR_ALIGN;
    qmm::RopeArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.positions = positions;
    a.slots = slots;
    a.inv_freq = inv_freq;
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.M = M;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.R = R;
    a.page_size = page_size;
    const qmm::MagicDiv d = qmm::magic_div(page_size);
    a.page_magic = d.magic;
    a.page_shift = d.shift;
    a.slot_count = num_pages * page_size;
    a.eps = eps;
    a.weight_offset = weight_offset;
    return qmm::launch_qk_norm_rope(a, in_type, out_type == QMM_BF16, interleaved != 0, stream) == hipSuccess
               ? QMM_OK
               : QMM_ERR_LAUNCH;
}

size_t qmm_paged_attention_workspace_bytes(int T, int B, int Hq, int Hkv, int D, int max_rows, int max_context,
                                           int window, int sinks)
{
    if (check_attention_sizes(T, B, Hq, Hkv, D, max_rows, max_context, window, sinks) != QMM_OK)
        return 0;
    // the largest that any block table needs
    return plan_of(B, Hq, Hkv, D, max_rows, max_context, window, sinks, 1, 1).workspace_bytes;
}

int qmm_paged_attention(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache, int type,
                        const int32_t *block_table, const int32_t *context_lens, const int32_t *row_starts, void *out,
                        float *lse, int T, int B, int Hq, int Hkv, int D, int num_pages, int page_size, int max_pages,
                        int max_rows, int max_context, float scale, int window, int sinks, void *workspace,
                        size_t workspace_bytes, hipStream_t stream)
{
    if (!q || !k_cache || !v_cache || !block_table || !context_lens || !row_starts || !out)
        return QMM_ERR_NULL;
    if (!output_type(type))
        return QMM_ERR_TYPE;
    int rc = check_attention_sizes(T, B, Hq, Hkv, D, max_rows, max_context, window, sinks);
    if (rc == QMM_OK)
        rc = check_cache(num_pages, page_size, Hkv);
    if (rc != QMM_OK)
        return rc;
    // Token numbers have 32 bits up to the end of a tile that begins at the
    // table's end, and loads run two tiles ahead.
    if (max_pages < 1 || (int64_t)max_pages * page_size > INT32_MAX - 4 * qmm::kAttnMostTile ||
        q_stride < (int64_t)Hq * D || !isfinite(scale))
        return QMM_ERR_SHAPE;
    const qmm::AttnPlan plan =
        plan_of(B, Hq, Hkv, D, max_rows, max_context, window, sinks, page_size, max_pages);
    if (plan.workspace_bytes > 0 && !workspace)
        return QMM_ERR_NULL;
    if (workspace_bytes < plan.workspace_bytes)
        return QMM_ERR_WORKSPACE;
    if (plan.blocks > INT32_MAX / 256 || plan.items > INT32_MAX / 256)  // the runtime's limit on threads of a launch
        return QMM_ERR_SHAPE;
    if (q_stride % 8 != 0 || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        (plan.workspace_bytes > 0 && !aligned(workspace, 16)) || !aligned(block_table, 4) ||
        !aligned(context_lens, 4) || !aligned(row_starts, 4) || !aligned(lse, 4))
        return QMM_ERR_ALIGN;
    qmm::AttnArgs a{};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.row_starts = row_starts;
    a.out = out;
    a.lse = lse;
    a.q_stride = q_stride;
    a.T = T;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.max_pages = max_pages;
    a.window = window < kFar ? window : 0;
    a.sinks = a.window > 0 ? (sinks < kFar ? sinks : kFar) : 0;
    a.scale_log2 = scale * 1.44269504088896340736f;
    const qmm::MagicDiv d = qmm::magic_div(page_size);
    a.page_magic = d.magic;
    a.page_shift = d.shift;
    return qmm::launch_paged_attention(a, plan, D, type == QMM_BF16, workspace, stream) == hipSuccess ? QMM_OK : QMM_ERR_LAUNCH;
}

size_t qmm_sample_workspace_bytes(int M, int V)
{
    return M < 1 || M > 65535 || !qmm::sample_size_supported(V) ? 0 : qmm::sample_workspace_bytes(M, V);
}

int qmm_sample(const void *logits, int64_t row_stride, int type, const float *u, const float *temperature,
               const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens, float *logprobs, int M,
               int V, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!logits || !u || !tokens || !workspace)
        return QMM_ERR_NULL;
    if (!any_type(type))
        return QMM_ERR_TYPE;
    if (M < 1 || M > 65535 || !qmm::sample_size_supported(V) || row_stride < V)
        return QMM_ERR_SHAPE;
    if (workspace_bytes < qmm::sample_workspace_bytes(M, V))
        return QMM_ERR_WORKSPACE;
    if (!aligned(logits, type == QMM_F32 ? 4 : 2) || !aligned(u, 4) || !aligned(temperature, 4) ||
        !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) ||
        !aligned(logprobs, 4) || !aligned(workspace, 16))
        return QMM_ERR_ALIGN;
    qmm::SampleArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.tokens = tokens;
    a.logprobs = logprobs;
    a.workspace = workspace;
    a.M = M;
    a.V = V;
    return qmm::launch_sample(a, type, stream) == hipSuccess ? QMM_OK : QMM_ERR_LAUNCH;
}

}  // extern "C"
