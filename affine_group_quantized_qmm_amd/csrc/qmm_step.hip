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
                      int page_size, int max_pages, int bits)
{
    return qmm::attn_plan(B, Hq, Hkv, D, max_rows, max_context, window < kFar ? window : 0, sinks, page_size,
                          max_pages, bits);
}

int check_lora_sizes(int count, const int *N, int M, int K, int r, int adapters)
{
    if (count < 1 || count > QMM_MAX_FUSED || M < 1 || K < 32 || K % 32 != 0 || r < 8 || r > 128 || r % 8 != 0 ||
        adapters < 1)
        return QMM_ERR_SHAPE;
    if (M > 65535 * 16 || K > (1 << 28))  // blocks of 16 rows along a grid's y
        return QMM_ERR_SHAPE;
    for (int i = 0; i < count; ++i)
        if (N[i] < 1 || N[i] > (1 << 28))
            return QMM_ERR_SHAPE;
    // the runtime counts a launch's threads in 32 bits
    const qmm::LoraPlan p = qmm::lora_plan(count, N, M, K, r, adapters);
    const uint64_t most = UINT32_MAX / 256;
    return (uint64_t)p.blocks * p.down_x * p.down_z > most || (uint64_t)p.blocks * p.up_x * p.up_z > most ? QMM_ERR_SHAPE
                                                                                                      : QMM_OK;
}

int check_logprobs_sizes(int M, int V, int n)
{
    if (M < 1 || V < 1 || V > (1 << 23) || n < 0 || n > 64)
        return QMM_ERR_SHAPE;
    // the runtime counts a launch's threads in 32 bits
    return M > (1 << 24) - 1 || qmm::logprobs_plan(M, V, n, 7).threads > (int64_t)UINT32_MAX ? QMM_ERR_SHAPE : QMM_OK;
}

qmm::RopeArgs rope_args(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                        const float *q_weight, const float *k_weight, float eps, float weight_offset,
                        const int32_t *positions, const float *inv_freq, int R, const int32_t *slots, void *q_out,
                        void *k_cache, void *v_cache, int M, int Hq, int Hkv, int D, int page_size)
{
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
    a.eps = eps;
    a.weight_offset = weight_offset;
    return a;
}

// Checks of the norm and rotation that do not depend on what the cache holds.
int check_rope(const qmm::RopeArgs &a, int in_type, int out_type, int num_pages)
{
    if (!a.q || !a.k || !a.v || !a.q_weight || !a.k_weight || !a.positions || !a.slots || !a.q_out || !a.k_cache ||
        !a.v_cache || (a.R > 0 && !a.inv_freq))
        return QMM_ERR_NULL;
    if (!any_type(in_type) || !output_type(out_type))
        return QMM_ERR_TYPE;
    // a workgroup of 256 threads for each row: the runtime counts a launch's threads in 32 bits
    if (a.M < 1 || a.Hq < 1 || a.M > (int)(UINT32_MAX / 256) || a.Hq > 65535 || a.Hkv > 65535)
        return QMM_ERR_SHAPE;
    const int rc = check_cache(num_pages, a.page_size, a.Hkv);
    if (rc != QMM_OK)
        return rc;
    if (a.D < 8 || a.D > 256 || a.D % 8 != 0 || a.R < 0 || a.R > a.D || a.R % 8 != 0)
        return QMM_ERR_HEAD;
    if (a.q_stride < (int64_t)a.Hq * a.D || a.k_stride < (int64_t)a.Hkv * a.D || a.v_stride < (int64_t)a.Hkv * a.D)
        return QMM_ERR_SHAPE;
    if (a.q_stride % 8 != 0 || a.k_stride % 8 != 0 || a.v_stride % 8 != 0 || !aligned(a.q, 16) || !aligned(a.k, 16) ||
        !aligned(a.v, 16) || !aligned(a.q_weight, 16) || !aligned(a.k_weight, 16) || !aligned(a.inv_freq, 16) ||
        !aligned(a.q_out, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.positions, 4) ||
        !aligned(a.slots, 4))
        return QMM_ERR_ALIGN;
    return QMM_OK;
}

int run_rope(qmm::RopeArgs &a, int in_type, int out_type, int interleaved, int num_pages, hipStream_t stream)
{
    const qmm::MagicDiv d = qmm::magic_div(a.page_size);
    a.page_magic = d.magic;
    a.page_shift = d.shift;
    a.slot_count = num_pages * a.page_size;
    return qmm::launch_qk_norm_rope(a, in_type, out_type == QMM_BF16, interleaved != 0, stream) == hipSuccess
               ? QMM_OK
               : QMM_ERR_LAUNCH;
}

// A quantized cache's format.
int check_format(int D, int bits, int G)
{
    if (bits != 4 && bits != 8)
        return QMM_ERR_BITS;
    if (G != 32 && G != 64 && G != 128)
        return QMM_ERR_GROUP;
    return D % G == 0 ? QMM_OK : QMM_ERR_HEAD;
}

// Checks and launch of attention over either kind of cache (bits 0: 16-bit rows).
// `a` holds the pointers, sizes and the format's words; the rest is set here.
int run_attention(qmm::AttnArgs &a, int type, int D, int bits, int max_rows, int max_context, float scale, int window,
                  int sinks, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!a.q || !a.k_cache || !a.v_cache || !a.block_table || !a.context_lens || !a.row_starts || !a.out)
        return QMM_ERR_NULL;
    if (!output_type(type))
        return QMM_ERR_TYPE;
    int rc = check_attention_sizes(a.T, a.B, a.Hq, a.Hkv, D, max_rows, max_context, window, sinks);
    if (rc == QMM_OK)
        rc = check_cache(a.num_pages, a.page_size, a.Hkv);
    if (rc != QMM_OK)
        return rc;
    // Token numbers have 32 bits up to the end of a tile that begins at the
    // table's end, and loads run two tiles ahead.
    if (a.max_pages < 1 || (int64_t)a.max_pages * a.page_size > INT32_MAX - 4 * qmm::kAttnMostTile ||
        a.q_stride < (int64_t)a.Hq * D || !isfinite(scale))
        return QMM_ERR_SHAPE;
    const qmm::AttnPlan plan =
        plan_of(a.B, a.Hq, a.Hkv, D, max_rows, max_context, window, sinks, a.page_size, a.max_pages, bits);
    if (plan.workspace_bytes > 0 && !workspace)
        return QMM_ERR_NULL;
    if (workspace_bytes < plan.workspace_bytes)
        return QMM_ERR_WORKSPACE;
    if (plan.blocks > INT32_MAX / 256 || plan.items > INT32_MAX / 256)  // the runtime's limit on threads of a launch
        return QMM_ERR_SHAPE;
    if (a.q_stride % 8 != 0 || !aligned(a.q, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) ||
        !aligned(a.out, 16) || (plan.workspace_bytes > 0 && !aligned(workspace, 16)) || !aligned(a.block_table, 4) ||
        !aligned(a.context_lens, 4) || !aligned(a.row_starts, 4) || !aligned(a.lse, 4) || !aligned(a.k_sb, 4) ||
        !aligned(a.v_sb, 4))
        return QMM_ERR_ALIGN;
    a.window = window < kFar ? window : 0;
    a.sinks = a.window > 0 ? (sinks < kFar ? sinks : kFar) : 0;
    a.scale_log2 = scale * 1.44269504088896340736f;
    const qmm::MagicDiv d = qmm::magic_div(a.page_size);
    a.page_magic = d.magic;
    a.page_shift = d.shift;
    return qmm::launch_paged_attention(a, plan, D, type == QMM_BF16, bits, workspace, stream) == hipSuccess
               ? QMM_OK
               : QMM_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int qmm_qk_norm_rope(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                     int in_type, const float *q_weight, const float *k_weight, float eps, float weight_offset,
                     const int32_t *positions, const float *inv_freq, int R, int interleaved, const int32_t *slots,
                     void *q_out, void *k_cache, void *v_cache, int out_type, int M, int Hq, int Hkv, int D,
                     int num_pages, int page_size, hipStream_t stream)
{
    qmm::RopeArgs a = rope_args(q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps, weight_offset, positions,
                                inv_freq, R, slots, q_out, k_cache, v_cache, M, Hq, Hkv, D, page_size);
    const int rc = check_rope(a, in_type, out_type, num_pages);
    return rc != QMM_OK ? rc : run_rope(a, in_type, out_type, interleaved, num_pages, stream);
}

int qmm_qk_norm_rope_quant(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, int in_type, const float *q_weight, const float *k_weight, float eps,
                           float weight_offset, const int32_t *positions, const float *inv_freq, int R, int interleaved,
                           const int32_t *slots, void *q_out, uint32_t *k_codes, uint32_t *k_sb, uint32_t *v_codes,
                           uint32_t *v_sb, int out_type, int M, int Hq, int Hkv, int D, int bits, int G, int num_pages,
                           int page_size, hipStream_t stream)
{
    qmm::RopeArgs a = rope_args(q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, eps, weight_offset, positions,
                                inv_freq, R, slots, q_out, k_codes, v_codes, M, Hq, Hkv, D, page_size);
    if (!k_sb || !v_sb)
        return QMM_ERR_NULL;
    int rc = check_rope(a, in_type, out_type, num_pages);
    if (rc == QMM_OK)
        rc = check_format(D, bits, G);
    if (rc != QMM_OK)
        return rc;
    if (!aligned(k_sb, 4) || !aligned(v_sb, 4))
        return QMM_ERR_ALIGN;
    a.k_sb = k_sb;
    a.v_sb = v_sb;
    a.bits = bits;
    a.group = G;
    return run_rope(a, in_type, out_type, interleaved, num_pages, stream);
}

int qmm_quant_cache_read(const uint32_t *k_codes, const uint32_t *k_sb, const uint32_t *v_codes, const uint32_t *v_sb,
                         const int32_t *slots, void *k_out, void *v_out, int out_type, int M, int Hkv, int D, int bits,
                         int G, int num_pages, int page_size, hipStream_t stream)
{
    if (!k_codes || !k_sb || !v_codes || !v_sb || !slots || !k_out || !v_out)
        return QMM_ERR_NULL;
    if (!output_type(out_type))
        return QMM_ERR_TYPE;
    int rc = M < 1 || Hkv > 65535 ? QMM_ERR_SHAPE : check_cache(num_pages, page_size, Hkv);
    if (rc == QMM_OK)
        rc = D < 32 || D > 256 ? QMM_ERR_HEAD : check_format(D, bits, G);
    if (rc != QMM_OK)
        return rc;
    // a thread for 8 codes of a row, at least a workgroup of 256 a row: the runtime counts a launch's threads in 32 bits
    const int64_t row_blocks = ((int64_t)2 * Hkv * (D / 8) + 255) / 256;
    if ((int64_t)M * row_blocks > UINT32_MAX / 256)
        return QMM_ERR_SHAPE;
    if (!aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
        !aligned(k_sb, 4) || !aligned(v_sb, 4) || !aligned(slots, 4))
        return QMM_ERR_ALIGN;
    qmm::ReadArgs a{};
    a.codes[0] = k_codes;
    a.codes[1] = v_codes;
    a.sb[0] = k_sb;
    a.sb[1] = v_sb;
    a.out[0] = k_out;
    a.out[1] = v_out;
    a.slots = slots;
    a.M = M;
    a.Hkv = Hkv;
    a.D = D;
    a.bits = bits;
    a.group = G;
    a.page_size = page_size;
    a.slot_count = num_pages * page_size;
    const qmm::MagicDiv d = qmm::magic_div(page_size);
    a.page_magic = d.magic;
    a.page_shift = d.shift;
    return qmm::launch_quant_cache_read(a, out_type == QMM_BF16, stream) == hipSuccess ? QMM_OK : QMM_ERR_LAUNCH;
}

size_t qmm_paged_attention_workspace_bytes(int T, int B, int Hq, int Hkv, int D, int max_rows, int max_context,
                                           int window, int sinks)
{
    if (check_attention_sizes(T, B, Hq, Hkv, D, max_rows, max_context, window, sinks) != QMM_OK)
        return 0;
    // the largest that any block table needs
    return plan_of(B, Hq, Hkv, D, max_rows, max_context, window, sinks, 1, 1, 0).workspace_bytes;
}

int qmm_paged_attention(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache, int type,
                        const int32_t *block_table, const int32_t *context_lens, const int32_t *row_starts, void *out,
                        float *lse, int T, int B, int Hq, int Hkv, int D, int num_pages, int page_size, int max_pages,
                        int max_rows, int max_context, float scale, int window, int sinks, void *workspace,
                        size_t workspace_bytes, hipStream_t stream)
{
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
    return run_attention(a, type, D, 0, max_rows, max_context, scale, window, sinks, workspace, workspace_bytes, stream);
}

size_t qmm_paged_attention_quant_workspace_bytes(int T, int B, int Hq, int Hkv, int D, int max_rows, int max_context,
                                                 int window, int sinks, int bits, int G)
{
    if (check_attention_sizes(T, B, Hq, Hkv, D, max_rows, max_context, window, sinks) != QMM_OK ||
        check_format(D, bits, G) != QMM_OK)
        return 0;
    return plan_of(B, Hq, Hkv, D, max_rows, max_context, window, sinks, 1, 1, bits).workspace_bytes;
}

int qmm_paged_attention_quant(const void *q, int64_t q_stride, const uint32_t *k_codes, const uint32_t *k_sb,
                              const uint32_t *v_codes, const uint32_t *v_sb, int type, const int32_t *block_table,
                              const int32_t *context_lens, const int32_t *row_starts, void *out, float *lse, int T,
                              int B, int Hq, int Hkv, int D, int bits, int G, int num_pages, int page_size,
                              int max_pages, int max_rows, int max_context, float scale, int window, int sinks,
                              void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!k_sb || !v_sb)
        return QMM_ERR_NULL;
    const int rc = check_format(D, bits, G);
    if (rc != QMM_OK)
        return rc;
    qmm::AttnArgs a{};
    a.q = q;
    a.k_cache = k_codes;
    a.v_cache = v_codes;
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
    a.k_sb = k_sb;
    a.v_sb = v_sb;
    a.code_shift = G == 32 ? 5 : G == 64 ? 6 : 7;
    for (int groups = D % 96 == 0 ? D / G / 3 : D / G; groups > 1; groups /= 2)
        ++a.words_shift;
    return run_attention(a, type, D, bits, max_rows, max_context, scale, window, sinks, workspace, workspace_bytes,
                         stream);
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

size_t qmm_lora_workspace_bytes(int count, const int *N, int M, int K, int r, int adapters)
{
    return !N || check_lora_sizes(count, N, M, K, r, adapters) != QMM_OK
               ? 0
               : qmm::lora_plan(count, N, M, K, r, adapters).workspace_bytes;
}

int qmm_lora(const void *x, int type, int count, const void *const *a, const void *const *b, float *const *y,
             const int *N, const int32_t *ids, const float *scales, int M, int K, int r, int adapters, void *workspace,
             size_t workspace_bytes, hipStream_t stream)
{
    if (!x || !a || !b || !y || !N || !ids)
        return QMM_ERR_NULL;
    if (!output_type(type))
        return QMM_ERR_TYPE;
    const int rc = check_lora_sizes(count, N, M, K, r, adapters);
    if (rc != QMM_OK)
        return rc;
    const qmm::LoraPlan plan = qmm::lora_plan(count, N, M, K, r, adapters);
    if (!workspace)
        return QMM_ERR_NULL;
    if (workspace_bytes < plan.workspace_bytes)
        return QMM_ERR_WORKSPACE;
    qmm::LoraArgs l{};
    for (int i = 0; i < count; ++i) {
        if (!a[i] || !b[i] || !y[i])
            return QMM_ERR_NULL;
        if (!aligned(a[i], 16) || !aligned(b[i], 16) || !aligned(y[i], 16))
            return QMM_ERR_ALIGN;
        l.proj[i] = qmm::LoraProj{a[i], b[i], y[i], N[i], 0};
    }
    if (!aligned(x, 16) || !aligned(workspace, 16) || !aligned(ids, 4) || !aligned(scales, 4))
        return QMM_ERR_ALIGN;
    for (int i = 0; i < count; ++i)  // both would be read, and added to, at once
        for (int j = 0; j < i; ++j)
            if (y[i] < y[j] + (int64_t)M * N[j] && y[j] < y[i] + (int64_t)M * N[i])
                return QMM_ERR_SHAPE;
    l.x = x;
    l.ids = ids;
    l.scales = scales;
    l.count = count;
    l.M = M;
    l.K = K;
    l.r = r;
    l.adapters = adapters;
    return qmm::launch_lora(l, plan, type == QMM_BF16, workspace, stream) == hipSuccess ? QMM_OK : QMM_ERR_LAUNCH;
}

size_t qmm_logprobs_workspace_bytes(int M, int V, int n)
{
    return check_logprobs_sizes(M, V, n) != QMM_OK ? 0 : qmm::logprobs_plan(M, V, n, 7).workspace_bytes;
}

int qmm_logprobs(const void *logits, int64_t row_stride, int type, const int32_t *tokens, float *logprobs,
                 int32_t *ranks, float *entropy, int n, int32_t *top_tokens, float *top_logprobs, int M, int V,
                 void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!logits || !tokens || !logprobs || (n > 0 && (!top_tokens || !top_logprobs)))
        return QMM_ERR_NULL;
    if (!any_type(type))
        return QMM_ERR_TYPE;
    const int rc = check_logprobs_sizes(M, V, n);
    if (rc != QMM_OK)
        return rc;
    if (row_stride < V)
        return QMM_ERR_SHAPE;
    const int size = type == QMM_F32 ? 4 : 2;
    const bool even = aligned(logits, 16) && row_stride * size % 16 == 0;
    const qmm::LogprobPlan plan = qmm::logprobs_plan(M, V, n, even ? 0 : 16 / size - 1);
    if (plan.workspace_bytes > 0 && !workspace)
        return QMM_ERR_NULL;
    if (workspace_bytes < plan.workspace_bytes)
        return QMM_ERR_WORKSPACE;
    if (!aligned(logits, type == QMM_F32 ? 4 : 2) || !aligned(tokens, 4) || !aligned(logprobs, 4) || !aligned(ranks, 4) ||
        !aligned(entropy, 4) || !aligned(top_tokens, 4) || !aligned(top_logprobs, 4) ||
        (plan.workspace_bytes > 0 && !aligned(workspace, 16)))
        return QMM_ERR_ALIGN;
    qmm::LogprobArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.tokens = tokens;
    a.logprobs = logprobs;
    a.ranks = ranks;
    a.entropy = entropy;
    a.top_tokens = top_tokens;
    a.top_logprobs = top_logprobs;
    a.M = M;
    a.V = V;
    a.n = n;
    return qmm::launch_logprobs(a, plan, type, workspace, stream) == hipSuccess ? QMM_OK : QMM_ERR_LAUNCH;
}

}  // extern "C"
