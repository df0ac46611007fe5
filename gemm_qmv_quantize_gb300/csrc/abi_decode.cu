// abi_decode.cu -- the C ABI of the operators beside the matmuls (include/qmv.h):
// argument validation before any CUDA call.
#include <cmath>
#include <cstring>

#include "decode_ops.h"
#include "qmv.h"

using namespace qmv;

namespace {

constexpr int64_t kMaxDim = 0x7fffffffLL;
constexpr int kMaxRows = 96;   // rows of a projection, as in the NVFP4 / FP8 calls

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

qmv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QMV_OK : QMV_ERR_CUDA; }

bool is_16bit(int type) { return type == QMV_F16 || type == QMV_BF16; }

bool lora_shape_ok(int M, int R, int64_t K)
{
    return M >= 0 && M <= kMaxRows && R >= 8 && R <= 256 && R % 8 == 0 && K >= 0 && K <= kMaxDim && K % 8 == 0;
}

bool attention_shape_ok(int B, int T, int Hq, int Hkv, int D, int64_t prefix_len, int64_t max_own)
{
    return B >= 0 && T >= 1 && Hq >= 1 && Hkv >= 1 && Hkv <= 65535 && Hq % Hkv == 0 && (D == 64 || D == 128) && prefix_len >= 0 &&
           max_own >= 0 && prefix_len <= kMaxDim && max_own <= kMaxDim &&
           static_cast<int64_t>(B) * T <= kMaxDim && static_cast<int64_t>(B) * T * Hq <= kMaxDim / 128;
}

// Of both appends with norms; codes: heads that the attention over them takes.
qmv_status norm_rope_shape(int type, int M, int Hq, int Hkv, int D, int rot, int axes, int n_positions, int64_t n_slots,
                           float eps, bool codes)
{
    if (!is_16bit(type) || M < 0 || Hq < 1 || Hkv < 1 || Hq > 65536 || Hkv > 65536) return QMV_ERR_SHAPE;
    if (D < 8 || D > 2 * kMaxRopePairs || D % 8 != 0 || rot < 0 || rot > D || rot % 8 != 0) return QMV_ERR_SHAPE;
    if (codes && ((D != 64 && D != 128) || n_slots % 16 != 0)) return QMV_ERR_SHAPE;
    if (axes < 1 || axes > kMaxRopeAxes || n_positions < (rot > 0 ? 1 : 0) || n_slots < 0) return QMV_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps)) return QMV_ERR_SHAPE;
    return QMV_OK;
}

qmv_status run_norm_rope(NormRopeArgs g, const uint8_t *axis_of_pair, int axes, qmv_stream_t stream)
{
    if (!g.qkv || !g.q || !g.slots || !g.k_cache || !g.v_cache) return QMV_ERR_NULL;
    if (g.rot > 0 && (!g.positions || !g.table || !axis_of_pair)) return QMV_ERR_NULL;
    if (misaligned(g.qkv, 16) || misaligned(g.q, 16) || misaligned(g.k_cache, 16) || misaligned(g.v_cache, 16) ||
        misaligned(g.table, 16) || misaligned(g.positions, 4) || misaligned(g.slots, 8) || misaligned(g.q_norm, 16) ||
        misaligned(g.k_norm, 16) || misaligned(g.k_scale, 4) || misaligned(g.v_scale, 4))
        return QMV_ERR_ALIGN;
    for (int i = 0; i < g.rot / 2; ++i) {
        if (axis_of_pair[i] >= axes) return QMV_ERR_SHAPE;
        g.axis_of_pair[i] = axis_of_pair[i];
    }
    return from_cuda(launch_norm_rope(g, stream));
}

bool paged_shape_ok(int B, int T, int Hq, int Hkv, int D, int64_t max_len)
{
    return B >= 0 && B <= 65535 && T >= 1 && Hq >= 1 && Hkv >= 1 && Hkv <= 65535 && Hq % Hkv == 0 && (D == 64 || D == 128) &&
           max_len >= 0 && max_len <= (1 << 30) && static_cast<int64_t>(T) * Hq <= (1 << 20) &&
           static_cast<int64_t>(B) * T * Hq <= kMaxDim;
}

}  // namespace

extern "C" {

int64_t qmv_lora_add_workspace(int M, int R, int64_t K)
{
    return lora_shape_ok(M, R, K) ? lora_workspace_bytes(M, R, K) : QMV_ERR_SHAPE;
}

qmv_status qmv_lora_add(const void *x, int x_type, const void *a, const void *b, int w_type, const int32_t *adapter,
                        const float *scale, const float *base, float *y, void *workspace, int64_t workspace_bytes,
                        int M, int64_t N, int64_t K, int R, int L, qmv_stream_t stream)
{
    if ((x_type != QMV_F32 && x_type != QMV_F16) || !is_16bit(w_type)) return QMV_ERR_SHAPE;
    if (!lora_shape_ok(M, R, K) || N < 0 || N > kMaxDim || L < 0) return QMV_ERR_SHAPE;
    if (M == 0 || N == 0) return QMV_OK;
    if (!base || !y) return QMV_ERR_NULL;
    if (misaligned(base, 4) || misaligned(y, 4)) return QMV_ERR_ALIGN;
    if (L == 0 || K == 0) {   // no adapter, or an empty sum
        if (y == base) return QMV_OK;
        return from_cuda(cudaMemcpyAsync(y, base, static_cast<size_t>(M) * static_cast<size_t>(N) * sizeof(float),
                                         cudaMemcpyDeviceToDevice, stream));
    }
    if (!x || !a || !b || !adapter || !scale || !workspace) return QMV_ERR_NULL;
    if (misaligned(x, 16) || misaligned(a, 16) || misaligned(b, 16) || misaligned(adapter, 4) || misaligned(scale, 4) ||
        misaligned(workspace, 16))
        return QMV_ERR_ALIGN;
    if (workspace_bytes < lora_workspace_bytes(M, R, K)) return QMV_ERR_SHAPE;
    return from_cuda(launch_lora(LoraArgs{x, a, b, adapter, scale, base, y, static_cast<float *>(workspace), x_type,
                                          w_type, M, R, L, N, K},
                                 stream));
}

qmv_status qmv_rope_append(const float *qkv, const int32_t *positions, const float *table, const uint8_t *axis_of_pair,
                           const int64_t *slots, void *q, void *k_cache, void *v_cache, int type, int interleaved,
                           int M, int Hq, int Hkv, int D, int rot, int axes, int n_positions, int64_t n_slots,
                           qmv_stream_t stream)
{
    if (!is_16bit(type) || M < 0 || Hq < 1 || Hkv < 1 || Hq > 65536 || Hkv > 65536) return QMV_ERR_SHAPE;
    if (D < 8 || D > 2 * kMaxRopePairs || D % 8 != 0 || rot < 0 || rot > D || rot % 8 != 0) return QMV_ERR_SHAPE;
    if (axes < 1 || axes > kMaxRopeAxes || n_positions < (rot > 0 ? 1 : 0) || n_slots < 0) return QMV_ERR_SHAPE;
    if (M == 0) return QMV_OK;
    if (!qkv || !q || !slots || !k_cache || !v_cache) return QMV_ERR_NULL;
    if (rot > 0 && (!positions || !table || !axis_of_pair)) return QMV_ERR_NULL;
    if (misaligned(qkv, 16) || misaligned(q, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) ||
        misaligned(table, 16) || misaligned(positions, 4) || misaligned(slots, 8))
        return QMV_ERR_ALIGN;
    RopeArgs g{qkv, positions, table, slots, q, k_cache, v_cache, n_slots, type, M, Hq, Hkv, D, rot, axes, n_positions,
               interleaved != 0, {}};
    for (int i = 0; i < rot / 2; ++i) {
        if (axis_of_pair[i] >= axes) return QMV_ERR_SHAPE;
        g.axis_of_pair[i] = axis_of_pair[i];
    }
    return from_cuda(launch_rope(g, stream));
}

qmv_status qmv_norm_rope_append(const float *qkv, const int32_t *positions, const float *table,
                                const uint8_t *axis_of_pair, const int64_t *slots, const float *q_norm,
                                const float *k_norm, float eps, void *q, void *k_cache, void *v_cache, int type,
                                int interleaved, int M, int Hq, int Hkv, int D, int rot, int axes, int n_positions,
                                int64_t n_slots, qmv_stream_t stream)
{
    const qmv_status st = norm_rope_shape(type, M, Hq, Hkv, D, rot, axes, n_positions, n_slots, eps, false);
    if (st != QMV_OK || M == 0) return st;
    return run_norm_rope(NormRopeArgs{qkv, positions, table, slots, q_norm, k_norm, q, k_cache, v_cache, nullptr, nullptr,
                                      n_slots, eps, 1.0f / static_cast<float>(D), type, M, Hq, Hkv, D, rot, n_positions, interleaved != 0, {}},
                         axis_of_pair, axes, stream);
}

qmv_status qmv_rope_append_e4m3(const float *qkv, const int32_t *positions, const float *table,
                                const uint8_t *axis_of_pair, const int64_t *slots, const float *q_norm,
                                const float *k_norm, float eps, void *q, void *k_cache, void *v_cache, float *k_scale,
                                float *v_scale, int type, int interleaved, int M, int Hq, int Hkv, int D, int rot,
                                int axes, int n_positions, int64_t n_slots, qmv_stream_t stream)
{
    const qmv_status st = norm_rope_shape(type, M, Hq, Hkv, D, rot, axes, n_positions, n_slots, eps, true);
    if (st != QMV_OK || M == 0) return st;
    if (!k_scale || !v_scale) return QMV_ERR_NULL;
    return run_norm_rope(NormRopeArgs{qkv, positions, table, slots, q_norm, k_norm, q, k_cache, v_cache, k_scale, v_scale,
                                      n_slots, eps, 1.0f / static_cast<float>(D), type, M, Hq, Hkv, D, rot, n_positions, interleaved != 0, {}},
                         axis_of_pair, axes, stream);
}

int64_t qmv_paged_attention_e4m3_workspace(int B, int T, int Hq, int Hkv, int D, int64_t max_len)
{
    return paged_shape_ok(B, T, Hq, Hkv, D, max_len) ? paged_workspace_bytes(B, T * (Hq / Hkv)) : QMV_ERR_SHAPE;
}

qmv_status qmv_paged_attention_e4m3(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                                    const float *v_scale, int type, int64_t n_pages, int page, const int32_t *table,
                                    int table_pages, const int32_t *lens, int64_t max_len, float scale, void *out,
                                    void *workspace, int64_t workspace_bytes, int B, int T, int Hq, int Hkv, int D,
                                    qmv_stream_t stream)
{
    if (!is_16bit(type) || !paged_shape_ok(B, T, Hq, Hkv, D, max_len)) return QMV_ERR_SHAPE;
    if (page < 16 || page > 256 || (page & (page - 1)) != 0 || n_pages < 0 || n_pages > kMaxDim || table_pages < 0)
        return QMV_ERR_SHAPE;
    if (max_len > static_cast<int64_t>(table_pages) * page) return QMV_ERR_SHAPE;
    if (n_pages == 0 && max_len > 0) return QMV_ERR_SHAPE;
    if (!(scale > 0.0f) || std::isinf(scale)) return QMV_ERR_SHAPE;
    if (B == 0) return QMV_OK;
    if (!q || !out || !lens) return QMV_ERR_NULL;
    if (max_len > 0 && (!k_cache || !v_cache || !k_scale || !v_scale || !table)) return QMV_ERR_NULL;
    if (misaligned(q, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) || misaligned(out, 16) ||
        misaligned(k_scale, 4) || misaligned(v_scale, 4) || misaligned(table, 4) || misaligned(lens, 4) ||
        misaligned(workspace, 16))
        return QMV_ERR_ALIGN;
    const int64_t need = paged_workspace_bytes(B, T * (Hq / Hkv));
    if (need > 0 && !workspace) return QMV_ERR_NULL;
    if (workspace_bytes < need) return QMV_ERR_SHAPE;
    return from_cuda(launch_paged_e4m3(PagedArgs{q, k_cache, v_cache, k_scale, v_scale, table, lens, out, workspace, n_pages,
                                                 max_len, scale, type, page, table_pages, B, T, Hq, Hkv, D},
                                       stream));
}

qmv_status qmv_sample(const float *logits, const float *u, const float *temperature, const int32_t *top_k,
                      const float *top_p, const float *min_p, int32_t *token, float *prob, int M, int V,
                      qmv_stream_t stream)
{
    if (M < 0 || M > 65535 || V < 1 || V > sample_max_vocabulary()) return QMV_ERR_SHAPE;
    if (M == 0) return QMV_OK;
    if (!logits || !u || !token) return QMV_ERR_NULL;
    if (misaligned(logits, 4) || misaligned(u, 4) || misaligned(temperature, 4) || misaligned(top_k, 4) ||
        misaligned(top_p, 4) || misaligned(min_p, 4) || misaligned(token, 4) || misaligned(prob, 4))
        return QMV_ERR_ALIGN;
    return from_cuda(launch_sample(SampleArgs{logits, u, temperature, top_k, top_p, min_p, token, prob, M, V}, stream));
}

int64_t qmv_prefix_attention_workspace(int B, int T, int Hq, int Hkv, int D, int64_t prefix_len, int64_t max_own)
{
    return attention_shape_ok(B, T, Hq, Hkv, D, prefix_len, max_own)
               ? attn_workspace_bytes(B, T, Hq, Hkv, D, prefix_len, max_own)
               : QMV_ERR_SHAPE;
}

qmv_status qmv_prefix_attention(const void *q, const void *k_cache, const void *v_cache, int type, int64_t n_pages,
                                int page, const int32_t *prefix_table, int64_t prefix_len, const int32_t *own_table,
                                int own_pages, const int32_t *own_len, int64_t max_own, float scale, void *out,
                                void *workspace, int64_t workspace_bytes, int B, int T, int Hq, int Hkv, int D,
                                qmv_stream_t stream)
{
    if (!is_16bit(type) || !attention_shape_ok(B, T, Hq, Hkv, D, prefix_len, max_own)) return QMV_ERR_SHAPE;
    if (page < 16 || page > 256 || (page & (page - 1)) != 0 || n_pages < 0 || n_pages > kMaxDim || own_pages < 0)
        return QMV_ERR_SHAPE;
    if (max_own > static_cast<int64_t>(own_pages) * page) return QMV_ERR_SHAPE;
    if (n_pages == 0 && (prefix_len > 0 || max_own > 0)) return QMV_ERR_SHAPE;
    if (!(scale > 0.0f) || std::isinf(scale)) return QMV_ERR_SHAPE;
    if (B == 0) return QMV_OK;
    if (!q || !out) return QMV_ERR_NULL;
    if ((prefix_len > 0 || max_own > 0) && (!k_cache || !v_cache)) return QMV_ERR_NULL;
    if ((prefix_len > 0 && !prefix_table) || (max_own > 0 && (!own_table || !own_len))) return QMV_ERR_NULL;
    if (misaligned(q, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) || misaligned(out, 16) ||
        misaligned(prefix_table, 4) || misaligned(own_table, 4) || misaligned(own_len, 4) || misaligned(workspace, 16))
        return QMV_ERR_ALIGN;
    const int64_t need = attn_workspace_bytes(B, T, Hq, Hkv, D, prefix_len, max_own);
    if (need > 0 && !workspace) return QMV_ERR_NULL;
    if (workspace_bytes < need) return QMV_ERR_SHAPE;
    return from_cuda(launch_attention(AttnArgs{q, k_cache, v_cache, prefix_table, own_table, own_len, out, workspace,
                                               n_pages, prefix_len, max_own, scale, type, page, own_pages, B, T, Hq,
                                               Hkv, D},
                                      stream));
}

qmv_status qmv_penalize_logits(const float *logits, const int32_t *tokens, int max_history, const int32_t *prompt_len,
                               const int32_t *total_len, const float *repetition, const float *presence,
                               const float *frequency, const int32_t *bias_tokens, const float *bias_values,
                               int max_bias, const uint32_t *mask, const int32_t *mask_row, int n_masks, float *y,
                               int M, int V, qmv_stream_t stream)
{
    if (M < 0 || M > 65535 || V < 0 || V > (1 << 30) || max_history < 0 || max_history > (1 << 29) || max_bias < 0 || n_masks < 0) return QMV_ERR_SHAPE;
    if (mask && !mask_row && n_masks < M) return QMV_ERR_SHAPE;
    if (M == 0 || V == 0) return QMV_OK;
    if (!logits || !y) return QMV_ERR_NULL;
    if (max_history > 0 && (!tokens || !prompt_len || !total_len)) return QMV_ERR_NULL;
    if (max_bias > 0 && (!bias_tokens || !bias_values)) return QMV_ERR_NULL;
    if (n_masks > 0 && !mask) return QMV_ERR_NULL;
    if (misaligned(logits, 4) || misaligned(y, 4) || misaligned(tokens, 4) || misaligned(prompt_len, 4) ||
        misaligned(total_len, 4) || misaligned(repetition, 4) || misaligned(presence, 4) || misaligned(frequency, 4) ||
        misaligned(bias_tokens, 4) || misaligned(bias_values, 4) || misaligned(mask, 4) || misaligned(mask_row, 4))
        return QMV_ERR_ALIGN;
    return from_cuda(launch_logits(LogitsArgs{logits, y, tokens, prompt_len, total_len, repetition, presence, frequency,
                                              bias_tokens, bias_values, mask, mask_row, M, V, max_history, max_bias,
                                              n_masks},
                                   stream));
}

}  // extern "C"
