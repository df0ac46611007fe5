// decode_ops.h -- host-side interface between the C ABI layer (abi_decode.cu) and the
// kernels of the operators that stand beside the matmuls in a decode step: adapters,
// rotary positions with the cache append, shared-prefix attention, logits. Not
// installed; not part of the ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qmv_internal.h"

namespace qmv {

// ---- low-rank adapters
struct LoraArgs {
    const void *x;           // [M][K]
    const void *a, *b;       // [L][R][K], [L][N][R]
    const int32_t *adapter;  // [M]
    const float *scale;      // [L]
    const float *base;       // [M][N]
    float *y;                // [M][N], may be base
    float *part;             // workspace: partial A x sums
    int x_type, w_type;      // QMV_F32 / QMV_F16 / QMV_BF16
    int M, R, L;
    int64_t N, K;
};
int64_t lora_workspace_bytes(int M, int R, int64_t K);
cudaError_t launch_lora(const LoraArgs &g, cudaStream_t s);

// ---- rotary positions and the cache append
constexpr int kMaxRopePairs = 128;
constexpr int kMaxRopeAxes = 4;
struct RopeArgs {
    const float *qkv;           // [M][(Hq + 2 Hkv) D]
    const int32_t *positions;   // [axes][M]
    const float *table;         // [n_positions][rot / 2][2]
    const int64_t *slots;       // [M]
    void *q, *k_cache, *v_cache;
    int64_t n_slots;
    int type, M, Hq, Hkv, D, rot, axes, n_positions, interleaved;
    uint8_t axis_of_pair[kMaxRopePairs];
};
cudaError_t launch_rope(const RopeArgs &g, cudaStream_t s);

// ---- attention over a shared prefix
struct AttnArgs {
    const void *q, *k_cache, *v_cache;
    const int32_t *prefix_table, *own_table, *own_len;
    void *out, *workspace;
    int64_t n_pages, prefix_len, max_own;
    float scale;
    int type, page, own_pages, B, T, Hq, Hkv, D;
};
int64_t attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int64_t prefix_len, int64_t max_own);
cudaError_t launch_attention(const AttnArgs &g, cudaStream_t s);

// ---- logits
struct LogitsArgs {
    const float *logits;
    float *y;
    const int32_t *tokens, *prompt_len, *total_len;
    const float *repetition, *presence, *frequency;
    const int32_t *bias_tokens;
    const float *bias_values;
    const uint32_t *mask;
    const int32_t *mask_row;
    int M, V, max_history, max_bias, n_masks;
};
cudaError_t launch_logits(const LogitsArgs &g, cudaStream_t s);

// Device error words of the operators that follow indices held in device memory.
cudaError_t read_error_word_rope(uint32_t *out, bool clear);
cudaError_t read_error_word_attention(uint32_t *out, bool clear);
cudaError_t read_error_word_logits(uint32_t *out, bool clear);

}  // namespace qmv
