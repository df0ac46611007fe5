// logits.cu -- penalties for repeated tokens, biases and grammar masks on logits, one
// row a request. For token v of row m, with seen = v is in the row's history and n = how
// often it is in the history from prompt_len on:
//   y = seen ? (x > 0 ? x / repetition : x repetition) : x
//   y = y - (frequency n + presence [n > 0]) + (sum of v's biases);  y = -inf where the mask's bit is 0
#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace qmv {
namespace {

__device__ uint32_t g_logits_error;

constexpr int kThreads = 256;
constexpr int kTile = 8192;          // tokens of the vocabulary a CTA
constexpr uint32_t kSeen = 1u << 31; // the bit above a token's count: it is in the history at all

__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LogitsArgs g)
{
    __shared__ uint32_t count[kTile];
    const int m = blockIdx.y, v0 = blockIdx.x * kTile, n = min(kTile, g.V - v0), tid = threadIdx.x;
    grid_launch_dependents();
    grid_dependency_wait();
    for (int i = tid; i < n; i += kThreads) count[i] = 0;
    __syncthreads();
    const int32_t *tokens = g.tokens + static_cast<int64_t>(m) * g.max_history;
    int total = g.total_len ? g.total_len[m] : 0;
    if (total > g.max_history) {
        if (tid == 0) atomicOr(&g_logits_error, kErrIndex);
        total = g.max_history;
    }
    const int prompt = total > 0 ? g.prompt_len[m] : 0;
    for (int i = tid; i < total; i += kThreads) {
        const int v = tokens[i];
        if (v >= g.V) {
            atomicOr(&g_logits_error, kErrIndex);
        } else if (v >= v0 && v < v0 + n) {
            atomicOr(&count[v - v0], kSeen);
            if (i >= prompt) atomicAdd(&count[v - v0], 1u);
        }
    }
    __syncthreads();
    const float rep = g.repetition ? g.repetition[m] : 1.0f;
    const float freq = g.frequency ? g.frequency[m] : 0.0f, pres = g.presence ? g.presence[m] : 0.0f;
    const int mr = g.mask ? (g.mask_row ? g.mask_row[m] : m) : -1;
    if (mr >= g.n_masks && g.mask && tid == 0) atomicOr(&g_logits_error, kErrIndex);
    const uint32_t *mask = mr >= 0 && mr < g.n_masks ? g.mask + static_cast<int64_t>(mr) * ((g.V + 31) / 32) : nullptr;
    const int32_t *bt = g.bias_tokens ? g.bias_tokens + static_cast<int64_t>(m) * g.max_bias : nullptr;
    const float *bv = g.bias_values + static_cast<int64_t>(m) * g.max_bias;
    for (int i = tid; i < n; i += kThreads) {
        const int v = v0 + i;
        const int64_t at = static_cast<int64_t>(m) * g.V + v;
        float x = g.logits[at];
        const uint32_t c = count[i];
        if (c) {
            x = x > 0.0f ? x / rep : x * rep;
            if (c & ~kSeen) x -= freq * static_cast<float>(c & ~kSeen) + pres;
        }
        if (bt)
            for (int j = 0; j < g.max_bias; ++j)
                if (bt[j] == v) x += bv[j];
        if (mask && !((mask[v >> 5] >> (v & 31)) & 1u)) x = -INFINITY;
        g.y[at] = x;
    }
}

}  // namespace

cudaError_t launch_logits(const LogitsArgs &g, cudaStream_t s)
{
    route_hit(kRouteLogits);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>((g.V + kTile - 1) / kTile), static_cast<unsigned>(g.M));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    return cudaLaunchKernelEx(&cfg, logits_kernel, g);
}

cudaError_t read_error_word_logits(uint32_t *out, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_logits_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_logits_error, &zero, sizeof(uint32_t));
}

}  // namespace qmv
