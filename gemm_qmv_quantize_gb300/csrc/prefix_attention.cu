// prefix_attention.cu -- attention of a batch whose requests share a long prefix: query
// rows see the prefix's keys and their request's own, both in a paged cache:
//   o = softmax(scale [q Kp^T, q Ko^T]) [Vp; Vo]
// with the softmax's maximum, sum and the output sums in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace qmv {
namespace {

__device__ uint32_t g_attention_error;

constexpr int kThreads = 128;   // keys a step

__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, __half *o) { *o = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(v); }

// One CTA a query row (token, head): 128 keys a step, one a thread, with the running
// maximum and sum of the softmax; then one output dimension a thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) attention_kernel(const __grid_constant__ AttnArgs g)
{
    __shared__ float q[128], p[kThreads], red[kThreads / 32];
    __shared__ int64_t at[kThreads];
    const int bt = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, b = bt / g.T, t = bt - b * g.T;
    const int hk = h / (g.Hq / g.Hkv);
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t row = (static_cast<int64_t>(bt) * g.Hq + h) * g.D;
    if (tid < g.D) q[tid] = to_f32(static_cast<const T *>(g.q)[row + tid]) * g.scale;
    int64_t own = g.max_own > 0 ? g.own_len[b] : 0;
    if (own > g.max_own) {
        if (tid == 0) atomicOr(&g_attention_error, kErrIndex);
        own = g.max_own;
    }
    own = max(static_cast<int64_t>(0), own - g.T + 1 + t);
    const int64_t keys = g.prefix_len + own;
    float top = -INFINITY, sum = 0.0f, acc = 0.0f;
    for (int64_t k0 = 0; k0 < keys; k0 += kThreads) {
        __syncthreads();
        const int64_t k = k0 + tid;
        float s = -INFINITY;
        if (k < keys) {
            const int64_t j = k < g.prefix_len ? k : k - g.prefix_len;
            const int32_t *table = k < g.prefix_len ? g.prefix_table : g.own_table + static_cast<int64_t>(b) * g.own_pages;
            int64_t pg = table[j / g.page];
            if (pg < 0 || pg >= g.n_pages) {
                atomicOr(&g_attention_error, kErrIndex);
                pg = 0;
            }
            at[tid] = ((pg * g.page + j % g.page) * g.Hkv + hk) * g.D;
            const T *kr = static_cast<const T *>(g.k_cache) + at[tid];
            s = 0.0f;
            for (int d = 0; d < g.D; ++d) s = fmaf(q[d], to_f32(kr[d]), s);
        }
        float m = s;
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((tid & 31) == 0) red[tid >> 5] = m;
        __syncthreads();
        m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float next = fmaxf(top, m), fix = __expf(top - next);
        const float e = k < keys ? __expf(s - next) : 0.0f;
        p[tid] = e;
        __syncthreads();
        acc *= fix;
        sum *= fix;
        const int n = static_cast<int>(min(keys - k0, static_cast<int64_t>(kThreads)));
        for (int i = 0; i < n; ++i) {
            sum += p[i];
            if (tid < g.D) acc = fmaf(p[i], to_f32(static_cast<const T *>(g.v_cache)[at[i] + tid]), acc);
        }
        top = next;
    }
    if (tid < g.D) from_f32(sum > 0.0f ? acc / sum : 0.0f, static_cast<T *>(g.out) + row + tid);
}

}  // namespace

int64_t attn_workspace_bytes(int, int, int, int, int, int64_t, int64_t) { return 0; }

cudaError_t launch_attention(const DeviceInfo &, const AttnArgs &g, cudaStream_t s)
{
    route_hit(kRoutePrefixAttention);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>(g.B * g.T), static_cast<unsigned>(g.Hq));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    return g.type == QMV_F16 ? cudaLaunchKernelEx(&cfg, attention_kernel<__half>, g)
                             : cudaLaunchKernelEx(&cfg, attention_kernel<__nv_bfloat16>, g);
}

cudaError_t read_error_word_attention(uint32_t *out, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_attention_error, sizeof(uint32_t));
    if (e != cudaSuccess || !clear) return e;
    const uint32_t zero = 0;
    return cudaMemcpyToSymbol(g_attention_error, &zero, sizeof(uint32_t));
}

}  // namespace qmv
