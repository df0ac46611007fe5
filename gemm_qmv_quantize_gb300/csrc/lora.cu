// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   y[m] = base[m] + scale[a] B[a] (A[a] x[m]),  a = adapter[m]
// with A[a] [R][K], B[a] [N][R]. Two launches: A x for every row, then B (A x) added to
// the projection's output. Sums and A x are held in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace qmv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// One warp a dot product A[a][r] . x[m].
template <typename X, typename W>
__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(LoraArgs g)
{
    const int m = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.y * (kThreads / 32) + warp;
    grid_dependency_wait();
    grid_launch_dependents();
    const int a = g.adapter[m];
    if (a < 0 || a >= g.L || r >= g.R) return;
    const X *x = static_cast<const X *>(g.x) + m * g.K;
    const W *w = static_cast<const W *>(g.a) + (static_cast<int64_t>(a) * g.R + r) * g.K;
    float sum = 0.0f;
    for (int64_t k = lane; k < g.K; k += 32) sum = fmaf(to_f32(w[k]), to_f32(x[k]), sum);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) g.part[m * g.R + r] = sum;
}

// One thread an output.
template <typename W>
__global__ void __launch_bounds__(kThreads) lora_expand_kernel(LoraArgs g)
{
    const int m = blockIdx.y;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    grid_launch_dependents();
    grid_dependency_wait();
    if (n >= g.N) return;
    const int a = g.adapter[m];
    float sum = 0.0f;
    if (a >= 0 && a < g.L) {
        const W *w = static_cast<const W *>(g.b) + (static_cast<int64_t>(a) * g.N + n) * g.R;
        for (int r = 0; r < g.R; ++r) sum = fmaf(to_f32(w[r]), g.part[m * g.R + r], sum);
        sum *= g.scale[a];
    }
    g.y[m * g.N + n] = g.base[m * g.N + n] + sum;
}

template <typename W>
cudaError_t launch_expand(const LoraArgs &g, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>((g.N + kThreads - 1) / kThreads), static_cast<unsigned>(g.M));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_expand_kernel<W>, g);
}

template <typename X, typename W>
cudaError_t launch_both(const LoraArgs &g, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>(g.M), static_cast<unsigned>((g.R + kThreads / 32 - 1) / (kThreads / 32)));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    cudaError_t e = cudaLaunchKernelEx(&cfg, lora_shrink_kernel<X, W>, g);
    return e != cudaSuccess ? e : launch_expand<W>(g, s);
}

}  // namespace

int64_t lora_workspace_bytes(int M, int R, int64_t) { return static_cast<int64_t>(M) * R * 4; }

cudaError_t launch_lora(const LoraArgs &g, cudaStream_t s)
{
    route_hit(kRouteLora);
    if (g.x_type == QMV_F32)
        return g.w_type == QMV_F16 ? launch_both<float, __half>(g, s) : launch_both<float, __nv_bfloat16>(g, s);
    return g.w_type == QMV_F16 ? launch_both<__half, __half>(g, s) : launch_both<__half, __nv_bfloat16>(g, s);
}

}  // namespace qmv
