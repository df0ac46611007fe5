// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   y[m] = base[m] + scale[a] B[a] (A[a] x[m]),  a = adapter[m]
// with A[a] [R][K], B[a] [N][R]. Two launches: A x for every row (partial sums over
// ranges of K), then B (A x) added to the projection's output.
//
// Rows that share an adapter are found on the device: each CTA compares the adapters of
// all M <= 96 rows with its own row's. The c rows of an adapter bring c CTAs a tile; they
// are cut into blocks of 8 rows, one tensor-core column each, so that the weights are
// read once for 8 rows and the number of working CTAs does not depend on who shares what.
//
// The products run on m16n8k8 TF32: 16-bit weights (binary16 or bfloat16) and binary16
// activations are exact in TF32, fp32 activations and A x go in as two terms whose sum
// keeps 22 bits, and sums are fp32. Bound by the weights' bytes: one row an adapter leaves
// 7 of the product's 8 columns empty and still reads memory at its rate.
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace qmv {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kBlockRows = 8;      // rows of a block: the product's columns
constexpr int kRankTile = 16;      // ranks of a shrink CTA, outputs of an expand step: the product's rows
constexpr int kMaxRows = 96, kMaxRank = 256;
constexpr int kSms = 152;

// D(16x8) += A(16x8, row) B(8x8, col) in TF32. A lane (g = lane / 4, t = lane % 4) holds
// a0 A[g][t], a1 A[g+8][t], a2 A[g][t+4], a3 A[g+8][t+4]; b0 B[t][g], b1 B[t+4][g];
// d0, d1 D[g][2t..], d2, d3 D[g+8][2t..].
__device__ __forceinline__ void mma_tf32(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// v as two TF32 terms: the first cut, the second rounded.
__device__ __forceinline__ void split_tf32(float v, float &hi, float &lo)
{
    hi = __uint_as_float(__float_as_uint(v) & 0xffffe000u);
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v - hi));
    lo = __uint_as_float(r);
}

template <typename W>
__device__ __forceinline__ float2 widen(uint32_t two)
{
    if constexpr (std::is_same_v<W, __half>) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&two));
    } else {
        return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
    }
}

// One step of 32 k on a 16 x 8 tile: lane (g, t) holds k 8t .. 8t + 7 of rows g and g + 8
// (w0, w1) and of column g (hi, and lo where `two` terms); the order of k within a product
// is free, as long as both operands have the same.
template <typename W, bool kTwo>
__device__ __forceinline__ void mma_step(float (&d)[4], uint4 w0, uint4 w1, const float (&hi)[8], const float (&lo)[8])
{
    const uint32_t a[4] = {w0.x, w0.y, w0.z, w0.w}, b[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 p = widen<W>(a[j]), q = widen<W>(b[j]);
        mma_tf32(d, p.x, q.x, p.y, q.y, hi[2 * j], hi[2 * j + 1]);
        if constexpr (kTwo) mma_tf32(d, p.x, q.x, p.y, q.y, lo[2 * j], lo[2 * j + 1]);
    }
}

// The rows that share row m's adapter, counted by one warp; rows[] gets those of its block.
struct Sharers {
    int adapter;       // -1: none
    int count, rank;   // rows that share it, of them before m
};
__device__ __forceinline__ Sharers find_sharers(const LoraArgs &g, int m, int lane)
{
    Sharers s;
    int a = __ldg(g.adapter + m);
    s.adapter = a >= 0 && a < g.L ? a : -1;
    s.count = s.rank = 0;
#pragma unroll
    for (int w = 0; w < kMaxRows / 32; ++w) {
        const int i = 32 * w + lane;
        const uint32_t same = __ballot_sync(0xffffffffu, i < g.M && __ldg(g.adapter + (i < g.M ? i : 0)) == a);
        const uint32_t before = m >= 32 * w + 32 ? 0xffffffffu : m <= 32 * w ? 0u : (1u << (m - 32 * w)) - 1u;
        s.count += __popc(same);
        s.rank += __popc(same & before);
    }
    return s;
}
// By one warp: the rows 8 block .. 8 block + 7 of those that share row m's adapter.
__device__ __forceinline__ void list_rows(const LoraArgs &g, int m, int lane, int block, int *rows)
{
    const int a = __ldg(g.adapter + m);
    int seen = 0;
#pragma unroll
    for (int w = 0; w < kMaxRows / 32; ++w) {
        const int i = 32 * w + lane;
        const bool mine = i < g.M && __ldg(g.adapter + (i < g.M ? i : 0)) == a;
        const uint32_t same = __ballot_sync(0xffffffffu, mine);
        const int at = seen + __popc(same & ((1u << lane) - 1u)) - kBlockRows * block;
        if (mine && at >= 0 && at < kBlockRows) rows[at] = i;
        seen += __popc(same);
    }
}

// Partial sums of A x: grid (rows, rank tiles, ranges of K). The CTA of a row's rank-th
// sharer takes block `rank` of the rows, if there is one; a warp a range of warp_k.
template <typename X, typename W>
__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(LoraArgs g, int warp_k)
{
    __shared__ float sums[kWarps][kRankTile][kBlockRows];
    __shared__ int rows[kBlockRows];
    const int m = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t = lane & 3;
    grid_dependency_wait();
    grid_launch_dependents();
    const Sharers s = find_sharers(g, m, lane);
    if (s.adapter < 0 || s.rank * kBlockRows >= s.count) return;
    const int nrows = min(kBlockRows, s.count - s.rank * kBlockRows);
    if (warp == 0) list_rows(g, m, lane, s.rank, rows);
    const int r0 = blockIdx.y * kRankTile;
    const int64_t k0 = (static_cast<int64_t>(blockIdx.z) * kWarps + warp) * warp_k, k1 = min(k0 + warp_k, g.K);
    const W *a0 = static_cast<const W *>(g.a) + (static_cast<int64_t>(s.adapter) * g.R + r0 + gid) * g.K;
    const bool has0 = r0 + gid < g.R, has1 = r0 + gid + 8 < g.R;
    __syncthreads();
    const bool has_x = gid < nrows;
    const X *x = static_cast<const X *>(g.x) + (has_x ? rows[gid] : 0) * g.K;
    const uint64_t stream = policy_evict_first();
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t kb = k0; kb < k1; kb += 128) {   // four steps' loads in flight
        uint4 w0[4], w1[4];
        constexpr int kXLoads = std::is_same_v<X, float> ? 2 : 1;
        uint4 xv[4][kXLoads];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int64_t k = kb + 32 * c + 8 * t;
            const bool in = k < k1;
            w0[c] = in && has0 ? ld_stream_v4(a0 + k, stream) : make_uint4(0, 0, 0, 0);
            w1[c] = in && has1 ? ld_stream_v4(a0 + 8 * g.K + k, stream) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kXLoads; ++i)
                xv[c][i] = in && has_x ? ld_shared_v4(reinterpret_cast<const uint4 *>(x + k) + i) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float hi[8], lo[8];
            if constexpr (std::is_same_v<X, float>) {
                const uint32_t v[8] = {xv[c][0].x, xv[c][0].y, xv[c][0].z, xv[c][0].w, xv[c][1].x, xv[c][1].y, xv[c][1].z, xv[c][1].w};
#pragma unroll
                for (int i = 0; i < 8; ++i) split_tf32(__uint_as_float(v[i]), hi[i], lo[i]);
            } else {
                const uint32_t v[4] = {xv[c][0].x, xv[c][0].y, xv[c][0].z, xv[c][0].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = widen<__half>(v[i]);
                    hi[2 * i] = f.x;
                    hi[2 * i + 1] = f.y;
                }
            }
            mma_step<W, std::is_same_v<X, float>>(d, w0[c], w1[c], hi, lo);
        }
    }
    sums[warp][gid][2 * t] = d[0];
    sums[warp][gid][2 * t + 1] = d[1];
    sums[warp][gid + 8][2 * t] = d[2];
    sums[warp][gid + 8][2 * t + 1] = d[3];
    __syncthreads();
    if (tid < kRankTile * kBlockRows) {
        const int r = tid % kRankTile, row = tid / kRankTile;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += sums[w][r][row];
        if (row < nrows && r0 + r < g.R) g.part[(static_cast<int64_t>(blockIdx.z) * g.M + rows[row]) * g.R + r0 + r] = sum;
    }
}

// y = base + scale B (A x): grid (rows, gridDim.y). The c sharers of an adapter have c x
// gridDim.y CTAs: those of block b of the rows are the sharers b, b + blocks, ...; their
// warps take the 16-output steps of N in turn.
template <typename W>
__global__ void __launch_bounds__(kThreads) lora_expand_kernel(LoraArgs g, int splits)
{
    __shared__ __align__(16) float ax[2][kBlockRows][kMaxRank + 4];   // scale A x as two TF32 terms
    __shared__ int rows[kBlockRows];
    const int m = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t = lane & 3;
    grid_launch_dependents();
    const Sharers s = find_sharers(g, m, lane);   // (the launch before began after whatever wrote these)
    if (s.adapter < 0) {
        grid_dependency_wait();
        if (g.y != g.base)
            for (int64_t n = static_cast<int64_t>(blockIdx.y) * kThreads + tid; n < g.N; n += static_cast<int64_t>(gridDim.y) * kThreads)
                g.y[m * g.N + n] = g.base[m * g.N + n];
        return;
    }
    const int blocks = (s.count + kBlockRows - 1) / kBlockRows, block = s.rank % blocks;
    const int nrows = min(kBlockRows, s.count - block * kBlockRows);
    const int mine = s.rank / blocks, ctas = (s.count - block + blocks - 1) / blocks;
    const int64_t steps = (g.N + kRankTile - 1) / kRankTile, stride = static_cast<int64_t>(ctas) * gridDim.y * kWarps;
    int64_t step = (static_cast<int64_t>(mine) * gridDim.y + blockIdx.y) * kWarps + warp;
    const W *b = static_cast<const W *>(g.b) + static_cast<int64_t>(s.adapter) * g.N * g.R;
    const uint64_t stream = policy_evict_first();
    // 64 ranks of a step: lane (g, t) holds ranks 32 c + 8 t .. + 7 of outputs g and g + 8
    uint4 w[2][2];
    auto load = [&](int64_t st, int r0) {
        const int64_t n = st * kRankTile + gid;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = r0 + 32 * c + 8 * t;
            w[c][0] = n < g.N && r < g.R ? ld_stream_v4(b + n * g.R + r, stream) : make_uint4(0, 0, 0, 0);
            w[c][1] = n + 8 < g.N && r < g.R ? ld_stream_v4(b + (n + 8) * g.R + r, stream) : make_uint4(0, 0, 0, 0);
        }
    };
    if (step < steps) load(step, 0);
    if (warp == 0) list_rows(g, m, lane, block, rows);
    __syncthreads();
    grid_dependency_wait();
    const float scale = __ldg(g.scale + s.adapter);
    const int ranks = (g.R + 63) & ~63;
    for (int i = tid; i < kBlockRows * ranks; i += kThreads) {
        const int row = i / ranks, r = i % ranks;
        float sum = 0.0f;
        if (row < nrows && r < g.R) {
            const float *p = g.part + static_cast<int64_t>(rows[row]) * g.R + r;
#pragma unroll 4
            for (int k = 0; k < splits; ++k) sum += p[static_cast<int64_t>(k) * g.M * g.R];
        }
        float hi, lo;
        split_tf32(sum * scale, hi, lo);
        ax[0][row][r] = hi;
        ax[1][row][r] = lo;
    }
    __syncthreads();
    for (; step < steps; step += stride) {
        // the projection's output for this step: rows 2 t and 2 t + 1, outputs g and g + 8
        float out[4];
        int64_t at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = step * kRankTile + gid + (i & 2 ? 8 : 0);
            const int row = 2 * t + (i & 1);
            at[i] = row < nrows && n < g.N ? rows[row] * g.N + n : -1;
            out[i] = at[i] >= 0 ? g.base[at[i]] : 0.0f;
        }
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int r0 = 0; r0 < g.R; r0 += 64) {
            uint4 now[2][2] = {{w[0][0], w[0][1]}, {w[1][0], w[1][1]}};
            const bool more = r0 + 64 < g.R;
            if (more || step + stride < steps) load(more ? step : step + stride, more ? r0 + 64 : 0);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    *reinterpret_cast<float4 *>(hi + i) = *reinterpret_cast<const float4 *>(&ax[0][gid][r0 + 32 * c + 8 * t + i]);
                    *reinterpret_cast<float4 *>(lo + i) = *reinterpret_cast<const float4 *>(&ax[1][gid][r0 + 32 * c + 8 * t + i]);
                }
                mma_step<W, true>(d, now[c][0], now[c][1], hi, lo);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at[i] >= 0) g.y[at[i]] = out[i] + d[i];
    }
}

// K of a shrink warp: 512 (at most 64 products in a chain of sums) where that fills the SMs
// twice, else 128, one round of loads.
int shrink_k(int M, int R, int64_t K)
{
    const int64_t ctas = static_cast<int64_t>(M) * ((R + kRankTile - 1) / kRankTile) * ((K + 512 * kWarps - 1) / (512 * kWarps));
    return ctas >= 2 * kSms ? 512 : 128;
}

int64_t shrink_splits(int M, int R, int64_t K)
{
    const int64_t per = static_cast<int64_t>(shrink_k(M, R, K)) * kWarps;
    return (K + per - 1) / per;
}

template <typename X, typename W>
cudaError_t launch_both(const LoraArgs &g, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    const int splits = static_cast<int>(shrink_splits(g.M, g.R, g.K));
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>(g.M), static_cast<unsigned>((g.R + kRankTile - 1) / kRankTile), static_cast<unsigned>(splits));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    cudaError_t e = cudaLaunchKernelEx(&cfg, lora_shrink_kernel<X, W>, g, shrink_k(g.M, g.R, g.K));
    if (e != cudaSuccess) return e;
    // starts beside the shrink launch, loads its first weights and waits for it; CTAs for
    // one step a warp, but no more than eight an SM
    const int64_t tiles = (g.N + kRankTile * kWarps - 1) / (kRankTile * kWarps);
    cfg.gridDim = dim3(static_cast<unsigned>(g.M), static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(tiles, 8 * kSms / g.M))));
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_expand_kernel<W>, g, splits);
}

}  // namespace

int64_t lora_workspace_bytes(int M, int R, int64_t K) { return shrink_splits(M, R, K) * M * R * 4; }

cudaError_t launch_lora(const LoraArgs &g, cudaStream_t s)
{
    route_hit(kRouteLora);
    if (g.x_type == QMV_F32)
        return g.w_type == QMV_F16 ? launch_both<float, __half>(g, s) : launch_both<float, __nv_bfloat16>(g, s);
    return g.w_type == QMV_F16 ? launch_both<__half, __half>(g, s) : launch_both<__half, __nv_bfloat16>(g, s);
}

}  // namespace qmv
