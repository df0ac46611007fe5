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
// keeps 22 bits. The tensor core cuts its running sums, so that a stage of 64 has sums of
// its own (8 products long) that are added in fp32, rounded: chains over all of K were off by
// 7e-7 of the outputs (5120 long). Bound by the weights' bytes: one row an adapter leaves
// 7 of the product's 8 columns empty and still reads memory at its rate. A lane's share of
// the operands comes by asynchronous copies into shared memory of its own, several stages
// ahead: 96 adapters of rank 64 beside 17408 x 5120 take 62 us, 4.7 TB/s (loads into
// registers: 65 us). The expand launch alone, 50 us for 227 MB, is short of issue slots
// (61 % used) as much as of bandwidth: weights are widened by hand and meet two terms each.
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
constexpr int kMaxRows = 96;
constexpr int kSms = 152;
constexpr int kSmShared = 228 * 1024, kCtaShared = 1024;   // shared memory of an SM; what a CTA takes beside its own
constexpr int kStages = 4;         // of 64 k or ranks, in flight for a warp

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

// v as two TF32 terms: the first cut (NaN as NaN: its payload may lie in what is cut), the
// second rounded (NaN beside an infinity).
__device__ __forceinline__ void split_tf32(float v, float &hi, float &lo)
{
    hi = v == v ? __uint_as_float(__float_as_uint(v) & 0xffffe000u) : v + v;
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v - hi));
    lo = __uint_as_float(r);
}

// Sums of first and of second terms. An infinity among the operands shows in the first
// terms' sum, and in the second's only as NaN (inf - inf, or 0 x inf).
__device__ __forceinline__ float both_terms(float first, float second) { return isfinite(first) ? first + second : first; }

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
// is free, as long as both operands have the same. The second terms have sums of their own.
template <typename W, bool kTwo>
__device__ __forceinline__ void mma_step(float (&d)[4], float (&e)[4], uint4 w0, uint4 w1, const float (&hi)[8], const float (&lo)[8])
{
    const uint32_t a[4] = {w0.x, w0.y, w0.z, w0.w}, b[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 p = widen<W>(a[j]), q = widen<W>(b[j]);
        mma_tf32(d, p.x, q.x, p.y, q.y, hi[2 * j], hi[2 * j + 1]);
        if constexpr (kTwo) mma_tf32(e, p.x, q.x, p.y, q.y, lo[2 * j], lo[2 * j + 1]);
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

// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void copy_or_zero(void *dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last n groups of this thread's copies have landed.
template <int n>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

template <typename X>
constexpr int kXPieces = std::is_same_v<X, float> ? 2 : 1;   // 16-byte pieces of 8 activations

template <typename X>
constexpr int shrink_smem() { return kWarps * kStages * (4 + 2 * kXPieces<X>) * 512; }

// Partial sums of A x: grid (rows, rank tiles, ranges of K). The CTA of a row's rank-th
// sharer takes block `rank` of the rows, if there is one; a warp a range of warp_k, in
// stages of 64.
template <typename X, typename W>
__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(LoraArgs g, int warp_k)
{
    extern __shared__ __align__(16) uint8_t ring[];   // [warp][stage][piece][lane] of 16 bytes
    __shared__ float sums[kWarps][kRankTile][kBlockRows];
    __shared__ int rows[kBlockRows];
    constexpr int kP = kXPieces<X>, kPieces = 4 + 2 * kP;
    const int m = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t = lane & 3;
    grid_dependency_wait();
    grid_launch_dependents();
    const Sharers s = find_sharers(g, m, lane);
    if (s.adapter < 0 || s.rank * kBlockRows >= s.count) return;
    const int nrows = min(kBlockRows, s.count - s.rank * kBlockRows);
    if (warp == 0) list_rows(g, m, lane, s.rank, rows);
    const int r0 = blockIdx.y * kRankTile;
    const int64_t k0 = (static_cast<int64_t>(blockIdx.z) * kWarps + warp) * warp_k, k1 = min(k0 + warp_k, g.K);
    const W *a = static_cast<const W *>(g.a) + (static_cast<int64_t>(s.adapter) * g.R + r0 + gid) * g.K;
    const bool has0 = r0 + gid < g.R, has1 = r0 + gid + 8 < g.R;
    const int stages = k1 > k0 ? static_cast<int>((k1 - k0 + 63) / 64) : 0;
    uint4 *mine = reinterpret_cast<uint4 *>(ring) + (warp * kStages * kPieces) * 32 + lane;
    auto piece = [&](int st, int i) { return mine + ((st % kStages) * kPieces + i) * 32; };
    auto load_a = [&](int st) {
        if (st >= stages) return;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int64_t k = k0 + 64 * st + 32 * c + 8 * t;
            const bool in = k < k1;
            copy_or_zero(piece(st, 2 * c), in && has0 ? a + k : g.a, in && has0);
            copy_or_zero(piece(st, 2 * c + 1), in && has1 ? a + 8 * g.K + k : g.a, in && has1);
        }
    };
    for (int st = 0; st < kStages - 1; ++st) load_a(st);
    __syncthreads();
    const bool has_x = gid < nrows;
    const X *x = static_cast<const X *>(g.x) + (has_x ? rows[gid] : 0) * g.K;
    auto load_x = [&](int st) {
        if (st < stages) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int64_t k = k0 + 64 * st + 32 * c + 8 * t;
                const bool in = k < k1 && has_x;
#pragma unroll
                for (int i = 0; i < kP; ++i)
                    copy_or_zero(piece(st, 4 + c * kP + i), in ? static_cast<const void *>(x + k + 4 * i) : g.x, in);
            }
        }
        copies_commit();
    };
    for (int st = 0; st < kStages - 1; ++st) load_x(st);
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int st = 0; st < stages; ++st) {
        copies_wait<kStages - 2>();
        load_a(st + kStages - 1);   // (into the stage that this lane read last)
        load_x(st + kStages - 1);
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}, rest[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float hi[8], lo[8];
            if constexpr (kP == 2) {
                const uint4 p = *piece(st, 4 + 2 * c), q = *piece(st, 5 + 2 * c);
                const uint32_t v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) split_tf32(__uint_as_float(v[i]), hi[i], lo[i]);
            } else {
                const uint4 p = *piece(st, 4 + c);
                const uint32_t v[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = widen<__half>(v[i]);
                    hi[2 * i] = f.x;
                    hi[2 * i + 1] = f.y;
                }
            }
            mma_step<W, kP == 2>(sum, rest, *piece(st, 2 * c), *piece(st, 2 * c + 1), hi, lo);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] += kP == 2 ? both_terms(sum[i], rest[i]) : sum[i];
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

// Shared memory of an expand CTA: its warps' stages, then scale A x as two TF32 terms,
// [2][8 rows][ranks + 4].
constexpr int kExpandRing = kWarps * kStages * 4 * 512;
int expand_smem(int R) { return kExpandRing + 2 * kBlockRows * (((R + 63) & ~63) + 4) * 4; }

// y = base + scale B (A x): grid (rows, gridDim.y). The c sharers of an adapter have c x
// gridDim.y CTAs: those of block b of the rows are the sharers b, b + blocks, ...; their
// warps take the 16-output steps of N in turn, in stages of 64 ranks.
template <typename W>
__global__ void __launch_bounds__(kThreads) lora_expand_kernel(LoraArgs g, int splits)
{
    extern __shared__ __align__(16) uint8_t ring[];
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
    const int64_t all = (g.N + kRankTile - 1) / kRankTile;
    const int stride = ctas * static_cast<int>(gridDim.y) * kWarps;
    const int first = (mine * static_cast<int>(gridDim.y) + static_cast<int>(blockIdx.y)) * kWarps + warp;
    const int steps = first < all ? static_cast<int>((all - first + stride - 1) / stride) : 0;   // of this warp
    const int per = (g.R + 63) / 64, stages = steps * per;   // stages a step, and of this warp
    const W *b = static_cast<const W *>(g.b) + static_cast<int64_t>(s.adapter) * g.N * g.R;
    uint4 *own = reinterpret_cast<uint4 *>(ring) + warp * kStages * 4 * 32 + lane;
    auto piece = [&](int st, int i) { return own + ((st % kStages) * 4 + i) * 32; };
    // the next stage to load: lane (g, t) has ranks 32 c + 8 t .. + 7 of outputs g and g + 8
    int next = 0, next_r = 0;
    int64_t next_n = static_cast<int64_t>(first) * kRankTile + gid;
    auto load = [&]() {
        if (next < stages) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = next_r + 32 * c + 8 * t;
                const bool in0 = next_n < g.N && r < g.R, in1 = next_n + 8 < g.N && r < g.R;
                copy_or_zero(piece(next, 2 * c), in0 ? b + next_n * g.R + r : b, in0);
                copy_or_zero(piece(next, 2 * c + 1), in1 ? b + (next_n + 8) * g.R + r : b, in1);
            }
        }
        copies_commit();
        ++next;
        next_r += 64;
        if (next_r >= g.R) {
            next_r = 0;
            next_n += static_cast<int64_t>(stride) * kRankTile;
        }
    };
    for (int i = 0; i < kStages - 1; ++i) load();
    if (warp == 0) list_rows(g, m, lane, block, rows);
    __syncthreads();
    grid_dependency_wait();
    const float scale = __ldg(g.scale + s.adapter);
    const int ranks = per * 64, pitch = ranks + 4;
    float *ax = reinterpret_cast<float *>(ring + kExpandRing), *ax_lo = ax + kBlockRows * pitch;
    for (int i = tid; i < kBlockRows * ranks; i += kThreads) {
        const int row = i / ranks, r = i % ranks;
        float sum = 0.0f;
        if (row < nrows && r < g.R) {
            const float *p = g.part + static_cast<int64_t>(rows[row]) * g.R + r;
#pragma unroll 4
            for (int k = 0; k < splits; ++k) sum += p[static_cast<int64_t>(k) * g.M * g.R];
        }
        split_tf32(sum * scale, ax[row * pitch + r], ax_lo[row * pitch + r]);
    }
    __syncthreads();
    // the projection's output for a step, loaded a step ahead: rows 2 t and 2 t + 1 (the
    // place of output 0, or -1), outputs g and g + 8
    const int64_t row0 = 2 * t < nrows ? rows[2 * t] * g.N : -1, row1 = 2 * t + 1 < nrows ? rows[2 * t + 1] * g.N : -1;
    float before[4];
    auto load_base = [&](int i) {
        const int64_t n = (static_cast<int64_t>(first) + static_cast<int64_t>(i) * stride) * kRankTile + gid;
        before[0] = i < steps && row0 >= 0 && n < g.N ? g.base[row0 + n] : 0.0f;
        before[1] = i < steps && row1 >= 0 && n < g.N ? g.base[row1 + n] : 0.0f;
        before[2] = i < steps && row0 >= 0 && n + 8 < g.N ? g.base[row0 + n + 8] : 0.0f;
        before[3] = i < steps && row1 >= 0 && n + 8 < g.N ? g.base[row1 + n + 8] : 0.0f;
    };
    load_base(0);
    for (int i = 0, st = 0; i < steps; ++i) {
        const float now[4] = {before[0], before[1], before[2], before[3]};
        load_base(i + 1);
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int r0 = 0; r0 < g.R; r0 += 64, ++st) {
            copies_wait<kStages - 2>();
            load();   // (into the stage that this lane read last)
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}, rest[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float hi[8], lo[8];
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    *reinterpret_cast<float4 *>(hi + j) = *reinterpret_cast<const float4 *>(ax + gid * pitch + r0 + 32 * c + 8 * t + j);
                    *reinterpret_cast<float4 *>(lo + j) = *reinterpret_cast<const float4 *>(ax_lo + gid * pitch + r0 + 32 * c + 8 * t + j);
                }
                mma_step<W, true>(sum, rest, *piece(st, 2 * c), *piece(st, 2 * c + 1), hi, lo);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] += both_terms(sum[j], rest[j]);
        }
        const int64_t n = (static_cast<int64_t>(first) + static_cast<int64_t>(i) * stride) * kRankTile + gid;
        if (n < g.N) {
            if (row0 >= 0) g.y[row0 + n] = now[0] + d[0];
            if (row1 >= 0) g.y[row1 + n] = now[1] + d[1];
        }
        if (n + 8 < g.N) {
            if (row0 >= 0) g.y[row0 + n + 8] = now[2] + d[2];
            if (row1 >= 0) g.y[row1 + n + 8] = now[3] + d[3];
        }
    }
}

// K of a shrink warp: 512 where that fills the SMs twice, else 128, one round of loads; more
// where a grid has no room for as many ranges (K above 2^28).
constexpr int kShortRange = 128, kLongRange = 512;
int shrink_k(int M, int R, int64_t K)
{
    const int64_t ctas = static_cast<int64_t>(M) * ((R + kRankTile - 1) / kRankTile) * ((K + kLongRange * kWarps - 1) / (kLongRange * kWarps));
    int range = ctas >= 2 * kSms ? kLongRange : kShortRange;
    while (K > static_cast<int64_t>(range) * kWarps * 65535) range *= 2;
    return range;
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
    const void *shrink = reinterpret_cast<const void *>(lora_shrink_kernel<X, W>);
    const void *expand = reinterpret_cast<const void *>(lora_expand_kernel<W>);
    cudaError_t e = ensure_smem_attr(shrink, shrink_smem<X>());
    if (e == cudaSuccess) e = ensure_smem_attr(expand, expand_smem(g.R));
    if (e != cudaSuccess) return e;
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>(g.M), static_cast<unsigned>((g.R + kRankTile - 1) / kRankTile), static_cast<unsigned>(splits));
    cfg.dynamicSmemBytes = static_cast<size_t>(shrink_smem<X>());
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = set_launch_overlap_attr(attr);
    if ((e = cudaLaunchKernelEx(&cfg, lora_shrink_kernel<X, W>, g, shrink_k(g.M, g.R, g.K))) != cudaSuccess) return e;
    // Starts beside the shrink launch, loads its first weights and waits for it. CTAs for one
    // step a warp, but no more than fit an SM: eight took 9.1 us for 7.0 (8 rows, 14336 x 4096)
    // and 20 for 15 (96 rows that share one adapter). By shared memory three fit, two above rank
    // 128, where a grid for three took 212 us for 196 (96 adapters of rank 256, 17408 x 5120).
    const int fit = kSms * std::min(3, kSmShared / (expand_smem(g.R) + kCtaShared));
    const int64_t tiles = (g.N + kRankTile * kWarps - 1) / (kRankTile * kWarps);
    cfg.gridDim = dim3(static_cast<unsigned>(g.M), static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(tiles, fit / g.M))));
    cfg.dynamicSmemBytes = static_cast<size_t>(expand_smem(g.R));
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_expand_kernel<W>, g, splits);
}

}  // namespace

// As for the shortest ranges at every size: a caller keeps the workspace of its largest batch,
// and a smaller one has the more of them.
int64_t lora_workspace_bytes(int M, int R, int64_t K)
{
    const int64_t per = kShortRange * kWarps;
    return (K + per - 1) / per * M * R * 4;
}

cudaError_t launch_lora(const LoraArgs &g, cudaStream_t s)
{
    route_hit(kRouteLora);
    if (g.x_type == QMV_F32)
        return g.w_type == QMV_F16 ? launch_both<float, __half>(g, s) : launch_both<float, __nv_bfloat16>(g, s);
    return g.w_type == QMV_F16 ? launch_both<__half, __half>(g, s) : launch_both<__half, __nv_bfloat16>(g, s);
}

}  // namespace qmv
