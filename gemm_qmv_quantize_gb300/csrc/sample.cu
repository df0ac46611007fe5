// sample.cu -- a token drawn from a row of logits x, with temperature T, top-k, top-p and
// min-p, from a random number u that the caller gives:
//   w_i = 2^(-t_i), t_i = (max x - x_i) log2(e) / T;  the order: w descending, equal logits by index
//   kept: the first k;  of these, those before which the sum of w is below p times their
//   sum;  of these, those with w_i >= min_p
//   token = the first i, by index, with (sum of kept w_j, j <= i) > u (sum of kept w_j)
//
// The choice has to be the one of exact arithmetic: tokens' shares of the sum are as small as
// 1e-7 or less, where sums in fp32 would move the borders between them by whole tokens. So weights are
// whole numbers, 2^44 for the largest token: t to 2^-33 or so by a two-term difference and
// product, 2^-t from a table of 256 and a short series, 2^-32 off its value; below 2^-44
// they are 0. Sums of whole numbers are exact, in any order, so the same call gives the
// same token, and nothing is sorted: the cuts are found by histograms.
//
// A row is a cluster's: each CTA keeps a slice of it in shared memory. Pass 1 finds the
// maximum. Pass 2, where there is a top-k or top-p, a histogram of 1024 bins of t, counts and
// sums; the first CTA adds them over the cluster and finds the bin that holds a cut; bins of
// more than 256 tokens are split again by the bits of (logit, index), then the bin's tokens are
// ranked. Pass 3 sums what is kept, in pieces of 128 tokens, and the piece that u falls to
// is gone through.
#include <algorithm>

#include <cooperative_groups.h>

#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace cg = cooperative_groups;

namespace qmv {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kRanked = 256;             // tokens that are ranked by comparing each with each
constexpr int kFraction = 44;            // bits of a weight below the point
constexpr float kMostT = 45.0f;          // from there on a weight is 0
constexpr int kMaxPieces = 512;          // of 128 tokens, of a CTA's slice
constexpr int64_t kMaxSlice = 32768 + 8; // tokens of a CTA
constexpr uint64_t kOne = 1ull << kFraction, kAll = ~0ull;

struct Found {                 // a bin with a cut in it
    uint64_t lo, hi;           // the codes of its tokens are in lo .. hi
    uint64_t need;             // tokens, or weight, up to the cut, of this bin
    uint64_t before;           // weight before the bin
    uint32_t count;            // its tokens; 0: there is no cut
};

struct alignas(16) Shared {
    uint32_t count[kBins], low[kBins], high[kBins];   // a histogram: tokens, and sums in two words
    uint64_t before[kBins + 1];                       // the first histogram's sums, added up (first CTA)
    uint32_t first_count[kBins];
    uint64_t table[256];                              // 2^(40 - j / 256)
    uint64_t list[kRanked];
    uint64_t piece[kMaxPieces];
    uint64_t warp_sum[kWarps];
    uint32_t warp_count[kWarps];
    uint64_t total, lo, hi;                           // of this CTA
    uint64_t cut, upto;
    Found found;
    uint32_t top, listed;
    int token;
};

// Logits in their order as whole numbers, NaN as -inf and -0 as 0.
__device__ __forceinline__ float cleaned(float x) { return x != x ? -INFINITY : x + 0.0f; }
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
// The order of tokens: the larger logit first, then the lower index.
__device__ __forceinline__ uint64_t code_of(float x, uint32_t index) { return static_cast<uint64_t>(~key_of(x)) << 32 | index; }

struct Row {
    float top, c_hi, c_lo;        // max x; log2(e) / T
    const uint64_t *table;
};

// t of a logit, rounded: not below that of a larger logit.
__device__ __forceinline__ float rough_t(const Row &r, float x) { return x == r.top ? 0.0f : (r.top - x) * r.c_hi; }

__device__ __forceinline__ uint64_t weight(const Row &r, float x)
{
    if (x == r.top) return kOne;
    const float d = r.top - x, t = d * r.c_hi;
    if (!(t <= kMostT)) return 0;   // and what is NaN
    const float back = r.top - d;   // what d's rounding left: top - x = d + d_lo, exactly
    const float d_lo = (back - x) + (r.top - (d + back));
    const float t_lo = fmaf(d, r.c_hi, -t) + fmaf(d, r.c_lo, d_lo * r.c_hi);
    const int k = __float2int_rn(t * 256.0f);
    const float z = ((t - static_cast<float>(k) * (1.0f / 256.0f)) + t_lo) * 0.693147180559945f;
    const float series = z * fmaf(z, fmaf(z, -1.0f / 6.0f, 0.5f), -1.0f);   // e^-z - 1, |z| <= 0.0014
    const uint64_t at = r.table[k & 255];
    const uint64_t w = at + static_cast<int64_t>(__float2int_rn(static_cast<float>(at) * series));
    return (w << (kFraction - 40)) >> (k >> 8);
}

__device__ __forceinline__ void add64(Shared &s, int bin, uint64_t w)
{
    const uint32_t lo = static_cast<uint32_t>(w), old = atomicAdd(&s.low[bin], lo);
    const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old ? 1u : 0u);
    if (hi) atomicAdd(&s.high[bin], hi);
}

__device__ __forceinline__ uint64_t shfl_up64(uint64_t v, int o) { return __shfl_up_sync(0xffffffffu, v, o); }

// Inclusive sums over the CTA's threads of a count and a weight.
__device__ __forceinline__ void scan(Shared &s, uint32_t &n, uint64_t &w)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t a = __shfl_up_sync(0xffffffffu, n, o);
        const uint64_t b = shfl_up64(w, o);
        if (lane >= o) n += a, w += b;
    }
    __syncthreads();
    if (lane == 31) s.warp_count[warp] = n, s.warp_sum[warp] = w;
    __syncthreads();
    for (int i = 0; i < warp; ++i) n += s.warp_count[i], w += s.warp_sum[i];
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void clear_histogram(Shared &s)
{
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.count[i] = s.low[i] = s.high[i] = 0;
}

// The first CTA: the cluster's histogram, and of it the bin in which the count, or the weight,
// reaches `need`. First level: kept for later cuts. Bins are [lo + (bin << shift), + 1 << shift).
__device__ void pick(cg::cluster_group &cluster, Shared &s, bool by_weight, bool first_level, uint64_t need, uint64_t lo,
                     uint64_t hi, int shift, uint64_t before)
{
    constexpr int kEach = kBins / kThreads;
    uint32_t n[kEach], n_sum = 0;
    uint64_t w[kEach], w_sum = 0;
    if (threadIdx.x == 0) s.found.count = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int bin = threadIdx.x * kEach + j;
        n[j] = 0, w[j] = 0;
        for (unsigned r = 0; r < cluster.num_blocks(); ++r) {
            const Shared &o = *cluster.map_shared_rank(&s, r);
            n[j] += o.count[bin];
            w[j] += (static_cast<uint64_t>(o.high[bin]) << 32) + o.low[bin];
        }
        n_sum += n[j], w_sum += w[j];
    }
    uint32_t n_at = n_sum;
    uint64_t w_at = w_sum;
    scan(s, n_at, w_at);
    n_at -= n_sum, w_at -= w_sum;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int bin = threadIdx.x * kEach + j;
        if (first_level) s.before[bin] = w_at, s.first_count[bin] = n[j];
        const uint64_t at = by_weight ? w_at : n_at, with = at + (by_weight ? w[j] : n[j]);
        if (at < need && need <= with) {
            s.found.count = n[j];
            s.found.need = need - at;
            s.found.before = before + w_at;
            s.found.lo = lo + (static_cast<uint64_t>(bin) << shift);
            s.found.hi = s.found.lo + ((static_cast<uint64_t>(1) << shift) - 1);
            if (s.found.hi > hi) s.found.hi = hi;
        }
        n_at += n[j], w_at += w[j];
    }
    if (first_level && threadIdx.x == kThreads - 1) s.before[kBins] = w_at;
    __syncthreads();
}

// Grid (C, M) in clusters of C. Dynamic shared memory: Shared, then the slice.
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleArgs g)
{
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    float *x = reinterpret_cast<float *>(smem + sizeof(Shared));
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, m = blockIdx.y;
    const unsigned rank = cluster.block_rank(), C = cluster.num_blocks();
    Shared &lead = *cluster.map_shared_rank(&s, 0);
    for (int j = tid; j < 256; j += kThreads) s.table[j] = static_cast<uint64_t>(__double2ll_rn(exp2(40.0 - j / 256.0)));
    clear_histogram(s);
    if (tid == 0) s.top = 0, s.lo = kAll, s.hi = 0, s.listed = 0, s.cut = kAll;
    grid_launch_dependents();
    grid_dependency_wait();
    // the slice: 16-byte pieces of the row from the boundary before it on; what is not the row's is -inf
    const float *row = g.logits + static_cast<int64_t>(m) * g.V;
    const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u) / 4;
    const int all = (g.V + skew + 3) / 4, each = (all + static_cast<int>(C) - 1) / static_cast<int>(C);
    const int from = min(all, static_cast<int>(rank) * each), pieces = min(all, from + each) - from;
    const int index0 = 4 * from - skew;   // of x[0]
    uint32_t top = 0;
#pragma unroll 4
    for (int i = tid; i < pieces; i += kThreads) {
        const int at = index0 + 4 * i;
        float4 v;
        if (at >= 0 && at + 4 <= g.V) {
            v = __ldg(reinterpret_cast<const float4 *>(row + at));
        } else {
            v.x = at >= 0 && at < g.V ? row[at] : -INFINITY;
            v.y = at + 1 >= 0 && at + 1 < g.V ? row[at + 1] : -INFINITY;
            v.z = at + 2 >= 0 && at + 2 < g.V ? row[at + 2] : -INFINITY;
            v.w = at + 3 >= 0 && at + 3 < g.V ? row[at + 3] : -INFINITY;
        }
        v = make_float4(cleaned(v.x), cleaned(v.y), cleaned(v.z), cleaned(v.w));
        reinterpret_cast<float4 *>(x)[i] = v;
        top = max(max(top, max(key_of(v.x), key_of(v.y))), max(key_of(v.z), key_of(v.w)));
    }
    const float T = g.temperature ? g.temperature[m] : 1.0f, u = g.u[m];
    const float top_p = g.top_p ? g.top_p[m] : 1.0f, min_p = g.min_p ? g.min_p[m] : 0.0f;
    int k = g.top_k ? g.top_k[m] : 0;
    if (k <= 0 || k > g.V) k = g.V;
    const bool greedy = !(T > 0.0f);
    if (greedy || top_p <= 0.0f || min_p > 1.0f) k = 1;
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();
    if (lane == 0) atomicMax(&s.top, top);
    cluster.sync();
    for (unsigned r = 0; r < C; ++r) top = max(top, cluster.map_shared_rank(&s, r)->top);
    Row r;
    r.top = of_key(top);
    r.table = s.table;
    const double c = 1.4426950408889634 / static_cast<double>(T);
    r.c_hi = static_cast<float>(c);
    r.c_lo = static_cast<float>(c - static_cast<double>(r.c_hi));
    const int n = 4 * pieces;
    if (top <= key_of(-INFINITY)) {   // no logit above -inf
        if (rank == 0 && tid == 0) {
            g.token[m] = -1;
            if (g.prob) g.prob[m] = 0.0f;
        }
        cluster.sync();   // nobody leaves while others read its memory
        return;
    }
    uint64_t cut = kAll;   // the last kept token's code
    const bool cut_p = top_p < 1.0f && k > 1, cut_k = k < g.V && k > 1;
    if (k == 1) {   // the first of the largest
        uint64_t first = kAll;
        for (int i = tid; i < n; i += kThreads)
            if (x[i] == r.top) first = min(first, code_of(x[i], static_cast<uint32_t>(index0 + i)));
        if (first != kAll) atomicMin(reinterpret_cast<unsigned long long *>(&s.lo), first);
        cluster.sync();
        for (unsigned q = 0; q < C; ++q) cut = min(cut, cluster.map_shared_rank(&s, q)->lo);
    } else if (cut_p || cut_k) {
        const float per_t = static_cast<float>(kBins) / kMostT;
        auto bin_of = [&](float t) { return min(static_cast<int>(t * per_t), kBins - 1); };
        for (int i = tid; i < n; i += kThreads) {
            const float t = rough_t(r, x[i]);
            if (!(t <= kMostT)) continue;
            const int bin = bin_of(t);
            atomicAdd(&s.count[bin], 1u);
            if (cut_p) add64(s, bin, weight(r, x[i]));
        }
        cluster.sync();
        bool first_level = true;
        for (int by_weight = cut_k ? 0 : 1; by_weight < (cut_p ? 2 : 1); ++by_weight) {
            if (rank == 0) {
                if (first_level) {   // without a top-k the share is of the whole sum, which is known after this
                    pick(cluster, s, false, true, static_cast<uint64_t>(k), 0, kAll, 0, 0);
                    if (tid == 0) s.upto = s.before[kBins];
                    __syncthreads();
                }
                if (by_weight) {
                    if (tid == 0) {
                        s.found.count = 0;
                        const uint64_t all_w = s.upto;
                        // the least whole number not below top_p all_w
                        const uint32_t bits = __float_as_uint(top_p);
                        const int e = static_cast<int>(bits >> 23);
                        const uint64_t mant = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
                        const int sh = 150 - max(e, 1);   // top_p = mant 2^-sh, 24 at least
                        const uint64_t lo = all_w * mant, hi = __umul64hi(all_w, mant);
                        uint64_t y;
                        if (sh < 64) {
                            y = (hi << (64 - sh)) | (lo >> sh);
                            if (lo & ((1ull << sh) - 1)) ++y;
                        } else {
                            y = sh < 128 ? (hi >> (sh - 64)) : 0;
                            if (y < 1) y = 1;
                        }
                        s.total = y;
                    }
                    __syncthreads();
                    const uint64_t y = s.total;
                    for (int bin = tid; bin < kBins; bin += kThreads) {
                        if (s.before[bin] < y && y <= s.before[bin + 1]) {
                            s.found.count = s.first_count[bin];
                            s.found.need = y - s.before[bin];
                            s.found.before = s.before[bin];
                            s.found.lo = static_cast<uint64_t>(bin);
                        }
                    }
                }
                __syncthreads();
            }
            first_level = false;
            cluster.sync();
            Found f = lead.found;
            cluster.sync();
            if (!f.count) continue;
            // the codes that the bin's tokens span
            const int bin = static_cast<int>(f.lo);   // the first level's
            if (tid == 0) s.lo = kAll, s.hi = 0;
            __syncthreads();
            uint64_t lo = kAll, hi = 0;
            for (int i = tid; i < n; i += kThreads) {
                const float t = rough_t(r, x[i]);
                if (!(t <= kMostT) || bin_of(t) != bin) continue;
                const uint64_t code = code_of(x[i], static_cast<uint32_t>(index0 + i));
                lo = min(lo, code), hi = max(hi, code);
            }
            if (lo != kAll) {
                atomicMin(reinterpret_cast<unsigned long long *>(&s.lo), lo);
                atomicMax(reinterpret_cast<unsigned long long *>(&s.hi), hi);
            }
            cluster.sync();
            for (unsigned q = 0; q < C; ++q) {
                const Shared &o = *cluster.map_shared_rank(&s, q);
                lo = min(lo, o.lo), hi = max(hi, o.hi);
            }
            f.lo = lo, f.hi = hi;
            cluster.sync();
            while (f.count > kRanked) {
                const int shift = max(0, 64 - __clzll(f.hi - f.lo) - 10);
                clear_histogram(s);
                __syncthreads();
                for (int i = tid; i < n; i += kThreads) {
                    const uint64_t code = code_of(x[i], static_cast<uint32_t>(index0 + i));
                    if (code < f.lo || code > f.hi) continue;
                    const int b = static_cast<int>((code - f.lo) >> shift);
                    atomicAdd(&s.count[b], 1u);
                    if (cut_p) add64(s, b, weight(r, x[i]));
                }
                cluster.sync();
                if (rank == 0) pick(cluster, s, by_weight, false, f.need, f.lo, f.hi, shift, f.before);
                cluster.sync();
                f = lead.found;
                cluster.sync();
            }
            // the bin's tokens, in no order, to the first CTA, which ranks them
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t code = code_of(x[i], static_cast<uint32_t>(index0 + i));
                if (code < f.lo || code > f.hi) continue;
                const uint32_t at = atomicAdd(&lead.listed, 1u);
                if (at < kRanked) lead.list[at] = code;
            }
            cluster.sync();
            if (rank == 0) {
                if (tid < static_cast<int>(f.count)) {
                    const uint64_t code = s.list[tid];
                    uint64_t rank_of = 0, w_before = 0;
                    for (uint32_t j = 0; j < f.count; ++j) {
                        const uint64_t o = s.list[j];
                        if (o >= code) continue;
                        ++rank_of;
                        if (cut_p) w_before += weight(r, of_key(~static_cast<uint32_t>(o >> 32)));
                    }
                    const uint64_t mine = cut_p ? weight(r, of_key(~static_cast<uint32_t>(code >> 32))) : 0;
                    const uint64_t at = by_weight ? w_before : rank_of, with = at + (by_weight ? mine : 1);
                    if (at < f.need && f.need <= with) {
                        s.cut = code;
                        s.upto = f.before + w_before + mine;
                    }
                }
                __syncthreads();
                if (tid == 0) s.listed = 0;
            }
            cluster.sync();
            cut = min(cut, lead.cut);
            cluster.sync();
        }
    }
    // what is kept, in pieces of 128 tokens
    const uint64_t least = min_p > 0.0f && k > 1 ? static_cast<uint64_t>(ceil(static_cast<double>(min_p) * static_cast<double>(kOne))) : 1;
    auto kept = [&](int i) -> uint64_t {
        const float v = x[i];
        if (code_of(v, static_cast<uint32_t>(index0 + i)) > cut) return 0;
        const uint64_t w = weight(r, v);
        return w >= least ? w : 0;
    };
    uint64_t mine = 0;
    for (int piece = warp; piece * 32 < pieces; piece += kWarps) {
        const int i = 4 * (piece * 32 + lane);
        uint64_t w = 0;
        if (i < n) w = kept(i) + kept(i + 1) + kept(i + 2) + kept(i + 3);
        w = warp_sum64(w);
        if (lane == 0) s.piece[piece] = w;
        mine += w;
    }
    __syncthreads();
    if (lane == 0) s.warp_sum[warp] = mine;
    __syncthreads();
    if (tid == 0) {
        uint64_t total = 0;
        for (int i = 0; i < kWarps; ++i) total += s.warp_sum[i];
        s.total = total;
    }
    cluster.sync();
    uint64_t before = 0, total = 0, own = 0;
    for (unsigned q = 0; q < C; ++q) {
        const uint64_t w = cluster.map_shared_rank(&s, q)->total;
        if (q < rank) before += w;
        if (q == rank) own = w;
        total += w;
    }
    // the largest whole number not above u total; u = mant 2^-sh
    uint64_t y;
    if (u >= 1.0f) {
        y = total - 1;
    } else {
        const uint32_t bits = u > 0.0f ? __float_as_uint(u) : 0u;
        const int e = static_cast<int>(bits >> 23), sh = 150 - max(e, 1);
        const uint64_t mant = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
        const uint64_t lo = total * mant, hi = __umul64hi(total, mant);
        y = sh < 64 ? (hi << (64 - sh)) | (lo >> sh) : sh < 128 ? hi >> (sh - 64) : 0;
    }
    if (warp == 0 && before <= y && y < before + own) {
        uint64_t at = before;
        int piece = 0;
        for (; piece * 32 < pieces; piece += 32) {
            uint64_t w = (piece + lane) * 32 < pieces ? s.piece[piece + lane] : 0, upto = w;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const uint64_t b = shfl_up64(upto, o);
                if (lane >= o) upto += b;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, at + upto > y);
            const int in = past ? __ffs(past) - 1 : 31;
            const uint64_t skip = __shfl_sync(0xffffffffu, upto - (past ? w : 0), in);
            at += skip;
            if (past) {
                piece += in;
                break;
            }
        }
        const int i = 4 * (piece * 32 + lane);
        uint64_t w[4] = {0, 0, 0, 0};
        if (i < n) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = kept(i + j);
        }
        const uint64_t sum4 = w[0] + w[1] + w[2] + w[3];
        uint64_t upto = sum4;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint64_t b = shfl_up64(upto, o);
            if (lane >= o) upto += b;
        }
        at += upto - sum4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (at <= y && y < at + w[j]) {
                g.token[m] = index0 + i + j;
                if (g.prob) g.prob[m] = static_cast<float>(static_cast<double>(w[j]) / static_cast<double>(total));
            }
            at += w[j];
        }
    }
    cluster.sync();   // nobody leaves while others read its memory
}

// CTAs of a row: slices of 4096 tokens or more, 8 CTAs at most, 16 where 8 slices do not fit.
int cluster_of(int V)
{
    if (V > 8 * (kMaxSlice - 8)) return 16;
    int C = 1;
    while (C < 8 && V > 4096 * C) C *= 2;
    return C;
}

}  // namespace

int sample_max_vocabulary() { return static_cast<int>(16 * (kMaxSlice - 8)); }

cudaError_t launch_sample(const SampleArgs &g, cudaStream_t s)
{
    route_hit(kRouteSample);
    const int C = cluster_of(g.V);
    const int slice = 4 * (((g.V + 3 + 3) / 4 + C - 1) / C);
    const size_t smem = sizeof(Shared) + static_cast<size_t>(slice) * 4;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(sample_kernel), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (C > 8) {
        e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3(static_cast<unsigned>(C), static_cast<unsigned>(g.M));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1 + set_launch_overlap_attr(attr + 1);
    return cudaLaunchKernelEx(&cfg, sample_kernel, g);
}

}  // namespace qmv
