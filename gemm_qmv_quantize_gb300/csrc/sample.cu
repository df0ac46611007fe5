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
// maximum. Pass 2, where there is a top-k or top-p, a histogram of 1024 bins of t (counts, and sums
// where a top-p needs them); the first CTA adds them over the cluster and finds the bin that
// holds the cut. Where the tokens up to that bin are few, as behind most top-k, they go to the
// first CTA, which ranks them and draws. Else only the bin's tokens do (bins of more than 256
// are split again by the bits of (logit, index)); then pass 3 sums what is kept, in pieces of
// 128 tokens, and the piece that u falls to is gone through.
//
// Bound by what it executes: 96 rows of 151936, four in five with a top-k of 50, take 61 us (the logits'
// bytes 8.6), eight rows with a top-p alone 29, one of 32000 with a top-k 9. A weight is 35
// instructions, a token of the histogram two or three atomics. (CTAs of 16 to a row, or 4, or of 1024 threads: 103, 93
// and 98 us for what then took 70; sums by 64-bit atomics of shared memory 72 for 57.)
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
    uint64_t lo, hi;           // the codes of its tokens are in lo .. hi; of the first histogram's: its number
    uint64_t need;             // tokens, or weight, up to the cut, of this bin
    uint64_t before;           // weight before the bin
    uint32_t count, upto;      // its tokens (0: there is no cut), and those of it and the bins before it
};

struct alignas(16) Power {     // 2^(40 - j / 256), whole and as fp32
    uint64_t whole;
    float rounded;
};

struct alignas(16) Shared {
    uint32_t count[kBins], low[kBins], high[kBins];   // a histogram: tokens, and sums in two words
    uint64_t before[kBins + 1];                       // the first histogram's sums, added up (first CTA)
    uint32_t first_count[kBins];
    Power table[256];
    uint64_t list[2][kRanked];                        // codes that were sent to the first CTA, for each cut
    uint64_t list_weight[kRanked];
    uint64_t piece[kMaxPieces];
    uint64_t warp_sum[kWarps];
    uint32_t warp_count[kWarps];
    uint64_t total, lo, hi;                           // of this CTA
    uint64_t cut[2], upto;
    Found found[2];
    uint32_t top, bottom, listed[2], counted;                 // counted: tokens of the first histogram (first CTA)
};

// The powers for j = 0 .. 255, worked out by the compiler: products of 2^(-2^k / 256), each the root of
// the one before it (Newton's iteration), in doubles.
struct Table {
    Power v[256];
    constexpr Table() : v()
    {
        double root[8] = {};
        double r = 0.5;
        for (int k = 7; k >= 0; --k) {
            double x = 1.0;
            for (int i = 0; i < 40; ++i) x = 0.5 * (x + r / x);
            root[k] = r = x;
        }
        for (int j = 0; j < 256; ++j) {
            double p = 1099511627776.0;
            for (int k = 0; k < 8; ++k)
                if (j >> k & 1) p *= root[k];
            v[j].whole = static_cast<uint64_t>(p + 0.5);
            v[j].rounded = static_cast<float>(p);
        }
    }
};
__device__ const Table g_table = Table();

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
    const Power *table;
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
    constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to a whole number, in the low bits
    const float shifted = fmaf(t, 256.0f, kMagic);
    const uint32_t k = __float_as_uint(shifted) - __float_as_uint(kMagic);
    const float z = (fmaf(shifted - kMagic, -1.0f / 256.0f, t) + t_lo) * 0.693147180559945f;
    const float series = z * fmaf(z, fmaf(z, -1.0f / 6.0f, 0.5f), -1.0f);   // e^-z - 1, |z| <= 0.0014
    const Power p = r.table[k & 255u];
    const uint64_t w = p.whole + static_cast<int64_t>(__float2int_rn(p.rounded * series));
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
__device__ void pick(cg::cluster_group &cluster, Shared &s, Found &found, bool weights, bool by_weight, bool first_level, uint64_t need,
                     uint64_t lo, uint64_t hi, int shift, uint64_t before)
{
    constexpr int kEach = kBins / kThreads;
    uint32_t n[kEach] = {}, n_sum = 0;
    uint64_t w[kEach] = {}, w_sum = 0;
    if (threadIdx.x == 0) found.count = 0;
#pragma unroll 4
    for (unsigned r = 0; r < cluster.num_blocks(); ++r) {
        const Shared &o = *cluster.map_shared_rank(&s, r);
        const uint2 c = reinterpret_cast<const uint2 *>(o.count)[threadIdx.x];
        n[0] += c.x, n[1] += c.y;
        if (weights) {
            const uint2 l = reinterpret_cast<const uint2 *>(o.low)[threadIdx.x], h = reinterpret_cast<const uint2 *>(o.high)[threadIdx.x];
            w[0] += (static_cast<uint64_t>(h.x) << 32) + l.x, w[1] += (static_cast<uint64_t>(h.y) << 32) + l.y;
        }
    }
    static_assert(kEach == 2, "two bins a thread");
    n_sum = n[0] + n[1], w_sum = w[0] + w[1];
    uint32_t n_at = n_sum;
    uint64_t w_at = w_sum;
    scan(s, n_at, w_at);
    n_at -= n_sum, w_at -= w_sum;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int bin = threadIdx.x * kEach + j;
        if (first_level) s.before[bin] = w_at, s.first_count[bin] = n[j];
        if (by_weight && first_level) need = 0;   // not known before all sums are
        const uint64_t at = by_weight ? w_at : n_at, with = at + (by_weight ? w[j] : n[j]);
        if (at < need && need <= with) {
            found.count = n[j];
            found.upto = n_at + n[j];
            found.need = need - at;
            found.before = before + w_at;
            found.lo = lo + (static_cast<uint64_t>(bin) << shift);
            found.hi = found.lo + ((static_cast<uint64_t>(1) << shift) - 1);
            if (found.hi > hi) found.hi = hi;
        }
        n_at += n[j], w_at += w[j];
    }
    if (first_level && threadIdx.x == kThreads - 1) s.before[kBins] = w_at, s.counted = n_at;
    __syncthreads();
}

// The largest whole number not above p w, and whether it is p w; 0 <= p < 1.
__device__ __forceinline__ uint64_t share_of(float p, uint64_t w, bool &exact)
{
    const uint32_t bits = __float_as_uint(p);
    const int e = static_cast<int>(bits >> 23), sh = 150 - max(e, 1);   // p = mant 2^-sh, sh is 24 at least
    const uint64_t mant = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const uint64_t lo = w * mant, hi = __umul64hi(w, mant);
    exact = sh < 64 ? (lo & ((static_cast<uint64_t>(1) << sh) - 1)) == 0 : mant == 0;
    return sh < 64 ? (hi << (64 - sh)) | (lo >> sh) : sh < 128 ? hi >> (sh - 64) : 0;
}
// The least whole number not below p w; 0 < p < 1.
__device__ __forceinline__ uint64_t share_above(float p, uint64_t w)
{
    bool exact;
    const uint64_t y = share_of(p, w, exact);
    return exact ? y : y + 1;
}
// a / b rounded about once: the quotient of both as fp32, and what that leaves.
__device__ __forceinline__ float ratio(uint64_t a, uint64_t b)
{
    const float ah = static_cast<float>(a), bh = static_cast<float>(b), q = ah / bh;
    const float al = static_cast<float>(static_cast<int64_t>(a - static_cast<uint64_t>(ah))), bl = static_cast<float>(static_cast<int64_t>(b - static_cast<uint64_t>(bh)));
    return q + (fmaf(-q, bh, ah) + fmaf(-q, bl, al)) / bh;
}
// The whole number that a kept token's running sum has to exceed.
__device__ __forceinline__ uint64_t drawn(float u, uint64_t total)
{
    bool exact;
    return u >= 1.0f ? total - 1 : u > 0.0f ? share_of(u, total, exact) : 0;
}

__device__ __forceinline__ uint64_t sum_over_cta(Shared &s, uint64_t v)
{
    v = warp_sum64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.warp_sum[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < kWarps; ++i) v += s.warp_sum[i];
    return v;
}

// The draw from the n codes of s.list[0], among which are the first k, or else all that a top-p keeps,
// whose share is of `whole`, the sum over the row.
__device__ void draw_from_list(Shared &s, const SampleArgs &g, const Row &r, int m, int n, int k, bool cut_k, bool cut_p, float top_p, uint64_t whole, uint64_t least, float u)
{
    const int tid = threadIdx.x;
    const uint64_t code = tid < n ? s.list[0][tid] : kAll;
    const uint64_t w = tid < n ? weight(r, of_key(~static_cast<uint32_t>(code >> 32))) : 0;
    if (tid < n) s.list_weight[tid] = w;
    __syncthreads();
    int rank = 0;
    uint64_t before = 0;
    if (tid < n) {
        for (int j = 0; j < n; ++j) {
            const bool b = s.list[0][j] < code;
            rank += b;
            before += b ? s.list_weight[j] : 0;
        }
    }
    bool kept = tid < n && rank < k;
    if (cut_p) {
        const uint64_t sum = sum_over_cta(s, kept ? w : 0);
        kept = kept && before < share_above(top_p, cut_k ? sum : whole);
    }
    kept = kept && w >= least;
    const uint64_t total = sum_over_cta(s, kept ? w : 0), y = drawn(u, total);
    if (tid < n) s.list_weight[tid] = kept ? w : 0;
    __syncthreads();
    if (!kept) return;
    const uint32_t index = static_cast<uint32_t>(code);
    uint64_t at = 0;
    for (int j = 0; j < n; ++j) at += static_cast<uint32_t>(s.list[0][j]) < index ? s.list_weight[j] : 0;
    if (at <= y && y < at + w) {
        g.token[m] = static_cast<int32_t>(index);
        if (g.prob) g.prob[m] = ratio(w, total);
    }
}

// Grid (C, M) in clusters of C. Dynamic shared memory: Shared, then the slice.
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleArgs g)
{
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    float *x = reinterpret_cast<float *>(smem + sizeof(Shared));
    float4 *x4 = reinterpret_cast<float4 *>(x);
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, m = blockIdx.y;
    const unsigned rank = cluster.block_rank(), C = cluster.num_blocks();
    Shared &lead = *cluster.map_shared_rank(&s, 0);
    if (tid < 256) s.table[tid] = g_table.v[tid];
    clear_histogram(s);
    if (tid == 0) s.top = 0, s.bottom = 0xffffffffu, s.lo = kAll, s.hi = 0, s.listed[0] = s.listed[1] = 0, s.cut[0] = s.cut[1] = kAll;
    grid_launch_dependents();
    grid_dependency_wait();
    // the slice: 16-byte pieces of the row from the boundary before it on; what is not the row's is -inf
    const float *row = g.logits + static_cast<int64_t>(m) * g.V;
    const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u) / 4;
    const int all = (g.V + skew + 3) / 4, each = (all + static_cast<int>(C) - 1) / static_cast<int>(C);
    const int from = min(all, static_cast<int>(rank) * each), pieces = min(all, from + each) - from;
    const int index0 = 4 * from - skew;   // of x[0]
    const int whole0 = max(0, (3 - index0) / 4), whole1 = max(whole0, min(pieces, (g.V - index0) / 4));   // pieces that are the row's
    for (int i = whole0 + tid; i < whole1; i += kThreads) cp_async_16(x4 + i, row + index0 + 4 * i);
    auto edge = [&](int i) {
        for (int j = 0; j < 4; ++j) {
            const int at = index0 + 4 * i + j;
            x[4 * i + j] = at >= 0 && at < g.V ? row[at] : -INFINITY;
        }
    };
    if (tid < min(whole0, pieces)) edge(tid);
    if (tid < pieces - whole1) edge(whole1 + tid);
    const float T = g.temperature ? g.temperature[m] : 1.0f, u = g.u[m];
    const float top_p = g.top_p ? g.top_p[m] : 1.0f, min_p = g.min_p ? g.min_p[m] : 0.0f;
    int k = g.top_k ? g.top_k[m] : 0;
    if (k <= 0 || k > g.V) k = g.V;
    if (!(T > 0.0f) || top_p <= 0.0f || min_p > 1.0f) k = 1;
    cp_async_wait_all();
    __syncthreads();
    float most = -INFINITY, lowest = INFINITY;   // lowest: above -inf
#pragma unroll 4
    for (int i = tid; i < pieces; i += kThreads) {
        float4 v = x4[i];
        v = make_float4(cleaned(v.x), cleaned(v.y), cleaned(v.z), cleaned(v.w));
        x4[i] = v;
        most = fmaxf(fmaxf(most, fmaxf(v.x, v.y)), fmaxf(v.z, v.w));
        const auto above = [](float a) { return a > -INFINITY ? a : INFINITY; };
        lowest = fminf(fminf(lowest, fminf(above(v.x), above(v.y))), fminf(above(v.z), above(v.w)));
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, key_of(most)), bottom = __reduce_min_sync(0xffffffffu, key_of(lowest));
    if (lane == 0) atomicMax(&s.top, top), atomicMin(&s.bottom, bottom);
    cluster.sync();
    // (a lane a CTA: reads of others' memory take a while)
    top = __reduce_max_sync(0xffffffffu, lane < static_cast<int>(C) ? cluster.map_shared_rank(&s, lane)->top : 0u);
    bottom = __reduce_min_sync(0xffffffffu, lane < static_cast<int>(C) ? cluster.map_shared_rank(&s, lane)->bottom : 0xffffffffu);
    // log2(e) / T in two terms, 2^-46 off
    constexpr float kLog2eHi = 1.44269502e+00f, kLog2eLo = 1.92596299e-08f;
    Row r;
    r.top = of_key(top);
    r.table = s.table;
    r.c_hi = kLog2eHi / T;
    r.c_lo = T < INFINITY ? (fmaf(-r.c_hi, T, kLog2eHi) + kLog2eLo) / T : 0.0f;
    if (top <= key_of(-INFINITY)) {   // no logit above -inf
        if (rank == 0 && tid == 0) {
            g.token[m] = -1;
            if (g.prob) g.prob[m] = 0.0f;
        }
        cluster.sync();   // nobody leaves while others read its memory
        return;
    }
    // f(logit, index) for every token of the slice
    auto each_token = [&](auto f) {
        for (int i = tid; i < pieces; i += kThreads) {
            const float4 v = x4[i];
            const uint32_t at = static_cast<uint32_t>(index0 + 4 * i);
            f(v.x, at), f(v.y, at + 1), f(v.z, at + 2), f(v.w, at + 3);
        }
    };
    // The histogram spans what the row's logits do, a vocabulary of nearly equal ones too.
    const float span = fminf(kMostT, fmaxf(1.001f * rough_t(r, of_key(bottom)), 1e-6f)), per_t = static_cast<float>(kBins) / span;
    auto bin_of = [&](float t) { return min(static_cast<int>(t * per_t), kBins - 1); };
    const uint64_t least = min_p > 0.0f && k > 1 ? (min_p >= 1.0f ? kOne : max(static_cast<unsigned long long>(1), static_cast<unsigned long long>(share_above(min_p, kOne)))) : 1;
    uint64_t cut = kAll;   // the last kept token's code
    const bool cut_p = top_p < 1.0f && k > 1, cut_k = k < g.V && k > 1;
    if (k == 1) {   // the first of the largest
        uint64_t first = kAll;
        each_token([&](float v, uint32_t at) {
            if (v == r.top) first = min(static_cast<unsigned long long>(first), static_cast<unsigned long long>(code_of(v, at)));
        });
        if (first != kAll) atomicMin(reinterpret_cast<unsigned long long *>(&s.lo), first);
        cluster.sync();
        for (unsigned q = 0; rank == 0 && tid == 0 && q < C; ++q) {
            const uint64_t o = cluster.map_shared_rank(&s, q)->lo;
            if (o < cut) cut = o;
        }
        if (rank == 0 && tid == 0) {
            g.token[m] = static_cast<int32_t>(static_cast<uint32_t>(cut));
            if (g.prob) g.prob[m] = 1.0f;
        }
        cluster.sync();
        return;
    }
    if (cut_p || cut_k) {
        // Behind a small top-k the tokens up to the cut are most likely few, and weights not needed for more than those.
        bool weights = cut_p && !(cut_k && k <= kRanked / 2);
        for (;;) {
            each_token([&](float v, uint32_t) {
                const float t = rough_t(r, v);
                if (!(t <= span)) return;
                const int bin = bin_of(t);
                atomicAdd(&s.count[bin], 1u);
                if (weights) add64(s, bin, weight(r, v));
            });
            cluster.sync();
            if (rank == 0) {
                pick(cluster, s, s.found[0], weights, !cut_k, true, static_cast<uint64_t>(k), 0, kAll, 0, 0);
                if (tid == 0) s.upto = s.before[kBins];
                // fewer tokens of any weight than k, and few: the last bin is taken for the cut's
                if (tid == 0 && cut_k && !s.found[0].count && s.counted <= kRanked) s.found[0] = Found{kBins - 1, 0, 0, 0, s.counted, s.counted};
                if (!cut_k) {   // the share of the whole sum
                    const uint64_t y = share_above(top_p, s.before[kBins]);
                    uint32_t n = 0;
                    for (int j = 0; j < kBins / kThreads; ++j) {
                        const int bin = tid * (kBins / kThreads) + j;
                        if (s.before[bin] < y) n += s.first_count[bin];   // bins up to the cut's, all of them
                    }
                    const uint32_t upto = static_cast<uint32_t>(sum_over_cta(s, n));
                    for (int bin = tid; bin < kBins; bin += kThreads) {
                        if (s.before[bin] >= y || y > s.before[bin + 1]) continue;
                        s.found[0] = Found{static_cast<uint64_t>(bin), 0, y - s.before[bin], s.before[bin], s.first_count[bin], upto};
                    }
                }
            }
            cluster.sync();
            const Found f = lead.found[0];
            if (f.count && f.upto <= kRanked) {   // few tokens: the first CTA sees to them
                const int last = static_cast<int>(f.lo);
                each_token([&](float v, uint32_t at) {
                    const float t = rough_t(r, v);
                    if (!(t <= span) || bin_of(t) > last) return;
                    const uint32_t i = atomicAdd(&lead.listed[0], 1u);
                    if (i < kRanked) lead.list[0][i] = code_of(v, at);
                });
                cluster.sync();
                if (rank == 0) draw_from_list(s, g, r, m, static_cast<int>(f.upto), k, cut_k, cut_p, top_p, s.upto, least, u);
                return;   // the others' memory is not read any more
            }
            if (weights || !cut_p) break;
            weights = true;   // more than a few after all
            clear_histogram(s);
            cluster.sync();
        }
        for (int by_weight = cut_k ? 0 : 1; by_weight < (cut_p ? 2 : 1); ++by_weight) {
            const int which = by_weight && cut_k ? 1 : 0;
            if (which) {   // a top-p behind a top-k
                if (rank == 0) {
                    if (tid == 0) s.found[1].count = 0;
                    const uint64_t y = share_above(top_p, s.upto);
                    __syncthreads();
                    for (int bin = tid; bin < kBins; bin += kThreads) {
                        if (s.before[bin] >= y || y > s.before[bin + 1]) continue;
                        s.found[1] = Found{static_cast<uint64_t>(bin), 0, y - s.before[bin], s.before[bin], s.first_count[bin], 0};
                    }
                }
                cluster.sync();
            }
            Found f = lead.found[which];
            if (!f.count) continue;
            const int bin = static_cast<int>(f.lo);   // the first histogram's
            const bool split = f.count > kRanked;
            if (split) {
                // the codes that the bin's tokens span
                if (tid == 0) s.lo = kAll, s.hi = 0;
                __syncthreads();
                unsigned long long lo = kAll, hi = 0;
                each_token([&](float v, uint32_t at) {
                    const float t = rough_t(r, v);
                    if (!(t <= span) || bin_of(t) != bin) return;
                    const unsigned long long code = code_of(v, at);
                    lo = min(lo, code), hi = max(hi, code);
                });
                if (lo != kAll) {
                    atomicMin(reinterpret_cast<unsigned long long *>(&s.lo), lo);
                    atomicMax(reinterpret_cast<unsigned long long *>(&s.hi), hi);
                }
                cluster.sync();
                for (unsigned q = 0; q < C; ++q) {
                    const Shared &o = *cluster.map_shared_rank(&s, q);
                    lo = min(lo, static_cast<unsigned long long>(o.lo)), hi = max(hi, static_cast<unsigned long long>(o.hi));
                }
                f.lo = lo, f.hi = hi;
                while (f.count > kRanked) {
                    const int shift = max(0, 64 - __clzll(static_cast<long long>(f.hi - f.lo)) - 10);
                    clear_histogram(s);
                    __syncthreads();
                    each_token([&](float v, uint32_t at) {
                        const uint64_t code = code_of(v, at);
                        if (code < f.lo || code > f.hi) return;
                        const int b = static_cast<int>((code - f.lo) >> shift);
                        atomicAdd(&s.count[b], 1u);
                        if (cut_p) add64(s, b, weight(r, v));
                    });
                    cluster.sync();
                    if (rank == 0) pick(cluster, s, s.found[which], cut_p, by_weight, false, f.need, f.lo, f.hi, shift, f.before);
                    cluster.sync();
                    f = lead.found[which];
                    cluster.sync();
                }
            }
            // the bin's tokens, in no order, to the first CTA, which ranks them
            each_token([&](float v, uint32_t at) {
                const uint64_t code = code_of(v, at);
                if (split) {
                    if (code < f.lo || code > f.hi) return;
                } else {
                    const float t = rough_t(r, v);
                    if (!(t <= span) || bin_of(t) != bin) return;
                }
                const uint32_t i = atomicAdd(&lead.listed[which], 1u);
                if (i < kRanked) lead.list[which][i] = code;
            });
            cluster.sync();
            if (rank == 0) {
                const int n = static_cast<int>(f.count);
                const uint64_t code = tid < n ? s.list[which][tid] : kAll;
                const uint64_t mine = tid < n && cut_p ? weight(r, of_key(~static_cast<uint32_t>(code >> 32))) : 0;
                if (tid < n) s.list_weight[tid] = mine;
                __syncthreads();
                if (tid < n) {
                    uint64_t rank_of = 0, w_before = 0;
                    for (int j = 0; j < n; ++j) {
                        const bool b = s.list[which][j] < code;
                        rank_of += b;
                        w_before += b ? s.list_weight[j] : 0;
                    }
                    const uint64_t at = by_weight ? w_before : rank_of, with = at + (by_weight ? mine : 1);
                    if (at < f.need && f.need <= with) {
                        s.cut[which] = code;
                        s.upto = f.before + w_before + mine;
                    }
                }
            }
            cluster.sync();
            if (lead.cut[which] < cut) cut = lead.cut[which];
        }
    }
    // what is kept, in pieces of 128 tokens
    // (first what one comparison of fp32 shows: below the last kept logit, or far below min_p)
    const float cut_x = cut == kAll ? -INFINITY : of_key(~static_cast<uint32_t>(cut >> 32));
    const float most_t = min_p > 0.0f && min_p < 1.0f ? fminf(kMostT, 0.001f - log2f(min_p)) : kMostT;
    auto kept = [&](float v, uint32_t at) -> uint64_t {
        if (v < cut_x || !(rough_t(r, v) <= most_t) || code_of(v, at) > cut) return 0;
        const uint64_t w = weight(r, v);
        return w >= least ? w : 0;
    };
    uint64_t mine = 0;
    for (int piece = warp; piece * 32 < pieces; piece += kWarps) {
        const int i = piece * 32 + lane;
        uint64_t w = 0;
        if (i < pieces) {
            const float4 v = x4[i];
            const uint32_t at = static_cast<uint32_t>(index0 + 4 * i);
            w = kept(v.x, at) + kept(v.y, at + 1) + kept(v.z, at + 2) + kept(v.w, at + 3);
        }
        // a sum of 32 weights' low 24 bits, and of what is above, fit 32 bits
        w = (static_cast<uint64_t>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w >> 24))) << 24) +
            __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w) & 0xffffffu);
        if (lane == 0) s.piece[piece] = w;
        mine += w;
    }
    mine = sum_over_cta(s, lane == 0 ? mine : 0);
    if (tid == 0) s.total = mine;
    cluster.sync();
    if (warp > 0) {
        cluster.sync();
        return;
    }
    uint64_t upto_rank = lane < static_cast<int>(C) ? cluster.map_shared_rank(&s, lane)->total : 0;
#pragma unroll
    for (int o = 1; o < 16; o *= 2) {
        const uint64_t b = shfl_up64(upto_rank, o);
        if (lane >= o) upto_rank += b;
    }
    const uint64_t total = __shfl_sync(0xffffffffu, upto_rank, C - 1), before = __shfl_sync(0xffffffffu, upto_rank, rank) - mine;
    const uint64_t y = drawn(u, total);
    if (before <= y && y < before + mine) {
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
            at += __shfl_sync(0xffffffffu, upto - (past ? w : 0), in);
            if (past) {
                piece += in;
                break;
            }
        }
        const int i = piece * 32 + lane;
        uint64_t w[4] = {0, 0, 0, 0};
        if (i < pieces) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = kept(x[4 * i + j], static_cast<uint32_t>(index0 + 4 * i + j));
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
                g.token[m] = index0 + 4 * i + j;
                if (g.prob) g.prob[m] = ratio(w[j], total);
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
