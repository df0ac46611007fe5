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
// product, 2^-t from a table of 256 and a short series, some 2^-32 off its value; below 2^-44
// they are 0. Sums of whole numbers are exact, in any order, so the same call gives the
// same token, and nothing is sorted: the cuts are found by histograms.
//
// A row is a cluster's: each CTA keeps a slice of it in shared memory. Pass 1 finds the
// maximum. A small top-k: a histogram of 512 bins of t of the threads' largest logits alone shows a
// bin up to which there are k tokens or more; those up to it go to the first CTA, which ranks
// them and draws. A top-p alone: all weights are summed; tokens so light that all of them together would
// not reach beyond 1 - p are behind the cut, the others' places go to lists, a warp each. Then, or with a
// larger top-k, a histogram of counts and sums of weights, added over the cluster by the first CTA, finds the
// bin that holds the cut. Where the tokens up to that bin are few they too go to the
// first CTA, which draws. Else only the bin's tokens do (bins of more than 256
// are split again by the bits of (logit, index)); then the last pass sums what is kept, in pieces of
// 64 tokens, and the piece that u falls to is gone through.
//
// Bound by what it executes: 96 rows of 151936, four in five with a top-k of 50, take 52 us (the logits'
// bytes 8.6), eight rows with a top-p alone 25, one of 32000 with a top-k 9. A weight is some 45
// instructions with its place in a table, a token of the histogram two or three atomics more: with a
// histogram of all tokens that was 61, 29 and 9 us. (CTAs of 16 to a row, or 4, or of 1024 threads: 103, 93
// and 98 us for what then took 70; 16 for up to four rows 5 % faster, for eight 6 % slower; sums by
// 64-bit atomics of shared memory 72 for 57.)
#include <algorithm>
#include <cfloat>

#include <cooperative_groups.h>

#include "decode_ops.h"
#include "qmv.h"
#include "qmv_device.cuh"

namespace cg = cooperative_groups;

namespace qmv {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = kThreads;
constexpr int kRanked = 256;             // tokens that are ranked by comparing each with each
constexpr int kFraction = 44;            // bits of a weight below the point
constexpr float kMostT = 45.0f;          // from there on a weight is 0
constexpr int64_t kMaxSlice = 32768 + 8; // tokens of a CTA
constexpr int kPiece = 64, kMaxPieces = (kMaxSlice / kWarps + kPiece) / kPiece;   // of a warp's share of the slice
constexpr int kListed = 320;             // tokens of a warp's list
constexpr uint64_t kOne = 1ull << kFraction, kAll = ~0ull;

struct Found {                 // a bin with a cut in it
    uint64_t lo, hi;           // the codes of its tokens are in lo .. hi; of the first histogram's: its number
    uint64_t need;             // tokens, or weight, up to the cut, of this bin
    uint64_t before;           // weight before the bin
    uint32_t count, upto;      // its tokens (0: there is no cut), and those of it and the bins before it
};

struct alignas(16) Shared {
    uint32_t count[kBins], low[kBins], high[kBins];   // a histogram: tokens, and sums in two words
    uint64_t before[kBins + 1];                       // the first histogram's sums, added up (first CTA)
    uint32_t first_count[kBins];
    uint64_t power[256];                              // 2^(44 - j / 256), of 2^4
    uint64_t list[2][kRanked];                        // codes that were sent to the first CTA, for each cut
    uint64_t list_weight[kRanked];
    uint64_t piece[kWarps][kMaxPieces];
    uint16_t listed_token[kWarps][kListed];           // of its share
    uint64_t warp_sum[kWarps];
    uint32_t warp_count[kWarps];
    uint64_t total, lo, hi;                           // of this CTA (total: of all weights, then of what is kept)
    uint64_t cut[2], upto;
    Found found[2];
    uint32_t top, bottom, listed[2], counted;                 // counted: tokens of the first histogram (first CTA)
};

// The powers for j = 0 .. 255, worked out by the compiler: products of 2^(-2^k / 256), each the root of
// the one before it (Newton's iteration), in doubles.
struct Table {
    uint64_t v[256];
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
            v[j] = static_cast<uint64_t>(p + 0.5) << (kFraction - 40);
        }
    }
};
__device__ const Table g_table = Table();

// Logits in their order as whole numbers, -0 as 0. (NaN have neither a place nor a weight: their t compares false.)
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
// The order of tokens: the larger logit first, then the lower index.
__device__ __forceinline__ uint64_t code_of(float x, uint32_t index) { return static_cast<uint64_t>(~key_of(x)) << 32 | index; }

struct Row {
    float top, c_hi, c_lo;        // max x; log2(e) / T
    const uint64_t *power;
};

// t of a logit, rounded: not below that of a larger logit.
__device__ __forceinline__ float rough_t(const Row &r, float x) { return x == r.top ? 0.0f : (r.top - x) * r.c_hi; }

__device__ __forceinline__ uint64_t weight(const Row &r, float x)
{
    const float d = r.top - x, t = d * r.c_hi;
    const float back = r.top - d;   // what d's rounding left: top - x = d + d_lo, exactly
    const float d_lo = (back - x) + (r.top - (d + back));
    const float t_lo = fmaf(d_lo, r.c_hi, fmaf(d, r.c_lo, fmaf(d, r.c_hi, -t)));
    constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to a whole number, in the low bits
    const float shifted = fmaf(fminf(t, kMostT), 256.0f, kMagic);
    const uint32_t k = __float_as_uint(shifted) - __float_as_uint(kMagic);
    const float z = fmaf(shifted - kMagic, -1.0f / 256.0f, t) + t_lo;   // |z| <= 0.002
    constexpr float kLn2 = 0.693147180559945f;
    const float series = z * fmaf(z, fmaf(z, -512.0f / 6.0f * kLn2 * kLn2 * kLn2, 256.0f * kLn2 * kLn2), -512.0f * kLn2);   // 2^9 (2^-z - 1)
    const uint64_t p = r.power[k & 255u];
    const uint64_t w = p + static_cast<int64_t>(__float2int_rn(__uint2float_rn(static_cast<uint32_t>(p >> (kFraction - 31))) * series)) * (1 << (kFraction - 40));
    return x == r.top ? kOne : t <= kMostT ? w >> (k >> 8) : 0;   // (t can be NaN)
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
    const int bin = threadIdx.x;
    uint32_t n = 0;
    uint64_t w = 0;
    if (threadIdx.x == 0) found.count = 0;
#pragma unroll 4
    for (unsigned r = 0; r < cluster.num_blocks(); ++r) {
        const Shared &o = *cluster.map_shared_rank(&s, r);
        n += o.count[bin];
        if (weights) w += (static_cast<uint64_t>(o.high[bin]) << 32) + o.low[bin];
    }
    uint32_t n_with = n;
    uint64_t w_with = w;
    scan(s, n_with, w_with);
    if (first_level) {
        s.before[bin] = w_with - w, s.first_count[bin] = n;
        if (bin == kBins - 1) s.before[kBins] = w_with, s.counted = n_with;
        if (by_weight) need = 0;   // not known before all sums are
    }
    const uint64_t with = by_weight ? w_with : n_with, at = with - (by_weight ? w : n);
    if (at < need && need <= with) {
        found.count = n;
        found.upto = n_with;
        found.need = need - at;
        found.before = before + w_with - w;
        found.lo = lo + (static_cast<uint64_t>(bin) << shift);
        found.hi = found.lo + ((static_cast<uint64_t>(1) << shift) - 1);
        if (found.hi > hi) found.hi = hi;
    }
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
    if (tid < 256) s.power[tid] = g_table.v[tid];
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
    if (!(T >= FLT_MIN) || top_p <= 0.0f || min_p > 1.0f) k = 1;   // (log2(e) / T is finite)
    cp_async_wait_all();
    __syncthreads();
    float most = -INFINITY, lowest = INFINITY;   // lowest: above -inf
#pragma unroll 4
    for (int i = tid; i < pieces; i += kThreads) {
        const float4 v = x4[i];
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
    r.power = s.power;
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
    const bool cut_p = top_p < 1.0f && k > 1, cut_k = k < g.V && k > 1;
    // The histogram spans what the row's logits do, a vocabulary of nearly equal ones too.
    const float range = 1.001f * rough_t(r, of_key(bottom));
    float span = fminf(kMostT, fmaxf(range, 1e-6f));
    // A warp's share of the slice, or a list of those of its tokens that can count, in their order
    const int share = 4 * ((pieces + kWarps - 1) / kWarps), first = warp * share;
    int tokens = max(0, min(share, 4 * pieces - first));
    bool listed = false;
    const uint16_t *list = s.listed_token[warp];
    // f(logit, index) for each of them
    auto each_token = [&](auto f) {
        if (listed) {
            for (int j = lane; j < tokens; j += 32) f(x[first + list[j]], static_cast<uint32_t>(index0 + first + list[j]));
            return;
        }
        for (int i = first + 4 * lane; i < first + tokens; i += 128) {
            const float4 v = *reinterpret_cast<const float4 *>(x + i);
            const uint32_t at = static_cast<uint32_t>(index0 + i);
            f(v.x, at), f(v.y, at + 1), f(v.z, at + 2), f(v.w, at + 3);
        }
    };
    const uint64_t least = min_p > 0.0f && k > 1 ? (min_p >= 1.0f ? kOne : max(static_cast<unsigned long long>(1), static_cast<unsigned long long>(share_above(min_p, kOne)))) : 1;
    uint64_t cut = kAll;   // the last kept token's code
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
    uint64_t whole = 0;   // all weights, where lists are made
    // Lists pay where most tokens are left out: by the row's range, as wide as that of normal logits of which a quarter is
    // listed. 32 rows of 151936 normal logits of standard deviation 3, 3.5 and 4, top-p 0.9: 55, 39 and 36 us for 59, 47 and
    // 41 without; 2 and 2.5, where lists would not hold them, 77 and 74 for 64 and 62. The range is that of all logits above -inf, so
    // masks of a finite value make any row wide: at 2, with one token masked by -1e9 76 us for 62, with half of them 64 (-inf 61), with
    // 98 of 100 masked by -1e4 31. (A pass that leaves them out of the range: 62 .. 66 in the first two, but 34 in the
    // last, 37 for 33 at 4, and for rows without masks 26.7 us for 25.9 with eight and 53 for 52 with 96.)
    const bool listing = cut_p && !cut_k && range > 23.0f - 3.6f * log2f(1.0f - top_p);
    if (listing) {
        uint64_t sum = 0;
        each_token([&](float v, uint32_t) { sum += weight(r, v); });
        sum = sum_over_cta(s, sum);
        if (tid == 0) s.total = sum;
        cluster.sync();
        whole = warp_sum64(lane < static_cast<int>(C) ? cluster.map_shared_rank(&s, lane)->total : 0);
        // Together, the tokens that are V / (1 - p) times lighter than the whole are behind the cut.
        span = fminf(span, log2f(static_cast<float>(g.V) * static_cast<float>(kOne) / ((1.0f - top_p) * static_cast<float>(whole))) + 0.01f);
        int n = 0;
#pragma unroll 4
        for (int j = lane; j - lane < tokens; j += 32) {
            const bool in = j < tokens && rough_t(r, x[first + j]) <= span;
            const uint32_t who = __ballot_sync(0xffffffffu, in);
            const int at = n + __popc(who & ((1u << lane) - 1));
            if (in && at < kListed) s.listed_token[warp][at] = static_cast<uint16_t>(j);
            n += __popc(who);
        }
        __syncwarp();
        listed = n <= kListed;
        if (listed) tokens = n;
    }
    const float per_t = static_cast<float>(kBins) / span;
    auto bin_of = [&](float t) { return min(static_cast<int>(t * per_t), kBins - 1); };
    if (cut_p || cut_k) {
        // Behind a small top-k, the histogram is of the threads' largest logits alone: as many of them as k are in
        // some first bins, so at least that many tokens are, and most likely few more. Those go to the first CTA.
        bool few = cut_k && k <= kRanked / 2;
        for (;;) {
            const bool weights = cut_p && !few;
            auto count = [&](float v, uint32_t) {
                const float t = rough_t(r, v);
                if (!(t <= span)) return;
                const int bin = bin_of(t);
                atomicAdd(&s.count[bin], 1u);
                if (weights) add64(s, bin, weight(r, v));
            };
            if (few) count(most, 0);
            else each_token(count);
            cluster.sync();
            if (rank == 0) {
                pick(cluster, s, s.found[0], weights, !cut_k, true, static_cast<uint64_t>(k), 0, kAll, 0, 0);
                if (tid == 0) s.upto = s.before[kBins];
                // fewer tokens of any weight than k, and few: the last bin is taken for the cut's
                if (tid == 0 && cut_k && !s.found[0].count && s.counted <= kRanked) s.found[0] = Found{kBins - 1, 0, 0, 0, s.counted, s.counted};
                if (!cut_k) {   // the share of the whole sum
                    if (!listing) whole = s.before[kBins];
                    const uint64_t y = share_above(top_p, whole);
                    const uint32_t upto = static_cast<uint32_t>(sum_over_cta(s, s.before[tid] < y ? s.first_count[tid] : 0));   // bins up to the cut's, all of them
                    if (s.before[tid] < y && y <= s.before[tid + 1])
                        s.found[0] = Found{static_cast<uint64_t>(tid), 0, y - s.before[tid], s.before[tid], s.first_count[tid], upto};
                    if (tid == 0) s.upto = whole;
                }
            }
            cluster.sync();
            const Found f = lead.found[0];
            if (f.count && f.upto <= kRanked) {   // few tokens: the first CTA sees to them
                const int last = static_cast<int>(f.lo);
                auto send = [&](float v, uint32_t at) {
                    const float t = rough_t(r, v);
                    if (!(t <= span) || bin_of(t) > last) return;
                    const uint32_t i = atomicAdd(&lead.listed[0], 1u);
                    if (i < kRanked) lead.list[0][i] = code_of(v, at);
                };
                if (listed) {
                    each_token(send);
                } else {
#pragma unroll 2
                    for (int i = first / 4 + lane; i < (first + tokens) / 4; i += 32) {
                        const float4 v = x4[i];
                        const float t = rough_t(r, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
                        if (!(t <= span) || bin_of(t) > last) continue;
                        const uint32_t at = static_cast<uint32_t>(index0 + 4 * i);
                        send(v.x, at), send(v.y, at + 1), send(v.z, at + 2), send(v.w, at + 3);
                    }
                }
                cluster.sync();
                const uint32_t n = few ? lead.listed[0] : f.upto;
                if (few) cluster.sync();   // all have read it
                if (n <= kRanked) {
                    if (rank == 0) draw_from_list(s, g, r, m, static_cast<int>(n), k, cut_k, cut_p, top_p, s.upto, least, u);
                    return;   // the others' memory is not read any more
                }
            }
            if (!few) break;
            few = false;   // more than a few after all
            clear_histogram(s);
            if (tid == 0) s.listed[0] = 0;
            cluster.sync();
        }
        for (int by_weight = cut_k ? 0 : 1; by_weight < (cut_p ? 2 : 1); ++by_weight) {
            const int which = by_weight && cut_k ? 1 : 0;
            if (which) {   // a top-p behind a top-k
                if (rank == 0) {
                    if (tid == 0) s.found[1].count = 0;
                    const uint64_t y = share_above(top_p, s.upto);
                    __syncthreads();
                    if (s.before[tid] < y && y <= s.before[tid + 1])
                        s.found[1] = Found{static_cast<uint64_t>(tid), 0, y - s.before[tid], s.before[tid], s.first_count[tid], 0};
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
                    const int shift = max(0, 64 - __clzll(static_cast<long long>(f.hi - f.lo)) - 9);
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
    // what is kept, in pieces
    // (first what one comparison of fp32 shows: below the last kept logit, or far below min_p)
    const float cut_x = cut == kAll ? -INFINITY : of_key(~static_cast<uint32_t>(cut >> 32));
    const float most_t = min_p > 0.0f && min_p < 1.0f ? fminf(kMostT, 0.001f - log2f(min_p)) : kMostT;
    auto kept = [&](float v, uint32_t at) -> uint64_t {
        if (v < cut_x || !(rough_t(r, v) <= most_t) || code_of(v, at) > cut) return 0;
        const uint64_t w = weight(r, v);
        return w >= least ? w : 0;
    };
    auto kept_at = [&](int j) -> uint64_t {
        if (j >= tokens) return 0;
        const int i = first + (listed ? list[j] : j);
        return kept(x[i], static_cast<uint32_t>(index0 + i));
    };
    uint64_t mine = 0;
    for (int p = 0; p * kPiece < tokens; ++p) {
        uint64_t w = kept_at(p * kPiece + lane) + kept_at(p * kPiece + 32 + lane);
        // a sum of 64 weights' low 24 bits, and of what is above, fit 32 bits
        w = (static_cast<uint64_t>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w >> 24))) << 24) +
            __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w) & 0xffffffu);
        if (lane == 0) s.piece[warp][p] = w;
        mine += w;
    }
    const uint64_t of_cta = sum_over_cta(s, lane == 0 ? mine : 0);
    if (tid == 0) s.total = of_cta;
    cluster.sync();
    // (inclusive sums over a warp's lanes)
    auto scanned = [&](uint64_t v) {
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint64_t b = shfl_up64(v, o);
            if (lane >= o) v += b;
        }
        return v;
    };
    const uint64_t upto_rank = scanned(lane < static_cast<int>(C) ? cluster.map_shared_rank(&s, lane)->total : 0);
    const uint64_t total = __shfl_sync(0xffffffffu, upto_rank, C - 1), y = drawn(u, total);
    uint64_t at = __shfl_sync(0xffffffffu, upto_rank, rank) - of_cta;
    for (int i = 0; i < warp; ++i) at += s.warp_sum[i];
    if (at <= y && y < at + mine) {
        __syncwarp();
        int p = 0;
        for (; y >= at + s.piece[warp][p]; ++p) at += s.piece[warp][p];
#pragma unroll 1
        for (int j = p * kPiece + lane; j < (p + 1) * kPiece; j += 32) {
            const uint64_t w = kept_at(j), upto = scanned(w);
            if (at + upto - w <= y && y < at + upto) {
                g.token[m] = index0 + first + (listed ? list[j] : j);
                if (g.prob) g.prob[m] = ratio(w, total);
            }
            at += __shfl_sync(0xffffffffu, upto, 31);
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
