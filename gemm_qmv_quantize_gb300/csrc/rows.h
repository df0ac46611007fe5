// rows.h -- counts of rows, which may be up to 2^31 - 1, in 32 bits that do not overflow:
// what is left is compared, not where it ends. For host and device code.
#pragma once

#ifdef __CUDACC__
#define QMV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define QMV_HOST_DEVICE inline
#endif

namespace qmv {

// Groups of n rows that M rows, one at least, make.
QMV_HOST_DEVICE constexpr int groups_of(int M, int n) { return (M - 1) / n + 1; }

// Whether row m + ahead is one of M; 0 <= m <= M, and ahead is not negative.
QMV_HOST_DEVICE constexpr bool row_ahead(int m, int ahead, int M) { return ahead < M - m; }

// Rows m, m + step, ..: `left` of them all, this one the first, are not gone through yet.
struct RowsInTurn {
    unsigned m;      // may pass 2^31 behind the last
    int step, left;
    // whether the row n steps on is there; n * step is small
    QMV_HOST_DEVICE bool ahead(int n) const { return n * step < left; }
    QMV_HOST_DEVICE int row(int n) const { return static_cast<int>(m + static_cast<unsigned>(n * step)); }   // of one that is
    QMV_HOST_DEVICE void next() { m += static_cast<unsigned>(step), left -= step; }
};

}  // namespace qmv
