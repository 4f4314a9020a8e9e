// Which sizes of the orthogonalised update go to its one-launch kernel (host only).
#pragma once

#include <stdint.h>

namespace bstq {

constexpr int kSmallRows = 128, kSmallCols = 256, kWidestCluster = 16;

// Blocks that share a matrix of q columns, up to 256 to a block.
inline int cluster_of(int64_t q)
{
    int blocks = 1;
    while ((int64_t)blocks * kSmallCols < q)
        blocks *= 2;
    return blocks;
}

// 128 rows, and 256 columns for each of up to 16 blocks of a cluster (64 x 4000 float
// 110 us against 184 in tiles, 3 x 128 x 4096 bf16 83 against 123), as far as the
// device places clusters of `widest` blocks.
inline bool is_small(int64_t m, int64_t n, int widest)
{
    const int64_t p = m < n ? m : n, q = m < n ? n : m;
    return p <= kSmallRows && cluster_of(q) <= (widest < kWidestCluster ? widest : kWidestCluster);
}

}  // namespace bstq
