// Host-side helpers that the entry points of every translation unit share.
#pragma once

#include <cuda_runtime.h>

#include <stdint.h>

namespace bstq {

struct DevInfo {
    int sms = 0;
    int max_smem_block = 0;
    int max_regs_sm = 0;
    int max_threads_sm = 0;
    int major = 0, minor = 0;
};

// Properties of the current device (false when there is none).
bool dev_info(DevInfo &out);

// Cycles after which a kernel's wait gives up (bstq_set_wait_limit).
long long wait_limit();

// Keeps the text of a CUDA error for bstq_last_error; returns BSTQ_ERR_CUDA.
int cuda_fail(cudaError_t err, const char *what);

// Whether an output's rows lie apart: `row` elements each, n0 of them s0 elements
// apart in each of n1 groups that are s1 apart.
inline bool rows_apart(int64_t row, int64_t n0, int64_t s0, int64_t n1, int64_t s1)
{
    if (n0 == 0 || n1 == 0)
        return true;
    if (n0 < n1) {
        const int64_t n = n0, s = s0;
        n0 = n1, s0 = s1, n1 = n, s1 = s;
    }
    if ((n0 > 1 && s0 < row) || (n1 > 1 && s1 < row))
        return false;
    if (n1 <= 1)
        return true;
    typedef __int128 wide;
    if (s1 >= (wide)(n0 - 1) * s0 + row || s0 >= (wide)(n1 - 1) * s1 + row)
        return true;
    // rows of both axes in turn: none within `row` of one that is k groups away
    for (int64_t k = 1; k < n1; ++k) {
        const wide d = (wide)k * s1, below = d / s0;
        if (below >= n0)
            return d - (wide)(n0 - 1) * s0 >= row;  // and so the groups further off
        if (d - below * s0 < row || (below + 1 < n0 && (below + 1) * s0 - d < row))
            return false;
    }
    return true;
}

inline bool misaligned_to(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace bstq
