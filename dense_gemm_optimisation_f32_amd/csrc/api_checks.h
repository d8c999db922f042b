// api_checks.h -- argument checks shared by the C-ABI layers (host code, no HIP call).
#pragma once

#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "../../include/mi355gemm.h"

namespace {

constexpr int kMaxSum = 1 << 30;   // a sum's length (K, or a weight gradient's R), a quantised side: positions in slices and tiles past the last stay ints

inline bool misaligned(const void *p, uintptr_t align)
{
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) % align) != 0;
}

// (rows-1)*ld + cols stays within 64 bits.
inline bool extent(long long rows, long long cols, long long ld, long long *out)
{
    *out = 0;
    if (rows == 0 || cols == 0) return true;
    if (rows > 1 && ld > (LLONG_MAX / 8 - cols) / (rows - 1)) return false;
    *out = (rows - 1) * ld + cols;
    return true;
}

// `members` matrices of `one` elements a `stride` apart: the stride holds one
// matrix and the whole extent stays within 64 bits.
inline int batch_extent(long long members, long long one, long long stride, bool apart)
{
    if (stride < 0 || (apart && members > 1 && stride < one)) return GEMM_ERR_LD;
    if (members > 1 && stride > 0 && members - 1 > (LLONG_MAX / 8 - one) / stride) return GEMM_ERR_SIZE;
    return GEMM_OK;
}

inline bool flag(int v)
{
    return v == 0 || v == 1;
}

inline int launched(hipError_t e)
{
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace
