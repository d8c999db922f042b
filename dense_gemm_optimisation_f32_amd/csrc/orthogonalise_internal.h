// orthogonalise_internal.h -- the launcher of the orthogonalised update, shared between the
// C-ABI layer (orthogonalise_api.cpp) and the kernels.  Not part of the public interface.
// Every problem has been checked by the C-ABI layer; sizes are positive.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

namespace mi355gemm {

constexpr int kMaxOrthoSide = 65536;
constexpr int kMaxOrthoSteps = 100;

struct OrthoProblem {
    int M, N, steps;
    const float *coefficients;   // host memory, three a step
    float alpha;
    const void *G;               // fp32 or bf16
    long long ldg, strideG;
    uint16_t *O;                 // bf16
    long long ldo, strideO;
    int batch;
    void *workspace;
};
bool ortho_fits(int M, int N, int batch);
size_t ortho_workspace(int M, int N, int batch);   // 0 where one workgroup holds a member
hipError_t launch_ortho(const OrthoProblem &p, bool bf, hipStream_t stream);

// One workgroup holds a member (orthogonalise_small.hip).
bool ortho_small(int M, int N);
hipError_t launch_ortho_small(const OrthoProblem &p, bool bf, hipStream_t stream);

// The fp16 copies of X are scaled by a power of two: its rows end up with a norm near 1 over n entries, entries near 1
// then.  (Those of A and B need none: their small entries are small beside a X.)
inline float ortho_x_scale(int M, int N)
{
    return std::exp2(std::floor(0.5f * std::log2((float)(M > N ? M : N))));
}

}  // namespace mi355gemm
