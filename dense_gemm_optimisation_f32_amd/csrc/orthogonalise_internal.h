// orthogonalise_internal.h -- the launcher of the orthogonalised update, shared between the
// C-ABI layer (orthogonalise_api.cpp) and the kernels.  Not part of the public interface.
// Every problem has been checked by the C-ABI layer; sizes are positive.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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
size_t ortho_workspace(int M, int N, int batch);
hipError_t launch_ortho(const OrthoProblem &p, bool bf, hipStream_t stream);

}  // namespace mi355gemm
