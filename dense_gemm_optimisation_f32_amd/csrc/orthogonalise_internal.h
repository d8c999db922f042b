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

// B's diagonal multiplies X in two parts: what this returns, in B's fp16 copy, X's fp16 copy X + E (E the copy's rounding), and
// the rest fp32's X.  B = b A + c A A, whole, times E stays in X's range (its left singular vectors) and shrinks with the singular
// value squared; a diagonal times E alone leaves that range, and what is outside grows by a factor a in every step.  So by default
// the diagonal goes with the rest of B.  Where row i of A has hardly anything beside its diagonal it need not: with P the
// projection onto X's range, A_ii^2 = <A e_i, P e_i>^2 <= |A e_i|^2 P_ii, so at most r / (1 + r) of e_i's square is outside, r = (sum of
// A_ij^2 over j != i) / A_ii^2.  There fp32's X takes the share 1 - 1024 r (if above 0), which leaves at most (1 - 1024 r) sqrt(r) <= 0.012
// of the diagonal times E outside.
// (All of it with fp32's X: 4e-2 off for two parallel rows.  None of it: single rows and orthogonal ones 1.4e-3, now 5e-4.)
// How exactly the share is computed does not matter: the caller leaves what this returns out of the rest.
constexpr float kAlone = 1024.f;
__device__ __forceinline__ _Float16 diagonal_of_copy(float b_ii, float a_ii, float others)
{
    const float q = kAlone * others, square = a_ii * a_ii;
    return (_Float16)(q < square ? b_ii * (q * __builtin_amdgcn_rcpf(fmaxf(square, 1e-37f))) : b_ii);
}

}  // namespace mi355gemm
