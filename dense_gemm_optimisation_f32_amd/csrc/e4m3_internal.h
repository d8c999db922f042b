// e4m3_internal.h -- launchers of the operators on 8-bit floats with a scale per block of
// 128, shared between the C-ABI layer (e4m3_api.cpp) and the kernels.  Not part of the
// public interface.  Every problem has been checked by the C-ABI layer; sizes are positive.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mi355gemm {

constexpr int kScaleBlock = 128;   // k per scale, and rows per scale of two-dimensional blocks

enum class QuantType { f32, f16, bf16 };

// Q = X or X^T in e4m3 with scales S[(k / 128) * lds + row / block].
struct QuantProblem {
    int transpose, block, M, K;   // Q is M x K
    const void *X;
    long long ldx, strideX;
    uint8_t *Q;
    long long ldq, strideQ;
    float *S;
    long long lds, strideS;
    int batch;
};
bool quant_fits(const QuantProblem &p, QuantType type);
hipError_t launch_quant(const QuantProblem &p, QuantType type, hipStream_t stream);

// C[r,:] = alpha * A[rows[r],:] B_g^T + beta * C[r,:] for offsets[g] <= r < offsets[g+1], the
// entries of A and B times their scales.  offsets == nullptr: one group of all R rows.
struct E4m3Problem {
    int blockB;                    // rows of B per scale: 1 or 128
    int groups, R, N, K;           // K = 0: no product (A and B are not read)
    float alpha, beta;
    const uint8_t *A;
    int M;                         // rows of A; a row index outside [0, M) reads as a row of zeros
    long long lda;
    const float *SA;
    long long ldsa;
    const int32_t *rows;           // R indices, or nullptr for r
    const uint8_t *B;              // groups members N x K
    long long ldb, strideB;
    const float *SB;
    long long ldsb, strideSB;
    const int32_t *offsets;        // groups + 1, or nullptr
    float *C;
    long long ldc;
};
bool e4m3_fits(const E4m3Problem &p);
hipError_t launch_e4m3(const E4m3Problem &p, hipStream_t stream);

}  // namespace mi355gemm
