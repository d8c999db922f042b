// routed_internal.h -- launchers of the products whose right operand is chosen
// per row (routing to experts, the experts' products, combining, low-rank
// adapters), shared between the C-ABI layer (routed_api.cpp) and the kernels.
// Not part of the public interface.  Every problem has been checked by the
// C-ABI layer; sizes are positive, offsets are 64-bit where they can be large.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mi355gemm {

// A launch is held below 2^31 threads (the runtime takes fewer than 2^32).
inline bool grid_holds(long long groups_of_threads, int threads)
{
    return groups_of_threads <= 0x7FFFFFFF / threads;
}

constexpr int kMaxExperts = 1024;   // route: experts, one wave holds a token's scores
constexpr int kMaxChoices = 32;     // route, combine: choices of a token
constexpr int kMaxRouteGroups = 64; // route: expert groups, one lane each
constexpr int kMaxRank = 128;       // lora

struct RouteProblem {
    int T, E, k;
    const float *logits;
    long long ldl;
    const float *bias;              // E values or nullptr
    int score;                      // 0 softmax, 1 sigmoid
    int groups, group_k, group_top;
    int renorm;
    float scale;
    int32_t *ids;                   // T x k
    float *weights;                 // T x k
    int32_t *offsets, *rows, *slots;   // E + 1, T*k, T x k; all three or none
    int32_t *counts;                // workspace: (chunks + 1) x (E + 1)
};
// Workspace bytes launch_route needs (0: none).
size_t route_workspace(int T, int E, int k);
hipError_t launch_route(const RouteProblem &p, hipStream_t stream);

struct RouteGradProblem {
    int T, E, k;
    const float *logits;
    long long ldl;
    int score, renorm;
    float scale;
    const int32_t *ids;
    const float *dweights;
    float *dlogits;
    long long lddl;
};
hipError_t launch_route_grad(const RouteGradProblem &p, hipStream_t stream);

struct CombineProblem {
    int T, k, N;
    const float *Y;
    int R;                          // rows of Y; slots outside [0, R) are skipped
    long long ldy;
    const int32_t *slots;           // T x k
    const float *weights;           // T x k, or nullptr for ones
    float beta;
    float *C;
    long long ldc;
};
hipError_t launch_combine(const CombineProblem &p, hipStream_t stream);

struct CombineGradProblem {
    int T, k, N;
    const float *dC;
    long long lddc;
    const float *Y;
    int R;
    long long ldy;
    const int32_t *slots;
    const float *weights;
    uint16_t *dY;
    long long lddy;
    float *dweights;
};
hipError_t launch_combine_grad(const CombineGradProblem &p, bool bf, hipStream_t stream);

// C[r,:] = alpha * A[rows[r],:] * op(B_g) + beta * C[r,:] for offsets[g] <= r < offsets[g+1].
struct GroupedProblem {
    int transB, groups, R, N, K;    // K = 0: no product (A and B are not read)
    float alpha, beta;
    const uint16_t *A;
    int M;                          // rows of A; a row index outside [0, M) reads as a row of zeros
    long long lda;
    const int32_t *rows;            // R indices, or nullptr for r
    const uint16_t *B;
    long long ldb, strideB;
    const int32_t *offsets;         // groups + 1
    float *C;
    long long ldc;
};
// A tile of the kernels that take this call has a grid that one launch holds.
bool grouped_fits(const GroupedProblem &p);
hipError_t launch_grouped(const GroupedProblem &p, bool bf, hipStream_t stream);

// C_g = alpha * sum over offsets[g] <= r < offsets[g+1] of A[rowsA[r],:]^T B[rowsB[r],:] + beta * C_g (M x N).
struct WgradProblem {
    int groups, R, M, N;            // R = 0: no product
    float alpha, beta;
    const uint16_t *A;
    int a_rows;
    long long lda;
    const int32_t *rowsA;
    const uint16_t *B;
    int b_rows;
    long long ldb;
    const int32_t *rowsB;
    const int32_t *offsets;
    float *C;
    long long ldc, strideC;
};
bool wgrad_fits(const WgradProblem &p);
hipError_t launch_wgrad(const WgradProblem &p, bool bf, hipStream_t stream);

// C[i,:] = alpha * (A[i,:] op(B) + scales[a] * (A[i,:] LA_a^T) LB_a^T) + beta * C[i,:], a = ids[i].
struct LoraProblem {
    int transB, M, N, K, rank, adapters;   // K = 0: no product
    float alpha, beta;
    const uint16_t *A;
    long long lda;
    const uint16_t *B;
    long long ldb;
    const uint16_t *LA;             // adapters x rank x K
    long long ldla, strideLA;
    const uint16_t *LB;             // adapters x N x rank
    long long ldlb, strideLB;
    const float *scales;            // adapters values, or nullptr for ones
    const int32_t *ranks;           // adapters values clamped to [0, rank], or nullptr for rank
    const int32_t *ids;             // M values; outside [0, adapters): no adapter
    float *C;
    long long ldc;
    float *t;                       // workspace
};
bool lora_fits(const LoraProblem &p);
size_t lora_workspace(int M, int N, int K, int rank);
hipError_t launch_lora(const LoraProblem &p, bool bf, hipStream_t stream);

}  // namespace mi355gemm
