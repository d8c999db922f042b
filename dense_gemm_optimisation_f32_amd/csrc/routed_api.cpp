// routed_api.cpp -- the exported C ABI of the products whose right operand is
// chosen per row (include/mi355gemm.h): argument checks, quick returns and
// dispatch to the kernel launchers.  Argument checks run before any HIP call, so
// they work on a host with no GPU.
#include <limits.h>
#include <stdint.h>

#include "../../include/mi355gemm.h"
#include "routed_internal.h"

namespace {

// Tokens of one call, and columns of the element-wise kernels: a launch holds
// fewer than 2^32 threads, and a grid's second axis 65535 blocks.  (The products'
// grids are checked for the tiles that take a call.)
constexpr int kMaxTokens = 1 << 23;
constexpr int kMaxCols = 1 << 25;
constexpr int kMaxSum = 1 << 30;   // a sum's length (K, or a weight gradient's R): positions in slices past the last stay ints

bool misaligned(const void *p, uintptr_t align)
{
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) % align) != 0;
}

// (rows-1)*ld + cols stays within 64 bits.
bool extent(long long rows, long long cols, long long ld, long long *out)
{
    *out = 0;
    if (rows == 0 || cols == 0) return true;
    if (rows > 1 && ld > (LLONG_MAX / 8 - cols) / (rows - 1)) return false;
    *out = (rows - 1) * ld + cols;
    return true;
}

// `members` matrices of `one` elements a `stride` apart: the stride holds one
// matrix and the whole extent stays within 64 bits.
int batch_extent(long long members, long long one, long long stride, bool apart)
{
    if (stride < 0 || (apart && members > 1 && stride < one)) return GEMM_ERR_LD;
    if (members > 1 && stride > 0 && members - 1 > (LLONG_MAX / 8 - one) / stride) return GEMM_ERR_SIZE;
    return GEMM_OK;
}

bool flag(int v)
{
    return v == 0 || v == 1;
}

int launched(hipError_t e)
{
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

bool route_sizes_ok(int T, int E, int k)
{
    return T >= 0 && T <= kMaxTokens && E >= 1 && E <= mi355gemm::kMaxExperts && k >= 1 && k <= mi355gemm::kMaxChoices &&
           k <= E;
}

int grouped(int transB, int groups, int R, int N, int K, float alpha, const uint16_t *A, int M, int lda,
            const int32_t *rows, const uint16_t *B, int ldb, long long strideB, const int32_t *offsets, float beta,
            float *C, int ldc, bool bf, hipStream_t stream)
{
    if (!flag(transB)) return GEMM_ERR_OP;
    if (groups < 0 || R < 0 || N < 0 || K < 0 || M < 0 || groups > 65535 || K > kMaxSum) return GEMM_ERR_SIZE;
    const long long b_rows = transB ? N : K, b_cols = transB ? K : N;
    if (lda < (K > 1 ? K : 1) || ldb < (b_cols > 1 ? b_cols : 1) || ldc < (N > 1 ? N : 1)) return GEMM_ERR_LD;
    long long ea, eb, ec;
    if (!extent(M, K, lda, &ea) || !extent(b_rows, b_cols, ldb, &eb) || !extent(R, N, ldc, &ec)) return GEMM_ERR_SIZE;
    if (const int rc = batch_extent(groups, eb, strideB, false); rc != GEMM_OK) return rc;
    if (groups == 0 || R == 0 || N == 0) return GEMM_OK;
    const bool product = K > 0 && alpha != 0.f && M > 0;
    mi355gemm::GroupedProblem p;
    p.transB = transB; p.groups = groups; p.R = R; p.N = N; p.K = product ? K : 0;
    p.alpha = alpha; p.beta = beta;
    p.A = A; p.M = M; p.lda = lda; p.rows = product ? rows : nullptr;   // (not read without a product)
    p.B = B; p.ldb = ldb; p.strideB = strideB;
    p.offsets = offsets;
    p.C = C; p.ldc = ldc;
    if (!mi355gemm::grouped_fits(p)) return GEMM_ERR_SIZE;
    if (!C || !offsets || (product && (!A || !B))) return GEMM_ERR_NULL;
    if (misaligned(C, 4) || misaligned(offsets, 4) || misaligned(rows, 4) ||
        (product && (misaligned(A, 2) || misaligned(B, 2))))
        return GEMM_ERR_ALIGN;
    return launched(mi355gemm::launch_grouped(p, bf, stream));
}

int wgrad(int groups, int R, int M, int N, float alpha, const uint16_t *A, int a_rows, int lda, const int32_t *rowsA,
          const uint16_t *B, int b_rows, int ldb, const int32_t *rowsB, const int32_t *offsets, float beta, float *C,
          int ldc, long long strideC, bool bf, hipStream_t stream)
{
    if (groups < 0 || R < 0 || M < 0 || N < 0 || a_rows < 0 || b_rows < 0 || groups > 65535 || R > kMaxSum)
        return GEMM_ERR_SIZE;
    if (lda < (M > 1 ? M : 1) || ldb < (N > 1 ? N : 1) || ldc < (N > 1 ? N : 1)) return GEMM_ERR_LD;
    long long ea, eb, ec;
    if (!extent(a_rows, M, lda, &ea) || !extent(b_rows, N, ldb, &eb) || !extent(M, N, ldc, &ec)) return GEMM_ERR_SIZE;
    if (const int rc = batch_extent(groups, ec, strideC, true); rc != GEMM_OK) return rc;
    if (groups == 0 || M == 0 || N == 0) return GEMM_OK;
    const bool product = R > 0 && alpha != 0.f && a_rows > 0 && b_rows > 0;
    mi355gemm::WgradProblem p;
    p.groups = groups; p.R = product ? R : 0; p.M = M; p.N = N;
    p.alpha = alpha; p.beta = beta;
    p.A = A; p.a_rows = a_rows; p.lda = lda; p.rowsA = rowsA;
    p.B = B; p.b_rows = b_rows; p.ldb = ldb; p.rowsB = rowsB;
    p.offsets = offsets;
    p.C = C; p.ldc = ldc; p.strideC = strideC;
    if (!mi355gemm::wgrad_fits(p)) return GEMM_ERR_SIZE;
    if (!C || (product && (!A || !B || !offsets))) return GEMM_ERR_NULL;
    if (misaligned(C, 4) || (product && (misaligned(A, 2) || misaligned(B, 2) || misaligned(offsets, 4) ||
                                         misaligned(rowsA, 4) || misaligned(rowsB, 4))))
        return GEMM_ERR_ALIGN;
    return launched(mi355gemm::launch_wgrad(p, bf, stream));
}

bool combine_sizes_ok(int T, int k, int N, int R)
{
    return T >= 0 && T <= kMaxTokens && k >= 1 && k <= mi355gemm::kMaxChoices && N >= 0 && N <= kMaxCols && R >= 0;
}

int combine_grad(int T, int k, int N, const float *dC, int lddc, const float *Y, int R, int ldy, const int32_t *slots,
                 const float *weights, uint16_t *dY, int lddy, float *dweights, bool bf, hipStream_t stream)
{
    if (!combine_sizes_ok(T, k, N, R)) return GEMM_ERR_SIZE;
    const int N1 = N > 1 ? N : 1;
    if (lddc < N1 || ldy < N1 || lddy < N1) return GEMM_ERR_LD;
    long long e;
    if (!extent(T, N, lddc, &e) || !extent(R, N, ldy, &e) || !extent(R, N, lddy, &e)) return GEMM_ERR_SIZE;
    if (T == 0) return GEMM_OK;
    if (!slots || !dweights || (N > 0 && (!dC || (R > 0 && (!Y || !dY))))) return GEMM_ERR_NULL;
    if (misaligned(slots, 4) || misaligned(dweights, 4) || misaligned(weights, 4) || misaligned(dC, 4) ||
        misaligned(Y, 4) || misaligned(dY, 2))
        return GEMM_ERR_ALIGN;
    mi355gemm::CombineGradProblem p;
    p.T = T; p.k = k; p.N = N;
    p.dC = dC; p.lddc = lddc;
    p.Y = Y; p.R = R; p.ldy = ldy;
    p.slots = slots; p.weights = weights;
    p.dY = dY; p.lddy = lddy;
    p.dweights = dweights;
    return launched(mi355gemm::launch_combine_grad(p, bf, stream));
}

bool lora_sizes_ok(int M, int N, int K, int rank)
{
    return M >= 0 && N >= 0 && K >= 0 && K <= kMaxSum && rank >= 1 && rank <= mi355gemm::kMaxRank && M <= kMaxTokens && N <= kMaxCols;
}

int lora(int transB, int M, int N, int K, int rank, int adapters, float alpha, const uint16_t *A, int lda,
         const uint16_t *B, int ldb, const uint16_t *LA, int ldla, long long strideLA, const uint16_t *LB, int ldlb,
         long long strideLB, const float *scales, const int32_t *ranks, const int32_t *ids, float beta, float *C, int ldc,
         void *workspace, long long workspace_bytes, bool bf, hipStream_t stream)
{
    if (!flag(transB)) return GEMM_ERR_OP;
    if (!lora_sizes_ok(M, N, K, rank) || adapters < 0) return GEMM_ERR_SIZE;
    const long long b_rows = transB ? N : K, b_cols = transB ? K : N;
    const int K1 = K > 1 ? K : 1;
    if (lda < K1 || ldb < (b_cols > 1 ? b_cols : 1) || ldc < (N > 1 ? N : 1) || ldla < K1 || ldlb < rank)
        return GEMM_ERR_LD;
    long long ea, eb, ec, ela, elb;
    if (!extent(M, K, lda, &ea) || !extent(b_rows, b_cols, ldb, &eb) || !extent(M, N, ldc, &ec) ||
        !extent(rank, K, ldla, &ela) || !extent(N, rank, ldlb, &elb))
        return GEMM_ERR_SIZE;
    if (const int rc = batch_extent(adapters, ela, strideLA, false); rc != GEMM_OK) return rc;
    if (const int rc = batch_extent(adapters, elb, strideLB, false); rc != GEMM_OK) return rc;
    if (M == 0 || N == 0) return GEMM_OK;
    const bool product = K > 0 && alpha != 0.f;
    mi355gemm::LoraProblem p;
    p.transB = transB; p.M = M; p.N = N; p.K = product ? K : 0; p.rank = rank; p.adapters = product ? adapters : 0;
    p.alpha = alpha; p.beta = beta;
    p.A = A; p.lda = lda; p.B = B; p.ldb = ldb;
    p.LA = LA; p.ldla = ldla; p.strideLA = strideLA;
    p.LB = LB; p.ldlb = ldlb; p.strideLB = strideLB;
    p.scales = scales; p.ranks = ranks; p.ids = ids;
    p.C = C; p.ldc = ldc;
    p.t = static_cast<float *>(workspace);
    if (!mi355gemm::lora_fits(p)) return GEMM_ERR_SIZE;
    if (!C) return GEMM_ERR_NULL;
    if (product && (!A || !B || (adapters > 0 && (!LA || !LB || !ids)))) return GEMM_ERR_NULL;
    if (misaligned(C, 4)) return GEMM_ERR_ALIGN;
    if (product && (misaligned(A, 2) || misaligned(B, 2) || misaligned(LA, 2) || misaligned(LB, 2) || misaligned(ids, 4) ||
                    misaligned(scales, 4) || misaligned(ranks, 4)))
        return GEMM_ERR_ALIGN;
    if (product && adapters > 0) {
        const size_t need = mi355gemm::lora_workspace(M, N, K, rank);
        if (workspace_bytes < 0 || (size_t)workspace_bytes < need) return GEMM_ERR_SCRATCH;
        if (need > 0 && !workspace) return GEMM_ERR_NULL;
        if (misaligned(workspace, 16)) return GEMM_ERR_ALIGN;
    }
    return launched(mi355gemm::launch_lora(p, bf, stream));
}

}  // namespace

extern "C" {

long long moe_route_workspace(int T, int E, int k)
{
    return route_sizes_ok(T, E, k) && T > 0 ? (long long)mi355gemm::route_workspace(T, E, k) : 0;
}

int moe_route_f32(int T, int E, const float *logits, int ldl, const float *bias, int score, int groups, int group_k,
                  int group_top, int k, int renorm, float scale, int32_t *ids, float *weights, int32_t *offsets,
                  int32_t *rows, int32_t *slots, void *workspace, long long workspace_bytes, hipStream_t stream)
{
    if (!flag(score) || !flag(renorm)) return GEMM_ERR_OP;
    if (!route_sizes_ok(T, E, k)) return GEMM_ERR_SIZE;
    if (groups < 1 || groups > mi355gemm::kMaxRouteGroups || E % groups != 0 || group_k < 1 || group_k > groups ||
        group_top < 1 || group_top > 2)
        return GEMM_ERR_SIZE;
    if (ldl < E) return GEMM_ERR_LD;
    long long e;
    if (!extent(T, E, ldl, &e)) return GEMM_ERR_SIZE;
    const bool layout = offsets || rows || slots;
    if (layout && (!offsets || (T > 0 && (!rows || !slots)))) return GEMM_ERR_NULL;
    if (T > 0 && (!logits || !ids || !weights)) return GEMM_ERR_NULL;
    if (misaligned(logits, 4) || misaligned(bias, 4) || misaligned(ids, 4) || misaligned(weights, 4) ||
        misaligned(offsets, 4) || misaligned(rows, 4) || misaligned(slots, 4))
        return GEMM_ERR_ALIGN;
    if (T == 0 && !layout) return GEMM_OK;
    if (T > 0 && layout) {
        const size_t need = mi355gemm::route_workspace(T, E, k);
        if (workspace_bytes < 0 || (size_t)workspace_bytes < need) return GEMM_ERR_SCRATCH;
        if (need > 0 && !workspace) return GEMM_ERR_NULL;
        if (misaligned(workspace, 4)) return GEMM_ERR_ALIGN;
    }
    mi355gemm::RouteProblem p;
    p.T = T; p.E = E; p.k = k;
    p.logits = logits; p.ldl = ldl; p.bias = bias;
    p.score = score; p.groups = groups; p.group_k = group_k; p.group_top = group_top;
    p.renorm = renorm; p.scale = scale;
    p.ids = ids; p.weights = weights;
    p.offsets = offsets; p.rows = rows; p.slots = slots;
    p.counts = static_cast<int32_t *>(workspace);
    return launched(mi355gemm::launch_route(p, stream));   // T = 0: the offsets are zeros
}

int moe_route_f32_grad(int T, int E, const float *logits, int ldl, int score, int k, int renorm, float scale,
                       const int32_t *ids, const float *dweights, float *dlogits, int lddl, hipStream_t stream)
{
    if (!flag(score) || !flag(renorm)) return GEMM_ERR_OP;
    if (!route_sizes_ok(T, E, k)) return GEMM_ERR_SIZE;
    if (ldl < E || lddl < E) return GEMM_ERR_LD;
    long long e;
    if (!extent(T, E, ldl, &e) || !extent(T, E, lddl, &e)) return GEMM_ERR_SIZE;
    if (T == 0) return GEMM_OK;
    if (!logits || !ids || !dweights || !dlogits) return GEMM_ERR_NULL;
    if (misaligned(logits, 4) || misaligned(ids, 4) || misaligned(dweights, 4) || misaligned(dlogits, 4))
        return GEMM_ERR_ALIGN;
    mi355gemm::RouteGradProblem p;
    p.T = T; p.E = E; p.k = k;
    p.logits = logits; p.ldl = ldl;
    p.score = score; p.renorm = renorm; p.scale = scale;
    p.ids = ids; p.dweights = dweights;
    p.dlogits = dlogits; p.lddl = lddl;
    return launched(mi355gemm::launch_route_grad(p, stream));
}

int gemm_grouped_f16_f32acc_ex(int transB, int groups, int R, int N, int K, float alpha, const uint16_t *A, int M, int lda,
                               const int32_t *rows, const uint16_t *B, int ldb, long long strideB, const int32_t *offsets,
                               float beta, float *C, int ldc, hipStream_t stream)
{
    return grouped(transB, groups, R, N, K, alpha, A, M, lda, rows, B, ldb, strideB, offsets, beta, C, ldc, false, stream);
}

int gemm_grouped_bf16_f32acc_ex(int transB, int groups, int R, int N, int K, float alpha, const uint16_t *A, int M,
                                int lda, const int32_t *rows, const uint16_t *B, int ldb, long long strideB,
                                const int32_t *offsets, float beta, float *C, int ldc, hipStream_t stream)
{
    return grouped(transB, groups, R, N, K, alpha, A, M, lda, rows, B, ldb, strideB, offsets, beta, C, ldc, true, stream);
}

int gemm_grouped_wgrad_f16_f32acc(int groups, int R, int M, int N, float alpha, const uint16_t *A, int a_rows, int lda,
                                  const int32_t *rowsA, const uint16_t *B, int b_rows, int ldb, const int32_t *rowsB,
                                  const int32_t *offsets, float beta, float *C, int ldc, long long strideC,
                                  hipStream_t stream)
{
    return wgrad(groups, R, M, N, alpha, A, a_rows, lda, rowsA, B, b_rows, ldb, rowsB, offsets, beta, C, ldc, strideC,
                 false, stream);
}

int gemm_grouped_wgrad_bf16_f32acc(int groups, int R, int M, int N, float alpha, const uint16_t *A, int a_rows, int lda,
                                   const int32_t *rowsA, const uint16_t *B, int b_rows, int ldb, const int32_t *rowsB,
                                   const int32_t *offsets, float beta, float *C, int ldc, long long strideC,
                                   hipStream_t stream)
{
    return wgrad(groups, R, M, N, alpha, A, a_rows, lda, rowsA, B, b_rows, ldb, rowsB, offsets, beta, C, ldc, strideC, true,
                 stream);
}

int moe_combine_f32(int T, int k, int N, const float *Y, int R, int ldy, const int32_t *slots, const float *weights,
                    float beta, float *C, int ldc, hipStream_t stream)
{
    if (!combine_sizes_ok(T, k, N, R)) return GEMM_ERR_SIZE;
    const int N1 = N > 1 ? N : 1;
    if (ldy < N1 || ldc < N1) return GEMM_ERR_LD;
    long long e;
    if (!extent(R, N, ldy, &e) || !extent(T, N, ldc, &e)) return GEMM_ERR_SIZE;
    if (T == 0 || N == 0) return GEMM_OK;
    if (!slots || !C || (R > 0 && !Y)) return GEMM_ERR_NULL;
    if (misaligned(Y, 4) || misaligned(slots, 4) || misaligned(weights, 4) || misaligned(C, 4)) return GEMM_ERR_ALIGN;
    mi355gemm::CombineProblem p;
    p.T = T; p.k = k; p.N = N;
    p.Y = Y; p.R = R; p.ldy = ldy;
    p.slots = slots; p.weights = weights;
    p.beta = beta;
    p.C = C; p.ldc = ldc;
    return launched(mi355gemm::launch_combine(p, stream));
}

int moe_combine_grad_f16(int T, int k, int N, const float *dC, int lddc, const float *Y, int R, int ldy,
                         const int32_t *slots, const float *weights, uint16_t *dY, int lddy, float *dweights,
                         hipStream_t stream)
{
    return combine_grad(T, k, N, dC, lddc, Y, R, ldy, slots, weights, dY, lddy, dweights, false, stream);
}

int moe_combine_grad_bf16(int T, int k, int N, const float *dC, int lddc, const float *Y, int R, int ldy,
                          const int32_t *slots, const float *weights, uint16_t *dY, int lddy, float *dweights,
                          hipStream_t stream)
{
    return combine_grad(T, k, N, dC, lddc, Y, R, ldy, slots, weights, dY, lddy, dweights, true, stream);
}

long long gemm_lora_workspace(int M, int N, int K, int rank)
{
    return lora_sizes_ok(M, N, K, rank) && M > 0 && N > 0 && K > 0 ? (long long)mi355gemm::lora_workspace(M, N, K, rank) : 0;
}

int gemm_lora_f16_f32acc_ex(int transB, int M, int N, int K, int rank, int adapters, float alpha, const uint16_t *A, int lda,
                            const uint16_t *B, int ldb, const uint16_t *LA, int ldla, long long strideLA,
                            const uint16_t *LB, int ldlb, long long strideLB, const float *scales, const int32_t *ranks,
                            const int32_t *ids, float beta, float *C, int ldc, void *workspace,
                            long long workspace_bytes, hipStream_t stream)
{
    return lora(transB, M, N, K, rank, adapters, alpha, A, lda, B, ldb, LA, ldla, strideLA, LB, ldlb, strideLB, scales, ranks,
                ids, beta, C, ldc, workspace, workspace_bytes, false, stream);
}

int gemm_lora_bf16_f32acc_ex(int transB, int M, int N, int K, int rank, int adapters, float alpha, const uint16_t *A, int lda,
                             const uint16_t *B, int ldb, const uint16_t *LA, int ldla, long long strideLA,
                             const uint16_t *LB, int ldlb, long long strideLB, const float *scales, const int32_t *ranks,
                             const int32_t *ids, float beta, float *C, int ldc, void *workspace,
                             long long workspace_bytes, hipStream_t stream)
{
    return lora(transB, M, N, K, rank, adapters, alpha, A, lda, B, ldb, LA, ldla, strideLA, LB, ldlb, strideLB, scales, ranks,
                ids, beta, C, ldc, workspace, workspace_bytes, true, stream);
}

}  // extern "C"
