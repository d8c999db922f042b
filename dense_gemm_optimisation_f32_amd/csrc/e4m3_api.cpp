// e4m3_api.cpp -- the exported C ABI of the operators on 8-bit floats with a scale per
// block of 128 (include/mi355gemm.h): argument checks, quick returns and dispatch to the
// kernel launchers.  Argument checks run before any HIP call, so they work on a host with
// no GPU.
#include "api_checks.h"
#include "e4m3_internal.h"

namespace {

int ceil_div(int a, int b)
{
    return a / b + (a % b != 0);
}

int at_least_1(int v)
{
    return v > 1 ? v : 1;
}

bool block_ok(int b)
{
    return b == 1 || b == mi355gemm::kScaleBlock;
}

int quant(int transpose, int block, int M, int K, const void *X, int ldx, long long strideX, uint8_t *Q, int ldq, long long strideQ,
          float *S, int lds, long long strideS, int batch_count, mi355gemm::QuantType type, hipStream_t stream)
{
    if (!flag(transpose)) return GEMM_ERR_OP;
    if (!block_ok(block) || M < 0 || K < 0 || M > kMaxSum || K > kMaxSum || batch_count < 0) return GEMM_ERR_SIZE;
    const int rows = transpose ? K : M, cols = transpose ? M : K, kb = ceil_div(K, 128), rb = ceil_div(M, block);
    if (ldx < at_least_1(cols) || ldq < at_least_1(K) || lds < at_least_1(rb)) return GEMM_ERR_LD;
    long long ex, eq, es;
    if (!extent(rows, cols, ldx, &ex) || !extent(M, K, ldq, &eq) || !extent(kb, rb, lds, &es)) return GEMM_ERR_SIZE;
    if (const int rc = batch_extent(batch_count, ex, strideX, false); rc != GEMM_OK) return rc;
    if (const int rc = batch_extent(batch_count, eq, strideQ, true); rc != GEMM_OK) return rc;
    if (const int rc = batch_extent(batch_count, es, strideS, true); rc != GEMM_OK) return rc;
    if (M == 0 || K == 0 || batch_count == 0) return GEMM_OK;
    mi355gemm::QuantProblem p;
    p.transpose = transpose; p.block = block; p.M = M; p.K = K;
    p.X = X; p.ldx = ldx; p.strideX = strideX;
    p.Q = Q; p.ldq = ldq; p.strideQ = strideQ;
    p.S = S; p.lds = lds; p.strideS = strideS;
    p.batch = batch_count;
    if (!mi355gemm::quant_fits(p, type)) return GEMM_ERR_SIZE;
    if (!X || !Q || !S) return GEMM_ERR_NULL;
    if (misaligned(X, type == mi355gemm::QuantType::f32 ? 4 : 2) || misaligned(S, 4)) return GEMM_ERR_ALIGN;
    return launched(mi355gemm::launch_quant(p, type, stream));
}

// Both products; offsets are read where `ragged`.
int product(bool ragged, int blockB, int groups, int R, int N, int K, float alpha, const uint8_t *A, int M, int lda, const float *SA,
            int ldsa, const int32_t *rows, const uint8_t *B, int ldb, long long strideB, const float *SB, int ldsb, long long strideSB,
            const int32_t *offsets, float beta, float *C, int ldc, hipStream_t stream)
{
    if (!block_ok(blockB) || groups < 0 || groups > 65535 || R < 0 || N < 0 || K < 0 || K > kMaxSum || M < 0) return GEMM_ERR_SIZE;
    const int kb = ceil_div(K, 128), nb = ceil_div(N, blockB);
    if (lda < at_least_1(K) || ldsa < at_least_1(M) || ldb < at_least_1(K) || ldsb < at_least_1(nb) || ldc < at_least_1(N))
        return GEMM_ERR_LD;
    long long ea, esa, eb, esb, ec;
    if (!extent(M, K, lda, &ea) || !extent(kb, M, ldsa, &esa) || !extent(N, K, ldb, &eb) || !extent(kb, nb, ldsb, &esb) ||
        !extent(R, N, ldc, &ec))
        return GEMM_ERR_SIZE;
    if (const int rc = batch_extent(groups, eb, strideB, false); rc != GEMM_OK) return rc;
    if (const int rc = batch_extent(groups, esb, strideSB, false); rc != GEMM_OK) return rc;
    if (groups == 0 || R == 0 || N == 0) return GEMM_OK;
    const bool multiplies = K > 0 && alpha != 0.f && M > 0;
    mi355gemm::E4m3Problem p;
    p.blockB = blockB; p.groups = groups; p.R = R; p.N = N; p.K = multiplies ? K : 0;
    p.alpha = alpha; p.beta = beta;
    p.A = A; p.M = M; p.lda = lda; p.SA = SA; p.ldsa = ldsa; p.rows = multiplies ? rows : nullptr;   // (not read without a product)
    p.B = B; p.ldb = ldb; p.strideB = strideB; p.SB = SB; p.ldsb = ldsb; p.strideSB = strideSB;
    p.offsets = offsets;
    p.C = C; p.ldc = ldc;
    if (!mi355gemm::e4m3_fits(p)) return GEMM_ERR_SIZE;
    if (!C || (ragged && !offsets) || (multiplies && (!A || !SA || !B || !SB))) return GEMM_ERR_NULL;
    if (misaligned(C, 4) || (ragged && misaligned(offsets, 4)) || misaligned(rows, 4) || (multiplies && (misaligned(SA, 4) || misaligned(SB, 4))))
        return GEMM_ERR_ALIGN;
    return launched(mi355gemm::launch_e4m3(p, stream));
}

}  // namespace

extern "C" {

int quant_e4m3_f32(int transpose, int block, int M, int K, const float *X, int ldx, long long strideX, uint8_t *Q, int ldq,
                   long long strideQ, float *S, int lds, long long strideS, int batch_count, hipStream_t stream)
{
    return quant(transpose, block, M, K, X, ldx, strideX, Q, ldq, strideQ, S, lds, strideS, batch_count, mi355gemm::QuantType::f32, stream);
}

int quant_e4m3_f16(int transpose, int block, int M, int K, const uint16_t *X, int ldx, long long strideX, uint8_t *Q, int ldq,
                   long long strideQ, float *S, int lds, long long strideS, int batch_count, hipStream_t stream)
{
    return quant(transpose, block, M, K, X, ldx, strideX, Q, ldq, strideQ, S, lds, strideS, batch_count, mi355gemm::QuantType::f16, stream);
}

int quant_e4m3_bf16(int transpose, int block, int M, int K, const uint16_t *X, int ldx, long long strideX, uint8_t *Q, int ldq,
                    long long strideQ, float *S, int lds, long long strideS, int batch_count, hipStream_t stream)
{
    return quant(transpose, block, M, K, X, ldx, strideX, Q, ldq, strideQ, S, lds, strideS, batch_count, mi355gemm::QuantType::bf16, stream);
}

int gemm_e4m3_f32acc(int blockB, int M, int N, int K, float alpha, const uint8_t *A, int lda, const float *SA, int ldsa, const uint8_t *B,
                     int ldb, const float *SB, int ldsb, float beta, float *C, int ldc, hipStream_t stream)
{
    return product(false, blockB, 1, M, N, K, alpha, A, M, lda, SA, ldsa, nullptr, B, ldb, 0, SB, ldsb, 0, nullptr, beta, C, ldc, stream);
}

int gemm_grouped_e4m3_f32acc(int blockB, int groups, int R, int N, int K, float alpha, const uint8_t *A, int M, int lda, const float *SA,
                             int ldsa, const int32_t *rows, const uint8_t *B, int ldb, long long strideB, const float *SB, int ldsb,
                             long long strideSB, const int32_t *offsets, float beta, float *C, int ldc, hipStream_t stream)
{
    return product(true, blockB, groups, R, N, K, alpha, A, M, lda, SA, ldsa, rows, B, ldb, strideB, SB, ldsb, strideSB, offsets, beta, C,
                   ldc, stream);
}

}  // extern "C"
