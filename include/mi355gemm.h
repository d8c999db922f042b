/*
 * mi355gemm.h -- row-major GEMM on one AMD Instinct MI355X (gfx950), C ABI.
 *
 * Every gemm_f32*, gemm_f16*, gemm_bf16* and gemm_batched_* entry point computes,
 * for row-major matrices (the calls whose right operand is chosen per row stand
 * at the end, with their own formulas),
 *
 *     C <- alpha * A * B + beta * C,      A: M x K,  B: K x N,  C: M x N
 *
 * which is the general matrix multiply C = alpha*op(A)op(B) + beta*C of the
 * MindNotes 'GEMM' page (section "core problem and arithmetic
 * characteristics") with op the identity.  That page's "cuBLAS engineering
 * interface" sections fix the other parts of the interface used here: a
 * leading dimension is the distance in elements between the starts of two
 * consecutive rows and may exceed the logical width (section "Leading
 * Dimension (lda, ldb, ldc)"); a strided batch is a set of same-shape GEMMs
 * placed a fixed element stride apart and run by one call, and mixed precision
 * means fp16 inputs with fp32 accumulation (section "Batched execution and
 * mixed precision").  Unlike cuBLAS the storage is row-major, there is no
 * handle, and alpha/beta are host values passed by value.
 *
 * Layout: element (i,k) of A is A[i*lda + k], (k,j) of B is B[k*ldb + j],
 * (i,j) of C is C[i*ldc + j].  Batched member b starts at A + b*strideA,
 * B + b*strideB, C + b*strideC (strides in elements).
 *
 * Ownership: A, B and C are device pointers owned by the caller.  The library
 * allocates no memory, keeps no state besides its loaded kernels, and never
 * synchronises: each call enqueues its kernels on `stream` (0 = the null
 * stream) and returns.  C must not overlap A or B, and batched C members must
 * not overlap one another.
 *
 * Semantics the pages leave open, taken from the BLAS reference:
 *   - beta == 0: C is written without being read (it may hold NaN);
 *   - K == 0 or alpha == 0: C <- beta*C (C <- 0 when beta == 0 too); A and B
 *     are not read;
 *   - M == 0, N == 0 or batch_count == 0: nothing is done.
 *
 * Errors: every entry point returns an int status.  Arguments are checked
 * before any HIP call; on an error nothing is enqueued.  Codes 0 to -4 are the
 * BLAS-style set (size, leading dimension or stride, NULL pointer, launch
 * refused); -5 and -6 report the two conditions that set has no code for (an
 * element-misaligned pointer, a transpose flag other than 0 or 1).
 */
#ifndef MI355GEMM_H
#define MI355GEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t *hipStream_t; /* the HIP runtime's stream handle */

enum {
    GEMM_OK = 0,
    GEMM_ERR_SIZE = -1,      /* M, N, K or batch_count negative, an extent overflows 64 bits, or
                                ceil(M/32)*ceil(N/32) exceeds INT_MAX (one launch's grid); for the
                                calls by row, a size outside the range they document */
    GEMM_ERR_LD = -2,        /* lda < max(1,K), ldb < max(1,N) (with transA: lda < max(1,M); with
                                transB: ldb < max(1,K)), ldc < max(1,N), negative stride, or
                                strideC smaller than one C member when batch_count > 1 */
    GEMM_ERR_NULL = -3,      /* NULL pointer for an operand that the call would read or write */
    GEMM_ERR_LAUNCH = -4,    /* the HIP runtime refused a kernel launch (hipGetLastError) */
    GEMM_ERR_ALIGN = -5,     /* pointer not aligned to its element size */
    GEMM_ERR_OP = -6,        /* transA or transB is neither 0 nor 1 */
    GEMM_ERR_SCRATCH = -7    /* gemm_f16_f32acc_noalloc: the call needs more scratch than the
                                library's static buffer holds; calls that take a workspace: it is
                                smaller than the call needs */
};

/*
 * gemm_f32 -- SGEMM: fp32 A, B, C; fp32 multiply-add.
 *   M, N, K    : logical sizes (>= 0).
 *   alpha, beta: fp32 scalars.
 *   A, lda     : device fp32, M x K row-major, lda >= max(1,K).
 *   B, ldb     : device fp32, K x N row-major, ldb >= max(1,N).
 *   C, ldc     : device fp32, M x N row-major, ldc >= max(1,N); read only when beta != 0.
 *   stream     : HIP stream the kernels are enqueued on.
 * Results agree with the fp64 definition to a normalized error
 * |C - ref| / (|alpha| sum_k |a_ik||b_kj| + |beta||c_ij|) <= 1e-5 and are
 * bit-identical from call to call for the same arguments.
 */
int gemm_f32(int M, int N, int K, float alpha,
             const float *A, int lda, const float *B, int ldb,
             float beta, float *C, int ldc, hipStream_t stream);

/*
 * gemm_f16_f32acc -- HGEMM: A and B hold IEEE binary16 values (bit patterns in
 * uint16_t), products are formed exactly and accumulated in fp32; alpha, beta
 * and C are fp32.  Arguments as for gemm_f32.
 */
int gemm_f16_f32acc(int M, int N, int K, float alpha,
                    const uint16_t *A, int lda, const uint16_t *B, int ldb,
                    float beta, float *C, int ldc, hipStream_t stream);

/*
 * gemm_batched_f16_f32acc -- batch_count independent HGEMMs of one shape.
 *   strideA, strideB, strideC: element distance between consecutive members
 *   (>= 0; strideA/strideB may be 0 to reuse one operand; strideC must be at
 *   least (M-1)*ldc + N when batch_count > 1).
 * Other arguments as for gemm_f16_f32acc; batch_count >= 0.
 */
int gemm_batched_f16_f32acc(int M, int N, int K, float alpha,
                            const uint16_t *A, int lda, long long strideA,
                            const uint16_t *B, int ldb, long long strideB,
                            float beta, float *C, int ldc, long long strideC,
                            int batch_count, hipStream_t stream);

/*
 * The _ex forms compute C <- alpha*op(A)*op(B) + beta*C, op(X) = X or X^T, the
 * general form of the MindNotes page's definition (section "core problem and
 * arithmetic characteristics").  op(A) is M x K and op(B) is K x N:
 *   transA = 0: A is stored M x K, element (i,k) at A[i*lda + k], lda >= max(1,K);
 *   transA = 1: A is stored K x M, element (i,k) at A[k*lda + i], lda >= max(1,M);
 *   transB = 0: B is stored K x N, element (k,j) at B[k*ldb + j], ldb >= max(1,N);
 *   transB = 1: B is stored N x K, element (k,j) at B[j*ldb + k], ldb >= max(1,K).
 * C is always M x N row-major.  Flags other than 0 or 1 return GEMM_ERR_OP.
 * Everything else is as for the entry points above (which are the _ex forms
 * with transA = transB = 0).
 */
int gemm_f32_ex(int transA, int transB, int M, int N, int K, float alpha,
                const float *A, int lda, const float *B, int ldb,
                float beta, float *C, int ldc, hipStream_t stream);

int gemm_f16_f32acc_ex(int transA, int transB, int M, int N, int K, float alpha,
                       const uint16_t *A, int lda, const uint16_t *B, int ldb,
                       float beta, float *C, int ldc, hipStream_t stream);

int gemm_batched_f16_f32acc_ex(int transA, int transB, int M, int N, int K, float alpha,
                               const uint16_t *A, int lda, long long strideA,
                               const uint16_t *B, int ldb, long long strideB,
                               float beta, float *C, int ldc, long long strideC,
                               int batch_count, hipStream_t stream);

/*
 * bfloat16 inputs.  The MindNotes page's mixed-precision interface (section
 * "Batched execution and mixed precision") takes either fp16 or bf16 inputs
 * with fp32 accumulation.  These four entry points are the bf16 forms of
 * gemm_f16_f32acc, gemm_batched_f16_f32acc, gemm_f16_f32acc_ex and
 * gemm_batched_f16_f32acc_ex, in that order: A and B hold bfloat16 values (the
 * upper 16 bits of an IEEE binary32, as uint16_t bit patterns), products are
 * formed exactly and accumulated in fp32; alpha, beta and C are fp32.
 * Arguments, layout, ownership, status codes and the accuracy statement are
 * as for the fp16 forms.
 */
int gemm_bf16_f32acc(int M, int N, int K, float alpha,
                     const uint16_t *A, int lda, const uint16_t *B, int ldb,
                     float beta, float *C, int ldc, hipStream_t stream);

int gemm_batched_bf16_f32acc(int M, int N, int K, float alpha,
                             const uint16_t *A, int lda, long long strideA,
                             const uint16_t *B, int ldb, long long strideB,
                             float beta, float *C, int ldc, long long strideC,
                             int batch_count, hipStream_t stream);

int gemm_bf16_f32acc_ex(int transA, int transB, int M, int N, int K, float alpha,
                        const uint16_t *A, int lda, const uint16_t *B, int ldb,
                        float beta, float *C, int ldc, hipStream_t stream);

int gemm_batched_bf16_f32acc_ex(int transA, int transB, int M, int N, int K, float alpha,
                                const uint16_t *A, int lda, long long strideA,
                                const uint16_t *B, int ldb, long long strideB,
                                float beta, float *C, int ldc, long long strideC,
                                int batch_count, hipStream_t stream);

/*
 * gemm_f16_f32acc_noalloc -- gemm_f16_f32acc for callers that cannot allocate
 * device memory (code under graph capture, tight serving loops, harnesses that
 * forbid hipMalloc).  Same arguments, results and status codes, plus
 * GEMM_ERR_SCRATCH.  Where gemm_f16_f32acc splits a tile's K range over several
 * workgroups it keeps the partial tiles and counters in scratch that the
 * library allocates per (device, stream) on first need; this form uses instead
 * one static device buffer per GPU, 8.25 MiB (256 KiB of tile counters and 128
 * fp32 partial tiles of 128 x 128), which covers every split the library makes,
 * and calls no allocating routine.  That buffer is shared by every call of this
 * entry point on the GPU and keeps the last call's contents: calls that overlap
 * on one GPU (different streams, or graphs replayed concurrently) race and must
 * not be made.  A call that would need more scratch returns GEMM_ERR_SCRATCH
 * and enqueues nothing.
 */
int gemm_f16_f32acc_noalloc(int M, int N, int K, float alpha,
                            const uint16_t *A, int lda, const uint16_t *B, int ldb,
                            float beta, float *C, int ldc, hipStream_t stream);

/*
 * Products whose right operand is chosen per row: routing tokens to experts,
 * the experts' products over the sorted rows, the weighted sum back to tokens,
 * and low-rank adapters beside a shared projection.
 *
 * Index arrays (int32) and offsets are device memory and are read by the
 * kernels only; a value that would lead outside an operand is never followed
 * (what happens instead stands with each call), so that they can come straight
 * from other kernels and be captured into a graph.  All matrices are row-major
 * with caller-chosen leading dimensions; C does not overlap another operand.
 * Calls that need scratch take it from the caller (`workspace`, at least
 * `workspace_bytes` = what the *_workspace function returns for the same sizes,
 * 16-byte aligned; contents before and after are of no account).  Two calls that
 * can overlap, replays of two captured graphs among them, need two workspaces.
 * Results are bit-identical from call to call for the same arguments.
 *
 * C of a product is at most what one launch's tiles cover, beyond it GEMM_ERR_SIZE: 2^23 - 1 tiles
 * of 64 x 64 (2^35 elements of C), of 128 x 128 with transB = 1 and for weight gradients; 2^22 - 1 of
 * 256 x 256 where rows start at dwords and hold whole 16-byte chunks (pointers at multiples of 4,
 * even leading dimensions and strides, K, or the N (M) of operands stored along it, a
 * multiple of 8).  Rows of groups count R / (tile rows) + min(groups, R) row tiles.
 */

/*
 * moe_route_f32 -- each of T tokens chooses k of E experts.
 *   logits         : fp32, T x E, ldl >= E.
 *   score          : 0: s = softmax over the token's E logits; 1: s = sigmoid(logit).
 *   bias           : E fp32 values or NULL.  c = s + bias ranks the experts; the
 *                    weights are made of s.
 *   groups, group_k, group_top: experts g*E/groups .. form group g.  A group's score
 *                    is the sum of its best group_top (1 or 2) available c; only the
 *                    group_k best groups' experts can be chosen.  groups = 1: no groups.
 *   renorm, scale  : weight_j = scale * s_j, or with renorm = 1
 *                    scale * s_j / (sum of the token's chosen s); 0 where that sum is 0.
 *   ids, weights   : T x k, contiguous: the choices in descending c, of equal ones
 *                    (and groups) the lowest index first; NaN ranks below every number.
 * An expert is unavailable to a token whose logit for it is -inf, and to all if its
 * bias is -inf.  Choices that find no available expert have id -1 and weight 0, so a
 * padded token is a row of -inf.  c is formed and compared in 64 bits (with softmax
 * or sigmoid scores, no bias and group_top 1 the logits order the experts alike).
 * The choices sorted by expert (offsets, rows and slots; all three or all NULL):
 *   offsets        : E + 1 values; expert e's rows are offsets[e] .. offsets[e+1]-1, in
 *                    the order of their tokens.
 *   rows           : T*k values: the token of each row; -1 from offsets[E] on.
 *   slots          : T x k: the row of each choice; -1 for an unfilled one.
 * Sizes: T <= 2^23, E <= 1024, k <= min(E, 32), groups <= 64 and a divisor of E.
 * The workspace is used for the sorted choices only.
 */
int moe_route_f32(int T, int E, const float *logits, int ldl, const float *bias, int score,
                  int groups, int group_k, int group_top, int k, int renorm, float scale,
                  int32_t *ids, float *weights, int32_t *offsets, int32_t *rows, int32_t *slots,
                  void *workspace, long long workspace_bytes, hipStream_t stream);
long long moe_route_workspace(int T, int E, int k);

/*
 * moe_route_f32_grad -- the gradient of moe_route_f32's weights in the logits:
 * dlogits (T x E, lddl >= E, every entry written) from dweights (T x k) and the ids
 * that were chosen (ids outside 0 .. E-1 get no gradient).  The choice itself and
 * the bias have none.  logits, score, renorm and scale as for moe_route_f32.
 */
int moe_route_f32_grad(int T, int E, const float *logits, int ldl, int score, int k, int renorm, float scale,
                       const int32_t *ids, const float *dweights, float *dlogits, int lddl, hipStream_t stream);

/*
 * gemm_grouped_*_f32acc_ex -- rows in groups, each group with its own right operand:
 *     C[r,:] <- alpha * A[rows[r],:] * op(B_g) + beta * C[r,:]   for offsets[g] <= r < offsets[g+1]
 *   R, N, K : C is R x N, op(B_g) is K x N.
 *   A, M    : M x K, lda >= max(1,K).
 *   rows    : R int32 indices of rows of A, or NULL for r itself; outside 0 .. M-1: the row's
 *             product is zeros, whatever B_g holds.
 *   B       : groups members strideB elements apart (0: one shared), each stored K x N
 *             (transB = 0, ldb >= max(1,N)) or N x K (transB = 1, ldb >= max(1,K)).
 *   offsets : groups + 1 ascending int32 values; they are clamped to 0 .. R.  Rows of C in no
 *             group are left as they are.
 * With transB flipped this is also the gradient in A's rows.  groups <= 65535, K <= 2^30.
 */
int gemm_grouped_f16_f32acc_ex(int transB, int groups, int R, int N, int K, float alpha,
                               const uint16_t *A, int M, int lda, const int32_t *rows,
                               const uint16_t *B, int ldb, long long strideB, const int32_t *offsets,
                               float beta, float *C, int ldc, hipStream_t stream);
int gemm_grouped_bf16_f32acc_ex(int transB, int groups, int R, int N, int K, float alpha,
                                const uint16_t *A, int M, int lda, const int32_t *rows,
                                const uint16_t *B, int ldb, long long strideB, const int32_t *offsets,
                                float beta, float *C, int ldc, hipStream_t stream);

/*
 * gemm_grouped_wgrad_*_f32acc -- the gradient in the groups' right operands:
 *     C_g <- alpha * sum over offsets[g] <= r < offsets[g+1] of A[rowsA[r],:]^T B[rowsB[r],:] + beta * C_g
 *   A : a_rows x M, lda >= max(1,M); B : b_rows x N, ldb >= max(1,N); rowsA, rowsB: R indices or
 *       NULL for r; outside the operand: a row of zeros (0 times an infinity is NaN here as
 *       elsewhere: where the other operand may hold one, take its row out too).
 *   C : groups members M x N, strideC apart (at least (M-1)*ldc + N); an empty group's is
 *       beta * C_g.
 * For weights stored N x K swap the two operands.  groups <= 65535, R <= 2^30.
 */
int gemm_grouped_wgrad_f16_f32acc(int groups, int R, int M, int N, float alpha,
                                  const uint16_t *A, int a_rows, int lda, const int32_t *rowsA,
                                  const uint16_t *B, int b_rows, int ldb, const int32_t *rowsB,
                                  const int32_t *offsets, float beta, float *C, int ldc, long long strideC,
                                  hipStream_t stream);
int gemm_grouped_wgrad_bf16_f32acc(int groups, int R, int M, int N, float alpha,
                                   const uint16_t *A, int a_rows, int lda, const int32_t *rowsA,
                                   const uint16_t *B, int b_rows, int ldb, const int32_t *rowsB,
                                   const int32_t *offsets, float beta, float *C, int ldc, long long strideC,
                                   hipStream_t stream);

/*
 * moe_combine_f32 -- the experts' rows back in token order:
 *     C[t,:] <- sum_j weights[t,j] * Y[slots[t,j],:] + beta * C[t,:]
 * in the order of j.  Y is R x N, C is T x N; slots T x k (outside 0 .. R-1: skipped, the
 * weight is then of no account); weights T x k or NULL for ones.  T <= 2^23, k <= 32,
 * N <= 2^25.  With NULL weights this is the gradient of a gathering grouped product's rows.
 */
int moe_combine_f32(int T, int k, int N, const float *Y, int R, int ldy, const int32_t *slots,
                    const float *weights, float beta, float *C, int ldc, hipStream_t stream);

/*
 * moe_combine_grad_* -- its gradient: dY[slots[t,j],:] = weights[t,j] * dC[t,:], rounded once
 * to the 16-bit type that the grouped products take, and dweights[t,j] = <dC[t,:], Y[slots[t,j],:]>
 * (0 for a skipped slot).  Rows of dY that no slot names are left as they are; slots of
 * one call are distinct (as moe_route_f32 makes them).
 */
int moe_combine_grad_f16(int T, int k, int N, const float *dC, int lddc, const float *Y, int R, int ldy,
                         const int32_t *slots, const float *weights, uint16_t *dY, int lddy, float *dweights,
                         hipStream_t stream);
int moe_combine_grad_bf16(int T, int k, int N, const float *dC, int lddc, const float *Y, int R, int ldy,
                          const int32_t *slots, const float *weights, uint16_t *dY, int lddy, float *dweights,
                          hipStream_t stream);

/*
 * gemm_lora_*_f32acc_ex -- one projection for all rows and a low-rank adapter per row:
 *     C[i,:] <- alpha * (A[i,:] op(B) + scales[a] * (A[i,:] LA_a^T) LB_a^T) + beta * C[i,:],  a = ids[i]
 *   A, B, C, transB : as for gemm_*_f32acc_ex with transA = 0.
 *   LA      : adapters members rank x K (ldla >= max(1,K)), strideLA apart.
 *   LB      : adapters members N x rank (ldlb >= rank), strideLB apart.
 *   scales  : a value per adapter, or NULL for ones.
 *   ranks   : a rank per adapter (clamped to 0 .. rank), or NULL for rank; what LA and LB hold
 *             past an adapter's rank is not used.
 *   ids     : M int32 values; outside 0 .. adapters-1: no adapter for that row.
 * The narrow product A LA^T is a sum in fp32 and stays in fp32 precision (fp16, more than 64 rows: values
 * below 2^-37 of their row's largest are held to 2^-61 of that).  A row's result depends on its own
 * adapter alone, whatever the others hold.  M <= 2^23, N <= 2^25, K <= 2^30, 1 <= rank <= 128.
 */
int gemm_lora_f16_f32acc_ex(int transB, int M, int N, int K, int rank, int adapters, float alpha,
                            const uint16_t *A, int lda, const uint16_t *B, int ldb,
                            const uint16_t *LA, int ldla, long long strideLA,
                            const uint16_t *LB, int ldlb, long long strideLB,
                            const float *scales, const int32_t *ranks, const int32_t *ids,
                            float beta, float *C, int ldc,
                            void *workspace, long long workspace_bytes, hipStream_t stream);
int gemm_lora_bf16_f32acc_ex(int transB, int M, int N, int K, int rank, int adapters, float alpha,
                             const uint16_t *A, int lda, const uint16_t *B, int ldb,
                             const uint16_t *LA, int ldla, long long strideLA,
                             const uint16_t *LB, int ldlb, long long strideLB,
                             const float *scales, const int32_t *ranks, const int32_t *ids,
                             float beta, float *C, int ldc,
                             void *workspace, long long workspace_bytes, hipStream_t stream);
long long gemm_lora_workspace(int M, int N, int K, int rank);

/*
 * 8-bit floating point (e4m3: four exponent bits, three fraction bits, 448 the largest value,
 * NaN but no infinity) with a scale for each block of 128 k.  The number at (i, k) of a matrix
 * is its 8-bit value times S[(k / 128) * lds + i / block]: a scale belongs to 128 k of one row
 * (block 1) or of 128 rows (block 128), and scales lie with the blocks of k outermost.
 * What a call writes (Q, S, C, O) overlaps none of its operands.
 */

/*
 * quant_e4m3_* -- Q and S from op(X), X in fp32, fp16 or bf16, for batch_count members:
 *   transpose = 0: X is stored M x K (ldx >= max(1,K)); 1: K x M (ldx >= max(1,M)), Q is of its transpose.
 *   Q : M x K, ldq >= max(1,K); bytes between rows are left as they are.
 *   S : ceil(K / 128) x ceil(M / block), lds >= max(1, ceil(M / block)); block is 1 or 128.
 *   strideX, strideQ, strideS: elements between members (strideQ and strideS at least a member).
 * A scale is the least power of two s with max|x| / s <= 448 over the block's finite values, at least 2^-126,
 * and 1 for a block of zeros; a value is x / s rounded to the nearest e4m3 value, ties to the even one (x / s itself
 * is not rounded).  Infinities and NaN become NaN and do not count for the scale.
 * M, K <= 2^30; fewer than 2^23 tiles of 128 x 128 (2^22 in fp32) over all members, of 32 x 512 with transpose = 0 and block 1.
 */
int quant_e4m3_f32(int transpose, int block, int M, int K, const float *X, int ldx, long long strideX,
                   uint8_t *Q, int ldq, long long strideQ, float *S, int lds, long long strideS,
                   int batch_count, hipStream_t stream);
int quant_e4m3_f16(int transpose, int block, int M, int K, const uint16_t *X, int ldx, long long strideX,
                   uint8_t *Q, int ldq, long long strideQ, float *S, int lds, long long strideS,
                   int batch_count, hipStream_t stream);
int quant_e4m3_bf16(int transpose, int block, int M, int K, const uint16_t *X, int ldx, long long strideX,
                    uint8_t *Q, int ldq, long long strideQ, float *S, int lds, long long strideS,
                    int batch_count, hipStream_t stream);

/*
 * gemm_e4m3_f32acc -- C <- alpha * A * B^T + beta * C for the numbers that A (M x K) and B (N x K) stand for:
 *     C[i,j] <- alpha * sum over kb of SA[kb,i] * SB[kb,j/blockB] * (sum over k in block kb of A[i,k] * B[j,k]) + beta * C[i,j]
 *   A, lda, SA, ldsa : 8-bit values, lda >= max(1,K), and a scale per row and 128 k, ldsa >= max(1,M).
 *   B, ldb, SB, ldsb : 8-bit values, ldb >= max(1,K), and a scale per blockB (1 or 128) rows and 128 k,
 *                      ldsb >= max(1, ceil(N / blockB)).
 * Scales are any fp32 values; a product of two scales is formed first, and rounded as fp32 rounds it.
 * C is fp32, M x N.  A layer's output is x W^T with blocks of 128 of W; its input gradient is g W with W turned
 * (quant_e4m3_* with transpose, or the same values and scales transposed), its weight gradient g^T x with both turned and blockB = 1.
 * The error is at most 1e-5 of |alpha| sum of |terms| + |beta C|, whatever K and the terms' signs are.
 * K <= 2^30; at most 2^23 - 1 tiles of 64 x 64 of C (2^35 elements).
 */
int gemm_e4m3_f32acc(int blockB, int M, int N, int K, float alpha,
                     const uint8_t *A, int lda, const float *SA, int ldsa,
                     const uint8_t *B, int ldb, const float *SB, int ldsb,
                     float beta, float *C, int ldc, hipStream_t stream);

/*
 * gemm_grouped_e4m3_f32acc -- the same for rows in groups, each group with its own right operand:
 *     C[r,:] <- alpha * A[rows[r],:] * B_g^T + beta * C[r,:]   for offsets[g] <= r < offsets[g+1]
 * rows, offsets, groups, R and M as for gemm_grouped_*_f32acc_ex (a row takes its own row's scales along); B and SB hold
 * groups members, strideB and strideSB apart (0: one shared).  groups <= 65535, K <= 2^30, R / 64 + min(groups, R) row tiles.
 */
int gemm_grouped_e4m3_f32acc(int blockB, int groups, int R, int N, int K, float alpha,
                             const uint8_t *A, int M, int lda, const float *SA, int ldsa, const int32_t *rows,
                             const uint8_t *B, int ldb, long long strideB, const float *SB, int ldsb, long long strideSB,
                             const int32_t *offsets, float beta, float *C, int ldc, hipStream_t stream);

/*
 * orthogonalise_* -- an update (momentum, gradient) with its singular values moved towards 1 by Newton-Schulz steps, for
 * batch_count members:
 *     X <- G / |G|_F;  for each step (a, b, c):  X <- a X + (b A + c A A) X,  A = X X^T;   O <- alpha * X
 *   G           : fp32 or bf16, M x N, ldg >= max(1,N), members strideG apart.
 *   coefficients: host memory, a, b, c of each of the `steps` (1 to 100) steps; read during the call.
 *   O           : bf16, M x N, ldo >= max(1,N), members strideO apart (at least a member).
 * M > N is computed from the other side (A = X^T X), which is the same X.  |G|_F is summed in 64 bits; G = 0 gives 0,
 * and an infinity or NaN in G makes its member NaN.  X is kept in fp32, the products are of fp16 copies, each value off by at most
 * 2^-11 of itself (see orthogonalise.hip).  Before it is rounded to bf16 the result is off by at most 5e-3 of its norm with the usual
 * five steps (3.4445, -4.7750, 2.0315), which amplify a rounding, and by at most 1e-3 with eight (1.875, -1.25, 0.375), which do not:
 * whatever G's rank, however unequal or parallel its rows are.  Only where the copies' roundings agree (entries of one size, or no more
 * than a few dozen that count) it can be 2e-2 and 2e-3.
 * fp16's range has to hold s^2, s sqrt(max(M,N)) and |b| s^2 + |c| s^4 for every singular value s on its way (to 1 and a
 * little above with the usual coefficients); what leaves it becomes infinite or NaN.
 * The workspace (orthogonalise_workspace bytes, 16-byte aligned) holds all members; 0 and NULL where one workgroup holds a member
 * (the smaller side up to 64 and the larger up to 1024, or up to 128 and 512).
 * M, N <= 65536; batch_count <= 65535; ceil(M / 64) * ceil(N / 64) * batch_count < 2^23.
 */
int orthogonalise_f32(int M, int N, int steps, const float *coefficients, float alpha,
                      const float *G, int ldg, long long strideG, uint16_t *O, int ldo, long long strideO,
                      int batch_count, void *workspace, long long workspace_bytes, hipStream_t stream);
int orthogonalise_bf16(int M, int N, int steps, const float *coefficients, float alpha,
                       const uint16_t *G, int ldg, long long strideG, uint16_t *O, int ldo, long long strideO,
                       int batch_count, void *workspace, long long workspace_bytes, hipStream_t stream);
long long orthogonalise_workspace(int M, int N, int batch_count);

/* gemm_status_string -- a static, NUL-terminated description of a status code. */
const char *gemm_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MI355GEMM_H */
