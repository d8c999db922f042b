// orthogonalise_api.cpp -- the exported C ABI of the orthogonalised update
// (include/mi355gemm.h): argument checks, quick returns and dispatch.  Argument checks run
// before any HIP call, so they work on a host with no GPU.
#include "api_checks.h"
#include "orthogonalise_internal.h"

namespace {

bool sizes_ok(int M, int N, int batch_count)
{
    return M >= 0 && N >= 0 && M <= mi355gemm::kMaxOrthoSide && N <= mi355gemm::kMaxOrthoSide && batch_count >= 0 && batch_count <= 65535 &&
           (M == 0 || N == 0 || batch_count == 0 || mi355gemm::ortho_fits(M, N, batch_count));
}

int orthogonalise(int M, int N, int steps, const float *coefficients, float alpha, const void *G, int ldg, long long strideG, uint16_t *O,
                  int ldo, long long strideO, int batch_count, void *workspace, long long workspace_bytes, bool bf, hipStream_t stream)
{
    if (!sizes_ok(M, N, batch_count) || steps < 1 || steps > mi355gemm::kMaxOrthoSteps) return GEMM_ERR_SIZE;
    const int N1 = N > 1 ? N : 1;
    if (ldg < N1 || ldo < N1) return GEMM_ERR_LD;
    long long eg, eo;
    if (!extent(M, N, ldg, &eg) || !extent(M, N, ldo, &eo)) return GEMM_ERR_SIZE;
    if (const int rc = batch_extent(batch_count, eg, strideG, false); rc != GEMM_OK) return rc;
    if (const int rc = batch_extent(batch_count, eo, strideO, true); rc != GEMM_OK) return rc;
    if (M == 0 || N == 0 || batch_count == 0) return GEMM_OK;
    if (!coefficients || !G || !O) return GEMM_ERR_NULL;
    if (misaligned(G, bf ? 2 : 4) || misaligned(O, 2)) return GEMM_ERR_ALIGN;
    const size_t need = mi355gemm::ortho_workspace(M, N, batch_count);
    if (workspace_bytes < 0 || (size_t)workspace_bytes < need) return GEMM_ERR_SCRATCH;
    if (need > 0 && !workspace) return GEMM_ERR_NULL;
    if (misaligned(workspace, 16)) return GEMM_ERR_ALIGN;
    mi355gemm::OrthoProblem p;
    p.M = M; p.N = N; p.steps = steps;
    p.coefficients = coefficients;
    p.alpha = alpha;
    p.G = G; p.ldg = ldg; p.strideG = strideG;
    p.O = O; p.ldo = ldo; p.strideO = strideO;
    p.batch = batch_count;
    p.workspace = workspace;
    return launched(mi355gemm::launch_ortho(p, bf, stream));
}

}  // namespace

extern "C" {

long long orthogonalise_workspace(int M, int N, int batch_count)
{
    return sizes_ok(M, N, batch_count) && M > 0 && N > 0 && batch_count > 0 ? (long long)mi355gemm::ortho_workspace(M, N, batch_count) : 0;
}

int orthogonalise_f32(int M, int N, int steps, const float *coefficients, float alpha, const float *G, int ldg, long long strideG,
                      uint16_t *O, int ldo, long long strideO, int batch_count, void *workspace, long long workspace_bytes,
                      hipStream_t stream)
{
    return orthogonalise(M, N, steps, coefficients, alpha, G, ldg, strideG, O, ldo, strideO, batch_count, workspace, workspace_bytes, false,
                         stream);
}

int orthogonalise_bf16(int M, int N, int steps, const float *coefficients, float alpha, const uint16_t *G, int ldg, long long strideG,
                       uint16_t *O, int ldo, long long strideO, int batch_count, void *workspace, long long workspace_bytes,
                       hipStream_t stream)
{
    return orthogonalise(M, N, steps, coefficients, alpha, G, ldg, strideG, O, ldo, strideO, batch_count, workspace, workspace_bytes, true,
                         stream);
}

}  // extern "C"
