// lora_mfma.hip -- a shared projection with a low-rank adapter per row:
//   C[i,:] = alpha (A[i,:] op(B) + scales[a] (A[i,:] LA_a^T) LB_a^T) + beta C[i,:],  a = ids[i]
#include "routed_internal.h"
#include "gemm_internal.h"
#include "stage16.h"

namespace mi355gemm {
namespace {

typedef float f32x4v __attribute__((ext_vector_type(4)));

template <bool BF>
__device__ __forceinline__ f32x4v mfma16x16(half8 a, half8 b, f32x4v c)
{
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

template <bool BF>
__device__ __forceinline__ float widen16(uint16_t h)
{
    if constexpr (BF)
        return __builtin_bit_cast(float, (unsigned)h << 16);
    else
        return (float)__builtin_bit_cast(_Float16, h);
}

// Eight values at p of which the first `valid` may be read; the others are zero.
__device__ __forceinline__ half8 load8_any(const uint16_t *p, int valid)
{
    u32x4 v;
    if (valid <= 0)
        v = u32x4{0u, 0u, 0u, 0u};
    else if (valid < 8)
        v = load8_masked(p, valid);
    else
        v = (reinterpret_cast<uintptr_t>(p) & 3) == 0 ? *reinterpret_cast<const u32x4_g *>(p) : load8_words(p);
    return __builtin_bit_cast(half8, v);
}

__device__ __forceinline__ int adapter_of(const LoraProblem &p, int row)
{
    const int a = row < p.M ? p.ids[row] : -1;
    return a >= 0 && a < p.adapters ? a : -1;
}
__device__ __forceinline__ int rank_of(const LoraProblem &p, int a)
{
    const int r = p.ranks ? p.ranks[a] : p.rank;
    return r < 0 ? 0 : r > p.rank ? p.rank : r;
}

// The narrow product t[i,:] = A[i,:] LA_a^T in 32 bits.  Block (b, j): the
// 16 rows of row block b that use its j-th distinct adapter; surplus blocks
// return.  The four waves share K and add up in wave order.
constexpr int kTPitch = kMaxRank;   // floats per row of t

template <bool BF, int NR>
__global__ __launch_bounds__(256) void lora_narrow_kernel(LoraProblem p)
{
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 15, lq = lane >> 4;
    const int row0 = blockIdx.x * 16;
    const int mine = adapter_of(p, row0 + li);
    // lanes whose adapter no earlier row of the block has
    bool first = lane < 16 && mine >= 0;
    for (int i = 0; i < 15; ++i) {
        const int o = __shfl(mine, i);
        if (i < lane && o == mine) first = false;
    }
    uint64_t firsts = __ballot(first);
    for (int j = 0; j < (int)blockIdx.y && firsts; ++j) firsts &= firsts - 1;
    if (!firsts) return;
    const int a = __builtin_amdgcn_readfirstlane(__shfl(mine, __builtin_ctzll(firsts)));
    const int ra = rank_of(p, a);
    const uint16_t *la = p.LA + (long long)a * p.strideLA;
    const int row = row0 + li;
    const uint16_t *x = row < p.M ? p.A + (long long)row * p.lda : nullptr;
    f32x4v acc[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[n] = f32x4v{0.f, 0.f, 0.f, 0.f};
    for (int k = 32 * wave; k < p.K; k += 128) {
        const int kq = k + 8 * lq;
        const half8 xb = x ? load8_any(x + kq, p.K - kq) : half8{};
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int j = 16 * n + li;
            const half8 f = load8_any(la + (long long)j * p.ldla + kq, j < ra ? p.K - kq : 0);
            acc[n] = mfma16x16<BF>(f, xb, acc[n]);
        }
    }
    __shared__ f32x4v part[4][NR][64];
#pragma unroll
    for (int n = 0; n < NR; ++n) part[wave][n][lane] = acc[n];
    __syncthreads();
    if (mine != a || row >= p.M) return;
    for (int n = wave; n < NR; n += 4) {
        const f32x4v s = (part[0][n][lane] + part[1][n][lane]) + (part[2][n][lane] + part[3][n][lane]);
        *reinterpret_cast<f32x4v *>(p.t + (long long)row * kTPitch + 16 * n + 4 * lq) = s;
    }
}

// C[i,n] += alpha * scale * sum_j t[i,j] LB_a[n,j].
template <bool BF>
__global__ __launch_bounds__(256) void lora_widen_kernel(LoraProblem p)
{
    const int row = blockIdx.y;
    const int a = adapter_of(p, row);
    if (a < 0) return;
    const int ra = rank_of(p, a);
    const float f = p.alpha * (p.scales ? p.scales[a] : 1.f);
    __shared__ float t[kMaxRank];
    if ((int)threadIdx.x < ra) t[threadIdx.x] = p.t[(long long)row * kTPitch + threadIdx.x];
    __syncthreads();
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= p.N) return;
    const uint16_t *b = p.LB + (long long)a * p.strideLB + (long long)n * p.ldlb;
    float s = 0.f;
    for (int j = 0; j < ra; ++j) s = __builtin_fmaf(t[j], widen16<BF>(b[j]), s);
    float *c = p.C + (long long)row * p.ldc + n;
    *c = __builtin_fmaf(f, s, *c);
}

template <bool BF>
hipError_t lora(const LoraProblem &p, hipStream_t stream)
{
    const dim3 ngrid((p.M + 15) / 16, p.adapters < 16 ? p.adapters : 16), block(256);
    if (p.K > 0 && p.adapters > 0) {
        if (p.rank <= 16)
            hipLaunchKernelGGL((lora_narrow_kernel<BF, 1>), ngrid, block, 0, stream, p);
        else if (p.rank <= 32)
            hipLaunchKernelGGL((lora_narrow_kernel<BF, 2>), ngrid, block, 0, stream, p);
        else if (p.rank <= 64)
            hipLaunchKernelGGL((lora_narrow_kernel<BF, 4>), ngrid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((lora_narrow_kernel<BF, 8>), ngrid, block, 0, stream, p);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    GemmProblem g = {};
    g.transB = p.transB;
    g.M = p.M; g.N = p.N; g.K = p.K; g.batch = 1;
    g.alpha = p.alpha; g.beta = p.beta;
    g.A = p.A; g.lda = p.lda;
    g.B = p.B; g.ldb = p.ldb;
    g.C = p.C; g.ldc = p.ldc;
    const hipError_t e = p.K == 0 ? launch_scale_c(g, stream) : BF ? launch_bgemm(g, stream) : launch_hgemm(g, stream);
    if (e != hipSuccess || p.K == 0 || p.adapters == 0) return e;
    for (int r0 = 0; r0 < p.M; r0 += 65535) {
        LoraProblem q = p;
        q.M = p.M - r0 < 65535 ? p.M - r0 : 65535;
        q.ids += r0;
        q.C += (long long)r0 * p.ldc;
        q.t += (long long)r0 * kTPitch;
        hipLaunchKernelGGL(lora_widen_kernel<BF>, dim3((p.N + 255) / 256, q.M), block, 0, stream, q);
    }
    return hipGetLastError();
}

}  // namespace

size_t lora_workspace(int M, int, int, int)
{
    return (size_t)M * kTPitch * sizeof(float);
}

hipError_t launch_lora(const LoraProblem &p, bool bf, hipStream_t stream)
{
    return bf ? lora<true>(p, stream) : lora<false>(p, stream);
}

}  // namespace mi355gemm
