// orthogonalise.hip -- an update with all its singular values moved to near 1 by matrix
// products alone (Newton-Schulz steps):
//   X <- G / |G|_F;  steps times:  X <- a X + (b A + c A A) X,  A = X X^T
// in which every singular value goes s <- a s + b s^3 + c s^5 and the singular vectors stay.
// X is the smaller way round (m x n, m <= n); a tall G is turned when it is read and turned
// back when the result is written.
//
// What is rounded where:
//   * X itself stays in fp32.  A rounding of X is noise in all directions, and a direction that G
//     hardly has grows by a factor a in every step (3.4445^5 = 485): rounded to 16 bits in
//     each step, a G of low rank came out 4e-2 off.
//   * The products' operands are fp16 copies.  There an error only multiplies X (from the left,
//     through A), and stays as small as it is.  The copies are scaled by powers of two into fp16's range.
//   * The diagonals of A and of B = b A + c A A, which come to be much larger than the rest, are
//     kept apart in fp32, and the fp16 copies hold zeros there: with A = D + O,
//       A A = D D + D O + O D + O O,   B X = diag(B) X + (B - diag(B)) X.
// Together the result is 4e-4 to 9e-4 off before it is rounded to bf16 (which costs 1.7e-3), 3e-3
// for a G of rank one.
#include "orthogonalise_internal.h"
#include "routed_internal.h"
#include "stage16.h"
#include "wave.h"

#include <cmath>

namespace mi355gemm {
namespace {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));

constexpr int kNormBlocks = 64;      // workgroups (and partial sums) of a matrix's norm
constexpr float kOffScale = 1024.f;  // of A's fp16 copy: entries are at most the largest singular value squared

// One matrix's part of the workspace.  Rows and columns are filled up to multiples of 64 with zeros,
// which the products keep.
struct Layout {
    long long m, n;                  // padded
    long long x, x16, xt[2], a16, b16, da, db, norm, bytes;   // byte offsets
};
long long up64(long long v) { return (v + 63) / 64 * 64; }
Layout layout(int M, int N)
{
    Layout l;
    l.m = up64(M < N ? M : N);
    l.n = up64(M < N ? N : M);
    long long at = 0;
    auto take = [&](long long bytes) {
        const long long here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    l.x = take(l.m * l.n * 4);
    l.x16 = take(l.m * l.n * 2);
    l.xt[0] = take(l.m * l.n * 2);
    l.xt[1] = take(l.m * l.n * 2);
    l.a16 = take(l.m * l.m * 2);
    l.b16 = take(l.m * l.m * 2);
    l.da = take(l.m * 4);
    l.db = take(l.m * 4);
    l.norm = take(kNormBlocks * 8);
    l.bytes = at;
    return l;
}

struct OrthoArgs {
    int M, N;                        // of G and O
    int m, n;                        // of X, padded
    bool tall, last;
    float a, b, c;                   // this step's coefficients
    float x_scale;                   // x16 and x hold x_scale * X
    float b_scale;                   // b16 holds b_scale * (B - diag(B))
    float alpha;
    const void *G;
    long long ldg, strideG;
    uint16_t *O;
    long long ldo, strideO;
    long long ws_stride;             // bytes per matrix
    float *x;
    _Float16 *x16, *xt_in, *xt_out, *a16, *b16;
    float *da, *db;
    double *norm;
};

template <class T>
__device__ __forceinline__ T *of_member(T *p, long long stride_bytes, int z)
{
    return reinterpret_cast<T *>(reinterpret_cast<uintptr_t>(p) + (uintptr_t)(z * stride_bytes));
}

template <bool BF>
__device__ __forceinline__ float g_at(const OrthoArgs &p, int z, long long r, long long c)
{
    const long long at = z * p.strideG + r * p.ldg + c;
    if constexpr (BF)
        return __builtin_bit_cast(float, (unsigned)reinterpret_cast<const uint16_t *>(p.G)[at] << 16);
    else
        return reinterpret_cast<const float *>(p.G)[at];
}

// Sums of squares in 64 bits: neither large nor small entries leave the range.
template <bool BF>
__global__ __launch_bounds__(256) void norm_kernel(OrthoArgs p)
{
    __shared__ double part[4];
    const int z = blockIdx.z, tid = threadIdx.x;
    double sum = 0;
    for (int r = blockIdx.x; r < p.M; r += kNormBlocks)
        for (int c = tid; c < p.N; c += 256) {
            const double v = g_at<BF>(p, z, r, c);
            sum = __builtin_fma(v, v, sum);
        }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) part[tid >> 6] = sum;
    __syncthreads();
    if (tid == 0) of_member(p.norm, p.ws_stride, z)[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X and its copies from G: a 64 x 64 tile of X per workgroup.
template <bool BF>
__global__ __launch_bounds__(256) void start_kernel(OrthoArgs p)
{
    __shared__ float tile[64][65];
    const int z = blockIdx.z, tid = threadIdx.x;
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // of X
    const double *norm = of_member(p.norm, p.ws_stride, z);
    double sum = 0;
    for (int i = 0; i < kNormBlocks; ++i) sum += norm[i];
    // zeros stay zeros; an infinity or NaN makes everything NaN
    const double f = sum == 0 ? 0 : sum < __builtin_inf() ? p.x_scale / __builtin_sqrt(sum) : __builtin_nan("");
    for (int e = tid; e < 64 * 64; e += 256) {
        // (consecutive threads along G's rows)
        const int i = p.tall ? e % 64 : e / 64, j = p.tall ? e / 64 : e % 64;
        const int gr = p.tall ? c0 + j : r0 + i, gc = p.tall ? r0 + i : c0 + j;
        tile[i][j] = gr < p.M && gc < p.N ? (float)(g_at<BF>(p, z, gr, gc) * f) : 0.f;
    }
    __syncthreads();
    float *x = of_member(p.x, p.ws_stride, z);
    _Float16 *x16 = of_member(p.x16, p.ws_stride, z), *xt = of_member(p.xt_out, p.ws_stride, z);
    for (int e = tid; e < 64 * 64; e += 256) {
        const int i = e / 64, j = e % 64;
        x[(long long)(r0 + i) * p.n + c0 + j] = tile[i][j];
        x16[(long long)(r0 + i) * p.n + c0 + j] = (_Float16)tile[i][j];
        xt[(long long)(c0 + i) * p.m + r0 + j] = (_Float16)tile[j][i];
    }
}

enum Product { kGram, kSquare, kApply };

// The three products of a step, each P Q^T of fp16 rows with k contiguous and whole slices of 64:
//   kGram    A = X X^T            P = Q = X
//   kSquare  B = b A + c A A      P = Q = A - diag(A)
//   kApply   X <- a X + B X       P = B - diag(B), Q = X^T
// 64 x 64 tiles of four waves of 32 x 32.
template <Product KIND>
__global__ __launch_bounds__(256) void product_kernel(OrthoArgs p)
{
    __shared__ __attribute__((aligned(16))) u32x4 lds[2][128 * 8];
    const int z = blockIdx.z, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
    const _Float16 *P = of_member(KIND == kGram ? p.x16 : KIND == kSquare ? p.a16 : p.b16, p.ws_stride, z);
    const _Float16 *Q = of_member(KIND == kGram ? p.x16 : KIND == kSquare ? p.a16 : p.xt_in, p.ws_stride, z);
    const int K = KIND == kGram ? p.n : p.m;
    const long long ld = K;
    const _Float16 *row[4];
    const int ch = tid & 7;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 3) + 32 * (i & 1);
        row[i] = (i < 2 ? P + (m0 + r) * ld : Q + (n0 + r) * ld) + 8 * ch;
    }
    u32x4 v[4];
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const u32x4 *>(row[i] + k0);
    };
    const int lr = lane & 31, lk = lane >> 5, wm = wave >> 1, wn = wave & 1;
    f32x16 acc = {};
    load(0);
    for (int t = 0; t < K / 64; ++t) {
        const int buf = t & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (tid >> 3) + 32 * i;
            lds[buf][r * 8 + (ch ^ swz_a<8>(r))] = v[i];
        }
        if (t + 1 < K / 64) load((t + 1) * 64);
        __syncthreads();
        const u32x4 *la = lds[buf] + (32 * wm + lr) * 8, *lb = lds[buf] + (64 + 32 * wn + lr) * 8;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int c = (2 * s + lk) ^ swz_a<8>(lr);
            acc = mfma16<false>(__builtin_bit_cast(half8, lb[c]), __builtin_bit_cast(half8, la[c]), acc);
        }
    }
    const int r = m0 + 32 * wm + lr;
    float *da = of_member(p.da, p.ws_stride, z), *db = of_member(p.db, p.ws_stride, z);
    _Float16 *a16 = of_member(p.a16, p.ws_stride, z), *b16 = of_member(p.b16, p.ws_stride, z);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int c = n0 + 32 * wn + 8 * g + 4 * lk;
        const f32x4_t s = {acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
        if constexpr (KIND == kGram) {
            const float back = 1.f / (p.x_scale * p.x_scale);
            half4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = s[e] * back;
                if (r == c + e) da[r] = v;
                h[e] = r == c + e ? (_Float16)0.f : (_Float16)(v * kOffScale);
            }
            *reinterpret_cast<half4 *>(a16 + (long long)r * p.m + c) = h;
        } else if constexpr (KIND == kSquare) {
            const half4 o = *reinterpret_cast<const half4 *>(a16 + (long long)r * p.m + c);
            half4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float off = (float)o[e] * (1.f / kOffScale), sq = s[e] * (1.f / (kOffScale * kOffScale));
                if (r == c + e) db[r] = p.b * da[r] + p.c * (da[r] * da[r] + sq);
                const float v = p.b * off + p.c * ((da[r] + da[c + e]) * off + sq);
                h[e] = r == c + e ? (_Float16)0.f : (_Float16)(v * p.b_scale);
            }
            *reinterpret_cast<half4 *>(b16 + (long long)r * p.m + c) = h;
        } else {
            float *x = of_member(p.x, p.ws_stride, z) + (long long)r * p.n + c;
            const f32x4_t old = *reinterpret_cast<const f32x4_t *>(x);
            const float f = p.a + db[r], back = 1.f / p.b_scale;
            f32x4_t v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f, old[e], back * s[e]);
            if (p.last) {
                const float out = p.alpha / p.x_scale;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row_o = p.tall ? c + e : r, col_o = p.tall ? r : c + e;
                    if (row_o < p.M && col_o < p.N)
                        p.O[z * p.strideO + (long long)row_o * p.ldo + col_o] = __builtin_bit_cast(uint16_t, (__bf16)(v[e] * out));
                }
            } else {
                *reinterpret_cast<f32x4_t *>(x) = v;
                half4 h;
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = (_Float16)v[e];
                *reinterpret_cast<half4 *>(of_member(p.x16, p.ws_stride, z) + (long long)r * p.n + c) = h;
                _Float16 *xt = of_member(p.xt_out, p.ws_stride, z);
#pragma unroll
                for (int e = 0; e < 4; ++e) xt[(long long)(c + e) * p.m + r] = h[e];
            }
        }
    }
}

template <Product KIND>
hipError_t launch_product(const OrthoArgs &a, int batch, hipStream_t stream)
{
    const int cols = KIND == kApply ? a.n : a.m;
    hipLaunchKernelGGL(product_kernel<KIND>, dim3(cols / 64, a.m / 64, batch), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <bool BF>
hipError_t launch(const OrthoProblem &q, hipStream_t stream)
{
    const Layout l = layout(q.M, q.N);
    OrthoArgs a = {};
    a.M = q.M; a.N = q.N;
    a.m = (int)l.m; a.n = (int)l.n;
    a.tall = q.M > q.N;
    // X's rows end up with a norm near 1 over n entries: entries near 2^0 after this
    a.x_scale = std::exp2(std::floor(0.5f * std::log2((float)(q.M > q.N ? q.M : q.N))));
    a.alpha = q.alpha;
    a.G = q.G; a.ldg = q.ldg; a.strideG = q.strideG;
    a.O = q.O; a.ldo = q.ldo; a.strideO = q.strideO;
    a.ws_stride = l.bytes;
    char *w = static_cast<char *>(q.workspace);
    a.x = reinterpret_cast<float *>(w + l.x);
    a.x16 = reinterpret_cast<_Float16 *>(w + l.x16);
    a.a16 = reinterpret_cast<_Float16 *>(w + l.a16);
    a.b16 = reinterpret_cast<_Float16 *>(w + l.b16);
    a.da = reinterpret_cast<float *>(w + l.da);
    a.db = reinterpret_cast<float *>(w + l.db);
    a.norm = reinterpret_cast<double *>(w + l.norm);
    _Float16 *xt[2] = {reinterpret_cast<_Float16 *>(w + l.xt[0]), reinterpret_cast<_Float16 *>(w + l.xt[1])};
    hipLaunchKernelGGL(norm_kernel<BF>, dim3(kNormBlocks, 1, q.batch), dim3(256), 0, stream, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    a.xt_out = xt[0];
    hipLaunchKernelGGL(start_kernel<BF>, dim3(a.n / 64, a.m / 64, q.batch), dim3(256), 0, stream, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    for (int s = 0; s < q.steps; ++s) {
        a.a = q.coefficients[3 * s];
        a.b = q.coefficients[3 * s + 1];
        a.c = q.coefficients[3 * s + 2];
        // entries of B for entries of A up to 4, below 2^15
        const float most = 4.f * std::fabs(a.b) + 16.f * std::fabs(a.c);
        a.b_scale = most > 0 && most < 32768.f ? std::exp2(std::floor(std::log2(32768.f / most))) : 1.f;
        if (a.b_scale > 1024.f) a.b_scale = 1024.f;
        a.xt_in = xt[s & 1];
        a.xt_out = xt[(s & 1) ^ 1];
        a.last = s + 1 == q.steps;
        if (hipError_t e = launch_product<kGram>(a, q.batch, stream); e != hipSuccess) return e;
        if (hipError_t e = launch_product<kSquare>(a, q.batch, stream); e != hipSuccess) return e;
        if (hipError_t e = launch_product<kApply>(a, q.batch, stream); e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

bool ortho_fits(int M, int N, int batch)
{
    const Layout l = layout(M, N);
    return grid_holds(l.m / 64 * (l.n / 64) * batch, 256);
}

size_t ortho_workspace(int M, int N, int batch)
{
    return (size_t)layout(M, N).bytes * batch;
}

hipError_t launch_ortho(const OrthoProblem &p, bool bf, hipStream_t stream)
{
    return bf ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace mi355gemm
