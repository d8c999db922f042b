// e4m3_mfma.hip -- products of 8-bit floating-point operands with a scale for each block
// of 128 k, fp32 accumulation and C:
//   C[r,:] = alpha A[rows[r],:] B_g^T + beta C[r,:],  offsets[g] <= r < offsets[g+1]
// for one group (a plain product) or ragged groups of rows.  Both operands are stored
// with k contiguous.  Within a block of 128 k the matrix cores sum exact products in
// fp32; each block's sum p then enters the result by
//   acc <- fma(sa[kb, row] * sb[kb, col], p, acc).
//
// The values go to the matrix cores as fp16, which holds every e4m3 value.  Their own 8-bit op
// has twice the rate, but it adds eight products at a time and keeps 14 bits below the largest of the
// eight: C came out 1.5e-5 of its norm off and single entries 3e-5 of the sum of their terms, where fp32
// sums are held to 1e-5 (and reach 1e-6 here).
#include "e4m3_internal.h"
#include "ragged_dma.h"

namespace mi355gemm {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct E4m3Args {
    int groups, R, N, K;
    float alpha, beta;
    const uint8_t *A;
    int a_rows;
    long long lda;
    const float *SA;
    long long ldsa;
    const int32_t *rows;
    const uint8_t *B;
    long long ldb, strideB;
    const float *SB;
    long long ldsb, strideSB;
    const int32_t *offsets;   // nullptr: one group of R rows
    float *C;
    long long ldc;
    int tiles_m, tiles_n;     // with offsets: tiles_m is what any ascending offsets can need
};

// Sixteen e4m3 values as fp16, exactly (NaN stays NaN), in order.
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
struct Half16 {
    half8 lo, hi;
};
__device__ __forceinline__ Half16 to_f16(const u32x4 &v)
{
    half2v h[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned w = v[i];
        h[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false);
        h[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true);
    }
    return __builtin_bit_cast(Half16, h);
}

// Sixteen bytes from p on, wherever p is; bytes at or past `valid` are zero.  The words
// read all hold one of the valid bytes.
__device__ __forceinline__ u32x4 load16_any(const uint8_t *p, int valid)
{
    if (valid <= 0) return u32x4{0u, 0u, 0u, 0u};
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const unsigned skip = (unsigned)(at & 3);
    const unsigned *w = reinterpret_cast<const unsigned *>(at & ~(uintptr_t)3);
    const int last = ((int)skip + (valid < 16 ? valid : 16) - 1) >> 2;
    unsigned x[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) x[i] = w[i < last ? i : last];
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __builtin_amdgcn_alignbit(x[i + 1], x[i], 8 * skip);
        const int left = valid - 4 * i;   // valid bytes of this word
        if (left < 4) v[i] = left <= 0 ? 0u : v[i] & (0xFFFFFFFFu >> (32 - 8 * left));
    }
    return v;
}

// ---------------------------------------------------------------------------
// The kernel for every shape, stride and alignment: a 64 x 64 tile of four waves of 32 x
// 32, slices of 128 k through registers into a double-buffered LDS.
template <int BLOCKB>
__global__ __launch_bounds__(256) void e4m3_any_kernel(E4m3Args p)
{
    constexpr int BM = 64, BN = 64, BK = 128;
    __shared__ __attribute__((aligned(16))) u32x4 lds[2][(BM + BN) * 8];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    int group = 0, m0, m_end, one, tm, tn;
    if (p.offsets) {
        const int total = count_row_tiles(p.offsets, p.groups, p.R, BM, p.tiles_m);
        if ((long long)blockIdx.x >= (long long)total * p.tiles_n) return;
        tile_coords((int)blockIdx.x, 0, 1, total, p.tiles_n, &one, &tm, &tn);
        const RowTile rt = find_row_tile(p.offsets, p.groups, p.R, BM, tm);
        if (rt.group < 0) return;
        group = rt.group;
        m0 = rt.first;
        m_end = rt.end;
    } else {
        tile_coords((int)blockIdx.x, 0, 1, p.tiles_m, p.tiles_n, &one, &tm, &tn);
        m0 = tm * BM;
        m_end = p.R;
    }
    const int n0 = tn * BN, N = p.N, K = p.K;
    const uint8_t *B = p.B + (long long)group * p.strideB;
    const float *SB = p.SB + (long long)group * p.strideSB;

    auto row_at = [&](int r) { return r >= m_end ? -1 : p.rows ? p.rows[r] : r; };
    // this thread's chunks: rows tid / 8 + 32 i of A (i < 2), then of B
    const uint8_t *row[4];
    const int ch = tid & 7;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 3) + 32 * (i & 1);
        if (i < 2) {
            const int at = row_at(m0 + r);
            row[i] = (unsigned)at < (unsigned)p.a_rows ? p.A + (long long)at * p.lda : nullptr;
        } else {
            row[i] = n0 + r < N ? B + (long long)(n0 + r) * p.ldb : nullptr;
        }
    }
    u32x4 v[4];
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + 16 * ch;
            v[i] = load16_any(row[i] + k, row[i] ? K - k : 0);
        }
    };
    auto store = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (tid >> 3) + 32 * i;   // (rows of B follow those of A)
            lds[buf][r * 8 + (ch ^ swz_a<8>(r))] = v[i];
        }
    };
    const int lr = lane & 31, lk = lane >> 5, wm = wave >> 1, wn = wave & 1;
    const int my_row = m0 + 32 * wm + lr, my_at = row_at(my_row);
    const bool held = (unsigned)my_at < (unsigned)p.a_rows;
    const float *sa = p.SA + (held ? my_at : 0);
    const int col0 = n0 + 32 * wn + 4 * lk;   // register r: column col0 + 8 (r / 4) + r % 4
    f32x16 acc = {};
    const int slices = (K + BK - 1) / BK;
    if (slices > 0) load(0);
    for (int t = 0; t < slices; ++t) {
        const int buf = t & 1;
        store(buf);
        if (t + 1 < slices) load((t + 1) * BK);
        const float fa = sa[(long long)t * p.ldsa];
        const float *sb = SB + (long long)t * p.ldsb;
        float fb[BLOCKB == 1 ? 16 : 1];
        if constexpr (BLOCKB == 1) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int c = col0 + 8 * (r >> 2) + (r & 3);
                fb[r] = sb[c < N ? c : N - 1];
            }
        } else {
            fb[0] = sb[n0 / 128];   // (64 columns lie in one block)
        }
        __syncthreads();   // the buffer written next was last read a step before, which every wave has left
        const u32x4 *la = lds[buf] + (32 * wm + lr) * 8, *lb = lds[buf] + (BM + 32 * wn + lr) * 8;
        f32x16 sum = {};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            // (lane halves take chunks 2 s and 2 s + 1: any order of the k will do that is the same for both operands)
            const int c = (2 * s + lk) ^ swz_a<8>(lr);
            const Half16 a = to_f16(la[c]), b = to_f16(lb[c]);
            sum = mfma16<false>(b.lo, a.lo, sum);
            sum = mfma16<false>(b.hi, a.hi, sum);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[r] = __builtin_fmaf(fa * fb[BLOCKB == 1 ? r : 0], sum[r], acc[r]);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        f32x4_t x = {acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
        if (!held) x = f32x4_t{0.f, 0.f, 0.f, 0.f};   // no such row: zeros, whatever B holds
        if (p.beta != 0.f)
            store_row4<true, true>(p.C, p.ldc, my_row, col0 + 8 * g, x, p.alpha, p.beta, m_end, N);
        else
            store_row4<true, false>(p.C, p.ldc, my_row, col0 + 8 * g, x, p.alpha, p.beta, m_end, N);
    }
}

E4m3Args arguments(const E4m3Problem &q)
{
    E4m3Args a = {};
    a.groups = q.groups; a.R = q.R; a.N = q.N; a.K = q.K;
    a.alpha = q.alpha; a.beta = q.beta;
    a.A = q.A; a.a_rows = q.M; a.lda = q.lda; a.SA = q.SA; a.ldsa = q.ldsa; a.rows = q.rows;
    a.B = q.B; a.ldb = q.ldb; a.strideB = q.strideB; a.SB = q.SB; a.ldsb = q.ldsb; a.strideSB = q.strideSB;
    a.offsets = q.offsets;
    a.C = q.C; a.ldc = q.ldc;
    return a;
}

// Row tiles of bm rows that any split of R rows over the groups can need.
long long row_tiles(const E4m3Problem &q, int bm)
{
    return q.offsets ? q.R / bm + (q.groups < q.R ? q.groups : q.R) : (q.R + (long long)bm - 1) / bm;
}

bool holds(const E4m3Problem &q, int bm, int bn, int threads)
{
    return grid_holds(row_tiles(q, bm) * ((q.N + (long long)bn - 1) / bn), threads);
}

hipError_t launch_any(const E4m3Problem &q, hipStream_t stream)
{
    E4m3Args a = arguments(q);
    a.tiles_m = (int)row_tiles(q, 64);
    a.tiles_n = (q.N + 63) / 64;
    const dim3 grid((unsigned)((long long)a.tiles_m * a.tiles_n));
    if (q.blockB == 1)
        hipLaunchKernelGGL(e4m3_any_kernel<1>, grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(e4m3_any_kernel<128>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

bool e4m3_fits(const E4m3Problem &q)
{
    return holds(q, 64, 64, 256);
}

hipError_t launch_e4m3(const E4m3Problem &q, hipStream_t stream)
{
    return launch_any(q, stream);
}

}  // namespace mi355gemm
