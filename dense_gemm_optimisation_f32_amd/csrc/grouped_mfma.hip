// grouped_mfma.hip -- products of ragged groups of rows, 16-bit inputs, fp32
// accumulation and C:
//   grouped  C[r,:] = alpha A[rows[r],:] op(B_g) + beta C[r,:],  offsets[g] <= r < offsets[g+1]
//   wgrad    C_g = alpha sum_r A[rowsA[r],:]^T B[rowsB[r],:] + beta C_g,  r in group g
// The offsets live on the device, so the host launches as many workgroups as
// any split of R rows over the groups can need, and each workgroup finds its
// group and tile from the offsets; surplus workgroups return at once.
#include "routed_internal.h"
#include "stage16.h"
#include "tile_order.h"

#include <limits.h>

namespace mi355gemm {
namespace {

// Group g's rows, clamped to [0, R] so that no offset leads outside C.
__device__ __forceinline__ void group_rows(const int32_t *offsets, int g, int R, int *lo, int *hi)
{
    const int a = offsets[g], b = offsets[g + 1];
    *lo = a < 0 ? 0 : a > R ? R : a;
    *hi = b < *lo ? *lo : b > R ? R : b;
}

// The row tiles (of BM rows, per group) of all groups, counted in order:
// `total` of them, and of tile `want` its group, first row and the group's end.
// Every wave does this by itself, 64 groups at a time, one per lane.
struct RowTile {
    int group, first, end;
};
__device__ __forceinline__ int count_row_tiles(const int32_t *offsets, int groups, int R, int bm)
{
    const int lane = threadIdx.x & 63;
    int total = 0;
    for (int g0 = 0; g0 < groups; g0 += 64) {
        int n = 0;
        if (g0 + lane < groups) {
            int lo, hi;
            group_rows(offsets, g0 + lane, R, &lo, &hi);
            n = (hi - lo + bm - 1) / bm;
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
        total += n;
    }
    return __builtin_amdgcn_readfirstlane(total);
}
__device__ __forceinline__ RowTile find_row_tile(const int32_t *offsets, int groups, int R, int bm, int want)
{
    const int lane = threadIdx.x & 63;
    for (int g0 = 0; g0 < groups; g0 += 64) {
        int lo = 0, hi = 0, n = 0;
        if (g0 + lane < groups) {
            group_rows(offsets, g0 + lane, R, &lo, &hi);
            n = (hi - lo + bm - 1) / bm;
        }
        int s = n;   // inclusive sum
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(s, d);
            if (lane >= d) s += o;
        }
        const uint64_t hit = __ballot(want >= s - n && want < s);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            const int first = __shfl(lo + (want - (s - n)) * bm, at);
            return {__builtin_amdgcn_readfirstlane(g0 + at), __builtin_amdgcn_readfirstlane(first),
                    __builtin_amdgcn_readfirstlane(__shfl(hi, at))};
        }
        want -= __builtin_amdgcn_readfirstlane(__shfl(s, 63));
    }
    return {-1, 0, 0};
}

// Eight consecutive values from column c of a row of `cols` (nullptr: zeros),
// wherever the row starts; columns at or past the end read as zero.
__device__ __forceinline__ u32x4 load8_row(const uint16_t *row, long long c, long long cols)
{
    if (row == nullptr || c >= cols) return u32x4{0u, 0u, 0u, 0u};
    const uint16_t *p = row + c;
    if (c + 8 > cols) return load8_masked(p, (int)(cols - c));
    return (reinterpret_cast<uintptr_t>(p) & 3) == 0 ? *reinterpret_cast<const u32x4_g *>(p) : load8_words(p);
}

struct RaggedArgs {
    int groups, R, M, N, K;   // grouped: K columns of A; wgrad: M columns of A
    float alpha, beta;
    const uint16_t *A;
    int a_rows;
    long long lda;
    const int32_t *rowsA;
    const uint16_t *B;
    int b_rows;               // wgrad
    long long ldb, strideB;
    const int32_t *rowsB;     // wgrad
    const int32_t *offsets;
    float *C;
    long long ldc, strideC;
    int tiles_m, tiles_n;
    bool product;             // false: C is only scaled
};

// ---------------------------------------------------------------------------
// The kernel for every shape, stride and alignment: 64x64 tiles of four waves,
// operand slices of 64 k read into registers and written to a double-buffered
// LDS (the register-staged scheme of hgemm_mfma.hip with rows addressed one by
// one).  WG = false: grouped (TB: B stored N x K per group); WG = true: wgrad,
// where both operands are stored with the k (the group's rows) outermost.
template <bool BF, bool WG, bool TB>
__global__ __launch_bounds__(256) void ragged_any_kernel(RaggedArgs p)
{
    using Cfg = HgCfg<64, 64>;
    constexpr int BM = Cfg::BM, BN = Cfg::BN, BK = Cfg::BK, NT = Cfg::NT;
    using TileA = HgTile<!WG, BM, BK, NT>;
    using TileB = HgTile<!WG && TB, BN, BK, NT>;
    constexpr int BUF_HALVES = TileA::HALVES + TileB::HALVES;
    __shared__ __attribute__((aligned(16))) uint16_t lds[2 * BUF_HALVES];

    const int tid = threadIdx.x;
    int group, m0, m_end, K, n0, k_lo = 0;
    if constexpr (WG) {
        int tm, tn;
        tile_coords(blockIdx.x, blockIdx.z, gridDim.z, p.tiles_m, p.tiles_n, &group, &tm, &tn);
        m0 = tm * BM;
        m_end = p.M;
        n0 = tn * BN;
        K = 0;
        if (p.product) {
            int hi;
            group_rows(p.offsets, group, p.R, &k_lo, &hi);
            K = hi - k_lo;
        }
    } else {
        const int total = count_row_tiles(p.offsets, p.groups, p.R, BM);
        if ((long long)blockIdx.x >= (long long)total * p.tiles_n) return;
        int one, tm, tn;
        // the XCD-aware order over the tiles that exist
        tile_coords((int)blockIdx.x, 0, 1, total, p.tiles_n, &one, &tm, &tn);
        const RowTile rt = find_row_tile(p.offsets, p.groups, p.R, BM, tm);
        if (rt.group < 0) return;
        group = rt.group;
        m0 = rt.first;
        m_end = rt.end;
        n0 = tn * BN;
        K = p.product ? p.K : 0;
    }
    const int N = p.N;
    const uint16_t *B = WG ? p.B : p.B + (long long)group * p.strideB;
    float *C = WG ? p.C + (long long)group * p.strideC : p.C;
    const long long lda = p.lda, ldb = p.ldb, ldc = p.ldc;

    u32x4 ra[TileA::LOADS], rb[TileB::LOADS];
    auto row_of = [](const uint16_t *X, long long ld, const int32_t *rows, int r, int end, int x_rows) -> const uint16_t * {
        if (r >= end) return nullptr;
        const int at = rows ? rows[r] : r;
        return at < 0 || at >= x_rows ? nullptr : X + (long long)at * ld;
    };
    // grouped: the rows of A this thread loads are fixed for the whole K loop
    const uint16_t *arow[TileA::LOADS];
    if constexpr (!WG) {
#pragma unroll
        for (int i = 0; i < TileA::LOADS; ++i)
            arow[i] = row_of(p.A, lda, p.rowsA, m0 + (i * NT + tid) / TileA::CPR, m_end, p.a_rows);
    }
    auto load_tiles = [&](int k0) {
#pragma unroll
        for (int i = 0; i < TileA::LOADS; ++i) {
            const int id = i * NT + tid;
            const int r = id / TileA::CPR, c = (id % TileA::CPR) * 8;
            if constexpr (WG)
                ra[i] = load8_row(row_of(p.A, lda, p.rowsA, k_lo + k0 + r, k_lo + K, p.a_rows), m0 + c, p.M);
            else
                ra[i] = load8_row(arow[i], k0 + c, K);
        }
#pragma unroll
        for (int i = 0; i < TileB::LOADS; ++i) {
            const int id = i * NT + tid;
            const int r = id / TileB::CPR, c = (id % TileB::CPR) * 8;
            if constexpr (WG)
                rb[i] = load8_row(row_of(p.B, ldb, p.rowsB, k_lo + k0 + r, k_lo + K, p.b_rows), n0 + c, N);
            else if constexpr (TB)
                rb[i] = load8_row(n0 + r < N ? B + (long long)(n0 + r) * ldb : nullptr, k0 + c, K);
            else
                rb[i] = load8_row(k0 + r < K ? B + (long long)(k0 + r) * ldb : nullptr, n0 + c, N);
        }
    };
    auto store_one = [&](auto tile, uint16_t *dst, int i, const u32x4 &v) {
        using T = decltype(tile);
        const int id = i * NT + tid;
        const int r = id / T::CPR, c = id % T::CPR;
        if constexpr (T::KCONTIG)
            *reinterpret_cast<u32x4 *>(dst + r * BK + 8 * swz(r, c)) = v;
        else
            *reinterpret_cast<u32x4 *>(dst + r * T::PITCH + 8 * c) = v;
    };
    auto store_tiles = [&](int buf) {
        uint16_t *la = lds + buf * BUF_HALVES;
        uint16_t *lb = la + TileA::HALVES;
#pragma unroll
        for (int i = 0; i < TileA::LOADS; ++i) store_one(TileA{}, la, i, ra[i]);
#pragma unroll
        for (int i = 0; i < TileB::LOADS; ++i) store_one(TileB{}, lb, i, rb[i]);
    };
    const int wave = tid >> 6, lane = tid & 63;
    const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;
    const int lr = lane & 31, lk = lane >> 5;
    const int q = lane >> 4, j = lane & 15;
    const int tr_row = 8 * (q >> 1) + (j >> 2);
    const int tr_col = 16 * (q & 1) + 4 * (j & 3);
    f32x16 acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.f;
    auto read_frag = [&](auto tile, const uint16_t *base, int first, int s) -> half8 {
        using T = decltype(tile);
        if constexpr (T::KCONTIG) {
            const int row = first + lr;
            return *reinterpret_cast<const half8 *>(base + row * BK + 8 * swz(row, 2 * s + lk));
        } else {
            const uint16_t *at = base + (16 * s + tr_row) * T::PITCH + first + tr_col;
            const short4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(at));
            const short4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(at + 4 * T::PITCH));
            const short4v both[2] = {lo, hi};
            return __builtin_bit_cast(half8, both);
        }
    };
    const int nk = (K + BK - 1) / BK;
    if (nk > 0) load_tiles(0);
    for (int t = 0; t < nk; ++t) {
        const int buf = t & 1;
        store_tiles(buf);
        if (t + 1 < nk) load_tiles((t + 1) * BK);
        // one barrier a step: the buffer written next was last read in the step
        // before this one, which every wave has left when it passes here
        __syncthreads();
        const uint16_t *la = lds + buf * BUF_HALVES;
        const uint16_t *lb = la + TileA::HALVES;
#pragma unroll
        for (int s = 0; s < BK / 16; ++s)
            acc = mfma16<BF>(read_frag(TileB{}, lb, wn * Cfg::TN, s), read_frag(TileA{}, la, wm * Cfg::TM, s), acc);
    }
    const long long row = m0 + wm * Cfg::TM + lr;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const long long col = n0 + wn * Cfg::TN + 8 * g + 4 * lk;
        const f32x4_t v = {acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
        if (p.beta != 0.f)
            store_row4<true, true>(C, ldc, row, col, v, p.alpha, p.beta, m_end, N);
        else
            store_row4<true, false>(C, ldc, row, col, v, p.alpha, p.beta, m_end, N);
    }
}

RaggedArgs grouped_args(const GroupedProblem &q)
{
    RaggedArgs a = {};
    a.groups = q.groups; a.R = q.R; a.N = q.N; a.K = q.K;
    a.alpha = q.alpha; a.beta = q.beta;
    a.A = q.A; a.a_rows = q.M; a.lda = q.lda; a.rowsA = q.rows;
    a.B = q.B; a.ldb = q.ldb; a.strideB = q.strideB;
    a.offsets = q.offsets;
    a.C = q.C; a.ldc = q.ldc;
    a.product = q.K > 0;
    return a;
}
RaggedArgs wgrad_args(const WgradProblem &q)
{
    RaggedArgs a = {};
    a.groups = q.groups; a.R = q.R; a.M = q.M; a.N = q.N;
    a.alpha = q.alpha; a.beta = q.beta;
    a.A = q.A; a.a_rows = q.a_rows; a.lda = q.lda; a.rowsA = q.rowsA;
    a.B = q.B; a.b_rows = q.b_rows; a.ldb = q.ldb; a.rowsB = q.rowsB;
    a.offsets = q.offsets;
    a.C = q.C; a.ldc = q.ldc; a.strideC = q.strideC;
    a.product = q.R > 0;
    return a;
}

// Row tiles of bm rows that any split of R rows over the groups can need: one
// per bm rows, and one part-filled one per group that holds rows.
long long most_row_tiles(int R, int groups, int bm)
{
    return R / bm + (groups < R ? groups : R);
}

}  // namespace

hipError_t launch_grouped(const GroupedProblem &q, bool bf, hipStream_t stream)
{
    RaggedArgs a = grouped_args(q);
    a.tiles_n = (q.N + 63) / 64;
    const long long tiles = most_row_tiles(q.R, q.groups, 64) * a.tiles_n;
    if (tiles > INT_MAX / 256) return hipErrorInvalidValue;   // a grid holds fewer than 2^32 threads
    const dim3 grid((unsigned)tiles), block(256);
    if (bf && q.transB)
        hipLaunchKernelGGL((ragged_any_kernel<true, false, true>), grid, block, 0, stream, a);
    else if (bf)
        hipLaunchKernelGGL((ragged_any_kernel<true, false, false>), grid, block, 0, stream, a);
    else if (q.transB)
        hipLaunchKernelGGL((ragged_any_kernel<false, false, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((ragged_any_kernel<false, false, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_wgrad(const WgradProblem &q, bool bf, hipStream_t stream)
{
    RaggedArgs a = wgrad_args(q);
    a.tiles_m = (q.M + 63) / 64;
    a.tiles_n = (q.N + 63) / 64;
    if ((long long)a.tiles_m * a.tiles_n > INT_MAX / 256 || q.groups > 65535) return hipErrorInvalidValue;
    const dim3 grid(a.tiles_m * a.tiles_n, 1, q.groups), block(256);
    if (bf)
        hipLaunchKernelGGL((ragged_any_kernel<true, true, false>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((ragged_any_kernel<false, true, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace mi355gemm
