// grouped_mfma.hip -- products of ragged groups of rows, 16-bit inputs, fp32
// accumulation and C:
//   grouped  C[r,:] = alpha A[rows[r],:] op(B_g) + beta C[r,:],  offsets[g] <= r < offsets[g+1]
//   wgrad    C_g = alpha sum_r A[rowsA[r],:]^T B[rowsB[r],:] + beta C_g,  r in group g
// The offsets live on the device, so the host launches as many workgroups as
// any split of R rows over the groups can need, and each workgroup finds its
// group and tile from the offsets; surplus workgroups return at once.
#include "routed_internal.h"
#include "ragged_dma.h"

#include <limits.h>

namespace mi355gemm {
namespace {

// Eight consecutive values from column c of a row, wherever the row starts, in two
// halves: the loads (words), whose results nothing touches while other loads are on
// their way, and the values (value8).  The words are the five dwords from the one that
// holds the first value on; past the last that holds one of the row's `cols` columns,
// that one again, so no load leaves the words the row occupies.  whole (the same in all
// lanes): no chunk of this slice ends before its eighth column, so four of the dwords are
// one load.  row == nullptr: zeros.
struct Words {
    unsigned w[5], shift;
};
__device__ __forceinline__ void words(const uint16_t *row, long long c, long long cols, bool whole, Words *out)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(row + c);
    if (whole) {
        const unsigned odd = row ? (unsigned)(p & 2) >> 1 : 0u;
        const unsigned *at = row ? reinterpret_cast<const unsigned *>(p & ~(uintptr_t)3) : zero_chunk;
        const u32x4 v = *reinterpret_cast<const u32x4_g *>(at);
#pragma unroll
        for (int i = 0; i < 4; ++i) out->w[i] = v[i];
        out->w[4] = at[3 + odd];
        out->shift = 16 * odd;
        return;
    }
    const int valid = row == nullptr || c >= cols ? 0 : cols - c < 8 ? (int)(cols - c) : 8;
    const unsigned odd = valid > 0 ? (unsigned)(p & 2) >> 1 : 0u;
    const int last = valid > 0 ? ((int)odd + valid - 1) >> 1 : 0;
    const unsigned *at = valid > 0 ? reinterpret_cast<const unsigned *>(p & ~(uintptr_t)3) : zero_chunk;
#pragma unroll
    for (int i = 0; i < 5; ++i) out->w[i] = at[i < last ? i : last];
    out->shift = 16 * odd;
}
__device__ __forceinline__ u32x4 value8(const Words &x, long long c, long long cols)
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_alignbit(x.w[i + 1], x.w[i], x.shift);
    if (cols - c < 8) {   // columns at or past the end are zero
        const int valid = (int)(cols - c);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = valid >= 2 * i + 2 ? v[i] : valid == 2 * i + 1 ? v[i] & 0xFFFFu : 0u;
    }
    return v;
}

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

    // operand slices on their way: AHEAD of them in registers
    constexpr int AHEAD = 2;
    Words ra[AHEAD][TileA::LOADS], rb[AHEAD][TileB::LOADS];
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
    auto load_tiles = [&](int k0, Words *ra, Words *rb) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < TileA::LOADS; ++i) {
            const int id = i * NT + tid;
            const int r = id / TileA::CPR, c = (id % TileA::CPR) * 8;
            if constexpr (WG)
                words(row_of(p.A, lda, p.rowsA, k_lo + k0 + r, k_lo + K, p.a_rows), m0 + c, p.M, m0 + BM <= p.M, &ra[i]);
            else
                words(arow[i], k0 + c, K, k0 + BK <= K, &ra[i]);
        }
#pragma unroll
        for (int i = 0; i < TileB::LOADS; ++i) {
            const int id = i * NT + tid;
            const int r = id / TileB::CPR, c = (id % TileB::CPR) * 8;
            if constexpr (WG)
                words(row_of(p.B, ldb, p.rowsB, k_lo + k0 + r, k_lo + K, p.b_rows), n0 + c, N, n0 + BN <= N, &rb[i]);
            else if constexpr (TB)
                words(n0 + r < N ? B + (long long)(n0 + r) * ldb : nullptr, k0 + c, K, k0 + BK <= K, &rb[i]);
            else
                words(k0 + r < K ? B + (long long)(k0 + r) * ldb : nullptr, n0 + c, N, n0 + BN <= N, &rb[i]);
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
    auto store_tiles = [&](int buf, int k0, const Words *ra, const Words *rb) __attribute__((always_inline)) {
        uint16_t *la = lds + buf * BUF_HALVES;
        uint16_t *lb = la + TileA::HALVES;
#pragma unroll
        for (int i = 0; i < TileA::LOADS; ++i) {
            const int c = (i * NT + tid) % TileA::CPR * 8;
            store_one(TileA{}, la, i, WG ? value8(ra[i], m0 + c, p.M) : value8(ra[i], k0 + c, K));
        }
#pragma unroll
        for (int i = 0; i < TileB::LOADS; ++i) {
            const int c = (i * NT + tid) % TileB::CPR * 8;
            store_one(TileB{}, lb, i, !WG && TB ? value8(rb[i], k0 + c, K) : value8(rb[i], n0 + c, N));
        }
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
#pragma unroll
    for (int d = 0; d < AHEAD; ++d)
        if (d < nk) load_tiles(d * BK, ra[d], rb[d]);
    auto step = [&](int t, Words *a, Words *b) __attribute__((always_inline)) {
        const int buf = t & 1;
        store_tiles(buf, t * BK, a, b);
        if (t + AHEAD < nk) load_tiles((t + AHEAD) * BK, a, b);
        // one barrier a step: the buffer written next was last read in the step
        // before this one, which every wave has left when it passes here
        __syncthreads();
        const uint16_t *la = lds + buf * BUF_HALVES;
        const uint16_t *lb = la + TileA::HALVES;
#pragma unroll
        for (int s = 0; s < BK / 16; ++s)
            acc = mfma16<BF>(read_frag(TileB{}, lb, wn * Cfg::TN, s), read_frag(TileA{}, la, wm * Cfg::TM, s), acc);
    };
    for (int t = 0; t < nk; t += AHEAD)
#pragma unroll
        for (int d = 0; d < AHEAD; ++d)
            if (t + d < nk) step(t + d, ra[d], rb[d]);
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

template <class Cfg, bool BF, bool TB>
__global__ __launch_bounds__(Cfg::NT) void grouped_stream_kernel(RaggedArgs p)
{
    __shared__ __attribute__((aligned(1024))) unsigned char lds[Cfg::LDS];
    stream_tile<Cfg, BF, kGrouped, TB>(p, lds, blockIdx.x, 0, 1);
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

bool dwords(const void *p, long long ld, long long stride)
{
    return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0 && stride % 2 == 0;
}

// The direct-to-LDS kernel takes these operands (see ragged_dma.h).
bool grouped_dma_ok(const GroupedProblem &q)
{
    return q.K > 0 && q.K % 8 == 0 && (q.transB || q.N % 8 == 0) && dwords(q.A, q.lda, 0) && dwords(q.B, q.ldb, q.strideB) &&
           256 * q.ldb * 2 < (1LL << 31);
}
bool wgrad_dma_ok(const WgradProblem &q)
{
    return q.R > 0 && q.M % 8 == 0 && q.N % 8 == 0 && dwords(q.A, q.lda, 0) && dwords(q.B, q.ldb, 0) &&
           64 * q.lda * 2 < (1LL << 31) && 64 * q.ldb * 2 < (1LL << 31);
}

// Rounds of 256 workgroups that the tiles take, in the time of a 256x256 tile:
// a 128x128 tile takes 0.4 of that, a 64x128 tile 0.25.
double tile_rounds(double tiles, double each)
{
    return (double)(long long)((tiles + 255) / 256) * each;
}

template <class Cfg, bool BF, int KIND, bool TB, bool GA = false, bool GB = false>
hipError_t launch_tiles(RaggedArgs a, long long row_tiles, int batch, hipStream_t stream)
{
    a.tiles_m = (int)row_tiles;
    a.tiles_n = (a.N + Cfg::BN - 1) / Cfg::BN;
    const long long tiles = row_tiles * a.tiles_n;
    if (tiles > INT_MAX / Cfg::NT) return hipErrorInvalidValue;   // a grid holds fewer than 2^32 threads
    hipLaunchKernelGGL((ragged_dma_kernel<Cfg, BF, KIND, TB, GA, GB>), dim3((unsigned)tiles, 1, batch), dim3(Cfg::NT), 0, stream, a);
    return hipGetLastError();
}

template <class Cfg, bool BF, bool TB>
hipError_t launch_stream(RaggedArgs a, hipStream_t stream)
{
    a.tiles_n = (a.N + Cfg::BN - 1) / Cfg::BN;
    const long long tiles = most_row_tiles(a.R, a.groups, Cfg::BM) * a.tiles_n;
    if (tiles > INT_MAX / Cfg::NT) return hipErrorInvalidValue;
    hipLaunchKernelGGL((grouped_stream_kernel<Cfg, BF, TB>), dim3((unsigned)tiles), dim3(Cfg::NT), 0, stream, a);
    return hipGetLastError();
}

template <bool BF, bool TB>
hipError_t grouped_tiles(const GroupedProblem &q, hipStream_t stream)
{
    const RaggedArgs a = grouped_args(q);
    const double rows = (double)q.R / q.groups;
    // Few rows per group: the time is the weights', streamed.  32 columns a workgroup for weights
    // stored N x K (two workgroups of 64 KB per CU; 64 groups x 2048 x 1024, 2 rows each: 56 us,
    // against 66 with 64 columns), 64 for K x N, whose rows would otherwise be read 64 bytes at a
    // time (53 against 58 us).  At 64 rows a group 128x128 and 64x128 tiles are as fast or faster
    // (57 us against 78), at 32 the streaming is (58 against 61).
    if (rows <= 32) return launch_stream<std::conditional_t<TB, StreamCfg<1, 1, 2, 4>, StreamCfg<1, 2, 3, 2>>, BF, TB>(a, stream);
    // tiles to expect: half of the part-filled ones
    const double part = 0.5 * (q.groups < q.R ? q.groups : q.R);
    const double n256 = (q.N + 255) / 256, n128 = (q.N + 127) / 128;
    const double c256 = tile_rounds((q.R / 256.0 + part) * n256, 1.0);
    const double c128 = tile_rounds((q.R / 128.0 + part) * n128, 0.4);
    const double c64 = tile_rounds((q.R / 64.0 + part) * n128, 0.25);
    if (c256 <= c128 && c256 <= c64) return launch_tiles<Ragged256, BF, kGrouped, TB>(a, most_row_tiles(q.R, q.groups, 256), 1, stream);
    if (c128 <= c64) return launch_tiles<Ragged128, BF, kGrouped, TB>(a, most_row_tiles(q.R, q.groups, 128), 1, stream);
    return launch_tiles<Ragged64, BF, kGrouped, TB>(a, most_row_tiles(q.R, q.groups, 64), 1, stream);
}

template <bool BF, bool TB>
hipError_t grouped_any(const GroupedProblem &q, hipStream_t stream)
{
    RaggedArgs a = grouped_args(q);
    a.tiles_n = (q.N + 63) / 64;
    const long long tiles = most_row_tiles(q.R, q.groups, 64) * a.tiles_n;
    if (tiles > INT_MAX / 256) return hipErrorInvalidValue;
    hipLaunchKernelGGL((ragged_any_kernel<BF, false, TB>), dim3((unsigned)tiles), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <bool BF>
hipError_t wgrad(const WgradProblem &q, hipStream_t stream)
{
    RaggedArgs a = wgrad_args(q);
    if (wgrad_dma_ok(q)) {
        const double c256 = tile_rounds((double)((q.M + 255) / 256) * ((q.N + 255) / 256) * q.groups, 1.0);
        const double c128 = tile_rounds((double)((q.M + 127) / 128) * ((q.N + 127) / 128) * q.groups, 0.4);
        auto tiles = [&](auto ga, auto gb) {
            constexpr bool GA = decltype(ga)::value, GB = decltype(gb)::value;
            if (c256 <= c128) return launch_tiles<Ragged256, BF, kWgrad, false, GA, GB>(a, (q.M + 255) / 256, q.groups, stream);
            return launch_tiles<Ragged128, BF, kWgrad, false, GA, GB>(a, (q.M + 127) / 128, q.groups, stream);
        };
        if (q.rowsA) return q.rowsB ? tiles(std::true_type{}, std::true_type{}) : tiles(std::true_type{}, std::false_type{});
        return q.rowsB ? tiles(std::false_type{}, std::true_type{}) : tiles(std::false_type{}, std::false_type{});
    }
    a.tiles_m = (q.M + 63) / 64;
    a.tiles_n = (q.N + 63) / 64;
    if ((long long)a.tiles_m * a.tiles_n > INT_MAX / 256) return hipErrorInvalidValue;
    hipLaunchKernelGGL((ragged_any_kernel<BF, true, false>), dim3(a.tiles_m * a.tiles_n, 1, q.groups), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped(const GroupedProblem &q, bool bf, hipStream_t stream)
{
    if (grouped_dma_ok(q)) {
        if (bf) return q.transB ? grouped_tiles<true, true>(q, stream) : grouped_tiles<true, false>(q, stream);
        return q.transB ? grouped_tiles<false, true>(q, stream) : grouped_tiles<false, false>(q, stream);
    }
    if (bf) return q.transB ? grouped_any<true, true>(q, stream) : grouped_any<true, false>(q, stream);
    return q.transB ? grouped_any<false, true>(q, stream) : grouped_any<false, false>(q, stream);
}

hipError_t launch_wgrad(const WgradProblem &q, bool bf, hipStream_t stream)
{
    return bf ? wgrad<true>(q, stream) : wgrad<false>(q, stream);
}

}  // namespace mi355gemm
