// grouped_mfma.hip -- products of ragged groups of rows, 16-bit inputs, fp32
// accumulation and C:
//   grouped  C[r,:] = alpha A[rows[r],:] op(B_g) + beta C[r,:],  offsets[g] <= r < offsets[g+1]
//   wgrad    C_g = alpha sum_r A[rowsA[r],:]^T B[rowsB[r],:] + beta C_g,  r in group g
// The offsets live on the device, so the host launches as many workgroups as
// any split of R rows over the groups can need, and each workgroup finds its
// group and tile from the offsets; surplus workgroups return at once.
#include "routed_internal.h"
#include "ragged_dma.h"

namespace mi355gemm {
namespace {

template <class Cfg, bool BF, bool TB>
__global__ __launch_bounds__(Cfg::NT) void grouped_stream_kernel(RaggedArgs p)
{
    __shared__ __attribute__((aligned(1024))) unsigned char lds[Cfg::LDS];
    stream_tile<Cfg, BF, kGrouped, TB>(p, lds, blockIdx.x, 0, 1);
}

// C of so many bytes goes past the caches.  The memory-side cache holds 256 MiB: with C of 128 MiB the product and
// the kernel that reads C next take 177 us together and 183 with such stores, with 256 MiB 351 and 346.
constexpr long long kPastCache = 192LL << 20;

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
    a.past_cache = 4LL * q.R * q.N >= kPastCache;
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
    a.past_cache = 4LL * q.M * q.N * q.groups >= kPastCache;
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

// Workgroups of Cfg's tiles, and whether one launch holds them.
template <class Cfg>
bool grouped_holds(const GroupedProblem &q)
{
    return grid_holds(most_row_tiles(q.R, q.groups, Cfg::BM) * ((q.N + Cfg::BN - 1LL) / Cfg::BN), Cfg::NT);
}
template <class Cfg>
bool wgrad_holds(const WgradProblem &q)
{
    return grid_holds((q.M + Cfg::BM - 1LL) / Cfg::BM * ((q.N + Cfg::BN - 1LL) / Cfg::BN), Cfg::NT);
}

template <class Cfg, bool BF, int KIND, bool TB, bool GA = false, bool GB = false>
hipError_t launch_tiles(RaggedArgs a, long long row_tiles, int batch, hipStream_t stream)
{
    a.tiles_m = (int)row_tiles;
    a.tiles_n = (a.N + Cfg::BN - 1) / Cfg::BN;
    const long long tiles = row_tiles * a.tiles_n;
    if (!grid_holds(tiles, Cfg::NT)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((ragged_dma_kernel<Cfg, BF, KIND, TB, GA, GB>), dim3((unsigned)tiles, 1, batch), dim3(Cfg::NT), 0, stream, a);
    return hipGetLastError();
}

template <class Cfg, bool BF, bool TB>
hipError_t launch_stream(RaggedArgs a, hipStream_t stream)
{
    const long long row_tiles = most_row_tiles(a.R, a.groups, Cfg::BM);
    a.tiles_m = (int)row_tiles;
    a.tiles_n = (a.N + Cfg::BN - 1) / Cfg::BN;
    const long long tiles = row_tiles * a.tiles_n;
    if (!grid_holds(tiles, Cfg::NT)) return hipErrorInvalidValue;
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
    // (57 us against 78), at 32 the streaming is (58 against 61).  The host knows the mean alone: a group
    // far above it has its weights read once for every 32 of its rows.
    // (Here and below: where one launch does not hold the tiles that would be fastest, larger ones.)
    using Stream = std::conditional_t<TB, StreamCfg<1, 1, 2, 4>, StreamCfg<1, 2, 3, 2>>;
    if (rows <= 32 && grouped_holds<Stream>(q)) return launch_stream<Stream, BF, TB>(a, stream);
    // tiles to expect: half of the part-filled ones
    const double part = 0.5 * (q.groups < q.R ? q.groups : q.R);
    const double n256 = (q.N + 255) / 256, n128 = (q.N + 127) / 128;
    const double c256 = tile_rounds((q.R / 256.0 + part) * n256, 1.0);
    const double c128 = tile_rounds((q.R / 128.0 + part) * n128, 0.4);
    const double c64 = tile_rounds((q.R / 64.0 + part) * n128, 0.25);
    const bool large = c256 <= c128 && c256 <= c64;
    if (!large && c64 < c128 && grouped_holds<Ragged64>(q))
        return launch_tiles<Ragged64, BF, kGrouped, TB>(a, most_row_tiles(q.R, q.groups, 64), 1, stream);
    if (!large && grouped_holds<Ragged128>(q))
        return launch_tiles<Ragged128, BF, kGrouped, TB>(a, most_row_tiles(q.R, q.groups, 128), 1, stream);
    return launch_tiles<Ragged256, BF, kGrouped, TB>(a, most_row_tiles(q.R, q.groups, 256), 1, stream);
}

template <class Cfg, bool BF, bool TB>
hipError_t grouped_any_tiles(const GroupedProblem &q, hipStream_t stream)
{
    RaggedArgs a = grouped_args(q);
    const long long row_tiles = most_row_tiles(q.R, q.groups, Cfg::BM);
    a.tiles_m = (int)row_tiles;
    a.tiles_n = (q.N + Cfg::BN - 1) / Cfg::BN;
    const long long tiles = row_tiles * a.tiles_n;
    if (!grid_holds(tiles, 256)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((ragged_any_kernel<Cfg, BF, kGrouped, TB>), dim3((unsigned)tiles), dim3(256), 0, stream, a);
    return hipGetLastError();
}
template <bool BF, bool TB>
hipError_t grouped_any(const GroupedProblem &q, hipStream_t stream)
{
    const double part = 0.5 * (q.groups < q.R ? q.groups : q.R);
    // 128x128 tiles where they fill the chip and B is stored N x K (16 groups, 8000 rows, 1001 x 1001, 564 tiles: 44
    // against 62 us; 8 groups, 4000 rows, 777 x 1001, 282 tiles: 26 against 30; 2000 rows, 157 tiles: 22 against 17.5);
    // stored K x N they gain nothing (564 tiles 76.3 against 75.6 us, 282 43 against 38)
    if constexpr (TB)
        if ((q.R / 128.0 + part) * ((q.N + 127) / 128) >= 256 || !grouped_holds<HgCfg<64, 64>>(q))
            return grouped_any_tiles<HgCfg<128, 128>, BF, TB>(q, stream);
    return grouped_any_tiles<HgCfg<64, 64>, BF, TB>(q, stream);
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
            if (c256 <= c128 || !wgrad_holds<Ragged128>(q))
                return launch_tiles<Ragged256, BF, kWgrad, false, GA, GB>(a, (q.M + 255) / 256, q.groups, stream);
            return launch_tiles<Ragged128, BF, kWgrad, false, GA, GB>(a, (q.M + 127) / 128, q.groups, stream);
        };
        if (q.rowsA) return q.rowsB ? tiles(std::true_type{}, std::true_type{}) : tiles(std::true_type{}, std::false_type{});
        return q.rowsB ? tiles(std::false_type{}, std::true_type{}) : tiles(std::false_type{}, std::false_type{});
    }
    auto any = [&](auto cfg) {
        using Cfg = decltype(cfg);
        a.tiles_m = (q.M + Cfg::BM - 1) / Cfg::BM;
        a.tiles_n = (q.N + Cfg::BN - 1) / Cfg::BN;
        if (!grid_holds((long long)a.tiles_m * a.tiles_n, 256)) return hipErrorInvalidValue;
        hipLaunchKernelGGL((ragged_any_kernel<Cfg, BF, kWgrad, false>), dim3(a.tiles_m * a.tiles_n, 1, q.groups), dim3(256), 0,
                           stream, a);
        return hipGetLastError();
    };
    // 128x128 tiles where there are several for a CU (1024 tiles: 16384 rows, 512 x 1023, 32 groups 63.5 against 75 us,
    // 4000 rows, 1001 x 1001, 16 groups 47 against 50; 560: 8000 rows, 513 x 777, 16 groups 45.5 against 41.5; 192: 6752
    // rows, 1024 x 341, 8 groups 37 against 29)
    if ((q.M + 127LL) / 128 * ((q.N + 127) / 128) * q.groups >= 768 || !wgrad_holds<HgCfg<64, 64>>(q)) return any(HgCfg<128, 128>{});
    return any(HgCfg<64, 64>{});
}

}  // namespace

bool grouped_fits(const GroupedProblem &q)
{
    if (grouped_dma_ok(q)) return grouped_holds<Ragged256>(q);
    return q.transB ? grouped_holds<HgCfg<128, 128>>(q) : grouped_holds<HgCfg<64, 64>>(q);
}

bool wgrad_fits(const WgradProblem &q)
{
    return wgrad_dma_ok(q) ? wgrad_holds<Ragged256>(q) : wgrad_holds<HgCfg<128, 128>>(q);
}

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
