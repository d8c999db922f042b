// lora_mfma.hip -- a shared projection with a low-rank adapter per row:
//   C[i,:] = alpha (A[i,:] op(B) + scales[a] (A[i,:] LA_a^T) LB_a^T) + beta C[i,:],  a = ids[i]
//
// The narrow product t = A LA^T is a few rank columns per row; it is kept in fp32
// precision throughout.  Two ways:
//   * up to 64 rows (decode), where the time is that of reading op(B) once: one
//     launch streams op(B) (stream_tile, the K range shared by several workgroups)
//     and, in further workgroups, forms t; a second adds up both, K share by K
//     share, multiplies t by LB's columns in fp32 and writes C;
//   * more rows: t first, split into 16-bit parts whose sum carries its 24 bits, then
//     the tiles of ragged_dma.h, which add the parts times LB's
//     columns after the K loop.
// Operands that direct-to-LDS loads cannot take (rows at odd halves, ragged
// 16-byte chunks) run the kernel for every alignment, then t and the product with LB.
//
// Measured (one MI355X, whole calls back to back): 1 row, 4096 x 4096 stored K x N, rank 16: 13.6 us, two
// kernels of 6.8 and 5.2 us under a tracer, the weights' 33.6 MB in 7.1 us at a copy's 4.7 TB/s; 48 rows over 32 adapters
// of rank 32, N x K: 18.2 us (12.3 + 6.8; every row's adapter is read in full, 50 MB in all: 10.9 us); 4096 rows,
// rank 16: 138 us, 1000 TFLOP/s (narrow product 11.7 us, tiles 124 to 133 us, against 114 us for a
// large matrix product of as many operations).  Tiles take a 32-row block's distinct adapters one after another, each
// a chain of loads: rows that each have their own adapter are the slowest.
#include "gemm_internal.h"
#include "ragged_dma.h"

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
template <bool BF>
__device__ __forceinline__ uint16_t round16(float v)
{
    if constexpr (BF)
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    else
        return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// Workspace.  pitch: rank rounded up to 16.
//   t: `shares` partial narrow products, each M x pitch fp32;
//   parts: kParts x M x pitch 16-bit values, then M factors (tiles);
//   sums: `splits` partial products, each M x N fp32 (decode).
__host__ __device__ inline int rank_pitch(int rank)
{
    return (rank + 15) / 16 * 16;
}

struct NarrowArgs {
    int M, K, adapters, rank, pitch;
    const uint16_t *A;
    long long lda;
    const uint16_t *LA;
    long long ldla, strideLA;
    const float *scales;
    const int32_t *ranks, *ids;
    float *t;             // shares x M x pitch, or
    uint16_t *parts;      // kParts x M x pitch with
    float *factor;        // M
};

// The narrow product of the rows of 16-row block `rb` that use its `nth` distinct
// adapter: t[i,:] = A[i,:] LA_a^T over share `share` of `shares` of K.  The NT / 64 waves
// take chunks of 64 k in turn and add up in wave order.  PARTS: the whole K, t
// rounded to 16-bit parts: of t / 2^e, 2^e such that the row's largest finite value is
// near 2^14 (fp16, whose exponents a row's t may leave), e = 0 for bf16.
// The parts hold t's 24 bits (see kPartStep).
// Bound by reading A (4096 x 4096, rank 16: 33.6 MB in 11.7 us, 2.9 TB/s).
template <bool BF, int NR, int NT, bool PARTS>
__device__ __forceinline__ void narrow_block(const NarrowArgs &p, unsigned char *lds, int rb, int nth, int share, int shares)
{
    constexpr int NW = NT / 64;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 15, lq = lane >> 4;
    const int row0 = rb * 16;
    const int mine = adapter_of(p.ids, p.adapters, row0 + li, p.M);
    // lanes whose adapter no earlier row of the block has
    bool first = lane < 16 && mine >= 0;
#pragma unroll
    for (int i = 0; i < 15; ++i) {
        const int o = __builtin_amdgcn_readlane(mine, i);
        if (i < lane && o == mine) first = false;
    }
    uint64_t firsts = __ballot(first);
    for (int j = 0; j < nth && firsts; ++j) firsts &= firsts - 1;
    if (!firsts) return;
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctzll(firsts));
    const int ra = rank_of(p.ranks, p.rank, a);
    const uint16_t *la = p.LA + (long long)a * p.strideLA;
    const int row = row0 + li;
    const uint16_t *x = p.A + (long long)(row < p.M ? row : p.M - 1) * p.lda;
    f32x4v acc[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[n] = f32x4v{0.f, 0.f, 0.f, 0.f};
    const int blocks = (p.K + 63) / 64, turn = NW * shares;
    // LA's rows that this lane loads; those past the adapter's rank are not read
    const uint16_t *lrow[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) lrow[n] = la + (long long)(16 * n + li) * p.ldla;
    const bool vec = p.K % 64 == 0 && p.lda % 2 == 0 && p.ldla % 2 == 0 && reinterpret_cast<uintptr_t>(x) % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(la) % 4 == 0;
    if (__builtin_amdgcn_readfirstlane(vec)) {
#pragma unroll(NR > 2 ? 1 : 2)
        for (int b = share * NW + wave; b < blocks; b += turn) {
            half8 xb[2], f[2][NR];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kq = 64 * b + 32 * h + 8 * lq;
                xb[h] = __builtin_bit_cast(half8, *reinterpret_cast<const u32x4_g *>(x + kq));
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    u32x4 v = {0u, 0u, 0u, 0u};
                    if (16 * n + li < ra) v = *reinterpret_cast<const u32x4_g *>(lrow[n] + kq);
                    f[h][n] = __builtin_bit_cast(half8, v);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NR; ++n) acc[n] = mfma16x16<BF>(f[h][n], xb[h], acc[n]);
        }
    } else {
        for (int b = share * NW + wave; b < blocks; b += turn)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kq = 64 * b + 32 * h + 8 * lq;
                const bool whole = 64 * (b + 1) <= p.K;
                Words xw, w[NR];
                words(x, kq, p.K, whole, &xw);
#pragma unroll
                for (int n = 0; n < NR; ++n) words(16 * n + li < ra ? lrow[n] : nullptr, kq, p.K, whole, &w[n]);
                const half8 xb = __builtin_bit_cast(half8, value8(xw, kq, p.K));
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    acc[n] = mfma16x16<BF>(__builtin_bit_cast(half8, value8(w[n], kq, p.K)), xb, acc[n]);
            }
    }
    // lane: columns 16n + 4*lq .. +3 of row li
    f32x4v *part = reinterpret_cast<f32x4v *>(lds);   // NW x NR x 64
#pragma unroll
    for (int n = 0; n < NR; ++n) part[(wave * NR + n) * 64 + lane] = acc[n];
    __syncthreads();
    if constexpr (!PARTS) {
        if (mine != a) return;
        for (int n = wave; n < NR; n += NW) {
            if (16 * n >= p.pitch) break;
            f32x4v s = part[n * 64 + lane];
#pragma unroll
            for (int w = 1; w < NW; ++w) s += part[(w * NR + n) * 64 + lane];
            *reinterpret_cast<f32x4v *>(p.t + ((long long)share * p.M + row) * p.pitch + 16 * n + 4 * lq) = s;
        }
    } else {
        if (wave != 0) return;
        // (columns past the adapter's rank are zeros, which a row's infinities times no row of LA are not)
        auto sum = [&](int n) {
            f32x4v v = part[n * 64 + lane];
#pragma unroll
            for (int w = 1; w < NW; ++w) v += part[(w * NR + n) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = 16 * n + 4 * lq + e < ra ? v[e] : 0.f;
            return v;
        };
        int ex = 0;
        if constexpr (!BF) {
            float most = 0.f;
            for (int n = 0; n < NR; ++n) {
                const f32x4v v = sum(n);
#pragma unroll
                for (int e = 0; e < 4; ++e) most = fabsf(v[e]) < INFINITY ? fmaxf(most, fabsf(v[e])) : most;
            }
            most = fmaxf(most, __shfl_xor(most, 16));
            most = fmaxf(most, __shfl_xor(most, 32));
            if (most > 0.f) {
                (void)frexpf(most, &ex);   // most = m 2^ex, 1/2 <= m < 1
                ex -= 15;
            }
        }
        if (mine != a) return;
        if (lq == 0) p.factor[row] = ldexpf(p.scales ? p.scales[a] : 1.f, ex);
        for (int n = 0; 16 * n < p.pitch; ++n) {
            const f32x4v v = sum(n);
            float rest[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) rest[e] = BF ? v[e] : ldexpf(v[e], -ex);
#pragma unroll
            for (int part_i = 0; part_i < kParts; ++part_i) {
                uint16_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[e] = round16<BF>(rest[e]);
                    const float got = widen16<BF>(h[e]);
                    rest[e] = got - got == 0.f ? (rest[e] - got) * (1.f / kPartStep<BF>) : 0.f;   // (infinities and NaN stand in the first part alone)
                }
                unsigned *dst = reinterpret_cast<unsigned *>(p.parts + ((long long)part_i * p.M + row) * p.pitch + 16 * n + 4 * lq);
                dst[0] = h[0] | ((unsigned)h[1] << 16);
                dst[1] = h[2] | ((unsigned)h[3] << 16);
            }
        }
    }
}

template <bool BF, int NR, bool PARTS>
__global__ __launch_bounds__(512) void narrow_kernel(NarrowArgs p)
{
    __shared__ __attribute__((aligned(16))) unsigned char lds[8 * NR * 64 * 16];
    narrow_block<BF, NR, 512, PARTS>(p, lds, blockIdx.x, blockIdx.y, 0, 1);
}

// Decode: the first `narrow` workgroups form t, the others stream op(B).  One launch, since t
// is needed only at the end: its loads share the chip with op(B)'s (48 rows, 4096 x 4096, 32
// adapters of rank 32: 12.6 us; bound by reading both).
template <class Cfg, bool BF, bool TB, int NR>
__global__ __launch_bounds__(Cfg::NT) void decode_kernel(RaggedArgs base, NarrowArgs thin, int narrow, int slots, int shares,
                                                         int splits)
{
    __shared__ __attribute__((aligned(1024))) unsigned char lds[Cfg::LDS];
    static_assert((Cfg::NT / 64) * NR * 64 * 16 <= Cfg::LDS, "the narrow product's sums fit");
    int b = blockIdx.x;
    if (b < narrow) {
        const int share = b % shares;
        b /= shares;
        narrow_block<BF, NR, Cfg::NT, false>(thin, lds, b / slots, b % slots, share, shares);
        return;
    }
    b -= narrow;
    stream_tile<Cfg, BF, kLora, TB>(base, lds, b / splits, b % splits, splits);
}

struct FinishArgs {
    int M, N, adapters, rank, pitch, shares, splits;
    float alpha, beta;
    const uint16_t *LB;
    long long ldlb, strideLB;
    const float *scales, *t, *sums;   // sums: splits x M x N, or nullptr: C holds alpha A op(B) + beta C already
    const int32_t *ranks, *ids;
    float *C;
    long long ldc;
};

// C[i,n] = alpha (sum of the products' shares + scale * sum_j t[i,j] LB_a[n,j]) + beta C[i,n].
// A thread per column, a block per row and NT columns.  Bound by latency: ids, then ranks, then
// LB's row, each waiting for the one before (48 x 4096, rank 32: 6.7 us for 10 MB of LB and 12.6 MB of sums;
// reading LB's row before the rank is known was no faster, 20.9 against 18.7 us for the call).
template <bool BF, int NT>
__global__ __launch_bounds__(NT) void finish_kernel(FinishArgs p)
{
    const int row = blockIdx.y;
    const int a = adapter_of(p.ids, p.adapters, row, p.M);
    if (a < 0 && p.sums == nullptr) return;
    const int ra = a < 0 ? 0 : rank_of(p.ranks, p.rank, a);
    __shared__ float t[kMaxRank];
    for (int j = threadIdx.x; j < kMaxRank; j += NT) {
        float s = 0.f;
        if (j < ra)
#pragma unroll 4
            for (int i = 0; i < p.shares; ++i) s += p.t[((long long)i * p.M + row) * p.pitch + j];
        t[j] = s;
    }
    // (loads first: they do not depend on one another)
    const int n = blockIdx.x * NT + threadIdx.x;
    const int nc = n < p.N ? n : p.N - 1;
    float base[4] = {0.f, 0.f, 0.f, 0.f};   // shares i, i + 4, ..., added in a fixed order
    if (p.sums) {
        const float *sum = p.sums + (long long)row * p.N + nc;
        const long long apart = (long long)p.M * p.N;
        for (int i = 0; i < p.splits; i += 4)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < p.splits) base[e] += sum[(i + e) * apart];
    }
    const uint16_t *b = p.LB + (a < 0 ? 0 : (long long)a * p.strideLB + (long long)nc * p.ldlb);
    float *c = p.C + (long long)row * p.ldc + nc;
    const float old = p.beta != 0.f || p.sums == nullptr ? *c : 0.f;
    const float scale = a >= 0 && p.scales ? p.scales[a] : 1.f;
    half8 h[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) h[x] = load8_any(b + 8 * x, ra - 8 * x);
    __syncthreads();
    float s = 0.f;
    for (int j = 0; j < ra; j += 16) {
        half8 next[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) next[x] = load8_any(b + j + 16 + 8 * x, ra - j - 16 - 8 * x);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const _Float16 v = h[x][e];   // (its 16 bits; past the rank t and v are zero)
                s = __builtin_fmaf(t[j + 8 * x + e], widen16<BF>(__builtin_bit_cast(uint16_t, v)), s);
            }
#pragma unroll
        for (int x = 0; x < 2; ++x) h[x] = next[x];
    }
    if (n >= p.N) return;
    if (p.sums) {
        const float v = p.alpha * (((base[0] + base[1]) + (base[2] + base[3])) + s * scale);
        *c = p.beta != 0.f ? __builtin_fmaf(p.beta, old, v) : v;
    } else {
        *c = __builtin_fmaf(p.alpha, s * scale, old);
    }
}

constexpr int kDecodeRows = 64;

// Workgroups that share a strip of 64 columns in decode, so that about 256 stream op(B) (4096 x 4096,
// 48 rows: 18.7 us, with twice as many 23.1): at least two slices of 64 k for each of their two waves, and 16
// workgroups at most, whose sums the join adds one after another (16 rows, 64 columns: K = 8192 14.2 us against
// 16.5 with 32, K = 65280 21 against 80 with 255).
int decode_splits(int N, int K)
{
    const int strips = (N + 63) / 64, most = (K + 255) / 256;
    int s = (256 + strips - 1) / strips;
    s = s > 16 ? 16 : s;
    return s < 1 ? 1 : s > most ? most : s;
}
// Workgroups that share K in a narrow product, at most: 256 k or more each.
int most_shares(int K)
{
    const int s = K / 256;
    return s < 1 ? 1 : s > 16 ? 16 : s;
}
// Distinct adapters that 16 rows can have.
int row_block_adapters(const LoraProblem &p)
{
    const int rows = p.M < 16 ? p.M : 16;
    return p.adapters < rows ? p.adapters : rows;
}

NarrowArgs narrow_args(const LoraProblem &p)
{
    NarrowArgs a = {};
    a.M = p.M; a.K = p.K; a.adapters = p.adapters; a.rank = p.rank; a.pitch = rank_pitch(p.rank);
    a.A = p.A; a.lda = p.lda;
    a.LA = p.LA; a.ldla = p.ldla; a.strideLA = p.strideLA;
    a.scales = p.scales; a.ranks = p.ranks; a.ids = p.ids;
    a.t = p.t;
    return a;
}
RaggedArgs base_args(const LoraProblem &p)
{
    RaggedArgs a = {};
    a.M = p.M; a.N = p.N; a.K = p.K; a.a_rows = p.M;
    a.alpha = p.alpha; a.beta = p.beta;
    a.A = p.A; a.lda = p.lda;
    a.B = p.B; a.ldb = p.ldb;
    a.C = p.C; a.ldc = p.ldc;
    return a;
}
FinishArgs finish_args(const LoraProblem &p)
{
    FinishArgs a = {};
    a.M = p.M; a.N = p.N; a.adapters = p.adapters; a.rank = p.rank; a.pitch = rank_pitch(p.rank);
    a.shares = 1; a.splits = 0;
    a.alpha = p.alpha; a.beta = p.beta;
    a.LB = p.LB; a.ldlb = p.ldlb; a.strideLB = p.strideLB;
    a.scales = p.scales; a.ranks = p.ranks; a.ids = p.ids;
    a.t = p.t;
    a.C = p.C; a.ldc = p.ldc;
    return a;
}

template <bool BF, bool PARTS>
hipError_t launch_narrow(const LoraProblem &p, const NarrowArgs &a, hipStream_t stream)
{
    const dim3 grid((p.M + 15) / 16, row_block_adapters(p)), block(512);
    if (p.rank <= 16)
        hipLaunchKernelGGL((narrow_kernel<BF, 1, PARTS>), grid, block, 0, stream, a);
    else if (p.rank <= 32)
        hipLaunchKernelGGL((narrow_kernel<BF, 2, PARTS>), grid, block, 0, stream, a);
    else if (p.rank <= 64)
        hipLaunchKernelGGL((narrow_kernel<BF, 4, PARTS>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((narrow_kernel<BF, 8, PARTS>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <bool BF>
hipError_t launch_finish(FinishArgs a, hipStream_t stream)
{
    const int M = a.M;
    for (int r0 = 0; r0 < M; r0 += 65535) {   // (rows from r0 on: t and sums are indexed by the whole M, with one share beyond 64 rows)
        FinishArgs q = a;
        const int rows = M - r0 < 65535 ? M - r0 : 65535;
        if (r0 > 0) {
            q.M = M - r0;
            q.ids += r0;
            q.t += (long long)r0 * a.pitch;
            q.C += (long long)r0 * a.ldc;
        }
        if (rows <= 8)   // (few rows: smaller blocks reach more CUs)
            hipLaunchKernelGGL((finish_kernel<BF, 64>), dim3((a.N + 63) / 64, rows), dim3(64), 0, stream, q);
        else
            hipLaunchKernelGGL((finish_kernel<BF, 256>), dim3((a.N + 255) / 256, rows), dim3(256), 0, stream, q);
    }
    return hipGetLastError();
}

bool dwords(const void *p, long long ld)
{
    return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0;
}
bool lora_dma_ok(const LoraProblem &p)
{
    return p.K > 0 && p.K % 8 == 0 && (p.transB || p.N % 8 == 0) && dwords(p.A, p.lda) && dwords(p.B, p.ldb) &&
           256 * p.ldb * 2 < (1LL << 31);
}

// Whether one launch holds Cfg's tiles.
template <class Cfg>
bool lora_holds(const LoraProblem &p)
{
    return grid_holds((p.M + Cfg::BM - 1LL) / Cfg::BM * ((p.N + Cfg::BN - 1LL) / Cfg::BN), Cfg::NT);
}

template <class Cfg, bool BF, bool TB>
hipError_t launch_decode(const LoraProblem &p, hipStream_t stream)
{
    RaggedArgs base = base_args(p);
    NarrowArgs thin = narrow_args(p);
    const int splits = decode_splits(p.N, p.K), slots = row_block_adapters(p), most = most_shares(p.K);
    // about 256 workgroups for the narrow product beside as many that stream: two per CU
    int shares = 256 / ((p.M + 15) / 16 * slots);
    shares = shares < 1 ? 1 : shares > most ? most : shares;
    float *sums = p.t + (size_t)shares * p.M * thin.pitch;
    base.tiles_m = (p.M + Cfg::BM - 1) / Cfg::BM;
    base.tiles_n = (p.N + Cfg::BN - 1) / Cfg::BN;
    base.C = sums; base.ldc = p.N; base.strideC = (long long)p.M * p.N;
    const int narrow = (p.M + 15) / 16 * slots * shares;
    const dim3 grid(narrow + base.tiles_m * base.tiles_n * splits), block(Cfg::NT);
    auto run = [&](auto nr) {
        hipLaunchKernelGGL((decode_kernel<Cfg, BF, TB, decltype(nr)::value>), grid, block, 0, stream, base, thin, narrow, slots,
                           shares, splits);
    };
    if (p.rank <= 16)
        run(std::integral_constant<int, 1>{});
    else if (p.rank <= 32)
        run(std::integral_constant<int, 2>{});
    else if (p.rank <= 64)
        run(std::integral_constant<int, 4>{});
    else
        run(std::integral_constant<int, 8>{});
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    FinishArgs f = finish_args(p);
    f.shares = shares; f.splits = splits; f.sums = sums;
    return launch_finish<BF>(f, stream);
}

template <class Cfg, bool BF, bool TB>
hipError_t launch_tiles(RaggedArgs a, hipStream_t stream)
{
    a.tiles_m = (a.M + Cfg::BM - 1) / Cfg::BM;
    a.tiles_n = (a.N + Cfg::BN - 1) / Cfg::BN;
    const long long tiles = (long long)a.tiles_m * a.tiles_n;
    if (!grid_holds(tiles, Cfg::NT)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((ragged_dma_kernel<Cfg, BF, kLora, TB, false, false>), dim3((unsigned)tiles), dim3(Cfg::NT), 0, stream, a);
    return hipGetLastError();
}

template <bool BF, bool TB>
hipError_t lora_tiles(const LoraProblem &p, hipStream_t stream)
{
    NarrowArgs thin = narrow_args(p);
    thin.parts = reinterpret_cast<uint16_t *>(p.t);
    thin.factor = reinterpret_cast<float *>(thin.parts + (size_t)kParts * p.M * thin.pitch);
    if (const hipError_t e = launch_narrow<BF, true>(p, thin, stream); e != hipSuccess) return e;
    RaggedArgs a = base_args(p);
    a.ad.ids = p.ids; a.ad.ranks = p.ranks; a.ad.adapters = p.adapters; a.ad.rank = p.rank;
    a.ad.LB = p.LB; a.ad.ldlb = p.ldlb; a.ad.strideLB = p.strideLB;
    a.ad.parts = thin.parts; a.ad.pitch = thin.pitch; a.ad.factor = thin.factor;
    auto rounds = [&](int bm, int bn) { return (((p.M + bm - 1LL) / bm) * ((p.N + bn - 1LL) / bn) + 255) / 256; };
    // in the time of a 256x256 tile: a 128x128 tile takes 0.4, a 64x128 tile 0.25
    const double c256 = rounds(256, 256), c128 = 0.4 * rounds(128, 128), c64 = 0.25 * rounds(64, 128);
    // (where one launch does not hold the tiles that would be fastest, larger ones)
    const bool large = c256 <= c128 && c256 <= c64;
    if (!large && c64 < c128 && lora_holds<Ragged64>(p)) return launch_tiles<Ragged64, BF, TB>(a, stream);
    if (!large && lora_holds<Ragged128>(p)) return launch_tiles<Ragged128, BF, TB>(a, stream);
    return launch_tiles<Ragged256, BF, TB>(a, stream);
}

// Any strides and alignments: the projection (few rows: K shared by several workgroups per
// tile), the narrow product, then both joined.
template <bool BF, bool TB>
hipError_t lora_any(const LoraProblem &p, hipStream_t stream)
{
    RaggedArgs a = base_args(p);
    FinishArgs f = finish_args(p);
    auto run = [&](auto cfg, int splits) {
        using Cfg = decltype(cfg);
        a.tiles_m = (p.M + Cfg::BM - 1) / Cfg::BM;
        a.tiles_n = (p.N + Cfg::BN - 1) / Cfg::BN;
        const long long tiles = (long long)a.tiles_m * a.tiles_n;
        if (!grid_holds(tiles, 256)) return hipErrorInvalidValue;
        hipLaunchKernelGGL((ragged_any_kernel<Cfg, BF, kLora, TB>), dim3((unsigned)tiles, splits), dim3(256), 0, stream, a);
        return hipGetLastError();
    };
    hipError_t e = hipSuccess;
    if (p.M <= kDecodeRows) {
        const int splits = decode_splits(p.N, p.K);
        if (splits > 1) {
            float *sums = p.t + (size_t)p.M * f.pitch;
            a.C = sums; a.ldc = p.N; a.strideC = (long long)p.M * p.N;
            f.splits = splits; f.sums = sums;
        }
        e = run(HgCfg<64, 64>{}, splits);
    } else {
        // (128x128 tiles as in the grouped product)
        bool large = false;
        if constexpr (TB) large = ((p.M + 127LL) / 128) * ((p.N + 127LL) / 128) >= 256 || !lora_holds<HgCfg<64, 64>>(p);
        if constexpr (TB)
            if (large) e = run(HgCfg<128, 128>{}, 1);
        if (!large) e = run(HgCfg<64, 64>{}, 1);
    }
    if (e != hipSuccess) return e;
    if (e = launch_narrow<BF, false>(p, narrow_args(p), stream); e != hipSuccess) return e;
    return launch_finish<BF>(f, stream);
}

template <bool BF>
hipError_t lora(const LoraProblem &p, hipStream_t stream)
{
    GemmProblem g = {};
    g.transB = p.transB;
    g.M = p.M; g.N = p.N; g.K = p.K; g.batch = 1;
    g.alpha = p.alpha; g.beta = p.beta;
    g.A = p.A; g.lda = p.lda;
    g.B = p.B; g.ldb = p.ldb;
    g.C = p.C; g.ldc = p.ldc;
    if (p.K == 0) return launch_scale_c(g, stream);
    if (p.adapters > 0 && lora_dma_ok(p)) {
        if (p.M <= 32) {
            if (p.transB) return launch_decode<StreamCfg<1, 2, 3, 2>, BF, true>(p, stream);
            return launch_decode<StreamCfg<1, 2, 3, 2>, BF, false>(p, stream);
        }
        if (p.M <= kDecodeRows) {
            if (p.transB) return launch_decode<StreamCfg<2, 2, 2, 2>, BF, true>(p, stream);
            return launch_decode<StreamCfg<2, 2, 2, 2>, BF, false>(p, stream);
        }
        return p.transB ? lora_tiles<BF, true>(p, stream) : lora_tiles<BF, false>(p, stream);
    }
    if (p.adapters == 0) return BF ? launch_bgemm(g, stream) : launch_hgemm(g, stream);
    return p.transB ? lora_any<BF, true>(p, stream) : lora_any<BF, false>(p, stream);
}

}  // namespace

bool lora_fits(const LoraProblem &p)
{
    if (p.K == 0 || p.M <= kDecodeRows) return true;   // (64 rows: N <= 2^25 is 2^19 strips)
    if (p.adapters == 0) return ((p.M + 31LL) / 32) * ((p.N + 31LL) / 32) <= 0x7FFFFFFF;   // (as gemm_*_f32acc_ex)
    if (lora_dma_ok(p)) return lora_holds<Ragged256>(p);
    return p.transB ? lora_holds<HgCfg<128, 128>>(p) : lora_holds<HgCfg<64, 64>>(p);
}

size_t lora_workspace(int M, int N, int K, int rank)
{
    const size_t cells = (size_t)M * rank_pitch(rank);
    if (M <= kDecodeRows)
        return (cells * most_shares(K) + (size_t)M * N * decode_splits(N, K)) * sizeof(float);
    return cells * kParts * sizeof(uint16_t) + (size_t)M * sizeof(float);   // at least the cells' fp32
}

hipError_t launch_lora(const LoraProblem &p, bool bf, hipStream_t stream)
{
    return bf ? lora<true>(p, stream) : lora<false>(p, stream);
}

}  // namespace mi355gemm
