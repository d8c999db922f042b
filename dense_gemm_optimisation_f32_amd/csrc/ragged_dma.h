// ragged_dma.h -- tiles of products whose right operand is chosen per row, fed by
// direct-to-LDS loads: ragged groups of rows (grouped_mfma.hip) and rows with
// low-rank adapters (lora_mfma.hip).
#pragma once

#include "routed_internal.h"
#include "row_tiles.h"
#include "stage16.h"
#include "tile_order.h"
#include "wave.h"

#include <type_traits>
#include <utility>

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
// `total` of them (at most `most`, the launch's), and of tile `want` its group, first row and the group's end.
// Every wave does this by itself, 64 groups at a time, one per lane.
struct RowTile {
    int group, first, end;
};
__device__ __forceinline__ int count_row_tiles(const int32_t *offsets, int groups, int R, int bm, int most)
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
        total = add_row_tiles(total, wave_sum((unsigned)n), most);
    }
    return total;
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
        const int s = wave_scan(n);
        const uint64_t hit = __ballot(want >= s - n && want < s);
        if (hit) {
            const int at = __builtin_ctzll(hit), first = lo + (want - (s - n)) * bm;
            return {g0 + at, __builtin_amdgcn_readlane(first, at), __builtin_amdgcn_readlane(hi, at)};
        }
        want -= __builtin_amdgcn_readlane(s, 63);
    }
    return {-1, 0, 0};
}

// The adapters of the rows (lora): the narrow product t of each row as three 16-bit
// parts, t / 2^e = part 0 + kPartStep (part 1 + kPartStep part 2), and the row's factor
// scale * 2^e.
struct AdapterArgs {
    const int32_t *ids, *ranks;
    int adapters, rank;
    const uint16_t *LB;
    long long ldlb, strideLB;
    const uint16_t *parts;    // 3 x M x pitch
    int pitch;                // halves per row: rank rounded up to 16
    const float *factor;      // M
};
// Parts of a 32-bit value: 24 bits as three pieces of 8 (bf16), or of 11 (fp16).  bf16 has fp32's exponents. In
// fp16 what a part leaves is scaled up by 2^11, so that it does not fall below fp16's smallest value
// (2^-24, with a row's largest near 2^14): a value keeps its 24 bits down to 2^-37 of the row's largest,
// and is off by 2^-61 of that below.  (Two fp16 parts held 22 bits; the third costs 1% of 2048 rows with rank 16,
// 2% of 4096 with rank 64, 5% of 1024 rows of 2048 x 2048 with rank 128.)
constexpr int kParts = 3;
template <bool BF>
constexpr float kPartStep = BF ? 1.f : 1.f / 2048;

__device__ __forceinline__ int adapter_of(const int32_t *ids, int adapters, int row, int M)
{
    const int a = row < M ? ids[row] : -1;
    return a >= 0 && a < adapters ? a : -1;
}
__device__ __forceinline__ int rank_of(const int32_t *ranks, int rank, int a)
{
    const int r = ranks ? ranks[a] : rank;
    return r < 0 ? 0 : r > rank ? rank : r;
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
    int tiles_m, tiles_n;     // grouped: tiles_m is what any ascending offsets can need
    bool product;             // false: C is only scaled
    bool past_cache;          // C is larger than what the memory-side cache keeps of it
    AdapterArgs ad;           // lora
};

// A direct-to-LDS load whose lanes each name a whole address (dma16 with one
// base for all lanes is in stage16.h; the notes there hold here too).
__device__ __forceinline__ void dma16_at(const void *p, unsigned lds_addr)
{
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(p), "s"(lds_addr) : "memory", "m0");
}

// A pointer that is the same in every lane, in scalar registers (dma16's base).
__device__ __forceinline__ const char *uniform(const char *p)
{
    const uint64_t b = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = (unsigned)__builtin_amdgcn_readfirstlane((int)b);
    const uint64_t hi = (unsigned)__builtin_amdgcn_readfirstlane((int)(b >> 32));
    return reinterpret_cast<const char *>(lo | (hi << 32));
}

// What a lane reads in place of a chunk outside its operand.
__device__ const unsigned zero_chunk[4] = {0u, 0u, 0u, 0u};

typedef const __attribute__((address_space(4))) int32_t *scalar_ints;   // read through the scalar cache

enum RaggedKind { kGrouped, kWgrad, kLora };

// ---------------------------------------------------------------------------
// The ring, its loads and its K loop are those of the whole-matrix kernel
// (hgemm_mfma.hip): slices of 64 k go straight from global memory into a ring of
// STAGES LDS slots, and the MFMAs of one 16-k substep run while the next one's
// fragments are read.  What differs is where rows come from:
//   * kGrouped, kLora: a lane's rows of A are fixed for the whole K loop, so their
//     addresses are formed once (rows[] looked up, clamped) and kept as pointers;
//   * kWgrad: the k are the group's rows.  With rows[] each slice's addresses
//     are formed from indices read by scalar loads one slice ahead; their counter is
//     not the one the ring's waits count;
//   * in a slice that the k range does not fill, chunks outside it are read from a
//     16-byte block of zeros, so nothing past an operand is read and whatever lies
//     between rows cannot reach a sum.  A group of fewer slices than the ring has
//     slots loads such zeros for the missing ones.
// Rows and columns of the tile outside the group or N re-read valid ones; their
// results are not stored.
// Needs: dword-aligned operand rows; K % 8 == 0 for K-contiguous operands and N (M) % 8
// == 0 for the others, so that no 16-byte chunk straddles an edge; 64 (BN) rows of B
// below 2^31 bytes apart.  K may be anything else.
// TB: B stored N x K (not wgrad).  GA, GB: the rows of A, B are looked up (wgrad).
//
// Measured under a tracer, bf16: 32768 gathered rows over 32 unequal groups, 2048 x 2048, B stored K x N: 294 us, 935
// TFLOP/s, matrix cores busy 53% of the cycles (79% in the whole-matrix kernel at 4096^3), the rest
// being part-filled tiles and five rounds of workgroups for four and a half of tiles; weight gradients of 16384
// rows over 32 groups, 2048 x 1024: 114 us, 600 TFLOP/s, 34%: each tile sums some 512 rows between a prologue and an
// epilogue, C's 268 MB are 57 us of a copy's time, and an XCD takes whole groups whatever their length; 4096
// rows with adapters of rank 16, 4096 x 4096: 133 us of tiles (124 at the least), 60%.  Two other tile shapes for
// the weight gradient: 128x256 138, 256x128 133, against 127 for 256x256 before C's stores left the caches.
template <class Cfg, bool BF, int KIND, bool TB, bool GA, bool GB>
__global__ __launch_bounds__(Cfg::NT) void ragged_dma_kernel(RaggedArgs p)
{
    constexpr int BM = Cfg::BM, BN = Cfg::BN, BK = Cfg::BK, S = Cfg::STAGES;
    constexpr bool WG = KIND == kWgrad;
    constexpr bool A_KC = !WG, B_KC = !WG && TB;
    static_assert((A_KC || BM >= 128) && (B_KC || BN >= 128), "MN-contiguous slices need 16 chunks per row");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S * Cfg::STAGE_BYTES];
    const unsigned lds0 = (unsigned)(uintptr_t)lds;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;

    int group = 0, m0, m_end, n0, K, k_lo = 0;   // K: this tile's k range [k_lo, k_lo + K)
    if constexpr (KIND == kGrouped) {
        const int total = count_row_tiles(p.offsets, p.groups, p.R, BM, p.tiles_m);
        if ((long long)blockIdx.x >= (long long)total * p.tiles_n) return;
        int one, tm, tn;
        tile_coords((int)blockIdx.x, 0, 1, total, p.tiles_n, &one, &tm, &tn);
        const RowTile rt = find_row_tile(p.offsets, p.groups, p.R, BM, tm);
        if (rt.group < 0) return;
        group = rt.group;
        m0 = rt.first;
        m_end = rt.end;
        n0 = tn * BN;
        K = p.K;
    } else {
        int tm, tn;
        tile_coords(blockIdx.x, blockIdx.z, gridDim.z, p.tiles_m, p.tiles_n, &group, &tm, &tn);
        m0 = tm * BM;
        m_end = p.M;
        n0 = tn * BN;
        K = p.K;
        if constexpr (WG) {
            int hi;
            group_rows(p.offsets, group, p.R, &k_lo, &hi);
            k_lo = __builtin_amdgcn_readfirstlane(k_lo);
            K = __builtin_amdgcn_readfirstlane(hi - k_lo);
        }
    }
    const int N = p.N;
    const long long lda = p.lda, ldb = p.ldb, ldc = p.ldc;
    float *C = WG ? p.C + (long long)group * p.strideC : p.C;
    const uint16_t *Bg = WG ? p.B : p.B + (long long)group * p.strideB;

    const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;
    const int lr = lane & 31, lk = lane >> 5;
    f32x16 acc[Cfg::FM][Cfg::FN];
#pragma unroll
    for (int i = 0; i < Cfg::FM; ++i)
#pragma unroll
        for (int jj = 0; jj < Cfg::FN; ++jj)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][jj][r] = 0.f;
    const int uwave = __builtin_amdgcn_readfirstlane(wave);
    const bool loader = uwave >= Cfg::NW - Cfg::LW;
    const int lw = loader ? uwave - (Cfg::NW - Cfg::LW) : 0;
    constexpr int A_LOADS = Cfg::A_LOADS, B_LOADS = Cfg::B_LOADS;
    constexpr int LOADS = A_LOADS + B_LOADS;
    const int limA = m_end - m0 < BM ? m_end - m0 : BM, limB = N - n0 < BN ? N - n0 : BN;

    // K-contiguous A: the lane's chunk of each of its rows.
    const uint16_t *rowA[A_KC ? A_LOADS : 1];
    if constexpr (A_KC) {
        constexpr int CPR = Cfg::A_CPR;
#pragma unroll
        for (int i = 0; i < A_LOADS; ++i) {
            const int r = (64 / CPR) * (lw * A_LOADS + i) + lane / CPR;
            int at = m0 + (r < limA ? r : limA - 1);
            if (KIND == kGrouped && p.rowsA) at = p.rowsA[at];
            if (at < 0 || at >= p.a_rows) at = 0;   // (its products are dropped in the epilogue)
            rowA[i] = p.A + (long long)at * lda + 8 * ((lane % CPR) ^ swz_a<CPR>(r));
        }
    }
    // Operands addressed from one base: byte offsets within a slice.
    unsigned offA[A_KC ? 1 : A_LOADS], offB[B_LOADS];
    if constexpr (!A_KC)
#pragma unroll
        for (int i = 0; i < A_LOADS; ++i) offA[i] = dma_offset<false, BM, BK, true>(lw * A_LOADS + i, lane, lda, limA);
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i) offB[i] = dma_offset<B_KC, BN, BK, true>(lw * B_LOADS + i, lane, ldb, limB);
    const long long stepA = BK * lda * 2, stepB = B_KC ? BK * 2 : BK * ldb * 2;
    const char *Ab = reinterpret_cast<const char *>(p.A + (WG ? (long long)k_lo * lda + m0 : 0));
    const char *Bb = reinterpret_cast<const char *>(Bg + (WG ? (long long)k_lo * ldb + n0 : B_KC ? (long long)n0 * ldb : n0));

    // k (of the slice) and column chunk of load g of an MN-contiguous operand.
    auto mn_k = [&](auto r, int g) -> int {
        constexpr int CPR = decltype(r)::value / 8;
        return (64 / CPR) * g + lane / CPR;
    };
    auto mn_col = [&](auto r, int g, int lim) -> int {
        constexpr int CPR = decltype(r)::value / 8;
        const int c = 8 * ((lane % CPR) ^ swz_b(mn_k(r, g)));
        return c < lim ? c : 0;
    };
    // wgrad, rows looked up: the indices of this wave's k rows of one slice, by scalar
    // loads all at once, one slice ahead of their use.  The lane then takes its row's.
    constexpr int RPL_A = 64 / (BM / 8), RPL_B = 64 / (BN / 8);   // k rows per load: 2 or 4
    // (vectors, so that they stay in registers)
    typedef int IdxA __attribute__((ext_vector_type(A_LOADS * RPL_A)));
    typedef int IdxB __attribute__((ext_vector_type(B_LOADS * RPL_B)));
    IdxA idxA = {};
    IdxB idxB = {};
    auto fetch = [&](const int32_t *rows, auto &idx, auto count_c, int kt) __attribute__((always_inline)) {
        constexpr int count = decltype(count_c)::value;
        const int first = kt * BK + lw * count;
        scalar_ints from = (scalar_ints)(const int32_t *)uniform((const char *)(rows + k_lo));
        if (first + count <= K) {
#pragma unroll
            for (int j = 0; j < count; ++j) idx[j] = from[first + j];
        } else {
#pragma unroll
            for (int j = 0; j < count; ++j) idx[j] = from[first + j < K ? first + j : K - 1];
        }
    };
    auto gathered = [&](auto r, const uint16_t *X, int cols0, long long ld, const auto &idx, int i, int x_rows, int kt, int g,
                        int lim) __attribute__((always_inline)) -> const void * {
        constexpr int RPL = 64 / (decltype(r)::value / 8);
        const int sub = lane / (64 / RPL);
        int at = idx[RPL * i];
#pragma unroll
        for (int j = 1; j < RPL; ++j) at = sub == j ? idx[RPL * i + j] : at;
        const bool ok = kt * BK + RPL * g + sub < K && (unsigned)at < (unsigned)x_rows;
        return ok ? (const void *)(X + (long long)at * ld + cols0 + mn_col(r, g, lim)) : (const void *)zero_chunk;
    };
    using RA = std::integral_constant<int, BM>;
    using RB = std::integral_constant<int, BN>;
    auto issue_slice = [&](int kt, int slot) __attribute__((always_inline)) {
        if (!loader) return;
        const unsigned la = __builtin_amdgcn_readfirstlane(lds0 + slot * Cfg::A_BYTES + lw * A_LOADS * 1024);
        const unsigned lb = __builtin_amdgcn_readfirstlane(lds0 + S * Cfg::A_BYTES + slot * Cfg::B_BYTES + lw * B_LOADS * 1024);
        const bool whole = (kt + 1) * BK <= K;
        const char *b = uniform(Bb + (long long)kt * stepB);
        if constexpr (!WG) {
            if (whole) {
#pragma unroll
                for (int i = 0; i < A_LOADS; ++i) dma16_at(rowA[i] + (long long)kt * BK, la + 1024 * i);
#pragma unroll
                for (int i = 0; i < B_LOADS; ++i) dma16(b, offB[i], lb + 1024 * i);
            } else {
                constexpr int CPR = BK / 8;
#pragma unroll
                for (int i = 0; i < A_LOADS; ++i) {
                    const int r = (64 / CPR) * (lw * A_LOADS + i) + lane / CPR;
                    const int k = kt * BK + 8 * ((lane % CPR) ^ swz_a<CPR>(r));
                    dma16_at(k < K ? (const void *)(rowA[i] + (long long)kt * BK) : (const void *)zero_chunk, la + 1024 * i);
                }
#pragma unroll
                for (int i = 0; i < B_LOADS; ++i) {
                    const int g = lw * B_LOADS + i;
                    int k;
                    if constexpr (B_KC) {
                        const int r = (64 / CPR) * g + lane / CPR;
                        k = kt * BK + 8 * ((lane % CPR) ^ swz_a<CPR>(r));
                    } else {
                        k = kt * BK + mn_k(RB{}, g);
                    }
                    dma16_at(k < K ? (const void *)(b + offB[i]) : (const void *)zero_chunk, lb + 1024 * i);
                }
            }
        } else {
            const char *a = Ab + (long long)kt * stepA;
            // without an index array, row r of the group is row k_lo + r, inside the operand
            auto plain = [&](auto r, const char *xb, const unsigned *off, auto loads_c, int x_rows, unsigned dst) __attribute__((always_inline)) {
                constexpr int loads = decltype(loads_c)::value;
                const char *x = uniform(xb);
                if (whole && k_lo + (kt + 1) * BK <= x_rows) {
#pragma unroll
                    for (int i = 0; i < loads; ++i) dma16(x, off[i], dst + 1024 * i);
                } else {
#pragma unroll
                    for (int i = 0; i < loads; ++i) {
                        const int k = kt * BK + mn_k(r, lw * loads + i);
                        dma16_at(k < K && k_lo + k < x_rows ? (const void *)(x + off[i]) : (const void *)zero_chunk, dst + 1024 * i);
                    }
                }
            };
            if constexpr (GA) {
#pragma unroll
                for (int i = 0; i < A_LOADS; ++i)
                    dma16_at(gathered(RA{}, p.A, m0, lda, idxA, i, p.a_rows, kt, lw * A_LOADS + i, limA), la + 1024 * i);
                fetch(p.rowsA, idxA, std::integral_constant<int, A_LOADS * RPL_A>{}, kt + 1);
            } else {
                plain(RA{}, a, offA, std::integral_constant<int, A_LOADS>{}, p.a_rows, la);
            }
            if constexpr (GB) {
#pragma unroll
                for (int i = 0; i < B_LOADS; ++i)
                    dma16_at(gathered(RB{}, p.B, n0, ldb, idxB, i, p.b_rows, kt, lw * B_LOADS + i, limB), lb + 1024 * i);
                fetch(p.rowsB, idxB, std::integral_constant<int, B_LOADS * RPL_B>{}, kt + 1);
            } else {
                plain(RB{}, b, offB, std::integral_constant<int, B_LOADS>{}, p.b_rows, lb);
            }
        }
    };

    constexpr int NS = BK / 16;
    constexpr int NFA = A_KC ? NS : Cfg::FM, NFB = B_KC ? NS : Cfg::FN;
    unsigned fragA[NFA], fragB[NFB];
#pragma unroll
    for (int x = 0; x < NFA; ++x)
        fragA[x] = A_KC ? frag_offset<true, BM, BK>(wm * Cfg::TM, lane, x)
                        : frag_offset<false, BM, BK>(wm * Cfg::TM + 32 * x, lane, 0);
#pragma unroll
    for (int x = 0; x < NFB; ++x)
        fragB[x] = S * Cfg::A_BYTES + (B_KC ? frag_offset<true, BN, BK>(wn * Cfg::TN, lane, x)
                                            : frag_offset<false, BN, BK>(wn * Cfg::TN + 32 * x, lane, 0));
    auto frag = [&](auto kc, auto rr, unsigned base, const unsigned *off, int x, int s) -> half8 {
        constexpr int R = decltype(rr)::value;
        if constexpr (decltype(kc)::value) {
            return *(const lds_half8 *)(uintptr_t)(base + off[s] + x * 32 * BK * 2);
        } else {
            const unsigned at = base + off[x] + 16 * s * R * 2;
            const short4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)at);
            const short4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)(at + 4 * R * 2));
            const short4v both[2] = {lo, hi};
            return __builtin_bit_cast(half8, both);
        }
    };
    half8 fa[2][Cfg::FM], fb[2][Cfg::FN];
    auto read_frags = [&](int slot, int s, half8 *a, half8 *b) {
        const unsigned base_a = lds0 + slot * Cfg::A_BYTES, base_b = lds0 + slot * Cfg::B_BYTES;
#pragma unroll
        for (int i = 0; i < Cfg::FM; ++i) a[i] = frag(std::bool_constant<A_KC>{}, RA{}, base_a, fragA, i, s);
#pragma unroll
        for (int jj = 0; jj < Cfg::FN; ++jj) b[jj] = frag(std::bool_constant<B_KC>{}, RB{}, base_b, fragB, jj, s);
    };
    auto mfmas = [&](const half8 *a, const half8 *b) {
#pragma unroll
        for (int i = 0; i < Cfg::FM; ++i)
#pragma unroll
            for (int jj = 0; jj < Cfg::FN; ++jj) acc[i][jj] = mfma16<BF>(b[jj], a[i], acc[i][jj]);
    };
    auto lds_barrier = [&]() {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    };
    auto interleave = [&]() {
#pragma unroll
        for (int i = 0; i < Cfg::FM * Cfg::FN; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
        }
    };
    const bool late = Cfg::STAGGER && uwave >= Cfg::NW / 2;
    auto step_in = [&](int t, auto pending, auto refill, bool late_refill, auto slot_c, auto works) __attribute__((always_inline)) {
        constexpr bool WORKS = decltype(works)::value;   // false: this wave only loads its share
        constexpr int SC = decltype(slot_c)::value;   // < 0: not known at compile time
        const int slot = SC >= 0 ? SC : t % S;
        const int next = SC >= 0 ? (SC + 1) % S : (t + 1) % S;
        const int prev = SC >= 0 ? (SC + S - 1) % S : (t - 1 + S) % S;
#pragma unroll
        for (int sub = 0; sub < NS; ++sub) {
            const int cur = sub & 1, nxt = cur ^ 1;
            if (sub + 1 < NS) {
                if constexpr (WORKS) read_frags(slot, sub + 1, fa[nxt], fb[nxt]);
                if (Cfg::STAGGER && sub == NS - 2 && late && late_refill) issue_slice(t - 1 + S, prev);
            } else {
                wait_vmcnt<LOADS * decltype(pending)::value>();
                __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave's slice-t reads are done
                lds_barrier();
                if (decltype(refill)::value && !late) issue_slice(t + S, slot);
                if constexpr (WORKS) read_frags(next, 0, fa[nxt], fb[nxt]);
            }
            if constexpr (WORKS) {
                mfmas(fa[cur], fb[cur]);
                interleave();
            }
        }
    };
    auto step = [&](int t, auto pending, auto refill, bool late_refill, auto works) __attribute__((always_inline)) {
        step_in(t, pending, refill, late_refill, std::integral_constant<int, -1>{}, works);
    };

    if (K > 0) {   // (uniform)
        // slices past the last are zeros: at least as many as the ring has slots
        const int slices = (K + BK - 1) / BK, nk = slices < S ? S : slices;
        if constexpr (WG) {
            if constexpr (GA) fetch(p.rowsA, idxA, std::integral_constant<int, A_LOADS * RPL_A>{}, 0);
            if constexpr (GB) fetch(p.rowsB, idxB, std::integral_constant<int, B_LOADS * RPL_B>{}, 0);
        }
#pragma unroll
        for (int st = 0; st < S; ++st) issue_slice(st, st);
        auto loop = [&](auto works) __attribute__((always_inline)) {
            constexpr bool WORKS = decltype(works)::value;
            wait_vmcnt<LOADS * (S - 1)>();
            lds_barrier();
            if constexpr (WORKS) read_frags(0, 0, fa[0], fb[0]);
            int t = 0;
            constexpr bool UNROLL = WORKS && BM >= 128 && !B_KC;   // (as in the whole-matrix kernel)
            for (; UNROLL && t + S - 1 + S < nk; t += S) {
                [&]<int... I>(std::integer_sequence<int, I...>) {
                    (step_in(t + I, std::integral_constant<int, S - 2>{}, std::true_type{}, t + I >= 1,
                             std::integral_constant<int, I>{}, works),
                     ...);
                }(std::make_integer_sequence<int, S>{});
            }
            for (; t + S < nk; ++t) step(t, std::integral_constant<int, S - 2>{}, std::true_type{}, t >= 1, works);
            const int t0 = nk - S;
            step(t0, std::integral_constant<int, S - 2>{}, std::false_type{}, t0 >= 1, works);
            if constexpr (S >= 3) step(t0 + 1, std::integral_constant<int, S - 3>{}, std::false_type{}, false, works);
            if constexpr (S >= 4) step(t0 + 2, std::integral_constant<int, S - 4>{}, std::false_type{}, false, works);
            if constexpr (WORKS) {
                const int slot = (nk - 1) % S;
#pragma unroll
                for (int sub = 0; sub < NS; ++sub) {
                    const int cur = sub & 1, nxt = cur ^ 1;
                    if (sub + 1 < NS) read_frags(slot, sub + 1, fa[nxt], fb[nxt]);
                    mfmas(fa[cur], fb[cur]);
                }
            }
        };
        // A wave whose rows all lie past the group's end only loads: the matrix cores
        // of a part-filled tile are left to the waves beside it on its SIMD.
        if (KIND == kGrouped && m0 + (uwave / Cfg::WN) * Cfg::TM >= m_end)
            loop(std::false_type{});
        else
            loop(std::true_type{});
    }

    // Epilogue by rows: straight from the accumulators a store instruction would write
    // 32 bytes of each of 32 rows; here each wave passes 32 rows at a time through its
    // part of the ring (free once every wave is past the barrier) and writes whole row
    // segments of its tile, TN * 4 bytes each.  16-byte chunk c of staged row r sits at
    // chunk c ^ (r % LPR), which keeps both directions off each other's banks.
    // past_cache: stores that leave the caches to A and B (32768 x 2048 x 2048 over 32 groups 332 -> 305 us, weight
    // gradients of 32 x 2048 x 1024 128 -> 108), where C is not kept for its reader anyway.
    const float alpha = p.alpha, beta = p.beta;
    constexpr int LPR = Cfg::TN / 4, RPI = 64 / LPR, NQ = 32 / RPI;
    static_assert(Cfg::NW * 32 * Cfg::TN * 4 <= S * Cfg::STAGE_BYTES, "staging area exceeds the ring");
    const unsigned stage = lds0 + wave * 32 * Cfg::TN * 4;
    lds_barrier();
    // The adapters of 32 rows: for each distinct one, LB's columns against the parts of its
    // rows (zeros for the others), added by the rows' factors to its own rows.  Here, where
    // the K loop's registers are free: before the loop the accumulators spilled (4096^3, bf16:
    // 154 us, here 134).
    const AdapterArgs &ad = p.ad;
    int aid[Cfg::FM];
    if constexpr (KIND == kLora)
#pragma unroll
        for (int i = 0; i < Cfg::FM; ++i)
            aid[i] = ad.adapters > 0 ? adapter_of(ad.ids, ad.adapters, m0 + wm * Cfg::TM + 32 * i + lr, p.M) : -1;
    auto add_adapters = [&](int first, int mine, f32x16 *sums) __attribute__((always_inline)) {
        const long long row = first + lr;
        const float f = mine >= 0 ? ad.factor[row] : 0.f;
        int todo = mine;
        for (uint64_t left = __ballot(todo >= 0); left; left = __ballot(todo >= 0)) {
            const int a = __builtin_amdgcn_readlane(todo, __builtin_ctzll(left));
            const int ra = rank_of(ad.ranks, ad.rank, a);
            const uint16_t *lb = ad.LB + (long long)a * ad.strideLB;
            f32x16 add[Cfg::FN];
#pragma unroll
            for (int jj = 0; jj < Cfg::FN; ++jj)
#pragma unroll
                for (int r = 0; r < 16; ++r) add[jj][r] = 0.f;
            for (int k0 = 0; k0 < ra; k0 += 16) {
                const int kq = k0 + 8 * lk;
                half8 ta[kParts], tb[Cfg::FN];
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    ta[part] = half8{};
                    if (mine == a)
                        ta[part] = *reinterpret_cast<const half8 *>(ad.parts + ((long long)part * p.M + row) * ad.pitch + kq);
                }
#pragma unroll
                for (int jj = 0; jj < Cfg::FN; ++jj) {
                    const int c = n0 + wn * Cfg::TN + 32 * jj + lr;
                    tb[jj] = load8_any(lb + (long long)(c < N ? c : N - 1) * ad.ldlb + kq, ra - kq);
                }
                if constexpr (BF) {
#pragma unroll
                    for (int part = 0; part < kParts; ++part)
#pragma unroll
                        for (int jj = 0; jj < Cfg::FN; ++jj) add[jj] = mfma16<BF>(tb[jj], ta[part], add[jj]);
                } else {
                    // (the last parts first, each sum scaled down to the part before it)
#pragma unroll
                    for (int jj = 0; jj < Cfg::FN; ++jj) {
                        f32x16 low = {};
#pragma unroll
                        for (int part = kParts - 1; part > 0; --part) {
                            low = mfma16<BF>(tb[jj], ta[part], low);
#pragma unroll
                            for (int r = 0; r < 16; ++r) low[r] *= kPartStep<BF>;
                        }
#pragma unroll
                        for (int r = 0; r < 16; ++r) add[jj][r] += low[r];
                        add[jj] = mfma16<BF>(tb[jj], ta[0], add[jj]);
                    }
                }
            }
            // (a lane holds values of its own row alone: another adapter's infinities stay out)
            if (todo == a) {
                todo = -1;
#pragma unroll
                for (int jj = 0; jj < Cfg::FN; ++jj)
#pragma unroll
                    for (int r = 0; r < 16; ++r) sums[jj][r] = __builtin_fmaf(f, add[jj][r], sums[jj][r]);
            }
        }
    };
    const int er = lane / LPR, ec = lane % LPR;   // row and chunk within RPI rows
    const int col = n0 + wn * Cfg::TN + 4 * ec;
#pragma unroll
    for (int i = 0; i < Cfg::FM; ++i) {
        const int first = m0 + wm * Cfg::TM + 32 * i;
        if (first >= m_end) break;   // (uniform)
        if constexpr (KIND == kLora) add_adapters(first, aid[i], acc[i]);
#pragma unroll
        for (int jj = 0; jj < Cfg::FN; ++jj)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4_t v = {acc[i][jj][4 * g], acc[i][jj][4 * g + 1], acc[i][jj][4 * g + 2], acc[i][jj][4 * g + 3]};
                *(lds_f32x4 *)(uintptr_t)(stage + lr * Cfg::TN * 4 + (((8 * jj + 2 * g + lk) ^ (lr & (LPR - 1))) * 16)) = v;
            }
        // a wave's LDS accesses complete in order; this orders the compiler's too
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        f32x4_t v[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int r = q * RPI + er;
            v[q] = *(const lds_f32x4 *)(uintptr_t)(stage + r * Cfg::TN * 4 + ((ec ^ (r & (LPR - 1))) * 16));
        }
        if constexpr (KIND == kGrouped) {
            // a row index outside A: a row of zeros
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int row = first + q * RPI + er;
                const int at = p.rowsA && row < m_end ? p.rowsA[row] : row;
                if (row < m_end && (unsigned)at >= (unsigned)p.a_rows) v[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
        }
        if (beta != 0.f) {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                store_row4<true, true>(C, ldc, first + q * RPI + er, col, v[q], alpha, beta, m_end, N);
        } else if (first + 32 <= m_end && n0 + BN <= N && p.past_cache) {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                __builtin_nontemporal_store(alpha * v[q], reinterpret_cast<f32x4_g *>(C + (long long)(first + q * RPI + er) * ldc + col));
        } else if (first + 32 <= m_end && n0 + BN <= N) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) store_row4<false, false>(C, ldc, first + q * RPI + er, col, v[q], alpha, beta, m_end, N);
        } else {
#pragma unroll
            for (int q = 0; q < NQ; ++q) store_row4<true, false>(C, ldc, first + q * RPI + er, col, v[q], alpha, beta, m_end, N);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// Eight consecutive values from column c of a row, wherever the row starts, in two
// halves: the loads (words), whose results nothing touches while other loads are on
// their way, and the values (value8).  The words are the five dwords from the one that
// holds the first value on; past the last that holds one of the row's `cols` columns,
// that one again, so no load leaves the words the row occupies.  whole (the same in all
// lanes): no chunk of this slice ends before its eighth column, so four of the dwords are
// one load.  row == nullptr: zeros.
// The pointers are named global: loads that may go to LDS too (flat ones, what a pointer
// made of a number gives) count as LDS accesses, and every barrier would wait for them.
struct Words {
    unsigned w[5], shift;
};
typedef const __attribute__((address_space(1))) unsigned *global_words;
typedef const __attribute__((address_space(1))) u32x4_g *global_chunk;
__device__ __forceinline__ void words(const uint16_t *row, long long c, long long cols, bool whole, Words *out)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(row + c);
    if (whole) {
        const unsigned odd = row ? (unsigned)(p & 2) >> 1 : 0u;
        const global_words at = (global_words)(row ? p & ~(uintptr_t)3 : reinterpret_cast<uintptr_t>(zero_chunk));
        const u32x4 v = *(global_chunk)at;
#pragma unroll
        for (int i = 0; i < 4; ++i) out->w[i] = v[i];
        out->w[4] = at[3 + odd];
        out->shift = 16 * odd;
        return;
    }
    const int valid = row == nullptr || c >= cols ? 0 : cols - c < 8 ? (int)(cols - c) : 8;
    const unsigned odd = valid > 0 ? (unsigned)(p & 2) >> 1 : 0u;
    const int last = valid > 0 ? ((int)odd + valid - 1) >> 1 : 0;
    const global_words at = (global_words)(valid > 0 ? p & ~(uintptr_t)3 : reinterpret_cast<uintptr_t>(zero_chunk));
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
// The kernel for every shape, stride and alignment: tiles of four waves,
// operand slices of 64 k read into registers two slices ahead and written to a
// double-buffered LDS (the register-staged scheme of hgemm_mfma.hip with rows
// addressed one by one).  kWgrad: both operands are stored with the k (the group's
// rows) outermost.  kLora: workgroup blockIdx.y takes its share of the slices, and
// with several the plain sums go to C + blockIdx.y * strideC.
// 64x64 tiles, or 128x128 (half the loads per product, the launchers say where).
// Bound by its loads through registers, two or five a chunk against one direct load, and at small sizes by one
// workgroup's chain of slices: fp16, 1001 rows over 5 groups, 777 x 513: 10.8 us (its bytes are 1.6 us of a copy);
// weight gradients of 11725 rows over 8 groups, 640 x 913: 68 us, 201 TFLOP/s.  Registers are held to what
// four waves per SIMD leave (wgrad: three, its LDS allows no more), or two with 128x128 tiles: else the
// sums were copied between register files in every slice.
template <class Cfg, bool BF, int KIND, bool TB>
__global__ __launch_bounds__(256, Cfg::BM == 64 ? (KIND == kWgrad ? 3 : 4) : 2) void ragged_any_kernel(RaggedArgs p)
{
    constexpr bool WG = KIND == kWgrad;
    constexpr int FM = Cfg::FM, FN = Cfg::FN;
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
    } else if constexpr (KIND == kLora) {
        int one, tm, tn;
        tile_coords((int)blockIdx.x, 0, 1, p.tiles_m, p.tiles_n, &one, &tm, &tn);
        group = 0;
        m0 = tm * BM;
        m_end = p.M;
        n0 = tn * BN;
        K = p.K;
    } else {
        const int total = count_row_tiles(p.offsets, p.groups, p.R, BM, p.tiles_m);
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
    float *C = p.C + (WG ? (long long)group : KIND == kLora ? (long long)blockIdx.y : 0) * p.strideC;
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
            arow[i] = row_of(p.A, lda, KIND == kLora ? nullptr : p.rowsA, m0 + (i * NT + tid) / TileA::CPR, m_end, p.a_rows);
    }
    // wgrad: the rows of the slice to load next, looked up a step before their loads and ahead of
    // the loads of that step, so that waiting for an index does not wait for those
    int na[TileA::LOADS], nb[TileB::LOADS];
    auto look_up = [&](int k0) __attribute__((always_inline)) {
        if constexpr (WG) {
            const int end = k_lo + K;   // (K > 0)
#pragma unroll
            for (int i = 0; i < TileA::LOADS; ++i) {
                const int r = k_lo + k0 + (i * NT + tid) / TileA::CPR, in = r < end ? r : end - 1;
                const int at = p.rowsA ? p.rowsA[in] : in;
                na[i] = r < end ? at : -1;
            }
#pragma unroll
            for (int i = 0; i < TileB::LOADS; ++i) {
                const int r = k_lo + k0 + (i * NT + tid) / TileB::CPR, in = r < end ? r : end - 1;
                const int at = p.rowsB ? p.rowsB[in] : in;
                nb[i] = r < end ? at : -1;
            }
        }
    };
    // whole: it is known that no chunk of the slice ends before its eighth column
    auto load_tiles = [&](auto whole_c, int k0, Words *ra, Words *rb) __attribute__((always_inline)) {
        constexpr bool WHOLE = decltype(whole_c)::value;
        int ia[TileA::LOADS], ib[TileB::LOADS];
        if constexpr (WG) {
#pragma unroll
            for (int i = 0; i < TileA::LOADS; ++i) ia[i] = na[i];
#pragma unroll
            for (int i = 0; i < TileB::LOADS; ++i) ib[i] = nb[i];
            look_up(k0 + BK);
        }
#pragma unroll
        for (int i = 0; i < TileA::LOADS; ++i) {
            const int id = i * NT + tid;
            const int c = (id % TileA::CPR) * 8;
            if constexpr (WG)
                words((unsigned)ia[i] < (unsigned)p.a_rows ? p.A + (long long)ia[i] * lda : nullptr, m0 + c, p.M, WHOLE || m0 + BM <= p.M, &ra[i]);
            else
                words(arow[i], k0 + c, K, WHOLE || k0 + BK <= K, &ra[i]);
        }
#pragma unroll
        for (int i = 0; i < TileB::LOADS; ++i) {
            const int id = i * NT + tid;
            const int r = id / TileB::CPR, c = (id % TileB::CPR) * 8;
            if constexpr (WG)
                words((unsigned)ib[i] < (unsigned)p.b_rows ? p.B + (long long)ib[i] * ldb : nullptr, n0 + c, N, WHOLE || n0 + BN <= N, &rb[i]);
            else if constexpr (TB)
                words(n0 + r < N ? B + (long long)(n0 + r) * ldb : nullptr, k0 + c, K, WHOLE || k0 + BK <= K, &rb[i]);
            else
                words(k0 + r < K ? B + (long long)(k0 + r) * ldb : nullptr, n0 + c, N, WHOLE || n0 + BN <= N, &rb[i]);
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
    auto store_tiles = [&](auto whole_c, int buf, int k0, const Words *ra, const Words *rb) __attribute__((always_inline)) {
        auto value = [&](const Words &x, long long c, long long cols) __attribute__((always_inline)) {
            return value8(x, c, decltype(whole_c)::value ? c + 8 : cols);
        };
        uint16_t *la = lds + buf * BUF_HALVES;
        uint16_t *lb = la + TileA::HALVES;
#pragma unroll
        for (int i = 0; i < TileA::LOADS; ++i) {
            const int c = (i * NT + tid) % TileA::CPR * 8;
            store_one(TileA{}, la, i, WG ? value(ra[i], m0 + c, p.M) : value(ra[i], k0 + c, K));
        }
#pragma unroll
        for (int i = 0; i < TileB::LOADS; ++i) {
            const int c = (i * NT + tid) % TileB::CPR * 8;
            store_one(TileB{}, lb, i, !WG && TB ? value(rb[i], k0 + c, K) : value(rb[i], n0 + c, N));
        }
    };
    const int wave = tid >> 6, lane = tid & 63;
    const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;
    const int lr = lane & 31, lk = lane >> 5;
    const int q = lane >> 4, j = lane & 15;
    const int tr_row = 8 * (q >> 1) + (j >> 2);
    const int tr_col = 16 * (q & 1) + 4 * (j & 3);
    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int x = 0; x < FN; ++x)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][x][r] = 0.f;
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
    // this workgroup's slices: all, or its share
    const int slices = (K + BK - 1) / BK;
    const int parts = KIND == kLora ? (int)gridDim.y : 1, part = KIND == kLora ? (int)blockIdx.y : 0;
    const int s0 = (int)((long long)slices * part / parts), nk = (int)((long long)slices * (part + 1) / parts);
    auto step = [&](auto whole_c, bool load, int t, Words *a, Words *b) __attribute__((always_inline)) {
        const int buf = (t - s0) & 1;
        store_tiles(whole_c, buf, t * BK, a, b);
        if (load) load_tiles(whole_c, (t + AHEAD) * BK, a, b);
        // one barrier a step: the buffer written next was last read in the step
        // before this one, which every wave has left when it passes here
        __syncthreads();
        const uint16_t *la = lds + buf * BUF_HALVES;
        const uint16_t *lb = la + TileA::HALVES;
#pragma unroll
        for (int s = 0; s < BK / 16; ++s) {
            half8 fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) fa[i] = read_frag(TileA{}, la, wm * Cfg::TM + 32 * i, s);
#pragma unroll
            for (int x = 0; x < FN; ++x) fb[x] = read_frag(TileB{}, lb, wn * Cfg::TN + 32 * x, s);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int x = 0; x < FN; ++x) acc[i][x] = mfma16<BF>(fb[x], fa[i], acc[i][x]);
        }
    };
    // Whole slices first, a loop whose steps all issue the same loads without a branch, so that the
    // waits for a slice's words leave the next slice's on their way; then the others.
    const int wholes = WG || (!TB && n0 + BN > N) ? s0 : K / BK > nk ? nk : K / BK;
    int t = s0;
    if (s0 < nk) look_up(s0 * BK);
    if (!WG && s0 + 2 * AHEAD <= wholes) {
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) load_tiles(std::true_type{}, (s0 + d) * BK, ra[d], rb[d]);
        for (; t + 2 * AHEAD <= wholes; t += AHEAD)
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) step(std::true_type{}, true, t + d, ra[d], rb[d]);
    } else {
#pragma unroll
        for (int d = 0; d < AHEAD; ++d)
            if (s0 + d < nk) load_tiles(std::false_type{}, (s0 + d) * BK, ra[d], rb[d]);
    }
    for (; t < nk; t += AHEAD)
#pragma unroll
        for (int d = 0; d < AHEAD; ++d)
            if (t + d < nk) step(std::false_type{}, t + d + AHEAD < nk, t + d, ra[d], rb[d]);
    const float alpha = parts > 1 ? 1.f : p.alpha, beta = parts > 1 ? 0.f : p.beta;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const long long row = m0 + wm * Cfg::TM + 32 * i + lr;
        // a row index outside A: a row of zeros, also where the group's weights hold infinities
        const int at = KIND == kGrouped && p.rowsA && row < m_end ? p.rowsA[row] : (int)row;
        const bool none = KIND == kGrouped && (unsigned)at >= (unsigned)p.a_rows;
#pragma unroll
        for (int x = 0; x < FN; ++x)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const long long col = n0 + wn * Cfg::TN + 32 * x + 8 * g + 4 * lk;
                f32x4_t v = {acc[i][x][4 * g], acc[i][x][4 * g + 1], acc[i][x][4 * g + 2], acc[i][x][4 * g + 3]};
                if (none) v = f32x4_t{0.f, 0.f, 0.f, 0.f};
                if (beta != 0.f)
                    store_row4<true, true>(C, ldc, row, col, v, alpha, beta, m_end, N);
                else
                    store_row4<true, false>(C, ldc, row, col, v, alpha, beta, m_end, N);
            }
    }
}

// ---------------------------------------------------------------------------
// Few rows: the weights are read once and multiplied by up to 32 FM rows, so the
// time is that of streaming them.  A workgroup takes 32 FN columns; its NW waves
// (and, lora, the gridDim.y workgroups of a strip) share the slices of 64 k in
// turn.  Every wave has a ring of S slots of its own that only it loads and reads:
// no barrier until the end, and S slices of loads in flight per wave.  The waves'
// sums are added in wave order.
//   kGrouped: C as in ragged_dma_kernel.  kLora: the plain sum of the
//   workgroup's slices goes to C + blockIdx.y * strideC (workspace), lora's last
//   kernel adds them up.
// Needs what ragged_dma_kernel needs.
// Bound by reading the weights: 64 groups of 2048 x 1024, 2 rows each, bf16, N x K: 268 MB in 35 us back to back (a part of
// the weights stays in the 256 MiB memory-side cache from one call to the next) and 46 with other weights
// each call, 5.9 TB/s, where a copy reaches 4.7 (it writes half of what it moves).
constexpr int kStreamBK = 64;

// XOR of an MN-contiguous slice's chunks in row k, rows of CPR chunks: the four rows
// that a transposed read touches fall on different banks.
template <int CPR>
__device__ __forceinline__ int swz_n(int k)
{
    return CPR == 8 ? 2 * (k & 3) : (k & 2);
}

template <int FM_, int FN_, int S_, int NW_>
struct StreamCfg {
    static constexpr int FM = FM_, FN = FN_, S = S_, NW = NW_;
    static constexpr int BM = 32 * FM, BN = 32 * FN, BK = kStreamBK, NT = 64 * NW;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE = A_BYTES + B_BYTES;
    static constexpr int A_LOADS = A_BYTES / 1024, B_LOADS = B_BYTES / 1024, LOADS = A_LOADS + B_LOADS;
    static constexpr int LDS = NW * S * STAGE;
    static_assert(FN == 1 || FN == 2, "rows of four or eight chunks");
    static_assert(NW * BM * BN * 4 <= LDS, "the waves' sums fit the rings");
    static_assert(LDS <= 160 * 1024 && LOADS * S < 64, "LDS, outstanding loads");
};

template <class Cfg, bool BF, int KIND, bool TB>
__device__ __forceinline__ void stream_tile(const RaggedArgs &p, unsigned char *lds, int block, int part, int parts)
{
    constexpr int FM = Cfg::FM, FN = Cfg::FN, S = Cfg::S, NW = Cfg::NW, BM = Cfg::BM, BN = Cfg::BN, BK = Cfg::BK;
    constexpr int A_LOADS = Cfg::A_LOADS, B_LOADS = Cfg::B_LOADS, LOADS = Cfg::LOADS;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int uwave = __builtin_amdgcn_readfirstlane(wave);
    const unsigned lds0 = (unsigned)(uintptr_t)lds;

    int group = 0, m0, m_end, n0;
    {
        int one, tm, tn;
        if constexpr (KIND == kGrouped) {
            const int total = count_row_tiles(p.offsets, p.groups, p.R, BM, p.tiles_m);
            if ((long long)block >= (long long)total * p.tiles_n) return;
            tile_coords(block, 0, 1, total, p.tiles_n, &one, &tm, &tn);
            const RowTile rt = find_row_tile(p.offsets, p.groups, p.R, BM, tm);
            if (rt.group < 0) return;
            group = rt.group;
            m0 = rt.first;
            m_end = rt.end;
        } else {
            tile_coords(block, 0, 1, p.tiles_m, p.tiles_n, &one, &tm, &tn);
            m0 = tm * BM;
            m_end = p.M;
        }
        n0 = tn * BN;
    }
    const int N = p.N, K = p.K;
    const long long lda = p.lda, ldb = p.ldb;
    const uint16_t *Bg = p.B + (long long)group * p.strideB;
    const int limA = m_end - m0 < BM ? m_end - m0 : BM, limB = N - n0 < BN ? N - n0 : BN;

    // chunk addresses of slice 0
    const uint16_t *rowA[A_LOADS];
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) {
        const int r = 8 * i + lane / 8;
        int at = m0 + (r < limA ? r : limA - 1);
        if (KIND == kGrouped && p.rowsA) at = p.rowsA[at];
        if ((unsigned)at >= (unsigned)p.a_rows) at = 0;   // (its products are dropped at the end)
        rowA[i] = p.A + (long long)at * lda + 8 * ((lane % 8) ^ swz_a<8>(r));
    }
    constexpr int BCPR = BN / 8, BRPL = 64 / BCPR;   // MN-contiguous B: chunks per k row, k rows per load
    unsigned offB[B_LOADS];
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i) {
        if constexpr (TB) {
            const int r = 8 * i + lane / 8;
            offB[i] = (unsigned)((r < limB ? r : limB - 1) * ldb + 8 * ((lane % 8) ^ swz_a<8>(r))) * 2u;
        } else {
            const int k = BRPL * i + lane / BCPR;
            int c = 8 * ((lane % BCPR) ^ swz_n<BCPR>(k));
            if (c >= limB) c = 0;
            offB[i] = (unsigned)(k * ldb + c) * 2u;
        }
    }
    const char *Bb = reinterpret_cast<const char *>(Bg + (TB ? (long long)n0 * ldb : n0));
    const long long stepB = TB ? BK * 2 : BK * ldb * 2;
    const unsigned ring = lds0 + uwave * S * Cfg::STAGE;
    auto issue = [&](int s, int slot) __attribute__((always_inline)) {
        const unsigned la = ring + slot * Cfg::STAGE, lb = la + Cfg::A_BYTES;
        const char *b = uniform(Bb + (long long)s * stepB);
        if ((s + 1) * BK <= K) {
#pragma unroll
            for (int i = 0; i < B_LOADS; ++i) dma16(b, offB[i], lb + 1024 * i);
#pragma unroll
            for (int i = 0; i < A_LOADS; ++i) dma16_at(rowA[i] + (long long)s * BK, la + 1024 * i);
        } else {
#pragma unroll
            for (int i = 0; i < B_LOADS; ++i) {
                const int k = s * BK + (TB ? 8 * ((lane % 8) ^ swz_a<8>(8 * i + lane / 8)) : BRPL * i + lane / BCPR);
                dma16_at(k < K ? (const void *)(b + offB[i]) : (const void *)zero_chunk, lb + 1024 * i);
            }
#pragma unroll
            for (int i = 0; i < A_LOADS; ++i) {
                const int k = s * BK + 8 * ((lane % 8) ^ swz_a<8>(8 * i + lane / 8));
                dma16_at(k < K ? (const void *)(rowA[i] + (long long)s * BK) : (const void *)zero_chunk, la + 1024 * i);
            }
        }
    };
    // fragment addresses within a slot (see frag_offset; rows 32 apart per block)
    const int lr = lane & 31, lk = lane >> 5, q = lane >> 4, j = lane & 15;
    auto kc_frag = [&](unsigned base, int x, int s) -> half8 {
        return *(const lds_half8 *)(uintptr_t)(base + (32 * x + lr) * BK * 2 + 16 * ((2 * s + lk) ^ swz_a<8>(lr)));
    };
    auto mn_frag = [&](unsigned base, int x, int s) -> half8 {
        const int k = 16 * s + 8 * (q >> 1) + (j >> 2), n = 32 * x + 16 * (q & 1) + 4 * (j & 3);
        const unsigned at = base + k * BN * 2 + 16 * ((n >> 3) ^ swz_n<BCPR>(k)) + 2 * (n & 7);
        const short4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)at);
        const short4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)(at + 4 * BN * 2));
        const short4v both[2] = {lo, hi};
        return __builtin_bit_cast(half8, both);
    };

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int x = 0; x < FN; ++x)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][x][r] = 0.f;

    // this wave's slices: first, first + turn, ...
    const int slices = (K + BK - 1) / BK, first = part * NW + uwave, turn = parts * NW;
    const int ns = slices > first ? (slices - first + turn - 1) / turn : 0;
#pragma unroll
    for (int i = 0; i < S; ++i)
        if (i < ns) issue(first + i * turn, i);
    auto compute = [&](int slot, bool refill, int s) __attribute__((always_inline)) {
        const unsigned la = ring + slot * Cfg::STAGE, lb = la + Cfg::A_BYTES;
        half8 fa[4][FM], fb[4][FN];
#pragma unroll
        for (int ss = 0; ss < 4; ++ss) {
#pragma unroll
            for (int i = 0; i < FM; ++i) fa[ss][i] = kc_frag(la, i, ss);
#pragma unroll
            for (int x = 0; x < FN; ++x) fb[ss][x] = TB ? kc_frag(lb, x, ss) : mn_frag(lb, x, ss);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read: it may be loaded again
        if (refill) issue(s, slot);
#pragma unroll
        for (int ss = 0; ss < 4; ++ss)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int x = 0; x < FN; ++x) acc[i][x] = mfma16<BF>(fb[ss][x], fa[ss][i], acc[i][x]);
    };
    int i = 0, slot = 0;
    for (; i + S < ns; ++i) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS * (S - 1)) : "memory");
        compute(slot, true, first + (i + S) * turn);
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    for (; i < ns; ++i) {   // the last slices: everything has been issued
        const int left = ns - 1 - i;
        if (S > 2 && left >= 2)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S > 2 ? LOADS * 2 : 0) : "memory");
        else if (left == 1)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        compute(slot, false, 0);
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    static_assert(S <= 3, "the last slices' waits");

    // the waves' sums, 16-byte chunk c of row r at chunk c ^ (r % CH), added in wave order
    constexpr int CH = BN / 4;   // chunks per row: 8 or 16
    __syncthreads();             // every wave has left its ring
#pragma unroll
    for (int i2 = 0; i2 < FM; ++i2)
#pragma unroll
        for (int x = 0; x < FN; ++x)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int r = 32 * i2 + lr, c = 8 * x + 2 * g + lk;
                const f32x4_t v = {acc[i2][x][4 * g], acc[i2][x][4 * g + 1], acc[i2][x][4 * g + 2], acc[i2][x][4 * g + 3]};
                *(lds_f32x4 *)(uintptr_t)(lds0 + wave * BM * BN * 4 + r * BN * 4 + ((c ^ (r & (CH - 1))) * 16)) = v;
            }
    __syncthreads();
    float *C = KIND == kLora ? p.C + (long long)part * p.strideC : p.C;
    for (int e = tid; e < limA * CH; e += Cfg::NT) {
        const int r = e / CH, c = e % CH;
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w)
            v += *(const lds_f32x4 *)(uintptr_t)(lds0 + w * BM * BN * 4 + r * BN * 4 + ((c ^ (r & (CH - 1))) * 16));
        const int row = m0 + r;
        if constexpr (KIND == kGrouped) {
            const int at = p.rowsA ? p.rowsA[row] : row;
            if ((unsigned)at >= (unsigned)p.a_rows) v = f32x4_t{0.f, 0.f, 0.f, 0.f};
            if (p.beta != 0.f)
                store_row4<true, true>(C, p.ldc, row, n0 + 4 * c, v, p.alpha, p.beta, m_end, N);
            else
                store_row4<true, false>(C, p.ldc, row, n0 + 4 * c, v, p.alpha, p.beta, m_end, N);
        } else {
            store_row4<true, false>(C, p.ldc, row, n0 + 4 * c, v, 1.f, 0.f, m_end, N);
        }
    }
}

using Ragged256 = HgDmaCfg<256, 256, 2, 2, 4, 64>;
using Ragged128 = HgDmaCfg<128, 128, 4, 2, 4, 64>;
using Ragged64 = HgDmaCfg<64, 128, 4, 2, 4, 64>;   // K-contiguous A alone

}  // namespace
}  // namespace mi355gemm
