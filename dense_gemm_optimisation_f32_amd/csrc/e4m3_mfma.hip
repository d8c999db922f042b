// e4m3_mfma.hip -- products of 8-bit floating-point operands with a scale for each block
// of 128 k, fp32 accumulation and C:
//   C[r,:] = alpha A[rows[r],:] B_g^T + beta C[r,:],  offsets[g] <= r < offsets[g+1]
// for one group (a plain product) or ragged groups of rows.  Both operands are stored
// with k contiguous.  Within a block of 128 k the matrix cores sum exact products in
// fp32; each block's sum p then enters the result by
//   acc <- fma(sa[kb, row] * sb[kb, col], p, acc).
// n additions of one sign are off by up to n/2 roundings of 2^-24, 8e-6 of the sum for 256: after that many acc is added to a
// sum of twice 32 bits and starts again (TwoSum below; K of 32768 and less needs none).
//
// The values go to the matrix cores as fp16, which holds every e4m3 value.  Their own 8-bit op
// has twice the rate, but it adds eight products at a time and keeps 14 bits below the largest of the
// eight: C came out 1.5e-5 of its norm off and single entries 3e-5 of the sum of their terms, where fp32
// sums are held to 1e-5 (and reach 1e-6 here).
#include "e4m3_internal.h"
#include "ragged_dma.h"

#include <cmath>

namespace mi355gemm {
namespace {

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
    bool past_cache;          // C is larger than what the memory-side cache keeps of it
};

// A sum in twice 32 bits: `hi` rounded to the nearest, and in `lo` what those roundings left.
constexpr int kChain = 256;   // additions in 32 bits at most
template <class V>            // of floats
struct TwoSum {
    V hi = {}, lo = {};
    // acc is added, and is zero then
    __device__ __forceinline__ void take(V &acc)
    {
#pragma unroll
        for (int r = 0; r < (int)(sizeof(V) / 4); ++r) {
            const float s = hi[r] + acc[r], back = s - hi[r];
            lo[r] += (hi[r] - (s - back)) + (acc[r] - back);
            hi[r] = s;
            acc[r] = 0.f;
        }
    }
    // the sum (one that has left the range has nothing to be corrected)
    __device__ __forceinline__ V value() const
    {
        V v;
#pragma unroll
        for (int r = 0; r < (int)(sizeof(V) / 4); ++r) v[r] = hi[r] + (fabsf(hi[r]) < INFINITY ? lo[r] : 0.f);
        return v;
    }
};
// Additions in one chain where `chains` share the slices of K.
constexpr long long chain_of(int K, int chains)
{
    return ((K + 127LL) / 128 + chains - 1) / chains;
}

// The workgroup's rows and column of tiles; group -1: none.  Up to 64 groups are read once, for the count of the tiles and for
// the workgroup's own.
struct E4m3Tile {
    int group, m0, m_end, tn;
};
__device__ __forceinline__ E4m3Tile tile_of(const E4m3Args &p, int bm)
{
    int one, tm, tn;
    if (!p.offsets) {
        tile_coords((int)blockIdx.x, 0, 1, p.tiles_m, p.tiles_n, &one, &tm, &tn);
        return {0, tm * bm, p.R, tn};
    }
    if (p.groups <= 64) {
        const int lane = threadIdx.x & 63;
        int lo = 0, hi = 0;
        if (lane < p.groups) group_rows(p.offsets, lane, p.R, &lo, &hi);
        const int n = (hi - lo + bm - 1) / bm, s = wave_scan(n);
        const int total = add_row_tiles(0, (unsigned)__builtin_amdgcn_readlane(s, 63), p.tiles_m);
        if ((long long)blockIdx.x >= (long long)total * p.tiles_n) return {-1, 0, 0, 0};
        tile_coords((int)blockIdx.x, 0, 1, total, p.tiles_n, &one, &tm, &tn);
        const int at = __builtin_ctzll(__ballot(tm >= s - n && tm < s));   // (tm is below the total)
        const int first = lo + (tm - (s - n)) * bm;
        return {at, __builtin_amdgcn_readlane(first, at), __builtin_amdgcn_readlane(hi, at), tn};
    }
    const int total = count_row_tiles(p.offsets, p.groups, p.R, bm, p.tiles_m);
    if ((long long)blockIdx.x >= (long long)total * p.tiles_n) return {-1, 0, 0, 0};
    tile_coords((int)blockIdx.x, 0, 1, total, p.tiles_n, &one, &tm, &tn);
    const RowTile rt = find_row_tile(p.offsets, p.groups, p.R, bm, tm);
    return {rt.group, rt.first, rt.end, tn};
}

// Sixteen e4m3 values as fp16, exactly (NaN stays NaN), in order.
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
struct Half16 {
    half8 lo, hi;
};
__device__ __forceinline__ Half16 to_f16(u32x4 v)
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

// The words of sixteen bytes from p on, wherever p is, of which `valid` are looked at: those read all hold one of these.  (With
// none a place that is always there is read: loads under a condition would wait for one another.)
struct Words16 {
    unsigned x[5];
};
__device__ __forceinline__ Words16 load_words(const uint8_t *p, int valid)
{
    const uintptr_t at = valid > 0 ? reinterpret_cast<uintptr_t>(p) : reinterpret_cast<uintptr_t>(&zero_chunk);
    const unsigned *w = reinterpret_cast<const unsigned *>(at & ~(uintptr_t)3);
    const int last = valid > 0 ? ((int)(at & 3) + (valid < 16 ? valid : 16) - 1) >> 2 : 0;
    Words16 v;
#pragma unroll
    for (int i = 0; i < 5; ++i) v.x[i] = w[i < last ? i : last];
    return v;
}
// The sixteen bytes; those at or past `valid` are zero.
__device__ __forceinline__ u32x4 bytes_of(const Words16 &w, const uint8_t *p, int valid)
{
    const unsigned skip = (unsigned)(reinterpret_cast<uintptr_t>(p) & 3);
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __builtin_amdgcn_alignbit(w.x[i + 1], w.x[i], 8 * skip);
        const int left = valid - 4 * i;   // valid bytes of this word
        if (left < 4) v[i] = left <= 0 ? 0u : v[i] & (0xFFFFFFFFu >> (32 - 8 * left));
    }
    return v;
}

// ---------------------------------------------------------------------------
// The kernel for what the others cannot address (rows 2^23 bytes apart and more, rows looked up in 4 GiB and more) and for
// K = 0: a 64 x 64 tile of four waves of 32 x 32, slices of 128 k through registers into a double-buffered LDS.  Each byte of
// an operand is loaded, shifted and stored by vector instructions: 581 us at 4096 x 4096 x 4096.
template <int BLOCKB>
__global__ __launch_bounds__(256) void e4m3_any_kernel(E4m3Args p)
{
    constexpr int BM = 64, BN = 64, BK = 128;
    __shared__ __attribute__((aligned(16))) u32x4 lds[2][(BM + BN) * 8];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const E4m3Tile tile = tile_of(p, BM);
    if (tile.group < 0) return;
    const int group = tile.group, m0 = tile.m0, m_end = tile.m_end;
    const int n0 = tile.tn * BN, N = p.N, K = p.K;
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
    Words16 v[4];
    auto valid = [&](int i, int k0) { return row[i] ? K - (k0 + 16 * ch) : 0; };
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load_words(row[i] + (k0 + 16 * ch), valid(i, k0));
    };
    auto store = [&](int buf, int k0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (tid >> 3) + 32 * i;   // (rows of B follow those of A)
            lds[buf][r * 8 + (ch ^ swz_a<8>(r))] = bytes_of(v[i], row[i] + (k0 + 16 * ch), valid(i, k0));
        }
    };
    const int lr = lane & 31, lk = lane >> 5, wm = wave >> 1, wn = wave & 1;
    const int my_row = m0 + 32 * wm + lr, my_at = row_at(my_row);
    const bool held = (unsigned)my_at < (unsigned)p.a_rows;
    const float *sa = p.SA + (held ? my_at : 0);
    const int col0 = n0 + 32 * wn + 4 * lk;   // register r: column col0 + 8 (r / 4) + r % 4
    f32x16 acc = {};
    TwoSum<f32x16> total;
    const int slices = (K + BK - 1) / BK;
    if (slices > 0) load(0);
    for (int t = 0; t < slices; ++t) {
        const int buf = t & 1;
        store(buf, t * BK);
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
        if ((t + 1) % kChain == 0) total.take(acc);
    }
    total.take(acc);
    acc = total.value();
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

// Direct-to-LDS load of a dword per lane (dma16 in stage16.h has the notes).
__device__ __forceinline__ void dma4_at(const void *p, unsigned lds_addr)
{
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, off" : : "v"(p), "s"(lds_addr) : "memory", "m0");
}
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) unsigned lds_unsigned;
// Sixteen bytes from byte `by` (0 to 3) of v on, of which `next` holds the last.
__device__ __forceinline__ u32x4 shifted(const u32x4 &v, unsigned next, unsigned by)
{
    return u32x4{__builtin_amdgcn_alignbyte(v.y, v.x, by), __builtin_amdgcn_alignbyte(v.z, v.y, by),
                 __builtin_amdgcn_alignbyte(v.w, v.z, by), __builtin_amdgcn_alignbyte(next, v.w, by)};
}
typedef __attribute__((address_space(3))) float lds_float;

// A BM x BN tile of KG groups of WM x WN waves; the groups take the slices of k in turn, each
// through a ring of STAGES slots.
template <int BM_, int BN_, int STAGES_, int WM_, int WN_, int KG_ = 1, bool LONG_ = false, bool SHIFT_ = false>
struct E4m3Cfg {
    static constexpr bool SHIFT = SHIFT_;   // rows at any byte
    static constexpr bool LONG = LONG_;     // sums of more than kChain slices
    using Shifted = E4m3Cfg<BM_, BN_, STAGES_, WM_, WN_, KG_, LONG_, true>;
    using Long = E4m3Cfg<BM_, BN_, STAGES_, WM_, WN_, KG_, true>;
    static constexpr int BM = BM_, BN = BN_, BK = 128, STAGES = STAGES_, WM = WM_, WN = WN_, KG = KG_;
    static constexpr int NW = WM * WN, NT = 64 * NW * KG;   // (waves of a group)
    static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
    static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;                            // a slice
    static constexpr int A_LOADS = A_BYTES / 1024 / NW, B_LOADS = B_BYTES / 1024 / NW;    // per wave
    static constexpr int S_LOADS = ((BM + BN) / 64 + NW - 1) / NW;                        // of 64 scales
    static constexpr int S_BYTES = 256 * NW * S_LOADS;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + (SHIFT ? 2 : 1) * S_BYTES;     // (SHIFT: and as many dwords)
    static constexpr int LOADS = A_LOADS + B_LOADS + S_LOADS;
    static constexpr int RING = STAGES * STAGE_BYTES, LDS = KG * RING;
    static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0 && BM % 64 == 0 && BN % 64 == 0,
                  "slices split evenly over the waves");
    static_assert(LDS <= 160 * 1024 && LOADS * STAGES < 64 && TN <= 128, "LDS, outstanding loads");
};

// ---------------------------------------------------------------------------
// Tiles fed by direct-to-LDS loads.  A slice of 128 k (one block of scales) of both
// operands, with the scales of its rows and columns, is a slot of a ring of STAGES; a lane
// reads 16 bytes of a row, makes fp16 of them and has the operands of two matrix-core ops.
// Needs: the rows' offsets from the operand's start (A, rows looked up) or from the tile's within 32 bits; without SHIFT
// dword-aligned rows and K % 16 == 0 (no chunk straddles the end).
// SHIFT: rows start at any byte.  A direct-to-LDS load takes whole dwords, so a row comes from the dword that holds its
// first byte on, with the dword behind each slice beside it; fragments are shifted into place when they are read.  The last k
// that do not fill a slice come through registers.
//
// Bound by the matrix cores and the vector instructions beside them: for a slice, a wave of the 128 x 128 tile has 32 matrix-core
// ops (1024 cycles) and 221 vector instructions (128 conversions, 64 multiply-adds; some 970 cycles with two waves a SIMD).
// 4096 x 4096 x 4096: 124 us (1.11 PFLOP/s, matrix cores busy 56% of the cycles; the fp16 product, which converts nothing, 113).
// Two workgroups a CU fill each other's gaps: with four slots and one 157, 256 x 128 and 128 x 256 tiles with three 127.5.
// 2048 x 4096 x 8192 with a scale for each row of B: 135 us, 64 products of two scales more a slice.  Shifted: 4096 x 4096 x 4001
// 160 us (through registers 488), 1001 x 777 x 513 7.3 us (12.1), a chain of 5 slices, KG = 2 of them at a time.
// Sums promoted in the next slice, beside its products: both sets of registers live, 64 moves a slice and spills.
template <class Cfg, int BLOCKB>
__global__ __launch_bounds__(Cfg::NT, 2) void e4m3_dma_kernel(E4m3Args p)
{
    constexpr bool SHIFT = Cfg::SHIFT;
    constexpr int BM = Cfg::BM, BN = Cfg::BN, BK = Cfg::BK, S = Cfg::STAGES, FM = Cfg::FM, FN = Cfg::FN;
    constexpr int A_LOADS = Cfg::A_LOADS, B_LOADS = Cfg::B_LOADS, S_LOADS = Cfg::S_LOADS;
    constexpr int LOADS = Cfg::LOADS + (SHIFT ? S_LOADS : 0);
    static_assert(LOADS * S < 64, "outstanding loads");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[Cfg::LDS];
    constexpr int KG = Cfg::KG;
    const int tid = threadIdx.x, lane = tid & 63, wave = (tid >> 6) % Cfg::NW;   // (of its group)
    const int uwave = __builtin_amdgcn_readfirstlane(wave), kg = __builtin_amdgcn_readfirstlane((tid >> 6) / Cfg::NW);
    const unsigned lds0 = (unsigned)(uintptr_t)lds + kg * Cfg::RING;
    const E4m3Tile tile = tile_of(p, BM);
    if (tile.group < 0) return;
    const int group = tile.group, m0 = tile.m0, m_end = tile.m_end;
    const int n0 = tile.tn * BN, N = p.N, K = p.K;
    const int limA = m_end - m0 < BM ? m_end - m0 : BM, limB = N - n0 < BN ? N - n0 : BN;

    // rows outside the tile's re-read valid ones; their results are not stored
    // (offsets count from this row; rows that A does not hold read it, and their products are dropped in the epilogue)
    const int base = p.rows ? 0 : m0 < p.a_rows ? m0 : p.a_rows - 1;
    auto row_of = [&](int r) {
        int at = m0 + (r < limA ? r : limA - 1);
        if (p.rows) at = p.rows[at];
        return (unsigned)at < (unsigned)p.a_rows ? at : base;
    };
    unsigned offA[A_LOADS], offB[B_LOADS];
    // the tile's first byte of each operand, and the dword that holds it
    const char *At = reinterpret_cast<const char *>(p.A) + base * p.lda;
    const char *Bt = reinterpret_cast<const char *>(p.B) + (long long)group * p.strideB + (long long)n0 * p.ldb;
    const unsigned skipA = SHIFT ? (unsigned)(reinterpret_cast<uintptr_t>(At) & 3) : 0u;
    const unsigned skipB = SHIFT ? (unsigned)(reinterpret_cast<uintptr_t>(Bt) & 3) : 0u;
    const char *Ab = At - skipA, *Bb = Bt - skipB;
    // a row's first byte, from there
    auto byteA = [&](int r) { return skipA + (unsigned)((row_of(r) - base) * p.lda); };
    auto byteB = [&](int c) { return skipB + (unsigned)((c < limB ? c : limB - 1) * p.ldb); };
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) {
        const int r = 8 * (uwave * A_LOADS + i) + lane / 8;
        offA[i] = (byteA(r) & (SHIFT ? ~3u : ~0u)) + 16 * ((lane % 8) ^ swz_a<8>(r));
    }
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i) {
        const int r = 8 * (uwave * B_LOADS + i) + lane / 8;
        offB[i] = (byteB(r) & (SHIFT ? ~3u : ~0u)) + 16 * ((lane % 8) ^ swz_a<8>(r));
    }
    // 64 rows' or columns' scales a load: those of A, then those of B, spread to one for each column
    const float *scale[S_LOADS];
    long long scale_step[S_LOADS];
    const char *behind[SHIFT ? S_LOADS : 1];   // the dword behind a row's slice 0 (that slice's last where all of it is inside)
#pragma unroll
    for (int i = 0; i < S_LOADS; ++i) {
        const int r = 64 * (uwave * S_LOADS + i) + lane;
        if (64 * (uwave * S_LOADS + i) < BM) {
            scale[i] = p.SA + row_of(r);
            scale_step[i] = p.ldsa;
            if constexpr (SHIFT) behind[i] = Ab + ((byteA(r) + (BK - 1)) & ~3u);
        } else {
            const int c = r - BM;
            scale[i] = p.SB + (long long)group * p.strideSB + (n0 + (c < limB ? c : limB - 1)) / BLOCKB;
            scale_step[i] = p.ldsb;
            if constexpr (SHIFT) behind[i] = Bb + ((byteB(c) + (BK - 1)) & ~3u);
        }
    }
    // this group's slices are kg, kg + KG, ..: nk steps, in which slices past the last are zeros
    const int slices = (K + BK - 1) / BK, looped = SHIFT ? K / BK : slices;   // (SHIFT: the whole ones)
    const int steps = (looped + KG - 1) / KG, nk = steps < S ? S : steps;
    auto issue = [&](int step, int slot) __attribute__((always_inline)) {
        const int t = step * KG + kg;
        const unsigned at = __builtin_amdgcn_readfirstlane(lds0 + slot * Cfg::STAGE_BYTES);
        const unsigned la = at + uwave * A_LOADS * 1024, lb = at + Cfg::A_BYTES + uwave * B_LOADS * 1024;
        const unsigned ls = at + Cfg::A_BYTES + Cfg::B_BYTES + uwave * S_LOADS * 256;
        const char *a = uniform(Ab + (long long)t * BK), *b = uniform(Bb + (long long)t * BK);
        // (a step without a slice: scales of zero too, an infinite one times its sum would be NaN)
#pragma unroll
        for (int i = 0; i < S_LOADS; ++i)
            dma4_at(t < looped ? (const void *)(scale[i] + t * scale_step[i]) : (const void *)zero_chunk, ls + 256 * i);
        if constexpr (SHIFT)
#pragma unroll
            for (int i = 0; i < S_LOADS; ++i)
                dma4_at(t < looped ? (const void *)(behind[i] + (long long)t * BK) : (const void *)zero_chunk, ls + Cfg::S_BYTES + 256 * i);
        if ((t + 1) * BK <= K) {
#pragma unroll
            for (int i = 0; i < A_LOADS; ++i) dma16(a, offA[i], la + 1024 * i);
#pragma unroll
            for (int i = 0; i < B_LOADS; ++i) dma16(b, offB[i], lb + 1024 * i);
        } else {   // (SHIFT: a step without a slice; the k that fill none come later)
#pragma unroll
            for (int i = 0; i < A_LOADS; ++i) {
                const int k = t * BK + 16 * ((lane % 8) ^ swz_a<8>(8 * (uwave * A_LOADS + i) + lane / 8));
                dma16_at(!SHIFT && k < K ? (const void *)(a + offA[i]) : (const void *)zero_chunk, la + 1024 * i);
            }
#pragma unroll
            for (int i = 0; i < B_LOADS; ++i) {
                const int k = t * BK + 16 * ((lane % 8) ^ swz_a<8>(8 * (uwave * B_LOADS + i) + lane / 8));
                dma16_at(!SHIFT && k < K ? (const void *)(b + offB[i]) : (const void *)zero_chunk, lb + 1024 * i);
            }
        }
    };

    const int wm = wave / Cfg::WN, wn = wave % Cfg::WN, lr = lane & 31, lk = lane >> 5;
    unsigned chunk[4];   // of substep s, within a row's 128 bytes (rows 32 apart have the same swizzle)
#pragma unroll
    for (int s = 0; s < 4; ++s) chunk[s] = 16 * ((2 * s + lk) ^ swz_a<8>(lr));
    const unsigned baseA = lds0 + (wm * Cfg::TM + lr) * BK, baseB = lds0 + Cfg::A_BYTES + (wn * Cfg::TN + lr) * BK;
    const unsigned baseS = lds0 + Cfg::A_BYTES + Cfg::B_BYTES;

    // SHIFT: bytes by which the lane's rows are off a dword (rows 32 apart alike, if not looked up), and where the dword behind a
    // chunk is: the next chunk's first, or the one behind the slice
    unsigned offbyA[SHIFT ? FM : 1], offbyB = 0, nextA[SHIFT ? 4 : 1], nextB[SHIFT ? 4 : 1];
    constexpr int STRIDE_BEHIND = 32 * 4;
    const bool last_chunk = lk == 1;   // (of substep 3)
    if constexpr (SHIFT) {
#pragma unroll
        for (int i = 0; i < FM; ++i) offbyA[i] = byteA(wm * Cfg::TM + 32 * i + lr) & 3;
        offbyB = byteB(wn * Cfg::TN + lr) & 3;
        const unsigned ex = lds0 + Cfg::A_BYTES + Cfg::B_BYTES + Cfg::S_BYTES;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const unsigned next = 16 * ((2 * s + lk + 1) ^ swz_a<8>(lr));
            nextA[s] = s == 3 && last_chunk ? ex + 4 * (wm * Cfg::TM + lr) : baseA + next;
            nextB[s] = s == 3 && last_chunk ? ex + 4 * (BM + wn * Cfg::TN + lr) : baseB + next;
        }
    }

    f32x16 acc[FM][FN], sum[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
    TwoSum<f32x16> total[Cfg::LONG ? FM : 1][Cfg::LONG ? FN : 1];
    auto fold = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) total[Cfg::LONG ? i : 0][Cfg::LONG ? j : 0].take(acc[i][j]);
    };
    u32x4 ra[FM], rb[FN];
    unsigned na[SHIFT ? FM : 1], nb[SHIFT ? FN : 1];
    Half16 fa[FM], fb[FN];
    auto read = [&](int slot, int s) __attribute__((always_inline)) {
        const unsigned at = slot * Cfg::STAGE_BYTES + chunk[s];
#pragma unroll
        for (int i = 0; i < FM; ++i) ra[i] = *(const lds_u32x4 *)(uintptr_t)(baseA + at + i * 32 * BK);
#pragma unroll
        for (int j = 0; j < FN; ++j) rb[j] = *(const lds_u32x4 *)(uintptr_t)(baseB + at + j * 32 * BK);
        if constexpr (SHIFT) {
            const int apart = s == 3 && last_chunk ? STRIDE_BEHIND : 32 * BK;
#pragma unroll
            for (int i = 0; i < FM; ++i) na[i] = *(const lds_unsigned *)(uintptr_t)(nextA[s] + slot * Cfg::STAGE_BYTES + i * apart);
#pragma unroll
            for (int j = 0; j < FN; ++j) nb[j] = *(const lds_unsigned *)(uintptr_t)(nextB[s] + slot * Cfg::STAGE_BYTES + j * apart);
        }
    };
    auto convert = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[i] = to_f16(SHIFT ? shifted(ra[i], na[SHIFT ? i : 0], offbyA[SHIFT ? i : 0]) : ra[i]);
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j] = to_f16(SHIFT ? shifted(rb[j], nb[SHIFT ? j : 0], offbyB) : rb[j]);
    };
    // the slice's scales
    float sa[FM], sb[BLOCKB == 1 ? 16 * FN : 1];
    auto read_scales = [&](int slot) __attribute__((always_inline)) {
        const unsigned at = baseS + slot * Cfg::STAGE_BYTES;
#pragma unroll
        for (int i = 0; i < FM; ++i) sa[i] = *(const lds_float *)(uintptr_t)(at + 4 * (wm * Cfg::TM + 32 * i + lr));
        const unsigned ab = at + 4 * (BM + wn * Cfg::TN);
        if constexpr (BLOCKB == 1) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4_t v = *(const lds_f32x4 *)(uintptr_t)(ab + 4 * (32 * j + 8 * g + 4 * lk));
#pragma unroll
                    for (int e = 0; e < 4; ++e) sb[16 * j + 4 * g + e] = v[e];
                }
        } else {
            sb[0] = *(const lds_float *)(uintptr_t)ab;   // (the wave's columns lie in one block)
#pragma unroll
            for (int i = 0; i < FM; ++i) sa[i] *= sb[0];
        }
    };
    auto add = [&](int i, int j) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
            acc[i][j][r] = __builtin_fmaf(BLOCKB == 1 ? sa[i] * sb[16 * j + r] : sa[i], sum[i][j][r], acc[i][j][r]);
    };
    auto lds_barrier = [&]() {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    };

    if (looped > 0) {
#pragma unroll
        for (int t = 0; t < S; ++t) issue(t, t);
        wait_vmcnt<LOADS * (S - 1)>();
        lds_barrier();
        read(0, 0);
        auto slice = [&](int t, int slot, auto pending, auto refill, auto more) __attribute__((always_inline)) {
            const int next = slot + 1 == S ? 0 : slot + 1;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                convert();
                if (s < 3) {
                    read(slot, s + 1);
                    if (s == 2) read_scales(slot);
                } else if constexpr (decltype(more)::value) {
                    wait_vmcnt<LOADS * decltype(pending)::value>();
                    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave has read its slot
                    lds_barrier();
                    if constexpr (decltype(refill)::value) issue(t + S, slot);
                    read(next, 0);
                }
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        sum[i][j] = mfma16<false>(fb[j].lo, fa[i].lo, s == 0 ? f32x16{} : sum[i][j]);
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) sum[i][j] = mfma16<false>(fb[j].hi, fa[i].hi, sum[i][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) add(i, j);
            if constexpr (Cfg::LONG)
                if ((t + 1) % kChain == 0) fold();
        };
        int t = 0, slot = 0;
        for (; t + S < nk; ++t) {
            slice(t, slot, std::integral_constant<int, S - 2>{}, std::true_type{}, std::true_type{});
            slot = slot + 1 == S ? 0 : slot + 1;
        }
        auto after = [&](int d) { return (slot + d) % S; };
        slice(t, slot, std::integral_constant<int, S - 2>{}, std::false_type{}, std::true_type{});
        if constexpr (S >= 3) slice(t + 1, after(1), std::integral_constant<int, S - 3>{}, std::false_type{}, std::true_type{});
        if constexpr (S >= 4) slice(t + 2, after(2), std::integral_constant<int, S - 4>{}, std::false_type{}, std::true_type{});
        slice(nk - 1, after(S - 1), std::integral_constant<int, 0>{}, std::false_type{}, std::false_type{});
    }

    if constexpr (SHIFT) {
        if (looped < slices) {   // the last k, by the first group
            lds_barrier();
            if (kg == 0) {
                constexpr int CHUNKS = (BM + BN) * 8 / (64 * Cfg::NW);
                const int ch = lane % 8, k = looped * BK + 16 * ch;
                auto row = [&](int i) { return i * 8 * Cfg::NW + wave * 8 + lane / 8; };   // (rows of B follow those of A)
                const uint8_t *from[CHUNKS];
                Words16 words[CHUNKS];
#pragma unroll
                for (int i = 0; i < CHUNKS; ++i) {
                    const int r = row(i);
                    from[i] = reinterpret_cast<const uint8_t *>(r < BM ? Ab + byteA(r) : Bb + byteB(r - BM)) + k;
                }
#pragma unroll
                for (int i = 0; i < CHUNKS; ++i) words[i] = load_words(from[i], K - k);
#pragma unroll
                for (int i = 0; i < CHUNKS; ++i)
                    *(lds_u32x4 *)(uintptr_t)(lds0 + row(i) * BK + 16 * (ch ^ swz_a<8>(row(i)))) = bytes_of(words[i], from[i], K - k);
                // (the scales of the last slice a wave has read, replaced)
                auto at = [&](int c) { return p.SB + (long long)group * p.strideSB + (long long)looped * p.ldsb + (c < N ? c : N - 1) / BLOCKB; };
#pragma unroll
                for (int i = 0; i < FM; ++i) sa[i] = p.SA[(long long)looped * p.ldsa + row_of(wm * Cfg::TM + 32 * i + lr)];
                if constexpr (BLOCKB == 1) {
#pragma unroll
                    for (int r = 0; r < 16 * FN; ++r) sb[r] = *at(n0 + wn * Cfg::TN + 32 * (r >> 4) + 8 * ((r >> 2) & 3) + 4 * lk + (r & 3));
                } else {
                    const float v = *at(n0 + wn * Cfg::TN);
#pragma unroll
                    for (int i = 0; i < FM; ++i) sa[i] *= v;
                }
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);
            lds_barrier();
            if (kg == 0) {
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) sum[i][j] = f32x16{};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
#pragma unroll
                    for (int i = 0; i < FM; ++i) fa[i] = to_f16(*(const lds_u32x4 *)(uintptr_t)(baseA + chunk[s] + i * 32 * BK));
#pragma unroll
                    for (int j = 0; j < FN; ++j) fb[j] = to_f16(*(const lds_u32x4 *)(uintptr_t)(baseB + chunk[s] + j * 32 * BK));
#pragma unroll
                    for (int i = 0; i < FM; ++i)
#pragma unroll
                        for (int j = 0; j < FN; ++j) {
                            sum[i][j] = mfma16<false>(fb[j].lo, fa[i].lo, sum[i][j]);
                            sum[i][j] = mfma16<false>(fb[j].hi, fa[i].hi, sum[i][j]);
                        }
                }
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) add(i, j);
            }
        }
    }
    if constexpr (Cfg::LONG) {
        fold();
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = total[i][j].value();
    }
    if constexpr (KG > 1) {
        // the groups' results, added in their order by the first
        lds_barrier();
        static_assert((KG - 1) * BM * BN * 4 <= Cfg::LDS, "the groups' results fit the rings");
        auto at = [&](int g, int i, int j, int c) {
            return (unsigned)(uintptr_t)lds + ((((g - 1) * Cfg::NW + wave) * FM + i) * FN + j) * 4096 + c * 1024 + lane * 16;
        };
        if (kg > 0)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *(lds_f32x4 *)(uintptr_t)at(kg, i, j, c) =
                            f32x4_t{acc[i][j][4 * c], acc[i][j][4 * c + 1], acc[i][j][4 * c + 2], acc[i][j][4 * c + 3]};
        __builtin_amdgcn_s_waitcnt(0xC07F);
        lds_barrier();
        if (kg > 0) return;
#pragma unroll
        for (int g = 1; g < KG; ++g)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const f32x4_t v = *(const lds_f32x4 *)(uintptr_t)at(g, i, j, c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][4 * c + e] += v[e];
                    }
        __builtin_amdgcn_s_waitcnt(0xC07F);
    }

    // Epilogue by rows through the ring: 32 rows of the wave's tile at a time, 16-byte chunk c of row r at
    // chunk c ^ (r % LPR).
    constexpr int LPR = Cfg::TN / 4, RPI = 64 / LPR, NQ = 32 / RPI;
    static_assert(Cfg::NW * 32 * Cfg::TN * 4 <= Cfg::RING, "staging area exceeds the ring");
    const unsigned stage = lds0 + wave * 32 * Cfg::TN * 4;
    lds_barrier();
    const int er = lane / LPR, ec = lane % LPR;
    const int col = n0 + wn * Cfg::TN + 4 * ec;
    const float alpha = p.alpha, beta = p.beta;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int first = m0 + wm * Cfg::TM + 32 * i;
        if (first >= m_end) break;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4_t v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                *(lds_f32x4 *)(uintptr_t)(stage + lr * Cfg::TN * 4 + (((8 * j + 2 * g + lk) ^ (lr & (LPR - 1))) * 16)) = v;
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        f32x4_t v[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int r = q * RPI + er;
            v[q] = *(const lds_f32x4 *)(uintptr_t)(stage + r * Cfg::TN * 4 + ((ec ^ (r & (LPR - 1))) * 16));
        }
        if (p.rows) {
            int at[NQ];   // (loads under a condition would wait for one another)
#pragma unroll
            for (int q = 0; q < NQ; ++q) at[q] = p.rows[first + q * RPI + er < m_end ? first + q * RPI + er : m_end - 1];
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                if ((unsigned)at[q] >= (unsigned)p.a_rows) v[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        } else if (m_end > p.a_rows) {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                if (first + q * RPI + er >= p.a_rows) v[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        if (beta != 0.f && first + 32 <= m_end && n0 + BN <= N) {
            f32x4_t c[NQ];   // (all of C that is read here on its way before the first is used)
#pragma unroll
            for (int q = 0; q < NQ; ++q) c[q] = load_row4<false>(p.C, p.ldc, first + q * RPI + er, col, m_end, N);
#pragma unroll
            for (int q = 0; q < NQ; ++q) store_row4_v(p.C, p.ldc, first + q * RPI + er, col, fma_row4(v[q], c[q], alpha, beta));
        } else if (beta != 0.f) {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                store_row4<true, true>(p.C, p.ldc, first + q * RPI + er, col, v[q], alpha, beta, m_end, N);
        } else if (first + 32 <= m_end && n0 + BN <= N && p.past_cache) {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                __builtin_nontemporal_store(alpha * v[q], reinterpret_cast<f32x4_g *>(p.C + (long long)(first + q * RPI + er) * p.ldc + col));
        } else if (first + 32 <= m_end && n0 + BN <= N) {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                store_row4<false, false>(p.C, p.ldc, first + q * RPI + er, col, v[q], alpha, beta, m_end, N);
        } else {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                store_row4<true, false>(p.C, p.ldc, first + q * RPI + er, col, v[q], alpha, beta, m_end, N);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

template <int RB_, int CB_, int NW_, int S_, bool LONG_ = false, bool SHIFT_ = false>
struct E4m3StreamCfg {
    static constexpr bool SHIFT = SHIFT_;   // rows at any byte
    static constexpr bool LONG = LONG_;     // sums of more than kChain slices
    using Shifted = E4m3StreamCfg<RB_, CB_, NW_, S_, LONG_, true>;
    using Long = E4m3StreamCfg<RB_, CB_, NW_, S_, true>;
    static constexpr int RB = RB_, CB = CB_, NW = NW_, S = S_;   // blocks of 16 rows and columns, waves, slots
    static constexpr int BM = 16 * RB, BN = 16 * CB, BK = 128, NT = 64 * NW;
    static constexpr int A_LOADS = 2 * RB, B_LOADS = 2 * CB, S_LOADS = (BM + BN + 63) / 64;
    static constexpr int LOADS = A_LOADS + B_LOADS + (SHIFT ? 2 : 1) * S_LOADS;
    static constexpr int STAGE = (A_LOADS + B_LOADS) * 1024 + (SHIFT ? 2 : 1) * S_LOADS * 256;
    static constexpr int LDS = NW * S * STAGE;
    static_assert(NW * BM * BN * 4 <= LDS, "the waves' sums fit the rings");
    static_assert(LDS <= 160 * 1024 && LOADS * S < 64 && S >= 2 && S <= 4 && BN <= 128, "LDS, outstanding loads");
};

// ---------------------------------------------------------------------------
// Few rows: the time is that of reading B once.  A workgroup takes 16 CB columns and up to
// 16 RB rows; its waves take the slices of 128 k in turn, each through a ring of S
// slots that only it loads and reads: no barrier until the end, S slices on their way per
// wave.  The waves' results are added in wave order.  Needs what e4m3_dma_kernel needs.  16 x 4096 x 4096: 5.9 us with its launch;
// 128 rows over 64 groups of 1024 x 2048: 19.7 us, 114 MB read at 5.8 TB/s (with 128 x 128 tiles 34); 16 x 4096 x 4001 8.3 us
// (through registers 61).
template <class Cfg, int BLOCKB>
__global__ __launch_bounds__(Cfg::NT) void e4m3_stream_kernel(E4m3Args p)
{
    constexpr int RB = Cfg::RB, CB = Cfg::CB, S = Cfg::S, NW = Cfg::NW, BM = Cfg::BM, BN = Cfg::BN, BK = Cfg::BK;
    constexpr int A_LOADS = Cfg::A_LOADS, B_LOADS = Cfg::B_LOADS, S_LOADS = Cfg::S_LOADS, LOADS = Cfg::LOADS;
    constexpr bool SHIFT = Cfg::SHIFT;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[Cfg::LDS];
    const unsigned lds0 = (unsigned)(uintptr_t)lds;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int uwave = __builtin_amdgcn_readfirstlane(wave);
    const E4m3Tile tile = tile_of(p, BM);
    if (tile.group < 0) return;
    const int group = tile.group, m0 = tile.m0, m_end = tile.m_end;
    const int n0 = tile.tn * BN, N = p.N, K = p.K;
    const int limA = m_end - m0 < BM ? m_end - m0 : BM, limB = N - n0 < BN ? N - n0 : BN;
    // (offsets count from this row; rows that A does not hold read it, and their products are dropped at the end)
    const int base = p.rows ? 0 : m0 < p.a_rows ? m0 : p.a_rows - 1;
    auto row_of = [&](int r) {
        int at = m0 + (r < limA ? r : limA - 1);
        if (p.rows) at = p.rows[at];
        return (unsigned)at < (unsigned)p.a_rows ? at : base;
    };
    unsigned offA[A_LOADS], offB[B_LOADS];
    const char *At = reinterpret_cast<const char *>(p.A) + base * p.lda;
    const char *Bt = reinterpret_cast<const char *>(p.B) + (long long)group * p.strideB + (long long)n0 * p.ldb;
    const unsigned skipA = SHIFT ? (unsigned)(reinterpret_cast<uintptr_t>(At) & 3) : 0u;
    const unsigned skipB = SHIFT ? (unsigned)(reinterpret_cast<uintptr_t>(Bt) & 3) : 0u;
    const char *Ab = At - skipA, *Bb = Bt - skipB;
    auto byteA = [&](int r) { return skipA + (unsigned)((row_of(r) - base) * p.lda); };
    auto byteB = [&](int c) { return skipB + (unsigned)((c < limB ? c : limB - 1) * p.ldb); };
    auto swizzled = [&](int load) { return 16 * ((lane % 8) ^ swz_a<8>(8 * load + lane / 8)); };   // byte of the lane's chunk
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i) {
        offB[i] = (byteB(8 * i + lane / 8) & (SHIFT ? ~3u : ~0u)) + swizzled(i);
    }
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) offA[i] = (byteA(8 * i + lane / 8) & (SHIFT ? ~3u : ~0u)) + swizzled(i);
    // scales: the rows', then the columns'
    const float *scale[S_LOADS];
    long long scale_step[S_LOADS];
    const char *behind[SHIFT ? S_LOADS : 1];   // the dword behind a row's slice (see e4m3_dma_kernel)
#pragma unroll
    for (int i = 0; i < S_LOADS; ++i) {
        const int r = 64 * i + lane, c = r - BM;
        scale[i] = r < BM ? p.SA + row_of(r) : p.SB + (long long)group * p.strideSB + (n0 + (c < limB ? c : limB - 1)) / BLOCKB;
        scale_step[i] = r < BM ? p.ldsa : p.ldsb;
        if constexpr (SHIFT) behind[i] = r < BM ? Ab + ((byteA(r) + (BK - 1)) & ~3u) : Bb + ((byteB(c) + (BK - 1)) & ~3u);
    }
    const int slices = (K + BK - 1) / BK, looped = SHIFT ? K / BK : slices;   // (SHIFT: the whole ones)
    const int my_row = m0 + (tid / (BN / 4) < limA ? tid / (BN / 4) : limA - 1), my_at = p.rows ? p.rows[my_row] : my_row;   // (of the epilogue)
    const unsigned ring = lds0 + uwave * S * Cfg::STAGE;
    auto issue = [&](int t, int slot) __attribute__((always_inline)) {
        const unsigned lb = __builtin_amdgcn_readfirstlane(ring + slot * Cfg::STAGE), la = lb + B_LOADS * 1024, ls = la + A_LOADS * 1024;
        const char *a = uniform(Ab + (long long)t * BK), *b = uniform(Bb + (long long)t * BK);
        if ((t + 1) * BK <= K) {
#pragma unroll
            for (int i = 0; i < B_LOADS; ++i) dma16(b, offB[i], lb + 1024 * i);
#pragma unroll
            for (int i = 0; i < A_LOADS; ++i) dma16(a, offA[i], la + 1024 * i);
        } else {
#pragma unroll
            for (int i = 0; i < B_LOADS; ++i)
                dma16_at(t * BK + swizzled(i) < K ? (const void *)(b + offB[i]) : (const void *)zero_chunk, lb + 1024 * i);
#pragma unroll
            for (int i = 0; i < A_LOADS; ++i)
                dma16_at(t * BK + swizzled(i) < K ? (const void *)(a + offA[i]) : (const void *)zero_chunk, la + 1024 * i);
        }
#pragma unroll
        for (int i = 0; i < S_LOADS; ++i) dma4_at(scale[i] + t * scale_step[i], ls + 256 * i);
        if constexpr (SHIFT)
#pragma unroll
            for (int i = 0; i < S_LOADS; ++i) dma4_at(behind[i] + (long long)t * BK, ls + S_LOADS * 256 + 256 * i);
    };
    const int lr = lane & 15, q = lane >> 4;
    unsigned offbyA[SHIFT ? RB : 1], offbyB = 0;   // bytes by which the lane's rows are off a dword (16 rows apart alike, if not looked up)
    if constexpr (SHIFT) {
#pragma unroll
        for (int i = 0; i < RB; ++i) offbyA[i] = byteA(16 * i + lr) & 3;
        offbyB = byteB(lr) & 3;
    }
    f32x4_t acc[RB][CB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    TwoSum<f32x4_t> total[Cfg::LONG ? RB : 1][Cfg::LONG ? CB : 1];
    auto fold = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) total[Cfg::LONG ? i : 0][Cfg::LONG ? j : 0].take(acc[i][j]);
    };
    // tail: a slice that came through registers, at its place
    auto compute = [&](int slot, bool refill, int t, auto tail) __attribute__((always_inline)) {
        constexpr bool MOVE = SHIFT && !decltype(tail)::value;
        const unsigned lb = ring + slot * Cfg::STAGE, la = lb + B_LOADS * 1024, ls = la + A_LOADS * 1024;
        u32x4 ra[RB][2], rb[CB][2];
        unsigned na[RB][2], nb[CB][2];
        float sa[RB];
        f32x4_t sb[CB];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const unsigned at = lr * BK + 16 * ((4 * s + q) ^ swz_a<8>(lr));   // (rows 16 apart: swizzles 2 apart)
#pragma unroll
            for (int j = 0; j < CB; ++j) rb[j][s] = *(const lds_u32x4 *)(uintptr_t)(lb + j * 16 * BK + (at ^ (32 * (j & 1))));
#pragma unroll
            for (int i = 0; i < RB; ++i) ra[i][s] = *(const lds_u32x4 *)(uintptr_t)(la + i * 16 * BK + (at ^ (32 * (i & 1))));
            if constexpr (MOVE) {
                // the dword behind each chunk: the next chunk's first, or the one behind the slice
                const unsigned next = lr * BK + 16 * ((4 * s + q + 1) ^ swz_a<8>(lr)), ex = ls + S_LOADS * 256;
                const bool over = s == 1 && q == 3;
#pragma unroll
                for (int j = 0; j < CB; ++j)
                    nb[j][s] = *(const lds_unsigned *)(uintptr_t)(over ? ex + 4 * (BM + 16 * j + lr) : lb + j * 16 * BK + (next ^ (32 * (j & 1))));
#pragma unroll
                for (int i = 0; i < RB; ++i)
                    na[i][s] = *(const lds_unsigned *)(uintptr_t)(over ? ex + 4 * (16 * i + lr) : la + i * 16 * BK + (next ^ (32 * (i & 1))));
            }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) sa[i] = *(const lds_float *)(uintptr_t)(ls + 4 * (16 * i + lr));
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            if constexpr (BLOCKB == 1) {
                sb[j] = *(const lds_f32x4 *)(uintptr_t)(ls + 4 * (BM + 16 * j + 4 * q));
            } else {
                const float v = *(const lds_float *)(uintptr_t)(ls + 4 * BM);   // (the columns lie in one block)
                sb[j] = f32x4_t{v, v, v, v};
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read: it may be loaded again
        if (refill) issue(t, slot);
        if constexpr (MOVE) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int j = 0; j < CB; ++j) rb[j][s] = shifted(rb[j][s], nb[j][s], offbyB);
#pragma unroll
                for (int i = 0; i < RB; ++i) ra[i][s] = shifted(ra[i][s], na[i][s], offbyA[SHIFT ? i : 0]);
            }
        }
        Half16 fa[RB][2];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s) fa[i][s] = to_f16(ra[i][s]);
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            const Half16 b0 = to_f16(rb[j][0]), b1 = to_f16(rb[j][1]);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
                sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(b0.lo, fa[i][0].lo, sum, 0, 0, 0);
                sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(b0.hi, fa[i][0].hi, sum, 0, 0, 0);
                sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(b1.lo, fa[i][1].lo, sum, 0, 0, 0);
                sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(b1.hi, fa[i][1].hi, sum, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(sa[i] * sb[j][r], sum[r], acc[i][j][r]);
            }
        }
    };
    const int ns = looped > uwave ? (looped - uwave + NW - 1) / NW : 0;   // this wave's slices: uwave, uwave + NW, ...
#pragma unroll
    for (int i = 0; i < S; ++i)
        if (i < ns) issue(uwave + i * NW, i);
    int i = 0, slot = 0;
    for (; i + S < ns; ++i) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS * (S - 1)) : "memory");
        compute(slot, true, uwave + (i + S) * NW, std::false_type{});
        if constexpr (Cfg::LONG)
            if ((i + 1) % kChain == 0) fold();
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    for (; i < ns; ++i) {   // the last slices: everything has been issued
        const int left = ns - 1 - i;
        if (S > 3 && left >= 3)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S > 3 ? LOADS * 3 : 0) : "memory");
        else if (S > 2 && left >= 2)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S > 2 ? LOADS * 2 : 0) : "memory");
        else if (left == 1)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        compute(slot, false, 0, std::false_type{});
        slot = slot + 1 == S ? 0 : slot + 1;
    }

    if constexpr (SHIFT) {
        if (looped < slices && uwave == looped % NW) {   // the last k, by the wave whose turn it is, into its first slot
            const unsigned lb = ring, la = lb + B_LOADS * 1024, ls = la + A_LOADS * 1024;
            const int k = looped * BK + 16 * (lane % 8);
            auto row = [&](int l) { return 8 * (l < B_LOADS ? l : l - B_LOADS) + lane / 8; };
            const uint8_t *from[A_LOADS + B_LOADS];
            Words16 words[A_LOADS + B_LOADS];
            float s[S_LOADS];
#pragma unroll
            for (int l = 0; l < A_LOADS + B_LOADS; ++l)
                from[l] = reinterpret_cast<const uint8_t *>(l < B_LOADS ? Bb + byteB(row(l)) : Ab + byteA(row(l))) + k;
#pragma unroll
            for (int l = 0; l < S_LOADS; ++l) s[l] = scale[l][looped * scale_step[l]];
#pragma unroll
            for (int l = 0; l < A_LOADS + B_LOADS; ++l) words[l] = load_words(from[l], K - k);
#pragma unroll
            for (int l = 0; l < A_LOADS + B_LOADS; ++l)
                *(lds_u32x4 *)(uintptr_t)((l < B_LOADS ? lb : la) + row(l) * BK + swizzled(l < B_LOADS ? l : l - B_LOADS)) = bytes_of(words[l], from[l], K - k);
#pragma unroll
            for (int l = 0; l < S_LOADS; ++l) *(lds_float *)(uintptr_t)(ls + 256 * l + 4 * lane) = s[l];
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            compute(0, false, 0, std::true_type{});
        }
    }

    if constexpr (Cfg::LONG) {
        fold();
#pragma unroll
        for (int i2 = 0; i2 < RB; ++i2)
#pragma unroll
            for (int j = 0; j < CB; ++j) acc[i2][j] = total[i2][j].value();
    }

    // the waves' results, 16-byte chunk c of row r at chunk c ^ (r % CH), added in wave order
    constexpr int CH = BN / 4;
    __syncthreads();   // every wave has left its ring
#pragma unroll
    for (int i2 = 0; i2 < RB; ++i2)
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            const int r = 16 * i2 + lr, c = 4 * j + q;
            *(lds_f32x4 *)(uintptr_t)(lds0 + wave * BM * BN * 4 + r * BN * 4 + ((c ^ (r & (CH - 1))) * 16)) = acc[i2][j];
        }
    __syncthreads();
    static_assert(BM * CH <= Cfg::NT, "four columns of a row a thread");
    if (tid < limA * CH) {
        const int r = tid / CH, c = tid % CH, row = m0 + r;
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w)
            v += *(const lds_f32x4 *)(uintptr_t)(lds0 + w * BM * BN * 4 + r * BN * 4 + ((c ^ (r & (CH - 1))) * 16));
        if ((unsigned)my_at >= (unsigned)p.a_rows) v = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (p.beta != 0.f)
            store_row4<true, true>(p.C, p.ldc, row, n0 + 4 * c, v, p.alpha, p.beta, m_end, N);
        else
            store_row4<true, false>(p.C, p.ldc, row, n0 + 4 * c, v, p.alpha, p.beta, m_end, N);
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
    a.past_cache = 4LL * q.R * q.N >= (192LL << 20);   // (the memory-side cache holds 256 MiB)
    return a;
}

// Row tiles of bm rows that any split of R rows over the groups can need.
long long row_tiles(const E4m3Problem &q, int bm)
{
    return q.offsets ? q.R / bm + (q.groups < q.R ? q.groups : q.R) : (q.R + (long long)bm - 1) / bm;
}

// The direct-to-LDS kernels take these operands ..
bool dma_ok(const E4m3Problem &q)
{
    return q.K > 0 && 256 * q.lda < (1LL << 31) && 256 * q.ldb < (1LL << 31) && (!q.rows || q.M * q.lda < (1LL << 32) - 4096);
}
// .. and these without shifting.
bool aligned(const E4m3Problem &q)
{
    auto words = [](const void *p, long long ld, long long stride) {
        return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 4 == 0 && stride % 4 == 0;
    };
    return q.K % 16 == 0 && words(q.A, q.lda, 0) && words(q.B, q.ldb, q.strideB);
}

template <class Cfg>
hipError_t launch_dma(const E4m3Problem &q, hipStream_t stream)
{
    if constexpr (!Cfg::SHIFT)
        if (!aligned(q)) return launch_dma<typename Cfg::Shifted>(q, stream);
    E4m3Args a = arguments(q);
    a.tiles_m = (int)row_tiles(q, Cfg::BM);
    a.tiles_n = (q.N + Cfg::BN - 1) / Cfg::BN;
    const dim3 grid((unsigned)((long long)a.tiles_m * a.tiles_n));
    if (q.blockB == 1)
        hipLaunchKernelGGL((e4m3_dma_kernel<Cfg, 1>), grid, dim3(Cfg::NT), 0, stream, a);
    else
        hipLaunchKernelGGL((e4m3_dma_kernel<Cfg, 128>), grid, dim3(Cfg::NT), 0, stream, a);
    return hipGetLastError();
}

template <class Cfg>
hipError_t launch_stream(const E4m3Problem &q, hipStream_t stream)
{
    if constexpr (!Cfg::LONG)
        if (chain_of(q.K, Cfg::NW) > kChain) return launch_stream<typename Cfg::Long>(q, stream);
    if constexpr (!Cfg::SHIFT)
        if (!aligned(q)) return launch_stream<typename Cfg::Shifted>(q, stream);
    E4m3Args a = arguments(q);
    a.tiles_m = (int)row_tiles(q, Cfg::BM);
    a.tiles_n = (q.N + Cfg::BN - 1) / Cfg::BN;
    const dim3 grid((unsigned)((long long)a.tiles_m * a.tiles_n));
    if (q.blockB == 1)
        hipLaunchKernelGGL((e4m3_stream_kernel<Cfg, 1>), grid, dim3(Cfg::NT), 0, stream, a);
    else
        hipLaunchKernelGGL((e4m3_stream_kernel<Cfg, 128>), grid, dim3(Cfg::NT), 0, stream, a);
    return hipGetLastError();
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

// The time of a tile's 128 k, of its start and end (us, one CU), and how many workgroups a CU holds: measured on
// square and flat plain products and on 8 to 64 groups of 10 to 500 rows each.
struct TileTime {
    double slice, fixed;
};
using Tile128 = E4m3Cfg<128, 128, 2, 2, 2>;
using Tile64x128 = E4m3Cfg<64, 128, 2, 1, 4, 2>;
using Tile64 = E4m3Cfg<64, 64, 2, 2, 2, 2>;
using Stream32 = E4m3StreamCfg<2, 2, 4, 2>;
using Stream16 = E4m3StreamCfg<1, 2, 4, 2>;
constexpr TileTime kTime128 = {1.15, 2}, kTime64x128 = {0.63, 4}, kTime64 = {0.42, 1}, kTime32 = {0.22, 1};

// Sums of more than kChain slices by the tile's long form: 1024 x 2048 x 131072 663 -> 686 us, 512 x 512 x 262144 263 -> 281.
template <class Cfg>
hipError_t launch_any_k(const E4m3Problem &q, hipStream_t stream)
{
    return chain_of(q.K, Cfg::KG) > kChain ? launch_dma<typename Cfg::Long>(q, stream) : launch_dma<Cfg>(q, stream);
}

// 128 x 128 tiles have no registers left for sums of twice 32 bits, so a longer K goes in pieces of kChain slices, each adding to C:
// 4096 x 4096 x 65536 2.10 ms in two, 2.13 in one (with such sums in eight waves, half a tile each and one workgroup a CU, 2.46).  At
// most 16, whose roundings in C then stay small beside those of a piece.
hipError_t launch_tile128(E4m3Problem q, hipStream_t stream)
{
    constexpr int PIECE = 128 * kChain;
    if (q.K > 16 * PIECE) return launch_any_k<Tile64x128>(q, stream);
    const int K = q.K;
    for (int k0 = 0; k0 < K; k0 += PIECE) {
        q.K = K - k0 < PIECE ? K - k0 : PIECE;
        if (hipError_t e = launch_dma<Tile128>(q, stream); e != hipSuccess) return e;
        q.A += PIECE;
        q.SA += kChain * q.ldsa;
        q.B += PIECE;
        q.SB += kChain * q.ldsb;
        q.beta = 1.f;
    }
    return hipSuccess;
}

hipError_t launch_tiles(const E4m3Problem &q, hipStream_t stream)
{
    const double rows = (double)q.R / q.groups, slices = (q.K + 127) / 128;
    // Up to 16 rows a group: streamed (64 groups, 128 rows, 1024 x 2048: 19.7 us, against 34 with 128x128 tiles; 512
    // rows 31.9 against 34.3 with the best tile; a plain 16 x 4096 x 4096 5.8 against 17).
    if (rows <= 16 && holds(q, Stream16::BM, Stream16::BN, Stream16::NT)) return launch_stream<Stream16>(q, stream);
    // Otherwise the tile whose rounds of 256 workgroups take the least time.  Groups part-fill half of their tiles,
    // and how many exist the host does not know: there the rounds are not whole numbers.
    auto time = [&](int bm, int bn, int threads, int per_round, TileTime t) {
        if (!holds(q, bm, bn, threads)) return 1e300;
        const double down = q.offsets ? (double)q.R / bm + 0.5 * (q.groups < q.R ? q.groups : q.R) : (q.R + bm - 1) / bm;
        const double rounds = down * ((q.N + bn - 1) / bn) / per_round;
        return (rounds <= 1 ? 1. : q.offsets ? rounds : std::ceil(rounds)) * (slices * t.slice + t.fixed);
    };
    const double c128 = time(128, 128, Tile128::NT, 256, kTime128), c64x128 = time(64, 128, Tile64x128::NT, 256, kTime64x128);
    const double c64 = time(64, 64, Tile64::NT, 256, kTime64);
    // (streaming 32 rows reads B once for each 32: for plain products, whose B then comes from the caches: 64 x 4096 x 4096
    // 7.4 us against 13, 512 x 512 x 4096 7.2 against 14; 64 groups of 47 rows 64 against 38)
    const double c32 = q.offsets ? 1e300 : time(32, 32, Stream32::NT, 512, kTime32);
    if (c32 < c64 && c32 < c64x128 && c32 < c128) return launch_stream<Stream32>(q, stream);
    if (c64 <= c64x128 && c64 <= c128) return launch_any_k<Tile64>(q, stream);
    if (c64x128 < c128) return launch_any_k<Tile64x128>(q, stream);
    return launch_tile128(q, stream);
}

}  // namespace

bool e4m3_fits(const E4m3Problem &q)
{
    return holds(q, 64, 64, 256);
}

hipError_t launch_e4m3(const E4m3Problem &q, hipStream_t stream)
{
    return dma_ok(q) ? launch_tiles(q, stream) : launch_any(q, stream);
}

}  // namespace mi355gemm
