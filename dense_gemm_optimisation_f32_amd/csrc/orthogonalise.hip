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
//   * The products' operands are fp16 copies, each value off by at most 2^-11 of itself.  An error of
//     A or B multiplies X from the left, and X's own copy X + E is multiplied by B, which is made of A:
//     neither brings in directions (left singular vectors) that X does not have.  X's is scaled by a power of two into fp16's range.
//   * The diagonal of A, which comes to be much larger than the rest, is kept apart in fp32, and the
//     fp16 copy holds zeros there: with A = D + O,  A A = D D + D O + O D + O O.
//   * The diagonal of B = b A + c A A is split: what goes with the rest of B in its fp16 copy, times X's copy, and what is left, in
//     fp32, times fp32's X (diagonal_of_copy in orthogonalise_internal.h has the rule and its reason).
// A model of this arithmetic against 64 bits, before the result is rounded to bf16 (which costs 1.7e-3): five steps of (3.4445, -4.775,
// 2.0315) 1.4e-3 off for gradients of full rank, mostly below 3e-3 for those of low rank, of few or of unequal rows (4.4e-3 at most);
// eight of (1.875, -1.25, 0.375), which bring back what is a little off, 2e-4 to 1e-3.  Where the copies' roundings all agree (entries of one size) the
// first steps, which amplify a relative error up to 10 times, are up to 1.2e-2 off.
#include "orthogonalise_internal.h"
#include "routed_internal.h"
#include "stage16.h"
#include "tile_order.h"
#include "wave.h"

#include <cmath>
#include <type_traits>

namespace mi355gemm {
namespace {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));

constexpr int kNormBlocks = 512;     // workgroups (and partial sums) of a matrix's norm at most

// One matrix's part of the workspace.  Rows and columns are filled up to multiples of 64 with zeros,
// which the products keep.
struct Layout {
    long long m, n;                  // padded
    long long x, x16[2], a16, b16, da, db, norm, bytes;   // byte offsets
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
    l.x16[0] = take(l.m * l.n * 2);   // (a step reads the one and writes the other)
    l.x16[1] = take(l.m * l.n * 2);
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
    int norm_blocks;
    float a, b, c;                   // this step's coefficients
    float x_scale;                   // x16 and x hold x_scale * X
    float alpha;
    const void *G;
    long long ldg, strideG;
    uint16_t *O;
    long long ldo, strideO;
    long long ws_stride;             // bytes per matrix
    float *x;
    _Float16 *x16, *x16_next, *a16, *b16;
    float *da, *db;
    double *norm;
};

template <class T>
__device__ __forceinline__ T *of_member(T *p, long long stride_bytes, int z)
{
    return reinterpret_cast<T *>(reinterpret_cast<uintptr_t>(p) + (uintptr_t)(z * stride_bytes));
}

__device__ __forceinline__ uint16_t bf16_bits(float v)
{
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// A pointer that is the same in every lane, in scalar registers (dma16's base).
__device__ __forceinline__ const char *uniform(const char *p)
{
    const uint64_t b = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = (unsigned)__builtin_amdgcn_readfirstlane((int)b);
    const uint64_t hi = (unsigned)__builtin_amdgcn_readfirstlane((int)(b >> 32));
    return reinterpret_cast<const char *>(lo | (hi << 32));
}
typedef __attribute__((address_space(3))) float lds_float;

template <bool BF>
__device__ __forceinline__ float g_at(const OrthoArgs &p, int z, long long r, long long c)
{
    const long long at = z * p.strideG + r * p.ldg + c;
    if constexpr (BF)
        return __builtin_bit_cast(float, (unsigned)reinterpret_cast<const uint16_t *>(p.G)[at] << 16);
    else
        return reinterpret_cast<const float *>(p.G)[at];
}

// Sums of squares in 64 bits: neither large nor small entries leave the range.  A wave takes 256 columns of a row at a
// time, four such pieces together: 12 us for 4096 x 4096 (5.4 TB/s; one entry a thread at a time 64).
template <bool BF, bool VEC>
__global__ __launch_bounds__(256) void norm_kernel(OrthoArgs p)
{
    __shared__ double part[4];
    const int z = blockIdx.z, tid = threadIdx.x, lane = tid & 63;
    const int across = (p.N + 255) / 256, turn = gridDim.x * 4;
    const int pieces = p.M * across;   // (at most 2^24)
    double sum = 0;
    for (int first = blockIdx.x * 4 + (tid >> 6); first < pieces; first += 4 * turn) {
        float v[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int piece = first + u * turn, r = piece / across, c = piece % across * 256 + 4 * lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[u][e] = 0.f;
            if (piece >= pieces) continue;
            if (VEC && c + 4 <= p.N) {
                const long long at = z * p.strideG + r * p.ldg + c;
                if constexpr (BF) {
                    typedef unsigned u32x2_g __attribute__((ext_vector_type(2), aligned(4)));
                    const u32x2_g w = *reinterpret_cast<const u32x2_g *>(reinterpret_cast<const uint16_t *>(p.G) + at);
                    const unsigned w0 = w.x, w1 = w.y;
                    v[u][0] = __builtin_bit_cast(float, w0 << 16);
                    v[u][1] = __builtin_bit_cast(float, w0 & 0xFFFF0000u);
                    v[u][2] = __builtin_bit_cast(float, w1 << 16);
                    v[u][3] = __builtin_bit_cast(float, w1 & 0xFFFF0000u);
                } else {
                    const f32x4_t w = *reinterpret_cast<const f32x4_g *>(reinterpret_cast<const float *>(p.G) + at);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[u][e] = w[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float at = g_at<BF>(p, z, r, c + e < p.N ? c + e : p.N - 1);   // (loaded in any case: loads under a
                    v[u][e] = c + e < p.N ? at : 0.f;                                    // condition would wait for one another)
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum = __builtin_fma((double)v[u][e], (double)v[u][e], sum);
    }
    sum = wave_sum(sum);
    if (lane == 0) part[tid >> 6] = sum;
    __syncthreads();
    if (tid == 0) of_member(p.norm, p.ws_stride, z)[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X and its copy from G: a 64 x 64 tile of X per workgroup.  4096 x 4096: 34 us, 168 MB at 4.9 TB/s.
template <bool BF>
__global__ __launch_bounds__(256) void start_kernel(OrthoArgs p)
{
    __shared__ float tile[64][65];
    const int z = blockIdx.z, tid = threadIdx.x;
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // of X
    const double *norm = of_member(p.norm, p.ws_stride, z);
    float g[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        // (consecutive threads along G's rows)
        const int e = tid + 256 * k, i = p.tall ? e % 64 : e / 64, j = p.tall ? e / 64 : e % 64;
        const int gr = p.tall ? c0 + j : r0 + i, gc = p.tall ? r0 + i : c0 + j;
        // (outside: a value inside, not counted below.  Loads under a condition would wait for one another.)
        g[k] = g_at<BF>(p, z, gr < p.M ? gr : p.M - 1, gc < p.N ? gc : p.N - 1);
    }
    double sum = 0;
    for (int i = tid & 63; i < p.norm_blocks; i += 64) sum += norm[i];
    sum = wave_sum(sum);
    // zeros stay zeros; an infinity or NaN makes everything NaN
    const double f = sum == 0 ? 0 : sum < __builtin_inf() ? p.x_scale / __builtin_sqrt(sum) : __builtin_nan("");
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int e = tid + 256 * k, i = p.tall ? e % 64 : e / 64, j = p.tall ? e / 64 : e % 64;
        const int gr = p.tall ? c0 + j : r0 + i, gc = p.tall ? r0 + i : c0 + j;
        tile[i][j] = gr < p.M && gc < p.N ? (float)(g[k] * f) : 0.f;
    }
    __syncthreads();
    float *x = of_member(p.x, p.ws_stride, z);
    _Float16 *x16 = of_member(p.x16, p.ws_stride, z);
    // four columns a thread
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int e = tid + 256 * k, i = e / 16, j = e % 16 * 4;
        f32x4_t v;
        half4 h;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            v[d] = tile[i][j + d];
            h[d] = (_Float16)v[d];
        }
        *reinterpret_cast<f32x4_t *>(x + (long long)(r0 + i) * p.n + c0 + j) = v;
        *reinterpret_cast<half4 *>(x16 + (long long)(r0 + i) * p.n + c0 + j) = h;
    }
}

constexpr int kGram = 0, kSquare = 1, kApply = 2;   // a step's products (below)

// The tile a workgroup takes.  XCD by XCD (see tile_order.h; here within 32 bits, whose divisions are short): the
// workgroups of one XCD take consecutive tiles, four tile rows at a time.  The symmetric products compute the tiles on and
// above the diagonal alone, row by row; a workgroup also stores its tile's mirror image.
template <int KIND>
__device__ __forceinline__ void tile_of(unsigned rows, unsigned cols, int *member, int *tm, int *tn)
{
    const unsigned each = KIND == kApply ? rows * cols : rows * (rows + 1) / 2;
    const unsigned total = each * gridDim.z, lin = blockIdx.z * each + blockIdx.x;   // (below 2^23)
    const unsigned xcd = lin % kNumXcd, per = total / kNumXcd, extra = total % kNumXcd;
    const unsigned logical = xcd * per + (xcd < extra ? xcd : extra) + lin / kNumXcd;
    const unsigned z = gridDim.z == 1 ? 0u : logical / each;
    unsigned left = logical - z * each;
    *member = (int)z;
    if constexpr (KIND == kApply) {
        const unsigned group = left / (kGroupM * cols), first = group * kGroupM;
        const unsigned down = rows - first < kGroupM ? rows - first : kGroupM;
        left -= group * kGroupM * cols;
        *tm = (int)(first + left % down);
        *tn = (int)(left / down);
    } else {
        unsigned r = 0;   // row r holds rows - r tiles (at most 1024 rows)
        while (left >= rows - r) {
            left -= rows - r;
            ++r;
        }
        *tm = (int)r;
        *tn = (int)(r + left);
    }
}

// An operand stored with k outermost (X as the right operand of B X), in slices of 64 k of R columns: 16-byte chunk c of row k
// sits at chunk c ^ swz_k(k), which puts the four rows that a transposed read touches on different banks.
template <int R>
__device__ __forceinline__ int swz_k(int k)
{
    return R == 64 ? 2 * (k & 3) : swz_b(k);
}
// Byte offset within a slice of the chunk that lane `lane` of wave load g fetches; chunks past the `lim` columns re-read the first.
template <int R>
__device__ __forceinline__ unsigned dma_offset_k(int g, int lane, long long ld, int lim)
{
    constexpr int CPR = R / 8;
    const int k = 64 / CPR * g + lane / CPR;
    const int c = 8 * ((lane % CPR) ^ swz_k<R>(k));
    return (unsigned)(k * ld + (c < lim ? c : 0)) * 2u;
}
// Where a lane reads four k of the columns from `first` on, of 16 k; four k further for the other four.
template <int R>
__device__ __forceinline__ unsigned frag_offset_k(int first, int lane)
{
    const int q = lane >> 4, l = lane & 15, k = 8 * (q >> 1) + (l >> 2), n = first + 16 * (q & 1) + 4 * (l & 3);
    return (unsigned)(k * R * 2 + 16 * ((n >> 3) ^ swz_k<R>(k)) + 2 * (n & 7));
}

// A member's arrays.
struct Parts {
    float *x, *da, *db;
    _Float16 *a16, *b16, *x16_next;
    uint16_t *O;
};
__device__ __forceinline__ Parts parts_of(const OrthoArgs &p, int z)
{
    return {of_member(p.x, p.ws_stride, z), of_member(p.da, p.ws_stride, z), of_member(p.db, p.ws_stride, z), of_member(p.a16, p.ws_stride, z),
            of_member(p.b16, p.ws_stride, z), of_member(p.x16_next, p.ws_stride, z), p.O + z * p.strideO};
}

// Four values of row r from column c on of a step's product: what comes of them (v, for the mirror image or a turned result), and
// their stores by rows.  xv, o, dr, dc: what stands there in X, in A's copy, and the diagonal's entries of the row and the columns.
template <int KIND>
__device__ __forceinline__ void finish(const OrthoArgs &p, const Parts &w, f32x4_t &v, int r, int c, const f32x4_t &xv, const half4 &o, float dr,
                                       const f32x4_t &dc)
{
    half4 h;
    if constexpr (KIND == kGram) {
        const float back = 1.f / (p.x_scale * p.x_scale);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] *= back;
            if (r == c + e) {
                w.da[r] = v[e];
                v[e] = 0.f;
            }
            h[e] = (_Float16)v[e];
        }
        *reinterpret_cast<half4 *>(w.a16 + (long long)r * p.m + c) = h;
    } else if constexpr (KIND == kSquare) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float off = o[e];
            if (r == c + e) {
                const float d = p.b * dr + p.c * (dr * dr + v[e]);
                v[e] = (float)diagonal_of_copy(d, dr, v[e]);
                w.db[r] = d - v[e];
            } else {
                v[e] = p.b * off + p.c * ((dr + dc[e]) * off + v[e]);
            }
            h[e] = (_Float16)v[e];
        }
        *reinterpret_cast<half4 *>(w.b16 + (long long)r * p.m + c) = h;
    } else {
        const float f = p.a + dr;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f, xv[e], v[e]);
        if (!p.last) {
            *reinterpret_cast<f32x4_t *>(w.x + (long long)r * p.n + c) = v;
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = (_Float16)v[e];
            *reinterpret_cast<half4 *>(w.x16_next + (long long)r * p.n + c) = h;
        } else if (!p.tall && r < p.M) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < p.N) w.O[(long long)r * p.ldo + c + e] = bf16_bits(v[e] * (p.alpha / p.x_scale));
        }
    }
}

// The three products of a step, of fp16 copies, k in whole slices of 64:
//   kGram    A = X X^T            P Q^T with P = Q = X
//   kSquare  B = b A + c A A      P Q^T with P = Q = A - diag(A)
//   kApply   X <- a X + B X       P Q   with P = B less the rest of its diagonal, Q = X
// The ring, its loads and its K loop are those of the whole-matrix kernel (hgemm_mfma.hip).  The epilogue passes 32 rows of
// a wave's tile at a time through LDS: by rows, and by columns for what is stored transposed.
//
// 4096 x 4096, a step: A 80 us, B 83, X 126 (1.09 PFLOP/s, matrix cores busy 68% of the cycles).  With all CUs multiplying
// the clock falls: a slice of a 256 x 256 tile takes 1.25 us on 136 CUs and 1.97 on 256, so leaving tiles out gains less than
// their count.  On 64 x 64 tiles a product of 1001 x 513 takes 5 to 6.7 us, a chain: 2 us to start and end, 0.8 until its loads
// are on their way, 1.3 to 3.8 in the loop (16 KB a slice into each CU), 1.4 for the epilogue; wave_kernel takes 3.3 to 4.7.
template <class Cfg, int KIND>
__global__ __launch_bounds__(Cfg::NT) void product_kernel(OrthoArgs p)
{
    constexpr int BM = Cfg::BM, BN = Cfg::BN, BK = 64, S = Cfg::STAGES, FM = Cfg::FM, FN = Cfg::FN;
    static_assert(KIND == kApply || BM == BN, "tiles of symmetric products are square");
    __shared__ __attribute__((aligned(1024))) unsigned char lds[S * Cfg::STAGE_BYTES];
    const unsigned lds0 = (unsigned)(uintptr_t)lds;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int uwave = __builtin_amdgcn_readfirstlane(wave);
    const int cols = KIND == kApply ? p.n : p.m, K = KIND == kGram ? p.n : p.m;
    int z, tm, tn;
    tile_of<KIND>((p.m + BM - 1) / BM, (cols + BN - 1) / BN, &z, &tm, &tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const _Float16 *P = of_member(KIND == kGram ? p.x16 : KIND == kSquare ? p.a16 : p.b16, p.ws_stride, z);
    const _Float16 *Q = of_member(KIND == kSquare ? p.a16 : p.x16, p.ws_stride, z);
    constexpr bool K_OUT = KIND == kApply;   // Q is stored with k outermost

    constexpr int A_LOADS = Cfg::A_LOADS, B_LOADS = Cfg::B_LOADS, LOADS = A_LOADS + B_LOADS;
    const bool loader = uwave >= Cfg::NW - Cfg::LW;
    const int lw = loader ? uwave - (Cfg::NW - Cfg::LW) : 0;
    unsigned offA[A_LOADS], offB[B_LOADS];
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) offA[i] = dma_offset<true, BM, BK, true>(lw * A_LOADS + i, lane, K, p.m - m0);
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i)
        offB[i] = K_OUT ? dma_offset_k<BN>(lw * B_LOADS + i, lane, p.n, cols - n0)
                        : dma_offset<true, BN, BK, true>(lw * B_LOADS + i, lane, K, cols - n0);
    const char *Pb = reinterpret_cast<const char *>(P + (long long)m0 * K);
    const char *Qb = reinterpret_cast<const char *>(Q + (K_OUT ? (long long)n0 : (long long)n0 * K));
    const long long stepQ = K_OUT ? (long long)BK * p.n * 2 : BK * 2;
    const int nk = K / BK;
    // loads `from` to `to` of slice t
    auto issue_part = [&](int t, int slot, int from, int to) __attribute__((always_inline)) {
        if (!loader) return;
        const unsigned la = __builtin_amdgcn_readfirstlane(lds0 + slot * Cfg::A_BYTES + lw * A_LOADS * 1024);
        const unsigned lb = __builtin_amdgcn_readfirstlane(lds0 + S * Cfg::A_BYTES + slot * Cfg::B_BYTES + lw * B_LOADS * 1024);
        // (a K of fewer slices than the ring has slots re-reads the last, which is not multiplied)
        const int at = t < nk ? t : nk - 1;
        const char *a = uniform(Pb + (long long)at * BK * 2), *b = uniform(Qb + at * stepQ);
#pragma unroll
        for (int i = 0; i < A_LOADS; ++i)
            if (i >= from && i < to) dma16(a, offA[i], la + 1024 * i);
#pragma unroll
        for (int i = 0; i < B_LOADS; ++i)
            if (A_LOADS + i >= from && A_LOADS + i < to) dma16(b, offB[i], lb + 1024 * i);
    };
    auto issue = [&](int t, int slot) __attribute__((always_inline)) { issue_part(t, slot, 0, LOADS); };
    const int wm = wave / Cfg::WN, wn = wave % Cfg::WN, lr = lane & 31, lk = lane >> 5;
    // What the epilogue reads (rows first + q RPI + er, columns c ..).  A wave of one block of 32 x 32 reads it here, ahead
    // of the K loop, which small matrices leave after a few microseconds.
    constexpr int TN = Cfg::TN, EP = TN % 64 == 0 ? 64 : 32, LPR = EP / 4, RPI = 64 / LPR, NQ = 32 / RPI;   // (EP columns at a time)
    constexpr bool EARLY = FM == 1 && FN == 1;
    const Parts w = parts_of(p, z);
    const int er = lane / LPR, c0 = n0 + wn * TN + 4 * (lane % LPR);
    f32x4_t xs[NQ], dcs;
    half4 os[NQ];
    float drs[NQ];
    auto read_epilogue = [&](int first, int c) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int r = first + q * RPI + er;
            if constexpr (KIND == kSquare) {
                os[q] = *reinterpret_cast<const half4 *>(w.a16 + (long long)r * p.m + c);
                drs[q] = w.da[r];
            } else if constexpr (KIND == kApply) {
                xs[q] = *reinterpret_cast<const f32x4_t *>(w.x + (long long)r * p.n + c);
                drs[q] = w.db[r];
            }
        }
        if constexpr (KIND == kSquare) dcs = *reinterpret_cast<const f32x4_t *>(w.da + c);
    };
    if constexpr (EARLY) read_epilogue(m0 + wm * Cfg::TM, c0);   // (64 x 64 tiles lie within the padded sizes)
    constexpr int NS = BK / 16;
    constexpr int NFB = K_OUT ? FN : NS;
    unsigned fragA[NS], fragB[NFB];
#pragma unroll
    for (int s = 0; s < NS; ++s) fragA[s] = lds0 + frag_offset<true, BM, BK>(wm * Cfg::TM, lane, s);
#pragma unroll
    for (int s = 0; s < NFB; ++s)
        fragB[s] = lds0 + S * Cfg::A_BYTES +
                   (K_OUT ? frag_offset_k<BN>(wn * Cfg::TN + 32 * s, lane) : frag_offset<true, BN, BK>(wn * Cfg::TN, lane, s));
    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
    half8 fa[2][FM], fb[2][FN];
    auto read = [&](int slot, int s, half8 *a, half8 *b) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i) a[i] = *(const lds_half8 *)(uintptr_t)(fragA[s] + slot * Cfg::A_BYTES + i * 32 * BK * 2);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if constexpr (K_OUT) {
                const unsigned at = fragB[j] + slot * Cfg::B_BYTES + 16 * s * BN * 2;
                const short4v both[2] = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)at),
                                         __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)(at + 4 * BN * 2))};
                b[j] = __builtin_bit_cast(half8, both);
            } else {
                b[j] = *(const lds_half8 *)(uintptr_t)(fragB[s] + slot * Cfg::B_BYTES + j * 32 * BK * 2);
            }
        }
    };
    auto mfmas = [&](const half8 *a, const half8 *b) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<false>(b[j], a[i], acc[i][j]);
#pragma unroll
        for (int i = 0; i < FM * FN; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
        }
    };
    auto lds_barrier = [&]() {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    };
    // One wave a SIMD (SPREAD) has nobody to multiply while it issues loads: its loads go out a few at a time between products.
    constexpr bool SPREAD = BM == 192;
    const bool late = SPREAD || (Cfg::STAGGER && uwave >= Cfg::NW / 2);
    auto step = [&](int t, auto pending, auto refill, bool late_refill) __attribute__((always_inline)) {
        const int slot = t % S, next = (t + 1) % S, prev = (t - 1 + S) % S;
#pragma unroll
        for (int sub = 0; sub < NS; ++sub) {
            const int cur = sub & 1, nxt = cur ^ 1;
            if (sub + 1 < NS) {
                read(slot, sub + 1, fa[nxt], fb[nxt]);
                if (SPREAD) {
                    if (late_refill) issue_part(t - 1 + S, prev, LOADS * sub / (NS - 1), LOADS * (sub + 1) / (NS - 1));
                } else if (Cfg::STAGGER && sub == NS - 2 && late && late_refill) {
                    issue(t - 1 + S, prev);
                }
            } else {
                wait_vmcnt<LOADS * decltype(pending)::value>();
                __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): this wave's slice-t reads are done
                lds_barrier();
                if (decltype(refill)::value && !late) issue(t + S, slot);
                read(next, 0, fa[nxt], fb[nxt]);
            }
            mfmas(fa[cur], fb[cur]);
        }
    };
#pragma unroll
    for (int st = 0; st < S; ++st) issue(st, st);
    wait_vmcnt<LOADS * (S - 1)>();
    lds_barrier();
    read(0, 0, fa[0], fb[0]);
    {
        // the last S - 1 of at least S steps find nothing left to load; a shorter K stops early
        int t = 0;
        for (; t + S < nk; ++t) step(t, std::integral_constant<int, S - 2>{}, std::true_type{}, t >= 1);
        const int t0 = t;
        auto tail = [&](int u, auto pending) __attribute__((always_inline)) {
            if (u + 1 < nk) step(u, pending, std::false_type{}, u == t0 && u >= 1);
        };
        tail(t0, std::integral_constant<int, S - 2>{});
        if constexpr (S >= 3) tail(t0 + 1, std::integral_constant<int, S - 3>{});
        if constexpr (S >= 4) tail(t0 + 2, std::integral_constant<int, S - 4>{});
        const int slot = (nk - 1) % S;
#pragma unroll
        for (int sub = 0; sub < NS; ++sub) {
            const int cur = sub & 1, nxt = cur ^ 1;
            if (sub + 1 < NS) read(slot, sub + 1, fa[nxt], fb[nxt]);
            mfmas(fa[cur], fb[cur]);
        }
    }

    static_assert(Cfg::NW * 32 * EP * 4 <= S * Cfg::STAGE_BYTES, "staging area exceeds the ring");
    static_assert(!EARLY || (BM == 64 && BN == 64), "early reads stay inside the padded matrices");
    const unsigned stage = lds0 + wave * 32 * EP * 4;
    wait_vmcnt<0>();   // (slices that a short K did not use)
    lds_barrier();
    // what also goes out by columns: a symmetric tile's mirror image, a tall result
    const bool turned = KIND == kApply ? p.last && p.tall : tm != tn;
    // chunk of the staged row: 16 bytes of columns 4 k.. at chunk k ^ (row % LPR)
    auto chunk = [&](int r, int k) { return stage + r * EP * 4 + 16 * (k ^ (r & (LPR - 1))); };
#pragma unroll
    for (int part = 0; part < FM * (TN / EP); ++part) {
        const int i = part / (TN / EP), jp = part % (TN / EP), first = m0 + wm * Cfg::TM + 32 * i, c = c0 + jp * EP;
        if (first >= p.m || n0 + wn * TN + jp * EP >= cols) continue;   // (uniform; padded sizes are multiples of 64)
        if constexpr (!EARLY) read_epilogue(first, c);
#pragma unroll
        for (int j = 0; j < EP / 32; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *(lds_f32x4 *)(uintptr_t)chunk(lr, 8 * j + 2 * g + lk) =
                    f32x4_t{acc[i][jp * EP / 32 + j][4 * g], acc[i][jp * EP / 32 + j][4 * g + 1], acc[i][jp * EP / 32 + j][4 * g + 2],
                            acc[i][jp * EP / 32 + j][4 * g + 3]};
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const int lrow = q * RPI + er, r = first + lrow;
            const unsigned at = chunk(lrow, lane % LPR);
            f32x4_t v = *(const lds_f32x4 *)(uintptr_t)at;
            finish<KIND>(p, w, v, r, c, xs[q], os[q], drs[q], dcs);
            if (turned) *(lds_f32x4 *)(uintptr_t)at = v;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (!turned) continue;
        // by columns: lane l has 32 rows of column l (EP = 64), or 16 of column l % 32 (EP = 32)
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        constexpr int HALF = EP / 2;
        const int cl = lane % EP, r0 = lane / EP * HALF, col = n0 + wn * TN + jp * EP + cl;
        float t[HALF];
#pragma unroll
        for (int e = 0; e < HALF; ++e) t[e] = *(const lds_float *)(uintptr_t)(chunk(r0 + e, cl >> 2) + 4 * (cl & 3));
        if constexpr (KIND == kApply) {
            if (col < p.M)
#pragma unroll
                for (int e = 0; e < HALF; ++e)
                    if (first + r0 + e < p.N) w.O[(long long)col * p.ldo + first + r0 + e] = bf16_bits(t[e] * (p.alpha / p.x_scale));
        } else {
            _Float16 *dst = (KIND == kGram ? w.a16 : w.b16) + (long long)col * p.m + first + r0;
#pragma unroll
            for (int e = 0; e < HALF; e += 8) {
                half8 h;
#pragma unroll
                for (int d = 0; d < 8; ++d) h[d] = (_Float16)t[e + d];
                *reinterpret_cast<half8 *>(dst + e) = h;
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// Small products: a 32 x 32 tile of four waves, which take the slices of 64 k in turn, each through a ring of two slots
// that only it loads and reads: no barrier until the waves' results are added, in wave order.  Against 64 x 64 tiles, four
// times the CUs read half as much each, and a wave's first slices are all on their way at once: 129 x 129 67.5 -> 52 us, 1001 x 513
// 105 -> 88, 300 x 2000 104 -> 81.5, 700 x 700 105 -> 86 (four slots: the same).
template <int KIND>
__global__ __launch_bounds__(256) void wave_kernel(OrthoArgs p)
{
    constexpr int T = 32, BK = 64, NW = 4, S = 2, SLICE = T * BK * 2, LOADS = 2 * SLICE / 1024;
    __shared__ __attribute__((aligned(1024))) unsigned char lds[NW * S * 2 * SLICE];
    const unsigned lds0 = (unsigned)(uintptr_t)lds;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int uwave = __builtin_amdgcn_readfirstlane(wave);
    const int K = KIND == kGram ? p.n : p.m, nk = K / BK;
    int z, tm, tn;
    tile_of<KIND>(p.m / T, p.n / T, &z, &tm, &tn);
    const int m0 = tm * T, n0 = tn * T;   // (padded sizes are multiples of 64: tiles are whole)
    const _Float16 *P = of_member(KIND == kGram ? p.x16 : KIND == kSquare ? p.a16 : p.b16, p.ws_stride, z) + (long long)m0 * K;
    const _Float16 *Q = of_member(KIND == kSquare ? p.a16 : p.x16, p.ws_stride, z);
    constexpr bool K_OUT = KIND == kApply;   // Q is stored with k outermost: rows of 32 columns, 64 bytes, whose four banks of a
                                             // transposed read differ as they lie
    const char *Pb = reinterpret_cast<const char *>(P), *Qb = reinterpret_cast<const char *>(Q + (K_OUT ? (long long)n0 : (long long)n0 * K));
    const long long stepQ = K_OUT ? (long long)BK * p.n * 2 : BK * 2;
    unsigned offP[LOADS / 2], offQ[LOADS / 2];
#pragma unroll
    for (int i = 0; i < LOADS / 2; ++i) {
        offP[i] = dma_offset<true, T, BK, false>(i, lane, K, T);
        offQ[i] = K_OUT ? (unsigned)((16 * i + lane / 4) * (long long)p.n + 8 * (lane % 4)) * 2u : offP[i];
    }
    const unsigned ring = lds0 + uwave * S * 2 * SLICE;
    auto issue = [&](int t, int slot) __attribute__((always_inline)) {
        const unsigned at = __builtin_amdgcn_readfirstlane(ring + slot * 2 * SLICE);
        const char *a = uniform(Pb + (long long)t * BK * 2), *b = uniform(Qb + t * stepQ);
#pragma unroll
        for (int i = 0; i < LOADS / 2; ++i) dma16(a, offP[i], at + 1024 * i);
#pragma unroll
        for (int i = 0; i < LOADS / 2; ++i) dma16(b, offQ[i], at + SLICE + 1024 * i);
    };
    // what the epilogue reads: four columns of a row a thread
    const Parts w = parts_of(p, z);
    const int er = tid / 8, ec = tid % 8, r = m0 + er, c = n0 + 4 * ec;
    f32x4_t xv = {}, dc = {};
    half4 o = {};
    float dr = 0.f;
    if constexpr (KIND == kSquare) {
        o = *reinterpret_cast<const half4 *>(w.a16 + (long long)r * p.m + c);
        dr = w.da[r];
        dc = *reinterpret_cast<const f32x4_t *>(w.da + c);
    } else if constexpr (KIND == kApply) {
        xv = *reinterpret_cast<const f32x4_t *>(w.x + (long long)r * p.n + c);
        dr = w.db[r];
    }
    unsigned fragP[BK / 16], fragQ[BK / 16];
#pragma unroll
    for (int s = 0; s < BK / 16; ++s) {
        const int q = lane >> 4, l = lane & 15;
        fragP[s] = frag_offset<true, T, BK>(0, lane, s);
        fragQ[s] = SLICE + (K_OUT ? (unsigned)((16 * s + 8 * (q >> 1) + (l >> 2)) * T + 16 * (q & 1) + 4 * (l & 3)) * 2u : fragP[s]);
    }
    f32x16 acc = {};
    const int ns = nk > uwave ? (nk - uwave + NW - 1) / NW : 0;   // this wave's slices: uwave, uwave + NW, ..
    auto compute = [&](int slot, bool refill, int t) __attribute__((always_inline)) {
        const unsigned at = ring + slot * 2 * SLICE;
        half8 a[BK / 16], b[BK / 16];
#pragma unroll
        for (int s = 0; s < BK / 16; ++s) {
            a[s] = *(const lds_half8 *)(uintptr_t)(at + fragP[s]);
            if constexpr (K_OUT) {
                const short4v both[2] = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)(at + fragQ[s])),
                                         __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)(at + fragQ[s] + 4 * T * 2))};
                b[s] = __builtin_bit_cast(half8, both);
            } else {
                b[s] = *(const lds_half8 *)(uintptr_t)(at + fragQ[s]);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot is read: it may be loaded again
        if (refill) issue(t, slot);
#pragma unroll
        for (int s = 0; s < BK / 16; ++s) acc = mfma16<false>(b[s], a[s], acc);
    };
#pragma unroll
    for (int i = 0; i < S; ++i)
        if (i < ns) issue(uwave + i * NW, i);
    int i = 0, slot = 0;
    for (; i + S < ns; ++i) {
        wait_vmcnt<LOADS *(S - 1)>();
        compute(slot, true, uwave + (i + S) * NW);
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    for (; i < ns; ++i) {   // the last slices: everything has been issued
        if (i + 1 < ns)
            wait_vmcnt<LOADS>();
        else
            wait_vmcnt<0>();
        compute(slot, false, 0);
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    // the waves' results: 16 bytes of columns 4 k.. of row r at chunk k ^ (r % 8)
    auto chunk = [&](int row, int k) { return lds0 + row * T * 4 + 16 * (k ^ (row & 7)); };
    __syncthreads();   // every wave has left its ring
#pragma unroll
    for (int g = 0; g < 4; ++g)
        *(lds_f32x4 *)(uintptr_t)(chunk(lane & 31, 2 * g + (lane >> 5)) + wave * T * T * 4) =
            f32x4_t{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
    __syncthreads();
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NW; ++k) v += *(const lds_f32x4 *)(uintptr_t)(chunk(er, ec) + k * T * T * 4);
    finish<KIND>(p, w, v, r, c, xv, o, dr, dc);
    const bool turned = KIND == kApply ? p.last && p.tall : tm != tn;
    if (!turned) return;
    *(lds_f32x4 *)(uintptr_t)chunk(er, ec) = v;   // (read by this thread alone until now)
    __syncthreads();
    // by columns: column er, rows 4 ec ..
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = *(const lds_float *)(uintptr_t)(chunk(4 * ec + e, er >> 2) + 4 * (er & 3));
    const int col = n0 + er, row = m0 + 4 * ec;
    if constexpr (KIND == kApply) {
        if (col < p.M)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (row + e < p.N) w.O[(long long)col * p.ldo + row + e] = bf16_bits(t[e] * (p.alpha / p.x_scale));
    } else {
        *reinterpret_cast<half4 *>((KIND == kGram ? w.a16 : w.b16) + (long long)col * p.m + row) = half4{(_Float16)t[0], (_Float16)t[1], (_Float16)t[2], (_Float16)t[3]};
    }
}

template <class Cfg, int KIND>
hipError_t launch_tiles(const OrthoArgs &a, int batch, hipStream_t stream)
{
    const int rows = (a.m + Cfg::BM - 1) / Cfg::BM, cols = (a.n + Cfg::BN - 1) / Cfg::BN;
    const int tiles = KIND == kApply ? rows * cols : rows * (rows + 1) / 2;
    hipLaunchKernelGGL((product_kernel<Cfg, KIND>), dim3(tiles, 1, batch), dim3(Cfg::NT), 0, stream, a);
    return hipGetLastError();
}

using Large = HgDmaCfg<256, 256, 2, 2, 4, 64>;
using Wide = HgDmaCfg<192, 192, 3, 2, 2, 64>;     // symmetric products only
using Middle = HgDmaCfg<128, 128, 4, 2, 4, 64>;
using Small = HgDmaCfg<64, 64, 4, 2, 2, 64>;

template <int KIND>
hipError_t launch_product(const OrthoArgs &a, int batch, hipStream_t stream)
{
    // Up to 512 tiles of 32 x 32 (two share a CU), those: 960 x 2000 156.5 -> 149.7 us with 465 for A and B; beyond, 1024 x 1024
    // with 528 126.8 -> 135.5, 300 x 2000 with 630 for X 82 -> 87.
    const long long rows32 = a.m / 32, tiles32 = KIND == kApply ? rows32 * (a.n / 32) : rows32 * (rows32 + 1) / 2;
    if (tiles32 * batch <= 512) {
        hipLaunchKernelGGL(wave_kernel<KIND>, dim3((unsigned)tiles32, 1, batch), dim3(256), 0, stream, a);
        return hipGetLastError();
    }
    // Otherwise rounds of 256 workgroups, each with so long for a slice and for its start and end (us, measured on products of 512 x
    // 512 to 4096 x 4096).  Two 64 x 64 tiles share a CU, so their rounds need not be whole.  (192 x 192 tiles fill a
    // round with one triangle of 4224 rows: 4096 x 4096 1593 -> 1480 us an update, 4096 x 8192 2819 -> 2522, against 256 x 256 on
    // 136 CUs.)
    auto time = [&](int side, double slice, double fixed, bool whole) {
        const double rows = (a.m + side - 1) / side, cols = (a.n + side - 1) / side;
        const double rounds = (KIND == kApply ? rows * cols : rows * (rows + 1) / 2) * batch / 256;
        const double slices = (KIND == kGram ? a.n : a.m) / 64;
        return (rounds <= 1 ? 1. : whole ? std::ceil(rounds) : rounds) * (slices * slice + fixed);
    };
    const double large = time(256, 1.4, 5, true), middle = time(128, 0.44, 4, true), small = time(64, 0.25, 1.4, false);
    if constexpr (KIND != kApply) {
        const double wide = time(192, 1.25, 5, true);
        if (wide < large && wide < middle && wide < small) return launch_tiles<Wide, KIND>(a, batch, stream);
    }
    if (large <= middle && large <= small) return launch_tiles<Large, KIND>(a, batch, stream);
    if (middle <= small) return launch_tiles<Middle, KIND>(a, batch, stream);
    return launch_tiles<Small, KIND>(a, batch, stream);
}

template <bool BF>
hipError_t launch(const OrthoProblem &q, hipStream_t stream)
{
    const Layout l = layout(q.M, q.N);
    OrthoArgs a = {};
    a.M = q.M; a.N = q.N;
    a.m = (int)l.m; a.n = (int)l.n;
    a.tall = q.M > q.N;
    a.x_scale = ortho_x_scale(q.M, q.N);
    a.alpha = q.alpha;
    a.G = q.G; a.ldg = q.ldg; a.strideG = q.strideG;
    a.O = q.O; a.ldo = q.ldo; a.strideO = q.strideO;
    a.ws_stride = l.bytes;
    char *w = static_cast<char *>(q.workspace);
    a.x = reinterpret_cast<float *>(w + l.x);
    a.a16 = reinterpret_cast<_Float16 *>(w + l.a16);
    a.b16 = reinterpret_cast<_Float16 *>(w + l.b16);
    a.da = reinterpret_cast<float *>(w + l.da);
    a.db = reinterpret_cast<float *>(w + l.db);
    a.norm = reinterpret_cast<double *>(w + l.norm);
    _Float16 *x16[2] = {reinterpret_cast<_Float16 *>(w + l.x16[0]), reinterpret_cast<_Float16 *>(w + l.x16[1])};
    // 4096 values a workgroup (four pieces of 256 for each wave), or more
    const long long share = ((long long)q.M * ((q.N + 255) / 256) + 15) / 16;
    a.norm_blocks = (int)(share < kNormBlocks ? share : kNormBlocks);
    const bool vec = !BF || (reinterpret_cast<uintptr_t>(q.G) % 4 == 0 && q.ldg % 2 == 0 && q.strideG % 2 == 0);
    if (vec)
        hipLaunchKernelGGL((norm_kernel<BF, true>), dim3(a.norm_blocks, 1, q.batch), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((norm_kernel<BF, false>), dim3(a.norm_blocks, 1, q.batch), dim3(256), 0, stream, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    a.x16 = x16[0];
    hipLaunchKernelGGL(start_kernel<BF>, dim3(a.n / 64, a.m / 64, q.batch), dim3(256), 0, stream, a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    for (int s = 0; s < q.steps; ++s) {
        a.a = q.coefficients[3 * s];
        a.b = q.coefficients[3 * s + 1];
        a.c = q.coefficients[3 * s + 2];
        a.x16 = x16[s & 1];
        a.x16_next = x16[(s & 1) ^ 1];
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
    return ortho_small(M, N) ? 0 : (size_t)layout(M, N).bytes * batch;
}

hipError_t launch_ortho(const OrthoProblem &p, bool bf, hipStream_t stream)
{
    if (ortho_small(p.M, p.N)) return launch_ortho_small(p, bf, stream);
    return bf ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace mi355gemm
