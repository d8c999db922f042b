// orthogonalise_small.hip -- the orthogonalised update (orthogonalise.hip has the method and what is
// rounded where) of matrices that one workgroup holds: one launch for all members and
// steps.
//
// X (m x n, fp32) stays in registers from the first step to the last, in blocks of 32 x 32 as the
// matrix core leaves them (lane: column lane % 32, register r: row 8 (r / 4) + 4 (lane / 32) + r % 4).
// A wave owns RB x CB blocks, WR x WC waves all of them.  A step:
//   the fp16 copy of X goes to LDS, column by column;                             barrier
//   A = X X^T, a block on or above the diagonal a wave; without its diagonal it goes to LDS
//   as fp16, the diagonal as fp32;                                                barrier
//   B = b A + c A A likewise, with a part of its diagonal, into a place of its own;  barrier
//   X <- (a + the rest of the diagonal) X + B X.                                  barrier
// Bound by the chain of a step (8.5 us at 128 x 512, 3.4 at 128 x 128, 1.7 at 64 x 64): four barriers, and between them LDS reads
// that the few blocks of A and B leave to some of the waves (10 of 16 at 128 x 512).  32 of 128 x 512, five steps: 55 us (53 with
// B's diagonal kept out of its copy); 128 x 128 22; 64 x 1024 37.  X X^T's sum shared by the idle waves costs a barrier more: 59.9 us against 55.9.
// X's copy is the right operand of the last product too.  Where LDS does not hold it beside A and B (more than 64 x 1024 or
// 96 x 512), they take its place, a wave owns all rows of its columns, and its own registers are that
// operand: eight rows of a lane's column are what a matrix-core op takes, in an order of rows that B's are
// then read in too.
#include "orthogonalise_internal.h"
#include "stage16.h"
#include "wave.h"

#include <type_traits>

namespace mi355gemm {
namespace {

typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) half4 lds_half4;
typedef __attribute__((address_space(3))) _Float16 lds_half;
typedef __attribute__((address_space(3))) float lds_float;
typedef __attribute__((address_space(3))) double lds_double;

struct SmallArgs {
    int M, N, steps;
    bool tall;                       // X = G^T
    float x_scale, alpha;
    const void *G;
    long long ldg, strideG;
    uint16_t *O;
    long long ldo, strideO;
    float step[kMaxOrthoSteps][3];   // a, b, c
};

template <int RB_, int CB_, int WR_, int WC_>
struct SmallCfg {
    static constexpr int RB = RB_, CB = CB_, WR = WR_, WC = WC_, NW = WR * WC, NT = 64 * NW;
    static constexpr int RF = RB * WR, M = 32 * RF, N = 32 * CB * WC;
    // X's copy, column by column: whole multiples of 128 bytes a column with 16-byte chunk c of column n at chunk c ^ swz(n) (SWZ),
    // or columns 32 bytes further apart: a transposed read's four columns are on different banks, a store's 16 on many
    static constexpr bool SWZ = RF % 2 == 0;
    static constexpr int X_PITCH = SWZ ? 2 * M : 2 * M + 32, A_PITCH = 2 * M + 16;
    static constexpr int X_BYTES = N * X_PITCH, A_BYTES = M * A_PITCH;
    static constexpr int SMALL = 8 * M + 8 * NW;   // the diagonals of A and B, and the waves' norms
    static constexpr bool KEEP = X_BYTES + 2 * A_BYTES + SMALL <= 160 * 1024;   // X's copy stays beside A and B
    static constexpr int BODY = KEEP ? X_BYTES + 2 * A_BYTES : X_BYTES > 2 * A_BYTES ? X_BYTES : 2 * A_BYTES;
    static constexpr int LDS = BODY + SMALL;
    static constexpr int BLOCKS = RF * (RF + 1) / 2, MINE = (BLOCKS + NW - 1) / NW;
    static_assert(LDS <= 160 * 1024 && (KEEP || WR == 1), "LDS");
    static_assert(KEEP == (M < 128 || N < 512), "X's copy gives way to A and B at 128 x 512 alone");
};

// Four registers as fp16, two a conversion.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ half4 to_half(const f32x16 &v, int r)
{
    const half2v h[2] = {__builtin_convertvector((f32x2{v[r], v[r + 1]}), half2v), __builtin_convertvector((f32x2{v[r + 2], v[r + 3]}), half2v)};
    return __builtin_bit_cast(half4, h);
}

// (four consecutive columns: different pairs of chunks; sixteen: eight chunks)
template <class Cfg>
__device__ __forceinline__ unsigned swz(int column)
{
    return Cfg::SWZ ? 16 * (2 * (column & 3) + ((column >> 2) & 1)) : 0;
}

template <class Cfg, bool BF>
__global__ __launch_bounds__(Cfg::NT) void small_kernel(SmallArgs p)
{
    constexpr int RB = Cfg::RB, CB = Cfg::CB, RF = Cfg::RF, NW = Cfg::NW, XP = Cfg::X_PITCH, AP = Cfg::A_PITCH, MINE = Cfg::MINE;
    constexpr bool KEEP = Cfg::KEEP;
    constexpr int AHEAD = KEEP ? 4 : 2;   // steps whose operands are read together
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const unsigned lds0 = (unsigned)(uintptr_t)lds, ldsA = lds0 + (KEEP ? Cfg::X_BYTES : 0), ldsB = ldsA + Cfg::A_BYTES;
    const unsigned ldsDa = lds0 + Cfg::BODY, ldsDb = ldsDa + 4 * Cfg::M, ldsN = ldsDb + 4 * Cfg::M;
    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, lk = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = p.tall ? p.N : p.M, n = p.tall ? p.M : p.N;
    const long long base = (long long)blockIdx.x * p.strideG;
    auto g_at = [&](long long at) -> float {
        if constexpr (BF)
            return __builtin_bit_cast(float, (unsigned)reinterpret_cast<const uint16_t *>(p.G)[at] << 16);
        else
            return reinterpret_cast<const float *>(p.G)[at];
    };
    const int rb0 = wave / Cfg::WC * RB, cb0 = wave % Cfg::WC * CB;   // the wave's first block
    f32x16 x[RB][CB];
    auto row_of = [&](int i, int r) { return 32 * (rb0 + i) + 8 * (r >> 2) + 4 * lk + (r & 3); };
    auto col_of = [&](int j) { return 32 * (cb0 + j) + lr; };

    // G by blocks: the lane's column, rows 4 (lane / 32) + 8 g + e
    const long long dr = p.tall ? 1 : p.ldg, dc = p.tall ? p.ldg : 1;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            const long long at = base + (32 * (rb0 + i) + 4 * lk) * dr + (long long)col_of(j) * dc;
            if (32 * (rb0 + i) + 32 <= m && 32 * (cb0 + j) + 32 <= n) {   // (uniform)
#pragma unroll
                for (int r = 0; r < 16; ++r) x[i][j][r] = g_at(at + (8 * (r >> 2) + (r & 3)) * dr);
            } else {
                // (outside: the first entry, dropped.  Loads under a condition would wait for one another.)
                const bool col_in = col_of(j) < n;
#pragma unroll
                for (int r = 0; r < 16; ++r) x[i][j][r] = g_at(col_in && row_of(i, r) < m ? at + (8 * (r >> 2) + (r & 3)) * dr : base);
#pragma unroll
                for (int r = 0; r < 16; ++r) x[i][j][r] = col_in && row_of(i, r) < m ? x[i][j][r] : 0.f;
            }
            __builtin_amdgcn_sched_barrier(0);   // (addresses of one block at a time in registers)
        }
    // The lane's sum of squares in 32 bits, of its values over the power of two of its largest; the rest in 64, so that
    // neither large nor small entries leave the range (64 bits for every entry: 13 us of 60 at 128 x 512).
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(x[i][j][r]));
    const int power = top > 0.f && top < INFINITY ? __builtin_amdgcn_frexp_expf(top) : 0;
    float squares = 0.f;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float v = __builtin_ldexpf(x[i][j][r], -power);
                squares = __builtin_fmaf(v, v, squares);
            }
    double sum = __builtin_ldexp((double)squares, 2 * power);
    sum = wave_sum(sum);
    if (lane == 0) *(lds_double *)(uintptr_t)(ldsN + 8 * wave) = sum;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += *(const lds_double *)(uintptr_t)(ldsN + 8 * w);
    // zeros stay zeros; an infinity or NaN makes everything NaN
    const double f = sum == 0 ? 0 : sum < __builtin_inf() ? p.x_scale / __builtin_sqrt(sum) : __builtin_nan("");
    // (f leaves 32 bits where G's entries are near their ends: its power of two is applied by itself)
    const int f_power = f > 0 ? __builtin_amdgcn_frexp_exp(f) : 0;
    const float f_rest = (float)__builtin_ldexp(f, -f_power);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) x[i][j][r] = __builtin_ldexpf(x[i][j][r], f_power) * f_rest;

    // this wave's blocks of A: number b = wave, wave + NW, .. of the upper triangle by rows
    int bi[MINE], bj[MINE];
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        int left = wave + k * NW, i = 0;
        while (i < RF && left >= RF - i) {
            left -= RF - i;
            ++i;
        }
        bi[k] = i;          // (RF: none)
        bj[k] = i + left;
    }
    const float back = 1.f / (p.x_scale * p.x_scale);
    // the register that holds the lane's entry of a diagonal block's diagonal, if the lane has it
    const int diag = ((lr >> 2) & 1) == lk ? 4 * (lr >> 3) + (lr & 3) : -1;
    for (int step = 0; step < p.steps; ++step) {
        // the lane's number anew: addresses formed from it are formed where they are used, not kept in registers over the loop
        int here = lane;
        asm volatile("" : "+v"(here));
        const int lr = here & 31, lk = here >> 5;
        auto col_of = [&](int j) { return 32 * (cb0 + j) + lr; };
        // the place of a block's column in the order of an operand from registers
        auto in_turn = [](int c) { return (c & 19) | ((c >> 2) & 1) << 3 | ((c >> 3) & 1) << 2; };
        // A block's values, fp16 and without the diagonal, to both of its places.  B for an operand from registers has its
        // columns in that operand's order.
        auto put = [&](unsigned to, int i, int j, const f32x16 &v, auto turned) __attribute__((always_inline)) {
            constexpr bool TURNED = decltype(turned)::value;
            const int col = TURNED ? in_turn(lr) : lr;
            const unsigned mine = to + (32 * j + lr) * AP + 2 * (32 * i + (TURNED ? 8 : 4) * lk), other = to + (32 * i + 4 * lk) * AP + 2 * (32 * j + col);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                half4 h = to_half(v, 4 * g);
                if (i == j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = diag == 4 * g + e ? (_Float16)0.f : h[e];
                *(lds_half4 *)(uintptr_t)(mine + (TURNED ? 32 * (g >> 1) + 8 * (g & 1) : 16 * g)) = h;
                if (i != j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) *(lds_half *)(uintptr_t)(other + (8 * g + e) * AP) = h[e];
            }
        };
        const float ca = p.step[step][0], cb = p.step[step][1], cc = p.step[step][2];
        // X's copy, column by column
#pragma unroll
        for (int j = 0; j < CB; ++j)
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const half4 h = to_half(x[i][j], 4 * g);
                    *(lds_half4 *)(uintptr_t)(lds0 + col_of(j) * XP + ((2 * (32 * (rb0 + i) + 8 * g + 4 * lk)) ^ swz<Cfg>(lr))) = h;
                }
        __syncthreads();
        f32x16 blk[MINE];
        {
            // transposed reads: four rows (columns of X) of 32 bytes for each 16 lanes
            const int q = here >> 4, l = here & 15;
            const unsigned col = 8 * (q >> 1) + (l >> 2), at = lds0 + col * XP, rows = 2 * (16 * (q & 1) + 4 * (l & 3));
            auto frag = [&](int b, int s) -> half8 {
                const unsigned lo = at + 16 * s * XP + ((64 * b + rows) ^ swz<Cfg>(col)), hi = at + (16 * s + 4) * XP + ((64 * b + rows) ^ swz<Cfg>(col + 4));
                const short4v both[2] = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)lo),
                                         __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(uintptr_t)hi)};
                return __builtin_bit_cast(half8, both);
            };
#pragma unroll
            for (int k = 0; k < MINE; ++k) {
                blk[k] = f32x16{};
                if (bi[k] < RF) {   // (uniform)
                    if (bi[k] == bj[k]) {
#pragma unroll AHEAD
                        for (int s = 0; s < Cfg::N / 16; ++s) {
                            const half8 a = frag(bi[k], s);
                            blk[k] = mfma16<false>(a, a, blk[k]);
                        }
                    } else {
#pragma unroll AHEAD
                        for (int s = 0; s < Cfg::N / 16; ++s) blk[k] = mfma16<false>(frag(bi[k], s), frag(bj[k], s), blk[k]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) blk[k][r] *= back;
            }
        }
        if constexpr (!KEEP) __syncthreads();
#pragma unroll
        for (int k = 0; k < MINE; ++k)
            if (bi[k] < RF) {
                if (bi[k] == bj[k]) {   // (uniform)
                    float mid = 0.f;
#pragma unroll
                    for (int r = 0; r < 16; ++r) mid = r == diag ? blk[k][r] : mid;
                    if (diag >= 0) *(lds_float *)(uintptr_t)(ldsDa + 4 * (32 * bi[k] + lr)) = mid;
                }
                put(ldsA, bi[k], bj[k], blk[k], std::false_type{});
            }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < MINE; ++k) {
            if (bi[k] >= RF) continue;
            const int i = bi[k], j = bj[k];
            f32x16 sq = {};
#pragma unroll AHEAD
            for (int s = 0; s < Cfg::M / 16; ++s) {
                const unsigned at = ldsA + lr * AP + 2 * (16 * s + 8 * lk);
                sq = mfma16<false>(*(const lds_half8 *)(uintptr_t)(at + 32 * i * AP), *(const lds_half8 *)(uintptr_t)(at + 32 * j * AP), sq);
            }
            const float dc = *(const lds_float *)(uintptr_t)(ldsDa + 4 * (32 * j + lr));
            float others = 0.f;   // the diagonal's entry, in the lanes that have one
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4_t dr = *(const lds_f32x4 *)(uintptr_t)(ldsDa + 4 * (32 * i + 8 * g + 4 * lk));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 4 * g + e;
                    const bool diagonal = i == j && r == diag;
                    const float v = blk[k][r];
                    // A A = D D + D O + O D + O O
                    blk[k][r] = cb * v + cc * ((diagonal ? dc * v : (dr[e] + dc) * v) + sq[r]);
                    others = diagonal ? sq[r] : others;
                }
            }
            put(ldsB, i, j, blk[k], std::bool_constant<!KEEP>{});
            if (i == j && diag >= 0) {   // (B's place, after its zero)
                const float b_ii = cb * dc + cc * (dc * dc + others);
                const _Float16 mid = diagonal_of_copy(b_ii, dc, others);
                const int at = KEEP ? lr : in_turn(lr);
                *(lds_float *)(uintptr_t)(ldsDb + 4 * (32 * i + lr)) = ca + (b_ii - (float)mid);
                *(lds_half *)(uintptr_t)(ldsB + (32 * i + lr) * AP + 2 * (32 * i + at)) = mid;
            }
        }
        __syncthreads();
        // X <- (a + the rest of B's diagonal) X + B X
        half8 xh[KEEP ? 1 : 2 * RF][CB];
        if constexpr (!KEEP)
            // the wave's columns: rows 16 s + 4 (lane / 32) .. + 3 and eight further
#pragma unroll
            for (int i = 0; i < RF; ++i)
#pragma unroll
                for (int j = 0; j < CB; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const half4 both[2] = {to_half(x[i][j], 8 * h), to_half(x[i][j], 8 * h + 4)};
                        xh[2 * i + h][j] = __builtin_bit_cast(half8, both);
                    }
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4_t d = *(const lds_f32x4 *)(uintptr_t)(ldsDb + 4 * (32 * (rb0 + i) + 8 * g + 4 * lk));
#pragma unroll
                for (int j = 0; j < CB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[i][j][4 * g + e] *= d[e];
            }
#pragma unroll
        for (int s = 0; s < 2 * RF; ++s) {
            if constexpr (KEEP)
#pragma unroll
                for (int j = 0; j < CB; ++j) xh[0][j] = *(const lds_half8 *)(uintptr_t)(lds0 + col_of(j) * XP + ((2 * (16 * s + 8 * lk)) ^ swz<Cfg>(lr)));
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const half8 b = *(const lds_half8 *)(uintptr_t)(ldsB + (32 * (rb0 + i) + lr) * AP + 2 * (16 * s + 8 * lk));
#pragma unroll
                for (int j = 0; j < CB; ++j) x[i][j] = mfma16<false>(b, xh[KEEP ? 0 : s][j], x[i][j]);
            }
            if constexpr (!KEEP) __builtin_amdgcn_sched_barrier(0);   // (else B's rows are read far ahead, and registers spill)
        }
        __syncthreads();   // X's copy and B are read
    }

    const float out = p.alpha / p.x_scale;
    uint16_t *O = p.O + (long long)blockIdx.x * p.strideO;
    const long long or_ = p.tall ? 1 : p.ldo, oc = p.tall ? p.ldo : 1;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            uint16_t *to = O + (32 * (rb0 + i) + 4 * lk) * or_ + (long long)col_of(j) * oc;
            const bool col_in = col_of(j) < n;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (col_in && row_of(i, r) < m)
                    to[(8 * (r >> 2) + (r & 3)) * or_] = __builtin_bit_cast(uint16_t, (__bf16)(x[i][j][r] * out));
            __builtin_amdgcn_sched_barrier(0);
        }
}

template <class Cfg>
hipError_t launch(const SmallArgs &a, int batch, bool bf, hipStream_t stream)
{
    if (bf)
        hipLaunchKernelGGL((small_kernel<Cfg, true>), dim3(batch), dim3(Cfg::NT), Cfg::LDS, stream, a);
    else
        hipLaunchKernelGGL((small_kernel<Cfg, false>), dim3(batch), dim3(Cfg::NT), Cfg::LDS, stream, a);
    return hipGetLastError();
}

}  // namespace

bool ortho_small(int M, int N)
{
    const int m = M < N ? M : N, n = M < N ? N : M;
    return (m <= 64 && n <= 1024) || (m <= 128 && n <= 512);
}

hipError_t launch_ortho_small(const OrthoProblem &q, bool bf, hipStream_t stream)
{
    const int m = q.M < q.N ? q.M : q.N, n = q.M < q.N ? q.N : q.M;
    SmallArgs a = {};
    a.M = q.M; a.N = q.N; a.steps = q.steps;
    a.tall = q.M > q.N;
    a.x_scale = ortho_x_scale(q.M, q.N);
    a.alpha = q.alpha;
    a.G = q.G; a.ldg = q.ldg; a.strideG = q.strideG;
    a.O = q.O; a.ldo = q.ldo; a.strideO = q.strideO;
    for (int s = 0; s < q.steps; ++s) {
        for (int k = 0; k < 3; ++k) a.step[s][k] = q.coefficients[3 * s + k];
    }
    auto go = [&](auto cfg) { return launch<decltype(cfg)>(a, q.batch, bf, stream); };
    // as many waves as the blocks give work, up to 16
    if (m <= 32) {
        if (n <= 128) return go(SmallCfg<1, 1, 1, 4>{});
        if (n <= 512) return go(SmallCfg<1, 1, 1, 16>{});
        return go(SmallCfg<1, 2, 1, 16>{});
    }
    if (m <= 64) {
        if (n <= 128) return go(SmallCfg<1, 1, 2, 4>{});
        if (n <= 256) return go(SmallCfg<1, 1, 2, 8>{});
        if (n <= 512) return go(SmallCfg<1, 2, 2, 8>{});
        return go(SmallCfg<2, 2, 1, 16>{});
    }
    if (m <= 96) {
        if (n <= 160) return go(SmallCfg<1, 1, 3, 5>{});
        if (n <= 320) return go(SmallCfg<1, 2, 3, 5>{});
        return go(SmallCfg<3, 1, 1, 16>{});
    }
    if (n <= 128) return go(SmallCfg<1, 1, 4, 4>{});
    if (n <= 256) return go(SmallCfg<2, 1, 2, 8>{});
    return go(SmallCfg<4, 1, 1, 16>{});
}

}  // namespace mi355gemm
