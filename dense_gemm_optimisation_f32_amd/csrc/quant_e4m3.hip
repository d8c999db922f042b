// quant_e4m3.hip -- a matrix, or its transpose, laid out in 8-bit floating point
// (e4m3: four exponent bits, three fraction bits, largest value 448, no infinity) with
// a scale for each block of 128 columns of one row or of 128 rows.
//
//   s = the least power of two with max|y| / s <= 448 over the block's finite values
//       (not below 2^-126; 1 for a block of zeros)
//   q = y / s rounded to the nearest e4m3 value, ties to the even one
//
// A power of two loses nothing against 448 / max|y|: the fraction bits are the same,
// only the block's smallest values reach 2^-9 half a step earlier.  y / s is then exact in
// fp32, so q is the nearest value of the quotient itself, with one rounding.
//
// Bound by memory: one pass, every value read once and written once.  What carries it is loads on their way, so values stay
// in registers as they are stored until their scale is known (as fp32 from the start, with a third of the waves: 8192 x 4096
// bf16 27.1 us).  Now 17.7 us there (5.7 TB/s; a large copy 4.7), 30.6 in fp32; 4096 x 8192 turned 18.1 in bf16, 31.6 in fp32;
// 4 of 4096 x 4096 in blocks of 128 rows 33.0 in bf16, 60.4 in fp32; 8191 x 4001 19.6; 16 x 4096 3.8, of which a launch is 3.
#include "e4m3_internal.h"
#include "routed_internal.h"
#include "stage16.h"
#include "wave.h"

#include <type_traits>

namespace mi355gemm {
namespace {

struct QuantArgs {
    int rows, cols;          // X as stored
    int tiles_r, tiles_c;
    const void *X;
    long long ldx, strideX;
    uint8_t *Q;
    long long ldq, strideQ;
    float *S;
    long long lds, strideS;
};

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
// 16 and 8 bytes at any address that holds the elements: loads and stores of this target need no other alignment
typedef unsigned int u32x4_h __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int u32x2_b __attribute__((ext_vector_type(2), aligned(1)));

// The element types by number, for the kernels' names: QuantType's order.
template <int TYPE>
using Stored = std::conditional_t<TYPE == 0, float, std::conditional_t<TYPE == 1, _Float16, __bf16>>;

template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
template <>
__device__ __forceinline__ float to_f32(__bf16 v)
{
    return __builtin_bit_cast(float, (unsigned)__builtin_bit_cast(uint16_t, v) << 16);
}

constexpr unsigned kInfinity = 0x7F800000u;

// The exponent bits of the block's scale from the bits of its largest magnitude
// 2^e m: 2^(e-8) if m <= 1.75 (448 = 1.75 * 2^8), else 2^(e-7).
__device__ __forceinline__ unsigned scale_exponent(unsigned top)
{
    if (top == 0) return 127u;
    const int e = (int)((top + 0x1FFFFFu) >> 23) - 8;
    return (unsigned)(e < 1 ? 1 : e);
}

// Four values to e4m3, in order from the lowest byte.  |y| <= 448 or NaN.
__device__ __forceinline__ unsigned to_e4m3(float a, float b, float c, float d)
{
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

__device__ __forceinline__ void store8_e4m3(uint8_t *dst, u32x2 v, int valid)
{
    if (valid >= 8) {
        *reinterpret_cast<u32x2_b *>(dst) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < valid) dst[e] = (uint8_t)(v[e >> 2] >> (8 * (e & 3)));
}

// The largest of 16 lanes' values, in each of the 16.
__device__ __forceinline__ unsigned row16_max(unsigned v)
{
    auto take = [&](unsigned o) { v = o > v ? o : v; };
    take(dpp<0x128, 0xF>(0u, v));   // rotations within the row by 8, 4, 2, 1
    take(dpp<0x124, 0xF>(0u, v));
    take(dpp<0x122, 0xF>(0u, v));
    take(dpp<0x121, 0xF>(0u, v));
    return v;
}

// Eight values of a row as they are stored.
template <class T>
struct Row8 {
    static constexpr int PER = 4 / sizeof(T);   // values a word
    unsigned w[8 / PER];
};
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Eight values of a row from column c on, or where that leaves the row from column cols - 8 on: into_place moves them then.
// (Loads under a condition would wait for one another; here all rows' are on their way together.)
template <class T>
__device__ __forceinline__ Row8<T> load8(const T *row, int c, int cols)
{
    Row8<T> v;
    if (cols >= 8) {   // (uniform)
        const T *from = row + (c < cols - 8 ? c : cols - 8);
#pragma unroll
        for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
            const u32x4 x = reinterpret_cast<const u32x4_h *>(from)[h];
#pragma unroll
            for (int e = 0; e < 4; ++e) v.w[4 * h + e] = x[e];
        }
        return v;
    }
    typedef std::conditional_t<sizeof(T) == 4, unsigned, uint16_t> Bits;
    const Bits *b = reinterpret_cast<const Bits *>(row);
    Bits x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = b[c + e < cols ? c + e : cols - 1];
#pragma unroll
    for (int i = 0; i < 8 / Row8<T>::PER; ++i) v.w[i] = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.w[e / Row8<T>::PER] |= (c + e < cols ? (unsigned)x[e] : 0u) << (sizeof(T) == 2 ? 16 * (e & 1) : 0);
    return v;
}
// The values `by` (1 and more) places down, zeros behind them.
template <class T>
__device__ __forceinline__ void move_down(Row8<T> &v, int by)
{
    constexpr int W = 8 / Row8<T>::PER;
    const int words = by / Row8<T>::PER;
#pragma unroll
    for (int step = W; step >= 1; step /= 2)
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const unsigned from = i + step < W ? v.w[i + step] : 0u;
            v.w[i] = (step == W ? words >= W : (words & step) != 0) ? from : v.w[i];
        }
    if constexpr (Row8<T>::PER == 2)
#pragma unroll
        for (int i = 0; i < W; ++i) v.w[i] = by & 1 ? __builtin_amdgcn_alignbit(i + 1 < W ? v.w[i + 1] : 0u, v.w[i], 16) : v.w[i];
}
template <class T, int R>
__device__ __forceinline__ void into_place(Row8<T> (&v)[R], int c, int cols)
{
    if (cols >= 8 && c > cols - 8)
#pragma unroll
        for (int i = 0; i < R; ++i) move_down(v[i], c - (cols - 8));
}
// Magnitudes of a word's values, and the larger of each: 16-bit values are compared as they are, two at a time.
template <class T>
constexpr unsigned kMagnitudes = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
template <class T>
__device__ __forceinline__ unsigned larger(unsigned a, unsigned b)
{
    if constexpr (sizeof(T) == 4)
        return a > b ? a : b;
    else
        return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
// A magnitude's bits as fp32, from those of value e of the words.
template <class T>
__device__ __forceinline__ unsigned as_f32(const unsigned *w, int e)
{
    if constexpr (sizeof(T) == 4)
        return w[e];
    else
        return __builtin_bit_cast(unsigned, to_f32(__builtin_bit_cast(T, (uint16_t)(w[e / 2] >> (16 * (e & 1))))));
}
// The largest of the words' magnitudes, as fp32.
template <class T>
__device__ __forceinline__ unsigned largest(const unsigned *w)
{
    unsigned t = 0;
#pragma unroll
    for (int e = 0; e < 8 / Row8<T>::PER; ++e) t = larger<T>(t, w[e] & kMagnitudes<T>);
    if constexpr (sizeof(T) == 2) t = larger<T>(t, t >> 16);
    return as_f32<T>(&t, 0);
}
// Infinities and NaN become NaN, or zeros.
template <class T>
__device__ __forceinline__ Row8<T> replaced(Row8<T> v, bool zeros)
{
    constexpr unsigned MASK = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFFu;
    const T inf = (T)__builtin_inff();
    unsigned least;
    if constexpr (sizeof(T) == 4)
        least = __builtin_bit_cast(unsigned, inf);
    else
        least = __builtin_bit_cast(uint16_t, inf);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int shift = sizeof(T) == 4 ? 0 : 16 * (e & 1);
        unsigned &w = v.w[e / Row8<T>::PER];
        if (((w >> shift) & MASK) >= least) w = zeros ? w & ~(MASK << shift) : w | (MASK << shift);
    }
    return v;
}
template <class T>
__device__ __forceinline__ float value(const Row8<T> &v, int e)
{
    if constexpr (sizeof(T) == 4)
        return __builtin_bit_cast(float, v.w[e]);
    else
        return to_f32(__builtin_bit_cast(T, (uint16_t)(v.w[e / 2] >> (16 * (e & 1)))));
}

// Scales of single rows of X as it is stored: a wave takes 8 rows of 512 columns, 1 KB of a 16-bit row at a time, and 16
// lanes a block (128 x 128 tiles, whose waves read 256 bytes of four rows: 27.3 us where this took 22.0).
constexpr int kRowsR = 32, kRowsC = 512;
template <int TYPE>
__global__ __launch_bounds__(256) void rows_kernel(QuantArgs p)
{
    typedef Stored<TYPE> T;
    const int tid = threadIdx.x, lane = tid & 63;
    const int tiles = p.tiles_r * p.tiles_c;
    const int z = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int r0 = tile / p.tiles_c * kRowsR + 8 * (tid >> 6), c0 = tile % p.tiles_c * kRowsC + 8 * lane;
    const T *X = reinterpret_cast<const T *>(p.X) + z * p.strideX;
    uint8_t *Q = p.Q + z * p.strideQ;
    Row8<T> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // (rows past the last are read from it)
        const int r = r0 + i < p.rows ? r0 + i : p.rows - 1;
        v[i] = load8<T>(X + r * p.ldx, c0, p.cols);
    }
    into_place(v, c0, p.cols);
    unsigned mine = 0;   // lane i of each 16: the exponent bits of row i's scale
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        unsigned top = row16_max(largest<T>(v[i].w));
        if (top >= kInfinity) {   // infinities and NaN do not count, and become NaN
            top = row16_max(largest<T>(replaced(v[i], true).w));
            v[i] = replaced(v[i], false);
        }
        const unsigned ex = scale_exponent(top);
        mine = (lane & 15) == i ? ex : mine;
        const float inv = __builtin_bit_cast(float, (254u - ex) << 23);   // y / s = y * 2^-(ex - 127)
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = value(v[i], e) * inv;
        const u32x2 q = {to_e4m3(y[0], y[1], y[2], y[3]), to_e4m3(y[4], y[5], y[6], y[7])};
        if (r0 + i < p.rows) store8_e4m3(Q + (r0 + i) * p.ldq + c0, q, p.cols - c0);
    }
    const int i = lane & 15;
    if (i < 8 && r0 + i < p.rows && c0 - 8 * i < p.cols)
        p.S[z * p.strideS + c0 / 128 * p.lds + r0 + i] = __builtin_bit_cast(float, mine << 23);
}

// A workgroup takes a 128 x 128 tile of X as it is stored: thread t holds 8 columns (8 (t % 16) ..) of R consecutive rows (R (t /
// 16) ..).  For scales of single rows of X^T (TRANS) or of 128 rows (SQUARE).  8 rows of fp32 would take 172 registers: 4096 x
// 8192 turned 33.9 us, against 31.8 with 4.
template <class T>
constexpr int kTileR = sizeof(T) == 4 ? 4 : 8;
template <class T>
constexpr int kTileThreads = 16 * 128 / kTileR<T>;

template <int TYPE, bool TRANS, bool SQUARE>
__global__ __launch_bounds__(kTileThreads<Stored<TYPE>>) void quant_kernel(QuantArgs p)
{
    typedef Stored<TYPE> T;
    constexpr int R = kTileR<T>, NW = kTileThreads<T> / 64, WORDS = 8 / Row8<T>::PER;
    __shared__ unsigned part[SQUARE ? NW : NW * 16 * WORDS];
    __shared__ __attribute__((aligned(16))) unsigned char turned[TRANS ? 128 * 128 : 16];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int tiles = p.tiles_r * p.tiles_c;
    const int z = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int tr = tile / p.tiles_c, tc = tile % p.tiles_c;
    static_assert(TRANS || SQUARE, "scales of single rows are rows_kernel's");
    const int r0 = tr * 128 + R * (tid >> 4), c0 = tc * 128 + 8 * (tid & 15);
    const T *X = reinterpret_cast<const T *>(p.X) + z * p.strideX;

    Row8<T> v[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        // (rows past the last are read from it)
        const int r = r0 + i < p.rows ? r0 + i : p.rows - 1;
        v[i] = load8<T>(X + r * p.ldx, c0, p.cols);
    }
    into_place(v, c0, p.cols);

    // exponent bits of the scales: of column e, or of the tile (SQUARE)
    unsigned ex[8];
    auto tops = [&](auto counted) __attribute__((always_inline)) {
        unsigned top[WORDS];
#pragma unroll
        for (int w = 0; w < WORDS; ++w) top[w] = 0u;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const Row8<T> c = counted(v[i]);
#pragma unroll
            for (int w = 0; w < WORDS; ++w) top[w] = larger<T>(top[w], c.w[w] & kMagnitudes<T>);
        }
        bool finite = true;
        __syncthreads();
        if constexpr (SQUARE) {
            const unsigned w = wave_max(largest<T>(top));
            if ((tid & 63) == 0) part[wave] = w;
            __syncthreads();
            unsigned all = part[0];
#pragma unroll
            for (int k = 1; k < NW; ++k) all = part[k] > all ? part[k] : all;
            finite = all < kInfinity;
            ex[0] = scale_exponent(all);
        } else {
#pragma unroll
            for (int w = 0; w < WORDS; ++w) {
                top[w] = larger<T>(top[w], (unsigned)__shfl_xor((int)top[w], 16));
                top[w] = larger<T>(top[w], (unsigned)__shfl_xor((int)top[w], 32));
            }
            if ((tid & 63) < 16)
#pragma unroll
                for (int w = 0; w < WORDS; ++w) part[(wave * 16 + (tid & 15)) * WORDS + w] = top[w];
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WORDS; ++w)
#pragma unroll
                for (int k = 0; k < NW; ++k) top[w] = larger<T>(top[w], part[(k * 16 + (tid & 15)) * WORDS + w]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned t = as_f32<T>(top, e);
                finite = finite && t < kInfinity;
                ex[e] = scale_exponent(t);
            }
        }
        return finite;
    };
    const bool finite = tops([](const Row8<T> &c) { return c; });
    if (__syncthreads_or(!finite)) {
        // infinities and NaN do not count, and become NaN
        tops([](const Row8<T> &c) { return replaced(c, true); });
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = replaced(v[i], false);
    }
    // y / s = y * 2^-(ex - 127)
    float inv[SQUARE ? 1 : 8];
#pragma unroll
    for (int e = 0; e < (SQUARE ? 1 : 8); ++e) inv[e] = __builtin_bit_cast(float, (254u - ex[e]) << 23);

    uint8_t *Q = p.Q + z * p.strideQ;
    float *S = p.S + z * p.strideS;
    if constexpr (!TRANS) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = value(v[i], e) * inv[0];
            const u32x2 q = {to_e4m3(y[0], y[1], y[2], y[3]), to_e4m3(y[4], y[5], y[6], y[7])};
            if (r0 + i < p.rows) store8_e4m3(Q + (long long)(r0 + i) * p.ldq + c0, q, p.cols - c0);
        }
        if (tid == 0) S[(long long)tc * p.lds + tr] = __builtin_bit_cast(float, ex[0] << 23);
    } else {
        // Q's rows are X's columns: R k of one row of Q per thread, 128 rows of 128 bytes
        // through LDS, 8-byte piece j of row m at piece j ^ (m / 8 % 16)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float y[R];
#pragma unroll
            for (int i = 0; i < R; ++i) y[i] = value(v[i], e) * inv[SQUARE ? 0 : e];
            const int m = 8 * (tid & 15) + e, k = R * (tid >> 4);
            unsigned char *to = turned + m * 128 + 8 * ((k >> 3) ^ ((m >> 3) & 15)) + (k & 7);
#pragma unroll
            for (int i = 0; i < R; i += 4) *reinterpret_cast<unsigned *>(to + i) = to_e4m3(y[i], y[i + 1], y[i + 2], y[i + 3]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int m = 128 / R * i + (tid >> 4), j = tid & 15;
            const u32x2 q = *reinterpret_cast<const u32x2 *>(turned + m * 128 + 8 * (j ^ ((m >> 3) & 15)));
            const int row = tc * 128 + m, k = tr * 128 + 8 * j;
            if (row < p.cols && k < p.rows) store8_e4m3(Q + (long long)row * p.ldq + k, q, p.rows - k);
        }
        if constexpr (SQUARE) {
            if (tid == 0) S[(long long)tr * p.lds + tc] = __builtin_bit_cast(float, ex[0] << 23);
        } else if (tid < 16) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c0 + e < p.cols) S[(long long)tr * p.lds + c0 + e] = __builtin_bit_cast(float, ex[e] << 23);
        }
    }
}

template <int TYPE, bool TRANS, bool SQUARE>
hipError_t launch(const QuantArgs &a, unsigned blocks, hipStream_t stream)
{
    if constexpr (TRANS || SQUARE)
        hipLaunchKernelGGL((quant_kernel<TYPE, TRANS, SQUARE>), dim3(blocks), dim3(kTileThreads<Stored<TYPE>>), 0, stream, a);
    else
        hipLaunchKernelGGL(rows_kernel<TYPE>, dim3(blocks), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <int TYPE>
hipError_t launch_type(const QuantProblem &q, const QuantArgs &a, unsigned blocks, hipStream_t stream)
{
    if (q.transpose) return q.block == 1 ? launch<TYPE, true, false>(a, blocks, stream) : launch<TYPE, true, true>(a, blocks, stream);
    return q.block == 1 ? launch<TYPE, false, false>(a, blocks, stream) : launch<TYPE, false, true>(a, blocks, stream);
}

// Rows and columns of X, as stored, that a workgroup takes.
int tile_rows(const QuantProblem &p)
{
    return !p.transpose && p.block == 1 ? kRowsR : 128;
}
int tile_cols(const QuantProblem &p)
{
    return !p.transpose && p.block == 1 ? kRowsC : 128;
}
long long quant_tiles(const QuantProblem &p)
{
    const long long rows = p.transpose ? p.K : p.M, cols = p.transpose ? p.M : p.K;
    return (rows + tile_rows(p) - 1) / tile_rows(p) * ((cols + tile_cols(p) - 1) / tile_cols(p));
}

}  // namespace

bool quant_fits(const QuantProblem &p, QuantType type)
{
    const long long tiles = quant_tiles(p);
    const int threads = type == QuantType::f32 && tile_cols(p) == 128 ? kTileThreads<float> : 256;
    return grid_holds(tiles, threads) && grid_holds(tiles * p.batch, threads);
}

hipError_t launch_quant(const QuantProblem &p, QuantType type, hipStream_t stream)
{
    QuantArgs a;
    a.rows = p.transpose ? p.K : p.M;
    a.cols = p.transpose ? p.M : p.K;
    a.tiles_r = (int)((a.rows + (long long)tile_rows(p) - 1) / tile_rows(p));
    a.tiles_c = (int)((a.cols + (long long)tile_cols(p) - 1) / tile_cols(p));
    a.X = p.X; a.ldx = p.ldx; a.strideX = p.strideX;
    a.Q = p.Q; a.ldq = p.ldq; a.strideQ = p.strideQ;
    a.S = p.S; a.lds = p.lds; a.strideS = p.strideS;
    const unsigned blocks = (unsigned)(quant_tiles(p) * p.batch);
    switch (type) {
    case QuantType::f32: return launch_type<0>(p, a, blocks, stream);
    case QuantType::f16: return launch_type<1>(p, a, blocks, stream);
    default: return launch_type<2>(p, a, blocks, stream);
    }
}

}  // namespace mi355gemm
