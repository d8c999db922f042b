// stage16.h -- device code shared by the kernels that multiply 16-bit operands
// (hgemm_mfma.hip, grouped_mfma.hip, lora_mfma.hip): the matrix-core op, global
// loads at dword and at half alignment, the LDS layouts of the operand tiles and
// the direct-to-LDS loads.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epilogue.h"

namespace mi355gemm {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// One 32x32x16 matrix-core op on eight 16-bit values of B and of A per lane:
// IEEE binary16 (BF = false) or bfloat16 (BF = true).  The kernels only move
// 16-bit payloads (half8 is their carrier type); the format matters here alone.
// Products of either format are exact in fp32, and the sum is accumulated in
// fp32 in both.
template <bool BF>
__device__ __forceinline__ f32x16 mfma16(half8 b, half8 a, f32x16 c)
{
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a),
                                                       c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(b, a, c, 0, 0, 0);
}
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes in global memory at dword (not 16-byte) alignment: multi-dword
// global loads need only dword alignment on CDNA
typedef unsigned int u32x4_g __attribute__((ext_vector_type(4), aligned(4)));
typedef __attribute__((address_space(3))) short4v lds_short4;

template <int BM_, int BN_>
struct HgCfg {
    static constexpr int BM = BM_, BN = BN_, BK = 64, WM = 2, WN = 2, NT = 256;
    static constexpr int TM = BM / WM, TN = BN / WN;
    static constexpr int FM = TM / 32, FN = TN / 32;
    static_assert(TM % 32 == 0 && TN % 32 == 0, "wave tile must be whole MFMA blocks");
};

// One operand tile of the register-staged kernel: R rows or columns of the
// output (BM for A, BN for B) by BK k.  KC: stored K-contiguous, kept in LDS
// as R rows of BK halves with swizzled 16-byte chunks; otherwise stored
// MN-contiguous, kept as BK rows of R halves plus a 64-byte pad.
template <bool KC, int R, int BK, int NT>
struct HgTile {
    static constexpr bool KCONTIG = KC;
    static constexpr int ROWS = KC ? R : BK;         // rows as stored
    static constexpr int COLS = KC ? BK : R;         // contiguous halves per stored row
    static constexpr int CPR = COLS / 8;             // 16-byte chunks per stored row
    static constexpr int LOADS = ROWS * CPR / NT;    // 16-byte chunks per thread
    static constexpr int PITCH = KC ? BK : R + 32;   // LDS row pitch (halves)
    static constexpr int HALVES = ROWS * PITCH;
    static_assert((ROWS * CPR) % NT == 0, "tile loads must split evenly");
    static_assert(!KC || BK == 64, "K-contiguous LDS rows are eight 16-byte chunks");
};

__device__ __forceinline__ int swz(int row, int chunk)
{
    return chunk ^ ((row ^ (row >> 3)) & 7);
}

// Eight fp16 values at p[0..7]; elements at or beyond `valid` read as zero.
__device__ __forceinline__ u32x4 load8_masked(const uint16_t *p, int valid)
{
    uint16_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (e < valid) ? p[e] : (uint16_t)0;
    u32x4 v;
    v.x = h[0] | ((unsigned)h[1] << 16);
    v.y = h[2] | ((unsigned)h[3] << 16);
    v.z = h[4] | ((unsigned)h[5] << 16);
    v.w = h[6] | ((unsigned)h[7] << 16);
    return v;
}

// Eight halves at p, which may start 2 bytes past a dword: a 16-byte load from
// the dword holding p[0] and a 4-byte load of the dword holding p[7], joined by
// a funnel shift of 0 or 16 bits.  Every dword read holds one of the eight
// halves, so no load leaves the words the matrix occupies.
__device__ __forceinline__ u32x4 load8_words(const uint16_t *p)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const unsigned sh = (unsigned)(a & 2) * 8;
    const unsigned *w = reinterpret_cast<const unsigned *>(a & ~(uintptr_t)3);
    const u32x4 lo = *reinterpret_cast<const u32x4_g *>(w);
    const unsigned hi = w[sh ? 4 : 3];
    return u32x4{__builtin_amdgcn_alignbit(lo.y, lo.x, sh), __builtin_amdgcn_alignbit(lo.z, lo.y, sh),
                 __builtin_amdgcn_alignbit(lo.w, lo.z, sh), __builtin_amdgcn_alignbit(hi, lo.w, sh)};
}

// Eight consecutive halves (r, c..c+7) of a row-major rows x cols matrix X;
// with MASK, elements outside it read as zero.  VEC: row starts are 4-byte
// aligned, so eight halves inside the matrix are one 16-byte load; otherwise
// they are two dword-aligned loads and a shift.
template <bool MASK, bool VEC>
__device__ __forceinline__ u32x4 load8(const uint16_t *X, long long ld, long long r, long long c, long long rows,
                                       long long cols)
{
    const uint16_t *src = X + r * ld + c;
    if (!MASK) return *reinterpret_cast<const u32x4_g *>(src);
    if (r >= rows || c >= cols) return u32x4{0u, 0u, 0u, 0u};
    if (c + 8 <= cols) return VEC ? *reinterpret_cast<const u32x4_g *>(src) : load8_words(src);
    return load8_masked(src, (int)(cols - c));
}

// A chunk swizzle.  64-byte rows (four chunks): rows that one LDS cycle
// serves get distinct (row, chunk) bank groups.  128-byte rows (eight chunks):
// the chunk is XORed with row bits 0-2 and 3-4, which keeps any aligned 16
// rows on distinct banks and is unchanged by the 32-row steps between the
// MFMA blocks of a wave.
template <int CPR>
__device__ __forceinline__ int swz_a(int r)
{
    return CPR == 8 ? ((r & 7) ^ ((r >> 3) & 3)) : (((r >> 1) ^ (r >> 3)) & 3);
}
__device__ __forceinline__ int swz_b(int k)
{
    // rows k..k+3 of an aligned group of four map to XOR patterns 0, 6, 10, 12
    return (0xCA60 >> (4 * (k & 3))) & 15;
}

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) half8 lds_half8;
typedef __attribute__((address_space(3))) f32x4_t lds_f32x4;

__device__ __forceinline__ lds_void *lds_ptr(unsigned byte)
{
    return (lds_void *)(uintptr_t)byte;
}

// One direct-to-LDS load: every lane fetches 16 bytes at sbase + voff and the
// wave's 1 KB lands contiguously at LDS byte lds_addr (lane l at +16*l).  It is
// issued through inline asm so that the compiler neither reorders LDS accesses
// around it (memory clobber) nor adds its own conservative vmcnt(0) before
// every later LDS read: completion is tracked explicitly with wait_vmcnt.  M0
// (the LDS destination) is set inside the statement; the compiler does not
// track that clobber, which is safe because these kernels give M0 no other use.
__device__ __forceinline__ void dma16(const void *sbase, unsigned voff, unsigned lds_addr)
{
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(voff), "s"(sbase), "s"(lds_addr)
                 : "memory", "m0");
}

// s_waitcnt with only the vector-memory counter constrained (gfx9 encoding:
// vmcnt bits [3:0] and [15:14], expcnt [6:4], lgkmcnt [11:8]).
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Per-lane byte offset (within one slice of global memory) of the 16-byte
// chunk that lane `lane` of wave load g fetches for an operand slice of R rows
// or columns and BK k; see the layouts above.  With CLAMP, `lim` is how many
// of the R rows (K-contiguous) or columns (MN-contiguous) lie inside M or N:
// a chunk past it re-reads a valid one (row lim-1, or chunk 0 of its row),
// whose products only reach C entries that are never stored.
template <bool KC, int R, int BK, bool CLAMP>
__device__ __forceinline__ unsigned dma_offset(int g, int lane, long long ld, int lim)
{
    if (KC) {
        constexpr int CPR = BK / 8;
        const int r = (64 / CPR) * g + lane / CPR;
        const int rr = (CLAMP && r >= lim) ? lim - 1 : r;
        return (unsigned)(rr * ld + 8 * ((lane % CPR) ^ swz_a<CPR>(r))) * 2u;
    }
    constexpr int CPR = R / 8, RPL = 64 / CPR;   // chunks per row, rows per wave load
    const int k = RPL * g + lane / CPR;
    int ch = (lane % CPR) ^ swz_b(k);
    if (CLAMP && 8 * ch >= lim) ch = 0;
    return (unsigned)(k * ld + 8 * ch) * 2u;
}

// Fragment read address (bytes within a slot, substep 0, MFMA block 0) for the
// lane; KC: the rows start at `first`, MN-contiguous: the columns do.
// K-contiguous fragments of substep s and block i add 16*(s-chunk XOR) and
// i*32 rows; MN-contiguous ones add 16*s rows and 32*i columns.
template <bool KC, int R, int BK>
__device__ __forceinline__ unsigned frag_offset(int first, int lane, int s)
{
    const int lr = lane & 31, lk = lane >> 5, q = lane >> 4, j = lane & 15;
    if (KC) {
        const int r = first + lr;
        return (unsigned)(r * BK * 2 + 16 * ((2 * s + lk) ^ swz_a<BK / 8>(r)));
    }
    const int kq = 8 * (q >> 1) + (j >> 2);     // row within a 16-row substep (plus 4*h)
    const int n = first + 16 * (q & 1) + 4 * (j & 3);
    return (unsigned)(kq * R * 2 + 16 * ((n >> 3) ^ swz_b(kq)) + 2 * (n & 7));
}

// A direct-to-LDS tile: BM x BN outputs of WM x WN waves, BK-k slices of both
// operands in a ring of STAGES slots.
template <int BM_, int BN_, int STAGES_, int WM_, int WN_, int BK_, bool SPLITS_ = false>
struct HgDmaCfg {
    static constexpr int BM = BM_, BN = BN_, BK = BK_, STAGES = STAGES_, WM = WM_, WN = WN_;
    static constexpr bool SPLITS = SPLITS_;   // also built with a K split over workgroups
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int A_CPR = BK / 8;                        // 16-byte chunks per A row
    static constexpr int TM = BM / WM, TN = BN / WN;
    static constexpr int FM = TM / 32, FN = TN / 32;
    static constexpr int A_BYTES = BM * BK * 2;                 // one A slice
    static constexpr int B_BYTES = BK * BN * 2;                 // one B slice
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    // A 1 KB direct-to-LDS load occupies the CU's vector-memory path for about
    // 16 cycles, and a wave blocked on issuing loads cannot issue MFMAs.  With
    // a two-slot ring the upper half of the waves (one per SIMD) issues every
    // load, right after the barrier that frees a slot, and the other wave on
    // each SIMD keeps the matrix core busy meanwhile.  With three or more
    // slots (STAGGER) every wave loads a share: the lower half right after the
    // barrier, the upper half two substeps before the next one, into the slot
    // that the previous barrier freed, so the two waves of a SIMD block on
    // their loads at different times.
    static constexpr bool STAGGER = STAGES >= 3;
    static constexpr int LW = STAGGER ? NW : NW / 2;            // loading waves
    static constexpr int A_LOADS = A_BYTES / 1024 / LW;         // per loading wave per slice
    static constexpr int B_LOADS = B_BYTES / 1024 / LW;
    static_assert(A_BYTES % (1024 * LW) == 0 && B_BYTES % (1024 * LW) == 0, "slices must split over the loaders");
    static_assert(A_CPR == 4 || A_CPR == 8, "K-contiguous rows of 64 or 128 bytes");
    static_assert(STAGES * STAGE_BYTES <= 160 * 1024, "LDS ring too large");
};

}  // namespace mi355gemm
