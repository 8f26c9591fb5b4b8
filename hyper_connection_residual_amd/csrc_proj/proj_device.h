// proj_device.h -- device helpers shared by the projections' kernels.
//
// Operand layout of every matrix product here: v_mfma_f32_16x16x32 with the
// weights as its first operand and the tokens as its second.  Lane l (l & 15 =
// r, l >> 4 = g) holds row r's 8 consecutive k at 8 g, of both operands, and of
// the product the 4 outputs 4 g + i of token r.  So one lane's results are
// neighbours of one token's row of out, and which adapter a token has is a
// matter of the lane.
#pragma once

#include "proj_internal.h"

#include <type_traits>

namespace hcp {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(1))) char* gbytes;

// What a row or a piece of a row that does not exist reads: zeros.
__device__ static const uint4 kZeros[1] = {{0, 0, 0, 0}};

__device__ __forceinline__ gbytes zeros() { return (gbytes)(const char*)kZeros; }

__device__ __forceinline__ u32x4 load16(gbytes p)
{
    return *(const __attribute__((address_space(1))) u32x4*)p;
}

template <bool H>
__device__ __forceinline__ f32x4_t mfma(u32x4 a, u32x4 b, f32x4_t c)
{
    if constexpr (H)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                      __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// 16-bit bits of x, to nearest even (NaN stays NaN, fp16 overflows to inf).
template <bool H>
__device__ __forceinline__ uint32_t bits16(float x)
{
    if constexpr (H)
        return __builtin_bit_cast(uint16_t, (_Float16)x);
    else
        return __builtin_bit_cast(uint16_t, (__bf16)x);
}

template <bool H>
__device__ __forceinline__ float from16(uint32_t b)
{
    if constexpr (H)
        return (float)__builtin_bit_cast(_Float16, (uint16_t)b);
    else
        return __builtin_bit_cast(float, b << 16);
}

// silu(g) u in fp32.  exp(-g) overflows to inf for g < -88, whose reciprocal is
// the zero that silu has there to within 1e-36.  The hardware's reciprocal (one
// unit in the last place) in place of a division: 64 of these per lane end a
// wide tile.
__device__ __forceinline__ float gated(float g, float u)
{
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Where row tile `want` (tiles of BM rows that start at each group's first
// row) lies.  Waves run it redundantly on their 64 lanes.
struct RowTile {
    int e, row0, rows;
};

__device__ __forceinline__ void group_range(const int32_t* off, int E, int M, int e, int& lo, int& hi)
{
    lo = hi = 0;
    if (e < E) {
        lo = min(max(off[e], 0), M);
        hi = min(max(off[e + 1], lo), M);
    }
}

// More tiles than any launch has workgroups: counts are cut there, so that those
// of offsets that are not in order stay in 32 bits too (64 lanes' sum: 2^30).
constexpr int kMostTiles = 1 << 24;

template <int BM>
__device__ __forceinline__ int count_tiles(const int32_t* off, int E, int M)
{
    if (!off)
        return (M + BM - 1) / BM;
    int sum = 0;
    for (int e = threadIdx.x & 63; e < E; e += 64) {
        int lo, hi;
        group_range(off, E, M, e, lo, hi);
        sum = min(sum + min((hi - lo + BM - 1) / BM, kMostTiles), kMostTiles);
    }
    for (int d = 32; d; d >>= 1)
        sum += __shfl_xor(sum, d);
    return __builtin_amdgcn_readfirstlane(sum);
}

template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* off, int E, int M, int want, RowTile& t)
{
    if (!off) {
        t.e = 0;
        t.row0 = want * BM;
        t.rows = min(BM, M - t.row0);
        return t.rows > 0;
    }
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int c = 0; c < E; c += 64) {
        int lo, hi;
        group_range(off, E, M, c + lane, lo, hi);
        const int n = min((hi - lo + BM - 1) / BM, kMostTiles);
        int upto = n;
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(upto, d);
            upto += lane >= d ? o : 0;
        }
        const unsigned long long past = __ballot(base + upto > want);
        if (past) {
            const int L = __builtin_ctzll(past);
            const int before = base + __builtin_amdgcn_readlane(upto, L) - __builtin_amdgcn_readlane(n, L);
            t.e = c + L;
            t.row0 = __builtin_amdgcn_readlane(lo, L) + (want - before) * BM;
            t.rows = min(BM, __builtin_amdgcn_readlane(hi, L) - t.row0);
            return true;
        }
        base += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// Row `i` of a tile: its bytes in x, or NULL where it has none (past the tile,
// or a gathered row that x does not have).
__device__ __forceinline__ gbytes x_row(const ProductArgs& a, const RowTile& t, int i)
{
    if (i >= t.rows)
        return nullptr;
    int64_t r = (int64_t)t.row0 + i;
    if (a.rows)
        r = a.rows[r];
    return r >= 0 && r < a.x_rows ? (gbytes)a.x + r * a.ldx : nullptr;
}

// 16 and 8 bytes at any address of their elements (rows of odd length lie so).
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef f32x4_t f32x4_at4 __attribute__((aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));

// COUNT results of one token from output n on, COUNT a multiple of 4.
template <bool H, int COUNT>
__device__ __forceinline__ void store_row(const ProductArgs& a, int64_t row, int n, const float (&y)[COUNT])
{
    if (n >= a.N)
        return;
    const int64_t at = row * a.ldo + n;
    if (n + COUNT <= a.N) {
        if (a.out32) {
            u32x4_at4* p = (u32x4_at4*)(a.out + 4 * at);
#pragma unroll
            for (int c = 0; c < COUNT / 4; ++c)
                p[c] = u32x4{__float_as_uint(y[4 * c]), __float_as_uint(y[4 * c + 1]),
                             __float_as_uint(y[4 * c + 2]), __float_as_uint(y[4 * c + 3])};
        } else {
            uint32_t w[COUNT / 2];
#pragma unroll
            for (int c = 0; c < COUNT / 2; ++c)
                w[c] = bits16<H>(y[2 * c]) | bits16<H>(y[2 * c + 1]) << 16;
            if constexpr (COUNT % 8 == 0) {
                u32x4_at2* p = (u32x4_at2*)(a.out + 2 * at);
#pragma unroll
                for (int c = 0; c < COUNT / 8; ++c)
                    p[c] = u32x4{w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]};
            } else {
                u32x2_at2* p = (u32x2_at2*)(a.out + 2 * at);
#pragma unroll
                for (int c = 0; c < COUNT / 4; ++c)
                    p[c] = u32x2{w[2 * c], w[2 * c + 1]};
            }
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < COUNT; ++c) {
        if (n + c < a.N) {
            if (a.out32)
                ((float*)a.out)[at + c] = y[c];
            else
                ((uint16_t*)a.out)[at + c] = (uint16_t)bits16<H>(y[c]);
        }
    }
}

// Piece `which` of x == p0 + p1 + p2 exactly, each a bf16 (the top 8 significant
// bits of what is left); an infinity or NaN is its first piece alone.
__device__ __forceinline__ uint32_t piece(float x, int which)
{
    const uint32_t b = __float_as_uint(x);
    const float r1 = x - __uint_as_float(b & 0xffff0000u);
    const uint32_t m = __float_as_uint(r1) & 0xffff0000u;
    const float r2 = r1 - __uint_as_float(m);
    const bool finite = (b & 0x7f800000u) != 0x7f800000u;
    const uint32_t first = b >> 16 | (!finite && (b & 0xffffu) ? 1u : 0u);  // (a NaN that the cut would make inf stays one)
    const uint32_t other = finite ? (which == 1 ? m : __float_as_uint(r2)) >> 16 : 0u;
    return which ? other : first;
}

// Of two fp16 numbers (exactly two bf16 pieces each) the first piece, their top 8
// significant bits, or the second.  (Of an infinity or NaN at least one piece is
// one, too.  The bits are those of the fp32 number: the smallest fp16 numbers, too,
// have a first piece other than zero, which an infinite v times it needs.)
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t half_piece(uint32_t both, bool second)
{
    const f16x2_t p = __builtin_bit_cast(f16x2_t, both);
    const float f0 = (float)p[0], f1 = (float)p[1];
    const uint32_t taken = second ? 0xffff0000u : 0u;
    const float r0 = f0 - __uint_as_float(__float_as_uint(f0) & taken), r1 = f1 - __uint_as_float(__float_as_uint(f1) & taken);
    return __float_as_uint(r0) >> 16 | (__float_as_uint(r1) & 0xffff0000u);
}

// Two numbers' exponents of ones: an infinity's or NaN's.
constexpr uint32_t exponents(bool half) { return half ? 0x7c007c00u : 0x7f807f80u; }

// 16-bit numbers with zeros for the infinities and NaNs among them.
template <bool H>
__device__ __forceinline__ u32x4 finite_of(u32x4 p)
{
    constexpr uint32_t low = exponents(H) & 0xffffu, high = exponents(H) & 0xffff0000u;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        p[c] &= ((p[c] & low) == low ? 0u : 0xffffu) | ((p[c] & high) == high ? 0u : 0xffff0000u);
    return p;
}

// 16-bit numbers with, for the infinities among them, the smallest normal numbers of
// their signs, and zeros for the NaNs.
template <bool H>
__device__ __forceinline__ u32x4 stand_ins(u32x4 p)
{
    constexpr uint32_t low = exponents(H) & 0xffffu;
    constexpr uint32_t least = low & ~(low << 1);
    const auto one = [](uint32_t b) { return (b & low) != low ? b : (b & 0x7fffu) == low ? (b & 0x8000u) | least : 0u; };
#pragma unroll
    for (int c = 0; c < 4; ++c)
        p[c] = one(p[c] & 0xffffu) | one(p[c] >> 16) << 16;
    return p;
}

}  // namespace hcp
