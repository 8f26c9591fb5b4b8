// attn_many.hip -- attention of many rows (prompts, and prefixes that requests
// share): tiles of 128 rows, keys and values through LDS.
//
// Four waves of 32 rows share a step's keys and values, 16 KB each (128, 64 or 32
// positions of heads of up to 64, 128 or 256 columns), which go from memory
// into LDS directly, one step ahead.  Products are v_mfma_f32_32x32x16: keys as the
// first operand, queries (in registers) as the second, so lane l (c = l & 31, h
// = l >> 5) has row c's scores at positions 8 b + 4 h + i: the second operand of the
// product with the values, as they lie.  That one's first operand, values by
// column, comes from LDS by transposing reads (four lanes give 4 positions' 16
// columns each; a lane gets one column's 4 positions).  Two workgroups share a
// compute unit: while one's waves exponentiate, the other's multiply.
#include "attn_device.h"

#pragma clang fp contract(off)

namespace hca {
namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kBytes = 16384;  // of a step's keys, and of its values

template <bool H>
__device__ __forceinline__ f32x16_t mfma32(u32x4 a, u32x4 b, f32x16_t c)
{
    if constexpr (H)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(hcp::f16x8_t, a), __builtin_bit_cast(hcp::f16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(hcp::bf16x8_t, a), __builtin_bit_cast(hcp::bf16x8_t, b), c, 0, 0, 0);
}

typedef __attribute__((address_space(3))) char* lbytes;

__device__ __forceinline__ u32x4 lds16(lbytes p) { return *(__attribute__((address_space(3))) u32x4*)p; }

__device__ __forceinline__ u32x2 lds_columns(lbytes p)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p));
}

__device__ __forceinline__ void dma16(gbytes from, lbytes to)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

// Ones where the numbers are infinities of the sign, or NaN.
template <bool H>
__device__ __forceinline__ u32x4 stray(u32x4 x, bool negative)
{
    constexpr uint32_t inf = H ? 0x7c00u : 0x7f80u, one = H ? 0x3c00u : 0x3f80u;
    const auto is = [&](uint32_t b) {
        const uint32_t m = b & 0x7fffu;
        return m > inf || (m == inf && (b >> 15) == (negative ? 1u : 0u)) ? one : 0u;
    };
#pragma unroll
    for (int c = 0; c < 4; ++c)
        x[c] = is(x[c] & 0xffffu) | is(x[c] >> 16) << 16;
    return x;
}

// Where 16-byte chunk c of row `row` lies in the row: eight rows' chunks in different
// banks (keys, read 16 bytes a lane), four rows' pairs of chunks (values).
template <int DP>
__device__ __forceinline__ int key_place(int c, int row) { return c ^ (row & 7); }
template <int DP>
__device__ __forceinline__ int value_place(int c, int row) { return c ^ 2 * (row & (DP == 64 ? 3 : 7)); }

template <int DP, bool H, bool FULL>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void many_rows(AttendArgs a)
{
    constexpr int UNIT = kBytes / (2 * DP), BLOCKS = UNIT / 32, KK = DP / 16, DB = DP / 32, ROW = 2 * DP;
    constexpr int CHUNKS = DP / 8, PER = 64 / CHUNKS, SENDS = 4;  // rows of one load, loads of a wave for each of a step's halves
    __shared__ __align__(1024) char k0[kBytes], k1[kBytes], v0[kBytes], v1[kBytes];
    __shared__ int sums[16];
    static_assert(2 * (kMaxSegments + 1) <= kBytes && 4 * (kMaxTiles + 1) <= 3 * kBytes, "the plan's lists");

    const int w = (blockIdx.x & 7) * (kWorkers / 8) + (blockIdx.x >> 3);  // neighbours on one XCD
    Start plan;
    if (threadIdx.x == 0)
        ((Record*)a.records)[w] = Record{};
    const auto at = [&](int i) -> int& {
        return i < kBytes / 4 ? ((int*)v0)[i] : i < kBytes / 2 ? ((int*)v1)[i - kBytes / 4] : ((int*)k1)[i - kBytes / 2];
    };
    if (!make_plan<kManyRows, UNIT, kThreads>(a, w, (uint16_t*)k0, at, sums, plan))
        return;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int c = lane & 31, h = lane >> 5;
    const int D = a.cache.dim;

    walk<kManyRows, UNIT>(a, plan, [&](const Segment& seg, int rt, int head, int u0, int u1, bool begins, bool ends, int last) {
        const Row row = row_of(a, seg, head, rt * kManyRows + 32 * wave + c);
        u32x4 q[KK];
        {
            const gbytes p = (gbytes)a.q.x + row.t * a.q.row + row.h * a.q.head;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                q[kk] = row.real && (FULL || 16 * kk + 8 * h < D) ? load16(p + 32 * kk + 16 * h) : u32x4{};
        }
        // positions that all of the wave's rows see, and that any sees
        int all_lo = row.real ? row.lo : 0, all_hi = row.real ? row.hi : 0x7fffffff;
        int any_lo = row.lo < row.hi ? row.lo : 0x7fffffff, any_hi = row.hi;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            all_lo = max(all_lo, __shfl_xor(all_lo, d));
            all_hi = min(all_hi, __shfl_xor(all_hi, d));
            any_lo = min(any_lo, __shfl_xor(any_lo, d));
            any_hi = max(any_hi, __shfl_xor(any_hi, d));
        }
        all_lo = __builtin_amdgcn_readfirstlane(all_lo);
        all_hi = __builtin_amdgcn_readfirstlane(all_hi);
        any_lo = __builtin_amdgcn_readfirstlane(any_lo);
        any_hi = __builtin_amdgcn_readfirstlane(any_hi);

        f32x16_t o[DB] = {};
        float m = kLowest, l = 0.0f;

        // This wave's rows of a step: UNIT / 4 neighbours, 16 of one page.
        constexpr int MINE = UNIT / 4, LOOKUPS = MINE > 16 ? MINE / 16 : 1;
        int32_t page[LOOKUPS];
        const auto look_up = [&](int u) {
            if (u < u1) {
#pragma unroll
                for (int i = 0; i < LOOKUPS; ++i)
                    page[i] = page_at(a, seg, u * UNIT + MINE * wave + 16 * i);
            }
        };
        const auto send = [&](int u, lbytes ks, lbytes vs) {
            const int in = lane / CHUNKS, ch = lane % CHUNKS;
#pragma unroll
            for (int x = 0; x < LOOKUPS; ++x) {
                const Page p = page_of(a, seg, head, u * UNIT + MINE * wave + 16 * x, page[x]);
#pragma unroll
                for (int i = x * SENDS / LOOKUPS; i < (x + 1) * SENDS / LOOKUPS; ++i) {
                    const int at = PER * i + in, there = min(at - 16 * x, p.last);  // row of this wave's, row from the page's on
                    const int tile_row = MINE * wave + at;
                    const int kc = key_place<DP>(ch, tile_row), vc = value_place<DP>(ch, tile_row);
                    const lbytes to_k = ks + (MINE * wave + PER * i) * ROW, to_v = vs + (MINE * wave + PER * i) * ROW;
                    const gbytes fk = p.k + (unsigned)(there * p.k_row + 16 * kc), fv = p.v + (unsigned)(there * p.v_row + 16 * vc);
                    dma16(FULL || 8 * kc < D ? fk : (gbytes)(const char*)kNoRow, to_k);
                    dma16(FULL || 8 * vc < D ? fv : (gbytes)(const char*)kNoRow, to_v);
                }
            }
        };

        const auto step = [&](int u, lbytes ks, lbytes vs) {
            const int j0 = u * UNIT;
            if (j0 + UNIT <= any_lo || j0 >= any_hi)
                return;
            f32x16_t s[BLOCKS];
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                s[b] = f32x16_t{};
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
                    s[b] = mfma32<H>(lds16(ks + (32 * b + c) * ROW + 16 * key_place<DP>(2 * kk + h, c)), q[kk], s[b]);
            }
            if (a.cap_out != 0.0f) {
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[b][i] = capped(a, s[b][i]);
            } else {
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[b][i] *= a.scale;
            }
            if (a.slopes) {
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[b][i] = fmaf(-row.slope, fabsf(row.p - (float)(j0 + 32 * b + 8 * (i >> 2) + 4 * h + (i & 3))), s[b][i]);
            }
            const bool some_hidden = j0 < all_lo || j0 + UNIT > all_hi;
            if (some_hidden) {
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = j0 + 32 * b + 8 * (i >> 2) + 4 * h + (i & 3);
                        s[b][i] = j >= row.lo && j < row.hi ? s[b][i] : -INFINITY;
                    }
            }
            float top = s[0][0];
#pragma unroll
            for (int i = 1; i < 16 * BLOCKS; ++i)
                top = fmaxf(top, s[i >> 4][i & 15]);
            top = max32(top);
            const bool past = top > m + kSlack;
            if (__any(past)) {
                const float to = past ? top : m, by = exp2_of(m - to);
                l *= by;
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    o[d] *= by;
                m = to;
            }
            u32x4 p[BLOCKS][2];
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float x = exp2_of(s[b][i] - m), y = exp2_of(s[b][i + 1] - m);
                    l += x + y;
                    p[b][i >> 3][(i >> 1) & 3] = pack2<H>(x, y);
                }
            // (a lane's address: position e of 4, half `hb` of 32 columns, 4 columns q)
            const int e = (lane & 15) >> 2, hb = (lane >> 4) & 1, qc = lane & 3;
            const lbytes from = vs + (4 * h + e) * ROW + 8 * (qc & 1);
            const auto values = [&](int d, int b, int x) {
                const lbytes at = from + 16 * value_place<DP>(4 * d + 2 * hb + (qc >> 1), 4 * h + e) + (32 * b + 16 * x) * ROW;
                const u32x2 lo = lds_columns(at), hi = lds_columns(at + 8 * ROW);
                return u32x4{lo[0], lo[1], hi[0], hi[1]};
            };
            if (!some_hidden) {
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int d = 0; d < DB; ++d)
                            o[d] = mfma32<H>(values(d, b, x), p[b][x], o[d]);
            } else {
                // A value that is no number reaches the rows that see its position alone: it is
                // left out of the product, and infinities and NaN are added where the product
                // of ones in their places with ones for what a row sees is not zero.
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        u32x4 sees;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = j0 + 32 * b + 16 * x + 8 * (i >> 1) + 4 * h + 2 * (i & 1);
                            constexpr uint32_t one = H ? 0x3c00u : 0x3f80u;
                            sees[i] = (j >= row.lo && j < row.hi ? one : 0u) | (j + 1 >= row.lo && j + 1 < row.hi ? one << 16 : 0u);
                        }
#pragma unroll
                        for (int d = 0; d < DB; ++d) {
                            const u32x4 y = values(d, b, x), finite = hcp::finite_of<H>(y);
                            const bool odd = (y[0] != finite[0]) | (y[1] != finite[1]) | (y[2] != finite[2]) | (y[3] != finite[3]);
                            o[d] = mfma32<H>(finite, p[b][x], o[d]);
                            if (__builtin_expect(__any(odd), 0)) {
                                const f32x16_t plus = mfma32<H>(stray<H>(y, false), sees, f32x16_t{}), minus = mfma32<H>(stray<H>(y, true), sees, f32x16_t{});
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    o[d][i] += (plus[i] > 0.0f ? INFINITY : 0.0f) + (minus[i] > 0.0f ? -INFINITY : 0.0f);
                            }
                        }
                    }
            }
        };

        // A step's loads have landed and the step before it is read, for all waves: the
        // next one's go where that one was.
        const auto turn = [&] {
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        look_up(u0);
        __syncthreads();  // (the plan's lists, or the item before, are read)
        send(u0, (lbytes)k0, (lbytes)v0);
        look_up(u0 + 1);
        for (int u = u0; u < u1; u += 2) {
            turn();
            if (u + 1 < u1)
                send(u + 1, (lbytes)k1, (lbytes)v1);
            look_up(u + 2);
            step(u, (lbytes)k0, (lbytes)v0);
            if (u + 1 == u1)
                break;
            turn();
            if (u + 2 < u1)
                send(u + 2, (lbytes)k0, (lbytes)v0);
            look_up(u + 3);
            step(u + 1, (lbytes)k1, (lbytes)v1);
        }

        const Target to = target_of<kManyRows>(a, w, seg, DP, begins, ends);
        const float sum = sum32(l);
        if (row.real) {
            const int mine = 32 * wave + c;
            if (to.sums) {
                const int64_t at = to.dense ? (int64_t)row.t * a.q_heads + row.h : mine;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (FULL || 32 * d + 8 * i < D)
                            *(f32x4_t*)(to.sums + at * DP + 32 * d + 8 * i + 4 * h) = f32x4_t{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
                if (h == 0)
                    to.ml[at] = float2{m, sum};
            } else {
                const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
                char* const out = a.out + row.t * a.out_row + row.h * a.out_head;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (FULL || 32 * d + 8 * i < D)
                            *(u32x2*)(out + 2 * (32 * d + 8 * i + 4 * h)) =
                                u32x2{pack2<H>(o[d][4 * i] * by, o[d][4 * i + 1] * by), pack2<H>(o[d][4 * i + 2] * by, o[d][4 * i + 3] * by)};
            }
        }
        if (begins && !ends && threadIdx.x == 0) {
            Record rec{};
            rec.t0 = seg.t0;
            rec.row0 = rt * kManyRows;
            rec.rows = min(kManyRows, seg.n * a.group - rt * kManyRows);
            rec.head = head;
            rec.last = last;
            ((Record*)a.records)[w] = rec;
        }
    });
}

template <int DP, bool H>
void run(const AttendArgs& a, hipStream_t s)
{
    if (a.cache.dim == DP)
        many_rows<DP, H, true><<<kWorkers, kThreads, 0, s>>>(a);
    else
        many_rows<DP, H, false><<<kWorkers, kThreads, 0, s>>>(a);
}

template <bool H>
void run(const AttendArgs& a, hipStream_t s)
{
    switch (padded(a.cache.dim)) {
    case 64: run<64, H>(a, s); break;
    case 128: run<128, H>(a, s); break;
    default: run<256, H>(a, s);
    }
}

}  // namespace

hipError_t launch_many(const AttendArgs& a, bool half, hipStream_t s)
{
    half ? run<true>(a, s) : run<false>(a, s);
    return hipGetLastError();
}

}  // namespace hca
