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

constexpr int kThreads = 256, kBytes = kStepBytes;  // of a step's keys, and of its values

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

// Where 16-byte chunk c of row `row` lies in the row: eight rows' chunks in different
// banks (keys, read 16 bytes a lane), four rows' pairs of chunks (values).
template <int DP>
__device__ __forceinline__ int key_place(int c, int row) { return c ^ (row & 7); }
template <int DP>
__device__ __forceinline__ int value_place(int c, int row) { return c ^ 2 * (row & (DP == 64 ? 3 : 7)); }

template <int DP, bool H, bool FULL>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void many_rows(AttendArgs)
{
    constexpr int UNIT = kBytes / (2 * DP), BLOCKS = UNIT / 32, KK = DP / 16, DB = DP / 32, ROW = 2 * DP;
    constexpr int CHUNKS = DP / 8, PER = 64 / CHUNKS, SENDS = 4;  // rows of one load, loads of a wave for each of a step's halves
    __shared__ __align__(1024) char k0[kBytes], k1[kBytes], v0[kBytes], v1[kBytes];
    __shared__ int sums[16];
    static_assert(2 * (kMaxSegments + 1) <= kBytes && 4 * (kMaxTiles + 1) <= 3 * kBytes, "the plan's lists");

    Start plan;
    int w;
    {
        Args& a = args();
        w = (blockIdx.x & 7) * (a.workers >> 3) + (blockIdx.x >> 3);  // neighbours on one XCD
        if (threadIdx.x == 0)
            ((Record*)a.records)[w] = Record{};
        const auto at = [&](int i) -> int& {
            return i < kBytes / 4 ? ((int*)v0)[i] : i < kBytes / 2 ? ((int*)v1)[i - kBytes / 4] : ((int*)k1)[i - kBytes / 2];
        };
        if (!make_plan<UNIT, kThreads>(a, w, (uint16_t*)k0, at, sums, plan))
            return;
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int c = lane & 31, h = lane >> 5;

    walk<UNIT>(args(), plan, [&](const Segment& seg, int rt, int head, int u0, int u1, bool begins, bool ends, int last) {
        Args& a = args();
        const int D = a.cache.dim;
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
        uint32_t odd = 0;
        const Stream str = stream_of(a, seg, head);
        const float scale = a.scale, cap_in = a.cap_in, cap_out = a.cap_out;
        const bool slopes = a.slopes != nullptr;

        // This wave's rows of a step: UNIT / 4 neighbours, 16 of one page.
        constexpr int MINE = UNIT / 4, LOOKUPS = MINE > 16 ? MINE / 16 : 1;
        int32_t page[LOOKUPS];
        const auto look_up = [&](int u) {
            if (u < u1) {
#pragma unroll
                for (int i = 0; i < LOOKUPS; ++i)
                    page[i] = page_at(str, u * UNIT + MINE * wave + 16 * i);
            }
        };
        const auto send = [&](int u, lbytes ks, lbytes vs) {
            const int in = lane / CHUNKS, ch = lane % CHUNKS;
#pragma unroll
            for (int x = 0; x < LOOKUPS; ++x) {
                const Page p = page_of(str, u * UNIT + MINE * wave + 16 * x, page[x]);
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

        // (a lane's address of values: position e of 4, half `hb` of 32 columns, 4 columns)
        const int e = (lane & 15) >> 2, hb = (lane >> 4) & 1;
        const auto values = [&](lbytes vs, int d, int at) {  // of the 16 positions from `at` on
            const lbytes from = vs + (4 * h + e) * ROW + 8 * (lane & 1) + 16 * value_place<DP>(4 * d + 2 * hb + ((lane & 3) >> 1), 4 * h + e) + at * ROW;
            const u32x2 lo = lds_columns(from), hi = lds_columns(from + 8 * ROW);
            return u32x4{lo[0], lo[1], hi[0], hi[1]};
        };
        const auto block = [&](int j0, lbytes ks, lbytes vs) {  // 32 positions
            f32x16_t s{};
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                s = mfma32<H>(lds16(ks + c * ROW + 16 * key_place<DP>(2 * kk + h, c)), q[kk], s);
            if (cap_out != 0.0f) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[i] = capped(s[i], cap_in, cap_out);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[i] *= scale;
            }
            if (slopes) {
                const float far = row.p - (float)(j0 + 4 * h);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[i] = fmaf(-row.slope, fabsf(far - (float)(8 * (i >> 2) + (i & 3))), s[i]);
            }
            const bool some_hidden = j0 < all_lo || j0 + 32 > all_hi;
            if (some_hidden) {
                const unsigned past_lo = j0 + 4 * h - row.lo, span = row.hi - row.lo;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[i] = past_lo + (unsigned)(8 * (i >> 2) + (i & 3)) < span ? s[i] : -INFINITY;
            }
            float top = s[0];
#pragma unroll
            for (int i = 1; i < 16; ++i)
                top = fmaxf(top, s[i]);
            top = max32(top);
            const bool past = top > m + kSlack;
            if (__any(past)) {
                const float to = past ? top : m, by = weight_of(m - to);
                l *= by;
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    o[d] *= by;
                m = to;
            }
            u32x4 p[2];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float x = exp2_of(s[i] - m), y = exp2_of(s[i + 1] - m);
                l += x + y;
                p[i >> 3][(i >> 1) & 3] = pack2<H>(x, y);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                u32x4 y[DB];
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    y[d] = values(vs, d, 16 * x);
                if (some_hidden) {  // a value that is no number is left out: it belongs to the rows that see it (see below)
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const u32x4 finite = hcp::finite_of<H>(y[d]);
                        odd |= (y[d][0] ^ finite[0]) | (y[d][1] ^ finite[1]) | (y[d][2] ^ finite[2]) | (y[d][3] ^ finite[3]);
                        y[d] = finite;
                    }
                }
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    o[d] = mfma32<H>(y[d], p[x], o[d]);
            }
        };
        const auto step = [&](int u, lbytes ks, lbytes vs) {
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                const int j0 = u * UNIT + 32 * b;
                if (j0 + 32 > any_lo && j0 < any_hi)
                    block(j0, ks + 32 * b * ROW, vs + 32 * b * ROW);
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

        // Infinities and NaN among values that some row of the wave does not see: added to the
        // rows that do.
        if (__builtin_expect(__any(odd != 0), 0)) {
            const unsigned span = row.hi - row.lo;
            for (int j0 = u0 * UNIT; j0 < u1 * UNIT; j0 += 16) {
                if ((j0 & ~31) >= all_lo && (j0 | 31) < all_hi)
                    continue;
                const Page p = page_of(str, j0, page_at(str, j0));
                for (int j = j0; j < min(j0 + 16, str.L); ++j) {
                    const bool sees = (unsigned)(j - row.lo) < span;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (FULL || 32 * d + 8 * i < D) {
                                const u32x2 y = load8(p.v + (unsigned)((j - j0) * p.v_row + 2 * (32 * d + 8 * i + 4 * h)));
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    o[d][4 * i + e] += odd_part<H>(y[e >> 1] >> 16 * (e & 1), sees);
                            }
                }
            }
        }

        Args& z = args();
        const Target to = target_of(z, w, seg, DP, begins, ends);
        const float sum = sum32(l);
        if (row.real) {
            const int mine = 32 * wave + c;
            if (to.sums) {
                const int64_t at = to.dense ? (int64_t)row.t * z.q_heads + row.h : mine;
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
                char* const out = z.out + row.t * z.out_row + row.h * z.out_head;
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
            rec.rows = min(kManyRows, seg.n * z.group - rt * kManyRows);
            rec.head = head;
            rec.last = last;
            ((Record*)z.records)[w] = rec;
        }
    });
}

template <int DP, bool H>
void run(const AttendArgs& a, hipStream_t s)
{
    if (a.cache.dim == DP)
        many_rows<DP, H, true><<<a.workers, kThreads, 0, s>>>(a);
    else
        many_rows<DP, H, false><<<a.workers, kThreads, 0, s>>>(a);
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
