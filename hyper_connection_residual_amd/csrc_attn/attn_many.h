// attn_many.h -- attention of many rows (prompts, and prefixes that requests
// share): tiles of 128 or 256 rows, keys and values through LDS.
//
// Four or eight waves of 32 rows share a step's keys and values, 16 KB each (128, 64
// or 32 positions of heads of up to 64, 128 or 256 columns), which go from memory
// into LDS directly, one step ahead.  Products are v_mfma_f32_32x32x16: keys as the
// first operand, queries (in registers) as the second, so lane l (c = l & 31, h
// = l >> 5) has row c's scores at positions 8 b + 4 h + i: the second operand of the
// product with the values, as they lie.  That one's first operand, values by
// column, comes from LDS by transposing reads (four lanes give 4 positions' 16
// columns each; a lane gets one column's 4 positions).  Of tiles of 128 rows and heads of up to 128
// columns, two workgroups share a compute unit: while one's waves exponentiate, the other's multiply.
// Tiles of 256 rows, and wider heads, have one each, for their registers.
//
// 8192 tokens of 3 requests over up to 6000 positions before them, 20 heads over 4 of 128
// columns (311 GFLOP): 354 us with the join, 0.88 PFLOP/s, the matrix cores 41 % busy;
// left are exponentials, a SIMD's two waves in step with each other behind the barrier, and
// the loads' sending.  128 rows take twice the bytes from L2 into LDS (386 us); 64 rows a
// wave leave each SIMD one wave, whose products cover nothing of its own exponentials (530).
#pragma once

#include "attn_device.h"

#pragma clang fp contract(off)

namespace hca {
namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// Where there is no cap and no bias, a product becomes a score in the subtraction of its row's maximum, unrounded; the
// maximum itself is rounded.  From this maximum on (over ln 2; that rounding moves the difference by up to
// 2^-5 there, and past the exponential's range from 2^31 on) scores are rounded before, as the maximum is.
constexpr float kLarge = 0x1p20f;

constexpr int kBytes = kStepBytes;  // of a step's keys, and of its values

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

// 16 bytes a lane from memory into LDS, at `to` + 16 lane.  In assembly, so that the compiler does
// not make every read of LDS wait for all of these loads: no register takes their
// results, and the waves wait before any of them is read.  (m0 is the compiler's.)
__device__ __forceinline__ void dma16(gbytes base, uint32_t offset, uint32_t to)
{
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "v"(offset), "s"(base), "s"(to)
                 : "memory");
}
// Four or eight of them: keys to `to` and the next KBs, values to 32 KB behind.
__device__ __forceinline__ void dma_step(const gbytes (&k)[4], const gbytes (&v)[4], const uint32_t (&k_at)[4], const uint32_t (&v_at)[4], uint32_t to)
{
    uint32_t m0;
    static_assert(kBytes == 16384, "32 KB from keys to values");
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %2, %10\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %3, %11\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %4, %12\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %5, %13\n\ts_add_u32 m0, m0, 0x7400\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %6, %14\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %7, %15\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %8, %16\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %9, %17\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(to), "v"(k_at[0]), "v"(k_at[1]), "v"(k_at[2]), "v"(k_at[3]), "v"(v_at[0]), "v"(v_at[1]), "v"(v_at[2]), "v"(v_at[3]),
                   "s"(k[0]), "s"(k[1]), "s"(k[2]), "s"(k[3]), "s"(v[0]), "s"(v[1]), "s"(v[2]), "s"(v[3])
                 : "memory", "scc");
}
__device__ __forceinline__ void dma_step(const gbytes (&k)[2], const gbytes (&v)[2], const uint32_t (&k_at)[2], const uint32_t (&v_at)[2], uint32_t to)
{
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %2, %6\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %3, %7\n\ts_add_u32 m0, m0, 0x7c00\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %4, %8\n\ts_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
                 "global_load_lds_dwordx4 %5, %9\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(to), "v"(k_at[0]), "v"(k_at[1]), "v"(v_at[0]), "v"(v_at[1]), "s"(k[0]), "s"(k[1]), "s"(v[0]), "s"(v[1])
                 : "memory", "scc");
}

// Where 16-byte chunk c of row `row` lies in its row (and the chunk that lies at place c), so that the
// lanes that LDS serves together find different banks: of keys (16 bytes a lane, chunk 2 kk
// + h of rows c) rows 0 .. 7 with rows 8 .. 15 and with the other h; of values (8 bytes a
// lane) four rows' pairs of chunks with their neighbours and with the next four rows.  Four
// neighbours stay together: their lanes' loads are 64 bytes of one line.
template <int DP>
__device__ __forceinline__ int key_place(int c, int row)
{
    return c ^ ((DP == 64 ? row & 6 : (row & 7) << 1) | (row >> 3 & 1));
}
template <int DP>
__device__ __forceinline__ int value_place(int c, int row)
{
    return c ^ 2 * (DP == 64 ? (row & 2) | (row >> 2 & 1) : (row & 3) << 1 | (row >> 2 & 1));
}

// What a wave keeps of its worker's items.
struct State {
    Start plan;
    Walk way;
    Item items[3];  // what is read, and what was fetched behind it: up to two, if the first has one unit
};

// WAVES: of 32 rows each.  FULL: dim is DP.  EXTRA: there is a cap, or there are slopes, or the scale is zero.
template <int DP, int WAVES, bool H, bool FULL, bool EXTRA>
__global__ __launch_bounds__(64 * WAVES, DP <= 128 ? 2 : 1) void many_rows(AttendArgs)
{
    constexpr int kThreads = 64 * WAVES;
    constexpr int UNIT = kBytes / (2 * DP), BLOCKS = UNIT / 32, KK = DP / 16, DB = DP / 32, ROW = 2 * DP;
    constexpr int CHUNKS = DP / 8, PER = 64 / CHUNKS, SENDS = 16 / WAVES;  // rows of one load, loads of a wave for each of a step's halves
    __shared__ __align__(1024) char lds[4 * kBytes];  // two stages of keys, two of values
    __shared__ int sums[16];
    static_assert(2 * (kMaxSegments + 1) <= kBytes && 4 * (kMaxTiles + 1) <= 3 * kBytes && 4 * kBytes <= 65536, "the plan's lists");

    Start plan;
    int w;
    {
        Args& a = args();
        // Neighbours on one XCD, which share keys and values (documents 75 us, spread 78); but prefixes' steps, with all waves'
        // rows full, are longer than own positions' and lie side by side: spread over all (64 tokens under a prefix 34 us for 38).
        w = a.prefix.groups ? blockIdx.x : (blockIdx.x & 7) * (a.workers >> 3) + (blockIdx.x >> 3);
        if (threadIdx.x == 0)
            ((Record*)a.records)[w] = Record{};
        const auto at = [&](int i) -> int& { return ((int*)(lds + kBytes))[i]; };
        if (!make_plan<UNIT, kThreads>(a, w, (uint16_t*)lds, at, sums, plan))
            return;
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    __shared__ State states[WAVES];
    State& state = states[wave];
    const auto next = [&](Item& to) {  // this wave's next item; false: there is none
        Start p = taken(&state.plan);
        Walk x = taken(&state.way);
        Item y;
        const bool some = next_item<UNIT>(args(), p, x, y);
        state.way = x;
        to = y;
        return some;
    };
    state.plan = plan;
    state.way = walk_from(plan);
    int now = 0, last = 0;  // the item that is read, the last one fetched
    const auto behind = [](int i) { return i == 2 ? 0 : i + 1; };
    if (!next(state.items[0]))
        return;

    // What goes into LDS runs one step ahead of what is read, from one item into the next.
    constexpr int MINE = UNIT / WAVES, LOOKUPS = MINE > 16 ? MINE / 16 : 1;  // this wave's rows of a step, neighbours, 16 of one page
    constexpr int EACH = MINE / LOOKUPS;                                 // rows of a lookup
    static_assert(PER * SENDS == MINE && PER * ROW == 1024, "a wave's loads: 1 KB each");
    Stream from;
    int ahead, end;  // the unit to be sent next, of those up to `end`
    const auto begin = [&](const Item* item) {
        const Item y = taken(item);
        from = stream_of(args(), y.g, y.head);
        ahead = y.u0;
        end = y.u1;
    };
    begin(&state.items[0]);
    int32_t page[LOOKUPS];
    const auto look_up = [&](int u) {
#pragma unroll
        for (int i = 0; i < LOOKUPS; ++i)
            page[i] = page_in_lanes(from, u * UNIT + MINE * wave + 16 * i);
    };
    const uint32_t at_lds = (uint32_t)(uintptr_t)(lbytes)lds;
    // Where a lane's loads begin from their lookup's first row: the row, and the chunk that goes to its place.
    uint32_t k_at[SENDS], v_at[SENDS];
    {
        Args& a = args();
        const int lane = threadIdx.x & 63, in = lane / CHUNKS, ch = lane % CHUNKS;
#pragma unroll
        for (int i = 0; i < SENDS; ++i) {
            const int at = PER * i + in, row = MINE * wave + at;
            int kc = key_place<DP>(ch, row), vc = value_place<DP>(ch, row);
            if constexpr (!FULL) {  // (columns that the head does not have: its first ones, times queries of zero or for no one)
                kc = 8 * kc < a.cache.dim ? kc : 0;
                vc = 8 * vc < a.cache.dim ? vc : 0;
            }
            k_at[i] = __umul24(at % EACH, a.cache.k_row) + 16 * kc;
            v_at[i] = __umul24(at % EACH, a.cache.v_row) + 16 * vc;
        }
    }
    const auto send = [&](int u, int stage) {
        const uint32_t to = at_lds + stage * kBytes + MINE * wave * ROW;
        const int j = u * UNIT + MINE * wave, mask = (1 << from.shift) - 1;
        gbytes k[SENDS], v[SENDS];
        bool whole = j + MINE <= from.L;
#pragma unroll
        for (int x = 0; x < LOOKUPS; ++x) {
            const uint32_t p = __builtin_amdgcn_readfirstlane(page[x]), row = (j + 16 * x) & mask;
            whole = whole && p < (uint64_t)from.pages;
            const gbytes kx = from.k + (uint64_t)p * (uint32_t)from.k_page + (uint64_t)row * (uint32_t)from.k_row;
            const gbytes vx = from.v + (uint64_t)p * (uint32_t)from.v_page + (uint64_t)row * (uint32_t)from.v_row;
#pragma unroll
            for (int i = x * SENDS / LOOKUPS; i < (x + 1) * SENDS / LOOKUPS; ++i) {
                k[i] = kx;
                v[i] = vx;
            }
        }
        if (whole) {
            dma_step(k, v, k_at, v_at, to);
        } else {  // rows that the segment or the cache does not have
            const int lane = threadIdx.x & 63, in = lane / CHUNKS;
#pragma unroll 1
            for (int i = 0; i < SENDS; ++i) {
                const int x = i * LOOKUPS / SENDS, at = PER * i + in - EACH * x;
                const Page p = page_of(from, j + EACH * x, __builtin_amdgcn_readfirstlane(LOOKUPS > 1 && x ? page[LOOKUPS - 1] : page[0]));
                const int less = at - min(at, p.last);  // rows that are not there: the last that is
                uint32_t ka = k_at[0], va = v_at[0];
#pragma unroll
                for (int y = 1; y < SENDS; ++y) {
                    ka = i == y ? k_at[y] : ka;
                    va = i == y ? v_at[y] : va;
                }
                // (a page that is not there: its row's chunk, of zeros)
                ka = p.k_row ? ka - __umul24(less, p.k_row) : ka - __umul24(at, from.k_row);
                va = p.v_row ? va - __umul24(less, p.v_row) : va - __umul24(at, from.v_row);
                dma16(p.k, ka, to + 1024 * i);
                dma16(p.v, va, to + 1024 * i + 2 * kBytes);
            }
        }
    };
    bool more = true;  // there is a unit to be sent
    const auto advance = [&] {  // to the unit behind the one that was sent: its pages are on their way when it is sent
        if (++ahead == end) {
            more = next(state.items[behind(last)]);
            if (!more)
                return;
            last = behind(last);
            begin(&state.items[last]);
        }
        look_up(ahead);
    };
    __syncthreads();  // (the plan's lists are read)
    look_up(ahead);
    send(ahead, 0);
    advance();
    int stage = 0;

    for (;;) {
        Args& a = args();
        const int D = a.cache.dim;
        const Item item = taken(&state.items[now]);
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));  // (what is made of it is made for each item: kept from item to item, it takes 30 registers)
        const int c = lane & 31, h = lane >> 5;
        const Row row = row_of(a, item.g, item.head, item.rt * (32 * WAVES) + 32 * wave + c);
        u32x4 q[KK];
        {
            const gbytes p = (gbytes)a.q.x + row.t * a.q.row + row.h * a.q.head;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {  // (from row or column 0 instead: a load under a condition is waited for by itself)
                const bool there = FULL || 16 * kk + 8 * h < D;
                const u32x4 x = load16(p + (there ? 32 * kk + 16 * h : 0)) ^ a.q_sign;
                q[kk] = row.real && there ? x : u32x4{};
            }
        }
        // positions that all of the wave's rows see, and that any sees
        const int all_lo = __builtin_amdgcn_readfirstlane(most_of<32>(row.real ? row.lo : 0));
        const int all_hi = __builtin_amdgcn_readfirstlane(least_of<32>(row.real ? row.hi : 0x7fffffff));
        const int any_lo = __builtin_amdgcn_readfirstlane(least_of<32>(row.lo < row.hi ? row.lo : 0x7fffffff));
        const int any_hi = __builtin_amdgcn_readfirstlane(most_of<32>(row.hi));

        f32x16_t o[DB] = {};
        float m = kLowest, l = 0.0f;
        [[maybe_unused]] float bar = kLowest;  // of a score that makes for another reference, or is to be rounded (see kLarge)
        uint32_t odd = 0;
        [[maybe_unused]] const float scale = a.scale, cap_in = a.cap_in, cap_out = a.cap_out;
        [[maybe_unused]] const bool slopes = a.slopes != nullptr;

        // Where this lane reads in the first stage: row c's chunk h of keys (chunk 2 kk + h: ^ 2 kk); of the first
        // 32 columns' values (those from 32 d on: ^ d) position e of 4, half `hb` of the columns, 4 columns.
        const uint32_t key_at = at_lds + c * ROW + 16 * key_place<DP>(h, c);
        uint32_t value_at;
        {
            const int e = (lane & 15) >> 2, hb = (lane >> 4) & 1;
            value_at = at_lds + 2 * kBytes + (4 * h + e) * ROW + 8 * (lane & 1) + 16 * value_place<DP>(2 * hb + ((lane & 3) >> 1), 4 * h + e);
        }
        const auto values = [&](uint32_t base, int d, int at) {  // of 16 positions from the stage's position `at` on
            const lbytes p = (lbytes)(uintptr_t)(base ^ 64 * d) + at * ROW;
            const u32x2 lo = lds_columns(p), hi = lds_columns(p + 8 * ROW);
            return u32x4{lo[0], lo[1], hi[0], hi[1]};
        };
        const auto keys = [&](uint32_t base, int at, u32x4 (&k)[KK]) {  // of the 32 positions from `at` on
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                k[kk] = lds16((lbytes)(uintptr_t)(base ^ 32 * kk) + at * ROW);
            asm volatile("" ::: "memory");  // (all on their way at once: left to itself, each read waits for the product before it)
            __builtin_amdgcn_sched_barrier(0);
        };
        // 32 positions: their keys are k; the next 32's, if there are, on their way when this returns
        const auto block = [&](int j0, u32x4 (&k)[KK], uint32_t ks, uint32_t vs, int at) {
            f32x16_t s{};
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                s = mfma32<H>(k[kk], q[kk], s);
            // the values are on their way while the scores are worked on
            constexpr int HALVES = DP == 256 ? 1 : 2;  // (of wide heads, the registers hold 16 positions' values)
            u32x4 y[HALVES][DB];
#pragma unroll
            for (int x = 0; x < HALVES; ++x)
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    y[x][d] = values(vs, d, at + 16 * x);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (EXTRA) {  // scores over ln 2
                if (cap_out > kLargeCap) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[i] = capped<true>(s[i], cap_in, cap_out);
                } else if (cap_out != 0.0f) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[i] = capped<false>(s[i], cap_in, cap_out);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[i] *= scale;
                }
                if (slopes) {
                    const float far = (float)(row.p - (j0 + 4 * h));
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[i] = fmaf(-row.slope, fabsf(far - (float)(8 * (i >> 2) + (i & 3))), s[i]);
                }
            }
            const bool some_hidden = j0 < all_lo || j0 + 32 > all_hi;
            if (some_hidden) {
                const int j = j0 + 4 * h, lo = min(max(row.lo - j, 0), 31), n = min(max(row.hi - j, 0), 32) - lo;
                const uint32_t seen = n <= 0 || row.lo - j > 31 ? 0u : (0xffffffffu >> (32 - n)) << lo;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[i] = score_if(seen, 8 * (i >> 2) + (i & 3), s[i]);
            }
            const auto finite_only = [&] {  // a value that is no number is left out: it belongs to the rows that see it (see below)
                bool some = false;
#pragma unroll
                for (int x = 0; x < HALVES; ++x)
                    some = some || some_odd<H>(y[x]);
                if (!__any(some))
                    return;
#pragma unroll
                for (int x = 0; x < HALVES; ++x)
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const u32x4 finite = hcp::finite_of<H>(y[x][d]);
                        odd |= (y[x][d][0] ^ finite[0]) | (y[x][d][1] ^ finite[1]) | (y[x][d][2] ^ finite[2]) | (y[x][d][3] ^ finite[3]);
                        y[x][d] = finite;
                    }
            };
            float top = s[0];
#pragma unroll
            for (int i = 1; i < 16; ++i)
                top = fmaxf(top, s[i]);
            top = max32(top);
            if constexpr (!EXTRA)
                top *= scale;
            [[maybe_unused]] float times = scale;
            if (__any(EXTRA ? top - m > kMost<H> : top > bar)) {
                const bool past = EXTRA ? top - m > kMost<H> : top > bar_of<H>(m);  // (of this row: the others' change nothing in it)
                const float to = past ? reference_of<H>(top) : m, by = weight_of(m - to);
                l *= by;
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    o[d] *= by;
                m = to;
                if constexpr (!EXTRA) {
                    const bool large = fabsf(m) > kLarge && m > kLowest;
                    bar = large ? kLowest : bar_of<H>(m);
                    if (__any(large)) {  // (other rows' stay as they are, bit for bit)
                        const float before = large ? scale : 1.0f;
                        times = large ? 1.0f : scale;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            s[i] *= before;
                    }
                }
            }
            // Rounded once to the type of the second product.  With a second piece of each, outputs would
            // be as near to 64 bits as their own rounding allows (bf16: a relative 0.0017, with one 0.0020 to 0.0022); its products
            // cost too much here: a prompt of 8192 tokens 346 us and 464, documents 80 and 90, single tokens under a prefix 44 and 47.
            u32x4 p[2];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float x = exp2_of(EXTRA ? s[i] - m : fmaf(s[i], times, -m)), z = exp2_of(EXTRA ? s[i + 1] - m : fmaf(s[i + 1], times, -m));
                l += x + z;
                p[i >> 3][(i >> 1) & 3] = pack2<H>(x, z);
            }
            if (some_hidden)
                finite_only();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (x == 1) {
                    if constexpr (HALVES == 1) {
#pragma unroll
                        for (int d = 0; d < DB; ++d)
                            y[0][d] = values(vs, d, at + 16);
                        if (some_hidden)
                            finite_only();
                    }
                    if (at + 32 < UNIT)
                        keys(ks, at + 32, k);
                }
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    o[d] = mfma32<H>(y[x % HALVES][d], p[x], o[d]);
            }
            asm volatile("" ::: "memory");
        };

        const int u1 = item.u1;
        for (int u = item.u0; u < u1; ++u) {
            // This step's loads have landed and the step before it is read, for all waves: the
            // next one's go where that one was.
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            if (more) {
                send(ahead, stage ^ 1);
                advance();
            }
            const int j0 = u * UNIT;
            if (j0 + UNIT > any_lo && j0 < any_hi) {
                const uint32_t ks = key_at + stage * kBytes, vs = value_at + stage * kBytes;
                // its blocks that some row sees
                const int b0 = max(any_lo - j0, 0) >> 5, b1 = min((any_hi - j0 + 31) >> 5, BLOCKS);
                u32x4 k[KK];
                keys(ks, 32 * b0, k);
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
                    if (b >= b0 && b < b1)
                        block(j0 + 32 * b, k, ks, vs, 32 * b);
            }
            stage ^= 1;
        }

        Args& z = args();
        const Item done = taken(&state.items[now]);
        const Target to = target_of(z, w, done, DP);
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
        // Infinities and NaN among values that some row of the wave does not see: to what is
        // stored of the rows that do.
        if (__builtin_expect(__any(odd != 0), 0)) {
            const unsigned span = row.hi - row.lo;
            const Stream str = stream_of(z, done.g, done.head);
            const int64_t at = to.dense ? (int64_t)row.t * z.q_heads + row.h : 32 * wave + c;
            for (int col = 4 * h; col < D; col += 8) {
                f32x4_t sum{};
                for (int j0 = done.u0 * UNIT; j0 < done.u1 * UNIT; j0 += 16) {
                    if ((j0 & ~31) >= all_lo && (j0 | 31) < all_hi)
                        continue;
                    const Page p = page_of(str, j0, page_at(str, j0));
                    for (int j = j0; j < min(j0 + 16, str.L); ++j) {
                        const u32x2 y = load8(p.v + (unsigned)((j - j0) * p.v_row + 2 * col));
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sum[e] += odd_part<H>(y[e >> 1] >> 16 * (e & 1), (unsigned)(j - row.lo) < span);
                    }
                }
                if (!row.real)
                    continue;
                if (to.sums) {
                    *(f32x4_t*)(to.sums + at * DP + col) += sum;
                } else {
                    uint32_t* const out = (uint32_t*)(z.out + row.t * z.out_row + row.h * z.out_head + 2 * col);
#pragma unroll
                    for (int e = 0; e < 4; e += 2)
                        out[e >> 1] = pack2<H>(from16<H>(out[e >> 1] & 0xffffu) + sum[e], from16<H>(out[e >> 1] >> 16) + sum[e + 1]);
                }
            }
        }
        if (done.begins && !done.ends && threadIdx.x == 0)
            leave_record(z, w, done);
        if (now == last)
            return;
        now = behind(now);
    }
}

template <int DP, int WAVES, bool H, bool EXTRA>
void run(const AttendArgs& a, hipStream_t s)
{
    if (a.cache.dim == DP)
        many_rows<DP, WAVES, H, true, EXTRA><<<a.workers, 64 * WAVES, 0, s>>>(a);
    else
        many_rows<DP, WAVES, H, false, EXTRA><<<a.workers, 64 * WAVES, 0, s>>>(a);
}

template <int DP, int WAVES, bool H>
void run(const AttendArgs& a, hipStream_t s)
{
    // (a scale of zero: the other way multiplies hidden scores, which are infinite, by it)
    a.cap_out != 0.0f || a.slopes || a.scale == 0.0f ? run<DP, WAVES, H, true>(a, s) : run<DP, WAVES, H, false>(a, s);
}

template <bool H>
hipError_t run_many(const AttendArgs& a, hipStream_t s)
{
    switch (padded(a.cache.dim)) {
    case 64: run<64, 4, H>(a, s); break;
    case 128: a.rows == 256 ? run<128, 8, H>(a, s) : run<128, 4, H>(a, s); break;
    default: run<256, 4, H>(a, s);
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace hca
