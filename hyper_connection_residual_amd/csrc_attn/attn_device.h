// attn_device.h -- what the attention's kernels share: which rows and positions
// a workgroup takes, what a row sees, scores, and where results go.
//
// A segment is one stretch of positions with the tokens that attend to it: a
// request's own positions with its new tokens, or a prefix with those of all of
// its group's requests.  A segment's rows, for one head of the cache, are its
// tokens times the `group` query heads that share that head: row i is token i /
// group, head i % group of them.  Rows are cut into tiles, and a tile's visible
// positions into units.  All units of all tiles and heads, one behind the
// other, are dealt to the workers (workgroups) in equal runs: so long and short
// requests cost each what they hold, and a tile that is cut between workers is
// joined by a second kernel.
#pragma once

#include "attn_internal.h"
#include "proj_device.h"

namespace hca {

using hcp::bits16;
using hcp::f32x4_t;
using hcp::from16;
using hcp::gbytes;
using hcp::load16;
using hcp::u32x2;
using hcp::u32x4;

typedef float f32x16_t __attribute__((ext_vector_type(16)));
// A kernel's one argument where it lies.  (Taken by value, the struct's hundred words are
// loaded at the kernel's start and kept: two hundred spilled scalar registers.)
typedef const __attribute__((address_space(4))) AttendArgs Args;
__device__ __forceinline__ Args& args()
{
    auto p = (Args*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));  // (what is loaded before this is not kept for after it)
    return *p;
}

// Lists of a batch, which no kernel writes: read by the scalar unit.
typedef const __attribute__((address_space(4))) int32_t* ints;
__device__ __forceinline__ ints scalars(const int32_t* p) { return (ints)p; }

__device__ __forceinline__ u32x2 load8(gbytes p)
{
    return *(const __attribute__((address_space(1))) u32x2*)p;
}

// A row that the cache does not have.
__device__ static const uint4 kNoRow[32] = {};
static_assert(sizeof(kNoRow) == 512, "HC_MAX_HEAD 16-bit numbers");

template <bool H>
__device__ __forceinline__ uint32_t pack2(float x, float y)
{
    if constexpr (H) {
        typedef _Float16 v2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, v2{(_Float16)x, (_Float16)y});
    } else {
        typedef __bf16 v2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, v2{(__bf16)x, (__bf16)y});
    }
}

// The other of the pairs of lanes l and l ^ 32 (l ^ 16): max and sum of the two.
__device__ __forceinline__ float max32(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max16(float x)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum32(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum16(float x)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The value of lane ^ D (D below 32).
template <int D>
__device__ __forceinline__ int other(int x) { return __builtin_amdgcn_ds_swizzle(x, D << 10 | 0x1f); }
// The same in lanes that agree but for their lowest bits: largest and smallest of LANES (up to 32).
template <int LANES>
__device__ __forceinline__ int most_of(int x)
{
    x = max(x, other<1>(x));
    x = max(x, other<2>(x));
    x = max(x, other<4>(x));
    x = max(x, other<8>(x));
    return LANES > 16 ? max(x, other<16>(x)) : x;
}
template <int LANES>
__device__ __forceinline__ int least_of(int x) { return ~most_of<LANES>(~x); }

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
// What sums under one maximum count for under a larger one.  Never zero: an infinity among
// them stays one (and a NaN, for which there is no maximum, stays NaN).  The smallest number there is: of
// sums that are numbers, no more than 2^-21 is left.
__device__ __forceinline__ float weight_of(float x) { return fmaxf(exp2_of(x), 0x1p-149f); }

// cap tanh(score / cap) over ln 2, from the product q k: tanh(y) = 1 - 2 / (1 + exp(2 y)), of
// which an infinite exponential makes 1 and a zero one -1.  Of scores far below the cap that difference
// leaves few digits, which tells under a large cap (an error of up to 2^-21 cap): there they take tanh(y) = y - y^3 / 3 +
// 2 y^5 / 15 (the next term: 2^-24 of y at 0.1).  Under a smaller one that is time for nothing: a shared
// prefix's windows 35 us, without it 30.
constexpr float kLargeCap = 64.0f * 1.44269504f;
template <bool LARGE>
__device__ __forceinline__ float capped(float product, float cap_in, float cap_out)
{
    const float z = product * cap_in;  // 2 y / ln 2
    const float far = fmaf(-2.0f * cap_out, __builtin_amdgcn_rcpf(1.0f + exp2_of(z)), cap_out);
    if constexpr (!LARGE)
        return far;
    const float y = 0.34657359f * z, yy = y * y;
    const float near = cap_out * (y * fmaf(yy, fmaf(yy, 0.13333333f, -0.33333333f), 1.0f));
    return fabsf(y) < 0.1f ? near : far;
}

// What rounding x and y to a pair of 16-bit numbers leaves of them, as another pair.
template <bool H>
__device__ __forceinline__ uint32_t rest2(float x, float y, uint32_t pair)
{
    return pack2<H>(x - from16<H>(pair & 0xffffu), y - from16<H>(pair >> 16));
}

// Whether infinities or NaN are among 16-bit numbers: by the largest of their magnitudes, two operations for
// two numbers (hcp::finite_of takes eight).
template <bool H, int N, class Words>
__device__ __forceinline__ bool some_odd(const Words (&y)[N])
{
    typedef uint16_t v2 __attribute__((ext_vector_type(2)));
    v2 top{};
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (unsigned i = 0; i < sizeof(Words) / 4; ++i)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(v2, (uint32_t)(y[n][i] & 0x7fff7fffu)));
    return max((int)top[0], (int)top[1]) >= (int)(hcp::exponents(H) & 0xffffu);
}

// A score, or -infinity where bit i of `seen` is clear.
__device__ __forceinline__ float score_if(uint32_t seen, int i, float s)
{
    const uint32_t all = (uint32_t)((int32_t)(seen << (31 - i)) >> 31);
    return __uint_as_float((all & __float_as_uint(s)) | (~all & 0xff800000u));
}

// The running maximum of a row that has seen nothing yet.  A finite number: its
// difference to a score is never NaN.  (Scores, over ln 2, are above it.)
constexpr float kLowest = -3.0e38f;
// Numerators are 2^(score - m), m the row's reference.  It is set so that the maximum's is 2^kAbove, and stays until a
// score's passes 2^kMost: rarely are sums scaled anew.  fp16 ends at 2^16 and counts in steps of 2^-24: with
// the largest numerator at 2^11 to 2^15, one of 2^-25 of it has its digits, and one that is lost is below 2^-35 of it (with the
// largest at 1 to 2^8, a long context's many small ones came out as nothing, next to sums that held them).  bf16 has
// fp32's range: with none above 1, weighted values' sums stay numbers wherever the values' own do.
template <bool H> constexpr float kAbove = H ? 11.0f : -8.0f;
template <bool H> constexpr float kMost = H ? 15.0f : 0.0f;
// (fp16, whose range ends there: not further than that, but for a rounding, where a reference has no digits for it.)
template <bool H>
__device__ __forceinline__ float reference_of(float top)
{
    const float m = top - kAbove<H>;
    return H && top - m > kAbove<H> + 0.5f ? top : m;
}
template <bool H>
__device__ __forceinline__ float bar_of(float m)
{
    const float bar = m + kMost<H>;
    return H && bar - m > kMost<H> + 0.5f ? m : bar;
}

// ---------------------------------------------------------------------------
// Segments

struct Segment {
    int t0, n;       // its tokens
    int L;           // its positions
    int at0;         // its token i's own position is at0 + i (own segments)
    int base;        // the sequence's position of its position 0
    int pre;         // whether it is a prefix
    const int32_t* row;  // of the table
};

// The group of request b: the last that starts at or before it, or -1.
template <class P>
__device__ __forceinline__ int group_of(Args& a, P starts, int b)
{
    int lo = 0, hi = a.prefix.groups;  // starts[lo - 1] <= b < starts[hi]
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (starts[mid] <= b)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo > 0 && b < starts[lo] ? lo - 1 : -1;
}

__device__ __forceinline__ int prefix_length(Args& a, int length)
{
    return (int)min((int64_t)max(length, 0), (int64_t)a.prefix.width << a.cache.shift);
}

__device__ __forceinline__ const int32_t* row_of_table(Args& a, int s)
{
    return s < a.batch.requests ? a.batch.table + s * a.batch.table_row : a.prefix.table + (s - a.batch.requests) * a.prefix.table_row;
}

// P: ints where s is the same in all lanes.
template <class P>
__device__ __forceinline__ Segment segment_of(Args& a, int s)
{
    const P off = (P)a.batch.offsets;
    Segment g;
    g.row = row_of_table(a, s);
    g.pre = s >= a.batch.requests;
    if (!g.pre) {
        clamped_range(a.T, off, s, s + 1, g.t0, g.n);
        g.n -= g.t0;
        const int length = max(((P)a.batch.lengths)[s], 0);
        g.L = (int)min((int64_t)length, (int64_t)a.batch.width << a.cache.shift);
        g.at0 = length - g.n;
        g.base = 0;
        if (a.prefix.groups) {
            const int p = group_of(a, (P)a.prefix.starts, s);
            g.base = p < 0 ? 0 : prefix_length(a, ((P)a.prefix.lengths)[p]);
        }
    } else {
        const int p = s - a.batch.requests;
        const int r0 = min(max(((P)a.prefix.starts)[p], 0), a.batch.requests);
        const int r1 = min(max(((P)a.prefix.starts)[p + 1], r0), a.batch.requests);
        clamped_range(a.T, off, r0, r1, g.t0, g.n);
        g.n -= g.t0;
        g.L = prefix_length(a, ((P)a.prefix.lengths)[p]);
        g.at0 = g.base = 0;
    }
    return g;
}

// The positions lo <= j < hi of segment g that its token i sees (lo == hi: none).
__device__ __forceinline__ void seen(Args& a, const Segment& g, int i, int& lo, int& hi)
{
    lo = 0;
    hi = g.pre ? g.L : g.at0 + i + 1;
    if (a.first)
        lo = max(a.first[g.t0 + i], 0) - g.base;
    if (a.last)
        hi = max(a.last[g.t0 + i], 0) - g.base;
    lo = max(lo, 0);
    hi = min(hi, g.L);
    if (lo >= hi)
        lo = hi = 0;
}

__device__ __forceinline__ int tiles_of(Args& a, const Segment& g)
{
    return tiles_of(g.n, a.group, a.rows);
}

// Tile rt of segment s: the place of its units in a.ranges.
__device__ __forceinline__ int range_at(Args& a, const Segment& g, int s, int rt)
{
    const int from = (int)((unsigned)(g.t0 * a.group) / (unsigned)a.rows) + s + rt;
    return g.pre ? from + (int)((unsigned)(a.T * a.group) / (unsigned)a.rows) + 1 : from;
}

// The units of UNIT positions that tile rt of segment g (the s-th) reads: at least one.
template <int UNIT>
__device__ __forceinline__ void units_of(Args& a, const Segment& g, int s, int rt, int& lo, int& hi)
{
    const int most = (g.L + UNIT - 1) / UNIT;
    if (a.ranges) {
        const int2 r = a.ranges[range_at(a, g, s, rt)];
        lo = min(max(r.x, 0), most);
        hi = min(r.y, most);
    } else {
        const int i = (int)((unsigned)(min(rt * a.rows + a.rows, g.n * a.group) - 1) / (unsigned)a.group);
        seen(a, g, i, lo, hi);
        lo /= UNIT;
        hi = (hi + UNIT - 1) / UNIT;
    }
    hi = max(hi, lo + 1);
}

// ---------------------------------------------------------------------------
// The plan: which units a worker takes

// Sum of x over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int x)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(x, d);
        x += lane >= d ? o : 0;
    }
    return x;
}

// The same over a workgroup of THREADS, and the sum of all; `sums`: LDS of one int a wave.
template <int THREADS>
__device__ __forceinline__ int block_scan(int x, int* sums, int& all)
{
    const int wave = threadIdx.x >> 6, up = wave_scan(x);
    if ((threadIdx.x & 63) == 63)
        sums[wave] = up;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        const int s = sums[w];
        before += w < wave ? s : 0;
        all += s;
    }
    __syncthreads();
    return up + before;
}

// An item, a tile for one head, counts as its units and `a.item_cost` more before its first, for its
// start and end.  Items lie segment by segment, in each head by head, in each tile by tile: workers of one
// XCD, which take neighbouring runs at the same time, then read all heads of the same
// positions (of 64 requests' single tokens head by head, the XCDs of one head took
// 20 % longer than the others), and many tiles of one head.
struct Start {
    int64_t all, from, to;  // all items' counts; this worker's
    int workers;
    int s, head, rt;        // the item (segment, head and tile) that `from` lies in ...
    int64_t at;             // ... and where that begins
    Segment g;
};

// Workers that get units: each `least` of them or more.
__device__ __forceinline__ int workers_of(Args& a, int64_t all)
{
    return (int)min((int64_t)a.workers, (int64_t)((uint64_t)(all + a.least - 1) / (uint32_t)a.least));
}
__device__ __forceinline__ int64_t first_unit(int64_t all, int workers, int w) { return all * w / workers; }
// The worker of unit u: the last whose first unit is at or before it.
__device__ __forceinline__ int worker_of(int64_t all, int workers, int64_t u)
{
    return (int)(((u + 1) * workers - 1) / all);
}

__device__ __forceinline__ bool deal(Args& a, int w, int units, Start& p)
{
    p.all = (int64_t)units * a.cache.heads;
    p.workers = workers_of(a, p.all);
    if (w >= p.workers)
        return false;
    p.from = first_unit(p.all, p.workers, w);
    p.to = first_unit(p.all, p.workers, w + 1);
    return true;
}

// Worker w's units; false: it has none.  All threads of the workgroup call it.  first:
// LDS, uint16 [kMaxSegments + 1]; at: accessor of an LDS list of kMaxTiles + 1 ints; sums:
// LDS ints, 16 of them.  Under prefixes the first worker leaves the lists for the join, which
// reads them as indexes: they are whole, or say that there are no units.
template <int UNIT, int THREADS, class At>
__device__ __forceinline__ bool make_plan(Args& a, int w, uint16_t* first, At at, int* sums, Start& p)
{
    const int S = a.batch.requests + a.prefix.groups, heads = a.cache.heads;
    const bool save = a.prefix.groups && w == 0;
    if (S <= 64) {  // a segment a lane, if each has one tile: no waiting for other waves (3.5 us to 1.9 for one token)
        const int lane = threadIdx.x & 63, s = min(lane, S - 1);
        const Segment g = segment_of<const int32_t*>(a, s);
        const int tiles = lane < S ? tiles_of(a, g) : 0;
        if (!__any(tiles > 1)) {
            int lo = 0, hi = 0;
            if (tiles)
                units_of<UNIT>(a, g, s, 0, lo, hi);
            const int n = tiles ? hi - lo + a.item_cost : 0, upto = wave_scan(n), units = __builtin_amdgcn_readlane(upto, 63);
            if (save && threadIdx.x < 64) {
                const int i = wave_scan(tiles);
                const int all_tiles = __builtin_amdgcn_readlane(i, 63);
                if (lane < S)
                    a.plan[2 + lane] = i - tiles;
                if (tiles)
                    a.plan[3 + S + i - 1] = upto - n;
                if (lane == 0) {
                    a.plan[0] = units;
                    a.plan[1] = a.plan[2 + S] = all_tiles;
                    a.plan[3 + S + all_tiles] = units;
                }
            }
            if (!deal(a, w, units, p))
                return false;
            const bool mine = (int64_t)heads * (upto - n) <= p.from && p.from < (int64_t)heads * upto;
            p.s = __builtin_ctzll(__ballot(mine));
            const int each = __builtin_amdgcn_readlane(n, p.s);
            const int64_t within = p.from - (int64_t)heads * (__builtin_amdgcn_readlane(upto, p.s) - each);
            p.head = (int)((uint64_t)within / (unsigned)each);
            p.at = p.from - within + (int64_t)p.head * each;
            p.rt = 0;
            p.g.t0 = __builtin_amdgcn_readlane(g.t0, p.s);
            p.g.n = __builtin_amdgcn_readlane(g.n, p.s);
            p.g.L = __builtin_amdgcn_readlane(g.L, p.s);
            p.g.at0 = __builtin_amdgcn_readlane(g.at0, p.s);
            p.g.base = __builtin_amdgcn_readlane(g.base, p.s);
            p.g.pre = p.s >= a.batch.requests;
            p.g.row = row_of_table(a, p.s);
            return true;
        }
    }
    int tiles = 0;
    for (int s0 = 0; s0 < S; s0 += THREADS) {
        const int s = s0 + threadIdx.x;
        const int n = s < S ? tiles_of(a, segment_of<const int32_t*>(a, s)) : 0;
        int all;
        const int upto = block_scan<THREADS>(n, sums, all);
        if (s < S)
            first[s] = (uint16_t)(tiles + upto - n);
        tiles += all;
    }
    if (!planned(tiles, a.tiles)) {
        if (save && threadIdx.x == 0)
            a.plan[0] = a.plan[1] = 0;
        return false;
    }
    if (threadIdx.x == 0)
        first[S] = (uint16_t)tiles;
    __syncthreads();
    int units = 0;
    for (int i0 = 0; i0 < tiles; i0 += THREADS) {
        const int i = i0 + threadIdx.x;
        int n = 0;
        if (i < tiles) {
            int lo = 0, hi = S;  // the last segment that begins at or before tile i: first[lo] <= i < first[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (first[mid] <= i)
                    lo = mid;
                else
                    hi = mid;
            }
            const int s = lo;
            units_of<UNIT>(a, segment_of<const int32_t*>(a, s), s, i - first[s], lo, hi);
            n = hi - lo + a.item_cost;
        }
        int all;
        const int upto = block_scan<THREADS>(n, sums, all);
        if (i < tiles)
            at(i) = units + upto - n;
        units += all;
    }
    if (threadIdx.x == 0)
        at(tiles) = units;
    __syncthreads();
    if (save) {
        for (int s = threadIdx.x; s <= S; s += THREADS)
            a.plan[2 + s] = first[s];
        for (int i = threadIdx.x; i <= tiles; i += THREADS)
            a.plan[3 + S + i] = at(i);
        if (threadIdx.x == 0) {
            a.plan[0] = units;
            a.plan[1] = tiles;
        }
    }
    if (!deal(a, w, units, p))
        return false;
    for (int s = threadIdx.x; s < S; s += THREADS)
        if ((int64_t)heads * at(first[s]) <= p.from && p.from < (int64_t)heads * at(first[s + 1]))
            sums[0] = s;
    __syncthreads();
    p.s = __builtin_amdgcn_readfirstlane(sums[0]);
    const int f0 = first[p.s], f1 = first[p.s + 1], from = at(f0), each = at(f1) - from;
    const int64_t within = p.from - (int64_t)heads * from;
    p.head = __builtin_amdgcn_readfirstlane((int)((uint64_t)within / (unsigned)each));
    const int rest = (int)(within - (int64_t)p.head * each) + from;
    for (int i = f0 + threadIdx.x; i < f1; i += THREADS)
        if (at(i) <= rest && rest < at(i + 1))
            sums[1] = i;
    __syncthreads();
    const int i = __builtin_amdgcn_readfirstlane(sums[1]);
    p.rt = i - __builtin_amdgcn_readfirstlane(f0);
    p.at = p.from - __builtin_amdgcn_readfirstlane(rest - at(i));
    p.g = segment_of<ints>(a, p.s);
    __syncthreads();
    return true;
}

// One worker's part of an item.
struct Item {
    Segment g;
    int s, head, rt;
    int u0, u1;        // its units
    int begins, ends;  // whether the item's first and last ones are among them
    int last;          // else: the worker that ends it
};

// A worker's way through its items.
struct Walk {
    int64_t at, u;  // where the next item begins, and from where on it is this worker's
    int s, head, rt;
    Segment g;
};
__device__ __forceinline__ Walk walk_from(const Start& p) { return Walk{p.at, p.from, p.s, p.head, p.rt, p.g}; }

template <int UNIT>
__device__ __forceinline__ bool next_item(Args& a, const Start& p, Walk& x, Item& y)
{
    for (;;) {
        if (x.u >= p.to)
            return false;
        if (x.rt == tiles_of(a, x.g)) {
            x.rt = 0;
            if (++x.head == a.cache.heads) {
                x.head = 0;
                do {
                    if (++x.s == a.batch.requests + a.prefix.groups)
                        return false;  // (never: the counts end before)
                    x.g = segment_of<ints>(a, x.s);
                } while (x.g.n == 0);
            }
        }
        int lo, hi;
        units_of<UNIT>(a, x.g, x.s, x.rt, lo, hi);
        lo = __builtin_amdgcn_readfirstlane(lo);
        hi = __builtin_amdgcn_readfirstlane(hi);
        const int64_t first = x.at + a.item_cost, end = first + (hi - lo);
        y.g = x.g;
        y.s = x.s;
        y.head = x.head;
        y.rt = x.rt;
        y.u0 = lo + (int)max(x.u - first, (int64_t)0);
        y.u1 = lo + (int)max(min(end, p.to) - first, (int64_t)0);
        y.begins = x.u <= first;
        y.ends = end <= p.to;
        y.last = y.ends ? 0 : worker_of(p.all, p.workers, end - 1);
        x.u = x.at = end;
        ++x.rt;
        if (y.u0 < y.u1)
            return true;
    }
}

// What a wave keeps in LDS from item to item, and the same in scalar registers.  (Kept in registers
// throughout, such states are spilled in the main loop.)
template <class T>
__device__ __forceinline__ T taken(const T* from)
{
    struct Words {
        uint32_t w[sizeof(T) / 4];
    } x;
    static_assert(sizeof(T) % 4 == 0, "whole words");
    __builtin_memcpy(&x, from, sizeof(T));
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 4; ++i)
        x.w[i] = __builtin_amdgcn_readfirstlane(x.w[i]);
    return __builtin_bit_cast(T, x);
}

// ---------------------------------------------------------------------------
// Rows

// A row of a tile, as one lane has it.
struct Row {
    bool real;       // it has a token
    int t, h;        // token, query head
    int lo, hi;      // the segment's positions that it sees
    float slope;     // with slopes: over ln 2 ...
    int p;           // ... and its position, from the segment's 0 (past 2^24 no number of fp32: distances are taken before)
};

__device__ __forceinline__ Row row_of(Args& a, const Segment& g, int head, int row)
{
    Row r;
    r.real = row < g.n * a.group;
    const int i = r.real ? (int)((unsigned)row / (unsigned)a.group) : 0;
    r.t = g.t0 + i;
    r.h = head * a.group + (r.real ? row - i * a.group : 0);
    r.lo = r.hi = 0;
    r.slope = 0.0f;
    r.p = 0;
    if (!r.real)
        return r;
    seen(a, g, i, r.lo, r.hi);
    if (a.slopes) {
        r.slope = a.slopes[r.h] * 1.44269504f;
        int64_t p = g.at0 + i;
        if (g.pre) {  // the token's request: the last that begins at or before it and is not empty
            int lo = 0, hi = a.batch.requests;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (a.batch.offsets[mid] <= r.t)
                    lo = mid;
                else
                    hi = mid;
            }
            int t0, t1;
            clamped_range(a.T, a.batch.offsets, lo, lo + 1, t0, t1);
            p = (int64_t)g.L + max(a.batch.lengths[lo], 0) - (t1 - r.t);
        }
        r.p = (int)min(p, (int64_t)0x7fffffff);  // (more only by lengths past the table; less than -2^18 never)
    }
    return r;
}

// Where the results of an item go.
struct Target {
    float* sums;   // NULL: the outputs themselves; else [rows][width] ...
    float2* ml;    // ... and [rows] (maximum over ln 2, sum)
    bool dense;    // rows by (token, head)
};

__device__ __forceinline__ Target target_of(Args& a, int w, const Item& y, int width)
{
    Target to{nullptr, nullptr, false};
    if (!(y.begins && y.ends)) {
        const int slot = 2 * w + y.begins;
        to.sums = a.part + (int64_t)slot * a.rows * width;
        to.ml = a.ml + slot * a.rows;
    } else if (a.prefix.groups) {
        const int64_t from = slot_rows(a.rows) + (y.g.pre ? (int64_t)a.T * a.q_heads : 0);
        to.sums = a.part + from * width;
        to.ml = a.ml + from;
        to.dense = true;
    }
    return to;
}

// The item that worker w begins and others end.
__device__ __forceinline__ void leave_record(Args& a, int w, const Item& y)
{
    Record r{};
    r.t0 = y.g.t0;
    r.row0 = y.rt * a.rows;
    r.rows = min(a.rows, y.g.n * a.group - r.row0);
    r.head = y.head;
    r.last = y.last;
    ((Record*)a.records)[w] = r;
}

// A segment's positions for one head, as the main loops go through them.
struct Stream {
    ints row;  // of the table
    gbytes k, v;
    int64_t k_page, v_page, pages;
    int k_row, v_row, shift, L;
};
__device__ __forceinline__ Stream stream_of(Args& a, const Segment& g, int head)
{
    Stream s;
    s.row = scalars(g.L > 0 ? g.row : (const int32_t*)kNoRow);
    s.k = (gbytes)a.cache.k + (int64_t)head * a.cache.k_head;
    s.v = (gbytes)a.cache.v + (int64_t)head * a.cache.v_head;
    s.k_page = a.cache.k_page;
    s.v_page = a.cache.v_page;
    s.pages = a.cache.pages;
    s.k_row = a.cache.k_row;
    s.v_row = a.cache.v_row;
    s.shift = a.cache.shift;
    s.L = g.L;
    return s;
}

// The table's entry for position j (which the segment may not have); j is the same in all lanes.
__device__ __forceinline__ int32_t page_at(const Stream& s, int j) { return j < s.L ? s.row[j >> s.shift] : -1; }
// The same in a vector register, where it can wait for its use (a scalar one that is spilled waits at
// once), and without a branch (whose two sides' registers would meet in a copy, which
// waits, too); of positions that the segment does not have, anything.
__device__ __forceinline__ int32_t page_in_lanes(const Stream& s, int j)
{
    uint32_t at = (max(min(j, s.L - 1), 0) >> s.shift) * 4;
    asm volatile("" : "+v"(at));
    return *(const __attribute__((address_space(1))) int32_t*)((gbytes)s.row + at);
}

// The rows from position j on, up to its page's end.
struct Page {
    gbytes k, v;
    int k_row, v_row;  // bytes from row to row (a page that is not there: 0, of zeros)
    int last;          // the last row, from this position on, that is there
};
__device__ __forceinline__ Page page_of(const Stream& s, int j, int32_t page)
{
    Page p;
    const bool there = j < s.L && (int64_t)(uint32_t)page < s.pages;
    const int64_t row = j & ((1 << s.shift) - 1);
    p.k = there ? s.k + page * s.k_page + row * s.k_row : (gbytes)(const char*)kNoRow;
    p.v = there ? s.v + page * s.v_page + row * s.v_row : (gbytes)(const char*)kNoRow;
    p.k_row = there ? s.k_row : 0;
    p.v_row = there ? s.v_row : 0;
    p.last = max(s.L - 1 - j, 0);
    return p;
}

// What a 16-bit number adds to a row's sum by being an infinity or NaN, where the row sees it.
template <bool H>
__device__ __forceinline__ float odd_part(uint32_t bits, bool sees)
{
    const float x = from16<H>(bits & 0xffffu);
    return sees && !(fabsf(x) < INFINITY) ? x : 0.0f;
}

}  // namespace hca
