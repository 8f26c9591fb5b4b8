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
typedef uint32_t u32x16 __attribute__((ext_vector_type(16)));
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

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
// What sums under one maximum count for under a larger one.  Never zero: an infinity among
// them stays one (and a NaN, for which there is no maximum, stays NaN).
__device__ __forceinline__ float weight_of(float x) { return fmaxf(exp2_of(x), 1.17549435e-38f); }

// cap tanh(score / cap) over ln 2, from the product q k: tanh(y) = 1 - 2 / (1 + exp(2 y)), of
// which an infinite exponential makes 1 and a zero one -1.
__device__ __forceinline__ float capped(float product, float cap_in, float cap_out)
{
    return fmaf(-2.0f * cap_out, __builtin_amdgcn_rcpf(1.0f + exp2_of(product * cap_in)), cap_out);
}

// The running maximum of a row that has seen nothing yet.  A finite number: its
// difference to a score is never NaN.  (Scores, over ln 2, are above it.)
constexpr float kLowest = -3.0e38f;
// A maximum stays the reference of its row until a score passes it by this much (over ln 2):
// numerators then stay under 2^8 and rarely are sums scaled anew.
constexpr float kSlack = 8.0f;

// ---------------------------------------------------------------------------
// Segments

struct Segment {
    int t0, n;       // its tokens
    int L;           // its positions
    int at0;         // its token i's own position is at0 + i (own segments)
    int base;        // the sequence's position of its position 0
    bool pre;        // a prefix
    const int32_t* row;  // of the table
};

template <class P>
__device__ __forceinline__ void clamped_range(Args& a, P off, int b0, int b1, int& lo, int& hi)
{
    lo = min(max(off[b0], 0), a.T);
    hi = min(max(off[b1], lo), a.T);
}

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

// P: ints where s is the same in all lanes.
template <class P>
__device__ __forceinline__ Segment segment_of(Args& a, int s)
{
    const P off = (P)a.batch.offsets;
    Segment g;
    g.pre = s >= a.batch.requests;
    if (!g.pre) {
        clamped_range(a, off, s, s + 1, g.t0, g.n);
        g.n -= g.t0;
        const int length = max(((P)a.batch.lengths)[s], 0);
        g.L = (int)min((int64_t)length, (int64_t)a.batch.width << a.cache.shift);
        g.at0 = length - g.n;
        g.row = a.batch.table + s * a.batch.table_row;
        g.base = 0;
        if (a.prefix.groups) {
            const int p = group_of(a, (P)a.prefix.starts, s);
            g.base = p < 0 ? 0 : prefix_length(a, ((P)a.prefix.lengths)[p]);
        }
    } else {
        const int p = s - a.batch.requests;
        const int r0 = min(max(((P)a.prefix.starts)[p], 0), a.batch.requests);
        const int r1 = min(max(((P)a.prefix.starts)[p + 1], r0), a.batch.requests);
        clamped_range(a, off, r0, r1, g.t0, g.n);
        g.n -= g.t0;
        g.L = prefix_length(a, ((P)a.prefix.lengths)[p]);
        g.at0 = g.base = 0;
        g.row = a.prefix.table + p * a.prefix.table_row;
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

// The units of UNIT positions that tile `rt` of segment g reads: at
// least one.  With first or last, LANES neighbouring lanes (of one tile) share its tokens.
template <int UNIT, int LANES>
__device__ __forceinline__ void units_of(Args& a, const Segment& g, int rt, int& lo_unit, int& hi_unit)
{
    const int i0 = (int)((unsigned)(rt * a.rows) / (unsigned)a.group);
    const int i1 = (int)((unsigned)(min(rt * a.rows + a.rows, g.n * a.group) - 1) / (unsigned)a.group);
    int lo = 0x7fffffff, hi = 0;
    if (a.first || a.last) {
        for (int i = i0 + (threadIdx.x & (LANES - 1)); i <= i1; i += LANES) {
            int l, h;
            seen(a, g, i, l, h);
            if (l < h) {
                lo = min(lo, l);
                hi = max(hi, h);
            }
        }
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) {
            lo = min(lo, __shfl_xor(lo, d));
            hi = max(hi, __shfl_xor(hi, d));
        }
    } else {
        seen(a, g, i1, lo, hi);
    }
    if (lo >= hi)
        lo = hi = 0;
    lo_unit = lo / UNIT;
    hi_unit = max((hi + UNIT - 1) / UNIT, lo_unit + 1);
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

// First: uint16 list in LDS of the segments' first tiles; Unit: int list of the
// tiles' first units (both with a last entry, the count of all).
struct Start {
    int64_t from, to;  // this worker's units, of `units` for each head
    int units, workers;
    int head, s, rt;   // the item (tile and head) of its first unit ...
    int64_t at;        // ... and that item's first unit
    int lo, hi;        // ... its units of positions
};

__device__ __forceinline__ int tiles_of(Args& a, int s)
{
    const Segment g = segment_of<const int32_t*>(a, s);
    return (int)((unsigned)(g.n * a.group + a.rows - 1) / (unsigned)a.rows);
}

// Workers that get units: each `least` of them or more.
__device__ __forceinline__ int workers_of(Args& a, int64_t all)
{
    return (int)min((int64_t)kWorkers, (int64_t)((uint64_t)(all + a.least - 1) / (uint32_t)a.least));
}
__device__ __forceinline__ int64_t first_unit(int64_t all, int workers, int w) { return all * w / workers; }
// The worker of unit u: the last whose first unit is at or before it.
__device__ __forceinline__ int worker_of(int64_t all, int workers, int64_t u)
{
    return (int)(((u + 1) * workers - 1) / all);
}

// Finds worker w's units; false: it has none.  All threads of the workgroup call
// it.  first: LDS, uint16 [kMaxSegments + 1]; at: accessor of an LDS list of kMaxTiles + 1
// ints; sums: LDS ints, 16 of them.  With `save`, the lists go to the scratch.
template <int UNIT, int THREADS, class At>
__device__ __forceinline__ bool make_plan(Args& a, int w, uint16_t* first, At at, int* sums, Start& p)
{
    const int S = a.batch.requests + a.prefix.groups;
    int tiles = 0;
    for (int s0 = 0; s0 < S; s0 += THREADS) {
        const int s = s0 + threadIdx.x;
        const int n = s < S ? tiles_of(a, s) : 0;
        int all;
        const int upto = block_scan<THREADS>(n, sums, all);
        if (s < S)
            first[s] = (uint16_t)min(tiles + upto - n, kMaxTiles);
        tiles = min(tiles + all, kMaxTiles);  // (more only where offsets are not in order)
    }
    if (threadIdx.x == 0)
        first[S] = (uint16_t)tiles;
    __syncthreads();
    const auto segment_at = [&](int i) {  // the last segment that begins at or before tile i
        int lo = 0, hi = S;               // first[lo] <= i < first[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (first[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    };
    int units = 0;
    // (masks of one's own: 16 lanes for a tile)
    const auto count = [&](auto lanes) {
        constexpr int LANES = decltype(lanes)::value;
        for (int i0 = 0; i0 < tiles; i0 += THREADS / LANES) {
            const int i = i0 + threadIdx.x / LANES;
            const bool mine = i < tiles && (threadIdx.x & (LANES - 1)) == 0;
            int n = 0;
            if (i < tiles) {
                const int s = segment_at(i);
                int lo, hi;
                units_of<UNIT, LANES>(a, segment_of<const int32_t*>(a, s), i - first[s], lo, hi);
                n = mine ? hi - lo : 0;
            }
            int all;
            const int upto = block_scan<THREADS>(n, sums, all);
            if (mine)
                at(i) = units + upto - n;
            units += all;
        }
    };
    if (a.first || a.last)
        count(std::integral_constant<int, 16>{});
    else
        count(std::integral_constant<int, 1>{});
    if (threadIdx.x == 0)
        at(tiles) = units;
    __syncthreads();
    if (a.prefix.groups && w == 0) {  // for the join
        for (int s = threadIdx.x; s <= S; s += THREADS)
            a.plan[2 + s] = first[s];
        for (int i = threadIdx.x; i <= tiles; i += THREADS)
            a.plan[3 + S + i] = at(i);
        if (threadIdx.x == 0) {
            a.plan[0] = units;
            a.plan[1] = tiles;
        }
    }
    const int64_t all = (int64_t)units * a.cache.heads;
    p.units = units;
    p.workers = workers_of(a, all);
    if (w >= p.workers)
        return false;
    p.from = first_unit(all, p.workers, w);
    p.to = first_unit(all, p.workers, w + 1);
    p.head = (int)(p.from / units);
    const int within = (int)(p.from - (int64_t)p.head * units);
    for (int i = threadIdx.x; i < tiles; i += THREADS)
        if (at(i) <= within && within < at(i + 1)) {
            sums[0] = i;
            sums[1] = segment_at(i);
        }
    __syncthreads();
    const int i = __builtin_amdgcn_readfirstlane(sums[0]);
    p.s = __builtin_amdgcn_readfirstlane(sums[1]);
    p.rt = i - __builtin_amdgcn_readfirstlane((int)first[p.s]);
    p.at = (int64_t)p.head * units + __builtin_amdgcn_readfirstlane(at(i));
    __syncthreads();
    return true;
}

// A worker's way through its items: f(segment, tile, head, first and last unit of
// positions, whether the item begins and ends here, the worker that ends it).
template <int UNIT, class F>
__device__ __forceinline__ void walk(Args& a, const Start& p, F f)
{
    int64_t at = p.at, u = p.from;
    int s = p.s, rt = p.rt, head = p.head;
    Segment g = segment_of<ints>(a, s);
    for (;;) {
        int lo, hi;
        units_of<UNIT, 64>(a, g, rt, lo, hi);
        lo = __builtin_amdgcn_readfirstlane(lo);
        hi = __builtin_amdgcn_readfirstlane(hi);
        const int64_t end = at + (hi - lo);
        const int k0 = lo + (int)(u - at), k1 = lo + (int)(min(end, p.to) - at);
        f(g, rt, head, k0, k1, u == at, end <= p.to,
          end <= p.to ? 0 : worker_of((int64_t)p.units * a.cache.heads, p.workers, end - 1));
        u = end;
        at = end;
        if (u >= p.to)
            return;
        if ((rt + 1) * a.rows < g.n * a.group) {
            ++rt;
            continue;
        }
        rt = 0;
        do {
            if (++s == a.batch.requests + a.prefix.groups) {
                s = 0;
                ++head;
            }
            g = segment_of<ints>(a, s);
        } while (g.n == 0);
    }
}

// ---------------------------------------------------------------------------
// Rows

// A row of a tile, as one lane has it.
struct Row {
    bool real;       // it has a token
    int t, h;        // token, query head
    int lo, hi;      // the segment's positions that it sees
    float slope, p;  // with slopes: over ln 2; its position, from the segment's 0
};

__device__ __forceinline__ Row row_of(Args& a, const Segment& g, int head, int row)
{
    Row r;
    r.real = row < g.n * a.group;
    const int i = r.real ? (int)((unsigned)row / (unsigned)a.group) : 0;
    r.t = g.t0 + i;
    r.h = head * a.group + (r.real ? row - i * a.group : 0);
    r.lo = r.hi = 0;
    r.slope = r.p = 0.0f;
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
            clamped_range(a, a.batch.offsets, lo, lo + 1, t0, t1);
            p = (int64_t)g.L + max(a.batch.lengths[lo], 0) - (t1 - r.t);
        }
        r.p = (float)p;
    }
    return r;
}

// Where the results of an item go.
struct Target {
    float* sums;   // NULL: the outputs themselves; else [rows][width] ...
    float2* ml;    // ... and [rows] (maximum over ln 2, sum)
    bool dense;    // rows by (token, head)
};

__device__ __forceinline__ Target target_of(Args& a, int w, const Segment& g, int width, bool begins, bool ends)
{
    Target to{nullptr, nullptr, false};
    if (!(begins && ends)) {
        const int slot = 2 * w + begins;
        to.sums = a.part + (int64_t)slot * a.rows * width;
        to.ml = a.ml + slot * a.rows;
    } else if (a.prefix.groups) {
        const int64_t from = slot_rows(a.rows) + (g.pre ? (int64_t)a.T * a.q_heads : 0);
        to.sums = a.part + from * width;
        to.ml = a.ml + from;
        to.dense = true;
    }
    return to;
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
    s.row = scalars(g.row);
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
