// attn_join.hip -- the parts of rows that several workers hold, or under
// prefixes two segments, become outputs.
//
// Bound by the latency of the parts' loads where they are few, by memory where
// they are many.  dim / 8 lanes (the next power of two) join one row, 8 columns a
// lane, so a wave joins 2, 4 or 8 rows at a time; four parts of each are on their
// way at once, and rows of more than 4 parts (of large tiles, 8) are shared by a workgroup's four waves.
// A prompt of 8192 tokens: 14 us, 62 MB of parts; 64 tokens' rows: 5.
#include "attn_device.h"

#include <algorithm>

#pragma clang fp contract(off)

namespace hca {
namespace {

constexpr int kThreads = kJoinThreads, kWaves = kThreads / 64;

// A row's parts, as its lanes join them: maximum over ln 2, sum, unscaled sums.
struct Joined {
    float top, sum;
    float y[8];
};

// Parts `from`, from + step, ... of n; of(i): the row of part i in a.ml and a.part.
template <int DP, class Of>
__device__ __forceinline__ Joined join_parts(Args& a, int from, int step, int n, Of of, int c)
{
    Joined r;
    r.top = kLowest;
    r.sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        r.y[e] = 0.0f;
    const float* const part = a.part;
    const float2* const ml = a.ml;
    for (int i0 = from; i0 < n; i0 += 4 * step) {
        float2 x[4];
        f32x4_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = of(min(i0 + i * step, n - 1));
            x[i] = ml[at];
            lo[i] = *(const f32x4_t*)(part + at * DP + 8 * c);
            hi[i] = *(const f32x4_t*)(part + at * DP + 8 * c + 4);
        }
        float top = r.top;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top = fmaxf(top, x[i].x);
        const float was = weight_of(r.top - top);
        r.top = top;
        r.sum *= was;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r.y[e] *= was;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float by = i0 + i * step < n ? weight_of(x[i].x - top) : 0.0f;
            if (by != 0.0f) {
                r.sum = fmaf(by, x[i].y, r.sum);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    r.y[e] = fmaf(by, lo[i][e], r.y[e]);
                    r.y[4 + e] = fmaf(by, hi[i][e], r.y[4 + e]);
                }
            }
        }
    }
    return r;
}

template <bool H>
__device__ __forceinline__ void store_row(Args& a, const Joined& r, int t, int head, int c)
{
    const float by = r.sum == 0.0f ? 0.0f : 1.0f / r.sum;
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w[e] = pack2<H>(r.y[2 * e] * by, r.y[2 * e + 1] * by);
    *(u32x4*)(a.out + t * a.out_row + head * a.out_head + 16 * c) = w;
}

// The four waves' shares of the same rows meet in LDS; wave 0 has them all.
template <int DP>
__device__ __forceinline__ void meet(Joined& r, float (&lds)[kWaves - 1][64][11])
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    __syncthreads();
    if (wave) {
        lds[wave - 1][lane][0] = r.top;
        lds[wave - 1][lane][1] = r.sum;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            lds[wave - 1][lane][2 + e] = r.y[e];
    }
    __syncthreads();
    if (wave)
        return;
    float top = r.top;
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w)
        top = fmaxf(top, lds[w][lane][0]);
    const float was = weight_of(r.top - top);
    r.top = top;
    r.sum *= was;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        r.y[e] *= was;
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w) {
        const float by = weight_of(lds[w][lane][0] - top);
        r.sum = fmaf(by, lds[w][lane][1], r.sum);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r.y[e] = fmaf(by, lds[w][lane][2 + e], r.y[e]);
    }
}

// The first and last unit of every tile, where tokens have ranges of their own: a wave
// for a tile's tokens.
__global__ __launch_bounds__(kThreads) void tile_ranges(AttendArgs, int unit)
{
    Args& a = args();
    const int s = blockIdx.x, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Segment g = segment_of<ints>(a, s);
    const int tiles = tiles_of(a, g);
    for (int rt = blockIdx.y * kWaves + wave; rt < tiles; rt += gridDim.y * kWaves) {
        const int i0 = (int)((unsigned)(rt * a.rows) / (unsigned)a.group);
        const int i1 = (int)((unsigned)(min(rt * a.rows + a.rows, g.n * a.group) - 1) / (unsigned)a.group);
        int lo = 0x7fffffff, hi = 0;
        for (int i = i0 + lane; i <= i1; i += 64) {
            int l, h;
            seen(a, g, i, l, h);
            if (l < h) {
                lo = min(lo, l);
                hi = max(hi, h);
            }
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            lo = min(lo, __shfl_xor(lo, d));
            hi = max(hi, __shfl_xor(hi, d));
        }
        if (lane == 0)
            a.ranges[range_at(a, g, s, rt)] = lo < hi ? int2{lo / unit, (hi + unit - 1) / unit} : int2{0, 0};
    }
}

// Tiles that were cut between workers: blockIdx.x is the worker that begins one.
// alone: as many parts a wave joins by itself.
template <int DP, bool H>
__global__ __launch_bounds__(kThreads) void join_tiles(AttendArgs, int alone)
{
    Args& a = args();
    __shared__ float lds[kWaves - 1][64][11];
    const Record rec = ((const Record*)a.records)[blockIdx.x];
    constexpr int LANES = DP / 8, EACH = 64 / LANES;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane % LANES, w = blockIdx.x;
    const int n = rec.last - w + 1;
    const bool together = n > alone;
    const int step = (together ? 1 : kWaves) * EACH;
    for (int i0 = blockIdx.y * step; i0 < rec.rows; i0 += gridDim.y * step) {  // (the same turns in all waves)
        const int i = i0 + (together ? 0 : wave * EACH) + lane / LANES;
        const bool live = i < rec.rows;
        const int in = live ? i : 0;
        // the first part is the beginning worker's second slot, the others' are their first
        const auto of = [&](int p) { return (int64_t)(2 * (w + p) + (p == 0)) * a.rows + in; };
        Joined r = join_parts<DP>(a, together ? wave : 0, together ? kWaves : 1, n, of, c);
        if (together) {
            meet<DP>(r, lds);
            if (wave)
                continue;
        }
        if (live && 8 * c < a.cache.dim) {
            const int row = rec.row0 + i, t = (int)((unsigned)row / (unsigned)a.group);
            store_row<H>(a, r, rec.t0 + t, rec.head * a.group + row - t * a.group, c);
        }
    }
}

// Under prefixes: every row, of its own positions and its prefix's.  A workgroup
// takes neighbouring rows; together: its waves share them.
template <int DP, bool H>
__global__ __launch_bounds__(kThreads) void join_shared(AttendArgs, bool together)
{
    Args& a = args();
    __shared__ float lds[kWaves - 1][64][11];
    constexpr int LANES = DP / 8, EACH = 64 / LANES;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane % LANES;
    const int64_t id = ((int64_t)blockIdx.x * (together ? 1 : kWaves) + (together ? 0 : wave)) * EACH + lane / LANES;
    bool live = id < (int64_t)a.T * a.q_heads;
    const int t = live ? (int)((uint64_t)id / (unsigned)a.q_heads) : 0, head = live ? (int)(id - (int64_t)t * a.q_heads) : 0;
    // the token's request: as many end at or before it
    const int32_t* const off = a.batch.offsets;
    int lo = 0, hi = a.batch.requests;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (off[mid + 1] <= t)
            lo = mid + 1;
        else
            hi = mid;
    }
    const int b = lo, last = a.batch.requests - 1;
    live = live && b <= last && t >= off[min(b, last)];
    const int32_t* const plan = a.plan;
    const int S = a.batch.requests + a.prefix.groups, units = plan[0], tiles = plan[1];
    const int64_t all = (int64_t)units * a.cache.heads;
    const int workers = workers_of(a, all);
    if (all == 0)
        return;
    // the parts of the row in segment s: whole, by (token, head); or in the slots of workers from .. to
    struct Parts {
        int from, n;
        int64_t at;
    };
    const auto parts_of = [&](int s, int t0) {
        const int row = (t - t0) * a.group + head % a.group, i = min(plan[2 + s] + row / a.rows, tiles - 1);
        const int from = plan[3 + S + plan[2 + s]], each = plan[3 + S + plan[3 + s]] - from;  // the segment's units of a head
        const int64_t u = (int64_t)a.cache.heads * from + (int64_t)(head / a.group) * each + plan[3 + S + i] - from;
        const int64_t end = u + plan[4 + S + i] - plan[3 + S + i];
        const int w0 = worker_of(all, workers, u + a.item_cost), w1 = worker_of(all, workers, end - 1);
        Parts p;
        p.from = w0;
        p.n = w1 - w0 + 1;
        p.at = w0 == w1 ? slot_rows(a.rows) + (s >= a.batch.requests ? (int64_t)a.T * a.q_heads : 0) + (int64_t)t * a.q_heads + head : row % a.rows;
        return p;
    };
    const auto place = [&](const Parts& p, int i) {
        return p.n == 1 ? p.at : (int64_t)(2 * (p.from + i) + (i == 0)) * a.rows + p.at;
    };
    Parts own{0, 0, 0}, pre{0, 0, 0};
    if (live) {
        own = parts_of(b, max(off[b], 0));
        const int g = group_of(a, a.prefix.starts, b);
        if (g >= 0) {
            const Segment p = segment_of<const int32_t*>(a, a.batch.requests + g);
            if (t >= p.t0 && t < p.t0 + p.n)  // (offsets that are not in order may leave it out)
                pre = parts_of(a.batch.requests + g, p.t0);
        }
    }
    Joined r = join_parts<DP>(a, together ? wave : 0, together ? kWaves : 1, own.n + pre.n,
                              [&](int i) { return i < own.n ? place(own, i) : place(pre, i - own.n); }, c);
    if (together) {
        meet<DP>(r, lds);
        if (wave)
            return;
    }
    if (live && 8 * c < a.cache.dim)
        store_row<H>(a, r, t, head, c);
}

template <int DP, bool H>
hipError_t run(const AttendArgs& a, hipStream_t s)
{
    constexpr int EACH = 64 / (DP / 8);
    if (a.prefix.groups) {
        // (few rows: four waves each, until there is one for every compute unit's four)
        const bool together = join_blocks(a.T, a.q_heads, EACH) <= 4096;
        const int64_t blocks = join_blocks(a.T, a.q_heads, together ? EACH : EACH * kWaves);
        join_shared<DP, H><<<(unsigned)blocks, kThreads, 0, s>>>(a, together);
    } else {
        // A turn each: rows of small tiles, or of so few that each is cut into four parts and more, by a workgroup's waves together (decode
        // 4.9 us, in turns 5.5; windows of wide heads 6.0 and 11.8), others', too many for that (requests of 500 rows 13.3 us and
        // 10.2), by a wave each.
        const bool few = a.rows < kManyRows || (a.T * a.group / a.rows + a.batch.requests) * (int64_t)a.cache.heads * 4 <= a.workers;
        const int turn = std::min(16, few ? EACH : EACH * kWaves);
        join_tiles<DP, H><<<dim3(a.workers, a.rows / turn), kThreads, 0, s>>>(a, few ? 4 : 8);
    }
    return hipGetLastError();
}

template <bool H>
hipError_t run(const AttendArgs& a, hipStream_t s)
{
    const int width = padded(a.cache.dim);
    return width == 64 ? run<64, H>(a, s) : width == 128 ? run<128, H>(a, s) : run<256, H>(a, s);
}

}  // namespace

hipError_t launch_ranges(const AttendArgs& a, int unit, hipStream_t s)
{
    // (one request may have all tiles; most have a few)
    const int64_t segments = a.batch.requests + a.prefix.groups, tiles = (int64_t)a.T * a.group / a.rows + 1;
    const int64_t each = (tiles + kWaves - 1) / kWaves;
    tile_ranges<<<dim3((unsigned)segments, (unsigned)(each > 64 ? 64 : each)), kThreads, 0, s>>>(a, unit);
    return hipGetLastError();
}

hipError_t launch_join(const AttendArgs& a, bool half, hipStream_t s)
{
    return half ? run<true>(a, s) : run<false>(a, s);
}

}  // namespace hca
