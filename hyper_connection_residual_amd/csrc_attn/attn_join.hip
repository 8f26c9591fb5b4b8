// attn_join.hip -- the parts of rows that several workers hold, or under
// prefixes two segments, become outputs.  A wave joins one row: the parts'
// (maximum, sum) by a lane each, then their sums, columns by lane.
#include "attn_device.h"

#pragma clang fp contract(off)

namespace hca {
namespace {

constexpr int kThreads = kJoinThreads;

__device__ __forceinline__ float wave_max(float x)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        x = fmaxf(x, __shfl_xor(x, d));
    return x;
}
__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        x += __shfl_xor(x, d);
    return x;
}

// of(i): the place of part i of n in a.ml and a.part.
template <int DP, bool H, class Of>
__device__ __forceinline__ void join_row(const AttendArgs& a, int n, Of of, int t, int head)
{
    constexpr int COLS = DP / 64;  // of a lane
    typedef float cols_t __attribute__((ext_vector_type(COLS)));
    const int lane = threadIdx.x & 63;
    float top = kLowest;
    for (int i = lane; i < n; i += 64)
        top = fmaxf(top, a.ml[of(i)].x);
    top = wave_max(top);
    float sum = 0.0f;
    cols_t y{};
    for (int i0 = 0; i0 < n; i0 += 64) {
        int64_t at = 0;
        float by = 0.0f;
        if (i0 + lane < n) {
            at = of(i0 + lane);
            const float2 ml = a.ml[at];
            by = exp2_of(ml.x - top);
            sum = fmaf(by, ml.y, sum);
        }
        // four parts on their way at a time; a part that counts for nothing adds nothing,
        // whatever it holds
        const int here = min(64, n - i0);
        for (int i = 0; i < here; i += 4) {
            cols_t part[4];
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int x = min(i + e, here - 1);
                const int64_t from = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)at, x) |
                                               (uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(at >> 32), x) << 32);
                f[e] = i + e < here ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(by), x)) : 0.0f;
                if constexpr (COLS == 1)
                    part[e][0] = a.part[from * DP + lane];
                else
                    part[e] = *(const cols_t*)(a.part + from * DP + COLS * lane);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < COLS; ++c)
                    y[c] = f[e] != 0.0f ? fmaf(f[e], part[e][c], y[c]) : y[c];
        }
    }
    sum = wave_sum(sum);
    if (COLS * lane >= a.cache.dim)
        return;
    const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
    char* const out = a.out + t * a.out_row + head * a.out_head + 2 * COLS * lane;
    if constexpr (COLS == 1)
        *(uint16_t*)out = (uint16_t)bits16<H>(y[0] * by);
    else
#pragma unroll
        for (int e = 0; e < COLS; e += 2)
            ((uint32_t*)out)[e / 2] = pack2<H>(y[e] * by, y[e + 1] * by);
}

// Tiles that were cut between workers: blockIdx.x is the worker that begins one.
template <int DP, int ROWS, bool H>
__global__ __launch_bounds__(kThreads) void join_tiles(AttendArgs a)
{
    const Record rec = ((const Record*)a.records)[blockIdx.x];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = blockIdx.x;
    for (int i = 4 * blockIdx.y + wave; i < rec.rows; i += 4 * gridDim.y) {
        const int row = rec.row0 + i, t = rec.t0 + row / a.group, head = rec.head * a.group + row % a.group;
        // the first part is the beginning worker's second slot, the others' are their first
        join_row<DP, H>(a, rec.last - w + 1, [&](int p) { return (int64_t)(2 * (w + p) + (p == 0)) * ROWS + i; }, t, head);
    }
}

// Under prefixes: every row, of its own positions and its prefix's.
template <int DP, int ROWS, bool H>
__global__ __launch_bounds__(kThreads) void join_shared(AttendArgs a)
{
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int t = __builtin_amdgcn_readfirstlane((int)(id / a.q_heads)), head = __builtin_amdgcn_readfirstlane((int)(id % a.q_heads));
    if (t >= a.T)
        return;
    const int lane = threadIdx.x & 63;
    const ints off = scalars(a.batch.offsets);
    // the token's request: as many end at or before it
    int b = 0;
    for (int i = 0; i < a.batch.requests; i += 64) {
        const bool before = i + lane < a.batch.requests && a.batch.offsets[min(i + lane, a.batch.requests - 1) + 1] <= t;
        const int n = __popcll(__ballot(before));
        b += n;
        if (n < 64)
            break;
    }
    if (b >= a.batch.requests || t < off[b] || t < 0)
        return;
    const ints plan = scalars(a.plan);
    const int S = a.batch.requests + a.prefix.groups, units = plan[0], tiles = plan[1];
    const int64_t all = (int64_t)units * a.cache.heads;
    if (all == 0)
        return;
    const int workers = (int)min((int64_t)a.workers, all);
    const int g = group_of(a, scalars(a.prefix.starts), b);
    // the parts of the row in segment s: whole, in the dense lists; or in the slots of workers from .. to
    struct Parts {
        int from, n;
        int64_t at;
    };
    const auto parts_of = [&](int s, int t0) {
        const int row = (t - t0) * a.group + head % a.group, i = min(plan[2 + s] + row / ROWS, tiles - 1);
        const int64_t u = (int64_t)(head / a.group) * units + plan[3 + S + i], end = u + plan[4 + S + i] - plan[3 + S + i];
        const int w0 = worker_of(all, workers, u), w1 = worker_of(all, workers, end - 1);
        Parts p;
        p.from = w0;
        p.n = w1 - w0 + 1;
        p.at = w0 == w1 ? slot_rows(ROWS) + (s >= a.batch.requests ? (int64_t)a.T * a.q_heads : 0) + (int64_t)t * a.q_heads + head : row % ROWS;
        return p;
    };
    const auto place = [&](const Parts& p, int i) {
        return p.n == 1 ? p.at : (int64_t)(2 * (p.from + i) + (i == 0)) * ROWS + p.at;
    };
    const Parts own = parts_of(b, max(off[b], 0));
    Parts pre{0, 0, 0};
    if (g >= 0) {
        const Segment seg = segment_of<ints>(a, a.batch.requests + g);
        pre = parts_of(a.batch.requests + g, seg.t0);
    }
    join_row<DP, H>(a, own.n + pre.n, [&](int i) { return i < own.n ? place(own, i) : place(pre, i - own.n); }, t, head);
}

template <int DP, int ROWS, bool H>
hipError_t run(const AttendArgs& a, hipStream_t s)
{
    if (a.prefix.groups) {
        join_shared<DP, ROWS, H><<<(unsigned)join_blocks(a.T, a.q_heads), kThreads, 0, s>>>(a);
    } else {
        join_tiles<DP, ROWS, H><<<dim3(kWorkers, ROWS / 16), kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <int DP, bool H>
hipError_t run(const AttendArgs& a, int rows, hipStream_t s)
{
    return rows == 16 ? run<DP, 16, H>(a, s) : rows == 32 ? run<DP, 32, H>(a, s) : rows == 64 ? run<DP, 64, H>(a, s) : run<DP, kManyRows, H>(a, s);
}

template <bool H>
hipError_t run(const AttendArgs& a, int rows, hipStream_t s)
{
    const int width = padded(a.cache.dim);
    return width == 64 ? run<64, H>(a, rows, s) : width == 128 ? run<128, H>(a, rows, s) : run<256, H>(a, rows, s);
}

}  // namespace

hipError_t launch_join(const AttendArgs& a, bool half, int rows, hipStream_t s)
{
    return half ? run<true>(a, rows, s) : run<false>(a, rows, s);
}

}  // namespace hca
