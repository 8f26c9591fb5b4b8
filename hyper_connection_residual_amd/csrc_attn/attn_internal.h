// attn_internal.h -- arguments and launchers shared by the host side
// (attn_api.hip) and the kernels of the attention.  Library-internal.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace hca {

// (strides in bytes)
struct CacheArgs {
    char *k, *v;
    int64_t pages, k_page, v_page;
    int k_row, k_head, v_row, v_head;
    int shift;  // page_size == 1 << shift
    int heads, dim;
};

struct BatchArgs {
    const int32_t *offsets, *lengths, *table;
    int64_t table_row;
    int requests, width;
};

struct PrefixArgs {
    const int32_t *starts, *lengths, *table;
    int64_t table_row;
    int groups, width;
};

struct HeadsArgs {
    const char* x;
    int64_t row, head;
};

struct RotateArgs {
    int T, dim, rotated, interleaved;
    HeadsArgs q, k, v;  // (k and v: with a cache)
    int q_heads;
    char* out;
    int64_t out_row, out_head;
    const int32_t* positions;
    const float *frequencies, *q_weight, *k_weight;
    float eps;
    int chunk;  // turns of a wave
    CacheArgs cache;
    BatchArgs batch;
};

struct AttendArgs {
    HeadsArgs q;
    char* out;
    int64_t out_row, out_head;
    CacheArgs cache;
    BatchArgs batch;
    PrefixArgs prefix;
    int T, q_heads, group;  // group: q_heads / cache.heads
    float scale;            // of a product, to its score over ln 2: not below zero ...
    uint32_t q_sign;        // ... the queries' signs are changed instead (both halves' sign bits, or none)
    float cap_in, cap_out;  // with a cap: score over ln 2 = cap_out tanh(product cap_in / 2 ln 2), see capped()
    const float* slopes;
    const int32_t *first, *last;
    // scratch: see Scratch
    int rows;     // of a tile
    int tiles;    // of all segments, at most (lists in order)
    int workers;  // workgroups
    int least;    // units that a worker gets at least
    int item_cost;  // see Start
    float* part;
    float2* ml;
    int32_t *records, *plan;
    int2* ranges;  // NULL without first and last
};

// Tokens off[b0] .. off[b1], of lists with any numbers in them.
template <class P>
__host__ __device__ inline void clamped_range(int T, P off, int b0, int b1, int& lo, int& hi)
{
    const int from = off[b0], to = off[b1];
    lo = from < 0 ? 0 : from < T ? from : T;
    hi = to < lo ? lo : to < T ? to : T;
}
__host__ __device__ inline int tiles_of(int tokens, int group, int rows) { return (int)((unsigned)(tokens * group + rows - 1) / (unsigned)rows); }
// Whether a plan of so many tiles is made.  The scratch and the counts of units have room for the tiles of lists in
// order, which share no token; of those that are not, segments may overlap (0, T, 0, T, ...: every second one
// has all tokens) and have any number of tiles.  Such a call computes nothing.
__host__ __device__ inline bool planned(int tiles, int room) { return tiles <= room; }
// Numbers of a.plan.
__host__ __device__ inline int64_t plan_numbers(int64_t segments, int64_t tiles) { return 2 + segments + 1 + tiles + 1; }

// Scratch of one call.  part and ml: `width` unscaled sums, and (maximum over ln
// 2, sum), of rows: first two slots of `rows` rows for each worker, for tiles that it
// does not hold whole (the first: one that it goes on with, the second: one that it
// begins); then, under prefixes, the rows of whole tiles by (token, head), those over
// own positions and those over prefixes.  records: the tile that a worker begins and
// others end; plan: the units and tiles in all, the first tile of each segment and the
// first unit of each tile; ranges: the first and last unit of each tile.
constexpr int kWorkers = 512;
struct Record {
    int32_t t0, row0, rows, head, last;  // rows 0: none
    int32_t pad[3];
};
struct Scratch {
    int64_t ml, records, plan, ranges, bytes;  // offsets
};
constexpr int64_t pad256(int64_t n) { return (n + 255) & ~int64_t(255); }
// Rows of the workers' two partial results each (of tiles of 256 rows, half the workers').
constexpr int64_t slot_rows(int rows) { return int64_t(2 * kWorkers) * (rows == 256 ? 128 : rows); }
// (tiles: T group / rows for the own segments and for the prefixes, and one for each segment)
inline Scratch scratch_of(int64_t T, int64_t q_heads, int rows, int width, int64_t segments, int64_t tiles, bool shared)
{
    const int64_t all = slot_rows(rows) + (shared ? 2 * T * q_heads : 0);
    Scratch s{};
    s.ml = pad256(4 * all * width);
    s.records = s.ml + pad256(8 * all);
    s.plan = s.records + pad256(int64_t(sizeof(Record)) * kWorkers);
    s.ranges = s.plan + (shared ? pad256(4 * plan_numbers(segments, tiles)) : 0);
    s.bytes = s.ranges + pad256(8 * (tiles + 2));
    return s;
}

// The most segments (requests and prefixes) and row tiles of a call: 16-bit and
// 32-bit lists in LDS.
constexpr int kMaxRequests = 2048, kMaxRows = 1 << 18;
constexpr int kManyRows = 128;                                           // rows of a tile of the many kernel, at least
constexpr int kMaxSegments = 2 * kMaxRequests;                           // requests and groups
constexpr int kMaxTiles = 2 * (kMaxRows / kManyRows) + kMaxSegments;     // own and under prefixes

inline int padded(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// Whether a launch's work-items can be counted in 32 bits.
inline bool fits(int64_t blocks, int threads) { return blocks * threads < (int64_t(1) << 32); }

// Lanes of a head in rotate, how many turns (of 64 lanes' heads) a wave takes of a
// token, and the launch's workgroups.  One turn until there are 16 waves for every
// compute unit, then more, which share their sines.
constexpr int kRotateThreads = 256;
inline int rotate_lanes(int dim) { return dim <= 32 ? 4 : dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }
inline int64_t rotate_turns(int64_t heads, int dim) { return (heads * rotate_lanes(dim) + 63) / 64; }
inline int64_t rotate_chunk(int64_t T, int64_t heads, int dim)
{
    const int64_t turns = rotate_turns(heads, dim), want = turns * T / 4096;
    return want < 1 ? 1 : want > turns ? turns : want;
}
inline int64_t rotate_blocks(int64_t T, int64_t heads, int dim)
{
    const int64_t chunk = rotate_chunk(T, heads, dim);
    return (T * ((rotate_turns(heads, dim) + chunk - 1) / chunk) + kRotateThreads / 64 - 1) / (kRotateThreads / 64);
}
constexpr int kJoinThreads = 256;
inline int64_t join_blocks(int64_t T, int64_t q_heads, int rows) { return (T * q_heads + rows - 1) / rows; }

hipError_t launch_rotate(const RotateArgs& a, bool half, bool append, hipStream_t s);
hipError_t launch_few(const AttendArgs& a, bool half, hipStream_t s);   // rows: 16, or (heads of more than 128 columns) 32
hipError_t launch_many_bf16(const AttendArgs& a, hipStream_t s);      // rows: 128 or (heads of up to 128 columns) 256
hipError_t launch_many_fp16(const AttendArgs& a, hipStream_t s);
hipError_t launch_ranges(const AttendArgs& a, int unit, hipStream_t s);
constexpr int kFewUnit = 32, kStepBytes = 16384;  // positions of a unit of the few kernel; bytes of keys of one of the many kernel
hipError_t launch_join(const AttendArgs& a, bool half, hipStream_t s);

}  // namespace hca
