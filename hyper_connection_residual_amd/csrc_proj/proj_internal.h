// proj_internal.h -- arguments and launchers shared by the host side
// (proj_api.hip) and the kernels of the projections.  Library-internal.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace hcp {

enum Type { kBf16 = 0, kFp16 = 1, kFp32 = 2 };
enum Mode { kPlain = 0, kGate = 1, kAdapt = 2 };

// The most splits of v = A x that the small and the tiled kernel add up; the
// wide one takes one.
constexpr int kSplitsSmall = 4, kSplitsTile = 2;

// One grouped product: out[i] = W[e] x[row of i], for the groups that offsets
// describes (E = 1 without offsets: all M rows).  16-bit operands.
struct ProductArgs {
    const char* x;           // [x_rows][K]
    int64_t ldx;             // bytes
    int64_t x_rows;
    const int32_t* rows;     // row of x per row of out, or NULL
    const char* W;           // [E][N or 2 N][K]
    const int32_t* offsets;  // [E + 1], or NULL
    int E, M, K, N;
    char* out;
    int64_t ldo;             // elements
    int out32;               // fp32 out
    // the adapters beside it (kAdapt)
    const int32_t* adapter;  // [M]
    int adapters, rank;
    const char* B;           // [adapters][N][rank]
    const float* scale;      // [adapters] or NULL
    const float* v;          // [v_splits][M][rank]: partial sums of A x
    int v_splits;
    const char* pieces;      // instead of v for the wide kernel: scale A x in pieces (see piece_chunks)
    // split K (tiles only): partial sums of the splits, [splits][M][N]
    float* part;
    int splits;
};

// scale A x as the wide kernel takes it: a row per token of 16-byte chunks (whole
// lines of 8), each 8 ranks of one of the three bf16 pieces whose sum it is; with
// fp16 weights, which are the sum of two pieces, each chunk twice: chunk q holds
// the ranks 8 (q mod (rank / 8)) and on, and of kind = q / (rank / 8) the piece kind
// (fp16: kind / 2, for the weights' piece kind mod 2; kind 1 without infinities and
// NaNs, see finite_of).
inline __host__ __device__ int piece_chunks(int rank, bool half) { return (half ? 6 : 3) * (rank / 8); }
inline __host__ __device__ int piece_bytes(int rank, bool half) { return (piece_chunks(rank, half) + 7) / 8 * 128; }

struct DownArgs {  // v[z][t][j] = sum over split z of A[adapter[t]][j] x[t]
    const char* x;
    int64_t ldx;  // bytes
    int M, K;
    const int32_t* adapter;
    int adapters, rank;
    const char* A;
    float* v;
    int splits;
    char* pieces;        // instead of v (splits == 1)
    const float* scale;  // (with pieces)
};

// Whether a launch's work-items can be counted in 32 bits.  Launchers return
// hipErrorInvalidConfiguration, and launch nothing, where they cannot.
inline bool fits(int64_t blocks, int threads)
{
    return blocks * threads < (int64_t(1) << 32);
}

// Workgroups of the products, and of each split (a multiple of 8, one for every XCD):
// tiles of `rows` tokens x `cols` outputs; groups: up to one more row tile for each.
inline int64_t product_blocks(int64_t M, int64_t groups, int rows, int64_t N, int cols)
{
    return (((M + rows - 1) / rows + groups) * ((N + cols - 1) / cols) + 7) / 8 * 8;
}
inline int64_t group_tiles(const ProductArgs& a) { return a.offsets ? (a.E < a.M ? a.E : a.M) : 0; }
// ... of the one token's product, of v = A x in its largest grid (many tokens: up to
// two workgroups, of 64 ranks, for each 16), and of join.
inline int64_t token_blocks(int64_t N) { return (N + 15) / 16; }
inline int64_t down_blocks(int64_t M) { return (M + 15) / 16 * 2; }
inline int64_t join_blocks(int64_t M, int64_t N) { return ((N + 3) / 4 * M + 255) / 256; }
constexpr int kSmallThreads = 256;  // (512 in grids of up to 256 workgroups)
constexpr int kSmallCols = 16, kTileThreads = 256, kTileCols = 128, kWideThreads = 512, kWideCols = 256;

hipError_t launch_adapter_down(const DownArgs& a, int type, hipStream_t s);
// one token with an adapter of rank up to kTokenRank (no v)
constexpr int kTokenRank = 64;
hipError_t launch_token(const ProductArgs& a, int type, const char* A, hipStream_t s);
// tokens: of a tile, 8, 16 or 32
hipError_t launch_small(const ProductArgs& a, int type, int mode, int tokens, hipStream_t s);
// tokens: of a tile, 64 or 128; stages: of the ring of 64 (with adapters 3; of 128: 2)
hipError_t launch_tile(const ProductArgs& a, int type, int mode, int tokens, int stages, hipStream_t s);
hipError_t launch_wide(const ProductArgs& a, int type, int mode, hipStream_t s);  // K > 64
hipError_t launch_join(const ProductArgs& a, int type, hipStream_t s);

struct RouteArgs {
    int T, E, k;
    const void* logits;
    int64_t ldl;  // elements
    int type, renorm;
    int vec;  // rows of logits are 16-byte aligned
    int32_t *ids, *offsets, *rows, *pos;
    float* weights;
    int32_t* hist;  // [blocks][E]
};
int route_blocks(int64_t T, int64_t E, int64_t k);  // 1: no scratch
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

struct CombineArgs {
    int T, k, C;
    const void* y;
    int64_t y_rows, ldy;  // elements
    int type;
    const int32_t* pos;
    const float* weights;
    void* out;
    int64_t ldo;
    int out_type;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t s);

}  // namespace hcp
