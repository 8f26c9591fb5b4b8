// proj_small.hip -- products of few tokens per group: decoded tokens and
// verify windows, through one projection or through many experts; and the
// adapters' inner product v = A x.
//
// With up to some tens of tokens a product is its weights' way from memory: a
// workgroup takes 16 or 32 rows of W whole, its 8 waves each an eighth of K,
// and every wave has its weights (8 loads of 16 bytes a lane and row block) in
// flight at once, straight into the registers that the matrix instructions
// read; the tokens come the same way from the L2.  The waves' sums meet in LDS.
#include "proj_device.h"

#pragma clang fp contract(off)

namespace hcp {
namespace {

constexpr int kWaves = 8;
constexpr int kUnit = 64;    // k per unit: one 128-byte line of a row, two matrix instructions
constexpr int kUnits = 4;    // units in flight per wave

// TM token blocks of 16, NJ row blocks of 16 (gated: NJ = 2, gate and up).
template <bool H, int MODE, int TM, int NJ>
__global__ __launch_bounds__(kWaves * 64) void small_product(ProductArgs a)
{
    static_assert(MODE != kGate || NJ == 2, "a gate and an up block");
    constexpr int BM = 16 * TM;
    constexpr int BN = MODE == kGate ? 16 : 16 * NJ;
    __shared__ f32x4_t sums[kWaves][TM * NJ][64];
    __shared__ float vs[MODE == kAdapt ? BM * 128 : 1];
    const unsigned cols = (unsigned)(a.N + BN - 1) / BN;
    RowTile t;
    if (!find_tile<BM>(a.offsets, a.E, a.M, blockIdx.x / cols, t))
        return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x % cols * BN;
    const int64_t row_bytes = 2 * (int64_t)a.K;
    const int64_t w_rows = MODE == kGate ? 2 * (int64_t)a.N : a.N;

    gbytes wp[NJ], xp[TM];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int n = n0 + (MODE == kGate ? r : 16 * j + r);
        const int64_t row = (MODE == kGate ? (int64_t)j * a.N : 0) + n;
        wp[j] = n < a.N ? (gbytes)a.W + (t.e * w_rows + row) * row_bytes : nullptr;
    }
#pragma unroll
    for (int m = 0; m < TM; ++m)
        xp[m] = x_row(a, t, 16 * m + r);

    f32x4_t acc[TM][NJ] = {};
    const int units = (a.K + kUnit - 1) / kUnit;
    for (int u0 = wave; u0 < units; u0 += kWaves * kUnits) {
        u32x4 w[kUnits][2][NJ], x[kUnits][2][TM];
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (u0 + u * kWaves) * kUnit + 32 * h + 8 * g;
                const bool in = k < a.K;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    w[u][h][j] = load16(in && wp[j] ? wp[j] + 2 * (int64_t)k : zeros());
#pragma unroll
                for (int m = 0; m < TM; ++m)
                    x[u][h][m] = load16(in && xp[m] ? xp[m] + 2 * (int64_t)k : zeros());
            }
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < TM; ++m)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        acc[m][j] = mfma<H>(w[u][h][j], x[u][h][m], acc[m][j]);
    }
    if constexpr (MODE == kAdapt) {
        // the tokens' v: the splits of the first kernel summed in their order
        for (int i = threadIdx.x; i < t.rows * a.rank; i += kWaves * 64) {
            const float* p = a.v + (int64_t)t.row0 * a.rank + i;
            float s = 0.0f;
            for (int z = 0; z < a.v_splits; ++z)
                s += p[(int64_t)z * a.M * a.rank];
            vs[i] = s;
        }
    }
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            sums[wave][m * NJ + j][lane] = acc[m][j];
    __syncthreads();

    constexpr int kParts = MODE == kGate ? TM : TM * NJ;
    for (int i = threadIdx.x; i < kParts * 64; i += kWaves * 64) {
        const int part = i >> 6, l = i & 63;
        const int m = MODE == kGate ? part : part / NJ, j = MODE == kGate ? 0 : part % NJ;
        const int token = 16 * m + (l & 15);
        const int n = n0 + 16 * j + 4 * (l >> 4);
        if (token >= t.rows || n >= a.N)
            continue;
        f32x4_t s = sums[0][m * NJ + j][l];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            s += sums[w][m * NJ + j][l];
        float y[4] = {s[0], s[1], s[2], s[3]};
        if constexpr (MODE == kGate) {
            f32x4_t up = sums[0][m * NJ + 1][l];
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                up += sums[w][m * NJ + 1][l];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                y[c] = gated(y[c], up[c]);
        }
        const int64_t row = (int64_t)t.row0 + token;
        if constexpr (MODE == kAdapt) {
            const int ad = a.adapter[row];
            if (ad >= 0 && ad < a.adapters) {
                float d[4] = {};
                for (int k = 0; k < a.rank; k += 8)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (n + c >= a.N)
                            break;
                        const u32x4 b = load16((gbytes)a.B + 2 * (((int64_t)ad * a.N + n + c) * a.rank + k));
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            d[c] = fmaf(from16<H>(b[q] & 0xffffu), vs[token * a.rank + k + 2 * q], d[c]);
                            d[c] = fmaf(from16<H>(b[q] >> 16), vs[token * a.rank + k + 2 * q + 1], d[c]);
                        }
                    }
                const float sc = a.scale ? a.scale[ad] : 1.0f;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    y[c] = fmaf(sc, d[c], y[c]);
            }
        }
        store_row<H, 4>(a, row, n, y);
    }
}

// v[z][t][j] for 16 tokens and the k units of split z; RJ row blocks of 16.
// The 16 tokens' adapters are shared out over the workgroups of one tile and
// split (the k-th adapter in order of appearance to workgroup k mod their
// number); each runs over all 16 tokens and keeps its own columns.
template <bool H, int RJ>
__global__ __launch_bounds__(kWaves * 64) void adapter_down(DownArgs a)
{
    __shared__ f32x4_t sums[kWaves][RJ][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int64_t token = (int64_t)blockIdx.x * 16 + r;
    const int ad = token < a.M ? a.adapter[token] : -1;
    bool open = ad >= 0 && ad < a.adapters;
    const gbytes xp = token < a.M ? (gbytes)a.x + token * a.ldx : nullptr;
    const int units = (a.K + kUnit - 1) / kUnit;
    const int u_lo = (int)((int64_t)units * blockIdx.y / a.splits);
    const int u_hi = (int)((int64_t)units * (blockIdx.y + 1) / a.splits);
    for (unsigned turn = 0;; ++turn) {
        const unsigned long long left = __ballot(open);  // (the same in every wave)
        if (!left)
            return;
        const int now = __builtin_amdgcn_readlane(ad, __builtin_ctzll(left));
        const bool mine = open && ad == now;
        open = open && !mine;
        if (turn % gridDim.z != blockIdx.z)
            continue;
        f32x4_t acc[RJ] = {};
        const gbytes A = (gbytes)a.A + 2 * ((int64_t)now * a.rank * a.K);
        for (int u0 = u_lo + wave; u0 < u_hi; u0 += kWaves * 2) {
            u32x4 w[2][2][RJ], x[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = (u0 + u * kWaves) * kUnit + 32 * h + 8 * g;
                    const bool in = u0 + u * kWaves < u_hi && k < a.K;
                    x[u][h] = load16(in && mine ? xp + 2 * (int64_t)k : zeros());
#pragma unroll
                    for (int j = 0; j < RJ; ++j) {
                        const int row = 16 * j + r;
                        w[u][h][j] = load16(in && row < a.rank ? A + 2 * ((int64_t)row * a.K + k) : zeros());
                    }
                }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < RJ; ++j)
                        acc[j] = mfma<H>(w[u][h][j], x[u][h], acc[j]);
        }
#pragma unroll
        for (int j = 0; j < RJ; ++j)
            sums[wave][j][lane] = acc[j];
        __syncthreads();
        for (int j = wave; j < RJ; j += kWaves) {
            f32x4_t s = sums[0][j][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                s += sums[w][j][lane];
            if (mine && 16 * j + 4 * g < a.rank)  // (rank is a multiple of 8)
                *(f32x4_t*)(a.v + ((int64_t)blockIdx.y * a.M + token) * a.rank + 16 * j + 4 * g) = s;
        }
        __syncthreads();
    }
}

// out = the splits' partial sums, in their order.
template <bool H>
__global__ __launch_bounds__(256) void join(ProductArgs a)
{
    const unsigned across = (unsigned)(a.N + 1023) / 1024;
    const int n = (blockIdx.x % across * 256 + threadIdx.x) * 4;
    const int64_t row = blockIdx.x / across;
    if (n >= a.N)
        return;
    float y[4] = {};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (n + c >= a.N)
            break;
        for (int z = 0; z < a.splits; ++z)
            y[c] += a.part[((int64_t)z * a.M + row) * a.N + n + c];
    }
    store_row<H, 4>(a, row, n, y);
}

template <bool H, int MODE>
hipError_t run_small(const ProductArgs& a, int tokens, hipStream_t s)
{
    const int64_t tiles = ((int64_t)a.M + tokens - 1) / tokens + (a.offsets ? (a.E < a.M ? a.E : a.M) : 0);
    constexpr int NJ = MODE == kGate ? 2 : 1;
    const int64_t blocks = tiles * ((a.N + 15) / 16);
    if (!fits(blocks, kWaves * 64))
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(kWaves * 64);
    if (tokens == 16)
        small_product<H, MODE, 1, NJ><<<grid, block, 0, s>>>(a);
    else if (tokens == 32)
        small_product<H, MODE, 2, NJ><<<grid, block, 0, s>>>(a);
    else
        small_product<H, MODE, 4, NJ><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

template <bool H>
void run_down(const DownArgs& a, hipStream_t s)
{
    const int tiles = (a.M + 15) / 16;
    const dim3 grid((unsigned)tiles, (unsigned)a.splits, tiles * a.splits < 256 ? 4u : 1u), block(kWaves * 64);
    if (a.rank <= 16)
        adapter_down<H, 1><<<grid, block, 0, s>>>(a);
    else if (a.rank <= 32)
        adapter_down<H, 2><<<grid, block, 0, s>>>(a);
    else if (a.rank <= 64)
        adapter_down<H, 4><<<grid, block, 0, s>>>(a);
    else
        adapter_down<H, 8><<<grid, block, 0, s>>>(a);
}

}  // namespace

hipError_t launch_small(const ProductArgs& a, int type, int mode, int tokens, hipStream_t s)
{
    if (type == kFp16)
        return mode == kPlain  ? run_small<true, kPlain>(a, tokens, s)
               : mode == kGate ? run_small<true, kGate>(a, tokens, s)
                               : run_small<true, kAdapt>(a, tokens, s);
    return mode == kPlain  ? run_small<false, kPlain>(a, tokens, s)
           : mode == kGate ? run_small<false, kGate>(a, tokens, s)
                           : run_small<false, kAdapt>(a, tokens, s);
}

hipError_t launch_adapter_down(const DownArgs& a, int type, hipStream_t s)
{
    type == kFp16 ? run_down<true>(a, s) : run_down<false>(a, s);
    return hipGetLastError();
}

hipError_t launch_join(const ProductArgs& a, int type, hipStream_t s)
{
    if (!fits((a.N + 1023) / 1024 * (int64_t)a.M, 256))
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)((a.N + 1023) / 1024 * a.M)), block(256);
    if (type == kFp16)
        join<true><<<grid, block, 0, s>>>(a);
    else
        join<false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace hcp
