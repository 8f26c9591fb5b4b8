// proj_small.hip -- products of few tokens per group: decoded tokens and
// verify windows, through one projection or through many experts; and the
// adapters' inner product v = A x.
//
// With up to some tens of tokens a product is its weights' way from memory.  A
// workgroup takes 16 rows of W whole, its 4 or 8 waves each their part of K;
// every wave streams its own units (128 bytes of each row, of W and of x) through
// a ring of its own in LDS and waits for no other wave until the sums meet at
// the end.  A grid that one round of workgroups holds takes 8 waves and all of
// LDS for each, everything on its way at once; a larger one 4 waves and a quarter
// of LDS, so that other workgroups load while one begins or ends (64 experts'
// gated products, 671 MB: 131 us with one or two workgroups of 8 waves on a
// compute unit, 109 us with three, 112 us with four of 4 waves, which are the
// faster ones for 16 and more tokens per tile: 119 us against 147 us).  The way through LDS is for the
// loads' sake: the matrix instructions want a row in every 16th lane, but the
// memory pipeline takes 64 cycles for a load whose neighbouring lanes read
// different rows, and 16 where 8 neighbours read one line (straight into
// registers, 10240 x 2560 took 16 us for 8 tokens and 30 us for 32).
#include "proj_tile.h"

#pragma clang fp contract(off)

namespace hcp {
namespace {

// Waits until at most `units` units of L loads each are in flight.
template <int L>
__device__ __forceinline__ void wait_units(int units)
{
    if (units >= 4)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(4 * L) : "memory");
    else if (units == 3)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * L) : "memory");
    else if (units == 2)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * L) : "memory");
    else if (units == 1)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L) : "memory");
    else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// One wave's part of a product: units u_lo + wave, + WAVES, ... below u_hi of 16 NJ
// rows of W and 8 TX tokens, through its ring of D units.  wp, xp: this lane's
// rows (8 i + lane / 8), at its chunk (lane & 7) ^ (row & 7).
template <bool H, int TX, int NJ, int D, int WAVES>
struct Stream {
    static constexpr int TM = (TX + 1) / 2;
    static constexpr int UNIT = (2 * NJ + 2 * TM) * 1024;  // (a half block of tokens leaves its other half as it is)
    static constexpr int LOADS = 2 * NJ + TX;
    static_assert(D >= 1 && D <= 5 && 4 * LOADS < 64, "wait_units, vmcnt");

    char* ring;
    gbytes wp[2 * NJ], xp[TX];

    __device__ __forceinline__ void send(int unit, int slot, int K)
    {
        if ((unit + 1) * kStep > K) {  // pieces past K are zeros
            const int lane = threadIdx.x & 63;
            if (unit * kStep + 8 * ((lane & 7) ^ (lane >> 3)) >= K) {
#pragma unroll
                for (int i = 0; i < 2 * NJ; ++i)
                    wp[i] = zeros();
#pragma unroll
                for (int i = 0; i < TX; ++i)
                    xp[i] = zeros();
            }
        }
#pragma unroll
        for (int i = 0; i < 2 * NJ; ++i) {
            dma16(wp[i], ring + slot * UNIT + i * 1024);
            wp[i] += 2 * kStep * WAVES;
        }
#pragma unroll
        for (int i = 0; i < TX; ++i) {
            dma16(xp[i], ring + slot * UNIT + (2 * NJ + i) * 1024);
            xp[i] += 2 * kStep * WAVES;
        }
    }

    // The first units are on their way after begin(); run() waits and multiplies.
    __device__ __forceinline__ void begin(int first, int u_hi, int K)
    {
#pragma unroll
        for (int i = 0; i < 2 * NJ; ++i)
            wp[i] += 2 * kStep * (int64_t)first;
#pragma unroll
        for (int i = 0; i < TX; ++i)
            xp[i] += 2 * kStep * (int64_t)first;
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (first + d * WAVES < u_hi)
                send(first + d * WAVES, d, K);
    }
    __device__ __forceinline__ void run(int first, int u_hi, int K, f32x4_t (&acc)[TM][NJ])
    {
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
        const uint32_t at = lds_addr(ring) + r * 128;
        const uint32_t c0 = 16 * (g ^ swizzle(r)), c1 = 16 * ((g + 4) ^ swizzle(r));
        int slot = 0;
        for (int u = first; u < u_hi; u += WAVES) {
            wait_units<LOADS>(min(D - 1, (u_hi - 1 - u) / WAVES));
            const uint32_t base = at + slot * UNIT;
            u32x4 w[2][NJ], x[2][TM];
            read_blocks<NJ>(base + c0, base + c1, w);
            read_blocks<TM>(base + NJ * 2048 + c0, base + NJ * 2048 + c1, x);
            if (u + D * WAVES < u_hi)
                send(u + D * WAVES, slot, K);
            slot = slot + 1 == D ? 0 : slot + 1;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int m = 0; m < TM; ++m)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        acc[m][j] = mfma<H>(w[h][j], x[h][m], acc[m][j]);
        }
    }
};

// Units per ring, of which all of a workgroup's have the 160 KB of LDS (one
// workgroup on a compute unit) or a quarter of it.
constexpr int ring_units(int unit_bytes, int waves, bool deep)
{
    const int d = (deep ? 160 : 40) * 1024 / (waves * unit_bytes);
    return d > 5 ? 5 : d < 1 ? 1 : d;
}

// The order of one group's tiles: each of the 8 XCDs (workgroup b runs on XCD
// b % 8) takes a contiguous eighth, in which the tiles that share the larger
// operand's rows follow each other, so that it is read from memory once (6140
// tokens x 6376 -> 35 outputs: 82 us in plain order).
__device__ __forceinline__ bool small_tile_of(const ProductArgs& a, unsigned rows_per_tile, unsigned cols, unsigned& row_tile,
                                              unsigned& col)
{
    const unsigned tiles = ((unsigned)a.M + rows_per_tile - 1) / rows_per_tile, total = tiles * cols, each = (total + 7) / 8;
    const unsigned id = (blockIdx.x & 7) * each + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= each || id >= total)
        return false;
    row_tile = a.M > a.N ? id / cols : id % tiles;
    col = a.M > a.N ? id % cols : id / tiles;
    return true;
}

// 8 TX tokens, 16 rows of W (gated: 16 of each).  Bound by memory: 8 experts of one
// token, gated 2560 -> 1024, 84 MB in 15.3 us, 5.5 TB/s; 64 rows of 64 experts,
// 1024 -> 2560, 227 MB in 44 us, 5.2 TB/s; 25 tokens, 2560 -> 10240, 56 MB in 17.4 us.
template <bool H, int MODE, int TX, bool DEEP>
__global__ __launch_bounds__(DEEP ? 512 : 256) void small_product(ProductArgs a)
{
    constexpr int WAVES = DEEP ? 8 : 4;
    constexpr int NJ = MODE == kGate ? 2 : 1;
    constexpr int TM = (TX + 1) / 2, BM = 8 * TX;
    constexpr int UNIT = (2 * NJ + 2 * TM) * 1024, D = ring_units(UNIT, WAVES, DEEP);
    __shared__ __align__(128) char lds[WAVES * D * UNIT];
    static_assert(D * UNIT >= TM * NJ * 1024, "the waves' sums take the rings' place");
    const unsigned cols = (unsigned)(a.N + 15) / 16;
    unsigned row_tile = blockIdx.x / cols, col = blockIdx.x % cols;
    if (!a.offsets && !small_tile_of(a, BM, cols, row_tile, col))
        return;
    RowTile t;
    if (!find_tile<BM>(a.offsets, a.E, a.M, row_tile, t))
        return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    const int n0 = col * 16;
    const int64_t row_bytes = 2 * (int64_t)a.K;
    const int64_t w_rows = MODE == kGate ? 2 * (int64_t)a.N : a.N;
    const int units = (a.K + kStep - 1) / kStep;

    // Rows past W and past the tile read one that exists; their results are not
    // stored.
    Stream<H, TX, NJ, D, WAVES> stream;
    stream.ring = lds + wave * D * UNIT;
    const int chunk = 16 * ((lane & 7) ^ (lane >> 3));
#pragma unroll
    for (int i = 0; i < 2 * NJ; ++i) {
        const int n = min(n0 + 8 * (i & 1) + (lane >> 3), a.N - 1);
        stream.wp[i] = (gbytes)a.W + (t.e * w_rows + (int64_t)(i >> 1) * a.N + n) * row_bytes + chunk;
    }
#pragma unroll
    for (int i = 0; i < TX; ++i) {
        const gbytes row = x_row(a, t, min(8 * i + (lane >> 3), t.rows - 1));
        stream.xp[i] = (row ? row : (gbytes)a.x) + chunk;
    }
    stream.begin(wave, units, a.K);

    f32x4_t acc[TM][NJ] = {};
    stream.run(wave, units, a.K, acc);

    if constexpr (MODE == kAdapt) {
        // the adapters' part: wave w adds the ranks 8 w and on, 8 at a time, to its sums.
        // (A scale that is not finite multiplies the sum over all ranks: wave 0 takes that.)
        bool odd = false;
        for (int k = 8 * wave; k < a.rank; k += 8 * WAVES)
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const int64_t token = (int64_t)t.row0 + min(16 * m + r, t.rows - 1);
                const int ad = a.adapter[token];
                const bool has = ad >= 0 && ad < a.adapters;
                const int own = has ? ad : 0;
                u32x4 b[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    b[c] = load16((gbytes)a.B + 2 * (((int64_t)own * a.N + min(n0 + 4 * g + c, a.N - 1)) * a.rank + k));
                // v: the splits of the first kernel summed in their order
                f32x4_t v[kSplitsSmall][2];
#pragma unroll
                for (int z = 0; z < kSplitsSmall; ++z) {
                    const gbytes p = (gbytes)a.v + 4 * (((int64_t)min(z, a.v_splits - 1) * a.M + token) * a.rank + k);
                    v[z][0] = __builtin_bit_cast(f32x4_t, load16(p));
                    v[z][1] = __builtin_bit_cast(f32x4_t, load16(p + 16));
                }
                const float sc = a.scale ? a.scale[own] : 1.0f;
                const bool add = has && !is_odd(sc);
                odd = (has && is_odd(sc)) || odd;
#pragma unroll
                for (int z = 1; z < kSplitsSmall; ++z)
                    if (z < a.v_splits) {
                        v[0][0] += v[z][0];
                        v[0][1] += v[z][1];
                    }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float d = 0.0f;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        d = fmaf(from16<H>(b[c][q] & 0xffffu), v[0][q >> 1][2 * (q & 1)], d);
                        d = fmaf(from16<H>(b[c][q] >> 16), v[0][q >> 1][2 * (q & 1) + 1], d);
                    }
                    acc[m][0][c] = add ? fmaf(sc, d, acc[m][0][c]) : acc[m][0][c];
                }
            }
        if (__builtin_expect(wave == 0 && __ballot(odd) != 0, 0)) {
#pragma unroll
            for (int m = 0; m < TM; ++m) {
                const int64_t token = (int64_t)t.row0 + min(16 * m + r, t.rows - 1);
                const int ad = a.adapter[token];
                const float sc = a.scale && ad >= 0 && ad < a.adapters ? a.scale[ad] : 1.0f;
                if (!is_odd(sc))
                    continue;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[m][0][c] += sc * rank_sum<H, false>(a, token, ad, min(n0 + 4 * g + c, a.N - 1), true);
            }
        }
    }
    __syncthreads();  // (every wave is done with its ring)
    f32x4_t* const sums = (f32x4_t*)lds;  // [wave][TM * NJ][64]
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            sums[(wave * TM * NJ + m * NJ + j) * 64 + lane] = acc[m][j];
    __syncthreads();
    static_assert(TM <= WAVES, "a wave for every block of tokens");
    if (wave >= TM)
        return;
    const int token = 16 * wave + r, n = n0 + 4 * g;
    if (token >= t.rows || n >= a.N)
        return;
    f32x4_t s[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        s[j] = sums[(wave * NJ + j) * 64 + lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            s[j] += sums[(w * TM * NJ + wave * NJ + j) * 64 + lane];
    }
    float y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
        y[c] = MODE == kGate ? gated(s[0][c], s[NJ - 1][c]) : s[0][c];
    if (a.rows && !x_row(a, t, token)) {  // a row that x does not have is zeros
#pragma unroll
        for (int c = 0; c < 4; ++c)
            y[c] = 0.0f;
    }
    store_row<H, 4>(a, (int64_t)t.row0 + token, n, y);
}

// One token with an adapter, in one launch: every workgroup takes 16 rows of W
// and, as 16 RJ rows more, all of its adapter's A, so that v is known where B
// needs it (the second kernel costs 5 us of 9 at 2560 x 2560; A is read by every
// workgroup, but from the L2).  5.7 us for rank 16, most of it a kernel's start and
// the way of the first bytes and the last.
template <bool H, int RJ, bool DEEP>
__global__ __launch_bounds__(DEEP ? 512 : 256) void token_product(ProductArgs a, const char* A)
{
    constexpr int WAVES = DEEP ? 8 : 4;
    using S0 = Stream<H, 1, 1 + RJ, 1, WAVES>;
    constexpr int D = ring_units(S0::UNIT, WAVES, DEEP);
    constexpr int UNIT = S0::UNIT;
    __shared__ __align__(128) char lds[WAVES * D * UNIT];
    __shared__ f32x4_t sums[WAVES][1 + RJ][4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n0 = blockIdx.x * 16, units = (a.K + kStep - 1) / kStep;
    const int ad = __builtin_amdgcn_readfirstlane(a.adapter[0]);
    const bool has = ad >= 0 && ad < a.adapters;
    const int own = has ? ad : 0;
    const int64_t row_bytes = 2 * (int64_t)a.K;

    Stream<H, 1, 1 + RJ, D, WAVES> stream;
    stream.ring = lds + wave * D * UNIT;
    const int chunk = 16 * ((lane & 7) ^ (lane >> 3));
#pragma unroll
    for (int i = 0; i < 2; ++i)
        stream.wp[i] = (gbytes)a.W + min(n0 + 8 * i + (lane >> 3), a.N - 1) * row_bytes + chunk;
#pragma unroll
    for (int i = 0; i < 2 * RJ; ++i)
        stream.wp[2 + i] = (gbytes)A + ((int64_t)own * a.rank + min(8 * i + (lane >> 3), a.rank - 1)) * row_bytes + chunk;
    stream.xp[0] = (gbytes)a.x + chunk;
    stream.begin(wave, units, a.K);

    // lane 4 n + q of the first wave ends output n0 + n; its ranks are 4 RJ q and on
    const int n = min(n0 + (lane >> 2), a.N - 1), j0 = 4 * RJ * (lane & 3);
    uint2 b[RJ];
#pragma unroll
    for (int i = 0; i < RJ; ++i)
        if (wave == 0)
            b[i] = *(const uint2*)(a.B + 2 * (((int64_t)own * a.N + n) * a.rank + min(j0 + 4 * i, a.rank - 4)));
    const float sc = a.scale ? a.scale[own] : 1.0f;

    f32x4_t acc[1][1 + RJ] = {};
    stream.run(wave, units, a.K, acc);
    if ((lane & 15) == 0) {  // (the token is column 0)
#pragma unroll
        for (int j = 0; j < 1 + RJ; ++j)
            sums[wave][j][lane >> 4] = acc[0][j];
    }
    __syncthreads();
    if (wave)
        return;
    const int i4 = (lane >> 2) & 3;
    float y = 0.0f, d = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        y += sums[w][0][lane >> 4][i4];
#pragma unroll
    for (int i = 0; i < RJ; ++i) {
        const int j = j0 + 4 * i;
        f32x4_t v = {};
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            v += sums[w][1 + (j >> 4)][(j >> 2) & 3];
        if (j < a.rank) {
            d = fmaf(from16<H>(b[i].x & 0xffffu), v[0], d);
            d = fmaf(from16<H>(b[i].x >> 16), v[1], d);
            d = fmaf(from16<H>(b[i].y & 0xffffu), v[2], d);
            d = fmaf(from16<H>(b[i].y >> 16), v[3], d);
        }
    }
    d += __shfl_xor(d, 1);
    d += __shfl_xor(d, 2);
    y = has ? fmaf(sc, d, y) : y;
    if ((lane & 3) == 0 && n0 + (lane >> 2) < a.N) {
        if (a.out32)
            ((float*)a.out)[n] = y;
        else
            ((uint16_t*)a.out)[n] = (uint16_t)bits16<H>(y);
    }
}

// v[z][t][j] (or its pieces) for 16 tokens, 16 NJ ranks and the k units of split z.  The 16
// tokens' adapters are shared out over the workgroups of one tile (the k-th in
// order of appearance to workgroup k mod their number); each runs over all 16
// tokens and keeps its own columns.  Bound by the ways of its few bytes: 25 tokens
// x 2560, rank 32, 5.8 us; 333 x 10240 of 24 requests, rank 64, 16 us; 8192 x 2560,
// 18 us for rank 16 and 28 us for rank 64 (x alone, 42 MB: 9 us; with x in the last
// level cache 11 and 19 us).
template <bool H, int NJ, bool DEEP>
__global__ __launch_bounds__(DEEP ? 512 : 256) void adapter_down(DownArgs a)
{
    constexpr int WAVES = DEEP ? 8 : 4;
    constexpr int UNIT = (2 * NJ + 2) * 1024, D = ring_units(UNIT, WAVES, DEEP);
    __shared__ __align__(128) char lds[WAVES * D * UNIT];
    f32x4_t* const sums = (f32x4_t*)lds;  // [wave][NJ][64], in the rings' place
    static_assert(D * UNIT >= NJ * 1024, "room for the sums");
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    const int64_t token = (int64_t)blockIdx.x * 16 + r;
    const int ad = token < a.M ? a.adapter[token] : -1;
    bool open = ad >= 0 && ad < a.adapters;
    const int blocks = (a.rank + 16 * NJ - 1) / (16 * NJ);
    const int z = blockIdx.y / blocks, j0 = blockIdx.y % blocks * 16 * NJ;
    const int units = (a.K + kStep - 1) / kStep;
    const int u_lo = (int)((int64_t)units * z / a.splits), u_hi = (int)((int64_t)units * (z + 1) / a.splits);
    const int chunk = 16 * ((lane & 7) ^ (lane >> 3));
    for (unsigned turn = 0;; ++turn) {
        const unsigned long long left = __ballot(open);  // (the same in every wave)
        if (!left)
            return;
        const int now = __builtin_amdgcn_readlane(ad, __builtin_ctzll(left));
        const bool mine = open && ad == now;
        open = open && !mine;
        if (turn % gridDim.z != blockIdx.z)
            continue;
        Stream<H, 2, NJ, D, WAVES> stream;
        stream.ring = lds + wave * D * UNIT;
#pragma unroll
        for (int i = 0; i < 2 * NJ; ++i)
            stream.wp[i] = (gbytes)a.A + chunk +
                           2 * ((int64_t)now * a.rank + min(j0 + 8 * i + (lane >> 3), a.rank - 1)) * a.K;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            stream.xp[i] = (gbytes)a.x + chunk + min((int64_t)blockIdx.x * 16 + 8 * i + (lane >> 3), (int64_t)a.M - 1) * a.ldx;
        f32x4_t acc[1][NJ] = {};
        stream.begin(u_lo + wave, u_hi, a.K);
        stream.run(u_lo + wave, u_hi, a.K, acc);
        __syncthreads();  // (every wave is done with its ring)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            sums[(wave * NJ + j) * 64 + lane] = acc[0][j];
        __syncthreads();
        for (int j = wave; j < NJ; j += WAVES) {
            f32x4_t s = sums[j * 64 + lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w)
                s += sums[(w * NJ + j) * 64 + lane];
            const int rank = j0 + 16 * j + 4 * g;
            if (!mine || rank >= a.rank)  // (rank is a multiple of 8)
                continue;
            if (a.pieces) {
                s *= a.scale ? finite_scale(a.scale[now]) : 1.0f;
                uint2* const to = (uint2*)(a.pieces + token * piece_bytes(a.rank, H) + 2 * rank);
#pragma unroll
                for (int kind = 0; kind < (H ? 6 : 3); ++kind) {
                    const int p = H ? kind >> 1 : kind;
                    uint2 both{piece(s[0], p) | piece(s[1], p) << 16, piece(s[2], p) | piece(s[3], p) << 16};
                    if (kind == 1 && H) {  // (the weights' second piece is mostly zero, and 0 times inf is a NaN)
                        const u32x4 f = finite_of<false>(u32x4{both.x, both.y, 0, 0});
                        both = uint2{f[0], f[1]};
                    }
                    to[kind * (a.rank / 4)] = both;
                }
            } else {
                *(f32x4_t*)(a.v + ((int64_t)z * a.M + token) * a.rank + rank) = s;
            }
        }
        __syncthreads();  // (the sums are read: the next adapter's rings may come)
    }
}

// out = the splits' partial sums, in their order.  A thread takes four outputs,
// its splits' loads together (333 x 2560, 4 splits: 17 MB in 5 us).
template <bool H, int Z>
__global__ __launch_bounds__(256) void join(ProductArgs a)
{
    const unsigned across = (unsigned)(a.N + 3) / 4;
    const unsigned i = blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / across;
    const int n = (int)(i - (unsigned)row * across) * 4;
    if (row >= a.M)
        return;
    const int64_t split = (int64_t)a.M * a.N;
    const float* p = a.part + row * a.N + n;
    float y[4] = {};
    if (n + 4 <= a.N) {
        f32x4_t v[Z];
#pragma unroll
        for (int z = 0; z < Z; ++z)
            v[z] = *(const f32x4_at4*)(p + z * split);
#pragma unroll
        for (int z = 1; z < Z; ++z)
            v[0] += v[z];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            y[c] = v[0][c];
    } else {
        for (int c = 0; n + c < a.N; ++c)
#pragma unroll
            for (int z = 0; z < Z; ++z)
                y[c] += p[z * split + c];
    }
    store_row<H, 4>(a, row, n, y);
}

template <bool H, int MODE, int TX>
hipError_t run_small(const ProductArgs& a, hipStream_t s)
{
    const int64_t blocks = product_blocks(a.M, group_tiles(a), 8 * TX, a.N, kSmallCols);
    if (!fits(blocks, kSmallThreads))
        return hipErrorInvalidConfiguration;
    if (blocks <= 256)
        small_product<H, MODE, TX, true><<<dim3((unsigned)blocks), dim3(512), 0, s>>>(a);
    else
        small_product<H, MODE, TX, false><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <bool H, int MODE>
hipError_t run_small(const ProductArgs& a, int tokens, hipStream_t s)
{
    return tokens == 8    ? run_small<H, MODE, 1>(a, s)
           : tokens == 16 ? run_small<H, MODE, 2>(a, s)
                          : run_small<H, MODE, 4>(a, s);
}

template <bool H, int NJ, bool DEEP>
void run_down(const DownArgs& a, int adapters_side, hipStream_t s)
{
    const dim3 grid((unsigned)((a.M + 15) / 16), (unsigned)(a.splits * ((a.rank + 16 * NJ - 1) / (16 * NJ))),
                    (unsigned)adapters_side);
    adapter_down<H, NJ, DEEP><<<grid, dim3(DEEP ? 512 : 256), 0, s>>>(a);
}

// Few tokens: 16 ranks per workgroup and a tile's adapters side by side, to fill
// the chip; more: 32 ranks, in workgroups of which a compute unit holds four;
// many: up to 64 ranks at once and no adapters side by side, so that x is read
// once or twice.
template <bool H>
void run_down(const DownArgs& a, hipStream_t s)
{
    const int tiles = (a.M + 15) / 16, blocks = (a.rank + 15) / 16;
    if (tiles * a.splits * blocks <= 96)
        run_down<H, 1, true>(a, 4, s);
    else if (tiles * a.splits < 256)
        a.rank <= 16 ? run_down<H, 1, false>(a, 4, s) : run_down<H, 2, false>(a, 4, s);
    else if (a.rank <= 16)
        run_down<H, 1, false>(a, 1, s);
    else if (a.rank <= 32)
        run_down<H, 2, false>(a, 1, s);
    else
        run_down<H, 4, false>(a, 1, s);
}

template <bool H, int RJ>
void run_token(const ProductArgs& a, const char* A, hipStream_t s)
{
    const unsigned blocks = (unsigned)token_blocks(a.N);
    if (blocks <= 256)
        token_product<H, RJ, true><<<dim3(blocks), dim3(512), 0, s>>>(a, A);
    else
        token_product<H, RJ, false><<<dim3(blocks), dim3(256), 0, s>>>(a, A);
}

template <bool H>
void run_token(const ProductArgs& a, const char* A, hipStream_t s)
{
    if (a.rank <= 16)
        run_token<H, 1>(a, A, s);
    else if (a.rank <= 32)
        run_token<H, 2>(a, A, s);
    else
        run_token<H, 4>(a, A, s);
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

hipError_t launch_token(const ProductArgs& a, int type, const char* A, hipStream_t s)
{
    if (!fits(token_blocks(a.N), 512))
        return hipErrorInvalidConfiguration;
    type == kFp16 ? run_token<true>(a, A, s) : run_token<false>(a, A, s);
    return hipGetLastError();
}

hipError_t launch_adapter_down(const DownArgs& a, int type, hipStream_t s)
{
    if (!fits(down_blocks(a.M), 256))
        return hipErrorInvalidConfiguration;
    type == kFp16 ? run_down<true>(a, s) : run_down<false>(a, s);
    return hipGetLastError();
}

namespace {

template <bool H>
hipError_t run_join(const ProductArgs& a, hipStream_t s)
{
    const int64_t blocks = join_blocks(a.M, a.N);
    if (!fits(blocks, 256))
        return hipErrorInvalidConfiguration;
    const auto kernel = a.splits == 2   ? join<H, 2>
                        : a.splits == 3 ? join<H, 3>
                        : a.splits == 4 ? join<H, 4>
                        : a.splits == 6 ? join<H, 6>
                                        : join<H, 8>;
    kernel<<<dim3((unsigned)blocks), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_join(const ProductArgs& a, int type, hipStream_t s)
{
    if (a.splits != 2 && a.splits != 3 && a.splits != 4 && a.splits != 6 && a.splits != 8)
        return hipErrorInvalidValue;
    return type == kFp16 ? run_join<true>(a, s) : run_join<false>(a, s);
}

}  // namespace hcp
