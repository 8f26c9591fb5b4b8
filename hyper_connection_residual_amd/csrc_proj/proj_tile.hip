// proj_tile.hip -- products of more tokens: LDS-tiled, a ring of K steps.
//
// What bounds such products is the way from the L2s to LDS, a tile's weights and
// tokens being read again by every other tile of its row and column, and a
// workgroup's start and end: 333 tokens, 10240 -> 2560 in 4 splits, move 460 MB in
// 41 us (139 MB from and to memory, matrix cores 26 % busy); 1806 rows of 32 experts,
// gated 2560 -> 1023, take 79 us (368 MB from and to memory, 4.7 TB/s).
//
// A workgroup of 4 waves computes BM tokens x BN rows of W.  Each K step of 64
// (one 128-byte line of every row) goes straight from memory into one stage of
// a ring in LDS (16 bytes a lane), NS - 1 steps ahead of its use.  Inside a
// stage chunk c of row r lies at slot c ^ swizzle(r), so that the 16 lanes that
// read one chunk of 16 rows hit different banks.
#include "proj_tile.h"

#pragma clang fp contract(off)

namespace hcp {
namespace {

// The reads of one step's operands and the products of another's, in one block of
// assembly that ends with the reads' wait, and with the wait states that the
// last product needs before other instructions use its sums.  (Dependent matrix
// instructions wait for each other by themselves.)
template <bool H>
__device__ __forceinline__ void read_multiply(uint32_t w0, uint32_t w1, uint32_t x0, uint32_t x1, const u32x4 (&w)[2][4],
                                              const u32x4 (&x)[2][2], u32x4 (&wn)[2][4], u32x4 (&xn)[2][2],
                                              f32x4_t (&acc)[2][4])
{
#define HCP_READS \
    "ds_read_b128 %[n0], %[w0]\n\tds_read_b128 %[n1], %[w0] offset:2048\n\tds_read_b128 %[n2], %[w0] offset:4096\n\t" \
    "ds_read_b128 %[n3], %[w0] offset:6144\n\tds_read_b128 %[y0], %[x0]\n\tds_read_b128 %[y1], %[x0] offset:2048\n\t" \
    "ds_read_b128 %[n4], %[w1]\n\tds_read_b128 %[n5], %[w1] offset:2048\n\tds_read_b128 %[n6], %[w1] offset:4096\n\t" \
    "ds_read_b128 %[n7], %[w1] offset:6144\n\tds_read_b128 %[y2], %[x1]\n\tds_read_b128 %[y3], %[x1] offset:2048\n\t"
#define HCP_M(OP, C, W, X) OP " %[" C "], %[" W "], %[" X "], %[" C "]\n\t"
#define HCP_PRODUCTS(OP) \
    HCP_M(OP, "c0", "v0", "u0") HCP_M(OP, "c1", "v1", "u0") HCP_M(OP, "c2", "v2", "u0") HCP_M(OP, "c3", "v3", "u0") \
    HCP_M(OP, "c4", "v0", "u1") HCP_M(OP, "c5", "v1", "u1") HCP_M(OP, "c6", "v2", "u1") HCP_M(OP, "c7", "v3", "u1") \
    HCP_M(OP, "c0", "v4", "u2") HCP_M(OP, "c1", "v5", "u2") HCP_M(OP, "c2", "v6", "u2") HCP_M(OP, "c3", "v7", "u2") \
    HCP_M(OP, "c4", "v4", "u3") HCP_M(OP, "c5", "v5", "u3") HCP_M(OP, "c6", "v6", "u3") HCP_M(OP, "c7", "v7", "u3") \
    "s_waitcnt lgkmcnt(0)\n\ts_nop 11"
#define HCP_OPERANDS \
    : [n0] "=&v"(wn[0][0]), [n1] "=&v"(wn[0][1]), [n2] "=&v"(wn[0][2]), [n3] "=&v"(wn[0][3]), [n4] "=&v"(wn[1][0]), \
      [n5] "=&v"(wn[1][1]), [n6] "=&v"(wn[1][2]), [n7] "=&v"(wn[1][3]), [y0] "=&v"(xn[0][0]), [y1] "=&v"(xn[0][1]), \
      [y2] "=&v"(xn[1][0]), [y3] "=&v"(xn[1][1]), [c0] "+v"(acc[0][0]), [c1] "+v"(acc[0][1]), [c2] "+v"(acc[0][2]), \
      [c3] "+v"(acc[0][3]), [c4] "+v"(acc[1][0]), [c5] "+v"(acc[1][1]), [c6] "+v"(acc[1][2]), [c7] "+v"(acc[1][3]) \
    : [w0] "v"(w0), [w1] "v"(w1), [x0] "v"(x0), [x1] "v"(x1), [v0] "v"(w[0][0]), [v1] "v"(w[0][1]), [v2] "v"(w[0][2]), \
      [v3] "v"(w[0][3]), [v4] "v"(w[1][0]), [v5] "v"(w[1][1]), [v6] "v"(w[1][2]), [v7] "v"(w[1][3]), [u0] "v"(x[0][0]), \
      [u1] "v"(x[0][1]), [u2] "v"(x[1][0]), [u3] "v"(x[1][1]) \
    : "memory"
    if constexpr (H)
        asm volatile(HCP_READS HCP_PRODUCTS("v_mfma_f32_16x16x32_f16") HCP_OPERANDS);
    else
        asm volatile(HCP_READS HCP_PRODUCTS("v_mfma_f32_16x16x32_bf16") HCP_OPERANDS);
#undef HCP_READS
#undef HCP_PRODUCTS
#undef HCP_OPERANDS
}

template <bool H>
__device__ __forceinline__ void read_multiply(uint32_t w0, uint32_t w1, uint32_t x0, uint32_t x1, const u32x4 (&w)[2][4],
                                              const u32x4 (&x)[2][4], u32x4 (&wn)[2][4], u32x4 (&xn)[2][4],
                                              f32x4_t (&acc)[4][4])
{
    read_blocks<4>(w0, w1, wn);
    read_blocks<4>(x0, x1, xn);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[m][j] = mfma<H>(w[h][j], x[h][m], acc[m][j]);
}

// The adapters' part of one wave's sums: acc[m][j] += scale B v of each token's
// own adapter.  The wave's adapters are taken one after the other, each in steps
// of 32 ranks whose B and v come straight from memory into registers; scale v
// (rounded to fp32) is the exact sum of three bf16 pieces, and an fp16 B that of
// two.  No other wave is waited for: a tile of a batch of short requests has
// several adapters, and passes through LDS cost it 2.3 us each (333 tokens of 24
// requests, rank 64: 35 us; so, with the splits' turns, some 10).  The splits of K take these steps in turn, too.
// `n`: output of this lane's row of every block of W.  Returns whether stray sums
// are left (then each split adds them: infinities and NaNs alone).
template <bool H, int MI, int NJ>
__device__ __forceinline__ bool add_adapters_direct(const ProductArgs& a, const RowTile& t, const int* of, int token0,
                                                    const int (&n)[NJ], int split, f32x4_t (&acc)[MI][NJ])
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    int ad[MI];
#pragma unroll
    for (int m = 0; m < MI; ++m)
        ad[m] = of[token0 + 16 * m + r];
    int k0 = 0, now = -1, turn = split;
    bool odd = false;
    const auto next = [&] {
        k0 += 32;
        if (k0 >= a.rank) {
            k0 = 0;
#pragma unroll
            for (int m = 0; m < MI; ++m)
                ad[m] = ad[m] == now ? -1 : ad[m];
        }
    };
    for (;;) {
        if (k0 == 0) {  // the first adapter that is left
            now = -1;
#pragma unroll
            for (int m = MI - 1; m >= 0; --m) {
                const unsigned long long left = __ballot(ad[m] >= 0);
                if (left)
                    now = __builtin_amdgcn_readlane(ad[m], __builtin_ctzll(left));
            }
            if (now < 0)
                return odd;
        }
        if (turn) {
            turn = turn + 1 == a.splits ? 0 : turn + 1;
            next();
            continue;
        }
        turn = a.splits > 1;
        const int k = k0 + 8 * g;
        u32x4 b[H ? 2 : 1][NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            b[0][j] = load16(k < a.rank ? (gbytes)a.B + 2 * (((int64_t)now * a.N + min(n[j], a.N - 1)) * a.rank + k) : zeros());
        f32x4_t v[MI][kSplitsTile][2];
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            const bool mine = ad[m] == now && k < a.rank;
#pragma unroll
            for (int z = 0; z < kSplitsTile; ++z) {
                const bool in = mine && z < a.v_splits;
                const gbytes p = in ? (gbytes)a.v + 4 * (((int64_t)z * a.M + t.row0 + token0 + 16 * m + r) * a.rank + k) : zeros();
                v[m][z][0] = __builtin_bit_cast(f32x4_t, load16(p));
                v[m][z][1] = __builtin_bit_cast(f32x4_t, load16(in ? p + 16 : p));
            }
        }
        const float sc = a.scale ? a.scale[now] : 1.0f;
        __builtin_amdgcn_sched_barrier(0);
        odd = is_odd(sc) || odd;
        odd = clean<H>(b[0]) || odd;
        if constexpr (H)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t both = b[0][j][c];
                    b[0][j][c] = half_piece(both, false);
                    b[1][j][c] = half_piece(both, true);
                }
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            const bool mine = ad[m] == now;
            if (__ballot(mine)) {
                const float by = mine ? finite_scale(sc) : 0.0f;
#pragma unroll
                for (int z = 1; z < kSplitsTile; ++z) {
                    v[m][0][0] += v[m][z][0];
                    v[m][0][1] += v[m][z][1];
                }
                v[m][0][0] *= by;
                v[m][0][1] *= by;
                u32x4 vp[3];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int c = 0; c < 3; ++c)
                        vp[c][q] = piece(v[m][0][q >> 1][2 * (q & 1)], c) | piece(v[m][0][q >> 1][2 * (q & 1) + 1], c) << 16;
                // (the second piece of an fp16 weight is mostly zero, and 0 times inf
                // would turn a sum that its first piece makes infinite into a NaN)
#pragma unroll
                for (int c = 2; c >= 0; --c)
#pragma unroll
                    for (int h = H ? 1 : 0; h >= 0; --h)
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
                            acc[m][j] = mfma<false>(b[h][j], h && c == 0 ? finite_of<false>(vp[0]) : vp[c], acc[m][j]);
            }
        }
        next();
    }
}

// (Registers for two workgroups on a compute unit: left to itself the compiler
// takes 264 for 128 tokens with fp16 adapters, one workgroup, 2000 x 2560 -> 2500
// 83 us instead of 54.)
template <bool H, int MODE, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN, 2) void tile_product(ProductArgs a)
{
    constexpr int MI = BM / WM / 16, NJ = BN / WN / 16, THREADS = 64 * WM * WN;
    constexpr int LX = BM * 8 / THREADS, LW = BN * 8 / THREADS;  // loads per thread and step
    constexpr int STAGE = (BM + BN) * 128;
    constexpr int OUT = MODE == kGate ? BN / 2 : BN;
    static_assert(LX * THREADS == BM * 8 && LW * THREADS == BN * 8 && NS >= 2, "whole loads");
    static_assert(MODE != kGate || NJ % 2 == 0, "gate and up blocks in pairs");
    __shared__ __align__(128) char lds[NS * STAGE];
    __shared__ int of[MODE == kAdapt ? BM : 1];

    int rt, ct;
    RowTile t;
    if (!tile_of<8>(blockIdx.x, count_tiles<BM>(a.offsets, a.E, a.M), (a.N + OUT - 1) / OUT, rt, ct) ||
        !find_tile<BM>(a.offsets, a.E, a.M, rt, t))
        return;
    if constexpr (MODE == kAdapt)
        load_adapters<BM, THREADS>(a, t, of);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4, wm = wave / WN, wn = wave % WN;
    const int n0 = ct * OUT + wn * (OUT / WN), token0 = wm * MI * 16;
    const int64_t row_bytes = 2 * (int64_t)a.K;
    const gbytes W = (gbytes)a.W + (int64_t)t.e * (MODE == kGate ? 2 : 1) * a.N * row_bytes;

    const int steps_all = (a.K + kStep - 1) / kStep;
    // (the splits take the steps in turn: together they read whole rows)
    const int s_lo = blockIdx.y, steps = (steps_all - s_lo + a.splits - 1) / a.splits;

    // this thread's pieces of a stage: chunk `chunk` of rows slot_row + i * THREADS / 8.
    // Rows past the tile or past W are given a row that exists: their results
    // are not stored.
    const int slot_row = threadIdx.x >> 3;
    const int chunk = (threadIdx.x & 7) ^ swizzle(slot_row);  // (the same for every i)
    static_assert(THREADS / 8 % 16 == 0, "rows of one thread share their swizzle");
    gbytes p[LX + LW];
#pragma unroll
    for (int i = 0; i < LX; ++i) {
        const gbytes row = x_row(a, t, slot_row + i * (THREADS / 8));
        p[i] = (row ? row : (gbytes)a.x) + 2 * (s_lo * kStep + 8 * chunk);
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
        const int row = slot_row + i * (THREADS / 8);
        int n, up;
        w_row<NJ, MODE == kGate>(row % (16 * NJ), n, up);
        n += ct * OUT + row / (16 * NJ) * (OUT / WN);
        n = n < a.N ? n : ct * OUT;
        p[LX + i] = W + ((int64_t)up * a.N + n) * row_bytes + 2 * (s_lo * kStep + 8 * chunk);
    }
    int fill = 0;  // the stage that is loaded next
    auto load = [&](int step) {
        // pieces past K, and steps past the last one, are zeros
        const int k0 = (s_lo + step * a.splits) * kStep;
        if (step >= steps || k0 + kStep > a.K) {
            if (step >= steps || k0 + 8 * chunk >= a.K) {
#pragma unroll
                for (int i = 0; i < LX + LW; ++i)
                    p[i] = zeros();
            }
        }
        char* stage = lds + fill * STAGE + wave * 1024;
        fill = fill + 1 == NS ? 0 : fill + 1;
#pragma unroll
        for (int i = 0; i < LX + LW; ++i) {
            dma16(p[i], stage + i * THREADS * 16);
            p[i] += 2 * kStep * a.splits;
        }
    };
    f32x4_t acc[MI][NJ] = {};
#pragma unroll
    for (int s = 0; s < NS; ++s)
        load(s);
    const uint32_t x_at = lds_addr(lds) + (token0 + r) * 128;
    const uint32_t w_at = lds_addr(lds) + BM * 128 + (wn * NJ * 16 + r) * 128;
    const uint32_t c0 = 16 * (g ^ swizzle(r)), c1 = 16 * ((g + 4) ^ swizzle(r));
    u32x4 wa[2][NJ], xa[2][MI], wb[2][NJ], xb[2][MI];
    wait_barrier<(NS - 1) * (LX + LW)>();
    read_blocks<NJ>(w_at + c0, w_at + c1, wa);
    read_blocks<MI>(x_at + c0, x_at + c1, xa);
    uint32_t stage = NS == 1 ? 0 : STAGE;  // the stage that is read next
    // One step: the operands of the next one are read while this one's are
    // multiplied.
    auto step = [&](int s, const u32x4 (&w)[2][NJ], const u32x4 (&x)[2][MI], u32x4 (&w_next)[2][NJ], u32x4 (&x_next)[2][MI]) {
        // the next step's loads are in (the later steps' may be on their way),
        // and every wave is done with the stage that is loaded now: this step's
        wait_barrier<(NS - 2) * (LX + LW)>();
        load(s + NS);
        read_multiply<H>(w_at + stage + c0, w_at + stage + c1, x_at + stage + c0, x_at + stage + c1, w, x, w_next, x_next, acc);
        stage = stage + STAGE == NS * STAGE ? 0 : stage + STAGE;
    };
    for (int s = 0; s < steps; s += 2) {  // (a step past the last one multiplies zeros)
        step(s, wa, xa, wb, xb);
        step(s + 1, wb, xb, wa, xa);
    }
    // (the zero loads past the last step land before the workgroup's LDS goes)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    bool odd = false;
    if constexpr (MODE == kAdapt) {
        int n[NJ], up;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            w_row<NJ, false>(16 * j + r, n[j], up);
            n[j] += n0;
        }
        // (always true; as code that may be passed by, it keeps its addresses out of the
        // main loop's registers, of which 128 tokens would spill 7)
        if (a.rank)
            odd = add_adapters_direct<H, MI, NJ>(a, t, of, token0, n, blockIdx.y, acc);
    }
    if (a.rows) {  // a row that x does not have is zeros
#pragma unroll
        for (int m = 0; m < MI; ++m)
            if (!x_row(a, t, token0 + 16 * m + r)) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[m][j] = f32x4_t{};
            }
    }
    ProductArgs to = a;
    if (a.splits > 1) {
        to.out = (char*)(a.part + (int64_t)blockIdx.y * a.M * a.N);
        to.ldo = a.N;
        to.out32 = 1;
    }
    store_block<H, MODE, MI, NJ>(to, t, token0, n0, acc);
    if constexpr (MODE == kAdapt)
        if (__builtin_expect(odd, 0))
            add_stray<H, MI, NJ, false>(to, t, token0, n0);
}

template <bool H, int MODE, int BM, int BN, int NS>
hipError_t run(const ProductArgs& a, hipStream_t s)
{
    constexpr int OUT = MODE == kGate ? BN / 2 : BN;
    static_assert(BN == kTileCols, "part_fits of the API");
    const int64_t tiles = product_blocks(a.M, group_tiles(a), BM, a.N, OUT);
    if (!fits(tiles * a.splits, kTileThreads))
        return hipErrorInvalidConfiguration;
    tile_product<H, MODE, BM, BN, 2, 2, NS><<<dim3((unsigned)tiles, (unsigned)a.splits), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <bool H, int MODE>
hipError_t run(const ProductArgs& a, int tokens, int stages, hipStream_t s)
{
    if (tokens == 128)
        return run<H, MODE, 128, 128, 2>(a, s);
    if constexpr (MODE != kAdapt)
        if (stages == 2)
            return run<H, MODE, 64, 128, 2>(a, s);
    return run<H, MODE, 64, 128, 3>(a, s);
}

}  // namespace

hipError_t launch_tile(const ProductArgs& a, int type, int mode, int tokens, int stages, hipStream_t s)
{
    if (type == kFp16)
        return mode == kPlain  ? run<true, kPlain>(a, tokens, stages, s)
               : mode == kGate ? run<true, kGate>(a, tokens, stages, s)
                               : run<true, kAdapt>(a, tokens, stages, s);
    return mode == kPlain  ? run<false, kPlain>(a, tokens, stages, s)
           : mode == kGate ? run<false, kGate>(a, tokens, stages, s)
                           : run<false, kAdapt>(a, tokens, stages, s);
}

}  // namespace hcp
