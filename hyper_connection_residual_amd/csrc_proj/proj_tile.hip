// proj_tile.hip -- products of more tokens: LDS-tiled, a ring of K steps.
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

// The adapters' part of one wave's sums: acc[m][j] += scale B v of each token's
// own adapter.  The wave's adapters are taken one after the other, each in steps
// of 32 ranks whose B and v come straight from memory into registers; scale v
// (rounded to fp32) is the exact sum of three bf16 pieces, and an fp16 B that of
// two.  No other wave is waited for: a tile of a batch of short requests has
// several adapters, and passes through LDS cost it 2.3 us each (333 tokens of 24
// requests, rank 64: 35 us).  `n`: output of this lane's row of every block of W.
// `kept`: 16 bytes of LDS for every lane.
template <bool H, int MI, int NJ>
__device__ __forceinline__ void add_adapters_direct(const ProductArgs& a, const RowTile& t, const int* of, u32x4* kept,
                                                    int token0, const int (&n)[NJ], f32x4_t (&acc)[MI][NJ])
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    int ad[MI];
#pragma unroll
    for (int m = 0; m < MI; ++m)
        ad[m] = of[token0 + 16 * m + r];
    const uint32_t keep_at = lds_addr(kept + lane);
    int k0 = 0, now = -1;
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
                break;
        }
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
        bool finite = true;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if constexpr (H) {
                    const uint32_t both = b[0][j][c];
                    b[0][j][c] = piece(from16<true>(both & 0xffffu), 0) | piece(from16<true>(both >> 16), 0) << 16;
                    b[1][j][c] = piece(from16<true>(both & 0xffffu), 1) | piece(from16<true>(both >> 16), 1) << 16;
                }
                finite = finite && (b[0][j][c] & 0x7f80u) != 0x7f80u && (b[0][j][c] & 0x7f800000u) != 0x7f800000u;
            }
        // A B that is finite everywhere adds zeros to the tokens whose v is not
        // here; else those tokens keep their sums.
        const bool keep = __ballot(!finite) != 0;
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            const bool mine = ad[m] == now;
            if (__ballot(mine)) {
                const float by = mine ? sc : 0.0f;
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
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if (keep)
                        keep_sum(keep_at, acc[m][j]);
#pragma unroll
                    for (int c = 2; c >= 0; --c)
#pragma unroll
                        for (int h = H ? 1 : 0; h >= 0; --h)
                            acc[m][j] = mfma<false>(b[h][j], vp[c], acc[m][j]);
                    if (keep && !mine)
                        restore_sum(keep_at, acc[m][j]);
                }
            }
        }
        k0 += 32;
        if (k0 >= a.rank) {
            k0 = 0;
#pragma unroll
            for (int m = 0; m < MI; ++m)
                ad[m] = ad[m] == now ? -1 : ad[m];
        }
    }
}

template <bool H, int MODE, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN) void tile_product(ProductArgs a)
{
    constexpr int MI = BM / WM / 16, NJ = BN / WN / 16, THREADS = 64 * WM * WN;
    constexpr int LX = BM * 8 / THREADS, LW = BN * 8 / THREADS;  // loads per thread and step
    constexpr int STAGE = (BM + BN) * 128;
    constexpr int OUT = MODE == kGate ? BN / 2 : BN;
    static_assert(LX * THREADS == BM * 8 && LW * THREADS == BN * 8 && NS >= 2, "whole loads");
    static_assert(MODE != kGate || NJ % 2 == 0, "gate and up blocks in pairs");
    __shared__ __align__(128) char lds[NS * STAGE];
    __shared__ int of[MODE == kAdapt ? BM : 1];
    __shared__ u32x4 kept[MODE == kAdapt ? THREADS : 1];

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
    const int s_lo = (int)((int64_t)steps_all * blockIdx.y / a.splits);
    const int steps = (int)((int64_t)steps_all * (blockIdx.y + 1) / a.splits) - s_lo;

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
        if (step >= steps || (s_lo + step + 1) * kStep > a.K) {
            if (step >= steps || (s_lo + step) * kStep + 8 * chunk >= a.K) {
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
            p[i] += 2 * kStep;
        }
    };
    f32x4_t acc[MI][NJ] = {};
#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
        load(s);
    const uint32_t x_at = lds_addr(lds) + (token0 + r) * 128;
    const uint32_t w_at = lds_addr(lds) + BM * 128 + (wn * NJ * 16 + r) * 128;
    const uint32_t c0 = 16 * (g ^ swizzle(r)), c1 = 16 * ((g + 4) ^ swizzle(r));
    uint32_t stage = 0;  // the stage that is read next
    for (int s = 0; s < steps; ++s) {
        // this step's loads are in (the later steps' may be on their way), and
        // every wave is done with the stage that is loaded next
        wait_barrier<(NS - 2) * (LX + LW)>();
        load(s + NS - 1);
        u32x4 w[2][NJ], x[2][MI];
        read_blocks<NJ>(w_at + stage + c0, w_at + stage + c1, w);
        read_blocks<MI>(x_at + stage + c0, x_at + stage + c1, x);
        stage = stage + STAGE == NS * STAGE ? 0 : stage + STAGE;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < MI; ++m)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[m][j] = mfma<H>(w[h][j], x[h][m], acc[m][j]);
    }
    // (the zero loads past the last step land before the workgroup's LDS goes)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if constexpr (MODE == kAdapt) {
        if (blockIdx.y == 0) {
            int n[NJ], up;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                w_row<NJ, false>(16 * j + r, n[j], up);
                n[j] += n0;
            }
            add_adapters_direct<H, MI, NJ>(a, t, of, kept + wave * 64, token0, n, acc);
        }
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
    if (a.splits == 1) {
        store_block<H, MODE, MI, NJ>(a, t, token0, n0, acc);
    } else if constexpr (MODE != kGate) {
        ProductArgs q = a;
        q.out = (char*)(a.part + (int64_t)blockIdx.y * a.M * a.N);
        q.ldo = a.N;
        q.out32 = 1;
        q.vec = a.N % 4 == 0;
        store_block<H, MODE, MI, NJ>(q, t, token0, n0, acc);
    }
}

template <bool H, int MODE, int BM, int BN, int NS>
hipError_t run(const ProductArgs& a, hipStream_t s)
{
    constexpr int OUT = MODE == kGate ? BN / 2 : BN;
    const int64_t rows = ((int64_t)a.M + BM - 1) / BM + (a.offsets ? (a.E < a.M ? a.E : a.M) : 0);
    const int64_t tiles = (rows * ((a.N + OUT - 1) / OUT) + 7) / 8 * 8;
    if (!fits(tiles * a.splits, 256))
        return hipErrorInvalidConfiguration;
    tile_product<H, MODE, BM, BN, 2, 2, NS><<<dim3((unsigned)tiles, (unsigned)a.splits), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <bool H, int MODE>
hipError_t run(const ProductArgs& a, int tokens, hipStream_t s)
{
    return tokens == 128 ? run<H, MODE, 128, 128, 2>(a, s) : run<H, MODE, 64, 128, 3>(a, s);
}

}  // namespace

hipError_t launch_tile(const ProductArgs& a, int type, int mode, int tokens, hipStream_t s)
{
    if (type == kFp16)
        return mode == kPlain  ? run<true, kPlain>(a, tokens, s)
               : mode == kGate ? run<true, kGate>(a, tokens, s)
                               : run<true, kAdapt>(a, tokens, s);
    return mode == kPlain  ? run<false, kPlain>(a, tokens, s)
           : mode == kGate ? run<false, kGate>(a, tokens, s)
                           : run<false, kAdapt>(a, tokens, s);
}

}  // namespace hcp
