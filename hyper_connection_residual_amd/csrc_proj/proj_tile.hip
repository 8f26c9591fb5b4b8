// proj_tile.hip -- products of more tokens: LDS-tiled, a ring of K steps.
//
// A workgroup of 4 waves computes BM tokens x BN rows of W.  Each K step of 64
// (one 128-byte line of every row) goes straight from memory into one stage of
// a ring in LDS (16 bytes a lane), NS - 1 steps ahead of its use.  Inside a
// stage chunk c of row r lies at slot c ^ swizzle(r), so that the 16 lanes that
// read one chunk of 16 rows hit different banks.
#include "proj_device.h"

#pragma clang fp contract(off)

namespace hcp {
namespace {

constexpr int kStep = 64;  // k per step

__device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)p; }

__device__ __forceinline__ void dma16(gbytes g, char* lds_wave_base)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                     (__attribute__((address_space(3))) void*)lds_wave_base, 16, 0, 0);
}

// COUNT row blocks (16 rows of 128 bytes, 2 KB apart), both halves of the
// step: the reads and their wait are one block of assembly, so that no
// register is used before its data is there.
template <int COUNT>
__device__ __forceinline__ void read_blocks(uint32_t a0, uint32_t a1, u32x4 (&v)[2][COUNT])
{
    static_assert(COUNT == 1 || COUNT == 2 || COUNT == 4, "row blocks per read");
    if constexpr (COUNT == 1)
        asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(v[0][0]), "=&v"(v[1][0])
                     : "v"(a0), "v"(a1)
                     : "memory");
    else if constexpr (COUNT == 2)
        asm volatile(
            "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:2048\n\t"
            "ds_read_b128 %2, %5\n\tds_read_b128 %3, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[1][0]), "=&v"(v[1][1])
            : "v"(a0), "v"(a1)
            : "memory");
    else
        asm volatile(
            "ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:2048\n\t"
            "ds_read_b128 %2, %8 offset:4096\n\tds_read_b128 %3, %8 offset:6144\n\t"
            "ds_read_b128 %4, %9\n\tds_read_b128 %5, %9 offset:2048\n\t"
            "ds_read_b128 %6, %9 offset:4096\n\tds_read_b128 %7, %9 offset:6144\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[0][2]), "=&v"(v[0][3]), "=&v"(v[1][0]), "=&v"(v[1][1]),
              "=&v"(v[1][2]), "=&v"(v[1][3])
            : "v"(a0), "v"(a1)
            : "memory");
}

template <int VM>
__device__ __forceinline__ void wait_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(VM) : "memory");
}

// Output n (gated: output f, and which product) of row `q` (0 .. 16 NJ - 1) of
// a wave's W rows: lane group g of the product holds rows 4 g + i of every
// block, and is given NJ * 4 neighbouring outputs, so that a lane stores them
// as whole 16-byte pieces and the four groups a whole line.
template <int NJ, bool GATE>
__device__ __forceinline__ void w_row(int q, int& n, int& up)
{
    const int j = q >> 4, g = (q >> 2) & 3, i = q & 3;
    up = GATE ? j & 1 : 0;
    n = GATE ? g * 2 * NJ + (j >> 1) * 4 + i : g * 4 * NJ + j * 4 + i;
}

// The adapters' part: acc[m][j] += scale B v of each token's own adapter.  The
// wave's distinct adapters are taken one after the other; a token's column
// takes only its own adapter's sum.  v is the exact sum of three bf16 pieces;
// fp16 weights are the exact sum of two.
template <bool H, int MI, int NJ>
__device__ __forceinline__ void add_adapters(const ProductArgs& a, const RowTile& t, int token0, const int (&n)[NJ],
                                             f32x4_t (&acc)[MI][NJ])
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    int ad[MI];
#pragma unroll
    for (int m = 0; m < MI; ++m) {
        const int token = token0 + 16 * m + r;
        ad[m] = token < t.rows ? a.adapter[t.row0 + token] : -1;
        if (ad[m] < 0 || ad[m] >= a.adapters)
            ad[m] = -1;
    }
    const int64_t split = (int64_t)a.M * a.rank;
    for (;;) {
        int now = -1;
#pragma unroll
        for (int m = MI - 1; m >= 0; --m) {
            const unsigned long long left = __ballot(ad[m] >= 0);
            if (left)
                now = __builtin_amdgcn_readlane(ad[m], __builtin_ctzll(left));
        }
        if (now < 0)
            return;
        const float sc = a.scale ? a.scale[now] : 1.0f;
        for (int k0 = 0; k0 < a.rank; k0 += 32) {
            const int k = k0 + 8 * g;
            u32x4 b[NJ], b2[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                b[j] = load16(n[j] < a.N && k < a.rank
                                  ? (gbytes)a.B + 2 * (((int64_t)now * a.N + n[j]) * a.rank + k)
                                  : zeros());
            if constexpr (H) {
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t p[2][3];
                        pieces(from16<true>(b[j][q] & 0xffffu), p[0]);
                        pieces(from16<true>(b[j][q] >> 16), p[1]);
                        b[j][q] = p[0][0] | p[1][0] << 16;
                        b2[j][q] = p[0][1] | p[1][1] << 16;
                    }
            }
#pragma unroll
            for (int m = 0; m < MI; ++m) {
                const bool mine = ad[m] == now;
                if (__ballot(mine)) {
                    f32x4_t v[2] = {};
                    if (mine && k < a.rank) {
                        const float* p = a.v + ((int64_t)t.row0 + token0 + 16 * m + r) * a.rank + k;
                        for (int z = 0; z < a.v_splits; ++z, p += split) {
                            v[0] += *(const f32x4_t*)p;
                            v[1] += *(const f32x4_t*)(p + 4);
                        }
                    }
                    u32x4 vp[3];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t lo[3], hi[3];
                        pieces(v[q >> 1][2 * (q & 1)], lo);
                        pieces(v[q >> 1][2 * (q & 1) + 1], hi);
#pragma unroll
                        for (int c = 0; c < 3; ++c)
                            vp[c][q] = lo[c] | hi[c] << 16;
                    }
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        f32x4_t s = {};
#pragma unroll
                        for (int c = 2; c >= 0; --c) {
                            s = mfma<false>(b[j], vp[c], s);
                            if constexpr (H)
                                s = mfma<false>(b2[j], vp[c], s);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[m][j][i] = mine ? fmaf(sc, s[i], acc[m][j][i]) : acc[m][j][i];
                    }
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MI; ++m)
            ad[m] = ad[m] == now ? -1 : ad[m];
    }
}

// Results of one wave: MI token blocks, NJ blocks of W rows, from output n0.
template <bool H, int MODE, int MI, int NJ>
__device__ __forceinline__ void store_block(const ProductArgs& a, const RowTile& t, int token0, int n0,
                                            const f32x4_t (&acc)[MI][NJ])
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int m = 0; m < MI; ++m) {
        const int token = token0 + 16 * m + r;
        constexpr int COUNT = MODE == kGate ? 2 * NJ : 4 * NJ;
        float y[COUNT];
#pragma unroll
        for (int c = 0; c < COUNT; ++c)
            y[c] = MODE == kGate ? gated(acc[m][c / 4 * 2][c % 4], acc[m][c / 4 * 2 + 1][c % 4])
                                 : acc[m][c / 4][c % 4];
        if (token < t.rows)
            store_row<H, COUNT>(a, (int64_t)t.row0 + token, n0 + g * COUNT, y);
    }
}

// The k-th tile in the order the tiles are worked on: the 8 XCDs (workgroup b
// runs on XCD b % 8) each take a contiguous eighth, and inside it groups of
// GROUP row tiles walk the columns together, so that an XCD's L2 holds what
// its workgroups share.
template <int GROUP>
__device__ __forceinline__ bool tile_of(int block, int row_tiles, int col_tiles, int& rt, int& ct)
{
    const int64_t total = (int64_t)row_tiles * col_tiles;
    const int64_t each = (total + 7) / 8;
    const int64_t id = (block & 7) * each + (block >> 3);
    if ((block >> 3) >= each || id >= total)
        return false;
    const int64_t per = (int64_t)GROUP * col_tiles;
    const int first = (int)(id / per) * GROUP;
    const int in_group = min(GROUP, row_tiles - first);
    const int rest = (int)(id % per);
    rt = first + rest % in_group;
    ct = rest / in_group;
    return true;
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

    int rt, ct;
    RowTile t;
    if (!tile_of<8>(blockIdx.x, count_tiles<BM>(a.offsets, a.E, a.M), (a.N + OUT - 1) / OUT, rt, ct) ||
        !find_tile<BM>(a.offsets, a.E, a.M, rt, t))
        return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const int n0 = ct * OUT + wn * (OUT / WN), token0 = wm * MI * 16;
    const int64_t row_bytes = 2 * (int64_t)a.K;
    const gbytes W = (gbytes)a.W + (int64_t)t.e * (MODE == kGate ? 2 : 1) * a.N * row_bytes;

    const int steps_all = (a.K + kStep - 1) / kStep;
    const int s_lo = (int)((int64_t)steps_all * blockIdx.y / a.splits);
    const int steps = (int)((int64_t)steps_all * (blockIdx.y + 1) / a.splits) - s_lo;

    // this thread's pieces of a stage: 16-byte slot i * THREADS + tid is chunk
    // (slot & 7) ^ swizzle(row) of row slot >> 3
    gbytes p[LX + LW];
    int k_of[LX + LW];  // its first k in step 0; past every K for a row that does not exist
#pragma unroll
    for (int i = 0; i < LX + LW; ++i) {
        const int slot = (i < LX ? i : i - LX) * THREADS + threadIdx.x;
        const int row = slot >> 3, c = (slot & 7) ^ swizzle(row);
        gbytes base;
        if (i < LX) {
            base = x_row(a, t, row);
        } else {
            int n, up;
            w_row<NJ, MODE == kGate>(row % (16 * NJ), n, up);
            n += ct * OUT + row / (16 * NJ) * (OUT / WN);
            base = n < a.N ? W + ((int64_t)up * a.N + n) * row_bytes : nullptr;
        }
        k_of[i] = base ? 8 * c : 1 << 30;
        p[i] = base + 16 * c;
    }
    auto load = [&](int step) {
        char* stage = lds + (step % NS) * STAGE + wave * 1024;
        const int k0 = (s_lo + step) * kStep;
#pragma unroll
        for (int i = 0; i < LX + LW; ++i) {
            const bool in = step < steps && k_of[i] + k0 < a.K;
            dma16(in ? p[i] + 2 * (int64_t)k0 : zeros(), stage + (i < LX ? i * THREADS * 16
                                                                         : BM * 128 + (i - LX) * THREADS * 16));
        }
    };
    f32x4_t acc[MI][NJ] = {};
#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
        load(s);
    const uint32_t x_at = lds_addr(lds) + (token0 + r) * 128;
    const uint32_t w_at = lds_addr(lds) + BM * 128 + (wn * NJ * 16 + r) * 128;
    const uint32_t c0 = 16 * (g ^ swizzle(r)), c1 = 16 * ((g + 4) ^ swizzle(r));
    for (int s = 0; s < steps; ++s) {
        // this step's loads are in (the later steps' may be on their way), and
        // every wave is done with the stage that is loaded next
        wait_barrier<(NS - 2) * (LX + LW)>();
        load(s + NS - 1);
        const uint32_t stage = (s % NS) * STAGE;
        u32x4 w[2][NJ], x[2][MI];
        read_blocks<NJ>(w_at + stage + c0, w_at + stage + c1, w);
        read_blocks<MI>(x_at + stage + c0, x_at + stage + c1, x);
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
            add_adapters<H, MI, NJ>(a, t, token0, n, acc);
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

template <bool H, int MODE>
hipError_t run(const ProductArgs& a, hipStream_t s)
{
    constexpr int BM = 64, BN = 128;
    constexpr int OUT = MODE == kGate ? BN / 2 : BN;
    const int64_t rows = ((int64_t)a.M + BM - 1) / BM + (a.offsets ? (a.E < a.M ? a.E : a.M) : 0);
    const int64_t tiles = rows * ((a.N + OUT - 1) / OUT);
    if (!fits((tiles + 7) / 8 * 8 * a.splits, 256))
        return hipErrorInvalidConfiguration;
    tile_product<H, MODE, BM, BN, 2, 2, 3><<<dim3((unsigned)((tiles + 7) / 8 * 8), (unsigned)a.splits), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tile(const ProductArgs& a, int type, int mode, hipStream_t s)
{
    if (type == kFp16)
        return mode == kPlain ? run<true, kPlain>(a, s) : mode == kGate ? run<true, kGate>(a, s) : run<true, kAdapt>(a, s);
    return mode == kPlain ? run<false, kPlain>(a, s) : mode == kGate ? run<false, kGate>(a, s) : run<false, kAdapt>(a, s);
}

}  // namespace hcp
