// proj_wide.hip -- products of many tokens: 256 tokens x 256 rows of W per
// workgroup, 8 waves of 128 x 64 each, K steps of 64.
//
// Such a product is bound by the matrix cores, and those by how they are fed:
// the 128 x 64 of a wave reads 24 KB of LDS per step for 64 matrix
// instructions.  The step is cut into four phases of 16 instructions (64
// tokens x 32 rows), and the two waves of a SIMD run half a phase apart: while
// one's matrix instructions run, the other reads the operands of its next phase
// and sends a quarter of the step after next on its way, straight from memory
// into LDS.  (8192 x 10240 x 2560 takes 315 us so, 1.36 PFLOP/s, and 356 us with the
// waves in step; a raised priority for the wave that multiplies costs 1 to 2 %.)  Two
// stages of 64 KB hold the steps; each is four units (W0, X0, W1,
// X1: what one phase reads), and a unit is overwritten by the same unit of the
// step after next in the phase after its last read, seven phases before it is
// read again.
//
//   phase   reads        sends       multiplies
//   0       X0(s)        W0(s + 2)   X0 W0
//   1       W1(s)        X0(s + 2)   X0 W1
//   2       X1(s)        W1(s + 2)   X1 W1
//   3       W0(s + 1)    X1(s + 2)   X1 W0
#include "proj_tile.h"

#pragma clang fp contract(off)

namespace hcp {
namespace {

constexpr int kUnit = 128 * 128;  // bytes: 128 rows of one step
constexpr int kStage = 4 * kUnit;
constexpr int kThreads = 512;
enum { kW0 = 0, kX0 = 1, kW1 = 2, kX1 = 3 };  // units, in the order they are sent

template <int VM>
__device__ __forceinline__ void landed_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(VM) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ void barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Loads that may be in flight at the end of a phase's reads, with `left` steps
// to go (2: or more): those of the last six phases.
constexpr int in_flight(int left, int phase)
{
    const int n = (left == 1 ? 10 : 2) - 2 * phase;
    return left == 2 ? 12 : n > 0 ? n : 0;
}

template <bool H, int M0, int J0>
__device__ __forceinline__ void multiply(bool any, f32x4_t (&acc)[8][4], const u32x4 (&x)[2][4], const u32x4 (&w)[2][2])
{
    if (!any)  // (no token of the tile: the last tile of a group)
        return;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[M0 + m][J0 + j] = mfma<H>(w[h][j], x[h][m], acc[M0 + m][J0 + j]);
}

// GROUPS: rows in groups, whose last tiles may be mostly empty: blocks of 64
// tokens without any skip their products (64 experts, 8192 rows: 187 us against
// 206; without groups the test costs the product 2 %).
// SPLITS of K: this workgroup's is blockIdx.y (8192 x 2560 x 10240 without any takes 4 %
// longer with the code for them).
template <bool H, int MODE, bool GROUPS, bool SPLITS>
__global__ __launch_bounds__(kThreads, 2) void wide_product(ProductArgs a)
{
    constexpr int OUT = MODE == kGate ? 128 : 256;
    __shared__ __align__(128) char lds[2 * kStage];
    __shared__ int of[MODE == kAdapt ? 256 : 1];

    int rt, ct;
    RowTile t;
    if (!tile_of<8>(blockIdx.x, count_tiles<256>(a.offsets, a.E, a.M), (a.N + OUT - 1) / OUT, rt, ct) ||
        !find_tile<256>(a.offsets, a.E, a.M, rt, t))
        return;
    if constexpr (MODE == kAdapt)
        load_adapters<256, kThreads>(a, t, of);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4, wm = wave >> 2, wn = wave & 3;
    const int n0 = ct * OUT + wn * (OUT / 4), token0 = wm * 128;
    const int64_t row_bytes = 2 * (int64_t)a.K;
    // this split's part of K, in pairs of steps (the two stages)
    const int pairs = (a.K + 2 * kStep - 1) / (2 * kStep), z = SPLITS ? blockIdx.y : 0;
    const int pair_lo = SPLITS ? (int)((int64_t)pairs * z / a.splits) : 0;
    const int steps = 2 * ((SPLITS ? (int)((int64_t)pairs * (z + 1) / a.splits) : pairs) - pair_lo);
    const int left = a.K - 2 * kStep * pair_lo, offset = 4 * kStep * pair_lo + 16 * ((threadIdx.x & 7) ^ swizzle(threadIdx.x >> 3));
    const gbytes W = (gbytes)a.W + (int64_t)t.e * (MODE == kGate ? 2 : 1) * a.N * row_bytes;

    // this thread's pieces of a unit: rows tid / 8 and 64 + tid / 8, one chunk.
    // Rows past the tile or past W are given the tile's first row: their
    // results are not stored.
    const int slot_row = threadIdx.x >> 3;
    const int chunk = (threadIdx.x & 7) ^ swizzle(slot_row);
    gbytes p[4][2];
    const gbytes first = a.rows ? nullptr : (gbytes)a.x + (int64_t)t.row0 * a.ldx;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 64 * i + slot_row;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const gbytes x = x_row(a, t, (row >> 6) * 128 + h * 64 + (row & 63));
            p[h ? kX1 : kX0][i] = (x ? x : first ? first : (gbytes)a.x) + offset;
            int n, up;
            w_row<4, MODE == kGate>(h * 32 + (row & 31), n, up);
            n += ct * OUT + (row >> 5) * (OUT / 4);
            n = n < a.N ? n : ct * OUT;
            p[h ? kW1 : kW0][i] = W + ((int64_t)up * a.N + n) * row_bytes + offset;
        }
    }
    char* const lds_wave = lds + wave * 1024;
    auto send = [&](int unit, int stage) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            dma16(p[unit][i], lds_wave + stage * kStage + unit * kUnit + i * (kUnit / 2));
            p[unit][i] += 2 * kStep;
        }
    };
    // pieces that lie past K are zeros
    auto before = [&](int step) {
        if ((step + 1) * kStep > left && step * kStep + 8 * chunk >= left) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                p[u][0] = p[u][1] = zeros();
        }
    };

    const uint32_t base = lds_addr(lds);
    const uint32_t c0 = 16 * (g ^ swizzle(r)), c1 = 16 * ((g + 4) ^ swizzle(r));
    const uint32_t x_at = base + (wm * 64 + r) * 128, w_at = base + (wn * 32 + r) * 128;
    auto read_x = [&](int unit, int stage, u32x4 (&v)[2][4]) {
        const uint32_t at = x_at + stage * kStage + unit * kUnit;
        read_blocks<4>(at + c0, at + c1, v);
    };
    auto read_w = [&](int unit, int stage, u32x4 (&v)[2][2]) {
        const uint32_t at = w_at + stage * kStage + unit * kUnit;
        read_blocks<2>(at + c0, at + c1, v);
    };

    const bool any0 = !GROUPS || token0 < t.rows, any1 = !GROUPS || token0 + 64 < t.rows;
    f32x4_t acc[8][4] = {};
    u32x4 x[2][4], wa[2][2], wb[2][2];

    // LEFT: steps after this one, 2 or more as 2.  w0 holds this step's W0; w1,
    // free until phase 1 and again from phase 3 on, then holds the next one's.
    auto step = [&](auto left, int stage, u32x4 (&w0)[2][2], u32x4 (&w1)[2][2]) {
        constexpr int LEFT = decltype(left)::value;
        read_x(kX0, stage, x);
        if constexpr (LEFT == 2)
            send(kW0, stage);
        landed_barrier<in_flight(LEFT, 0)>();
        multiply<H, 0, 0>(any0, acc, x, w0);
        barrier();
        read_w(kW1, stage, w1);
        if constexpr (LEFT == 2)
            send(kX0, stage);
        landed_barrier<in_flight(LEFT, 1)>();
        multiply<H, 0, 2>(any0, acc, x, w1);
        barrier();
        read_x(kX1, stage, x);
        if constexpr (LEFT == 2)
            send(kW1, stage);
        landed_barrier<in_flight(LEFT, 2)>();
        multiply<H, 4, 2>(any1, acc, x, w1);
        barrier();
        if constexpr (LEFT > 0)
            read_w(kW0, stage ^ 1, w1);
        if constexpr (LEFT == 2)
            send(kX1, stage);
        landed_barrier<in_flight(LEFT, 3)>();
        multiply<H, 4, 0>(any1, acc, x, w0);
        barrier();
    };
    using Two = std::integral_constant<int, 2>;
    using One = std::integral_constant<int, 1>;
    using None = std::integral_constant<int, 0>;

    auto send_first = [&] {
        before(0);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            send(u, 0);
    };
    bool odd = false, sent = false;
    if constexpr (MODE == kAdapt) {
        // the adapters' part comes first, while nothing else is in the sums (after
        // the product it is 41 registers too many, and 8192 x 10240 x 2560 takes
        // 371 us instead of 355)
        __syncthreads();  // (the tile's adapters are in LDS)
        const auto row_of = [&](int q) {
            int n, up;
            w_row<4, false>(q & 63, n, up);
            return n + (q >> 6) * 64;
        };
        if (z == 0)
            odd = add_adapters<H, 256, 256, kThreads, 8, 4>(a, t, lds, of, token0, wn * 64, ct * OUT, row_of, send_first, sent, acc);
    }
    if (!sent)
        send_first();
    before(1);
#pragma unroll
    for (int u = 0; u < 4; ++u)
        send(u, 1);
    landed_barrier<12>();
    read_w(kW0, 0, wa);
    barrier();
    if (wave >= 4)
        barrier();  // the second wave of every SIMD runs half a phase behind
    for (int s = 2; s < steps; s += 2) {
        before(s);
        step(Two{}, 0, wa, wb);
        before(s + 1);
        step(Two{}, 1, wb, wa);
    }
    step(One{}, 0, wa, wb);
    step(None{}, 1, wb, wa);
    if (wave < 4)
        barrier();

    if (a.rows) {  // a row that x does not have is zeros
#pragma unroll
        for (int m = 0; m < 8; ++m)
            if (!x_row(a, t, token0 + 16 * m + r)) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[m][j] = f32x4_t{};
            }
    }
    ProductArgs to = a;
    if constexpr (SPLITS) {
        to.out = (char*)(a.part + (int64_t)z * a.M * a.N);
        to.ldo = a.N;
        to.out32 = 1;
    }
    // (whether a scale of the wave's tokens is not finite: on its way while the results
    // are stored; asked for in every step of the adapters it cost 5 % at rank 128, once
    // ahead of them up to 1 %)
    float scale[2] = {1.0f, 1.0f};
    if constexpr (MODE == kAdapt)
        if (a.scale && z == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                scale[i] = a.scale[max(of[token0 + 64 * i + lane], 0)];
        }
    store_block<H, MODE, 8, 4>(to, t, token0, n0, acc);
    if constexpr (MODE == kAdapt)
        if (__builtin_expect(odd || __ballot(is_odd(scale[0]) || is_odd(scale[1])) != 0, 0))
            add_stray<H, 8, 4, true>(to, t, token0, n0);
}

template <bool H, int MODE>
hipError_t run(const ProductArgs& a, hipStream_t s)
{
    constexpr int OUT = MODE == kGate ? 128 : 256;
    static_assert(kThreads == kWideThreads && (MODE == kGate || OUT == kWideCols), "part_fits of the API");
    const int64_t blocks = product_blocks(a.M, group_tiles(a), 256, a.N, OUT);
    if (!fits(blocks * a.splits, kThreads))
        return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks, (unsigned)a.splits);
    if (a.offsets) {
        if constexpr (MODE != kAdapt)
            wide_product<H, MODE, true, false><<<grid, kThreads, 0, s>>>(a);
    } else if constexpr (MODE != kGate) {
        if (a.splits > 1)
            wide_product<H, MODE, false, true><<<grid, kThreads, 0, s>>>(a);
        else
            wide_product<H, MODE, false, false><<<grid, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_wide(const ProductArgs& a, int type, int mode, hipStream_t s)
{
    if (type == kFp16)
        return mode == kPlain ? run<true, kPlain>(a, s) : mode == kGate ? run<true, kGate>(a, s) : run<true, kAdapt>(a, s);
    return mode == kPlain ? run<false, kPlain>(a, s) : mode == kGate ? run<false, kGate>(a, s) : run<false, kAdapt>(a, s);
}

}  // namespace hcp
