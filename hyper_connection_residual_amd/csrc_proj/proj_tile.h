// proj_tile.h -- what the LDS-tiled products (proj_tile.hip, proj_wide.hip)
// share: the layout of a K step in LDS, its reads, the adapters' part, the
// stores and the order of the tiles.
//
// Inside LDS a row of a K step is one 128-byte line of 8 chunks; chunk c of row
// r lies at slot c ^ (r & 7).  A 16-byte read serves 16 lanes at a time, but not
// 16 in a row: lanes 0-3 and 12-15 (one chunk of rows 0-3 and 12-15) together
// with 20-27 (the next chunk of rows 4-11).  Over those this swizzle meets every
// bank once; with row bit 3 mixed in as well (right for 16 lanes in a row) half
// of all LDS cycles were bank conflicts.
#pragma once

#include "proj_device.h"

#pragma clang fp contract(off)

namespace hcp {

constexpr int kStep = 64;  // k per step

__device__ __forceinline__ int swizzle(int row) { return row & 7; }

__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)p; }

__device__ __forceinline__ void dma16(gbytes g, char* lds_wave_base)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                     (__attribute__((address_space(3))) void*)lds_wave_base, 16, 0, 0);
}

// COUNT row blocks (16 rows of 128 bytes, 2 KB apart), both halves of the
// step, into v[][AT ..]: the reads and their wait are one block of assembly, so
// that no register is used before its data is there.
template <int COUNT, int AT = 0, int ALL>
__device__ __forceinline__ void read_blocks(uint32_t a0, uint32_t a1, u32x4 (&v)[2][ALL])
{
    static_assert(AT + COUNT <= ALL, "inside v");
    if constexpr (COUNT == 1) {
        asm volatile("ds_read_b128 %0, %2 offset:%4\n\tds_read_b128 %1, %3 offset:%4\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(v[0][AT]), "=&v"(v[1][AT])
                     : "v"(a0), "v"(a1), "n"(AT * 2048)
                     : "memory");
    } else if constexpr (COUNT == 2) {
        asm volatile(
            "ds_read_b128 %0, %4 offset:%6\n\tds_read_b128 %1, %4 offset:%7\n\t"
            "ds_read_b128 %2, %5 offset:%6\n\tds_read_b128 %3, %5 offset:%7\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(v[0][AT]), "=&v"(v[0][AT + 1]), "=&v"(v[1][AT]), "=&v"(v[1][AT + 1])
            : "v"(a0), "v"(a1), "n"(AT * 2048), "n"((AT + 1) * 2048)
            : "memory");
    } else if constexpr (COUNT == 4) {
        static_assert(AT == 0, "the first four");
        asm volatile(
            "ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:2048\n\t"
            "ds_read_b128 %2, %8 offset:4096\n\tds_read_b128 %3, %8 offset:6144\n\t"
            "ds_read_b128 %4, %9\n\tds_read_b128 %5, %9 offset:2048\n\t"
            "ds_read_b128 %6, %9 offset:4096\n\tds_read_b128 %7, %9 offset:6144\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[0][2]), "=&v"(v[0][3]), "=&v"(v[1][0]), "=&v"(v[1][1]),
              "=&v"(v[1][2]), "=&v"(v[1][3])
            : "v"(a0), "v"(a1)
            : "memory");
    } else {
        static_assert(COUNT == 3 || COUNT == 5, "row blocks per read");
        read_blocks<COUNT - 1>(a0, a1, v);
        read_blocks<1, COUNT - 1>(a0, a1, v);
    }
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

// The tokens' adapters, -1 for none, before the product: they wait in LDS for
// its end.
template <int BM, int THREADS>
__device__ __forceinline__ void load_adapters(const ProductArgs& a, const RowTile& t, int* of)
{
    for (int i = threadIdx.x; i < BM; i += THREADS) {
        const int ad = i < t.rows ? a.adapter[t.row0 + i] : -1;
        of[i] = ad >= 0 && ad < a.adapters ? ad : -1;
    }
}

// A B that is not finite everywhere.  The tokens of other adapters, whose v here
// is zeros, must not see it, so its infinities and NaNs are taken out of the
// matrix product (clean says whether there were any) and their products are
// added to their own tokens' results after these have been stored (add_stray).
// What stands in for an infinity is a tiny number of its sign, so that an infinite v
// times it is infinite still, not NaN.
template <bool H, int NJ>
__device__ __forceinline__ bool clean(u32x4 (&w)[NJ])
{
    constexpr uint32_t ones = exponents(H);
    uint32_t any = 0;  // (an exponent of ones and one more reach the bit above)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            any |= (w[j][c] & ones) + (ones & ~(ones << 1));
    const bool odd = __ballot((any & 0x80008000u) != 0) != 0;
    if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            w[j] = stand_ins<H>(w[j]);
    }
    return odd;
}
// A scale that is not finite.  It multiplies the whole sum over the ranks, and is
// none of a matrix product: its sign stands in for it there, and the sum itself is
// added to the results after these have been stored (add_stray).
__device__ __forceinline__ bool is_odd(float scale) { return !(fabsf(scale) < INFINITY); }
__device__ __forceinline__ float finite_scale(float scale) { return is_odd(scale) ? copysignf(1.0f, scale) : scale; }

// The lowest of a tile's adapters above `last`: lane l has those of tokens l, 64 + l, ...
constexpr int kNoAdapter = 1 << 30;
template <int COUNT>
__device__ __forceinline__ int next_adapter(const int (&ad)[COUNT], int last)
{
    int next = kNoAdapter;
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
        next = ad[i] > last ? min(next, ad[i]) : next;
    for (int d = 32; d; d >>= 1)
        next = min(next, __shfl_xor(next, d));
    return __builtin_amdgcn_readfirstlane(next);
}

// The adapters' part: acc[m][j] += scale B v of each token's own adapter, ahead of
// the product itself.  The tile's adapters are taken one after the other (in
// ascending order); for each, scale v's pieces and B go through LDS as one more K
// step, or a few (a step's 8 chunks: see piece_chunks; an fp16 B is cut into its
// pieces on the way).  The steps alternate between the two stages at `lds`, of
// (BM + BN) * 128 bytes each; while one is multiplied the next one is on its way,
// and beside the last one, if it is in the second stage, the product's own first
// (send_first, which sends as many loads).  `row_of(q)`: the output of row q of W in
// the tile, after the tile's first, n_first.  Returns whether stray sums are left, and in `sent` whether the first
// step is on its way.
template <bool H, int BM, int BN, int THREADS, int MI, int NJ, typename RowOf, typename SendFirst>
__device__ __forceinline__ bool add_adapters(const ProductArgs& a, const RowTile& t, char* lds, const int* of,
                                             int token0, int w_row0, int n_first, RowOf row_of, SendFirst send_first, bool& sent,
                                             f32x4_t (&acc)[MI][NJ])
{
    constexpr int PX = BM * 8 / THREADS, PW = BN * 8 / THREADS;  // chunks per thread and step
    constexpr int STAGE = (BM + BN) * 128;
    static_assert(NJ == 4 && MI % 2 == 0 && PX + PW == 8, "reads and waits below");
    static_assert(THREADS / 8 % 8 == 0, "rows of one thread share their swizzle");
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    // this thread's slots: chunk cx of rows row0 + i * THREADS / 8
    const int row0 = threadIdx.x >> 3, cx = threadIdx.x & 7;
    int all[BM / 64], own[PX];  // (read before any load into LDS, on which reads of LDS would wait)
#pragma unroll
    for (int i = 0; i < BM / 64; ++i)
        all[i] = of[64 * i + lane];
#pragma unroll
    for (int i = 0; i < PX; ++i)
        own[i] = of[row0 + i * (THREADS / 8)];
    int now = next_adapter(all, -1);
    sent = false;
    if (now == kNoAdapter)
        return false;
    const int eighths = a.rank >> 3, chunks = piece_chunks(a.rank, H), pitch = piece_bytes(a.rank, H);
    const uint32_t at_x = lds_addr(lds) + (token0 + r) * 128, at_w = lds_addr(lds) + BM * 128 + (w_row0 + r) * 128;
    const uint32_t c0 = 16 * (g ^ swizzle(r)), c1 = 16 * ((g + 4) ^ swizzle(r));
    u32x4 b[H ? PW : 1];
    const gbytes pieces = (gbytes)a.pieces + (int64_t)t.row0 * pitch;
    auto kind_of = [&](int q) {  // q / eighths, below 6
        int kind = 0;
#pragma unroll
        for (int i = 1; i < (H ? 6 : 3); ++i)
            kind += q >= i * eighths;
        return kind;
    };
    auto send = [&](int ad, int q0, int stage) {
        const int q = q0 + (cx ^ swizzle(row0)), k = q < chunks ? 8 * (q - kind_of(q) * eighths) : 0;
        char* const to = lds + stage * STAGE + (threadIdx.x & ~63) * 16;
        const gbytes B = (gbytes)a.B + 2 * (((int64_t)ad * a.N + n_first) * a.rank);
#pragma unroll
        for (int i = 0; i < PW; ++i) {
            // (a row past B: any other, its results are not stored; a chunk past the
            // last: any other, v's is zeros)
            const int n = min(row_of(row0 + i * (THREADS / 8)), a.N - n_first - 1);
            const gbytes p = B + 2u * (unsigned)(__mul24(n, a.rank) + k);
            if constexpr (H)
                b[i] = load16(p);
            else
                dma16(p, to + BM * 128 + i * THREADS * 16);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < PX; ++i) {
            const int row = row0 + i * (THREADS / 8);
            const gbytes p = q < chunks && own[i] == ad ? pieces + (unsigned)(__mul24(row, pitch) + 16 * q) : zeros();
            dma16(p, to + i * THREADS * 16);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    bool odd = false;
    int q0 = 0, stage = (chunks + 7) / 8 & 1;  // (one adapter's last step is in the second stage)
    send(now, 0, stage);
    for (;;) {
        if constexpr (H) {
            const bool second = kind_of(q0 + (cx ^ swizzle(row0))) & 1;
            const uint32_t to = lds_addr(lds) + stage * STAGE + BM * 128 + row0 * 128 + 16 * cx;
#pragma unroll
            for (int i = 0; i < PW; ++i) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    b[i][c] = half_piece(b[i][c], second);
                asm volatile("ds_write_b128 %0, %1 offset:%2" ::"v"(to), "v"(b[i]), "n"(i * THREADS * 16) : "memory");
            }
        }
        int next = now, q1 = q0 + 8;
        if (q1 >= chunks) {
            q1 = 0;
            next = next_adapter(all, now);
        }
        const bool last = next == kNoAdapter;
        sent = last && stage == 1;
        if (!last)
            send(next, q1, stage ^ 1);
        else if (sent)
            send_first();
        // (this step's loads are in, the next one's 8 may be on their way; the waves' stores are seen)
        if (last && !sent)
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        u32x4 w[2][NJ];
        read_blocks<NJ>(at_w + stage * STAGE + c0, at_w + stage * STAGE + c1, w);
        odd = clean<false>(w[0]) || odd;
        odd = clean<false>(w[1]) || odd;
#pragma unroll
        for (int m = 0; m < MI; m += 2) {
            u32x4 x[2][2];
            read_blocks<2>(at_x + stage * STAGE + 2048 * m + c0, at_x + stage * STAGE + 2048 * m + c1, x);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        acc[m + i][j] = mfma<false>(w[h][j], x[h][i], acc[m + i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("s_barrier" ::: "memory");  // (its reads are done)
        __builtin_amdgcn_sched_barrier(0);
        if (last)
            return odd;
        now = next;
        q0 = q1;
        stage ^= 1;
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

// The sum of B v over the ranks for one token and output, one after the other: all
// of them, or those whose weight is an infinity or NaN.
template <bool H, bool PIECES>
__device__ __forceinline__ float rank_sum(const ProductArgs& a, int64_t row, int ad, int n, bool all)
{
    const uint16_t* B = (const uint16_t*)a.B + ((int64_t)ad * a.N + n) * a.rank;
    float sum = 0.0f;
#pragma clang loop unroll(disable)
    for (int k = 0; k < a.rank; ++k) {
        const float b = from16<H>(B[k]);
        if (!all && fabsf(b) < INFINITY)
            continue;
        float v = 0.0f;
        if constexpr (PIECES) {
            const uint16_t* p = (const uint16_t*)(a.pieces + row * piece_bytes(a.rank, H)) + k;
            for (int i = 2; i >= 0; --i)
                v += from16<false>(p[(H ? 2 * i : i) * a.rank]);
        } else {
            for (int z = 0; z < a.v_splits; ++z)
                v += a.v[((int64_t)z * a.M + row) * a.rank + k];
        }
        sum += b * v;
    }
    return sum;
}

// After store_block: the products that clean took out, and those of a scale that is
// not finite, to the results that this lane has stored.
template <bool H, int MI, int NJ, bool PIECES>
__device__ __forceinline__ void add_stray(const ProductArgs& a, const RowTile& t, int token0, int n0)
{
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma clang loop unroll(disable)
    for (int i = 0; i < MI * 4 * NJ; ++i) {
        const int token = token0 + i / (4 * NJ) * 16 + r, n = n0 + g * 4 * NJ + i % (4 * NJ);
        if (token >= t.rows || n >= a.N)
            continue;
        const int64_t row = (int64_t)t.row0 + token;
        const int ad = a.adapter[row];
        if (ad < 0 || ad >= a.adapters)
            continue;
        const float sc = a.scale ? a.scale[ad] : 1.0f;
        // (the pieces are of v times the finite scale)
        const float sum = rank_sum<H, PIECES>(a, row, ad, n, is_odd(sc)) * (!PIECES ? sc : is_odd(sc) ? fabsf(sc) : 1.0f);
        if (fabsf(sum) < INFINITY)
            continue;
        const int64_t at = row * a.ldo + n;
        if (a.out32)
            ((float*)a.out)[at] += sum;
        else
            ((uint16_t*)a.out)[at] = (uint16_t)bits16<H>(from16<H>(((uint16_t*)a.out)[at]) + sum);
    }
}

// The k-th tile in the order the tiles are worked on: the 8 XCDs (workgroup b
// runs on XCD b % 8) each take a contiguous eighth, and inside it groups of
// GROUP row tiles walk the columns together, so that an XCD's L2 holds what
// its workgroups share.
template <int GROUP>
__device__ __forceinline__ bool tile_of(unsigned block, unsigned row_tiles, unsigned col_tiles, int& rt, int& ct)
{
    // (32 bits hold the number of workgroups of any launch)
    const unsigned total = row_tiles * col_tiles;
    const unsigned each = (total + 7) / 8;
    const unsigned id = (block & 7) * each + (block >> 3);
    if ((block >> 3) >= each || id >= total)
        return false;
    const unsigned per = GROUP * col_tiles;
    const unsigned group = id / per, rest = id - group * per;
    const unsigned in_group = min((unsigned)GROUP, row_tiles - group * GROUP);
    ct = rest / in_group;
    rt = group * GROUP + rest - ct * in_group;
    return true;
}

}  // namespace hcp
