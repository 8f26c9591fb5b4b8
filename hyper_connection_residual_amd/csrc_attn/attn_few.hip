// attn_few.hip -- attention of few rows (single tokens; verify windows of wide heads): tiles
// of 16 or 32 rows, keys and values straight from memory into registers.
//
// Such a call is bound by reading the cache once: 64 requests' tokens over
// 262000 positions of 4 heads of 128 are 0.54 GB and 2.7 GFLOP.  So nothing is
// staged: a wave takes 16 rows and 32 positions at a time, keys as rows of a matrix
// instruction's first operand, whose product with the queries leaves lane l
// (r = l & 15, g = l >> 4) with row r's scores at positions 4 g + i and 16 + 4 g
// + i: what it needs, as they lie, as the second operand of the product with the
// values.  That one's first operand is values by column, 8 positions a lane: a
// lane loads 8 neighbouring columns of its 8 positions, in whole rows by 16
// lanes, and transposes them in its registers, 32 byte permutations for 8 KB.
// Numerators enter it in two pieces of 16 bits each, since the matrix cores have the
// time: results then differ from those of fp32 numerators by a relative 0.00003 to 0.00009
// (with one piece 0.001 to 0.0022 in bf16, next to 0.0017 of the outputs' own rounding).
// With the join, 64 requests' tokens take 114.5 us for 113.8, windows of wide heads 57.5 for 56.4.
// Its keys' registers are free again once the scores are there, its values' after
// the second product: loads of the next 32 positions then start.  A workgroup's
// four waves take its units in turn and join their sums through LDS; with 32
// rows, two waves take the same unit at about the same time, other rows each, so that
// one finds it in the caches.  Those 64 requests take 108 us, 5.0 TB/s; one token over 5000
// positions 11, most of it the way to the first product.
#include "attn_device.h"

#pragma clang fp contract(off)

namespace hca {
namespace {

constexpr int kUnit = kFewUnit, kThreads = 256, kWaves = 4;

// Of 8 positions' neighbouring columns, column c.
template <int WORDS>
__device__ __forceinline__ u32x4 column(const uint32_t (&v)[8][WORDS], int c)
{
    const uint32_t pick = c & 1 ? 0x07060302u : 0x05040100u;
    u32x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        y[e] = __builtin_amdgcn_perm(v[2 * e + 1][c >> 1], v[2 * e][c >> 1], pick);
    return y;
}

// FULL: dim is DP.
template <int DP, bool H, bool FULL>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void few_rows(AttendArgs)
{
    constexpr int KK = DP / 32, WORDS = DP / 32, COLS = 2 * WORDS;  // WORDS: of a lane's columns of one row
    constexpr int PITCH = DP + 4;
    constexpr int JOIN = 4 * kWaves * 16 * PITCH, PLAN = 4 * (kMaxTiles + 1) + 2 * (kMaxSegments + 2);
    __shared__ __align__(16) char lds[JOIN > PLAN ? JOIN : PLAN];
    __shared__ float2 ml[kWaves][16];
    __shared__ int sums[16];

    Start plan;
    int w;
    {
        Args& a = args();
        w = (blockIdx.x & 7) * (a.workers >> 3) + (blockIdx.x >> 3);  // neighbours on one XCD
        int* const at = (int*)lds;
        if (threadIdx.x == 0)
            ((Record*)a.records)[w] = Record{};
        if (!make_plan<kUnit, kThreads>(a, w, (uint16_t*)(at + kMaxTiles + 1), [&](int i) -> int& { return at[i]; }, sums, plan))
            return;
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    Walk way = walk_from(plan);
    Item item;
    while (next_item<kUnit>(args(), plan, way, item)) {
        const Segment& seg = item.g;
        const int rt = item.rt, head = item.head, u0 = item.u0, u1 = item.u1;
        Args& a = args();
        const int D = a.cache.dim;
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));  // (what is made of it is made for each item, not kept from item to item)
        const int r = lane & 15, g = lane >> 4;
        // (columns that the head does not have: its first ones, times queries of zero or for no one)
        const int k_at = 16 * g, v_at = FULL || COLS / (DP == 256 ? 2 : 1) * r < D ? (DP == 64 ? 8 : 16) * r : 0;
        const int shares = a.rows >> 4, turns = kWaves / shares;  // waves of one unit; units at a time
        const int block = wave & (shares - 1);                    // this wave's rows
        const Row row = row_of(a, seg, head, rt * a.rows + 16 * block + r);
        u32x4 q[KK];
        {
            const gbytes p = (gbytes)a.q.x + row.t * a.q.row + row.h * a.q.head;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {  // (from row or column 0 instead: a load under a condition is waited for by itself)
                const bool there = FULL || 8 * g + 32 * kk < D;
                const u32x4 x = load16(p + (there ? 16 * g + 64 * kk : 0)) ^ a.q_sign;
                q[kk] = row.real && there ? x : u32x4{};
            }
        }
        // positions that all rows see
        const int all_lo = __builtin_amdgcn_readfirstlane(most_of<16>(row.real ? row.lo : 0));
        const int all_hi = __builtin_amdgcn_readfirstlane(least_of<16>(row.real ? row.hi : 0x7fffffff));

        f32x4_t o[COLS] = {};
        float m = kLowest, l = 0.0f;
        uint32_t odd = 0;
        u32x4 k[2][KK];
        uint32_t v[8][WORDS];
        const Stream str = stream_of(a, seg, head);
        const float scale = a.scale, cap_in = a.cap_in, cap_out = a.cap_out;
        const bool slopes = a.slopes != nullptr;
        const auto load_k = [&](const Page& A, const Page& B) {
            const int r0 = __umul24(min(r, A.last), A.k_row) + k_at, r1 = __umul24(min(r, B.last), B.k_row) + k_at;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const bool there = FULL || 8 * g + 32 * kk < D;
                k[0][kk] = load16(A.k + (unsigned)(r0 + (FULL ? 64 * kk : there ? 64 * kk : -k_at)));
                k[1][kk] = load16(B.k + (unsigned)(r1 + (FULL ? 64 * kk : there ? 64 * kk : -k_at)));
            }
        };
        const auto load_v = [&](const Page& A, const Page& B) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const Page& p = e < 4 ? A : B;
                const gbytes from = p.v + (unsigned)(__umul24(min(4 * g + (e & 3), p.last), p.v_row) + v_at);
                if constexpr (DP == 64) {
                    const u32x2 x = load8(from);
                    v[e][0] = x[0];
                    v[e][1] = x[1];
                } else {
#pragma unroll
                    for (int c = 0; c < WORDS; c += 4) {
                        const u32x4 x = load16(from + (c && (FULL || 128 + 8 * r < D) ? 256 : 0));
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[e][c + i] = x[i];
                    }
                }
            }
        };
        Page A, B;
        int32_t pa = -1, pb = -1;
        const auto pages = [&](int u) {
            A = page_of(str, u * kUnit, pa);
            B = page_of(str, u * kUnit + 16, pb);
        };
        const auto look_up = [&](int u) {
            if (u < u1) {
                pa = page_at(str, u * kUnit);
                pb = page_at(str, u * kUnit + 16);
            }
        };
        int u = u0 + wave / shares;
        if (u < u1) {
            look_up(u);
            pages(u);
            load_k(A, B);
            load_v(A, B);
            look_up(u + turns);
        }
        for (; u < u1; u += turns) {
            const int j0 = u * kUnit;
            const bool more = u + turns < u1;
            f32x4_t s[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                s[b] = f32x4_t{};
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
                    s[b] = hcp::mfma<H>(k[b][kk], q[kk], s[b]);
            }
            if (more) {
                pages(u + turns);
                look_up(u + 2 * turns);
                load_k(A, B);
            }
            // scores over ln 2
            if (cap_out > kLargeCap) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[i >> 2][i & 3] = capped<true>(s[i >> 2][i & 3], cap_in, cap_out);
            } else if (cap_out != 0.0f) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[i >> 2][i & 3] = capped<false>(s[i >> 2][i & 3], cap_in, cap_out);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[i >> 2][i & 3] *= scale;
            }
            if (slopes) {
                const float far = (float)(row.p - (j0 + 4 * g));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[i >> 2][i & 3] = fmaf(-row.slope, fabsf(far - (float)(16 * (i >> 2) + (i & 3))), s[i >> 2][i & 3]);
            }
            const bool some_hidden = j0 < all_lo || j0 + kUnit > all_hi;
            if (some_hidden) {
                const unsigned past_lo = j0 + 4 * g - row.lo, span = row.hi - row.lo;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    s[i >> 2][i & 3] = past_lo + (unsigned)(16 * (i >> 2) + (i & 3)) < span ? s[i >> 2][i & 3] : -INFINITY;
            }
            float top = s[0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i)
                top = fmaxf(top, s[i >> 2][i & 3]);
            top = max32(max16(top));
            const bool past = top - m > kMost<H>;
            if (__any(past)) {
                const float to = past ? reference_of<H>(top) : m, by = weight_of(m - to);
                l *= by;
#pragma unroll
                for (int c = 0; c < COLS; ++c)
                    o[c] *= by;
                m = to;
            }
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] = exp2_of(s[i >> 2][i & 3] - m);
                l += y[i];
            }
            u32x4 p, rest;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = pack2<H>(y[2 * i], y[2 * i + 1]);
                rest[i] = rest2<H>(y[2 * i], y[2 * i + 1], p[i]);
            }
            // A value that is no number, where a row does not see it, is left out: it belongs to the rows that do (see below).  Where all
            // do, it stays in the first piece's product alone: the second's, or nothing, times an infinity is NaN.
            if (__builtin_expect(!some_hidden && !__any(some_odd<H>(v)), 1)) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    const u32x4 x = column(v, c);
                    o[c] = hcp::mfma<H>(x, rest, hcp::mfma<H>(x, p, o[c]));
                }
            } else {
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    const u32x4 x = column(v, c), finite = hcp::finite_of<H>(x);
                    if (some_hidden)
                        odd |= (x[0] ^ finite[0]) | (x[1] ^ finite[1]) | (x[2] ^ finite[2]) | (x[3] ^ finite[3]);
                    o[c] = hcp::mfma<H>(finite, rest, hcp::mfma<H>(some_hidden ? finite : x, p, o[c]));
                }
            }
            if (more)
                load_v(A, B);
        }
        // The waves' sums meet in LDS.
        {
            const float sum = sum32(sum16(l));
            if (g == 0)
                ml[wave][r] = float2{m, sum};
            float* const to = (float*)lds + (wave * 16 + r) * PITCH;
            constexpr int EACH = DP == 256 ? 8 : COLS;  // neighbouring columns
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < COLS; c += 4)
                    *(f32x4_t*)(to + (c >= EACH ? 128 : 0) + EACH * (4 * g + i) + (c & (EACH - 1))) =
                        f32x4_t{o[c][i], o[c + 1][i], o[c + 2][i], o[c + 3][i]};
            // Infinities and NaN among values that some row of the wave does not see: added to the
            // rows that do.
            if (__builtin_expect(__any(odd != 0), 0)) {
                const unsigned span = row.hi - row.lo;
                for (int col = 4 * g; col < D; col += 16) {
                    f32x4_t add{};
                    for (u = u0 + wave / shares; u < u1; u += turns)
                        for (int j0 = u * kUnit; j0 < (u + 1) * kUnit; j0 += 16) {
                            if ((j0 & ~31) >= all_lo && (j0 | 31) < all_hi)
                                continue;
                            const Page at = page_of(str, j0, page_at(str, j0));
                            for (int j = j0; j < min(j0 + 16, str.L); ++j) {
                                const u32x2 x = load8(at.v + (unsigned)((j - j0) * at.v_row + 2 * col));
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    add[e] += odd_part<H>(x[e >> 1] >> 16 * (e & 1), (unsigned)(j - row.lo) < span);
                            }
                        }
                    *(f32x4_t*)(to + col) += add;
                }
            }
        }
        __syncthreads();
        Args& b = args();
        const Target to = target_of(b, w, item, DP);
        constexpr int PER = DP / 4;  // threads of a row, 4 columns each
        for (int i = threadIdx.x; i < b.rows * PER; i += kThreads) {
            const int in = i / PER, c = 4 * (i % PER), ri = rt * b.rows + in;
            if (ri >= seg.n * b.group || c >= D)
                continue;
            const int from = in >> 4, at = in & 15;  // the first of the row's waves, `shares` apart
            float top = ml[from][at].x, sum = 0.0f;
            for (int x = from + shares; x < kWaves; x += shares)
                top = fmaxf(top, ml[x][at].x);
            f32x4_t y{};
            for (int x = from; x < kWaves; x += shares) {
                const float by = weight_of(ml[x][at].x - top);
                sum = fmaf(by, ml[x][at].y, sum);
                const f32x4_t part = *(const f32x4_t*)((const float*)lds + (x * 16 + at) * PITCH + c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = fmaf(by, part[e], y[e]);
            }
            if (to.sums) {
                *(f32x4_t*)(to.sums + (int64_t)in * DP + c) = y;
                if (c == 0)
                    to.ml[in] = float2{top, sum};
            } else {
                const int i_ = (int)((unsigned)ri / (unsigned)b.group), t = seg.t0 + i_, h = head * b.group + ri - i_ * b.group;
                const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
                *(u32x2*)(b.out + t * b.out_row + h * b.out_head + 2 * c) =
                    u32x2{pack2<H>(y[0] * by, y[1] * by), pack2<H>(y[2] * by, y[3] * by)};
            }
        }
        if (item.begins && !item.ends && threadIdx.x == 0)
            leave_record(b, w, item);
        __syncthreads();
    }
}

template <int DP, bool H>
void run(const AttendArgs& a, hipStream_t s)
{
    if (a.cache.dim == DP)
        few_rows<DP, H, true><<<a.workers, kThreads, 0, s>>>(a);
    else
        few_rows<DP, H, false><<<a.workers, kThreads, 0, s>>>(a);
}

template <bool H>
void run(const AttendArgs& a, hipStream_t s)
{
    switch (padded(a.cache.dim)) {
    case 64: run<64, H>(a, s); break;
    case 128: run<128, H>(a, s); break;
    default: run<256, H>(a, s);
    }
}

}  // namespace

hipError_t launch_few(const AttendArgs& a, bool half, hipStream_t s)
{
    half ? run<true>(a, s) : run<false>(a, s);
    return hipGetLastError();
}

}  // namespace hca
