// attn_few.hip -- attention of few rows (single tokens, verify windows): tiles of
// 16 NB rows, keys and values straight from memory into registers.
//
// Such a call is bound by reading the cache once: 64 requests' tokens over
// 262000 positions of 4 heads of 128 are 0.54 GB and 2.7 GFLOP.  So nothing is
// staged: a wave takes 32 positions at a time, keys as rows of a matrix
// instruction's first operand, whose product with the queries leaves lane l
// (r = l & 15, g = l >> 4) with row r's scores at positions 4 g + i and 16 + 4 g
// + i: what it needs, as they lie, as the second operand of the product with the
// values.  That one's first operand is values by column, 8 positions a lane: a
// lane loads 8 neighbouring columns of its 8 positions, in whole rows by 16
// lanes, and transposes them in its registers, 32 byte permutations for 8 KB.
// Its keys' registers are free again once the scores are there, its values' after
// the second product: loads of the next 32 positions then start.  The four waves
// of a workgroup take its units in turn and join their sums through LDS.
#include "attn_device.h"

#pragma clang fp contract(off)

namespace hca {
namespace {

constexpr int kUnit = 32, kThreads = 256, kWaves = 4;

// Of D positions' neighbours: column c of each lane's 8 positions, from their rows.
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

// Ones where the numbers are infinities of the sign, or NaN.
template <bool H>
__device__ __forceinline__ u32x4 stray(u32x4 x, bool negative)
{
    constexpr uint32_t inf = H ? 0x7c00u : 0x7f80u, one = H ? 0x3c00u : 0x3f80u;
    const auto is = [&](uint32_t b) {
        const uint32_t m = b & 0x7fffu;
        return m > inf || (m == inf && (b >> 15) == (negative ? 1u : 0u)) ? one : 0u;
    };
#pragma unroll
    for (int c = 0; c < 4; ++c)
        x[c] = is(x[c] & 0xffffu) | is(x[c] >> 16) << 16;
    return x;
}

// FULL: dim is DP.
template <int DP, int NB, bool H, bool FULL>
__global__ __launch_bounds__(kThreads, DP * NB <= 128 ? 2 : 1) void few_rows(AttendArgs a)
{
    constexpr int ROWS = 16 * NB, KK = DP / 32, WORDS = DP / 32, COLS = 2 * WORDS;  // WORDS: of a lane's columns of one row
    constexpr int PITCH = DP + 4;
    constexpr int JOIN = 4 * kWaves * ROWS * PITCH, PLAN = 4 * (kMaxTiles + 1) + 2 * (kMaxSegments + 2);
    __shared__ __align__(16) char lds[JOIN > PLAN ? JOIN : PLAN];
    __shared__ float2 ml[kWaves][ROWS];
    __shared__ int sums[16];

    const int w = (blockIdx.x & 7) * (kWorkers / 8) + (blockIdx.x >> 3);  // neighbours on one XCD
    Start plan;
    int* const at = (int*)lds;
    if (threadIdx.x == 0)
        ((Record*)a.records)[w] = Record{};
    if (!make_plan<ROWS, kUnit, kThreads>(a, w, (uint16_t*)(at + kMaxTiles + 1), [&](int i) -> int& { return at[i]; }, sums, plan))
        return;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;
    const int D = a.cache.dim;
    // (columns that the head does not have: its first ones, and then zeros or left out)
    const int k_at = 16 * g, v_at = FULL || COLS / (DP == 256 ? 2 : 1) * r < D ? (DP == 64 ? 8 : 16) * r : 0;

    walk<ROWS, kUnit>(a, plan, [&](const Segment& seg, int rt, int head, int u0, int u1, bool begins, bool ends, int last) {
        Row rows[NB];
        u32x4 q[NB][KK];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            rows[nb] = row_of(a, seg, head, rt * ROWS + 16 * nb + r);
            const gbytes p = (gbytes)a.q.x + rows[nb].t * a.q.row + rows[nb].h * a.q.head;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                q[nb][kk] = rows[nb].real && (FULL || 8 * g + 32 * kk < D) ? load16(p + 16 * g + 64 * kk) : u32x4{};
        }
        // positions that all rows see, and that any sees
        int all_lo = 0, all_hi = 0x7fffffff;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            if (rows[nb].real) {
                all_lo = max(all_lo, rows[nb].lo);
                all_hi = min(all_hi, rows[nb].hi);
            }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            all_lo = max(all_lo, __shfl_xor(all_lo, d));
            all_hi = min(all_hi, __shfl_xor(all_hi, d));
        }
        all_lo = __builtin_amdgcn_readfirstlane(all_lo);
        all_hi = __builtin_amdgcn_readfirstlane(all_hi);

        f32x4_t o[NB][COLS] = {};
        float m[NB], l[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb] = kLowest;
            l[nb] = 0.0f;
        }
        u32x4 k[2][KK];
        uint32_t v[8][WORDS];
        const auto load_k = [&](const Page& A, const Page& B) {
            const int r0 = min(r, A.last) * A.k_row + k_at, r1 = min(r, B.last) * B.k_row + k_at;
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
                const gbytes from = p.v + (unsigned)(min(4 * g + (e & 3), p.last) * p.v_row + v_at);
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
        const auto pages = [&](int u, int32_t pa, int32_t pb) {
            A = page_of(a, seg, head, u * kUnit, pa);
            B = page_of(a, seg, head, u * kUnit + 16, pb);
        };
        int32_t pa = -1, pb = -1;
        const auto look_up = [&](int u) {
            if (u < u1) {
                pa = page_at(a, seg, u * kUnit);
                pb = page_at(a, seg, u * kUnit + 16);
            }
        };
        int u = u0 + wave;
        if (u < u1) {
            look_up(u);
            pages(u, pa, pb);
            load_k(A, B);
            load_v(A, B);
            look_up(u + kWaves);
        }
        for (; u < u1; u += kWaves) {
            const int j0 = u * kUnit;
            const bool more = u + kWaves < u1;
            if constexpr (!FULL) {
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
                    if (8 * g + 32 * kk >= D)
                        k[0][kk] = k[1][kk] = u32x4{};
            }
            f32x4_t s[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    s[nb][b] = f32x4_t{};
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk)
                        s[nb][b] = hcp::mfma<H>(k[b][kk], q[nb][kk], s[nb][b]);
                }
            if (more) {
                pages(u + kWaves, pa, pb);
                look_up(u + 2 * kWaves);
                load_k(A, B);
            }
            // scores over ln 2
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (a.cap_out != 0.0f) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[nb][b][i] = capped(a, s[nb][b][i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[nb][b][i] *= a.scale;
                    }
                    if (a.slopes) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[nb][b][i] = fmaf(-rows[nb].slope, fabsf(rows[nb].p - (float)(j0 + 16 * b + 4 * g + i)), s[nb][b][i]);
                    }
                }
            const bool some_hidden = j0 < all_lo || j0 + kUnit > all_hi;
            if (some_hidden) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = j0 + 16 * b + 4 * g + i;
                            s[nb][b][i] = j >= rows[nb].lo && j < rows[nb].hi ? s[nb][b][i] : -INFINITY;
                        }
            }
            u32x4 p[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float top = s[nb][0][0];
#pragma unroll
                for (int i = 1; i < 8; ++i)
                    top = fmaxf(top, s[nb][i >> 2][i & 3]);
                top = max32(max16(top));
                const bool past = top > m[nb] + kSlack;
                if (__any(past)) {
                    const float to = past ? top : m[nb], by = exp2_of(m[nb] - to);
                    l[nb] *= by;
#pragma unroll
                    for (int c = 0; c < COLS; ++c)
                        o[nb][c] *= by;
                    m[nb] = to;
                }
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] = exp2_of(s[nb][i >> 2][i & 3] - m[nb]);
                    l[nb] += y[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    p[nb][i] = pack2<H>(y[2 * i], y[2 * i + 1]);
            }
            if (!some_hidden) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    const u32x4 x = column(v, c);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        o[nb][c] = hcp::mfma<H>(x, p[nb], o[nb][c]);
                }
            } else {
                // A value that is no number reaches the rows that see its position alone: it is
                // left out of the product, and infinities and NaN are added where the product
                // of ones in their places with ones for what a row sees is not zero.
                u32x4 sees[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = j0 + 16 * (i >> 1) + 4 * g + 2 * (i & 1);
                        constexpr uint32_t one = H ? 0x3c00u : 0x3f80u;
                        sees[nb][i] = (j >= rows[nb].lo && j < rows[nb].hi ? one : 0u) | (j + 1 >= rows[nb].lo && j + 1 < rows[nb].hi ? one << 16 : 0u);
                    }
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    const u32x4 x = column(v, c), finite = hcp::finite_of<H>(x);
                    const bool odd = (x[0] != finite[0]) | (x[1] != finite[1]) | (x[2] != finite[2]) | (x[3] != finite[3]);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        o[nb][c] = hcp::mfma<H>(finite, p[nb], o[nb][c]);
                    if (__builtin_expect(__any(odd), 0)) {
                        const u32x4 up = stray<H>(x, false), down = stray<H>(x, true);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            const f32x4_t plus = hcp::mfma<H>(up, sees[nb], f32x4_t{}), minus = hcp::mfma<H>(down, sees[nb], f32x4_t{});
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                o[nb][c][i] += (plus[i] > 0.0f ? INFINITY : 0.0f) + (minus[i] > 0.0f ? -INFINITY : 0.0f);
                        }
                    }
                }
            }
            if (more)
                load_v(A, B);
        }

        // The waves' sums meet in LDS.
        float* const mine = (float*)lds + wave * ROWS * PITCH;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const float sum = sum32(sum16(l[nb]));
            if (g == 0)
                ml[wave][16 * nb + r] = float2{m[nb], sum};
            float* const to = mine + (16 * nb + r) * PITCH;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < COLS; c += 4) {
                    constexpr int EACH = DP == 256 ? 8 : COLS;  // neighbouring columns
                    *(f32x4_t*)(to + (c >= EACH ? 128 : 0) + EACH * (4 * g + i) + (c & (EACH - 1))) =
                        f32x4_t{o[nb][c][i], o[nb][c + 1][i], o[nb][c + 2][i], o[nb][c + 3][i]};
                }
        }
        __syncthreads();
        const Target to = target_of<ROWS>(a, w, seg, DP, begins, ends);
        constexpr int PER = DP / 4;  // threads of a row, 4 columns each
#pragma unroll
        for (int i = threadIdx.x; i < ROWS * PER; i += kThreads) {
            const int row = i / PER, c = 4 * (i % PER);
            if (rt * ROWS + row >= seg.n * a.group || c >= D)
                continue;
            float top = ml[0][row].x, sum = 0.0f;
#pragma unroll
            for (int x = 1; x < kWaves; ++x)
                top = fmaxf(top, ml[x][row].x);
            f32x4_t y{};
#pragma unroll
            for (int x = 0; x < kWaves; ++x) {
                const float by = exp2_of(ml[x][row].x - top);
                sum = fmaf(by, ml[x][row].y, sum);
                const f32x4_t part = *(const f32x4_t*)((const float*)lds + (x * ROWS + row) * PITCH + c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = fmaf(by, part[e], y[e]);
            }
            if (to.sums) {
                *(f32x4_t*)(to.sums + (int64_t)row * DP + c) = y;
                if (c == 0)
                    to.ml[row] = float2{top, sum};
            } else {
                const int ri = rt * ROWS + row, t = seg.t0 + ri / a.group, h = head * a.group + ri % a.group;
                const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
                *(u32x2*)(a.out + t * a.out_row + h * a.out_head + 2 * c) =
                    u32x2{pack2<H>(y[0] * by, y[1] * by), pack2<H>(y[2] * by, y[3] * by)};
            }
        }
        if (begins && !ends && threadIdx.x == 0) {
            Record rec{};
            rec.t0 = seg.t0;
            rec.row0 = rt * ROWS;
            rec.rows = min(ROWS, seg.n * a.group - rt * ROWS);
            rec.head = head;
            rec.last = last;
            ((Record*)a.records)[w] = rec;
        }
        __syncthreads();
    });
}

template <int DP, int NB, bool H>
void run(const AttendArgs& a, hipStream_t s)
{
    if (a.cache.dim == DP)
        few_rows<DP, NB, H, true><<<kWorkers, kThreads, 0, s>>>(a);
    else
        few_rows<DP, NB, H, false><<<kWorkers, kThreads, 0, s>>>(a);
}

template <bool H>
void run(const AttendArgs& a, int rows, hipStream_t s)
{
    switch (padded(a.cache.dim)) {
    case 64: rows <= 16 ? run<64, 1, H>(a, s) : rows <= 32 ? run<64, 2, H>(a, s) : run<64, 4, H>(a, s); break;
    case 128: rows <= 16 ? run<128, 1, H>(a, s) : rows <= 32 ? run<128, 2, H>(a, s) : run<128, 4, H>(a, s); break;
    default: rows <= 16 ? run<256, 1, H>(a, s) : run<256, 2, H>(a, s);
    }
}

}  // namespace

hipError_t launch_few(const AttendArgs& a, bool half, int rows, hipStream_t s)
{
    half ? run<true>(a, rows, s) : run<false>(a, rows, s);
    return hipGetLastError();
}

}  // namespace hca
