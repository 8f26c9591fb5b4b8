// attn_rotate.hip -- heads normed and turned by their positions, and appended to
// the cache.
//
// Bound by memory: every head is read once and written once.  A head takes the
// next power of two of dim / 8 lanes, 8 columns a lane: the columns of 4 pairs, or 8
// that pass.  A wave takes one token and several of its heads at a time, so the
// angles' sines and cosines (in 64 bits up to their fraction of a turn: 20
// operations a pair) are computed once for all of the token's heads.  8192 tokens of 40
// heads of 64 columns take 16.3 us, of 28 heads of 128 into a cache 22.9: 5.1 TB/s.
#include "attn_device.h"

#pragma clang fp contract(off)

namespace hca {
namespace {

constexpr int kThreads = kRotateThreads;

// Lane c of a head's: its two runs of 4 columns begin at lo and hi.
struct Columns {
    int lo, hi;
    bool turns;
};

__device__ __forceinline__ Columns columns_of(const RotateArgs& a, int c)
{
    const int eighths = a.rotated / 8;
    if (c >= eighths || a.interleaved)
        return Columns{8 * c, 8 * c + 4, c < eighths};
    return Columns{4 * c, a.rotated / 2 + 4 * c, true};
}

template <bool H>
__device__ __forceinline__ void unpack4(u32x2 x, float* y)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        y[2 * i] = from16<H>(x[i] & 0xffffu);
        y[2 * i + 1] = from16<H>(x[i] >> 16);
    }
}

// Sine and cosine of position * frequency: the product is exact in 64 bits but for
// a last bit, and so is its fraction of a turn to 2^-53 of the turns; the fraction's
// in 32 bits.
__device__ __forceinline__ void turn_of(int position, float frequency, float& sine, float& cosine)
{
    const double turns = (double)position * (double)frequency * 0.15915494309189535;
    const float part = (float)(turns - __builtin_rint(turns));
    sincospif(2.0f * part, &sine, &cosine);
}

// LANES: of a head.  APPEND: heads are the queries', then the keys', then the values'.  PAST: results pass the caches.
template <bool H, int LANES, bool APPEND, bool PAST>
__global__ __launch_bounds__(kThreads) void rotate(RotateArgs a)
{
    constexpr int EACH = 64 / LANES;  // heads of a wave at a time
    const int lane = threadIdx.x & 63, c = lane % LANES, in = lane / LANES;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int heads = a.q_heads + (APPEND ? 2 * a.cache.heads : 0);
    const int turns = (heads + EACH - 1) / EACH, chunks = (turns + a.chunk - 1) / a.chunk;
    const int64_t id = (int64_t)blockIdx.x * (kThreads / 64) + wave;
    const int t = __builtin_amdgcn_readfirstlane((int)(id / chunks)), first = __builtin_amdgcn_readfirstlane((int)(id % chunks) * a.chunk);
    if (t >= a.T)
        return;
    // the token's request and position, and where its key and value go
    int position = 0;
    char *to_k = nullptr, *to_v = nullptr;
    if constexpr (APPEND) {
        const ints off = scalars(a.batch.offsets);
        int b = 0;
        for (int i = 0; i < a.batch.requests; i += 64) {
            const bool before = i + lane < a.batch.requests && a.batch.offsets[min(i + lane, a.batch.requests - 1) + 1] <= t;
            const int n = __popcll(__ballot(before));
            b += n;
            if (n < 64)
                break;
        }
        if (b >= a.batch.requests || t < off[b])
            return;  // (of no request)
        const int end = min(off[b + 1], a.T), at = max(scalars(a.batch.lengths)[b], 0) - (end - t);
        position = at;
        if (at >= 0 && (at >> a.cache.shift) < a.batch.width) {
            const int page = scalars(a.batch.table + b * a.batch.table_row)[at >> a.cache.shift];
            if ((int64_t)(uint32_t)page < a.cache.pages) {
                const int64_t row = at & ((1 << a.cache.shift) - 1);
                to_k = a.cache.k + page * a.cache.k_page + row * a.cache.k_row;
                to_v = a.cache.v + page * a.cache.v_page + row * a.cache.v_row;
            }
        }
    }
    if (a.positions)
        position = scalars(a.positions)[t];
    const bool there = c < a.dim / 8;
    const Columns at = columns_of(a, there ? c : 0);
    float sine[4], cosine[4];
    if (a.frequencies && at.turns) {
        const f32x4_t f = *(const hcp::f32x4_at4*)(a.frequencies + 4 * (there ? c : 0));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            turn_of(position, f[i], sine[i], cosine[i]);
    }
    for (int turn = first; turn < min(first + a.chunk, turns); ++turn) {
        const int head = turn * EACH + in;
        const bool is_q = !APPEND || head < a.q_heads, is_v = APPEND && head >= a.q_heads + a.cache.heads;
        const int h = is_q ? head : head - a.q_heads - (is_v ? a.cache.heads : 0);
        const HeadsArgs& from = is_q ? a.q : is_v ? a.v : a.k;
        char* to = is_q ? a.out + t * a.out_row + h * a.out_head
                   : is_v ? (to_v ? to_v + (int64_t)h * a.cache.v_head : nullptr)
                          : (to_k ? to_k + (int64_t)h * a.cache.k_head : nullptr);
        const bool live = there && head < heads && to;
        u32x2 lo{}, hi{};
        if (live) {
            const gbytes x = (gbytes)from.x + t * from.row + h * from.head;
            lo = load8(x + 2 * at.lo);
            hi = load8(x + 2 * at.hi);
        }
        const float* const weight = is_q ? a.q_weight : a.k_weight;
        if (!is_v) {
            float x[8];
            unpack4<H>(lo, x);
            unpack4<H>(hi, x + 4);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum = fmaf(x[i], x[i], sum);
#pragma unroll
            for (int d = 1; d < LANES; d <<= 1)
                sum += __shfl_xor(sum, d);
            if (weight) {
                const float by = 1.0f / sqrtf(sum / (float)a.dim + a.eps);
                const f32x4_t w0 = *(const hcp::f32x4_at4*)(weight + at.lo), w1 = *(const hcp::f32x4_at4*)(weight + at.hi);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = x[i] * by * w0[i];
                    x[4 + i] = x[4 + i] * by * w1[i];
                }
            }
            if (a.frequencies && at.turns) {
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u = x[2 * i], v = x[2 * i + 1];
                        x[2 * i] = u * cosine[i] - v * sine[i];
                        x[2 * i + 1] = v * cosine[i] + u * sine[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u = x[i], v = x[4 + i];
                        x[i] = u * cosine[i] - v * sine[i];
                        x[4 + i] = v * cosine[i] + u * sine[i];
                    }
                }
            }
            lo = u32x2{pack2<H>(x[0], x[1]), pack2<H>(x[2], x[3])};
            hi = u32x2{pack2<H>(x[4], x[5]), pack2<H>(x[6], x[7])};
        }
        if (live) {
            u32x2 *const to_lo = (u32x2*)(to + 2 * at.lo), *const to_hi = (u32x2*)(to + 2 * at.hi);
            if constexpr (PAST) {
                __builtin_nontemporal_store(lo, to_lo);
                __builtin_nontemporal_store(hi, to_hi);
            } else {
                *to_lo = lo;
                *to_hi = hi;
            }
        }
    }
}

template <bool H, int LANES, bool APPEND>
hipError_t run(RotateArgs a, hipStream_t s)
{
    const int64_t heads = a.q_heads + (APPEND ? 2 * a.cache.heads : 0);
    a.chunk = (int)rotate_chunk(a.T, heads, a.dim);
    // Of a long chunk, results that pass the caches leave them to what is read (8192 tokens of 28 heads of 128 columns,
    // 117 MB: 23.6 us, through the caches 34.6); of a short one, they are there for the attention that follows.
    const bool past = a.T * heads * a.dim * 2 > (16 << 20);
    const int64_t blocks = rotate_blocks(a.T, heads, a.dim);
    if (past)
        rotate<H, LANES, APPEND, true><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    else
        rotate<H, LANES, APPEND, false><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <bool H, bool APPEND>
hipError_t run(const RotateArgs& a, hipStream_t s)
{
    const int lanes = rotate_lanes(a.dim);
    return lanes == 4    ? run<H, 4, APPEND>(a, s)
           : lanes == 8  ? run<H, 8, APPEND>(a, s)
           : lanes == 16 ? run<H, 16, APPEND>(a, s)
                         : run<H, 32, APPEND>(a, s);
}

}  // namespace

hipError_t launch_rotate(const RotateArgs& a, bool half, bool append, hipStream_t s)
{
    if (append)
        return half ? run<true, true>(a, s) : run<false, true>(a, s);
    return half ? run<true, false>(a, s) : run<false, false>(a, s);
}

}  // namespace hca
