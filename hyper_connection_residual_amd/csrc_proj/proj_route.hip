// proj_route.hip -- the router's choice and sort, and the experts' join.
//
// Both are bound by memory at length and by launches when short.  The choice
// gives a wave four tokens at a time (16 lanes each, up to 128 experts), their
// logits in registers and the next four's on their way; the sort is a counting
// sort by expert that keeps the tokens' order: every block ranks its own slots
// per expert and counts them, and a second kernel adds what lies before the
// block.  A batch that one block holds is done in one launch.  What bounds the
// choice is its instructions, some hundred per token: with one token per wave
// 32768 x 128, 8 of them, took 38 us, and now takes 19, the second kernel 8.  One
// block's batch (8 x 64) takes 4.2 us.
#include "proj_device.h"

#pragma clang fp contract(off)

namespace hcp {
namespace {

constexpr int kWaves = 16;  // at most
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxE = 512;

// Lanes per token: 8 experts for each, 4 up to 64 experts, and a lane for every slot.
int token_lanes(int64_t E, int64_t k)
{
    return E <= 128 && k <= 16 ? 16 : E <= 256 ? 32 : 64;
}

// Tokens of a block: one block, and so one launch, while that takes no longer (128 x
// 128, 8 each: 12.8 us, 9.8 us in two launches, of which the second costs the host 3;
// 128 x 256: 24, 11); then a block for every compute unit, from 16 tokens each (in
// blocks of 128 a batch of 2048 x 128 took 17 us, now 10), up to 128; then as many as
// make 512 blocks, whose counts the second kernel reads.
int block_tokens(int64_t T, int G)
{
    if (T <= (G == 16 ? 128 : 64))
        return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
    const int64_t few = (T + 255) / 256, many = (T + 511) / 512;
    const int64_t each = few <= 128 ? few : many < 128 ? 128 : many;
    return each <= 16 ? 16 : each <= 32 ? 32 : (int)((each + 63) / 64 * 64);
}

// Waves of a block: as many as it has tokens for at once, G lanes each.
int block_waves(int each, int G)
{
    const int waves = each * G / 64;
    return waves < kWaves ? waves : kWaves;
}

// Larger keys are larger logits; 0 is a masked expert (-inf, NaN).
__device__ __forceinline__ uint32_t key_of(float f)
{
    if (!(f > -INFINITY))
        return 0;
    const uint32_t b = __float_as_uint(fminf(f, 3.402823466e38f) + 0.0f);  // (-0 equals 0)
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// Over the G neighbouring lanes (16, 32 or 64) that have one token, in all of them.
template <int ROTATE>
__device__ __forceinline__ uint32_t rotated(uint32_t v)  // from the lane ROTATE before, around 16 lanes
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + ROTATE, 0xf, 0xf, false);
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    v = max(v, rotated<1>(v));
    v = max(v, rotated<2>(v));
    v = max(v, rotated<4>(v));
    v = max(v, rotated<8>(v));
    if constexpr (G > 16)
        v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    if constexpr (G > 32)
        v = max(v, (uint32_t)__shfl_xor((int)v, 32));
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v)
{
    for (int d = 1; d < G; d <<= 1)
        v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t at)
{
    return a.type == kFp32 ? ((const float*)a.logits)[at]
                           : a.type == kFp16 ? from16<true>(((const uint16_t*)a.logits)[at])
                                             : from16<false>(((const uint16_t*)a.logits)[at]);
}

// V neighbouring logits of one token from expert e on, as keys; 0 past E.
template <int V>
__device__ __forceinline__ void load_keys(const RouteArgs& a, int64_t token, int e, uint32_t (&key)[V])
{
    const int64_t at = token * a.ldl + e;
    if (a.vec && e + V <= a.E) {
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            if (a.type == kFp32) {
                const f32x4_t f = *(const f32x4_t*)((const float*)a.logits + at + q);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    key[q + c] = __float_as_uint(f[c]);
            } else {
                const uint2 w = *(const uint2*)((const uint16_t*)a.logits + at + q);
                const uint32_t u[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    key[q + c] = __float_as_uint(a.type == kFp16 ? from16<true>(u[c]) : from16<false>(u[c]));
            }
        }
#pragma unroll
        for (int q = 0; q < V; ++q)
            key[q] = key_of(__uint_as_float(key[q]));
    } else {
#pragma unroll
        for (int q = 0; q < V; ++q)
            key[q] = e + q < a.E ? key_of(load_logit(a, at + q)) : 0;
    }
}

// The choice of 64 / G tokens by one wave, G lanes each: lane l of a token holds
// experts V l and on, so that of equal logits the lowest lane's, and in a lane
// the lowest register's, is the lower expert.  Lane s returns slot s's expert (-1:
// none) and its weight.
template <int G, int V>
__device__ __forceinline__ void choose(const RouteArgs& a, uint32_t (&key)[V], int& id, float& weight)
{
    const int lane = threadIdx.x & 63, l = lane & (G - 1), base = lane & ~(G - 1);
    id = -1;
    uint32_t mine = 0, top = 0;
    float sum = 0.0f;
    for (int s = 0; s < a.k; ++s) {
        uint32_t head = key[0];
#pragma unroll
        for (int q = 1; q < V; ++q)
            head = max(head, key[q]);
        const uint32_t best = group_max<G>(head);
        if (s == 0) {
            top = best;
            if (!a.renorm) {
#pragma unroll
                for (int q = 0; q < V; ++q)
                    sum += key[q] ? expf(logit_of(key[q]) - logit_of(top)) : 0.0f;
            }
        }
        // (a token without any expert left has best = 0, a key that no expert has)
        const int first = __builtin_ctzll(__ballot(head == best) >> base);
        int e = 0;
#pragma unroll
        for (int q = V - 1; q >= 0; --q)
            e = key[q] == best ? q : e;
#pragma unroll
        for (int q = 0; q < V; ++q)
            key[q] = l == first && e == q ? 0 : key[q];
        const int chosen = __shfl(e, base + first) + V * first;
        if (l == s && best) {
            id = chosen;
            mine = best;
        }
    }
    const float w = id >= 0 ? expf(logit_of(mine) - logit_of(top)) : 0.0f;
    sum = group_sum<G>(a.renorm ? w : sum);
    weight = id >= 0 ? w / sum : 0.0f;
}

// Between turns of a wave's lanes at the same words of LDS: what the earlier lanes
// stored is there for the later ones.  (The wave's LDS instructions run in order; this
// keeps the compiler from merging or reordering the turns.  No instruction comes of it.)
__device__ __forceinline__ void next_turn()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The choice of a block's tokens; each slot's rank among the block's slots of
// its expert; and the block's counts.  ONE: the whole batch is this block, and
// the sort is finished here.
template <int G, int V, bool ONE>
__global__ __launch_bounds__(kThreads) void route_choose(RouteArgs a, int each)
{
    constexpr int TOKENS = 64 / G;  // of a wave at once
    __shared__ int count[kWaves][kMaxE];  // per wave, then what lies before the wave
    __shared__ int start[ONE ? kMaxE + 1 : 1];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l = lane & (G - 1), group = lane / G;
    // a wave's tokens are neighbours, so that its slots are in order
    const int threads = blockDim.x, waves = threads >> 6;
    const int64_t first = (int64_t)blockIdx.x * each + wave * (each / waves);
    const int64_t last = min(first + each / waves, (int64_t)a.T);
    uint32_t key[V], next[V];
    if (first < last)
        load_keys<V>(a, min(first + group, last - 1), V * l, next);
    for (int i = threadIdx.x; i < waves * kMaxE; i += threads)
        (&count[0][0])[i] = 0;
    __syncthreads();
    for (int64_t t0 = first; t0 < last; t0 += TOKENS) {
#pragma unroll
        for (int q = 0; q < V; ++q)
            key[q] = next[q];
        if (t0 + TOKENS < last)  // the next tokens' logits, while these are chosen from
            load_keys<V>(a, min(t0 + TOKENS + group, last - 1), V * l, next);
        int id;
        float weight;
        choose<G, V>(a, key, id, weight);
        const int64_t t = t0 + group;
        const bool slot = t < last && l < a.k;
        int rank = -1;
#pragma unroll
        for (int i = 0; i < TOKENS; ++i) {  // one token after the other; a token's experts differ
            if (group == i && slot && id >= 0) {
                rank = count[wave][id];
                count[wave][id] = rank + 1;
            }
            next_turn();
        }
        if (slot) {
            a.ids[t * a.k + l] = id;
            a.weights[t * a.k + l] = weight;
            a.pos[t * a.k + l] = rank;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += threads) {
        int sum = 0;
#pragma unroll 4
        for (int w = 0; w < waves; ++w) {  // (4, 8 or 16)
            const int c = count[w][e];
            count[w][e] = sum;
            sum += c;
        }
        if constexpr (ONE)
            start[e] = sum;
        else
            a.hist[(int64_t)blockIdx.x * a.E + e] = sum;
    }
    __syncthreads();
    if constexpr (ONE) {
        if (wave == 0) {
            int base = 0;
            for (int c = 0; c < a.E; c += 64) {
                const int n = c + lane < a.E ? start[c + lane] : 0;
                int upto = n;
                for (int d = 1; d < 64; d <<= 1) {
                    const int o = __shfl_up(upto, d);
                    upto += lane >= d ? o : 0;
                }
                if (c + lane < a.E) {
                    start[c + lane] = base + upto - n;
                    a.offsets[c + lane] = base + upto - n;
                }
                base += __shfl(upto, 63);
            }
            if (lane == 0) {
                start[kMaxE] = base;
                a.offsets[a.E] = base;
            }
        }
        __syncthreads();
    }
    // (each slot by the lane that stored it)
    for (int64_t t = first + group; t < last; t += TOKENS) {
        if (l >= a.k)
            continue;
        const int64_t slot = t * a.k + l;
        const int id = a.ids[slot];
        if (id < 0)
            continue;
        const int at = a.pos[slot] + count[wave][id] + (ONE ? start[id] : 0);
        a.pos[slot] = at;
        if constexpr (ONE)
            a.rows[at] = (int)t;
    }
    if constexpr (ONE)
        for (int i = start[kMaxE] + threadIdx.x; i < a.T * a.k; i += threads)
            a.rows[i] = -1;
}

// Adds what lies before the block: the lower experts' slots, and the expert's
// slots of earlier blocks.
__global__ __launch_bounds__(kThreads) void route_place(RouteArgs a, int each, int blocks)
{
    __shared__ int before[kMaxE], total[kMaxE], start[kMaxE + 1];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (int i = threadIdx.x; i < kMaxE; i += kThreads)
        before[i] = total[i] = 0;
    __syncthreads();
    // the block's threads share the counts' reading: neighbouring experts in
    // neighbouring lanes, some blocks each (whole numbers: any order)
    const int lanes = (a.E + 63) / 64 * 64, groups = kThreads / lanes;
    const int e = threadIdx.x % lanes, part = threadIdx.x / lanes;
    if (e < a.E && part < groups) {
        int b4 = 0, all = 0;
        for (int b0 = part; b0 < blocks; b0 += 16 * groups) {
            int c[16];  // (16 loads on their way together)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                c[i] = a.hist[(int64_t)min(b0 + i * groups, blocks - 1) * a.E + e];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int b = b0 + i * groups;
                all += b < blocks ? c[i] : 0;
                b4 += b < min(blocks, (int)blockIdx.x) ? c[i] : 0;
            }
        }
        atomicAdd(&before[e], b4);
        atomicAdd(&total[e], all);
    }
    __syncthreads();
    if (wave == 0) {
        int base = 0;
        for (int c = 0; c < a.E; c += 64) {
            const int n = c + lane < a.E ? total[c + lane] : 0;
            int upto = n;
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(upto, d);
                upto += lane >= d ? o : 0;
            }
            if (c + lane < a.E) {
                before[c + lane] += base + upto - n;
                if (blockIdx.x == 0)
                    a.offsets[c + lane] = base + upto - n;
            }
            base += __shfl(upto, 63);
        }
        if (lane == 0) {
            start[kMaxE] = base;
            if (blockIdx.x == 0)
                a.offsets[a.E] = base;
        }
    }
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * each, last = min(first + each, (int64_t)a.T);
    for (int64_t i = first * a.k + threadIdx.x; i < last * a.k; i += kThreads) {
        const int id = a.ids[i];
        if (id >= 0) {
            const int at = a.pos[i] + before[id];
            a.pos[i] = at;
            a.rows[at] = (int)(i / a.k);
        }
        if (i >= start[kMaxE])
            a.rows[i] = -1;
    }
}

template <int G, int V>
void run_route(const RouteArgs& a, hipStream_t s)
{
    const int each = block_tokens(a.T, G), blocks = (int)(((int64_t)a.T + each - 1) / each);
    const int threads = 64 * block_waves(each, G);
    if (blocks == 1) {
        route_choose<G, V, true><<<1, threads, 0, s>>>(a, each);
    } else {
        route_choose<G, V, false><<<blocks, threads, 0, s>>>(a, each);
        route_place<<<blocks, kThreads, 0, s>>>(a, each, blocks);
    }
}

__device__ __forceinline__ float load_value(const void* y, int type, int64_t at)
{
    return type == kFp32 ? ((const float*)y)[at]
                         : type == kFp16 ? from16<true>(((const uint16_t*)y)[at])
                                         : from16<false>(((const uint16_t*)y)[at]);
}

__device__ __forceinline__ void store_value(void* out, int type, int64_t at, float v)
{
    if (type == kFp32)
        ((float*)out)[at] = v;
    else
        ((uint16_t*)out)[at] = (uint16_t)(type == kFp16 ? bits16<true>(v) : bits16<false>(v));
}

// 8 neighbouring values of a row, of which `there` exist.
template <int TYPE>
__device__ __forceinline__ void load8(const void* y, int64_t at, int there, float (&v)[8])
{
    if (there < 8) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            v[q] = q < there ? load_value(y, TYPE, at + q) : 0.0f;
    } else if constexpr (TYPE == kFp32) {
        const f32x4_at4* p = (const f32x4_at4*)((const float*)y + at);
        const f32x4_t v0 = p[0], v1 = p[1];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] = v0[q];
            v[4 + q] = v1[q];
        }
    } else {
        const u32x4 w = *(const u32x4_at2*)((const uint16_t*)y + at);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = from16<TYPE == kFp16>(w[q] & 0xffffu);
            v[2 * q + 1] = from16<TYPE == kFp16>(w[q] >> 16);
        }
    }
}

// A thread sums 8 neighbouring columns of one token.  Bound by memory: 8192 x 2560, 8
// rows each, 364 MB in 79 us, 4.6 TB/s (a copy's rate).
template <int TYPE>
__global__ __launch_bounds__(256) void combine(CombineArgs a)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int cols = (a.C + 7) / 8;
    const int64_t t = i / cols;
    const int c = (int)(i % cols) * 8, there = min(8, a.C - c);
    if (t >= a.T)
        return;
    float sum[8] = {};
    for (int s = 0; s < a.k; ++s) {
        const int64_t row = a.pos[t * a.k + s];
        if (row < 0 || row >= a.y_rows)
            continue;
        const float w = a.weights[t * a.k + s];
        float v[8];
        load8<TYPE>(a.y, row * a.ldy + c, there, v);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            sum[q] = fmaf(w, v[q], sum[q]);
    }
    const int64_t at = t * a.ldo + c;
    if (there < 8) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < there)
                store_value(a.out, a.out_type, at + q, sum[q]);
    } else if (a.out_type == kFp32) {
        f32x4_at4* p = (f32x4_at4*)((float*)a.out + at);
        p[0] = f32x4_t{sum[0], sum[1], sum[2], sum[3]};
        p[1] = f32x4_t{sum[4], sum[5], sum[6], sum[7]};
    } else {
        u32x4 w;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            w[q] = a.out_type == kFp16 ? bits16<true>(sum[2 * q]) | bits16<true>(sum[2 * q + 1]) << 16
                                       : bits16<false>(sum[2 * q]) | bits16<false>(sum[2 * q + 1]) << 16;
        *(u32x4_at2*)((uint16_t*)a.out + at) = w;
    }
}

template <int TYPE>
hipError_t run_combine(const CombineArgs& a, hipStream_t s)
{
    const int64_t blocks = ((int64_t)a.T * ((a.C + 7) / 8) + 255) / 256;
    if (!fits(blocks, 256))
        return hipErrorInvalidConfiguration;
    combine<TYPE><<<(unsigned)blocks, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int route_blocks(int64_t T, int64_t E, int64_t k)
{
    const int each = block_tokens(T, token_lanes(E, k));
    return (int)((T + each - 1) / each);
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s)
{
    const int lanes = token_lanes(a.E, a.k);
    if (lanes == 16 && a.E <= 64)
        run_route<16, 4>(a, s);
    else if (lanes == 16)
        run_route<16, 8>(a, s);
    else if (lanes == 32)
        run_route<32, 8>(a, s);
    else
        run_route<64, 8>(a, s);
    return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t s)
{
    return a.type == kFp32   ? run_combine<kFp32>(a, s)
           : a.type == kFp16 ? run_combine<kFp16>(a, s)
                             : run_combine<kBf16>(a, s);
}

}  // namespace hcp
