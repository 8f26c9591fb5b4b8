// proj_api.hip -- host side of the C ABI declared in include/hc_proj.h:
// argument checks, the choice of the kernel, and the launches.  Nothing is
// allocated and no state is kept but which devices are gfx950.
#include "hc_proj.h"
#include "proj_internal.h"

#include <atomic>
#include <cstring>

namespace {

using namespace hcp;

thread_local int g_last_hip_error = 0;

int record(hipError_t e, int status)
{
    g_last_hip_error = static_cast<int>(e);
    return status;
}

bool aligned(const void* p, uintptr_t to)
{
    return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}

int64_t size_of(int type)
{
    return type == kFp32 ? 4 : 2;
}

// The current device must be a gfx950 part.
int check_device()
{
    constexpr int kDevices = 64;
    static std::atomic<signed char> known[kDevices];  // 0: not asked yet
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return record(e, HC_ERR_DEVICE);
    signed char ok = dev < kDevices ? known[dev].load(std::memory_order_relaxed) : 0;
    if (!ok) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, dev);
        if (e != hipSuccess)
            return record(e, HC_ERR_DEVICE);
        ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
        if (dev < kDevices)
            known[dev].store(ok, std::memory_order_relaxed);
    }
    return ok > 0 ? HC_OK : record(hipSuccess, HC_ERR_DEVICE);
}

int done(hipError_t e)
{
    return e == hipSuccess                       ? HC_OK
           : e == hipErrorInvalidConfiguration ? record(e, HC_ERR_SIZE)  // (see fits)
                                                 : record(e, HC_ERR_LAUNCH);
}

constexpr int64_t kMost = (int64_t(1) << 31) - 65536;  // rows and columns: 32-bit tile arithmetic
constexpr int64_t kMostK = int64_t(1) << 28;           // a row's bytes: 32-bit offsets

int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

// Whether the adapter's inner product is part of the one kernel: one token, and
// A's way from the L2 to every workgroup shorter than a launch (1 x 2560 x 2560,
// rank 16: 5.5 us against 9.3; 1 x 10240 x 2560, rank 32, 20480 rows of A in
// all: 18.3 us against 17.3).
bool one_launch(int64_t T, int64_t N, int64_t rank)
{
    return T == 1 && rank <= kTokenRank && ceil_div(N, 16) * rank <= 12288;
}

int64_t pad16(int64_t bytes)
{
    return (bytes + 15) & ~int64_t(15);
}

// How a product is taken: by the wide kernel; by the small one (tokens of a tile
// 8, 16 or 32); or by the tiled one (64 or 128), with splits of K.
enum Kernel { kSmall, kTiled, kWide };
struct Plan {
    Kernel kernel;
    int tokens, splits;
    double us;
};

// What a product of `tiles` row tiles of 32 takes by the small kernel, in us: 3 us,
// and the longer of its waves' way through K (0.55 us a unit in grids of one round,
// 0.6 us in larger ones) and what it moves from the L2, 20 TB/s; 1.5 ns per workgroup.
double small_us(double tiles, int64_t K, int64_t N, bool gate)
{
    const double groups = tiles * (double)ceil_div(N, 16), units = (double)ceil_div(K, 64);
    const double way = groups <= 256 ? 0.55 * units / 8 : 0.6 * units / 4;
    const double moved = groups * (gate ? 64 : 48) * 2.0 * (double)K / 20e6;
    return 3.0 + (way > moved ? way : moved) + 0.0015 * groups;
}

// What `tiles` tiles of the tiled kernel take, in us.  The chip holds 512 workgroups,
// two on a compute unit, which then share the way into its LDS: a step of 64 takes
// 0.38 us with 64 tokens and 0.8 us with 128 in a last round of up to 256
// workgroups, 0.75 and 1.1 us in others, and a workgroup's start and end 4 us;
// splits cost the second kernel's 4 us and their partial sums' way, 6 TB/s.
double tiled_us(double tiles, int tokens, int64_t K, int z, double outputs)
{
    const int64_t groups = (int64_t)tiles * z, rest = groups % 512;
    const double steps = (double)ceil_div(ceil_div(K, 64), z);
    const double alone = 4.0 + (tokens == 64 ? 0.38 : 0.8) * steps, shared = 4.0 + (tokens == 64 ? 0.75 : 1.1) * steps;
    return (double)(groups / 512) * shared + (rest == 0 ? 0.0 : rest <= 256 ? alone : shared) +
           (z > 1 ? 4.0 + outputs * z * 8.0 / 6e6 : 0.0);
}

// What `tiles` tiles of the wide kernel take, in us: rounds of 256 workgroups (of 32 for
// each XCD, which takes an eighth of the tiles), a step of 64 1.15 us, a workgroup's
// start and end 11 us; splits as above, and slower.
double wide_us(double tiles, int64_t K, int z, double outputs)
{
    return (double)ceil_div(ceil_div((int64_t)tiles, 8) * z, 32) * (11.0 + 1.15 * (double)ceil_div(ceil_div(K, 64), z)) +
           (z > 1 ? 8.0 + outputs * z * 8.0 / 5e6 : 0.0);
}

// The plan that takes the least time by what its parts measured; the small kernel
// takes the benefit of the doubt.  How many adapters a tile has is not known here:
// assumed are, for every 32 ranks, 3 us (and 2) of the tiled kernel's workgroups, which
// the splits share, and some more in tiles of 128 tokens; 3 us of the wide one's; 6 ns
// for each of the small one's.  (5 and 7 splits are left out: 45 x 8720
// x 4215 takes 34 us with 7 and 25 us with 6.)  Over 530 products of 33 to 4000 tokens
// the plan takes 1.5 % longer than the best of all, over 490 with adapters 1.5 %.  Both
// sides measured, in us: 128 x 2560 x 2560 small 10.9, tiled 14.0; 100 x 674 x 3584 8.0,
// 12.7; 1500 x 33 x 1744 7.0, 9.6; 400 x 2560 x 2560 26, 22; 100 x 10240 x 2560 34, 23; of the
// tilings, 512 x 5600 x 4096: 41 with 64 tokens and no splits, 48 with 128 tokens and 3,
// 69 with 128 and none; 3633 x 1384 x 2418: 36 with wide tiles, 50 with 64 tokens; 2000
// x 10240 x 2560: 108 with wide tiles and 3 splits, 139 with 64 tokens; with adapters, 1341 x 280 x 1394, rank 64: small 70, tiled 17.
Plan plan(int64_t T, int64_t K, int64_t N, int64_t rank)
{
    const double small = small_us((double)ceil_div(T, 32), K, N, false);
    if (T <= 32)
        return Plan{kSmall, T <= 8 ? 8 : T <= 16 ? 16 : 32, 1, small};
    Plan best{kTiled, 64, 1, 0.0};
    const double ranks = (double)rank / 32;
    for (int tokens = 64; tokens <= 128; tokens += 64)
        for (int z : {1, 2, 3, 4, 6, 8}) {
            if (z > 1 && z * 256 > K)
                break;
            const int64_t tiles = ceil_div(T, tokens) * ceil_div(N, 128);
            double us = tiled_us((double)tiles, tokens, K, z, (double)T * (double)N);
            if (rank)
                us = (tokens == 64 ? us : 1.15 * us) + (2.0 + 3.0 * ranks) / z * (double)ceil_div(tiles * z, 512);
            if (best.us == 0 || us < best.us)
                best = Plan{kTiled, tokens, z, us};
        }
    const int64_t tiles = ceil_div(T, 256) * ceil_div(N, 256), groups = ceil_div(T, 32) * ceil_div(N, 16);
    for (int z : {1, 2, 3, 4, 6, 8}) {
        if (K <= 64 || (z > 1 && z * 512 > K))
            break;
        const double us = wide_us((double)tiles, K, z, (double)T * (double)N) + 3.0 * ranks * (double)ceil_div(tiles, 256);
        if (us < best.us)
            best = Plan{kWide, 256, z, us};
    }
    if (small + 0.006 * ranks * (double)groups < 1.2 * best.us)
        return Plan{kSmall, 32, 1, small};
    return best;
}

// The tokens that are taken first, in whole rounds of the wide kernel, where the
// rest by itself takes less time than in its last round; 0: all together.  6656 x
// 10240 x 2560, 260 tiles: 378 us in two rounds, 275 us as 250 tiles and 256 tokens;
// 6600 x 2568 x 2560: 126, 87.
int64_t head_of(int64_t T, int64_t K, int64_t N, int64_t rank)
{
    const int64_t cols = ceil_div(N, 256), tiles = ceil_div(T, 256) * cols, head = tiles / 256 * 256 / cols * 256;
    if (tiles % 256 == 0 || head == 0 || head >= T)
        return 0;
    return plan(head, K, N, rank).us + plan(T - head, K, N, rank).us + (rank ? 10.0 : 5.0) < 0.97 * plan(T, K, N, rank).us
               ? head
               : 0;
}

// Splits of K for v = A x: 4096 of K for each, as many as the kernel that adds
// them up takes; none once the tokens fill the chip.
int down_splits(const Plan& by, int64_t T, int64_t K)
{
    const int64_t most = T > 2048 || by.kernel == kWide ? 1 : by.kernel == kSmall ? kSplitsSmall : kSplitsTile;
    const int64_t z = ceil_div(K, 4096);
    return (int)(z > most ? most : z);
}

// Scratch of a product: v or its pieces first, then the splits' partial sums.
int64_t v_bytes(const Plan& by, int64_t T, int64_t K, int64_t rank, bool half)
{
    return by.kernel == kWide ? T * piece_bytes((int)rank, half) : pad16(4 * (int64_t)down_splits(by, T, K) * T * rank);
}

// Scratch of the tokens that are taken together.
int64_t part_work(int64_t T, int64_t K, int64_t N, int64_t rank)
{
    if (rank && one_launch(T, N, rank))
        return 0;
    const Plan by = plan(T, K, N, rank);
    return (rank ? v_bytes(by, T, K, rank, true) : 0) + (by.splits > 1 ? 4 * by.splits * T * N : 0);
}

// Whether all launches for these tokens can take place (see fits).
bool part_fits(int64_t T, int64_t K, int64_t N, int64_t rank)
{
    if (rank && one_launch(T, N, rank))
        return fits(token_blocks(N), 512);
    const Plan by = plan(T, K, N, rank);
    if ((rank && !fits(down_blocks(T), 256)) || (by.splits > 1 && !fits(join_blocks(T, N), 256)))
        return false;
    const int cols = by.kernel == kSmall ? kSmallCols : by.kernel == kWide ? kWideCols : kTileCols;
    const int threads = by.kernel == kSmall ? kSmallThreads : by.kernel == kWide ? kWideThreads : kTileThreads;
    return fits(product_blocks(T, 0, by.tokens, N, cols) * by.splits, threads);
}

// The launches for the tokens that are taken together, all of `a`'s.
int project_part(ProductArgs a, int type, const char* A, float* v, hipStream_t s)
{
    const int64_t T = a.M, K = a.K, N = a.N, rank = a.rank;
    if (rank && one_launch(T, N, rank))
        return done(launch_token(a, type, A, s));
    const Plan by = plan(T, K, N, rank);
    if (rank) {
        DownArgs d{a.x, a.ldx, a.M, a.K, a.adapter, a.adapters, a.rank, A, v, down_splits(by, T, K), nullptr, a.scale};
        if (by.kernel == kWide)
            d.pieces = reinterpret_cast<char*>(v);
        const hipError_t e = launch_adapter_down(d, type, s);
        if (e != hipSuccess)
            return done(e);
        a.v = v;
        a.v_splits = d.splits;
        a.pieces = d.pieces;
    }
    const int mode = rank ? kAdapt : kPlain;
    a.splits = by.splits;
    a.part = v + (rank ? v_bytes(by, T, K, rank, type == HC_FP16) / 4 : 0);
    hipError_t e = by.kernel == kSmall  ? launch_small(a, type, mode, by.tokens, s)
                   : by.kernel == kWide ? launch_wide(a, type, mode, s)
                                        : launch_tile(a, type, mode, by.tokens, 3, s);
    if (e == hipSuccess && a.splits > 1)
        e = launch_join(a, type, s);
    return done(e);
}

}  // namespace

extern "C" {

HC_API int64_t hc_project_work(int64_t T, int64_t K, int64_t N, int64_t rank)
{
    if (T < 1 || K < 1 || N < 1 || rank < 0 || rank > HC_MAX_RANK || T > kMost || N > kMost || K > kMostK)
        return 0;
    const int64_t head = head_of(T, K, N, rank), rest = part_work(T - head, K, N, rank);
    const int64_t first = head ? part_work(head, K, N, rank) : 0;
    return first > rest ? first : rest;
}

HC_API int hc_project(int64_t T, int64_t K, int64_t N, int type, const void* x, int64_t ldx, const void* W,
                      const int32_t* adapter, int64_t adapters, int64_t rank, const void* A, const void* B,
                      const float* scale, void* out, int64_t ldo, int out_type, void* work, int64_t work_bytes,
                      void* stream)
{
    const bool beside = adapter && adapters > 0;
    if (T < 1 || K < 1 || N < 1 || adapters < 0 || !x || !W || !out || (type != HC_BF16 && type != HC_FP16) ||
        (out_type != type && out_type != HC_FP32) || ldx < K || ldo < N)
        return HC_ERR_ARG;
    if (beside && (!A || !B || rank < 1))
        return HC_ERR_ARG;
    if (T > kMost || N > kMost || K > kMostK || K % 8 || ldx % 8 || adapters > kMost ||
        (beside && (rank % 8 || rank > HC_MAX_RANK)))
        return HC_ERR_SIZE;
    if (!beside)
        rank = 0;
    const int64_t need = hc_project_work(T, K, N, rank);
    if (need && !work)
        return HC_ERR_ARG;
    if (work_bytes < need)
        return HC_ERR_SIZE;
    const int64_t head = head_of(T, K, N, rank);
    if ((head && !part_fits(head, K, N, rank)) || !part_fits(T - head, K, N, rank))
        return HC_ERR_SIZE;
    if (!aligned(x, 16) || !aligned(W, 16) || (need && !aligned(work, 16)) || !aligned(out, size_of(out_type)) ||
        (beside && (!aligned(A, 16) || !aligned(B, 16) || !aligned(adapter, 4) || !aligned(scale, 4))))
        return HC_ERR_ALIGN;
    const int st = check_device();
    if (st != HC_OK)
        return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    float* v = static_cast<float*>(work);
    ProductArgs a{};
    a.x = static_cast<const char*>(x);
    a.ldx = 2 * ldx;
    a.x_rows = T;
    a.W = static_cast<const char*>(W);
    a.E = 1;
    a.M = (int)T;
    a.K = (int)K;
    a.N = (int)N;
    a.out = static_cast<char*>(out);
    a.ldo = ldo;
    a.out32 = out_type == HC_FP32;
    a.splits = 1;
    if (beside) {
        a.adapter = adapter;
        a.adapters = (int)adapters;
        a.rank = (int)rank;
        a.B = static_cast<const char*>(B);
        a.scale = scale;
    }
    // (the second part's v takes the first's place when the stream has passed it)
    if (head) {
        a.M = (int)head;
        const int first = project_part(a, type, static_cast<const char*>(A), v, s);
        if (first != HC_OK)
            return first;
        a.x += head * a.ldx;
        a.x_rows = a.M = (int)(T - head);
        a.out += head * ldo * size_of(out_type);
        if (beside)
            a.adapter += head;
    }
    return project_part(a, type, static_cast<const char*>(A), v, s);
}

HC_API int hc_expert_project(int64_t R, int64_t K, int64_t N, int64_t E, int type, const void* x, int64_t x_rows,
                             int64_t ldx, const int32_t* rows, const void* W, const int32_t* offsets, int gate,
                             void* out, int64_t ldo, int out_type, void* stream)
{
    if (R < 1 || K < 1 || N < 1 || E < 1 || x_rows < 1 || !x || !W || !offsets || !out ||
        (type != HC_BF16 && type != HC_FP16) || (out_type != type && out_type != HC_FP32) || ldx < K || ldo < N)
        return HC_ERR_ARG;
    if (!rows && x_rows < R)
        return HC_ERR_ARG;
    if (R > kMost || N > kMost / 2 || K > kMostK || E > kMost || K % 8 || ldx % 8)
        return HC_ERR_SIZE;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(out, size_of(out_type)) || !aligned(offsets, 4) ||
        !aligned(rows, 4))
        return HC_ERR_ALIGN;
    const int st = check_device();
    if (st != HC_OK)
        return st;
    ProductArgs a{};
    a.x = static_cast<const char*>(x);
    a.ldx = 2 * ldx;
    a.x_rows = x_rows;
    a.rows = rows;
    a.W = static_cast<const char*>(W);
    a.offsets = offsets;
    a.E = (int)E;
    a.M = (int)R;
    a.K = (int)K;
    a.N = (int)N;
    a.out = static_cast<char*>(out);
    a.ldo = ldo;
    a.out32 = out_type == HC_FP32;
    a.splits = 1;
    const int mode = gate ? kGate : kPlain;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // The groups' sizes are on the device: the rules go by their mean, and by a
    // last tile of each group that is half full.
    const int64_t mean = ceil_div(R, E), wn = gate ? 2 * N : N;
    const double halves = 0.5 * (double)(E < R ? E : R);
    if (R <= 8 || mean <= 4)
        return done(launch_small(a, type, mode, 8, s));
    if (mean <= 12)
        return done(launch_small(a, type, mode, 16, s));
    if (mean <= 24)
        return done(launch_small(a, type, mode, 32, s));
    // The least time by what the kernels' parts measured (15 % less of the doubt for
    // the small one, which gathers x once for every 16 outputs), or by the way of
    // all experts' weights from memory, which each kernel takes at a rate of its own.
    // Over 700 calls of 25 to 40000 rows this takes 2.7 % longer than the best of all, and
    // 7 % less than tiles of 64 rows up to a mean of 128, and 128 or 256 from there on.
    // Both sides measured, in us: 9168 rows of 39 experts, gated 2712 -> 75: small 84,
    // 64 rows 41; 18830 of 44, gated 392 -> 64: 18, 128 rows 11; 2688 of 16, 1296 -> 4089:
    // 64 rows 77, 128 rows 66, wide 48; 1806 of 32, gated 2560 -> 1023 (335 MB of weights):
    // small 111, 64 rows 79, 128 rows 106, wide 78.
    const auto us = [&](double parts, double rate) {
        const double way = (double)(E < R ? E : R) * (double)K * (double)wn * 2e-6 / rate;  // (rate: TB/s)
        return parts > way ? parts : way;
    };
    const double tiles64 = ((double)ceil_div(R, 64) + halves) * (double)ceil_div(wn, 128);
    const double tiles128 = ((double)ceil_div(R, 128) + halves) * (double)ceil_div(wn, 128);
    const double us32 = us(small_us((double)ceil_div(R, 32) + halves, K, N, gate) / 0.85, 4.0);
    const double us64 = us(tiled_us(tiles64, 64, K, 1, 0), 4.7);
    const double us128 = us(tiled_us(tiles128, 128, K, 1, 0), 3.0);
    const double us256 = us(wide_us(((double)ceil_div(R, 256) + halves) * (double)ceil_div(wn, 256), K, 1, 0), 4.5);
    const double tiled = us64 < us128 ? us64 : us128;
    if (K > 64 && us256 < us32 && us256 < tiled)
        return done(launch_wide(a, type, mode, s));
    if (us32 < tiled)
        return done(launch_small(a, type, mode, 32, s));
    if (us128 < us64)
        return done(launch_tile(a, type, mode, 128, 2, s));
    // Rings of two stages let a compute unit hold three workgroups, of three
    // stages two: the shorter ring where all workgroups then run at once.  1806
    // rows of 32 experts, gated 2560 -> 1023: 704 workgroups, 81 us against 90;
    // 3600 rows, 1152: 127 us against 115; 900 rows, 480: 82 us against 79.
    return done(launch_tile(a, type, mode, 64, tiles64 > 512 && tiles64 <= 768 ? 2 : 3, s));
}

HC_API int64_t hc_route_work(int64_t T, int64_t E, int64_t k)
{
    if (T < 1 || E < 1 || k < 1 || E > HC_MAX_EXPERTS || k > HC_MAX_TOPK || T > kMost / k)
        return 0;
    const int blocks = route_blocks(T, E, k);
    return blocks > 1 ? 4 * blocks * E : 0;
}

HC_API int hc_route(int64_t T, int64_t E, int64_t k, const void* logits, int64_t ldl, int type, int renorm,
                    int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, void* work,
                    int64_t work_bytes, void* stream)
{
    if (T < 1 || E < 1 || k < 1 || k > E || !logits || !ids || !weights || !offsets || !rows || !pos ||
        (type != HC_BF16 && type != HC_FP16 && type != HC_FP32) || ldl < E)
        return HC_ERR_ARG;
    if (E > HC_MAX_EXPERTS || k > HC_MAX_TOPK || T > kMost / k)
        return HC_ERR_SIZE;
    const int64_t need = hc_route_work(T, E, k);
    if (need && !work)
        return HC_ERR_ARG;
    if (work_bytes < need)
        return HC_ERR_SIZE;
    if (!aligned(logits, size_of(type)) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(offsets, 4) ||
        !aligned(rows, 4) || !aligned(pos, 4) || (need && !aligned(work, 16)))
        return HC_ERR_ALIGN;
    const int st = check_device();
    if (st != HC_OK)
        return st;
    const RouteArgs a{(int)T, (int)E, (int)k, logits, ldl, type, renorm != 0,
                      aligned(logits, 16) && ldl * size_of(type) % 16 == 0, ids, offsets, rows, pos, weights,
                      static_cast<int32_t*>(work)};
    return done(launch_route(a, static_cast<hipStream_t>(stream)));
}

HC_API int hc_expert_combine(int64_t T, int64_t k, int64_t C, const void* y, int64_t y_rows, int64_t ldy, int type,
                             const int32_t* pos, const float* weights, void* out, int64_t ldo, int out_type,
                             void* stream)
{
    const auto known = [](int t) { return t == HC_BF16 || t == HC_FP16 || t == HC_FP32; };
    if (T < 1 || k < 1 || C < 1 || y_rows < 1 || !y || !pos || !weights || !out || !known(type) ||
        !known(out_type) || ldy < C || ldo < C)
        return HC_ERR_ARG;
    if (T > kMost / k || C > kMost || ceil_div(T * C, 256) > kMost || k > HC_MAX_EXPERTS)
        return HC_ERR_SIZE;
    if (!aligned(y, size_of(type)) || !aligned(out, size_of(out_type)) || !aligned(pos, 4) || !aligned(weights, 4))
        return HC_ERR_ALIGN;
    const int st = check_device();
    if (st != HC_OK)
        return st;
    const CombineArgs a{(int)T, (int)k, (int)C, y, y_rows, ldy, type, pos, weights, out, ldo, out_type};
    return done(launch_combine(a, static_cast<hipStream_t>(stream)));
}

HC_API const char* hc_proj_status_string(int status)
{
    switch (status) {
    case HC_OK: return "ok";
    case HC_ERR_ARG: return "invalid argument (a size below 1, a required pointer that is NULL, a type that the call does not take, "
                            "a row stride shorter than its row, or k above E)";
    case HC_ERR_ALIGN: return "a pointer is not aligned (16 bytes for x, W, A, B and work, its own type for the others)";
    case HC_ERR_DEVICE: return "the current device is not a gfx950 (MI355X) GPU or could not be queried";
    case HC_ERR_LAUNCH: return "a kernel launch failed";
    case HC_ERR_SIZE: return "a size is outside its limits (K, ldx and rank are multiples of 8, rank up to 128, 512 experts, "
                             "32 per token, fewer than 2^31 rows, fewer than 2^32 threads), or work_bytes is too small";
    default: return "unknown status";
    }
}

HC_API int hc_proj_last_hip_error(void)
{
    return g_last_hip_error;
}

}  // extern "C"
