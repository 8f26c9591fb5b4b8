// attn_api.hip -- host side of the C ABI declared in include/hc_attn.h: argument
// checks, the choice of the kernel, and the launches.  Nothing is allocated and
// no state is kept but which devices are gfx950.
#include "hc_attn.h"
#include "attn_internal.h"

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstring>

namespace {

using namespace hca;

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
    return e == hipSuccess ? HC_OK : record(e, HC_ERR_LAUNCH);
}

constexpr int64_t kMost = (int64_t(1) << 31) - 65536;
constexpr int64_t kMostStride = int64_t(1) << 23;  // elements from row to row and head to head of a cache (bytes: 24 bits)
constexpr float kMostScale = 0x1p100f;  // scale and cap: what they are multiplied by stays a number

int64_t ceil_div(int64_t a, int64_t b)
{
    return (a + b - 1) / b;
}

// Heads [T][heads][dim] in memory.
int check_heads(const void* x, int64_t row, int64_t head, int64_t heads, int64_t dim)
{
    if (!x || (heads > 1 && head < dim) || row < dim)
        return HC_ERR_ARG;
    if (row % 8 || head % 8)
        return HC_ERR_SIZE;
    return HC_OK;
}

int check_cache(const hc_cache* c)
{
    if (!c || !c->keys || !c->values || c->pages < 1 || c->heads < 1 || c->dim < 1 || c->page_size < 1 ||
        (c->type != HC_BF16 && c->type != HC_FP16) || c->key_row < c->dim || c->value_row < c->dim || c->key_page < 0 ||
        c->value_page < 0 || (c->heads > 1 && (c->key_head < c->dim || c->value_head < c->dim)))
        return HC_ERR_ARG;
    if (c->dim > HC_MAX_HEAD || c->dim % 8 || c->page_size < HC_MIN_PAGE || c->page_size > HC_MAX_PAGE ||
        (c->page_size & (c->page_size - 1)) || c->pages > kMost || c->key_page >= kMost || c->value_page >= kMost || c->heads > 65536 || (c->key_row | c->value_row | c->key_head | c->value_head) >= kMostStride ||
        (c->key_row | c->value_row | c->key_head | c->value_head | c->key_page | c->value_page) % 8)
        return HC_ERR_SIZE;
    return HC_OK;
}

int check_batch(const hc_batch* b)
{
    if (!b || b->requests < 1 || !b->offsets || !b->lengths || b->width < 0 || (b->width > 0 && !b->table) ||
        (b->requests > 1 && b->table_row < b->width))
        return HC_ERR_ARG;
    return b->requests > HC_MAX_REQUESTS || b->width > kMost || b->table_row > (int64_t(1) << 40) ? HC_ERR_SIZE : HC_OK;
}

int check_prefix(const hc_prefix* p)
{
    if (!p || p->groups < 1 || !p->starts || !p->lengths || p->width < 0 || (p->width > 0 && !p->table) ||
        (p->groups > 1 && p->table_row < p->width))
        return HC_ERR_ARG;
    return p->groups > HC_MAX_REQUESTS || p->width > kMost || p->table_row > (int64_t(1) << 40) ? HC_ERR_SIZE : HC_OK;
}

CacheArgs cache_of(const hc_cache* c)
{
    CacheArgs a{};
    a.k = static_cast<char*>(c->keys);
    a.v = static_cast<char*>(c->values);
    a.pages = c->pages;
    a.k_page = 2 * c->key_page;
    a.v_page = 2 * c->value_page;
    a.k_row = (int)(2 * c->key_row);
    a.k_head = (int)(2 * c->key_head);
    a.v_row = (int)(2 * c->value_row);
    a.v_head = (int)(2 * c->value_head);
    while ((int64_t(1) << a.shift) < c->page_size)
        ++a.shift;
    a.heads = (int)c->heads;
    a.dim = (int)c->dim;
    return a;
}

BatchArgs batch_of(const hc_batch* b)
{
    return BatchArgs{b->offsets, b->lengths, b->table, b->table_row, (int)b->requests, (int)b->width};
}

bool batch_aligned(const hc_batch* b)
{
    return aligned(b->offsets, 4) && aligned(b->lengths, 4) && aligned(b->table, 4);
}

// Which kernel, and how many rows its tiles have: those that hold the new tokens'
// rows of a request on average.
struct Choice {
    int rows;  // kManyRows and more: the many kernel
    int64_t tiles;  // no more than these, of all segments
};
Choice choose(int64_t rows, int64_t dim, int64_t requests, int64_t groups)
{
    const int64_t mean = ceil_div(rows, requests);
    // The cache straight into registers pays for short calls of single tokens, whose start is shorter (one token over 300 positions
    // of 4 heads of 128 columns 12.6 us, through LDS 14.4; 64 tokens over up to 500 15.5 and 17.1; up to 16000 114.8 and 112.0), and, of wide heads, whose
    // values take twice the time through LDS, for windows (24 rows each, capped: 57.1 us and 61.5; not capped 56.9 and 55.2).  From 10
    // rows of up to 128 columns LDS takes less: 10 rows 47.1 and 51.4, 40 rows 48.4 and 75.6.  The mean is of the whole batch, whatever its requests are: 256
    // single tokens with a chunk of 150 (a mean of 8) take 153 us, through LDS 134, as two calls 175.
    const int few = dim > 128 ? (mean <= 16 ? 16 : mean <= 32 ? 32 : 0) : mean <= 8 ? 16 : 0;
    if (few && !groups)
        return Choice{few, rows / few + requests};
    // Eight waves on a step's keys and values halve what goes into LDS: a prompt of 8192 tokens 357 us, four waves 386; 20
    // requests of 500 rows 48.3 and 47.8, of 300 (tiles half empty) 42.8 and 40.1.  Smaller heads, more arithmetic for
    // what they load, gain nothing (documents 90 and 87 when it was tried), and wider ones have no registers for it.
    const int many = mean > 256 && padded((int)dim) == 128 && !groups ? 256 : kManyRows;
    return Choice{many, (groups ? 2 : 1) * (rows / many) + requests + groups};
}

bool sizes_fit(int64_t T, int64_t q_heads, int64_t heads, int64_t requests, int64_t groups)
{
    return T >= 1 && heads >= 1 && q_heads >= heads && q_heads % heads == 0 && q_heads <= 65536 && T <= kMaxRows && q_heads / heads <= kMaxRows &&
           T * (q_heads / heads) <= kMaxRows && requests >= 1 && requests <= HC_MAX_REQUESTS && groups <= HC_MAX_REQUESTS;
}

int attend(int64_t T, int64_t q_heads, const void* q, int64_t q_row, int64_t q_head, const hc_cache* cache, const hc_batch* batch,
           const hc_prefix* prefix, float scale, float cap, const float* slopes, const int32_t* first, const int32_t* last, void* out,
           int64_t out_row, int64_t out_head, void* work, int64_t work_bytes, void* stream)
{
    int st = check_cache(cache);
    if (st == HC_OK)
        st = check_batch(batch);
    if (st != HC_OK)
        return st;
    if (T < 1 || q_heads < 1 || q_heads % cache->heads || !work || !(cap >= 0.0f && cap <= kMostScale) || !(std::fabs(scale) <= kMostScale))
        return HC_ERR_ARG;
    st = check_heads(q, q_row, q_head, q_heads, cache->dim);
    if (st == HC_OK)
        st = check_heads(out, out_row, out_head, q_heads, cache->dim);
    if (st != HC_OK)
        return st;
    const int64_t groups = prefix ? prefix->groups : 0;
    if (!sizes_fit(T, q_heads, cache->heads, batch->requests, groups))
        return HC_ERR_SIZE;
    if (groups && !fits(join_blocks(T, q_heads, 8), kJoinThreads))
        return HC_ERR_SIZE;
    const int64_t group = q_heads / cache->heads;
    const Choice to = choose(T * group, cache->dim, batch->requests, groups);
    // (positions of a sequence are counted in 32 bits, to the end of its last unit, and so are units of all tiles, with up to 4 more
    // for each; the smallest unit has 32 positions)
    const int64_t prefix_width = prefix ? prefix->width : 0, width = std::max(prefix_width, batch->width);
    if (prefix_width + batch->width > kMost / cache->page_size || to.tiles * (ceil_div(width * cache->page_size, 32) + 8) >= (int64_t(1) << 31))
        return HC_ERR_SIZE;
    const Scratch at = scratch_of(T, q_heads, to.rows, padded((int)cache->dim), batch->requests + groups, to.tiles, groups > 0);
    if (work_bytes < at.bytes)
        return HC_ERR_SIZE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache->keys, 16) || !aligned(cache->values, 16) || !aligned(work, 16) || !batch_aligned(batch) ||
        !aligned(slopes, 4) || !aligned(first, 4) || !aligned(last, 4) ||
        (prefix && !(aligned(prefix->starts, 4) && aligned(prefix->lengths, 4) && aligned(prefix->table, 4))))
        return HC_ERR_ALIGN;
    st = check_device();
    if (st != HC_OK)
        return st;
    AttendArgs a{};
    a.q = HeadsArgs{static_cast<const char*>(q), 2 * q_row, 2 * q_head};
    a.out = static_cast<char*>(out);
    a.out_row = 2 * out_row;
    a.out_head = 2 * out_head;
    a.cache = cache_of(cache);
    a.batch = batch_of(batch);
    if (prefix)
        a.prefix = PrefixArgs{prefix->starts, prefix->lengths, prefix->table, prefix->table_row, (int)groups, (int)prefix->width};
    a.T = (int)T;
    a.q_heads = (int)q_heads;
    a.group = (int)group;
    constexpr double log2e = 1.4426950408889634;
    a.scale = (float)(std::fabs(scale) * log2e);
    a.q_sign = scale < 0.0f ? 0x80008000u : 0u;
    if (cap > 0.0f) {
        a.cap_in = (float)std::min(2.0 * log2e * std::fabs(scale) / cap, (double)FLT_MAX);
        a.cap_out = (float)(cap * log2e);
    }
    a.slopes = slopes;
    a.first = first;
    a.last = last;
    a.rows = to.rows;
    a.tiles = (int)to.tiles;
    const int unit = to.rows >= kManyRows ? kStepBytes / (2 * padded((int)cache->dim)) : kFewUnit;  // positions
    a.least = to.rows >= kManyRows ? 1 : 64 / to.rows;  // (few: one for each of a workgroup's waves that share a row)
    // An item's start and end, in units: of many rows 128 positions' time, of 256 rows (alone on their compute unit) 256 positions'.
    a.item_cost = to.rows >= kManyRows ? to.rows / unit : 3;
    // as many as are on the card at once: two on a compute unit, or one with the registers that wide heads need
    a.workers = cache->dim > 128 || to.rows == 256 ? kWorkers / 2 : kWorkers;
    char* const w = static_cast<char*>(work);
    a.part = reinterpret_cast<float*>(w);
    a.ml = reinterpret_cast<float2*>(w + at.ml);
    a.records = reinterpret_cast<int32_t*>(w + at.records);
    a.plan = reinterpret_cast<int32_t*>(w + at.plan);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool half = cache->type == HC_FP16;
    if (first || last) {
        a.ranges = reinterpret_cast<int2*>(w + at.ranges);
        st = done(launch_ranges(a, unit, s));
        if (st != HC_OK)
            return st;
    }
    st = done(to.rows < kManyRows ? launch_few(a, half, s) : half ? launch_many_fp16(a, s) : launch_many_bf16(a, s));
    return st == HC_OK ? done(launch_join(a, half, s)) : st;
}

}  // namespace

extern "C" {

HC_API int hc_rotate_heads(int64_t T, int64_t heads, int64_t dim, int type, const void* x, int64_t x_row, int64_t x_head,
                           const int32_t* positions, const float* frequencies, int64_t rotated, int interleaved, const float* weight,
                           float eps, void* out, int64_t out_row, int64_t out_head, void* stream)
{
    if (T < 1 || heads < 1 || dim < 1 || (type != HC_BF16 && type != HC_FP16) || (frequencies && (!positions || rotated < 1 || rotated > dim)) || !(eps >= 0.0f))
        return HC_ERR_ARG;
    int st = check_heads(x, x_row, x_head, heads, dim);
    if (st == HC_OK)
        st = check_heads(out, out_row, out_head, heads, dim);
    if (st != HC_OK)
        return st;
    if (T > kMost || heads > 65536 || dim > HC_MAX_HEAD || dim % 8 || (frequencies && rotated % 8) ||
        !fits(rotate_blocks(T, heads, (int)dim), kRotateThreads))
        return HC_ERR_SIZE;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(positions, 4) || !aligned(frequencies, 4) || !aligned(weight, 4))
        return HC_ERR_ALIGN;
    st = check_device();
    if (st != HC_OK)
        return st;
    RotateArgs a{};
    a.T = (int)T;
    a.dim = (int)dim;
    a.rotated = frequencies ? (int)rotated : 0;
    a.interleaved = interleaved != 0;
    a.q = HeadsArgs{static_cast<const char*>(x), 2 * x_row, 2 * x_head};
    a.q_heads = (int)heads;
    a.out = static_cast<char*>(out);
    a.out_row = 2 * out_row;
    a.out_head = 2 * out_head;
    a.positions = frequencies ? positions : nullptr;
    a.frequencies = frequencies;
    a.q_weight = weight;
    a.eps = eps;
    return done(launch_rotate(a, type == HC_FP16, false, static_cast<hipStream_t>(stream)));
}

HC_API int hc_append_heads(int64_t T, int64_t q_heads, const void* q, int64_t q_row, int64_t q_head, const void* k, int64_t k_row,
                           int64_t k_head, const void* v, int64_t v_row, int64_t v_head, const hc_cache* cache, const hc_batch* batch,
                           const int32_t* positions, const float* frequencies, int64_t rotated, int interleaved, const float* q_weight,
                           const float* k_weight, float eps, void* out, int64_t out_row, int64_t out_head, void* stream)
{
    int st = check_cache(cache);
    if (st == HC_OK)
        st = check_batch(batch);
    if (st != HC_OK)
        return st;
    if (T < 1 || q_heads < 0 || (frequencies && (rotated < 1 || rotated > cache->dim)) || !(eps >= 0.0f))
        return HC_ERR_ARG;
    if (q_heads) {
        st = check_heads(q, q_row, q_head, q_heads, cache->dim);
        if (st == HC_OK)
            st = check_heads(out, out_row, out_head, q_heads, cache->dim);
    }
    if (st == HC_OK)
        st = check_heads(k, k_row, k_head, cache->heads, cache->dim);
    if (st == HC_OK)
        st = check_heads(v, v_row, v_head, cache->heads, cache->dim);
    if (st != HC_OK)
        return st;
    if (T > kMost || q_heads > 65536 || (frequencies && rotated % 8) ||
        !fits(rotate_blocks(T, q_heads + 2 * cache->heads, (int)cache->dim), kRotateThreads))
        return HC_ERR_SIZE;
    if ((q_heads && !(aligned(q, 16) && aligned(out, 16))) || !aligned(k, 16) || !aligned(v, 16) || !aligned(cache->keys, 16) ||
        !aligned(cache->values, 16) || !batch_aligned(batch) || !aligned(positions, 4) || !aligned(frequencies, 4) || !aligned(q_weight, 4) ||
        !aligned(k_weight, 4))
        return HC_ERR_ALIGN;
    st = check_device();
    if (st != HC_OK)
        return st;
    RotateArgs a{};
    a.T = (int)T;
    a.dim = (int)cache->dim;
    a.rotated = frequencies ? (int)rotated : 0;
    a.interleaved = interleaved != 0;
    a.q = HeadsArgs{static_cast<const char*>(q), 2 * q_row, 2 * q_head};
    a.k = HeadsArgs{static_cast<const char*>(k), 2 * k_row, 2 * k_head};
    a.v = HeadsArgs{static_cast<const char*>(v), 2 * v_row, 2 * v_head};
    a.q_heads = (int)q_heads;
    a.out = static_cast<char*>(out);
    a.out_row = 2 * out_row;
    a.out_head = 2 * out_head;
    a.positions = positions;
    a.frequencies = frequencies;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.cache = cache_of(cache);
    a.batch = batch_of(batch);
    return done(launch_rotate(a, cache->type == HC_FP16, true, static_cast<hipStream_t>(stream)));
}

HC_API int64_t hc_attend_work(int64_t T, int64_t q_heads, int64_t heads, int64_t dim, int64_t requests, int64_t groups)
{
    if (!sizes_fit(T, q_heads, heads, requests, groups) || groups < 0 || dim < 1 || dim > HC_MAX_HEAD || dim % 8)
        return 0;
    const Choice to = choose(T * (q_heads / heads), dim, requests, groups);
    return scratch_of(T, q_heads, to.rows, padded((int)dim), requests + groups, to.tiles, groups > 0).bytes;
}

HC_API int hc_attend(int64_t T, int64_t q_heads, const void* q, int64_t q_row, int64_t q_head, const hc_cache* cache, const hc_batch* batch,
                     float scale, float cap, const float* slopes, const int32_t* first, const int32_t* last, void* out, int64_t out_row,
                     int64_t out_head, void* work, int64_t work_bytes, void* stream)
{
    return attend(T, q_heads, q, q_row, q_head, cache, batch, nullptr, scale, cap, slopes, first, last, out, out_row, out_head, work,
                  work_bytes, stream);
}

HC_API int hc_attend_shared(int64_t T, int64_t q_heads, const void* q, int64_t q_row, int64_t q_head, const hc_cache* cache,
                            const hc_batch* batch, const hc_prefix* prefix, float scale, float cap, const float* slopes, const int32_t* first,
                            const int32_t* last, void* out, int64_t out_row, int64_t out_head, void* work, int64_t work_bytes, void* stream)
{
    const int st = check_prefix(prefix);
    if (st != HC_OK)
        return st;
    return attend(T, q_heads, q, q_row, q_head, cache, batch, prefix, scale, cap, slopes, first, last, out, out_row, out_head, work,
                  work_bytes, stream);
}

HC_API const char* hc_attn_status_string(int status)
{
    switch (status) {
    case HC_OK: return "ok";
    case HC_ERR_ARG: return "invalid argument (a size below 1, a required pointer that is NULL, a type that the call does not take, "
                            "a stride shorter than what it steps over, query heads that are no multiple of the cache's, more "
                            "rotated columns than a head has, or a scale, cap or eps that is no number of its range)";
    case HC_ERR_ALIGN: return "a pointer is not aligned (16 bytes for heads, cache and work, its own type for the others)";
    case HC_ERR_DEVICE: return "the current device is not a gfx950 (MI355X) GPU or could not be queried";
    case HC_ERR_LAUNCH: return "a kernel launch failed";
    case HC_ERR_SIZE: return "a size is outside its limits (columns, strides and rotated columns are multiples of 8, heads of up to 256 "
                             "columns, pages of a power of two from 16 to 65536 positions, 2048 requests, 262144 rows, fewer than 2^32 "
                             "threads, up to 2^31 - 65536 positions of a sequence, fewer than 2^31 positions in all tiles' tables over 32), "
                             "or work_bytes is too small";
    default: return "unknown status";
    }
}

HC_API int hc_attn_last_hip_error(void)
{
    return g_last_hip_error;
}

}  // extern "C"
