// C-ABI layer of the paged Q4_0 KV cache and its attention: argument
// validation on the host, before any HIP call, and dispatch to the kernels.
#include <climits>
#include <cmath>

#include "../../include/qmm.h"
#include "qmm_kv.h"

namespace {

using qmm::fail;

constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxGroup = 64;
constexpr int64_t kMaxBatch = 1 << 20;

bool misaligned(const void *p, uintptr_t to) { return (uintptr_t)p % to != 0; }

bool overlaps(const void *a, uint64_t a_len, const void *b, uint64_t b_len)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + b_len && y < x + a_len;
}

bool page_size_ok(int64_t p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }

bool head_dim_ok(int64_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

uint64_t cache_bytes(const qmm::KvCache &c)
{
    return (uint64_t)c.num_pages * (uint64_t)c.kv_heads *
           (uint64_t)qmm::kv_chunk_bytes(c.page_size, c.head_dim);
}

int check_cache(const char *fn, const qmm_kv_cache *c, qmm::KvCache *out, bool need_pages)
{
    if (!c) return fail(QMM_EINVAL, "%s: null pointer (cache)", fn);
    if (need_pages && !c->pages) return fail(QMM_EINVAL, "%s: null pointer (cache->pages)", fn);
    if (!page_size_ok(c->page_size))
        return fail(QMM_EUNSUPPORTED, "%s: page_size=%lld unsupported (16, 32, 64, 128 or 256)",
                    fn, (long long)c->page_size);
    if (!head_dim_ok(c->head_dim))
        return fail(QMM_EUNSUPPORTED,
                    "%s: head_dim=%lld unsupported (64, 96, 128, 192 or 256)", fn,
                    (long long)c->head_dim);
    if (c->kv_heads < 1 || c->kv_heads > kMaxHeads || c->num_pages < 1 ||
        c->num_pages > INT_MAX)
        return fail(QMM_EINVAL,
                    "%s: need 1 <= kv_heads <= %lld and 1 <= num_pages < 2^31 (%lld, %lld)", fn,
                    (long long)kMaxHeads, (long long)c->kv_heads, (long long)c->num_pages);
    if (need_pages && misaligned(c->pages, 16))
        return fail(QMM_EALIGN, "%s: misaligned pointer (the cache needs 16-byte alignment)", fn);
    *out = {(uint8_t *)c->pages, (int)c->num_pages, (int)c->page_size, (int)c->kv_heads,
            (int)c->head_dim};
    return QMM_OK;
}

// cols: values of a row (0: none to check); the launches need T * cols < 2^40.
int check_rows(const char *fn, int64_t T, int64_t cols = 0)
{
    if (T < 0 || T > INT_MAX)
        return fail(QMM_EINVAL, "%s: need 0 <= T < 2^31 (T=%lld)", fn, (long long)T);
    if (cols && T >= ((int64_t)1 << 40) / cols)
        return fail(QMM_EUNSUPPORTED, "%s: T=%lld rows of %lld values pass 2^40", fn,
                    (long long)T, (long long)cols);
    return QMM_OK;
}

// Bytes from the first to the last value of T rows of `cols` floats.
uint64_t rows_bytes(int64_t T, int64_t stride, int64_t cols)
{
    return ((uint64_t)(T - 1) * (uint64_t)stride + (uint64_t)cols) * 4u;
}

int check_stride(const char *fn, const char *name, int64_t T, int64_t stride, int64_t cols)
{
    if (stride < cols || stride % 4 || stride > INT64_MAX / 8 / (T > 0 ? T : 1))
        return fail(QMM_EINVAL,
                    "%s: %s=%lld (need a multiple of 4, at least %lld, without overflow)", fn,
                    name, (long long)stride, (long long)cols);
    return QMM_OK;
}

int finish(const char *fn, hipError_t err)
{
    if (err != hipSuccess)
        return fail(QMM_EHIP, "%s: launch failed: %s", fn, hipGetErrorString(err));
    return QMM_OK;
}

int check_attend_sizes(const char *fn, const qmm::KvCache &c, int64_t T, int64_t B,
                       int64_t q_heads, int64_t max_q, int64_t max_len, int64_t window)
{
    if (int st = check_rows(fn, T)) return st;
    if (B < 1 || B > kMaxBatch)
        return fail(QMM_EINVAL, "%s: need 1 <= B <= 2^20 (B=%lld)", fn, (long long)B);
    if (q_heads < 1 || q_heads % c.kv_heads || q_heads / c.kv_heads > kMaxGroup)
        return fail(QMM_EINVAL,
                    "%s: q_heads=%lld must be a multiple of kv_heads=%d, at most %lld times it",
                    fn, (long long)q_heads, c.kv_heads, (long long)kMaxGroup);
    if (max_q < 1 || max_q > INT_MAX || max_len < 1 || max_len > INT_MAX)
        return fail(QMM_EINVAL,
                    "%s: max_q and max_len must be at least 1 and below 2^31 (%lld, %lld)", fn,
                    (long long)max_q, (long long)max_len);
    if (window < 0 || window > INT_MAX)
        return fail(QMM_EINVAL, "%s: need 0 <= window < 2^31 (window=%lld)", fn,
                    (long long)window);
    // the row index of the (T, q_heads) grid and the packed rows of a request
    if (T > INT_MAX / q_heads || max_q > INT_MAX / kMaxGroup)
        return fail(QMM_EUNSUPPORTED, "%s: T * q_heads or 64 * max_q passes 2^31", fn);
    return QMM_OK;
}

uint64_t workspace_bytes_of(const qmm::AttendShape &s, int64_t rows, int head_dim)
{
    return s.splits > 1 ? (uint64_t)s.splits * (uint64_t)rows * (uint64_t)(head_dim + 2) * 4u : 0;
}

}  // namespace

extern "C" {

QMM_API int64_t qmm_kv_chunk_bytes_q4_0(int64_t page_size, int64_t head_dim)
{
    if (!page_size_ok(page_size) || !head_dim_ok(head_dim)) return 0;
    return qmm::kv_chunk_bytes((int)page_size, (int)head_dim);
}

QMM_API int qmm_kv_plan(const int32_t *want, const int32_t *lens, int32_t *table, int32_t *ring,
                        const int64_t *pool, int32_t *new_lens, int64_t *new_pool, int32_t *cu,
                        int64_t *slots, int32_t *positions, int32_t *status, int64_t B,
                        int64_t T, int64_t width, int64_t ring_size, int64_t page_size,
                        hipStream_t stream)
{
    const char *fn = "qmm_kv_plan";
    if (!want || !lens || !table || !ring || !pool || !new_lens || !new_pool || !cu || !status ||
        (T > 0 && !slots))
        return fail(QMM_EINVAL, "%s: null pointer", fn);
    if (int st = check_rows(fn, T)) return st;
    if (B < 1 || B > kMaxBatch)
        return fail(QMM_EINVAL, "%s: need 1 <= B <= 2^20 (B=%lld)", fn, (long long)B);
    if (!page_size_ok(page_size))
        return fail(QMM_EUNSUPPORTED, "%s: page_size=%lld unsupported (16, 32, 64, 128 or 256)",
                    fn, (long long)page_size);
    if (width < 1 || width > INT_MAX / page_size)
        return fail(QMM_EINVAL, "%s: need width >= 1 and width * page_size < 2^31 (width=%lld)",
                    fn, (long long)width);
    if (ring_size < 1 || ring_size > INT_MAX)
        return fail(QMM_EINVAL, "%s: need 1 <= ring_size < 2^31 (ring_size=%lld)", fn,
                    (long long)ring_size);
    for (const void *p : {(const void *)want, (const void *)lens, (const void *)table,
                          (const void *)ring, (const void *)new_lens, (const void *)cu,
                          (const void *)positions, (const void *)status})
        if (misaligned(p, 4))
            return fail(QMM_EALIGN, "%s: misaligned pointer (int32 arrays need 4 bytes)", fn);
    for (const void *p : {(const void *)pool, (const void *)new_pool, (const void *)slots})
        if (misaligned(p, 8))
            return fail(QMM_EALIGN, "%s: misaligned pointer (int64 arrays need 8 bytes)", fn);
    enum { kWant, kLens, kPool, kTable, kRing, kNewLens, kNewPool, kCu, kSlots, kPositions, kStatus };
    const struct { const void *p; uint64_t n; } parts[] = {
        {want, 4u * (uint64_t)B},
        {lens, 4u * (uint64_t)B},
        {pool, 16},
        {table, 4u * (uint64_t)B * (uint64_t)width},
        {ring, 4u * (uint64_t)ring_size},
        {new_lens, 4u * (uint64_t)B},
        {new_pool, 16},
        {cu, 4u * ((uint64_t)B + 1)},
        {slots, 8u * (uint64_t)T},
        {positions, positions ? 4u * (uint64_t)T : 0},
        {status, 4u * (uint64_t)B},
    };
    for (int x = kWant; x <= kStatus; ++x)
        for (int y = x + 1; y <= kStatus; ++y) {
            if (y < kTable || !parts[x].n || !parts[y].n) continue;     // two inputs, or nothing
            // in place, and only these arrays (with want = lens nothing changes)
            const bool twins = (x == kLens && y == kNewLens) || (x == kPool && y == kNewPool) ||
                               (x == kWant && y == kNewLens && want == lens);
            if (twins && parts[x].p == parts[y].p) continue;
            if (overlaps(parts[x].p, parts[x].n, parts[y].p, parts[y].n))
                return fail(QMM_EINVAL, "%s: an output overlaps another array", fn);
        }
    return finish(fn, qmm::launch_kv_plan({want, lens, table, ring, pool, new_lens, new_pool, cu,
                                           slots, positions, status, (int)B, (int)T, (int)width,
                                           (int)ring_size, (int)page_size},
                                          stream));
}

QMM_API int qmm_kv_append_q4_0(const float *k, int64_t k_stride, const float *v,
                               int64_t v_stride, const qmm_kv_cache *cache,
                               const int64_t *slots, int64_t T, hipStream_t stream)
{
    const char *fn = "qmm_kv_append_q4_0";
    qmm::KvCache c;
    if (int st = check_cache(fn, cache, &c, T != 0)) return st;
    const int64_t cols = (int64_t)c.kv_heads * c.head_dim;
    if (int st = check_rows(fn, T, cols)) return st;
    if (int st = check_stride(fn, "k_stride", T, k_stride, cols)) return st;
    if (int st = check_stride(fn, "v_stride", T, v_stride, cols)) return st;
    if (T == 0) return QMM_OK;
    if (!k || !v || !slots) return fail(QMM_EINVAL, "%s: null pointer", fn);
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 8))
        return fail(QMM_EALIGN,
                    "%s: misaligned pointer (k and v need 16-byte, slots 8-byte alignment)", fn);
    const uint64_t n = cache_bytes(c);
    if (overlaps(c.pages, n, k, rows_bytes(T, k_stride, cols)) ||
        overlaps(c.pages, n, v, rows_bytes(T, v_stride, cols)) ||
        overlaps(c.pages, n, slots, 8u * (uint64_t)T))
        return fail(QMM_EINVAL, "%s: the cache overlaps k, v or slots", fn);
    return finish(fn, qmm::launch_kv_append(c, k, k_stride, v, v_stride, slots, (int)T, stream));
}

QMM_API int qmm_kv_read_q4_0(const qmm_kv_cache *cache, const int64_t *slots, float *k,
                             float *v, int64_t T, hipStream_t stream)
{
    const char *fn = "qmm_kv_read_q4_0";
    qmm::KvCache c;
    if (int st = check_cache(fn, cache, &c, T != 0)) return st;
    const int64_t cols = (int64_t)c.kv_heads * c.head_dim;
    if (int st = check_rows(fn, T, cols)) return st;
    if (T == 0) return QMM_OK;
    if (!k || !v || !slots) return fail(QMM_EINVAL, "%s: null pointer", fn);
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(slots, 8))
        return fail(QMM_EALIGN,
                    "%s: misaligned pointer (k and v need 16-byte, slots 8-byte alignment)", fn);
    const uint64_t n = cache_bytes(c), rows = rows_bytes(T, cols, cols);
    if (overlaps(k, rows, c.pages, n) || overlaps(v, rows, c.pages, n) ||
        overlaps(k, rows, v, rows) || overlaps(k, rows, slots, 8u * (uint64_t)T) ||
        overlaps(v, rows, slots, 8u * (uint64_t)T))
        return fail(QMM_EINVAL, "%s: an output overlaps another array", fn);
    return finish(fn, qmm::launch_kv_read(c, slots, k, v, (int)T, stream));
}

QMM_API int64_t qmm_attend_q4_0_workspace(const qmm_kv_cache *cache, int64_t T, int64_t B,
                                          int64_t q_heads, int64_t max_q, int64_t max_len,
                                          int64_t window)
{
    const char *fn = "qmm_attend_q4_0_workspace";
    qmm::KvCache c;
    if (int st = check_cache(fn, cache, &c, false)) return -st;
    if (int st = check_attend_sizes(fn, c, T, B, q_heads, max_q, max_len, window)) return -st;
    const auto s = qmm::attend_shape((int)T, (int)B, c.kv_heads, (int)(q_heads / c.kv_heads),
                                     c.head_dim, max_q, max_len, window);
    return (int64_t)workspace_bytes_of(s, T * q_heads, c.head_dim);
}

QMM_API int qmm_attend_q4_0(const float *q, int64_t q_stride, const qmm_kv_cache *cache,
                            const int32_t *table, int64_t width, const int32_t *lens,
                            const int32_t *cu, float *out, float *lse, void *workspace,
                            int64_t workspace_bytes, int64_t T, int64_t B, int64_t q_heads,
                            int64_t max_q, int64_t max_len, float scale, int causal,
                            int64_t window, hipStream_t stream)
{
    const char *fn = "qmm_attend_q4_0";
    qmm::KvCache c;
    if (int st = check_cache(fn, cache, &c, T != 0)) return st;
    if (int st = check_attend_sizes(fn, c, T, B, q_heads, max_q, max_len, window)) return st;
    const int64_t cols = q_heads * c.head_dim;
    if (int st = check_stride(fn, "q_stride", T, q_stride, cols)) return st;
    if (width < 1 || width > INT_MAX / c.page_size)
        return fail(QMM_EINVAL, "%s: need width >= 1 and width * page_size < 2^31 (width=%lld)",
                    fn, (long long)width);
    if (!std::isfinite(scale)) return fail(QMM_EINVAL, "%s: scale must be finite", fn);
    if (causal != 0 && causal != 1)
        return fail(QMM_EINVAL, "%s: causal must be 0 or 1 (%d)", fn, causal);
    if (T == 0) return QMM_OK;
    if (!q || !table || !lens || !cu || !out) return fail(QMM_EINVAL, "%s: null pointer", fn);
    if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lse, 4) || misaligned(table, 4) ||
        misaligned(lens, 4) || misaligned(cu, 4) || misaligned(workspace, 16))
        return fail(QMM_EALIGN,
                    "%s: misaligned pointer (q, out and workspace need 16-byte, the others "
                    "4-byte alignment)", fn);
    const auto s = qmm::attend_shape((int)T, (int)B, c.kv_heads, (int)(q_heads / c.kv_heads),
                                     c.head_dim, max_q, max_len, window);
    const uint64_t need = workspace_bytes_of(s, T * q_heads, c.head_dim);
    if (need && (!workspace || workspace_bytes < 0 || (uint64_t)workspace_bytes < need))
        return fail(QMM_EINVAL, "%s: the workspace needs %llu bytes (%lld given)", fn,
                    (unsigned long long)need, workspace ? (long long)workspace_bytes : 0LL);
    const uint64_t out_len = rows_bytes(T, cols, cols);
    const uint64_t lse_len = lse ? (uint64_t)(T * q_heads) * 4u : 0;
    const struct { const void *p; uint64_t n; bool out; } parts[] = {
        {q, rows_bytes(T, q_stride, cols), false},
        {c.pages, cache_bytes(c), false},
        {table, 4u * (uint64_t)B * (uint64_t)width, false},
        {lens, 4u * (uint64_t)B, false},
        {cu, 4u * ((uint64_t)B + 1), false},
        {out, out_len, true},
        {lse, lse_len, true},
        {workspace, need, true},
    };
    for (const auto &x : parts)
        for (const auto &y : parts)
            if (&x < &y && (x.out || y.out) && x.n && y.n && overlaps(x.p, x.n, y.p, y.n))
                return fail(QMM_EINVAL, "%s: out, lse or the workspace overlaps another array",
                            fn);
    qmm::AttendArgs a = {};
    a.q = q;
    a.q_stride = q_stride;
    a.cache = c;
    a.table = table;
    a.width = (int)width;
    a.lens = lens;
    a.cu = cu;
    a.out = out;
    a.lse = lse;
    a.part_o = (float *)workspace;
    a.part_ml = need ? (float *)workspace + (uint64_t)s.splits * (uint64_t)(T * cols) : nullptr;
    a.tokens = (int)T;
    a.batch = (int)B;
    a.q_heads = (int)q_heads;
    a.group = (int)(q_heads / c.kv_heads);
    a.tiles = s.tiles;
    a.tile_rows = s.tile_rows;
    a.splits = s.splits;
    a.min_part = s.min_part;
    a.waves = s.waves;
    a.few = s.few;
    a.scale = scale;
    a.causal = causal;
    a.window = (int)window;
    return finish(fn, qmm::launch_attend(a, stream));
}

}  // extern "C"
