// Internal declarations of the paged Q4_0 KV cache and its attention, shared
// by their C-ABI layer (qmm_kv_api.hip) and kernels. Not installed; the
// public interface is include/qmm.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {

// Sets the thread's error string (qmm_last_error) and returns status.
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

// A cache whose geometry the C-ABI layer has checked.
struct KvCache {
    uint8_t *pages;
    int num_pages;
    int page_size;      // 16 .. 256, a power of two
    int kv_heads;
    int head_dim;       // 64, 96, 128, 192 or 256
};

// One (page, head) chunk: byte offsets of its planes. Codes take D / 2 bytes
// per token, scales D / 16; the K half and the V half have the same size.
__host__ __device__ constexpr int64_t kv_chunk_bytes(int page_size, int head_dim)
{
    return (int64_t)page_size * head_dim * 9 / 8;
}

// Integers that live on the device are trusted nowhere: every page, slot and
// row that a kernel follows comes out of the functions below.

__host__ __device__ inline bool kv_slot_ok(const KvCache &c, int64_t slot)
{
    return slot >= 0 && slot < (int64_t)c.num_pages * c.page_size;
}

// A request's rows of the batch and its tokens in the cache, inside the T rows
// and the table whatever cu and lens hold.
struct KvRequest {
    int q0, count, len;
};

__host__ __device__ inline KvRequest kv_request(const int32_t *cu, const int32_t *lens, int b,
                                                int tokens, int width, int page_shift)
{
    const int first = cu[b] < 0 ? 0 : cu[b] < tokens ? cu[b] : tokens;
    const int end = cu[b + 1] < first ? first : cu[b + 1] < tokens ? cu[b + 1] : tokens;
    const int64_t most = (int64_t)width << page_shift;      // below 2^31
    const int64_t len = lens[b] < 0 ? 0 : lens[b];
    return {first, end - first, (int)(len < most ? len : most)};
}

// The table entry of token t >= 0, inside a row whose last entry is `last`. What
// it holds is a page only if the cache has it; past a request's end it may be any
// page, and the tokens there are hidden by their places.
__host__ __device__ inline int kv_entry(int t, int page_shift, int last)
{
    const int at = t >> page_shift;
    return at < last ? at : last;
}

__host__ __device__ inline bool kv_page_exists(int page, int num_pages)
{
    return (unsigned)page < (unsigned)num_pages;
}

// As many of n rows or pages as there is room for. Both are sums over lengths
// that the device holds, up to 2^52, and room is negative once more has been
// asked for than there is; only what is left of them is narrowed.
__host__ __device__ inline int kv_fitting(int64_t n, int64_t room)
{
    const int64_t most = n < room ? n : room;
    return (int)(most < 0 ? 0 : most < INT32_MAX ? most : INT32_MAX);
}

// The place `after` entries behind a ring's head, head and after at most `size`
// (together past 32 bits in a ring of more than 2^30).
__host__ __device__ inline int kv_ring_place(int head, int64_t after, int size)
{
    const int64_t at = head + after;
    return (int)(at >= size ? at - size : at);
}

// Workgroups of `threads` for n items, n up to 2^31 - 1.
__host__ __device__ inline unsigned kv_groups(int n, int threads)
{
    return ((unsigned)n + (unsigned)threads - 1) / (unsigned)threads;
}

struct KvPlanArgs {
    const int32_t *want, *lens;
    int32_t *table, *ring;
    const int64_t *pool;
    int32_t *new_lens;
    int64_t *new_pool;
    int32_t *cu;
    int64_t *slots;
    int32_t *positions;     // may be null
    int32_t *status;
    int batch, tokens, width, ring_size, page_size;
};

struct AttendArgs {
    const float *q;
    int64_t q_stride;
    KvCache cache;
    const int32_t *table;
    int width;              // table entries per request
    const int32_t *lens, *cu;
    float *out, *lse;       // lse may be null
    float *part_o;          // [splits][tokens * q_heads][head_dim], splits > 1
    float *part_ml;         // [splits][tokens * q_heads][2]
    int tokens, batch, q_heads, group;
    int first, requests;    // those of this launch
    int tiles;              // row tiles per (request, KV head) in the grid
    int tile_rows;          // rows of such a tile
    int splits;             // parts of a request's keys
    int min_part;           // least keys of a part
    int waves;              // of a workgroup of the kernel for few rows, 4 or 8
    bool few;               // attend_few_kernel, with tiles of 8 or 16 rows
    float scale;
    int causal;
    int window;             // 0: none
};

// How an attention call is launched, from the sizes that the host knows.
struct AttendShape {
    int tiles, splits, min_part, tile_rows, waves;
    bool few;               // up to 16 rows: attend_few_kernel
};
AttendShape attend_shape(int tokens, int batch, int kv_heads, int group, int head_dim,
                         int64_t max_q, int64_t max_len, int64_t window);

// Launchers; arguments are validated by the C-ABI layer.
hipError_t launch_kv_plan(const KvPlanArgs &a, hipStream_t stream);
hipError_t launch_kv_append(const KvCache &c, const float *k, int64_t k_stride, const float *v,
                            int64_t v_stride, const int64_t *slots, int tokens,
                            hipStream_t stream);
hipError_t launch_kv_read(const KvCache &c, const int64_t *slots, float *k, float *v, int tokens,
                          hipStream_t stream);
hipError_t launch_attend(const AttendArgs &a, hipStream_t stream);
// ... its kernel for tiles of 16 rows, or of 32 up to 128 dims (head_dim is one of
// those above)
void launch_attend_many(const AttendArgs &a, unsigned grid, hipStream_t stream);

}  // namespace qmm
