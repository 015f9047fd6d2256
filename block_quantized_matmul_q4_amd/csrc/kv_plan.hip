// Planning one serving step of the paged KV cache: pages taken and given
// back, first rows, slots and positions.
//
// Per request three sums over the requests before it are needed: new rows
// (grow), pages asked for (ask) and pages given back (back). One scan gives
// all three, because what is refused forms a suffix: the sum of asks only
// grows, so the granted asks are those up to the first that does not fit and
// the pages of a granted request start at (sum of all asks before it); and a
// request whose rows end past T has only such requests after it that grow.
// A request that gives pages back asks for none, so nothing can refuse it.
//
// The work is a few bytes per request, page and token: latency is all there
// is to it. One workgroup scans the requests, 1024 at a time: 8 requests that
// decode 5 us, 512 that decode, grow by chunks of up to 500 tokens or end 10.6 us,
// and 4 us for a second launch that fills more than 4096 rows (8356 rows filled by
// the one workgroup: 18.8 us in all; an empty launch takes 1.7 us).
#include "qmm_kv.h"

namespace qmm {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;

struct Sums {
    int64_t grow, ask, back;
};

__device__ __forceinline__ int32_t capped(int64_t v)
{
    return (int32_t)(v < INT32_MAX ? v : INT32_MAX);
}

__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b)
{
    return {a.grow + b.grow, a.ask + b.ask, a.back + b.back};
}

// Inclusive sums over the workgroup's threads; total: over all of them.
__device__ Sums block_scan(Sums v, Sums *wave_sums, Sums &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const Sums o = {__shfl_up(v.grow, d), __shfl_up(v.ask, d), __shfl_up(v.back, d)};
        if (lane >= d) v = v + o;
    }
    if (lane == 63) wave_sums[wave] = v;
    __syncthreads();
    if (wave == 0) {                    // the waves' sums, inclusive
        Sums s = {};
        if (lane < kWaves) s = wave_sums[lane];
#pragma unroll
        for (int d = 1; d < kWaves; d *= 2) {
            const Sums o = {__shfl_up(s.grow, d), __shfl_up(s.ask, d), __shfl_up(s.back, d)};
            if (lane >= d) s = s + o;
        }
        if (lane < kWaves) wave_sums[lane] = s;
    }
    __syncthreads();
    total = wave_sums[kWaves - 1];
    if (wave > 0) v = v + wave_sums[wave - 1];
    __syncthreads();
    return v;
}

// First index i < n with a[i] > x (a non-decreasing, a[n - 1] > x).
template <typename T>
__device__ __forceinline__ int upper(const T *a, int n, T x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] > x) hi = mid; else lo = mid + 1;
    }
    return lo;
}

struct Request {
    int32_t lens;
    int32_t have;           // pages before the step
    int32_t need;
    int32_t granted;
};

// FILL: also the slots and positions (few tokens); else a second launch.
template <bool FILL>
__global__ void __launch_bounds__(kThreads) plan_kernel(KvPlanArgs a, int shift)
{
    __shared__ Sums wave_sums[kWaves];
    __shared__ Request req[kThreads];
    __shared__ int32_t take_end[kThreads], back_end[kThreads], row_end[kThreads];
    __shared__ int64_t taken_all;
    const int tid = threadIdx.x;
    const int size = a.ring_size;
    const int64_t pool_head = a.pool[0], pool_count = a.pool[1];
    const int head = pool_head < 0 || pool_head >= size ? 0 : (int)pool_head;
    const int count = (int)(pool_count < 0 ? 0 : pool_count > size ? size : pool_count);
    const int64_t limit = (int64_t)a.width << shift;
    Sums carry = {};
    int64_t taken = 0;
    if (tid == 0) a.cu[0] = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + tid;
        const bool on = b < a.batch;
        const int64_t want = on ? a.want[b] : 0, lens = on ? a.lens[b] : 0;
        const bool bad = lens < 0 || lens > limit || want < 0 || want > limit;
        const int mask = (1 << shift) - 1;
        const int have = bad ? 0 : (int)((lens + mask) >> shift);
        const int need = bad ? 0 : (int)((want + mask) >> shift);
        const int grow = !bad && want > lens ? (int)(want - lens) : 0;
        const int ask = need > have ? need - have : 0;
        const int back = need < have ? have - need : 0;
        Sums total;
        const Sums upto = carry + block_scan({grow, ask, back}, wave_sums, total);
        const bool late = grow > 0 && upto.grow > a.tokens;
        const bool lacking = !late && ask > 0 && upto.ask > count;
        const bool granted = !(bad || late || lacking);
        const int take = granted ? ask : 0;
        if (on) {
            a.cu[b + 1] = capped(upto.grow);
            a.new_lens[b] = granted ? (int)want : (int)lens;
            a.status[b] = bad ? 2 : late ? 3 : lacking ? 1 : 0;
        }
        // ends of this chunk's ranges; refused asks take nothing, and only
        // refused ones follow
        req[tid] = {(int32_t)lens, have, need, granted};
        if (tid == 0) taken_all = taken;
        __syncthreads();
        if (take > 0) atomicMax((unsigned long long *)&taken_all, (unsigned long long)upto.ask);
        __syncthreads();
        const int64_t taken_now = taken_all;
        const int64_t upto_taken = upto.ask < taken_now ? upto.ask : taken_now;
        const unsigned takes = (unsigned)(taken_now - taken);    // at most count
        take_end[tid] = (int32_t)(upto_taken - taken);
        back_end[tid] = capped(upto.back - carry.back);
        row_end[tid] = capped(upto.grow - carry.grow);
        __syncthreads();
        for (unsigned i = tid; i < takes; i += kThreads) {
            const int r = upper(take_end, kThreads, (int)i);
            const int nth = (int)i - (r ? take_end[r - 1] : 0);
            a.table[(int64_t)(b0 + r) * a.width + req[r].have + nth] =
                a.ring[kv_ring_place(head, taken + i, size)];
        }
        // places of the ring that are free (the pages taken are still in theirs)
        const unsigned backs = kv_fitting(total.back, size - count - carry.back);
        for (unsigned i = tid; i < backs; i += kThreads) {
            const int r = upper(back_end, kThreads, (int)i);
            const int nth = (int)i - (r ? back_end[r - 1] : 0);
            a.ring[kv_ring_place(head, count + carry.back + i, size)] =
                a.table[(int64_t)(b0 + r) * a.width + req[r].need + nth];
        }
        if constexpr (FILL) {
            const int rows = kv_fitting(total.grow, a.tokens - carry.grow);
            for (int i = tid; i < rows; i += kThreads) {
                const int row = (int)carry.grow + i;    // below T: there are rows left
                const int r = upper(row_end, kThreads, i);
                const Request q = req[r];
                int64_t slot = -1;
                int pos = -1;
                if (q.granted) {
                    pos = q.lens + i - (r ? row_end[r - 1] : 0);
                    const int at = pos >> shift;
                    const int page =
                        at < q.have
                            ? a.table[(int64_t)(b0 + r) * a.width + at]
                            : a.ring[kv_ring_place(
                                  head, taken + (r ? take_end[r - 1] : 0) + at - q.have, size)];
                    slot = (int64_t)page * (1 << shift) + (pos & mask);
                }
                a.slots[row] = slot;
                if (a.positions) a.positions[row] = pos;
            }
        }
        carry = carry + total;
        taken = taken_now;
        __syncthreads();
    }
    if constexpr (FILL)
        for (int64_t row = carry.grow + tid; row < a.tokens; row += kThreads) {
            a.slots[row] = -1;
            if (a.positions) a.positions[row] = -1;
        }
    if (tid == 0) {
        const int64_t room = size - count;
        a.new_pool[0] = kv_ring_place(head, taken, size);
        a.new_pool[1] = count - taken + (carry.back < room ? carry.back : room);
    }
}

// Slots and positions from the first kernel's outputs, one thread per row.
__global__ void __launch_bounds__(256) fill_kernel(KvPlanArgs a, int shift)
{
    const int row = blockIdx.x * 256 + threadIdx.x;
    if (row >= a.tokens) return;
    int64_t slot = -1;
    int pos = -1;
    if (row < a.cu[a.batch]) {
        const int r = upper(a.cu + 1, a.batch, row);
        if (a.status[r] == 0) {
            pos = a.want[r] - (a.cu[r + 1] - row);
            const int page = a.table[(int64_t)r * a.width + (pos >> shift)];
            slot = (int64_t)page * (1 << shift) + (pos & ((1 << shift) - 1));
        }
    }
    a.slots[row] = slot;
    if (a.positions) a.positions[row] = pos;
}

}  // namespace

hipError_t launch_kv_plan(const KvPlanArgs &a, hipStream_t stream)
{
    const int shift = __builtin_ctz(a.page_size);
    if (a.tokens <= 4096) {
        plan_kernel<true><<<1, kThreads, 0, stream>>>(a, shift);
        return hipGetLastError();
    }
    plan_kernel<false><<<1, kThreads, 0, stream>>>(a, shift);
    if (hipError_t err = hipGetLastError()) return err;
    fill_kernel<<<kv_groups(a.tokens, 256), 256, 0, stream>>>(a, shift);
    return hipGetLastError();
}

}  // namespace qmm
