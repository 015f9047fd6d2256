// Which rows and keys the attention kernels' workgroups take: arithmetic on a
// request's integers, for the device and for checks of it on the host.
#pragma once

#include "qmm_kv.h"

namespace qmm {

constexpr int kKeys = 32;           // keys per wave and step

// The rows of a tile and the keys they see. Rows of a request that share a KV
// head are numbered token after token, the group's heads next to each other.
struct Reach {
    int lo, hi;             // keys [lo, hi) that the tile's rows span
    int all_lo, all_hi;     // keys that every row sees
};

struct Rows {
    int count, group, base, len, causal, window, rows;

    __host__ __device__ __forceinline__ Rows(const AttendArgs &a, const KvRequest &r)
        : count(r.count), group(a.group), base(r.len - r.count), len(r.len), causal(a.causal),
          window(a.window), rows(r.count * a.group)
    {
    }
    // end (start) of the keys that token `token` sees
    __host__ __device__ __forceinline__ int end(int token) const
    {
        return causal ? min(max(base + token + 1, 0), len) : len;
    }
    __host__ __device__ __forceinline__ int begin(int token) const
    {
        // (base is negative where a request has more new rows than tokens: the window
        // comes off what is left of the place, which stays within 32 bits)
        return window ? max(max(base + token + 1, 0) - window, 0) : 0;
    }
    __host__ __device__ __forceinline__ Reach reach(int row0, int n) const
    {
        const int first = row0 / group, last = min(row0 + n - 1, rows - 1) / group;
        return {begin(first), end(last), begin(last), end(first)};
    }
};

// The unit (request, KV head) of workgroup `id`; each run of `units` workgroups
// has every unit once. Workgroups go to the 8 XCDs in turn and, within one, to
// its shader engines in turn, so the same order in each run would give all the
// parts of one long request to the same engines (measured: four prompt chunks
// of unlike lengths, half of the wave slots empty). Each run starts 8 units
// further: another engine, and the same XCD, whose L2 has the unit's codes.
__host__ __device__ __forceinline__ int unit_of(unsigned id, int units)
{
    const unsigned run = id / units;
    return (int)((id % units + 8 * (run % units)) % units);
}

// The part of a tile's keys that split `split` of `splits` takes, in steps of
// `step` keys from a multiple of 32 on. Places are unsigned here: a wave's next
// step may start past 2^31 - 1, where it ends.
struct Part {
    unsigned from, to;
};

__host__ __device__ __forceinline__ Part part_of(const Reach &r, int split, int splits, int min_part,
                                                 int step)
{
    const int start = r.lo & ~(kKeys - 1);
    const unsigned span = max(r.hi - start, 0);
    const unsigned each = (span + (unsigned)splits - 1) / (unsigned)splits;
    const unsigned part = each > (unsigned)min_part ? each : (unsigned)min_part;
    const unsigned keys = (part + step - 1) / step * step;      // at most 2^31
    // (from the end backwards, so that no sum passes 32 bits)
    const uint64_t before = (uint64_t)keys * (unsigned)split;
    const unsigned left = before < span ? span - (unsigned)before : 0;
    const unsigned mine = left < keys ? left : keys;
    const unsigned from = (unsigned)r.hi - left;
    return {from, from + mine};
}

// The step after t0 < to, or t0 again if that is the last one.
__host__ __device__ __forceinline__ unsigned step_after(unsigned t0, unsigned to, unsigned step)
{
    return to - t0 > step ? t0 + step : t0;
}

}  // namespace qmm
