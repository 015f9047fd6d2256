// How an attention call is launched, from the sizes that the host knows (for the
// library and for checks of the rules).
#pragma once

#include "qmm_kv.h"

namespace qmm {

// Most parts of a request's keys.
constexpr int kMaxSplits = 2048;

// A launch has to hold less than 2^32 threads, i.e. 2^23 workgroups of 512. Tiles
// of rows make at most 2^20 of them, 2^11 times what the chip holds at once;
// requests beyond 2^22 workgroups and rows to be joined beyond 2^20 take further
// launches.
constexpr int64_t kLaunchTiles = 1 << 20;
constexpr int64_t kLaunchGroups = 1 << 22;
constexpr int64_t kJoinRows = 1 << 20;

inline int requests_per_launch(int kv_heads, int tiles, int splits)
{
    const int64_t most = kLaunchGroups / ((int64_t)kv_heads * tiles * splits);
    return most > 1 ? (int)most : 1;
}

// Workgroups of four waves that the chip holds at once with two waves per SIMD, as
// the kernels for many rows have. Those for 8 rows have room for three up to 128
// dims and for four at 64, which no rule here uses: 131072 keys of 32/8 heads
// of 128 make 1024 workgroups, where 768 run at once.
constexpr int64_t kResident = 512;

inline AttendShape attend_shape_of(int tokens, int batch, int kv_heads, int group, int head_dim,
                                   int64_t max_q, int64_t max_len, int64_t window)
{
    if (max_q > tokens) max_q = tokens > 0 ? tokens : 1;
    if (window > 0 && max_len > window + max_q) max_len = window + max_q;
    const int64_t packed = max_q * group;
    // Two tiles of 16 rows share each decoded key where their registers leave room
    // for two waves per SIMD, and where there is work for every workgroup slot (a
    // prompt of 2048, 32/8 heads of 128: 147 -> 133 us; of 512, 16 heads of 64, which
    // has less: 8.9 -> 15.5 us; 8/2 heads of 256, one wave per SIMD: 79 -> 91 us; all
    // with a kernel trace attached, without which these calls take 113, 8.5 and 68 us).
    //
    // 9 to 16 rows by the kernel for few rows -> by the other one, whole calls in a
    // graph, 4 rows x group 4: where requests fill the chip, up to 128 dims, it is the
    // faster (64 requests of 4000 keys, 8 KV heads of 64: 49 -> 67 us, of 128: 91 -> 117
    // us); 16 requests of 2000 20.5 -> 20.2, of 8000 46.9 -> 44.4 us at 128 dims. At 256
    // dims its tiles of 16 rows spill 24 registers and lose throughout (16 requests of
    // 8000 keys, 2 KV heads: 37.7 -> 30.8 us).
    const bool few = packed <= 16;
    const bool twice = head_dim <= 128 && (int64_t)batch * kv_heads * ((packed + 31) / 32) >= kResident;
    const int rows = packed <= 8 ? 8 : twice && !few ? 32 : 16;
    // (a workgroup walks on to the tiles that the grid leaves out: where max_q is far
    // above what most requests bring, most of its tiles have no rows)
    int64_t tiles = (packed + rows - 1) / rows;
    const int64_t most = kLaunchTiles / ((int64_t)batch * kv_heads);
    if (tiles > most) tiles = most > 1 ? most : 1;
    const int64_t units = (int64_t)batch * kv_heads * tiles;
    // Keys of a part: few enough that every workgroup slot has one, and, once
    // there is enough work, so few that ragged requests even out (four parts
    // to a slot), but no less than what pays for joining them
    const int64_t all = units * max_len;
    int64_t part;
    if (!few) {
        part = all / (16 * kResident);
        // (300 rows over 3000 keys, 32/8 heads of 128, parts of 2048 -> of one per
        // slot: 89 -> 81 us)
        const int64_t each = all / kResident;
        if (part < 2048) part = each < 256 ? 256 : each < 2048 ? each : 2048;
    } else if (units <= kResident / 2 && max_len * head_dim <= 512 * 256) {
        // Short requests: eight waves and one launch, a launch less for the host (3 to 4
        // us a call outside of graphs). Parts of four waves and a join -> this, in a
        // graph: 32 requests of 1024 keys, 32/8 heads of 64, 12.9 -> 10.0 us, of 512 at
        // 128 dims 12.8 -> 9.8 us; but one of 512 at 256 dims 12.6 -> 13.5 us, one of
        // 1024 at 128 dims 9.8 -> 12.3 us, and one of 2048 at 64 dims 8.6 -> 13.7 us.
        return {(int)tiles, 1, (int)max_len, rows, 8, few};
    } else {
        part = all / (4 * kResident);
        if (part < 1024) part = all / kResident < 1024 ? all / kResident : 1024;
        if (part < 256) part = 256;
    }
    int64_t splits = (max_len + part - 1) / part;
    if (splits > kMaxSplits) splits = kMaxSplits;
    return {(int)tiles, (int)splits, (int)(part < INT32_MAX ? part : INT32_MAX), rows, 4, few};
}

}  // namespace qmm
