// Runs the index arithmetic that the kernels of the paged KV cache share
// (csrc/qmm_kv.h, csrc/qmm_attend_rows.h) and the rules by which attention is
// launched (csrc/qmm_attend_shape.h) on the host, built with AddressSanitizer and
// UndefinedBehaviorSanitizer, over sums and lengths next to and past the ends of
// 32 bits. Exits non-zero on the first failed check. With the eight sizes of a
// call as arguments it prints that call's launch instead.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../block_quantized_matmul_q4_amd/csrc/qmm_attend_rows.h"
#include "../../block_quantized_matmul_q4_amd/csrc/qmm_attend_shape.h"
#include "../../block_quantized_matmul_q4_amd/csrc/qmm_kv.h"

namespace {
long g_checks = 0;

#define CHECK(cond)                                                              \
    do {                                                                         \
        ++g_checks;                                                              \
        if (!(cond)) {                                                           \
            std::fprintf(stderr, "FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond); \
            std::exit(1);                                                        \
        }                                                                        \
    } while (0)

// Rows (pages) that a plan writes at `before`, the sum of all earlier ones, into
// an array of `size`.
void fitting()
{
    std::vector<int64_t> sums = {0, 1, 7, 1023, 1024};
    for (int64_t at : {(int64_t)1 << 12, (int64_t)1 << 31, (int64_t)1 << 32, (int64_t)1 << 33,
                       (int64_t)3 << 31, (int64_t)1024 * 4194303, (int64_t)1024 * 3000000,
                       (int64_t)1 << 52})
        for (int64_t d : {-4096, -11, -10, -1, 0, 1, 9, 10, 4096}) sums.push_back(at + d);
    for (int64_t size : {(int64_t)0, (int64_t)1, (int64_t)10, (int64_t)4096, (int64_t)INT_MAX})
        for (int64_t before : sums)
            for (int64_t n : sums) {
                const int got = qmm::kv_fitting(n, size - before);
                CHECK(got >= 0 && got <= n);
                CHECK(got == 0 || before + got <= size);
                // all of them, or all that there is room for
                CHECK(got == n || before + got == size || before >= size);
            }
}

// Places of a ring, also of one whose head and count add up to more than 2^31.
void ring_places()
{
    for (int size : {1, 2, 50, 1 << 30, (1 << 30) + 7, INT_MAX})
        for (int head : {0, 1, size / 2, size - 1})
            for (int64_t after : {(int64_t)0, (int64_t)1, (int64_t)size / 2, (int64_t)size - 1, (int64_t)size}) {
                if (head >= size || after > size) continue;
                CHECK(qmm::kv_ring_place(head, after, size) == (head + after) % size);
            }
}

// Workgroups for up to 2^31 - 1 rows, whose last thread still has a 32-bit number.
void groups()
{
    for (int threads : {64, 256, 512, 1024})
        for (int64_t n : {(int64_t)0, (int64_t)1, (int64_t)255, (int64_t)256, (int64_t)257,
                          (int64_t)INT_MAX - 256, (int64_t)INT_MAX - 255, (int64_t)INT_MAX}) {
            const int64_t got = qmm::kv_groups((int)n, threads);
            CHECK(got == (n + threads - 1) / threads && got * threads - 1 <= INT_MAX);
        }
}

// The keys that a row sees, by the definition in 64 bits: j <= p if causal, j > p -
// window if there is one, 0 <= j < len.
void visible_keys()
{
    const int most = INT_MAX - 15;
    for (int len : {0, 1, 3, 50, 300, most})
        for (int count : {1, 5, 70, 1000, most})
            for (int causal : {0, 1})
                for (int window : {0, 1, 5, 299, INT_MAX - 50, INT_MAX - 2, INT_MAX}) {
                    qmm::AttendArgs a = {};
                    a.group = 1;
                    a.causal = causal;
                    a.window = window;
                    const qmm::Rows rows(a, {0, count, len});
                    for (int64_t token : {(int64_t)0, (int64_t)1, (int64_t)4, (int64_t)69,
                                          (int64_t)count - 51, (int64_t)count - 2, (int64_t)count - 1}) {
                        if (token < 0 || token >= count) continue;
                        const int64_t p = (int64_t)len - count + token;
                        int64_t lo = 0, hi = len;
                        if (causal && p + 1 < hi) hi = p + 1 > 0 ? p + 1 : 0;
                        if (window && p - window + 1 > 0) lo = p - window + 1;
                        CHECK(rows.begin((int)token) == lo && rows.end((int)token) == hi);
                    }
                }
}

// Parts and steps cover a tile's keys once, in order, at every length; the places
// that a step looks up lie before the part's end. The last steps of long parts
// stand for the others.
void parts_and_steps()
{
    const int most = INT_MAX - 15;
    for (int hi : {0, 1, 31, 32, 33, 257, 5000, 1 << 30, most - 256, most - 1, most})
        for (int lo : {0, 5, 64, hi - 1000, hi - 300, hi - 32, hi - 1, hi, hi + 7})
            for (int splits : {1, 2, 17, 2048})
                for (int min_part : {1, 256, 2048, INT_MAX})
                    for (int waves : {4, 8}) {
                        if (lo < 0 || lo > most) continue;
                        const unsigned step = (unsigned)waves * qmm::kKeys;
                        const unsigned start = (unsigned)lo / 32 * 32;
                        const qmm::Reach reach = {lo, hi, lo, hi};
                        unsigned end = start < (unsigned)hi ? start : (unsigned)hi;
                        for (int split = 0; split < splits; ++split) {
                            const auto [from, to] = qmm::part_of(reach, split, splits, min_part, (int)step);
                            CHECK(from == end && to >= from && to <= (unsigned)hi);
                            CHECK(from == to || from % 32 == 0);
                            end = to;
                            for (unsigned wave = 0; wave < (unsigned)waves; ++wave) {
                                unsigned t0 = from + wave * qmm::kKeys;
                                if (t0 < to && to - t0 > 4 * step) t0 += (to - t0) / step * step - 2 * step;
                                for (int n = 0; t0 < to; t0 += step, ++n) {
                                    CHECK(n < 4 && t0 + qmm::kKeys - 1 <= (unsigned)INT_MAX);
                                    const unsigned next = qmm::step_after(t0, to, step);
                                    CHECK(next < to && (next == t0 + step || (next == t0 && t0 + step >= to)));
                                    CHECK(qmm::kv_entry((int)next + 16, 4, most / 16 - 1) < most / 16);
                                }
                            }
                        }
                        CHECK(end == (unsigned)hi);
                    }
}

// Every launch of every accepted size holds less than 2^32 threads, and the launches
// of a call have each request once.
void launches()
{
    for (int batch : {1, 7, 512, 513, 1 << 16, 600000, 1 << 20})
        for (int kv_heads : {1, 8, 1024})
            for (int group : {1, 8, 64})
                for (int64_t tokens : {(int64_t)1, (int64_t)16384, (int64_t)INT_MAX / (kv_heads * group)})
                    for (int64_t max_q : {(int64_t)1, (int64_t)33, (int64_t)16384, (int64_t)INT_MAX / 64})
                        for (int64_t max_len : {(int64_t)1, (int64_t)5000, (int64_t)1 << 20, (int64_t)INT_MAX})
                            for (int64_t window : {(int64_t)0, (int64_t)4096, (int64_t)INT_MAX})
                                for (int dim : {64, 256}) {
                                    const auto s = qmm::attend_shape_of((int)tokens, batch, kv_heads, group, dim,
                                                                        max_q, max_len, window);
                                    CHECK(s.tiles >= 1 && s.splits >= 1 && s.splits <= qmm::kMaxSplits);
                                    CHECK(s.min_part >= 1 && (s.waves == 4 || s.waves == 8));
                                    const int most = qmm::requests_per_launch(kv_heads, s.tiles, s.splits);
                                    const int64_t n = most < batch ? most : batch;
                                    CHECK(n >= 1 && n * kv_heads * s.tiles * s.splits * s.waves * 64 < (int64_t)1 << 32);
                                    const int64_t rows = tokens * kv_heads * group;
                                    const int64_t joined = rows < qmm::kJoinRows ? rows : qmm::kJoinRows;
                                    CHECK(joined * 512 < (int64_t)1 << 32);
                                    // rows that one workgroup would walk on to although the chip is not full
                                    const int64_t groups = (int64_t)batch * kv_heads * s.tiles;
                                    const int64_t packed = (max_q < tokens ? max_q : tokens) * group;
                                    CHECK((int64_t)s.tiles * s.tile_rows >= packed || groups > qmm::kLaunchTiles / 2);
                                }
}

}  // namespace

int main(int argc, char **argv)
{
    if (argc == 9) {
        int64_t v[8];
        for (int i = 0; i < 8; ++i) v[i] = std::atoll(argv[i + 1]);
        const auto s = qmm::attend_shape_of((int)v[0], (int)v[1], (int)v[2], (int)v[3], (int)v[4], v[5], v[6], v[7]);
        std::printf("%d %d %d %d %d %d\n", s.tiles, s.splits, s.min_part, s.tile_rows, s.waves, (int)s.few);
        return 0;
    }
    launches();
    fitting();
    parts_and_steps();
    visible_keys();
    groups();
    ring_places();
    std::printf("kv bounds passed (%ld)\n", g_checks);
    return 0;
}
