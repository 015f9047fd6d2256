// Attention of f32 queries over the paged Q4_0 cache, for more than 16 rows of a
// request per KV head: drafted tokens of large groups, prompts and prompt chunks.
//
// The products and the lane order are those of the kernel for few rows
// (attend.hip). What differs is what the rows share: a wave works on QT tiles
// of 16 rows against the same 32 keys, so that decoding is done once for all of
// them, and whatever is done per row and key is kept small:
//   K: the exact codes q - 8, two terms of q, the block's scale on the result;
//   V: each value q d is made once, as two fp16 terms that hold it exactly (d
//      has 11 bits and q - 8 four: hi = fp16(q d), lo = q d - hi), and p as two
//      terms: O += lo p1 + hi p2 + hi p1, the omitted lo p2 being 2^-24 of it.
// So a row costs per key and 32 dims two matrix instructions' share for S and
// three for O, and the vector ALU no more than the scale on S, the softmax and
// the two terms of p.
//
// p is carried times 2^12 (fp16's subnormals); where a |d| of V reaches 512 the
// step takes d / 8, and O times 1 / 8 before and 8 after the product. A scale that
// is NaN or infinite may reach only rows that see its key, while all rows share the
// values made of it: the step takes it as 0 and marks the block of the rows that
// see it, whose results are set to NaN at the end.
//
// A workgroup of four waves has one tile of rows; each wave takes every fourth
// 32 keys by itself, without a barrier, and the four join through LDS. Tiles
// are started from the last, which see the most keys.
//
// Bound: the vector ALU (per 32 keys and 32 rows at 128 dims 80 matrix
// instructions of 16 cycles and 520 other operations of 4), two waves per SIMD.
// Up to 128 dims QT = 2 where there is work for every workgroup slot; wider rows
// take QT = 1, since two tiles' registers leave one wave per SIMD (a prompt of
// 2048 tokens, 8/2 heads of 256: 87 us, with QT = 1 78 us, both with a kernel trace
// attached; a whole call takes 68 us without). Four chunks of up to 512 tokens over
// 5000 to 16384 keys, 32/8 heads of 128, 901 us (0.32 PFLOP/s; the matrix cores are
// busy 32 % of the time and the vector ALU 59 %, one after the other) and 20 us for
// the join. Decoding once per 128 rows into LDS, a barrier every 32 keys, was built:
// half of the vector operations, at 128 dims the same time, twice the time for 512
// tokens, and for four chunks of 512 over 16384 keys, 8/2 heads of 256, 787 us where
// this kernel takes 837; it is not kept.
#include "qmm_attend.h"

namespace qmm {
namespace {

constexpr int kWaves = 4;
// How far scores may pass the running maximum (in units of log 2) before it is
// moved: p 2^12 stays below fp16's end with p up to 8
constexpr float kSlack = 3.0f;

__device__ __forceinline__ f32x4 mfma(const Frag &a, const Frag &b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v, b.v, c, 0, 0, 0);
}

__device__ __forceinline__ bool not_finite(uint32_t half) { return (half & 0x7C00u) == 0x7C00u; }

template <int NB, int QT>
__global__ void __launch_bounds__(kWaves * 64, 2) attend_many_kernel(AttendArgs a)
{
    constexpr int D = 32 * NB;
    constexpr int kRows = 16 * QT;
    constexpr int kPad = D + 4;
    constexpr int kStep = kWaves * kKeys;
    __shared__ float s_o[kWaves][16][kPad];
    __shared__ float s_m[kWaves][16], s_l[kWaves][16];

    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int units = a.requests * a.cache.kv_heads;
    const int unit = unit_of(blockIdx.x, units);
    const int split = blockIdx.x / units % a.splits;
    const int tile0 = a.tiles - 1 - (int)(blockIdx.x / units / a.splits);
    const int b = a.first + unit / a.cache.kv_heads, kvh = unit % a.cache.kv_heads;
    const int shift = __builtin_ctz(a.cache.page_size);
    const KvRequest request = kv_request(a.cu, a.lens, b, a.tokens, a.width, shift);
    const int q0 = request.q0;
    const Rows rows_of(a, request);
    const int rows = rows_of.rows;
    const Keys<NB, true> keys(a.cache, a.table + (int64_t)b * a.width, a.width, shift, kvh, n, g);
    const Patterns patterns;

    for (int tile = tile0; tile * kRows < rows; tile += a.tiles) {
        const Reach reach = rows_of.reach(tile * kRows, kRows);
        const auto [from, to] = part_of(reach, split, a.splits, a.min_part, kStep);

        // this lane's row of each tile; the last rows repeat the request's last one
        Query<NB, false> q[QT];
        int lo[QT], hi[QT];
        float m[QT], l[QT];
        uint32_t poison[QT];
        f32x4 o[QT][NB][2] = {};
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int row = min(tile * kRows + 16 * t + n, rows - 1);
            const int token = row / a.group, head = kvh * a.group + row % a.group;
            lo[t] = rows_of.begin(token);
            hi[t] = min(rows_of.end(token), (int)to);
            q[t].load(a.q + (int64_t)(q0 + token) * a.q_stride + head * D, g, a.scale, -1.0f);
            m[t] = kLowest;
            l[t] = 0.0f;
            poison[t] = 0;
        }

        unsigned t0 = from + wave * kKeys;
        Half<NB> kx[2], vx[2];
        Pages pages = {{-1, -1}}, entries = {{-1, -1}};    // of the next step
        if (t0 < to) {
            pages = keys.pages(keys.look_up(t0));
            entries = keys.look_up(step_after(t0, to, kStep));
#pragma unroll
            for (int h = 0; h < 2; ++h) keys.load_k(kx[h], pages.at[h], t0 + 16 * h);
#pragma unroll
            for (int h = 0; h < 2; ++h) keys.load_v(vx[h], pages.at[h], t0 + 16 * h);
        }

        for (; t0 < to; t0 += kStep) {
            // the last step loads its own keys again, which costs less than the
            // registers that loads under a condition take
            const unsigned next = step_after(t0, to, kStep);
            const Pages next_pages = keys.pages(entries);
            entries = keys.look_up(step_after(next, to, kStep));

            f32x4 s[QT][2] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h)
                unrolled<NB>([&](auto block) {
                    constexpr int i = decltype(block)::value;
                    Frag f;
                    codes_of(patterns, kx[h].codes.w[i], f.h, f.h + 2);
                    const uint32_t d[2] = {from_lane<2 * i>(kx[h].scales),
                                           from_lane<2 * i + 1>(kx[h].scales)};
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        const f32x4 acc = mfma(f, q[t].second[i], mfma(f, q[t].first[i], f32x4{}));
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            s[t][h][2 * c] = fmaf(half_lo(d[c]), acc[2 * c], s[t][h][2 * c]);
                            s[t][h][2 * c + 1] =
                                fmaf(half_hi(d[c]), acc[2 * c + 1], s[t][h][2 * c + 1]);
                        }
                    }
                });
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int h = 0; h < 2; ++h) keys.load_k(kx[h], next_pages.at[h], next + 16 * h);

            const bool whole = pages.at[0] >= 0 && pages.at[1] >= 0 && t0 >= (unsigned)reach.all_lo &&
                               t0 + kKeys <= (unsigned)reach.all_hi && t0 + kKeys <= to;
            uint32_t seen[QT];                  // bit 4 h + r: key 16 h + 4 g + r is visible
#pragma unroll
            for (int t = 0; t < QT; ++t) seen[t] = 0xFF;
            if (!whole) {
                keep_branch();
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    seen[t] = 0;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int at = (int)t0 + 16 * h + 4 * g + r;
                            const bool ok = pages.at[h] >= 0 && at >= lo[t] && at < hi[t];
                            seen[t] |= (uint32_t)ok << (4 * h + r);
                            s[t][h][r] = ok ? s[t][h][r] : kNone;
                        }
                }
            }

            // V scales of keys that no row sees may hold anything; a scale from
            // 512 on (bits 14 and 13 of the fp16) takes the step aside
            uint32_t d[2] = {vx[0].scales, vx[1].scales};
            if (!whole) {
                keep_branch();
                uint32_t some = seen[0];
#pragma unroll
                for (int t = 1; t < QT; ++t) some |= seen[t];
                some |= (uint32_t)__builtin_amdgcn_mov_dpp((int)some, 0x128, 0xF, 0xF, true);
                some |= (uint32_t)__builtin_amdgcn_mov_dpp((int)some, 0x124, 0xF, 0xF, true);
                some |= (uint32_t)__builtin_amdgcn_mov_dpp((int)some, 0x122, 0xF, 0xF, true);
                some |= (uint32_t)__builtin_amdgcn_mov_dpp((int)some, 0x121, 0xF, 0xF, true);
#pragma unroll
                for (int h = 0; h < 2; ++h) {   // lane n has keys 2 (n % 2) and the next
                    const uint32_t two = some >> (4 * h + 2 * (n & 1));
                    d[h] &= (two & 1 ? 0xFFFFu : 0) | (two & 2 ? 0xFFFF0000u : 0);
                }
            }
            const bool aside = __any(((d[0] & (d[0] << 1)) | (d[1] & (d[1] << 1))) & 0x40004000u);

            // exponents of 2 of the row's p, and whether they pass the limit
            float e[QT][2][4];
            bool grows = false;
            const float limit = kUpLog + kSlack;
            auto exponents = [&] {
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; ++r) e[t][h][r] = fmaf(s[t][h][r], q[t].factor, kUpLog - m[t]);
            };
            exponents();
#pragma unroll
            for (int t = 0; t < QT; ++t) grows |= largest(e[t]) > limit;
            if (__any(grows)) {
                keep_branch();
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    // (only rows that pass it, so that none depends on its neighbours)
                    const bool passes = groups_max(largest(e[t])) > limit;
                    const float m_new = passes ? groups_max(largest(s[t])) * q[t].factor : m[t];
                    const float shrink = __builtin_amdgcn_exp2f(m[t] - m_new);
                    m[t] = m_new;
                    l[t] *= shrink;
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        o[t][i][0] *= shrink;
                        o[t][i][1] *= shrink;
                    }
                }
                exponents();
            }
            float p[QT][2][4];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        p[t][h][r] = __builtin_amdgcn_exp2f(e[t][h][r]);
                        l[t] += p[t][h][r];
                    }
            }

            auto scale_all = [&](float f) {
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        o[t][i][0] *= f;
                        o[t][i][1] *= f;
                    }
            };
            if (aside) {
                keep_branch();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    unrolled<2 * NB>([&](auto pair) {
                        constexpr int i = decltype(pair)::value / 2, c = decltype(pair)::value % 2;
                        const uint32_t two = from_lane<2 * i + c>(d[h]);
                        const uint32_t bad = (uint32_t)not_finite(two) | (uint32_t)not_finite(two >> 16) << 1;
#pragma unroll
                        for (int t = 0; t < QT; ++t)
                            if (bad & seen[t] >> (4 * h + 2 * c)) poison[t] |= 1u << i;
                    });
                    const f16x2 eighth = {(_Float16)0.125f, (_Float16)0.125f};
                    if (not_finite(d[h])) d[h] &= 0xFFFF0000u;
                    if (not_finite(d[h] >> 16)) d[h] &= 0xFFFFu;
                    d[h] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, d[h]) * eighth);
                }
                scale_all(0.125f);
            }

            Frag p1[QT], p2[QT];
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float y0 = p[t][h][2 * c], y1 = p[t][h][2 * c + 1];
                        p1[t].u[2 * h + c] = two_halves(y0, y1);
                        p2[t].u[2 * h + c] = second_terms(y0, y1, p1[t].u[2 * h + c]);
                    }
            unrolled<NB>([&](auto block) {
                constexpr int i = decltype(block)::value;
                __builtin_amdgcn_sched_barrier(0);
                Frag v[2], rest[2];             // low and high nibbles' values
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    codes_of(patterns, vx[h].codes.w[i], v[0].h + 2 * h, v[1].h + 2 * h);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f16x2 d2[2] = {__builtin_bit_cast(f16x2, from_lane<2 * i>(d[h])),
                                         __builtin_bit_cast(f16x2, from_lane<2 * i + 1>(d[h]))};
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const f16x2 code = v[x].h[2 * h + c];
                            v[x].h[2 * h + c] = code * d2[c];
                            rest[x].h[2 * h + c] =
                                __builtin_elementwise_fma(code, d2[c], -v[x].h[2 * h + c]);
                        }
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int t = 0; t < QT; ++t)
                        o[t][i][x] = mfma(v[x], p1[t], mfma(v[x], p2[t], mfma(rest[x], p1[t], o[t][i][x])));
            });
            __builtin_amdgcn_sched_barrier(0);
            if (aside) {
                keep_branch();
                scale_all(8.0f);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) keys.load_v(vx[h], next_pages.at[h], next + 16 * h);
            pages = next_pages;
        }

        // the waves' parts meet in LDS, 16 rows at a time
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            uint32_t marked = poison[t];        // any lane group's keys
            marked |= (uint32_t)__shfl_xor((int)marked, 16);
            marked |= (uint32_t)__shfl_xor((int)marked, 32);
            const float sum_l = groups_sum(l[t]);
            if (g == 0) {
                s_m[wave][n] = m[t] == kLowest ? kNone : m[t];
                s_l[wave][n] = sum_l;
            }
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 nan = {NAN, NAN, NAN, NAN};
                    *(f32x4 *)&s_o[wave][n][32 * i + 16 * h + 4 * g] =
                        marked >> i & 1 ? nan : o[t][i][h];
                }
            __syncthreads();
            const int row0 = tile * kRows + 16 * t;
            const int stored = min(16, rows - row0);
            for (int at = threadIdx.x; at < stored * (D / 4); at += kWaves * 64) {
                const int r = at / (D / 4), c = at % (D / 4) * 4;
                float mm = kNone, ll = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, s_m[w][r]);
                f32x4 sum = {};
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    const float f = weight(s_m[w][r], mm);
                    ll = fmaf(f, s_l[w][r], ll);
                    sum += f * *(const f32x4 *)&s_o[w][r][c];
                }
                store_row(a, q0, kvh, row0 + r, split, D, c, sum, mm, ll);
            }
            __syncthreads();
        }
    }
}

}  // namespace

template <int NB>
static void launch_many(const AttendArgs &a, unsigned grid, hipStream_t stream)
{
    if constexpr (NB <= 4) {
        if (a.tile_rows == 32) {
            attend_many_kernel<NB, 2><<<grid, kWaves * 64, 0, stream>>>(a);
            return;
        }
    }
    attend_many_kernel<NB, 1><<<grid, kWaves * 64, 0, stream>>>(a);
}

void launch_attend_many(const AttendArgs &a, unsigned grid, hipStream_t stream)
{
    switch (a.cache.head_dim) {
    case 64: launch_many<2>(a, grid, stream); break;
    case 96: launch_many<3>(a, grid, stream); break;
    case 128: launch_many<4>(a, grid, stream); break;
    case 192: launch_many<6>(a, grid, stream); break;
    default: launch_many<8>(a, grid, stream); break;
    }
}

}  // namespace qmm
