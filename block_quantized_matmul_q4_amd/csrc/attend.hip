// Attention of f32 queries over the paged Q4_0 cache, for few rows per request
// (decoding and checking drafted tokens).
//
// The rows of a request that share a KV head (its new tokens x the group's
// query heads, token after token) are packed into tiles of 16, so one pass
// over the codes serves them all. A tile's keys are taken 32 at a time:
//   S^T = K Q^T   per block of 32 dims one v_mfma_f32_16x16x32_f16 per term of
//                 q: A = the codes of 16 keys, B = q of 16 rows; the block's
//                 fp16 scale multiplies the result in f32, so no key is
//                 rounded;
//   p = exp2(S f - m), m the running maximum, moved only where the exponents
//                 pass it by a limit;
//   O^T += V^T P^T   per block of 32 dims: A = the codes of 32 keys, B = p d of
//                 16 rows, d the block's scales of those keys.
// A lane holds one row throughout (row = lane % 16, MFMA column), so the
// softmax exchanges lanes only where the maximum moves, and the P that
// comes out of the first product has the lane order that the second takes,
// with keys {4 g + r, 16 + 4 g + r} in lane group g = lane / 16.
//
// f32 accuracy on fp16 matrix cores: the codes q - 8 are exact in fp16; q
// (scaled by a power of two per row, so that its largest magnitude lies in
// [8, 16)) and p d enter as two fp16 terms, hi = fp16(x), lo = fp16(x - hi).
// Up to 8 rows are PACKed: columns 0-7 carry the first terms, columns 8-15 the
// second ones of the same rows, so each product takes one instruction instead
// of two and q half the registers; the two columns of a row are added where S
// and, at the end, O leave the matrix cores.
// p is carried times 2^12 (in O and in the sum alike, so it cancels) to keep
// the low terms of small weights out of fp16's subnormals. A step whose V
// scales reach 2 would push p d towards fp16's end; there p is taken without
// that factor and the codes carry it.
//
// Decoding a nibble: shifted into mantissa bits 6-9 under the exponent of 16
// it reads as 16 + q; in bits 4-7 under that of 64 as 64 + q, in bits 0-3 under
// that of 1024 as 1024 + q. For K the offset 24 leaves with the accumulator's
// start, -24 sum(q) of the block, which takes one operation per code; for V it
// would have to be removed from sums over the whole context, where it would
// cost accuracy, so a packed addition takes it off each pair of codes, and the
// forms that need fewer shifts are used.
//
// Bound: HBM in principle (a key costs 9/8 D bytes per KV head), the vector ALU
// in practice (per 32 keys and tile about 12 operations per lane and 32 dims for
// K, 22 for V, half of them for p d and its two terms). Hence the split of the
// work: one wave works on 32 keys by itself, its next keys' codes in flight
// meanwhile (K from the moment S is done, V from the moment O is), the block
// table's entries a step further ahead, the waves of a workgroup share a part of
// the keys and join through LDS, and long requests are split over workgroups
// whose parts a second launch joins.
// Measured, 32/8 heads of 128: 64 requests up to 8192 keys (335 MB of codes) 88
// us, 3.8 TB/s, and 5 us for the join; one of 131072 keys 36 + 7 us. 8/2 heads of
// 256, 32 requests up to 2351 keys 18 + 4 us. What a call takes apart from its keys
// (in a graph, where an empty kernel takes 2.4 us), at 256 dims: 8.8 us for 576
// workgroups of four waves, 15.3 with one step of 128 keys, 4.5 us for each further
// one; 6.0 us for 32 of eight waves, 10.2 with one step of 256 keys, 3.0 us for each
// further one. At 64 dims 4.6, 6.8 and 1.4 us; 4.0, 5.6 and 1.0 us. With tiles of 16
// rows at 256 dims 24 registers are spilled, some of them in the key loop; all other
// forms spill no vector register. Steps that paid: the table read through the
// constant address space and a step ahead (a vector load waits for all loads in
// flight, 109 -> 96 us), the running maximum moved only when the exponents pass
// it by 2 and compared through them (96 -> 89 us), scales shared by DPP
// broadcasts, accumulators in ordinary registers.
#include "qmm_attend.h"
#include "qmm_attend_shape.h"

namespace qmm {
namespace {

// How far scores may pass the running maximum (in units of log 2) before it is
// moved: p 2^12 d stays below fp16's end with p up to 4 and d up to 2
constexpr float kSlack = 2.0f;

// Waves of a SIMD that the registers leave room for.
template <int NB, bool PACK, int WAVES>
constexpr int kWavesPerSimd = WAVES == 8 ? (NB <= 2 && PACK ? 4 : 2)
                              : NB <= 2 ? (PACK ? 4 : 3)
                                        : NB <= 4 && PACK ? 3 : 2;

template <int NB, bool PACK, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, (kWavesPerSimd<NB, PACK, WAVES>)) attend_few_kernel(AttendArgs a)
{
    constexpr int D = 32 * NB;
    constexpr int kRows = PACK ? 8 : 16;            // rows of a tile
    constexpr int kPad = D + 4;
    constexpr int kStep = WAVES * kKeys;
    // From 192 dims on the registers of the accumulators' starts would spill,
    // and K codes are made as V's (two more operations per word)
    constexpr bool kOffset = NB < 6;
    __shared__ float s_o[WAVES][kRows][kPad];
    __shared__ float s_m[WAVES][kRows], s_l[WAVES][kRows];

    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int units = a.requests * a.cache.kv_heads;
    const int unit = unit_of(blockIdx.x, units);
    const int split = blockIdx.x / units % a.splits;
    const int tile0 = blockIdx.x / units / a.splits;
    const int b = a.first + unit / a.cache.kv_heads, kvh = unit % a.cache.kv_heads;
    const int shift = __builtin_ctz(a.cache.page_size);
    const KvRequest request = kv_request(a.cu, a.lens, b, a.tokens, a.width, shift);
    const int q0 = request.q0;
    const Rows rows_of(a, request);
    const int rows = rows_of.rows;
    const Keys<NB, (NB > 4)> keys(a.cache, a.table + (int64_t)b * a.width, a.width, shift, kvh, n, g);
    const Patterns patterns;
    // PACK: columns 8-15 take x - hi where columns 0-7 take x
    const float minus = n < 8 ? 0.0f : -1.0f;

    for (int tile = tile0; tile * kRows < rows; tile += a.tiles) {
        // this lane's row; the tile's last rows repeat the request's last one
        const int row = min(tile * kRows + (n & (kRows - 1)), rows - 1);
        const int token = row / a.group, head = kvh * a.group + row % a.group;
        const int hi = rows_of.end(token), lo = rows_of.begin(token);   // its keys
        const Reach reach = rows_of.reach(tile * kRows, kRows);
        const auto [from, to] = part_of(reach, split, a.splits, a.min_part, kStep);

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

        const float *q = a.q + (int64_t)(q0 + token) * a.q_stride + head * D;
        Query<NB, PACK> x;
        x.load(q, g, a.scale, minus);
        const float factor = x.factor;
        // -24 sum(q) of each block, in all of a column's places
        f32x4 start_s[kOffset ? NB : 1] = {};
        Frag minus24;
#pragma unroll
        for (int c = 0; c < 4; ++c) minus24.u[c] = 0xCE00CE00u;
#pragma unroll
        for (int i = 0; kOffset && i < NB; ++i) {
            start_s[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(minus24.v, x.first[i].v, f32x4{}, 0, 0, 0);
            if constexpr (!PACK)
                start_s[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(minus24.v, x.second[i].v,
                                                                    start_s[i], 0, 0, 0);
        }

        f32x4 o[NB][2] = {};
        float m = kLowest, l = 0.0f;            // l: this lane's keys only

        for (; t0 < to; t0 += kStep) {
            // the last step loads its own keys again, which costs less than the
            // registers that loads under a condition take
            const unsigned next = step_after(t0, to, kStep);
            const Pages next_pages = keys.pages(entries);
            entries = keys.look_up(step_after(next, to, kStep));

            f32x4 s[2] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                unrolled<NB>([&](auto block) {
                    constexpr int i = decltype(block)::value;
                    Frag f;
                    if constexpr (kOffset)
                        offset_codes(patterns, kx[h].codes.w[i], f);
                    else
                        codes_of(patterns, kx[h].codes.w[i], f.h, f.h + 2);
                    f32x4 acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        f.v, x.first[i].v, start_s[kOffset ? i : 0], 0, 0, 0);
                    if constexpr (!PACK)
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.v, x.second[i].v, acc, 0, 0, 0);
                    unrolled<2>([&](auto pair) {
                        constexpr int c = decltype(pair)::value;
                        const uint32_t d = from_lane<2 * i + c>(kx[h].scales);
                        s[h][2 * c] = fmaf(half_lo(d), acc[2 * c], s[h][2 * c]);
                        s[h][2 * c + 1] = fmaf(half_hi(d), acc[2 * c + 1], s[h][2 * c + 1]);
                    });
                });
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int h = 0; h < 2; ++h) keys.load_k(kx[h], next_pages.at[h], next + 16 * h);
            if constexpr (PACK)                 // first and second terms' columns
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[h][r] += dpp_f<0x128, 0xF>(s[h][r]);

            const bool whole = pages.at[0] >= 0 && pages.at[1] >= 0 && t0 >= (unsigned)reach.all_lo &&
                               t0 + kKeys <= (unsigned)reach.all_hi && t0 + kKeys <= to;
            uint32_t seen = 0xFF;               // bit 4 h + r: key 16 h + 4 g + r is visible
            if (!whole) {
                keep_branch();
                seen = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int t = (int)t0 + 16 * h + 4 * g + r;
                        const bool ok = pages.at[h] >= 0 && t >= lo && t < min(hi, (int)to);
                        seen |= (uint32_t)ok << (4 * h + r);
                        s[h][r] = ok ? s[h][r] : kNone;
                    }
            }

            const ValueScales<NB> d[2] = {ValueScales<NB>(vx[0].scales),
                                          ValueScales<NB>(vx[1].scales)};
            // a V scale of 2 or more (of keys that some row sees): p without its
            // factor, the codes with it
            uint32_t some = seen;               // keys that some row sees
            if (!whole) {
                keep_branch();
                some |= (uint32_t)__builtin_amdgcn_mov_dpp((int)some, 0x128, 0xF, 0xF, true);
                some |= (uint32_t)__builtin_amdgcn_mov_dpp((int)some, 0x124, 0xF, 0xF, true);
                some |= (uint32_t)__builtin_amdgcn_mov_dpp((int)some, 0x122, 0xF, 0xF, true);
                some |= (uint32_t)__builtin_amdgcn_mov_dpp((int)some, 0x121, 0xF, 0xF, true);
            }
            bool large = false;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < ValueScales<NB>::kRegs; ++j)
                    large |= (some >> (4 * h + ValueScales<NB>::key(n, j)) & 1) &&
                             !(fabsf(d[h].d[j]) < 2.0f);
            const bool big = __any(large);

            float e[2][4];              // exponents of 2 of p
            auto exponents = [&] {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) e[h][r] = fmaf(s[h][r], factor, kUpLog - m);
            };
            exponents();
            const float limit = kUpLog + (big ? 0.0f : kSlack);
            if (__any(largest(e) > limit)) {
                keep_branch();
                // (only rows that pass it, so that none depends on its neighbours)
                const bool passes = groups_max(largest(e)) > limit;
                const float m_new = passes ? groups_max(largest(s)) * factor : m;
                const float shrink = __builtin_amdgcn_exp2f(m - m_new);
                m = m_new;
                l *= shrink;
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    o[i][0] *= shrink;
                    o[i][1] *= shrink;
                }
                exponents();
            }
            float p[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    p[h][r] = __builtin_amdgcn_exp2f(e[h][r]);
                    l += p[h][r];
                }

            const bool plain = whole && !big;
            f16x2 up = {(_Float16)1.0f, (_Float16)1.0f};
            if (!plain) {
                keep_branch();
                up = big ? f16x2{(_Float16)kUp, (_Float16)kUp} : up;
                const float down = big ? 1.0f / kUp : 1.0f;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 4; ++r) p[h][r] *= down;
            }

            // O += V^T (p d)^T
            auto values = [&](auto is_plain) {
                unrolled<NB>([&](auto block) {
                    constexpr int i = decltype(block)::value;
                    __builtin_amdgcn_sched_barrier(0);
                    Frag p1, p2, low, high;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float y[4];
                        unrolled<4>([&](auto key) {
                            constexpr int r = decltype(key)::value;
                            y[r] = p[h][r] * d[h].template get<i, r>();
                            // a scale that is NaN may not meet the p = 0 of a hidden key
                            if constexpr (!decltype(is_plain)::value) y[r] = seen >> (4 * h + r) & 1 ? y[r] : 0.0f;
                        });
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float y0 = y[2 * c], y1 = y[2 * c + 1];
                            const uint32_t first = two_halves(y0, y1);
                            if constexpr (PACK) {
                                p1.u[2 * h + c] = second_terms(y0, y1, first, minus);
                            } else {
                                p1.u[2 * h + c] = first;
                                p2.u[2 * h + c] = second_terms(y0, y1, first);
                            }
                        }
                        uint32_t w = vx[h].codes.w[i];
                        if constexpr (!decltype(is_plain)::value) keep_apart(w);
                        codes_of(patterns, w, low.h + 2 * h, high.h + 2 * h);
                    }
                    if constexpr (!decltype(is_plain)::value) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            low.h[c] *= up;
                            high.h[c] *= up;
                        }
                    }
                    o[i][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(low.v, p1.v, o[i][0], 0, 0, 0);
                    o[i][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(high.v, p1.v, o[i][1], 0, 0, 0);
                    if constexpr (!PACK) {
                        o[i][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(low.v, p2.v, o[i][0], 0, 0, 0);
                        o[i][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(high.v, p2.v, o[i][1], 0, 0, 0);
                    }
                });
            };
            if (plain) values(std::true_type{}); else values(std::false_type{});
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int h = 0; h < 2; ++h) keys.load_v(vx[h], next_pages.at[h], next + 16 * h);
            pages = next_pages;
        }

        // the waves' parts meet in LDS
        l = groups_sum(l);
        if (g == 0 && n < kRows) {
            s_m[wave][n] = m == kLowest ? kNone : m;
            s_l[wave][n] = l;
        }
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (PACK)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[i][h][r] += dpp_f<0x128, 0xF>(o[i][h][r]);
                if (n < kRows) *(f32x4 *)&s_o[wave][n][32 * i + 16 * h + 4 * g] = o[i][h];
            }
        __syncthreads();
        const int stored = min(kRows, rows - tile * kRows);
        for (int at = threadIdx.x; at < stored * (D / 4); at += WAVES * 64) {
            const int r = at / (D / 4), c = at % (D / 4) * 4;
            float mm = kNone, ll = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) mm = fmaxf(mm, s_m[w][r]);
            f32x4 sum = {};
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const float f = weight(s_m[w][r], mm);
                ll = fmaf(f, s_l[w][r], ll);
                sum += f * *(const f32x4 *)&s_o[w][r][c];
            }
            store_row(a, q0, kvh, tile * kRows + r, split, D, c, sum, mm, ll);
        }
        __syncthreads();
    }
}

// Rows before cu[0] and from cu[B] on belong to no request: no part of them is
// written, and they are not either.
__device__ __forceinline__ bool of_a_request(const AttendArgs &a, int64_t row)
{
    const int64_t token = row / a.q_heads;
    return token >= a.cu[0] && token < a.cu[a.batch];
}

// A few parts: D / 4 threads per row, each for itself.
constexpr int kFewSplits = 16;

__global__ void __launch_bounds__(256) join_few_kernel(AttendArgs a, int64_t first)
{
    const int D = a.cache.head_dim, wide = D / 4;
    const int64_t rows_all = (int64_t)a.tokens * a.q_heads;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, row = first + id / wide;
    if (row >= rows_all || !of_a_request(a, row)) return;
    const int c = (int)(id % wide) * 4;
    const float2 *ml = (const float2 *)a.part_ml + row;
    float m = kNone;
    // eight parts at a time, all their loads in flight; m moves as it does in the
    // softmax
    f32x4 sum = {};
    float l = 0.0f;
    for (int s0 = 0; s0 < a.splits; s0 += 8) {
        float2 part[8];
        f32x4 o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int s = min(s0 + i, a.splits - 1);
            part[i] = ml[s * rows_all];
            o[i] = *(const f32x4 *)(a.part_o + (s * rows_all + row) * D + c);
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, part[i].x);
        const float shrink = weight(m, top);
        m = top;
        l *= shrink;
        sum *= shrink;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // a part that has seen nothing has l = 0, and its o is anything
            const bool counts = s0 + i < a.splits && part[i].y != 0.0f;
            const float w = counts ? weight(part[i].x, m) : 0.0f;
            l = fmaf(w, counts ? part[i].y : 0.0f, l);
#pragma unroll
            for (int x = 0; x < 4; ++x) sum[x] = fmaf(w, counts ? o[i][x] : 0.0f, sum[x]);
        }
    }
    *(f32x4 *)(a.out + row * D + c) = l == 0.0f ? f32x4{} : sum / l;
    if (a.lse && c == 0) a.lse[row] = log_sum(m, l);
}

// Joins the parts of each row: out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
// One workgroup per row: the parts' weights first, then groups of D / 4 threads
// share the parts out, so that many parts are many loads in flight.
constexpr int kJoinThreads = 512;

__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttendArgs a, int64_t first)
{
    __shared__ float s_w[kMaxSplits], s_wave[kJoinThreads / 64];
    __shared__ float s_l[kMaxSplits];
    __shared__ f32x4 s_o[kJoinThreads];
    const int D = a.cache.head_dim, tid = threadIdx.x, wave = tid >> 6;
    const int64_t rows_all = (int64_t)a.tokens * a.q_heads, row = first + blockIdx.x;
    if (!of_a_request(a, row)) return;
    float m = kNone;
    for (int s = tid; s < a.splits; s += kJoinThreads) {
        const float *ml = a.part_ml + (s * rows_all + row) * 2;
        s_w[s] = ml[0];
        s_l[s] = ml[1];
        m = fmaxf(m, ml[0]);
    }
#pragma unroll
    for (int d = 32; d; d /= 2) m = fmaxf(m, __shfl_xor(m, d));
    if ((tid & 63) == 0) s_wave[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinThreads / 64; ++w) m = fmaxf(m, s_wave[w]);
    // A part that has seen nothing has l = 0 and is left out, by a weight below 0: one
    // whose weight is 0 because its scores are far lower has to bring its NaNs.
    for (int s = tid; s < a.splits; s += kJoinThreads) {
        const float w = s_l[s] == 0.0f ? -1.0f : weight(s_w[s], m);
        s_w[s] = w;
        s_l[s] *= w;
    }
    __syncthreads();
    const int wide = D / 4, groups = kJoinThreads / wide, group = tid / wide;
    const int c = tid % wide * 4;
    f32x4 sum = {};
    if (group < groups)
#pragma unroll 8
        for (int s = group; s < a.splits; s += groups) {
            const f32x4 o = *(const f32x4 *)(a.part_o + (s * rows_all + row) * D + c);
            if (!(s_w[s] < 0.0f)) sum += s_w[s] * o;
        }
    s_o[tid] = sum;
    float l = 0.0f;
    for (int s = tid & 63; s < a.splits; s += 64) l += s_l[s];
#pragma unroll
    for (int d = 32; d; d /= 2) l += __shfl_xor(l, d);
    __syncthreads();
    if (tid < wide) {
        for (int i = 1; i < groups; ++i) sum += s_o[i * wide + tid];
        *(f32x4 *)(a.out + row * D + c) = l == 0.0f ? f32x4{} : sum / l;
        if (a.lse && tid == 0) a.lse[row] = log_sum(m, l);
    }
}

}  // namespace

AttendShape attend_shape(int tokens, int batch, int kv_heads, int group, int head_dim,
                         int64_t max_q, int64_t max_len, int64_t window)
{
    return attend_shape_of(tokens, batch, kv_heads, group, head_dim, max_q, max_len, window);
}

template <int NB, bool PACK>
static void launch_few(const AttendArgs &a, unsigned grid, hipStream_t stream)
{
    if (a.waves == 8)
        attend_few_kernel<NB, PACK, 8><<<grid, 512, 0, stream>>>(a);
    else
        attend_few_kernel<NB, PACK, 4><<<grid, 256, 0, stream>>>(a);
}

template <int NB>
static void launch_few(const AttendArgs &a, unsigned grid, hipStream_t stream)
{
    if (a.tile_rows == 8)
        launch_few<NB, true>(a, grid, stream);
    else
        launch_few<NB, false>(a, grid, stream);
}

static hipError_t launch_requests(const AttendArgs &a, hipStream_t stream)
{
    const unsigned grid = (unsigned)a.requests * a.cache.kv_heads * a.tiles * a.splits;
    if (!a.few) {
        launch_attend_many(a, grid, stream);
    } else {
        switch (a.cache.head_dim) {
        case 64: launch_few<2>(a, grid, stream); break;
        case 96: launch_few<3>(a, grid, stream); break;
        case 128: launch_few<4>(a, grid, stream); break;
        case 192: launch_few<6>(a, grid, stream); break;
        case 256: launch_few<8>(a, grid, stream); break;
        default: return hipErrorInvalidValue;
        }
    }
    return hipGetLastError();
}

hipError_t launch_attend(const AttendArgs &args, hipStream_t stream)
{
    AttendArgs a = args;
    const int most = requests_per_launch(a.cache.kv_heads, a.tiles, a.splits);
    for (a.first = 0; a.first < a.batch; a.first += a.requests) {
        a.requests = a.batch - a.first < most ? a.batch - a.first : most;
        if (hipError_t err = launch_requests(a, stream)) return err;
    }
    const int64_t rows = (int64_t)a.tokens * a.q_heads;
    for (int64_t first = 0; a.splits > 1 && first < rows; first += kJoinRows) {
        const int64_t n = rows - first < kJoinRows ? rows - first : kJoinRows;
        if (a.splits <= kFewSplits) {
            const int64_t threads = n * (a.cache.head_dim / 4);
            join_few_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, stream>>>(a, first);
        } else {
            join_kernel<<<(unsigned)n, kJoinThreads, 0, stream>>>(a, first);
        }
    }
    return hipGetLastError();
}

}  // namespace qmm
