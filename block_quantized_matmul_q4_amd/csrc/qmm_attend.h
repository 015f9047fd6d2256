// Device code shared by the attention kernels over the paged Q4_0 cache
// (attend.hip: few rows per request; attend_many.hip: more).
#pragma once

#include <utility>

#include "qmm_attend_rows.h"
#include "qmm_internal.h"
#include "qmm_kv.h"

namespace qmm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kNone = -INFINITY;
// The running maximum of a row that has seen nothing: the first score passes it,
// and what is added to scores stays finite
constexpr float kLowest = -3.4028234e38f;
constexpr float kUpLog = 12.0f;     // p is carried times 2^12
constexpr float kUp = 4096.0f;

union Frag {
    f16x8 v;
    f16x2 h[4];
    uint32_t u[4];
};

// Largest value over the four lane groups, in every lane.
__device__ __forceinline__ float groups_max(float v)
{
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float groups_sum(float v)
{
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Largest of a lane's eight values (NaNs left out).
template <typename T>
__device__ __forceinline__ float largest(const T (&v)[2])
{
    return fmaxf(fmaxf(fmaxf(fmaxf(v[0][0], v[0][1]), v[0][2]), fmaxf(fmaxf(v[0][3], v[1][0]), v[1][1])),
                 fmaxf(v[1][2], v[1][3]));
}

// x + f * (fp16 half HIGH of w), in f32 (one rounding)
template <int HIGH>
__device__ __forceinline__ float plus_half(float x, float f, uint32_t w)
{
    float y;
    if constexpr (HIGH)
        asm("v_fma_mix_f32 %0, %1, %2, %3 op_sel:[0,1,0] op_sel_hi:[0,1,0]"
            : "=v"(y) : "v"(f), "v"(w), "v"(x));
    else
        asm("v_fma_mix_f32 %0, %1, %2, %3 op_sel_hi:[0,1,0]" : "=v"(y) : "v"(f), "v"(w), "v"(x));
    return y;
}

// Two values as fp16, to nearest (even).
__device__ __forceinline__ uint32_t two_halves(float x0, float x1)
{
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)x0, (_Float16)x1});
}

// The second terms of two values whose first terms are hi: fp16(x - hi).
__device__ __forceinline__ uint32_t second_terms(float x0, float x1, uint32_t hi, float minus = -1.0f)
{
    return two_halves(plus_half<0>(x0, minus, hi), plus_half<1>(x1, minus, hi));
}

// Factor of a part with maximum m where the whole has the maximum `all`. Both
// are -inf where a row has seen nothing (its sums are 0) or only NaN scores
// (its sums are NaN and have to stay).
__device__ __forceinline__ float weight(float m, float all)
{
    return all == kNone ? 1.0f : __builtin_amdgcn_exp2f(m - all);
}

// log of the sum of exp(s), from the maximum in units of log 2 and the sum of
// 2^12 exp(s - max)
__device__ __forceinline__ float log_sum(float m, float l)
{
    return l == 0.0f ? kNone : (m - kUpLog + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

// Constants that an instruction can take next to each other (one from a scalar
// register, one from a vector register), so that (x & mask) | bits is one.
struct Patterns {
    uint32_t mid_mask = 0x03C003C0u, mid = 0x4C004C00u;     // bits 6-9: 16 + q
    uint32_t low_mask = 0x000F000Fu, low = 0x64006400u;     // bits 0-3: 1024 + q
    uint32_t high_mask = 0x00F000F0u, high = 0x54005400u;   // bits 4-7: 64 + q
    __device__ __forceinline__ Patterns()
    {
        asm("" : "+s"(mid_mask), "+s"(low_mask), "+s"(high_mask));
        asm("" : "+v"(mid), "+v"(low), "+v"(high));
    }
};

// 16 + q of a word's nibbles, the order in which q's fragments are laid out:
// low nibbles of bytes 0, 2 and 1, 3, then the high ones.
__device__ __forceinline__ void offset_codes(const Patterns &c, uint32_t w, Frag &f)
{
    f.u[0] = ((w << 6) & c.mid_mask) | c.mid;
    f.u[1] = ((w >> 2) & c.mid_mask) | c.mid;
    f.u[2] = ((w << 2) & c.mid_mask) | c.mid;
    f.u[3] = ((w >> 6) & c.mid_mask) | c.mid;
}

// q - 8 of a V word (bytes: keys 0, 2, 1, 3 of four): the low nibbles of keys
// 0, 1 and 2, 3, and the high ones.
__device__ __forceinline__ void codes_of(const Patterns &c, uint32_t w, f16x2 *low, f16x2 *high)
{
    const f16x2 from1024 = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    const f16x2 from64 = {(_Float16)-72.0f, (_Float16)-72.0f};
    const uint32_t w8 = w >> 8;
    low[0] = __builtin_bit_cast(f16x2, (w & c.low_mask) | c.low) + from1024;
    low[1] = __builtin_bit_cast(f16x2, (w8 & c.low_mask) | c.low) + from1024;
    high[0] = __builtin_bit_cast(f16x2, (w & c.high_mask) | c.high) + from64;
    high[1] = __builtin_bit_cast(f16x2, (w8 & c.high_mask) | c.high) + from64;
}

template <int N>
struct Words {
    uint32_t w[N];
};

template <int N>
__device__ __forceinline__ void load(Words<N> &to, const uint8_t *from)
{
    const uint32_t *p = (const uint32_t *)from;
#pragma unroll
    for (int i = 0; i + 4 <= N; i += 4) {
        const u32x4_a4 v = *(const u32x4_a4 *)(p + i);
        for (int c = 0; c < 4; ++c) to.w[i + c] = v[c];
    }
    if constexpr (N % 4 >= 2) {
        const u32x2_a4 v = *(const u32x2_a4 *)(p + N / 4 * 4);
        to.w[N / 4 * 4] = v[0];
        to.w[N / 4 * 4 + 1] = v[1];
    }
    if constexpr (N % 2) to.w[N - 1] = p[N - 1];
}

// v of lane LANE of each group of 16, in all of them
template <int LANE, typename T>
__device__ __forceinline__ T from_lane(T v)
{
    return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v),
                                                          0x150 + LANE, 0xF, 0xF, true));
}

// The 4 NB scales of keys 4 g .. 4 g + 3 (block after block) are shared out
// over the 16 lanes of group g and come to the others by DPP broadcasts; loaded
// whole into every lane they would take 4 times the registers and loads.
//
// K: a pair of scales per lane, so that a broadcast serves two multiply-adds.
// V: one fp16 per lane, or two from 17 scales on; converted to f32 they are
// broadcast by the multiplications themselves.
template <int NB>
struct ValueScales {
    static constexpr int kRegs = NB > 4 ? 2 : 1;
    float d[kRegs];

    __device__ __forceinline__ explicit ValueScales(uint32_t raw)
    {
        d[0] = half_lo(raw);
        if constexpr (kRegs == 2) d[1] = half_hi(raw);
    }
    // which of the four keys register j of lane n holds a scale of
    __device__ __forceinline__ static int key(int n, int j) { return (n * kRegs + j) & 3; }
    // scale of block I of key 4 g + R
    template <int I, int R>
    __device__ __forceinline__ float get() const
    {
        constexpr int at = 4 * I + R;
        return from_lane<at / kRegs>(d[at % kRegs]);
    }
};

// f(0), f(1), .. f(N - 1) with constants
template <typename F, int... I>
__device__ __forceinline__ void unrolled_over(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}

template <int N, typename F>
__device__ __forceinline__ void unrolled(F f)
{
    unrolled_over(f, std::make_integer_sequence<int, N>{});
}

// What a wave works on: the keys of 16 rows' tile that one part has.
template <int NB>
struct Half {               // codes and scales of 16 keys, of K or of V
    Words<NB> codes;
    uint32_t scales;
};

// Keeps the code around it where it is: not executed speculatively, not merged
// with the same code of another branch.
__device__ __forceinline__ void keep_branch() { asm volatile(""); }

__device__ __forceinline__ void keep_apart(uint32_t &v) { asm volatile("" : "+v"(v)); }

// Where 32 keys lie: their pages, -1 where none is to be read.
struct Pages {
    int at[2];
};

// The block table is read through the constant address space: its entries are
// the same for a whole wave and no kernel here writes them, and as vector loads
// they would make every step wait for all of its loads in flight (vector loads
// return in order).
typedef const __attribute__((address_space(4))) int32_t *TableEntries;

// The lane's own part of an address, kept a 32-bit number inside loops: an
// address is then a scalar base and that, without 64-bit additions.
__device__ __forceinline__ uint32_t offset(uint32_t v)
{
    asm("" : "+v"(v));
    return v;
}

// Finds and loads a request's keys for one wave (V_PAIRS: the scales of V in
// pairs, as those of K). A load's address is a scalar
// base and the lane's own offset, which stays the same throughout.
template <int NB, bool V_PAIRS>
struct Keys {
    static constexpr int D = 32 * NB;
    const uint8_t *base;            // the head's first chunk
    uint32_t page_bytes;            // below 2^27
    int num_pages, shift;
    TableEntries table;
    int last;                       // entry of the row
    uint32_t k_at, k_scale_at, v_at, v_scale_at;

    __device__ __forceinline__ Keys(const KvCache &cache, const int32_t *table, int width,
                                    int shift, int kvh, int n, int g)
        : base(cache.pages + (int64_t)kvh * ((D << shift) * 9 / 8)),
          page_bytes((uint32_t)cache.kv_heads * (uint32_t)((D << shift) * 9 / 8)),
          num_pages(cache.num_pages), shift(shift),
          table((TableEntries)(uintptr_t)table), last(width - 1)
    {
        // K: word g of each block of key n. V: byte n of each block of keys 4 g ..
        k_at = n * (D / 2) + g * NB * 4;
        v_at = g * (2 * D) + n * NB * 4;
        k_scale_at = g * NB * 8 + 4 * (n < 2 * NB ? n : n & 1);
        v_scale_at = V_PAIRS ? k_scale_at : g * NB * 8 + 2 * (n < 4 * NB ? n : n & 3);
    }
    // The table's entries for keys t0 .. t0 + 31 (t0 a multiple of 32), to be
    // looked up a step before they are used; pages() makes pages of them. Past the
    // request's end the table may hold anything; keys there are hidden by their
    // places.
    __device__ __forceinline__ Pages look_up(int t0) const
    {
        return {{table[kv_entry(t0, shift, last)], table[kv_entry(t0 + 16, shift, last)]}};
    }
    __device__ __forceinline__ Pages pages(const Pages &entries) const
    {
        Pages p;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            p.at[h] = kv_page_exists(entries.at[h], num_pages) ? entries.at[h] : -1;
        return p;
    }
    __device__ __forceinline__ const uint8_t *chunk(int page) const
    {
        return base + (uint64_t)(uint32_t)max(page, 0) * page_bytes;
    }
    __device__ __forceinline__ int place(int t) const { return t & ((1 << shift) - 1); }
    __device__ __forceinline__ void load_k(Half<NB> &to, int page, int t) const
    {
        const uint8_t *from = chunk(page), *scales = from + ((D / 2) << shift);
        load(to.codes, from + place(t) * (D / 2) + offset(k_at));
        to.scales = *(const uint32_t *)(scales + place(t) * (NB * 2) + offset(k_scale_at));
    }
    __device__ __forceinline__ void load_v(Half<NB> &to, int page, int t) const
    {
        const uint8_t *from = chunk(page) + ((D * 9 / 16) << shift);
        const uint8_t *scales = from + ((D / 2) << shift);
        load(to.codes, from + place(t) * (D / 2) + offset(v_at));
        if constexpr (V_PAIRS)
            to.scales = *(const uint32_t *)(scales + place(t) * (NB * 2) + offset(v_scale_at));
        else
            to.scales = *(const uint16_t *)(scales + place(t) * (NB * 2) + offset(v_scale_at));
    }
};

// The 32 NB values of a row of q that a lane holds, as the matrix cores take
// them: scaled by a power of two, so that the row's largest magnitude lies in
// [8, 16), two fp16 terms each. Scores times `factor` are in units of log 2.
template <int NB, bool PACK>
struct Query {
    Frag first[NB], second[PACK ? 1 : NB];
    float factor;

    // PACK: columns 8-15 take the second terms (minus = -1), columns 0-7 the
    // first (minus = 0) of the same rows
    __device__ __forceinline__ void load(const float *q, int g, float scale, float minus)
    {
        f32x4 x[NB][2];
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                x[i][h] = *(const f32x4 *)(q + 32 * i + 16 * h + 4 * g);
#pragma unroll
                for (int c = 0; c < 4; ++c) top = fmaxf(top, fabsf(x[i][h][c]));
            }
        top = groups_max(top);
        // 2^e with top 2^-e in [8, 16); rows of zeros or subnormals are taken as 2^-100
        const int e = max((int)(__float_as_uint(top) >> 23), 27) - 127 - 3;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        factor = fabsf(scale) * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
        // scores that are all 0: the factor may not be, it multiplies -inf too
        const float sign = factor == 0 ? 0.0f : scale < 0 ? -down : down;
        if (factor == 0) factor = 1.0f;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 y = x[i][h] * sign;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t hi = two_halves(y[c], y[c + 2]);
                    if constexpr (PACK) {
                        first[i].u[2 * h + c] = second_terms(y[c], y[c + 2], hi, minus);
                    } else {
                        first[i].u[2 * h + c] = hi;
                        second[i].u[2 * h + c] = second_terms(y[c], y[c + 2], hi);
                    }
                }
            }
    }
};

// Writes the joined result of row `packed` (of KV head kvh), columns c .. c + 3.
__device__ __forceinline__ void store_row(const AttendArgs &a, int q0, int kvh, int packed,
                                          int split, int D, int c, f32x4 sum, float m, float l)
{
    const int64_t row = (int64_t)(q0 + packed / a.group) * a.q_heads + kvh * a.group +
                        packed % a.group;
    if (a.splits == 1) {
        *(f32x4 *)(a.out + row * D + c) = l == 0.0f ? f32x4{} : sum / l;
        if (a.lse && c == 0) a.lse[row] = log_sum(m, l);
    } else {
        const int64_t at = split * ((int64_t)a.tokens * a.q_heads) + row;
        // a part in which the row has seen nothing leaves its sums unwritten
        if (l != 0.0f) *(f32x4 *)(a.part_o + at * D + c) = sum;
        if (c == 0) {
            a.part_ml[2 * at] = m;
            a.part_ml[2 * at + 1] = l;
        }
    }
}

}  // namespace
}  // namespace qmm
