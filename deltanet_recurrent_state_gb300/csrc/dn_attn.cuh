// Shared by the attention kernels over a paged cache: their arguments, how the work is cut into
// units, and where a unit's partial result goes.
//
// Rows. The G query heads of a key head see the same keys, so a request's n tokens x G heads of one
// key head are n * G rows of one product; row r is token r / G, head h * G + r % G. A tile is M rows.
//
// Units. A unit is a tile, a key head and a range of cached tokens, the work of one CTA. Lengths are
// known on the device only, so every CTA finds its own unit: its warps read the B requests' lengths,
// sum the work (tiles x tokens x heads), choose a range length C, and look their unit up in the running
// count. If there are fewer tiles than half the CTAs that run at once, C makes one wave of equal ranges (a
// single request's long cache: D = 256, one token over 25,000, took 27.7 us so and 39.5 in four waves).
// Else it is the longest span divided by the f that an estimate of the time likes best (attn_time), a lane to
// each: more ranges even out a batch's end, and each costs its CTA's beginning and end. A request's ranges
// are of one length. The host sizes the grid by a bound; CTAs past the last unit leave.
//
// Partials. A tile seen in one range is finished by its unit. Otherwise every range leaves the running
// maximum, the sum and the unnormalised output of its rows (32 bits) in a slot of the workspace,
// and attn_join_kernel adds them in the order of the ranges, so results repeat bit for bit. Only
// requests with at least two ranges own slots, and those have about 2 * max(target, wave) of them at
// most (a request of span > C has fewer than 2 span / C ranges), whatever B and the lengths are.
#pragma once

#include "dn.h"
#include "dn_device.cuh"
#include "dn_kv.cuh"

namespace dn {

constexpr int kAttnSms = 152;  // GB300

// 2^x within 2 units in the last place; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct AttnArgs {
    KvPool p;
    const void *q;
    long long q_stride;  // elements between packed rows of q
    const void *kc, *vc;
    const uint8_t *ke, *ve;
    void *out;
    float *lse;   // may be null
    float *part;  // slots of attn_slot(M, D) floats
    int G;
    float scale_log2;  // scale * log2(e): scores are kept in powers of two
    int window;        // 0: none
    int M;             // rows of a tile
    int align;         // ranges start at multiples of this many tokens (a power of two)
    int wave, target;  // units: CTAs that run at once, and of a batch (at least as many)
    int min_range;
    int unit_cost, join_cost;  // of a unit's beginning and end, and of joining, in tokens of a CTA's work
    bool soft;                 // memory-bound: a wave that is not full runs faster
};

struct AttnUnit {
    int b, h, t, c;        // request, key head, tile, range
    int s, n, first, len;  // packed rows [s, s + n); position of the first; cached tokens
    int lo, hi;            // cached tokens of this unit; lo is rounded down to a multiple of align
    int see;               // the first that any row of the tile sees: what a window leaves in lo .. see - 1 may hold anything
    int ranges;            // ranges of this tile that see anything (at least 1)
    int slot;              // workspace slot of range 0 of this tile (ranges > 1)
};

// Floats of a slot: M rows of D, then M pairs (maximum, sum). Rows are read and written four floats at a time, so
// every slot begins on 16 bytes, also where a tile has an odd number of rows (D = 256 with 5 heads: 125).
__host__ __device__ constexpr size_t attn_slot(int M, int D) { return ((size_t)M * (D + 2) + 3) / 4 * 4; }

__host__ __device__ inline long long attn_tiles_bound(int B, int total, int G, int M) {
    const long long rows = (long long)total * G;
    return rows / M + (B < total ? B : total);
}
// a / b for a >= 0, b > 0. Most of a unit's search is divisions, and an integer one takes about 100 cycles:
// below 2^21 the quotient of 32-bit floats (2 units in the last place) is off by less than one before it is
// cut, so by one at most before the correction.
__device__ __forceinline__ int attn_div(int a, int b) {
    if (a >= 1 << 21 || b >= 1 << 24) return a / b;
    int q = (int)__fdividef((float)a, (float)b);
    const int r = a - q * b;
    q += r >= b ? 1 : r < 0 ? -1 : 0;
    return q;
}
__device__ __forceinline__ int attn_ceil_div(int a, int b) { return attn_div(a + b - 1, b); }

// A request's packed rows, cached tokens, tiles and the most tokens that one of its tiles sees.
struct AttnRequest {
    int s, n, first, len, tiles, span;
};
__device__ __forceinline__ AttnRequest attn_request(const AttnArgs &a, int b) {
    AttnRequest r;
    packed_rows(a.p, b, r.s, r.n);
    const int held = held_tokens(a.p, b);
    r.first = held - r.n;
    r.len = min(held, a.p.max_pages << a.p.page_shift);
    r.tiles = attn_ceil_div(r.n * a.G, a.M);  // (the host bounds total * heads by 2^31 - 1 - 1024)
    r.span = a.window ? min(r.len, a.window + attn_div(a.M - 1, a.G) + 1 + a.align) : r.len;  // (window <= 2^30)
    return r;
}

// Estimated time, in tokens of one CTA, of tiles (with heads) of `all` tokens together and at most `longest` each,
// cut into ranges of C.
__device__ __forceinline__ float attn_time(const AttnArgs &a, float tiles, float all, float longest, float C) {
    const float mean = __fdividef(all, tiles), wave = (float)a.wave, cost = (float)a.unit_cost;
    const bool even = mean >= 0.9f * longest;
    const float units = tiles * fmaxf(1.f, ceilf(even ? __fdividef(longest, C) - 1e-3f : __fdividef(mean, C) - 0.1f));
    const float waves = __fdividef(units, wave);
    float t;
    if (a.soft) t = fmaxf(C, __fdividef(all, wave) + 0.5f * C) + cost * fmaxf(1.f, waves);
    else if (waves <= 1.f) t = C + cost;
    else if (even) t = ceilf(waves) * (C + cost);
    else t = __fdividef(all, wave) + 0.5f * C + cost * waves;
    return C < longest ? t + (float)a.join_cost : t;
}

// The unit with this number (JOIN: the tile and head with this number among those of requests with
// several ranges), found by one warp; false if there is none.
template <bool JOIN>
__device__ __forceinline__ bool attn_unit(const AttnArgs &a, int idx, AttnUnit &u) {
    const int lane = threadIdx.x % 32, B = a.p.B, unit_log2 = 31 - __clz(a.align);
    AttnRequest r = {};
    long long work = 0;
    int whole = 0, longest = 0;  // tiles; the longest span
    if (B == 1) {   // (every lane has the one request: nothing to add up or to hand round)
        r = attn_request(a, 0);
        work = (long long)r.tiles * r.span;
        whole = r.tiles;
        longest = r.span;
    } else {
        for (int i = 0; i < B; i += 32) {
            r = AttnRequest{};
            if (i + lane < B) r = attn_request(a, i + lane);
            work += (long long)r.tiles * r.span;
            whole += r.tiles;
            longest = max(longest, r.tiles ? r.span : 0);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) work += __shfl_xor_sync(0xffffffffu, work, off);
        whole = __reduce_add_sync(0xffffffffu, whole);
        longest = __reduce_max_sync(0xffffffffu, longest);
    }
    // C in units of align tokens (2^24 at most), not below all / target, which bounds the units and slots; 2^-20 less,
    // so that what fits is not rounded up, which the slots' margin covers
    // (a 64-bit integer to float goes through the fp64 pipe, so it goes in two parts)
    const float all = ((float)(int)(work >> 24) * 16777216.f + (float)(int)(work & 0xffffff)) * (float)a.p.heads, tiles_all = (float)whole * (float)a.p.heads;
    const bool few = 2 * (long long)whole * a.p.heads < a.wave;
    auto at_least = [&](int units) {
        return (int)fminf(ceilf(__fdividef(all, (float)units * (float)a.align) * (1.f - 0x1p-20f)), 16777215.f);
    };
    const int least = a.min_range >> unit_log2;
    int most = max(at_least(few ? a.wave : a.target), least);
    if (few && longest <= (most << unit_log2) + a.join_cost) most = 16777215;  // joining would take longer than the rest
    if (!few) {
        const int units = (longest + a.align - 1) >> unit_log2, mine = attn_ceil_div(max(units, 1), lane + 1);
        const float t = attn_time(a, tiles_all, all, (float)longest, (float)mine * (float)a.align);
        // (the time in 27 bits, the lane in five: the fewest ranges of the best)
        const unsigned key = (mine >= most || lane == 0 ? (unsigned)fminf(t, 67108863.f) << 5 : 0xffffffe0u) | lane;
        most = max(__shfl_sync(0xffffffffu, mine, __reduce_min_sync(0xffffffffu, key) & 31), least);
    }
    // equal ranges of at most `most`
    auto cut = [&](int span, int &step) {
        const int units = (span + a.align - 1) >> unit_log2;
        step = units;
        if (units > most) step = attn_ceil_div(units, attn_ceil_div(units, most));
        step = max(step, least);
        return units > step ? attn_ceil_div(units, step) : 1;
    };
    int before = 0, slots_before = 0;
    for (int i = 0; i < B; i += 32) {
        if (B > 32) {  // (else the values of the loop above)
            r = AttnRequest{};
            if (i + lane < B) r = attn_request(a, i + lane);
        }
        int step;
        const int ranges = cut(r.span, step);
        const int slots = ranges > 1 ? r.tiles * ranges * a.p.heads : 0;
        const int units = JOIN ? (ranges > 1 ? r.tiles * a.p.heads : 0) : r.tiles * ranges * a.p.heads;
        int upto = units, slots_upto = slots;
        if (B > 1) {
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, off), y = __shfl_up_sync(0xffffffffu, slots_upto, off);
                if (lane >= off) {
                    upto += x;
                    slots_upto += y;
                }
            }
        }
        const unsigned past = __ballot_sync(0xffffffffu, idx < before + upto);
        if (past) {
            const int at = __ffs(past) - 1;
            auto from = [&](int x) { return B == 1 ? x : __shfl_sync(0xffffffffu, x, at); };
            u.b = i + at;
            u.s = from(r.s);
            u.n = from(r.n);
            u.first = from(r.first);
            u.len = from(r.len);
            const int T = from(r.tiles), R = from(ranges);
            step = from(step) << unit_log2;  // (2^30 + align at most)
            int local = idx - before - from(upto - units);
            // neighbours in the grid are tiles of one range, so they share its pages in L2; the
            // last tile of a prompt, which sees most, comes first
            int q = T > 1 ? attn_div(local, T) : local;
            u.t = T - 1 - (local - q * T);
            local = q;
            q = JOIN || R == 1 ? local : attn_div(local, R);
            u.c = JOIN ? 0 : local - q * R;
            u.h = q;
            u.slot = slots_before + from(slots_upto - slots) + (u.h * T + u.t) * R;
            const int r0 = u.t * a.M, r1 = min(a.M, u.n * a.G - r0) - 1 + r0;
            const int hi = min(max(u.first + attn_div(r1, a.G) + 1, 0), u.len);
            u.see = a.window ? max(u.first + attn_div(r0, a.G) - a.window + 1, 0) : 0;
            const int lo = min(u.see & ~(a.align - 1), hi);
            u.ranges = hi - lo > step ? attn_ceil_div(hi - lo, step) : 1;
            u.lo = u.c < u.ranges ? lo + u.c * step : hi;
            u.hi = hi - u.lo > step ? u.lo + step : hi;
            return true;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
        slots_before += __shfl_sync(0xffffffffu, slots_upto, 31);
    }
    return false;
}

// Entry of the join kernel (dn_attn.cu), shared by both attention kernels.
void launch_attn_join(const AttnArgs &a, int D, bool bf, cudaStream_t st);
// Tiles of 128 rows on tcgen05 (dn_attn_tc.cu).
dn_status launch_attn_tc(const AttnArgs &a, int D, bool bf, bool kv8, unsigned grid, cudaStream_t st);

}  // namespace dn
