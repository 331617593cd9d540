// Shared by the attention kernels over a paged cache: their arguments, how the work is cut into
// units, and where a unit's partial result goes.
//
// Rows. The G query heads of a key head see the same keys, so a request's n tokens x G heads of one
// key head are n * G rows of one product; row r is token r / G, head h * G + r % G. A tile is M rows.
//
// Units. A unit is a tile, a key head and a range of cached tokens, the work of one CTA. Lengths are
// known on the device only, so every CTA finds its own unit: its warps read the B requests' lengths,
// sum the work (tiles x tokens x heads), take the range length C that makes so many units of it, and look
// their unit up in the running count. If there are fewer tiles than half the CTAs that run at once, that
// is one wave of equal ranges (a single request's long cache: D = 256, one token over 25,000, took 27.7 us so
// and 39.5 in four waves); else it is a few waves, whose ends even out requests of all lengths (64
// requests: 173 us against 191 in one wave). A request's ranges are of one length. The host sizes the grid
// by a bound; CTAs past the last unit leave.
//
// Partials. A tile seen in one range is finished by its unit. Otherwise every range leaves the running
// maximum, the sum and the unnormalised output of its rows (32 bits) in a slot of the workspace,
// and attn_join_kernel adds them in the order of the ranges, so results repeat bit for bit. Only
// requests with at least two ranges own slots, and those have fewer than 2 * max(target, wave) of them
// (a request of span > C has fewer than 2 span / C ranges), whatever B and the lengths are.
#pragma once

#include "dn.h"
#include "dn_device.cuh"
#include "dn_kv.cuh"

namespace dn {

constexpr int kAttnSms = 152;  // GB300

struct AttnArgs {
    KvPool p;
    const void *q;
    long long q_stride;  // elements between packed rows of q
    const void *kc, *vc;
    const uint8_t *ke, *ve;
    void *out;
    float *lse;   // may be null
    float *part;  // slots of M * (D + 2) floats
    int G;
    float scale_log2;  // scale * log2(e): scores are kept in powers of two
    int window;        // 0: none
    int M;             // rows of a tile
    int align;         // ranges start at multiples of this many tokens (a power of two)
    int wave, target;  // units: CTAs that run at once, and of a batch (at least as many)
    int min_range;
};

struct AttnUnit {
    int b, h, t, c;        // request, key head, tile, range
    int s, n, first, len;  // packed rows [s, s + n); position of the first; cached tokens
    int lo, hi;            // cached tokens of this unit
    int ranges;            // ranges of this tile that see anything (at least 1)
    int slot;              // workspace slot of range 0 of this tile (ranges > 1)
};

__host__ __device__ inline long long attn_tiles_bound(int B, int total, int G, int M) {
    const long long rows = (long long)total * G;
    return rows / M + (B < total ? B : total);
}
// A request's packed rows, cached tokens, tiles and the most tokens that one of its tiles sees.
__device__ __forceinline__ void attn_request(const AttnArgs &a, int b, int &s, int &n, int &first, int &len, int &tiles,
                                             int &span) {
    packed_rows(a.p, b, s, n);
    const int held = min(max(__ldg(&a.p.kv_len[b]), 0), 1 << 30);
    first = held - n;
    len = min(held, a.p.max_pages << a.p.page_shift);
    tiles = (n * a.G + a.M - 1) / a.M;  // (the host bounds total * heads by 2^31 - 1 - M)
    span = a.window ? min(len, a.window + (a.M - 1) / a.G + 1 + a.align) : len;  // (window <= 2^30)
}

// The unit with this number (JOIN: the tile and head with this number among those of requests with
// several ranges), found by one warp; false if there is none.
template <bool JOIN>
__device__ __forceinline__ bool attn_unit(const AttnArgs &a, int idx, AttnUnit &u) {
    const int lane = threadIdx.x % 32, B = a.p.B;
    long long work = 0;
    int whole = 0;  // tiles
    int s = 0, n = 0, first = 0, len = 0, tiles = 0, span = 0;
    for (int i = 0; i < B; i += 32) {
        tiles = span = 0;
        if (i + lane < B) attn_request(a, i + lane, s, n, first, len, tiles, span);
        work += (long long)tiles * span;
        whole += tiles;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) work += __shfl_xor_sync(0xffffffffu, work, off);
    whole = __reduce_add_sync(0xffffffffu, whole);
    const int target = 2 * (long long)whole * a.p.heads < a.wave ? a.wave : a.target;
    // C = work * heads / target, rounded up to a multiple of align: in 32 bits unless the work is huge
    work = work * a.p.heads + target - 1;
    const long long C = work < 0x7fffffff ? (int)work / target : work / target;
    const int most = max((int)min((C + a.align - 1) & ~(long long)(a.align - 1), 1ll << 30), a.min_range);
    int before = 0, slots_before = 0;
    for (int i = 0; i < B; i += 32) {
        if (B > 32) {  // (else the values of the loop above)
            tiles = span = 0;
            if (i + lane < B) attn_request(a, i + lane, s, n, first, len, tiles, span);
        }
        // equal ranges of at most `most` tokens (all at most 2^30)
        const int cut = max(1, (span + most - 1) / most), range = max(a.min_range, ((span + cut - 1) / cut + a.align - 1) & ~(a.align - 1));
        const int ranges = max(1, (span + range - 1) / range);
        const int slots = ranges > 1 ? tiles * ranges * a.p.heads : 0;
        const int units = JOIN ? (ranges > 1 ? tiles * a.p.heads : 0) : tiles * ranges * a.p.heads;
        int upto = units, slots_upto = slots;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, off), y = __shfl_up_sync(0xffffffffu, slots_upto, off);
            if (lane >= off) {
                upto += x;
                slots_upto += y;
            }
        }
        const unsigned past = __ballot_sync(0xffffffffu, idx < before + upto);
        if (past) {
            const int at = __ffs(past) - 1;
            auto from = [&](int x) { return __shfl_sync(0xffffffffu, x, at); };
            u.b = i + at;
            u.s = from(s);
            u.n = from(n);
            u.first = from(first);
            u.len = from(len);
            const int T = from(tiles), R = from(ranges), step = from(range);
            int local = idx - before - from(upto - units);
            // neighbours in the grid are tiles of one range, so they share its pages in L2; the
            // last tile of a prompt, which sees most, comes first
            u.t = T - 1 - local % T;
            local /= T;
            u.c = JOIN ? 0 : local % R;
            u.h = JOIN ? local : local / R;
            u.slot = slots_before + from(slots_upto - slots) + (u.h * T + u.t) * R;
            const int r0 = u.t * a.M, r1 = min(a.M, u.n * a.G - r0) - 1 + r0;
            const int hi = min(max(u.first + r1 / a.G + 1, 0), u.len);
            int lo = a.window ? max(u.first + r0 / a.G - a.window + 1, 0) : 0;
            lo = min(lo & ~(a.align - 1), hi);  // (align is a power of two)
            u.ranges = max(1, (hi - lo + step - 1) / step);
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
