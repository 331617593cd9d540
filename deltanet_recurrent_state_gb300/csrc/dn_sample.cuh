// The kernels of dn_accept_sampled, compiled for one type of logits in each of dn_sample_f16.cu, dn_sample_bf16.cu and dn_sample_f32.cu.
//
// A row's tokens are ordered by value (the lower index first among equal ones), and every filter keeps a prefix of
// that order: the first top_k, those of weight >= min_p, the shortest prefix with a mass of top_p. So what is kept is
// {x > tau} and the first r tokens with x == tau, and no sorting is needed: tau and r are found by counting, and the token
// is the first in index order at which the kept mass passes u times the total.
//
// One cluster of CTAs a row (one CTA where the rows alone fill the GPU). Each CTA reads its part of the row from HBM once, keeps the largest
// value of every 16-byte vector, and the part itself if it fits into shared memory (else it is read again, from L2, where
// that is needed). A warp has a run of vectors and its lanes one each at a step. CTAs exchange what follows through
// distributed shared memory, one cluster barrier an exchange.
//   Near the maximum. What the filters keep is nearly always a few tokens of many. A bound that at least k tokens reach comes from the
//   lanes' largest tokens alone: the k-th largest of one CTA's is one, and so is the least of all CTAs' (k / CTAs)-th. The
//   tokens above it are listed in index order; without a top_k (then some 64 are hoped to do) the mass of all tokens is summed in the
//   same step. If the lists hold all that the filters keep, one CTA takes them, compares each token with each for its place
//   and the mass before it, and finishes alone.
//   The whole row, where nothing is filtered or more is kept than the lists hold: a histogram of all tokens (of counts, then of
//   masses in 16 bits a token), and of a bin's parts while a bin holds more tokens than are listed, guesses tau, and a pass over the row sums
//   the exact masses above it and in all. They decide; a guess that was wrong moves to the next value, then by growing steps and halvings,
//   so the approximations cost time at most.
// Calls of many rows leave rows that need several such passes to a second kernel with eight CTAs for each of them.
//
// Exact masses. Which token a random number means is decided by sums over the vocabulary against borders that lie as dense as
// its tokens, so weights are taken to 2^-33 of themselves, 2^-36.7 in the mean square (a pair of floats: reduced argument, table, short
// series; P. T. P. Tang, "Table-driven implementation of the exponential function in IEEE floating-point arithmetic", 1989), and
// summed on fixed grids, 2^-43 of the largest over a row, where the order of a sum does not matter. 32-bit arithmetic would give another
// token than 64 bits do for one random number in some thousands over a flat row; this does for one in 10^7.
// That costs some 57 issue slots a token, and 32-bit arithmetic 13. So tokens of less than 2^-14 of the largest weight are summed in
// 32 bits at first, and the result counts only if no border lies within their error's bound (errors of equal tokens, and that of the
// scale, have one sign, so their averaging out is not counted on). The row is summed again exactly if one does: where light tokens make up a share f of
// a row, that is a row in 1 / f or fewer. With a top_p all tokens are taken exactly at once where that share is above 2^-10.
//
// What bounds it: a call of few rows is a chain of dependent steps (loads, four block and three cluster barriers, the comparison);
// one of many rows the arithmetic of those that need the mass of the whole row, with HBM's share at 11.5 us for 256 rows of 151,936 in
// 16 bits. Measured on a GB300, us: one row of 151,936 in fp16 with top_k 40 and top_p 0.9 11.3, with top_p 0.95 alone 13.4,
// without filters 13.6, at temperature 4 with top_p 0.95 50; 16 rows 14.1, 17.4, 18.2, 71; 256 rows in bf16 26.4, 47.5, 55.3, 568, and 48 with a
// mixture of the first three (88 if a row of it keeps thousands of tokens, or has to be summed again exactly).
// Registers: 64 a thread in every kernel, so that two CTAs fit an SM. Spilled, bytes of stores and loads: kEasy 16 to 48 and 24 to 80, kAll held 190 and
// 200, not held 510 to 570 and 740 to 800, kHard held 320 to 360 and 690 to 800, not held 1,600 to 1,650 and 1,460 to 1,630.
// (With 128 registers and one CTA an SM kHard, held, spills nothing: one flat row among 256 then takes 80 for 87, but 256 of them 773 for 580.)
#pragma once

#include <algorithm>
#include <type_traits>
#include <utility>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dn.h"
#include "dn_device.cuh"
#include "dn_internal.h"
#include "dn_sample.h"
#include "dn_vec.cuh"

namespace dn {
namespace sample {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kMaxSteps = 256;       // vectors of a lane, at most
constexpr int kListed = 1024;        // tokens (or values of a bin) that a CTA lists
constexpr int kMerged = 2560;        // values of a bin that all of them do
constexpr int kNear = 64;            // tokens to list where top_k does not say how many
constexpr int kSome = 512;           // listed tokens that are put together beside the part of the row, not in its place
constexpr int kFew = 256;            // listed tokens that are compared each with each
constexpr float kTail = 14.f;        // the negative binary logarithm of a weight that is summed in 32 bits at first
constexpr int kTailShift = 10;       // all of those make up much of a row from 2^-10 of it on
constexpr int kTailError = 16;       // their sum is off by less than 2^-16: y by 2^-22.3 of itself (at 60, where 400,000 such weights make up 2^-41, 2^-16.9
                                     // of the weight), the exponential by 2^-22, a sum of 32 by 2^-19
constexpr int kFixed = 43;           // sums over a row are in units of 2^-43 of the largest weight: 2^19 of them fit 64 bits
constexpr int kList = 50;            // over listed tokens, and a warp's tokens: units of 2^-50, 12,500 tokens
constexpr int kFine = 56;            // a token's own weight, and what a warp adds up below the units of a row: 2^-56
constexpr float kCountScale = 32.f;  // bins a unit of distance, for counts

// kAll: a kernel for all that a row may need. kEasy leaves rows that take several passes over all of their tokens to kHard, which
// has more CTAs for each of them.
enum Mode { kAll, kEasy, kHard };
constexpr unsigned kHeavy = 1u << 31;  // beside a row's number: its light tokens make up much of it

template <typename E> constexpr int kVecOf = 16 / (int)sizeof(E);
// Values of a 16-bit type differ, as 32-bit floats, above these bits.
template <typename E> constexpr int kKeyShift = sizeof(E) == 4 ? 0 : kIsBf16<E> ? 16 : 13;

template <typename E> __device__ __forceinline__ void decode(uint4 u, float (&x)[kVecOf<E>]) {
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(E) == 4) {
            x[i] = __uint_as_float(w[i]);
        } else {
            const float2 f = unpack2<kIsBf16<E>>(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}
template <typename E> __device__ __forceinline__ float2 pair_of(uint4 u, int j) {  // tokens 2 j and 2 j + 1
    if constexpr (sizeof(E) == 4) {
        return j ? make_float2(__uint_as_float(u.z), __uint_as_float(u.w)) : make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    } else {
        return unpack2<kIsBf16<E>>(j < 2 ? j < 1 ? u.x : u.y : j < 3 ? u.z : u.w);
    }
}
// The largest value of a vector, NaN where it holds nothing else.
template <typename E> __device__ __forceinline__ float largest(uint4 u) {
    if constexpr (sizeof(E) == 4) {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    } else {
        using E2 = typename std::conditional<kIsBf16<E>, __nv_bfloat162, __half2>::type;
        const E2 *h = reinterpret_cast<const E2 *>(&u);
        const E2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(static_cast<float>(m.x), static_cast<float>(m.y));
    }
}
template <typename E> __device__ __forceinline__ unsigned lowest_bits() {  // -infinity, twice for 16 bits
    return sizeof(E) == 4 ? 0xff800000u : kIsBf16<E> ? 0xff80ff80u : 0xfc00fc00u;
}

// Order-preserving integers of values (no NaN); -0 counts as +0.
template <typename E> __device__ __forceinline__ unsigned key_of(float x) {
    const unsigned b = __float_as_uint(x == 0.f ? 0.f : x);
    return ((b & 0x80000000u) ? ~b : (b | 0x80000000u)) >> kKeyShift<E>;
}
template <typename E> __device__ __forceinline__ float value_of(unsigned key) {
    const unsigned k = key << kKeyShift<E>;
    if (k & 0x80000000u) return __uint_as_float(k & 0x7fffffffu);
    return __uint_as_float(~(k | ((1u << kKeyShift<E>) - 1u)));
}

__device__ __forceinline__ float exp2_fast(float y) {  // to 2^-22; 0 below 2^-126
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return r;
}

// 2^(j / 16) as pairs of floats: 16 of 8 bytes lie in different banks of shared memory.
static __constant__ float2 kPowers[16] = {
    {1.f, 0.f}, {1.04427373f, 4.83347016e-08f}, {1.09050775f, -1.30775399e-08f}, {1.13878858f, 5.38622231e-08f},
    {1.18920708f, 3.79763527e-08f}, {1.24185777f, 4.4968381e-08f}, {1.29683959f, -4.01899953e-08f}, {1.35425556f, -1.01233493e-08f},
    {1.41421354f, 2.4203235e-08f}, {1.47682619f, -4.50089885e-08f}, {1.54221082f, 8.07090483e-09f}, {1.61049032f, 9.83621717e-09f},
    {1.68179286f, -2.47553267e-08f}, {1.75625217f, -9.23577037e-09f}, {1.8340081f, -1.1239278e-08f}, {1.91520655f, 9.84532811e-09f},
};

// A token's weight is 2^y, y = (x - top) (ch + cl). `least`: what lies below it is taken as this far down, 2^-60. `sharp`: only the
// largest has a weight, because it is infinite or the next float below it is less than 2^-60.
struct Scale {
    float top, ch, cl, least;
    bool sharp;
};

struct Entry {  // a token near the maximum
    unsigned key;
    int token;
    u64 weight;
};

struct Shared {
    u64 kept[2][kMaxCluster], all[2][kMaxCluster], tail[2][kMaxCluster];  // exchanged masses, two sets used in turn
    unsigned eq[2][kMaxCluster];
    float top[kMaxCluster], share[kMaxCluster], alone[kMaxCluster];
    u64 scan64[kWarps], scan64b[kWarps], scan64c[kWarps];
    unsigned scan32[kWarps], scan32b[kWarps];
    float scanf[kWarps];
    double floor_distance;  // what min_p leaves below the maximum
    u64 key_weight;
    int bin, reach[2], done, chosen, place;
    uint4 ends[2];  // the row's first and last vector, which it may share with its neighbours
    float before;
    unsigned lo, hi, listed, next;
    float2 powers[16];
    alignas(16) unsigned hist[kBins];
    union {
        struct {
            uint2 near[kListed];  // key and token
            Entry some[kSome];
        };
        struct {
            unsigned list[kListed], merged[kMerged];
        };
        struct {
            u64 part[kFew];
            unsigned part_rank[kFew];
        };
        struct {
            u64 step_mass[kMaxSteps];
            unsigned step_alike[kMaxSteps], step_kept[kMaxSteps];
        };
    };
};

// The weights of two tokens, each as a sum of two floats right to 2^-33 of itself. y = n + j / 16 + f with |f| <= 1/32; all in packed
// arithmetic, two tokens an instruction, with no sign to change on the way.
struct Weights {
    float2 hi, lo;
};
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
__device__ __forceinline__ Weights weights_of(float x0, float x1, const Scale &c, const float2 *powers) {
    if (c.sharp) return Weights{make_float2(x0 == c.top ? 1.f : 0.f, x1 == c.top ? 1.f : 0.f), two(0.f)};
    const float2 x = make_float2(fmaxf(x0, c.least), fmaxf(x1, c.least)), nt = two(-c.top);  // (NaN: least)
    const float2 s = __fadd2_rn(x, nt);
    const float2 bb = __fadd2_rn(s, two(c.top));                          // x as s has it
    const float2 ns = __fmul2_rn(s, two(-1.f));
    const float2 e = __fadd2_rn(__ffma2_rn(bb, two(-1.f), x), __fadd2_rn(nt, __fadd2_rn(bb, ns)));  // x - top = s + e
    const float2 p = __fmul2_rn(s, two(c.ch)), np = __fmul2_rn(ns, two(c.ch));
    const float2 q = __ffma2_rn(e, two(c.ch), __ffma2_rn(s, two(c.cl), __ffma2_rn(s, two(c.ch), np)));  // y = p + q
    const float2 t = __ffma2_rn(p, two(16.f), two(12582912.f));           // rounds to an integer
    const int k0 = __float_as_int(t.x) - 0x4b400000, k1 = __float_as_int(t.y) - 0x4b400000;
    const float2 f = __ffma2_rn(__fadd2_rn(t, two(-12582912.f)), two(-0.0625f), p);
    // 2^(f + q) = 1 + gh + zl,  g = (f + q) ln 2 = gh + gl,  e^g - 1 = g + g^2 (1/2 + g/6 + g^2/24 + g^3/120)
    const float2 gh = __fmul2_rn(f, two(0.693147182f)), ngh = __fmul2_rn(f, two(-0.693147182f));
    const float2 gl = __fadd2_rn(__ffma2_rn(f, two(0.693147182f), ngh), __ffma2_rn(f, two(-1.90465431e-09f), __fmul2_rn(q, two(0.693147182f))));
    const float2 g = __fadd2_rn(gh, gl);
    const float2 zl = __ffma2_rn(__fmul2_rn(g, g), __ffma2_rn(g, __ffma2_rn(g, __ffma2_rn(g, two(0.00833333333f), two(0.0416666667f)), two(0.166666667f)), two(0.5f)), gl);
    const float2 b0 = powers[k0 & 15], b1 = powers[k1 & 15];
    const float2 bh = make_float2(b0.x, b1.x), bl = make_float2(b0.y, b1.y);
    // (no product that is rounded by itself meets a sum: the compiler may make one operation of the two, and hi + lo would then count its rounding twice)
    const float2 hi = __ffma2_rn(bh, gh, bh);
    const float2 lo = __fadd2_rn(__ffma2_rn(bh, gh, __ffma2_rn(hi, two(-1.f), bh)), __fadd2_rn(bl, __ffma2_rn(bl, gh, __fmul2_rn(bh, zl))));
    const float2 power = make_float2(__int_as_float((127 + (k0 >> 4)) << 23), __int_as_float((127 + (k1 >> 4)) << 23));
    return Weights{__fmul2_rn(hi, power), __fmul2_rn(lo, power)};
}

// Two sums of up to 32 weights each. Parts on grids of 2^-18 and 2^-37 add up exactly in floats; the rest, of 2^-38 and 2^-25 of the weight at most, has
// an error of 2^-45 of the weights. (Equal tokens round alike, so a plain float sum of them is off by up to 2^-20 of itself however many lanes share it.)
struct Sum {
    float2 a = {0.f, 0.f}, b = {0.f, 0.f}, c = {0.f, 0.f};
    __device__ __forceinline__ void add(const Weights &w, bool first, bool second) {
        const float2 hi = make_float2(first ? w.hi.x : 0.f, second ? w.hi.y : 0.f), lo = make_float2(first ? w.lo.x : 0.f, second ? w.lo.y : 0.f);
        const float2 on = __fadd2_rn(__fadd2_rn(hi, two(48.f)), two(-48.f));  // the floats of 32 .. 64 have steps of 2^-18
        const float2 rest = __ffma2_rn(on, two(-1.f), hi);                    // (exact)
        const float2 mid = __fadd2_rn(__fadd2_rn(rest, two(0x1.8p-14f)), two(-0x1.8p-14f));  // those of 2^-14 .. 2^-13 of 2^-37
        a = __fadd2_rn(a, on);
        b = __fadd2_rn(b, mid);
        c = __fadd2_rn(c, __fadd2_rn(__ffma2_rn(mid, two(-1.f), rest), lo));
    }
    __device__ __forceinline__ u64 fixed() const {  // the parts on the grids, in units of 2^-kFixed (the two sums' sums are of 24 bits)
        return ((u64)(long long)__float2int_rn((a.x + a.y) * 0x1p18f) << (kFixed - 18)) +
               ((u64)(long long)__float2int_rn((b.x + b.y) * 0x1p37f) << (kFixed - 37));
    }
    // the rest, in units of 2^-kFine, and a sum of light tokens
    __device__ __forceinline__ long long fine(float2 light) const { return __float2ll_rn(((c.x + c.y) + (light.x + light.y)) * 0x1p56f); }
};
__device__ __forceinline__ u64 weight_of(float x, const Scale &c, const float2 *powers) {  // one token's, in units of 2^-kFine
    Sum s;
    s.add(weights_of(x, x, c, powers), true, false);
    return (s.fixed() << (kFine - kFixed)) + (u64)s.fine(two(0.f));
}
// Units of 2^-kFine as coarser ones of 2^-bits.
__device__ __forceinline__ u64 coarser(u64 fine, int bits) { return (fine + (1ull << (kFine - bits - 1))) >> (kFine - bits); }
__device__ __forceinline__ u64 rest_of(long long fine) { return (u64)((fine + (1ll << (kFine - kFixed - 1))) >> (kFine - kFixed)); }  // (below 0, too)
// The mass of n tokens alike, rounded down to units of 2^-kFixed, and the fewest of them with a mass of `need` (above 0; enough of them have it).
__device__ __forceinline__ u64 mass_of(unsigned n, u64 weight) {
    return (__umul64hi(n, weight) << (64 - kFine + kFixed)) | (n * weight >> (kFine - kFixed));
}
static __device__ __noinline__ unsigned fewest_of(u64 need, u64 weight) {
    unsigned n = (unsigned)(__ull2float_rn(need) * (float)(1 << (kFine - kFixed)) / __ull2float_rn(weight));  // 2^19 at most, so off by one at most
    while (mass_of(n, weight) < need) ++n;
    while (n > 0 && mass_of(n - 1, weight) >= need) --n;
    return n;
}

// Whether a value's tokens, with the mass before them and that up to them, begin before the goal or not, and reach it or not, and after
// how many, whichever way the masses and the goal are off by less than `error` of one another.
static __device__ __noinline__ bool certain(u64 before, u64 upto, u64 goal, u64 error, u64 weight) {
    auto apart = [&](u64 mass) { return mass >= goal + error || goal >= mass + error; };
    if (!apart(before) || !apart(upto)) return false;
    if (before >= goal || upto < goal) return true;
    const u64 need = goal - before;
    return need > error && fewest_of(need - error, weight) == fewest_of(need + error, weight);
}

static __device__ __noinline__ u64 weight_called(float x, Scale c, const float2 *powers) { return weight_of(x, c, powers); }
template <bool CALLED> __device__ __forceinline__ u64 weight_at(float x, const Scale &c, const float2 *powers) {
    return CALLED ? weight_called(x, c, powers) : weight_of(x, c, powers);
}

// The first bin at which the sum over bins from bin 0 on, `before` included, reaches the goal: its number (kBins if none) and what
// lies before it, in s.bin and s.before. v0, v1: bins 2 t and 2 t + 1 of thread t. Counts stay exact: they are below 2^24.
__device__ __forceinline__ void find_bin_here(Shared &s, float before, float goal, float v0, float v1) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float upto = v0 + v1;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float o = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += o;
    }
    if (lane == 31) s.scanf[warp] = upto;
    if (threadIdx.x == 0) s.bin = kBins;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += s.scanf[w];
    upto += before;
    const int mine = upto - v1 >= goal ? 2 * threadIdx.x : upto >= goal ? 2 * threadIdx.x + 1 : kBins;
    if (mine < kBins) atomicMin(&s.bin, mine);
    __syncthreads();
    if (s.bin == mine && mine < kBins) s.before = mine & 1 ? upto - v1 : upto - v1 - v0;
    __syncthreads();
}

static __device__ __noinline__ void find_bin_called(Shared &s, float before, float goal, float v0, float v1) { find_bin_here(s, before, goal, v0, v1); }
template <bool CALLED> __device__ __forceinline__ void find_bin(Shared &s, float before, float goal, float v0, float v1) {
    if (CALLED) find_bin_called(s, before, goal, v0, v1);
    else find_bin_here(s, before, goal, v0, v1);
}

// floor(f * all) for 0 < f < 1, and whether that left something off.
__device__ __forceinline__ u64 part_of(u64 all, float f, bool &part) {
    const int bits = __float_as_int(f), e = bits >> 23;
    const u64 m = (bits & 0x7fffff) | (e ? 0x800000 : 0);
    const int shift = 150 - max(e, 1);  // f = m 2^-shift, 24 <= shift <= 149
    const u64 hi = __umul64hi(all, m), lo = all * m;
    if (shift >= 128) {
        part = (hi | lo) != 0;
        return 0;
    }
    if (shift >= 64) {
        const u64 r = hi >> (shift - 64);
        part = lo != 0 || (r << (shift - 64)) != hi;
        return r;
    }
    part = (lo << (64 - shift)) != 0;
    return (hi << (64 - shift)) | (lo >> shift);
}

// One row. HELD: a CTA's part of it stays in shared memory. Else it is read again, from L2, where that is needed.
template <typename E, bool HELD, Mode MODE>
__device__ __forceinline__ void sample_row(const SampleArgs &a, Shared &s, uint4 *slice, int row, bool all_exact) {
    constexpr int VEC = kVecOf<E>;
    // The second kernel runs a row or two on an SM, so much of its time is that of fetching instructions: its loops over pairs of tokens
    // and over warps stay loops, and what it needs in several places is called. (A flat row: 60 us in a single call before, 38 after.)
    constexpr bool kShort = MODE == kHard;
    constexpr int kUnroll = kShort ? 1 : VEC / 2, kUnrollWarps = kShort ? 1 : kWarps;
    // the vectors if they are held, then their largest values, rounded up to bf16
    unsigned short *const crest = reinterpret_cast<unsigned short *>(slice + (HELD ? a.room : 0));
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = row / a.T;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const float kInf = __int_as_float(0x7f800000);

    auto here = cluster.barrier_arrive();  // before a peer's memory is written, the peer has to be at this row

    // ---- the slice, the request's parameters, the row's maximum ----
    const float given = a.temperature[b];
    const bool greedy = !(given > 0.f);
    // far from either end of the floats, where neither a token's distance times the scale nor min_p's distance overflows
    const float temp = greedy ? 1.f : fminf(fmaxf(given, 1e-30f), 1e36f);
    int k = a.top_k ? a.top_k[b] : 0;
    float p = a.top_p ? a.top_p[b] : 1.f;
    const float min_p = a.min_p ? a.min_p[b] : 0.f;
    const float uniform = a.uniform[row];
    const long long first = (long long)row * a.V;  // the row's first token in the tensor
    const int head = (int)(first % VEC);           // and its place in a vector
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const E *>(a.logits) + (first - head));
    const int vecs = (head + a.V + VEC - 1) / VEC, per_cta = (vecs + ranks - 1) / ranks;
    const int base = rank * per_cta, held = max(0, min(per_cta, vecs - base));  // this CTA's first vector, and how many it has
    // a warp has a run of them, of which its lanes take one each at a step: the order of the tokens is that of warp, step and lane
    const int per_warp = (per_cta + kWarps - 1) / kWarps, from = warp * per_warp, mine_end = min(from + per_warp, held);
    auto fetch = [&](int i) {  // vector i of this CTA
        if (HELD) return slice[i];
        const int v = base + i;
        return v == 0 ? s.ends[0] : v == vecs - 1 ? s.ends[1] : src[v];
    };
    float run_top = -kInf;  // the largest of this thread's tokens
    auto take = [&](int i, uint4 u) {
        if (HELD) slice[i] = u;
        const float m = largest<E>(u);
        crest[i] = __bfloat16_as_ushort(__float2bfloat16_ru(m));
        run_top = fmaxf(run_top, m);  // (not a NaN)
    };
    constexpr int kLoads = 8;  // of a thread in flight
    for (int i0 = from + lane; i0 < mine_end; i0 += 32 * kLoads) {
        uint4 u[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int i = i0 + j * 32, v = base + i;
            u[j] = make_uint4(0, 0, 0, 0);
            if (i < mine_end && v > 0 && v < vecs - 1) u[j] = HELD ? __ldcs(src + v) : src[v];
        }
        if (threadIdx.x == 0 && i0 == from && min_p > 0.f)  // 64-bit arithmetic is slow: one thread's, while the loads are on their way
            s.floor_distance = min_p < 1.f ? (double)temp * log((double)min_p) : 0.0;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int i = i0 + j * 32, v = base + i;
            if (i < mine_end && v > 0 && v < vecs - 1) take(i, u[j]);
        }
    }
    for (int v = 0; v < vecs; v += max(vecs - 1, 1)) {  // the row's ends may share a vector with its neighbours, or with nobody
        const int i = v - base;
        if (i < from || i >= mine_end || (i - from) % 32 != lane) continue;
        unsigned w[4] = {lowest_bits<E>(), lowest_bits<E>(), lowest_bits<E>(), lowest_bits<E>()};
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int at = v * VEC + j - head;
            if (at < 0 || at >= a.V) continue;
            if constexpr (sizeof(E) == 4) {
                w[j] = static_cast<const unsigned *>(a.logits)[first + at];
            } else {
                const unsigned h = static_cast<const unsigned short *>(a.logits)[first + at];
                w[j / 2] = j & 1 ? (w[j / 2] & 0xffffu) | (h << 16) : (w[j / 2] & 0xffff0000u) | h;
            }
        }
        const uint4 u = make_uint4(w[0], w[1], w[2], w[3]);
        s.ends[v ? 1 : 0] = u;
        take(i, u);
    }
    // what is kept of a request's filters; y of the weights: log2(e) / temperature as a pair of floats
    if (greedy || p <= 0.f) k = 1;  // the first of the largest alone
    if (!(p < 1.f) || k == 1) p = 1.f;
    if (k < 1 || k > a.V) k = a.V;
    const bool by_count = k < a.V, floors = k > 1 && min_p > 0.f;
    Scale scale = {0.f, 1.44269502f / temp, 0.f, 0.f, false};
    scale.cl = (fmaf(-scale.ch, temp, 1.44269502f) + 1.92596303e-8f) / temp;
    __syncthreads();

    // The token, and the accepted length by the last row of the request. One warp.
    auto finish = [&](int token, float logprob) {
        unsigned done = 0;
        if (lane == 0) {
            a.target[row] = token;
            if (a.logprob) a.logprob[row] = logprob;
            if (a.T > 1) {
                __threadfence();
                done = atomicAdd(&a.counters[b], 1u);
            }
        }
        done = __shfl_sync(0xffffffffu, done, 0);
        if (a.T > 1 && done != (unsigned)a.T - 1) return;
        __threadfence();
        int length = a.T;
        for (int t0 = 0; t0 < a.T && length == a.T; t0 += 32) {
            const int t = t0 + lane;
            const long long at = (long long)b * a.T + t;
            const bool miss = t < a.T && __ldg(&a.draft[at]) != (a.T > 1 ? __ldcg(&a.target[at]) : token);
            const unsigned m = __ballot_sync(0xffffffffu, miss);
            if (m) length = t0 + __ffs(m) - 1;
        }
        if (lane == 0) {
            a.accepted[b] = length;
            if (a.T > 1) a.counters[b] = 0;
        }
    };
    float top = run_top;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) s.scanf[warp] = top;
    __syncthreads();
    top = s.scanf[lane % kWarps];
#pragma unroll
    for (int off = kWarps / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    // A bound that at least `want` tokens reach, the first k or as many as are hoped to do: such a number of this CTA's threads' largest
    // reach `alone`, and the CTA's part of that number `share`. They are a bin's lower end, below it whatever was rounded.
    const int want = by_count ? k : min(kNear, ranks * kThreads / 4);
    const bool seek = MODE != kHard && k > 1 && want <= ranks * kThreads / 2 && (by_count || p < 1.f);
    float share = -kInf, alone = -kInf;
    if (seek) {
        const float y = run_top == top ? 0.f : (top - run_top) * kCountScale;
        if (y < (float)kBins && top > -kInf) atomicAdd(&s.hist[(int)y], 1u);
        __syncthreads();
        const int v0 = (int)s.hist[2 * threadIdx.x], v1 = (int)s.hist[2 * threadIdx.x + 1];
        int upto = v0 + v1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += o;
        }
        if (lane == 31) s.scan32[warp] = (unsigned)upto;
        if (threadIdx.x < 2) s.reach[threadIdx.x] = kBins;
        __syncthreads();
        for (int w = 0; w < warp; ++w) upto += (int)s.scan32[w];
        const int goals[2] = {(want + ranks - 1) / ranks, want};
#pragma unroll
        for (int g = 0; g < 2; ++g)
            if (upto >= goals[g] && upto - v0 - v1 < goals[g]) s.reach[g] = 2 * threadIdx.x + (upto - v1 < goals[g]);
        __syncthreads();
        const float step = (1.f + 0x1p-21f) / kCountScale;
        if (s.reach[0] < kBins) share = __fsub_rd(top, (float)(s.reach[0] + 1) * step);
        if (s.reach[1] < kBins) alone = __fsub_rd(top, (float)(s.reach[1] + 1) * step);
    }
    cluster.barrier_wait(std::move(here));
    if ((int)threadIdx.x < ranks) {
        *cluster.map_shared_rank(&s.top[rank], threadIdx.x) = top;
        *cluster.map_shared_rank(&s.share[rank], threadIdx.x) = share;
        *cluster.map_shared_rank(&s.alone[rank], threadIdx.x) = alone;
    }
    cluster.sync();
    share = kInf;
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i)
        if (i < ranks) top = fmaxf(top, s.top[i]), share = fminf(share, s.share[i]), alone = fmaxf(alone, s.alone[i]);
    if (top == -kInf) {  // nothing but masked tokens: the first
        if (rank == 0 && warp == 0) finish(0, 0.f);
        return;
    }
    scale.top = top;
    scale.least = fmaxf(top - 60.f / scale.ch, -3.4e38f);
    scale.sharp = !(scale.least < top) || top == kInf;
    const float floor = floors ? __double2float_ru((double)top + s.floor_distance) : -kInf;  // no token below it is kept
    const float lowest = fmaxf(floor, -3.40282347e38f);                                      // nor a masked one

    auto distance = [&](float x) { return x == top ? 0.f : top - x; };  // (infinity less itself)
    // a token's bin, kBins or more where it has none, for counts and for masses; NaN has none
    auto count_bin = [&](float x) {
        const float y = distance(x) * kCountScale;
        return y < (float)kBins ? (int)y : kBins;
    };
    // the bin of a mass is given by its exponent and the upper four bits of its fraction, and its share by its upper 16 bits; fewer for
    // a CTA of more than 2^16 tokens, all of which may lie in one bin of 32 bits
    const int dropped = max(0, 16 - __clz(per_cta * VEC - 1));
    auto mass_bits = [&](float x) { return (unsigned)__float_as_int(exp2_fast(scale.sharp ? (x == top ? 0.f : -200.f) : (x - top) * scale.ch)); };
    auto mass_bin = [&](unsigned bits) { return 0x7f0 - (int)(bits >> 19); };
    auto mass_share = [&](unsigned bits) { return ((bits & 0x7fffffu) | 0x800000u) >> (8 + dropped); };
    auto mass_unit = [&](int bin) { return __int_as_float(((0x3f800000 - (bin << 19)) & 0x7f800000) + (dropped << 23)); };  // of 2^-15, in the weight's octave
    // this thread's vectors f(u), and its tokens f(x)
    auto each_vector = [&](auto f) {
        if (HELD) {
            for (int i = from + lane; i < mine_end; i += 32) f(slice[i]);
            return;
        }
        uint4 now, next;  // two loads ahead of the work
        if (from + lane < mine_end) now = fetch(from + lane);
        if (from + lane + 32 < mine_end) next = fetch(from + lane + 32);
#pragma unroll 1
        for (int i = from + lane; i < mine_end; i += 32) {
            const uint4 u = now;
            now = next;
            if (i + 64 < mine_end) next = fetch(i + 64);
            f(u);
        }
    };
    auto each = [&](auto f) {
        each_vector([&](uint4 u) {
            float x[VEC];
            decode<E>(u, x);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f(x[j]);
        });
    };
    auto clear = [&]() {
        for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[i] = 0;
        if (threadIdx.x == 0) s.lo = 0xffffffffu, s.hi = 0;
        __syncthreads();
    };
    // The histograms are whole, and the lists of the last selection have been read by all: then is s.listed cleared. Bins 2 t and
    // 2 t + 1 over the cluster.
    auto merged_bins = [&]() {
        cluster.sync();
        if (threadIdx.x == 0) s.listed = 0;  // (find_bin's barriers come before it is counted up)
        uint2 v[kMaxCluster];
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i)
            v[i] = i < ranks ? *reinterpret_cast<const uint2 *>(cluster.map_shared_rank(&s.hist[2 * threadIdx.x], i)) : make_uint2(0, 0);
        float2 n = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) n.x += (float)v[i].x, n.y += (float)v[i].y;
        return n;
    };
    // The values that the CTAs have listed, of the chosen bin, side by side in s.merged: how many, or -1 if they are too many.
    auto merge_lists = [&]() {
        cluster.sync();
        int n = 0, starts[kMaxCluster];
        bool fits = true;
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) starts[i] = i < ranks ? (int)*cluster.map_shared_rank(&s.listed, i) : 0;
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) {
            const int m = starts[i];
            fits = fits && m <= kListed;
            starts[i] = n;
            n += m;
        }
        fits = fits && n <= kMerged;
        if (fits)
            for (int j = threadIdx.x; j < n; j += kThreads) {
                int owner = 0, start = 0;
#pragma unroll
                for (int i = 1; i < kMaxCluster; ++i)
                    if (i < ranks && j >= starts[i]) owner = i, start = starts[i];
                s.merged[j] = *cluster.map_shared_rank(&s.list[j - start], owner);
            }
        return fits ? n : -1;
    };
    // The key of n at which the running sum from the largest on reaches the goal, and what lies before it. share(j): the j-th's
    // part, in units. (s.lo and s.hi are set back before.)
    auto find_key = [&](int n, float before, float goal, float unit, auto key_at, auto share, float &at) {
        unsigned lo = 0xffffffffu, hi = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < n; j += kThreads) lo = min(lo, key_at(j)), hi = max(hi, key_at(j));
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) atomicMin(&s.lo, lo), atomicMax(&s.hi, hi);
        __syncthreads();
        lo = s.lo, hi = s.hi;
        while (lo < hi) {
            const int shift = max(0, 22 - __clz(hi - lo));
            for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[i] = 0;
            __syncthreads();
            for (int j = threadIdx.x; j < n; j += kThreads) {
                const unsigned key = key_at(j);
                if (key >= lo && key <= hi) atomicAdd(&s.hist[(hi - key) >> shift], share(j));
            }
            __syncthreads();
            find_bin<kShort>(s, before, goal, unit * (float)s.hist[2 * threadIdx.x], unit * (float)s.hist[2 * threadIdx.x + 1]);
            if (s.bin == kBins) {  // (a sum of masses in another order may end below its goal)
                hi = lo;
                break;
            }
            before = s.before;
            hi -= (unsigned)s.bin << shift;
            lo = hi - lo >= (1u << shift) ? hi - (1u << shift) + 1 : lo;
            // (a bin of several keys that holds one: the next round's finer bins find it)
        }
        at = before;
        return hi;
    };
    auto merged_key = [&](int j) { return s.merged[j]; };
    // The key, lo .. hi, at which the running sum of the shares, in units, of the tokens that member() takes reaches the goal, from the largest on:
    // from a list of them if they fit (n: how many; else 0 or less), after a histogram of that range's parts as long as they do not. 0 if
    // it is not reached; and what lies before the key.
    auto find_in_row = [&](unsigned lo, unsigned hi, float &before, float goal, float unit, auto member, auto share, int &n, bool counts) {
        for (;;) {
            const float from_x = value_of<E>(lo), to_x = value_of<E>(hi);
            each_vector([&](uint4 u) {  // (nearly all tokens are outside)
                float x[VEC];
                decode<E>(u, x);
                unsigned some = 0;
#pragma unroll
                for (int j = 0; j < VEC; ++j) some |= (unsigned)(x[j] >= from_x && x[j] <= to_x) << j;
                for (; some; some &= some - 1) {
                    const int j = __ffs(some) - 1;
                    const float2 pair = pair_of<E>(u, j / 2);
                    const float mine = j % 2 ? pair.y : pair.x;
                    if (!member(mine)) continue;
                    const unsigned at = atomicAdd(&s.listed, 1u);
                    if (at < kListed) s.list[at] = key_of<E>(mine);
                }
            });
            n = merge_lists();
            if (counts && n >= 0 && before + (float)n < goal) return 0u;
            if (n > 0) return find_key(n, before, goal, unit, merged_key, [&](int j) { return share(value_of<E>(s.merged[j])); }, before);
            if (n == 0 || lo == hi) return hi;
            const int shift = max(0, 22 - __clz(hi - lo));
            clear();
            each([&](float x) {
                if (x >= from_x && x <= to_x && member(x)) atomicAdd(&s.hist[(hi - key_of<E>(x)) >> shift], share(x));
            });
            const float2 bins = merged_bins();
            find_bin<kShort>(s, before, goal, unit * bins.x, unit * bins.y);
            if (s.bin == kBins) {
                cluster.sync();  // (others may be reading the histogram)
                return 0u;
            }
            before = s.before;
            hi -= (unsigned)s.bin << shift;
            lo = hi - lo >= (1u << shift) ? hi - (1u << shift) + 1 : lo;
        }
    };
    // The mass of a lane's vectors: of the tokens that in() takes, and with BOTH of those of above() among them. Pairs of tokens of less than
    // 2^-kTail are added up in 32 bits, unless all_exact.
    const float tail_top = top - kTail / scale.ch;
    struct Mass {
        Sum exact, exact_above;
        float2 small, small_above;
        int n;
        u64 all, kept;
        long long rest, rest_kept;  // (light tokens, and what lies below the units, of all and of those above)
    };
    auto flush_mass = [&](auto both, Mass &m) {
        m.all += m.exact.fixed();
        m.rest += m.exact.fine(m.small);
        if (decltype(both)::value) {
            m.kept += m.exact_above.fixed();
            m.rest_kept += m.exact_above.fine(m.small_above);
        }
    };
    auto add_mass = [&](auto both, auto unroll, Mass &m, uint4 u, auto in, auto above, bool all_exact) {
        constexpr bool BOTH = decltype(both)::value;
        constexpr int UNROLL = decltype(unroll)::value;
#pragma unroll UNROLL
        for (int j = 0; j < VEC / 2; ++j) {
            const float2 x = pair_of<E>(u, j);
            const bool in0 = in(x.x), in1 = in(x.y);
            const bool above0 = BOTH && in0 && above(x.x), above1 = BOTH && in1 && above(x.y);
            if (all_exact || fmaxf(x.x, x.y) >= tail_top) {
                const Weights w = weights_of(x.x, x.y, scale, s.powers);
                m.exact.add(w, in0, in1);
                if (BOTH) m.exact_above.add(w, above0, above1);
            } else {
                const float2 y = __fmul2_rn(__fadd2_rn(x, two(-top)), two(scale.ch));
                const float w0 = exp2_fast(y.x), w1 = exp2_fast(y.y);
                if (in0) m.small.x += w0;
                if (in1) m.small.y += w1;
                if (above0) m.small_above.x += w0;
                if (above1) m.small_above.y += w1;
            }
        }
        if ((m.n += VEC) == 64) {
            flush_mass(both, m);
            m.exact = Sum();
            m.small = two(0.f);
            if (BOTH) m.exact_above = Sum(), m.small_above = two(0.f);
            m.n = 0;
        }
    };
    // The warp's mass of its lanes', and that of its light tokens.
    auto end_mass = [&](auto both, Mass &m, bool all_exact, u64 &tail) {
        flush_mass(both, m);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            m.all += __shfl_xor_sync(0xffffffffu, m.all, off), m.rest += __shfl_xor_sync(0xffffffffu, m.rest, off);
            if (decltype(both)::value) m.kept += __shfl_xor_sync(0xffffffffu, m.kept, off), m.rest_kept += __shfl_xor_sync(0xffffffffu, m.rest_kept, off);
        }
        const u64 rest = rest_of(m.rest);
        m.all += rest;
        if (decltype(both)::value) m.kept += rest_of(m.rest_kept);
        tail = all_exact || m.rest < 0 ? 0 : rest;
    };
    const std::true_type both{};
    const std::false_type one{};
    const std::integral_constant<int, kUnroll> pairs{};
    auto nucleus = [&](u64 all) {  // the least mass that top_p keeps
        bool part;
        const u64 m = part_of(all, p, part);
        return m + part;
    };
    auto draw = [&](u64 all) {  // the random number's place in the kept mass
        bool part;
        return !(uniform > 0.f) ? 0 : uniform < 1.f ? part_of(all, uniform, part) : all - 1;
    };
    auto log_share = [&](float x, u64 all, int bits) {  // of a token's weight in the kept mass, which is 1 or more, in units of 2^-bits
        const float over = __ull2float_rn(all - (1ull << bits)) * __int_as_float((127 - bits) << 23);
        return (x == top ? 0.f : (x - top) / temp) - log1pf(over);
    };

    // ---- near the maximum ----
    int parity = 0;          // of the exchanged sets
    // the listed tokens are those from here on
    const float bound = k == 1 ? top : seek ? fmaxf(share, alone) : floor;
    if (MODE != kHard && bound > -kInf && (by_count ? k <= ranks * kThreads / 2 : p < 1.f || floors)) {
        const bool floored = floor >= bound;       // min_p keeps nothing that is not listed
        const bool whole = !by_count && !floored;  // the mass of the others counts
        const float least = fmaxf(bound, floor);
        // this CTA's vectors with such tokens, in order: where the histogram was
        unsigned *const queue = s.hist;
        auto promising = [&](int i) { return i < mine_end && __uint_as_float((unsigned)crest[i] << 16) >= least; };
        unsigned found = 0;
        for (int i = from; i < mine_end; i += 32) found += __popc(__ballot_sync(0xffffffffu, promising(i + lane)));
        u64 all = 0, tail = 0;
        if (whole) {
            Mass m = {};
            each_vector([&](uint4 u) { add_mass(one, pairs, m, u, [&](float x) { return x >= lowest; }, [](float) { return true; }, false); });
            end_mass(one, m, false, tail);
            if (lane == 0) s.scan64[warp] = m.all, s.scan64b[warp] = tail;
        }
        __syncthreads();
        if (lane == 0) s.scan32[warp] = found;
        __syncthreads();
        unsigned queued = 0, at = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) at = queued;
            queued += s.scan32[w];
        }
        if (found && queued <= kBins)
            for (int i = from; i < mine_end; i += 32) {
                const unsigned who = __ballot_sync(0xffffffffu, promising(i + lane));
                if ((who >> lane) & 1) queue[at + __popc(who & ((1u << lane) - 1u))] = (unsigned)(i + lane);
                at += __popc(who);
            }
        __syncthreads();
        // and their tokens: two vectors a thread
        constexpr int kEach = kBins / kThreads;
        uint4 u[kEach];
        unsigned mine = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const unsigned q = threadIdx.x * kEach + j;
            u[j] = make_uint4(lowest_bits<E>(), lowest_bits<E>(), lowest_bits<E>(), lowest_bits<E>());
            if (queued <= kBins && q < queued) u[j] = fetch((int)queue[q]);
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            float x[VEC];
            decode<E>(u[j], x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) mine += x[e] >= least;
        }
        unsigned upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const unsigned o = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += o;
        }
        if (lane == 31) s.scan32[warp] = upto;
        __syncthreads();
        unsigned count = 0;
        at = upto - mine;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += s.scan32[w];
            count += s.scan32[w];
        }
        if (queued > kBins) count = kListed + 1;
        if (mine && count <= kListed) {
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const unsigned q = threadIdx.x * kEach + j;
                if (q >= queued) continue;
                const int token = (base + (int)queue[q]) * VEC - head;
                float x[VEC];
                decode<E>(u[j], x);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (x[e] >= least) s.near[at++] = make_uint2(key_of<E>(x[e]), (unsigned)(token + e));
            }
        }
        if ((int)threadIdx.x < ranks) {
            *cluster.map_shared_rank(&s.eq[0][rank], threadIdx.x) = count;
            if (whole) {
                all = tail = 0;
                for (int w = 0; w < kWarps; ++w) all += s.scan64[w], tail += s.scan64b[w];
                *cluster.map_shared_rank(&s.all[0][rank], threadIdx.x) = all;
                *cluster.map_shared_rank(&s.tail[0][rank], threadIdx.x) = tail;
            }
        }
        cluster.sync();
        parity = 1;
        int n = 0, starts[kMaxCluster];
        bool fits = true;
        all = tail = 0;
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) {
            starts[i] = n;
            if (i >= ranks) continue;
            n += (int)s.eq[0][i];
            fits = fits && s.eq[0][i] <= kListed;
            if (whole) all += s.all[0][i], tail += s.tail[0][i];
        }
        fits = fits && n <= (whole ? kFew : max(kSome, (HELD ? a.room : a.room / 8)));
        if (whole) all_exact = tail > all >> kTailShift;
        // the lists side by side in the first CTA, where its part of the row was if they are long (and are known to be enough)
        Entry *entry = n <= kSome ? s.some : reinterpret_cast<Entry *>(slice);  // (16 bytes each)
        const bool few = n <= kFew;
        u64 keep = 0;  // this thread's token's weight if it is kept (if few)
        // A few tokens are compared each with each, for a token's place in the order and the mass before it. Those that the filters keep;
        // false if the light tokens' error makes that uncertain.
        auto keep_few = [&]() {
            const int me = threadIdx.x % kFew, part = threadIdx.x / kFew;
            u64 mass = 0;
            unsigned place = 0;
            Entry e = {};
            if (me - lane < n) {
                if (me < n) e = entry[me];
                const int begin = part ? n / 2 : 0, end = part ? n : n / 2;
#pragma unroll 4
                for (int j = begin; j < end; ++j) {
                    const Entry o = entry[j];
                    if (o.key > e.key || (o.key == e.key && j < me)) mass += o.weight, ++place;
                }
            }
            __syncthreads();  // (s.near lies where s.part does)
            if (part) s.part[me] = mass, s.part_rank[me] = place;
            __syncthreads();
            const bool have = !part && me < n;
            if (have) mass += s.part[me], place += s.part_rank[me];
            keep = have && place < (unsigned)k ? e.weight : 0;
            if (!(p < 1.f)) return true;
            // the mass that top_p takes its part of: that of the tokens kept so far, and of those that are not listed
            u64 sum = keep;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) s.scan64[warp] = sum;
            __syncthreads();
            sum = 0;
            for (int w = 0; w < kFew / 32; ++w) sum += s.scan64[w];
            __syncthreads();
            if (!whole) {
                if (keep && mass >= nucleus(sum)) keep = 0;
                return true;
            }
            const u64 error = tail >> kTailError, goal = nucleus(all), most = nucleus(all + error);
            mass >>= kList - kFixed;  // (a goal of whole units is reached or not)
            const bool doubt = keep && (mass >= nucleus(all - error)) != (mass >= most);
            if (keep && mass >= goal) keep = 0;
            return !__syncthreads_or(doubt) && most <= sum >> (kList - kFixed);
        };
        if (fits) {
            if (rank == 0) {
                for (int j = threadIdx.x; j < n; j += kThreads) {
                    int owner = 0, start = 0;
#pragma unroll
                    for (int i = 1; i < kMaxCluster; ++i)
                        if (i < ranks && j >= starts[i]) owner = i, start = starts[i];
                    const uint2 e = *cluster.map_shared_rank(&s.near[j - start], owner);
                    entry[j] = Entry{e.x, (int)e.y, k == 1 ? 1ull << kList : coarser(weight_of(value_of<E>(e.x), scale, s.powers), kList)};
                }
                __syncthreads();
                if (whole) {
                    const bool sure = keep_few();
                    if ((int)threadIdx.x < ranks) *cluster.map_shared_rank(&s.done, threadIdx.x) = sure;
                }
            }
            cluster.sync();  // the others wait until they have been read
            fits = !whole || s.done;
            if (fits && rank != 0) return;
        }
        if (fits) {
            unsigned key = 0, r = 0;  // tokens above this key and the first r of it are kept (unless few)
            u64 weight = 0;           // of a token of this key
            if (few) {
                if (!whole) keep_few();
            } else {
                auto key_at = [&](int j) { return entry[j].key; };
                auto reset = [&]() {
                    __syncthreads();
                    if (threadIdx.x == 0) s.lo = 0xffffffffu, s.hi = 0;
                };
                // tokens above key1, and the first ties of key1
                unsigned key1 = 0, ties = 0;
                if (by_count && n > k) {
                    reset();
                    float before;
                    key1 = find_key(n, 0.f, (float)k, 1.f, key_at, [](int) { return 1u; }, before);
                    ties = (unsigned)(k - (int)before);
                }
                key = key1;
                r = ties;
                u64 sum;
                unsigned alike;
                auto above = [&](unsigned than) {  // the mass above a key, and the tokens at it
                    sum = 0;
                    alike = 0;
                    for (int j = threadIdx.x; j < n; j += kThreads) {
                        const Entry e = entry[j];
                        if (e.key > than) sum += e.weight;
                        if (e.key == than) ++alike, s.key_weight = e.weight;
                    }
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                    alike = __reduce_add_sync(0xffffffffu, alike);
                    __syncthreads();
                    if (lane == 0) s.scan64[warp] = sum, s.scan32[warp] = alike;
                    __syncthreads();
                    sum = 0;
                    alike = 0;
                    for (int w = 0; w < kWarps; ++w) sum += s.scan64[w], alike += s.scan32[w];
                    weight = alike ? s.key_weight : 0;
                };
                above(key);
                if (p < 1.f) {
                    all = sum + (u64)r * weight;  // (not whole: those lists are short)
                    const u64 goal = nucleus(all);
                    const int shift = max(0, 33 - (int)__clzll((long long)all));  // shares add up to less than 2^31
                    if (sum >= goal) {  // (else some of the ties complete it)
                        reset();
                        float before;
                        key = max(key1, find_key(n, 0.f, (float)(goal >> shift), 1.f, key_at,
                                                 [&](int j) { return entry[j].key > key1 ? (unsigned)(entry[j].weight >> shift) : 0u; }, before));
                    }
                    for (;;) {  // the shares are rounded: the next key, where they were wrong
                        above(key);
                        r = key > key1 ? alike : ties;
                        const bool up = sum >= goal;
                        if (!up && sum + (u64)r * weight >= goal) break;
                        unsigned next = up ? 0xffffffffu : 0u;
                        for (int j = threadIdx.x; j < n; j += kThreads) {
                            const unsigned o = entry[j].key;
                            if (up ? o > key : o < key) next = up ? min(next, o) : max(next, o);
                        }
                        next = up ? __reduce_min_sync(0xffffffffu, next) : __reduce_max_sync(0xffffffffu, next);
                        reset();
                        __syncthreads();
                        if (lane == 0) up ? atomicMin(&s.lo, next) : atomicMax(&s.hi, next);
                        __syncthreads();
                        key = up ? s.lo : s.hi;
                    }
                    r = (unsigned)((goal - sum + weight - 1) / weight);
                }
            }
            // the first token in index order at which the kept mass passes u times the total
            const int per = few ? 1 : (n + kThreads - 1) / kThreads, begin = threadIdx.x * per, end = min(n, begin + per);
            u64 part = keep;
            unsigned same = 0;
            if (!few)
                for (int j = begin; j < end; ++j) {
                    if (entry[j].key > key) part += entry[j].weight;
                    same += entry[j].key == key;
                }
            u64 part_upto = part;
            unsigned same_upto = same;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const u64 o = __shfl_up_sync(0xffffffffu, part_upto, off);
                const unsigned q = __shfl_up_sync(0xffffffffu, same_upto, off);
                if (lane >= off) part_upto += o, same_upto += q;
            }
            __syncthreads();
            if (lane == 31) s.scan64[warp] = part_upto, s.scan32[warp] = same_upto;
            __syncthreads();
            u64 total = 0, mass_at = part_upto - part;
            unsigned same_all = 0, same_at = same_upto - same;
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) mass_at += total, same_at += same_all;
                total += s.scan64[w], same_all += s.scan32[w];
            }
            total += (u64)r * weight;
            // (the range of a thread's tokens is looked at by the one whose mass holds the place)
            const u64 goal = draw(total);
            const u64 lower = mass_at + (u64)min(same_at, r) * weight, upper = mass_at + part + (u64)min(same_at + same, r) * weight;
            const unsigned here = __ballot_sync(0xffffffffu, lower <= goal && goal < upper);
            if (!here) return;
            int token = 0;
            unsigned token_key = 0;
            if (lower <= goal && goal < upper) {
                u64 m = lower;
                for (int j = begin; j < end; ++j) {
                    const Entry e = entry[j];
                    u64 w = few ? keep : e.key > key ? e.weight : 0;
                    if (!few && e.key == key && same_at++ < r) w = weight;
                    m += w;
                    if (w && m > goal) {
                        token = e.token;
                        token_key = e.key;
                        break;
                    }
                }
            }
            token = __shfl_sync(0xffffffffu, token, __ffs(here) - 1);
            token_key = __shfl_sync(0xffffffffu, token_key, __ffs(here) - 1);
            finish(token, lane == 0 ? log_share(value_of<E>(token_key), total, kList) : 0.f);
            return;
        }
    }

    auto leave = [&]() {  // to the second kernel
        if (rank != 0 || threadIdx.x != 0) return;
        const unsigned at = atomicAdd(&a.hard[0], 1u);
        if (at < (unsigned)(a.B * a.T)) a.hard[3 + at] = (unsigned)row | (all_exact ? kHeavy : 0u);  // (less, if the workspace was zeros)
    };
    if (MODE == kEasy && (by_count || p < 1.f)) {
        leave();
        return;
    }

    // ---- the whole row; top_k and min_p: the tokens x > tau1 and the first r1 with x == tau1 ----
    float tau1 = -kInf;
    unsigned r1 = 0;
    if (k == 1) {
        tau1 = top;
        r1 = 1;
    } else if (MODE != kEasy && k < a.V) {
        clear();
        each([&](float x) {
            const int bin = count_bin(x);
            if (bin < kBins) atomicAdd(&s.hist[bin], 1u);
        });
        const float2 bins = merged_bins();
        find_bin<kShort>(s, 0.f, (float)k, bins.x, bins.y);
        const int bin = s.bin;
        float before = 0.f;
        unsigned lo = key_of<E>(-kInf) + 1, hi = key_of<E>(top);
        if (bin < kBins) {  // (else they are far below the maximum)
            before = s.before;
            lo = max(lo, key_of<E>(__fsub_rd(top, (float)(bin + 1) * ((1.f + 0x1p-21f) / kCountScale))));
            hi = min(hi, key_of<E>(__fsub_ru(top, (float)bin * ((1.f - 0x1p-21f) / kCountScale))));
        }
        int n;
        const unsigned key = find_in_row(lo, hi, before, (float)k, 1.f, [&](float x) { return bin == kBins || count_bin(x) == bin; }, [](float) { return 1u; }, n, true);
        if (key) {  // (else fewer than k tokens are not masked, and all of them are kept)
            tau1 = value_of<E>(key);
            r1 = (unsigned)(k - (int)before);
        }
    }
    if (floor > tau1) {
        tau1 = floor == 0.f ? -1.4e-45f : __uint_as_float(__float_as_uint(floor) + (floor > 0.f ? -1 : 1));  // the float below
        // and the type's value there or below it: a negative float between two values has the key of the upper one, which may be kept
        const unsigned key = key_of<E>(tau1);
        tau1 = value_of<E>(value_of<E>(key) > tau1 ? key - 1 : key);
        r1 = 0;
    }

    // ---- top_p: a guess of the last value that it keeps ----
    float tau = tau1;
    int listed = 0;
    if (MODE != kEasy && p < 1.f) {
        clear();
        each([&](float x) {
            const unsigned bits = mass_bits(x);
            const int bin = mass_bin(bits);
            if (x > tau1 && bin < kBins) atomicAdd(&s.hist[bin], mass_share(bits));
        });
        const float2 bins = merged_bins();
        const int i0 = 2 * threadIdx.x;
        const float v0 = mass_unit(i0) * bins.x, v1 = mass_unit(i0 + 1) * bins.y;
        float sum = v0 + v1;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) s.scanf[warp] = sum;
        __syncthreads();
        sum = 0.f;
        for (int w = 0; w < kWarps; ++w) sum += s.scanf[w];
        if (r1) sum += (float)r1 * ((float)weight_at<kShort>(tau1, scale, s.powers) * (0x1p-56f * 32768.f));
        __syncthreads();
        const float goal = p * sum;
        find_bin<kShort>(s, 0.f, goal, v0, v1);
        const int bin = s.bin;
        float before = s.before;
        if (bin < kBins) {  // (else the tokens at tau1 are reached)
            // (the bin's range, a little wide)
            const float most = __uint_as_float((0x7f1u - (unsigned)bin) << 19), least_of = __uint_as_float((0x7f0u - (unsigned)bin) << 19);
            const float high = top + (log2f(most) * (1.f - 0x1p-20f) + 0x1p-20f) / scale.ch, low = top + (log2f(least_of) * (1.f + 0x1p-20f) - 0x1p-20f) / scale.ch;
            const float slack = 0x1p-22f * fmaxf(fabsf(top), fabsf(low));
            const unsigned key = find_in_row(key_of<E>(fmaxf(low - slack, tau1)), key_of<E>(fminf(high + slack, top)), before, goal, mass_unit(bin),
                                             [&](float x) { return x > tau1 && mass_bin(mass_bits(x)) == bin; }, [&](float x) { return mass_share(mass_bits(x)); }, listed, false);
            tau = fmaxf(key ? value_of<E>(key) : fminf(value_of<E>(key_of<E>(low)), top), tau1);
        }
    }

    // ---- the exact masses, and what top_p keeps ----
    u64 error;  // twice that of the light tokens' 32-bit sums: of a running mass and of its share of the whole
    u64 kept, kept_before, all_kept, tau_weight, tail;  // this warp's, of the warps before it, of the row; of a token at tau (2^-kFine)
    unsigned alike, alike_before, r;
    auto above_tau = [&](float x) { return x > tau; };
    unsigned lo = key_of<E>(tau1), hi = key_of<E>(top), now = key_of<E>(tau);  // tau's key is now, and in the end one of lo .. hi
    for (;;) {
        for (int tries = 0;; ++tries) {
            Mass m = {};
            alike = 0;
            u64 mine;  // of all that count, with a top_p
            if (p < 1.f) {
                each_vector([&](uint4 u) { add_mass(both, pairs, m, u, [&](float x) { alike += x == tau; return x > tau1; }, above_tau, all_exact); });
                end_mass(both, m, all_exact, tail);
                mine = m.all, kept = m.kept;
            } else {
                each_vector([&](uint4 u) { add_mass(one, pairs, m, u, [&](float x) { alike += x == tau; return x > tau; }, above_tau, all_exact); });
                end_mass(one, m, all_exact, tail);
                mine = kept = m.all;
            }
            alike = __reduce_add_sync(0xffffffffu, alike);
            __syncthreads();
            if (lane == 0) s.scan64[warp] = kept, s.scan32[warp] = alike, s.scan64b[warp] = mine, s.scan64c[warp] = tail;
            __syncthreads();
            u64 cta_kept = 0, cta_all = 0, cta_tail = 0;
            unsigned cta_alike = 0;
#pragma unroll kUnrollWarps
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) kept_before = cta_kept, alike_before = cta_alike;
                cta_kept += s.scan64[w], cta_alike += s.scan32[w], cta_all += s.scan64b[w], cta_tail += s.scan64c[w];
            }
            if (threadIdx.x == 0) s.done = 0;  // (until the CTA that has the token says otherwise, after the exchange)
            if ((int)threadIdx.x < ranks) {
                *cluster.map_shared_rank(&s.kept[parity][rank], threadIdx.x) = cta_kept;
                *cluster.map_shared_rank(&s.all[parity][rank], threadIdx.x) = cta_all;
                *cluster.map_shared_rank(&s.tail[parity][rank], threadIdx.x) = cta_tail;
                *cluster.map_shared_rank(&s.eq[parity][rank], threadIdx.x) = cta_alike;
            }
            cluster.sync();
            all_kept = 0;
            u64 all = 0;
            tail = 0;
            unsigned all_alike = 0;
            for (int i = 0; i < ranks; ++i) {
                if (i == rank) kept_before += all_kept, alike_before += all_alike;
                all_kept += s.kept[parity][i], all += s.all[parity][i], tail += s.tail[parity][i], all_alike += s.eq[parity][i];
            }
            parity ^= 1;
            error = tail >> (kTailError - 1);
            if (tail > all >> kTailShift && p < 1.f) {
                all_exact = true;
                --tries;
                continue;
            }
            tau_weight = weight_at<kShort>(tau, scale, s.powers);
            r = tau > tau1 ? all_alike : r1;  // tokens at tau that may be kept
            if (!(p < 1.f)) break;
            if (r1) all += mass_of(r1, weight_at<kShort>(tau1, scale, s.powers));
            const u64 goal = nucleus(all), with_all = all_kept + mass_of(r, tau_weight);
            const bool more = all_kept >= goal, fewer = with_all < goal;  // tau is higher, or lower
            if (error && !certain(all_kept, with_all, goal, error, tau_weight)) {
                all_exact = true;
                --tries;
                continue;
            }
            if (!more && !fewer) {
                r = fewest_of(goal - all_kept, tau_weight);
                break;
            }
            if (more) lo = now + 1;
            else hi = now - 1;
            // No value is left where the sum over a value's tokens and their number times one's weight, which differ by some units, lie on
            // either side of the goal: then all of them are kept and none below. (And 16 growing steps and 32 halvings are not passed.)
            if (lo > hi || tries > 60) {
                if (more) r = 0;
                break;
            }
            // the next value in the bin, at first; then in steps that grow, to the middle of what is left at most
            unsigned next = lo == hi ? lo : 0;
            if (!next && tries < 3 && listed > 0) {
                unsigned best = more ? 0xffffffffu : 0u;
                for (int j = lane; j < listed; j += 32) {
                    const unsigned key = s.merged[j];
                    if (more ? key > now : key < now) best = more ? min(best, key) : max(best, key);
                }
                best = more ? __reduce_min_sync(0xffffffffu, best) : __reduce_max_sync(0xffffffffu, best);
                if (best >= lo && best <= hi) next = best;
            }
            if (!next) {
                const unsigned step = min((hi - lo) / 2, tries < 16 ? (1u << 2 * tries) - 1u : 0xffffffffu);
                next = more ? lo + step : hi - step;
            }
            now = next;
            tau = fmaxf(value_of<E>(now), tau1);
        }

        // ---- the token: the first at which the kept mass passes u times the total. Light tokens' errors may move that beyond a border ----
        const u64 all = all_kept + mass_of(r, tau_weight), goal = draw(all);
        auto mass = [&](u64 m, unsigned alike_upto) { return m + mass_of(min(alike_upto, r), tau_weight); };
        // the warp that has it; then its steps, which all warps share
        if (threadIdx.x == 0) s.chosen = s.place = -1;
        __syncthreads();
        if (lane == 0 && mass(kept_before, alike_before) <= goal && goal < mass(kept_before + kept, alike_before + alike)) {
            s.chosen = warp;
            s.scan64[0] = kept_before;
            s.scan32[0] = alike_before;
        }
        __syncthreads();
        const int chosen = s.chosen;
        int token = -1;
        float token_x = top;
        bool sure = false;
        if (chosen >= 0) {
            int begin = chosen * per_warp, end = min(begin + per_warp, held);
            u64 kept_upto = s.scan64[0];
            unsigned alike_upto = s.scan32[0];
            if (!kShort) {  // the step that has it, first; the last with a kept token where the warp's sum was some units more
                const int steps = (end - begin + 31) / 32;
                for (int step = warp; step < steps; step += kWarps) {
                    const int i = begin + step * 32 + lane;
                    Mass m = {};
                    unsigned same = 0, some = 0;
                    if (i < end) add_mass(one, pairs, m, fetch(i), [&](float x) { same += x == tau; some += x > tau; return x > tau; }, above_tau, all_exact);
                    u64 light;
                    end_mass(one, m, true, light);
                    same = __reduce_add_sync(0xffffffffu, same);
                    some = __reduce_add_sync(0xffffffffu, some);
                    if (lane == 0) s.step_mass[step] = m.all, s.step_alike[step] = same, s.step_kept[step] = some;
                }
                __syncthreads();
                int step = 0;
                u64 kept_at = kept_upto;
                unsigned alike_at = alike_upto;
                for (int j = 0; j < steps; ++j) {
                    const bool any = s.step_kept[j] || (s.step_alike[j] && alike_at < r);
                    if (any) step = j, kept_upto = kept_at, alike_upto = alike_at;
                    kept_at += s.step_mass[j], alike_at += s.step_alike[j];
                    if (any && mass(kept_at, alike_at) > goal) break;
                }
                begin += step * 32;
                end = min(begin + 32, end);
            }
            // a token a thread at a time; the last kept one if none passes
            constexpr int kFound = 1 << 30;
            int mine = -1;
            float mine_x = top;
            bool clear_of = false;
            u64 listed_upto = 0;  // of the tokens so far, in units of 2^-kList
            for (int v = begin; v < end; v += kThreads / VEC) {
                const int i = v + (int)threadIdx.x / VEC;
                float x = -kInf;
                if (i < end) {
                    const float2 pair = pair_of<E>(fetch(i), (int)threadIdx.x % VEC / 2);
                    x = threadIdx.x % 2 ? pair.y : pair.x;
                }
                const u64 w = x > tau ? coarser(weight_at<kShort>(x, scale, s.powers), kList) : 0;
                const unsigned equal = __ballot_sync(0xffffffffu, x == tau);
                u64 upto = w;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const u64 o = __shfl_up_sync(0xffffffffu, upto, off);
                    if (lane >= off) upto += o;
                }
                if (lane == 31) s.scan64b[warp] = upto, s.scan32b[warp] = __popc(equal);
                __syncthreads();
                u64 listed_at = upto - w;
                unsigned alike_at = __popc(equal & ((1u << lane) - 1u));
#pragma unroll 1
                for (int o = 0; o < kWarps; ++o) {
                    if (o == warp) listed_at += listed_upto, alike_at += alike_upto;
                    listed_upto += s.scan64b[o], alike_upto += s.scan32b[o];
                }
                const u64 before = mass(kept_upto + (listed_at >> (kList - kFixed)), alike_at);
                const u64 after = mass(kept_upto + ((listed_at + w) >> (kList - kFixed)), alike_at + (x == tau));
                int at = -1;
                if (x > tau || (x == tau && alike_at < r)) {
                    at = mine = i * VEC + (int)threadIdx.x % VEC;
                    mine_x = x;
                    if (before <= goal && goal < after) {
                        at |= kFound;
                        clear_of = before + error <= goal && goal + error < after;
                    }
                }
                at = __reduce_max_sync(0xffffffffu, at);
                if (lane == 0 && at >= 0) atomicMax(&s.place, at);
                __syncthreads();
                if (s.place >= kFound) break;
            }
            const int place = s.place;
            const unsigned who = __ballot_sync(0xffffffffu, mine >= 0 && mine == (place & (kFound - 1)));
            if (who) {
                const int owner = __ffs(who) - 1;
                sure = place >= kFound && __shfl_sync(0xffffffffu, (int)clear_of, owner);
                token_x = __shfl_sync(0xffffffffu, mine_x, owner);
                token = base * VEC - head + (place & (kFound - 1));
                if (error && lane < ranks) *cluster.map_shared_rank(&s.done, lane) = sure;
            }
        }
        if (error) {  // all have to know whether the row is summed again
            auto told = cluster.barrier_arrive();
            if (token >= 0 && sure) finish(token, lane == 0 ? log_share(token_x, all, kFixed) : 0.f);
            cluster.barrier_wait(std::move(told));
            if (s.done) return;
            all_exact = true;
            if (MODE == kEasy) {
                leave();
                return;
            }
            continue;
        }
        if (token >= 0) finish(token, lane == 0 ? log_share(token_x, all, kFixed) : 0.f);
        return;
    }
}

template <typename E, bool HELD, Mode MODE>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint4 slice[];
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    const unsigned ranks = cluster.num_blocks();
    if (threadIdx.x < 16) s.powers[threadIdx.x] = kPowers[threadIdx.x];
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.hist[i] = 0;
    grid_dep_wait();
    grid_dep_trigger();
    if (MODE != kHard) {
        sample_row<E, HELD, MODE>(a, s, slice, (int)(blockIdx.x / ranks), false);
        return;
    }
    const unsigned rows = (unsigned)(a.B * a.T), n = min(__ldcg(&a.hard[0]), rows);  // (and rows below that, if the workspace was zeros)
    const unsigned clusters = gridDim.x / ranks, self = blockIdx.x / ranks;
    // A row a cluster, of the first ones, which start first. More rows than clusters are taken as they come: some clusters may start only when
    // others have ended.
    const bool dealt = n <= clusters;
    if (dealt && self >= n) return;
    const bool leader = cluster.block_rank() == 0 && threadIdx.x == 0;
    unsigned i = self;
    cluster.sync();
    do {
        if (!dealt) {
            if (leader) {
                const unsigned next = atomicAdd(&a.hard[1], 1u);
                for (unsigned o = 0; o < ranks; ++o) *cluster.map_shared_rank(&s.next, o) = next;
            }
            cluster.sync();
            i = s.next;
            if (i >= n) break;
        }
        const unsigned which = __ldcg(&a.hard[3 + i]);
        if ((which & ~kHeavy) < rows) sample_row<E, HELD, MODE>(a, s, slice, (int)(which & ~kHeavy), which & kHeavy);
        cluster.sync();
        if (leader) a.hard[3 + i] = 0;  // (a later call of other sizes may have a counter there)
    } while (!dealt);
    if (leader) {  // all clusters have read the numbers: they are set back
        __threadfence();
        if (atomicAdd(&a.hard[2], 1u) == (dealt ? n : clusters) - 1) a.hard[0] = a.hard[1] = a.hard[2] = 0;
    }
}

constexpr int kHeldBytes = 192 * 1024;  // of a CTA's part of a row, with the crests

template <typename E, bool HELD, Mode MODE> dn_status launch_sample_as(const SampleArgs &a, long long clusters, int ranks, cudaStream_t st) {
    const size_t smem = ((size_t)a.room * (HELD ? 18 : 2) + 15) / 16 * 16;
    if (cudaFuncSetAttribute(sample_kernel<E, HELD, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
        cudaGetLastError();
        return DN_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(clusters * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaLaunchKernelEx(&cfg, sample_kernel<E, HELD, MODE>, a);
    return launch_status();
}

// A row gets as many CTAs as the rows leave of one wave, each with a vector a thread at least. Rows that fill the GPU with one CTA
// each, of more than a vector a thread, leave the hard ones to a second kernel.
// Measured, us, rows of 151,936: top_k 40 with top_p 0.9 and 1, 2, 4, 8 CTAs a row: 16 rows 17.5, 15.3, 13.5, 13.2; 80 rows 17.3, 27.2, 24.0,
// 33.5; 256 rows 25.1, 56.8, 58.3, 89.3. The second kernel costs 1.8 where no row is hard; 256 rows of which one keeps thousands of tokens take
// 165 without it and 88 with it. Clusters of 16 in it: 83, but those need not fit every GPU.
template <typename E> dn_status launch_sample(SampleArgs a, cudaStream_t st) {
    const int vecs = (a.V + 2 * kVecOf<E> - 2) / kVecOf<E>;  // wherever a row begins
    const long long rows = (long long)a.B * a.T;
    const int sms = device_sm_count();
    int ranks = 1;
    while (ranks < kMaxCluster && vecs > ranks * kThreads && 2 * ranks * rows <= sms) ranks *= 2;
    a.room = (vecs + ranks - 1) / ranks;
    bool held = (size_t)a.room * 18 <= kHeldBytes;
    if (ranks > 1 || vecs <= kThreads)
        return held ? launch_sample_as<E, true, kAll>(a, rows, ranks, st) : launch_sample_as<E, false, kAll>(a, rows, ranks, st);
    const dn_status easy = held ? launch_sample_as<E, true, kEasy>(a, rows, 1, st) : launch_sample_as<E, false, kEasy>(a, rows, 1, st);
    if (easy != DN_OK) return easy;
    a.room = (vecs + kMaxCluster - 1) / kMaxCluster;
    held = (size_t)a.room * 18 <= kHeldBytes;
    const long long clusters = std::min<long long>(rows, std::max(1, 2 * sms / kMaxCluster));
    return held ? launch_sample_as<E, true, kHard>(a, clusters, kMaxCluster, st) : launch_sample_as<E, false, kHard>(a, clusters, kMaxCluster, st);
}

}  // namespace sample
}  // namespace dn
