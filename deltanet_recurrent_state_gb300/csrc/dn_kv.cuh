// Shared by the paged-cache kernels: addresses in the pool, the packed rows of the requests,
// and the 8-bit form of a key or value row.
//
// 8-bit rows. A row x (one token's keys or values of one head, D elements) is stored as e4m3
// values y and one byte E: x ~ y * 2^(E - 127), with E - 127 the smallest exponent e for which
// max |x| <= 448 * 2^e (448 is the largest e4m3 value). A power of two costs nothing against an
// arbitrary scale, because e4m3 has the same relative step in every binade; it makes y * 2^e exact
// in 32 bits, lets the attention kernels apply it to a score or a probability by an exponent, and
// takes one byte a row instead of four.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dn.h"

namespace dn {

// Where a request's cached tokens are.
struct KvPool {
    const int *start;   // [B + 1] packed rows of each request's newest tokens
    const int *kv_len;  // [B] cached tokens, the newest included
    const int *table;   // [B][max_pages] pool pages
    int B, total, max_pages, pages, page_shift, heads;
};

// The pool page of position pos of request b; -1 where there is none (never followed).
__device__ __forceinline__ int pool_page(const KvPool &p, int b, int pos) {
    const int i = pos >> p.page_shift;
    if (pos < 0 || i >= p.max_pages) return -1;
    const int g = __ldg(&p.table[(long long)b * p.max_pages + i]);
    return (unsigned)g < (unsigned)p.pages ? g : -1;
}

// Cached tokens of request b, 0 .. DN_KV_MAX_TOKENS whatever the value of kv_len.
__device__ __forceinline__ int held_tokens(const KvPool &p, int b) { return min(max(__ldg(&p.kv_len[b]), 0), DN_KV_MAX_TOKENS); }

// The packed rows [s, s + n) of request b, inside 0 .. total whatever the values of start.
__device__ __forceinline__ void packed_rows(const KvPool &p, int b, int &s, int &n) {
    s = min(max(__ldg(&p.start[b]), 0), p.total);
    n = max(min(__ldg(&p.start[b + 1]), p.total) - s, 0);
}

// 2^(E - 127) for a stored exponent byte (E = 0 is the subnormal 2^-127).
__device__ __forceinline__ float exp_byte(int E) { return __int_as_float(E ? E << 23 : 0x00400000); }

// scale * 2^e, the factor of a row's scores, kept away from 0 and infinity: masked scores are -inf before they are
// multiplied, and -inf * 0 is NaN, as is the product of infinity and a score of 0.
__device__ __forceinline__ float score_factor(float scale, int e) {
    e = min(max(e, -252), 252);
    const int h = e >> 1;  // in two steps, each a normal power
    return fminf(fmaxf(scale * __int_as_float((127 + h) << 23) * __int_as_float((127 + e - h) << 23), 0x1p-149f), 3e38f);
}

// The exponent byte of a row whose largest magnitude is `big`: the fraction bits of 448 are 1.75,
// so a larger fraction carries into the exponent. Zero, subnormal and tiny rows give 0.
__device__ __forceinline__ int exponent_of(float big) {
    const int e = (int)((__float_as_uint(big) + 0x1fffffu) >> 23) - 127 - 8;
    return min(max(e, -127), 127) + 127;
}

// Two floats to two e4m3 (the first in the low byte): to nearest, ties to even, beyond 448 to 448.
__device__ __forceinline__ unsigned short pack_e4m3(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 to two fp16, exactly.
__device__ __forceinline__ unsigned unpack_e4m3(unsigned short v) {
    unsigned r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

template <bool BF> __device__ __forceinline__ float2 unpack2(unsigned u) {
    if (BF) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
template <bool BF> __device__ __forceinline__ unsigned pack2(float lo, float hi) {
    if (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const unsigned *>(&h);
    }
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&h);
}

}  // namespace dn
