// dn_kv_append, dn_kv_gather: the keys and values of packed tokens to and from a paged cache.
//
// The pool is [pages][heads][page][D]: one head's page is contiguous, so an attention tile of one
// head reads whole pages and a token's row of one head is one aligned segment of D elements.
//
// Both are copies (append rounds to 8 bits on the way if the cache holds e4m3), bound by memory: one
// warp moves one token's keys and values of up to 1,024 elements, 8 elements a lane and pass, with
// the loads of all its passes issued before the first store. The row maximum that the 8-bit form
// needs is a shuffle over the D / 8 lanes that hold the row. The request of a packed row is found by the
// whole warp at once (32 entries of start a step), in the shadow of the data loads.
// Measured on a GB300: 25,000 tokens of 8 x 128-wide heads from bf16 to 8 bits 27.6 us, 5.6 TB/s, 82 % of the copy rate;
// 25,000 of 4 x 256 read back from 8 bits 26.4 us, 5.8 TB/s, 86 %. Small calls are latency.
#include <type_traits>

#include <cuda_runtime.h>

#include "dn.h"
#include "dn_device.cuh"
#include "dn_internal.h"
#include "dn_kv.cuh"
#include "dn_kv_host.h"

namespace dn {
namespace {

constexpr int kWarps = 4;   // tokens (or 1,024-element pieces of tokens) per CTA
constexpr int kPasses = 4;  // 256-element passes of a warp

// The request that packed row t belongs to, by the whole warp; -1 if none.
__device__ __forceinline__ int request_of(const KvPool &p, int t, int lane) {
    int b = 0;
    for (int i = 0; i < p.B; i += 32) {
        const int e = i + lane < p.B ? __ldg(&p.start[i + lane + 1]) : 0x7fffffff;
        b += __popc(__ballot_sync(0xffffffffu, e <= t));
    }
    return b < p.B && __ldg(&p.start[b]) <= t ? b : -1;
}

// Offset in rows of D elements of packed row t's place in the pool (head 0), or -1.
__device__ __forceinline__ long long place_of(const KvPool &p, int t, int lane) {
    const int b = request_of(p, t, lane);
    if (b < 0) return -1;
    int s, n;
    packed_rows(p, b, s, n);
    if (t < s || t >= s + n) return -1;
    const int pos = held_tokens(p, b) - n + (t - s);
    const int g = pool_page(p, b, pos);
    if (g < 0) return -1;
    return (((long long)g * p.heads) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

template <int D, bool BF, bool KV8>
__global__ void __launch_bounds__(32 * kWarps)
kv_append_kernel(KvPool p, const uint4 *__restrict__ k, const uint4 *__restrict__ v, long long k_stride8,
                 long long v_stride8, int pieces, void *__restrict__ kc, void *__restrict__ vc,
                 uint8_t *__restrict__ ke, uint8_t *__restrict__ ve) {
    constexpr int LPR = D / 8;  // lanes (of 8 elements) per row
    const int lane = threadIdx.x % 32;
    const long long unit = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
    const long long t = unit / pieces;
    const int first = (int)(unit % pieces) * kPasses * 32;  // this warp's first 8-element group of the token
    grid_dep_wait();
    grid_dep_trigger();
    if (t >= p.total) return;
    const int groups = p.heads * LPR;
    uint4 rk[kPasses], rv[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int j = first + i * 32 + lane;
        rk[i] = rv[i] = make_uint4(0, 0, 0, 0);
        if (j < groups) {
            rk[i] = __ldcs(k + t * k_stride8 + j);
            rv[i] = __ldcs(v + t * v_stride8 + j);
        }
    }
    const long long at = place_of(p, (int)t, lane);
    if (at < 0) return;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int j = first + i * 32 + lane;
        const int h = j / LPR;
        const long long row = at + ((long long)h << p.page_shift);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint4 r = kv ? rv[i] : rk[i];
            void *dst = kv ? vc : kc;
            if (!KV8) {
                if (j < groups) reinterpret_cast<uint4 *>(dst)[row * LPR + j % LPR] = r;
                continue;
            }
            const unsigned u[4] = {r.x, r.y, r.z, r.w};
            float x[8], big = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2<BF>(u[e]);
                x[2 * e] = f.x;
                x[2 * e + 1] = f.y;
                big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));  // a NaN does not count
            }
#pragma unroll
            for (int off = LPR / 2; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
            const int E = exponent_of(big);
            const float s = exp_byte(254 - E);  // 2^-(E - 127), exact
            uint2 w;
            w.x = pack_e4m3(x[0] * s, x[1] * s) | ((unsigned)pack_e4m3(x[2] * s, x[3] * s) << 16);
            w.y = pack_e4m3(x[4] * s, x[5] * s) | ((unsigned)pack_e4m3(x[6] * s, x[7] * s) << 16);
            if (j < groups) {
                reinterpret_cast<uint2 *>(dst)[row * LPR + j % LPR] = w;
                if (j % LPR == 0) (kv ? ve : ke)[row] = (uint8_t)E;
            }
        }
    }
}

// 8 bits hold no infinity, and none comes back: a row whose largest value is near the type's largest may
// have been rounded up beyond it.
template <bool BF> __device__ __forceinline__ float in_range(float x) {
    const float most = BF ? 3.38953139e38f : 65504.f;
    return x > most ? most : x < -most ? -most : x;  // NaN stays
}

template <int D, bool BF, bool KV8>
__global__ void __launch_bounds__(32 * kWarps)
kv_gather_kernel(KvPool p, const void *__restrict__ kc, const void *__restrict__ vc, const uint8_t *__restrict__ ke,
                 const uint8_t *__restrict__ ve, int pieces, uint4 *__restrict__ k, uint4 *__restrict__ v) {
    constexpr int LPR = D / 8;
    const int lane = threadIdx.x % 32;
    const long long unit = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
    const long long t = unit / pieces;
    const int first = (int)(unit % pieces) * kPasses * 32;
    grid_dep_wait();
    grid_dep_trigger();
    if (t >= p.total) return;
    const int groups = p.heads * LPR;
    const long long at = place_of(p, (int)t, lane);
    uint4 r[2][kPasses];
    int E[2][kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int j = first + i * 32 + lane;
        const long long row = at + ((long long)(j / LPR) << p.page_shift);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            r[kv][i] = make_uint4(0, 0, 0, 0);
            E[kv][i] = 127;
            if (j >= groups || at < 0) continue;
            const void *src = kv ? vc : kc;
            if (KV8) {
                const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(src) + row * LPR + j % LPR);
                r[kv][i].x = w.x;
                r[kv][i].y = w.y;
                E[kv][i] = __ldg((kv ? ve : ke) + row);
            } else {
                r[kv][i] = __ldcs(reinterpret_cast<const uint4 *>(src) + row * LPR + j % LPR);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int j = first + i * 32 + lane;
        if (j >= groups) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            uint4 o = r[kv][i];
            if (KV8) {
                const float s = exp_byte(E[kv][i]);
                unsigned u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack2<false>(unpack_e4m3((unsigned short)((e < 2 ? o.x : o.y) >> (16 * (e & 1)))));
                    u[e] = pack2<BF>(in_range<BF>(f.x * s), in_range<BF>(f.y * s));
                }
                o = make_uint4(u[0], u[1], u[2], u[3]);
            }
            __stcs((kv ? v : k) + t * groups + j, o);
        }
    }
}

// What append and gather check alike. DN_OK: go on.
dn_status check_pool(int B, int total, int heads, int D, int page, dn_dtype io_dt, dn_dtype cache_dt) {
    if (B < 0 || total < 0 || total > DN_KV_MAX_ROWS || heads < 1) return DN_ERR_INVALID_ARG;
    if (!kv_dtypes_known(io_dt, cache_dt)) return DN_ERR_INVALID_ARG;
    if (!kv_shape_ok(D, page) || !kv_dtypes_ok(io_dt, cache_dt)) return DN_ERR_UNSUPPORTED;
    if ((long long)heads * D > (1 << 24)) return DN_ERR_INVALID_ARG;
    return DN_OK;
}

}  // namespace
}  // namespace dn

#define DN_KV_LAUNCH(kernel, ...)                                                                                \
    do {                                                                                                         \
        const bool bf = io_dt == DN_BF16, kv8 = cache_dt == DN_E4M3;                                             \
        auto go = [&](auto d) {                                                                                  \
            constexpr int DD = decltype(d)::value;                                                               \
            if (bf && kv8) launch_pdl(kernel<DD, true, true>, dim3((unsigned)blocks), dim3(32 * kWarps), 0, st, __VA_ARGS__);        \
            else if (bf) launch_pdl(kernel<DD, true, false>, dim3((unsigned)blocks), dim3(32 * kWarps), 0, st, __VA_ARGS__);         \
            else if (kv8) launch_pdl(kernel<DD, false, true>, dim3((unsigned)blocks), dim3(32 * kWarps), 0, st, __VA_ARGS__);        \
            else launch_pdl(kernel<DD, false, false>, dim3((unsigned)blocks), dim3(32 * kWarps), 0, st, __VA_ARGS__);                \
        };                                                                                                       \
        if (D == 64) go(std::integral_constant<int, 64>{});                                                      \
        else if (D == 128) go(std::integral_constant<int, 128>{});                                               \
        else go(std::integral_constant<int, 256>{});                                                             \
    } while (0)

extern "C" dn_status dn_kv_append(int B, int total, int heads, int D, int page, int max_pages, int pages,
                                  dn_dtype io_dt, dn_dtype cache_dt, const void *k, const void *v, int64_t k_stride,
                                  int64_t v_stride, const int32_t *start, const int32_t *kv_len,
                                  const int32_t *page_table, void *k_cache, void *v_cache, uint8_t *k_exp,
                                  uint8_t *v_exp, dn_stream_t stream) {
    using namespace dn;
    const dn_status ok = check_pool(B, total, heads, D, page, io_dt, cache_dt);
    if (ok != DN_OK) return ok;
    if (!kv_pages_ok(max_pages, pages, page) || k_stride < (int64_t)heads * D || v_stride < (int64_t)heads * D ||
        k_stride % 8 || v_stride % 8)
        return DN_ERR_INVALID_ARG;
    if (B == 0 || total == 0) return DN_OK;
    if (!kv_pointers_ok(B, start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp, cache_dt, pages, max_pages) ||
        !k || !v || !aligned(k, 16) || !aligned(v, 16))
        return DN_ERR_INVALID_ARG;
    if (pages == 0 || max_pages == 0) return DN_OK;  // no place for any token
    KvPool p = {start, kv_len, page_table, B, total, max_pages, pages, page_log2(page), heads};
    const int pieces = (heads * (D / 8) + 32 * kPasses - 1) / (32 * kPasses);
    const long long blocks = ((long long)total * pieces + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return DN_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    DN_KV_LAUNCH(kv_append_kernel, p, static_cast<const uint4 *>(k), static_cast<const uint4 *>(v),
                 (long long)(k_stride / 8), (long long)(v_stride / 8), pieces, k_cache, v_cache, k_exp, v_exp);
    return launch_status();
}

extern "C" dn_status dn_kv_gather(int B, int total, int heads, int D, int page, int max_pages, int pages,
                                  dn_dtype io_dt, dn_dtype cache_dt, const int32_t *start, const int32_t *kv_len,
                                  const int32_t *page_table, const void *k_cache, const void *v_cache,
                                  const uint8_t *k_exp, const uint8_t *v_exp, void *k, void *v, dn_stream_t stream) {
    using namespace dn;
    const dn_status ok = check_pool(B, total, heads, D, page, io_dt, cache_dt);
    if (ok != DN_OK) return ok;
    if (!kv_pages_ok(max_pages, pages, page)) return DN_ERR_INVALID_ARG;
    if (total == 0) return DN_OK;
    if (!kv_pointers_ok(B, start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp, cache_dt, pages, max_pages) || !k || !v || !aligned(k, 16) || !aligned(v, 16))
        return DN_ERR_INVALID_ARG;
    KvPool p = {start, kv_len, page_table, B, total, max_pages, pages, page_log2(page), heads};
    const int pieces = (heads * (D / 8) + 32 * kPasses - 1) / (32 * kPasses);
    const long long blocks = ((long long)total * pieces + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return DN_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    DN_KV_LAUNCH(kv_gather_kernel, p, k_cache, v_cache, k_exp, v_exp, pieces, static_cast<uint4 *>(k),
                 static_cast<uint4 *>(v));
    return launch_status();
}
