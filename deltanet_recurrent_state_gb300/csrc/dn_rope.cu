// dn_rope_append: new tokens' queries and keys turned by their positions, keys and values to the paged cache.
//
// One pass over the packed rows. A lane holds two groups of 8 elements of a head's row, D / 16 lanes a row; in the half layout
// the two are partners (element j and the one rot / 2 on; rot is a multiple of 16), so pairs meet in a lane in both layouts and one
// sine and cosine serves two elements. A row is normed (a shuffle sums the squares), turned, rounded once and stored in one
// go, a query to q_out and a key or value to its place in the pool.
//
// Angles. A frequency is given as turns a token in 64-bit fractions of a turn, so position * frequency in 64-bit integers drops
// the whole turns exactly, however far the position; the upper 32 bits, as a signed fraction of a turn, are the angle
// to 2^-32 of a turn. Its sine and cosine come from the special function unit: in -pi .. pi its absolute error is
// below 2^-21. With the products a turned element is off by less than 2^-19.5 of its pair's size, 1/360 of the unit in the last place
// that fp16 has for the larger of the two. (One 8-bit element in 10^5 is rounded to another value than from an angle of 64 bits.)
// A lane holds the same columns of every head of its token, so a warp computes them once for all its passes.
//
// What bounds it: memory at a prompt (every element read once and written once), latency at a verify block, where a
// token's heads are spread over more warps. Measured on a GB300: 25,000 tokens of 32 + 8 + 8 heads of 128 from bf16 into 8 bits 91 us,
// 6.2 TB/s, 91 % of the copy rate; of 24 + 4 + 4 heads of 256 in fp16, 64 elements turned, 120 us, the copy rate; a verify
// block 2.8 us.
#include <type_traits>

#include <cuda_runtime.h>

#include "dn.h"
#include "dn_device.cuh"
#include "dn_internal.h"
#include "dn_kv.cuh"
#include "dn_kv_host.h"

namespace dn {
namespace {

constexpr int kWarps = 4;
constexpr int kPasses = 4;  // passes of 512 elements whose loads are in flight together

struct RopeArgs {
    KvPool pool;
    int heads_q, rot, pieces;  // warps of a token
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;  // in 8-element groups
    const int *positions;
    const unsigned long long *freqs;
    float amplitude, eps;
    const void *q_weight, *k_weight;
    void *kc, *vc;
    uint8_t *ke, *ve;
    void *q_out;
};

template <bool BF> __device__ __forceinline__ void unpack8(uint4 r, float (&x)[8]) {
    const unsigned u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = unpack2<BF>(u[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
    }
}

template <int D, bool BF, bool KV8, bool PAIRS, int PASSES>
__global__ void __launch_bounds__(32 * kWarps)
rope_append_kernel(const RopeArgs a) {
    constexpr int LPR = D / 8, LANES = LPR / 2;  // groups of 8 elements, and lanes, of a row
    const KvPool &p = a.pool;
    const int lane = threadIdx.x % 32, u = lane % LANES;
    const unsigned unit = blockIdx.x * kWarps + threadIdx.x / 32;
    const int t = (int)(unit / (unsigned)a.pieces);
    const int piece = (int)(unit - (unsigned)t * (unsigned)a.pieces);
    // this lane's two groups of every row: partners among the turned ones, and the halves of the others
    const int half = a.rot / 16;
    const bool turned = u < half;
    const int g0 = turned ? u : half + u, g1 = turned ? u + half : g0 + LANES - half;
    grid_dep_wait();
    grid_dep_trigger();
    if (t >= p.total) return;
    const int rows = a.heads_q + 2 * p.heads, first = piece * PASSES * (32 / LANES) + lane / LANES;
    uint4 raw[PASSES][2];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        int row = first + i * (32 / LANES);
        const uint4 *from = static_cast<const uint4 *>(a.q) + t * a.q_stride;
        bool any = row < a.heads_q;
        if (!any) {
            row -= a.heads_q;
            any = row < 2 * p.heads;
            from = row < p.heads ? static_cast<const uint4 *>(a.k) + t * a.k_stride : static_cast<const uint4 *>(a.v) + t * a.v_stride;
            if (row >= p.heads) row -= p.heads;
        }
        raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
        if (any) {
            raw[i][0] = __ldcs(from + row * LPR + g0);
            raw[i][1] = __ldcs(from + row * LPR + g1);
        }
    }
    // the rest of the set-up is in the shadow of these loads
    const int b = request_of(p, t, lane);
    if (b < 0) return;  // rows of no request are left as they are
    int s, n;
    packed_rows(p, b, s, n);
    if (t < s || t >= s + n) return;
    const int place = held_tokens(p, b) - n + (t - s);
    const int g = pool_page(p, b, place);
    const long long at = (((long long)g * p.heads) << p.page_shift) + (place & ((1 << p.page_shift) - 1));

    // sine and cosine of this lane's pairs: (group 0, group 1) of 8, or neighbours, 4 of each group
    float cs[8], sn[8];
    if (turned) {
        const unsigned long long pos = (unsigned long long)(long long)(a.positions ? __ldg(&a.positions[t]) : place);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const unsigned long long f = __ldg(&a.freqs[PAIRS ? (e < 4 ? g0 * 4 + e : g1 * 4 + e - 4) : u * 8 + e]);
            const float angle = (float)(int)((pos * f) >> 32) * 1.46291807926715968e-9f;  // 2 pi 2^-32
            cs[e] = __cosf(angle) * a.amplitude;
            sn[e] = __sinf(angle) * a.amplitude;
        }
    }

#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int row = first + i * (32 / LANES);
        if (row - lane / LANES >= rows) break;  // the whole warp
        const bool is_q = row < a.heads_q, is_v = row >= a.heads_q + p.heads;
        float x[2][8];
        unpack8<BF>(raw[i][0], x[0]);
        unpack8<BF>(raw[i][1], x[1]);
        const void *w = is_v ? nullptr : is_q ? a.q_weight : a.k_weight;
        if (a.q_weight) {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) sum = fmaf(x[e / 8][e % 8], x[e / 8][e % 8], sum);
#pragma unroll
            for (int off = LANES / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            const float f = rsqrtf(fmaf(sum, 1.f / D, a.eps));
            if (w) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float m[8];
                    unpack8<BF>(__ldg(static_cast<const uint4 *>(w) + (h ? g1 : g0)), m);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[h][e] *= f * m[e];
                }
            }
        }
        const bool turn = turned && !is_v;
        if (turn) {
            if (PAIRS) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float &lo = x[e / 4][2 * (e % 4)], &hi = x[e / 4][2 * (e % 4) + 1];
                    const float y = lo * cs[e] - hi * sn[e];
                    hi = hi * cs[e] + lo * sn[e];
                    lo = y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 lo = make_float2(x[0][e], x[0][e + 1]), hi = make_float2(x[1][e], x[1][e + 1]);
                    const float2 c = make_float2(cs[e], cs[e + 1]), sp = make_float2(sn[e], sn[e + 1]);
                    const float2 y0 = __ffma2_rn(hi, make_float2(-sp.x, -sp.y), __fmul2_rn(lo, c));
                    const float2 y1 = __ffma2_rn(lo, sp, __fmul2_rn(hi, c));
                    x[0][e] = y0.x, x[0][e + 1] = y0.y;
                    x[1][e] = y1.x, x[1][e + 1] = y1.y;
                }
            }
        }
        uint4 r[2] = {raw[i][0], raw[i][1]};
        if (turn || w) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                r[h] = make_uint4(pack2<BF>(x[h][0], x[h][1]), pack2<BF>(x[h][2], x[h][3]), pack2<BF>(x[h][4], x[h][5]), pack2<BF>(x[h][6], x[h][7]));
        }
        int E = 0;
        if (KV8 && row - lane / LANES + 32 / LANES > a.heads_q) {  // (not for a pass of queries alone)
            float big = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) big = fmaxf(big, fabsf(x[e / 8][e % 8]));  // a NaN does not count
#pragma unroll
            for (int off = LANES / 2; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
            E = exponent_of(big);
        }
        if (row >= rows) continue;
        if (is_q) {
            uint4 *to = static_cast<uint4 *>(a.q_out) + ((long long)t * a.heads_q + row) * LPR;
            to[g0] = r[0];
            to[g1] = r[1];
            continue;
        }
        if (g < 0) continue;
        const int head = row - a.heads_q - (is_v ? p.heads : 0);
        const long long place_row = at + ((long long)head << p.page_shift);
        void *dst = is_v ? a.vc : a.kc;
        if (!KV8) {
            uint4 *to = static_cast<uint4 *>(dst) + place_row * LPR;
            to[g0] = r[0];
            to[g1] = r[1];
        } else {
            const float sc = exp_byte(254 - E);
            uint2 *to = static_cast<uint2 *>(dst) + place_row * LPR;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint2 c;
                c.x = pack_e4m3(x[h][0] * sc, x[h][1] * sc) | ((unsigned)pack_e4m3(x[h][2] * sc, x[h][3] * sc) << 16);
                c.y = pack_e4m3(x[h][4] * sc, x[h][5] * sc) | ((unsigned)pack_e4m3(x[h][6] * sc, x[h][7] * sc) << 16);
                to[h ? g1 : g0] = c;
            }
            if (u == 0) (is_v ? a.ve : a.ke)[place_row] = (uint8_t)E;
        }
    }
}

template <int D, bool BF, bool KV8, bool PAIRS> void launch_rope(RopeArgs a, cudaStream_t st) {
    const int passes = (a.heads_q + 2 * a.pool.heads + 512 / D - 1) / (512 / D);  // of one token
    auto go = [&](auto per) {
        constexpr int P = decltype(per)::value;
        a.pieces = (passes + P - 1) / P;
        const unsigned blocks = (unsigned)(((long long)a.pool.total * a.pieces + kWarps - 1) / kWarps);
        launch_pdl(rope_append_kernel<D, BF, KV8, PAIRS, P>, dim3(blocks), dim3(32 * kWarps), 0, st, a);
    };
    // few rows: one pass a warp, so that they run at once (16 tokens 2.8 us); many: four (three 95, two 101, six 91 us for 25,000 tokens).
    // One against four at 1,200, 2,400, 4,900 and 9,700 warps of one pass: 48 heads of 128 into 8 bits 2.9, 3.2, 3.9, 6.5 against 3.5, 3.6, 4.1, 5.4 us;
    // into 16 bits 2.6, 3.1, 3.7, 6.2 against 3.0, 3.1, 3.5, 4.8; 24 heads of 64 2.6, 2.9, 3.5, 5.9 against 2.8, 3.0, 3.9, 5.5;
    // 32 heads of 256 3.0, 3.4, 4.8, 7.9 against 3.2, 3.2, 3.7, 4.9
    if ((long long)a.pool.total * passes <= 32ll * device_sm_count()) {
        go(std::integral_constant<int, 1>{});
    } else {
        go(std::integral_constant<int, kPasses>{});
    }
}

}  // namespace
}  // namespace dn

extern "C" dn_status dn_rope_append(int B, int total, int heads, int group, int D, int rot, int page, int max_pages, int pages,
                                    dn_dtype io_dt, dn_dtype cache_dt, int interleaved, const void *q, int64_t q_stride,
                                    const void *k, int64_t k_stride, const void *v, int64_t v_stride, const int32_t *positions,
                                    const int64_t *freqs, float amplitude, const void *q_weight, const void *k_weight, float eps,
                                    const int32_t *start, const int32_t *kv_len, const int32_t *page_table, void *k_cache,
                                    void *v_cache, uint8_t *k_exp, uint8_t *v_exp, void *q_out, dn_stream_t stream) {
    using namespace dn;
    if (B < 0 || total < 0 || total > DN_KV_MAX_ROWS || heads < 1 || group < 1) return DN_ERR_INVALID_ARG;
    if (!kv_dtypes_known(io_dt, cache_dt)) return DN_ERR_INVALID_ARG;
    if (!kv_shape_ok(D, page) || !kv_dtypes_ok(io_dt, cache_dt)) return DN_ERR_UNSUPPORTED;
    if (rot < 16 || rot > D || rot % 16) return DN_ERR_UNSUPPORTED;
    const int64_t wide_k = (int64_t)heads * D;
    // (the product of all three is taken only where it is known to fit)
    if (wide_k > (1 << 24) || group > (1 << 24) / wide_k || !kv_pages_ok(max_pages, pages, page)) return DN_ERR_INVALID_ARG;
    const int64_t wide_q = wide_k * group;
    if (q_stride < wide_q || k_stride < wide_k || v_stride < wide_k || (q_stride | k_stride | v_stride) % 8) return DN_ERR_INVALID_ARG;
    if (!(amplitude > 0.f) || !(amplitude < 3e38f) || !q_weight != !k_weight || (q_weight && (!(eps > 0.f) || !(eps < 3e38f)))) return DN_ERR_INVALID_ARG;
    // a warp's number fits 32 bits even where each has one pass
    if ((int64_t)total * ((wide_q + 2 * wide_k) / 256 + 1) > 0x7fffffffLL) return DN_ERR_INVALID_ARG;
    if (B == 0 || total == 0) return DN_OK;
    if (!kv_pointers_ok(B, start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp, cache_dt, pages, max_pages)) return DN_ERR_INVALID_ARG;
    if (!q || !k || !v || !q_out || !freqs || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
        !aligned(freqs, 8) || !aligned(positions, 4) || !aligned(q_weight, 16) || !aligned(k_weight, 16))
        return DN_ERR_INVALID_ARG;
    RopeArgs a = {};
    a.pool = {start, kv_len, page_table, B, total, max_pages, pages, page_log2(page), heads};
    a.heads_q = heads * group;
    a.rot = rot;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride / 8;
    a.k_stride = k_stride / 8;
    a.v_stride = v_stride / 8;
    a.positions = positions;
    a.freqs = reinterpret_cast<const unsigned long long *>(freqs);
    a.amplitude = amplitude;
    a.eps = eps;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.kc = k_cache;
    a.vc = v_cache;
    a.ke = k_exp;
    a.ve = v_exp;
    a.q_out = q_out;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool bf = io_dt == DN_BF16, kv8 = cache_dt == DN_E4M3, pairs = interleaved != 0;
    auto pick = [&](auto d, auto b16, auto k8) {
        constexpr int DD = decltype(d)::value;
        constexpr bool BF = decltype(b16)::value, KV8 = decltype(k8)::value;
        if (pairs) launch_rope<DD, BF, KV8, true>(a, st);
        else launch_rope<DD, BF, KV8, false>(a, st);
    };
    auto types = [&](auto d) {
        if (bf && kv8) pick(d, std::true_type{}, std::true_type{});
        else if (bf) pick(d, std::true_type{}, std::false_type{});
        else if (kv8) pick(d, std::false_type{}, std::true_type{});
        else pick(d, std::false_type{}, std::false_type{});
    };
    if (D == 64) types(std::integral_constant<int, 64>{});
    else if (D == 128) types(std::integral_constant<int, 128>{});
    else types(std::integral_constant<int, 256>{});
    return launch_status();
}
