// dn_attn_paged: attention of each request's newest tokens over its paged cache.
//
//   x_j = scale q . k_j over the cached positions j that the row sees,
//   out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),   lse = m + log sum_j e^(x_j - m),  m = max_j x_j
//
// in one pass over the cache: m, the sum and the output are running values, rescaled when m grows.
// Powers of two are used throughout (x log2(e), exp2). How the work is cut is in dn_attn.cuh.
//
// attn_rows_kernel, here, is for few rows: tiles of 16 or 32 rows with warp MMAs. With so few rows the
// cache is read once and used little, so the kernel is bound by those reads: each warp streams its own
// 16- or 32-token pieces of the range through a private ring in shared memory (cp.async, XOR-swizzled
// chunks) and never waits for another warp until the end, where the warps' m, sums and outputs are
// merged. Pages are multiples of 16 tokens, so 16 tokens are one contiguous segment of the pool.
// Measured on a GB300: 64 single tokens over ragged caches of up to 8,000 bf16 tokens (8 x 4 heads of 128) 178 us,
// 6.1 TB/s, 90 % of the copy rate; 64 blocks of 1 to 4 tokens over up to 25,000 in 8 bits 379 us, 5.1 TB/s (counters of
// 24 such requests: ALU pipe 53 %, issue slots 39 %, 2.6 warps a scheduler). One token over 1,000 (24 x 256 heads) takes
// about 9.8 us on the device for 0.6 us of bytes: latency.
//
// fp16 probabilities are held as 2^15 p, which fp16 has room for (p <= 1): those below 2^-39 are lost to the product with the
// values, not those below 2^-24, which many tokens of a long cache may have while the sum counts them.
//
// 8-bit caches. The e4m3 values go to fp16 in registers, exactly; the rows' powers of two never
// touch them. A key's exponent multiplies its score in 32 bits. A value's exponent multiplies its
// probability: p 2^(E - R + 15) <= 2^15 with R the largest exponent so far, rounded to fp16 for the
// MMA. Those 15 binades keep a probability's full 11 bits until the product is 2^-29 of the largest.
// q is brought to fp16 by a power of two for each row (exact for all but elements 2^-14 of the row's
// largest), so bf16 inputs take the same path. An 8x8 ldmatrix tile of bytes gives a thread four
// neighbouring bytes of one row: for the keys the four are two k-pairs of the MMA (the same order is
// used for q, and a dot product has no order), for the values they are two tokens' pairs of columns.
#include <algorithm>
#include <type_traits>

#include <cuda_runtime.h>

#include "dn.h"
#include "dn_attn.cuh"
#include "dn_internal.h"
#include "dn_kv_host.h"
#include "dn_mma.cuh"

namespace dn {
namespace {

template <bool BF>
__device__ __forceinline__ void mma_rows(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Chunk c (16 bytes) of row r in a tile of CPR chunks a row: conflict-free for 8-row ldmatrix reads.
template <int CPR>
__device__ __forceinline__ int chunk_at(int r, int c) {
    return CPR >= 8 ? r * CPR + (c ^ (r & 7)) : r * CPR + (c ^ ((r >> 1) & (CPR - 1)));
}

template <int D, int MT, bool KV8>
struct RowsShape {
    static constexpr int W = 4;                               // warps
    static constexpr int EB = KV8 ? 1 : 2;                    // bytes of a cached element
    // Tokens of a warp's step, in halves of 16 (a page is a multiple of that): 32 where 16 tokens are few
    // bytes and the instructions of a step weigh (8 bits, D = 64), 16 where the ring would leave too few warps.
    static constexpr int H = D * EB <= 128 ? 2 : 1, P = 16 * H;
    static constexpr int HALF = 16 * D * EB;                  // bytes of 16 tokens' keys
    static constexpr int TILE = H * HALF;
    static constexpr int STAGE = 2 * TILE + (KV8 ? 32 * H : 0);   // keys, values, exponent bytes
    // Ring stages. Two leave three CTAs an SM (96 KB in flight, and 12 warps to compute): with four, one CTA of
    // 4 warps, the batch of 64 single tokens (D = 128, 16-bit) took 266 us instead of 193.
    static constexpr int ST = D * EB >= 256 && !(D == 128) ? 3 : 2;
    static constexpr int CTAS = MT == 2 ? 2 : D == 64 ? 4 : D == 128 ? 3 : KV8 ? 2 : 1;  // an SM: bounds the registers
    static constexpr int M = 16 * MT;
    static constexpr bool QREG = D * MT <= 128;               // q fragments in registers, else shared
    static constexpr size_t RING = (size_t)W * ST * STAGE;
    static constexpr size_t MERGE = (size_t)W * M * (D + 2) * 4;  // the warps' outputs, in the ring's place
    static constexpr size_t QOFF = ((RING > MERGE ? RING : MERGE) + 15) / 16 * 16;
    static constexpr size_t SMEM = QOFF + (QREG ? 0 : (size_t)MT * (D / 16) * 32 * 16);
};

template <int D, int MT, bool BF, bool KV8>
__global__ void __launch_bounds__(128, RowsShape<D, MT, KV8>::CTAS)
attn_rows_kernel(const __grid_constant__ AttnArgs a, bool io_bf) {
    using S = RowsShape<D, MT, KV8>;
    constexpr int W = S::W, ST = S::ST, KS = D / 16, CPR = D * S::EB / 16, M = S::M, H = S::H, P = S::P;
    constexpr bool MB = BF && !KV8;  // type of the MMAs
    constexpr float P_UP = MB || KV8 ? 0.f : 15.f, P_DOWN = MB || KV8 ? 1.f : 0x1p-15f;  // binades of the probabilities (KV8: in vf)
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane >> 2, t4 = lane & 3;
    grid_dep_wait();
    grid_dep_trigger();
    AttnUnit u;
    if (!attn_unit<false>(a, blockIdx.x, u)) return;
    if (u.c >= u.ranges) return;
    const int row0 = u.t * M, rows = min(M, u.n * a.G - row0);  // (the host bounds total * heads)

    // ---- the ring: piece i of this warp is tokens lo + P (warp + W i) .. + P - 1 of the range
    unsigned char *ring = smem + (size_t)warp * ST * S::STAGE;
    const int pieces = max(0, ((u.hi - u.lo + P - 1) / P - warp + W - 1) / W);
    int page_ahead = -1;  // lane l: the pool page of this warp's 16 tokens number 32 * batch + l
    // Tokens before the window are in the warps' first pieces alone: the range begins less than 64 tokens before it.
    static_assert(P * W >= 64, "ranges begin at multiples of 64");
    auto load = [&](int i, auto first) {
        if (i < pieces) {
            if (((i * H) & 31) == 0) page_ahead = pool_page(a.p, u.b, u.lo + P * (warp + W * (i + lane / H)) + 16 * (lane % H));
            unsigned char *st = ring + (i % ST) * S::STAGE;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int pg = __shfl_sync(0xffffffffu, page_ahead, (i * H + h) & 31);
                const int j0 = u.lo + P * (warp + W * i) + 16 * h;
                const long long row0 = ((((long long)max(pg, 0) * a.p.heads + u.h)) << a.p.page_shift) + (j0 & ((1 << a.p.page_shift) - 1));
                const int live = pg < 0 ? 0 : min(16, u.hi - j0);  // rows past the range are zeros,
                const int dead = first ? u.see - j0 : 0;           // as are those before the window
                const unsigned char *ks = static_cast<const unsigned char *>(a.kc) + row0 * (D * S::EB) + lane * 16;
                const unsigned char *vs = static_cast<const unsigned char *>(a.vc) + row0 * (D * S::EB) + lane * 16;
#pragma unroll
                for (int x = 0; x < 16 * CPR / 32; ++x) {
                    const int e = x * 32 + lane, at = h * S::HALF + 16 * chunk_at<CPR>(e / CPR, e % CPR);
                    if (live >= 16 && dead <= 0) {
                        cp_async16(st + at, ks + x * 512, 16);
                        cp_async16(st + S::TILE + at, vs + x * 512, 16);
                    } else {  // (nothing is read where the count is 0)
                        const int bytes = e / CPR < live && e / CPR >= dead ? 16 : 0;
                        cp_async16(st + at, bytes ? ks + x * 512 : static_cast<const unsigned char *>(a.q), bytes);
                        cp_async16(st + S::TILE + at, bytes ? vs + x * 512 : static_cast<const unsigned char *>(a.q), bytes);
                    }
                }
                if (KV8 && lane < 2)
                    cp_async16(st + 2 * S::TILE + 32 * h + 16 * lane, live > 0 ? (lane ? a.ve : a.ke) + row0 : static_cast<const uint8_t *>(a.q), live > 0 ? 16 : 0);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) {
        if (i == 0) load(i, std::true_type{});
        else load(i, std::false_type{});
    }

    // ---- q fragments: rows g and g + 8 of each 16-row tile
    unsigned qf[S::QREG ? MT : 1][S::QREG ? KS : 1][4];
    uint4 *qs = reinterpret_cast<uint4 *>(smem + S::QOFF);
    float row_scale[MT][2];  // factor of a row's scores
    int pos[MT][2];          // position of the row's token, INT_MIN/2 for rows that are not there
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const unsigned short *src[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r = 16 * mt + g + 8 * hh;
            const int tok = (row0 + r) / a.G;
            src[hh] = r < rows ? static_cast<const unsigned short *>(a.q) + (u.s + tok) * a.q_stride +
                                     (long long)(u.h * a.G + row0 + r - tok * a.G) * D
                               : nullptr;
            pos[mt][hh] = r < rows ? u.first + tok : -(1 << 30) - (1 << 29);
            row_scale[mt][hh] = a.scale_log2;
        }
        if (!KV8) {
            if (S::QREG || warp == 0) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    unsigned f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)  // a0, a1: rows g, g + 8 at k = 2 t4; a2, a3: at k = 2 t4 + 8
                        f[e] = src[e & 1] ? __ldg(reinterpret_cast<const unsigned *>(src[e & 1] + 16 * ks + 2 * t4 + 8 * (e >> 1))) : 0u;
                    if (S::QREG) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) qf[S::QREG ? mt : 0][S::QREG ? ks : 0][e] = f[e];
                    } else {
                        qs[(mt * KS + ks) * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
                    }
                }
            }
        } else {
            // a thread holds k = 16 ks + 4 t4 .. + 3 of its rows (the order of the key bytes)
            float s2[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float big = 0.f;
#pragma unroll 4
                for (int ks = 0; ks < KS; ++ks) {
                    const uint2 w = src[hh] ? __ldg(reinterpret_cast<const uint2 *>(src[hh] + 16 * ks + 4 * t4)) : make_uint2(0, 0);
                    const float2 x = io_bf ? unpack2<true>(w.x) : unpack2<false>(w.x), y = io_bf ? unpack2<true>(w.y) : unpack2<false>(w.y);
                    big = fmaxf(fmaxf(big, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(y.x), fabsf(y.y)));
                }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                // q = (q 2^-e) 2^e with the largest of the row in [1, 2)
                const int e = min(max((int)(__float_as_uint(big) >> 23) - 127, -126), 126);
                s2[hh] = __int_as_float((127 - e) << 23);
                row_scale[mt][hh] = score_factor(a.scale_log2, e);
            }
            if (S::QREG || warp == 0) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    unsigned f[4];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const uint2 w = src[hh] ? __ldg(reinterpret_cast<const uint2 *>(src[hh] + 16 * ks + 4 * t4)) : make_uint2(0, 0);
                        const float2 x = io_bf ? unpack2<true>(w.x) : unpack2<false>(w.x), y = io_bf ? unpack2<true>(w.y) : unpack2<false>(w.y);
                        f[hh] = pack2<false>(x.x * s2[hh], x.y * s2[hh]);
                        f[2 + hh] = pack2<false>(y.x * s2[hh], y.y * s2[hh]);
                    }
                    if (S::QREG) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) qf[S::QREG ? mt : 0][S::QREG ? ks : 0][e] = f[e];
                    } else {
                        qs[(mt * KS + ks) * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
                    }
                }
            }
        }
    }
    if (!S::QREG) __syncthreads();
    const int row0_pos = u.first + row0 / a.G;  // positions of the tile's first and last token
    const int last = u.first + (row0 + rows - 1) / a.G;

    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
        m[mt][0] = m[mt][1] = -INFINITY;
        l[mt][0] = l[mt][1] = 0.f;
    }
    int ref = 0;  // 8 bits: the largest value exponent so far

    for (int i = 0; i < pieces; ++i) {
        cp_async_wait<ST - 2>();
        __syncwarp();
        load(i + ST - 1, std::false_type{});
        const unsigned char *st = ring + (i % ST) * S::STAGE;
        const int j0 = u.lo + P * (warp + W * i);
        // ---- scores
        float s[MT][2 * H][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 8 * H; ++x) s[mt][x >> 2][x & 3] = 0.f;
        unsigned kb[H][4];  // 8 bits: key bytes of two k-steps
#pragma unroll
        for (int ks = 0; ks < KS; ks += KV8 ? 2 : 1) {
#pragma unroll
            for (int x = 0; x < (KV8 ? 2 : 1); ++x) {
                unsigned f[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if (S::QREG) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[mt][e] = qf[S::QREG ? mt : 0][S::QREG ? ks + x : 0][e];
                    } else {
                        const uint4 w = qs[(mt * KS + ks + x) * 32 + lane];
                        f[mt][0] = w.x; f[mt][1] = w.y; f[mt][2] = w.z; f[mt][3] = w.w;
                    }
                }
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    unsigned b[2][2];
                    if (!KV8) {
                        // matrices: tokens 0-7 at k 0-7, k 8-15, tokens 8-15 at k 0-7, k 8-15
                        unsigned r[4];
                        ldsm_x4(r, st + h * S::HALF + 16 * chunk_at<CPR>((lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
                        b[0][0] = r[0]; b[0][1] = r[1]; b[1][0] = r[2]; b[1][1] = r[3];
                    } else {
                        // matrices: tokens 0-7, 8-15 at bytes 16 ks .., then at bytes 16 (ks + 1) ..
                        if (x == 0) ldsm_x4(kb[h], st + h * S::HALF + 16 * chunk_at<CPR>((lane & 7) + (((lane >> 3) & 1) << 3), ks + (lane >> 4)));
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            b[nt][0] = unpack_e4m3((unsigned short)kb[h][2 * x + nt]);
                            b[nt][1] = unpack_e4m3((unsigned short)(kb[h][2 * x + nt] >> 16));
                        }
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma_rows<MB>(s[mt][2 * h], f[mt], b[0][0], b[0][1]);
                        mma_rows<MB>(s[mt][2 * h + 1], f[mt], b[1][0], b[1][1]);
                    }
                }
            }
        }
        // ---- exponents of the keys and values (tokens 8 nt + 2 t4, + 1 of this thread)
        float vf[2 * H][2];
        if (KV8) {
            // bytes past the range or before the window are not of the rows'
            const int see = a.window && i == 0 ? row0_pos - a.window + 1 : 0;
            const bool part = j0 + P > u.hi || j0 < see;
            const unsigned char *ex = st + 2 * S::TILE;  // of each half: 16 keys', 16 values'
            unsigned top = 0;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const uint4 all = *reinterpret_cast<const uint4 *>(ex + 32 * h + 16);
                unsigned w[4] = {all.x, all.y, all.z, all.w};
                if (part) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int livebytes = min(max(u.hi - j0 - 16 * h - 4 * x, 0), 4), deadbytes = min(max(see - j0 - 16 * h - 4 * x, 0), 4);
                        if (livebytes < 4) w[x] &= (1u << (8 * livebytes)) - 1u;
                        w[x] = deadbytes < 4 ? w[x] & (0xffffffffu << (8 * deadbytes)) : 0u;
                    }
                }
                top = __vmaxu4(top, __vmaxu4(__vmaxu4(w[0], w[1]), __vmaxu4(w[2], w[3])));
            }
            top = __vmaxu4(top, top >> 16);
            top = max(top & 0xffu, (top >> 8) & 0xffu);
            if ((int)top > ref) {  // the same in every lane
                const float f = exp2_fast((float)(ref - (int)top));
                ref = (int)top;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < D / 8; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[mt][j][e] *= f;
            }
#pragma unroll
            for (int nt = 0; nt < 2 * H; ++nt) {
                const unsigned char *at = ex + 32 * (nt / 2) + 8 * (nt & 1) + 2 * t4;
                const unsigned k2 = *reinterpret_cast<const unsigned short *>(at), v2 = *reinterpret_cast<const unsigned short *>(at + 16);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float kf = exp_byte((k2 >> (8 * e)) & 0xffu);
                    const int x = (int)((v2 >> (8 * e)) & 0xffu) - ref + 15 + 127;
                    vf[nt][e] = __int_as_float(max(x, 0) << 23);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        s[mt][nt][e] *= kf;
                        s[mt][nt][2 + e] *= kf;
                    }
                }
            }
            if (part) {
#pragma unroll
                for (int x = 0; x < 4 * H; ++x) {
                    const int j = j0 + 8 * (x / 2) + 2 * t4 + x % 2;
                    if (j >= u.hi || j < see) vf[x / 2][x % 2] = 0.f;
                }
            }
        }
        // ---- masks: only pieces that some row does not see in full
        const bool edge = j0 + P - 1 > row0_pos || j0 + P > u.hi || (a.window && j0 <= last - a.window);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                if (edge) {
#pragma unroll
                    for (int nt = 0; nt < 2 * H; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = j0 + 8 * nt + 2 * t4 + e;
                            if (j > pos[mt][hh] || j >= u.hi || (a.window && j <= pos[mt][hh] - a.window)) s[mt][nt][2 * hh + e] = -INFINITY;
                        }
                }
                float big = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < 2 * H; ++nt) big = fmaxf(fmaxf(big, s[mt][nt][2 * hh]), s[mt][nt][2 * hh + 1]);
                big *= row_scale[mt][hh];
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                const float mn = fmaxf(m[mt][hh], big);
                const float base = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every p is 0
                const bool grew = mn > m[mt][hh];
                if (__any_sync(0xffffffffu, grew)) {
                    const float f = exp2_fast(m[mt][hh] - base);
                    l[mt][hh] *= f;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        o[mt][j][2 * hh] *= f;
                        o[mt][j][2 * hh + 1] *= f;
                    }
                    m[mt][hh] = mn;
                }
#pragma unroll
                for (int nt = 0; nt < 2 * H; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = s[mt][nt][2 * hh + e];
                        x = exp2_fast(fmaf(x, row_scale[mt][hh], P_UP - base));
                        l[mt][hh] += x;
                        if (KV8) x *= vf[nt][e];
                    }
            }
        // ---- output: p (16 rows x 16 tokens, rounded to 16 bits) times the values
#pragma unroll
        for (int h = 0; h < H; ++h) {
            unsigned pf[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) pf[mt][e] = pack2<MB>(s[mt][2 * h + (e >> 1)][2 * (e & 1)], s[mt][2 * h + (e >> 1)][2 * (e & 1) + 1]);
            const unsigned char *sv = st + S::TILE + h * S::HALF;
#pragma unroll
            for (int c = 0; c < CPR; c += 2) {
                // matrices: tokens 0-7, 8-15 at chunk c, then at chunk c + 1, transposed
                unsigned r[4];
                ldsm_x4_t(r, sv + 16 * chunk_at<CPR>((lane & 7) + (((lane >> 3) & 1) << 3), c + (lane >> 4)));
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!KV8) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) mma_rows<MB>(o[mt][c + x], pf[mt], r[2 * x], r[2 * x + 1]);
                    } else {
                        // bytes (token, column): (0, 0) (0, 1) (1, 0) (1, 1) -> the even and the odd columns
                        const unsigned w0 = __byte_perm(r[2 * x], 0, 0x3120), w1 = __byte_perm(r[2 * x + 1], 0, 0x3120);
                        const unsigned e0 = unpack_e4m3((unsigned short)w0), e1 = unpack_e4m3((unsigned short)w1);
                        const unsigned d0 = unpack_e4m3((unsigned short)(w0 >> 16)), d1 = unpack_e4m3((unsigned short)(w1 >> 16));
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            mma_rows<MB>(o[mt][2 * (c + x)], pf[mt], e0, e1);
                            mma_rows<MB>(o[mt][2 * (c + x) + 1], pf[mt], d0, d1);
                        }
                    }
                }
            }
        }
        __syncwarp();
    }

    // ---- merge the warps
    cp_async_wait<0>();
    __syncthreads();
    float *mo = reinterpret_cast<float *>(smem);           // [W][M][D]
    float2 *ml = reinterpret_cast<float2 *>(mo + W * M * D);  // [W][M]
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r = 16 * mt + g + 8 * hh;
            float sum = l[mt][hh] * P_DOWN;
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (t4 == 0) ml[warp * M + r] = make_float2(m[mt][hh], sum);
            float *dst = mo + (warp * M + r) * D;
            // 2^(ref - 127 - 15) in two steps: the power itself may be below the smallest float, and the outputs are not
            const float unit = exp_byte(ref);
            auto out = [&](float x) { return x * 0x1p-15f * unit; };
            if (!KV8) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    *reinterpret_cast<float2 *>(dst + 8 * j + 2 * t4) = make_float2(o[mt][j][2 * hh] * P_DOWN, o[mt][j][2 * hh + 1] * P_DOWN);
            } else {
#pragma unroll
                for (int c = 0; c < D / 16; ++c)  // columns 16 c + 4 t4 .. + 3: even, odd, even, odd
                    *reinterpret_cast<float4 *>(dst + 16 * c + 4 * t4) =
                        make_float4(out(o[mt][2 * c][2 * hh]), out(o[mt][2 * c + 1][2 * hh]), out(o[mt][2 * c][2 * hh + 1]),
                                    out(o[mt][2 * c + 1][2 * hh + 1]));
            }
        }
    __syncthreads();
    const bool final = u.ranges == 1;
    float *part = a.part + (u.slot + u.c) * attn_slot(M, D);
    for (int x = threadIdx.x; x < rows * (D / 4); x += 32 * W) {
        const int r = x / (D / 4), d = 4 * (x % (D / 4));
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w * M + r].x);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float2 y = ml[w * M + r];
            const float f = exp2_fast(y.x - base);
            const float4 v = *reinterpret_cast<const float4 *>(mo + (w * M + r) * D + d);
            sum = fmaf(f, y.y, sum);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
        }
        if (final) {
            const int tok = (row0 + r) / a.G;
            const size_t at = (u.s + tok) * (a.p.heads * a.G) + u.h * a.G + row0 + r - tok * a.G;
            const float inv = sum > 0.f ? 1.f / sum : 0.f;
            if (sum != sum) acc.x = acc.y = acc.z = acc.w = sum;
            uint2 w;
            const bool bf = KV8 ? io_bf : BF;
            w.x = bf ? pack2<true>(acc.x * inv, acc.y * inv) : pack2<false>(acc.x * inv, acc.y * inv);
            w.y = bf ? pack2<true>(acc.z * inv, acc.w * inv) : pack2<false>(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(a.out) + at * D + d) = w;
            if (d == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
        } else {
            *reinterpret_cast<float4 *>(part + r * D + d) = acc;
            if (d == 0) *reinterpret_cast<float2 *>(part + M * D + 2 * r) = make_float2(top, sum);
        }
    }
}

// ---- join: the ranges of a tile, in their order ----------------------------------------------
// A CTA joins ROWS rows of one tile and head, its eight warps in equal groups a row: each warp adds
// an eighth (or fewer) of the ranges, a lane holding D / 32 columns, and the warps' sums are added in order.
// The partials were written by the launch before and are in L2; a row is few loads deep.
template <int D, int ROWS>
__global__ void __launch_bounds__(256)
attn_join_kernel(const __grid_constant__ AttnArgs a, bool bf) {
    constexpr int E = D / 32, WPR = 8 / ROWS;
    __shared__ float sh[8][D];
    __shared__ float2 sml[8];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    grid_dep_wait();
    grid_dep_trigger();
    AttnUnit u;
    if (!attn_unit<true>(a, blockIdx.x, u) || u.ranges < 2) return;
    const int M = a.M, row0 = u.t * M, rows = min(M, u.n * a.G - row0);
    const int r = blockIdx.y * ROWS + warp / WPR, w = warp % WPR;
    if ((int)(blockIdx.y * ROWS) >= rows) return;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    float top = -INFINITY, sum = 0.f;
    if (r < rows) {
        const size_t slot = attn_slot(M, D);
        const float *p = a.part + u.slot * slot;
        const int per = (u.ranges + WPR - 1) / WPR, c0 = w * per, c1 = min(u.ranges, c0 + per);
#pragma unroll 4
        for (int c = c0; c < c1; ++c) {
            const float2 y = __ldg(reinterpret_cast<const float2 *>(p + c * slot + M * D + 2 * r));
            const float *v = p + c * slot + (size_t)r * D + E * lane;
            float x[E];
            if (E == 2) {
                const float2 q = __ldg(reinterpret_cast<const float2 *>(v));
                x[0] = q.x; x[E - 1] = q.y;
            } else {
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const float4 q = __ldg(reinterpret_cast<const float4 *>(v + e));
                    x[e] = q.x; x[(e + 1) % E] = q.y; x[(e + 2) % E] = q.z; x[(e + 3) % E] = q.w;
                }
            }
            const float most = fmaxf(top, y.x), base = most == -INFINITY ? 0.f : most;
            const float f0 = exp2_fast(top - base), f1 = exp2_fast(y.x - base);
            top = most;
            sum = fmaf(f1, y.y, f0 * sum);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(f1, x[e], f0 * acc[e]);
        }
    }
    if (w) {
#pragma unroll
        for (int e = 0; e < E; ++e) sh[warp][E * lane + e] = acc[e];
        if (lane == 0) sml[warp] = make_float2(top, sum);
    }
    __syncthreads();
    if (w || r >= rows) return;
    float all = top;
#pragma unroll
    for (int i = 1; i < WPR; ++i) all = fmaxf(all, sml[warp + i].x);
    const float base = all == -INFINITY ? 0.f : all, f0 = exp2_fast(top - base);
    sum *= f0;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f0;
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
        const float f = exp2_fast(sml[warp + i].x - base);
        sum = fmaf(f, sml[warp + i].y, sum);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(f, sh[warp + i][E * lane + e], acc[e]);
    }
    const float inv = sum > 0.f ? 1.f / sum : sum != sum ? sum : 0.f;  // NaN stays NaN
    const int tok = (row0 + r) / a.G;
    const size_t at = (u.s + tok) * (a.p.heads * a.G) + u.h * a.G + row0 + r - tok * a.G;
    unsigned *dst = reinterpret_cast<unsigned *>(static_cast<unsigned short *>(a.out) + at * D + E * lane);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = bf ? pack2<true>(acc[e] * inv, acc[e + 1] * inv) : pack2<false>(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (all + log2f(sum)) * 0.693147180559945f;
}

// ---- host: which kernel, and how many units ---------------------------------------------------

// Tiles' ranges are of 256 tokens or more. 64 rows over 1,200 tokens of 8 x 128-wide heads took 17.5, 14.5 and 13.3 us
// with at least 1,024, 512 and 256; over 600 tokens not to cut was better (11.2 us against 12.8), which join_cost
// is for. Over 96 shapes of 600 to 5,000 tokens, 256 was 8 % faster than 512 and 1,024 9 % slower.
struct AttnPlan {
    bool tc;
    int M, wave, target, align, min_range, unit_cost, join_cost;
};

AttnPlan attn_plan(int B, int total, int G, int D, bool kv8) {
    // rows of a request, on average over the batch
    const long long rows = B > 0 ? ((long long)total * G + B - 1) / B : 0;
    // Warp MMAs up to 16 rows, and up to 32 where tcgen05 tiles are no faster: 64 requests x 8,000 tokens, 24 rows of
    // each of 4 key heads: D = 128 in 16 bits 218 us on warps and 201 in tiles, in 8 bits 198 and 349, D = 64 128 and 163.
    // D = 256 holds 16 rows a warp. A group of more than 128 heads has more rows than a tcgen05 tile: warp MMAs.
    const int most = D == 256 || (D == 128 && !kv8) ? 16 : 32;
    if (rows > most && G <= 128)
        return {true, 128 / G * G * (D == 256 ? 1 : 2), kAttnSms, kAttnSms, D == 256 ? 64 : 128, 256, 600, 150};
    const int resident = D == 256 ? (kv8 ? 2 : 1) : 3;  // CTAs an SM
    return {false, rows <= 16 ? 16 : most, resident * kAttnSms, 8 * kAttnSms, 64, 64, 400, 100};
}

// Sizes that the attention takes, as far as they are products.
bool attn_sizes_ok(int total, int heads_kv, int group) {
    const long long heads = (long long)heads_kv * group;
    return heads <= (1 << 20) && total * heads <= 0x7fffffffLL - 1024;
}

template <int D, int MT, bool BF, bool KV8>
void launch_rows(const AttnArgs &a, bool io_bf, unsigned grid, cudaStream_t st) {
    using S = RowsShape<D, MT, KV8>;
    cudaFuncSetAttribute(attn_rows_kernel<D, MT, BF, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::SMEM);
    launch_pdl(attn_rows_kernel<D, MT, BF, KV8>, dim3(grid), dim3(128), S::SMEM, st, a, io_bf);
}

template <int D, int MT>
bool launch_rows(const AttnArgs &a, bool bf, bool kv8, unsigned grid, cudaStream_t st) {
    if (a.M != 16 * MT) return false;
    if (kv8) launch_rows<D, MT, false, true>(a, bf, grid, st);
    else if constexpr (D == 64 || MT == 1) {
        if (bf) launch_rows<D, MT, true, false>(a, bf, grid, st);
        else launch_rows<D, MT, false, false>(a, bf, grid, st);
    } else return false;
    return true;
}

}  // namespace

template <int ROWS>
void launch_join(const AttnArgs &a, int D, bool bf, unsigned pairs, unsigned rows, cudaStream_t st) {
    const dim3 grid(pairs, (rows + ROWS - 1) / ROWS);
    if (D == 64) launch_pdl(attn_join_kernel<64, ROWS>, grid, dim3(256), 0, st, a, bf);
    else if (D == 128) launch_pdl(attn_join_kernel<128, ROWS>, grid, dim3(256), 0, st, a, bf);
    else launch_pdl(attn_join_kernel<256, ROWS>, grid, dim3(256), 0, st, a, bf);
}

// Few tiles have many ranges each: a CTA a row, as long as that is at most a few waves of CTAs. Many tiles
// have few ranges, and most CTAs of a grid that covers them all have nothing to join: eight rows a CTA.
void launch_attn_join(const AttnArgs &a, int D, bool bf, cudaStream_t st) {
    const long long pairs = std::min((long long)std::max(a.target, a.wave), attn_tiles_bound(a.p.B, a.p.total, a.G, a.M) * a.p.heads);
    const long long rows = std::min((long long)a.M, (long long)a.p.total * a.G);
    if (pairs * rows <= 8 * kAttnSms) launch_join<1>(a, D, bf, (unsigned)pairs, (unsigned)rows, st);
    else launch_join<8>(a, D, bf, (unsigned)pairs, (unsigned)rows, st);
}

}  // namespace dn

extern "C" size_t dn_attn_workspace_bytes(int B, int total, int heads_kv, int group, int D) {
    using namespace dn;
    if (B < 1 || total < 1 || total > DN_KV_MAX_ROWS || heads_kv < 1 || group < 1 || !kv_shape_ok(D, 16) ||
        !attn_sizes_ok(total, heads_kv, group))
        return 0;
    size_t most = 0;
    for (int kv8 = 0; kv8 < 2; ++kv8) {
        const AttnPlan p = attn_plan(B, total, group, D, kv8);
        most = std::max(most, (2 * std::max(p.target, p.wave) + 64) * attn_slot(p.M, D) * sizeof(float));
    }
    return most;
}

extern "C" dn_status dn_attn_paged(int B, int total, int heads_kv, int group, int D, int page, int max_pages, int pages,
                                   dn_dtype io_dt, dn_dtype cache_dt, const void *q, int64_t q_stride,
                                   const int32_t *start, const int32_t *kv_len, const int32_t *page_table,
                                   const void *k_cache, const void *v_cache, const uint8_t *k_exp,
                                   const uint8_t *v_exp, float scale, int window, void *out, float *lse,
                                   void *workspace, size_t workspace_bytes, dn_stream_t stream) {
    using namespace dn;
    if (B < 0 || total < 0 || total > DN_KV_MAX_ROWS || heads_kv < 1 || group < 1 || window < 0 ||
        !(scale > 0.f) || !(scale < 2e38f) || !kv_dtypes_known(io_dt, cache_dt))
        return DN_ERR_INVALID_ARG;
    if (!kv_shape_ok(D, page) || !kv_dtypes_ok(io_dt, cache_dt)) return DN_ERR_UNSUPPORTED;
    if (!attn_sizes_ok(total, heads_kv, group) || !kv_pages_ok(max_pages, pages, page) || q_stride < (int64_t)heads_kv * group * D || q_stride % 8)
        return DN_ERR_INVALID_ARG;
    if (B == 0 || total == 0) return DN_OK;
    if (!kv_pointers_ok(B, start, kv_len, page_table, k_cache, v_cache, k_exp, v_exp, cache_dt, pages, max_pages) || !q ||
        !out || !workspace || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16) ||
        workspace_bytes < dn_attn_workspace_bytes(B, total, heads_kv, group, D))
        return DN_ERR_INVALID_ARG;
    AttnPlan p = attn_plan(B, total, group, D, cache_dt == DN_E4M3);
    if (pages == 0 || max_pages == 0) p = {false, 16, kAttnSms, kAttnSms, 64, 64, 400, 100};  // nothing is cached: no pool to copy from
    // At most this many units: few tiles are cut for one wave (CTAs without a unit still cost their launch),
    // and a table of few pages bounds the ranges of a tile.
    const long long whole = attn_tiles_bound(B, total, group, p.M) * heads_kv;
    if (2 * whole < p.wave) p.target = p.wave;
    const long long units = std::min(std::max(p.target, p.wave) + whole,
                                     whole * std::max(1LL, ((long long)max_pages * page + p.min_range - 1) / p.min_range));
    if (units > 0x7fffffffLL) return DN_ERR_INVALID_ARG;
    AttnArgs a;
    a.p = {start, kv_len, page_table, B, total, max_pages, pages, page_log2(page), heads_kv};
    a.q = q;
    a.q_stride = q_stride;
    a.kc = k_cache;
    a.vc = v_cache;
    a.ke = k_exp;
    a.ve = v_exp;
    a.out = out;
    a.lse = lse;
    a.part = static_cast<float *>(workspace);
    a.G = group;
    a.scale_log2 = scale * 1.44269504088896f;
    a.window = window >= DN_KV_MAX_TOKENS ? 0 : window;
    a.M = p.M;
    a.align = p.align;
    a.wave = p.wave;
    a.target = p.target;
    a.min_range = p.min_range;
    a.unit_cost = p.unit_cost;
    a.join_cost = p.join_cost;
    a.soft = !p.tc;
    const bool bf = io_dt == DN_BF16, kv8 = cache_dt == DN_E4M3;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    bool launched = true;
    if (p.tc && pages > 0 && max_pages > 0) {
        const dn_status ok = launch_attn_tc(a, D, bf, kv8, (unsigned)units, st);
        if (ok != DN_OK) return ok;
    } else if (D == 64 && p.M == 16) launched = launch_rows<64, 1>(a, bf, kv8, (unsigned)units, st);
    else if (D == 64) launched = launch_rows<64, 2>(a, bf, kv8, (unsigned)units, st);
    else if (D == 128 && p.M == 16) launched = launch_rows<128, 1>(a, bf, kv8, (unsigned)units, st);
    else if (D == 128) launched = launch_rows<128, 2>(a, bf, kv8, (unsigned)units, st);
    else launched = launch_rows<256, 1>(a, bf, kv8, (unsigned)units, st);
    if (!launched) return DN_ERR_UNSUPPORTED;  // (a plan for a kernel that is not there)
    if (units > whole) launch_attn_join(a, D, bf, st);  // (else no tile can have two ranges)
    return launch_status();
}
