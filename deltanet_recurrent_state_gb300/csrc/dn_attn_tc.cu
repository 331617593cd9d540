// dn_attn_paged for tiles of many rows, on tcgen05 tensor cores.
//
// The mathematics is in dn_attn.cu, the cutting of the work in dn_attn.cuh. A unit is one CTA that
// has an SM's tensor memory to itself: S = Q K^T of 128 rows by BN cached tokens, P = exp2(S - m),
// O += P V, with S, P and O in tensor memory and nothing but Q, K and V in shared memory.
//
// Steps and streams. Step j computes S into buffer j & 1; its softmax turns that into P (16 bits, in the
// same columns if D = 128); P V is added to an accumulator. S(j + 2) may overwrite P(j) because products of
// one shape run in the order of their issue; for the other D the shapes differ and P has its own columns.
// The tensor core runs S(0), S(1), then P V(j), S(j + 2), .., so one step's softmax always has another
// step's products beside it. For D <= 128 the even and the odd steps are two streams with a warpgroup and an
// accumulator each: if the unit has more than 128 rows (a prompt's chunk) the streams are its two halves of
// rows over the same keys, else (a verify block) they are the even and the odd key tiles of the same rows,
// merged at the end. For D = 256 an accumulator takes half of the tensor memory: one stream, key tiles of
// 64 tokens, of which each of the two warpgroups has half of the columns.
//
// Copies. K and V tiles pass through one ring of shared-memory slots in the order in which the products take
// them. Pages come in by TMA, one box per page and 64 columns, with the 128-byte swizzle that the MMA
// descriptors read; the producer's lanes look the pages up 32 at a time. A page that a
// request does not have is an out-of-range coordinate, which the copy fills with zeros. Rows of the last
// page past the range, and of the first one before a window, may hold anything: their scores are masked, and
// their values are zeroed in shared memory before the product (0 x NaN is not 0). q comes the same way, G heads
// by 128 / G tokens a box, so a tile is as many whole tokens as 128 rows hold.
//
// 8-bit caches. The boxes land in a ring of raw tiles, and a warpgroup turns them into fp16 tiles, multiplied
// by the powers of two 2^(E - R + 7) of the tokens: R is the tile's largest exponent for the keys, whose
// 2^R joins the score's factor, and the largest so far for the values, so that tiles add up. The largest e4m3,
// 448, becomes 57,344 at most, inside fp16's range; at the other end elements are rounded once, to multiples of 2^-24,
// which is 2^-40 of that (without the 7 binades, 2^-33). The largest element may be one that a row does not
// see. bf16 q is brought to fp16 by a power of two for each row, as in dn_attn.cu.
//
// Running maximum. O is rescaled only when a row's maximum grows by more than 2^8: until then its
// probabilities are at most 2^8, rounded to 16 bits with the same relative step, and the division by the
// sum at the end takes the factor out again. fp16 ones are held as 2^7 p, up to 2^15: fp16's smallest number is then
// 2^-31 (see dn_attn.cu).
//
// Measured on a GB300. A prompt's chunk (2,048 tokens, 25,000 cached with them, 32 x 128 heads, bf16) takes 589 us,
// 1,370 TFLOP/s, 71 % of cuBLAS's rate (about 565 back to back on one input): its 256 units are 1.7 waves of 152,
// 84 % of two, and a chunk of 1,216 over 8,192 keeps the tensor pipe active 64 % of the cycles. A verify block
// (96 rows of D = 256 over 25,000 tokens, 16 bits) takes 34 us for 15 us of bytes: one wave, of which about 8 us
// are its end and the join. Over 268,000 tokens in 8 bits it takes 172 us for 81: a 64-token tile took 2,750 to 3,300
// cycles by clock stamps at 175 us, 1,400 would be the copy rate; three 16-bit slots are what fits beside q.
//
// Every wait is bounded in time; a wait that runs out raises the CTA's abort flag, and every role
// leaves after its own copies and products have landed.
#include <type_traits>

#include <cuda_runtime.h>

#include "dn.h"
#include "dn_attn.cuh"
#include "dn_internal.h"
#include "dn_mma.cuh"
#include "dn_tc05.cuh"
#include "dn_tmap.h"

namespace dn {
namespace {

__device__ unsigned int g_attn_timeouts;

// D += A B with A in tensor memory (16-bit elements, two to a column).
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
                 :: "r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}

#define DN_R32(r)                                                                                                  \
    "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),    \
        "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),     \
        "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),    \
        "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])

// 32 lanes x 32 columns; the registers may be read after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
                   "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
                   "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
                   "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[N][32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : DN_R32(r[0])::"memory");
#pragma unroll
    for (int i = 1; i < N; ++i) asm volatile("" : DN_R32(r[i])::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                    "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
                    "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_3d(void *smem, const void *tmap, int c0, int c1, int c2, unsigned long long *mb) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(smem_addr(smem)), "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(mb)) : "memory");
}
__device__ __forceinline__ void mbar_arrive(unsigned long long *mb) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(smem_addr(mb)) : "memory");
}
__device__ __forceinline__ bool mbar_test(unsigned long long *mb, unsigned parity) {
    unsigned ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(smem_addr(mb)), "r"(parity) : "memory");
    return ok;
}
// mbar_wait_guarded for a whole warp, which sees one answer; the timer is read only if the phase is not
// complete at once.
__device__ __forceinline__ bool wait_for(unsigned long long *mb, unsigned parity, volatile int *abort) {
    bool ok = mbar_test(mb, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    if (!ok) ok = mbar_wait_guarded(mb, parity, abort, &g_attn_timeouts);
    return __all_sync(0xffffffffu, ok);
}
// The same for a single thread.
__device__ __forceinline__ bool wait_one(unsigned long long *mb, unsigned parity, volatile int *abort) {
    return mbar_test(mb, parity) || mbar_wait_guarded(mb, parity, abort, &g_attn_timeouts);
}

__device__ __forceinline__ bool elect_one() {
    unsigned r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r;
}

constexpr int P_UP = 7;     // binades that fp16 probabilities, at most 2^8, are raised by
constexpr int TILE_UP = 7;  // binades that an 8-bit tile's elements are raised by: 448 * 2^7 = 57,344 is inside fp16's range

template <int D, bool KV8>
struct TileShape {
    static constexpr int NS = D <= 128 ? 2 : 1;      // streams
    static constexpr int BN = D <= 128 ? 128 : 64;   // tokens of a key tile
    static constexpr int HALVES = D / 64;            // 64-column boxes of a tile
    static constexpr int TILE = BN * D * 2;          // bytes of a 16-bit K or V tile
    static constexpr int QTILE = 128 * D * 2;
    static constexpr int SLOTS = KV8 ? (D == 64 ? 4 : 3) : (D == 64 ? 6 : D == 128 ? 5 : 4);
    static constexpr int RAW = KV8 ? BN * D : 0;     // bytes of an 8-bit tile
    static constexpr int RAWS = KV8 ? (D == 64 ? 4 : 3) : 0;
    static constexpr int SOFTMAX = 256;              // threads of the softmax warpgroups: a row each, or half a row (D = 256)
    static constexpr int CN = BN * NS / 2;           // columns of S that a thread has
    // Threads that turn 8-bit tiles into fp16: one group for the keys and one for the values, so that one's
    // waits pass beside the other's work. The more elements a token has, the more of the block's registers
    // they are worth: for D = 64 the softmax keeps its scores in registers (three prompts' window of 1,000 took
    // 88 us so, and 104 with 14 such warps), for D = 128 it reads them twice (32 verify blocks of 64 rows: 256 us
    // with 14 warps, 328 with 6).
    static constexpr int CVT = KV8 ? (D == 64 ? 64 : 192) : 0;
    static constexpr bool TWICE = KV8 && D == 128;
    static constexpr int THREADS = SOFTMAX + 128 + 2 * CVT;
    static_assert(THREADS % 128 == 0, "register splits go by warpgroups");
    // columns of tensor memory: S at 0 and BN, P in the place of S for D = 128 (where that fills the
    // 512 columns), else beside it
    static constexpr int COL_P = D == 128 ? 0 : D == 64 ? 384 : 128, P_STEP = D == 128 ? BN : BN / 2, COL_O = 256, O_STEP = D;
    // registers of a softmax thread and of the others; the sum stays within the launch's
    static constexpr bool SPLIT = NS == 2 || KV8;
    static constexpr int R_SOFTMAX = !KV8 ? 208 : D == 64 ? 176 : D == 128 ? 112 : 96, R_OTHER = !KV8 ? 88 : D == 64 ? 80 : D == 128 ? 64 : 72;
    static constexpr int R_LAUNCH = 65536 / THREADS / 8 * 8;
    static_assert(!SPLIT || SOFTMAX * R_SOFTMAX + (THREADS - SOFTMAX) * R_OTHER <= THREADS * R_LAUNCH, "registers");
    static constexpr int OFF_RING = NS * QTILE;
    static constexpr int OFF_RAW = OFF_RING + SLOTS * TILE;
    static constexpr int OFF_POW = OFF_RAW + RAWS * RAW;  // [2][4][BN]: powers of two of a key or value tile's tokens
    static constexpr int OFF_BAR = OFF_POW + (KV8 ? 2 * 4 * BN * 4 : 0);
    static constexpr int OFF_ROW = OFF_BAR + 2048;  // D = 256: [2][2][128] maxima of half rows, [2][128] their sums
    static constexpr int BYTES = OFF_ROW + (NS == 1 ? 3072 : 0) + 1024;                        // and the alignment of the base
    static_assert(BYTES <= 232448, "shared memory of one CTA");
    // Barriers go by tile modulo 4, so a tile's copy must not be issued before the tile four earlier has been
    // used: key tile 4 is the eighth copy of a ring (see seq_k), tile 0 the first.
    static_assert(SLOTS + (NS == 2) <= 7 && RAWS <= 7, "a ring holds fewer copies than lie between tiles t and t + 4");
    static_assert(NS == 1 || QTILE == TILE, "a q tile's place is a slot");
    static constexpr int STAGE = 32 * ((KV8 || D == 64 ? 32 : 64) + 4) * 4;  // a warp's rows on their way out, from the first byte
    static_assert(NS == 1 || 8 * STAGE <= OFF_RING + 8192, "rows on their way out lie before the merge");
    static_assert(NS == 1 || 8192 + 2 * 128 * (D / 2 + 4) * 4 + 2048 <= SLOTS * TILE, "the streams merge in the ring");
};

struct Bars {
    // by kind (keys, values) and tile modulo 4
    unsigned long long full[2][4], empty[2][4], raw_full[2][4], raw_empty[2][4], pow_full[2][4], ref_full[4], s_full[2], p_full[2], most_full[2], pv, q_full, q_ready, first_v, last_v, fin;
    uint32_t tmem;
    int abort, k_ref[4], v_ref[4], tiny[2][4];
    AttnUnit unit[8];  // the unit again, for the end (a copy a warp: held in registers it would cost the softmax some)
    signed char q_exp[256];  // powers of two of bf16 q rows brought to fp16
};
static_assert(sizeof(Bars) <= 2048, "barriers");

// Place of K (or V) tile t of n in the ring's order, and the other way round.
__device__ __forceinline__ int seq_k(bool two_q, int t) { return two_q ? 2 * t : (t == 0 ? 0 : 2 * t - 1); }
__device__ __forceinline__ int seq_v(bool two_q, int t, int n) { return two_q ? 2 * t + 1 : min(2 * t + 2, 2 * n - 1); }
__device__ __forceinline__ void seq_tile(bool two_q, int seq, int n, int &t, bool &is_v) {
    if (two_q) {
        t = seq >> 1;
        is_v = seq & 1;
    } else {
        is_v = seq == 2 * n - 1 || (seq > 0 && !(seq & 1));
        t = seq == 2 * n - 1 ? n - 1 : (seq & 1) ? (seq + 1) >> 1 : seq == 0 ? 0 : (seq - 2) >> 1;
    }
}

// A copy from shared memory that is not what the compiler still holds in registers.
__device__ __forceinline__ AttnUnit again(AttnUnit &from) {
    AttnUnit u;
    int *to = reinterpret_cast<int *>(&u);
    const volatile int *at = reinterpret_cast<const volatile int *>(&from);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(AttnUnit) / 4); ++i) to[i] = at[i];
    return u;
}

// One warp's 32 rows (lane: row) x `cols` columns of an accumulator, times f0 and (8 bits) then `unit`, whose product may
// be below the smallest float where the outputs are not, plus f1 times `other` (the row's values in shared memory, or null), to out (part null) or to a slot of the workspace; `at` is the row of out,
// -1 where there is none. EC columns at a time pass through shared memory, so that EC / 4 lanes write a row's
// neighbouring columns: a lane writing its own row would touch 32 lines a store. Tensor-memory loads are the
// whole warp's, whatever its rows.
template <int D, bool KV8>
__device__ __forceinline__ void put_rows(const AttnArgs &a, void *shared, uint32_t addr, int c0, int cols, float f0, float unit, bool any,
                                         float f1, const float *other, float *part, int row0, int at, bool bf) {
    constexpr int EC = KV8 || D == 64 ? 32 : 64, ER = 128 / EC;  // columns at a time, rows a store
    const int lane = threadIdx.x % 32;
    if (!__any_sync(0xffffffffu, at >= 0)) return;
    float *stage = static_cast<float *>(shared);
#pragma unroll 1
    for (int d = 0; d < cols; d += EC) {
        uint32_t y[EC / 32][32];
        if (any) {
#pragma unroll
            for (int i = 0; i < EC / 32; ++i) tmem_ld32_start(addr + d + 32 * i, y[i]);
            tmem_wait_ld(y);
        }
#pragma unroll
        for (int e = 0; e < EC; e += 4) {
            float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            if (any)
                z = make_float4(f0 * __uint_as_float(y[e / 32][e % 32]), f0 * __uint_as_float(y[e / 32][e % 32 + 1]),
                                f0 * __uint_as_float(y[e / 32][e % 32 + 2]), f0 * __uint_as_float(y[e / 32][e % 32 + 3]));
            if (KV8) z = make_float4(z.x * unit, z.y * unit, z.z * unit, z.w * unit);
            if (other) {
                const float4 w = *reinterpret_cast<const float4 *>(other + d + e);
                z = make_float4(fmaf(f1, w.x, z.x), fmaf(f1, w.y, z.y), fmaf(f1, w.z, z.z), fmaf(f1, w.w, z.w));
            }
            *reinterpret_cast<float4 *>(stage + lane * (EC + 4) + e) = z;
        }
        __syncwarp();
#pragma unroll 8
        for (int i = 0; i < 32 / ER; ++i) {
            const int r = ER * i + lane / (EC / 4), e = 4 * (lane % (EC / 4));
            const int row_at = __shfl_sync(0xffffffffu, at, r);
            const float4 w = *reinterpret_cast<const float4 *>(stage + r * (EC + 4) + e);
            if (row_at < 0) continue;
            if (!part) {
                uint2 h;
                h.x = bf ? pack2<true>(w.x, w.y) : pack2<false>(w.x, w.y);
                h.y = bf ? pack2<true>(w.z, w.w) : pack2<false>(w.z, w.w);
                *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(a.out) + (size_t)row_at * D + c0 + d + e) = h;
            } else {
                *reinterpret_cast<float4 *>(part + (size_t)(row0 + r) * D + c0 + d + e) = w;
            }
        }
        __syncwarp();
    }
}

template <int D, bool BF, bool KV8>
__global__ void __launch_bounds__(TileShape<D, KV8>::THREADS, 1)
attn_tile_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap mq,
                 const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, bool io_bf) {
    using S = TileShape<D, KV8>;
    constexpr int BN = S::BN, CN = S::CN, NS = S::NS, SLOTS = S::SLOTS, TILE = S::TILE;
    constexpr bool MB = BF && !KV8;
    constexpr int W_TMA = S::SOFTMAX / 32, W_MMA = W_TMA + 1;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    unsigned char *raw = smem + S::OFF_RAW;
    Bars &bar = *reinterpret_cast<Bars *>(smem + S::OFF_BAR);
    float *row_most = reinterpret_cast<float *>(smem + S::OFF_ROW), *row_sum = row_most + 512;  // (D = 256)
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(&bar.full[i >> 2][i & 3], KV8 ? S::CVT : 1);
            mbar_init(&bar.empty[i >> 2][i & 3], 1);
            mbar_init(&bar.raw_full[i >> 2][i & 3], 1);
            mbar_init(&bar.raw_empty[i >> 2][i & 3], KV8 ? S::CVT : 1);
            mbar_init(&bar.pow_full[i >> 2][i & 3], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&bar.ref_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], NS == 1 ? 256 : 128);
            mbar_init(&bar.most_full[i], 256);
        }
        mbar_init(&bar.pv, 1);
        mbar_init(&bar.q_full, 1);
        mbar_init(&bar.q_ready, S::SOFTMAX);
        mbar_init(&bar.first_v, 1);
        mbar_init(&bar.last_v, 1);
        mbar_init(&bar.fin, 1);
        bar.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == W_MMA) tmem_alloc<512>(&bar.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = bar.tmem;
    volatile int *abort = &bar.abort;
    // (all of this beside the launch before; from here on every warp goes its own way)
    grid_dep_wait();
    grid_dep_trigger();
    AttnUnit u;
    if (!attn_unit<false>(a, blockIdx.x, u) || u.c >= u.ranges) {
        if (warp == W_MMA) tmem_free<512>(tm);
        return;
    }
    if (warp < 8 && lane == 0) bar.unit[warp] = u;
    __syncwarp();
    const int mq_rows = a.M / NS;                                 // rows of a q tile: whole tokens, at most 128
    const int row0 = u.t * a.M, rows = min(a.M, u.n * a.G - row0);  // (the host bounds total * heads)
    const bool two_q = NS == 2 && rows > mq_rows;
    const int tiles = (u.hi - u.lo + BN - 1) / BN;
    const int steps = two_q ? 2 * tiles : tiles;
    const int head = max(u.see - u.lo, 0);  // tokens of the first tile that no row sees (fewer than a tile)
    // the ring; without a second q tile, its place is one more slot
    const bool wide = NS == 2 && !two_q;
    unsigned char *ring = smem + S::OFF_RING - (wide ? S::QTILE : 0);
    const int slots = wide ? SLOTS + 1 : SLOTS;
    auto slot_of = [&](int seq) { return wide ? seq % (SLOTS + 1) : seq % SLOTS; };

    if (warp == W_TMA || (!KV8 && warp == W_TMA + 3)) {
        if (S::SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::R_OTHER));
        // ---- producers. Issuing a copy takes a thread over 100 cycles, so keys and values have a warp each; for 8 bits,
        // whose boxes are whole rows, one warp does for both.
        const bool values = warp != W_TMA;
        const int page = 1 << a.p.page_shift, R = min(page, BN);  // tokens of a box
        const int NB = KV8 ? S::RAWS : slots;
        int issued = 0;
        if (tiles > 0 && !values && elect_one()) {
            const int tokens = 128 / a.G, boxes_q = S::HALVES * (two_q ? 2 : 1);
            mbar_arrive_expect_tx(&bar.q_full, boxes_q * mq_rows * 128);
            for (int i = 0; i < boxes_q; ++i)
                tma_load_3d(smem + i / S::HALVES * S::QTILE + i % S::HALVES * (128 * 128), &mq, i % S::HALVES * 64, u.h * a.G,
                            u.s + row0 / a.G + i / S::HALVES * tokens, &bar.q_full);
        }
        __syncwarp();
        // pool pages of this unit, 32 boxes' worth a batch, a lane each: the batch in use and the next, which the
        // keys may be ahead in
        const int per_log2 = (BN == 128 ? 7 : 6) - min(a.p.page_shift, BN == 128 ? 7 : 6), per = 1 << per_log2;  // boxes of a tile
        auto look = [&](int x) {
            const int j = u.lo + (32 * x + lane) * R, pg = j < u.hi ? pool_page(a.p, u.b, j) : -1;
            return pg < 0 ? a.p.pages : pg;  // past the last page: zeros
        };
        int pages_even = look(0), pages_odd = look(1);
        for (int seq = 0; seq < 2 * tiles; ++seq) {
            int t;
            bool is_v;
            seq_tile(two_q, seq, tiles, t, is_v);
            if (!KV8 && is_v != values) continue;
            const int x = (t << per_log2) >> 5;
            if ((!KV8 || is_v) && x > 0 && ((t << per_log2) & 31) == 0) {
                if (x & 1) pages_even = look(x + 1);
                else pages_odd = look(x + 1);
            }
            const int ids = x & 1 ? pages_odd : pages_even;
            const int slot = KV8 ? seq % (KV8 ? S::RAWS : 1) : slot_of(seq), j0 = u.lo + t * BN;
            unsigned long long *full = KV8 ? &bar.raw_full[is_v][t & 3] : is_v && t == tiles - 1 ? &bar.last_v
                                       : is_v && t == 0 && head > 0 ? &bar.first_v : &bar.full[is_v][t & 3];
            if (seq >= NB) {  // what was in the slot before
                int t0;
                bool v0;
                seq_tile(two_q, seq - NB, tiles, t0, v0);
                if (!wait_for(KV8 ? &bar.raw_empty[v0][t0 & 3] : &bar.empty[v0][t0 & 3], (t0 >> 2) & 1, abort)) break;
            }
            if (elect_one()) mbar_arrive_expect_tx(full, KV8 ? S::RAW : TILE);
            const int y0 = u.h * page + (j0 & (page - 1));  // (a tile starts a page, or lies in one)
            for (int box = 0; box < per; ++box) {
                const int pg = __shfl_sync(0xffffffffu, ids, ((t << per_log2) + box) & 31);
                if (elect_one()) {
                    unsigned char *dst = KV8 ? raw + slot * S::RAW + box * R * D : ring + slot * TILE + box * R * 128;
#pragma unroll
                    for (int half = 0; half < (KV8 ? 1 : S::HALVES); ++half)
                        tma_load_3d(dst + half * BN * 128, is_v ? &mv : &mk, half * 64, y0, pg, full);
                }
            }
            __syncwarp();
            issued = seq + 1;
        }
        if (*abort) {  // what was copied has to land before the CTA leaves
            if (tiles > 0 && !values) mbar_drain(&bar.q_full, 0);
            for (int seq = max(0, issued - 2 * NB); seq < issued; ++seq) {
                int t;
                bool is_v;
                seq_tile(two_q, seq, tiles, t, is_v);
                if (!KV8 && is_v != values) continue;
                if (!KV8 && is_v && t == tiles - 1) mbar_drain(&bar.last_v, 0);
                else if (!KV8 && is_v && t == 0 && head > 0) mbar_drain(&bar.first_v, 0);
                else if (seq >= issued - NB) mbar_drain(KV8 ? &bar.raw_full[is_v][t & 3] : &bar.full[is_v][t & 3], (t >> 2) & 1);
            }
        }
    } else if (warp == W_MMA) {
        if (S::SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::R_OTHER));
        // ---- products, all by one thread
        constexpr uint32_t type = MB ? (1u << 7) | (1u << 10) : 0u;
        constexpr uint32_t id_s = umma_idesc(128, BN, 0, 0) | type, id_o = umma_idesc(128, D, 0, 1) | type;
        if (steps > 0 && elect_one()) {
            bool ok = wait_one(&bar.q_full, 0, abort) && (!(KV8 && io_bf) || wait_one(&bar.q_ready, 0, abort));
            tc_fence_after();
            // (a descriptor's address field is in 16-byte units)
            const uint64_t q_desc = desc_kmajor(smem_addr(smem)), k_desc = desc_kmajor(smem_addr(ring)),
                           v_desc = desc_mnmajor(smem_addr(ring), BN * 128);
            auto scores = [&](int j) {
                const int t = two_q ? j >> 1 : j, slot = slot_of(seq_k(two_q, t));
                if (!wait_one(&bar.full[0][t & 3], (t >> 2) & 1, abort)) return false;
                tc_fence_after();
                const uint64_t qd = q_desc + (two_q ? (j & 1) * (S::QTILE / 16) : 0), kd = k_desc + slot * (TILE / 16);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_f16(tm + (j & 1) * BN, qd + (k / 4) * (128 * 128 / 16) + (k % 4) * 2, kd + (k / 4) * (BN * 128 / 16) + (k % 4) * 2, id_s, k > 0);
                umma_commit(&bar.s_full[j & 1]);
                if (!two_q || (j & 1)) umma_commit(&bar.empty[0][t & 3]);
                return true;
            };
            auto outputs = [&](int j) {
                const int t = two_q ? j >> 1 : j, slot = slot_of(seq_v(two_q, t, tiles));
                if (!wait_one(&bar.full[1][t & 3], (t >> 2) & 1, abort)) return false;
                if (!wait_one(&bar.p_full[j & 1], (j >> 1) & 1, abort)) return false;
                tc_fence_after();
                const uint64_t vd = v_desc + slot * (TILE / 16);
                const uint32_t o = tm + S::COL_O + (NS == 2 ? (j & 1) * S::O_STEP : 0), p = tm + S::COL_P + (j & 1) * S::P_STEP;
#pragma unroll
                for (int k = 0; k < BN / 16; ++k) umma_ts(o, p + 8 * k, vd + k * (2048 / 16), id_o, k > 0 || j >= NS);
                if (NS == 1) umma_commit(&bar.pv);
                if (!two_q || (j & 1)) umma_commit(&bar.empty[1][t & 3]);
                return true;
            };
            ok = ok && scores(0);
            if (ok && steps > 1) ok = scores(1);
            for (int j = 0; ok && j < steps; ++j) {
                ok = outputs(j);
                if (ok && j + 2 < steps) ok = scores(j + 2);
            }
            umma_commit(&bar.fin);
            if (!ok) mbar_drain(&bar.fin, 0);
        }
        __syncwarp();
    } else if (!KV8 && warp >= W_TMA) {
        if (S::SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::R_OTHER));
        if (warp == W_TMA + 2 && tiles > 0) {
            // ---- the first tile's values before a window and the last one's past the range, whose copies land on
            // barriers of their own
            auto clear = [&](int t, int r0, int r1) {  // rows r0 .. r1 - 1 of value tile t
                const int slot = slot_of(seq_v(two_q, t, tiles));
                for (int i = lane; i < (r1 - r0) * 8 * S::HALVES; i += 32) {
                    const int r = r0 + i / (8 * S::HALVES), c = i % (8 * S::HALVES);
                    *reinterpret_cast<uint4 *>(ring + slot * TILE + (c / 8) * BN * 128 + r * 128 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
                }
            };
            auto hand_on = [&](int t) {
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.full[1][t & 3]);
            };
            if (head > 0 && tiles > 1 && wait_for(&bar.first_v, 0, abort)) {
                clear(0, 0, head);
                hand_on(0);
            }
            if (wait_for(&bar.last_v, 0, abort)) {
                if (tiles == 1) clear(0, 0, min(head, BN));
                clear(tiles - 1, u.hi - (u.lo + (tiles - 1) * BN), BN);
                hand_on(tiles - 1);
            }
        }
    } else if (KV8 && warp >= W_TMA && warp < W_TMA + 4) {
        if (S::SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::R_OTHER));
        // ---- the tokens' powers of two, up to four tiles ahead: a warp for the keys, one for the values
        const bool is_v = warp == W_TMA + 3;
        int most = 0;  // the values' largest exponent so far
        for (int t = 0; t < tiles; ++t) {
            // exponents of tokens 4 lane .. + 3; bytes past the range or before the window are not of the rows'
            const int j = u.lo + t * BN + 4 * lane, live = u.hi - j, dead = u.see - j;
            unsigned ek = 0, ev = 0;
            if (4 * lane < BN && live > 0) {
                const int pg = pool_page(a.p, u.b, j);
                if (pg >= 0) {
                    const long long at = ((((long long)pg * a.p.heads + u.h)) << a.p.page_shift) + (j & ((1 << a.p.page_shift) - 1));
                    const unsigned mask = (live >= 4 ? 0xffffffffu : (1u << (8 * live)) - 1u) &
                                          (dead <= 0 ? 0xffffffffu : dead >= 4 ? 0u : 0xffffffffu << (8 * dead));
                    ev = __ldg(reinterpret_cast<const unsigned *>(a.ve + at)) & mask;
                    if (!is_v) ek = __ldg(reinterpret_cast<const unsigned *>(a.ke + at)) & mask;
                }
            }
            auto largest = [](unsigned e) {
                const unsigned m = __vmaxu4(e, e >> 16);
                return (int)__reduce_max_sync(0xffffffffu, max(m & 0xffu, (m >> 8) & 0xffu));
            };
            most = max(most, largest(ev));
            const int R = is_v ? most : largest(ek);
            // tile t - 4 is done with: its values multiplied (so its softmax is past), its keys or values turned
            if (t >= 4 && (!wait_for(&bar.empty[1][t & 3], ((t - 4) >> 2) & 1, abort) ||
                           !wait_for(&bar.raw_empty[is_v][t & 3], ((t - 4) >> 2) & 1, abort)))
                break;
            bool tiny = false;
            if (4 * lane < BN) {
                // 2^(E - R + 7) in fp16, twice: subnormal below 2^-14. Below 2^-24 it comes as 2^-24 in the low half and the
                // rest in the high one, with its sign set; from 2^-34 on even 448 times it rounds to 0
                unsigned f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int E = (int)(((is_v ? ev : ek) >> (8 * e)) & 0xffu) - R + TILE_UP;
                    f[e] = E >= -24 ? (E >= -14 ? (unsigned)(15 + E) << 10 : 1u << (24 + E)) * 0x10001u
                                    : E >= -33 ? 0x80000001u | (unsigned)(15 + 24 + E) << 26 : 0u;
                    tiny |= (int)f[e] < 0;
                }
                *reinterpret_cast<uint4 *>(smem + S::OFF_POW + ((is_v * 4 + (t & 3)) * BN + 4 * lane) * 4) = make_uint4(f[0], f[1], f[2], f[3]);
            }
            if (!is_v && lane == 0) {  // the softmax learns both
                bar.k_ref[t & 3] = R;
                bar.v_ref[t & 3] = most;
                mbar_arrive(&bar.ref_full[t & 3]);
            }
            tiny = __any_sync(0xffffffffu, tiny);
            __syncwarp();
            if (lane == 0) {
                bar.tiny[is_v][t & 3] = tiny;
                mbar_arrive(&bar.pow_full[is_v][t & 3]);
            }
        }
    } else if (KV8 && warp >= W_TMA + 4) {
        if (S::SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::R_OTHER));
        // ---- 8-bit tiles to fp16
        const bool is_v = tid - (W_TMA + 4) * 32 >= S::CVT;
        const int c = tid - (W_TMA + 4) * 32 - (is_v ? S::CVT : 0);
        for (int t = 0; t < tiles; ++t) {
            const int seq = is_v ? seq_v(two_q, t, tiles) : seq_k(two_q, t), live = min(BN, u.hi - (u.lo + t * BN)), dead = t == 0 ? head : 0;
            const int slot = slot_of(seq), rs = seq % (KV8 ? S::RAWS : 1);
            if (seq >= slots) {
                int t0;
                bool v0;
                seq_tile(two_q, seq - slots, tiles, t0, v0);
                if (!wait_for(&bar.empty[v0][t0 & 3], (t0 >> 2) & 1, abort)) break;
            }
            if (!wait_for(&bar.pow_full[is_v][t & 3], (t >> 2) & 1, abort)) break;
            if (!wait_for(&bar.raw_full[is_v][t & 3], (t >> 2) & 1, abort)) break;
            const unsigned *mine = reinterpret_cast<const unsigned *>(smem + S::OFF_POW) + (is_v * 4 + (t & 3)) * BN;
            const unsigned char *src = raw + rs * S::RAW;
            unsigned char *dst = ring + slot * TILE;
            constexpr int CHUNKS = BN * D / 16, PER = KV8 ? (CHUNKS + S::CVT - 1) / (KV8 ? S::CVT : 1) : 1, BATCH = 2;
#pragma unroll
            for (int i0 = 0; i0 < PER; i0 += BATCH) {
                uint4 w[BATCH];
                unsigned f[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int x = (i0 + i) * S::CVT + c, r = x / (D / 16);
                    w[i] = make_uint4(0, 0, 0, 0);
                    if (i0 + i < PER && x < CHUNKS) {  // (a warp's 32 chunks at once)
                        f[i] = mine[r];
                        if (r < live && r >= dead) w[i] = *reinterpret_cast<const uint4 *>(src + x * 16);  // rows past the range or before the window are zeros
                    }
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int x = (i0 + i) * S::CVT + c, r = x / (D / 16), e = x % (D / 16) * 16, half = e / 64, ch = e % 64 / 8;
                    if (i0 + i >= PER || x >= CHUNKS) break;
                    auto two = [&](unsigned v) {
                        const unsigned h = unpack_e4m3((unsigned short)v);
                        const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&f[i]));
                        return *reinterpret_cast<const unsigned *>(&y);
                    };
                    uint4 o[2];
                    o[0] = make_uint4(two(w[i].x), two(w[i].x >> 16), two(w[i].y), two(w[i].y >> 16));
                    o[1] = make_uint4(two(w[i].z), two(w[i].z >> 16), two(w[i].w), two(w[i].w >> 16));
                    unsigned char *row = dst + half * BN * 128 + r * 128;
                    const int first = half & 1;  // lanes of neighbouring halves store to different banks
                    *reinterpret_cast<uint4 *>(row + (((ch + first) ^ (r & 7)) << 4)) = first ? o[1] : o[0];
                    *reinterpret_cast<uint4 *>(row + (((ch + 1 - first) ^ (r & 7)) << 4)) = first ? o[0] : o[1];
                }
            }
            if (bar.tiny[is_v][t & 3]) {
                // rows whose power is below 2^-24, again: its high half first, exactly (e4m3 are multiples of 2^-9)
#pragma unroll 1
                for (int x = c; x < CHUNKS; x += KV8 ? S::CVT : 1) {
                    const int r = x / (D / 16), e = x % (D / 16) * 16, half = e / 64, ch = e % 64 / 8;
                    const unsigned f = mine[r], hi = (f >> 16 & 0x7fffu) * 0x10001u, lo = 0x10001u;
                    if ((int)f >= 0 || r >= live || r < dead) continue;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const unsigned h = unpack_e4m3(*reinterpret_cast<const unsigned short *>(src + x * 16 + 2 * i));
                        const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&hi));
                        *reinterpret_cast<__half2 *>(dst + half * BN * 128 + r * 128 + (((ch + i / 4) ^ (r & 7)) << 4) + i % 4 * 4) =
                            __hmul2(y, *reinterpret_cast<const __half2 *>(&lo));
                    }
                }
            }
            fence_proxy_async();
            mbar_arrive(&bar.full[is_v][t & 3]);
            mbar_arrive(&bar.raw_empty[is_v][t & 3]);
        }
    } else {
        // ---- softmax: a thread per row, or (D = 256, one stream) two threads with half of its columns each
        if (S::SPLIT) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::R_SOFTMAX));
        const int s = warp / 4, row = tid % 128;
        const int r_unit = two_q ? s * mq_rows + row : row;  // this thread's row of the unit
        const int tok = (row0 + r_unit) / a.G, pos = u.first + tok;
        // positions of the first and last row of the stream, for whole tiles without a mask
        const int tok_first = (row0 + (two_q ? s * mq_rows : 0)) / a.G, pos_first = u.first + tok_first, pos_last = pos_first + 128 / a.G - 1;
        int q_exp = 0;
        bool ok = true, any = false;
        if (KV8 && io_bf && tiles > 0) {
            // bf16 rows to fp16 by a power of two, in place (which chunk is which does not matter here)
            ok = wait_for(&bar.q_full, 0, abort);
            if (two_q || s == 0) {
                unsigned char *mine = smem + (two_q ? s * S::QTILE : 0) + row * 128;
                constexpr int N = 8;  // chunks held at a time
                float big = 0.f;
                uint4 w[N];
#pragma unroll 1
                for (int x0 = 8 * S::HALVES - N; x0 >= 0; x0 -= N)
#pragma unroll
                    for (int x = 0; x < N; ++x) {
                        w[x] = *reinterpret_cast<const uint4 *>(mine + (x0 + x) / 8 * (128 * 128) + ((x + row) & 7) * 16);
                        const unsigned v[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = unpack2<true>(v[e]);
                            big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
                        }
                    }
                const int e2 = min(max((int)(__float_as_uint(big) >> 23) - 127, -126), 126);
                const float f2 = __int_as_float((127 - e2) << 23);
                bar.q_exp[two_q ? tid : row] = (signed char)e2;
#pragma unroll 1
                for (int x0 = 0; x0 < 8 * S::HALVES; x0 += N)  // (the first ones are still held)
#pragma unroll
                    for (int x = 0; x < N; ++x) {
                        uint4 *at = reinterpret_cast<uint4 *>(mine + (x0 + x) / 8 * (128 * 128) + ((x + row) & 7) * 16);
                        const uint4 y = x0 ? *at : w[x];
                        unsigned v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = unpack2<true>(v[e]);
                            v[e] = pack2<false>(f.x * f2, f.y * f2);
                        }
                        *at = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                fence_proxy_async();
            }
            mbar_arrive(&bar.q_ready);
            bar_sync(1, S::SOFTMAX);
            q_exp = bar.q_exp[two_q ? tid : row];
        }
        const uint32_t lanes = (uint32_t)(32 * (warp % 4)) << 16;
        const uint32_t o_addr = tm + lanes + S::COL_O + (NS == 2 ? s * S::O_STEP : 0);
        float m = -INFINITY, l = 0.f;
        int ref = 0;
        for (int j = NS == 2 ? s : 0; ok && j < steps; j += NS) {
            const int t = two_q ? j >> 1 : j, j0 = u.lo + t * BN;
            const uint32_t s_addr = tm + lanes + (j & 1) * BN + (NS == 1 ? s * CN : 0), p_addr = tm + lanes + S::COL_P + (j & 1) * S::P_STEP + (NS == 1 ? s * CN / 2 : 0);
            float factor = a.scale_log2;
            int ref_now = 0;
            if (KV8) {  // (known up to four tiles ahead of the scores)
                if (!wait_for(&bar.ref_full[t & 3], (t >> 2) & 1, abort)) { ok = false; break; }
                factor = score_factor(a.scale_log2, q_exp + bar.k_ref[t & 3] - 127 - TILE_UP);
                ref_now = bar.v_ref[t & 3];
            }
            if (!wait_for(&bar.s_full[j & 1], (j >> 1) & 1, abort)) { ok = false; break; }
            tc_fence_after();
            constexpr int HELD = S::TWICE ? 2 : CN / 32;  // groups of 32 columns held in registers
            uint32_t x[HELD][32];
#pragma unroll
            for (int i = 0; i < HELD; ++i) tmem_ld32_start(s_addr + 32 * i, x[i]);
            tmem_wait_ld(x);
            // columns least < i <= most are seen, as bits of each 32
            const bool edge = j0 + BN - 1 > pos_first || j0 + BN > u.hi || (a.window && j0 <= pos_last - a.window);
            const int c0 = NS == 1 ? s * CN : 0, most = min(pos, u.hi - 1) - j0 - c0, least = a.window ? pos - a.window - j0 - c0 : -1 - c0;
            auto hide = [&](uint32_t(&y)[32], int i) {
                const int up = most - 32 * i, down = least - 32 * i;
                const unsigned keep = (up >= 31 ? 0xffffffffu : up < 0 ? 0u : (2u << up) - 1u) &
                                      ~(down >= 31 ? 0xffffffffu : down < 0 ? 0u : (2u << down) - 1u);
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = keep & (1u << e) ? y[e] : 0xff800000u;  // -inf
            };
            float b[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i0 = 0; i0 < CN / 32; i0 += HELD) {
                if (i0 > 0) {
#pragma unroll
                    for (int i = 0; i < HELD; ++i) tmem_ld32_start(s_addr + 32 * (i0 + i), x[i]);
                    tmem_wait_ld(x);
                }
                if (edge) {
#pragma unroll
                    for (int i = 0; i < HELD; ++i) hide(x[i], i0 + i);
                }
#pragma unroll
                for (int i = 0; i < HELD * 32; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        b[e] = fmaxf(fmaxf(b[e], __uint_as_float(x[i / 32][i % 32 + 2 * e])), __uint_as_float(x[i / 32][i % 32 + 2 * e + 1]));
            }
            float big = fmaxf(fmaxf(b[0], b[1]), fmaxf(b[2], b[3])) * factor;
            if (NS == 1) {  // with the other half of the row's columns
                row_most[((j & 1) * 2 + s) * 128 + row] = big;
                mbar_arrive(&bar.most_full[j & 1]);
                if (!wait_for(&bar.most_full[j & 1], (j >> 1) & 1, abort)) { ok = false; break; }
                big = fmaxf(big, row_most[((j & 1) * 2 + 1 - s) * 128 + row]);
            }
            if (!any) {
                any = true;
                m = big;
                ref = ref_now;
            } else {
                const bool grew = big > m + 8.f;
                const float base_old = m;
                if (grew) m = big;
                float f = grew ? exp2_fast(base_old - m) : 1.f;
                const bool moved = KV8 && ref_now != ref;
                if (__any_sync(0xffffffffu, grew) || moved) {
                    l *= f;
                    if (moved) f *= exp2_fast((float)(ref - ref_now));
                    ref = ref_now;
                    if (NS == 1) {  // the product of the step before may be under way
                        if (!wait_for(&bar.pv, (j - 1) & 1, abort)) { ok = false; break; }
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int d = NS == 1 ? s * (D / 2) : 0; d < (NS == 1 ? (s + 1) * (D / 2) : D); d += 32) {
                        uint32_t y[1][32];
                        tmem_ld32_start(o_addr + d, y[0]);
                        tmem_wait_ld(y);
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[0][e] = __float_as_uint(__uint_as_float(y[0][e]) * f);
                        tmem_st32(o_addr + d, y[0]);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
            const float2 f2 = make_float2(factor, factor), b2 = make_float2((MB ? 0.f : (float)P_UP) - base, (MB ? 0.f : (float)P_UP) - base);
            float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            if (HELD < CN / 32) {
                uint32_t(&y)[1][32] = reinterpret_cast<uint32_t(&)[1][32]>(x[0]);
                tmem_ld32_start(s_addr, x[0]);
                tmem_wait_ld(y);
                if (edge) hide(x[0], 0);
            }
#pragma unroll
            for (int i = 0; i < CN / 32; ++i) {
                uint32_t p[16], (&now)[32] = x[HELD < CN / 32 ? i & 1 : i], (&next)[32] = x[HELD < CN / 32 ? (i + 1) & 1 : 0];
                if (HELD < CN / 32 && i + 1 < CN / 32) tmem_ld32_start(s_addr + 32 * (i + 1), next);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float2 y = __ffma2_rn(make_float2(__uint_as_float(now[e]), __uint_as_float(now[e + 1])), f2, b2);
                    y = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                    l2[(e >> 1) & 1] = __fadd2_rn(l2[(e >> 1) & 1], y);
                    p[e / 2] = pack2<MB>(y.x, y.y);
                }
                if (HELD < CN / 32 && i + 1 < CN / 32) {
                    tmem_wait_ld(reinterpret_cast<uint32_t(&)[1][32]>(next));
                    if (edge) hide(next, i + 1);
                }
                tmem_st16(p_addr + 16 * i, p);
            }
            l += (l2[0].x + l2[1].x) + (l2[0].y + l2[1].y);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bar.p_full[j & 1]);
        }
        // ---- the outputs
        if (steps > 0 && ok) ok = wait_for(&bar.fin, 0, abort);
        tc_fence_after();
        constexpr float p_down = MB ? 1.f : 1.f / (1 << P_UP);
        const float up = KV8 ? p_down / (1 << TILE_UP) : p_down, unit = KV8 ? exp_byte(ref) : 1.f;  // one after the other: see put_rows
        l *= p_down;
        const AttnUnit v = again(bar.unit[warp]);
        const int first = v.t * a.M, r_here = (NS == 2 && two_q ? s * mq_rows : 0) + row;
        const bool merge = NS == 2 && !two_q, final = v.ranges == 1;
        constexpr int HALF = D / 2, PITCH = HALF + 4;
        // two streams of the same rows: each hands the other half of its columns, and finishes the rest
        unsigned char *mine = smem + S::OFF_RING + 8192;  // (rows on their way out may take the bytes before)
        float *to = reinterpret_cast<float *>(mine) + s * 128 * PITCH, *from = reinterpret_cast<float *>(mine) + (1 - s) * 128 * PITCH;
        float2 *ml = reinterpret_cast<float2 *>(mine + 2 * 128 * PITCH * 4);
        float top = m, f0 = up, f1 = 0.f, sum = l;
        if (NS == 1) {  // the sum of the other half of the columns
            row_sum[s * 128 + row] = l;
            bar_sync(2, 256);
            sum = row_sum[row] + row_sum[128 + row];
        }
        if (merge) {
            ml[s * 128 + row] = make_float2(m, l);
#pragma unroll 1
            for (int d = 0; ok && any && d < HALF; d += 32) {
                uint32_t y[1][32];
                tmem_ld32_start(o_addr + (1 - s) * HALF + d, y[0]);
                tmem_wait_ld(y);
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4 *>(to + row * PITCH + d + e) =
                        make_float4(__uint_as_float(y[0][e]) * up * unit, __uint_as_float(y[0][e + 1]) * up * unit,
                                    __uint_as_float(y[0][e + 2]) * up * unit, __uint_as_float(y[0][e + 3]) * up * unit);
            }
            bar_sync(2, 256);
            const float2 y = ml[(1 - s) * 128 + row];
            top = fmaxf(m, y.x);
            const float base = top == -INFINITY ? 0.f : top;
            f0 = exp2_fast(m - base);
            f1 = exp2_fast(y.x - base);
            sum = s ? f1 * y.y + f0 * l : f0 * l + f1 * y.y;
            f0 *= up;
        }
        if (final) {
            const float inv = sum > 0.f ? 1.f / sum : sum != sum ? sum : 0.f;  // NaN stays NaN
            f0 *= inv;
            f1 *= inv;
        }
        // the row's place in out and lse; a slot's rows are dense
        const bool live = row < mq_rows && r_here < v.n * a.G - first;
        const int token = (first + r_here) / a.G, at = (v.s + token) * (a.p.heads * a.G) + v.h * a.G + (first + r_here - token * a.G);
        float *part = a.part + (v.slot + v.c) * attn_slot(a.M, D);
        if (ok && live && !((merge || NS == 1) && s == 1)) {
            if (!final) *reinterpret_cast<float2 *>(part + (size_t)a.M * D + 2 * r_here) = make_float2(top, sum);
            else if (a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
        }
        const int c0 = merge || NS == 1 ? s * HALF : 0;
        const bool other = merge && (s ? tiles > 0 : tiles > 1);
        if (ok)
            put_rows<D, KV8>(a, smem + warp * S::STAGE, o_addr + c0, c0, NS == 1 || merge ? HALF : D, f0, unit, any, f1, other ? from + row * PITCH : nullptr,
                             final ? nullptr : part, r_here - lane, live ? at : -1, KV8 ? io_bf : BF);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == W_MMA) tmem_free<512>(tm);
}

// [pages][heads * page][D] of a pool: boxes of 64 columns with the 128-byte swizzle (16-bit), or whole
// rows without (8-bit), min(page, BN) rows high.
bool pool_map(CUtensorMap *m, const void *base, const AttnArgs &a, int D, int eb, int rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t page = 1ull << a.p.page_shift;
    const cuuint64_t dims[3] = {(cuuint64_t)D, a.p.heads * page, (cuuint64_t)a.p.pages};
    const cuuint64_t strides[2] = {(cuuint64_t)D * eb, a.p.heads * page * D * eb};
    const cuuint32_t box[3] = {(cuuint32_t)(eb == 1 ? D : 64), (cuuint32_t)rows, 1}, es[3] = {1, 1, 1};
    return enc(m, eb == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base), dims, strides,
               box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, eb == 1 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as [total][heads][D]: boxes of 64 columns, G heads and 128 / G tokens.
bool q_map(CUtensorMap *m, const AttnArgs &a, int D) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.p.heads * a.G, (cuuint64_t)a.p.total};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)(128 / a.G)}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(a.q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF, bool KV8>
dn_status launch_tile(const AttnArgs &a, bool io_bf, unsigned grid, cudaStream_t st) {
    using S = TileShape<D, KV8>;
    const int rows = 1 << a.p.page_shift < S::BN ? 1 << a.p.page_shift : S::BN;
    CUtensorMap mq, mk, mv;
    if (!q_map(&mq, a, D) || !pool_map(&mk, a.kc, a, D, KV8 ? 1 : 2, rows) || !pool_map(&mv, a.vc, a, D, KV8 ? 1 : 2, rows)) return DN_ERR_CUDA;
    cudaFuncSetAttribute(attn_tile_kernel<D, BF, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    launch_pdl(attn_tile_kernel<D, BF, KV8>, dim3(grid), dim3(S::THREADS), S::BYTES, st, a, mq, mk, mv, io_bf);
    return DN_OK;
}

template <int D>
dn_status launch_tile(const AttnArgs &a, bool bf, bool kv8, unsigned grid, cudaStream_t st) {
    if (kv8) return launch_tile<D, false, true>(a, bf, grid, st);
    return bf ? launch_tile<D, true, false>(a, bf, grid, st) : launch_tile<D, false, false>(a, bf, grid, st);
}

}  // namespace

dn_status launch_attn_tc(const AttnArgs &a, int D, bool bf, bool kv8, unsigned grid, cudaStream_t st) {
    if (D == 64) return launch_tile<64>(a, bf, kv8, grid, st);
    if (D == 128) return launch_tile<128>(a, bf, kv8, grid, st);
    return launch_tile<256>(a, bf, kv8, grid, st);
}

}  // namespace dn

extern "C" unsigned int dn_attn_wait_timeouts(void) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, dn::g_attn_timeouts, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return 0xffffffffu;
    }
    return v;
}
