// dn_head_norm, dn_residual_norm: the norms, gates and residual additions between a step's large calls.
//
// Both read every input once and write every output once, with the sums of squares and all arithmetic in 32 bits
// and one rounding at each store, so memory bounds large calls and the launch bounds small ones.
// Measured on a GB300: 25,000 x 48 heads of 128 in fp16 136 us, 6.77 TB/s, the copy rate; 25,000 rows of 2,560 in bf16 with
// a 32-bit residual, own norm and gate 128 us, 7.0 TB/s.
//
// dn_head_norm: a head's row of D elements lies on D / 8 lanes of one warp (8 elements a lane), and its sum of squares is
// a shuffle among them; nothing is shared between warps. Small calls have one piece of 256 elements a warp, large ones four (two in
// fp32) with their loads in flight together: eight CTAs of 128 threads an SM measured best (136 us; seven 141; other
// numbers of pieces 143 to 166).
//
// dn_residual_norm: a row of C elements stays in the registers of one warp (C <= 512) or one CTA between the reads and
// the writes. The sums of squares of the block's output and of the new residual are two reductions, the second over
// what the first has scaled: taking both from one pass over products would cancel where the new residual is small.
#include <cuda_runtime.h>

#include "dn.h"
#include "dn_device.cuh"
#include "dn_internal.h"
#include "dn_vec.cuh"

namespace dn {
namespace {

// act(z) of 8 values. 1 / (1 + e^-z) is taken from e^-|z|, which cannot overflow; fp32 tensors get the accurate exponential.
template <typename T> __device__ __forceinline__ void activate(int act, float (&z)[8]) {
    if (act == DN_ACT_NONE) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float e = sizeof(T) == 4 ? expf(-fabsf(z[i])) : __expf(-fabsf(z[i]));
        const float y = __fdividef(z[i] < 0.f ? e : 1.f, 1.f + e);
        z[i] = act == DN_ACT_SILU ? z[i] * y : y;
    }
}

__device__ __forceinline__ float sum_squares(const float (&x)[8]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
    return s;
}

__device__ __forceinline__ void times(float (&v)[8], const float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 p = __fmul2_rn(make_float2(v[i], v[i + 1]), make_float2(w[i], w[i + 1]));
        v[i] = p.x;
        v[i + 1] = p.y;
    }
}

constexpr int kHeadWarps = 4;

// PASSES 256-element pieces of the packed heads a warp, all of their loads in flight at once.
template <typename T, int PASSES>
__global__ void __launch_bounds__(32 * kHeadWarps, 8)
head_norm_kernel(unsigned groups, unsigned groups_row, int lanes_row, int order, int act, const T *x, long long x_stride,
                 const T *__restrict__ gate, long long gate_stride, const T *__restrict__ weight, float inv_d, float eps,
                 T *out) {
    const int lane = threadIdx.x % 32;
    const unsigned first = (blockIdx.x * kHeadWarps + threadIdx.x / 32) * (PASSES * 32u) + lane;
    grid_dep_wait();
    grid_dep_trigger();
    Vec8<T> rx[PASSES], rg[PASSES];
    unsigned row = first / groups_row, at = first - row * groups_row;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        rx[i] = rg[i] = Vec8<T>{};
        if (first + i * 32 < groups) {
            rx[i] = load_vec(x + (long long)row * x_stride + at * 8ll);
            if (gate) rg[i] = load_vec(gate + (long long)row * gate_stride + at * 8ll);
        }
        at += 32;
        const unsigned rows = groups_row >= 32 ? at >= groups_row : at / groups_row;
        row += rows;
        at -= rows * groups_row;
    }
    float w[8];
    if (weight) {
        to_floats(load_vec(weight + (lane & (lanes_row - 1)) * 8), w);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const unsigned j = first + i * 32;
        float v[8], z[8];
        to_floats(rx[i], v);
        if (gate) {
            to_floats(rg[i], z);
            activate<T>(act, z);
        }
        if (gate && order != DN_NORM_GATE) times(v, z);
        if (order != DN_GATE) {
            float s = sum_squares(v);
            for (int off = lanes_row / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            const float f = rsqrtf(fmaf(s, inv_d, eps));
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= f;
            if (weight) times(v, w);
            if (gate && order == DN_NORM_GATE) times(v, z);
        }
        if (j < groups) store_vec(out + j * 8ll, v);
    }
}

// Sum over a row's threads; every thread gets it. `red` is written before the one barrier and read after it, so two
// sums in a row need two arrays.
template <bool WARP> __device__ __forceinline__ float row_sum(float s, float *red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (WARP) return s;
    const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (lane == 0) red[threadIdx.x / 32] = s;
    __syncthreads();
    s = lane < warps ? red[lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
}

// One row a warp (WARP: blockDim = (32, rows)) or a CTA; PER groups of 8 elements a thread.
template <typename T, typename R, int PER, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024)
residual_norm_kernel(int rows, int groups, int act, const T *__restrict__ y, long long y_stride, const T *__restrict__ gate,
                     long long gate_stride, const T *__restrict__ after, float scale, const R *residual, R *residual_out,
                     const T *__restrict__ weight, float inv_c, float eps, T *__restrict__ out) {
    __shared__ float red[2][32];
    const long long row = WARP ? (long long)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    const int step = WARP ? 32 : blockDim.x;
    grid_dep_wait();
    grid_dep_trigger();
    if (WARP && row >= rows) return;
    Vec8<T> ry[PER], rg[PER];
    Vec8<R> rr[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int j = threadIdx.x + i * step;
        ry[i] = rg[i] = Vec8<T>{};
        rr[i] = Vec8<R>{};
        if (j < groups) {
            rr[i] = load_vec(residual + (row * groups + j) * 8);
            if (y) ry[i] = load_vec(y + row * y_stride + j * 8);
            if (gate) rg[i] = load_vec(gate + row * gate_stride + j * 8);
        }
    }
    float f = scale;
    if (after) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            float v[8];
            to_floats(ry[i], v);
            s += sum_squares(v);
        }
        f = rsqrtf(fmaf(row_sum<WARP>(s, red[0]), inv_c, eps));
    }
    float v[PER][8], s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int j = threadIdx.x + i * step;
        to_floats(rr[i], v[i]);
        if (y) {
            float a[8], b[8];
            to_floats(ry[i], a);
            if (after) {
                to_floats(j < groups ? load_vec(after + j * 8) : Vec8<T>{}, b);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] *= f * b[e];
            }
            if (gate) {
                to_floats(rg[i], b);
                activate<T>(act, b);
                times(a, b);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = fmaf(scale, a[e], v[i][e]);
            if (j < groups) store_vec(residual_out + (row * groups + j) * 8, v[i]);
        }
        s += sum_squares(v[i]);
    }
    f = rsqrtf(fmaf(row_sum<WARP>(s, red[1]), inv_c, eps));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int j = threadIdx.x + i * step;
        if (j >= groups) continue;
        if (weight) {
            float w[8];
            to_floats(load_vec(weight + j * 8), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] *= f * w[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] *= f;
        }
        store_vec(out + (row * groups + j) * 8, v[i]);
    }
}

inline bool io_dtype_known(dn_dtype t) { return t >= DN_F16 && t <= DN_E4M3; }
inline bool act_known(int act) { return act == DN_ACT_NONE || act == DN_ACT_SIGMOID || act == DN_ACT_SILU; }

struct HeadArgs {
    unsigned groups, groups_row;
    int lanes_row, order, act;
    const void *x, *gate, *weight;
    long long x_stride, gate_stride;
    float eps, inv_d;
    void *out;
    cudaStream_t st;
};

template <typename T> void launch_head(const HeadArgs &a) {
    auto go = [&](auto passes) {
        constexpr int P = decltype(passes)::value;
        const unsigned blocks = (unsigned)((a.groups + (unsigned long long)(P * 32 * kHeadWarps) - 1) / (P * 32 * kHeadWarps));
        launch_pdl(head_norm_kernel<T, P>, dim3(blocks), dim3(32 * kHeadWarps), 0, a.st, a.groups, a.groups_row, a.lanes_row,
                   a.order, a.act, static_cast<const T *>(a.x), a.x_stride, static_cast<const T *>(a.gate), a.gate_stride,
                   static_cast<const T *>(a.weight), a.inv_d, a.eps, static_cast<T *>(a.out));
    };
    // one piece a warp against four (16 bits): 680 rows of 48 heads of 128 (2^19 groups) 5.4 against 5.6 us, 1,020 rows 7.4 against 7.0, 2,000 rows 13.6
    // against 11.8; against two (fp32): 170 rows 2.95 against 3.00, 680 rows 6.3 and 6.3, 1,020 rows 8.8 against 8.5, 2,000 rows 22.0 against 21.6
    if (a.groups <= 1u << 19) go(std::integral_constant<int, 1>{});
    else go(std::integral_constant<int, sizeof(T) == 4 ? 2 : 4>{});
}

struct ResidualArgs {
    int rows, groups, act;
    const void *y, *gate, *after, *residual, *weight;
    long long y_stride, gate_stride;
    float scale, inv_c, eps;
    void *residual_out, *out;
    cudaStream_t st;
};

template <typename T, typename R> void launch_residual(const ResidualArgs &a) {
    auto go = [&](auto per, auto warp) {
        constexpr int P = decltype(per)::value;
        constexpr bool W = decltype(warp)::value;
        const dim3 block = W ? dim3(32, 4) : dim3((unsigned)((a.groups + 32 * P - 1) / (32 * P) * 32));
        const unsigned blocks = W ? (unsigned)(((long long)a.rows + 3) / 4) : (unsigned)a.rows;
        launch_pdl(residual_norm_kernel<T, R, P, W>, dim3(blocks), block, 0, a.st, a.rows, a.groups, a.act,
                   static_cast<const T *>(a.y), a.y_stride, static_cast<const T *>(a.gate), a.gate_stride,
                   static_cast<const T *>(a.after), a.scale, static_cast<const R *>(a.residual), static_cast<R *>(a.residual_out),
                   static_cast<const T *>(a.weight), a.inv_c, a.eps, static_cast<T *>(a.out));
    };
    using Y = std::true_type;
    using N = std::false_type;
    // 16 rows and many, us, in bf16. A warp a row against a CTA: C = 512 1.9 and 24.7 (40,000 rows) against 1.9 and 41; C = 1,024 2.6 and 48.5
    // against 1.8 and 48.0. One group a thread against two: C = 5,120 2.1 and 73.4 (12,000 rows) against 2.3 and 73.1; C = 8,192 2.4
    // and 81.1 (8,000 rows) against 2.6 and 79.2.
    if (a.groups <= 32) go(std::integral_constant<int, 1>{}, Y{});
    else if (a.groups <= 64) go(std::integral_constant<int, 2>{}, Y{});
    else if (a.groups <= 640) go(std::integral_constant<int, 1>{}, N{});
    else go(std::integral_constant<int, 2>{}, N{});
}

constexpr int kMaxWidth = 2 * 1024 * 8;  // residual_norm's elements a row: two groups of 8 for each of 1,024 threads

}  // namespace
}  // namespace dn

extern "C" dn_status dn_head_norm(int rows, int heads, int D, dn_dtype io_dt, dn_norm_order order, dn_act act, const void *x,
                                  int64_t x_stride, const void *gate, int64_t gate_stride, const void *weight, float eps,
                                  void *out, dn_stream_t stream) {
    using namespace dn;
    if (rows < 0 || heads < 1 || !io_dtype_known(io_dt) || !act_known(act) || !(eps > 0.f) || !(eps < 3e38f)) return DN_ERR_INVALID_ARG;
    if (order != DN_NORM_GATE && order != DN_GATE_NORM && order != DN_GATE) return DN_ERR_INVALID_ARG;
    if ((D != 64 && D != 128 && D != 256) || io_dt == DN_E4M3) return DN_ERR_UNSUPPORTED;
    const int64_t wide = (int64_t)heads * D;
    const int64_t vec = io_dt == DN_F32 ? 4 : 8;
    if (wide > (1 << 24) || (int64_t)rows * (wide / 8) > 0x7fffffffLL) return DN_ERR_INVALID_ARG;
    if (x_stride < wide || x_stride % vec || (gate && (gate_stride < wide || gate_stride % vec))) return DN_ERR_INVALID_ARG;
    if (order != DN_NORM_GATE && !gate) return DN_ERR_INVALID_ARG;
    if (order == DN_GATE && weight) return DN_ERR_INVALID_ARG;
    if (rows == 0) return DN_OK;
    if (!x || !out || !aligned(x, 16) || !aligned(out, 16) || !aligned(gate, 16) || !aligned(weight, 16)) return DN_ERR_INVALID_ARG;
    const HeadArgs a = {(unsigned)(rows * (wide / 8)), (unsigned)(wide / 8), D / 8, order, act, x, gate, weight, x_stride, gate_stride, eps,
                        1.f / D, out, reinterpret_cast<cudaStream_t>(stream)};
    if (io_dt == DN_F16) launch_head<__half>(a);
    else if (io_dt == DN_BF16) launch_head<__nv_bfloat16>(a);
    else launch_head<float>(a);
    return launch_status();
}

extern "C" dn_status dn_residual_norm(int rows, int C, dn_dtype io_dt, dn_dtype res_dt, dn_act act, const void *y, int64_t y_stride,
                                      const void *gate, int64_t gate_stride, const void *after_weight, float scale,
                                      const void *residual, void *residual_out, const void *weight, float eps, void *out,
                                      dn_stream_t stream) {
    using namespace dn;
    if (rows < 0 || C < 1 || !io_dtype_known(io_dt) || !io_dtype_known(res_dt) || !act_known(act)) return DN_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !(eps < 3e38f) || !(scale > -3e38f) || !(scale < 3e38f)) return DN_ERR_INVALID_ARG;
    if (io_dt == DN_E4M3 || (res_dt != io_dt && res_dt != DN_F32) || C % 8 || C > kMaxWidth) return DN_ERR_UNSUPPORTED;
    const int64_t vec = io_dt == DN_F32 ? 4 : 8;
    if (!y && (gate || after_weight)) return DN_ERR_INVALID_ARG;
    if ((y && (y_stride < C || y_stride % vec)) || (gate && (gate_stride < C || gate_stride % vec))) return DN_ERR_INVALID_ARG;
    if (rows == 0) return DN_OK;
    if (!residual || !out || (y && !residual_out)) return DN_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(gate, 16) || !aligned(after_weight, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) ||
        !aligned(weight, 16) || !aligned(out, 16))
        return DN_ERR_INVALID_ARG;
    const ResidualArgs a = {rows, C / 8, act, y, gate, after_weight, residual, weight, y_stride, gate_stride, scale, 1.f / C, eps, residual_out,
                            out, reinterpret_cast<cudaStream_t>(stream)};
    const bool wide = res_dt == DN_F32;
    if (io_dt == DN_F32) launch_residual<float, float>(a);
    else if (io_dt == DN_F16 && wide) launch_residual<__half, float>(a);
    else if (io_dt == DN_F16) launch_residual<__half, __half>(a);
    else if (wide) launch_residual<__nv_bfloat16, float>(a);
    else launch_residual<__nv_bfloat16, __nv_bfloat16>(a);
    return launch_status();
}
