// kda_gated_rms_norm: the RMS norm of each head's output row, its gate, and the
// rounding to e4m3 with one scale per row of 128, in one pass.
//
//     n = x / sqrt(mean(x^2) + eps) * w * act(gate);  y_scale = max|n| / 448;  y = e4m3(n / y_scale)
//
// Sum and maximum come from one reduction: with m = x w act(gate), the codes are e4m3(m 448 / max|m|) and the scale is max|m| / sqrt(
// mean(x^2) + eps) / 448, so a row is read once and stays in registers (where max|m| is far from 1, which n need not be, it is read
// again and n formed in the order above). Sixteen lanes take a row, eight channels each (one 16-byte
// access of x, gate and, half as wide, y), a row each: what hides the memory's latency is the number of warps.
//
// Bound by memory: 5 bytes per channel with bf16 x (2 + 2 in, 1 out), 7 with fp32. The sigmoid is the hardware's 2^x and reciprocal (a
// few units in the last place; expf and an IEEE division made the kernel wait for its instructions, 53 an element). 8192 tokens, 16 heads,
// bf16, in turn on six sets of tensors: 16.2 us, 5.2 TB/s of a copy's 6.65 (on one set, partly from L2, 13.5; fp32 20.8 and 17.6), in 6.7
// waves of CTAs that each load, reduce and store once (CTAs of 256 threads were 8 % slower, of 512 13 %).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda.h"
#include "kda_checks.h"
#include "kda_common.cuh"
#include "kda_e4m3.cuh"
#include "kda_linear.cuh"

namespace kda {
namespace gatednorm {

constexpr float TINY = 7.888609052210118e-31f;  // 2^-100: below it a row counts as zero
constexpr float E4M3_MAX = 448.f;
constexpr int THREADS = 128, PER_SM = 16;  // every warp an SM has; two rows a half warp and half the warps: 22 % slower
constexpr int CTA_ROWS = THREADS / 16;

using lin::add2;
using lin::f2;
using lin::fma2;
using lin::mul2;
using lin::of_bf16;
using lin::pair;
using lin::split;

// read once: past the first cache (4 % less time in turn, 11 % of a call)
__device__ __forceinline__ uint4 load_once(const void *p) {
    uint4 u;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
    return u;
}
// eight channels, in pairs
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, f2 (&v)[4]) {
    const uint4 u = load_once(p);
    v[0] = of_bf16(u.x), v[1] = of_bf16(u.y), v[2] = of_bf16(u.z), v[3] = of_bf16(u.w);
}
__device__ __forceinline__ void load8(const float *p, f2 (&v)[4]) {
    const uint4 a = load_once(p), b = load_once(p + 4);
    v[0] = pair(a.x, a.y), v[1] = pair(a.z, a.w), v[2] = pair(b.x, b.y), v[3] = pair(b.z, b.w);
}
__device__ __forceinline__ void load_weight(const float *p, f2 (&v)[4]) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(p)[0], b = reinterpret_cast<const ulonglong2 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}
using kda::max_abs_nan;
__device__ __forceinline__ float max_abs_nan(float m, float x, float y) {  // NaN once any is
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(x)), "f"(fabsf(y)));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <bool SILU>
__device__ __forceinline__ f2 act(f2 gate) {
    float a, b;
    split(mul2(gate, pair(-LOG2E, -LOG2E)), a, b);
    split(add2(pair(ex2(a), ex2(b)), pair(1.f, 1.f)), a, b);  // (2^x infinite: closed)
    const f2 s = pair(rcp(a), rcp(b));
    return SILU ? mul2(s, gate) : s;
}
__device__ __forceinline__ float max_abs_nan(float m, f2 x) {
    float a, b;
    split(x, a, b);
    return max_abs_nan(m, a, b);
}

// STRIDED: the gate's tokens lie gate_stride elements apart; otherwise like x.
template <typename X, bool STRIDED, bool SILU>
__global__ void __launch_bounds__(THREADS, PER_SM)
    kda_gated_rms_norm_kernel(const X *__restrict__ x, const __nv_bfloat16 *__restrict__ gate, int64_t gate_stride,
                              const float *__restrict__ weight, int32_t rows, int32_t heads, float eps, uint8_t *__restrict__ y,
                              float *__restrict__ y_scale) {
    const int c = 8 * (threadIdx.x & 15);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * CTA_ROWS + threadIdx.x / 16;
    f2 v[4] = {}, g[4] = {}, w[4];
    auto load_row = [&] {
        load8(x + row * DV + c, v);
        int64_t at = row * DV;
        if (STRIDED) {
            const uint32_t t = static_cast<uint32_t>(row) / static_cast<uint32_t>(heads);
            at = t * gate_stride + static_cast<int64_t>(static_cast<uint32_t>(row) - t * heads) * DV;
        }
        load8(gate + at + c, g);
    };
    if (row < rows) load_row();
    load_weight(weight + c, w);
    f2 sums = 0;
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        sums = fma2(v[j], v[j], sums);
        v[j] = mul2(v[j], mul2(w[j], act<SILU>(g[j])));
        mx = max_abs_nan(mx, v[j]);
    }
    float sum, half;
    split(sums, sum, half);
    sum += half;
#pragma unroll
    for (int s = 8; s; s >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, s);
        mx = max_abs_nan(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    }
    if (row >= rows) return;  // (a whole half warp)
    const float rstd = rsqrtf(sum * (1.f / DV) + eps);
    float amax = mx * rstd, mul = E4M3_MAX * rcp(mx);
    if (!(mx > 1e-30f && mx < 1e30f)) {  // the products, or a quotient by them, may be out of range where n is not
        load_row();
        load_weight(weight + c, w);
        amax = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = mul2(mul2(mul2(v[j], pair(rstd, rstd)), w[j]), act<SILU>(g[j]));
            amax = max_abs_nan(amax, v[j]);
        }
#pragma unroll
        for (int s = 8; s; s >>= 1) amax = max_abs_nan(amax, __shfl_xor_sync(0xffffu << (threadIdx.x & 16), amax, s));
        mul = E4M3_MAX / amax;
    }
    // A sum that is not finite, by a NaN, an infinity or an overflow, marks the whole row; so does an infinite n.
    const bool good = sum <= 3.402823466e38f && amax <= 3.402823466e38f, tiny = good && amax < TINY;
    if (tiny) mul = 0.f;
    if (!good) mul = __int_as_float(0x7fc00000);
    if (c == 0) y_scale[row] = tiny ? 0.f : good ? amax * (1.f / E4M3_MAX) : mul;
    float q[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) split(mul2(v[j], pair(mul, mul)), q[2 * j], q[2 * j + 1]);
    *reinterpret_cast<uint2 *>(y + row * DV + c) = make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
}

template <typename X>
void launch(const X *x, const __nv_bfloat16 *gate, int64_t gs, const float *w, int rows, int heads, float eps, bool silu,
            uint8_t *y, float *ys, cudaStream_t s) {
    const int grid = (rows - 1) / CTA_ROWS + 1;
    const bool strided = gs != static_cast<int64_t>(heads) * DV;
    auto run = [&](auto kernel) { kernel<<<grid, THREADS, 0, s>>>(x, gate, gs, w, rows, heads, eps, y, ys); };
    if (strided)
        silu ? run(kda_gated_rms_norm_kernel<X, true, true>) : run(kda_gated_rms_norm_kernel<X, true, false>);
    else
        silu ? run(kda_gated_rms_norm_kernel<X, false, true>) : run(kda_gated_rms_norm_kernel<X, false, false>);
}

}  // namespace gatednorm
}  // namespace kda

extern "C" kda_status_t kda_gated_rms_norm(const void *x, const void *gate, int64_t gate_token_stride, const float *weight,
                                           int64_t tokens, int32_t num_heads, int32_t head_dim_v, float eps, int32_t x_fp32,
                                           int32_t silu, void *y, float *y_scale, kda_stream_t stream) {
    using kda::checks::aligned;
    if (head_dim_v != KDA_HEAD_DIM) return KDA_ERR_UNSUPPORTED;
    if (tokens < 0 || num_heads < 1 || (x_fp32 != 0 && x_fp32 != 1) || (silu != 0 && silu != 1)) return KDA_ERR_INVALID_ARG;
    if (tokens > 0x7fffffffLL / num_heads) return KDA_ERR_UNSUPPORTED;
    if (!(eps >= 1e-40f && eps < 3.0e38f)) return KDA_ERR_INVALID_ARG;
    if (gate_token_stride < static_cast<int64_t>(num_heads) * KDA_HEAD_DIM || gate_token_stride % 8) return KDA_ERR_INVALID_ARG;
    if (tokens == 0) return KDA_OK;
    if (gate_token_stride > (int64_t{1} << 40) / tokens) return KDA_ERR_UNSUPPORTED;
    if (!x || !gate || !weight || !y || !y_scale) return KDA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(gate, 16) || !aligned(weight, 16) || !aligned(y, 16) || !aligned(y_scale, 4))
        return KDA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const auto *gb = static_cast<const __nv_bfloat16 *>(gate);
    const int rows = static_cast<int>(tokens * num_heads);
    if (x_fp32)
        kda::gatednorm::launch(static_cast<const float *>(x), gb, gate_token_stride, weight, rows, num_heads, eps, silu != 0,
                               static_cast<uint8_t *>(y), y_scale, s);
    else
        kda::gatednorm::launch(static_cast<const __nv_bfloat16 *>(x), gb, gate_token_stride, weight, rows, num_heads, eps,
                               silu != 0, static_cast<uint8_t *>(y), y_scale, s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
