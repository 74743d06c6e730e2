// kda_gated_rms_norm: the RMS norm of each head's output row, its gate, and the
// rounding to e4m3 with one scale per row of 128, in one pass.
//
//     n = x / sqrt(mean(x^2) + eps) * w * act(gate);  y_scale = max|n| / 448;  y = e4m3(n / y_scale)
//
// Sum and maximum come from one reduction: with m = x w act(gate), the codes are e4m3(m 448 / max|m|) and the scale is max|m| / sqrt(
// mean(x^2) + eps) / 448, so a row is read once and stays in registers. Sixteen lanes take a row, eight channels each (one 16-byte
// access of x, gate and, half as wide, y); the weight's eight values stay in registers for the two rows that a half warp takes.
//
// Bound by memory: 5 bytes per channel with bf16 x (2 + 2 in, 1 out), 7 with fp32. The sigmoid is the hardware's 2^x and reciprocal (a
// few units in the last place; expf and an IEEE division made the kernel wait for its instructions, 53 an element).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda.h"
#include "kda_checks.h"
#include "kda_common.cuh"

namespace kda {
namespace gatednorm {

constexpr float TINY = 7.888609052210118e-31f;  // 2^-100: below it a row counts as zero
constexpr float E4M3_MAX = 448.f;
constexpr int THREADS = 256;
constexpr int ROWS = 2;                              // of a half warp
constexpr int CTA_ROWS = THREADS / 16 * ROWS;

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;  // saturating, round to nearest even; NaN stays NaN
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// STRIDED: the gate's tokens lie gate_stride elements apart; otherwise like x.
template <typename X, bool STRIDED, bool SILU>
__global__ void __launch_bounds__(THREADS)
    kda_gated_rms_norm_kernel(const X *__restrict__ x, const __nv_bfloat16 *__restrict__ gate, int64_t gate_stride,
                              const float *__restrict__ weight, int32_t rows, int32_t heads, float eps, uint8_t *__restrict__ y,
                              float *__restrict__ y_scale) {
    const int c = 8 * (threadIdx.x & 15);
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * CTA_ROWS + threadIdx.x / 16;
    float w[8], v[ROWS][8], g[ROWS][8];
    load8(weight + c, w);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t row = row0 + i * (THREADS / 16);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = g[i][j] = 0.f;
        if (row >= rows) continue;
        load8(x + row * DV + c, v[i]);
        int64_t at = row * DV;
        if (STRIDED) {
            const uint32_t t = static_cast<uint32_t>(row) / static_cast<uint32_t>(heads);
            at = t * gate_stride + static_cast<int64_t>(static_cast<uint32_t>(row) - t * heads) * DV;
        }
        load8(gate + at + c, g[i]);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t row = row0 + i * (THREADS / 16);
        float sum = 0.f, mx = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum = fmaf(v[i][j], v[i][j], sum);
            const float sig = rcp(1.f + ex2(g[i][j] * -LOG2E));  // (2^x infinite: closed)
            v[i][j] *= w[j] * (SILU ? g[i][j] * sig : sig);
            mx = max_abs_nan(mx, v[i][j]);
        }
#pragma unroll
        for (int s = 8; s; s >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, s);
            mx = max_abs_nan(mx, __shfl_xor_sync(0xffffffffu, mx, s));
        }
        if (row >= rows) continue;  // (a whole half warp)
        // A sum that is not finite, by a NaN, an infinity or an overflow, marks the whole row; so does an infinite product.
        const bool fine = sum <= 3.402823466e38f && mx <= 3.402823466e38f;
        const float rstd = rsqrtf(sum * (1.f / DV) + eps), amax = fine ? mx * rstd : __int_as_float(0x7fc00000);
        const bool good = amax <= 3.402823466e38f, tiny = amax < TINY;
        float mul = E4M3_MAX * rcp(mx);
        if (!(mx > 1e-30f && mx < 1e30f)) {  // where the quotient, or its reciprocal, is out of range: in two factors
            const float first = mx < 1.f ? 0x1p80f : 0x1p-80f;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= first;
            mul = E4M3_MAX / (mx * first);
        }
        if (tiny) mul = 0.f;
        if (!good) mul = __int_as_float(0x7fc00000);
        if (c == 0) y_scale[row] = tiny ? 0.f : good ? amax * (1.f / E4M3_MAX) : mul;
        const uint32_t a = e4m3x4(v[i][0] * mul, v[i][1] * mul, v[i][2] * mul, v[i][3] * mul);
        const uint32_t b = e4m3x4(v[i][4] * mul, v[i][5] * mul, v[i][6] * mul, v[i][7] * mul);
        *reinterpret_cast<uint2 *>(y + row * DV + c) = make_uint2(a, b);
    }
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
    if (!(eps > 0.f && eps < 3.0e38f)) return KDA_ERR_INVALID_ARG;
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
