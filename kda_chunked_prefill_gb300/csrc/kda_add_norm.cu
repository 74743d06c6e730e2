// kda_add_rms_norm: the residual's addition, the RMS norm and the rounding to
// e4m3 with one scale per row, in one pass over the row.
//
//     h = x + r;  n = h / sqrt(mean(h^2) + eps) * w;  y_scale = max|n| / 448;  y = e4m3(n / y_scale)
//
// Sum and maximum come from one reduction: max|n| = max|h w| / sqrt(mean(h^2) +
// eps), so a row is read once, kept in registers, reduced once and written once.
// Bound by memory: 7 bytes per element (2 + 2 in, 2 + 1 out; 11 with an fp32
// residual).
//
// 8192 rows of 2048 (calls replayed from a graph): with a bf16 residual 20.5 us, 5.7 TB/s (86 % of a copy); with an fp32 residual
// 30.8 us, 6.0 TB/s (90 %).
//
// Rows are cut at multiples of 8 elements of the whole tensor, not of the row:
// with 16-byte-aligned tensors every such group is one aligned access of x, r, r'
// and y whatever the width; a group that two rows share is handled element by
// element at both ends.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda.h"
#include "kda_checks.h"
#include "kda_common.cuh"

namespace kda {
namespace addnorm {

constexpr float TINY = 7.888609052210118e-31f;  // 2^-100: below it a row counts as zero
constexpr float E4M3_MAX = 448.f;
constexpr int NARROW = 4;  // rows of a CTA where a warp takes one

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;  // saturating, round to nearest even; NaN stays NaN
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ void load_weight(const float *p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store_res(__nv_bfloat16 *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store_res(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <typename R>
struct Raw {  // eight elements as they lie in memory
    uint4 u[sizeof(R) / 2];
};
template <typename R>
__device__ __forceinline__ void load_raw(Raw<R> &r, const R *p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(R) / 2); ++i) r.u[i] = reinterpret_cast<const uint4 *>(p)[i];
}
__device__ __forceinline__ void add_raw(float (&v)[8], const Raw<__nv_bfloat16> &r) {
    const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16(w[i]);
        v[2 * i] += f.x;
        v[2 * i + 1] += f.y;
    }
}
__device__ __forceinline__ void add_raw(float (&v)[8], const Raw<float> &r) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[4 * i] += __uint_as_float(r.u[i].x);
        v[4 * i + 1] += __uint_as_float(r.u[i].y);
        v[4 * i + 2] += __uint_as_float(r.u[i].z);
        v[4 * i + 3] += __uint_as_float(r.u[i].w);
    }
}
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }

// THREADS threads per row, a warp or whole CTAs; a thread holds NV groups of 8 elements.
// ALIGNED: width is a multiple of 8 (no shared groups, weight loads are vectors).
template <typename R, int THREADS, int NV, bool ALIGNED>
__global__ void __launch_bounds__(THREADS == 32 ? 32 * NARROW : THREADS)
    kda_add_rms_norm_kernel(const __nv_bfloat16 *__restrict__ x, const R *res, const float *__restrict__ weight, int32_t rows,
                            int32_t width, float eps, R *res_out, uint8_t *__restrict__ y, float *__restrict__ y_scale) {
    constexpr int WARPS = THREADS / 32;
    __shared__ float s_sum[WARPS], s_max[WARPS];
    const int tid = threadIdx.x % THREADS;
    const int64_t row = THREADS == 32 ? static_cast<int64_t>(blockIdx.x) * NARROW + threadIdx.x / 32 : blockIdx.x;
    if (row >= rows) return;
    const int64_t f0 = row * width, f1 = f0 + width;
    const int64_t v0 = f0 >> 3;
    float h[NV][8];
    float sum = 0.f, mx = 0.f;
    // All loads before the first store, where the registers hold them: the residual may be updated in place, and no load moves
    // past a store by itself.
    constexpr bool AHEAD = THREADS <= 512;
    Raw<__nv_bfloat16> xr[NV];
    Raw<R> rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t f = (v0 + tid + i * THREADS) << 3;
        if (AHEAD && f + 8 <= f1 && (ALIGNED || f >= f0)) {
            load_raw(xr[i], x + f);
            load_raw(rr[i], res + f);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t f = (v0 + tid + i * THREADS) << 3;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
        if (f >= f1) continue;
        if (ALIGNED || (f >= f0 && f + 8 <= f1)) {
            if (!AHEAD) {
                load_raw(xr[i], x + f);
                load_raw(rr[i], res + f);
            }
            add_raw(h[i], xr[i]);
            add_raw(h[i], rr[i]);
            store_res(res_out + f, h[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = f + j >= f0 && f + j < f1;
                h[i][j] = in ? as_float(x[f + j]) + as_float(res[f + j]) : 0.f;
                if (in) put(res_out + f + j, h[i][j]);
            }
        }
    }
    // h becomes h * w
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t f = (v0 + tid + i * THREADS) << 3;
        if (f >= f1) continue;
        float w[8];
        if (ALIGNED) {
            load_weight(weight + (f - f0), w);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = (f + j >= f0 && f + j < f1) ? __ldg(weight + (f + j - f0)) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum = fmaf(h[i][j], h[i][j], sum);
            h[i][j] *= w[j];
            mx = max_abs_nan(mx, h[i][j]);
        }
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, s);
        mx = max_abs_nan(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    }
    if (WARPS > 1) {
        if ((tid & 31) == 0) {
            s_sum[tid >> 5] = sum;
            s_max[tid >> 5] = mx;
        }
        __syncthreads();
        sum = 0.f;
        mx = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            sum += s_sum[i];
            mx = max_abs_nan(mx, s_max[i]);
        }
    }
    // (a sum that is not finite, by a NaN, an infinity or an overflow, marks the whole row)
    const float rstd = sum <= 3.402823466e38f ? 1.f / sqrtf(sum / static_cast<float>(width) + eps) : __int_as_float(0x7fc00000);
    const float amax = max_abs_nan(0.f, mx * rstd);  // max|n|; NaN once anything in the row is not finite
    const bool tiny = amax < TINY;
    float mul = tiny ? 0.f : rstd * (E4M3_MAX / amax);
    if (mul > 3.402823466e38f) {  // small elements and a small eps: in two factors
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] *= rstd;
        mul = E4M3_MAX / amax;
    }
    if (tid == 0) y_scale[row] = tiny ? 0.f : amax / E4M3_MAX;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t f = (v0 + tid + i * THREADS) << 3;
        if (f >= f1) continue;
        const uint32_t a = e4m3x4(h[i][0] * mul, h[i][1] * mul, h[i][2] * mul, h[i][3] * mul);
        const uint32_t b = e4m3x4(h[i][4] * mul, h[i][5] * mul, h[i][6] * mul, h[i][7] * mul);
        if (ALIGNED || (f >= f0 && f + 8 <= f1)) {
            *reinterpret_cast<uint2 *>(y + f) = make_uint2(a, b);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (f + j >= f0 && f + j < f1) y[f + j] = static_cast<uint8_t>((j < 4 ? a : b) >> (8 * (j & 3)));
        }
    }
}

template <typename R, int THREADS, int NV>
void launch_width(bool al, const __nv_bfloat16 *x, const R *res, const float *w, int rows, int width, float eps,
                  R *res_out, uint8_t *y, float *ys, cudaStream_t s) {
    constexpr int PER_CTA = THREADS == 32 ? NARROW : 1;
    const int grid = (rows - 1) / PER_CTA + 1;
    if (al)
        kda_add_rms_norm_kernel<R, THREADS, NV, true><<<grid, THREADS * PER_CTA, 0, s>>>(x, res, w, rows, width, eps, res_out, y, ys);
    else
        kda_add_rms_norm_kernel<R, THREADS, NV, false><<<grid, THREADS * PER_CTA, 0, s>>>(x, res, w, rows, width, eps, res_out, y, ys);
}
template <typename R>
void launch(const __nv_bfloat16 *x, const R *res, const float *w, int rows, int width, float eps, R *res_out,
            uint8_t *y, float *ys, cudaStream_t s) {
    const bool al = width % 8 == 0;
    const int groups = al ? width / 8 : width / 8 + 2;  // groups a row may touch
    // Two groups a thread or three, as far as that is a warp to 512 threads a row. Measured with 8192 rows of 2048 (bf16 residual): 20.5
    // us, with one group 22.4 and four 23.8; 2048 rows of 12288: three groups 31.5, two (1024 threads) 45.1, six 38.7.
    if (groups <= 32)
        launch_width<R, 32, 1>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
    else if (groups <= 64)
        launch_width<R, 32, 2>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
    else if (groups <= 128)
        launch_width<R, 64, 2>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
    else if (groups <= 256)
        launch_width<R, 128, 2>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
    else if (groups <= 384)
        launch_width<R, 128, 3>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
    else if (groups <= 512)
        launch_width<R, 256, 2>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
    else if (groups <= 768)
        launch_width<R, 256, 3>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
    else if (groups <= 1024)
        launch_width<R, 512, 2>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
    else if (groups <= 1536)
        launch_width<R, 512, 3>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
    else if (groups <= 2048)
        launch_width<R, 512, 4>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
    else
        launch_width<R, 1024, 5>(al, x, res, w, rows, width, eps, res_out, y, ys, s);
}

}  // namespace addnorm
}  // namespace kda

extern "C" kda_status_t kda_add_rms_norm(const void *x, const void *residual, const float *weight, int64_t rows,
                                         int32_t width, float eps, int32_t residual_fp32, void *residual_out, void *y,
                                         float *y_scale, kda_stream_t stream) {
    using kda::checks::aligned;
    if (rows < 0 || rows > 0x7fffffffLL || width < 1) return KDA_ERR_INVALID_ARG;
    if (width > KDA_NORM_MAX_WIDTH) return KDA_ERR_UNSUPPORTED;
    if (!(eps > 0.f && eps < 3.0e38f) || (residual_fp32 != 0 && residual_fp32 != 1)) return KDA_ERR_INVALID_ARG;
    if (rows == 0) return KDA_OK;
    if (!x || !residual || !weight || !residual_out || !y || !y_scale) return KDA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
        !aligned(y, 16) || !aligned(y_scale, 4))
        return KDA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const auto *xb = static_cast<const __nv_bfloat16 *>(x);
    auto *y8 = static_cast<uint8_t *>(y);
    const int n = static_cast<int>(rows);
    if (residual_fp32)
        kda::addnorm::launch<float>(xb, static_cast<const float *>(residual), weight, n, width, eps,
                                    static_cast<float *>(residual_out), y8, y_scale, s);
    else
        kda::addnorm::launch<__nv_bfloat16>(xb, static_cast<const __nv_bfloat16 *>(residual), weight, n, width, eps,
                                            static_cast<__nv_bfloat16 *>(residual_out), y8, y_scale, s);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
