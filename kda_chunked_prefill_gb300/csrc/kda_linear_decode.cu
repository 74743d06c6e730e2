// kda_linear_decode_fwd: the recurrence of the linear attention with one decay
// per head, token after token, state in and out:
//     S <- e^{g_t} S + k_t v_t^T ;  o_t = scale S^T q_t
//
// One CTA per (sequence, head, quarter of the value columns), state in
// registers. Unlike the delta rule the update needs no k^T S, so a token costs
// one reduction: every thread updates its 8 key rows x 4 columns (in pairs) and
// adds up q_c S_cv over them, lanes that share columns add by shuffles, the four
// warps through shared memory, four tokens at a time; the next four tokens'
// operands come meanwhile. Everything is fp32; o is rounded once.
//
// Bound by memory: 64 KB of state read and written per (sequence, head) and
// call. A warp reads 4 key rows x 128 bytes per access, 8 accesses in flight.
// 256 sequences x 1 token, 16 heads: 80 us, a copy's time. A further token of the
// same call costs 12 to 14 us (issue: 150 instructions a warp).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda.h"
#include "kda_checks.h"
#include "kda_common.cuh"
#include "kda_linear.cuh"
#include "kda_linear.h"

namespace kda {
namespace lin {
namespace dec {

constexpr int THREADS = 128;
constexpr int PER_SM = 7;  // at most 72 registers: 256 sequences x 8 tokens take 162 us, with 6 or 8 CTAs 172 and 174
constexpr int QUARTERS = 4;
constexpr int COLS = DV / QUARTERS;
constexpr int BATCH = 4;  // tokens staged in shared memory at a time: a warp's outputs each
static_assert(BATCH == THREADS / 32 && COLS == 32, "a lane has a column");

template <bool VARLEN>
__global__ void __launch_bounds__(THREADS, PER_SM) kda_linear_recurrent_kernel(const Params p) {
    __shared__ alignas(16) float sk[BATCH][DK], sq[BATCH][DK], sv[BATCH][COLS];
    __shared__ float sd[BATCH];
    __shared__ alignas(16) float part[BATCH][4][COLS];
    const int quarter = blockIdx.x % QUARTERS;
    const int64_t chain = blockIdx.x / QUARTERS;  // n * H + h
    const int n = static_cast<int>(chain / p.H), h = static_cast<int>(chain % p.H), hk = h / p.rep;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int col = COLS * quarter + 4 * (lane & 7);
    const int row0 = 32 * warp + 8 * (lane >> 3);  // eight rows

    int64_t bos, len;
    if (VARLEN) {
        const int64_t b = p.cu[n], e = p.cu[n + 1];
        if (b < 0 || e < b || e > p.T || p.cu[0] != 0) {
            if (tid == 0) set_status(p.status, KDA_ERR_BAD_SEQLENS);
            return;
        }
        bos = b;
        len = e - b;
        if (p.longest >= 0 && len > p.longest) return;  // runs in chunks
    } else {
        bos = static_cast<int64_t>(n) * p.steps;
        len = p.steps;
    }

    const size_t sbase = static_cast<size_t>(chain) * (DK * DV) + static_cast<size_t>(row0) * DV + col;
    f2 S[8][2];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const float4 x = p.s0 ? *reinterpret_cast<const float4 *>(p.s0 + sbase + r * DV) : make_float4(0.f, 0.f, 0.f, 0.f);
        S[r][0] = pair(x.x, x.y);
        S[r][1] = pair(x.z, x.w);
    }

    __nv_bfloat16 k[BATCH], q[BATCH], v;  // the batch to come: this thread's channel of each token, its column of one token
    float g = 0.f;
    bool gate_bad = false;
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int64_t t = bos + t0 + u;
            if (t0 + u >= len) continue;
            k[u] = p.k[t * p.ks + hk * DK + tid];
            q[u] = p.q[t * p.qs + hk * DK + tid];
            if (warp == u) v = p.v[t * p.vs + h * DV + COLS * quarter + lane];
            if (tid == u) g = p.g[p.g_per_token ? t * p.H + h : h];
        }
    };
    if (len > 0) load(0);
    for (int64_t t0 = 0; t0 < len; t0 += BATCH) {
        const int steps = static_cast<int>(len - t0 < BATCH ? len - t0 : BATCH);
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            if (u >= steps) continue;
            sk[u][tid] = __bfloat162float(k[u]);
            sq[u][tid] = __bfloat162float(q[u]);
            if (warp == u) sv[u][lane] = __bfloat162float(v);
            if (tid == u) {
                gate_bad |= !(g <= 0.f);
                sd[u] = g < G_FLOOR ? 0.f : expf(g);
            }
        }
        __syncthreads();  // (and the last batch's part[] has been read)
        if (t0 + BATCH < len) load(t0 + BATCH);
#pragma unroll 1
        for (int u = 0; u < steps; ++u) {
            const f2 d = pair(sd[u], sd[u]);
            const float4 vv = *reinterpret_cast<const float4 *>(&sv[u][4 * (lane & 7)]);
            const f2 v0 = pair(vv.x, vv.y), v1 = pair(vv.z, vv.w);
            f2 a0 = 0, a1 = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&sk[u][row0 + 4 * i]);
                const float4 q4 = *reinterpret_cast<const float4 *>(&sq[u][row0 + 4 * i]);
                const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f2(&s)[2] = S[4 * i + j];
                    const f2 k2 = pair(kk[j], kk[j]), q2 = pair(qq[j], qq[j]);
                    s[0] = fma2(k2, v0, mul2(d, s[0]));
                    s[1] = fma2(k2, v1, mul2(d, s[1]));
                    a0 = fma2(q2, s[0], a0);
                    a1 = fma2(q2, s[1], a1);
                }
            }
            float4 a;
            split(a0, a.x, a.y);
            split(a1, a.z, a.w);
#pragma unroll
            for (int s = 8; s <= 16; s <<= 1) {
                a.x += __shfl_xor_sync(0xffffffffu, a.x, s);
                a.y += __shfl_xor_sync(0xffffffffu, a.y, s);
                a.z += __shfl_xor_sync(0xffffffffu, a.z, s);
                a.w += __shfl_xor_sync(0xffffffffu, a.w, s);
            }
            if (lane < 8) *reinterpret_cast<float4 *>(&part[u][warp][4 * lane]) = a;
        }
        __syncthreads();  // (and sk, sq, sv and sd have been read)
        if (warp < steps) {  // a token's columns each
            const float o = p.scale * ((part[warp][0][lane] + part[warp][1][lane]) + (part[warp][2][lane] + part[warp][3][lane]));
            p.o[((bos + t0 + warp) * p.H + h) * DV + COLS * quarter + lane] = __float2bfloat16_rn(o);
        }
    }
    if (p.sT) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float4 x;
            split(S[r][0], x.x, x.y);
            split(S[r][1], x.z, x.w);
            *reinterpret_cast<float4 *>(p.sT + sbase + r * DV) = x;
        }
    }
    if (gate_bad) set_status(p.status, KDA_ERR_GATE_RANGE);
}

}  // namespace dec

cudaError_t launch_recurrent(const Params &p, cudaStream_t stream) {
    const int grid = p.N * p.H * dec::QUARTERS;  // the caller has checked that this fits
    if (p.cu)
        dec::kda_linear_recurrent_kernel<true><<<grid, dec::THREADS, 0, stream>>>(p);
    else
        dec::kda_linear_recurrent_kernel<false><<<grid, dec::THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace lin
}  // namespace kda
