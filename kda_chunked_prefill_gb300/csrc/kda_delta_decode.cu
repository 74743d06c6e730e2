// kda_gated_delta_decode_fwd: the delta rule with one decay per head, token after
// token, state in and out:
//     S <- e^{g_t} S;  d = beta_t (v_t - S^T k_t);  S <- S + k_t d^T;  o_t = scale S^T q_t
//
// A warp owns 16 value columns of one (sequence, head): column j of S, d and o
// depends on column j of the state alone, so no warp waits for another and there
// is no barrier. A lane holds 16 key rows x 4 columns in registers. A token costs one
// reduction: k^T S and q^T S come from the state before the update, and
//     o = scale (e^g q^T S + (q.k) d)
// needs no second pass over it. The eight sums of a lane are reduced over the eight
// lanes that share its columns by halves (4 + 2 + 1 shuffles), which leaves each of
// them with one. Everything is fp32; o is rounded once.
//
// Bound by memory: 64 KB of state read and written per (sequence, head) and
// call. A warp reads 8 rows x 64 bytes per access, 16 accesses in flight. (32 columns a warp, 4 rows x 128 bytes per access and half
// as many warps: 8 % slower.) 256 sequences x 1 token, 16 heads: 82 us, a copy's time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda.h"
#include "kda_common.cuh"
#include "kda_delta.h"
#include "kda_linear.cuh"

namespace kda {
namespace delta {
namespace dec {

using lin::f2;
using lin::fma2;
using lin::mul2;
using lin::pair;
using lin::split;

constexpr int THREADS = 64;
constexpr int PER_SM = 8;  // 128 registers: 16 warps an SM; with the 158 the compiler takes otherwise, 12, and 94 us instead of 82
constexpr int COLS = 16;                                 // value columns of a warp
constexpr int CTA_COLS = COLS * THREADS / 32;
constexpr int PARTS = DV / CTA_COLS;                     // CTAs of a (sequence, head)
constexpr int ROWS = 16;                                 // key rows of a lane
static_assert(ROWS * 8 == DK, "eight lanes share a column");

struct Token {
    uint4 k[2], q[2];  // 16 rows each
    uint2 v;           // 4 columns
    float g, beta;
};

// The sequences that are left out, by one CTA beside the others: 64 bounds a round, about 0.7 us, where the recurrence takes 0.02 us for each
// sequence and head. (Every CTA of the launches behind looking for its own in all bounds: 4096 sequences of 16 tokens, 16 heads 4500 us
// instead of 4040, 20,000 of one token, 2 heads 1460 instead of 780.)
__device__ __noinline__ void list_long(const Params &p) {
    __shared__ int32_t total;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    bool bad = false;
#pragma unroll 1
    for (int64_t n0 = 0; n0 < p.N; n0 += THREADS) {
        const int64_t n = n0 + threadIdx.x;
        int chunks = 0;
        if (n < p.N) {
            const int64_t b = p.cu[n], e = p.cu[n + 1];
            if (b < 0 || e < b || e > p.T || p.cu[0] != 0)
                bad = true;
            else if (e - b > p.longest)
                chunks = static_cast<int>((e - b + CHUNK - 1) / CHUNK);
        }
        const int first = chunks ? atomicAdd(&total, chunks) : 0;
        for (unsigned left = __ballot_sync(0xffffffffu, chunks > 0); left; left &= left - 1) {
            const int l = __ffs(left) - 1, count = __shfl_sync(0xffffffffu, chunks, l), to = __shfl_sync(0xffffffffu, first, l);
            // (bounds that are not in order may hold more chunks than there is room for)
            for (int i = lane; i < count && to >= 0 && to + static_cast<int64_t>(i) < p.most; i += 32)
                p.list[to + i] = make_int2(static_cast<int>(n) - lane + l, i);
        }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) p.listed[0] = total, p.listed[1] = bad;
}

template <bool VARLEN>
__global__ void __launch_bounds__(THREADS, PER_SM) kda_gated_delta_recurrent_kernel(const Params p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t index = blockIdx.x;
    if (VARLEN && p.listed) {
        if (index == 0) {
            list_long(p);
            return;
        }
        --index;
    }
    const int part = index % PARTS;
    const int64_t chain = index / PARTS;  // n * H + h
    const int n = static_cast<int>(chain / p.H), h = static_cast<int>(chain % p.H), hk = h / p.rep;
    const int rg = lane >> 2;                                        // rows 16 rg ..
    const int col = CTA_COLS * part + COLS * warp + 4 * (lane & 3);  // columns col .. col + 3

    int64_t bos, len;
    if (VARLEN) {
        const int64_t b = p.cu[n], e = p.cu[n + 1];
        if (b < 0 || e < b || e > p.T || p.cu[0] != 0) {
            if (threadIdx.x == 0) set_status(p.status, KDA_ERR_BAD_SEQLENS);
            return;
        }
        bos = b;
        len = e - b;
        if (p.longest >= 0 && len > p.longest) return;  // runs in chunks
    } else {
        bos = static_cast<int64_t>(n) * p.steps;
        len = p.steps;
    }

    const size_t sbase = static_cast<size_t>(chain) * (DK * DV) + static_cast<size_t>(ROWS * rg) * DV + col;
    f2 S[ROWS][2];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float4 x = p.s0 ? *reinterpret_cast<const float4 *>(p.s0 + sbase + r * DV) : make_float4(0.f, 0.f, 0.f, 0.f);
        S[r][0] = pair(x.x, x.y);
        S[r][1] = pair(x.z, x.w);
    }
    Token next;
    auto load = [&](int64_t t) {
        const uint4 *k = reinterpret_cast<const uint4 *>(p.k + t * p.ks + hk * DK + ROWS * rg);
        const uint4 *q = reinterpret_cast<const uint4 *>(p.q + t * p.qs + hk * DK + ROWS * rg);
        next.k[0] = k[0], next.k[1] = k[1];
        next.q[0] = q[0], next.q[1] = q[1];
        next.v = *reinterpret_cast<const uint2 *>(p.v + t * p.vs + h * DV + col);
        next.g = p.g[t * p.H + h];
        next.beta = p.beta[t * p.H + h];
    };
    bool gate_bad = false;
    if (len > 0) load(bos);
    for (int64_t t = bos; t < bos + len; ++t) {
        const Token x = next;
        if (t + 1 < bos + len) load(t + 1);
        const uint32_t kw[8] = {x.k[0].x, x.k[0].y, x.k[0].z, x.k[0].w, x.k[1].x, x.k[1].y, x.k[1].z, x.k[1].w};
        const uint32_t qw[8] = {x.q[0].x, x.q[0].y, x.q[0].z, x.q[0].w, x.q[1].x, x.q[1].y, x.q[1].z, x.q[1].w};
        f2 a0 = 0, a1 = 0, o0 = 0, o1 = 0;
        float qk = 0.f;
#pragma unroll
        for (int i = 0; i < ROWS / 2; ++i) {
            const float2 kk = unpack_bf16(kw[i]), qq = unpack_bf16(qw[i]);
            qk = fmaf(qq.x, kk.x, qk);
            qk = fmaf(qq.y, kk.y, qk);
            a0 = fma2(pair(kk.x, kk.x), S[2 * i][0], a0);
            a1 = fma2(pair(kk.x, kk.x), S[2 * i][1], a1);
            o0 = fma2(pair(qq.x, qq.x), S[2 * i][0], o0);
            o1 = fma2(pair(qq.x, qq.x), S[2 * i][1], o1);
            a0 = fma2(pair(kk.y, kk.y), S[2 * i + 1][0], a0);
            a1 = fma2(pair(kk.y, kk.y), S[2 * i + 1][1], a1);
            o0 = fma2(pair(qq.y, qq.y), S[2 * i + 1][0], o0);
            o1 = fma2(pair(qq.y, qq.y), S[2 * i + 1][1], o1);
        }
        // over the eight row groups: lane 16 bit 4 keeps k^T S or q^T S, bits 3 and 2 one of the four columns
        float s[8];
        split(a0, s[0], s[1]);
        split(a1, s[2], s[3]);
        split(o0, s[4], s[5]);
        split(o1, s[6], s[7]);
        const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
        float r4[4], r2[2], r1;
#pragma unroll
        for (int j = 0; j < 4; ++j) r4[j] = (b4 ? s[4 + j] : s[j]) + __shfl_xor_sync(0xffffffffu, b4 ? s[j] : s[4 + j], 16);
#pragma unroll
        for (int j = 0; j < 2; ++j) r2[j] = (b3 ? r4[2 + j] : r4[j]) + __shfl_xor_sync(0xffffffffu, b3 ? r4[j] : r4[2 + j], 8);
        r1 = (b2 ? r2[1] : r2[0]) + __shfl_xor_sync(0xffffffffu, b2 ? r2[0] : r2[1], 4);
#pragma unroll
        for (int m = 4; m <= 16; m <<= 1) qk += __shfl_xor_sync(0xffffffffu, qk, m);

        gate_bad |= !(x.g <= 0.f);
        const float d = expf(x.g);  // 0 for -inf
        const float2 v01 = unpack_bf16(x.v.x), v23 = unpack_bf16(x.v.y);
        const float v[4] = {v01.x, v01.y, v23.x, v23.y};
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = x.beta * fmaf(-d, __shfl_sync(0xffffffffu, r1, 4 * j + (lane & 3)), v[j]);
        const float mine = b3 ? (b2 ? w[3] : w[2]) : (b2 ? w[1] : w[0]);
        if (b4) {
            const float o = p.scale * fmaf(d, r1, qk * mine);
            p.o[(t * p.H + h) * DV + col + (rg & 3)] = __float2bfloat16_rn(o);
        }
        const f2 d2 = pair(d, d), w0 = pair(w[0], w[1]), w1 = pair(w[2], w[3]);
#pragma unroll
        for (int i = 0; i < ROWS / 2; ++i) {
            const float2 kk = unpack_bf16(kw[i]);
            S[2 * i][0] = fma2(pair(kk.x, kk.x), w0, mul2(d2, S[2 * i][0]));
            S[2 * i][1] = fma2(pair(kk.x, kk.x), w1, mul2(d2, S[2 * i][1]));
            S[2 * i + 1][0] = fma2(pair(kk.y, kk.y), w0, mul2(d2, S[2 * i + 1][0]));
            S[2 * i + 1][1] = fma2(pair(kk.y, kk.y), w1, mul2(d2, S[2 * i + 1][1]));
        }
    }
    if (p.sT) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            float4 x;
            split(S[r][0], x.x, x.y);
            split(S[r][1], x.z, x.w);
            *reinterpret_cast<float4 *>(p.sT + sbase + r * DV) = x;
        }
    }
    if (gate_bad && lane == 0) set_status(p.status, KDA_ERR_GATE_RANGE);
}

}  // namespace dec

cudaError_t launch_recurrent(const Params &p, cudaStream_t stream) {
    const int grid = p.N * p.H * dec::PARTS + (p.listed ? 1 : 0);  // the caller has checked that this fits
    if (p.cu)
        dec::kda_gated_delta_recurrent_kernel<true><<<grid, dec::THREADS, 0, stream>>>(p);
    else
        dec::kda_gated_delta_recurrent_kernel<false><<<grid, dec::THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace delta
}  // namespace kda
