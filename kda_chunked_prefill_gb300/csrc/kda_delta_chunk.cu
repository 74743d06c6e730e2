// Chunked form of the delta rule with one decay per head (kda_gated_delta_chunk_fwd) on tcgen05.
//
// For a chunk of 64 tokens with G_i the sum of its g up to token i (all g <= 0) and L_ij = e^{G_i - G_j}, j <= i:
//     A_ij = [j < i] beta_i L_ij (k_i.k_j);   T = (I + A)^-1 diag(beta);   P_ij = [j <= i] scale L_ij (q_i.k_j)
//     Z    = V - diag(e^G) K S                what the entry state leaves of the values
//     X    = T Z                              what each token writes:  x_i = beta_i (v_i - e^{g_i} k_i^T S_{i-1})
//     O    = scale diag(e^G) Q S + (P T) Z
//     S    = e^{G_end} S + K^T diag(e^{G_end - G}) X
//
// T, P T and the decays do not depend on the state. A first launch makes them for every chunk and head at once, into the
// workspace, as the shared-memory tiles that the second's tensor cores read. The second walks the chunks of each sequence and
// head: four dependent products a chunk, two of them (K S and Q S; T Z and P T Z) one MMA each on stacked operands.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "kda.h"
#include "kda_delta.h"
#include "kda_linear.cuh"
#include "kda_tensor_map.h"

namespace kda {
namespace delta {

namespace {

using lin::f2;
using lin::pair;
using lin::split;

constexpr int C = 64;  // tokens of a chunk

// What the first launch leaves of a chunk and head. The tiles are rows of 64 bf16 (128 bytes), 128-byte swizzled.
struct Decays {
    float upto[C];    // e^{G_t}
    float after[C];   // e^{G_end - G_t}
    float whole, less;  // e^{G_end}, and minus 1
    float pad[30];
};
constexpr int TILE = C * 128;  // 64 x 64 bf16
constexpr int OFF_T = 0, OFF_PT = TILE, OFF_TLO = 2 * TILE, OFF_DECAYS = 3 * TILE;  // in this order in a stage, too
constexpr int IMAGE = OFF_DECAYS + sizeof(Decays);
static_assert(IMAGE % 128 == 0 && sizeof(Decays) % 16 == 0, "bulk copies");

// 16-byte group c of row r of a tile
__device__ __forceinline__ int swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// Workspace slots of chunks: those of sequence n begin at cu[n] / 64 + n, which leaves each as many as it can need.
__device__ __forceinline__ int64_t slot_base(int64_t bos, int64_t n) { return bos / C + n; }

struct ChunkParams {
    Params a;
    CUtensorMap tq, tk, tv;
    unsigned char *images;  // [slot][head]
    int64_t slots;
};

// ------------------------------------------------------------------ first launch: T, P T and the decays of each chunk
namespace prep {

constexpr int THREADS = 256;
constexpr int LD = 68;  // floats of a row of A and T in shared memory
constexpr int OFF_K = 0, OFF_Q = C * 256;          // k and q, rows of 256 bytes; then, over them, A and T
constexpr int OFF_A = 0, OFF_TF = C * LD * 4;
constexpr int OFF_M = 2 * C * LD * 4;              // 32 x LD floats: A21 T11
constexpr int OFF_IMG = OFF_M + 32 * LD * 4;
constexpr int OFF_G = OFF_IMG + IMAGE;             // float2 [64]: log2 prefix in two terms; beta
constexpr int SMEM = OFF_G + C * 8 + C * 4;
static_assert(OFF_M >= 2 * C * 256 && OFF_IMG % 128 == 0, "layout");

__device__ __forceinline__ int kq_at(int r, int c) { return r * 256 + ((c & 8) << 4) + (((c ^ r) & 7) << 4); }  // 16-byte group c

// The sequence whose slots hold `slot`: the last n with slot_base(cu[n], n) <= slot (whole warp).
__device__ __forceinline__ int find_sequence(const Params &p, int64_t slot, int lane) {
    int lo = 0, n = p.N;  // among lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + step * lane;
        const bool ok = step * lane < n && slot_base(__ldg(p.cu + at), at) <= slot;
        const unsigned b = __ballot_sync(0xffffffffu, ok);
        const int last = b ? 31 - __clz(b) : 0;
        lo += step * last;
        n = n - step * last < step ? n - step * last : step;
    }
    return lo;
}

// 2^(x + y), |y| far below 1
__device__ __forceinline__ float ex2_2(float x, float y) { return ex2(x) * fmaf(y, 0.6931471805599453f, 1.f); }

__global__ void __launch_bounds__(THREADS, 3) kda_gated_delta_prepare_kernel(const __grid_constant__ ChunkParams cp) {
    const Params &p = cp.a;
    extern __shared__ __align__(128) unsigned char smem[];
    float *A = reinterpret_cast<float *>(smem + OFF_A), *T = reinterpret_cast<float *>(smem + OFF_TF);
    float *M = reinterpret_cast<float *>(smem + OFF_M);
    unsigned char *img = smem + OFF_IMG;
    float2 *G = reinterpret_cast<float2 *>(smem + OFF_G);
    float *beta = reinterpret_cast<float *>(smem + OFF_G + C * 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t slot = blockIdx.x / p.H;
    const int h = static_cast<int>(blockIdx.x % p.H), hk = h / p.rep;

    const int n = find_sequence(p, slot, lane);
    const int64_t bos = p.cu[n], eos = p.cu[n + 1];
    if (bos < 0 || eos < bos || eos > p.T || p.cu[0] != 0) {
        if (tid == 0) set_status(p.status, KDA_ERR_BAD_SEQLENS);
        return;
    }
    const int64_t t0 = bos + (slot - slot_base(bos, n)) * C;
    if (t0 < bos || t0 >= eos) return;
    const int left = eos - t0 < C ? static_cast<int>(eos - t0) : C;

#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int idx = tid + i * THREADS, r = (idx >> 4) & 63, c = idx & 15;
        const bool is_q = idx >= 1024, in = r < left;
        const __nv_bfloat16 *src = is_q ? p.q + (t0 + (in ? r : 0)) * p.qs : p.k + (t0 + (in ? r : 0)) * p.ks;
        cp_async16(smem + (is_q ? OFF_Q : OFF_K) + kq_at(r, c), src + hk * DK + 8 * c, in ? 16 : 0);
    }
    if (warp == 0) {  // log2 decays, summed in 64 bits: differences of far sums keep their last bits
        double x[2];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const float g = t < left ? p.g[(t0 + t) * p.H + h] : 0.f;
            beta[t] = t < left ? p.beta[(t0 + t) * p.H + h] : 0.f;
            bad |= !(g <= 0.f);
            x[i] = (g < -138.f ? -200.0 : static_cast<double>(g) * 1.4426950408889634);  // (2^-200 is 0 in fp32)
        }
        double s = x[0] + x[1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        const double end = __shfl_sync(0xffffffffu, s, 31);
        const double g1 = s, g0 = s - x[1];
        Decays *d = reinterpret_cast<Decays *>(img + OFF_DECAYS);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const double gt = i ? g1 : g0, rest = end - gt;
            const float hi = static_cast<float>(gt), lo = static_cast<float>(gt - hi);
            G[2 * lane + i] = make_float2(hi, lo);
            d->upto[2 * lane + i] = ex2_2(hi, lo);
            const float rhi = static_cast<float>(rest);
            d->after[2 * lane + i] = ex2_2(rhi, static_cast<float>(rest - rhi));
        }
        if (lane == 0) {
            const float hi = static_cast<float>(end), lo = static_cast<float>(end - hi);
            d->whole = ex2_2(hi, lo);
            d->less = expm1f(static_cast<float>(end * 0.6931471805599453));
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(p.status, KDA_ERR_GATE_RANGE);
    }
    cp_async_commit();
    cp_async_wait_all();
    __syncthreads();

    // rows 16 rb .. of K K^T (warps 0-3) or Q K^T (4-7), up to the diagonal
    const int rb = warp & 3;
    float acc[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    {
        const unsigned char *rows = smem + (warp < 4 ? OFF_K : OFF_Q);
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
            uint32_t a[4];
            ldsm_x4(a, rows + kq_at(16 * rb + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j > rb) continue;
                uint32_t b[4];
                ldsm_x4(b, smem + OFF_K + kq_at(16 * j + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)));
                mma16816(acc[2 * j], a, b[0], b[1]);
                mma16816(acc[2 * j + 1], a, b[2], b[3]);
            }
        }
    }
    const int i0 = 16 * rb + (lane >> 2);
    const float2 gi[2] = {G[i0], G[i0 + 8]};
    const float mul[2] = {warp < 4 ? beta[i0] : p.scale, warp < 4 ? beta[i0 + 8] : p.scale};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = i0 + (c >> 1) * 8, s = 8 * j + 2 * (lane & 3) + (c & 1);
            const float2 gs = G[s];
            const float d = (gi[c >> 1].x - gs.x) + (gi[c >> 1].y - gs.y);
            const bool in = warp < 4 ? s < i : s <= i;
            acc[j][c] = in ? mul[c >> 1] * ex2(d) * acc[j][c] : 0.f;
        }
    }
    __syncthreads();  // (k and q have been read: A and T go over them)
    if (warp < 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                *reinterpret_cast<float2 *>(A + (i0 + 8 * c) * LD + 8 * j + 2 * (lane & 3)) =
                    make_float2(acc[j][2 * c], acc[j][2 * c + 1]);
        __syncwarp();
        // the diagonal block of these rows, inverted by substitution: a lane has a column
        if (lane < 16) {
            const float *a = A + 16 * rb * LD + 16 * rb;
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float s0 = r == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                for (int m = 0; m < r; m += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(a + r * LD + m);
                    s0 = fmaf(-v.x, x[m], s0);
                    if (m + 1 < r) s1 = fmaf(-v.y, x[m + 1], s1);
                    if (m + 2 < r) s0 = fmaf(-v.z, x[m + 2], s0);
                    if (m + 3 < r) s1 = fmaf(-v.w, x[m + 3], s1);
                }
                x[r] = s0 + s1;
                T[(16 * rb + r) * LD + 16 * rb + lane] = x[r];
            }
        }
    }
    __syncthreads();
    {  // the blocks below the diagonal of both halves: -T22 (A21 T11), 16 x 16
        const int half = tid >> 7, i = (tid >> 3) & 15, j = 2 * (tid & 7);
        const float *a = A + (32 * half + 16) * LD + 32 * half, *t11 = T + 32 * half * LD + 32 * half;
        float *m = M + 16 * half * LD;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float av = a[i * LD + k];
            const float2 t = *reinterpret_cast<const float2 *>(t11 + k * LD + j);
            s0 = fmaf(av, t.x, s0);
            s1 = fmaf(av, t.y, s1);
        }
        *reinterpret_cast<float2 *>(m + i * LD + j) = make_float2(s0, s1);
        __syncthreads();
        const float *t22 = T + (32 * half + 16) * LD + 32 * half + 16;
        s0 = s1 = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float av = t22[i * LD + k];
            const float2 t = *reinterpret_cast<const float2 *>(m + k * LD + j);
            s0 = fmaf(-av, t.x, s0);
            s1 = fmaf(-av, t.y, s1);
        }
        *reinterpret_cast<float2 *>(T + (32 * half + 16 + i) * LD + 32 * half + j) = make_float2(s0, s1);
        // (above the diagonal blocks: zeros, that the next step multiplies)
        *reinterpret_cast<float2 *>(T + (32 * half + i) * LD + 32 * half + 16 + j) = make_float2(0.f, 0.f);
        __syncthreads();
    }
    {  // and of the whole, 32 x 32
        const int i = tid >> 3, j = 4 * (tid & 7);
        auto product = [&](const float *a, const float *b) {
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int k = 0; k < 32; ++k) {
                const float av = a[i * LD + k];
                const float4 t = *reinterpret_cast<const float4 *>(b + k * LD + j);
                s.x = fmaf(av, t.x, s.x);
                s.y = fmaf(av, t.y, s.y);
                s.z = fmaf(av, t.z, s.z);
                s.w = fmaf(av, t.w, s.w);
            }
            return s;
        };
        *reinterpret_cast<float4 *>(M + i * LD + j) = product(A + 32 * LD, T);
        __syncthreads();
        const float4 s = product(T + 32 * LD + 32, M);
        *reinterpret_cast<float4 *>(T + (32 + i) * LD + j) = make_float4(-s.x, -s.y, -s.z, -s.w);
        __syncthreads();
    }
    {  // T diag(beta) in two bf16 terms
        const int r = tid >> 2, c0 = 16 * (tid & 3);
#pragma unroll
        for (int c = 0; c < 16; c += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int s = c0 + c + 2 * j;
                const float2 t = *reinterpret_cast<const float2 *>(T + r * LD + s);
                const float x = s <= r ? t.x * beta[s] : 0.f, y = s + 1 <= r ? t.y * beta[s + 1] : 0.f;
                hi[j] = pack_bf16(x, y);
                const float2 f = unpack_bf16(hi[j]);
                lo[j] = pack_bf16(x - f.x, y - f.y);
            }
            const int at = swz(r, (c0 + c) / 8);
            *reinterpret_cast<uint4 *>(img + OFF_T + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(img + OFF_TLO + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    __syncthreads();
    if (warp >= 4) {  // P T, rows 16 rb ..: P's accumulators are its fragments, both factors in two terms
        float pt[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) pt[j][i] = 0.f;
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
            if (kb > rb) continue;
            uint32_t ph[4], pl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *v = &acc[2 * kb + (i >> 1)][2 * (i & 1)];
                ph[i] = pack_bf16(v[0], v[1]);
                const float2 f = unpack_bf16(ph[i]);
                pl[i] = pack_bf16(v[0] - f.x, v[1] - f.y);
            }
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
                if (nb > kb) continue;
                uint32_t bh[4], bl[4];
                const int at = swz(16 * kb + (lane & 15), 2 * nb + (lane >> 4));
                ldsm_x4_t(bh, img + OFF_T + at);
                ldsm_x4_t(bl, img + OFF_TLO + at);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    mma16816(pt[2 * nb + u], ph, bh[2 * u], bh[2 * u + 1]);
                    mma16816(pt[2 * nb + u], ph, bl[2 * u], bl[2 * u + 1]);
                    mma16816(pt[2 * nb + u], pl, bh[2 * u], bh[2 * u + 1]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                *reinterpret_cast<uint32_t *>(img + OFF_PT + swz(i0 + 8 * c, j) + 4 * (lane & 3)) =
                    pack_bf16(pt[j][2 * c], pt[j][2 * c + 1]);
    }
    fence_proxy_async_shared();
    __syncthreads();
    if (tid == 0) {
        bulk_s2g(cp.images + (slot * p.H + h) * IMAGE, img, IMAGE);
        bulk_commit();
        bulk_wait_all();
    }
}

}  // namespace prep

// ------------------------------------------------------------------ second launch: the state from chunk to chunk
namespace walk {

// Everything is transposed: lanes of the accumulators are the 128 value columns. What depends on the state (S, Z, X, each in two bf16
// terms) is then the operand that tensor memory holds, and never passes through shared memory, whose bandwidth would bound this
// kernel otherwise; K, Q, T and P T are read from the tiles as they arrive.
constexpr int WARPS = 16;   // warp = lanes 32 (w % 4) .., part w / 4: 32 keys of the state, 16 tokens of a chunk
constexpr int KEYS = 32, TOKS = 16;
constexpr int WARP_LOAD = WARPS, WARP_MMA = WARPS + 1, THREADS = 32 * (WARPS + 2);
constexpr int STAGES = 3;
// a stage: [K ; Q] and V as panels of 64 channels; [T ; P T]; second term of T; decays
constexpr int PANEL = 2 * TILE;
constexpr int OFF_KQ = 0, OFF_V = 2 * PANEL, OFF_TT = OFF_V + 2 * TILE, OFF_TL = OFF_TT + 2 * TILE, OFF_D = OFF_TL + TILE;
constexpr int STAGE = OFF_D + 1024;
static_assert(sizeof(Decays) <= 1024, "stage");
constexpr int STAGE_BYTES = 2 * PANEL + 2 * TILE + IMAGE;  // that arrive
constexpr int OFF_MISC = STAGES * STAGE;
// Tensor memory columns: S (first terms of 128 keys, then second); (K S)^T, under it Z, and (Q S)^T; X^T, under it X in two terms, and
// (P T Z)^T; the update (K^T X)^T. Of Z and X, 16 tokens take 8 columns of first terms and 8 of second, over their sums.
constexpr uint32_t COL_S = 0, COL_KS = 128, COL_QS = 192, COL_X = 256, COL_O = 320, COL_U = 384;

struct Misc {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t s[2], z, x;           // written; S by halves of the keys
    uint64_t ks, xs, u;            // MMAs complete: K S and Q S; T Z and P T Z; the update
    uint64_t drained;
    uint32_t tmem;
    int32_t abort;
};
constexpr int SMEM = OFF_MISC + static_cast<int>(sizeof(Misc)) + 1024;
static_assert(SMEM <= 227 * 1024, "one CTA's shared memory");

// waits of up to 0.1 ms each before a role gives up; and before one that has given up takes its own copies for complete
constexpr int WAITS = 20000, WAITS_DRAIN = 100;
__device__ __forceinline__ bool wait(Misc *m, uint64_t *bar, uint32_t parity) {
    int i = 0;
#pragma unroll 1
    while (!lin::mbar_wait_some(bar, parity)) {
        if (++i == WAITS) *reinterpret_cast<volatile int32_t *>(&m->abort) = 1;
        if (*reinterpret_cast<volatile int32_t *>(&m->abort)) return false;
    }
    return true;
}
__device__ __forceinline__ void wait_drain(uint64_t *bar, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < WAITS_DRAIN && !lin::mbar_wait_some(bar, parity); ++i) {
    }
}
__device__ __forceinline__ bool wait_warp(Misc *m, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(m, bar, parity));
}
__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) lin::mbar_arrive(bar);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[8]) { tmem_st8(t, r); }
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&r)[16]) { tmem_st16(t, r); }
// v in two bf16 terms: N columns of pairs at `hi` and at `lo`, and on to the MMAs
template <int N>
__device__ __forceinline__ void store_split(uint32_t hi, uint32_t lo, const f2 (&v)[N]) {
    uint32_t h[N], l[N];
    const f2 minus = pair(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = lin::bf16_of(v[i]);
    tmem_st(hi, h);
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = lin::bf16_of(lin::fma2(lin::of_bf16(h[i]), minus, v[i]));
    tmem_st(lo, l);
    tmem_wait_st();
    tc_fence_before();
}

__global__ void __launch_bounds__(THREADS, 1) kda_gated_delta_chunk_kernel(const __grid_constant__ ChunkParams cp) {
    const Params &p = cp.a;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    Misc *m = reinterpret_cast<Misc *>(smem + OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t chain = blockIdx.x;
    const int n = static_cast<int>(chain / p.H), h = static_cast<int>(chain % p.H), hk = h / p.rep;
    const int64_t bos = p.cu[n], eos = p.cu[n + 1];
    if (bos < 0 || eos < bos || eos > p.T || p.cu[0] != 0) {
        if (tid == 0) set_status(p.status, KDA_ERR_BAD_SEQLENS);
        return;
    }
    const int chunks = static_cast<int>((eos - bos + C - 1) / C);

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) mbar_init(&m->full[i], 1), mbar_init(&m->empty[i], WARPS + 1);
        for (int i = 0; i < 2; ++i) mbar_init(&m->s[i], WARPS / 2);
        mbar_init(&m->z, WARPS), mbar_init(&m->x, WARPS), mbar_init(&m->ks, 1), mbar_init(&m->xs, 1), mbar_init(&m->u, 1);
        mbar_init(&m->drained, 1);
        m->abort = 0;
        mbar_fence_init();
    }
    if (warp == WARP_MMA) tmem_alloc(&m->tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem;

    if (warp == WARP_LOAD) {
        if (lane == 0) {
            const unsigned char *images = cp.images + (slot_base(bos, n) * p.H + h) * IMAGE;
            bool ok = true;
            int it = 0;
            for (; it < chunks; ++it) {
                const int st = it % STAGES, t = static_cast<int>(bos) + it * C;
                if (!(ok = wait(m, &m->empty[st], ((it / STAGES) & 1) ^ 1))) break;
                unsigned char *s = smem + st * STAGE;
                uint64_t *bar = &m->full[st];
                const uint64_t first = lin::evict_first();
                mbar_arrive_expect_tx(bar, STAGE_BYTES);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    lin::tma_load_3d(s + OFF_KQ + c * PANEL, &cp.tk, 64 * c, hk, t, bar, first);
                    lin::tma_load_3d(s + OFF_KQ + c * PANEL + TILE, &cp.tq, 64 * c, hk, t, bar, first);
                    lin::tma_load_3d(s + OFF_V + c * TILE, &cp.tv, 64 * c, h, t, bar, first);
                }
                bulk_g2s(s + OFF_TT, images + static_cast<int64_t>(it) * p.H * IMAGE, IMAGE, bar);
            }
            if (!ok)  // what is in flight lands before the CTA ends
                for (int i = it < STAGES ? 0 : it - STAGES; i < it; ++i) wait_drain(&m->full[i % STAGES], (i / STAGES) & 1);
        }
    } else if (warp == WARP_MMA) {
        const uint32_t base = smem_u32(smem);
        constexpr uint32_t ID = lin::idesc_bf16(false, false, 128, 128), ID_LO = lin::idesc_bf16(false, false, 128, 64),
                           ID_U = lin::idesc_bf16(false, true, 128, 128);
        bool ok = true;
        for (int it = 0; it < chunks; ++it) {
            const int st = it % STAGES;
            const uint32_t ph = it & 1, s = base + st * STAGE;
            if (!(ok = wait_warp(m, &m->full[st], (it / STAGES) & 1))) break;
            const int64_t left = eos - bos - static_cast<int64_t>(it) * C;
            if (left < C) {  // the rows of K behind are another sequence's, or anything: as zeros
                unsigned char *kq = smem + st * STAGE + OFF_KQ;
                for (int i = static_cast<int>(left) * 8 + lane; i < TILE / 16; i += 32) {
                    *reinterpret_cast<uint4 *>(kq + i * 16) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(kq + PANEL + i * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_shared();
                __syncwarp();
            }
            auto kq_at = [&](int k) { return umma_desc_sw128(s + OFF_KQ + (k >> 2) * PANEL + (k & 3) * 32, 16, 1024); };
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!(ok = wait_warp(m, &m->s[half], ph))) break;
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int k = 4 * half; k < 4 * half + 4; ++k) {
                        lin::umma_ts(tmem + COL_KS, tmem + COL_S + 8 * k, kq_at(k), ID, k > 0);
                        lin::umma_ts(tmem + COL_KS, tmem + COL_S + 64 + 8 * k, kq_at(k), ID, 1);
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
            if (lane == 0) {
                umma_commit(&m->ks);
            }
            __syncwarp();
            if (!(ok = wait_warp(m, &m->z, ph))) break;
            tc_fence_after();
            if (lane == 0) {
                auto t_at = [&](int off, int k) { return umma_desc_sw128(s + off + k * 32, 16, 1024); };
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lin::umma_ts(tmem + COL_X, tmem + COL_KS + 16 * k, t_at(OFF_TT, k), ID, k > 0);
                    lin::umma_ts(tmem + COL_X, tmem + COL_KS + 16 * k + 8, t_at(OFF_TT, k), ID, 1);
                    lin::umma_ts(tmem + COL_X, tmem + COL_KS + 16 * k, t_at(OFF_TL, k), ID_LO, 1);
                }
                umma_commit(&m->xs);
            }
            __syncwarp();
            if (!(ok = wait_warp(m, &m->x, ph))) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t b = umma_desc_sw128(s + OFF_KQ + k * 2048, PANEL, 1024);
                    lin::umma_ts(tmem + COL_U, tmem + COL_X + 16 * k, b, ID_U, k > 0);
                    lin::umma_ts(tmem + COL_U, tmem + COL_X + 16 * k + 8, b, ID_U, 1);
                }
                umma_commit(&m->u);
                umma_commit(&m->empty[st]);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) {
            umma_commit(&m->drained);
            wait_drain(&m->drained, 0);
        }
        __syncwarp();
    } else {
        const int quad = warp & 3, part = warp >> 2, half = part >> 1;
        const int val = 32 * quad + lane;  // the value column
        const uint32_t t = tmem + (static_cast<uint32_t>(32 * quad) << 16);
        const int k0 = KEYS * part, t0 = TOKS * part;
        f2 S[KEYS / 2];  // keys k0 + 2 i, k0 + 2 i + 1
        {
            const float *s0 = p.s0 ? p.s0 + static_cast<size_t>(chain) * (DK * DV) + k0 * DV + val : nullptr;
#pragma unroll
            for (int i = 0; i < KEYS / 2; ++i) S[i] = s0 ? pair(s0[2 * i * DV], s0[(2 * i + 1) * DV]) : 0;
        }
        bool ok = true;
        for (int it = 0; it < chunks; ++it) {
            const int st = it % STAGES;
            const uint32_t ph = it & 1;
            const int64_t rest = eos - bos - static_cast<int64_t>(it) * C;
            const int left = rest < C ? static_cast<int>(rest) : C;
            const unsigned char *stage = smem + st * STAGE;
            const Decays *d = reinterpret_cast<const Decays *>(stage + OFF_D);
            store_split(t + COL_S + k0 / 2, t + COL_S + 64 + k0 / 2, S);
            arrive_warp(&m->s[half]);
            if (!(ok = wait_warp(m, &m->full[st], (it / STAGES) & 1))) break;
            f2 z[TOKS / 2], w[TOKS / 2];
            {
                const unsigned char *v = stage + OFF_V + (val >> 6) * TILE + t0 * 128 + (val & 7) * 2;
                const int c = (val & 63) >> 3;
                auto at = [&](int i) {
                    return static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(v + i * 128 + ((c ^ (i & 7)) << 4))) << 16;
                };
#pragma unroll
                for (int i = 0; i < TOKS / 2; ++i) z[i] = pair(at(2 * i), at(2 * i + 1));
            }
            const float whole = d->whole, less = d->less;
            uint32_t r[16];
            if (!(ok = wait_warp(m, &m->ks, ph))) break;
            tc_fence_after();
            tmem_ld16(t + COL_KS + t0, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < TOKS / 2; ++i) {
                const float2 e = *reinterpret_cast<const float2 *>(&d->upto[t0 + 2 * i]);
                z[i] = lin::fma2(pair(-e.x, -e.y), pair(r[2 * i], r[2 * i + 1]), z[i]);
            }
            auto mask = [&](f2(&v)[TOKS / 2]) {  // tokens behind the sequence: zeros, whatever they are
                if (left == C) return;
#pragma unroll
                for (int i = 0; i < TOKS / 2; ++i) {
                    float x, y;
                    split(v[i], x, y);
                    v[i] = pair(t0 + 2 * i < left ? x : 0.f, t0 + 2 * i + 1 < left ? y : 0.f);
                }
            };
            mask(z);
            store_split(t + COL_KS + t0, t + COL_KS + t0 + 8, z);
            arrive_warp(&m->z);
            if (!(ok = wait_warp(m, &m->xs, ph))) break;
            tc_fence_after();
            tmem_ld16(t + COL_X + t0, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < TOKS / 2; ++i) {
                const float2 e = *reinterpret_cast<const float2 *>(&d->after[t0 + 2 * i]);
                w[i] = lin::mul2(pair(e.x, e.y), pair(r[2 * i], r[2 * i + 1]));
            }
            mask(w);
            store_split(t + COL_X + t0, t + COL_X + t0 + 8, w);
            arrive_warp(&m->x);
            {
                uint32_t q[16];
                tmem_ld16(t + COL_QS + t0, q);
                tmem_ld16(t + COL_O + t0, r);
                tmem_wait_ld();
                tc_fence_before();
                __nv_bfloat16 *o = p.o + ((bos + static_cast<int64_t>(it) * C + t0) * p.H + h) * DV + val;
#pragma unroll
                for (int i = 0; i < TOKS; ++i) {
                    const float x = fmaf(p.scale * d->upto[t0 + i], __uint_as_float(q[i]), __uint_as_float(r[i]));
                    if (t0 + i < left) o[static_cast<int64_t>(i) * p.H * DV] = __float2bfloat16_rn(x);
                }
            }
            arrive_warp(&m->empty[st]);
            if (!(ok = wait_warp(m, &m->u, ph))) break;
            tc_fence_after();
            uint32_t u[32];
            lin::tmem_ld32(t + COL_U + k0, u);
            tmem_wait_ld();
            if (less < -0.5f) {
                const f2 f = pair(whole, whole);
#pragma unroll
                for (int i = 0; i < KEYS / 2; ++i) S[i] = lin::fma2(S[i], f, pair(u[2 * i], u[2 * i + 1]));
            } else {  // (a slow decay is not rounded away chunk after chunk)
                const f2 f = pair(less, less);
#pragma unroll
                for (int i = 0; i < KEYS / 2; ++i) S[i] = lin::add2(S[i], lin::fma2(S[i], f, pair(u[2 * i], u[2 * i + 1])));
            }
        }
        if (p.sT && ok) {
            float *sT = p.sT + static_cast<size_t>(chain) * (DK * DV) + k0 * DV + val;
#pragma unroll
            for (int i = 0; i < KEYS / 2; ++i) {
                float x, y;
                split(S[i], x, y);
                sT[2 * i * DV] = x, sT[(2 * i + 1) * DV] = y;
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && m->abort) set_status(p.status, KDA_ERR_TIMEOUT);
    if (warp == WARP_MMA) tmem_dealloc(tmem, 512);
}

}  // namespace walk

// [tokens][heads][128] bf16 with a token stride; boxes of 64 channels x 1 head x 64 tokens
bool encode_heads(CUtensorMap *m, const __nv_bfloat16 *x, int64_t tokens, int heads, int64_t stride) {
    const cuuint64_t dims[3] = {DK, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {DK * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, 1, C};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, 3, dims, strides, box);
}

}  // namespace

size_t chunked_workspace_bytes(int64_t N, int64_t T, int64_t H) { return static_cast<size_t>((T / C + N) * H) * IMAGE; }

cudaError_t launch_chunked(const Params &a, void *workspace, cudaStream_t stream) {
    if (a.T < 1) return launch_recurrent(a, stream);  // (states pass through)
    ChunkParams p{};
    p.a = a;
    p.images = static_cast<unsigned char *>(workspace);
    p.slots = a.T / C + a.N;
    const int hk = a.H / a.rep;
    if (!encode_heads(&p.tq, a.q, a.T, hk, a.qs) || !encode_heads(&p.tk, a.k, a.T, hk, a.ks) ||
        !encode_heads(&p.tv, a.v, a.T, a.H, a.vs))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(prep::kda_gated_delta_prepare_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, prep::SMEM);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(walk::kda_gated_delta_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, walk::SMEM);
    if (e != cudaSuccess) return e;
    prep::kda_gated_delta_prepare_kernel<<<static_cast<unsigned>(p.slots * a.H), prep::THREADS, prep::SMEM, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    walk::kda_gated_delta_chunk_kernel<<<static_cast<unsigned>(a.N) * a.H, walk::THREADS, walk::SMEM, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace delta
}  // namespace kda
