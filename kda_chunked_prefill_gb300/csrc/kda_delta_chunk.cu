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
// head: K S, T Z and K^T X one after the other, Q S and P T Z beside them. Where there are few sequences, long ones are cut: a pass over
// the parts' states from zero and their maps, and a join, come before the walk (see plan).
//
// Bound by latency. 4 x 2048 tokens, 16 heads: 35 us for the 2112 chunks (5 CTAs an SM, 12 us each: substitutions and products of 16
// rows that wait for one another), 72 for 32 chunks one after the other on 64 SMs, 2.1 us each: three products of 45 to 70 cycles an MMA,
// and after each the accumulators' way through registers, split in two bf16 terms, back to tensor memory. The tensor pipe is busy in
// 46 % of a walking SM's cycles. In all 111 us; 1 x 65536 tokens, 4 heads: 60, states 119, join 58, walk 71, in all 315.
// (Z, X and S in halves, so that MMAs start on the first: 3 % slower, as each half's hand-over costs what it hides. Operands through shared
// memory with 64 value columns a CTA: 5300 cycles a chunk for half of the columns, against 4400 for all.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "kda.h"
#include "kda_delta.h"
#include "kda_linear.cuh"
#include "kda_tensor_map.h"
#include "kda_waits.cuh"

namespace kda {
namespace delta {

namespace {

using lin::f2;
using lin::pair;
using lin::split;

constexpr int C = CHUNK;

// What the first launch leaves of a chunk and head. The tiles are rows of 64 bf16 (128 bytes), 128-byte swizzled.
struct Decays {
    float minus[C];   // -e^{G_t}
    float out[C];     // scale e^{G_t}
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

// Workspace slots of chunks: those of sequence n begin at cu[n] / 64 + n, which leaves each as many as it can need. (Where only the long
// sequences run in chunks, the recurrence's launch before these has listed their chunks, one after the other.)
__device__ __forceinline__ int64_t slot_base(int64_t bos, int64_t n) { return bos / C + n; }

__device__ __forceinline__ uint64_t evict_normal() {  // (the second launch reads them again)
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// A launch may be set up while the one before ends: what that one wrote is read behind this.
__device__ __forceinline__ void wait_for_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A part of a sequence that a CTA walks: chunks c0 .. c0 + len - 1 of sequence n.
struct Segment {
    int32_t n, c0, len;
    int32_t slot;   // of its first chunk
    int32_t from;   // the state it begins with: after a cut, its number; -1: the sequence's initial one; -2 - i: cut i's copy of it
    int32_t to;     // of the pass over the states: the cut that its state goes to
    int32_t kind;   // 0: outputs and the sequence's last state, 3: outputs; of the pass over the states, 1: the state, 2: its map
};
// The cuts of a sequence: numbers first .. first + count - 1.
struct Cuts {
    int32_t n, first, count;
};

struct ChunkParams {
    Params a;
    CUtensorMap tq, tk, tv;
    unsigned char *images;  // [slot][head]
    int64_t slots;          // of chunks
    // sequences that are cut (device memory in the workspace)
    int32_t longer;         // sequences of no more tokens are left out (the recurrence runs them, and lists the others); -1: none is
    int32_t withhold;       // tests: the chunk of each CTA whose Z is not handed on (-1: none)
    int32_t shortest;       // shortest cut that the workspace is sized for, in chunks; 0: none is cut
    int32_t sms;
    int32_t from;           // first of the outputs' jobs that are run in rounds
    int32_t *counts;        // [0] segments, [1] those of the pass over the states, [2] sequences to join
    const int32_t *listed;  // the long sequences' chunks, where only those run here: see Params
    const int2 *list;
    Segment *segs, *segs_s;
    Cuts *cuts;
    // [cut][head][2][128][128]: the state after it (from zero; joined: the true one); the map of the part before it, transposed, or, for a
    // sequence's first cut, the initial state (which the last part may have overwritten when the first begins with it)
    float *states;
};

// ------------------------------------------------------------------ which sequences are cut, and where
namespace plan {

// Cuts that are estimated: the shortest times these, over 2; and none.
constexpr int CUTS = 8;
__host__ __device__ constexpr int cut_length(int i, int shortest) {
    constexpr int twice[CUTS] = {2, 3, 4, 6, 8, 12, 16, 24};
    return shortest * twice[i] / 2;
}
struct Work {
    int32_t jobs, longest;
    int64_t chunks;
    int32_t cuts;
};
__host__ __device__ inline void add(Work &w, int64_t count, int len) {
    if (count < 1) return;
    w.jobs += static_cast<int32_t>(count);
    w.chunks += count * len;
    if (len > w.longest) w.longest = len;
}
// A sequence of `chunks` cut to `len` or less: its parts' length, and how many.
__host__ __device__ inline void parts_of(int chunks, int len, int &one, int &k) {
    one = chunks;
    k = 1;
    if (chunks <= len) return;
    one = (chunks - 1) / ((chunks - 1) / len + 1) + 1;
    k = (chunks - 1) / one + 1;
}
// Its jobs in the outputs' pass, and in the pass over the states: all parts but the last, the state from zero and, but for the first, the
// map.
__host__ __device__ inline void add_sequence(Work &out, Work &states, int &most, int chunks, int len) {
    int one, k;
    parts_of(chunks, len, one, k);
    add(out, k, one);
    if (k > 1) add(states, 2 * k - 3, one);
    states.cuts += k - 1;
    if (k > most) most = k;
}
// The time of a pass on `sms` CTAs, in chunks (2.1 us): a job takes its own and one for its start and end.
__host__ __device__ inline float pass_time(const Work &w, int heads, int sms) {
    const float jobs = static_cast<float>(w.jobs) * heads, one = w.longest + 1.f;
    const float even = (static_cast<float>(w.chunks) * heads + jobs) / sms + (jobs > sms ? 0.5f * one : 0.f);
    const float rounds = ceilf(jobs / sms) * one;
    const float t = even < rounds ? even : rounds;
    return w.jobs == 0 ? 0.f : t > one ? t : one;
}
// With the join (0.9 of a chunk's time a part) and two more launches. With these three figures the cut taken was within 5 % of the best
// of those tried in 28 batches. 1 sequence of 65,536 tokens: 1 head in parts of 14, 21, 28, 54 chunks 216, 198, 206, 280 us and 2124
// whole; 4 heads 27, 40, 54: 315, 372, 329 and 2174. 16 of 1 to 3853 tokens, 16 heads: the longest in 3 parts 176, whole 191. 4 of
// 2048, 16 heads: in 2 parts 125, whole 112.
__host__ __device__ inline float time_of(const Work &out, const Work &states, int most, int heads, int sms) {
    return pass_time(out, heads, sms) + (most > 1 ? pass_time(states, heads, sms) + 0.9f * most + 2.f : 0.f);
}

constexpr int THREADS = 128, BUCKETS = 64, HELD = 4096;
struct Shared {
    Work out[CUTS + 1], states[CUTS + 1];
    int32_t most[CUTS + 1];
    int32_t bucket[2][BUCKETS];  // first segments of each length, long ones first: of the outputs' pass, of the states'
    int32_t cuts, joined, len, longest;
    int32_t held[HELD];          // chunks of the first items
};

// -1: bounds that are not in order; -2: a sequence that is left out
__device__ __forceinline__ int chunks_of(const ChunkParams &cp, int n) {
    const Params &p = cp.a;
    const int64_t b = p.cu[n], e = p.cu[n + 1];
    if (b < 0 || e < b || e > p.T || p.cu[0] != 0) return -1;
    return e - b <= cp.longer ? -2 : static_cast<int>((e - b + C - 1) / C);
}
__device__ __forceinline__ int warp_sum(int x) { return __reduce_add_sync(0xffffffffu, x); }
__device__ __forceinline__ int warp_max(int x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ Work warp_work(Work w) {
    long long chunks = w.chunks;
#pragma unroll
    for (int d = 16; d; d >>= 1) chunks += __shfl_xor_sync(0xffffffffu, chunks, d);
    return {warp_sum(w.jobs), warp_max(w.longest), chunks, warp_sum(w.cuts)};
}

// Some bounds of the batch are not in order (whole CTA).
__device__ __forceinline__ bool malformed(const ChunkParams &cp) {
    bool bad = false;
    if (cp.longer >= 0)
        bad = cp.listed[1];
    else
        for (int n = threadIdx.x; n < cp.a.N; n += blockDim.x) bad |= chunks_of(cp, n) == -1;
    return __syncthreads_or(bad);
}

// One CTA: the cut by estimates from the lengths, and the segments of both passes, long ones first. (The other CTAs' chunks take longer
// than this only if it is quick: lengths are read once, a warp estimates a cut. 5 to 11 us; as code of its own, out of the chunks' way, a call
// takes 1 to 3 % less.)
__device__ __noinline__ void make(const ChunkParams &cp, Shared *sh) {
    const Params &p = cp.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < 2 * BUCKETS; i += THREADS) sh->bucket[i / BUCKETS][i % BUCKETS] = 0;
    if (tid == 0) sh->cuts = sh->joined = 0;
    // Slots of chunks are found, and the workspace is large enough, where bounds are in order; otherwise this launch runs what it can itself.
    if (malformed(cp)) {
        if (tid == 0) set_status(p.status, KDA_ERR_BAD_SEQLENS);
        if (tid < 3) cp.counts[tid] = 0;
        return;
    }
    // items: the sequences, or the long ones' chunks, of which the first stands for its sequence
    const bool listed = cp.longer >= 0;
    const int items = listed ? cp.listed[0] : p.N;
    auto sequence = [&](int i) { return listed ? cp.list[i].x : i; };
    auto chunks_at = [&](int i) { return listed && cp.list[i].y != 0 ? -2 : chunks_of(cp, sequence(i)); };
    for (int i = tid; i < items && i < HELD; i += THREADS) sh->held[i] = chunks_at(i);
    __syncthreads();
    auto length = [&](int i) { return i < HELD ? sh->held[i] : chunks_at(i); };
    const int candidates = cp.shortest ? CUTS + 1 : 1;  // the last: none is cut
    for (int c = warp; c < candidates; c += THREADS / 32) {
        const int len = c == candidates - 1 ? 0x7fffffff : cut_length(c, cp.shortest);
        Work out{0, 0, 0, 0}, states{0, 0, 0, 0};
        int most = 0;
        for (int i = lane; i < items; i += 32) {
            const int chunks = length(i);
            if (chunks >= 0) add_sequence(out, states, most, chunks, len);
        }
        out = warp_work(out), states = warp_work(states), most = warp_max(most);
        if (lane == 0) sh->out[c] = out, sh->states[c] = states, sh->most[c] = most;
    }
    __syncthreads();
    if (warp == 0) {
        const float t = lane < candidates ? time_of(sh->out[lane], sh->states[lane], sh->most[lane], p.H, cp.sms) : 3.0e38f;
        float least = t;
#pragma unroll
        for (int d = 16; d; d >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, d));
        const int best = 31 - __clz(__ballot_sync(0xffffffffu, t == least && lane < candidates));
        if (lane == 0) {
            sh->len = best == candidates - 1 ? 0x7fffffff : cut_length(best, cp.shortest);
            sh->longest = sh->out[best].longest > 0 ? sh->out[best].longest : 1;
        }
    }
    __syncthreads();
    auto bucket_of = [&](int len) { return BUCKETS - 1 - static_cast<int>(static_cast<int64_t>(len) * (BUCKETS - 1) / sh->longest); };
    auto for_each = [&](auto &&f) {
        for (int i = tid; i < items; i += THREADS) {
            const int chunks = length(i);
            if (chunks < 0) continue;
            int one, k;
            parts_of(chunks, sh->len, one, k);
            f(i, chunks, k, one);
        }
    };
    for_each([&](int, int chunks, int k, int one) {  // (all parts but the last are of one length)
        const int whole = bucket_of(one), last = bucket_of(chunks - (k - 1) * one);
        if (k > 1) {
            atomicAdd(&sh->bucket[0][whole], k - 1);
            atomicAdd(&sh->bucket[1][whole], 2 * k - 3);
        }
        atomicAdd(&sh->bucket[0][last], 1);
    });
    __syncthreads();
    if (warp < 2) {
        int *bucket = sh->bucket[warp];
        const int x = bucket[2 * lane], y = bucket[2 * lane + 1];
        int sum = x + y;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += z;
        }
        bucket[2 * lane] = sum - x - y;
        bucket[2 * lane + 1] = sum - y;
        if (lane == 31) cp.counts[warp] = sum;
    }
    __syncthreads();
    for_each([&](int item, int chunks, int k, int one) {
        const int n = sequence(item), slot = listed ? item : static_cast<int>(slot_base(p.cu[n], n));
        int first = -1, at = 0, at_s = 0;
        if (k > 1) {
            first = atomicAdd(&sh->cuts, k - 1);
            cp.cuts[atomicAdd(&sh->joined, 1)] = {n, first, k - 1};
            at = atomicAdd(&sh->bucket[0][bucket_of(one)], k - 1);
            at_s = atomicAdd(&sh->bucket[1][bucket_of(one)], 2 * k - 3);
        }
        for (int i = 0; i < k - 1; ++i) {
            const int c0 = i * one;
            cp.segs[at++] = {n, c0, one, slot + c0, i ? first + i - 1 : -2 - first, -1, 3};
            cp.segs_s[at_s++] = {n, c0, one, slot + c0, -1, first + i, 1};
            if (i) cp.segs_s[at_s++] = {n, c0, one, slot + c0, -1, first + i, 2};
        }
        const int c0 = (k - 1) * one, len = chunks - c0;
        cp.segs[atomicAdd(&sh->bucket[0][bucket_of(len)], 1)] = {n, c0, len, slot + c0, k > 1 ? first + k - 2 : -1, -1, 0};
    });
    __syncthreads();
    if (tid == 0) cp.counts[2] = sh->joined;
}

}  // namespace plan

// ------------------------------------------------------------------ first launch: T, P T and the decays of each chunk; the plan
namespace prep {

// Four warps to a chunk and head, each with 16 rows of A and P, in blocks of 16 x 16 that stay in registers as fragments. T's
// diagonal blocks by substitution in fp32; below it, T_ij = -T_ii sum_{j <= k < i} A_ik T_kj, one block diagonal after another, on
// operands of two bf16 terms (three products: 2^-16). Scaled by beta from the start: (T diag(beta))_kj does as well for T_kj.
constexpr int THREADS = 128;
constexpr int PER_SM = 5;
constexpr int SB = 16, BLOCKS = C / SB;
constexpr int LD = 20;                                   // floats of a row of a diagonal block
constexpr int OFF_K = 0, OFF_Q = 2 * TILE, OFF_IMG = 0;  // k and q, two panels of 64 channels each; over them, what leaves
constexpr int OFF_MISC = 4 * TILE;
static_assert(IMAGE <= OFF_MISC, "layout");
static_assert(sizeof(plan::Shared) <= OFF_MISC && plan::THREADS == THREADS, "the plan's CTA");

struct Misc {
    alignas(16) float diag[BLOCKS][SB * LD];
    float2 G[C];                        // log2 prefix in two terms
    float beta[C];
    float row[C];                       // e^{G_i - (G before i's block)}
    float col[BLOCKS - 1][C - SB];      // e^{(G before block b + 1) - G_j}
    uint64_t full;
};
constexpr int SMEM = OFF_MISC + static_cast<int>(sizeof(Misc)) + 1024;
static_assert(SMEM * PER_SM <= 227 * 1024, "shared memory");

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

// A sum in two terms, the second what the first leaves.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two add(Two a, Two b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo), hi = s + e;
    return {hi, e - (hi - s)};
}
// 2^(x + y), |y| far below 1
__device__ __forceinline__ float ex2_2(float x, float y) { return ex2(x) * fmaf(y, 0.6931471805599453f, 1.f); }
// 2^(a - b)
__device__ __forceinline__ float ex2_diff(float2 a, float2 b) { return ex2((a.x - b.x) + (a.y - b.y)); }

__device__ __forceinline__ uint32_t transpose(uint32_t a) {  // an 8 x 8 matrix of 16-bit elements
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// two values in two bf16 terms
__device__ __forceinline__ void split_pair(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(x, y);
    const float2 f = unpack_bf16(hi);
    lo = pack_bf16(x - f.x, y - f.y);
}
// A 16 x 16 block as the tensor core's left operand: first and second terms. c[0..1]: rows g and g + 8 of columns 2 q, 2 q + 1 in the
// accumulators' order; c[2..3] of columns 8 further.
struct Left {
    uint32_t hi[4], lo[4];
};
__device__ __forceinline__ void to_left(Left &f, const float (&a)[4], const float (&b)[4]) {
    split_pair(a[0], a[1], f.hi[0], f.lo[0]);
    split_pair(a[2], a[3], f.hi[1], f.lo[1]);
    split_pair(b[0], b[1], f.hi[2], f.lo[2]);
    split_pair(b[2], b[3], f.hi[3], f.lo[3]);
}
// d += left x (hi + lo), without the product of the second terms; hi, lo: right operand's fragments of two tiles of 8 columns
__device__ __forceinline__ void product(float (&d)[2][4], const Left &f, const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        mma16816(d[u], f.hi, hi[2 * u], hi[2 * u + 1]);
        mma16816(d[u], f.hi, lo[2 * u], lo[2 * u + 1]);
        mma16816(d[u], f.lo, hi[2 * u], hi[2 * u + 1]);
    }
}

// Malformed batches: the last CTAs of this launch run the sequences whose own bounds are in order, token
// after token by the recurrence's formulas in fp32: 32 value columns of a sequence and head, a lane a column, a warp 32 keys of it; one
// sum over the warps a token, about 1 us. Nothing in the workspace is used, as where a chunk's images lie presupposes order. (The
// same code in the walk's kernel, never called, took 2 to 3 % of every well-formed call; here 0 to 1 %.)
__device__ __noinline__ void token_by_token(const ChunkParams &cp, int first, int ctas, float *sums) {
    const Params &p = cp.a;
    constexpr int PARTS = THREADS / 32, KEYS = DK / PARTS, BLOCKS = DV / 32, BUF = PARTS * 65;  // k^T S, q^T S and q.k by parts of the keys
    const int part = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!plan::malformed(cp)) return;
    const int64_t jobs = static_cast<int64_t>(p.N) * p.H * BLOCKS;
    uint32_t buf = 0;
#pragma unroll 1
    for (int64_t job = first; job < jobs; job += ctas) {
        const int val = 32 * static_cast<int>(job % BLOCKS) + lane, h = static_cast<int>(job / BLOCKS % p.H), n = static_cast<int>(job / BLOCKS / p.H);
        if (plan::chunks_of(cp, n) < 0) continue;  // (its own bounds are bad, or the recurrence runs it)
        const int64_t bos = p.cu[n], eos = p.cu[n + 1];
        const size_t state = (static_cast<size_t>(n) * p.H + h) * (DK * DV) + static_cast<size_t>(KEYS * part) * DV + val;
        const int c = h / p.rep * DK + KEYS * part;
        float S[KEYS];
#pragma unroll
        for (int i = 0; i < KEYS; ++i) S[i] = p.s0 ? p.s0[state + i * DV] : 0.f;
#pragma unroll 1
        for (int64_t t = bos; t < eos; ++t, buf ^= 1) {
            float *at = sums + buf * BUF;  // (its last use was read before the barrier of the token before)
            const uint4 *kp = reinterpret_cast<const uint4 *>(p.k + t * p.ks + c), *qp = reinterpret_cast<const uint4 *>(p.q + t * p.qs + c);
            uint32_t k[KEYS / 2];
            float ks = 0.f, qs = 0.f, qk = 0.f;
#pragma unroll
            for (int i = 0; i < KEYS / 8; ++i) {
                const uint4 x = kp[i], y = qp[i];
                const uint32_t q[4] = {y.x, y.y, y.z, y.w};
                k[4 * i] = x.x, k[4 * i + 1] = x.y, k[4 * i + 2] = x.z, k[4 * i + 3] = x.w;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 kk = unpack_bf16(k[4 * i + j]), qq = unpack_bf16(q[j]);
                    const float s0 = S[8 * i + 2 * j], s1 = S[8 * i + 2 * j + 1];
                    ks = fmaf(kk.y, s1, fmaf(kk.x, s0, ks));
                    qs = fmaf(qq.y, s1, fmaf(qq.x, s0, qs));
                    qk = fmaf(qq.y, kk.y, fmaf(qq.x, kk.x, qk));
                }
            }
            at[65 * part + lane] = ks;
            at[65 * part + 32 + lane] = qs;
            if (lane == 0) at[65 * part + 64] = qk;
            __syncthreads();
            ks = qs = qk = 0.f;
#pragma unroll
            for (int i = 0; i < PARTS; ++i) ks += at[65 * i + lane], qs += at[65 * i + 32 + lane], qk += at[65 * i + 64];
            const float d = expf(p.g[t * p.H + h]), v = __bfloat162float(p.v[t * p.vs + h * DV + val]);
            const float x = p.beta[t * p.H + h] * fmaf(-d, ks, v);
            if (part == 0) p.o[(t * p.H + h) * DV + val] = __float2bfloat16_rn(p.scale * fmaf(d, qs, qk * x));
#pragma unroll
            for (int i = 0; i < KEYS / 2; ++i) {
                const float2 kk = unpack_bf16(k[i]);
                S[2 * i] = fmaf(kk.x, x, d * S[2 * i]);
                S[2 * i + 1] = fmaf(kk.y, x, d * S[2 * i + 1]);
            }
        }
        if (p.sT) {
#pragma unroll
            for (int i = 0; i < KEYS; ++i) p.sT[state + i * DV] = S[i];
        }
    }
}
// their number: an SM each, and no more than they have jobs
int spare_ctas(int64_t N, int64_t H, int sms) { return static_cast<int>(4 * N * H < sms ? 4 * N * H : sms); }

__global__ void __launch_bounds__(THREADS, PER_SM) kda_gated_delta_prepare_kernel(const __grid_constant__ ChunkParams cp) {
    const Params &p = cp.a;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    unsigned char *img = smem + OFF_IMG;
    Misc *m = reinterpret_cast<Misc *>(smem + OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    let_next_launch();
    if (blockIdx.x == 0) {
        plan::make(cp, reinterpret_cast<plan::Shared *>(smem));
        return;
    }
    if (blockIdx.x > cp.slots * p.H) {
        const int first = static_cast<int>(1 + cp.slots * p.H);
        token_by_token(cp, static_cast<int>(blockIdx.x) - first, static_cast<int>(gridDim.x) - first, reinterpret_cast<float *>(smem));
        return;
    }
    const int64_t slot = (blockIdx.x - 1) / p.H;
    const int h = static_cast<int>((blockIdx.x - 1) % p.H), hk = h / p.rep;

    int n, chunk = 0;
    if (cp.longer >= 0) {
        if (slot >= cp.listed[0]) return;
        const int2 at = cp.list[slot];
        n = at.x, chunk = at.y;
    } else {
        n = find_sequence(p, slot, lane);
    }
    const int64_t bos = p.cu[n], eos = p.cu[n + 1];
    if (bos < 0 || eos < bos || eos > p.T || p.cu[0] != 0) return;  // (the batch is malformed: the plan reports it)
    const int64_t t0 = bos + (cp.longer >= 0 ? chunk : slot - slot_base(bos, n)) * C;
    if (t0 < bos || t0 >= eos) return;
    const int left = eos - t0 < C ? static_cast<int>(eos - t0) : C;  // rows behind are anything: what they enter is set to zero

    if (tid == 0) {
        mbar_init(&m->full, 1);
        mbar_fence_init();
        mbar_arrive_expect_tx(&m->full, 4 * TILE);
        const uint64_t keep = evict_normal();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            lin::tma_load_3d(smem + OFF_K + c * TILE, &cp.tk, 64 * c, hk, static_cast<int>(t0), &m->full, keep);
            lin::tma_load_3d(smem + OFF_Q + c * TILE, &cp.tq, 64 * c, hk, static_cast<int>(t0), &m->full, keep);
        }
    }
    __syncthreads();  // (the barrier is set up)
    float decays[4];  // of tokens 2 lane, 2 lane + 1: to the token, after it (warp 0)
    float whole = 0.f, less = 0.f;
    if (warp == 0) {
        // log2 decays, summed in two fp32 terms: differences of far sums keep their last bits. (In 64 bits, floating or fixed point, the
        // sums took two to three times as long, and every warp waits for them.) Below -138 a gate counts as -inf: 2^-200 is 0 in fp32.
        Two x[2];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const float g = t < left ? p.g[(t0 + t) * p.H + h] : 0.f;
            m->beta[t] = t < left ? p.beta[(t0 + t) * p.H + h] : 0.f;
            bad |= !(g <= 0.f);
            const float y = g * LOG2E;
            x[i] = g < -138.f ? Two{-200.f, 0.f} : Two{y, fmaf(g, LOG2E, -y) + g * 1.925963e-8f};  // (log2 e beyond LOG2E)
        }
        Two s = add(x[0], x[1]);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Two y{__shfl_up_sync(0xffffffffu, s.hi, d), __shfl_up_sync(0xffffffffu, s.lo, d)};
            if (lane >= d) s = add(s, y);
        }
        const Two end{__shfl_sync(0xffffffffu, s.hi, 31), __shfl_sync(0xffffffffu, s.lo, 31)};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const Two gt = i ? s : add(s, {-x[1].hi, -x[1].lo}), rest = add(end, {-gt.hi, -gt.lo});
            m->G[2 * lane + i] = make_float2(gt.hi, gt.lo);
            decays[i] = ex2_2(gt.hi, gt.lo);
            decays[2 + i] = ex2_2(rest.hi, rest.lo);
        }
        whole = ex2_2(end.hi, end.lo);
        less = expm1f((end.hi + end.lo) * 0.6931471805599453f);
        if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(p.status, KDA_ERR_GATE_RANGE);
        __syncwarp();
        // decays between blocks, in two factors that meet at the row's block
        const float2 zero = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < C; i += 32) m->row[i + lane] = ex2_diff(m->G[i + lane], i + lane >= SB ? m->G[((i + lane) & ~(SB - 1)) - 1] : zero);
#pragma unroll
        for (int i = 0; i < 6 * SB; i += 32) {
            const int e = i + lane, b = e < SB ? 0 : e < 3 * SB ? 1 : 2, j = e - (b == 0 ? 0 : b == 1 ? SB : 3 * SB);
            m->col[b][j] = ex2_diff(m->G[SB * (b + 1) - 1], m->G[j]);
        }
    }
    bool here = mbar_try_wait(&m->full, 0);
#pragma unroll 1
    for (int i = 0; i < 200000 && !here; ++i) here = lin::mbar_wait_some(&m->full, 0);

    // rows 16 w .. of K K^T and Q K^T, up to the diagonal
    const int w = warp, g = lane >> 2, q2 = 2 * (lane & 3);
    auto kq_at = [](int r, int c) { return (c >> 3) * TILE + swz(r, c & 7); };  // 16-byte group c of row r
    float sk[2 * BLOCKS][4], sq[2 * BLOCKS][4];
#pragma unroll
    for (int j = 0; j < 2 * BLOCKS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sk[j][i] = sq[j][i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < DK / 16; ++kk) {
        uint32_t a[4], c[4];
        ldsm_x4(a, smem + OFF_K + kq_at(SB * w + (lane & 15), 2 * kk + (lane >> 4)));
        ldsm_x4(c, smem + OFF_Q + kq_at(SB * w + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j) {
            if (j > w) continue;
            uint32_t b[4];
            ldsm_x4(b, smem + OFF_K + kq_at(SB * j + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)));
            mma16816(sk[2 * j], a, b[0], b[1]);
            mma16816(sk[2 * j + 1], a, b[2], b[3]);
            mma16816(sq[2 * j], c, b[0], b[1]);
            mma16816(sq[2 * j + 1], c, b[2], b[3]);
        }
    }
    // (the copies end at the latest with the kernel: never false)
    if (!__syncthreads_and(here)) {
        if (tid == 0) set_status(p.status, KDA_ERR_TIMEOUT);
        return;
    }
    const int i0 = SB * w + g;
    const float bi[2] = {m->beta[i0], m->beta[i0 + 8]};
    const bool in[2] = {i0 < left, i0 + 8 < left};
    Left A[BLOCKS - 1], P[BLOCKS];
    {
        const float rf[2] = {m->row[i0], m->row[i0 + 8]};
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j) {
            if (j > w) continue;
            if (j < w) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float2 cf = *reinterpret_cast<const float2 *>(&m->col[w - 1][SB * j + 8 * u + q2]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float l = rf[c >> 1] * ((c & 1) ? cf.y : cf.x);
                        sk[2 * j + u][c] = in[c >> 1] ? bi[c >> 1] * l * sk[2 * j + u][c] : 0.f;
                        sq[2 * j + u][c] = in[c >> 1] ? p.scale * l * sq[2 * j + u][c] : 0.f;
                    }
                }
                to_left(A[j < BLOCKS - 1 ? j : 0], sk[2 * j], sk[2 * j + 1]);
            } else {
                const float2 gi[2] = {m->G[i0], m->G[i0 + 8]};
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int r = g + 8 * (c >> 1), s = 8 * u + q2 + (c & 1);
                        const float l = ex2_diff(gi[c >> 1], m->G[SB * w + s]);
                        sk[2 * j + u][c] = in[c >> 1] && s < r ? bi[c >> 1] * l * sk[2 * j + u][c] : 0.f;
                        sq[2 * j + u][c] = in[c >> 1] && s <= r ? p.scale * l * sq[2 * j + u][c] : 0.f;
                    }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        *reinterpret_cast<float2 *>(&m->diag[w][(g + 8 * c) * LD + 8 * u + q2]) =
                            make_float2(sk[2 * j + u][2 * c], sk[2 * j + u][2 * c + 1]);
            }
            to_left(P[j], sq[2 * j], sq[2 * j + 1]);
        }
    }
    // (k and q have been read: what leaves goes over them)
    Left D;           // -T_ww
    {
        float *a = m->diag[w];
        float x[SB];
        if (lane < SB) {  // a column each
#pragma unroll
            for (int r = 0; r < SB; ++r) {
                float s0 = r == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                for (int k = 0; k < r; k += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(a + r * LD + k);
                    s0 = fmaf(-v.x, x[k], s0);
                    if (k + 1 < r) s1 = fmaf(-v.y, x[k + 1], s1);
                    if (k + 2 < r) s0 = fmaf(-v.z, x[k + 2], s0);
                    if (k + 3 < r) s1 = fmaf(-v.w, x[k + 3], s1);
                }
                x[r] = s0 + s1;
            }
        }
        __syncwarp();
        if (lane < SB) {
#pragma unroll
            for (int r = 0; r < SB; ++r) a[r * LD + lane] = r >= lane ? x[r] : 0.f;
        }
        __syncwarp();
        float t[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float2 be = *reinterpret_cast<const float2 *>(&m->beta[SB * w + 8 * u + q2]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float2 v = *reinterpret_cast<const float2 *>(a + (g + 8 * c) * LD + 8 * u + q2);
                t[u][2 * c] = -v.x, t[u][2 * c + 1] = -v.y;
                uint32_t hi, lo;
                split_pair(v.x * be.x, v.y * be.y, hi, lo);
                const int at = swz(i0 + 8 * c, 2 * w + u) + 2 * q2;
                *reinterpret_cast<uint32_t *>(img + OFF_T + at) = hi;
                *reinterpret_cast<uint32_t *>(img + OFF_TLO + at) = lo;
            }
        }
        to_left(D, t[0], t[1]);
    }
    {  // above the diagonal blocks: zeros
        const int r = tid & (C - 1), second = tid / C;
        for (int c = 2 * (r / SB) + 2; c < 2 * BLOCKS; ++c) {
            *reinterpret_cast<uint4 *>(img + (second ? OFF_TLO : OFF_T) + swz(r, c)) = make_uint4(0, 0, 0, 0);
            if ((c & 1) == second) *reinterpret_cast<uint4 *>(img + OFF_PT + swz(r, c)) = make_uint4(0, 0, 0, 0);
        }
    }
    if (warp == 0) {
        Decays *d = reinterpret_cast<Decays *>(img + OFF_DECAYS);
        *reinterpret_cast<float2 *>(&d->minus[2 * lane]) = make_float2(-decays[0], -decays[1]);
        *reinterpret_cast<float2 *>(&d->out[2 * lane]) = make_float2(p.scale * decays[0], p.scale * decays[1]);
        *reinterpret_cast<float2 *>(&d->after[2 * lane]) = make_float2(decays[2], decays[3]);
        if (lane == 0) d->whole = whole, d->less = less;
    }
    __syncthreads();
    // the right operand's fragments of block (k, j) of T
    auto load_t = [&](int k, int j, uint32_t(&hi)[4], uint32_t(&lo)[4]) {
        const int at = swz(SB * k + (lane & 15), 2 * j + (lane >> 4));
        ldsm_x4_t(hi, img + OFF_T + at);
        ldsm_x4_t(lo, img + OFF_TLO + at);
    };
#pragma unroll
    for (int d = 1; d < BLOCKS; ++d) {
        if (w >= d) {
            const int j = w - d;
            float r[2][4] = {};
#pragma unroll
            for (int k = 0; k < BLOCKS - 1; ++k) {
                if (k < j || k >= w) continue;
                uint32_t hi[4], lo[4];
                load_t(k, j, hi, lo);
                product(r, A[k], hi, lo);
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x, y;
                    split_pair(r[u][2 * c], r[u][2 * c + 1], x, y);
                    hi[2 * u + c] = transpose(x);
                    lo[2 * u + c] = transpose(y);
                }
            float t[2][4] = {};
            product(t, D, hi, lo);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x, y;
                    split_pair(t[u][2 * c], t[u][2 * c + 1], x, y);
                    const int at = swz(i0 + 8 * c, 2 * j + u) + 2 * q2;
                    *reinterpret_cast<uint32_t *>(img + OFF_T + at) = x;
                    *reinterpret_cast<uint32_t *>(img + OFF_TLO + at) = y;
                }
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j) {  // P T
        if (j > w) continue;
        float t[2][4] = {};
#pragma unroll
        for (int k = j; k < BLOCKS; ++k) {
            if (k > w) continue;
            uint32_t hi[4], lo[4];
            load_t(k, j, hi, lo);
            product(t, P[k], hi, lo);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                *reinterpret_cast<uint32_t *>(img + OFF_PT + swz(i0 + 8 * c, 2 * j + u) + 2 * q2) =
                    pack_bf16(t[u][2 * c], t[u][2 * c + 1]);
    }
    __syncthreads();
    // (by all threads: a bulk copy would hold the CTA for 2000 cycles more)
    uint4 *to = reinterpret_cast<uint4 *>(cp.images + (slot * p.H + h) * IMAGE);
#pragma unroll 4
    for (int i = tid; i < IMAGE / 16; i += THREADS) to[i] = reinterpret_cast<const uint4 *>(img)[i];
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
// Tensor memory columns: S; (K S)^T, under it Z, and (Q S)^T; X^T, under it X, and (P T Z)^T; the update (K^T X)^T. Of S, Z and X, 16 keys
// or tokens take 8 columns of first terms and 8 of second.
constexpr uint32_t COL_S = 0, COL_KS = 128, COL_QS = 192, COL_X = 256, COL_O = 320, COL_U = 384;

struct Misc {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t s[2], z, x;           // written; S by halves of the keys
    uint64_t ks, xs, o, u;         // MMAs complete: K S; T Z; Q S and P T Z; the update
    uint64_t drained;
    uint32_t tmem;
    int32_t abort;
};
constexpr int SMEM = OFF_MISC + static_cast<int>(sizeof(Misc)) + 1024;
static_assert(SMEM <= 227 * 1024, "one CTA's shared memory");

__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    lin::mbar_arrive_if(bar, (threadIdx.x & 31) == 0);
}
// x - a, y - b for the pair (a, b) of bf16
__device__ __forceinline__ uint32_t rest_of(f2 v, uint32_t h) {
    float x, y;
    split(v, x, y);
    asm("{\n\t.reg .b16 a, b, m;\n\tmov.b32 {a, b}, %2;\n\tmov.b16 m, 0xBF80;\n\t"  // -1
        "fma.rn.f32.bf16 %0, a, m, %0;\n\tfma.rn.f32.bf16 %1, b, m, %1;\n\t}"
        : "+f"(x), "+f"(y)
        : "r"(h));
    return pack_bf16(x, y);
}
// 16 values in two bf16 terms: 8 columns of pairs and 8 more (by two stores of 8 columns: 2 % slower)
__device__ __forceinline__ void put_split(uint32_t at, const f2 *v) {
    uint32_t x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = lin::bf16_of(v[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[8 + i] = rest_of(v[i], x[i]);
    tmem_st16(at, x);
}
// what this warp has put is there for the MMAs
__device__ __forceinline__ void hand_on(uint64_t *bar) {
    tmem_wait_st();
    tc_fence_before();
    arrive_warp(bar);
}

__device__ __forceinline__ void set_up(Misc *m) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&m->full[i], 1), mbar_init(&m->empty[i], WARPS + 1);
    for (int i = 0; i < 2; ++i) mbar_init(&m->s[i], WARPS / 2);
    mbar_init(&m->z, WARPS), mbar_init(&m->x, WARPS), mbar_init(&m->ks, 1), mbar_init(&m->xs, 1), mbar_init(&m->o, 1), mbar_init(&m->u, 1);
    mbar_init(&m->drained, 1);
    mbar_fence_init();
}

// A segment, by the whole CTA. STATES: of the pass over the states of cut sequences.
// ROUNDS: another segment may follow.
template <bool STATES, bool ROUNDS>
__device__ __forceinline__ void walk(const ChunkParams &cp, const Segment &seg, int h, unsigned char *smem, Misc *m, uint32_t tmem) {
    const Params &p = cp.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hk = h / p.rep;
    const bool is_map = STATES && seg.kind == 2;
    const int64_t chain = static_cast<int64_t>(seg.n) * p.H + h;
    const int64_t begin = p.cu[seg.n], bos = begin + static_cast<int64_t>(seg.c0) * C, eos = p.cu[seg.n + 1];  // from the segment on
    const int chunks = seg.len;

    if (warp == WARP_LOAD) {
        if (lane == 0) {
            const unsigned char *images = cp.images + (static_cast<int64_t>(seg.slot) * p.H + h) * IMAGE;
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
            else if (ROUNDS)  // the barriers are set up anew for the next segment: no arrival is left out
                for (int i = it < STAGES ? 0 : it - STAGES; i < it && ok; ++i) ok = wait(m, &m->empty[i % STAGES], (i / STAGES) & 1);
        }
    } else if (warp == WARP_MMA) {
        // The whole warp goes through the loop, so that descriptors are made in uniform registers; one lane issues.
        const uint32_t base = smem_u32(smem);
        constexpr uint32_t ID = lin::idesc_bf16(false, false, 128, 64), ID_U = lin::idesc_bf16(false, true, 128, 128);
        bool ok = true;
        uint32_t st = 0, use = 0;
#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            const uint32_t ph = it & 1, s = base + st * STAGE;
            if (!(ok = wait_warp(m, &m->full[st], use & 1))) break;
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
            const uint64_t kq = umma_desc_sw128(s + OFF_KQ, 16, 1024), tt = umma_desc_sw128(s + OFF_TT, 16, 1024);
            const uint64_t kt = umma_desc_sw128(s + OFF_KQ, PANEL, 1024);
            // (additions to the address field: bytes / 16)
            // What the chain waits for goes first, N = 64 (an MMA takes 45 to 50 cycles then, 65 to 70 with N = 128); Q S and P T Z follow
            // while the warps make Z and X.
            if (!(ok = wait_warp(m, &m->s[0], ph))) break;
            tc_fence_after();
            if (lin::elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lin::umma_ts(tmem + COL_KS, tmem + COL_S + 16 * k, kq + k * 2, ID, k > 0);
                    lin::umma_ts(tmem + COL_KS, tmem + COL_S + 16 * k + 8, kq + k * 2, ID, 1);
                }
            }
            if (!(ok = wait_warp(m, &m->s[1], ph))) break;
            tc_fence_after();
            if (lin::elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lin::umma_ts(tmem + COL_KS, tmem + COL_S + 64 + 16 * k, kq + PANEL / 16 + k * 2, ID, 1);
                    lin::umma_ts(tmem + COL_KS, tmem + COL_S + 72 + 16 * k, kq + PANEL / 16 + k * 2, ID, 1);
                }
                umma_commit(&m->ks);
                if (!STATES) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint64_t q = kq + TILE / 16 + (k >> 2) * (PANEL / 16) + (k & 3) * 2;
                        lin::umma_ts(tmem + COL_QS, tmem + COL_S + 16 * k, q, ID, k > 0);
                        lin::umma_ts(tmem + COL_QS, tmem + COL_S + 16 * k + 8, q, ID, 1);
                    }
                }
            }
            if (!(ok = wait_warp(m, &m->z, ph))) break;
            tc_fence_after();
            if (lin::elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lin::umma_ts(tmem + COL_X, tmem + COL_KS + 16 * k, tt + k * 2, ID, k > 0);
                    lin::umma_ts(tmem + COL_X, tmem + COL_KS + 16 * k + 8, tt + k * 2, ID, 1);
                    lin::umma_ts(tmem + COL_X, tmem + COL_KS + 16 * k, tt + (OFF_TL - OFF_TT) / 16 + k * 2, ID, 1);
                }
                umma_commit(&m->xs);
                if (!STATES) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        lin::umma_ts(tmem + COL_O, tmem + COL_KS + 16 * k, tt + TILE / 16 + k * 2, ID, k > 0);
                        lin::umma_ts(tmem + COL_O, tmem + COL_KS + 16 * k + 8, tt + TILE / 16 + k * 2, ID, 1);
                    }
                    umma_commit(&m->o);
                }
            }
            if (!(ok = wait_warp(m, &m->x, ph))) break;
            tc_fence_after();
            if (lin::elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lin::umma_ts(tmem + COL_U, tmem + COL_X + 16 * k, kt + k * 128, ID_U, k > 0);
                    lin::umma_ts(tmem + COL_U, tmem + COL_X + 16 * k + 8, kt + k * 128, ID_U, 1);
                }
                umma_commit(&m->u);
                umma_commit(&m->empty[st]);
            }
            if (++st == STAGES) st = 0, ++use;
        }
        __syncwarp();
        if (!ok) {
            if (lin::elect_one()) umma_commit(&m->drained);  // (by the lane that issued the MMAs: a commit tracks its own thread's)
            __syncwarp();
            wait_drain(&m->drained, 0);
        }
        __syncwarp();
    } else {
        const int quad = warp & 3, part = warp >> 2, half = part >> 1;
        const int val = 32 * quad + lane;  // the value column
        const uint32_t t = tmem + (static_cast<uint32_t>(32 * quad) << 16);
        const int k0 = KEYS * part, t0 = TOKS * part;
        f2 S[KEYS / 2];  // keys k0 + 2 i, k0 + 2 i + 1
        constexpr size_t STATE = DK * DV;
        {
            const float *s0 = STATES ? (seg.c0 == 0 ? p.s0 : nullptr) : p.s0;
            if (s0) s0 += chain * STATE;
            if (!STATES && seg.from >= 0) s0 = cp.states + (static_cast<size_t>(seg.from) * p.H + h) * 2 * STATE;
            if (!STATES && seg.from < -1 && s0) s0 = cp.states + (static_cast<size_t>(-2 - seg.from) * p.H + h) * 2 * STATE + STATE;
            if (s0) s0 += k0 * DV + val;
#pragma unroll
            for (int i = 0; i < KEYS / 2; ++i) {
                S[i] = s0 ? pair(s0[2 * i * DV], s0[(2 * i + 1) * DV]) : 0;
                if (is_map) S[i] = pair(k0 + 2 * i == val ? 1.f : 0.f, k0 + 2 * i + 1 == val ? 1.f : 0.f);
            }
        }
        bool ok = true;
        if (chunks > 0) {
            put_split(t + COL_S + k0, S);
            put_split(t + COL_S + k0 + 16, S + 8);
            hand_on(&m->s[half]);
        }
        int rest = static_cast<int>(eos - bos);  // tokens, from this chunk on
        uint32_t st = 0, use = 0;
#pragma unroll 1
        for (int it = 0; it < chunks; ++it, rest -= C) {
            const uint32_t ph = it & 1;
            const int left = rest < C ? rest : C;
            const unsigned char *stage = smem + st * STAGE;
            const Decays *d = reinterpret_cast<const Decays *>(stage + OFF_D);
            if (!(ok = wait_warp(m, &m->full[st], use & 1))) break;
            // (what does not depend on the MMAs is done while they run)
            const float whole = d->whole, less = d->less;
            if (less < -0.5f) {
                const f2 f = pair(whole, whole);
#pragma unroll
                for (int i = 0; i < KEYS / 2; ++i) S[i] = lin::mul2(S[i], f);
            } else {  // (a slow decay is not rounded away chunk after chunk)
                const f2 f = pair(less, less);
#pragma unroll
                for (int i = 0; i < KEYS / 2; ++i) S[i] = lin::fma2(S[i], f, S[i]);
            }
            f2 z[TOKS / 2], e[TOKS / 2];
            {
                const unsigned char *v = stage + OFF_V + (val >> 6) * TILE + t0 * 128 + (val & 7) * 2;
                const int c = (val & 63) >> 3;
                auto at = [&](int i) {
                    return static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(v + i * 128 + ((c ^ (i & 7)) << 4))) << 16;
                };
#pragma unroll
                for (int i = 0; i < TOKS / 2; ++i) z[i] = is_map ? 0 : pair(at(2 * i), at(2 * i + 1));
                if (left < C) {  // tokens behind the sequence: zeros, whatever they are; so are their rows of T and of K, and then of X
#pragma unroll
                    for (int i = 0; i < TOKS / 2; ++i) {
                        float x, y;
                        split(z[i], x, y);
                        z[i] = pair(t0 + 2 * i < left ? x : 0.f, t0 + 2 * i + 1 < left ? y : 0.f);
                    }
                }
            }
            auto load_decays = [&](const float *x) {
#pragma unroll
                for (int i = 0; i < TOKS / 4; ++i) {
                    const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(x + t0 + 4 * i);
                    e[2 * i] = u.x, e[2 * i + 1] = u.y;
                }
            };
            uint32_t r[16];
            if (!(ok = wait_warp(m, &m->ks, ph))) break;
            tc_fence_after();
            tmem_ld16(t + COL_KS + t0, r);
            load_decays(d->minus);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < TOKS / 2; ++i) z[i] = lin::fma2(e[i], pair(r[2 * i], r[2 * i + 1]), z[i]);
            put_split(t + COL_KS + t0, z);
            if (it != cp.withhold) hand_on(&m->z);
            load_decays(d->after);
            if (!(ok = wait_warp(m, &m->xs, ph))) break;
            tc_fence_after();
            tmem_ld16(t + COL_X + t0, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < TOKS / 2; ++i) z[i] = lin::mul2(e[i], pair(r[2 * i], r[2 * i + 1]));
            put_split(t + COL_X + t0, z);
            hand_on(&m->x);
            if (!STATES) {
                if (!(ok = wait_warp(m, &m->o, ph))) break;
                tc_fence_after();
                uint32_t q[16];
                tmem_ld16(t + COL_QS + t0, q);
                tmem_ld16(t + COL_O + t0, r);
                load_decays(d->out);
                tmem_wait_ld();
                tc_fence_before();
                // Two tokens of two neighbouring columns lie in two lanes: each stores both columns of one token.
                const bool odd = lane & 1;
                const int64_t ld = static_cast<int64_t>(p.H) * DV;
                __nv_bfloat16 *o = p.o + (bos + static_cast<int64_t>(it) * C + t0 + odd) * ld + h * DV + (val & ~1);
                const int mine = left - t0 - odd;  // tokens from this lane's first on
#pragma unroll
                for (int i = 0; i < TOKS / 2; ++i) {
                    const uint32_t a = lin::bf16_of(lin::fma2(e[i], pair(q[2 * i], q[2 * i + 1]), pair(r[2 * i], r[2 * i + 1])));
                    const uint32_t b = __shfl_xor_sync(0xffffffffu, a, 1);
                    const uint32_t x = odd ? __byte_perm(b, a, 0x7632) : __byte_perm(a, b, 0x5410);
                    if (2 * i < mine) *reinterpret_cast<uint32_t *>(o) = x;
                    o += 2 * ld;
                }
            }
            arrive_warp(&m->empty[st]);
            if (!(ok = wait_warp(m, &m->u, ph))) break;
            tc_fence_after();
            // the update, and the next chunk's operand: the second half of the keys is read while the first is split
            uint32_t u[2][16];
            tmem_ld16(t + COL_U + k0, u[0]);
            tmem_wait_ld();
            tmem_ld16(t + COL_U + k0 + 16, u[1]);
            const bool more = it + 1 < chunks;
#pragma unroll
            for (int i = 0; i < 8; ++i) S[i] = lin::add2(S[i], pair(u[0][2 * i], u[0][2 * i + 1]));
            if (more) put_split(t + COL_S + k0, S);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) S[8 + i] = lin::add2(S[8 + i], pair(u[1][2 * i], u[1][2 * i + 1]));
            if (more) {
                put_split(t + COL_S + k0 + 16, S + 8);
                hand_on(&m->s[half]);
            }
            if (++st == STAGES) st = 0, ++use;
        }
        if (is_map) {  // by the columns that it maps from
            if (ok) {
                float *sT = cp.states + ((static_cast<size_t>(seg.to) * p.H + h) * 2 + 1) * STATE + val * DK + k0;
#pragma unroll
                for (int i = 0; i < KEYS / 2; i += 2) {
                    float4 x;
                    split(S[i], x.x, x.y);
                    split(S[i + 1], x.z, x.w);
                    *reinterpret_cast<float4 *>(sT + 2 * i) = x;
                }
            }
        } else if (float *sT = STATES ? cp.states + (static_cast<size_t>(seg.to) * p.H + h) * 2 * STATE
                                      : seg.kind == 0 && p.sT ? p.sT + chain * STATE : nullptr;
                   sT && ok) {
            sT += k0 * DV + val;
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
}

// The outputs' CTAs have a segment each; those of the pass over the states, no more of them than SMs, one in each round, there and back,
// as long ones are listed first. So have those of the outputs' jobs from `from` on: where most sequences run token after token, and the host
// does not know how many do not, only the first jobs have a CTA each (16,384 that end at once take 75 us). (Where no sequence is cut, this
// launch and the join's end at once, the sooner the fewer CTAs they have:
// with one for each segment and for each part of the join's columns they took 4.9 us of 16 x 64 tokens and 16 heads, 9.6 of 8 x 1024 and
// 7.6 of 4 x 2048, and as many as SMs 2.5, 4.8 and 6.0. The outputs' CTAs in rounds as well took 9 to 18 % longer for a chunk: the loop
// costs registers.)
template <bool STATES, bool ROUNDS>
__global__ void __launch_bounds__(THREADS, 1) kda_gated_delta_chunk_kernel(const __grid_constant__ ChunkParams cp) {
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    Misc *m = reinterpret_cast<Misc *>(smem + OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, H = cp.a.H;
    if (tid == 0) {
        set_up(m);
        m->abort = 0;
    }
    const int from = ROUNDS && !STATES ? cp.from : 0;
    int index = from + static_cast<int>(blockIdx.x);
    let_next_launch();
    wait_for_launch();
    const Segment *segs = STATES ? cp.segs_s : cp.segs;  // (the plan's)
    const int jobs = cp.counts[STATES ? 1 : 0] * H;
    if (index >= jobs) return;
    Segment seg = segs[index / H];
    if (warp == WARP_MMA) tmem_alloc(&m->tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem;
    walk<STATES, ROUNDS>(cp, seg, index % H, smem, m, tmem);
    if (ROUNDS) {
#pragma unroll 1
        for (int round = 1;; ++round) {
            index = from + round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            if (index >= jobs || m->abort) break;
            if (tid == 0) {  // (every arrival has come)
                for (uint64_t *bar = m->full; bar <= &m->drained; ++bar) lin::mbar_inval(bar);
                set_up(m);
            }
            seg = segs[index / H];
            __syncthreads();
            walk<STATES, ROUNDS>(cp, seg, index % H, smem, m, tmem);
        }
    }
    if (tid == 0 && m->abort) set_status(cp.a.status, KDA_ERR_TIMEOUT);
    if (warp == WARP_MMA) tmem_dealloc(tmem, 512);
}

}  // namespace walk

// ------------------------------------------------------------------ between the passes: the states that the parts begin with
namespace join {

constexpr int COLS = 8, PARTS = DV / COLS;
constexpr int KEYS = 2, SHARES = 8, SHARE = DK / SHARES, THREADS = DK / KEYS * SHARES;
constexpr int STAGES = 2;
struct Shared {
    alignas(16) float F[STAGES][DK][DK];         // maps, transposed
    alignas(16) float E[DK][COLS];
    alignas(16) float sums[SHARES][2][DK][COLS / 2];  // by halves of the columns: neighbouring keys are neighbours
};
static_assert(COLS == 8, "two halves of four columns");

__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups() {  // for all but the last N
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// After a cut, E = F E' + N, with E' the state after the cut before, F the map of the part between them and N its state from zero. One
// CTA has 8 value columns of a sequence and head, and an SM's registers; a thread two keys and an eighth of the sum's terms. fp32
// throughout, the sums in one order. One cut waits for the one before; F (64 KB) comes two cuts ahead. 37 cuts of 4 heads: 58 us, 1.6 a
// cut, the time of a thread's 260 instructions at four warps a scheduler. (F in registers, one cut ahead: 65 us. Three tf32 products on
// mma.sync, with F split by each CTA: 74.)
__global__ void __launch_bounds__(THREADS, 1) kda_gated_delta_join_kernel(const __grid_constant__ ChunkParams cp) {
    extern __shared__ __align__(16) unsigned char raw[];
    Shared *m = reinterpret_cast<Shared *>(raw);
    const int key = threadIdx.x % (DK / KEYS), share = threadIdx.x / (DK / KEYS);  // keys key and key + 64
    const int mk = threadIdx.x / 4, mc = 2 * (threadIdx.x % 4);  // this thread's two columns of E and N
    constexpr size_t STATE = DK * DV;
    const size_t step = 2 * STATE * cp.a.H;
    let_next_launch();
    wait_for_launch();
    const int64_t jobs = static_cast<int64_t>(cp.counts[2]) * cp.a.H * PARTS;
#pragma unroll 1
    for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const int part = static_cast<int>(job % PARTS), h = static_cast<int>(job / PARTS % cp.a.H);
        const Cuts cuts = cp.cuts[job / PARTS / cp.a.H];
        float *at = cp.states + (static_cast<size_t>(cuts.first) * cp.a.H + h) * 2 * STATE;
        const size_t mine = static_cast<size_t>(mk) * DV + COLS * part + mc;
        if (const float *s0 = cp.a.s0)
            *reinterpret_cast<float2 *>(at + STATE + mine) =
                *reinterpret_cast<const float2 *>(s0 + (static_cast<int64_t>(cuts.n) * cp.a.H + h) * STATE + mine);
        auto load = [&](int s) {  // cut s's map
            if (s < cuts.count) {
                const float *from = at + step * s + STATE + 4 * threadIdx.x;
                float *to = &m->F[s % STAGES][0][0] + 4 * threadIdx.x;
#pragma unroll
                for (int i = 0; i < DK * DK / 4 / THREADS; ++i) copy16(to + 4 * THREADS * i, from + 4 * THREADS * i);
            }
            end_group();
        };
        auto load_n = [&](int s) {
            return s < cuts.count ? *reinterpret_cast<const float2 *>(at + step * s + mine) : make_float2(0.f, 0.f);
        };
        load(1);
        load(2);
        float2 n = load_n(0), ahead = load_n(1);
        *reinterpret_cast<float2 *>(&m->E[mk][mc]) = n;
#pragma unroll 1
        for (int s = 1; s < cuts.count; ++s) {
            n = ahead;
            ahead = load_n(s + 1);
            wait_groups<1>();
            __syncthreads();
            const float(*F)[DK] = m->F[s % STAGES] + SHARE * share;
            f2 x[KEYS][COLS / 2];
#pragma unroll
            for (int k = 0; k < KEYS; ++k)
#pragma unroll
                for (int c = 0; c < COLS / 2; ++c) x[k][c] = 0;
#pragma unroll
            for (int j = 0; j < SHARE; ++j) {
                const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(&m->E[SHARE * share + j][0]);
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&m->E[SHARE * share + j][4]);
#pragma unroll
                for (int k = 0; k < KEYS; ++k) {
                    const float f = F[j][key + k * (DK / KEYS)];
                    const f2 a = pair(f, f);
                    x[k][0] = lin::fma2(a, u.x, x[k][0]);
                    x[k][1] = lin::fma2(a, u.y, x[k][1]);
                    x[k][2] = lin::fma2(a, v.x, x[k][2]);
                    x[k][3] = lin::fma2(a, v.y, x[k][3]);
                }
            }
#pragma unroll
            for (int k = 0; k < KEYS; ++k)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    *reinterpret_cast<ulonglong2 *>(m->sums[share][half][key + k * (DK / KEYS)]) =
                        make_ulonglong2(x[k][2 * half], x[k][2 * half + 1]);
            __syncthreads();
            load(s + 2);
#pragma unroll
            for (int r = 0; r < SHARES; ++r) {
                const float2 u = *reinterpret_cast<const float2 *>(&m->sums[r][mc / 4][mk][mc % 4]);
                n.x += u.x;
                n.y += u.y;
            }
            *reinterpret_cast<float2 *>(at + step * s + mine) = n;
            *reinterpret_cast<float2 *>(&m->E[mk][mc]) = n;
        }
    }
}

}  // namespace join

// [tokens][heads][128] bf16 with a token stride; boxes of 64 channels x 1 head x 64 tokens
bool encode_heads(CUtensorMap *m, const __nv_bfloat16 *x, int64_t tokens, int heads, int64_t stride) {
    const cuuint64_t dims[3] = {DK, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {DK * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, 1, C};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, 3, dims, strides, box);
}

// The shortest cut worth a try, an SM's share of all chunks; 0 where none pays, which spares two launches (3 us of the 112 of
// 4 x 2048 tokens and 16 heads, where the host cannot rule it out). Cuts gain most where one sequence holds all tokens: if none pays for
// that one, none is tried.
int shortest_cut(int64_t N, int64_t T, int64_t H, int sms) {
    const int64_t longest = (T + C - 1) / C, all = (T / C + N) * H;
    int64_t len = (all + sms - 1) / sms;
    if (len < 4) len = 4;
    auto time = [&](int cut) {
        plan::Work out{0, 0, 0, 0}, states{0, 0, 0, 0};
        int most = 0;
        plan::add_sequence(out, states, most, static_cast<int>(longest), cut);
        return plan::time_of(out, states, most, static_cast<int>(H), sms);
    };
    bool pays = false;
    for (int i = 0; i < plan::CUTS; ++i) {
        const int cut = plan::cut_length(i, static_cast<int>(len));
        pays |= cut < longest && time(cut) < time(0x7fffffff);
    }
    return pays ? static_cast<int>(len) : 0;
}

// Batches of few tokens a sequence run the recurrence, which takes a time for each token where a chunk takes the same for 1 as for 64. In
// us, the recurrence and chunks: 256 sequences of 8 tokens, 4 heads 47 and 72, of 16 79 and 74, of 24 112 and 75; 16 heads 168 and 262, 275
// and 268, 386 and 274; 32 heads 315 and 522, 523 and 529, 745 and 534. 1024 of 16, 16 heads 1022 and 1041; 64 of 16, 1, 16 and 96 heads 17
// and 19, 77 and 70, 397 and 410; 16 of 16, 16 heads 27 and 23 (the furthest from the better).
// A batch of so few tokens on average may hold long sequences among many short ones (prompts among single tokens), and the host does
// not know: those of more than FEW_LONGEST tokens run as chunks all the same. The recurrence's launch lists their chunks; where there are none,
// the launches behind it take 5 us of 16 sequences of 16 tokens, 17 of 256 and 50 of 4096 (16 heads; the sequences themselves 21, 260 and 3990).
bool few_tokens(int64_t N, int64_t T) { return T <= 16 * N; }
constexpr int FEW_LONGEST = KDA_DECODE_MAX_TOKENS;  // what the recurrence's own entry point takes
constexpr int OWN_CTAS = 4;  // of the outputs' pass with a segment of their own, an SM
int64_t most_long(int64_t N, int64_t T) { return T / (FEW_LONGEST + 1) < N ? T / (FEW_LONGEST + 1) : N; }

struct Layout {
    int64_t slots, segs, cuts;  // of chunks; parts: ceil(c / L) <= c' / L + 1 summed over the sequences; cuts: (c - 1) / L
    int shortest;
    size_t images, list, seg, seg_s, cut, states, bytes;
};
Layout layout_of(int64_t N, int64_t T, int64_t H, int sms) {
    Layout l;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const bool few = few_tokens(N, T);
    if (few) N = most_long(N, T);
    l.shortest = shortest_cut(N, T, H, sms);
    l.slots = T / C + N;
    l.cuts = l.shortest ? T / (static_cast<int64_t>(C) * l.shortest) : 0;
    l.segs = N + l.cuts;
    l.images = 256;
    l.list = up(l.images + static_cast<size_t>(l.slots * H) * IMAGE);
    l.seg = up(l.list + (few ? sizeof(int2) * l.slots : 0));
    l.seg_s = up(l.seg + sizeof(Segment) * l.segs);
    l.cut = up(l.seg_s + sizeof(Segment) * 2 * l.cuts);
    l.states = up(l.cut + sizeof(Cuts) * l.cuts);
    l.bytes = l.states + sizeof(float) * 2 * DK * DV * static_cast<size_t>(l.cuts * H);
    return l;
}
// nothing runs as chunks
bool recurrence_only(int64_t N, int64_t T) { return T < 1 || (few_tokens(N, T) && T <= FEW_LONGEST); }

// `after`: its CTAs may be set up while the launch before ends (they wait for it before they read what it wrote).
cudaError_t launch(void (*kernel)(ChunkParams), int64_t ctas, int threads, int smem, bool after, const ChunkParams &p, cudaStream_t stream) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

size_t chunked_workspace_bytes(int64_t N, int64_t T, int64_t H) {
    const int sms = sm_count();
    return sms < 1 || recurrence_only(N, T) ? 0 : layout_of(N, T, H, sms).bytes;
}

cudaError_t launch_chunked(const Params &a, void *workspace, cudaStream_t stream, int withhold) {
    if (recurrence_only(a.N, a.T)) return launch_recurrent(a, stream);
    const int sms = sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    ChunkParams p{};
    p.a = a;
    const int hk = a.H / a.rep;
    if (!encode_heads(&p.tq, a.q, a.T, hk, a.qs) || !encode_heads(&p.tk, a.k, a.T, hk, a.ks) ||
        !encode_heads(&p.tv, a.v, a.T, a.H, a.vs))
        return cudaErrorInvalidValue;
    p.withhold = withhold;
    const bool few = few_tokens(a.N, a.T);
    p.longer = few ? FEW_LONGEST : -1;
    const Layout l = layout_of(a.N, a.T, a.H, sms);
    p.shortest = l.shortest;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    p.counts = reinterpret_cast<int32_t *>(ws);
    int32_t *listed = p.counts + 4;
    int2 *list = reinterpret_cast<int2 *>(ws + l.list);
    p.listed = listed;
    p.list = list;
    p.images = ws + l.images;
    p.slots = l.slots;
    p.sms = sms;
    p.segs = reinterpret_cast<Segment *>(ws + l.seg);
    p.segs_s = reinterpret_cast<Segment *>(ws + l.seg_s);
    p.cuts = reinterpret_cast<Cuts *>(ws + l.cut);
    p.states = reinterpret_cast<float *>(ws + l.states);
    cudaError_t e = cudaSuccess;
    if (few) {
        Params rest = a;
        rest.longest = FEW_LONGEST;
        rest.listed = listed;
        rest.list = list;
        rest.most = l.slots;
        e = launch_recurrent(rest, stream);
        if (e != cudaSuccess) return e;
    }
    e = launch(prep::kda_gated_delta_prepare_kernel, 1 + l.slots * a.H + prep::spare_ctas(a.N, a.H, sms), prep::THREADS, prep::SMEM, false, p, stream);
    if (e == cudaSuccess && p.shortest) {
        const int64_t parts = 2 * l.cuts * a.H, joins = (l.cuts < a.N ? l.cuts : a.N) * a.H * join::PARTS;
        e = launch(walk::kda_gated_delta_chunk_kernel<true, true>, parts < sms ? parts : sms, walk::THREADS, walk::SMEM, true, p, stream);
        if (e == cudaSuccess)
            e = launch(join::kda_gated_delta_join_kernel, joins < sms ? joins : sms, join::THREADS, sizeof(join::Shared), true, p, stream);
    }
    // (a long sequence among many short ones needs few of the CTAs that there might have to be)
    const int64_t jobs = l.segs * a.H, own = few && jobs > OWN_CTAS * sms ? OWN_CTAS * sms : jobs;
    if (e == cudaSuccess) e = launch(walk::kda_gated_delta_chunk_kernel<false, false>, own, walk::THREADS, walk::SMEM, true, p, stream);
    if (e == cudaSuccess && own < jobs) {
        p.from = static_cast<int32_t>(own);
        e = launch(walk::kda_gated_delta_chunk_kernel<false, true>, sms, walk::THREADS, walk::SMEM, true, p, stream);
    }
    return e;
}

}  // namespace delta
}  // namespace kda
