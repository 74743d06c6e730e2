// Chunked form of the linear attention with one decay per head (kda_linear_chunk_fwd) on tcgen05.
//
// For a chunk of 128 tokens with G_i the sum of its g up to token i (all g <= 0):
//     A    = q k^T                                MMA, 128 x 128 x 128, into tensor memory
//     P_ij = [j <= i] e^{G_i - G_j} A_ij          bf16, over A
//     O    = diag(e^G) q S + P v                  two MMAs into one accumulator, S in bf16
//     U^T  = v~^T k,  v~_j = e^{G_end - G_j} v_j  MMA, v~ in two bf16 terms
//     S    = e^{G_end} S + U                      fp32 registers
//
// A CTA per SM walks (segment, head) tasks: a segment is a sequence or, where there are few, a part of one. Roles run side by
// side, each a chunk or two ahead of the next:
//   load    one thread: q, k and v tiles by TMA into a ring of six 32 KB tiles, two chunks of the three kinds
//   decays  one warp: the chunk's decay tables from g
//   v~      8 warps: v~, transposed into tensor memory, in stages of 32 tokens
//   scores  8 warps: P, and half of o
//   state   8 warps: S, and the other half of o; o leaves by TMA from the chunk's q tile
//   MMAs    one warp for q k^T, q S and P v, one for U
//
// Why this split. U does not depend on S, so the recurrence from chunk to chunk is one fused multiply-add per state element and
// its rounding to bf16 for the next q S: S stays in fp32 registers (two threads share a value column) and is never accumulated
// by the tensor cores over many chunks. v~ in two bf16 terms, both multiplied by the exact bf16 k, keeps the final state within
// 4e-6 (relative, against 64 bits; one term: 2e-3; three: 2e-7, and 10 to 13 % more time); P and the copy of S that q
// multiplies are rounded once to bf16, like o.
//
// Decays: every factor is 2^x with x a sum of same-signed terms that starts at the nearer end (prefixes within 32 tokens,
// suffixes within 32 tokens plus whole-block totals), so its absolute error is a few units in the last place of x itself, never
// of the chunk's total, and no factor exceeds 1 (but see EASY). Scores between tokens of one block of 32 are the exception: their x
// is the difference of two prefixes from the block's start, off by a few units in the last place of those. That is 1e-5 where the
// block forgets once, and 5e-4 at most (32 tokens of -inf): below the rounding of P.
//
// Cut sequences (one or few long prompts): a launch makes the segments' states from zero (v, k and g alone), joins them to entry
// states, E' = decay E + N, and then makes the outputs. That reads k and v twice, and takes 1.7 us more a chunk.
//
// Bound by latency: one chunk takes an SM 2.6 us, with 1.5 us of MMAs and 0.8 us of memory at an SM's share. The chain is
// q k^T -> P (1.2 us) -> P v (0.6) -> o (0.4) -> q k^T of the next chunk (0.4), because P lies over the scores: q k^T waits behind P v.
// (Columns of P's own would need v~ in two stages instead of four.) 4 sequences of 2048, 16 heads (64 tasks): 50 us; 8 of 2048: 56 us,
// 4.9 TB/s; one of 65536, 4 heads (cut in 37): 105 us; one of 16384, 96 heads: 356 us, 4.6 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include <atomic>
#include <cmath>

#include "kda.h"
#include "kda_linear.cuh"
#include "kda_linear.h"

namespace kda {
namespace lin {

namespace {

constexpr int C = CHUNK;
constexpr int TILE = C * DK * 2;  // one 128 x 128 bf16 tile: two panels of 64 channels, 128-byte rows, swizzled
constexpr int PANEL = TILE / 2;
constexpr int TILES = 6;
constexpr int OFF_S = TILES * TILE;   // bf16 copy of S: [value][key], two panels of 64 keys
constexpr int STAGES = 4, STAGE_ROWS = C / STAGES;  // stages of a chunk's v~
constexpr int OFF_MISC = OFF_S + TILE;

struct ChunkParams {
    Params a;
    CUtensorMap tq, tk, tv, to;
    int32_t tasks;  // WHOLE: (sequence, head) pairs
    Withhold withhold;
    // the rest only with segments (device memory in the workspace)
    int32_t seg_chunks;  // shortest cut that the workspace is sized for
    int32_t most_segs;   // that the workspace holds
    int32_t most_slots;  // states of cut sequences' segments that it holds
    int32_t sms;
    int32_t *counts;     // [0] segments, [1] barrier between the passes, [2] segments of the pass over the states (0: nothing is cut),
                         // [3] CTAs that have the plan, [6] sequences to join
    unsigned long long *go, token;  // the plan is there
    int2 *first;         // first slot and number of segments of each sequence to join
    Segment *segs;       // the segments, long ones first
    Segment *segs_s;     // those of the pass over the states, long ones first
    float *decays;       // [slot][head], as decay_factor() gives them
    float *states;       // [slot][head][128][128]
};

struct Misc {
    uint64_t full[6];                 // a tile has come, by its kind and its chunk's number
    uint64_t empty[TILES];            // a slot is free
    uint64_t qk, qs, u, o, vfree[STAGES];  // tensor core -> warps (commits)
    uint64_t decw[2], dect;           // decay tables written: w and factor; tab, pre and start
    uint64_t vt[STAGES], s, p;        // v~ stage, bf16 state, scores written (and q S scaled)
    uint64_t wfree[2], zeroed;        // w read; rows behind a segment zeroed
    uint64_t go;                      // the first g have been read
    uint64_t ufree;                   // U read
    uint64_t ofree;                   // O read, and written to the q tile
    uint32_t tmem;                    // address of the tensor memory
    int32_t abort;                    // a wait ran out
    int32_t easy;                     // this chunk's decay is above EASY
    int32_t products;                 // -1, or how many chunks' P v have been issued in all (their warp has ended)
    // slow chunks (EASY): tab[j] = 2^-(sum of g up to j), pre[j] = log2 sum of g up to j, start = 0; others: tab, for anchors
    // 1..3 from tab_at(), 2^(sum of g after j up to the start of block a), j before it, and pre the log2 prefix within j's block
    alignas(16) float tab[192];
    alignas(16) float pre[C];
    alignas(16) uint32_t w[2][C];     // 2^(sum of g after j up to the chunk's end), a chunk ahead: for a pair of tokens two bf16
                                      // values and what they leave, in bf16
    float start[4];                   // log2 sum of g up to the start of each block
    float factor[4];                  // the chunk's decay as decay_factor() gives it, of the last four chunks
};
__host__ __device__ constexpr int tab_at(int anchor) { return anchor == 1 ? 0 : anchor == 2 ? 32 : 96; }
static_assert(offsetof(Misc, tab) % 16 == 0 && offsetof(Misc, pre) % 16 == 0 && offsetof(Misc, w) % 16 == 0 && OFF_MISC % 16 == 0,
              "read as float4");
constexpr int SMEM = OFF_MISC + static_cast<int>(sizeof(Misc));
static_assert(SMEM <= 227 * 1024, "one CTA's shared memory");

// tensor memory columns: q k^T, and P in the first half of each block's; the outputs; U; v~ (hi of 128 tokens, then lo)
constexpr uint32_t COL_QK = 0, COL_O = 128, COL_U = 256, COL_VT = 384;
// warps: 0-7 scores, 8-15 state, 16-23 v~, then one each
constexpr int GROUP = 256;
constexpr int WARP_LOAD = 24, WARP_DECAY = 25, WARP_MMA_OUT = 26, WARP_MMA_U = 27, THREADS = 896;
constexpr int WARP_STORE = 4;  // of the scores' warps, the one with only masked scores
// Registers: 28 warps launch with 72; the roles' shares add up to no more.
constexpr int REGS = 72, REGS_SCORES = 72, REGS_STATE = 104, REGS_V = 48, REGS_AUX = 56;
static_assert(8 * REGS_SCORES + 8 * REGS_STATE + 8 * REGS_V + 4 * REGS_AUX <= 28 * REGS, "the launch's registers");
// A chunk whose whole decay is above 2^EASY needs no anchors: its scores are A_ij 2^-(sum of g up to j), at most 2^48 times
// their size, and the row's 2^(sum of g up to i) is left to the output, so that q S and P v add up as they are.
// (A_ij v_j must stay below 2^79 then. Without this, q S is scaled in tensor memory between the two MMAs: 4 % more a chunk.)
constexpr float EASY = -48.f;
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr int GRID_POLLS = 1 << 24;
// waits of up to WAIT_NS each before a role gives up; and before one that has given up takes its own copies for complete
constexpr int WAITS = 20000, WAITS_DRAIN = 100;
constexpr int MMAS_END = 200000;  // cycles; a chunk's MMAs, the most that are ever queued, take 3000

struct Task {
    int64_t t0;
    int32_t len, h;
    const float *sin;  // NULL: zeros
    float *sout;       // NULL: not wanted
    float *decay;      // NULL, or where the segment's decay_factor() goes
    bool skip;
};

// The roles' code is shared by the two passes of a launch with segments (SEG): `states` is true in the first. One copy of each:
// an SM's instruction cache holds about one copy of all roles, and a role's first run through cold code costs as much as two
// chunks.
template <bool SEG>
__device__ __forceinline__ int tasks_of(const ChunkParams &p, bool states) {
    return SEG ? p.counts[states ? 2 : 0] * p.a.H : p.tasks;
}
// The CTA's k-th task. Segments are sorted by length: back and forth over the CTAs, each gets about the same number of chunks.
__device__ __forceinline__ int nth_task(int k, int cta, int ctas) { return k * ctas + (k & 1 ? ctas - 1 - cta : cta); }
template <bool SEG>
__device__ __forceinline__ int nth_task(int k) {
    return SEG ? nth_task(k, blockIdx.x, gridDim.x) : k * gridDim.x + blockIdx.x;
}

template <bool SEG>
__device__ __forceinline__ Task task_of(const ChunkParams &p, int id, bool states) {
    const Params &a = p.a;
    Task t;
    const int seg = id / a.H;
    t.h = id - seg * a.H;
    t.decay = nullptr;
    constexpr size_t SZ = static_cast<size_t>(DK) * DV;
    if (!SEG) {
        const int64_t b = a.cu[seg], e = a.cu[seg + 1];
        t.skip = b < 0 || e < b || e > a.T || a.cu[0] != 0;
        t.t0 = b;
        t.len = static_cast<int32_t>(e - b);
        const size_t at = static_cast<size_t>(id) * SZ;
        t.sin = a.s0 ? a.s0 + at : nullptr;
        t.sout = a.sT ? a.sT + at : nullptr;
        return t;
    }
    const Segment sg = (states ? p.segs_s : p.segs)[seg];
    t.t0 = sg.t0;
    t.len = sg.len;
    t.skip = false;
    const int own = sg.slot * a.H + t.h;
    const size_t at = (static_cast<size_t>(sg.seq) * a.H + t.h) * SZ, ws = static_cast<size_t>(own) * SZ;
    const bool last = sg.index == sg.count - 1;
    // With the states updated in place, a cut sequence's entry state is read by one
    // CTA and overwritten by another: the last segment's slot, else unused, keeps it (a task without tokens).
    const bool keep = sg.count > 1 && a.s0 && a.s0 == a.sT;
    if (states) {
        if (last) t.len = 0;
        t.sin = (last || sg.index == 0) && a.s0 ? a.s0 + at : nullptr;
        t.sout = p.states + ws;
        t.decay = p.decays + own;
    } else {
        const size_t row = static_cast<size_t>(a.H) * SZ;
        t.sin = sg.index > 0 ? p.states + ws - row : keep ? p.states + ws + (sg.count - 1) * row : a.s0 ? a.s0 + at : nullptr;
        t.sout = last && a.sT ? a.sT + at : nullptr;
    }
    return t;
}

constexpr int TQ = 0, TV = 1, TK = 2;
// The six slots hold the three tiles of two chunks, or the two (v, k) of three. A slot's barriers are numbered by the chunks
// that have used it.
__device__ __forceinline__ int slot_of(int kind, uint32_t it, bool states) {
    return states ? 2 * static_cast<int>(it % 3) + kind - TV : 3 * static_cast<int>(it % 2) + kind;
}
__device__ __forceinline__ uint32_t use_of(uint32_t it, bool states) { return states ? it / 3 : it / 2; }

// A bounded wait for a barrier's phase. (A parity wait takes the phase before
// last for the next: every role that waits on a barrier waits for each of its
// phases in turn, or has seen the one before complete through another wait.)
// False: it ran out, or another role has given up. A warp that gets false leaves its role at once: roles meet at these barriers
// alone (but see give_up), where those that stay behind give up in their turn, until all threads have come to the end of the pass.
__device__ __forceinline__ bool wait(Misc *m, uint64_t *bar, uint32_t parity) {
    int i = 0;
#pragma unroll 1
    while (!mbar_wait_some(bar, parity)) {
        if (++i == WAITS) *reinterpret_cast<volatile int32_t *>(&m->abort) = 1;
        if (*reinterpret_cast<volatile int32_t *>(&m->abort)) return false;
    }
    return true;
}
// a role that has given up waits for what it has in flight
__device__ __forceinline__ void wait_drain(uint64_t *bar, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < WAITS_DRAIN && !mbar_wait_some(bar, parity); ++i) {
    }
}
// a wait() of a whole warp, with one answer
__device__ __forceinline__ bool wait_warp(Misc *m, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(m, bar, parity));
}
// one arrival for the whole warp
__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    mbar_arrive_if(bar, (threadIdx.x & 31) == 0);
}

// g of token `row` of a chunk (0 behind the segment)
__device__ __forceinline__ float gate_raw(const Params &a, int64_t t0, int row, int left, int h) {
    if (row >= left) return 0.f;
    return __ldg(a.g + (a.g_per_token ? (t0 + row) * a.H + h : h));
}
__device__ __forceinline__ float log2_decay(float g) {  // 2^-200 is 0 in fp32; a NaN stays one and shows in what it decays
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(g * LOG2E), "f"(-200.f));
    return r;
}
// The decay 2^x of a state that many steps multiply, with all of fp32's relative precision: down to 1/2 (and for growth, which a
// gate above 0 gives) 2^x - 1, below -2^-x. (Minus one, so that a slow decay is not rounded away step after step; not for a fast one,
// whose difference from 1 has lost its last bits: at 2^-13 3 % of them, below 2^-24 all.)
__device__ __forceinline__ float decay_factor(float x) {
    const float less = expm1f(x * (1.f / LOG2E));
    return less < -0.5f ? -ex2(-x) : less;
}
__device__ __forceinline__ bool is_fast(float factor) { return factor < -0.5f; }
__device__ __forceinline__ float fast_decay(float factor) {  // (one instruction, off by one unit in the last place)
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(-factor));
    return r;
}

// Operand descriptors: a tile's own, and the step to k-block kk of 16 added to it (within the address field: no carry leaves it).
__device__ __forceinline__ uint64_t desc_k(uint32_t tile) { return umma_desc_sw128(tile, 16, 1024); }  // K-major
__device__ __forceinline__ uint64_t desc_mn(uint32_t tile, uint32_t panel) {  // MN-major: rows are k
    return umma_desc_sw128(tile, panel, 1024);
}
__device__ __forceinline__ constexpr uint64_t step_k(int kk) { return ((kk >> 2) * PANEL + (kk & 3) * 32) >> 4; }
__device__ __forceinline__ constexpr uint64_t step_mn(int kk) { return (kk * 2048) >> 4; }

// ---- one thread: tile loads, a chunk ahead (two in the pass over the states)
template <bool SEG>
__device__ __forceinline__ void role_load(const ChunkParams &p, unsigned char *smem, Misc *m, bool states) {
    const uint64_t policy = evict_first();
    uint32_t it = 0, part = 0;  // whole chunks issued, and which kinds of a chunk that was given up
    bool ok = true;
    const int tasks = tasks_of<SEG>(p, states), first = states ? TV : TQ;
#pragma unroll 1
    for (int nth = 0, id; ok && (id = nth_task<SEG>(nth)) < tasks; ++nth) {
        const Task t = task_of<SEG>(p, id, states);
        if (t.skip) continue;
        const int hk = t.h / p.a.rep;
        if (t.sin) prefetch_l2(t.sin, DK * DV * sizeof(float));  // (the state's warps come for it a chunk or two later)
#pragma unroll 1
        for (int c = 0; ok && c < t.len; c += C) {
            const int row = static_cast<int>(t.t0 + c);
            part = 0;
            // the first decay table waits for a few bytes of g: they go ahead of all SMs' first tiles
            if (it == 0 && !wait(m, &m->go, 0)) {
                ok = false;
                break;
            }
            const uint32_t use = use_of(it, states);
#pragma unroll 1
            for (int i = first; i < 3; ++i) {  // v, k, q: q's slot is free last, when an output has been stored
                const int kind = states ? i : i == 2 ? TQ : i + 1;
                const int slot = slot_of(kind, it, states);
                if (use > 0 && !wait(m, &m->empty[slot], (use - 1) & 1)) {
                    ok = false;
                    break;
                }
                unsigned char *dst = smem + slot * TILE;
                const CUtensorMap *map = kind == TV ? &p.tv : kind == TK ? &p.tk : &p.tq;
                const int head = kind == TV ? t.h : hk;
                mbar_arrive_expect_tx(&m->full[slot], TILE);
                tma_load_3d(dst, map, 0, head, row, &m->full[slot], policy);
                tma_load_3d(dst + PANEL, map, 64, head, row, &m->full[slot], policy);
                part |= 1u << kind;
            }
            if (ok) ++it, part = 0;
        }
    }
    // no copy and no commit of this CTA is in flight when it ends
    const uint32_t back = states ? 3 : 2;
#pragma unroll 1
    for (uint32_t k = it > back ? it - back : 0; k < it; ++k)
#pragma unroll 1
        for (int kind = first; ok && kind < 3; ++kind) ok = wait(m, &m->empty[slot_of(kind, k, states)], use_of(k, states) & 1);
    if (ok) return;
#pragma unroll 1
    for (uint32_t k = it > back ? it - back : 0; k <= it; ++k)
#pragma unroll 1
        for (int kind = first; kind < 3; ++kind) {
            const bool again = part >> kind & 1;  // chunk `it` has this kind's tile, where that of `it - back` was
            if (k == it ? again : !(again && k + back == it)) wait_drain(&m->full[slot_of(kind, k, states)], use_of(k, states) & 1);
        }
}

// ---- two warps: MMAs, one the scores' and the outputs' (q k^T, q S, P v), one U. Each walks the tasks as a whole warp, with
// everything that makes an address the same in all lanes, and one lane issues. (A 128 x 128 x 16 MMA runs 70 cycles; from one
// warp the waits and descriptors between groups of four or eight cost as much again.)
template <bool SEG>
__device__ __forceinline__ uint32_t role_mma_out(const ChunkParams &p, unsigned char *smem, Misc *m, uint32_t tmem) {
    constexpr bool states = false;
    constexpr uint32_t ID_KK = idesc_bf16(false, false, C, C), ID_PV = idesc_bf16(false, true, C, DV);
    uint32_t it = 0;
    const uint32_t base = smem_u32(smem);
    const uint64_t s = desc_k(base + OFF_S);
    const int tasks = __shfl_sync(0xffffffffu, tasks_of<SEG>(p, states), 0);
    tmem = __shfl_sync(0xffffffffu, tmem, 0);
#pragma unroll 1
    for (int nth = 0, id; (id = nth_task<SEG>(nth)) < tasks; ++nth) {
        const Task t = task_of<SEG>(p, id, states);
        const int len = __shfl_sync(0xffffffffu, t.skip ? 0 : t.len, 0);
#pragma unroll 1
        for (int c = 0; c < len; c += C, ++it) {
            const uint32_t ph = it & 1, up = use_of(it, states) & 1;
            const int iq = slot_of(TQ, it, states), iv = slot_of(TV, it, states), ik = slot_of(TK, it, states);
            const uint64_t q = desc_k(base + iq * TILE), k = desc_k(base + ik * TILE);
            if (!wait_warp(m, &m->full[iq], up)) return it;
            if (!wait_warp(m, &m->full[ik], up)) return it;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk) umma_f16(tmem + COL_QK, q + step_k(kk), k + step_k(kk), ID_KK, kk > 0);
                umma_commit(&m->qk);
                umma_commit(&m->empty[ik]);
            }
            if (!wait_warp(m, &m->s, ph)) return it;
            if (it > 0 && !wait_warp(m, &m->ofree, ph ^ 1)) return it;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk) umma_f16(tmem + COL_O, q + step_k(kk), s + step_k(kk), ID_KK, kk > 0);
                umma_commit(&m->qs);
            }
            // P v onto the scaled q S; after U: by then v~ has been made of v
            const uint64_t v = desc_mn(base + iv * TILE, PANEL);
            if (!wait_warp(m, &m->u, ph)) return it;
            if (!wait_warp(m, &m->p, ph)) return it;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                    umma_ts(tmem + COL_O, tmem + COL_QK + 32 * (kk >> 1) + 8 * (kk & 1), v + step_mn(kk), ID_PV, 1);
                umma_commit(&m->o);
                umma_commit(&m->empty[iv]);
            }
        }
    }
    return it;
}
template <bool SEG>
__device__ __forceinline__ void role_mma_state(const ChunkParams &p, unsigned char *smem, Misc *m, uint32_t tmem, bool states) {
    constexpr uint32_t ID_U = idesc_bf16(false, true, DV, DK);
    uint32_t it = 0;
    const uint32_t base = smem_u32(smem);
    const int tasks = __shfl_sync(0xffffffffu, tasks_of<SEG>(p, states), 0);
    tmem = __shfl_sync(0xffffffffu, tmem, 0);
#pragma unroll 1
    for (int nth = 0, id; (id = nth_task<SEG>(nth)) < tasks; ++nth) {
        const Task t = task_of<SEG>(p, id, states);
        const int len = __shfl_sync(0xffffffffu, t.skip ? 0 : t.len, 0);
#pragma unroll 1
        for (int c = 0; c < len; c += C, ++it) {
            const uint32_t ph = it & 1;
            const int iv = slot_of(TV, it, states), ik = slot_of(TK, it, states);
            const uint64_t kt = desc_mn(base + ik * TILE, PANEL);
            if (!wait_warp(m, &m->full[ik], use_of(it, states) & 1)) return;
            if (it > 0 && !wait_warp(m, &m->ufree, ph ^ 1)) return;
#pragma unroll 1
            for (int st = 0; st < STAGES; ++st) {
                const uint64_t k = kt + st * step_mn(STAGE_ROWS / 16);
                const uint32_t vt = tmem + COL_VT + st * (STAGE_ROWS / 2);
                if (!wait_warp(m, &m->vt[st], ph)) return;
                // U is not complete before the last chunk's output is read: nobody that waits for u is a phase late
                if (!states && st == STAGES - 1 && it > 0 && !wait_warp(m, &m->ofree, ph ^ 1)) return;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < STAGE_ROWS / 16; ++kk) {
                        umma_ts(tmem + COL_U, vt + 8 * kk, k + step_mn(kk), ID_U, st > 0 || kk > 0);
                        umma_ts(tmem + COL_U, vt + C / 2 + 8 * kk, k + step_mn(kk), ID_U, 1);
                    }
                    umma_commit(&m->vfree[st]);
                    if (st == STAGES - 1) {
                        umma_commit(&m->u);
                        umma_commit(&m->empty[ik]);
                        if (states) umma_commit(&m->empty[iv]);
                    }
                }
            }
        }
    }
}
// ---- one warp: decay tables. Lane l has tokens 4 l .. 4 l + 3, eight lanes a block of 32.
template <bool SEG>
__device__ __forceinline__ void role_decay(const ChunkParams &p, Misc *m, bool states) {
    const Params &a = p.a;
    const int lane = threadIdx.x & 31, in = lane & 7, block = lane >> 3;
    uint32_t it = 0;
    bool bad = false;
    const int tasks = tasks_of<SEG>(p, states);
#pragma unroll 1
    for (int nth = 0, id; (id = nth_task<SEG>(nth)) < tasks; ++nth) {
        const Task t = task_of<SEG>(p, id, states);
        if (t.skip) continue;
        float raw[4], sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[j] = gate_raw(a, t.t0, 4 * lane + j, t.len, t.h);
#pragma unroll 1
        for (int c = 0; c < t.len; c += C, ++it) {
            float pre[4], suf[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bad |= !(raw[j] <= 0.f);
                pre[j] = log2_decay(raw[j]);
            }
            if (it == 0) {
                bad = __any_sync(0xffffffffu, bad);  // (they have come)
                arrive_warp(&m->go);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) raw[j] = gate_raw(a, t.t0 + c + C, 4 * lane + j, t.len - c - C, t.h);
            suf[3] = 0.f;  // after the token, within the lane
#pragma unroll
            for (int j = 2; j >= 0; --j) suf[j] = suf[j + 1] + pre[j + 1];
            const float own = suf[0] + pre[0];
#pragma unroll
            for (int j = 1; j < 4; ++j) pre[j] += pre[j - 1];
            float up = own, down = own;  // sums over the block's lanes up to this one, from this one on
#pragma unroll
            for (int s = 1; s < 8; s <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, up, s), y = __shfl_down_sync(0xffffffffu, down, s);
                if (in >= s) up += x;
                if (in + s < 8) down += y;
            }
            float before = __shfl_up_sync(0xffffffffu, up, 1), after = __shfl_down_sync(0xffffffffu, down, 1);
            if (in == 0) before = 0.f;  // the block's lanes before this one
            if (in == 7) after = 0.f;   // and behind it
            float tot[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) tot[b] = __shfl_sync(0xffffffffu, down, 8 * b);
            const float total = (tot[0] + tot[1]) + (tot[2] + tot[3]);
            sum += total;
            float to_end = after;  // whole blocks added one by one, the nearer first
#pragma unroll
            for (int b = 1; b < 4; ++b)
                if (b > block) to_end += tot[b];
            const int buf = it & 1;
            if (it > 1 && !wait_warp(m, &m->wfree[buf], ((it >> 1) - 1) & 1)) return;
            const f2 w0 = pair(ex2(suf[0] + to_end), ex2(suf[1] + to_end)), w1 = pair(ex2(suf[2] + to_end), ex2(suf[3] + to_end));
            const uint32_t h0 = bf16_of(w0), h1 = bf16_of(w1);
            const f2 minus = pair(-1.f, -1.f);
            *reinterpret_cast<uint4 *>(&m->w[buf][4 * lane]) =
                make_uint4(h0, bf16_of(fma2(of_bf16(h0), minus, w0)), h1, bf16_of(fma2(of_bf16(h1), minus, w1)));
            // (the state's warps have read the entry of four chunks ago: U of three chunks ago came after their read, and v~ of two
            // chunks ago, whose end wfree tells, after it)
            if (lane == 0) m->factor[it & 3] = decay_factor(total);
            if (it != static_cast<uint32_t>(states ? p.withhold.states : p.withhold.outputs)) arrive_warp(&m->decw[buf]);
            if (states) continue;
            if (it > 0 && !wait_warp(m, &m->p, (it - 1) & 1)) return;
            const bool easy = total > EASY;
            if (easy) {
                float from = before;  // this block's earlier lanes, then the blocks before it
#pragma unroll
                for (int b = 2; b >= 0; --b)
                    if (b < block) from += tot[b];
                *reinterpret_cast<float4 *>(&m->tab[4 * lane]) =
                    make_float4(ex2(-pre[0] - from), ex2(-pre[1] - from), ex2(-pre[2] - from), ex2(-pre[3] - from));
                before = from;
            } else {
#pragma unroll 1
                for (int x = block + 1; x < 4; ++x) {
                    *reinterpret_cast<float4 *>(&m->tab[tab_at(x) + 4 * lane]) =
                        make_float4(ex2(suf[0] + after), ex2(suf[1] + after), ex2(suf[2] + after), ex2(suf[3] + after));
                    after += x == 1 ? tot[1] : tot[2];
                }
            }
            *reinterpret_cast<float4 *>(&m->pre[4 * lane]) =
                make_float4(pre[0] + before, pre[1] + before, pre[2] + before, pre[3] + before);
            if (lane == 0) {
                float from = 0.f;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    m->start[b] = easy ? 0.f : from;
                    from += tot[b];
                }
                m->easy = easy;
            }
            arrive_warp(&m->dect);
        }
        if (states && lane == 0) *t.decay = decay_factor(sum);
    }
    if (bad) set_status(a.status, KDA_ERR_GATE_RANGE);
}

// ---- warps 16-23: v~_j = 2^(sum of g after j) v_j in two bf16 terms, transposed into tensor memory. A warp has 32 value channels
// (its quarter of the lanes) and 16 of every 32 tokens: ldmatrix transposes 8 x 8 blocks, and a tensor-memory store of the same
// fragment shape puts each pair of tokens into its channel's lane.
// With w = a + b in bf16, off by 2^-16 w at most: h = bf16(v a), and l = bf16(v b + (v a - h)), where v a - h has no more than 8
// bits and is exact, and l, of 2^-7 v w at most, is rounded by 2^-8 of itself. So h + l is off by 3 / 2^16 of v w at most (4e-6 of
// a state in all), in three instructions for a pair of tokens; from fp32 products it took eight, and 2.3e-6.
template <bool SEG>
__device__ __forceinline__ void role_v(const ChunkParams &p, unsigned char *smem, Misc *m, uint32_t tmem, bool states) {
    const int gtid = threadIdx.x & (GROUP - 1), lane = gtid & 31, quad = (gtid >> 5) & 3, half = gtid >> 7;
    const uint32_t dst = tmem + (static_cast<uint32_t>(quad) << 21) + COL_VT + 8 * half;
    // this lane's row of the blocks: token lane % 8, channels 8 (lane / 8) .. of the quarter; swizzle: 16-byte piece ^ row % 8
    const uint32_t row0 = (quad >> 1) * PANEL + (16 * half + (lane & 7)) * 128 + (((4 * (quad & 1) + (lane >> 3)) ^ (lane & 7)) << 4);
    const int pair0 = 16 * half + 2 * (lane & 3);  // the fragments' tokens
    uint32_t it = 0, ends = 0;  // chunks, and those that a segment does not fill
    const int tasks = tasks_of<SEG>(p, states);
#pragma unroll 1
    for (int nth = 0, id; (id = nth_task<SEG>(nth)) < tasks; ++nth) {
        const Task t = task_of<SEG>(p, id, states);
        if (t.skip) continue;
#pragma unroll 1
        for (int c = 0; c < t.len; c += C, ++it) {
            const int left = t.len - c, iv = slot_of(TV, it, states), ik = slot_of(TK, it, states);
            const uint32_t up = use_of(it, states) & 1;
            unsigned char *tv = smem + iv * TILE;
            if (!wait_warp(m, &m->full[iv], up)) return;
            if (left < C) {  // rows behind the segment are someone else's: zeros in v and k
                if (!wait_warp(m, &m->full[ik], up)) return;
                unsigned char *tk = smem + ik * TILE;
#pragma unroll 1
                for (int i = gtid; i < (C - left) * 16; i += GROUP) {
                    const int at = (i & 8 ? PANEL : 0) + (left + (i >> 4)) * 128 + (i & 7) * 16;
                    *reinterpret_cast<uint4 *>(tv + at) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(tk + at) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_shared();
                arrive_warp(&m->zeroed);
                if (!wait_warp(m, &m->zeroed, ends++ & 1)) return;
            }
            if (!wait_warp(m, &m->decw[it & 1], (it >> 1) & 1)) return;
#pragma unroll 1
            for (int st = 0; st < STAGES; ++st) {
                if (it > 0 && !wait_warp(m, &m->vfree[st], (it - 1) & 1)) return;
                tc_fence_after();
                uint32_t hi[8], lo[8];  // [8 tokens][8 channels]
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t x[4];
                    ldsm_x4_t(x, tv + row0 + st * (STAGE_ROWS * 128) + g * 1024);
                    const uint2 w2 = *reinterpret_cast<const uint2 *>(&m->w[it & 1][STAGE_ROWS * st + 8 * g + pair0]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t y = mul_bf16(x[i], w2.x);
                        hi[4 * g + i] = y;
                        lo[4 * g + i] = fma_bf16(x[i], w2.y, fma_bf16(x[i], w2.x, y ^ 0x80008000u));
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // 16 lanes each
                    const uint32_t at = dst + (h << 20) + st * (STAGE_ROWS / 2);
                    tmem_st_frag2(at, hi[2 * h], hi[2 * h + 1], hi[4 + 2 * h], hi[5 + 2 * h]);
                    tmem_st_frag2(at + C / 2, lo[2 * h], lo[2 * h + 1], lo[4 + 2 * h], lo[5 + 2 * h]);
                }
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(&m->vt[st]);
            }
            arrive_warp(&m->wfree[it & 1]);
        }
    }
}

// The scores' and the state's warps meet at one named barrier, which has no limit, and where the storing warp alone waits: for a
// chunk's output in the q tile. It comes there after that chunk's P v, so every other warp has arrived at the chunk's p by then, and
// none can pass the next chunk's o before it is back. So a warp that gives up behind p still arrives for a chunk whose P v is issued,
// and for no other, and the storing warp finds just the arrivals that it waits for.
// at: what the role returned, the number of the chunk behind whose p it gave up, plus one, or 0
__device__ __forceinline__ void give_up(Misc *m, uint32_t at) {
    if (at == 0 || threadIdx.x >> 5 == WARP_STORE) return;
#pragma unroll 1
    for (int i = 0; i < GRID_POLLS; ++i) {  // (the warp of P v gives up in its turn)
        const int products = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int32_t *>(&m->products), 0);
        if (products >= 0) {
            if (static_cast<int>(at) <= products) named_bar_arrive(2, 2 * GROUP);
            return;
        }
        __nanosleep(64);
    }
}

// A chunk's output from tensor memory into the q tile, and out. The scores' and the state's warps share it: four threads a token
// row, 32 values each (half, part). False: given up.
__device__ __forceinline__ bool output_part(const ChunkParams &p, unsigned char *smem, Misc *m, uint32_t tmem_lanes, const Task &t, int c,
                                            int slot, int tid, int half, int part, float factor, uint32_t ph) {
    unsigned char *tile = smem + slot * TILE + half * PANEL;
    const int left = t.len - c, lane = threadIdx.x & 31;
    tc_fence_after();
    const f2 s2 = pair(factor, factor);
#pragma unroll 1
    for (int b = 0; b < 2; ++b) {
        uint32_t o[16];
        tmem_ld16(tmem_lanes + COL_O + 64 * half + 32 * part + 16 * b, o);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // the tile's swizzle: 16-byte piece ^ row % 8
            const int i = 8 * j;
            *reinterpret_cast<uint4 *>(tile + tid * 128 + (((4 * part + 2 * b + j) ^ (tid & 7)) << 4)) =
                make_uint4(bf16_of(mul2(s2, pair(o[i], o[i + 1]))), bf16_of(mul2(s2, pair(o[i + 2], o[i + 3]))),
                           bf16_of(mul2(s2, pair(o[i + 4], o[i + 5]))), bf16_of(mul2(s2, pair(o[i + 6], o[i + 7]))));
        }
    }
    tc_fence_before();
    arrive_warp(&m->ofree);
    if (left < C) {  // rows behind the segment are not written
        if (!wait_warp(m, &m->ofree, ph)) return false;
#pragma unroll 1
        for (int i = 128 * part + tid; i < left * 8; i += 256) {
            const int r = i >> 3, j = i & 7;
            *reinterpret_cast<uint4 *>(p.a.o + ((t.t0 + c + r) * p.a.H + t.h) * DV + 64 * half + 8 * j) =
                *reinterpret_cast<const uint4 *>(tile + r * 128 + ((j ^ (r & 7)) << 4));
        }
    } else {
        fence_proxy_async_shared();
    }
    // one warp stores a whole chunk's o and frees the tile; the others go on
    if (threadIdx.x >> 5 != WARP_STORE) {
        named_bar_arrive(2, 2 * GROUP);
    } else {
        named_bar_sync(2, 2 * GROUP);
        if (lane == 0) {
            if (left >= C) {
                const unsigned char *src = smem + slot * TILE;
                tma_store_3d(&p.to, src, 0, t.h, static_cast<int>(t.t0 + c), evict_first());
                tma_store_3d(&p.to, src + PANEL, 64, t.h, static_cast<int>(t.t0 + c), evict_first());
                bulk_commit();
                bulk_wait_read();
            }
            mbar_arrive(&m->empty[slot]);
        }
        __syncwarp();
    }
    return true;
}

// ---- warps 0-7: decayed scores. Two threads share a token row: key blocks 0 and 3, or 1 and 2.
template <bool SEG>
__device__ __forceinline__ uint32_t role_scores(const ChunkParams &p, unsigned char *smem, Misc *m, uint32_t tmem) {
    constexpr bool states = false;
    const int half = threadIdx.x >> 7, tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
    const uint32_t lanes = static_cast<uint32_t>(warp) << 21;  // TMEM lane offset 32 * warp in bits 16..31
    uint32_t it = 0;
    const int tasks = tasks_of<SEG>(p, states);
#pragma unroll 1
    for (int nth = 0, id; (id = nth_task<SEG>(nth)) < tasks; ++nth) {
        const Task t = task_of<SEG>(p, id, states);
        if (t.skip) continue;
#pragma unroll 1
        for (int c = 0; c < t.len; c += C, ++it) {
            const uint32_t ph = it & 1;
            if (!wait_warp(m, &m->dect, ph) || !wait_warp(m, &m->qk, ph)) return 0;
            tc_fence_after();
            const float pre = m->pre[tid], row = ex2(pre);
            const bool easy = m->easy;
            const float out = p.a.scale * (easy ? row : 1.f);  // what the row's output is multiplied by
            // key blocks of 32: 0 and 3, or 1 and 2
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int b = i ? 3 - half : half;
                uint32_t s[32];
                if (b <= warp) tmem_ld32(tmem + lanes + COL_QK + 32 * b, s);
                if (b > warp) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = 0;
                } else if (easy) {
                    const float4 *f = reinterpret_cast<const float4 *>(&m->tab[32 * b]);
                    const int see = b == warp ? lane : 32;
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 w = f[j];
                        const uint32_t x = bf16_of(mul2(pair(s[4 * j], s[4 * j + 1]), pair(w.x, w.y)));
                        const uint32_t y = bf16_of(mul2(pair(s[4 * j + 2], s[4 * j + 3]), pair(w.z, w.w)));
                        s[2 * j] = 4 * j + 1 <= see ? x : 4 * j <= see ? x & 0xffffu : 0u;
                        s[2 * j + 1] = 4 * j + 3 <= see ? y : 4 * j + 2 <= see ? y & 0xffffu : 0u;
                    }
                } else if (b < warp) {
                    const float4 *f = reinterpret_cast<const float4 *>(&m->tab[tab_at(warp) + 32 * b]);
                    const f2 r2 = pair(row, row);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 w = f[j];
                        s[2 * j] = bf16_of(mul2(pair(s[4 * j], s[4 * j + 1]), mul2(r2, pair(w.x, w.y))));
                        s[2 * j + 1] = bf16_of(mul2(pair(s[4 * j + 2], s[4 * j + 3]), mul2(r2, pair(w.z, w.w))));
                    }
                } else {
                    const float4 *f = reinterpret_cast<const float4 *>(&m->pre[32 * b]);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 w = f[j];
                        // (selected, not multiplied by zero: a score behind the row, and its weight, may be anything)
                        const float x = 4 * j <= lane ? __uint_as_float(s[4 * j]) * ex2(pre - w.x) : 0.f;
                        const float y = 4 * j + 1 <= lane ? __uint_as_float(s[4 * j + 1]) * ex2(pre - w.y) : 0.f;
                        const float z = 4 * j + 2 <= lane ? __uint_as_float(s[4 * j + 2]) * ex2(pre - w.z) : 0.f;
                        const float q = 4 * j + 3 <= lane ? __uint_as_float(s[4 * j + 3]) * ex2(pre - w.w) : 0.f;
                        s[2 * j] = pack_bf16(x, y);
                        s[2 * j + 1] = pack_bf16(z, q);
                    }
                }
                tmem_st16(tmem + lanes + COL_QK + 32 * b, s);  // over the scores they come from
            }
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&m->p);
            if (!wait_warp(m, &m->o, ph)) return it + 1;
            if (!output_part(p, smem, m, tmem + lanes, t, c, slot_of(TQ, it, states), tid, half, 0, out, ph)) return it + 1;
        }
    }
    if (threadIdx.x == 32 * WARP_STORE) bulk_wait_all();
    return 0;
}

// ---- warps 8-15: the state, transposed as U is. Two threads share a value column of S, one half of its keys each.
template <bool SEG>
__device__ __forceinline__ uint32_t role_state(const ChunkParams &p, unsigned char *smem, Misc *m, uint32_t tmem, bool states) {
    constexpr int NK = DK / 2;
    const Params &a = p.a;
    const int gtid = threadIdx.x - GROUP, half = gtid >> 7, tid = gtid & 127, warp = tid >> 5;
    const uint32_t lanes = static_cast<uint32_t>(warp) << 21;
    unsigned char *sS = smem + OFF_S + half * PANEL + tid * 128;
    uint32_t it = 0;
    f2 S[NK / 2];
    const int tasks = tasks_of<SEG>(p, states);
#pragma unroll 1
    for (int nth = 0, id; (id = nth_task<SEG>(nth)) < tasks; ++nth) {
        const Task t = task_of<SEG>(p, id, states);
        if (t.skip) {
            if (!SEG && gtid == 0 && t.h == 0) set_status(a.status, KDA_ERR_BAD_SEQLENS);
            continue;
        }
        const size_t at = static_cast<size_t>(half * NK) * DV + tid;  // and every 128th value behind it
        if (t.sin) {
#pragma unroll
            for (int j = 0; j < NK / 2; ++j) S[j] = pair(__ldcg(t.sin + at + 2 * j * DV), __ldcg(t.sin + at + (2 * j + 1) * DV));
        } else {
#pragma unroll
            for (int j = 0; j < NK / 2; ++j) S[j] = 0;
        }
        auto publish = [&]() {  // the bf16 copy that q multiplies
#pragma unroll
            for (int j = 0; j < NK / 8; ++j)
                *reinterpret_cast<uint4 *>(sS + ((j ^ (tid & 7)) << 4)) =
                    make_uint4(bf16_of(S[4 * j]), bf16_of(S[4 * j + 1]), bf16_of(S[4 * j + 2]), bf16_of(S[4 * j + 3]));
            fence_proxy_async_shared();
            arrive_warp(&m->s);
        };
        if (!states && t.len > 0) publish();
#pragma unroll 1
        for (int c = 0; c < t.len; c += C, ++it) {
            const uint32_t ph = it & 1;
            float out = a.scale;  // what the row's output is multiplied by
            if (!states) {
                if (!wait_warp(m, &m->dect, ph)) return 0;
                const float entry = ex2(m->pre[tid] + m->start[warp]);
                if (m->easy) {
                    out *= entry;
                } else {  // q S by the row's decay since the chunk began; P v is added onto it
                    if (!wait_warp(m, &m->qs, ph)) return 0;
                    tc_fence_after();
                    const f2 e2 = pair(entry, entry);
#pragma unroll 1
                    for (int b = 0; b < 4; ++b) {
                        uint32_t x[16];
                        tmem_ld16(tmem + lanes + COL_O + 64 * half + 16 * b, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float y, z;
                            split(mul2(e2, pair(x[2 * j], x[2 * j + 1])), y, z);
                            x[2 * j] = __float_as_uint(y);
                            x[2 * j + 1] = __float_as_uint(z);
                        }
                        tmem_st16(tmem + lanes + COL_O + 64 * half + 16 * b, x);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                arrive_warp(&m->p);
            }
            if (!wait_warp(m, &m->u, ph)) return it + 1;
            tc_fence_after();
            float less = m->factor[it & 3];
            if (is_fast(less)) {  // by itself
                const float whole = fast_decay(less);
                const f2 w2 = pair(whole, whole);
#pragma unroll
                for (int j = 0; j < NK / 2; ++j) S[j] = mul2(S[j], w2);
                less = 0.f;
            }
            const f2 d2 = pair(less, less);
#pragma unroll
            for (int b = 0; b < NK / 16; ++b) {
                uint32_t u[16];
                tmem_ld16(tmem + lanes + COL_U + NK * half + 16 * b, u);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) S[8 * b + j] = add2(fma2(S[8 * b + j], d2, S[8 * b + j]), pair(u[2 * j], u[2 * j + 1]));
            }
            tc_fence_before();
            arrive_warp(&m->ufree);
            if (!states) {
                if (!wait_warp(m, &m->qs, ph)) return it + 1;  // q has been multiplied by the last copy
                if (c + C < t.len) publish();
                if (!wait_warp(m, &m->o, ph)) return it + 1;
                if (!output_part(p, smem, m, tmem + lanes, t, c, slot_of(TQ, it, states), tid, half, 1, out, ph)) return it + 1;
            }
        }
        if (t.sout) {
#pragma unroll
            for (int j = 0; j < NK / 2; ++j) {
                float x, y;
                split(S[j], x, y);
                t.sout[at + 2 * j * DV] = x;
                t.sout[at + (2 * j + 1) * DV] = y;
            }
        }
    }
    return 0;
}

// ---- segments: between the two passes of one launch
// all threads of the CTA (from whichever role)
__device__ __forceinline__ void cta_sync() {
    __syncwarp();  // (a warp comes to a barrier as a whole)
    named_bar_sync(0, THREADS);
}
// all CTAs of the launch (one thread of each; all are resident); false: a wait ran out
__device__ __forceinline__ bool grid_sync(int32_t *count, int32_t target) {
    __threadfence();
    atomicAdd(count, 1);
#pragma unroll 1
    for (int i = 0; i < GRID_POLLS; ++i) {
        // (relaxed polls, one fence: an acquire load per poll invalidates the L1 cache each time, and the SM's next loads
        // wait for all of them)
        if (ld_relaxed(count) >= target) {
            __threadfence();
            return true;
        }
        __nanosleep(64);
    }
    return false;
}

// Entry states: E_{s+1} = decay_s E_s + N_s along a sequence, in place over the segments' states N_s. Each of the launch's
// 256 x CTAs threads takes a pair of values through all segments of a head, with BATCH loads in flight. (The first segment's
// state is whole already, and the last one's is not needed.)
__device__ __forceinline__ void join_states(const ChunkParams &p, int gtid) {
    constexpr int BATCH = 8, UNITS = DK * DV / 2;
    const int H = p.a.H;
    const size_t step = static_cast<size_t>(H) * UNITS;  // from segment to segment
#pragma unroll 1
    for (int n = 0; n < p.counts[6]; ++n) {
        const int2 f = p.first[n];
#pragma unroll 1
        for (uint32_t u = blockIdx.x * GROUP + gtid; u < static_cast<uint32_t>(H) * UNITS; u += gridDim.x * GROUP) {
            f2 *s = reinterpret_cast<f2 *>(p.states) + f.x * step + u;
            const float *d = p.decays + static_cast<int64_t>(f.x) * H + u / UNITS;
            f2 e = __ldcg(s);
#pragma unroll 1
            for (int left = f.y - 2; left > 0; left -= BATCH) {
                f2 x[BATCH];
                float dd[BATCH];
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    const int at = 1 + (j < left ? j : 0);
                    x[j] = __ldcg(s + at * step);
                    dd[j] = __ldcg(d + at * H);
                }
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    const float keep = is_fast(dd[j]) ? 0.f : 1.f, times = is_fast(dd[j]) ? fast_decay(dd[j]) : dd[j];
                    e = add2(fma2(e, pair(times, times), mul2(e, pair(keep, keep))), x[j]);
                    if (j < left) s[(1 + j) * step] = e;
                }
                s += BATCH * step;
                d += BATCH * H;
            }
        }
    }
}

constexpr int BARRIERS = offsetof(Misc, tmem) / sizeof(uint64_t);  // they come first in Misc
__device__ __forceinline__ int arrivals_of(int i, bool states) {
    constexpr int E0 = offsetof(Misc, empty) / 8, V0 = offsetof(Misc, vt) / 8, P0 = offsetof(Misc, p) / 8,
                  W0 = offsetof(Misc, wfree) / 8, U0 = offsetof(Misc, ufree) / 8;
    if (i >= E0 && i < E0 + TILES) return !states && (i - E0) % 3 == TK ? 2 : 1;  // a k tile is read by q k^T and by U
    if (i == P0 || i == U0 + 1) return 2 * GROUP / 32;                              // warps of the scores' and the state's groups
    return ((i >= V0 && i < P0) || (i >= W0 && i < W0 + 3) || i == U0) ? GROUP / 32 : 1;  // warps of one group
}
__device__ __forceinline__ void init_barriers(Misc *m, bool states) {  // warp 0
    for (int i = threadIdx.x; i < BARRIERS; i += 32) mbar_init(reinterpret_cast<uint64_t *>(m) + i, arrivals_of(i, states));
    mbar_fence_init();
}

// From the pass over the states to the pass over the outputs, for the role of thread 0 (LEADS), the state's (JOINS) and the
// others; false: the launch has given up.
template <bool LEADS, bool JOINS>
__device__ __forceinline__ bool next_pass(const ChunkParams &p, Misc *m) {
    cta_sync();
    if (LEADS && threadIdx.x == 0 && !grid_sync(p.counts + 1, gridDim.x)) m->abort = 1;
    cta_sync();
    if (JOINS) join_states(p, threadIdx.x - GROUP);
    cta_sync();
    if (LEADS && threadIdx.x < 32) {
        if (*reinterpret_cast<volatile int32_t *>(&m->abort) == 0) {
            for (int i = threadIdx.x; i < BARRIERS; i += 32) mbar_inval(reinterpret_cast<uint64_t *>(m) + i);  // (every arrival has come)
            init_barriers(m, false);
        }
        __syncwarp();
        if (threadIdx.x == 0 && !grid_sync(p.counts + 1, 2 * gridDim.x)) m->abort = 1;
    }
    cta_sync();
    return *reinterpret_cast<volatile int32_t *>(&m->abort) == 0;
}

// ---- segments: one CTA decides whether and how to cut, and sorts. Sequence n of c chunks gets ceil(c / L) segments of about
// equal length, for the L of a few that is estimated to be fastest with these lengths. The estimate of a cut into no more than
// SORTED segments is that of the busiest SM under the order in which the segments will be taken, found by sorting them; more
// segments stay in the order of the sequences, and are taken to be of average length.
constexpr int CUTS = 7, SORTED = 384, PLAN_GROUP = THREADS / CUTS;
static_assert(PLAN_GROUP == 128, "four warps a candidate");
// Fitted to 90 timings on GB300 (15 batches, each with the six cuts), in microseconds: a chunk and a task of the pass over the
// outputs and of that over the states, the outputs' chunks when memory bounds all SMs, the join and its barriers, and the join of
// a segment. Each of the 15 was within 1 % of the best of its six. (A task costs this much where tasks are few: its first chunk
// goes alone through all roles.)
constexpr float T_OUT = 2.7f, T_OUT_TASK = 9.f, T_STATES = 1.7f, T_STATES_TASK = 6.f, T_OUT_ALL = 3.2f, T_CUT = 8.f, T_JOIN = 0.2f;

__host__ __device__ inline int cut_length(int i, int shortest) {  // candidates: no cut, then 1, 1.5, 2, 3, 4, 5 times the shortest
    return i == 0 ? 0x3fffffff : i == 1 ? shortest : i == 2 ? shortest + (shortest + 1) / 2 : shortest * (i - 1);
}
__host__ __device__ inline int pieces(int c, int len) { return c <= len ? 1 : (c + len - 1) / len; }
struct Cut {
    int longest, most, tasks, all, tasks_s, all_s;  // longest segment, most segments of a sequence; segments and their chunks in either pass
};
__host__ __device__ inline float pass_time(int longest, float all, float tasks, int sms, float chunk, float task) {
    const float mean = all / fmaxf(tasks, 1.f) * chunk + task, rounds = tasks / sms;
    return fmaxf(longest * chunk + task + fmaxf(floorf(rounds) - 1.f, 0.f) * mean, ceilf(rounds) * mean);
}
__host__ __device__ inline float cut_time(const Cut &c, int H, int sms, float out, float states) {
    out = fmaxf(out, static_cast<float>(c.all) * H / sms * T_OUT_ALL);
    return c.tasks_s > 0 ? out + states + T_CUT + T_JOIN * c.most : out;
}
__host__ __device__ inline float cut_time(const Cut &c, int H, int sms) {
    const float h = static_cast<float>(H);
    return cut_time(c, H, sms, pass_time(c.longest, c.all * h, c.tasks * h, sms, T_OUT, T_OUT_TASK),
                    pass_time(c.longest, c.all_s * h, c.tasks_s * h, sms, T_STATES, T_STATES_TASK));
}

// the segments of a candidate, by number, and the numbers in order of length (tables of both passes)
struct Sorted {
    alignas(16) uint32_t key[2][SORTED];  // in either pass (outputs, states): chunks << 16 | 0xffff - number, larger ones first; 0: not in it
    uint16_t seq[SORTED], index[SORTED];
    uint16_t order[2][SORTED];            // the numbers by key
};
struct PlanShared {
    Sorted sorted[CUTS];
    Cut cuts[CUTS];
    int slots[CUTS];    // segments of cut sequences
    int slot[SORTED];   // of the chosen candidate: the first state of the (cut) sequence whose first segment has this number
    int next;           // states that have been given to sequences
    int time[CUTS][2];  // of the passes: bits of a positive float
    int warps[CUTS][PLAN_GROUP / 32];
    int count[CUTS], total_s, best, cut;  // segments of the pass over the states; sequences cut in more than two
};

// every sequence as long as the next
__device__ __forceinline__ bool equal_lengths(const ChunkParams &p) {
    const int64_t each = p.a.T / p.a.N;
    bool equal = true;
    for (int n = threadIdx.x; n <= p.a.N; n += THREADS) equal = equal && p.a.cu[n] == n * each;
    return __syncthreads_and(equal);
}

// some sequence is not left out (or its offsets say so, valid or not)
__device__ __forceinline__ bool some_longer(const ChunkParams &p) {
    bool longer = false;
    for (int n = threadIdx.x; n < p.a.N; n += THREADS) longer = longer || static_cast<int64_t>(p.a.cu[n + 1]) - p.a.cu[n] > p.a.longest;
    return __syncthreads_or(longer);
}

// all threads of one CTA; the others wait for it
__device__ __forceinline__ void plan(const ChunkParams &p, PlanShared &m) {
    const Params &a = p.a;
    const int tid = threadIdx.x, i = tid / PLAN_GROUP, x0 = tid % PLAN_GROUP;  // candidate, and thread of its group
    const int len = cut_length(i, p.seg_chunks);
    const bool start_ok = a.cu[0] == 0;
    const bool keep = a.s0 && a.s0 == a.sT;
    auto chunks = [&](int n) -> int {  // -1: no valid offsets; -2: left out
        const int64_t b = a.cu[n], e = a.cu[n + 1];
        if (!(start_ok && b >= 0 && e >= b && e <= a.T)) return -1;
        return e - b <= a.longest ? -2 : static_cast<int>((e - b + C - 1) / C);
    };
    if (tid < CUTS) m.cuts[tid] = Cut{}, m.slots[tid] = 0;
    if (tid < 2 * CUTS) m.time[tid >> 1][tid & 1] = 0;
    if (tid < CUTS) m.count[tid] = 0;
    if (tid == 0) m.total_s = m.cut = m.next = 0;
    __syncthreads();
    // each group: its candidate's segments, and the number of the first segment of each thread's sequences
    const int per = (a.N + PLAN_GROUP - 1) / PLAN_GROUP, n0 = x0 * per, n1 = n0 + per < a.N ? n0 + per : a.N;
    Cut own{};
    int mine = 0, kept = 0;  // (saturating: offsets that are no offsets can add up to anything)
    for (int n = n0; n < n1; ++n) {
        const int c = chunks(n);
        if (c < 0) continue;
        const int k = pieces(c, len), one = (c + k - 1) / k;
        mine = min(mine + k, p.most_segs + 1);
        if (k > 1) kept = min(kept + k, p.most_slots + 1);
        own.longest = max(own.longest, one);
        own.most = max(own.most, k);
        own.all += c;
        own.tasks_s += k - 1;
        own.all_s += c - one;  // (0 of a sequence that is not cut)
    }
    if (n0 < n1) {
        atomicMax(&m.cuts[i].longest, own.longest);
        atomicMax(&m.cuts[i].most, own.most);
        atomicAdd(&m.slots[i], kept);
        atomicAdd(&m.cuts[i].all, own.all);
        atomicAdd(&m.cuts[i].tasks_s, own.tasks_s);
        atomicAdd(&m.cuts[i].all_s, own.all_s);
    }
    int upto = mine;  // sums over the threads up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if ((tid & 31) >= o) upto = min(upto + y, p.most_segs + 1);
    }
    if ((tid & 31) == 31) m.warps[i][x0 >> 5] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < PLAN_GROUP / 32; ++w) {
        if (w == x0 >> 5) upto += total;
        total = min(total + m.warps[i][w], p.most_segs + 1);
    }
    const int first = upto - mine;
    // more than valid offsets can need: sequences overlap (cu_seqlens goes back), and nothing runs
    const bool overlap = __syncthreads_or(total > p.most_segs || m.slots[i] > p.most_slots);
    if (overlap) {
        if (tid == 0) {
            set_status(a.status, KDA_ERR_BAD_SEQLENS);
            p.counts[0] = p.counts[1] = p.counts[2] = 0;
        }
        return;
    }
    if (x0 == 0) m.cuts[i].tasks = total;
    Sorted &t = m.sorted[i];
    const bool sort = total <= SORTED && a.N <= 0xffff;  // (a table's entry has 16 bits)
    if (sort) {
        int at = first;
        for (int n = n0; n < n1; ++n) {
            const int c = chunks(n), k = c < 0 ? 0 : pieces(c, len);
            for (int j = 0; j < k; ++j, ++at) t.seq[at] = static_cast<uint16_t>(n), t.index[at] = static_cast<uint16_t>(j);
        }
    }
    __syncthreads();
    // the first chunk of segment j of k; and a segment's chunks in the pass over the states, where the last one of a cut sequence
    // comes without tokens, if at all, to keep the sequence's entry state
    auto begin = [](int c, int k, int j) { return j * (c / k) + min(j, c % k); };
    auto states_len = [&](int l, int k, int j) { return j < k - 1 ? l : k > 1 && keep ? 0 : -1; };
    if (sort)
        for (int x = x0; x < (total + 3 & ~3); x += PLAN_GROUP) {
            const int c = x < total ? chunks(t.seq[x]) : 0, k = pieces(c, len), j = t.index[x];
            const int l = x < total ? min(begin(c, k, j + 1) - begin(c, k, j), 0x7fff) : -1, ls = l < 0 ? -1 : states_len(l, k, j);
            t.key[0][x] = l < 0 ? 0 : l << 16 | 0xffff - x;
            t.key[1][x] = ls < 0 ? 0 : ls << 16 | 0xffff - x;
            if (ls >= 0) atomicAdd(&m.count[i], 1);
        }
    __syncthreads();
    if (sort)
        for (int x = x0; x < total; x += PLAN_GROUP)
#pragma unroll
            for (int pass = 0; pass < 2; ++pass) {
                const uint32_t own = t.key[pass][x];
                int rank = 0;
#pragma unroll 4
                for (int y = 0; y < total; y += 4) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(&t.key[pass][y]);
                    rank += (v.x > own) + (v.y > own) + (v.z > own) + (v.w > own);
                }
                if (own) t.order[pass][rank] = static_cast<uint16_t>(x);
            }
    __syncthreads();
    if (sort)
        for (int b = x0; b < 2 * p.sms; b += PLAN_GROUP) {  // both passes' tasks of every SM
            const int pass = b >= p.sms, sm = b - pass * p.sms, tasks = (pass ? m.count[i] : total) * a.H;
            float time = 0.f;
            for (int k = 0, id; (id = nth_task(k, sm, p.sms)) < tasks; ++k)
                time += (t.key[pass][t.order[pass][id / a.H]] >> 16) * (pass ? T_STATES : T_OUT) + (pass ? T_STATES_TASK : T_OUT_TASK);
            atomicMax(&m.time[i][pass], __float_as_int(time));
        }
    __syncthreads();
    if (tid == 0) {
        float least = 3.0e38f;
        m.best = 0;
        for (int j = 0; j < CUTS; ++j) {
            const Cut &c = m.cuts[j];
            const float time = c.tasks <= SORTED && a.N <= 0xffff ? cut_time(c, a.H, p.sms, __int_as_float(m.time[j][0]), __int_as_float(m.time[j][1]))
                                                 : cut_time(c, a.H, p.sms);
            if (time < least) least = time, m.best = j;
        }
    }
    __syncthreads();
    if (i == m.best) {  // the chosen candidate's group writes
        auto segment = [&](int n, int j, int slot) {
            const int64_t from = a.cu[n], to = a.cu[n + 1];
            const int c = static_cast<int>((to - from + C - 1) / C), k = pieces(c, len);
            Segment s;
            s.t0 = static_cast<int32_t>(from + static_cast<int64_t>(begin(c, k, j)) * C);
            s.len = static_cast<int32_t>(j == k - 1 ? to - s.t0 : (begin(c, k, j + 1) - begin(c, k, j)) * C);
            s.seq = n;
            s.index = j;
            s.count = k;
            s.slot = slot;
            return s;
        };
        int at = first;
        for (int n = n0; n < n1; ++n) {
            const int c = chunks(n), k = c < 0 ? 0 : pieces(c, len);
            if (c == -1) set_status(a.status, KDA_ERR_BAD_SEQLENS);
            const int slot = k > 1 ? atomicAdd(&m.next, k) : 0;
            if (k > 2) p.first[atomicAdd(&m.cut, 1)] = make_int2(slot, k);
            if (sort && k > 0) m.slot[at] = slot;
            for (int j = 0; !sort && j < k; ++j) {
                const Segment s = segment(n, j, slot + j);
                p.segs[at + j] = s;
                if (states_len(0, k, j) >= 0) p.segs_s[atomicAdd(&m.total_s, 1)] = s;
            }
            at += k;
        }
        named_bar_sync(1, PLAN_GROUP);
        auto numbered = [&](int x) {
            const int j = t.index[x];
            return segment(t.seq[x], j, m.slot[x - j] + j);
        };
        if (sort)
            for (int r = x0; r < total; r += PLAN_GROUP) {
                p.segs[r] = numbered(t.order[0][r]);
                if (r < m.count[i]) p.segs_s[r] = numbered(t.order[1][r]);
            }
        named_bar_sync(1, PLAN_GROUP);
        if (x0 == 0) {
            p.counts[0] = total;
            p.counts[1] = 0;
            p.counts[2] = sort ? m.count[i] : m.total_s;
            p.counts[6] = m.cut;
        }
    }
    fence_proxy_async_shared();  // the tiles come to the same place
}

// SEGMENTS: the plan's segments, states first if something is cut; else every sequence as a whole
template <bool SEGMENTS>
__device__ __forceinline__ void run_roles(const ChunkParams &p, unsigned char *smem) {
    Misc *m = reinterpret_cast<Misc *>(smem + OFF_MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool cut = SEGMENTS && p.counts[2] > 0;  // two passes
    if (warp == 0) {
        init_barriers(m, cut);
        m->abort = 0;
        m->products = -1;
    }
    if (warp == WARP_MMA_U) tmem_alloc(&m->tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m->tmem;
    // every role: the pass over the states, the join, the pass over the outputs; or the last alone
    if (warp < 8) {
        if (!cut || next_pass<true, false>(p, m)) give_up(m, role_scores<SEGMENTS>(p, smem, m, tmem));
    } else if (warp < 16) {
        more_registers<REGS_STATE>();
#pragma unroll 1
        for (int pass = cut ? 0 : 1; pass < 2; ++pass) {
            const uint32_t at = role_state<SEGMENTS>(p, smem, m, tmem, SEGMENTS && pass == 0);
            if (pass == 1) give_up(m, at);
            if (SEGMENTS && pass == 0 && !next_pass<false, true>(p, m)) break;
        }
    } else if (warp < 24) {
        fewer_registers<REGS_V>();
#pragma unroll 1
        for (int pass = cut ? 0 : 1; pass < 2; ++pass) {
            role_v<SEGMENTS>(p, smem, m, tmem, SEGMENTS && pass == 0);
            if (SEGMENTS && pass == 0 && !next_pass<false, false>(p, m)) break;
        }
    } else {
        fewer_registers<REGS_AUX>();
#pragma unroll 1
        for (int pass = cut ? 0 : 1; pass < 2; ++pass) {
            const bool states = SEGMENTS && pass == 0;
            if (warp == WARP_LOAD) {
                if (lane == 0) role_load<SEGMENTS>(p, smem, m, states);
            } else if (warp == WARP_DECAY) {
                role_decay<SEGMENTS>(p, m, states);
            } else if (warp == WARP_MMA_U) {
                role_mma_state<SEGMENTS>(p, smem, m, tmem, states);
            } else if (warp == WARP_MMA_OUT && !states) {
                const uint32_t products = role_mma_out<SEGMENTS>(p, smem, m, tmem);
                if (lane == 0) *reinterpret_cast<volatile int32_t *>(&m->products) = static_cast<int32_t>(products);
            }
            __syncwarp();
            if (SEGMENTS && pass == 0 && !next_pass<false, false>(p, m)) break;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && m->abort) set_status(p.a.status, KDA_ERR_TIMEOUT);
    if (warp == WARP_MMA_U) {
        if (m->abort)  // what has been issued may have nobody left that waited for it: it ends, then the CTA does
            for (const long long from = clock64(); clock64() - from < MMAS_END;) __nanosleep(1000);
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

// CTA 0 plans, and the others wait for the launch's token in the workspace, which the last of them takes away again: the memory
// may hold anything, or what an earlier launch with the same arguments left (a replayed graph). False: the wait ran out.
__device__ __forceinline__ bool wait_for_plan(const ChunkParams &p, unsigned char *smem) {
    if (blockIdx.x == 0) {
        plan(p, *reinterpret_cast<PlanShared *>(smem));
        __syncthreads();
        if (threadIdx.x == 0) {
            p.counts[3] = 0;
            __threadfence();
            *reinterpret_cast<volatile unsigned long long *>(p.go) = gridDim.x > 1 ? p.token : 0;
        }
        __syncthreads();
        return true;
    }
    bool ok = true;
    if (threadIdx.x == 0) {
        ok = false;
#pragma unroll 1
        for (int i = 0; !ok && i < GRID_POLLS; ++i) {
            ok = *reinterpret_cast<volatile unsigned long long *>(p.go) == p.token;
            if (!ok) __nanosleep(64);
        }
        __threadfence();
        if (ok && atomicAdd(p.counts + 3, 1) == gridDim.x - 2) *reinterpret_cast<volatile unsigned long long *>(p.go) = 0;
    }
    return __syncthreads_and(ok);
}

static_assert(sizeof(PlanShared) <= OFF_MISC, "the plan lies where the tiles will");
// What a launch may turn out to be. Two copies of the roles where it may be either: in the code with both passes, whole sequences
// take 10 % longer. A kernel with only one of them takes 1 to 5 % less than one with both.
enum Mode { WHOLE, PLANNED, EITHER };
template <Mode MODE>
__global__ void __launch_bounds__(THREADS, 1) kda_linear_chunk_kernel(const __grid_constant__ ChunkParams p) {
    extern __shared__ __align__(1024) unsigned char smem[];
    if (MODE == WHOLE || (MODE == EITHER && equal_lengths(p))) {
        if (MODE != PLANNED) run_roles<false>(p, smem);
    } else if (MODE != WHOLE) {
        if (MODE == PLANNED && p.a.longest >= 0 && !some_longer(p)) return;
        if (wait_for_plan(p, smem))
            run_roles<true>(p, smem);
        else if (threadIdx.x == 0)
            set_status(p.a.status, KDA_ERR_TIMEOUT);
    }
}

}  // namespace

// ------------------------------------------------------------------ host side
namespace {
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {  // looked up once through the runtime (no link to the driver library)
    static const EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}
// [tokens][heads][128] bf16 with a token stride; box 64 channels x 1 head x 128 tokens, 128-byte swizzle
bool encode(CUtensorMap *m, const __nv_bfloat16 *x, int64_t tokens, int heads, int64_t stride) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {DK, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {DK * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, 1, C}, estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16 *>(x), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int num_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return sms;
}

template <Mode MODE>
cudaError_t run(const ChunkParams &p, int64_t most_tasks, int sms, cudaStream_t stream) {
    const auto kernel = kda_linear_chunk_kernel<MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    static const int regs = [] {
        cudaFuncAttributes at{};
        return cudaFuncGetAttributes(&at, kda_linear_chunk_kernel<MODE>) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs != REGS) return cudaErrorInvalidConfiguration;  // the roles' register split adds up to this
    const int grid = static_cast<int>(most_tasks < sms ? most_tasks : sms);
    if (MODE != WHOLE) {
        void *args[] = {const_cast<ChunkParams *>(&p)};
        return cudaLaunchCooperativeKernel(reinterpret_cast<const void *>(kernel), dim3(grid), dim3(THREADS), args, SMEM, stream);
    }
    kernel<<<grid, THREADS, SMEM, stream>>>(p);
    return cudaGetLastError();
}

// Sequences of few tokens run the recurrence, which takes a time for each token where a chunk takes the same for 1 as for 128.
// 16 heads, 17 tokens each: 16 sequences 21 us and as chunks 14, 64 sequences 78 and 50, 256 sequences 276 and 178; a token
// more or less is 1.0, 3.7 and 13.5 us of the recurrence, so they meet at 9 to 10 tokens.
//
// That is for sequences of like lengths. A batch of so few tokens on average may hold long sequences beside many short ones (prompts
// among single tokens), and the host does not know. Those of more than FEW_LONGEST tokens then run as chunks, in a second launch that
// ends at once where there are none. 256 sequences of one token, 16 heads: 83.3 us with it, 81.6 without; 255 of one token and one of
// 2049: 136 us, and 1660 by the recurrence alone.
bool few_tokens(int64_t N, int64_t T) { return T <= 9 * N; }
constexpr int FEW_LONGEST = KDA_DECODE_MAX_TOKENS;  // what the recurrence's own entry point takes

// Sequences of equal lengths are estimated to be as fast whole as cut (4 x 2048, 16 heads: 50 us, cut 60). Every CTA
// then looks whether they are equal, and none plans if so: the host does not know, and a padded batch looks the same to it.
bool whole_if_equal(int64_t N, int64_t T, int64_t H, int len, int sms) {
    if (T % N) return false;
    const int64_t each = (T / N + C - 1) / C;
    auto time_of = [&](int64_t cut) {
        const int64_t k = (each + cut - 1) / cut, one = (each + k - 1) / k;
        return cut_time({static_cast<int>(one), static_cast<int>(k), static_cast<int>(k * N), static_cast<int>(each * N),
                         static_cast<int>((k - 1) * N), static_cast<int>((each - one) * N)}, static_cast<int>(H), sms);
    };
    float best = 3.0e38f;
    for (int i = 1; i < CUTS; ++i) best = std::fmin(best, time_of(cut_length(i, len)));
    return time_of(each) <= best;
}
// The shortest cut of sequences worth a try, about half an SM's share of the chunks; 0 when no sequence can be longer, or there
// is one, as fast whole.
int segment_chunks(int64_t N, int64_t T, int64_t H, int sms) {
    const int64_t longest = (T + C - 1) / C, all = (T / C + N) * H;
    int64_t len = (all + 2 * sms - 1) / (2 * sms);
    if (len < 4) len = 4;
    if (longest <= len || (N == 1 && whole_if_equal(N, T, H, static_cast<int>(len), sms))) return 0;
    return static_cast<int>(len);
}

// The same for what a batch of few tokens on average holds of long sequences, at most long_sequences(): always planned.
int64_t long_sequences(int64_t N, int64_t T) { return T / (FEW_LONGEST + 1) < N ? T / (FEW_LONGEST + 1) : N; }
int segment_chunks_of_long(int64_t longer, int64_t T, int64_t H, int sms) {
    const int len = segment_chunks(longer, T, H, sms);
    return len ? len : static_cast<int>((T + C - 1) / C);
}

struct Layout {
    int64_t most;   // segments at most: ceil(c / L) <= c' / L + 1 summed over the sequences
    int64_t slots;  // of cut sequences (c > L): ceil(c / L) <= 2 c' / L
    size_t first, segs, segs_s, decays, states, bytes;
};
Layout layout_of(int64_t N, int64_t T, int64_t H, int len) {
    Layout l;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    l.most = T / (static_cast<int64_t>(C) * len) + N;
    l.slots = 2 * T / (static_cast<int64_t>(C) * len);
    if (l.slots > l.most) l.slots = l.most;
    l.first = 256;
    l.segs = up(l.first + sizeof(int2) * N);
    l.segs_s = up(l.segs + sizeof(Segment) * l.most);
    l.decays = up(l.segs_s + sizeof(Segment) * l.most);
    l.states = up(l.decays + sizeof(float) * l.slots * H);
    l.bytes = l.states + sizeof(float) * DK * DV * l.slots * H;
    return l;
}
}  // namespace

size_t chunked_workspace_bytes(int64_t N, int64_t T, int64_t H) {
    if (N < 1 || T < 1 || H < 1) return 0;
    const bool few = few_tokens(N, T);
    if (few && T <= FEW_LONGEST) return 0;
    const int sms = num_sms();
    if (sms < 1) return 0;
    if (few) N = long_sequences(N, T);
    const int len = few ? segment_chunks_of_long(N, T, H, sms) : segment_chunks(N, T, H, sms);
    return len ? layout_of(N, T, H, len).bytes : 0;
}

cudaError_t launch_chunked(const Params &a, void *workspace, cudaStream_t stream, Withhold withhold) {
    const bool few = few_tokens(a.N, a.T);
    if (few && a.T <= FEW_LONGEST) return launch_recurrent(a, stream);
    const int sms = num_sms();
    if (sms < 1) return cudaErrorInvalidDevice;
    ChunkParams p{};
    p.a = a;
    const int64_t N = few ? long_sequences(a.N, a.T) : a.N;
    const int hk = a.H / a.rep;
    if (!encode(&p.tq, a.q, a.T, hk, a.qs) || !encode(&p.tk, a.k, a.T, hk, a.ks) || !encode(&p.tv, a.v, a.T, a.H, a.vs) ||
        !encode(&p.to, a.o, a.T, a.H, static_cast<int64_t>(a.H) * DV))
        return cudaErrorInvalidValue;
    if (few) {
        p.a.longest = FEW_LONGEST;
        const cudaError_t e = launch_recurrent(p.a, stream);
        if (e != cudaSuccess) return e;
    }
    p.seg_chunks = few ? segment_chunks_of_long(N, a.T, a.H, sms) : segment_chunks(N, a.T, a.H, sms);
    p.tasks = a.N * a.H;
    p.withhold = withhold;
    if (!p.seg_chunks) return run<WHOLE>(p, p.tasks, sms, stream);
    const Layout l = layout_of(N, a.T, a.H, p.seg_chunks);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    p.most_segs = static_cast<int32_t>(l.most);
    p.most_slots = static_cast<int32_t>(l.slots);
    p.sms = sms;
    p.counts = reinterpret_cast<int32_t *>(ws);
    p.first = reinterpret_cast<int2 *>(ws + l.first);
    p.segs = reinterpret_cast<Segment *>(ws + l.segs);
    p.segs_s = reinterpret_cast<Segment *>(ws + l.segs_s);
    p.decays = reinterpret_cast<float *>(ws + l.decays);
    p.states = reinterpret_cast<float *>(ws + l.states);
    p.go = reinterpret_cast<unsigned long long *>(ws + 32);
    static std::atomic<unsigned long long> calls{0};
    p.token = (++calls + static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(&calls))) * 0x9e3779b97f4a7c15ull;
    return !few && whole_if_equal(a.N, a.T, a.H, p.seg_chunks, sms) ? run<EITHER>(p, l.most * a.H, sms, stream)
                                                            : run<PLANNED>(p, l.most * a.H, sms, stream);
}

}  // namespace lin
}  // namespace kda
