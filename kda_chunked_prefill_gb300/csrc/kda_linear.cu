// Chunked form of the linear attention with one decay per head (kda_linear_chunk_fwd) on tcgen05.
//
// For a chunk of 128 tokens with G_i the sum of its g up to token i (all g <= 0):
//     A   = q k^T                                 MMA  [128 x 128 x 128]
//     P_ij = [j <= i] e^{G_i - G_j} A_ij          warpgroup 0, bf16 into tensor memory
//     O1  = q S,  O2 = P v                        MMA, MMA
//     o_i = scale (e^{G_i} O1_i + O2_i)           warpgroup 0
//     U   = k^T v~,  v~_j = e^{G_end - G_j} v_j   warpgroup 1 forms v~, MMA
//     S   = e^{G_end} S + U                       warpgroup 1, fp32 registers
//
// One CTA per SM walks (segment, head) tasks: a segment is a sequence or a part
// of one. Roles run side by side, each a chunk or two ahead of the next:
//   load    one thread: q, k and v tiles by TMA into a ring of five 32 KB tiles
//   decays  one warp: the chunk's decay tables from g
//   v~      8 warps: v~ in stages of 32 tokens
//   scores  8 warps: P, half of o_i
//   state   8 warps: S, the other half of o_i; o leaves from the chunk's q tile
//   MMAs    one warp for q k^T, q S and P v, one for U
//
// Why this split. U does not depend on S, so the recurrence from chunk to chunk
// is one fused multiply-add per state element and its rounding to bf16 for the
// next q S: S stays in fp32 registers (a key row shared by two threads), is
// never accumulated by the tensor cores over many chunks, and a chunk's MMAs
// are all off the critical path. v~ is split in two bf16 terms (hi + lo, both
// multiplied by the exact bf16 k), which keeps the final state within about
// 3e-6; P and the copy of S that q multiplies are rounded once to bf16, like o.
//
// Decays: every factor is 2^x with x a sum of same-signed terms that starts at
// the nearer end (prefixes within 32 tokens, suffixes within 32 tokens plus
// whole-block totals), so its absolute error is a few units in the last place of
// x itself, never of the chunk's total, and no factor exceeds 1.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include <atomic>

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
constexpr int STAGES = 2, STAGE_ROWS = C / STAGES;  // stages of a chunk's v~
constexpr int OFF_MISC = OFF_S + TILE;

struct ChunkParams {
    Params a;
    CUtensorMap tq, tk, tv, to;
    int32_t tasks;  // WHOLE: (sequence, head) pairs
    // the rest only with segments (device memory in the workspace)
    int32_t seg_chunks;
    int32_t most_segs;  // that the workspace holds
    int32_t *num_segs;  // and, behind it, the count of the launch's barrier
    int2 *first;     // [N] first segment and number of segments
    Segment *segs;
    float *decays;   // [segment][head], minus one
    float *states;   // [segment][head][128][128]
};

struct Misc {
    uint64_t full[6];                 // a tile has come, by its kind and its chunk's number
    uint64_t empty[TILES];            // a slot is free
    uint64_t qk, qs, u, o, vfree[STAGES];  // tensor core -> warps (commits)
    uint64_t decw[2], dect;           // decay tables written: w and dm1; tab, pre and start
    uint64_t vt[STAGES], s, p;        // v~ stage, bf16 state, scores written (and q S scaled, if need be)
    uint64_t wfree[2];                // w read
    uint64_t go;                      // the first g have been read
    uint64_t ufree, ofree;            // U read; O read
    uint32_t tmem;                    // address of the tensor memory
    int32_t abort;                    // a wait ran out
    int32_t easy, pad;                // this chunk's decay is above EASY
    // slow chunks (EASY): tab[j] = 2^-(sum of g up to j), pre[j] = log2 sum of g up to j, start = 0; others: tab, for anchors
    // 1..3 from tab_at(), 2^(sum of g after j up to the start of block a), j before it, and pre the log2 prefix within j's block
    alignas(16) float tab[192];
    alignas(16) float pre[C];
    alignas(16) float w[2][C];        // 2^(sum of g after j up to the chunk's end), a chunk ahead
    float start[4];                   // log2 sum of g up to the start of each block
    float dm1[4];                     // 2^(the chunk's sum) - 1, of the last four chunks
};
__host__ __device__ constexpr int tab_at(int anchor) { return anchor == 1 ? 0 : anchor == 2 ? 32 : 96; }
static_assert(offsetof(Misc, tab) % 16 == 0 && offsetof(Misc, pre) % 16 == 0 && offsetof(Misc, w) % 16 == 0 && OFF_MISC % 16 == 0,
              "read as float4");
constexpr int SMEM = OFF_MISC + static_cast<int>(sizeof(Misc));
static_assert(SMEM <= 227 * 1024, "one CTA's shared memory");

// tensor memory columns: q k^T, and P in the first half of each block's; the outputs; U; v~ (hi of 128 tokens, then lo)
constexpr uint32_t COL_QK = 0, COL_O = 128, COL_U = 256, COL_VT = 384;
// threads: four warps with a role each, then three groups of eight
constexpr int WARP_LOAD = 0, WARP_DECAY = 1, WARP_MMA_OUT = 2, WARP_MMA_U = 3;
constexpr int GROUP = 256, T_SCORES = 128, T_STATE = T_SCORES + GROUP, T_V = T_STATE + GROUP, THREADS = T_V + GROUP;
constexpr int WARP_STORE = T_SCORES / 32 + 4;  // of the scores' warps, the one with only masked scores
// Registers: 28 warps launch with 72; the roles' shares add up to no more.
constexpr int REGS = 72, REGS_SCORES = 72, REGS_STATE = 104, REGS_V = 48, REGS_AUX = 56;
static_assert(8 * REGS_SCORES + 8 * REGS_STATE + 8 * REGS_V + 4 * REGS_AUX <= 28 * REGS, "the launch's registers");
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
// A chunk whose whole decay is above 2^EASY needs no anchors: its scores are A_ij 2^-(sum of g up to j), at most 2^80 times
// their size, and the row's 2^(sum of g up to i) is left to the output, so that q S and P v add up as they are.
constexpr float EASY = -80.f;
constexpr int GRID_POLLS = 1 << 24;
constexpr int WAITS = 20000;  // waits of up to WAIT_NS each before a role gives up

struct Task {
    int64_t t0;
    int32_t len, h;
    const float *sin;  // NULL: zeros
    float *sout;       // NULL: not wanted
    float *decay;      // NULL, or where the segment's decay minus one goes
    bool skip;
};

// The roles' code is shared by the two passes of a segmented launch (SEG): `states` is true in the first. One copy of each:
// an SM's instruction cache holds about one copy of all roles, and a role's first run through cold code costs as much as
// two chunks.
template <bool SEG>
__device__ __forceinline__ int tasks_of(const ChunkParams &p) {
    return SEG ? *p.num_segs * p.a.H : p.tasks;
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
    const Segment sg = p.segs[seg];
    t.t0 = sg.t0;
    t.len = sg.len;
    const size_t at = (static_cast<size_t>(sg.seq) * a.H + t.h) * SZ, ws = static_cast<size_t>(id) * SZ;
    const bool last = sg.index == sg.count - 1;
    // With the states updated in place, a cut sequence's entry state is read by one
    // CTA and overwritten by another: the last segment's slot, else unused, keeps it.
    const bool keep = sg.count > 1 && a.s0 && a.s0 == a.sT;
    if (states) {
        t.skip = last && !keep;
        if (last) t.len = 0;
        t.sin = (last || sg.index == 0) && a.s0 ? a.s0 + at : nullptr;
        t.sout = p.states + ws;
        t.decay = p.decays + id;
    } else {
        const size_t row = static_cast<size_t>(a.H) * SZ;
        t.skip = false;
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
// False: it ran out, or another role has given up
__device__ __forceinline__ bool wait(Misc *m, uint64_t *bar, uint32_t parity) {
    int i = 0;
#pragma unroll 1
    while (!mbar_wait_some(bar, parity)) {
        if (++i == WAITS) *reinterpret_cast<volatile int32_t *>(&m->abort) = 1;
        if (*reinterpret_cast<volatile int32_t *>(&m->abort)) return false;
    }
    return true;
}
// the same for a whole warp, with one answer
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
__device__ __forceinline__ float log2_decay(float g) { return fmaxf(g * LOG2E, -200.f); }  // 2^-200 is 0 in fp32

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
    const int tasks = tasks_of<SEG>(p), first = states ? TV : TQ;
#pragma unroll 1
    for (int id = blockIdx.x; ok && id < tasks; id += gridDim.x) {
        const Task t = task_of<SEG>(p, id, states);
        if (t.skip) continue;
        const int hk = t.h / p.a.rep;
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
            if (ok) ++it;
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
    for (int kind = first; kind < 3; ++kind) {
        if (it > 0) (void)mbar_wait_some(&m->full[slot_of(kind, it - 1, states)], use_of(it - 1, states) & 1);
        if (part >> kind & 1) (void)mbar_wait_some(&m->full[slot_of(kind, it, states)], use_of(it, states) & 1);
    }
}

// ---- two warps: MMAs, one the scores' and the outputs' (q k^T, q S, P v), one U. Each walks the tasks as a whole warp, and one
// lane issues. Tile addresses are constants, by the slot as a template argument: with addresses from registers an MMA takes 140
// to 280 cycles to issue, with constants 61, and a 128 x 128 x 16 MMA runs 70.
template <int SLOT>
__device__ __forceinline__ void issue_qk(uint32_t base, Misc *m) {
    const uint64_t q = desc_k(base + SLOT * TILE), k = desc_k(base + (SLOT + TK) * TILE);
#pragma unroll
    for (int kk = 0; kk < DK / 16; ++kk) umma_f16(COL_QK, q + step_k(kk), k + step_k(kk), idesc_bf16(false, false, C, C), kk > 0);
    umma_commit(&m->qk);
    umma_commit(&m->empty[SLOT + TK]);
}
template <int SLOT>
__device__ __forceinline__ void issue_qs(uint32_t base, Misc *m) {
    const uint64_t q = desc_k(base + SLOT * TILE), s = desc_k(base + OFF_S);
#pragma unroll
    for (int kk = 0; kk < DK / 16; ++kk) umma_f16(COL_O, q + step_k(kk), s + step_k(kk), idesc_bf16(false, false, C, DV), kk > 0);
    umma_commit(&m->qs);
}
template <int SLOT>
__device__ __forceinline__ void issue_pv(uint32_t base, Misc *m) {
    const uint64_t v = desc_mn(base + (SLOT + TV) * TILE, PANEL);
#pragma unroll
    for (int kk = 0; kk < C / 16; ++kk)
        umma_ts(COL_O, COL_QK + 32 * (kk >> 1) + 8 * (kk & 1), v + step_mn(kk), idesc_bf16(false, true, C, DV), 1);
    umma_commit(&m->o);
    umma_commit(&m->empty[SLOT + TV]);
}
template <int SLOT, int ST>
__device__ __forceinline__ void issue_u(uint32_t base, Misc *m) {
    const uint64_t k = desc_mn(base + SLOT * TILE, PANEL) + step_mn(ST * STAGE_ROWS / 16);
    constexpr uint32_t VT = COL_VT + ST * (STAGE_ROWS / 2), ID = idesc_bf16(false, true, DV, DK);
#pragma unroll
    for (int kk = 0; kk < STAGE_ROWS / 16; ++kk) {
        umma_ts(COL_U, VT + 8 * kk, k + step_mn(kk), ID, ST > 0 || kk > 0);
        umma_ts(COL_U, VT + C / 2 + 8 * kk, k + step_mn(kk), ID, 1);
    }
    umma_commit(&m->vfree[ST]);
}
template <int ST>
__device__ __forceinline__ void issue_u(uint32_t base, Misc *m, int slot) {  // a k tile's slot
    if (slot == 2)
        issue_u<2, ST>(base, m);
    else if (slot == 5)
        issue_u<5, ST>(base, m);
    else if (slot == 1)
        issue_u<1, ST>(base, m);
    else
        issue_u<3, ST>(base, m);
}

template <bool SEG>
__device__ __forceinline__ void role_mma_out(const ChunkParams &p, unsigned char *smem, Misc *m) {
    constexpr bool states = false;
    uint32_t it = 0;
    const uint32_t base = smem_u32(smem);
    const int tasks = __shfl_sync(0xffffffffu, tasks_of<SEG>(p), 0);
#pragma unroll 1
    for (int id = blockIdx.x; id < tasks; id += gridDim.x) {
        const Task t = task_of<SEG>(p, id, states);
        const int len = __shfl_sync(0xffffffffu, t.skip ? 0 : t.len, 0);
#pragma unroll 1
        for (int c = 0; c < len; c += C, ++it) {
            const uint32_t ph = it & 1, up = use_of(it, states) & 1;
            if (!wait_warp(m, &m->full[slot_of(TQ, it, states)], up)) return;
            if (!wait_warp(m, &m->full[slot_of(TK, it, states)], up)) return;
            tc_fence_after();
            if (elect_one()) {
                if (ph)
                    issue_qk<3>(base, m);
                else
                    issue_qk<0>(base, m);
            }
            __syncwarp();
            if (!wait_warp(m, &m->s, ph)) return;
            if (it > 0 && !wait_warp(m, &m->ofree, ph ^ 1)) return;
            tc_fence_after();
            if (elect_one()) {
                if (ph)
                    issue_qs<3>(base, m);
                else
                    issue_qs<0>(base, m);
            }
            __syncwarp();
            // P v onto q S; after U: by then v~ has been made of v
            if (!wait_warp(m, &m->u, ph)) return;
            if (!wait_warp(m, &m->p, ph)) return;
            tc_fence_after();
            if (elect_one()) {
                if (ph)
                    issue_pv<3>(base, m);
                else
                    issue_pv<0>(base, m);
            }
            __syncwarp();
        }
    }
}
template <bool SEG>
__device__ __forceinline__ void role_mma_state(const ChunkParams &p, unsigned char *smem, Misc *m, bool states) {
    uint32_t it = 0;
    const uint32_t base = smem_u32(smem);
    const int tasks = __shfl_sync(0xffffffffu, tasks_of<SEG>(p), 0);
#pragma unroll 1
    for (int id = blockIdx.x; id < tasks; id += gridDim.x) {
        const Task t = task_of<SEG>(p, id, states);
        const int len = __shfl_sync(0xffffffffu, t.skip ? 0 : t.len, 0);
#pragma unroll 1
        for (int c = 0; c < len; c += C, ++it) {
            const uint32_t ph = it & 1;
            const int ik = slot_of(TK, it, states);
            if (!wait_warp(m, &m->full[ik], use_of(it, states) & 1)) return;
            if (it > 0 && !wait_warp(m, &m->ufree, ph ^ 1)) return;
            if (!wait_warp(m, &m->vt[0], ph)) return;
            tc_fence_after();
            if (elect_one()) issue_u<0>(base, m, ik);
            __syncwarp();
            if (!wait_warp(m, &m->vt[1], ph)) return;
            // U is not complete before the last chunk's output is read: nobody that waits for u is a phase late
            if (!states && it > 0 && !wait_warp(m, &m->ofree, ph ^ 1)) return;
            tc_fence_after();
            if (elect_one()) {
                issue_u<1>(base, m, ik);
                umma_commit(&m->u);
                umma_commit(&m->empty[ik]);
                if (states) umma_commit(&m->empty[slot_of(TV, it, states)]);
            }
            __syncwarp();
        }
    }
}
static_assert(STAGES == 2, "role_mma_state");

// ---- one warp: decay tables. Lane l has tokens 4 l .. 4 l + 3, eight lanes a block of 32.
template <bool SEG>
__device__ __forceinline__ void role_decay(const ChunkParams &p, Misc *m, bool states) {
    const Params &a = p.a;
    const int lane = threadIdx.x & 31, in = lane & 7, block = lane >> 3;
    uint32_t it = 0;
    bool bad = false;
    const int tasks = tasks_of<SEG>(p);
#pragma unroll 1
    for (int id = blockIdx.x; id < tasks; id += gridDim.x) {
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
            *reinterpret_cast<float4 *>(&m->w[buf][4 * lane]) =
                make_float4(ex2(suf[0] + to_end), ex2(suf[1] + to_end), ex2(suf[2] + to_end), ex2(suf[3] + to_end));
            // (minus one, so that a slow decay is not rounded away chunk after chunk; the state's warps have read the
            // entry of four chunks ago: the scores of two chunks ago came after their read)
            if (lane == 0) m->dm1[it & 3] = expm1f(total * (1.f / LOG2E));
            arrive_warp(&m->decw[buf]);
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
        if (states && lane == 0) *t.decay = expm1f(sum * (1.f / LOG2E));
    }
    if (bad) set_status(a.status, KDA_ERR_GATE_RANGE);
}

// ---- eight warps: v~_j = 2^(sum of g after j) v_j in two bf16 terms, transposed into tensor memory. A warp has 32 value channels
// (its quarter of the lanes) and 16 of every 32 tokens: ldmatrix transposes 8 x 8 blocks, and a tensor-memory store of the same
// fragment shape puts each pair of tokens into its channel's lane.
template <bool SEG>
__device__ __forceinline__ void role_v(const ChunkParams &p, unsigned char *smem, Misc *m, uint32_t tmem, bool states) {
    const int gtid = threadIdx.x - T_V, lane = gtid & 31, quad = (gtid >> 5) & 3, half = gtid >> 7;
    const uint32_t dst = tmem + (static_cast<uint32_t>(quad) << 21) + COL_VT + 8 * half;
    // this lane's row of the blocks: token lane % 8, channels 8 (lane / 8) .. of the quarter; swizzle: 16-byte piece ^ row % 8
    const uint32_t row0 = (quad >> 1) * PANEL + (16 * half + (lane & 7)) * 128 + (((4 * (quad & 1) + (lane >> 3)) ^ (lane & 7)) << 4);
    const int pair0 = 16 * half + 2 * (lane & 3);  // the fragments' tokens
    const f2 minus = pair(-1.f, -1.f);
    bool fail = false;  // (a warp that gives up still comes to the barriers)
    uint32_t it = 0;
    const int tasks = tasks_of<SEG>(p);
#pragma unroll 1
    for (int id = blockIdx.x; id < tasks; id += gridDim.x) {
        const Task t = task_of<SEG>(p, id, states);
        if (t.skip) continue;
#pragma unroll 1
        for (int c = 0; c < t.len; c += C, ++it) {
            const int left = t.len - c, iv = slot_of(TV, it, states), ik = slot_of(TK, it, states);
            const uint32_t up = use_of(it, states) & 1;
            unsigned char *tv = smem + iv * TILE;
            fail = fail || !wait_warp(m, &m->full[iv], up);
            if (left < C) {  // rows behind the segment are someone else's: zeros in v and k
                fail = fail || !wait_warp(m, &m->full[ik], up);
                unsigned char *tk = smem + ik * TILE;
#pragma unroll 1
                for (int i = gtid; !fail && i < (C - left) * 16; i += GROUP) {
                    const int at = (i & 8 ? PANEL : 0) + (left + (i >> 4)) * 128 + (i & 7) * 16;
                    *reinterpret_cast<uint4 *>(tv + at) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(tk + at) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_shared();
                if (named_bar_or(3, GROUP, fail)) return;
            }
            fail = fail || !wait_warp(m, &m->decw[it & 1], (it >> 1) & 1);
#pragma unroll 1
            for (int st = 0; st < STAGES; ++st) {
                fail = fail || (it > 0 && !wait_warp(m, &m->vfree[st], (it - 1) & 1));
                if (fail) break;
                tc_fence_after();
#pragma unroll 1
                for (int t0 = STAGE_ROWS * st; t0 < STAGE_ROWS * (st + 1); t0 += 32) {
                    uint32_t hi[8], lo[8];  // [8 tokens][8 channels]
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint32_t x[4];
                        ldsm_x4_t(x, tv + row0 + t0 * 128 + g * 1024);
                        const f2 w2 = *reinterpret_cast<const f2 *>(&m->w[it & 1][t0 + 8 * g + pair0]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const f2 y = mul2(of_bf16(x[i]), w2);
                            hi[4 * g + i] = bf16_of(y);
                            lo[4 * g + i] = bf16_of(fma2(of_bf16(hi[4 * g + i]), minus, y));
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // 16 lanes each
                        const uint32_t at = dst + (h << 20) + t0 / 2;
                        tmem_st_frag2(at, hi[2 * h], hi[2 * h + 1], hi[4 + 2 * h], hi[5 + 2 * h]);
                        tmem_st_frag2(at + C / 2, lo[2 * h], lo[2 * h + 1], lo[4 + 2 * h], lo[5 + 2 * h]);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(&m->vt[st]);
            }
            if (!fail) arrive_warp(&m->wfree[it & 1]);
        }
    }
}

// A chunk's output from tensor memory into the q tile, and out. The scores' and the state's warps share it: four threads a token
// row, 32 values each (half, part). True: some warp has given up. (A warp that gives up still comes to the barriers.)
__device__ __forceinline__ bool output_part(const ChunkParams &p, unsigned char *smem, Misc *m, uint32_t tmem_lanes, const Task &t, int c,
                                            int slot, int tid, int half, int part, float factor, bool fail) {
    unsigned char *tile = smem + slot * TILE + half * PANEL;
    const int left = t.len - c, lane = threadIdx.x & 31;
    if (!fail) {
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
    }
    if (left < C) {  // rows behind the segment are not written
        if (named_bar_or(1, 2 * GROUP, fail)) return true;
#pragma unroll 1
        for (int i = 128 * part + tid; i < left * 8; i += 256) {
            const int r = i >> 3, j = i & 7;
            *reinterpret_cast<uint4 *>(p.a.o + ((t.t0 + c + r) * p.a.H + t.h) * DV + 64 * half + 8 * j) =
                *reinterpret_cast<const uint4 *>(tile + r * 128 + ((j ^ (r & 7)) << 4));
        }
    } else {
        fence_proxy_async_shared();
    }
    // one warp stores a whole chunk's o and frees the tile; the others go on (none of them comes here again before that warp's
    // scores of the next chunk)
    if (threadIdx.x >> 5 != WARP_STORE) {
        named_bar_arrive(2, 2 * GROUP);
    } else {
        named_bar_sync(2, 2 * GROUP);
        if (lane == 0) {
            if (left >= C && !fail) {
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
    return false;
}

// ---- eight warps: decayed scores. Two threads share a token row: key blocks 0 and 3, or 1 and 2.
template <bool SEG>
__device__ __forceinline__ void role_scores(const ChunkParams &p, unsigned char *smem, Misc *m, uint32_t tmem) {
    constexpr bool states = false;
    const int half = (threadIdx.x - T_SCORES) >> 7, tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
    const uint32_t lanes = static_cast<uint32_t>(warp) << 21;  // TMEM lane offset 32 * warp in bits 16..31
    uint32_t it = 0;
    bool fail = false;  // (a warp that gives up still comes to the barriers and tells the others there)
    const int tasks = tasks_of<SEG>(p);
#pragma unroll 1
    for (int id = blockIdx.x; id < tasks; id += gridDim.x) {
        const Task t = task_of<SEG>(p, id, states);
        if (t.skip) continue;
#pragma unroll 1
        for (int c = 0; c < t.len; c += C, ++it) {
            const uint32_t ph = it & 1;
            fail = fail || !wait_warp(m, &m->dect, ph) || !wait_warp(m, &m->qk, ph);
            float out = 0.f;  // what the row's output is multiplied by
            if (!fail) {
                tc_fence_after();
                const float pre = m->pre[tid];
                const bool easy = m->easy;
                out = p.a.scale * (easy ? ex2(pre) : 1.f);
                const float row = easy ? 1.f : ex2(pre);
                // key blocks of 32, half a block at a time: blocks 0 and 3, or 1 and 2 (small loop bodies: with six roles
                // on it, a scheduler fetches most instructions it meets once a chunk from beyond its own cache)
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    const int b = (i & 2) ? 3 - half : half, j0 = 32 * b + 16 * (i & 1);
                    uint32_t s[16], x[8];
                    if (b > warp) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = 0;
                    } else {
                        tmem_ld16(tmem + lanes + COL_QK + j0, s);
                        if (easy) {
                            const f2 *f = reinterpret_cast<const f2 *>(&m->tab[j0]);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 8; ++j) x[j] = bf16_of(mul2(pair(s[2 * j], s[2 * j + 1]), f[j]));
                        } else {
                            const bool near = b == warp;
                            const float2 *f = reinterpret_cast<const float2 *>((near ? m->pre : m->tab + tab_at(warp)) + j0);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                float2 w = f[j];
                                w = near ? make_float2(ex2(pre - w.x), ex2(pre - w.y)) : make_float2(row * w.x, row * w.y);
                                x[j] = bf16_of(mul2(pair(s[2 * j], s[2 * j + 1]), pair(w.x, w.y)));
                            }
                        }
                        if (b == warp) {  // (cleared, not multiplied by zero: a score behind the row, and its weight, may be anything)
                            const int see = lane + 1 - 16 * (i & 1);
#pragma unroll
                            for (int j = 0; j < 8; ++j) x[j] = 2 * j + 1 < see ? x[j] : 2 * j < see ? x[j] & 0xffffu : 0u;
                        }
                    }
                    tmem_st8(tmem + lanes + COL_QK + 32 * b + 8 * (i & 1), x);  // over the scores they come from
                }
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(&m->p);
            }
            fail = fail || !wait_warp(m, &m->o, ph);
            if (output_part(p, smem, m, tmem + lanes, t, c, slot_of(TQ, it, states), tid, half, 0, out, fail)) return;
        }
    }
    if (threadIdx.x == 32 * WARP_STORE) bulk_wait_all();
}

// ---- eight warps: the state, transposed as U is. Two threads share a value column of S, one half of its keys each.
template <bool SEG>
__device__ __forceinline__ void role_state(const ChunkParams &p, unsigned char *smem, Misc *m, uint32_t tmem, bool states) {
    constexpr int NK = DK / 2;
    const Params &a = p.a;
    const int gtid = threadIdx.x - T_STATE, half = gtid >> 7, tid = gtid & 127, warp = tid >> 5;
    const uint32_t lanes = static_cast<uint32_t>(warp) << 21;
    unsigned char *sS = smem + OFF_S + half * PANEL + tid * 128;
    uint32_t it = 0;
    bool fail = false;
    f2 S[NK / 2];
    const int tasks = tasks_of<SEG>(p);
#pragma unroll 1
    for (int id = blockIdx.x; id < tasks; id += gridDim.x) {
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
                fail = fail || !wait_warp(m, &m->dect, ph);
                if (!fail) {
                    const float entry = ex2(m->pre[tid] + m->start[warp]);
                    if (m->easy) {
                        out *= entry;
                    } else if (wait_warp(m, &m->qs, ph)) {  // q S by the row's decay since the chunk began; P v is added onto it
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
                    } else {
                        fail = true;
                    }
                    arrive_warp(&m->p);
                }
            }
            fail = fail || !wait_warp(m, &m->u, ph);
            if (!fail) {
                tc_fence_after();
                const float dm1 = m->dm1[it & 3];
                const f2 d2 = pair(dm1, dm1);
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
                    fail = !wait_warp(m, &m->qs, ph);  // q has been multiplied by the last copy
                    if (!fail && c + C < t.len) publish();
                }
            }
            if (!states) {
                fail = fail || !wait_warp(m, &m->o, ph);
                if (output_part(p, smem, m, tmem + lanes, t, c, slot_of(TQ, it, states), tid, half, 1, out, fail)) return;
            }
        }
        if (fail) return;
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
    for (int n = 0; n < p.a.N; ++n) {
        const int2 f = p.first[n];
#pragma unroll 1
        for (uint32_t u = blockIdx.x * GROUP + gtid; f.y > 2 && u < static_cast<uint32_t>(H) * UNITS; u += gridDim.x * GROUP) {
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
                    e = add2(fma2(e, pair(dd[j], dd[j]), e), x[j]);
                    if (j < left) s[(1 + j) * step] = e;
                }
                s += BATCH * step;
                d += BATCH * H;
            }
        }
    }
}

// Touches the pages that this CTA's part of the join and its first output task begin in, from warps that the pass over the
// states leaves idle: an SM's first access to a page costs microseconds when all SMs make theirs at once.
__device__ __forceinline__ void touch(const void *p) {
    asm volatile("{\n\t.reg .b32 x;\n\tld.volatile.global.u32 x, [%0];\n\t}" ::"l"(p) : "memory");
}
__device__ __forceinline__ void touch_ahead(const ChunkParams &p) {
    const int tid = threadIdx.x - T_SCORES;
    const int tasks = tasks_of<true>(p), id = blockIdx.x;
    constexpr size_t SZ = static_cast<size_t>(DK) * DV;
    if (id >= tasks) return;
    const Task t = task_of<true>(p, id, false);
    if (t.len > 0) {
        const int hk = t.h / p.a.rep;
        if (tid == 0) touch(p.a.q + t.t0 * p.a.qs + hk * DK);
        if (tid == 1) touch(p.a.o + (t.t0 * p.a.H + t.h) * DV);
        if (tid == 2) touch(p.a.g + (p.a.g_per_token ? t.t0 * p.a.H + t.h : t.h));
    }
    if (tid == 3 && t.sin) touch(t.sin);
    if (tid == 4 && t.sout) touch(t.sout);
    if (tid < 64) {
        const size_t all = static_cast<size_t>(tasks) * SZ, at = static_cast<size_t>(tid) << 19;  // every 2 MB of the states
        if (at < all) touch(p.states + at);
    }
}

constexpr int BARRIERS = offsetof(Misc, tmem) / sizeof(uint64_t);  // they come first in Misc
__device__ __forceinline__ int arrivals_of(int i, bool states) {
    constexpr int E0 = offsetof(Misc, empty) / 8, V0 = offsetof(Misc, vt) / 8, P0 = offsetof(Misc, p) / 8,
                  W0 = offsetof(Misc, wfree) / 8, U0 = offsetof(Misc, ufree) / 8;
    if (i >= E0 && i < E0 + TILES) return !states && (i - E0) % 3 == TK ? 2 : 1;  // a k tile is read by q k^T and by U
    if (i == P0 || i == U0 + 1) return 2 * GROUP / 32;                              // warps of the scores' and the state's groups
    return ((i >= V0 && i < P0) || (i >= W0 && i < W0 + 2) || i == U0) ? GROUP / 32 : 1;  // warps of one group
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
    if (LEADS && threadIdx.x == 0 && !grid_sync(p.num_segs + 1, gridDim.x)) m->abort = 1;
    cta_sync();
    if (JOINS) join_states(p, threadIdx.x - T_STATE);
    cta_sync();
    if (LEADS && threadIdx.x < 32) {
        for (int i = threadIdx.x; i < BARRIERS; i += 32) mbar_inval(reinterpret_cast<uint64_t *>(m) + i);  // (every arrival has come)
        init_barriers(m, false);
        __syncwarp();
        if (threadIdx.x == 0 && !grid_sync(p.num_segs + 1, 2 * gridDim.x)) m->abort = 1;
    }
    cta_sync();
    return *reinterpret_cast<volatile int32_t *>(&m->abort) == 0;
}

// SEGMENTS: sequences in segments, states first (a cooperative launch); else every sequence as a whole
template <bool SEGMENTS>
__global__ void __launch_bounds__(THREADS, 1) kda_linear_chunk_kernel(const __grid_constant__ ChunkParams p) {
    extern __shared__ __align__(1024) unsigned char smem[];
    Misc *m = reinterpret_cast<Misc *>(smem + OFF_MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) {
        init_barriers(m, SEGMENTS);
        m->abort = 0;
    }
    if (warp == WARP_MMA_U) tmem_alloc(&m->tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;  // all 512 columns were allocated: they begin at column 0
    // every role: the pass over the states, the join, the pass over the outputs; or the last alone
    if (threadIdx.x < T_SCORES) {
        fewer_registers<REGS_AUX>();
#pragma unroll 1
        for (int pass = SEGMENTS ? 0 : 1; pass < 2; ++pass) {
            const bool states = SEGMENTS && pass == 0;
            if (warp == WARP_LOAD) {
                if (lane == 0) role_load<SEGMENTS>(p, smem, m, states);
            } else if (warp == WARP_DECAY) {
                role_decay<SEGMENTS>(p, m, states);
            } else if (warp == WARP_MMA_U) {
                role_mma_state<SEGMENTS>(p, smem, m, states);
            } else if (warp == WARP_MMA_OUT && !states) {
                role_mma_out<SEGMENTS>(p, smem, m);
            }
            __syncwarp();
            if (SEGMENTS && pass == 0 && !next_pass<true, false>(p, m)) break;
        }
    } else if (threadIdx.x < T_STATE) {
        if (SEGMENTS) touch_ahead(p);
        if (!SEGMENTS || next_pass<false, false>(p, m)) role_scores<SEGMENTS>(p, smem, m, tmem);
    } else if (threadIdx.x < T_V) {
        more_registers<REGS_STATE>();
#pragma unroll 1
        for (int pass = SEGMENTS ? 0 : 1; pass < 2; ++pass) {
            role_state<SEGMENTS>(p, smem, m, tmem, SEGMENTS && pass == 0);
            if (SEGMENTS && pass == 0 && !next_pass<false, true>(p, m)) break;
        }
    } else {
        fewer_registers<REGS_V>();
#pragma unroll 1
        for (int pass = SEGMENTS ? 0 : 1; pass < 2; ++pass) {
            role_v<SEGMENTS>(p, smem, m, tmem, SEGMENTS && pass == 0);
            if (SEGMENTS && pass == 0 && !next_pass<false, false>(p, m)) break;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && m->abort) set_status(p.a.status, KDA_ERR_TIMEOUT);
    if (warp == WARP_MMA_U) tmem_dealloc(tmem, 512);
}

// ---- segments: one CTA. Sequence n of c chunks gets ceil(c / L) segments of about equal length.
__global__ void __launch_bounds__(256) kda_linear_plan_kernel(const ChunkParams p) {
    __shared__ int part[256], total;
    const Params &a = p.a;
    const int tid = threadIdx.x;
    const int per = (a.N + 255) / 256, n0 = tid * per, n1 = n0 + per < a.N ? n0 + per : a.N;
    const bool start_ok = a.cu[0] == 0;
    auto chunks = [&](int n) -> int64_t {
        const int64_t b = a.cu[n], e = a.cu[n + 1];
        return start_ok && b >= 0 && e >= b && e <= a.T ? (e - b + C - 1) / C : -1;
    };
    int mine = 0;
    for (int n = n0; n < n1; ++n) {
        const int64_t c = chunks(n);
        mine += c < 0 ? 0 : c == 0 ? 1 : static_cast<int>((c + p.seg_chunks - 1) / p.seg_chunks);
    }
    part[tid] = mine;
    __syncthreads();
    if (tid == 0) {
        int s = 0;
        for (int i = 0; i < 256; ++i) {
            const int v = part[i];
            part[i] = s;
            s += v;
        }
        // more than valid offsets can need: sequences overlap (cu_seqlens goes back), and nothing runs
        if (s > p.most_segs) {
            set_status(a.status, KDA_ERR_BAD_SEQLENS);
            s = -1;
        }
        p.num_segs[0] = s < 0 ? 0 : s;
        p.num_segs[1] = 0;
        total = s;
    }
    __syncthreads();
    if (total < 0) {
        for (int n = n0; n < n1; ++n) p.first[n] = make_int2(0, 0);
        return;
    }
    int at = part[tid];
    for (int n = n0; n < n1; ++n) {
        const int64_t c = chunks(n);
        if (c < 0) {
            set_status(a.status, KDA_ERR_BAD_SEQLENS);
            p.first[n] = make_int2(at, 0);
            continue;
        }
        const int k = c == 0 ? 1 : static_cast<int>((c + p.seg_chunks - 1) / p.seg_chunks);
        const int64_t step = (c + k - 1) / k * C, len = a.cu[n + 1] - a.cu[n];
        p.first[n] = make_int2(at, k);
        for (int i = 0; i < k; ++i, ++at) {
            Segment sg;
            const int64_t b = i * step < len ? i * step : len, e = b + step < len ? b + step : len;
            sg.t0 = static_cast<int32_t>(a.cu[n] + b);
            sg.len = static_cast<int32_t>(e - b);
            sg.seq = n;
            sg.index = i;
            sg.count = k;
            p.segs[at] = sg;
        }
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

int device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) (void)cudaGetLastError();
    return dev;
}
// SMs of the current device (0: no usable device); asked once for each of the first MAX_DEVICES
constexpr int MAX_DEVICES = 64;
int num_sms() {
    static std::atomic<int> known[MAX_DEVICES];
    const int dev = device();
    if (dev < 0) return 0;
    int sms = dev < MAX_DEVICES ? known[dev].load(std::memory_order_relaxed) : 0;
    if (sms) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    if (dev < MAX_DEVICES) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

template <bool SEGMENTS>
cudaError_t run(const ChunkParams &p, int64_t most_tasks, int sms, cudaStream_t stream) {
    const auto kernel = kda_linear_chunk_kernel<SEGMENTS>;
    static std::atomic<bool> ready[MAX_DEVICES];
    const int dev = device();
    if (dev < 0 || dev >= MAX_DEVICES || !ready[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        cudaFuncAttributes at{};
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, kernel);
        if (e != cudaSuccess) return e;
        if (at.numRegs != REGS) return cudaErrorInvalidConfiguration;  // the roles' register split adds up to this
        if (dev >= 0 && dev < MAX_DEVICES) ready[dev].store(true, std::memory_order_release);
    }
    const int grid = static_cast<int>(most_tasks < sms ? most_tasks : sms);
    if (SEGMENTS) {
        void *args[] = {const_cast<ChunkParams *>(&p)};
        return cudaLaunchCooperativeKernel(reinterpret_cast<const void *>(kernel), dim3(grid), dim3(THREADS), args, SMEM, stream);
    }
    kernel<<<grid, THREADS, SMEM, stream>>>(p);
    return cudaGetLastError();
}

// Sequences of few tokens run the recurrence.
bool few_tokens(int64_t N, int64_t T) { return T <= 16 * N; }

// Chunks per segment so that every SM gets about one (segment, head); 0 when no
// sequence can be longer than that.
int segment_chunks(int64_t N, int64_t T, int64_t H, int sms) {
    const int64_t longest = (T + C - 1) / C, all = (T / C + N) * H;
    int64_t len = (all + sms - 1) / sms;
    if (len < 4) len = 4;
    return longest <= len ? 0 : static_cast<int>(len);
}

struct Layout {
    int64_t most;  // segments at most: ceil(c / L) <= c' / L + 1 summed over the sequences
    size_t first, segs, decays, states, bytes;
};
Layout layout_of(int64_t N, int64_t T, int64_t H, int len) {
    Layout l;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    l.most = T / (static_cast<int64_t>(C) * len) + N;
    l.first = 256;
    l.segs = up(l.first + sizeof(int2) * N);
    l.decays = up(l.segs + sizeof(Segment) * l.most);
    l.states = up(l.decays + sizeof(float) * l.most * H);
    l.bytes = l.states + sizeof(float) * DK * DV * l.most * H;
    return l;
}
}  // namespace

size_t chunked_workspace_bytes(int64_t N, int64_t T, int64_t H) {
    if (N < 1 || T < 1 || H < 1 || few_tokens(N, T)) return 0;
    const int sms = num_sms();
    const int len = sms > 0 ? segment_chunks(N, T, H, sms) : 0;
    return len ? layout_of(N, T, H, len).bytes : 0;
}

cudaError_t launch_chunked(const Params &a, void *workspace, cudaStream_t stream) {
    if (few_tokens(a.N, a.T)) return launch_recurrent(a, stream);
    const int sms = num_sms();
    if (sms < 1) return cudaErrorInvalidDevice;
    ChunkParams p{};
    p.a = a;
    const int hk = a.H / a.rep;
    if (!encode(&p.tq, a.q, a.T, hk, a.qs) || !encode(&p.tk, a.k, a.T, hk, a.ks) || !encode(&p.tv, a.v, a.T, a.H, a.vs) ||
        !encode(&p.to, a.o, a.T, a.H, static_cast<int64_t>(a.H) * DV))
        return cudaErrorInvalidValue;
    p.seg_chunks = segment_chunks(a.N, a.T, a.H, sms);
    p.tasks = a.N * a.H;
    if (!p.seg_chunks) return run<false>(p, p.tasks, sms, stream);
    const Layout l = layout_of(a.N, a.T, a.H, p.seg_chunks);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    p.most_segs = static_cast<int32_t>(l.most);
    p.num_segs = reinterpret_cast<int32_t *>(ws);
    p.first = reinterpret_cast<int2 *>(ws + l.first);
    p.segs = reinterpret_cast<Segment *>(ws + l.segs);
    p.decays = reinterpret_cast<float *>(ws + l.decays);
    p.states = reinterpret_cast<float *>(ws + l.states);
    kda_linear_plan_kernel<<<1, 256, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? run<true>(p, l.most * a.H, sms, stream) : e;
}

}  // namespace lin
}  // namespace kda
