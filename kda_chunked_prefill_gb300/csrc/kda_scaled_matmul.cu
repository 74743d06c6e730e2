// kda_scaled_matmul on tcgen05: e4m3 activations times an e4m3 weight, with fp32 scales.
//
//     y[t, n] = sum over blocks b of 128 channels:  xs[t, b] ws[n / 128, b] sum_{k in b} x[t, k] w[n, k]      bf16, rounded once
//
// The scales are any fp32 numbers, so the tensor core cannot apply them. It forms each block's inner sum (four MMAs of 32 channels)
// in one of two accumulators in tensor memory; eight warps read it while it forms the next block's in the other, and add it,
// times its scale, to their fp32 registers: acc += (xs ws) D.
//
// A CTA makes tiles of 128 lanes x BN columns of the accumulator. Roles:
//   load    one thread: 128-byte wide tiles of both operands by TMA into a ring of stages
//   MMAs    two threads, every second block each: waiting for its operands and issuing takes one as long as the tensor core
//   scales  one warp: xs ws of each block, to shared memory, a few blocks ahead
//   sums    eight warps: a lane and half of the columns each; then y
//
// Which operand takes the lanes. For more than 64 rows the rows of x do, columns are outputs: a thread needs one scale a block
// (its 128 columns share the weight's), and y leaves by tiled stores. For up to 64 rows (decode) the weight's rows do and x's are
// the columns, as few as 16: no lane of the tensor core idles, and the weight, which is what bounds these calls, is read by
// as many CTAs as there are. Where these tiles are fewer than the SMs, the CTAs of a cluster share one: each takes a part of the
// channels, and they add up their sums through distributed shared memory, in the order of their ranks.
//
// Wide tiles are a pair's: two CTAs make 256 x 256, each has its 128 lanes' accumulators and half of the columns' operand. An SM takes
// 54 bytes a cycle into shared memory (measured by loads alone): a tile of 128 x 256 by one CTA needs 48 KB a block, 920 cycles, where its
// MMAs take 512; of a pair, each CTA needs 32 KB, 610. The two halves of the columns have barriers of their own.
//
// What bounds it. Many rows: the round trip of the accumulators, two of which fill tensor memory (read by the sums' warps, arrival at the
// first CTA, MMAs, commit to both), 800 cycles a block: 8192 rows, 2048 channels to 6144 outputs 78 us at 2070 MHz, 2.65 PFLOP/s, and 85 to 88
// after some tens of milliseconds of it, when the power cap holds the SMs at 1800 to 1940 MHz, replayed or not. (At the full clock: columns in one
// piece 88 us; one CTA's tiles 86; the pair without the sums 73; sixteen warps for the sums 92.) Few rows: reading the weight (7 rows, 12288
// to 12288: 28 us, 5.4 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda.h"
#include "kda_checks.h"
#include "kda_linear.cuh"
#include "kda_tensor_map.h"
#include "kda_waits.cuh"

namespace kda {
namespace mm {

using lin::f2;
using lin::mbar_arrive;

constexpr int LANES = 128;  // of an accumulator
constexpr int KB = 128;     // channels of a block: a row of a stage's tile is 128 bytes
constexpr int THREADS = 384;
constexpr int SUM_WARPS = 8, FIRST_SUM_WARP = 4;
constexpr int AHEAD = 4;    // blocks whose scales are loaded and handed on at a time (a wait a block for them was a third of the sums' time)
constexpr int SCALES = 2;   // such groups in shared memory
constexpr int MAX_SPLITS = 8;
constexpr int SWAP_ROWS = 64;

template <int BN, bool SWAP>
struct Cfg {
    // of a pair's columns, each CTA has the first or the second 64 of both halves
    static constexpr bool PAIR = BN == 256;
    static constexpr int HALVES = PAIR ? 2 : 1;  // of the columns: accumulators with barriers of their own
    static constexpr int A_BYTES = LANES * KB, B_BOX = PAIR ? BN / 4 : BN, B_BYTES = HALVES * B_BOX * KB, STAGE = A_BYTES + B_BYTES;
    static constexpr int CTAS = BN <= 64 ? 2 : 1;  // per SM
    static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 5 : SWAP ? (BN == 64 ? 4 : 5) : 3;
    static constexpr int GROUPS = BN == 256 ? 2 : 1;  // column groups with a weight scale of their own
    static constexpr int SCALE_FLOATS = SWAP ? BN : GROUPS * LANES;
    static constexpr int STAGING = SWAP ? 0 : LANES * BN * 2;  // y's tile, a warp's part after another's
    static constexpr int COLS = BN / 2;                        // of a thread
    static constexpr int PANEL = COLS < 64 ? COLS : 64;        // columns of y's tile that are stored at a time
    // where columns c .. c + 7 of a warp's row r lie: rows of 128 bytes with the 128-byte swizzle, or of 64 with the 64-byte one
    static __device__ __forceinline__ int staged(int r, int c) {
        return (c / PANEL) * (32 * PANEL * 2) + r * (PANEL * 2) + ((((c % PANEL) / 8) ^ (PANEL == 64 ? r & 7 : (r >> 1) & 3)) << 4);
    }
    static constexpr int RED_LD = LANES + 1;                   // a column of the sums that a cluster adds up
    static constexpr int TMEM = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int OFF_STAGING = STAGES * STAGE, OFF_SCALES = OFF_STAGING + STAGING;
    static constexpr int OFF_MISC = OFF_SCALES + SCALES * AHEAD * SCALE_FLOATS * 4;
    // registers of the sums' warps and the others, where an even share is too few
    static constexpr bool UNEVEN = BN == 256;
    static constexpr int REGS_SUM = 208, REGS_AUX = 80, REGS = 168;
    static_assert(!UNEVEN || 8 * REGS_SUM + 4 * REGS_AUX <= 12 * REGS, "the launch's registers");
};

struct Misc {
    uint64_t full[5], empty[5];              // a stage
    uint64_t tfull[4], tempty[4];            // an accumulator
    uint64_t sfull[SCALES], sempty[SCALES];  // a group's scales
    uint64_t drained[2];
    uint32_t tmem;
    int32_t abort;
};

struct Params {
    CUtensorMap a, b, y;  // the lanes' operand, the columns', and (rows in the lanes) the output
    const float *xs, *ws;
    int64_t xs_row;   // floats from one row's scales to the next
    int32_t xs_block; // and from one block's to the next (0: one scale a row)
    int32_t blocks;   // of channels
    int32_t rows, outs;
    int32_t lane_tiles, col_tiles, tiles;
    int32_t splits;   // CTAs of a cluster that share a tile
    int32_t tiled_y;  // y leaves by tiled stores
    int32_t withhold; // tests: the group of blocks of each CTA whose scales are not handed on (-1: none)
    __nv_bfloat16 *out;
    int32_t *status;
};

__device__ __forceinline__ bool is_complete(uint64_t *bar, uint32_t parity) {  // (does not wait)
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int c0, int c1, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(smem_u32(src))
                 : "memory");
}
// the same address in the first CTA of a pair
__device__ __forceinline__ uint32_t in_leader(const void *p) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}
// a CTA's half of a pair's stage: its bytes count at the first CTA's barrier
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, int c0, int c1, uint32_t leader_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(leader_bar)
        : "memory");
}
// What this arrival hands over is tensor memory alone: the products that wait for it write the accumulator that the warps have read, and no
// warp's other memory is read behind it. That order is tcgen05's own: tcgen05.wait::ld completes the warp's loads (their values are in
// registers), tcgen05.fence::before_thread_sync puts them before the arrival, and after_thread_sync puts the products behind the wait for it.
// So release at cluster scope, which waits for the warps' accesses to all memory, is not needed: 8192 rows, 2048 channels to 6144 outputs
// 167 us with it, 80 in this form (release at the CTA's scope) and 80 relaxed.
__device__ __forceinline__ void arrive_remote_if(uint32_t bar, bool yes) {  // (no branch)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(static_cast<uint32_t>(yes))
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void alloc(uint32_t *slot, uint32_t ncols) {  // whole warp
    if (!PAIR) {
        tmem_alloc(slot, ncols);
        return;
    }
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <bool PAIR>
__device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t ncols) {
    if (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
    else
        tmem_dealloc(taddr, ncols);
}
// kind::f8f6f4 with e4m3 A and B (K-major) and fp32 D: 32 channels
template <bool PAIR>
__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}
// arrives at `bar`, of a pair at the barriers of this address of the CTAs in `mask`, once the MMAs so far are complete
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar, uint16_t mask = 3) {
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
            "h"(mask)
            : "memory");
    else
        umma_commit(bar);
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[8]) { tmem_ld8(t, r); }
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&r)[16]) { tmem_ld16(t, r); }
__device__ __forceinline__ void cluster_sync() {  // all threads of the cluster's CTAs
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

// Tiles in the order they are made: bands of BAND lanes, in a band column after column, so that what runs at one time shares few rows of
// both operands.
constexpr uint32_t BAND = 2048;
template <bool PAIR>
__device__ __forceinline__ void tile_at(const Params &p, int32_t i, int &lane_tile, int &col_tile) {
    constexpr uint32_t MOST = BAND / LANES / (PAIR ? 2 : 1);
    const uint32_t wide = MOST * static_cast<uint32_t>(p.col_tiles), band = static_cast<uint32_t>(i) / wide, in = i - band * wide;
    const uint32_t first = band * MOST, rest = p.lane_tiles - first, height = rest < MOST ? rest : MOST, col = in / height;
    lane_tile = static_cast<int>(first + in - col * height);
    col_tile = static_cast<int>(col);
}

template <int BN, bool SWAP>
__global__ void __launch_bounds__(THREADS, Cfg<BN, SWAP>::CTAS) kda_scaled_matmul_kernel(const __grid_constant__ Params p) {
    using C = Cfg<BN, SWAP>;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    float *scales = reinterpret_cast<float *>(smem + C::OFF_SCALES);
    Misc *m = reinterpret_cast<Misc *>(smem + C::OFF_MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) mbar_init(&m->full[i], 1), mbar_init(&m->empty[i], 1);
        for (int i = 0; i < 2 * C::HALVES; ++i) mbar_init(&m->tfull[i], 1), mbar_init(&m->tempty[i], SUM_WARPS);
        for (int i = 0; i < SCALES; ++i) mbar_init(&m->sfull[i], 1), mbar_init(&m->sempty[i], SUM_WARPS);
        mbar_init(&m->drained[0], 1), mbar_init(&m->drained[1], 1);
        m->abort = 0;
        mbar_fence_init();
    }
    if (warp == 3) alloc<C::PAIR>(&m->tmem, C::TMEM);
    tc_fence_before();
    __syncthreads();
    if (C::PAIR) cluster_sync();  // (both CTAs' barriers are set up)
    tc_fence_after();
    const uint32_t tmem = m->tmem;

    // this CTA's tiles, and its part of their blocks or, of a pair, of their lanes
    const int splits = SWAP ? p.splits : 1, rank = splits > 1 ? static_cast<int>(blockIdx.x) % splits : 0;
    const int peer = C::PAIR ? static_cast<int>(blockIdx.x) & 1 : 0;
    const int32_t tile0 = C::PAIR ? blockIdx.x / 2 : blockIdx.x / splits, tile_step = C::PAIR ? gridDim.x / 2 : gridDim.x / splits;
    const int b0 = static_cast<int>(static_cast<int64_t>(p.blocks) * rank / splits);
    const int b1 = static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / splits);

    if (warp < FIRST_SUM_WARP) {
        if (C::UNEVEN) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_AUX));
        if (warp == 0 && lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int32_t tile = tile0; ok && tile < p.tiles; tile += tile_step) {
                int lt, ct;
                tile_at<C::PAIR>(p, tile, lt, ct);
                if (C::PAIR) lt = 2 * lt + peer;
                for (int b = b0; b < b1; ++b, ++it) {
                    const uint32_t st = it % C::STAGES, use = it / C::STAGES;
                    if (!(ok = wait(m, &m->empty[st], (use & 1) ^ 1))) break;
                    unsigned char *s = smem + st * C::STAGE;
                    if (C::PAIR) {
                        const uint32_t bar = in_leader(&m->full[st]);
                        if (!peer) mbar_arrive_expect_tx(&m->full[st], 2 * C::STAGE);
                        tma_load_2d_pair(s, &p.a, b * KB, lt * LANES, bar);
#pragma unroll
                        for (int h = 0; h < C::HALVES; ++h)
                            tma_load_2d_pair(s + C::A_BYTES + h * C::B_BOX * KB, &p.b, b * KB, ct * BN + (2 * h + peer) * C::B_BOX, bar);
                    } else {
                        mbar_arrive_expect_tx(&m->full[st], C::STAGE);
                        tma_load_2d(s, &p.a, b * KB, lt * LANES, &m->full[st]);
                        tma_load_2d(s + C::A_BYTES, &p.b, b * KB, ct * BN, &m->full[st]);
                    }
                }
            }
            if (C::PAIR)  // the first CTA's commits arrive here: none may be on its way when this CTA ends
                for (uint32_t i = it < C::STAGES ? 0 : it - C::STAGES; ok && i < it; ++i)
                    ok = wait(m, &m->empty[i % C::STAGES], (i / C::STAGES) & 1);
            if (!ok && !peer)  // what is in flight lands before the CTA, or both of a pair, end
                for (uint32_t i = it < C::STAGES ? 0 : it - C::STAGES; i < it; ++i)
                    wait_drain(&m->full[i % C::STAGES], (i / C::STAGES) & 1);
        } else if ((warp == 1 || warp == 3) && !peer) {
            // The whole warp goes through the loop, so that descriptors are made in uniform registers; one lane issues. Its instructions
            // count: the sums' push them out of the first instruction cache.
            constexpr uint32_t M = C::PAIR ? 2 * LANES : LANES, N = BN / C::HALVES, ID = (1u << 4) | (N >> 3 << 17) | (M >> 4 << 24);
            const uint32_t buf = static_cast<uint32_t>(warp >> 1), d = tmem + buf * BN;
            const uint64_t a0 = umma_desc_sw128(smem_u32(smem), 16, 1024);
            const int32_t tiles = tile0 < p.tiles ? (p.tiles - 1 - tile0) / tile_step + 1 : 0;
            const int64_t blocks = static_cast<int64_t>(tiles) * (b1 - b0);  // in all; every second is this thread's
            uint32_t st = buf % C::STAGES, use = buf / C::STAGES, n = 0;
            bool ok = true;
#pragma unroll 1
            for (int64_t it = buf; it < blocks; it += 2, ++n) {
                const uint64_t a = a0 + st * (C::STAGE / 16), b = a + C::A_BYTES / 16;
                // The accumulators first: that the sums are through with block it - 2, and so with every block before, says that this stage's
                // last use, perhaps the other warp's, is over. Its parity alone would take the phase before last for this one. (Of a pair, each
                // of these warps has stages of its own, and asks for the operands ahead.)
                if (C::PAIR && !(ok = wait_warp(m, &m->full[st], use & 1))) break;
#pragma unroll
                for (int h = 0; h < C::HALVES; ++h) {
                    const uint32_t i = buf * C::HALVES + h;
                    ok = wait_warp(m, &m->tempty[i], (n & 1) ^ 1) && (C::PAIR || wait_warp(m, &m->full[st], use & 1));
                    if (!ok) break;
                    tc_fence_after();
                    if (lin::elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_e4m3<C::PAIR>(d + h * (BN / 2), a + 2 * k, b + h * (C::B_BOX * KB / 16) + 2 * k, ID, k > 0);
                        if (h == C::HALVES - 1) commit<C::PAIR>(&m->empty[st]);
                        commit<C::PAIR>(&m->tfull[i]);
                    }
                }
                if (!ok) break;
                st += 2;
                if (st >= C::STAGES) st -= C::STAGES, ++use;
            }
            __syncwarp();
            if (!ok) {
                if (lin::elect_one()) commit<C::PAIR>(&m->drained[buf], 1);
                __syncwarp();
                wait_drain(&m->drained[buf], 0);
            }
        } else if (warp == 2) {
            uint32_t it = 0;
            bool ok = true;
            for (int32_t tile = tile0; ok && tile < p.tiles; tile += tile_step) {
                int lt, ct;
                tile_at<C::PAIR>(p, tile, lt, ct);
                if (C::PAIR) lt = 2 * lt + peer;
                const int row0 = SWAP ? ct * BN : lt * LANES;
                const int out_block = SWAP ? lt : ct * BN / KB;
                const int out_blocks = (p.outs + KB - 1) / KB;
                constexpr int PER = SWAP ? (BN + 31) / 32 : LANES / 32;  // rows of a lane
                for (int b = b0; ok && b < b1; b += AHEAD) {
                    float xs[AHEAD][PER], ws[AHEAD][C::GROUPS];
#pragma unroll
                    for (int a = 0; a < AHEAD; ++a) {
                        const int bb = b + a < b1 ? b + a : b1 - 1;
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const int64_t row = row0 + 32 * i + lane;
                            xs[a][i] = row < p.rows ? __ldg(p.xs + row * p.xs_row + static_cast<int64_t>(bb) * p.xs_block) : 0.f;
                        }
#pragma unroll
                        for (int g = 0; g < C::GROUPS; ++g)
                            ws[a][g] = out_block + g < out_blocks
                                           ? __ldg(p.ws + static_cast<int64_t>(out_block + g) * p.blocks + bb) : 0.f;
                    }
                    const uint32_t slot = it % SCALES;
                    if (!(ok = wait_warp(m, &m->sempty[slot], ((it / SCALES) & 1) ^ 1))) break;
                    float *s = scales + slot * (AHEAD * C::SCALE_FLOATS);
#pragma unroll
                    for (int a = 0; a < AHEAD; ++a)
#pragma unroll
                        for (int g = 0; g < C::GROUPS; ++g)
#pragma unroll
                            for (int i = 0; i < PER; ++i)
                                if (!SWAP || BN >= 32 || lane < BN)
                                    s[a * C::SCALE_FLOATS + g * LANES + 32 * i + lane] = xs[a][i] * ws[a][g];
                    if (static_cast<int32_t>(it) != p.withhold) arrive_warp(&m->sfull[slot]);
                    ++it;
                }
            }
        }
    } else {
        if (C::UNEVEN) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SUM));
        const int e = warp - FIRST_SUM_WARP, quad = warp & 3, half = e >> 2;
        const int my_lane = 32 * quad + lane, col0 = half * C::COLS;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * quad) << 16) + col0;
        const uint32_t tempty = C::PAIR ? in_leader(&m->tempty[0]) : 0, mine_of = C::PAIR ? half : 0;  // its accumulator of a buffer's
        constexpr int LD = C::COLS < 16 ? C::COLS : 16;  // columns read at a time
        uint32_t it = 0, group = 0;
        bool ok = true, ready = false;  // ready: the next block's sum is there
        for (int32_t tile = tile0; ok && tile < p.tiles; tile += tile_step) {
            int lt, ct;
            tile_at<C::PAIR>(p, tile, lt, ct);
            if (C::PAIR) lt = 2 * lt + peer;
            f2 acc[C::COLS / 2];  // of neighbouring columns
#pragma unroll
            for (int i = 0; i < C::COLS / 2; ++i) acc[i] = 0;
            float mine[AHEAD];
            const float *s = scales;  // the block's
            int handed = 0;           // blocks of this group to come
#pragma unroll 1
            for (int left = b1 - b0; left > 0; --left, ++it) {
                const uint32_t buf = it & 1, slot = group % SCALES;
                if (handed == 0) {
                    if (!(ok = wait_warp(m, &m->sfull[slot], (group / SCALES) & 1))) break;
                    handed = AHEAD;
                    s = scales + slot * (AHEAD * C::SCALE_FLOATS);
                    if (!SWAP) {
#pragma unroll
                        for (int a = 0; a < AHEAD; ++a) mine[a] = s[a * C::SCALE_FLOATS + (col0 / KB) * LANES + my_lane];
                        __syncwarp();
                        lin::mbar_arrive_if(&m->sempty[slot], lane == 0);
                        ++group;
                    }
                }
                --handed;
                if (!__all_sync(0xffffffffu, ready) && !(ok = wait_warp(m, &m->tfull[buf * C::HALVES + mine_of], (it >> 1) & 1))) break;
                tc_fence_after();
                uint32_t d[2][LD];
                tmem_ld(taddr + buf * BN, d[0]);
                const float one = mine[0];
#pragma unroll
                for (int a = 0; a + 1 < AHEAD; ++a) mine[a] = mine[a + 1];
#pragma unroll
                for (int c = 0; c < C::COLS; c += LD) {  // (the next columns come while these are added)
                    const uint32_t(&x)[LD] = d[c / LD & 1];
                    tmem_wait_ld();
                    if (c + LD < C::COLS) {
                        tmem_ld(taddr + buf * BN + c + LD, d[c / LD + 1 & 1]);
                    } else {  // all is read: the accumulator is handed back, and the other one asked for, before the last columns are added
                        tc_fence_before();
                        __syncwarp();
                        if (C::PAIR)
                            arrive_remote_if(tempty + 8 * (buf * C::HALVES + mine_of), lane == 0);
                        else
                            lin::mbar_arrive_if(&m->tempty[buf], lane == 0);
                        ready = is_complete(&m->tfull[(buf ^ 1) * C::HALVES + mine_of], ((it + 1) >> 1) & 1);
                    }
#pragma unroll
                    for (int i = 0; i < LD; i += 4) {
                        float4 f = make_float4(one, one, one, one);
                        if (SWAP) f = *reinterpret_cast<const float4 *>(s + col0 + c + i);
                        f2 &a0 = acc[(c + i) / 2], &a1 = acc[(c + i) / 2 + 1];
                        a0 = lin::fma2(lin::pair(x[i], x[i + 1]), lin::pair(f.x, f.y), a0);
                        a1 = lin::fma2(lin::pair(x[i + 2], x[i + 3]), lin::pair(f.z, f.w), a1);
                    }
                }
                s += C::SCALE_FLOATS;
                if (SWAP && (handed == 0 || left == 1)) {
                    __syncwarp();
                    lin::mbar_arrive_if(&m->sempty[slot], lane == 0);
                    ++group;
                    handed = 0;
                }
            }
            if (!ok) break;
            if (SWAP && splits > 1) {  // (one tile a CTA; the stages are done with)
                float *red = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int i = 0; i < C::COLS; i += 2) {
                    float u, v;
                    lin::split(acc[i / 2], u, v);
                    red[(col0 + i) * C::RED_LD + my_lane] = u;
                    red[(col0 + i + 1) * C::RED_LD + my_lane] = v;
                }
            } else if (SWAP) {
                const int64_t n = static_cast<int64_t>(lt) * LANES + my_lane;
#pragma unroll
                for (int i = 0; i < C::COLS; ++i) {
                    const int64_t t = static_cast<int64_t>(ct) * BN + col0 + i;
                    float u, v;
                    lin::split(acc[i / 2], u, v);
                    if (n < p.outs && t < p.rows) p.out[t * p.outs + n] = __float2bfloat16_rn(i & 1 ? v : u);
                }
            } else {
                // the warp's own 32 rows of y, as panels of PANEL columns, swizzled
                unsigned char *staging = smem + C::OFF_STAGING + e * (32 * C::COLS * 2);
                if (lane == 0) bulk_wait_read();  // (the tile before has left)
                __syncwarp();
#pragma unroll
                for (int c = 0; c < C::COLS; c += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = lin::bf16_of(acc[c / 2 + j]);
                    *reinterpret_cast<uint4 *>(staging + C::staged(lane, c)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async_shared();
                __syncwarp();
                const int64_t t0 = static_cast<int64_t>(lt) * LANES + 32 * quad;
                const int n0 = ct * BN + col0;
                if (p.tiled_y) {
                    if (lane == 0) {
#pragma unroll
                        for (int c = 0; c < C::COLS; c += C::PANEL)
                            if (n0 + c < p.outs && t0 < p.rows)
                                tma_store_2d(&p.y, staging + C::staged(0, c), n0 + c, static_cast<int>(t0));
                        bulk_commit();
                    }
                } else {
#pragma unroll 1
                    for (int r = 0; r < 32 && t0 + r < p.rows; ++r)
                        for (int c = lane; c < C::COLS && n0 + c < p.outs; c += 32)
                            p.out[(t0 + r) * p.outs + n0 + c] =
                                *reinterpret_cast<const __nv_bfloat16 *>(staging + C::staged(r, c & ~7) + (c & 7) * 2);
                    __syncwarp();
                }
            }
        }
        if (!SWAP && lane == 0) bulk_wait_read();
    }

    // (every thread comes here, one that has given up as well)
    __syncwarp();
    if (SWAP && splits > 1) {
        cluster_sync();
        if (warp >= FIRST_SUM_WARP) {
            int lt, ct;
            tile_at<C::PAIR>(p, tile0, lt, ct);
            const int c0 = BN * rank / splits, n = BN * (rank + 1) / splits - c0;
            const uint32_t red = smem_u32(smem);
#pragma unroll 4
            for (int i = threadIdx.x - 32 * FIRST_SUM_WARP; i < n * LANES; i += 32 * SUM_WARPS) {
                const int c = c0 + i / LANES, l = i % LANES;
                const int64_t t = static_cast<int64_t>(ct) * BN + c, o = static_cast<int64_t>(lt) * LANES + l;
                if (t >= p.rows || o >= p.outs) continue;
                float part[MAX_SPLITS], s = 0.f;
#pragma unroll
                for (int r = 0; r < MAX_SPLITS; ++r)
                    if (r < splits) part[r] = ld_cluster(red + 4 * (c * C::RED_LD + l), r);
#pragma unroll
                for (int r = 0; r < MAX_SPLITS; ++r)
                    if (r < splits) s += part[r];
                p.out[t * p.outs + o] = __float2bfloat16_rn(s);
            }
        }
        cluster_sync();  // (the others have read this CTA's sums)
    }
    tc_fence_before();
    __syncthreads();
    if (C::PAIR) cluster_sync();  // (the pair's products have read this CTA's tiles, and nothing arrives at its barriers any more)
    tc_fence_after();
    if (threadIdx.x == 0 && m->abort) set_status(p.status, KDA_ERR_TIMEOUT);
    if (warp == 3) dealloc<C::PAIR>(tmem, C::TMEM);
}

template <int BN, bool SWAP>
cudaError_t launch(Params &p, const void *x, const void *w, int64_t width, int splits, int sms, cudaStream_t stream) {
    using C = Cfg<BN, SWAP>;
    constexpr int SMEM = C::OFF_MISC + static_cast<int>(sizeof(Misc)) + 1024;
    static_assert(SMEM * C::CTAS <= 227 * 1024, "shared memory");
    static_assert(AHEAD == 4, "a block's scale is picked among four");
    static_assert(C::STAGES >= 2 && (!C::PAIR || C::STAGES % 2 == 0) && C::STAGES * C::STAGE / 16 < 0x3fff, "see the MMAs' warps");
    static_assert(!SWAP || BN * C::RED_LD * 4 <= C::STAGES * C::STAGE, "a cluster's sums lie over the stages");
    const auto kernel = kda_scaled_matmul_kernel<BN, SWAP>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    if (C::UNEVEN) {
        static const int regs = [] {
            cudaFuncAttributes f{};
            return cudaFuncGetAttributes(&f, kda_scaled_matmul_kernel<BN, SWAP>) == cudaSuccess ? f.numRegs : 0;
        }();
        if (regs != C::REGS) return cudaErrorInvalidConfiguration;  // the warps' register split adds up to this
    }
    const int lanes = SWAP ? p.outs : p.rows, cols = SWAP ? p.rows : p.outs;
    auto operand = [&](CUtensorMap *m, const void *at, int64_t n, int box_rows) {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(n)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(width)};
        const cuuint32_t box[2] = {KB, static_cast<cuuint32_t>(box_rows)};
        return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, at, 2, dims, strides, box);
    };
    if (!operand(&p.a, SWAP ? w : x, lanes, LANES) || !operand(&p.b, SWAP ? x : w, cols, C::B_BOX)) return cudaErrorInvalidValue;
    p.tiled_y = 0;
    if (!SWAP && p.outs % 8 == 0) {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.outs), static_cast<cuuint64_t>(p.rows)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.outs) * 2};
        const cuuint32_t box[2] = {static_cast<cuuint32_t>(C::PANEL), 32};
        if (!encode_map(&p.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.out, 2, dims, strides, box,
                        C::PANEL == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
        p.tiled_y = 1;
    }
    p.lane_tiles = (lanes - 1) / (C::PAIR ? 2 * LANES : LANES) + 1;
    p.col_tiles = (cols - 1) / BN + 1;
    const int64_t tiles = static_cast<int64_t>(p.lane_tiles) * p.col_tiles;
    if (tiles > 0x7fffffffLL / 16) return cudaErrorInvalidValue;  // (y would be larger than any memory)
    p.tiles = static_cast<int32_t>(tiles);
    p.splits = splits;
    if (splits == 1 && !C::PAIR) {
        const int64_t most = static_cast<int64_t>(sms) * C::CTAS;
        kernel<<<static_cast<int>(tiles < most ? tiles : most), THREADS, SMEM, stream>>>(p);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(C::PAIR ? 2 * (p.tiles < sms / 2 ? p.tiles : sms / 2) : p.tiles * splits));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(C::PAIR ? 2 : splits);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const Params &>(p));
}

struct Choice {
    int bn, splits;
};
// The least estimated time, in cycles: rounds of CTAs x (blocks x a block's time + a tile's start and end). It is there to order the choices
// and is below what a call takes, most of all for few rows, where reading the weight is not in it. Measured, us a call, in turn on sets of
// tensors larger than L2, * what is taken:
//   rows, channels to outputs    tiles of 64   128    256      rows, channels to outputs    splits 1    2     3     4     5     6     8
//   8192,  2048 to  6144            134.2   111.2   80.5*        7, 12288 to 12288             31.0  29.9  28.7*
//   8192,  2048 to  2048             49.4    40.4   33.0*        7,  8192 to  1024             17.0  11.8   9.4   8.0   7.5   6.9   6.0*
//  16384,  1024 to  1024             29.3    24.8   21.9*       16,  4096 to  4096             11.3   9.6   8.7   8.2*  9.0   9.2   8.9
//   3000,  1024 to 12288             58.7    49.7   38.3*       30, 12288 to  2048             26.5  17.5  13.7  12.0  11.1  10.6  11.2*
//   1024,  2048 to  6144             23.2    20.0   20.1*       32,  4096 to  4096             12.1  10.7   9.4   8.9*  9.8   9.8   9.6
//   1024,  2048 to  2048             10.5     9.4*  11.8        64, 12288 to  2048             34.0  22.8  17.1  14.5  13.1  12.4  13.4*
//    512,  2048 to  2048              8.8*    8.7   10.9        64,  2048 to 12288             11.4* 14.6  13.4
//    256,  2048 to  6176             11.1     9.6*  13.0        64,  2048 to  6176             10.3  11.0  11.5* 10.3  10.1  14.3
//    128, 12288 to  2048             37.1*   31.1   43.0        50,  8192 to  8192             25.2  21.3* 20.0  18.8
// At most 8 % from the best but for the last two of the right and the last of the left (13 to 19 %).
Choice choose(int64_t rows, int64_t outs, int blocks, int sms) {
    auto over = [](int64_t a, int64_t b) { return (a - 1) / b + 1; };
    Choice best{0, 1};
    double least = 0;
    auto offer = [&](int bn, int splits, double t) {
        if (!best.bn || t < least) best = {bn, splits}, least = t;
    };
    if (rows <= SWAP_ROWS) {
        const int bn = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
        const int64_t tiles = over(outs, LANES);
        for (int s = 1; s <= MAX_SPLITS && s <= blocks && (s == 1 || tiles * s <= 2 * static_cast<int64_t>(sms)); ++s)
            offer(bn, s, static_cast<double>(over(tiles * s, sms)) * over(blocks, s) * 500. + (s > 1 ? 2500. : 0.));
        return best;
    }
    auto wide = [&](int bn, int64_t slots, int64_t tiles, double block) {
        offer(bn, 1, static_cast<double>(over(tiles, slots)) * (blocks * block + 1200.));
    };
    const int64_t high = over(rows, LANES), t64 = high * over(outs, 64);
    if (sms > 1) wide(256, sms / 2, over(rows, 2 * LANES) * over(outs, 256), 800.);
    wide(128, sms, high * over(outs, 128), 680.);
    wide(64, 2 * sms, t64, t64 <= sms ? 560. : 830.);
    return best;
}

}  // namespace mm
}  // namespace kda

static kda_status_t scaled_matmul(const void *x, const float *x_scale, int32_t x_scale_per_block, const void *weight,
                                  const float *weight_scale, int64_t rows, int32_t width, int32_t outs, void *y,
                                  int32_t *status_dev, kda_stream_t stream, int32_t withhold) {
    using kda::checks::aligned;
    if (rows < 0 || width < 1 || outs < 1 || (x_scale_per_block != 0 && x_scale_per_block != 1)) return KDA_ERR_INVALID_ARG;
    if (width % 16 != 0) return KDA_ERR_UNSUPPORTED;
    if (rows > 0x7fffffffLL - 128 || width > KDA_MATMUL_MAX || outs > KDA_MATMUL_MAX) return KDA_ERR_UNSUPPORTED;
    if (status_dev && !aligned(status_dev, 4)) return KDA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows > 0) {
        if (!x || !x_scale || !weight || !weight_scale || !y) return KDA_ERR_INVALID_ARG;
        if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(y, 16) || !aligned(x_scale, 4) || !aligned(weight_scale, 4))
            return KDA_ERR_INVALID_ARG;
    }
    if (status_dev && cudaMemsetAsync(status_dev, 0, sizeof(int32_t), s) != cudaSuccess) return KDA_ERR_CUDA;
    if (rows == 0) return KDA_OK;
    const int sms = kda::sm_count();
    if (sms < 1) return KDA_ERR_CUDA;
    kda::mm::Params p{};
    p.xs = x_scale;
    p.ws = weight_scale;
    p.blocks = (width - 1) / kda::mm::KB + 1;
    p.xs_row = x_scale_per_block ? p.blocks : 1;
    p.xs_block = x_scale_per_block;
    p.rows = static_cast<int32_t>(rows);
    p.outs = outs;
    p.out = static_cast<__nv_bfloat16 *>(y);
    p.status = status_dev;
    p.withhold = withhold;
    const kda::mm::Choice c = kda::mm::choose(rows, outs, p.blocks, sms);
    cudaError_t e;
    if (rows <= kda::mm::SWAP_ROWS)
        e = c.bn == 16   ? kda::mm::launch<16, true>(p, x, weight, width, c.splits, sms, s)
            : c.bn == 32 ? kda::mm::launch<32, true>(p, x, weight, width, c.splits, sms, s)
                         : kda::mm::launch<64, true>(p, x, weight, width, c.splits, sms, s);
    else
        e = c.bn == 64    ? kda::mm::launch<64, false>(p, x, weight, width, c.splits, sms, s)
            : c.bn == 128 ? kda::mm::launch<128, false>(p, x, weight, width, c.splits, sms, s)
                          : kda::mm::launch<256, false>(p, x, weight, width, c.splits, sms, s);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status_t kda_scaled_matmul(const void *x, const float *x_scale, int32_t x_scale_per_block, const void *weight,
                                          const float *weight_scale, int64_t rows, int32_t width, int32_t outs, void *y,
                                          int32_t *status_dev, kda_stream_t stream) {
    return scaled_matmul(x, x_scale, x_scale_per_block, weight, weight_scale, rows, width, outs, y, status_dev, stream, -1);
}

extern "C" kda_status_t kda_scaled_matmul_debug(const void *x, const float *x_scale, int32_t x_scale_per_block,
                                                const void *weight, const float *weight_scale, int64_t rows, int32_t width,
                                                int32_t outs, void *y, int32_t *status_dev, kda_stream_t stream,
                                                int32_t withhold) {
    if (withhold < -1) return KDA_ERR_INVALID_ARG;
    return scaled_matmul(x, x_scale, x_scale_per_block, weight, weight_scale, rows, width, outs, y, status_dev, stream, withhold);
}
