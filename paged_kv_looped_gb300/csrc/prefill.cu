// Causal attention over packed prompts for sm_103a.
//
// "Faster fuzzy minds", "LOTUS" / packed prefill: the prompts' tokens lie one sequence after
// another; token i of a sequence attends to its keys 0..i:
//     out_i = sum_{j <= i} softmax_j(scale <q_i, k_j>) v_j,   lse_i = log sum_{j <= i} exp(scale <q_i, k_j>).
// The keys and values are the projection's own rows (or an append's k_out, v_out), not the
// paged pool.
//
// One CTA takes two tiles of 128 query rows that share their keys: at an even group of query heads
// two heads of one kv head at the same tokens, else one head at 256 consecutive tokens.  It
// walks the keys in tiles of 128:
//     S = Q K^T   (128 x 128, K = head_dim)      O += P V   (128 x head_dim, K = 128)
// on tcgen05 (fp32 accumulators in tensor memory: S of both tiles, O of both tiles, 512 columns).
// 4 * 128 * 128 * head_dim flops a tile and key tile take the tensor pipe 1024 clocks at head_dim 128.
// A tile's chain (softmax, then P V and the next S, and the hand-overs between them) takes 2600 clocks where
// two tiles' products alone would take 2048, so the chain bounds long prompts, the tensor pipe 80 %
// busy: 15973 tokens x 64 heads 2510-2575 us (1620-1665 TFLOP/s, 82-84 % of a large cuBLAS product's measured rate).
// Short prompts lose more to each item's first and last key tiles, whose chain is half empty (16 prompts
// of 1024-2000 tokens x 32 heads: 294-302 us, 955-980 TFLOP/s, tensor pipe 52 % busy).
//
// Roles: warps 0-3 / 4-7 softmax of tile 0 / 1 (a thread owns one row = one tensor-memory lane: row maxima and
// sums need no exchange), warp 8 / 9 the MMAs of tile 0 / 1, warp 10 the works and the copies.  The CTAs are
// persistent: each takes over blocks the hardware has not started yet (cluster launch control), so
// that the copies and the first S of the next item run beside the end of the last (8192 tokens x 32
// heads 351 -> 333 us; 16 prompts of 1024-2000 tokens 407 -> 328).  P (bf16) is written over the S
// it came from, in two halves that the products take one by one.  The reference maximum of a row moves only when
// the running maximum exceeds it by 2^8, so O is rescaled rarely, by the row's own thread.
// P in bf16 is the one rounding besides the output's (both operands of a product have one type, and V is bf16): outputs
// are off by 0.0019-0.0020 of themselves where fp32 weights leave 0.0015-0.0016.  The weights' sum is fp32, taken before
// their rounding: taken after it, it would cost the softmax two more instructions a pair, and help only rows in which
// one weight outweighs the rest.
//
// Tried and slower or equal at 8192 tokens x 32 heads: polling instead of suspended waits in the MMA threads
// (351 -> 419 us), no maximum but a limit on the weights' sum (376), one MMA thread for both tiles (350), the
// output written behind the next item's first softmax (326 -> 349), four further warps for the output (320 -> 335:
// the softmax warps then have 176 registers instead of 208), two threads a row (411: the units bound the
// softmax, not one thread's latency).
#include <cuda.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>
#include <vector>

#include "rlt.h"
#include "rlt_device.cuh"
#include "rlt_internal.h"
#include "rlt_tc.cuh"

namespace rlt {
namespace {

constexpr int kTile = 128;                   // query rows, keys of a tile
constexpr int kMmaWarp = 8, kLoadWarp = 10;  // MMA warps 8 and 9: one a tile
constexpr int kThreads = 12 * 32;            // warp 11 only fills the third warpgroup
// Registers a thread: 168 at launch (384 threads); the softmax warpgroups take up what the third one
// gives back: 2 * 208 + 88 = 3 * 168.
constexpr int kRegsSoftmax = 208, kRegsRest = 88;
constexpr float kRescaleThreshold = 8.f;     // log2 units: weights of up to 2^8
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;
constexpr int kPartsFrom = 6;                // items of the largest size an SM's share has to hold
constexpr int64_t kL2Share = 48 << 20;       // of K and V in use at a time (L2 is 126 MB)
constexpr int kOutBytes = 32 * 128;
constexpr int kItemFields = 4;               // first row of the sequence, its length, first query of the item, 0

// The output's staging takes the place of a fifth ring slot at head_dim 128: five slots and no staging 326 us, four
// slots 330, four and the staging 320 (8192 tokens x 32 heads).
template <int D>
struct PCfg {
    static constexpr int kStages = D == 128 ? 4 : 8;             // K/V ring slots
    static constexpr int kBlock = kTile * 128;                   // a 64-dim column block of a tile
    static constexpr int kTileBytes = D / 64 * kBlock;
    static constexpr int kRingOff = 2 * kTileBytes;              // behind the two Q tiles
    static constexpr int kOutOff = kRingOff + kStages * kTileBytes;   // 32 rows x 64 dims of output a softmax warp
    static constexpr int kBarOff = kOutOff + 8 * kOutBytes;
    enum Bar {
        kQFull = 0,                          // [tile] the item's Q landed
        kQFree = kQFull + 2,                 // [tile] read by its last S
        kFull = kQFree + 2,                  // [ring slot] K or V landed
        kFree = kFull + kStages,             // [ring slot] read by both tiles' products
        kSFull = kFree + kStages,            // [tile] S of a key tile written
        kPFull = kSFull + 2,                 // [tile][64 keys] P written by the tile's 4 warps
        kODone = kPFull + 4,                 // [tile] the item's last P V complete
        kOFree = kODone + 2,                 // [tile] O read out by the tile's 4 warps
        kWorkFull = kOFree + 2,              // [2] a work descriptor published
        kWorkFree = kWorkFull + 2,           // [2] every role is done with it
        kNext = kWorkFree + 2,               // the scheduler's answer landed
        kClean = kNext + 1,                  // [2 works][tile] V of the tile's last keys looked at (a pair's tiles: [0])
        kNumBars = kClean + 4
    };
    static constexpr int kWorkOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;   // two Work
    static constexpr int kNextOff = kWorkOff + 32;               // the scheduler's 16-byte answer
    static constexpr int kBadOff = kNextOff + 16;                // [2 works][softmax warp] rows with non-finite values
    static constexpr int kFlagOff = kBadOff + 64;
    static constexpr int kSmem = kFlagOff + 16 + 1024;
    static_assert(kNumBars <= kThreads, "a thread a barrier at the start");
};

// One work item: query rows q0.. of a sequence (rows row0 .. row0 + len - 1) for one unit of heads.
struct Work {
    int32_t row0, len, q0, unit;             // len 0: nothing to do; -1: no more work
};

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z,
                                            uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// The box at (x, y, z) from shared memory, as a bulk group of the calling thread.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int32_t x, int32_t y, int32_t z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
                 : "memory");
}

// Cluster launch control: asks the hardware scheduler for the block of this grid it would start next.  The
// 16-byte answer lands in shared memory and completes 16 bytes of the barrier's transaction count.
__device__ __forceinline__ void ask_for_block(void *answer, uint64_t *bar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}

// The block number of an answer, or -1 when the grid has no block left to start.
__device__ __forceinline__ int answered_block(const void *answer)
{
    int32_t x, got;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.b32 %1, 1, 0, p;\n\t"
        "mov.b32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, h;\n\t}"
        : "=r"(x), "=r"(got)
        : "r"(smem_u32(answer))
        : "memory");
    return got != 0 ? x : -1;
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const volatile int *abort, uint64_t limit)
{
    return __all_sync(kFullMask, mbar_wait_or_abort(bar, parity, abort, limit));
}

// 2^x, kept in program order among volatile instructions.
__device__ __forceinline__ float exp2_in_order(float x)
{
    float r;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 32 bytes to a 32-byte aligned address.
__device__ __forceinline__ void store_sector(void *dst, const uint32_t (&y)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(y[0]), "r"(y[1]), "r"(y[2]),
                 "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                 : "memory");
}

// Whether a word of two bf16 values holds an infinity or NaN, from the larger magnitude's bits.
__device__ __forceinline__ bool not_finite(uint32_t bits) { return (bits & 0xffffu) >= 0x7f80u || bits >= 0x7f800000u; }

// kFault: the timeout test's instance (rlt_debug_fault_next_decode): one copy left unissued, the limit from the call.
template <int D, bool kFault>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap,
                   const PrefillParams p)
{
    using C = PCfg<D>;
    constexpr int kBlocks = D / 64;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *base =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + C::kBarOff);
    volatile Work *works = reinterpret_cast<volatile Work *>(base + C::kWorkOff);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(base + C::kFlagOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + C::kFlagOff + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // The CTA is set up while the kernel ahead ends. Without the early start nothing is read before it has, and
    // the kernel behind starts no earlier either.
    if (p.early != 0)
        pdl_launch_dependents();

    const int G = p.num_q_heads / p.num_kv_heads;
    const bool pair = G % 2 == 0;                // tile 1: the next head, else the next 128 tokens
    const int units = pair ? p.num_q_heads / 2 : p.num_q_heads;
    const int head_step = pair ? 1 : 0, tok_step = pair ? 0 : kTile;

    // The load warp's first round trips go out before the CTA is set up: the maps, and the first work's item.
    auto find = [&](int block) -> Work {
        // items in the plan's order for chunk_units units of heads, then for the next ones
        const int chunk = block / (p.num_items * p.chunk_units), first = chunk * p.chunk_units;
        const int rest = block - p.num_items * first, width = min(p.chunk_units, units - first);
        const int item = rest / width;
        const int32_t *it = p.items + (int64_t)item * kItemFields;
        return Work{it[0], it[1], it[2], first + rest - item * width};
    };
    Work first_work{0, 0, 0, 0};
    if (warp == kLoadWarp) {
        if (lane == 0) {
            tc::prefetch_tmap(&qmap);
            tc::prefetch_tmap(&kmap);
            tc::prefetch_tmap(&vmap);
            tc::prefetch_tmap(&omap);
        }
        if (p.early != 0)
            first_work = find(blockIdx.x);
    }
    if (tid < C::kNumBars) {
        const int i = tid;
        int count = 1;
        if (i >= C::kFree && i < C::kSFull)
            count = 2;                           // both tiles' MMA threads
        else if ((i >= C::kPFull && i < C::kODone) || (i >= C::kOFree && i < C::kWorkFull))
            count = 4;                           // the tile's softmax warps
        else if (i >= C::kWorkFree && i < C::kNext)
            count = 10;                          // two MMA threads, eight softmax warps
        else if (i >= C::kClean)
            count = pair ? 8 : 4;                // the softmax warps that look
        mbar_init(&bars[i], count);
        *abort_flag = 0;
        *(abort_flag + 1) = 0;
        mbar_init_fence();
    }
    if (tid < 16)
        reinterpret_cast<uint32_t *>(base + C::kBadOff)[tid] = 0u;
    if (warp == kMmaWarp) {
        pdl_wait();                              // the kernel ahead may still have tensor memory to allocate
        tc::tmem_alloc(tslot, kTmemCols);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;
    bool ok = true;
    const uint64_t limit = kFault ? p.wait_limit_ns : kWaitLimitNs;

    // Every role goes through the same works; key tiles of tile s: up to its last row's own key.
    auto take = [&](int d, Work &w) {            // (the barrier has been waited for)
        w.row0 = works[d & 1].row0;
        w.len = works[d & 1].len;
        w.q0 = works[d & 1].q0;
        w.unit = works[d & 1].unit;
    };
    auto key_tiles = [&](const Work &w, int s) -> int {
        return w.len <= w.q0 + s * tok_step ? 0 : w.q0 / kTile + 1 + s * (tok_step / kTile);
    };

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp == kLoadWarp && tc::elect_one()) {
            // ------------------------------------------------- works and copies
            // The CTA's own block first, then the ones the hardware scheduler hands over instead of starting
            // them: the items keep their order, and a CTA's start is paid once.  The next work is asked
            // for while this one's copies are issued.  Ring order K0, V0, K1, V1, ...; rows behind
            // the last one of the array read as zeros.
            pdl_wait();
            if (p.early == 0) {
                pdl_launch_dependents();
                first_work = find(blockIdx.x);
            }
            auto load = [&](unsigned char *dst, const CUtensorMap *map, int head, int row, uint64_t *bar) {
                mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
                    tma_load_3d(dst + b * C::kBlock, map, b * 64, head, row, bar);
            };
            int block = blockIdx.x, st = 0, issued = 0, queries[2] = {0, 0};
            bool asked = false;
            uint32_t parity = 1;                 // of the slot's previous release (none in the first round)
            for (int d = 0;; ++d) {
                if (d >= 2 && !(ok = mbar_wait_or_abort(&bars[C::kWorkFree + (d & 1)], (d / 2 - 1) & 1u, abort_flag, limit)))
                    break;
                Work w{0, -1, 0, 0};
                if (block >= 0) {
                    w = d == 0 ? first_work : find(block);
                    if (w.row0 < 0 || w.len < 1 || w.len > p.num_rows - w.row0 || w.q0 < 0 || w.q0 >= w.len ||
                        w.q0 % kTile != 0) {
                        record_error(p.err, RLT_DEVERR_BAD_LEN);   // a plan of other sequences
                        w.len = w.q0 = 0;
                    }
                }
                works[d & 1].row0 = w.row0;
                works[d & 1].len = w.len;
                works[d & 1].q0 = w.q0;
                works[d & 1].unit = w.unit;
                mbar_arrive(&bars[C::kWorkFull + (d & 1)]);
                if (w.len < 0)
                    break;
                mbar_arrive_expect_tx(&bars[C::kNext], 16);
                ask_for_block(base + C::kNextOff, &bars[C::kNext]);
                asked = true;
                const int head0 = pair ? 2 * w.unit : w.unit, kv_head = head0 / G;
                const int n = max(key_tiles(w, 0), key_tiles(w, 1));
                for (int i = 0; ok && i < 2 * n; ++i) {
                    if (i < 2) {
                        if (d > 0 && !(ok = mbar_wait_or_abort(&bars[C::kQFree + i], (d - 1) & 1u, abort_flag, limit)))
                            break;
                        if (key_tiles(w, i) > 0) {
                            load(base + i * C::kTileBytes, &qmap, head0 + i * head_step, w.row0 + w.q0 + i * tok_step,
                                 &bars[C::kQFull + i]);
                            queries[i] = 1;
                        } else {
                            mbar_arrive(&bars[C::kQFull + i]);
                        }
                    }
                    if (issued >= C::kStages && !(ok = mbar_wait_or_abort(&bars[C::kFree + st], parity, abort_flag, limit)))
                        break;
                    if (kFault && blockIdx.x == 0 && d == 0 && i == 1)
                        mbar_arrive_expect_tx(&bars[C::kFull + st], C::kTileBytes);   // these bytes never arrive
                    else
                        load(base + C::kRingOff + st * C::kTileBytes, (i & 1) ? &vmap : &kmap, kv_head,
                             w.row0 + (i >> 1) * kTile, &bars[C::kFull + st]);
                    ++issued;
                    if (++st == C::kStages) {
                        st = 0;
                        parity ^= 1u;
                    }
                }
                if (n == 0) {                    // (keeps the Q barriers' phases one a work)
                    for (int i = 0; ok && i < 2; ++i) {
                        if (d > 0)
                            ok = mbar_wait_or_abort(&bars[C::kQFree + i], (d - 1) & 1u, abort_flag, limit);
                        mbar_arrive(&bars[C::kQFull + i]);
                    }
                }
                if (!ok || !(ok = mbar_wait_or_abort(&bars[C::kNext], d & 1u, abort_flag, limit)))
                    break;
                asked = false;
                block = answered_block(base + C::kNextOff);
                fence_proxy_async();             // the answer has been read before the next one is written
            }
            if (!ok) {
                *abort_flag = 1;
                // every copy and the scheduler's answer have landed before the CTA gives up its memory (bounded;
                // on the normal path the other roles have waited for all of them)
                for (int i = max(0, issued - C::kStages); i < issued; ++i)
                    mbar_wait(&bars[C::kFull + i % C::kStages], (i / C::kStages) & 1u, limit);
                for (uint64_t t0 = global_ns(); (asked || queries[0] || queries[1]) && global_ns() - t0 < kWaitLimitNs / 100;)
                    ;
            }
        } else if (warp < kLoadWarp && tc::elect_one()) {
            // ---------------------------------------------------------- products
            // One thread a tile, in the order S | PV S' | PV' S'' ...: MMAs of one thread run in issue order, so S of
            // the next key tile may overwrite the P that the PV before it reads.  An MMA keeps the tensor pipe 64
            // clocks, so its issue has to take less: descriptors advance by constants (computed anew for each
            // MMA, they bounded the kernel: 476 us where these take 376, 8192 tokens x 32 heads).
            const int s = warp - kMmaWarp;
            constexpr uint32_t id_s = tc::instr_desc_bf16(128, 128, false);
            constexpr uint32_t id_o = tc::instr_desc_bf16(128, D, true);
            // Descriptors: the low words (address and leading offset, both in 16 bytes) advance, the high word
            // (stride 1024, 128-byte swizzle) is tc::smem_desc's constant.
            constexpr uint32_t kTileStep = C::kTileBytes >> 4, kBlockStep = C::kBlock >> 4;
            const uint32_t qd = (uint32_t)tc::smem_desc(smem_u32(base), 16, 1024) + s * kTileStep;
            const uint32_t kd = (uint32_t)tc::smem_desc(smem_u32(base + C::kRingOff), 16, 1024);
            const uint32_t vd = (uint32_t)tc::smem_desc(smem_u32(base + C::kRingOff), C::kBlock, 1024);
            auto desc = [&](uint32_t low) -> uint64_t {
                constexpr uint32_t kHigh = (1024 >> 4) | (1u << 14) | (2u << 29);
                return ((uint64_t)kHigh << 32) | low;
            };
            const uint32_t t_s = tmem + kColS + s * kTile, t_o = tmem + kColO + s * kTile;
            auto issue_s = [&](int slot) {
                const uint32_t b = kd + slot * kTileStep;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t at = (kk >> 2) * kBlockStep + (kk & 3) * 2;
                    tc::mma_bf16(t_s, desc(qd + at), desc(b + at), id_s, kk > 0);
                }
                tc::mma_commit(&bars[C::kSFull + s]);
            };
            auto issue_pv = [&](int half, int slot, bool first) {             // 64 keys
                const uint32_t b = vd + slot * kTileStep + half * (4 * 2048 >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc::mma_bf16_ta(t_o, t_s + half * 32 + kk * 8, desc(b + kk * (2048 >> 4)), id_o, kk > 0 || !first);
            };
            // ring slot and parity of the next copy to be waited for
            int st = 0;
            uint32_t parity = 0;
            auto wait_slot = [&](int &slot) -> bool {
                slot = st;
                if (!mbar_wait_or_abort(&bars[C::kFull + st], parity, abort_flag, limit))
                    return false;
                if (++st == C::kStages) {
                    st = 0;
                    parity ^= 1u;
                }
                return true;
            };
            // a tile without work on a copy lets it go at once
            auto release = [&](int bar, bool used) {
                if (used)
                    tc::mma_commit(&bars[bar]);
                else
                    mbar_arrive(&bars[bar]);
            };
            // P V and the S behind it are issued as one: the two threads' MMAs would else alternate, both tiles' S
            // would come at the same time, and both softmaxes would then want the same units at once (8 ragged
            // prompts 171 -> 164 us, 8192 tokens x 16 heads of 2 kv heads 200 -> 166).
            volatile int *turn = abort_flag + 1;
            auto take_turn = [&]() -> bool {
                for (uint32_t it = 1; it != 0; ++it) {
                    if (atomicCAS(const_cast<int *>(turn), 0, 1) == 0)
                        return true;
                    if ((it & 1023u) == 0u && *abort_flag != 0)
                        return false;
                }
                return false;
            };
            auto pass_turn = [&]() { *turn = 0; };
            int tiles = 0, items = 0, s_issued = 0;   // key tiles and works with rows, over all works
            for (int d = 0;; ++d) {
                if (!(ok = mbar_wait_or_abort(&bars[C::kWorkFull + (d & 1)], (d / 2) & 1u, abort_flag, limit)))
                    break;
                Work w;
                take(d, w);
                if (w.len < 0)
                    break;
                const int ns0 = key_tiles(w, 0), ns = key_tiles(w, s), n = max(ns0, key_tiles(w, 1));
                uint64_t *clean = &bars[C::kClean + (d & 1) * 2];
                int k_slot = 0, v_slot = 0;
                if (!(ok = mbar_wait_or_abort(&bars[C::kQFull + s], d & 1u, abort_flag, limit)))
                    break;
                if (n > 0) {
                    if (!(ok = wait_slot(k_slot)))
                        break;
                    if (ns > 0) {
                        issue_s(k_slot);
                        ++s_issued;
                    }
                    release(C::kFree + k_slot, ns > 0);
                }
                if (ns <= 1)
                    release(C::kQFree + s, ns > 0);
                for (int j = 0; ok && j < n; ++j) {
                    if (!(ok = wait_slot(v_slot)) || (j + 1 < n && !(ok = wait_slot(k_slot))))
                        break;
                    if (j < ns) {
                        // The values of the last keys have been looked at: a pair's tiles share them, and at an odd group
                        // tile 0's last keys are ordinary ones of tile 1.  (Waited for before the turn is taken.)
                        if (j == ns0 - 1 && !(ok = mbar_wait_or_abort(&clean[0], (d / 2) & 1u, abort_flag, limit)))
                            break;
                        if (!pair && s == 1 && j == ns - 1 &&
                            !(ok = mbar_wait_or_abort(&clean[1], (d / 2) & 1u, abort_flag, limit)))
                            break;
                        // the item before has left O
                        if (j == 0 && items > 0 &&
                            !(ok = mbar_wait_or_abort(&bars[C::kOFree + s], (items - 1) & 1u, abort_flag, limit)))
                            break;
                        if (!(ok = mbar_wait_or_abort(&bars[C::kPFull + 2 * s], tiles & 1u, abort_flag, limit)))
                            break;
                        if (!(ok = take_turn()))
                            break;
                        tc::fence_after_sync();
                        issue_pv(0, v_slot, j == 0);
                        if (!(ok = mbar_wait_or_abort(&bars[C::kPFull + 2 * s + 1], tiles & 1u, abort_flag, limit)))
                            break;
                        tc::fence_after_sync();
                        issue_pv(1, v_slot, false);
                        ++tiles;
                        if (j + 1 < ns) {
                            issue_s(k_slot);
                            ++s_issued;
                            if (j + 2 == ns)
                                tc::mma_commit(&bars[C::kQFree + s]);
                        } else {
                            tc::mma_commit(&bars[C::kODone + s]);
                            ++items;
                        }
                        pass_turn();
                    }
                    release(C::kFree + v_slot, j < ns);
                    if (j + 1 < n)
                        release(C::kFree + k_slot, j + 1 < ns);
                }
                if (!ok)
                    break;
                mbar_arrive(&bars[C::kWorkFree + (d & 1)]);
            }
            if (!ok)
                *abort_flag = 1;
            // every issued MMA is complete before the CTA gives up its memory (bounded).  On the normal path the
            // last ODone covers all; after an abort, the last S and some time for a P V half behind it
            if (ok) {
                if (items > 0)
                    mbar_wait(&bars[C::kODone + s], (items - 1) & 1u, limit);
            } else {
                if (s_issued > 0)
                    mbar_wait(&bars[C::kSFull + s], (s_issued - 1) & 1u, limit);
                for (uint64_t t0 = global_ns(); global_ns() - t0 < kWaitLimitNs / 100;)
                    ;
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---------------------------------------------------------- softmax
        const int s = warp >> 2, quarter = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t t_s = t_lane + kColS + s * kTile, t_o = t_lane + kColO + s * kTile;
        auto p_ready = [&](int half) {           // this warp's P of 64 keys is in tensor memory
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars[C::kPFull + 2 * s + half]);
        };
        int tiles = 0, items = 0, copies = 0;    // of this tile, and of the ring before this work
        for (int d = 0;; ++d) {
            if (!(ok = warp_wait(&bars[C::kWorkFull + (d & 1)], (d / 2) & 1u, abort_flag, limit)))
                break;
            Work wk;
            take(d, wk);
            if (wk.len < 0)
                break;
            const int ns = key_tiles(wk, s), n = max(key_tiles(wk, 0), key_tiles(wk, 1));
            const int q_tok = wk.q0 + s * tok_step + quarter * 32 + lane;    // this thread's query, in its sequence
            const int head0 = pair ? 2 * wk.unit : wk.unit;
            volatile uint32_t *bad = reinterpret_cast<volatile uint32_t *>(base + C::kBadOff) + (d & 1) * 8;
            if (ns == 0 && lane == 0)
                mbar_arrive(&bars[C::kClean + (d & 1) * 2 + (pair ? 0 : s)]);
            float m_ref = 0.f, l_run = 0.f;
            bool m_set = false;
            for (int j = 0; j < ns; ++j, ++tiles) {
                if (j == ns - 1) {
                    // The tile of the row's own keys: weights of masked keys are 0, but 0 times an infinity or NaN
                    // would stay.  Rows of V past the sequence (they may hold anything) become zeros, and so do
                    // single values that are not finite; their rows are noted, and the epilogue adds what
                    // a query may see of them.  It is done while S is computed, each row by one warp, and every product
                    // that reads these values waits for all of them.  A pair's tiles have the same last keys: 16 rows a
                    // warp, two lanes a row (at head_dim 128 the second starts four chunks on, in other banks); else
                    // 32 rows of the tile's own, a lane a row.  (One further warp for all of it took 321 us where this
                    // takes 298, 16 prompts of 1024-2000 tokens x 32 heads.)
                    const int i = copies + 2 * j + 1;
                    if (!(ok = warp_wait(&bars[C::kFull + i % C::kStages], (i / C::kStages) & 1u, abort_flag, limit)))
                        break;
                    unsigned char *vt = base + C::kRingOff + i % C::kStages * C::kTileBytes;
                    const int r = pair ? warp * 16 + (lane >> 1) : quarter * 32 + lane;
                    const bool inside = r < wk.len - j * kTile;
                    auto chunk = [&](int half, int c) -> uint4 * {
                        const int at = D == 128 ? half * C::kBlock + r * 128 + (((c ^ (half << 2) ^ r) & 7) << 4)
                                                : r * 128 + ((((half << 2) + c) ^ r) & 7) * 16;
                        return reinterpret_cast<uint4 *>(vt + at);
                    };
                    uint32_t big = 0u;
#pragma unroll 1
                    for (int half = pair ? lane & 1 : 0; half < (pair ? (lane & 1) + 1 : 2); ++half)
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            const uint4 x = *chunk(half, c);
                            big = __vmaxu2(big, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                                         __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
                        }
                    const unsigned odd = __ballot_sync(kFullMask, inside && not_finite(big));
                    if (lane == 0)
                        bad[warp] = odd;
                    if (!inside || not_finite(big)) {
#pragma unroll 1
                        for (int c = 0; c < (pair ? D / 16 : D / 8); ++c) {
                            uint4 *at = pair ? chunk(lane & 1, c) : chunk(c / (D / 16), c % (D / 16));
                            uint4 x = *at;
                            auto finite = [&](uint32_t y) -> uint32_t {
                                if (!inside)
                                    return 0u;
                                return ((y & 0x7f80u) == 0x7f80u ? 0u : y & 0xffffu) |
                                       ((y & 0x7f800000u) == 0x7f800000u ? 0u : y & 0xffff0000u);
                            };
                            *at = make_uint4(finite(x.x), finite(x.y), finite(x.z), finite(x.w));
                        }
                        fence_proxy_async();     // (generic writes before the products' reads)
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bars[C::kClean + (d & 1) * 2 + (pair ? 0 : s)]);
                }
                if (!(ok = warp_wait(&bars[C::kSFull + s], tiles & 1u, abort_flag, limit)))
                    break;
                tc::fence_after_sync();
                // P = 2^(s - m), 32 columns at a time.  The exponentials of the next columns are issued ahead of the
                // conversions of the last ones.
                uint64_t sum2[2] = {0ull, 0ull};
                auto raise = [&](const float (&x)[32], float (&y)[32]) {
                    const uint64_t sc2 = f2_pack(p.qscale, p.qscale), off2 = f2_pack(-m_ref, -m_ref);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 z = f2_unpack(f2_fma(f2_pack(x[2 * i], x[2 * i + 1]), sc2, off2));
                        y[2 * i] = exp2_in_order(z.x);
                        y[2 * i + 1] = exp2_in_order(z.y);
                    }
                };
                auto store = [&](const float (&y)[32], int c) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[i] = cvt_bf16x2(y[2 * i], y[2 * i + 1]);
                    tc::tmem_st_nowait<16>(t_s + c * 16, w);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sum2[i & 1] = f2_add(sum2[i & 1], f2_pack(y[2 * i], y[2 * i + 1]));
                };
                auto top = [&](float m, const float (&x)[32]) -> float {     // the larger of m and the columns', four chains
                    float mx[4] = {m, x[0], x[1], x[2]};
#pragma unroll
                    for (int i = 3; i < 31; i += 2)
                        mx[(i >> 1) & 3] = fmaxf(fmaxf(mx[(i >> 1) & 3], x[i]), x[i + 1]);
                    return fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), x[31]);
                };
                // The reference moves up to the row's maximum where that exceeds it by 2^8, and O and the sum with it;
                // the first finite score sets it.  (S of this tile is behind the products of the last: O is at
                // rest.)
                auto move = [&](float mx, bool up) {
                    const float m_next = up ? mx : m_ref;
                    const float by = up && m_set ? fast_exp2(m_ref - m_next) : 1.f;
                    m_ref = m_next;
                    m_set = m_set || up;
                    if (j == 0)
                        return;
                    l_run *= by;
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        float o[16];
                        uint32_t ow[16];
                        tc::tmem_ld<16>(t_o + c * 16, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            ow[i] = __float_as_uint(o[i] * by);
                        tc::tmem_st_nowait<16>(t_o + c * 16, ow);
                    }
                };
                // (a row without a finite score waits for one; NaN scores stay NaN)
                auto must_move = [&](float mx) -> bool {
                    return mx > -CUDART_INF_F && (!m_set || mx > m_ref + kRescaleThreshold);
                };
                if (j < ns - 1) {
                    float v[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tc::tmem_ld32_nowait(t_s + c * 32, v[c]);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        tc::tmem_wait_ld(v[c]);
                    // The first columns' weights are made against the reference the row has, beside the row's
                    // maximum: it moves rarely, and then they are made again.
                    float y0[32];
                    raise(v[0], y0);
                    const float mx = fmaxf(fmaxf(top(-CUDART_INF_F, v[0]), top(-CUDART_INF_F, v[1])),
                                           fmaxf(top(-CUDART_INF_F, v[2]), top(-CUDART_INF_F, v[3]))) * p.qscale;
                    if (__any_sync(kFullMask, must_move(mx))) {
                        move(mx, must_move(mx));
                        raise(v[0], y0);
                    }
                    raise(v[1], v[1]);
                    store(y0, 0);
                    raise(v[2], v[2]);
                    store(v[1], 1);
                    p_ready(0);                  // the first 64 keys' weights
                    raise(v[3], v[3]);
                    store(v[2], 2);
                    store(v[3], 3);
                    p_ready(1);
                } else {
                    // The row's own keys: a warp's rows see the 32 columns before its quarter whole, its quarter's up
                    // to their own, and none behind, whose weights are zeros without an exponential.
                    // Read twice, 32 columns at a time: P of columns c is stored over scores of columns c / 2.
                    float mx = -CUDART_INF_F;
#pragma unroll 1
                    for (int c = 0; c <= quarter; ++c) {
                        float v[32];
                        tc::tmem_ld32(t_s + c * 32, v);
                        if (c == quarter) {
#pragma unroll
                            for (int i = 1; i < 32; ++i)
                                v[i] = i <= lane ? v[i] : -CUDART_INF_F;
                        }
                        mx = top(mx, v);
                    }
                    mx *= p.qscale;
                    if (__any_sync(kFullMask, must_move(mx)))
                        move(mx, must_move(mx));
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        if (c <= quarter) {
                            float v[32];
                            tc::tmem_ld32(t_s + c * 32, v);
                            if (c == quarter) {
#pragma unroll
                                for (int i = 1; i < 32; ++i)
                                    v[i] = i <= lane ? v[i] : -CUDART_INF_F;
                            }
                            raise(v, v);
                            store(v, c);
                        } else {
                            tc::tmem_zero_nowait<16>(t_s + c * 16);
                        }
                        if (c & 1)
                            p_ready(c >> 1);
                    }
                }
                const float2 sum = f2_unpack(f2_add(sum2[0], sum2[1]));
                l_run += sum.x + sum.y;
            }
            if (ok && ns > 0 && (ok = warp_wait(&bars[C::kODone + s], items & 1u, abort_flag, limit))) {
                tc::fence_after_sync();
                ++items;
                const float inv = 1.f / l_run;
                const int64_t at = (int64_t)(wk.row0 + q_tok) * p.num_q_heads + head0 + s * head_step;
                // Rows of V with values that are not finite, of the keys from q0 on: the last ones of a pair, or of tile
                // 0 (ordinary ones of tile 1) and then of tile 1.  P V has waited for these barriers, so they have
                // completed; the probes order the notes' reads behind them (waits here took 303 us for 298).
                const int words = pair || s == 1 ? 8 : 4;
                mbar_test_wait(&bars[C::kClean + (d & 1) * 2], (d / 2) & 1u);
                mbar_test_wait(&bars[C::kClean + (d & 1) * 2 + s], (d / 2) & 1u);
                uint32_t any_bad = 0u;
                for (int i = 0; i < words; ++i)
                    any_bad |= bad[i];
                float o[D / 32][32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    tc::tmem_ld32_nowait(t_o + c * 32, o[c]);
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    tc::tmem_wait_ld(o[c]);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars[C::kOFree + s]);
                if (any_bad != 0u) {
#pragma unroll 1
                    for (int b = 0; b < words * 32; b += pair ? 2 : 1) {     // (a pair: a row has two bits, for its halves)
                        const int key = wk.q0 + (pair ? b >> 1 : b);
                        if (((bad[b >> 5] >> (b & 31)) & (pair ? 3u : 1u)) == 0u || key > q_tok || key >= wk.len)
                            continue;
                        const uint16_t *vr = p.v + (int64_t)(wk.row0 + key) * p.v_stride + (int64_t)(head0 / G) * D;
#pragma unroll
                        for (int c = 0; c < D; ++c) {
                            const uint32_t x = vr[c];
                            if ((x & 0x7f80u) == 0x7f80u)
                                o[c / 32][c % 32] += __uint_as_float(x << 16);
                        }
                    }
                }
                // The warp's rows, 64 dims at a time, through shared memory and a tensor copy: a lane's row is a line
                // of its own for every store instruction, and 8 warps' stores of that kind held up the shared-
                // memory pipe (and with it every barrier of the CTA) for 2300 clocks a tile.  Rows at the end
                // of a sequence are stored directly: the copy's box would reach into the next one's.
                if (q_tok - lane + 31 < wk.len) {
                    unsigned char *mine = base + C::kOutOff + warp * kOutBytes;
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) {
                        if (lane == 0)
                            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the last copy has read it
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float *x = &o[2 * b + c / 4][c % 4 * 8];
                            *reinterpret_cast<uint4 *>(mine + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                                make_uint4(cvt_bf16x2(x[0] * inv, x[1] * inv), cvt_bf16x2(x[2] * inv, x[3] * inv),
                                           cvt_bf16x2(x[4] * inv, x[5] * inv), cvt_bf16x2(x[6] * inv, x[7] * inv));
                        }
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0)
                            tma_store_3d(&omap, mine, b * 64, head0 + s * head_step, wk.row0 + q_tok);
                    }
                } else if (q_tok < wk.len) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const float *x = &o[i / 2][i % 2 * 16];
                        uint32_t y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            y[k] = cvt_bf16x2(x[2 * k] * inv, x[2 * k + 1] * inv);
                        store_sector(p.out + at * D + i * 16, y);
                    }
                }
                if (q_tok < wk.len) {
                    if (p.lse_out != nullptr)
                        p.lse_out[at] = (m_ref + log2f(l_run)) * 0.6931471805599453f;
                }
            }
            if (!ok)
                break;
            copies += 2 * n;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars[C::kWorkFree + (d & 1)]);
        }
        if (!ok) {
            *abort_flag = 1;
            tc::tmem_wait_st();                  // (no store is under way when the tensor memory is given back)
        }
        if (lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");        // the output has left shared memory
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (tid == 0 && *abort_flag != 0)
        record_error(p.err, RLT_DEVERR_TIMEOUT);
    if (warp == kMmaWarp)
        tc::tmem_dealloc(tmem, kTmemCols);
}

// Token rows of `heads` x D bf16, `stride` elements apart; boxes of box_rows tokens x 64 dims of one head.
bool make_rows_map(CUtensorMap *map, const uint16_t *ptr, int64_t rows, int heads, int D, int64_t stride,
                   int box_rows = kTile)
{
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    const tc::EncodeTiledFn fn = tc::encode_tiled_fn();
    return fn != nullptr && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(ptr), dims, strides, box,
                               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kFault>
cudaError_t launch_prefill_typed(const PrefillParams &p, cudaStream_t stream, bool early)
{
    using C = PCfg<D>;
    static_assert(C::kSmem <= 227 * 1024, "shared memory of one CTA");
    CUtensorMap qmap, kmap, vmap, omap;
    if (!make_rows_map(&qmap, p.q, p.num_rows, p.num_q_heads, D, p.q_stride) ||
        !make_rows_map(&kmap, p.k, p.num_rows, p.num_kv_heads, D, p.k_stride) ||
        !make_rows_map(&vmap, p.v, p.num_rows, p.num_kv_heads, D, p.v_stride) ||
        !make_rows_map(&omap, p.out, p.num_rows, p.num_q_heads, D, (int64_t)p.num_q_heads * D, 32))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit == 0 || (configured.load(std::memory_order_acquire) & bit) == 0) {
        e = cudaFuncSetAttribute(prefill_kernel<D, kFault>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess)
            return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    // The items of a unit re-read its kv head's rows.  Where the rows of all kv heads overflow L2, and the largest
    // item is small beside an SM's share of the work (the order by size then starts anew a few times), as
    // many kv heads run through the plan at a time as keep theirs in L2.  16 prompts of 1024-2000 tokens, 32 kv
    // heads, 400 MB of K and V: 299 us in parts, 318 in one; one prompt of 2048 tokens, 128 kv heads: 131
    // in parts, 123 in one (an item is a quarter of an SM's share there).
    const int G = p.num_q_heads / p.num_kv_heads, per_kv = G % 2 == 0 ? G / 2 : G;
    const int64_t kv_bytes = (int64_t)p.num_rows * D * 4;
    int64_t kv_heads = std::min<int64_t>(std::max<int64_t>(kL2Share / kv_bytes, 1), p.num_kv_heads);
    if ((int64_t)p.total_tiles * per_kv * p.num_kv_heads < (int64_t)kPartsFrom * p.num_sms * p.max_tiles)
        kv_heads = p.num_kv_heads;
    PrefillParams c = p;
    c.chunk_units = (int32_t)kv_heads * per_kv;
    c.early = early ? 1 : 0;
    return launch_kernel(prefill_kernel<D, kFault>, dim3(p.num_items * per_kv * p.num_kv_heads), dim3(kThreads), C::kSmem,
                         stream, true, qmap, kmap, vmap, omap, c);
}

}  // namespace

cudaError_t launch_prefill(const PrefillParams &p, int head_dim, cudaStream_t stream, bool early)
{
    if (p.wait_limit_ns != 0)
        return head_dim == 128 ? launch_prefill_typed<128, true>(p, stream, early)
                               : launch_prefill_typed<64, true>(p, stream, early);
    return head_dim == 128 ? launch_prefill_typed<128, false>(p, stream, early)
                           : launch_prefill_typed<64, false>(p, stream, early);
}

}  // namespace rlt

// ------------------------------------------------------------- host planner

extern "C" RLT_API rlt_status rlt_plan_prefill(const int32_t *seq_lens, int32_t batch, int32_t query_group,
                                               int32_t *items, int32_t max_items, int32_t *sizes)
{
    if (batch < 0 || (batch > 0 && seq_lens == nullptr) || query_group < 1 || sizes == nullptr || max_items < 0 ||
        (max_items > 0 && items == nullptr))
        return RLT_ERR_INVALID_ARG;
    const int64_t step = query_group % 2 == 0 ? 128 : 256;
    int64_t rows = 0, count = 0, longest = 0, tiles = 0;
    for (int32_t b = 0; b < batch; ++b) {
        if (seq_lens[b] < 0)
            return RLT_ERR_INVALID_ARG;
        rows += seq_lens[b];
        count += (seq_lens[b] + step - 1) / step;
        const int64_t all = (seq_lens[b] + 127) / 128;           // key tiles of the items: step/128, 2 step/128, ..
        for (int64_t n = step / 128; n < all + step / 128; n += step / 128)
            tiles += std::min(n, all);
        longest = std::max<int64_t>(longest, seq_lens[b]);
    }
    if (rows > INT32_MAX)
        return RLT_ERR_UNSUPPORTED;
    sizes[0] = (int32_t)count;
    sizes[1] = (int32_t)rows;
    sizes[2] = (int32_t)((longest + 127) / 128);
    sizes[3] = (int32_t)std::min<int64_t>(tiles, INT32_MAX);
    if (count > max_items)
        return RLT_ERR_OUT_OF_RANGE;
    // The items with the most keys first, so that the grid ends on short ones: from the longest
    // sequence's last step down, each step's items in the order of the batch.
    int64_t at = 0;
    try {
        std::vector<std::pair<int32_t, int32_t>> order;         // (length, index), longest first
        std::vector<int32_t> first;
        int32_t row = 0;
        for (int32_t b = 0; b < batch; ++b) {
            order.emplace_back(seq_lens[b], b);
            first.push_back(row);
            row += seq_lens[b];
        }
        std::stable_sort(order.begin(), order.end(), [](const auto &x, const auto &y) { return x.first > y.first; });
        for (int64_t q0 = longest > 0 ? (longest - 1) / step * step : -1; q0 >= 0; q0 -= step)
            for (const auto &o : order) {
                if (o.first <= q0)
                    break;
                int32_t *it = items + at++ * 4;
                it[0] = first[o.second];
                it[1] = o.first;
                it[2] = (int32_t)q0;
                it[3] = 0;
            }
    } catch (...) {
        return RLT_ERR_INVALID_ARG;              // no host memory for the order
    }
    return RLT_OK;
}
