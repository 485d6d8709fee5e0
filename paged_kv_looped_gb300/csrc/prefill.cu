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
// on tcgen05 (fp32 accumulators in tensor memory).  4 * 128 * 128 * head_dim flops a tile and key
// tile take the tensor pipe 1024 clocks at head_dim 128, the softmax of one tile fits beside the
// products of the other, so the tensor pipe bounds long prompts; short ones are bound by the start of
// a CTA (first copies, no overlap) and by their ragged last tiles.
//
// Roles: warps 0-3 / 4-7 softmax of tile 0 / 1 (a thread owns one row = one tensor-memory lane:
// row maxima and sums need no exchange), warp 8 / 9 the MMAs of tile 0 / 1, warp 10 the copies.  P (bf16)
// is written over the S it came from.  The reference maximum of a row moves only when the running
// maximum exceeds it by 2^8, so O is rescaled rarely, by the row's own thread.
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
constexpr float kRescaleThreshold = 8.f;     // log2 units
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;
constexpr int kItemFields = 4;               // first row of the sequence, its length, first query of the item, 0

template <int D>
struct PCfg {
    static constexpr int kStages = D == 128 ? 5 : 8;             // K/V ring slots
    static constexpr int kBlock = kTile * 128;                   // a 64-dim column block of a tile
    static constexpr int kTileBytes = D / 64 * kBlock;
    static constexpr int kRingOff = 2 * kTileBytes;              // behind the two Q tiles
    static constexpr int kBarOff = kRingOff + kStages * kTileBytes;
    enum Bar { kQFull = 0, kFull = 2, kFree = kFull + kStages, kSFull = kFree + kStages, kPFull = kSFull + 2,
               kPvDone = kPFull + 4, kNumBars = kPvDone + 2 };
    static constexpr int kFlagOff = kBarOff + kNumBars * 8;
    static constexpr int kSmem = kFlagOff + 16 + 1024;
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

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const volatile int *abort)
{
    return __all_sync(kFullMask, mbar_wait_or_abort(bar, parity, abort));
}

// 2^x, kept in program order among volatile instructions.
__device__ __forceinline__ float exp2_in_order(float x)
{
    float r;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const PrefillParams p)
{
    using C = PCfg<D>;
    constexpr int kBlocks = D / 64;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *base =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + C::kBarOff);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(base + C::kFlagOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + C::kFlagOff + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();

    const int G = p.num_q_heads / p.num_kv_heads;
    const bool pair = G % 2 == 0;                // tile 1: the next head, else the next 128 tokens
    const int units = pair ? p.num_q_heads / 2 : p.num_q_heads;
    const int item = blockIdx.x / units, unit = blockIdx.x - item * units;
    const int32_t *it = p.items + (int64_t)item * kItemFields;
    const int row0 = it[0], len = it[1], q0 = it[2];
    if (row0 < 0 || len < 1 || len > p.num_rows - row0 || q0 < 0 || q0 >= len || q0 % kTile != 0) {
        if (tid == 0)
            record_error(p.err, RLT_DEVERR_BAD_LEN);   // a plan of other sequences
        return;
    }
    const int head0 = pair ? 2 * unit : unit, kv_head = head0 / G;
    const int head_step = pair ? 1 : 0, tok_step = pair ? 0 : kTile;
    // key tiles of each query tile: up to its last row's own key
    const int n0 = q0 / kTile + 1;
    const int n1 = q0 + tok_step < len ? n0 + tok_step / kTile : 0;
    const int n = max(n0, n1);

    if (tid == 0) {
        for (int i = 0; i < C::kSFull; ++i)
            mbar_init(&bars[i], i < C::kFree ? 1 : 2);   // a slot is free once both tiles' products have read it
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[C::kSFull + i], 1);
            mbar_init(&bars[C::kPFull + 2 * i], 4);
            mbar_init(&bars[C::kPFull + 2 * i + 1], 4);
            mbar_init(&bars[C::kPvDone + i], 1);
        }
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == kMmaWarp)
        tc::tmem_alloc(tslot, kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;
    bool ok = true;

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp == kLoadWarp && tc::elect_one()) {
            // ---------------------------------------------------------- copies
            // Ring order K0, V0, K1, V1, ...; rows behind the last one of the array read as zeros.
            tc::prefetch_tmap(&qmap);
            tc::prefetch_tmap(&kmap);
            tc::prefetch_tmap(&vmap);
            pdl_wait();
            auto load = [&](unsigned char *dst, const CUtensorMap *map, int head, int row, uint64_t *bar) {
                mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
                    tma_load_3d(dst + b * C::kBlock, map, b * 64, head, row, bar);
            };
            int st = 0, issued = 0, queries = 0;
            uint32_t parity = 1;                 // of the slot's previous release (none in the first round)
            for (int i = 0; i < 2 * n; ++i) {
                if (queries < 2 && (queries == 0 || n1 > 0)) {
                    load(base + queries * C::kTileBytes, &qmap, head0 + queries * head_step,
                         row0 + q0 + queries * tok_step, &bars[C::kQFull + queries]);
                    ++queries;
                }
                if (i >= C::kStages && !(ok = mbar_wait_or_abort(&bars[C::kFree + st], parity, abort_flag)))
                    break;
                load(base + C::kRingOff + st * C::kTileBytes, (i & 1) ? &vmap : &kmap, kv_head,
                     row0 + (i >> 1) * kTile, &bars[C::kFull + st]);
                issued = i + 1;
                if (++st == C::kStages) {
                    st = 0;
                    parity ^= 1u;
                }
            }
            if (!ok)
                *abort_flag = 1;
            // every copy has landed before the CTA gives up its memory (bounded; on the normal path
            // the products have waited for all of them)
            for (int i = max(0, issued - C::kStages); i < issued; ++i)
                mbar_wait(&bars[C::kFull + i % C::kStages], (i / C::kStages) & 1u);
            for (int i = 0; i < queries; ++i)
                mbar_wait(&bars[C::kQFull + i], 0);
        } else if (warp < kLoadWarp && tc::elect_one()) {
            // ---------------------------------------------------------- products
            // One thread a tile, in the order S | PV S' | PV' S'' ...: MMAs of one thread run in issue order,
            // so S of the next key tile may overwrite the P that the PV before it reads.  A wait costs a thread
            // about 75 clocks and a full MMA queue holds it up; with a thread a tile neither delays the
            // other tile's products (one thread for both measured 352 us where two take 322: 8192
            // tokens, 32 heads).  An MMA keeps the tensor pipe 64 clocks, so its issue has to take
            // less: the descriptors are the tile's plus constants.
            const int s = warp - kMmaWarp;
            const int ns = s == 0 ? n0 : n1;
            constexpr uint32_t id_s = tc::instr_desc_bf16(128, 128, false);
            constexpr uint32_t id_o = tc::instr_desc_bf16(128, D, true);
            constexpr uint64_t kTileStep = C::kTileBytes >> 4;
            const uint64_t qd = tc::smem_desc(smem_u32(base), 16, 1024) + s * kTileStep;
            const uint64_t kd = tc::smem_desc(smem_u32(base + C::kRingOff), 16, 1024);
            const uint64_t vd = tc::smem_desc(smem_u32(base + C::kRingOff), C::kBlock, 1024);
            const uint32_t t_s = tmem + kColS + s * kTile, t_o = tmem + kColO + s * kTile;
            auto issue_s = [&](int slot) {
                const uint64_t b = kd + slot * kTileStep;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    constexpr uint64_t kStep = C::kBlock >> 4;
                    tc::mma_bf16(t_s, qd + (kk >> 2) * kStep + (kk & 3) * 2, b + (kk >> 2) * kStep + (kk & 3) * 2, id_s,
                                 kk > 0);
                }
                tc::mma_commit(&bars[C::kSFull + s]);
            };
            auto issue_pv = [&](int half, int slot, bool first) {             // 64 keys
                const uint64_t b = vd + slot * kTileStep + half * (4 * 2048 >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc::mma_bf16_ta(t_o, t_s + half * 32 + kk * 8, b + kk * (2048 >> 4), id_o, kk > 0 || !first);
            };
            // ring slot and parity of the next copy to be waited for
            int st = 0;
            uint32_t parity = 0;
            auto wait_slot = [&](int &slot) -> bool {
                slot = st;
                if (!mbar_wait_or_abort(&bars[C::kFull + st], parity, abort_flag))
                    return false;
                if (++st == C::kStages) {
                    st = 0;
                    parity ^= 1u;
                }
                return true;
            };
            // a tile without work on a copy lets it go at once
            auto release = [&](int slot, bool used) {
                if (used)
                    tc::mma_commit(&bars[C::kFree + slot]);
                else
                    mbar_arrive(&bars[C::kFree + slot]);
            };
            int k_slot = 0, v_slot = 0, s_issued = 0, pv_issued = 0;
            ok = wait_slot(k_slot) && (ns == 0 || mbar_wait_or_abort(&bars[C::kQFull + s], 0, abort_flag));
            if (ok) {
                if (ns > 0) {
                    issue_s(k_slot);
                    s_issued = 1;
                }
                release(k_slot, ns > 0);
            }
            for (int j = 0; ok && j < n; ++j) {
                if (!(ok = wait_slot(v_slot)) || (j + 1 < n && !(ok = wait_slot(k_slot))))
                    break;
                if (j < ns) {
                    if (!(ok = mbar_wait_or_abort(&bars[C::kPFull + 2 * s], j & 1u, abort_flag)))
                        break;
                    tc::fence_after_sync();
                    issue_pv(0, v_slot, j == 0);
                    pv_issued = j + 1;
                    ok = mbar_wait_or_abort(&bars[C::kPFull + 2 * s + 1], j & 1u, abort_flag);
                    tc::fence_after_sync();
                    if (ok)
                        issue_pv(1, v_slot, false);
                    tc::mma_commit(&bars[C::kPvDone + s]);
                    if (!ok)
                        break;
                    if (j + 1 < ns) {
                        issue_s(k_slot);
                        s_issued = j + 2;
                    }
                }
                release(v_slot, j < ns);
                if (j + 1 < n)
                    release(k_slot, j + 1 < ns);
            }
            if (!ok)
                *abort_flag = 1;
            // every issued MMA is complete before the CTA gives up its memory (bounded)
            if (pv_issued > 0)
                mbar_wait(&bars[C::kPvDone + s], (pv_issued - 1) & 1u);
            if (s_issued > pv_issued)
                mbar_wait(&bars[C::kSFull + s], (s_issued - 1) & 1u);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---------------------------------------------------------- softmax
        const int s = warp >> 2, quarter = warp & 3;
        const int ns = s == 0 ? n0 : n1;
        const int q_tok = q0 + s * tok_step + quarter * 32 + lane;       // this thread's query, in its sequence
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t t_s = t_lane + kColS + s * kTile, t_o = t_lane + kColO + s * kTile;
        float m_ref = -CUDART_INF_F, l_run = 0.f;
        auto p_ready = [&](int half) {           // this warp's P of 64 keys is in tensor memory
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bars[C::kPFull + 2 * s + half]);
        };
        for (int j = 0; j < ns; ++j) {
            if (!(ok = warp_wait(&bars[C::kSFull + s], j & 1u, abort_flag)))
                break;
            tc::fence_after_sync();
            if (j == ns - 1 && (j + 1) * kTile > len && quarter == 0) {
                // ragged end of the sequence: the V rows past it may hold anything (0 * NaN would
                // poison O): zeros, once the copy has landed
                const int i = 2 * j + 1;
                if (!(ok = warp_wait(&bars[C::kFull + i % C::kStages], (i / C::kStages) & 1u, abort_flag)))
                    break;
                unsigned char *vt = base + C::kRingOff + i % C::kStages * C::kTileBytes;
                const int valid = len - j * kTile;
                for (int c = lane; c < (kTile - valid) * kBlocks * 8; c += 32) {
                    const int r = valid + c / (kBlocks * 8), c16 = c % (kBlocks * 8);
                    *reinterpret_cast<uint4 *>(vt + (c16 >> 3) * C::kBlock + r * 128 + (c16 & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
            }
            float v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                tc::tmem_ld32_nowait(t_s + c * 32, v[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                tc::tmem_wait_ld(v[c]);
            if (j == ns - 1) {                   // the diagonal: keys behind the query
                const int last = q_tok - j * kTile;
#pragma unroll
                for (int i = 0; i < kTile; ++i)
                    v[i / 32][i % 32] = i <= last ? v[i / 32][i % 32] : -CUDART_INF_F;
            }
            // P = 2^(s - m), 32 columns at a time.  The first ones are made against the reference the row has,
            // beside the row's maximum: it moves rarely, and then they are made again.  The exponentials
            // of the next columns are issued ahead of the conversions of the last ones: the unit
            // that makes them (8 lanes a clock) is what a warp waits for.
            auto raise = [&](const float (&x)[32], float (&y)[32], float m) {
                const float m_sub = m == -CUDART_INF_F ? 0.f : m;
                const uint64_t sc2 = f2_pack(p.qscale, p.qscale), off2 = f2_pack(-m_sub, -m_sub);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 z = f2_unpack(f2_fma(f2_pack(x[2 * i], x[2 * i + 1]), sc2, off2));
                    y[2 * i] = exp2_in_order(z.x);
                    y[2 * i + 1] = exp2_in_order(z.y);
                }
            };
            uint64_t sum2[2] = {0ull, 0ull};
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
            float y0[32];
            raise(v[0], y0, m_ref);
            float mx4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int i = 0; i < 32; i += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx4[k] = fmaxf(fmaxf(mx4[k], v[c][i + k]), v[c][i + 4 + k]);
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.qscale;
            const bool up = mx > m_ref + kRescaleThreshold;
            if (__any_sync(kFullMask, up)) {
                const float m_next = up ? mx : m_ref;
                const float scale_o = m_next == m_ref ? 1.f : fast_exp2(m_ref - m_next);
                if (j > 0) {
                    if (!(ok = warp_wait(&bars[C::kPvDone + s], (j - 1) & 1u, abort_flag)))
                        break;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        float o[16];
                        uint32_t ow[16];
                        tc::tmem_ld<16>(t_o + c * 16, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            ow[i] = __float_as_uint(o[i] * scale_o);
                        tc::tmem_st_nowait<16>(t_o + c * 16, ow);
                    }
                }
                l_run *= scale_o;
                m_ref = m_next;
                raise(v[0], y0, m_ref);
            }
            raise(v[1], v[1], m_ref);
            store(y0, 0);
            raise(v[2], v[2], m_ref);
            store(v[1], 1);
            p_ready(0);                          // the first 64 keys' weights
            raise(v[3], v[3], m_ref);
            store(v[2], 2);
            store(v[3], 3);
            p_ready(1);
            const float2 sum = f2_unpack(f2_add(sum2[0], sum2[1]));
            l_run += sum.x + sum.y;
        }
        if (ok && ns > 0 && (ok = warp_wait(&bars[C::kPvDone + s], (ns - 1) & 1u, abort_flag))) {
            tc::fence_after_sync();
            const float inv = 1.f / l_run;
            const int64_t at = (int64_t)(row0 + q_tok) * p.num_q_heads + head0 + s * head_step;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                tc::tmem_ld<32>(t_o + c * 32, o);
                if (q_tok < len) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + at * D + c * 32);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dst[i] = make_uint4(cvt_bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv),
                                            cvt_bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                            cvt_bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                            cvt_bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
                }
            }
            if (q_tok < len && p.lse_out != nullptr)
                p.lse_out[at] = (m_ref + log2f(l_run)) * 0.6931471805599453f;
        }
        if (!ok)
            *abort_flag = 1;
    }

    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (tid == 0 && *abort_flag != 0)
        record_error(p.err, RLT_DEVERR_TIMEOUT);
    if (warp == kMmaWarp)
        tc::tmem_dealloc(tmem, kTmemCols);
}

// Token rows of `heads` x D bf16, `stride` elements apart; boxes of 128 tokens x 64 dims of one head.
bool make_rows_map(CUtensorMap *map, const uint16_t *ptr, int64_t rows, int heads, int D, int64_t stride)
{
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, kTile};
    const cuuint32_t estr[3] = {1, 1, 1};
    const tc::EncodeTiledFn fn = tc::encode_tiled_fn();
    return fn != nullptr && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(ptr), dims, strides, box,
                               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_prefill_typed(const PrefillParams &p, cudaStream_t stream, bool early)
{
    using C = PCfg<D>;
    static_assert(C::kSmem <= 227 * 1024, "shared memory of one CTA");
    CUtensorMap qmap, kmap, vmap;
    if (!make_rows_map(&qmap, p.q, p.num_rows, p.num_q_heads, D, p.q_stride) ||
        !make_rows_map(&kmap, p.k, p.num_rows, p.num_kv_heads, D, p.k_stride) ||
        !make_rows_map(&vmap, p.v, p.num_rows, p.num_kv_heads, D, p.v_stride))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit == 0 || (configured.load(std::memory_order_acquire) & bit) == 0) {
        e = cudaFuncSetAttribute(prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess)
            return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    const int G = p.num_q_heads / p.num_kv_heads;
    const unsigned units = G % 2 == 0 ? p.num_q_heads / 2 : p.num_q_heads;
    return launch_kernel(prefill_kernel<D>, dim3(p.num_items * units), dim3(kThreads), C::kSmem, stream, early, qmap,
                         kmap, vmap, p);
}

}  // namespace

cudaError_t launch_prefill(const PrefillParams &p, int head_dim, cudaStream_t stream, bool early)
{
    return head_dim == 128 ? launch_prefill_typed<128>(p, stream, early) : launch_prefill_typed<64>(p, stream, early);
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
    int64_t rows = 0, count = 0, longest = 0;
    for (int32_t b = 0; b < batch; ++b) {
        if (seq_lens[b] < 0)
            return RLT_ERR_INVALID_ARG;
        rows += seq_lens[b];
        count += (seq_lens[b] + step - 1) / step;
        longest = std::max<int64_t>(longest, seq_lens[b]);
    }
    if (rows > INT32_MAX)
        return RLT_ERR_UNSUPPORTED;
    sizes[0] = (int32_t)count;
    sizes[1] = (int32_t)rows;
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
