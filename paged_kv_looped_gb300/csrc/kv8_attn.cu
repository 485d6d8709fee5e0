// Paged decode attention over the 8-bit cache for sm_103a: split-K partials and their join.
//
// "Faster fuzzy minds", "When scheduler does the work" and "Recurrent depth": one new token per
// request attends over its cached tokens, read page by page from one (layer, plane) bank.  The
// cache holds value = e4m3 * 2^e with one e per (token, kv head) (rlt_fp8.cuh), so with x8 the
// held e4m3 numbers and everything in log2 units
//     s_j = qscale <q, k8_j> 2^(ke_j),     out = sum_j 2^(s_j) 2^(ve_j) v8_j / sum_j 2^(s_j).
// The value's scale rides in the exponent: w_j = s_j + ve_j, and P_j = 2^(w_j - m + 14) against a
// running maximum m of w multiplies v8_j.  A row of zero values carries the scale 2^0 whatever its neighbours'
// scales are; it would raise m and cost the others' weights their bits, so it counts with 2^-100.
//
// What bounds it: the cache's bytes, 2 (D + 1) per token and kv head; 4 G flop for each pair of
// them.  At 6.7 TB/s an SM takes in about 21 bytes a clock, and a CUDA-core kernel would have to
// convert and multiply each with G queries; so the products run on the warp-level tensor
// instruction (m16n8k16, fp16 operands, fp32 sums), whose 8 columns hold the G <= 8 query heads
// of a kv head: the instructions per byte do not depend on G.  (tcgen05 wants 64 or 128 query rows,
// and 8-bit operands on both sides.)
//   S^T = K q^T   A = 16 tokens x 16 dims, e4m3 -> fp16 in registers (exact); B = the queries,
//                 fp16 after a power-of-two scale per head that brings the head's largest
//                 magnitude into [2^14, 2^15) (a bf16 query keeps its bits there down to 2^-38 of it)
//   O^T = V^T P^T A = 16 dims x 16 tokens, pairs of tokens interleaved byte by byte; B = P^T,
//                 S^T's accumulator transposed by movmatrix.  P is rounded to fp16 (2^-11
//                 relative down to 2^-28 of the largest weight, thanks to the 2^14 above)
// Which of a lane's k, tokens and dims an instruction's slots name is free as long as both operands
// agree, so every shared-memory read is 16 contiguous bytes of a row (8 for V at head_dim 64);
// tiles land swizzled by the tensor copy (16-byte chunks XORed by row), and the token order below
// makes the reads of both K and V free of bank conflicts at head_dim 128.
//
// Measured: 64 requests x 16 kv heads x 512-4096 tokens (599 MB) 98.6 us, 256 log-normal requests x 8 (1.84 GB)
// 279.5 us, 8 x 32k-131k tokens x 8 (1.16 GB) 180.3 us with the join: 91, 98 and 96 % of a copy's 6.7 TB/s; what is
// left of the first is the grid's start and its last CTAs (7 us).  At head_dim 64 a tile is 2 KB for the same
// copies and instructions: 302 MB in 67.5 us (4.5 TB/s), 928 MB in 181 (5.1).
// Three CTAs an SM with two stages of two tiles a warp; in an earlier form, whose calls in a row started only at the
// end of the kernel ahead, they took 100 / 275 / 178 us, 118 / 318 / 198 with two CTAs of three such stages,
// 110 / 301 / 190 with four stages of one tile, 101 / 277 / 181 with four CTAs of three stages of one tile.
// The zero rows' look costs 0.3 to 0.6 %; at every tile, not only where the maximum rises, it took 1 to 1.7 %.
#include <cuda.h>
#include <math_constants.h>

#include <atomic>

#include "rlt_device.cuh"
#include "rlt_fp8.cuh"
#include "rlt_internal.h"
#include "rlt_merge.cuh"
#include "rlt_tc.cuh"

namespace rlt {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;                   // copy ring depth per warp
constexpr int kStageTiles = 2;               // 16-token tiles per stage
constexpr int kStageTokens = kStageTiles * kTileTokens;
constexpr float kPOffset = 14.f;             // P's largest value is 2^14
constexpr float kZeroRowExp = -100.f;        // of a row of zero values: l stays below 2^(100 + 21) of 2^m
constexpr int kMaxGroup = 8;
constexpr int kNarrowSplits = 16;            // up to this many splits (two rounds of loads) a warp joins a row alone

template <int D>
struct Cfg8 {
    static constexpr int kTileBytes = kTileTokens * D;           // K (or V) of a tile
    static constexpr int kSideBytes = kStageTokens * D;
    static constexpr int kStageBytes = 2 * kSideBytes;
    static constexpr int kPipeBytes = kWarps * kStages * kStageBytes;
    static constexpr int kMergeStride = D + 4;
    static constexpr int kMergeBytes = kWarps * kMaxGroup * kMergeStride * 4;
    static constexpr int kExpOffset = kPipeBytes > kMergeBytes ? kPipeBytes : kMergeBytes;
    static constexpr int kExpBytes = kWarps * kStages * 2 * kStageTokens;   // K and V exponents
    static constexpr int kBarOffset = kExpOffset + kExpBytes;
    static constexpr int kSmemBytes = kBarOffset + kWarps * kStages * 8 + 1024;   // + alignment
};

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), fp16 operands.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The token of a tile that accumulator row r of an 8-row half stands for.  At head_dim 128 rows 2j
// and 2j + 1 differ in bit 2, so that the 8 lanes of one shared-memory phase (two rows, four
// chunks each) meet all 8 chunk places under the swizzle, and the even (and the odd) rows
// differ in bits 1 and 2, which does the same for V's phases (four rows, two chunks each).
template <int D>
__device__ __forceinline__ int token_of(int r)
{
    if constexpr (D == 128)
        return (((r ^ (r >> 2)) & 1) << 2) | (r & 2) | (r >> 2);
    else
        return r;
}

// Byte offset of 16-byte chunk c of row r of a tile (tensor-copy swizzle of the row's width).
template <int D>
__device__ __forceinline__ int chunk_offset(int r, int c)
{
    if constexpr (D == 128)
        return r * 128 + ((c ^ (r & 7)) << 4);
    else
        return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// kFault: the timeout test's instance (rlt_debug_fault_next_decode): one copy left unissued, the limit from the call.
template <int D, bool kFault>
__global__ void __launch_bounds__(kThreads, 3)
    kv8_partial_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const DecodeParams p, const uint8_t *__restrict__ k_exp, const uint8_t *__restrict__ v_exp, int early)
{
    using C = Cfg8<D>;
    constexpr int kHalves = D / 64;              // 64-dim halves of a K row
    constexpr int kDimTiles = D / 16;            // 16-dim tiles of O^T
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    // The grid starts while the kernel ahead ends.  Without the early start nothing is read before it has, and
    // the kernel behind starts no earlier either.
    if (early == 0)
        pdl_wait();
    pdl_launch_dependents();
    const int split = blockIdx.x, head = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;       // accumulator row and column pair of this lane
    const int G = p.num_q_heads / p.num_kv_heads;

    const Span sp = request_span(p, b, split == 0 && head == 0 && threadIdx.x == 0);
    const int L = sp.L;
    const int n_tiles = (L + kTileTokens - 1) / kTileTokens;
    const int n_splits = split_count(p, sp);
    if (split >= n_splits) {
        if (split == 0) {                        // empty request: out = 0, lse = -inf
            pdl_wait();
            const int64_t bh = (int64_t)b * p.num_q_heads + head * G;
            for (int d = threadIdx.x; d < G * D / 2; d += kThreads)
                reinterpret_cast<uint32_t *>(p.out + bh * D)[d] = 0u;
            if (p.lse_out != nullptr && threadIdx.x < G)
                p.lse_out[bh + threadIdx.x] = -CUDART_INF_F;
        }
        return;
    }

    const int tile_begin = split * p.tiles_per_split;
    const int tile_end = min(tile_begin + p.tiles_per_split, n_tiles);
    const int groups = (tile_end - tile_begin + kStageTiles - 1) / kStageTiles;
    const int my_count = warp < groups ? (groups - warp + kWarps - 1) / kWarps : 0;

    unsigned char *pipe = smem + warp * kStages * C::kStageBytes;
    uint8_t *exps = smem + C::kExpOffset + warp * kStages * 2 * kStageTokens;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOffset) + warp * kStages;
    if (lane == 0) {
        for (int s = 0; s < kStages; ++s)
            mbar_init(&bars[s], 1);
        mbar_init_fence();
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
    }
    __syncwarp();

    // Lane j holds the pool row (slot row of this kv head) of this warp's j-th tile, -1 where
    // there is none: a page outside the pool is skipped and recorded.
    int my_row = -1;
    {
        const int tile = tile_begin + kStageTiles * (warp + kWarps * (lane / kStageTiles)) + lane % kStageTiles;
        if (lane < kStageTiles * my_count && tile < tile_end) {
            const int tok = tile * kTileTokens;
            const int page = p.page_table[(int64_t)b * p.max_pages + tok / p.page_size];
            if (page >= 0 && (int64_t)page < p.num_pages)
                my_row = (int)(((int64_t)page * p.num_kv_heads + head) * p.page_size + tok % p.page_size);
            else
                record_error(p.err, RLT_DEVERR_BAD_PAGE);
        }
    }
    const unsigned have = __ballot_sync(kFullMask, my_row >= 0);

    // Stage i: this lane's tile of it, if any, as four copies.
    auto issue = [&](int i) {
        uint64_t *bar = &bars[i % kStages];
        const unsigned mine = (have >> (kStageTiles * i)) & ((1u << kStageTiles) - 1u);
        if (lane == 0)
            mbar_arrive_expect_tx(bar, __popc(mine) * 2 * (C::kTileBytes + kTileTokens));
        __syncwarp();
        if (lane / kStageTiles == i && my_row >= 0) {
            unsigned char *dst = pipe + (i % kStages) * C::kStageBytes + (lane % kStageTiles) * C::kTileBytes;
            uint8_t *de = exps + (i % kStages) * 2 * kStageTokens + (lane % kStageTiles) * kTileTokens;
            if (!(kFault && i == 0 && lane == 0 && warp == 0 && split == 0 && head == 0 && b == 0))
                tc::tma_load_2d_once(dst, &kmap, 0, my_row, bar);
            tc::tma_load_2d_once(dst + C::kSideBytes, &vmap, 0, my_row, bar);
            bulk_load_once(de, k_exp + my_row, kTileTokens, bar);
            bulk_load_once(de + kStageTokens, v_exp + my_row, kTileTokens, bar);
        }
    };
    int issued = 0;
    for (; issued < min(my_count, kStages); ++issued)
        issue(issued);
    pdl_wait();

    // The queries as B operands: column g is query head g; slot pairs (2t, 2t + 1) and (2t + 8,
    // 2t + 9) of instruction (hh, kk) are dims 64 hh + 16 t + 4 kk + 0..3, the four bytes
    // that word kk of this lane's K chunk holds.
    uint32_t qb[kHalves * 4][2];
    float sc0, sc1;                              // score scales of heads 2t and 2t + 1
    {
        uint2 raw[kHalves * 4];
        uint32_t amax = 0u;
        const uint16_t *src = p.q + ((int64_t)b * p.num_q_heads + head * G + min(g, G - 1)) * D + 16 * t;
#pragma unroll
        for (int i = 0; i < kHalves * 4; ++i) {
            raw[i] = *reinterpret_cast<const uint2 *>(src + 64 * (i / 4) + 4 * (i % 4));
            amax = max(max(amax, max(raw[i].x & 0x7fffu, (raw[i].x >> 16) & 0x7fffu)),
                       max(raw[i].y & 0x7fffu, (raw[i].y >> 16) & 0x7fffu));
        }
        amax = max(amax, __shfl_xor_sync(kFullMask, amax, 1));
        amax = max(amax, __shfl_xor_sync(kFullMask, amax, 2));
        const int eq = max((int)(amax >> 7) - 127 - 14, -100);
        const float down = __uint_as_float((uint32_t)(127 - eq) << 23);
#pragma unroll
        for (int i = 0; i < kHalves * 4; ++i) {
            qb[i][0] = f16x2(bf16_lo(raw[i].x) * down, bf16_hi(raw[i].x) * down);
            qb[i][1] = f16x2(bf16_lo(raw[i].y) * down, bf16_hi(raw[i].y) * down);
        }
        const float own = p.qscale * __uint_as_float((uint32_t)(127 + eq) << 23);
        sc0 = __shfl_sync(kFullMask, own, 8 * t);
        sc1 = __shfl_sync(kFullMask, own, 8 * t + 4);
    }

    float acc[kDimTiles][4];
#pragma unroll
    for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            acc[i][c] = 0.f;
    float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;   // heads 2t, 2t + 1; l: this lane's tokens

    const int tok_g = token_of<D>(g);            // this lane's tokens of a tile's scores: tok_g, tok_g + 8
    const int tok_a = token_of<D>(2 * t), tok_b = token_of<D>(2 * t + 1);   // and of its values (and + 8)
    const uint64_t limit = kFault ? p.wait_limit_ns : kWaitLimitNs;
    uint32_t phase = 0;
    bool failed = false;
    int i = 0;
    for (; i < my_count; ++i) {
        const int s = i % kStages;
        if (!__all_sync(kFullMask, mbar_wait(&bars[s], (phase >> s) & 1u, limit))) {
            failed = true;
            break;
        }
        phase ^= 1u << s;
        const unsigned char *ks = pipe + s * C::kStageBytes;
        const unsigned char *vs = ks + C::kSideBytes;
        const uint8_t *es = exps + s * 2 * kStageTokens;
        const int tok0 = (tile_begin + kStageTiles * (warp + kWarps * i)) * kTileTokens;

        int valid[kStageTiles];                  // tokens of each tile (warp-uniform)
        float sv[kStageTiles][4], wv[kStageTiles][4];
        float x0 = -CUDART_INF_F, x1 = -CUDART_INF_F;
        bool one = false;                        // a value scale of 2^0 among this lane's tokens
#pragma unroll
        for (int u = 0; u < kStageTiles; ++u) {
            valid[u] = ((have >> (kStageTiles * i + u)) & 1u) ? min(kTileTokens, L - tok0 - u * kTileTokens) : 0;
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            if (valid[u] > 0) {
                const unsigned char *kt = ks + u * C::kTileBytes;
#pragma unroll
                for (int hh = 0; hh < kHalves; ++hh) {
                    const uint4 lo = *reinterpret_cast<const uint4 *>(kt + chunk_offset<D>(tok_g, t + 4 * hh));
                    const uint4 hi = *reinterpret_cast<const uint4 *>(kt + chunk_offset<D>(tok_g + 8, t + 4 * hh));
                    const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f16(c, f16x2_of_e4m3(lw[kk]), f16x2_of_e4m3(hw[kk]), f16x2_of_e4m3(lw[kk] >> 16),
                                f16x2_of_e4m3(hw[kk] >> 16), qb[hh * 4 + kk][0], qb[hh * 4 + kk][1]);
                }
            }
            const float ka = exp_scale(es[u * kTileTokens + tok_g]), kb = exp_scale(es[u * kTileTokens + tok_g + 8]);
            const float va = (float)((int)es[kStageTokens + u * kTileTokens + tok_g] - kExpBias);
            const float vb = (float)((int)es[kStageTokens + u * kTileTokens + tok_g + 8] - kExpBias);
            const bool in_a = tok_g < valid[u], in_b = tok_g + 8 < valid[u];
            one |= va == 0.f || vb == 0.f;
            sv[u][0] = in_a ? c[0] * sc0 * ka : -CUDART_INF_F;
            sv[u][1] = in_a ? c[1] * sc1 * ka : -CUDART_INF_F;
            sv[u][2] = in_b ? c[2] * sc0 * kb : -CUDART_INF_F;
            sv[u][3] = in_b ? c[3] * sc1 * kb : -CUDART_INF_F;
            wv[u][0] = sv[u][0] + va;
            wv[u][1] = sv[u][1] + va;
            wv[u][2] = sv[u][2] + vb;
            wv[u][3] = sv[u][3] + vb;
            x0 = fmaxf(x0, fmaxf(wv[u][0], wv[u][2]));
            x1 = fmaxf(x1, fmaxf(wv[u][1], wv[u][3]));
        }
        x0 = fmaxf(m0, warp_max_xor(x0, 4));
        x1 = fmaxf(m1, warp_max_xor(x1, 4));
        if (__any_sync(kFullMask, x0 != m0 || x1 != m1)) {
            // The maximum rises, but not for a row of zeros.  (Where it does not rise they do no harm.)
            if (__any_sync(kFullMask, one)) {
                x0 = x1 = -CUDART_INF_F;
#pragma unroll
                for (int u = 0; u < kStageTiles; ++u) {
                    // Scale 2^0: zeros, or (rarely) values of 128 to 256.  The four lanes of a token look at a quarter
                    // of its row each; negative zeros count too.
                    const uint8_t *ve = es + kStageTokens + u * kTileTokens;
                    uint32_t ra = 0u, rb = 0u;
#pragma unroll
                    for (int hh = 0; hh < kHalves; ++hh) {
                        const unsigned char *vt = vs + u * C::kTileBytes;
                        const uint4 x = *reinterpret_cast<const uint4 *>(vt + chunk_offset<D>(tok_g, t + 4 * hh));
                        const uint4 y = *reinterpret_cast<const uint4 *>(vt + chunk_offset<D>(tok_g + 8, t + 4 * hh));
                        ra |= x.x | x.y | x.z | x.w;
                        rb |= y.x | y.y | y.z | y.w;
                    }
                    ra |= __shfl_xor_sync(kFullMask, ra, 1);
                    ra |= __shfl_xor_sync(kFullMask, ra, 2);
                    rb |= __shfl_xor_sync(kFullMask, rb, 1);
                    rb |= __shfl_xor_sync(kFullMask, rb, 2);
                    if (ve[tok_g] == kExpBias && (ra & 0x7f7f7f7fu) == 0u) {
                        wv[u][0] = sv[u][0] + kZeroRowExp;
                        wv[u][1] = sv[u][1] + kZeroRowExp;
                    }
                    if (ve[tok_g + 8] == kExpBias && (rb & 0x7f7f7f7fu) == 0u) {
                        wv[u][2] = sv[u][2] + kZeroRowExp;
                        wv[u][3] = sv[u][3] + kZeroRowExp;
                    }
                    x0 = fmaxf(x0, fmaxf(wv[u][0], wv[u][2]));
                    x1 = fmaxf(x1, fmaxf(wv[u][1], wv[u][3]));
                }
                x0 = fmaxf(m0, warp_max_xor(x0, 4));
                x1 = fmaxf(m1, warp_max_xor(x1, 4));
            }
            // 2^(m - x) in two halves: it may be below fp32's smallest where l (up to 2^121) times it is not
            const float h0 = x0 == m0 ? 1.f : fast_exp2(0.5f * (m0 - x0)), h1 = x1 == m1 ? 1.f : fast_exp2(0.5f * (m1 - x1));
            const float a0 = h0 * h0, a1 = h1 * h1;
            l0 = l0 * h0 * h0;
            l1 = l1 * h1 * h1;
#pragma unroll
            for (int d = 0; d < kDimTiles; ++d) {
                acc[d][0] *= a0;
                acc[d][1] *= a1;
                acc[d][2] *= a0;
                acc[d][3] *= a1;
            }
            m0 = x0;
            m1 = x1;
        }
        const float r0 = m0 == -CUDART_INF_F ? 0.f : m0, r1 = m1 == -CUDART_INF_F ? 0.f : m1;
#pragma unroll
        for (int u = 0; u < kStageTiles; ++u) {
            if (valid[u] <= 0)
                continue;
            l0 += fast_exp2(sv[u][0] - r0) + fast_exp2(sv[u][2] - r0);
            l1 += fast_exp2(sv[u][1] - r1) + fast_exp2(sv[u][3] - r1);
            const uint32_t pa = f16x2(fast_exp2(wv[u][0] - r0 + kPOffset), fast_exp2(wv[u][1] - r1 + kPOffset));
            const uint32_t pb = f16x2(fast_exp2(wv[u][2] - r0 + kPOffset), fast_exp2(wv[u][3] - r1 + kPOffset));
            const uint32_t b0 = transpose_8x8(pa), b1 = transpose_8x8(pb);
            const unsigned char *vt = vs + u * C::kTileBytes;
            constexpr int kWords = D / 32;       // words of a token's row that this lane takes
            uint32_t va[kWords], vb[kWords], vc[kWords], vd[kWords];
            auto take = [&](uint32_t (&w)[kWords], int tok) {
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(vt + chunk_offset<D>(tok, g));
                    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(vt + chunk_offset<D>(tok, g >> 1) + (g & 1) * 8);
                    w[0] = x.x; w[1] = x.y;
                }
                // rows behind the request's end hold anything, NaN among it: 0 * NaN would stay
                if (valid[u] < kTileTokens && tok >= valid[u]) {
#pragma unroll
                    for (int k = 0; k < kWords; ++k)
                        w[k] = 0u;
                }
            };
            take(va, tok_a);
            take(vb, tok_b);
            take(vc, tok_a + 8);
            take(vd, tok_b + 8);
#pragma unroll
            for (int d = 0; d < kDimTiles; ++d) {
                // bytes 2(d & 1) and + 1 of word d / 2: dims (D / 8) g + 2 d and + 1, tokens side by side
                const uint32_t sel = (d & 1) ? 0x7362u : 0x5140u;
                const uint32_t ab = __byte_perm(va[d / 2], vb[d / 2], sel), cd = __byte_perm(vc[d / 2], vd[d / 2], sel);
                mma_f16(acc[d], f16x2_of_e4m3(ab), f16x2_of_e4m3(ab >> 16), f16x2_of_e4m3(cd), f16x2_of_e4m3(cd >> 16),
                        b0, b1);
            }
        }
        __syncwarp();
        fence_proxy_async();                     // our reads of stage s before its next refill
        if (issued < my_count) {
            issue(issued);
            ++issued;
        }
    }
    if (failed) {
        // A copy never arrived: record it, then wait (bounded) for the copies still in flight
        // before the shared memory is given up; this warp's tokens are left out.
        if (lane == 0)
            record_error(p.err, RLT_DEVERR_TIMEOUT);
        for (int k = i; k < issued; ++k) {
            mbar_wait(&bars[k % kStages], (phase >> (k % kStages)) & 1u, limit);
            phase ^= 1u << (k % kStages);
        }
        m0 = m1 = -CUDART_INF_F;
        l0 = l1 = 0.f;
#pragma unroll
        for (int d = 0; d < kDimTiles; ++d)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[d][c] = 0.f;
    }
    l0 = warp_sum_xor(l0, 4);
    l1 = warp_sum_xor(l1, 4);

    // Merge the 4 warps through shared memory (aliases the copy rings).
    __syncthreads();
    float *mg = reinterpret_cast<float *>(smem);
    float *h0 = mg + (warp * kMaxGroup + 2 * t) * C::kMergeStride, *h1 = h0 + C::kMergeStride;
#pragma unroll
    for (int d = 0; d < kDimTiles; ++d) {
        *reinterpret_cast<float2 *>(h0 + (D / 8) * g + 2 * d) = make_float2(acc[d][0], acc[d][2]);
        *reinterpret_cast<float2 *>(h1 + (D / 8) * g + 2 * d) = make_float2(acc[d][1], acc[d][3]);
    }
    if (g == 0) {
        h0[D] = m0;
        h0[D + 1] = l0;
        h1[D] = m1;
        h1[D + 1] = l1;
    }
    __syncthreads();
    for (int item = threadIdx.x; item < G * D / 4; item += kThreads) {
        const int h = item / (D / 4);
        const int d0 = (item % (D / 4)) * 4;
        float M = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            M = fmaxf(M, mg[(w * kMaxGroup + h) * C::kMergeStride + D]);
        float ls = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
        M = M == -CUDART_INF_F ? 0.f : M;        // no token, or NaN scores only: they stay NaN
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float *row = mg + (w * kMaxGroup + h) * C::kMergeStride;
            const float half = exp2f(0.5f * (row[D] - M)), sc = half * half;   // (as the running rescale)
            ls = fmaf(row[D + 1] * half, half, ls);
            o0 = fmaf(row[d0 + 0], sc, o0);
            o1 = fmaf(row[d0 + 1], sc, o1);
            o2 = fmaf(row[d0 + 2], sc, o2);
            o3 = fmaf(row[d0 + 3], sc, o3);
        }
        const float inv = ls == 0.f ? 0.f : 0x1p-14f / ls;   // (kPOffset)
        const float lse2 = ls == 0.f ? -CUDART_INF_F : M + log2f(ls);
        const int64_t bh = (int64_t)b * p.num_q_heads + head * G + h;
        if (n_splits == 1) {
            *reinterpret_cast<uint2 *>(p.out + bh * D + d0) =
                make_uint2(cvt_bf16x2(o0 * inv, o1 * inv), cvt_bf16x2(o2 * inv, o3 * inv));
            if (d0 == 0 && p.lse_out != nullptr)
                p.lse_out[bh] = lse2 * kLn2;
        } else {
            const int64_t slot = bh * p.part_stride + split;
            *reinterpret_cast<float4 *>(p.o_part + slot * D + d0) =
                make_float4(o0 * inv, o1 * inv, o2 * inv, o3 * inv);
            if (d0 == 0)
                p.lse_part[slot] = lse2;
        }
    }
}

// Joins a row's split partials (rlt_merge.cuh's identity): every split below the request's count has
// written its slot.  kWide: the four warps of a CTA share one row's slots, else each has a row of
// its own.  NaN partials make NaN outputs.  Latency-bound: every partial is read once, from L2.
template <int D, bool kWide>
__global__ void __launch_bounds__(kThreads) kv8_combine_kernel(const DecodeParams p)
{
    constexpr int DPL = D / 32, kLoads = 8;
    __shared__ float part[kWarps][D + 1];
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t bh = kWide ? blockIdx.x : (int64_t)blockIdx.x * kWarps + warp;
    const bool live = bh < (int64_t)p.batch * p.num_q_heads;
    const int n = live ? split_count(p, request_span(p, (int)(bh / p.num_q_heads), false)) : 0;
    pdl_wait();                                  // the partial kernel of this call is done
    if (n <= 1)
        return;                                  // written by the partial kernel (uniform over a wide CTA)
    const float *lse = p.lse_part + bh * p.part_stride;
    const float *o = p.o_part + bh * p.part_stride * D + lane * DPL;
    float M = -CUDART_INF_F;
    for (int s = lane; s < n; s += 32)
        M = fmaxf(M, __ldcg(lse + s));
    M = warp_max_xor(M, 1);
    M = M == -CUDART_INF_F ? 0.f : M;
    float acc[DPL], ls = 0.f;
#pragma unroll
    for (int d = 0; d < DPL; ++d)
        acc[d] = 0.f;
    constexpr int kStep = kWide ? kWarps : 1;
    for (int s0 = kWide ? warp : 0; s0 < n; s0 += kLoads * kStep) {
        float v[kLoads][DPL], w[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int s = s0 + i * kStep;
            w[i] = -CUDART_INF_F;
#pragma unroll
            for (int d = 0; d < DPL; ++d)
                v[i][d] = 0.f;
            if (s < n) {
                w[i] = __ldcg(lse + s);
                if constexpr (DPL == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(o + (int64_t)s * D));
                    v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2 *>(o + (int64_t)s * D));
                    v[i][0] = x.x; v[i][1] = x.y;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            w[i] = exp2f(w[i] - M);
            ls += w[i];
#pragma unroll
            for (int d = 0; d < DPL; ++d)
                acc[d] = fmaf(w[i], v[i][d], acc[d]);
        }
    }
    if constexpr (kWide) {
#pragma unroll
        for (int d = 0; d < DPL; ++d)
            part[warp][lane * DPL + d] = acc[d];
        if (lane == 0)
            part[warp][D] = ls;
        __syncthreads();
        if (warp != 0)
            return;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            ls += part[w][D];
#pragma unroll
            for (int d = 0; d < DPL; ++d)
                acc[d] += part[w][lane * DPL + d];
        }
    }
    const float inv = ls == 0.f ? 0.f : 1.f / ls;
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + bh * D + lane * DPL);
#pragma unroll
    for (int d = 0; d < DPL / 2; ++d)
        dst[d] = cvt_bf16x2(acc[2 * d] * inv, acc[2 * d + 1] * inv);
    if (lane == 0 && p.lse_out != nullptr)
        p.lse_out[bh] = ls == 0.f ? -CUDART_INF_F : (M + log2f(ls)) * kLn2;
}

// One bank side as rows of D bytes; boxes of a 16-token tile, swizzled by the row's width.
bool make_map8(CUtensorMap *map, const uint8_t *bank, int64_t rows, int head_dim)
{
    const cuuint64_t dims[2] = {(cuuint64_t)head_dim, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)head_dim};
    const cuuint32_t box[2] = {(cuuint32_t)head_dim, (cuuint32_t)kTileTokens};
    const cuuint32_t estr[2] = {1, 1};
    const tc::EncodeTiledFn fn = tc::encode_tiled_fn();
    return fn != nullptr &&
           fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(bank), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kFault>
cudaError_t launch_typed8(const DecodeParams &p, const Kv8Bank &bank, cudaStream_t stream, bool early)
{
    using C = Cfg8<D>;
    static_assert(C::kSmemBytes <= 227 * 1024, "shared memory budget");
    CUtensorMap kmap, vmap;
    const int64_t rows = p.num_pages > 0 ? p.num_pages * p.num_kv_heads * p.page_size : 1;   // (an empty pool: never read)
    if (!make_map8(&kmap, bank.k, rows, D) || !make_map8(&vmap, bank.v, rows, D))
        return cudaErrorInvalidValue;
    // The shared-memory opt-in is per function and device: set it once per device.
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (bit == 0 || (configured.load(std::memory_order_acquire) & bit) == 0) {
        e = cudaFuncSetAttribute(kv8_partial_kernel<D, kFault>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess)
            return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    e = launch_kernel(kv8_partial_kernel<D, kFault>, dim3(p.max_splits, p.num_kv_heads, p.batch), dim3(kThreads),
                      C::kSmemBytes, stream, true, kmap, vmap, p, bank.k_exp, bank.v_exp, early ? 1 : 0);
    if (e != cudaSuccess || p.max_splits <= 1)
        return e;
    const int64_t q_rows = (int64_t)p.batch * p.num_q_heads;
    if (p.max_splits > kNarrowSplits)
        return launch_kernel(kv8_combine_kernel<D, true>, dim3((unsigned)q_rows), dim3(kThreads), 0, stream, true, p);
    return launch_kernel(kv8_combine_kernel<D, false>, dim3((unsigned)((q_rows + kWarps - 1) / kWarps)),
                         dim3(kThreads), 0, stream, true, p);
}

}  // namespace

bool kv8_decode_supported(int head_dim, int group)
{
    return (head_dim == 64 || head_dim == 128) && group >= 1 && group <= kMaxGroup;
}

cudaError_t launch_kv8_decode(const DecodeParams &p, const Kv8Bank &bank, int head_dim, cudaStream_t stream, bool early)
{
    if (p.debug_drop_copy != 0)
        return head_dim == 128 ? launch_typed8<128, true>(p, bank, stream, early)
                               : launch_typed8<64, true>(p, bank, stream, early);
    return head_dim == 128 ? launch_typed8<128, false>(p, bank, stream, early)
                           : launch_typed8<64, false>(p, bank, stream, early);
}

}  // namespace rlt
