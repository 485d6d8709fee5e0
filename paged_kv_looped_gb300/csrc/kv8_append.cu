// Append of a step's or a prompt's keys and values to the 8-bit paged cache, with the position
// rotation of queries and keys, for sm_103a.
//
// "Faster fuzzy minds", "LOTUS": store_kv writes each token's rows to the slots it is handed;
// "Recurrent depth": a token keeps one RoPE position across all its banks.  Per token: its query
// heads are rotated to bf16, its keys rotated and quantised, its values quantised (rlt_fp8.cuh).
//
// The angle of pair i at position p is p * base^(-2i/rot) radians.  Its turns, p * base^(-2i/rot)
// / 2 pi, matter modulo 1 only: with the frequency as a 64-bit fixed-point fraction F_i of a turn,
// the low 64 bits of p * F_i are that fraction of a turn, exactly reduced for any position (F_i is made
// in extended precision: at position 2^31 the angle is off by 2^-29 rad).  The nearest quarter
// turn goes to the quadrant, the rest, at most pi/4, to the Taylor polynomials of sin and cos.
#include <cmath>

#include "rlt_device.cuh"
#include "rlt_fp8.cuh"
#include "rlt_internal.h"

namespace rlt {
namespace {

constexpr int kAppendWarps = 4;
// Warps that fill the SMs: fewer tokens than this are split by heads.  Splitting more (2 warps a token at 16389
// tokens of 80 heads) took 130 us where this took 118: a token's angles are then made twice.
constexpr int kSpreadWarps = 152 * 16;

// cos and sin of `turns` / 2^64 turns, to a little over half an ulp: the angle x + dx in two parts (dx: what
// the 24 bits of x leave of it), the polynomials' small terms added last.  Their first dropped terms
// are below 2e-9 and 2e-10 for |x| <= pi/4.  Of 67 million keys 68 are then held one e4m3 step off the exact
// rotation's (they lie next to a tie), 85 with plain fp32 products of correctly rounded cosines.  Sums in two
// parts, rounded to the odd neighbour, left 2 and took 131 us where this takes 115 (16389 tokens of 64 + 16 heads).
__device__ __forceinline__ void turn_cos_sin(uint64_t turns, float &c, float &s)
{
    constexpr float kUnit = 6.283185307179586f / 8589934592.f;            // 2 pi / 2^33
    constexpr float kUnitLo = (float)(6.283185307179586 / 8589934592. - (double)kUnit);
    const uint32_t quadrant = (uint32_t)((turns + (1ull << 61)) >> 62);
    const int32_t rest = (int32_t)((int64_t)(turns - ((uint64_t)quadrant << 62)) >> 31);
    const float hi = (float)(rest & ~127), lo = (float)(rest & 127);      // hi: 24 bits, exact
    const float x = hi * kUnit;
    const float dx = fmaf(hi, kUnit, -x) + fmaf(hi, kUnitLo, lo * kUnit);
    const float y = x * x, dy = fmaf(x, x, -y);
    const float ps = fmaf(fmaf(fmaf(y, 1.f / 362880.f, -1.f / 5040.f), y, 1.f / 120.f), y, -1.f / 6.f) * (y * x);
    const float pc = fmaf(fmaf(fmaf(y, -1.f / 3628800.f, 1.f / 40320.f), y, -1.f / 720.f), y, 1.f / 24.f) * y;
    const float w = fmaf(y, -0.5f, 1.f), dw = (1.f - w) - 0.5f * y;       // 1 - y/2 and what its rounding left
    const float sp = x + (ps + fmaf(dx, -0.5f * y, dx));
    const float cp = w + (dw + fmaf(pc, y, -fmaf(dx, x, 0.5f * dy)));
    const float cc = (quadrant & 1u) ? sp : cp, ss = (quadrant & 1u) ? cp : sp;
    c = ((quadrant + 1u) & 2u) ? -cc : cc;
    s = (quadrant & 2u) ? -ss : ss;
}

// Where row h of a token (its query heads, then its key heads, then its value heads) comes from.
struct RowAt {
    const uint16_t *src;
    int kind, g;                                 // 0 query, 1 key, 2 value; head
};

__device__ __forceinline__ RowAt row_at(const Kv8AppendParams &p, int64_t i, int h, int D)
{
    const int kind = h < p.num_q_heads ? 0 : h < p.num_q_heads + p.num_kv_heads ? 1 : 2;
    const int g = kind == 0 ? h : h - p.num_q_heads - (kind - 1) * p.num_kv_heads;
    const uint16_t *src = kind == 0   ? p.q + i * p.q_stride
                          : kind == 1 ? p.k_new + i * p.k_stride
                                      : p.v_new + i * p.v_stride;
    return {src + (int64_t)g * D, kind, g};
}

// The token's slot, or -1 where nothing is written for it; a slot past the pool is recorded once.
__device__ __forceinline__ int64_t token_slot(const Kv8AppendParams &p, int64_t i, bool report)
{
    const int64_t slot = p.out_loc[i];
    if (slot < p.num_slots)
        return slot < 0 ? -1 : slot;
    if (report)
        record_error(p.err, RLT_DEVERR_BAD_SLOT);
    return -1;
}

// The request's counter becomes at least the position + 1, as an int32 holds it; a position below 0 counts nothing.
__device__ __forceinline__ void count_written(const Kv8AppendParams &p, int64_t i)
{
    const int32_t r = p.request[i];
    if (r >= 0 && r < p.batch)
        atomicMax(&p.written[r], (int32_t)min(max(p.positions[i], (int64_t)-1), (int64_t)INT32_MAX - 1) + 1);
    else
        record_error(p.err, RLT_DEVERR_BAD_SLOT);
}

// 16 values of a row from one 16-byte chunk pair: fp32, and the largest magnitude's bf16 bits.
__device__ __forceinline__ void unpack8(const uint4 &w, float (&f)[8])
{
    f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
}

__device__ __forceinline__ uint32_t amax2(const uint4 &w)
{
    return __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8], float by)
{
    return make_uint4(cvt_bf16x2(f[0] * by, f[1] * by), cvt_bf16x2(f[2] * by, f[3] * by),
                      cvt_bf16x2(f[4] * by, f[5] * by), cvt_bf16x2(f[6] * by, f[7] * by));
}

// Rotations whose halves are whole 16-byte chunks (rot_dim a multiple of 16; so is head_dim).  A lane holds the
// two chunks of a row that turn into each other (or two neighbouring chunks behind rot_dim) and D / 16
// lanes a row, so a row needs no exchange but its largest magnitude.  A warp stays with one token: its
// angles are computed once and used for every head; the rows of kBatch rounds are loaded before the
// first is worked on.  Bound by memory: 2 (hq + 2 hkv) D bytes in, as many out, and the cache: 16389 tokens
// of 64 + 16 heads (705 MB) 115 us, 6.1 TB/s (a copy's rate is 6.7).  Rounds: 3 and 4 take 115 us
// here, 27 and 29 us for 16000 tokens of 6 + 4 heads (90 MB, 13.5 us of bytes: a warp's one round of rows leaves
// nothing in flight while it is worked on; before the angles were shared: 2 rounds 125 us where 4
// took 118).  A lane computing all its eight angles itself took 118 and 34 us, a kernel of one row a warp 863.
constexpr int kBatch = 3;

template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32) kv8_append_chunks_kernel(const Kv8AppendParams p, int splits)
{
    constexpr int kLanes = D / 16, kRows = 32 / kLanes;
    pdl_wait();                                  // (launched while the kernel ahead ends)
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const int64_t i = w / splits;
    if (i >= p.n_tokens)
        return;
    const int part = (int)(w - i * splits);
    const int t = lane % kLanes, r0 = part * kRows + lane / kLanes, step = splits * kRows;
    __shared__ __align__(16) float2 angles[kAppendWarps][64];
    float2 *mine = angles[threadIdx.x >> 5];
    const int turned = p.rot_dim / 16;
    const bool turns = t < turned;
    const int ca = turns ? t : 2 * t, cb = turns ? t + turned : 2 * t + 1;   // this lane's chunks
    const int heads = p.num_q_heads + 2 * p.num_kv_heads;

    uint4 a[kBatch], b[kBatch];
    auto load = [&](int r) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = r + u * step;
            if (h < heads) {
                const uint4 *src = reinterpret_cast<const uint4 *>(row_at(p, i, h, D).src);
                a[u] = __ldcs(src + ca);
                b[u] = __ldcs(src + cb);
            } else {
                a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    };
    const uint64_t pos = turned > 0 ? (uint64_t)p.positions[i] : 0ull;
    load(r0);                                    // (rows of an unused entry are read too: one round trip fewer)
    const int64_t slot = token_slot(p, i, part == 0 && lane == 0);
    if (slot < 0)
        return;
    // A lane makes at most two of the token's rot_dim / 2 angles and takes its eight from the warp's.
    float c[8], s[8];
    for (int k = lane; k < p.rot_dim / 2; k += 32)
        turn_cos_sin(pos * p.freq[k], mine[k].x, mine[k].y);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        const float4 x = turns ? *reinterpret_cast<const float4 *>(&mine[t * 8 + k]) : make_float4(0.f, 0.f, 0.f, 0.f);
        c[k] = x.x;
        s[k] = x.y;
        c[k + 1] = x.z;
        s[k + 1] = x.w;
    }
    const int64_t page = slot / p.page_size;
    const int64_t at0 = page * p.num_kv_heads * p.page_size + (slot - page * p.page_size);
    for (int r = r0; r - r0 < heads - part * kRows; r += step * kBatch) {   // (uniform over the warp)
        if (r != r0)
            load(r);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = r + u * step;
            uint32_t m2 = __vmaxu2(amax2(a[u]), amax2(b[u]));
            uint32_t amax = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
                amax = max(amax, __shfl_xor_sync(kFullMask, amax, o));
            if (h >= heads)
                continue;
            const RowAt row = row_at(p, i, h, D);
            float fa[8], fb[8];
            unpack8(a[u], fa);
            unpack8(b[u], fb);
            if (turns && row.kind < 2) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float x = fa[k], y = fb[k];
                    fa[k] = fmaf(x, c[k], -(y * s[k]));
                    fb[k] = fmaf(y, c[k], x * s[k]);
                }
            }
            if (row.kind == 0) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.q_out + (i * p.num_q_heads + row.g) * D);
                dst[ca] = pack8(fa, 1.f);
                dst[cb] = pack8(fb, 1.f);
                continue;
            }
            const uint32_t byte = row_exponent(amax);
            const float scale = exp_scale(byte), inv = exp_inverse(byte);
            const int64_t at = at0 + (int64_t)row.g * p.page_size;
            uint2 *dst = reinterpret_cast<uint2 *>((row.kind == 1 ? p.k_bank : p.v_bank) + at * D);
            uint16_t *held = row.kind == 1 ? p.k_out : p.v_out;
            uint4 *hd = reinterpret_cast<uint4 *>(held + (held != nullptr ? (i * p.num_kv_heads + row.g) * D : 0));
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                float (&f)[8] = side == 0 ? fa : fb;
                uint32_t x8[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x8[k] = e4m3x2(f[2 * k] * inv, f[2 * k + 1] * inv);
                dst[side == 0 ? ca : cb] = make_uint2(x8[0] | (x8[1] << 16), x8[2] | (x8[3] << 16));
                if (held != nullptr) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 v = f32x2_of_f16(f16x2_of_e4m3(x8[k]));
                        f[2 * k] = v.x;
                        f[2 * k + 1] = v.y;
                    }
                    hd[side == 0 ? ca : cb] = pack8(f, scale);
                }
            }
            if (t == 0) {
                (row.kind == 1 ? p.k_exp : p.v_exp)[at] = (uint8_t)byte;
                if (row.kind == 1 && row.g == 0 && p.written != nullptr)
                    count_written(p, i);
            }
        }
    }
}

template <int N>
__device__ __forceinline__ void load_words(const uint32_t *src, uint32_t (&x)[N])
{
    if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(src);
        x[0] = v.x;
        x[1] = v.y;
    } else {
        x[0] = *src;
    }
}

template <int N>
__device__ __forceinline__ void store_words(uint16_t *row, int lane, const uint32_t (&y)[N])
{
    if constexpr (N == 2)
        reinterpret_cast<uint2 *>(row)[lane] = make_uint2(y[0], y[1]);
    else
        reinterpret_cast<uint32_t *>(row)[lane] = y[0];
}

// Any even rot_dim: a row passes through shared memory, where a lane finds the other member of its pairs.
// A warp stays with one token; its angles (at most two pairs a lane) are computed once.  16000 tokens of 32 + 16
// heads at rot_dim 62 (426 MB, 64 us of bytes) 105 us; one row at a time took 128.
template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32) kv8_append_pairs_kernel(const Kv8AppendParams p, int splits)
{
    constexpr int kWords = D / 64;               // 32-bit words of a row that a lane loads
    __shared__ __align__(16) float rows[kAppendWarps][kBatch][D];
    pdl_wait();                                  // (launched while the kernel ahead ends)
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const int64_t i = w / splits;
    if (i >= p.n_tokens)
        return;
    const int part = (int)(w - i * splits), half = p.rot_dim / 2;
    const int64_t slot = token_slot(p, i, part == 0 && lane == 0);
    if (slot < 0)
        return;
    float (*row)[D] = rows[threadIdx.x >> 5];
    const int heads = p.num_q_heads + 2 * p.num_kv_heads;
    float c[2], s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (lane + 32 * k < half)
            turn_cos_sin((uint64_t)p.positions[i] * p.freq[lane + 32 * k], c[k], s[k]);
    const int64_t page = slot / p.page_size;
    const int64_t at0 = page * p.num_kv_heads * p.page_size + (slot - page * p.page_size);
    for (int h0 = part; h0 < heads; h0 += splits * kBatch) {
        uint32_t x[kBatch][kWords];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = min(h0 + u * splits, heads - 1);       // (a row past the last is loaded, not written)
            const uint32_t *src = reinterpret_cast<const uint32_t *>(row_at(p, i, h, D).src) + lane * kWords;
            load_words(src, x[u]);
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if constexpr (kWords == 2)
                *reinterpret_cast<float4 *>(row[u] + lane * 4) =
                    make_float4(bf16_lo(x[u][0]), bf16_hi(x[u][0]), bf16_lo(x[u][1]), bf16_hi(x[u][1]));
            else
                *reinterpret_cast<float2 *>(row[u] + lane * 2) = make_float2(bf16_lo(x[u][0]), bf16_hi(x[u][0]));
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (h0 + u * splits >= p.num_q_heads + p.num_kv_heads)
                break;                           // values
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = lane + 32 * k;
                if (j < half) {
                    const float a = row[u][j], b = row[u][j + half];
                    row[u][j] = fmaf(a, c[k], -(b * s[k]));
                    row[u][j + half] = fmaf(b, c[k], a * s[k]);
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = h0 + u * splits;
            if (h >= heads)
                break;
            const RowAt r = row_at(p, i, h, D);
            uint32_t amax = 0u;
#pragma unroll
            for (int k = 0; k < kWords; ++k)
                amax = max(amax, max(x[u][k] & 0x7fffu, (x[u][k] >> 16) & 0x7fffu));
            if (r.kind != 0)
                amax = __reduce_max_sync(kFullMask, amax);
            const uint32_t byte = row_exponent(amax);
            const float scale = exp_scale(byte), inv = exp_inverse(byte);
            const int64_t at = at0 + (int64_t)r.g * p.page_size;
            uint16_t *held = r.kind == 1 ? p.k_out : p.v_out;
            float f[2 * kWords];
            if constexpr (kWords == 2) {
                const float4 v = *reinterpret_cast<const float4 *>(row[u] + lane * 4);
                f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(row[u] + lane * 2);
                f[0] = v.x; f[1] = v.y;
            }
            uint32_t y[kWords], x8 = 0u;
            if (r.kind == 0) {
#pragma unroll
                for (int k = 0; k < kWords; ++k)
                    y[k] = cvt_bf16x2(f[2 * k], f[2 * k + 1]);
                store_words(p.q_out + (i * p.num_q_heads + r.g) * D, lane, y);
                continue;
            }
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                const uint32_t pair = e4m3x2(f[2 * k] * inv, f[2 * k + 1] * inv);
                const float2 v = f32x2_of_f16(f16x2_of_e4m3(pair));
                y[k] = cvt_bf16x2(v.x * scale, v.y * scale);
                x8 |= pair << (16 * k);
            }
            uint8_t *dst = (r.kind == 1 ? p.k_bank : p.v_bank) + at * D;
            if constexpr (kWords == 2)
                reinterpret_cast<uint32_t *>(dst)[lane] = x8;
            else
                reinterpret_cast<uint16_t *>(dst)[lane] = (uint16_t)x8;
            if (held != nullptr)
                store_words(held + (i * p.num_kv_heads + r.g) * D, lane, y);
            if (lane == 0) {
                (r.kind == 1 ? p.k_exp : p.v_exp)[at] = (uint8_t)byte;
                if (r.kind == 1 && r.g == 0 && p.written != nullptr)
                    count_written(p, i);
            }
        }
    }
}

template <int D>
cudaError_t launch_append_typed(const Kv8AppendParams &p, cudaStream_t stream)
{
    const int heads = p.num_q_heads + 2 * p.num_kv_heads;
    const bool chunks = p.rot_dim % 16 == 0;
    const int rounds = chunks ? (heads * (D / 16) + 31) / 32 : heads;
    // Warps per token: few tokens are spread over the SMs, row by row; many keep one warp each, whose
    // angles then serve all heads.
    const int64_t want = kSpreadWarps / (p.n_tokens > 0 ? p.n_tokens : 1);
    const int splits = (int)(want < 1 ? 1 : want < rounds ? want : rounds);
    const int64_t blocks = ((int64_t)p.n_tokens * splits + kAppendWarps - 1) / kAppendWarps;
    return launch_kernel(chunks ? kv8_append_chunks_kernel<D> : kv8_append_pairs_kernel<D>, dim3((unsigned)blocks),
                         dim3(kAppendWarps * 32), 0, stream, true, p, splits);
}

}  // namespace

// F_i = base^(-2i/rot) / 2 pi turns per position, modulo one turn, as a 64-bit fraction.  Positions multiply its
// error, so it needs all 64 bits: long double (a mantissa of 64 bits or more), one power and a product a pair.
void rope_frequencies(int rot_dim, double base, uint64_t *freq)
{
    if (rot_dim < 2)
        return;
    const long double step = std::pow((long double)base, -2.0L / rot_dim);
    long double turns = 0.1591549430918953357688837633725143620L;
    for (int i = 0; i < rot_dim / 2; ++i, turns *= step)
        freq[i] = (uint64_t)(std::fmod(turns, 1.0L) * 18446744073709551616.0L);
}

cudaError_t launch_kv8_append(const Kv8AppendParams &p, cudaStream_t stream)
{
    return p.head_dim == 128 ? launch_append_typed<128>(p, stream) : launch_append_typed<64>(p, stream);
}

}  // namespace rlt
