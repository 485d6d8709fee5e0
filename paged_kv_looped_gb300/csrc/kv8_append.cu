// Append of a step's or a prompt's keys and values to the 8-bit paged cache, with the position
// rotation of queries and keys, for sm_103a.
//
// "Faster fuzzy minds", "LOTUS": store_kv writes each token's rows to the slots it is handed;
// "Recurrent depth": a token keeps one RoPE position across all its banks.  Per token: its query
// heads are rotated to bf16, its keys rotated and quantised, its values quantised (rlt_fp8.cuh).
//
// The angle of pair i at position p is p * base^(-2i/rot) radians.  Its turns, p * base^(-2i/rot)
// / 2 pi, matter modulo 1 only: with the frequency as a 64-bit fixed-point fraction F_i of a turn,
// the low 64 bits of p * F_i are that fraction of a turn, exactly reduced for any position (F_i
// carries fp64's rounding, 2^-53 relative: 2^-36 turns at position 2^17).  The nearest quarter
// turn goes to the quadrant, the rest, at most pi/4, to the Taylor polynomials of sin and cos.
#include <cmath>

#include "rlt_device.cuh"
#include "rlt_fp8.cuh"
#include "rlt_internal.h"

namespace rlt {
namespace {

constexpr int kAppendWarps = 8;

// cos and sin of `turns` / 2^64 turns.  x is off by at most 2^-33 turns and its fp32 rounding; the
// polynomials' first dropped terms are below 2e-9 and 2e-10 for |x| <= pi/4.
__device__ __forceinline__ void turn_cos_sin(uint64_t turns, float &c, float &s)
{
    const uint32_t quadrant = (uint32_t)((turns + (1ull << 61)) >> 62);
    const int32_t rest = (int32_t)((int64_t)(turns - ((uint64_t)quadrant << 62)) >> 31);
    const float x = (float)rest * (6.283185307179586f / 8589934592.f);   // 2 pi / 2^33
    const float y = x * x;
    const float sp = fmaf(fmaf(fmaf(fmaf(y, 1.f / 362880.f, -1.f / 5040.f), y, 1.f / 120.f), y, -1.f / 6.f), y * x, x);
    const float cp = fmaf(
        fmaf(fmaf(fmaf(fmaf(y, -1.f / 3628800.f, 1.f / 40320.f), y, -1.f / 720.f), y, 1.f / 24.f), y, -0.5f), y, 1.f);
    const float cc = (quadrant & 1u) ? sp : cp, ss = (quadrant & 1u) ? cp : sp;
    c = ((quadrant + 1u) & 2u) ? -cc : cc;
    s = (quadrant & 2u) ? -ss : ss;
}

// One warp per row (a head of q, k or v of one token).
__global__ void __launch_bounds__(kAppendWarps * 32) kv8_append_kernel(const Kv8AppendParams p)
{
    __shared__ float rows[kAppendWarps][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = p.head_dim, half = p.rot_dim / 2;
    const int heads = p.num_q_heads + 2 * p.num_kv_heads;
    const int64_t total = (int64_t)p.n_tokens * heads;
    float *row = rows[warp];
    for (int64_t w = (int64_t)blockIdx.x * kAppendWarps + warp; w < total; w += (int64_t)gridDim.x * kAppendWarps) {
        const int64_t i = w / heads;
        const int h = (int)(w - i * heads);
        const int64_t slot = p.out_loc[i];
        if (slot < 0)
            continue;                            // no token for this entry
        if (slot >= p.num_slots) {
            if (h == 0 && lane == 0)
                record_error(p.err, RLT_DEVERR_BAD_SLOT);
            continue;
        }
        const int kind = h < p.num_q_heads ? 0 : h < p.num_q_heads + p.num_kv_heads ? 1 : 2;
        const int g = kind == 0 ? h : h - p.num_q_heads - (kind - 1) * p.num_kv_heads;
        const uint16_t *src = kind == 0   ? p.q + i * p.q_stride + (int64_t)g * D
                              : kind == 1 ? p.k_new + i * p.k_stride + (int64_t)g * D
                                          : p.v_new + i * p.v_stride + (int64_t)g * D;
        uint32_t amax = 0u;
        __syncwarp();
        for (int d = lane; d < D; d += 32) {
            const uint32_t b = src[d];
            amax = max(amax, b & 0x7fffu);
            row[d] = __uint_as_float(b << 16);
        }
        amax = __reduce_max_sync(kFullMask, amax);
        __syncwarp();
        const uint64_t pos = kind < 2 && half > 0 ? (uint64_t)p.positions[i] : 0ull;
        if (kind < 2) {
            for (int j = lane; j < half; j += 32) {
                float c, s;
                turn_cos_sin(pos * p.freq[j], c, s);
                const float a = row[j], b = row[j + half];
                row[j] = fmaf(a, c, -(b * s));
                row[j + half] = fmaf(b, c, a * s);
            }
            __syncwarp();
        }
        if (kind == 0) {
            for (int d = lane * 2; d < D; d += 64)
                reinterpret_cast<uint32_t *>(p.q_out)[((i * p.num_q_heads + g) * D + d) / 2] =
                    cvt_bf16x2(row[d], row[d + 1]);
            continue;
        }
        const uint32_t byte = row_exponent(amax);
        const float scale = exp_scale(byte), inv = exp_inverse(byte);
        const int64_t page = slot / p.page_size;
        const int64_t at = (page * p.num_kv_heads + g) * p.page_size + (slot - page * p.page_size);
        uint8_t *dst = (kind == 1 ? p.k_bank : p.v_bank) + at * D;
        uint16_t *held = kind == 1 ? p.k_out : p.v_out;
        for (int d = lane * 2; d < D; d += 64) {
            const uint32_t x8 = e4m3x2(row[d] * inv, row[d + 1] * inv);
            *reinterpret_cast<uint16_t *>(dst + d) = (uint16_t)x8;
            if (held != nullptr) {
                const float2 f = f32x2_of_f16(f16x2_of_e4m3(x8));
                reinterpret_cast<uint32_t *>(held)[((i * p.num_kv_heads + g) * D + d) / 2] =
                    cvt_bf16x2(f.x * scale, f.y * scale);
            }
        }
        if (lane == 0) {
            (kind == 1 ? p.k_exp : p.v_exp)[at] = (uint8_t)byte;
            if (kind == 1 && g == 0 && p.written != nullptr) {
                const int32_t r = p.request[i];
                if (r >= 0 && r < p.batch)
                    atomicMax(&p.written[r], (int32_t)min(p.positions[i] + 1, (int64_t)INT32_MAX));
                else
                    record_error(p.err, RLT_DEVERR_BAD_SLOT);
            }
        }
    }
}

}  // namespace

// F_i = base^(-2i/rot) / 2 pi turns per position, modulo one turn, as a 64-bit fraction.
void rope_frequencies(int rot_dim, double base, uint64_t *freq)
{
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double turns = std::fmod(std::pow(base, -2.0 * i / rot_dim) * 0.15915494309189535, 1.0);
        freq[i] = (uint64_t)(turns * 18446744073709551616.0);
    }
}

cudaError_t launch_kv8_append(const Kv8AppendParams &p, cudaStream_t stream)
{
    const int64_t rows = (int64_t)p.n_tokens * (p.num_q_heads + 2 * p.num_kv_heads);
    int64_t blocks = (rows + kAppendWarps - 1) / kAppendWarps;
    if (blocks > (1 << 20))
        blocks = 1 << 20;
    kv8_append_kernel<<<(unsigned)blocks, kAppendWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace rlt
