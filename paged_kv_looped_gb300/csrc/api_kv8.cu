// extern "C" entry points of the 8-bit cache and of packed prompts: host-side argument checks and dispatch to the
// kernels.  Nothing here allocates device memory.
#include <cuda_runtime.h>

#include <cmath>

#include "rlt.h"
#include "rlt_internal.h"

namespace {

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

rlt_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RLT_OK : RLT_ERR_CUDA; }

rlt_status check_pool8(const rlt_kv8_pool *pool, int32_t bank)
{
    if (pool == nullptr || pool->k == nullptr || pool->v == nullptr || pool->k_exp == nullptr || pool->v_exp == nullptr)
        return RLT_ERR_INVALID_ARG;
    if (pool->num_pages < 0 || pool->num_banks < 1 || pool->num_kv_heads < 1 || pool->page_size < 1 ||
        pool->head_dim < 1)
        return RLT_ERR_INVALID_ARG;
    if (!aligned16(pool->k) || !aligned16(pool->v) || !aligned16(pool->k_exp) || !aligned16(pool->v_exp))
        return RLT_ERR_INVALID_ARG;
    // a 16-token tile of one kv head is the unit of every copy; its first row has to fit an int32
    if ((pool->head_dim != 64 && pool->head_dim != 128) || pool->page_size % rlt::kTileTokens != 0 ||
        pool->num_pages > (INT64_C(0x7fffffff) / pool->num_kv_heads) / pool->page_size)
        return RLT_ERR_UNSUPPORTED;
    if (bank < 0 || bank >= pool->num_banks)
        return RLT_ERR_OUT_OF_RANGE;
    return RLT_OK;
}

// A rows x width block of bf16 elements, `stride` elements from row to row.
struct Block {
    const void *ptr;
    int64_t rows, width, stride;
    uintptr_t begin() const { return reinterpret_cast<uintptr_t>(ptr); }
    uintptr_t end() const { return begin() + (uintptr_t)((rows - 1) * stride + width) * 2; }
};

// An output may lie exactly on its own input (every row is read before it is written), but on
// nothing else.
bool clashes(const Block &out, const Block &in, bool own_input)
{
    if (out.ptr == nullptr || in.ptr == nullptr || out.end() <= in.begin() || in.end() <= out.begin())
        return false;
    return !(own_input && out.ptr == in.ptr && out.stride == in.stride);
}

}  // namespace

extern "C" {

RLT_API rlt_status rlt_kv8_append_rope(const rlt_kv8_pool *pool, int32_t bank, const void *q, int32_t num_q_heads,
                                       int64_t q_stride, const void *k_new, int64_t k_stride, const void *v_new,
                                       int64_t v_stride, const int64_t *positions, const int64_t *out_loc,
                                       int32_t n_tokens, int32_t rot_dim, double rope_base, void *q_out, void *k_out,
                                       void *v_out, const int32_t *request, int32_t *written, int32_t batch,
                                       void *stream)
{
    rlt_status st = check_pool8(pool, bank);
    if (st != RLT_OK)
        return st;
    const int64_t kv_width = (int64_t)pool->num_kv_heads * pool->head_dim;
    const int64_t q_width = (int64_t)num_q_heads * pool->head_dim;
    if (n_tokens < 0 || rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > pool->head_dim ||
        (rot_dim > 0 && (!(rope_base > 0.0) || !std::isfinite(rope_base))) ||
        (written != nullptr && (request == nullptr || batch < 1)) || (q != nullptr) != (q_out != nullptr) ||
        (q != nullptr && num_q_heads < 1))
        return RLT_ERR_INVALID_ARG;
    if (n_tokens == 0)
        return RLT_OK;
    if (k_new == nullptr || v_new == nullptr || out_loc == nullptr ||
        (positions == nullptr && (rot_dim > 0 || written != nullptr)))
        return RLT_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q_out) || !aligned16(k_out) ||
        !aligned16(v_out) || reinterpret_cast<uintptr_t>(out_loc) % 8 != 0 ||
        reinterpret_cast<uintptr_t>(positions) % 8 != 0 || reinterpret_cast<uintptr_t>(request) % 4 != 0 ||
        reinterpret_cast<uintptr_t>(written) % 4 != 0)
        return RLT_ERR_INVALID_ARG;
    if (k_stride < kv_width || v_stride < kv_width || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        (q != nullptr && (q_stride < q_width || q_stride % 8 != 0)))
        return RLT_ERR_INVALID_ARG;
    const Block in[3] = {{q, n_tokens, q_width, q_stride}, {k_new, n_tokens, kv_width, k_stride},
                         {v_new, n_tokens, kv_width, v_stride}};
    const Block out[3] = {{q_out, n_tokens, q_width, q_width}, {k_out, n_tokens, kv_width, kv_width},
                          {v_out, n_tokens, kv_width, kv_width}};
    for (int o = 0; o < 3; ++o)
        for (int i = 0; i < 3; ++i)
            if (clashes(out[o], in[i], o == i) || (i < o && clashes(out[o], out[i], false)))
                return RLT_ERR_INVALID_ARG;
    const int64_t slots = pool->num_pages * pool->page_size;
    // nor on the pool's own arrays (in 2-byte elements, rounded up)
    const int64_t pool_rows = (int64_t)pool->num_banks * slots * pool->num_kv_heads;
    const Block held[4] = {{pool->k, 1, pool_rows * pool->head_dim / 2, 0}, {pool->v, 1, pool_rows * pool->head_dim / 2, 0},
                           {pool->k_exp, 1, (pool_rows + 1) / 2, 0}, {pool->v_exp, 1, (pool_rows + 1) / 2, 0}};
    for (int o = 0; o < 3; ++o)
        for (int i = 0; i < 4; ++i)
            if (clashes(out[o], held[i], false))
                return RLT_ERR_INVALID_ARG;
    if ((st = rlt::validate_slots(out_loc, n_tokens, slots, static_cast<cudaStream_t>(stream))) != RLT_OK)
        return st;

    rlt::Kv8AppendParams p{};
    if ((st = rlt::current_device_info(&p.err, nullptr)) != RLT_OK)
        return st;
    const int64_t rows = (int64_t)bank * slots * pool->num_kv_heads;
    p.q = static_cast<const uint16_t *>(q);
    p.k_new = static_cast<const uint16_t *>(k_new);
    p.v_new = static_cast<const uint16_t *>(v_new);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.positions = positions;
    p.out_loc = out_loc;
    p.k_bank = static_cast<uint8_t *>(pool->k) + rows * pool->head_dim;
    p.v_bank = static_cast<uint8_t *>(pool->v) + rows * pool->head_dim;
    p.k_exp = pool->k_exp + rows;
    p.v_exp = pool->v_exp + rows;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.v_out = static_cast<uint16_t *>(v_out);
    p.request = request;
    p.written = written != nullptr ? written + (int64_t)bank * batch : nullptr;
    p.num_slots = slots;
    p.n_tokens = n_tokens;
    p.num_q_heads = q != nullptr ? num_q_heads : 0;
    p.num_kv_heads = pool->num_kv_heads;
    p.page_size = pool->page_size;
    p.head_dim = pool->head_dim;
    p.rot_dim = rot_dim;
    p.batch = batch;
    // the frequencies depend on (rot_dim, rope_base) alone, a model's constants: each host thread keeps
    // its last ones (up to 64 powers are a few microseconds of a step's launch)
    static thread_local struct { int32_t rot = -1; double base = 0.0; uint64_t freq[64]; } last;
    if (last.rot != rot_dim || last.base != rope_base) {
        rlt::rope_frequencies(rot_dim, rope_base, last.freq);
        last.rot = rot_dim;
        last.base = rope_base;
    }
    for (int i = 0; i < rot_dim / 2; ++i)
        p.freq[i] = last.freq[i];
    return from_cuda(rlt::launch_kv8_append(p, static_cast<cudaStream_t>(stream)));
}

RLT_API size_t rlt_paged_decode_kv8_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                                   int32_t head_dim, int32_t max_seq_len, int32_t split_tokens)
{
    return rlt_paged_decode_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, split_tokens);
}

RLT_API rlt_status rlt_paged_decode_attn_kv8(const rlt_kv8_pool *pool, int32_t bank, const void *q,
                                             int32_t num_q_heads, const int32_t *page_table, int32_t max_pages,
                                             const int32_t *seq_lens, int32_t batch, int32_t max_seq_len, float scale,
                                             void *out, float *lse_out, void *workspace, size_t workspace_bytes,
                                             int32_t split_tokens, uint32_t flags, void *stream)
{
    if ((flags & ~RLT_ATTN_EARLY_START) != 0)
        return RLT_ERR_INVALID_ARG;
    rlt_status st = check_pool8(pool, bank);
    if (st != RLT_OK)
        return st;
    if (batch < 0 || max_seq_len < 0 || max_pages < 0 || num_q_heads < 1 || split_tokens < 0 ||
        split_tokens % rlt::kTileTokens != 0 || split_tokens > 128 * rlt::kTileTokens ||
        num_q_heads % pool->num_kv_heads != 0)
        return RLT_ERR_INVALID_ARG;
    if (!rlt::kv8_decode_supported(pool->head_dim, num_q_heads / pool->num_kv_heads) || batch > 65535 ||
        pool->num_kv_heads > 65535)
        return RLT_ERR_UNSUPPORTED;
    if (batch == 0)
        return RLT_OK;
    if (q == nullptr || page_table == nullptr || seq_lens == nullptr || out == nullptr || max_pages < 1 ||
        !aligned16(q) || !aligned16(out) || !aligned16(workspace) || !std::isfinite(scale) ||
        reinterpret_cast<uintptr_t>(page_table) % 4 != 0 || reinterpret_cast<uintptr_t>(seq_lens) % 4 != 0 ||
        reinterpret_cast<uintptr_t>(lse_out) % 4 != 0)
        return RLT_ERR_INVALID_ARG;
    if ((st = rlt::validate_lengths(page_table, max_pages, seq_lens, batch, pool->num_pages, pool->page_size,
                                    static_cast<cudaStream_t>(stream))) != RLT_OK)
        return st;
    rlt::DecodeParams p{};
    int sms = 0;
    if ((st = rlt::current_device_info(&p.err, &sms)) != RLT_OK)
        return st;
    const rlt::DecodePlan plan = rlt::plan_decode(batch, num_q_heads, pool->num_kv_heads, pool->head_dim, max_seq_len,
                                                  split_tokens, sms);
    if (plan.workspace_bytes > 0 && (workspace == nullptr || workspace_bytes < plan.workspace_bytes))
        return RLT_ERR_WORKSPACE_TOO_SMALL;
    const int64_t rows = (int64_t)bank * pool->num_pages * pool->num_kv_heads * pool->page_size;
    const rlt::Kv8Bank b8{static_cast<const uint8_t *>(pool->k) + rows * pool->head_dim,
                          static_cast<const uint8_t *>(pool->v) + rows * pool->head_dim, pool->k_exp + rows,
                          pool->v_exp + rows};
    p.q = static_cast<const uint16_t *>(q);
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.out = static_cast<uint16_t *>(out);
    p.lse_out = lse_out;
    p.lse_part = static_cast<float *>(workspace);
    p.o_part = workspace != nullptr ? reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.lse_part_bytes)
                                    : nullptr;
    p.num_pages = pool->num_pages;
    p.num_kv_heads = pool->num_kv_heads;
    p.num_q_heads = num_q_heads;
    p.page_size = pool->page_size;
    p.max_pages = max_pages;
    p.batch = batch;
    p.tiles_per_split = plan.tiles_per_split;
    p.max_splits = plan.max_splits;
    p.part_stride = plan.max_splits;
    if ((p.wait_limit_ns = rlt::take_fault_limit()) != 0)
        p.debug_drop_copy = 1;
    const double s = scale > 0.f ? (double)scale : 1.0 / std::sqrt((double)pool->head_dim);
    p.qscale = (float)(s * 1.4426950408889634);   // log2(e): softmax in base 2
    return from_cuda(rlt::launch_kv8_decode(p, b8, pool->head_dim, static_cast<cudaStream_t>(stream),
                                            (flags & RLT_ATTN_EARLY_START) != 0));
}

RLT_API rlt_status rlt_prefill_attn(const void *q, int32_t num_q_heads, int64_t q_stride, const void *k,
                                    int64_t k_stride, const void *v, int64_t v_stride, int32_t num_kv_heads,
                                    int32_t head_dim, int32_t num_rows, const int32_t *items, int32_t num_items,
                                    int32_t max_key_tiles, int32_t total_key_tiles, float scale, void *out, float *lse_out, uint32_t flags, void *stream)
{
    if ((flags & ~RLT_ATTN_EARLY_START) != 0 || num_rows < 0 || num_items < 0 || max_key_tiles < 0 ||
        total_key_tiles < 0 || num_kv_heads < 1 || num_q_heads < 1 ||
        num_q_heads % num_kv_heads != 0 || !std::isfinite(scale))
        return RLT_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || (int64_t)num_items * num_q_heads > INT32_MAX)
        return RLT_ERR_UNSUPPORTED;
    if (num_items == 0)
        return RLT_OK;
    const int64_t q_width = (int64_t)num_q_heads * head_dim, kv_width = (int64_t)num_kv_heads * head_dim;
    if (num_rows < 1 || q == nullptr || k == nullptr || v == nullptr || items == nullptr || out == nullptr ||
        !aligned16(q) || !aligned16(k) || !aligned16(v) || reinterpret_cast<uintptr_t>(out) % 32 != 0 ||
        reinterpret_cast<uintptr_t>(items) % 4 != 0 || reinterpret_cast<uintptr_t>(lse_out) % 4 != 0)
        return RLT_ERR_INVALID_ARG;
    if (q_stride < q_width || k_stride < kv_width || v_stride < kv_width || q_stride % 8 != 0 || k_stride % 8 != 0 ||
        v_stride % 8 != 0)
        return RLT_ERR_INVALID_ARG;
    const Block to{out, num_rows, q_width, q_width};
    if (clashes(to, {q, num_rows, q_width, q_stride}, false) || clashes(to, {k, num_rows, kv_width, k_stride}, false) ||
        clashes(to, {v, num_rows, kv_width, v_stride}, false))
        return RLT_ERR_INVALID_ARG;
    rlt::PrefillParams p{};
    int sms = 0;
    rlt_status st = rlt::current_device_info(&p.err, &sms);
    if (st != RLT_OK)
        return st;
    p.max_tiles = max_key_tiles;
    p.total_tiles = total_key_tiles;
    p.num_sms = sms;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.items = items;
    p.out = static_cast<uint16_t *>(out);
    p.lse_out = lse_out;
    p.num_rows = num_rows;
    p.num_items = num_items;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.wait_limit_ns = rlt::take_fault_limit();
    const double s = scale > 0.f ? (double)scale : 1.0 / std::sqrt((double)head_dim);
    p.qscale = (float)(s * 1.4426950408889634);   // log2(e): softmax in base 2
    return from_cuda(rlt::launch_prefill(p, head_dim, static_cast<cudaStream_t>(stream),
                                         (flags & RLT_ATTN_EARLY_START) != 0));
}

}  // extern "C"
