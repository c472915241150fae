// mx_kv_api.cpp -- the C ABI of the key/value-cache operators (declared in include/mx_kv.h):
// argument validation, dispatch and error mapping.  Host code only; no allocation, no
// synchronization, no global state.
#include "mx_kv.h"

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "mx_kv_internal.h"

namespace {

constexpr int64_t kMaxDim = 512;
// Kernels number their units of work in 31 bits.  Writes and reads have two tensors' elements in units of 8 or
// 16: below 2^31 for any dense tensor that is accepted.  A rotation may have a unit for each element.
constexpr int64_t kMaxElems = int64_t(1) << 32;               // of a dense tensor
constexpr int64_t kMaxRopeElems = (int64_t(1) << 31) - 1;     // of a rotation's launch: larger ones go in parts
constexpr int64_t kMaxRows = int64_t(1) << 24;   // rows of an attention call

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool valid_g(float g) { return std::isfinite(g) && std::isnormal(g) && g > 0.0f; }
bool valid_type(mx_dtype t) { return t == MX_F32 || t == MX_BF16; }

// a non-negative product of non-negative numbers stays within `most`
bool within(int64_t a, int64_t b, int64_t most) { return a == 0 || b <= most / a; }

mx_status check_cache(const mxkv_cache* c)
{
    if (!c) return MX_ERR_INVALID_ARG;
    if (c->num_pages < 0 || c->heads < 1 || c->page_size < 1 || c->dim < 1) return MX_ERR_INVALID_ARG;
    if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128 && c->block != 256) return MX_ERR_INVALID_ARG;
    if (c->dim % c->block != 0) return MX_ERR_INVALID_ARG;
    if (c->element != MXKV_FP4 && c->element != MXKV_FP8) return MX_ERR_INVALID_ARG;
    if (c->fmt != MX_SCALE_E4M3 && c->fmt != MX_SCALE_UE5M3 && c->fmt != MX_SCALE_E8M0) return MX_ERR_INVALID_ARG;
    if (!valid_g(c->k_scale) || !valid_g(c->v_scale)) return MX_ERR_INVALID_ARG;
    if (!within(c->num_pages, c->page_size, INT32_MAX)) return MX_ERR_INVALID_ARG;
    if (c->dim > kMaxDim || c->heads > 65535) return MX_ERR_UNSUPPORTED;
    return MX_OK;
}

mx_status check_cache_memory(const mxkv_cache* c)
{
    if (c->num_pages == 0) return MX_OK;  // no slot exists, nothing of it is touched
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return MX_ERR_INVALID_ARG;
    if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales))
        return MX_ERR_ALIGNMENT;
    return MX_OK;
}

mxk::KvPool pool_of(const mxkv_cache* c)
{
    mxk::KvPool p{};
    p.codes[0] = c->k_codes;
    p.codes[1] = c->v_codes;
    p.scales[0] = c->k_scales;
    p.scales[1] = c->v_scales;
    p.g[0] = c->k_scale;
    p.g[1] = c->v_scale;
    p.num_pages = (uint32_t)c->num_pages;
    p.heads = (uint32_t)c->heads;
    p.page = (uint32_t)c->page_size;
    p.dim = (uint32_t)c->dim;
    p.block = (uint32_t)c->block;
    p.fp8 = c->element == MXKV_FP8;
    p.fmt = (int)c->fmt;
    return p;
}

mx_status check_rope(const int32_t* positions, const float* table, int64_t max_pos, int rot_dim, int64_t dim)
{
    if (rot_dim < 0 || (rot_dim & 1) || rot_dim > dim) return MX_ERR_INVALID_ARG;
    if (rot_dim == 0) return MX_OK;
    if (max_pos < 1 || max_pos > INT32_MAX || !positions || !table) return MX_ERR_INVALID_ARG;
    if (!aligned16(table) || !aligned4(positions)) return MX_ERR_ALIGNMENT;
    return MX_OK;
}

mxk::RopePart rope_of(const int32_t* positions, const float* table, int64_t max_pos, int rot_dim, int inter, int transpose)
{
    mxk::RopePart r{};
    r.positions = positions;
    r.table = rot_dim ? table : nullptr;
    r.max_pos = (uint32_t)max_pos;
    r.rot = (uint32_t)rot_dim;
    r.inter = inter != 0;
    r.transpose = transpose != 0;
    return r;
}

// tokens x heads x dim with unit stride along dim
mx_status check_dense(int64_t tokens, int64_t heads, int64_t dim)
{
    if (tokens < 0 || heads < 0 || dim < 0) return MX_ERR_INVALID_ARG;
    if (dim > kMaxDim) return MX_ERR_UNSUPPORTED;
    if (!within(tokens, heads, kMaxElems) || !within(tokens * heads, dim, kMaxElems - 1)) return MX_ERR_UNSUPPORTED;
    return MX_OK;
}

}  // namespace

extern "C" {

mx_status mxkv_rope_table(float* table, int64_t max_pos, int rot_dim, double base, mxkv_scaling scaling,
                          double factor, double original_len, double low, double high, double magnitude,
                          void* stream)
{
    if (max_pos < 0 || rot_dim < 0 || (rot_dim & 1)) return MX_ERR_INVALID_ARG;
    if (!std::isfinite(base) || !(base > 0) || !std::isfinite(factor) || !(factor > 0) || !std::isfinite(magnitude))
        return MX_ERR_INVALID_ARG;
    if (scaling != MXKV_SCALING_NONE && scaling != MXKV_SCALING_LINEAR && scaling != MXKV_SCALING_BASE &&
        scaling != MXKV_SCALING_PARTS)
        return MX_ERR_INVALID_ARG;
    if (scaling == MXKV_SCALING_BASE && rot_dim <= 2) return MX_ERR_INVALID_ARG;
    if (scaling == MXKV_SCALING_PARTS && (!std::isfinite(original_len) || !(original_len > 0) || !std::isfinite(low) ||
                                          !std::isfinite(high) || !(high > low)))
        return MX_ERR_INVALID_ARG;
    if (rot_dim > kMaxDim || !within(max_pos, rot_dim / 2, INT32_MAX)) return MX_ERR_UNSUPPORTED;
    if (max_pos == 0 || rot_dim == 0) return MX_OK;
    if (!table) return MX_ERR_INVALID_ARG;
    if (!aligned16(table)) return MX_ERR_ALIGNMENT;
    const mxk::RopeTableArgs a{table, (uint32_t)max_pos, (uint32_t)rot_dim / 2, base, factor, original_len, low, high,
                               magnitude, (int)scaling};
    return mxk::launch_rope_table(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MX_OK : MX_ERR_HIP;
}

mx_status mxkv_rope(const void* x, mx_dtype type, int64_t tokens, int64_t heads, int64_t dim, int64_t ld_x_token,
                    int64_t ld_x_head, const int32_t* positions, const float* table, int64_t max_pos, int rot_dim,
                    int interleaved, int transpose, void* y, int64_t ld_y_token, int64_t ld_y_head, void* stream)
{
    mx_status st = check_dense(tokens, heads, dim);
    if (st != MX_OK) return st;
    if (!valid_type(type)) return MX_ERR_INVALID_ARG;
    if (ld_x_token < 0 || ld_x_head < 0 || ld_y_token < 0 || ld_y_head < 0) return MX_ERR_INVALID_ARG;
    if (rot_dim < 0 || (rot_dim & 1) || rot_dim > dim) return MX_ERR_INVALID_ARG;
    if (tokens == 0 || heads == 0 || dim == 0) return MX_OK;
    if (!x || !y) return MX_ERR_INVALID_ARG;
    if ((st = check_rope(positions, table, max_pos, rot_dim, dim)) != MX_OK) return st;
    if (!aligned16(x) || !aligned16(y)) return MX_ERR_ALIGNMENT;
    mxk::RopeArgs a{};
    a.bf16 = type == MX_BF16;
    a.dim = (uint32_t)dim;
    a.ldx_t = ld_x_token;
    a.ldx_h = ld_x_head;
    a.ldy_t = ld_y_token;
    a.ldy_h = ld_y_head;
    a.r = rope_of(positions, table, max_pos, rot_dim, interleaved, transpose);
    const int64_t size = a.bf16 ? 2 : 4;
    const int64_t some_heads = std::min(heads, kMaxRopeElems / dim), some_tokens = std::min(tokens, kMaxRopeElems / (some_heads * dim));
    for (int64_t t = 0; t < tokens; t += some_tokens) {
        for (int64_t h = 0; h < heads; h += some_heads) {
            a.x = static_cast<const uint8_t*>(x) + (t * ld_x_token + h * ld_x_head) * size;
            a.y = static_cast<uint8_t*>(y) + (t * ld_y_token + h * ld_y_head) * size;
            a.tokens = (uint32_t)std::min(some_tokens, tokens - t);
            a.heads = (uint32_t)std::min(some_heads, heads - h);
            a.r.positions = rot_dim ? positions + t : nullptr;
            if (mxk::launch_rope(a, static_cast<hipStream_t>(stream)) != hipSuccess) return MX_ERR_HIP;
        }
    }
    return MX_OK;
}

mx_status mxkv_write(const mxkv_cache* cache, const void* k, const void* v, mx_dtype type, int64_t tokens,
                     int64_t ld_k_token, int64_t ld_k_head, int64_t ld_v_token, int64_t ld_v_head,
                     const int32_t* slots, const int32_t* positions, const float* table, int64_t max_pos,
                     int rot_dim, int interleaved, void* k_hat, void* v_hat, void* stream)
{
    mx_status st = check_cache(cache);
    if (st != MX_OK) return st;
    if ((st = check_dense(tokens, cache->heads, cache->dim)) != MX_OK) return st;
    if (!valid_type(type)) return MX_ERR_INVALID_ARG;
    if (ld_k_token < 0 || ld_k_head < 0 || ld_v_token < 0 || ld_v_head < 0) return MX_ERR_INVALID_ARG;
    if ((k_hat == nullptr) != (v_hat == nullptr)) return MX_ERR_INVALID_ARG;
    const int rot = table ? rot_dim : 0;
    if (rot_dim < 0 || (rot & 1) || rot > cache->dim) return MX_ERR_INVALID_ARG;
    if (tokens == 0) return MX_OK;
    if (!k || !v || !slots) return MX_ERR_INVALID_ARG;
    if ((st = check_cache_memory(cache)) != MX_OK) return st;
    if ((st = check_rope(positions, table, max_pos, rot, cache->dim)) != MX_OK) return st;
    if (!aligned16(k) || !aligned16(v) || !aligned4(slots) || (k_hat && (!aligned16(k_hat) || !aligned16(v_hat))))
        return MX_ERR_ALIGNMENT;
    mxk::KvWriteArgs a{};
    a.c = pool_of(cache);
    a.x[0] = k;
    a.x[1] = v;
    a.bf16 = type == MX_BF16;
    a.tokens = (uint32_t)tokens;
    a.ld_t[0] = ld_k_token;
    a.ld_t[1] = ld_v_token;
    a.ld_h[0] = ld_k_head;
    a.ld_h[1] = ld_v_head;
    a.slots = slots;
    a.r = rope_of(positions, table, max_pos, rot, interleaved, 0);
    a.hat[0] = k_hat;
    a.hat[1] = v_hat;
    return mxk::launch_kv_write(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MX_OK : MX_ERR_HIP;
}

mx_status mxkv_read(const mxkv_cache* cache, const int32_t* slots, int64_t tokens, void* k, void* v, mx_dtype type,
                    void* stream)
{
    mx_status st = check_cache(cache);
    if (st != MX_OK) return st;
    if ((st = check_dense(tokens, cache->heads, cache->dim)) != MX_OK) return st;
    if (!valid_type(type)) return MX_ERR_INVALID_ARG;
    if (tokens == 0) return MX_OK;
    if (!k || !v || !slots) return MX_ERR_INVALID_ARG;
    if ((st = check_cache_memory(cache)) != MX_OK) return st;
    if (!aligned16(k) || !aligned16(v) || !aligned4(slots)) return MX_ERR_ALIGNMENT;
    mxk::KvReadArgs a{};
    a.c = pool_of(cache);
    a.slots = slots;
    a.tokens = (uint32_t)tokens;
    a.y[0] = k;
    a.y[1] = v;
    a.bf16 = type == MX_BF16;
    return mxk::launch_kv_read(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MX_OK : MX_ERR_HIP;
}

static mx_status attention_sizes(const mxkv_cache* cache, int64_t batch, int64_t new_tokens, int64_t q_heads,
                                 int64_t max_pages, mxk::KvAttnArgs* a)
{
    const mx_status st = check_cache(cache);
    if (st != MX_OK) return st;
    if (batch < 0 || new_tokens < 0 || q_heads < 0 || q_heads % cache->heads != 0 || max_pages < 0) return MX_ERR_INVALID_ARG;
    if (!within(max_pages, cache->page_size, INT32_MAX)) return MX_ERR_INVALID_ARG;
    if (!within(batch, new_tokens, kMaxRows) || !within(batch * new_tokens, q_heads, kMaxRows - 1) || batch > 65535)
        return MX_ERR_UNSUPPORTED;
    a->c = pool_of(cache);
    a->batch = (uint32_t)batch;
    a->nt = (uint32_t)new_tokens;
    a->q_heads = (uint32_t)q_heads;
    a->max_pages = (uint32_t)max_pages;
    if (batch > 0 && new_tokens > 0 && q_heads > 0 && !mxk::kv_attention_fits(*a)) return MX_ERR_UNSUPPORTED;
    return MX_OK;
}

size_t mxkv_attention_workspace_size(const mxkv_cache* cache, int64_t batch, int64_t new_tokens, int64_t q_heads,
                                     int64_t max_pages)
{
    mxk::KvAttnArgs a{};
    if (attention_sizes(cache, batch, new_tokens, q_heads, max_pages, &a) != MX_OK) return 0;
    if (batch == 0 || new_tokens == 0 || q_heads == 0) return 0;
    return mxk::kv_attention_work_bytes(a);
}

mx_status mxkv_attention(const mxkv_cache* cache, const void* q, int64_t batch, int64_t new_tokens, int64_t q_heads,
                         int64_t ld_q_batch, int64_t ld_q_token, int64_t ld_q_head, const int32_t* block_table,
                         int64_t max_pages, int64_t ld_table, const int32_t* lens, const int32_t* n_new,
                         const uint8_t* mask, int64_t ld_mask_batch, int64_t ld_mask_row, float softmax_scale,
                         void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream)
{
    mxk::KvAttnArgs a{};
    mx_status st = attention_sizes(cache, batch, new_tokens, q_heads, max_pages, &a);
    if (st != MX_OK) return st;
    if (ld_q_batch < 0 || ld_q_token < 0 || ld_q_head < 0 || ld_table < 0 || !std::isfinite(softmax_scale))
        return MX_ERR_INVALID_ARG;
    if (mask && (ld_mask_batch < 0 || ld_mask_row < 0)) return MX_ERR_INVALID_ARG;
    if (batch == 0 || new_tokens == 0 || q_heads == 0) return MX_OK;
    if (!q || !lens || !out || (max_pages > 0 && !block_table)) return MX_ERR_INVALID_ARG;
    if ((st = check_cache_memory(cache)) != MX_OK) return st;
    const size_t need = mxk::kv_attention_work_bytes(a);
    if (need && (!workspace || workspace_bytes < need)) return MX_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(lse) || (need && !aligned16(workspace))) return MX_ERR_ALIGNMENT;
    if (!aligned4(lens) || !aligned4(n_new) || !aligned4(block_table)) return MX_ERR_ALIGNMENT;
    a.q = static_cast<const uint16_t*>(q);
    a.ldq_b = ld_q_batch;
    a.ldq_t = ld_q_token;
    a.ldq_h = ld_q_head;
    a.table = block_table;
    a.ld_table = ld_table;
    a.lens = lens;
    a.n_new = n_new;
    a.mask = mask;
    a.ldm_b = ld_mask_batch;
    a.ldm_r = ld_mask_row;
    a.scale = softmax_scale;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.work = workspace;
    return mxk::launch_kv_attention(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MX_OK : MX_ERR_HIP;
}

}  // extern "C"
