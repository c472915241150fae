/*
 * mx_kv.h -- the microscaled key/value cache of libmx: rotary positions, quantized write and
 * read of the cache, and the attention of new tokens over it, on AMD MI355X (gfx950).
 *
 * The cache holds the block formats of mx.h: blocks of `block` consecutive elements of one
 * head's key or value share a scale byte (E4M3, UE5M3 or E8M0), the elements are E2M1 codes
 * (two per byte, the even element in the low nibble) or E4M3 bytes, and codes and scales are
 * those that mx_quantize / mx_quantize_fp8 give for the same blocks, bit for bit.
 *
 * Layout.  A cache is a pool of num_pages pages of page_size tokens:
 *   codes : num_pages x heads x page_size x (dim/2 bytes for MXKV_FP4, dim for MXKV_FP8)
 *   scales: num_pages x heads x page_size x dim/block bytes
 * for keys and for values, all contiguous.  Slot s is place s % page_size of page
 * s / page_size.  A sequence's token j lives in place j % page_size of the page that entry
 * j / page_size of its block table row names.
 *
 * Conventions are those of mx.h: device pointers owned by the caller, no allocation, no
 * synchronization, arguments validated on the host before any launch, empty calls return MX_OK
 * and launch nothing.  Dense tensors, cache tensors, tables and workspaces must be 16-byte
 * aligned (MX_ERR_ALIGNMENT otherwise); arrays of int32 and masks need the alignment of their
 * elements only.  The mxkv_cache itself is host memory, read during the call.
 * Numbers that only the device knows are made safe there: slots outside the pool are passed
 * over, positions outside the table take its first or last row, a block table entry that
 * names no page of the pool holds no tokens, and lengths are cut to what the block table holds.
 */
#ifndef MX_KV_H
#define MX_KV_H

#include "mx.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MXKV_FP4 = 0, MXKV_FP8 = 1 } mxkv_element; /* E2M1 codes / E4M3 bytes */

typedef struct {
    uint8_t* k_codes;
    uint8_t* k_scales;
    uint8_t* v_codes;
    uint8_t* v_scales;
    int64_t num_pages;
    int32_t heads;     /* key/value heads */
    int32_t page_size; /* tokens of a page, >= 1 */
    int32_t dim;       /* elements of a head, a multiple of block, <= 512 */
    int32_t block;     /* 16, 32, 64, 128 or 256 */
    mxkv_element element;
    mx_scale_fmt fmt;
    float k_scale;     /* per-tensor scales g of keys and of values (1.0 for none) */
    float v_scale;
} mxkv_cache;

/* How frequencies are stretched for contexts longer than the trained one. */
typedef enum {
    MXKV_SCALING_NONE = 0,
    MXKV_SCALING_LINEAR = 1, /* every frequency divided by factor */
    MXKV_SCALING_BASE = 2,   /* base multiplied by factor^(R / (R - 2)) */
    MXKV_SCALING_PARTS = 3   /* frequency f divided by factor where it makes few turns in
                                original_len positions: with t = original_len f / 2 pi and
                                w = clamp((t - low) / (high - low), 0, 1) it becomes
                                f w + f / factor (1 - w) */
} mxkv_scaling;

/*
 * mxkv_rope_table -- cos | sin of position * frequency: max_pos rows of rot_dim fp32, first the
 * rot_dim / 2 cosines, then the sines.  Frequency i is base^(-2 i / rot_dim), stretched as
 * `scaling` says; `magnitude` multiplies every entry (1.0 for a plain rotation).  Angles,
 * sines and cosines are formed in fp64 and rounded once.
 * Errors: MX_ERR_INVALID_ARG for a negative size, an odd or negative rot_dim, base <= 0,
 * factor <= 0, an unknown scaling, PARTS without original_len > 0 and high > low, BASE with
 * rot_dim <= 2, a non-finite argument or a null table; MX_ERR_UNSUPPORTED for
 * rot_dim > 512 or max_pos * rot_dim / 2 >= 2^31; MX_ERR_ALIGNMENT.
 */
mx_status mxkv_rope_table(float* table, int64_t max_pos, int rot_dim, double base, mxkv_scaling scaling,
                          double factor, double original_len, double low, double high, double magnitude,
                          void* stream);

/*
 * mxkv_rope -- rotary positions.  For every token and head the first rot_dim elements are
 * taken in pairs (a, b) = elements (i, i + rot_dim / 2), or (2 i, 2 i + 1) if `interleaved`,
 * and become (a c - b s, b c + a s) with c, s the table's entries i of the token's position;
 * with `transpose` s is negated, which is the gradient: dx from dy.  The other elements are
 * copied.  Products and sums are single fp32 operations, each rounded (no fused
 * multiply-add), and the result is rounded once to x's type, so that quantizing y gives the same
 * codes on every path.
 *  x, y : tokens x heads x dim, element type `type`, unit stride along dim; ld_*_token and
 *         ld_*_head are strides in elements (>= 0 for x; y's rows must not overlap).  y may
 *         be x itself (same strides).
 *  positions: tokens int32.
 * Errors: MX_ERR_INVALID_ARG for null pointers, negative sizes or strides, rot_dim odd,
 * negative or above dim, max_pos < 1, an unknown type; MX_ERR_UNSUPPORTED for dim > 512
 * or tokens * heads * dim >= 2^32; MX_ERR_ALIGNMENT.
 */
mx_status mxkv_rope(const void* x, mx_dtype type, int64_t tokens, int64_t heads, int64_t dim, int64_t ld_x_token,
                    int64_t ld_x_head, const int32_t* positions, const float* table, int64_t max_pos, int rot_dim,
                    int interleaved, int transpose, void* y, int64_t ld_y_token, int64_t ld_y_head, void* stream);

/*
 * mxkv_write -- quantize the keys and values of `tokens` tokens into their slots.  With a
 * table (not NULL) the keys are rotated first, exactly as mxkv_rope rotates them (rounding to
 * `type` included).
 *  k, v  : tokens x heads x dim, strides in elements as for mxkv_rope; finite, as for mx_quantize (what a slot
 *          holds that was written from other numbers is unspecified).
 *  slots : tokens int32; a slot outside the pool is passed over (nothing is written for that
 *          token, its k_hat / v_hat rows are written all the same).  What a slot holds that two tokens of one
 *          call share is unspecified: codes and scale bytes of both, mixed.
 *  k_hat, v_hat: optional outputs (both or neither), contiguous tokens x heads x dim of `type`: the values
 *          that the written codes stand for, rounded as mx_dequantize rounds them.
 * Errors: MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED and MX_ERR_ALIGNMENT as above; a cache whose
 * dim % block != 0, block is not listed, page_size < 1, num_pages < 0, a scale that mx_quantize would refuse,
 * or num_pages * page_size >= 2^31 is MX_ERR_INVALID_ARG.
 */
mx_status mxkv_write(const mxkv_cache* cache, const void* k, const void* v, mx_dtype type, int64_t tokens,
                     int64_t ld_k_token, int64_t ld_k_head, int64_t ld_v_token, int64_t ld_v_head,
                     const int32_t* slots, const int32_t* positions, const float* table, int64_t max_pos,
                     int rot_dim, int interleaved, void* k_hat, void* v_hat, void* stream);

/*
 * mxkv_read -- keys and values of `tokens` slots as dense contiguous tensors tokens x heads x dim
 * of `type`: e * s * g rounded as mx_dequantize rounds it.  A slot outside the pool gives
 * zeros.  Errors as for mxkv_write.
 */
mx_status mxkv_read(const mxkv_cache* cache, const int32_t* slots, int64_t tokens, void* k, void* v, mx_dtype type,
                    void* stream);

/*
 * mxkv_attention -- attention of new tokens over the cache.  Every sequence b has lens[b]
 * cached tokens and, after them, n_new[b] new ones (new_tokens for all where n_new is NULL), whose
 * keys and values are in the cache already, at token numbers lens[b] ... lens[b] + n_new[b] - 1.
 * New token i of a sequence sees all its cached tokens, and new token j where
 * mask[b][i][j] is not 0 -- a tree of drafted tokens: j an ancestor of i or i itself --
 * or, where mask is NULL, every j <= i.  For every query head h, with key/value head
 * h / (q_heads / heads):
 *     out = sum_j p_j v_j / sum_j p_j,   p_j = exp(softmax_scale q . k_j - max),
 * and lse = log sum_j exp(softmax_scale q . k_j).  A token that sees nothing, and a token
 * i >= n_new[b], gives out = 0 and lse = -inf.  Slots past a sequence's tokens are not used,
 * whatever they hold, and a token that does not see new token j is free of what slot j holds, NaN bytes
 * and values past bf16's range among it.  In a token that is seen, a NaN byte (never written by mxkv_write) of a code or an E8M0 scale
 * gives NaN; one of an E4M3 or UE5M3 scale gives NaN or the value of the bits.
 *  q     : batch x new_tokens x q_heads x dim bf16, unit stride along dim, other strides given.
 *  block_table: batch rows of max_pages int32, row stride ld_table.
 *  lens, n_new: batch int32 each.
 *  mask  : bytes, batch x new_tokens x new_tokens, unit stride along the last; ld_mask_batch may
 *          be 0 (one mask for all sequences).
 *  out   : bf16, contiguous batch x new_tokens x q_heads x dim; lse: optional fp32, batch x
 *          new_tokens x q_heads.
 *  workspace: mxkv_attention_workspace_size(...) bytes (contents unspecified before and after).
 * Scores, the p_j and sums are fp32 (the product with the values keeps each p_j to 2^-16 of itself), and the
 * result is rounded once, to bf16.  The order of sums is fixed by the sizes and lengths: repeated calls give the
 * same bits.
 * Errors: MX_ERR_INVALID_ARG for null pointers, negative sizes or strides, q_heads not a
 * multiple of heads, a softmax_scale that is not finite, a missing or short workspace;
 * MX_ERR_UNSUPPORTED for batch * new_tokens * q_heads >= 2^24, batch > 65535, or a block table so
 * wide that batch * heads * tiles * (max_pages * page_size / 128 + 8) >= 2^31 with tiles =
 * ceil(new_tokens * q_heads / heads / 16);
 * MX_ERR_ALIGNMENT.
 */
size_t mxkv_attention_workspace_size(const mxkv_cache* cache, int64_t batch, int64_t new_tokens, int64_t q_heads,
                                     int64_t max_pages);
mx_status mxkv_attention(const mxkv_cache* cache, const void* q, int64_t batch, int64_t new_tokens, int64_t q_heads,
                         int64_t ld_q_batch, int64_t ld_q_token, int64_t ld_q_head, const int32_t* block_table,
                         int64_t max_pages, int64_t ld_table, const int32_t* lens, const int32_t* n_new,
                         const uint8_t* mask, int64_t ld_mask_batch, int64_t ld_mask_row, float softmax_scale,
                         void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MX_KV_H */
