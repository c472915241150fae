// mx_kv_attn.h -- the matrix-core attention kernel over the quantized cache, instantiated for
// one head size per translation unit.  Private to libmx.
//
// One workgroup of four waves takes 16 NQ rows (new token, query head) that share a key/value
// head, and a run of the sequence's tokens; a wave takes 32 tokens at a time, which asynchronous loads
// bring into its part of LDS two tiles ahead.  Both products run
// transposed on bf16 MFMA 16x16x32,
//     S^T = K Q^T  (tokens x rows),    O^T += V^T P^T  (elements x rows),
// and every operand is in the lane that needs it as read or as computed, with nothing
// exchanged between lanes:
//  * lane 16 g + n reads elements g D/4 ... of its token's key, a run of D/4 consecutive codes: the
//    contraction order of a product is free as long as both sides share it, so MFMA step st takes
//    elements g D/4 + 8 st + 0..7 of Q and K in lane group g;
//  * the scores of S^T come out with row n and tokens 4 g + r in lane 16 g + n, which is the
//    layout that the second product wants of P^T, for the tokens that its group's lanes then
//    have to hold of V;
//  * the same lane reads elements n D/16 ... of those tokens' values, so that MFMA j makes elements
//    n D/16 + j for all n.  The converter gives a token's element pair; a byte permute of two
//    tokens' pairs makes the token pairs that the product contracts.
// Matrix row m of half s is token 16 s + 4 (m % 4) + m / 4, which gives both products the same tokens.
//
// The running maximum is raised only when a score passes it by 8 (in powers of two): p then stays
// below 2^8, sums stay far from overflow, and the accumulators are rarely rescaled.  Sums, maxima and scores
// are fp32.  The product with the values takes bf16, in which codes times scales are exact and p is not: p goes
// in as two parts, its nearest bf16 and the nearest bf16 of the rest, which leaves 2^-16 of it.  One part, 2^-8
// of a term, was as large an error as the rounding of the result, which is the only one to bf16 now.  The second
// products are free where memory is waited for (32 sequences up to 8192: 41.9 and 42.4 us) and cost the
// many-row cases 13 to 22% (8 trees over FP8: 68.2 and 77.7 us; 512 rows of a head over 131072 tokens: 390 and 462).
//
// What bounds it.  Few rows (decode): HBM, 5.4 TB/s of FP4 and 5.9 of FP8 per added token (32 sequences of 8192
// and of 16384: 71.8 and 124.5 us, 115.3 and 209.5), besides some 20 us of a call: two launches, loads that wait
// for each other before the first tile and after the last, workgroups that end at different times.  Many rows:
// issue.  Over FP4 a tile of 32 tokens x 32 rows x 128 elements takes 48 MFMAs (768 cycles) and 277 other vector
// instructions (64 to decode, 32 to pair tokens, 16 exponentials, 48 to split p), for two waves of a SIMD: vector
// units 54%, matrix units 37% of the cycles, 0.60 PFLOP/s at a clock that falls to 2.1 GHz.  What was tried there
// and measured alike: decoding a pair of elements between the products of the last, table entries read a tile
// ahead, all LDS reads before the first use, two or four waves on one tile behind a barrier, Q in LDS with three
// waves of a SIMD.  64 rows of a wave spill: 2.6 times the time.
#pragma once

#include <type_traits>

#include "mx_device.h"
#include "mx_kv_internal.h"

namespace mxk {
namespace kv {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float NO_MAX = -1e30f;  // the maximum of a row that has seen no key
constexpr float RAISE = 8.0f;
constexpr uint32_t STEP = 128;    // tokens of a workgroup's step: four waves of 32

// What no kernel of the call writes and every lane reads alike comes through the scalar cache, whose
// loads are counted apart from the tiles' own.
typedef const __attribute__((address_space(4))) int32_t* ScalarInts;
__device__ __forceinline__ int32_t read_uniform(const int32_t* p, uint64_t i)
{
    return reinterpret_cast<ScalarInts>(reinterpret_cast<uintptr_t>(p))[i];
}

struct Seq {
    uint32_t cached, held;  // tokens before the new ones; all tokens
    uint32_t fresh;         // new tokens
};

// A value that is the same in all lanes, as the compiler is to know
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// A sequence's lengths, cut to what the call and the block table hold
__device__ __forceinline__ Seq seq_of(const KvAttnArgs& a, uint32_t b)
{
    const uint32_t cap = a.max_pages * a.c.page;
    const int32_t l = a.lens[b], n = a.n_new ? a.n_new[b] : (int32_t)a.nt;
    Seq s;
    s.cached = l < 0 ? 0u : ((uint32_t)l < cap ? (uint32_t)l : cap);
    s.fresh = n < 0 ? 0u : ((uint32_t)n < a.nt ? (uint32_t)n : a.nt);
    s.held = s.cached + s.fresh < cap ? s.cached + s.fresh : cap;
    return s;
}

__device__ __forceinline__ Seq seq_uniform(const KvAttnArgs& a, uint32_t b)
{
    b = uniform(b);
    const uint32_t cap = a.max_pages * a.c.page;
    const int32_t l = read_uniform(a.lens, b), n = a.n_new ? read_uniform(a.n_new, b) : (int32_t)a.nt;
    Seq s;
    s.cached = l < 0 ? 0u : ((uint32_t)l < cap ? (uint32_t)l : cap);
    s.fresh = n < 0 ? 0u : ((uint32_t)n < a.nt ? (uint32_t)n : a.nt);
    s.held = s.cached + s.fresh < cap ? s.cached + s.fresh : cap;
    return s;
}

// How a call is cut into pieces of equal length.  A segment is as many row tiles of a sequence, in the order
// (key/value head, tile), as a team has workgroups: a tile each, over the same tokens at the same time, so that
// what one of them reads the others find in L2.  A call's work is the list of all units: sequences, for each
// the segments, for each `begin` units that stand for what beginning
// and ending a segment costs, and the steps over the sequence's tokens (one at least, so that every
// output is written).  Team w takes units start(w) ... start(w + 1) - 1 of
// that list, whatever segments they fall in; a segment that lies in one team is finished
// there, the pieces of a cut one go to the workspace and are joined in order.  The workspace begins with
// the number of all units and of those before each sequence, which workgroup 0 writes for the
// kernel that joins.
struct AttnPlan {
    FastDiv page_div, group_div;
    uint32_t teams;       // of `team` workgroups each
    uint32_t team;
    uint32_t row_tiles;   // row tiles of a key/value head
    uint32_t group;       // query heads of a key/value head
    uint64_t most;        // units that the block table has room for
    uint32_t block_shift, scale_shift;  // log2 of the block, of a row's scale bytes
    uint32_t begin;       // steps that take as long as beginning and ending a segment
    float c;              // |softmax scale * key scale| * log2 e
    uint32_t flip;        // 0x80008000 where that is negative: queries change sign
    uint32_t s_bits, s_sign;  // E4M3 / UE5M3 scale bytes: magnitude and sign bits,
    float s_mul;              // and the factor that moves their exponent to fp32's
};

// bytes of the counts that the workspace begins with
__host__ __device__ constexpr uint64_t meta_bytes(uint32_t batch) { return ((uint64_t)(batch + 1) * 4 + 255) & ~uint64_t(255); }

struct Cut {
    uint32_t quot, rem;  // units = quot * teams + rem: the first rem teams take one more
    __device__ __forceinline__ uint32_t start(uint32_t w) const { return w * quot + (w < rem ? w : rem); }
    __device__ __forceinline__ uint32_t owner(uint32_t p) const
    {
        const uint32_t long_ones = rem * (quot + 1);
        return p < long_ones ? p / (quot + 1) : rem + (p - long_ones) / quot;
    }
};

// Teams that a list of `units` is shared by: all, unless that leaves them fewer than 3 units and every CU has a
// workgroup without them.  A piece costs its beginning, its end and its part of the join: one head's 8 rows over
// 131072 FP4 tokens took 13 + 12 us by 342 workgroups and 15 + 22 by 768; 8 heads over 2047 are best off with a
// unit each (6.6 + 5.3 us, with 3 units 8.4 + 4.8).
__device__ __forceinline__ uint32_t teams_for(const AttnPlan& p, uint32_t units)
{
    const uint32_t few = 256 / p.team, n = units / 3 > few ? units / 3 : few;
    return n < p.teams ? n : p.teams;
}

// A sequence's part of the list: the row tiles that its new tokens fill, for each head.
struct Part {
    uint32_t tiles;  // row tiles of a head
    uint32_t steps;  // of a segment
    uint32_t units;
};

__device__ __forceinline__ Part part_of(const AttnPlan& p, const Seq& s, uint32_t heads, uint32_t tile_rows)
{
    Part t;
    const uint32_t n = (s.held + STEP - 1) / STEP;
    t.tiles = (s.fresh * p.group + tile_rows - 1) / tile_rows;
    t.steps = n ? n : 1u;
    t.units = (heads * t.tiles + p.team - 1) / p.team * (t.steps + p.begin);
    return t;
}

// The rows of tokens past a sequence's n_new: 0, and no score.
__device__ __forceinline__ void fill_rest(const KvAttnArgs& a)
{
    for (uint32_t k = blockIdx.x; k < a.batch * a.nt; k += gridDim.x) {
        const uint32_t b = k / a.nt;
        const int32_t n = read_uniform(a.n_new, b);
        if (n > 0 && k - b * a.nt < (uint32_t)n) continue;
        u32x4* out = reinterpret_cast<u32x4*>(a.out + (uint64_t)k * a.q_heads * a.c.dim);
        for (uint32_t i = threadIdx.x; i < a.q_heads * a.c.dim / 8; i += 256) out[i] = u32x4{0u, 0u, 0u, 0u};
        if (a.lse)
            for (uint32_t h = threadIdx.x; h < a.q_heads; h += 256) a.lse[(uint64_t)k * a.q_heads + h] = -INFINITY;
    }
}

// Inclusive sum over the wave's lanes
__device__ __forceinline__ uint32_t wave_scan(uint32_t v)
{
    const uint32_t lane = threadIdx.x & 63;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)v, off);
        if (lane >= (uint32_t)off) v += o;
    }
    return v;
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, uint32_t lane)
{
    return (uint32_t)__builtin_amdgcn_readlane((int)v, (int)lane);
}

// Units up to and with sequence b0 + lane, `before` of them before b0
__device__ __forceinline__ uint32_t scan_64(const KvAttnArgs& a, const AttnPlan& p, uint32_t b0, uint32_t before, uint32_t tile_rows)
{
    const uint32_t b = b0 + (threadIdx.x & 63);
    const uint32_t n = b < a.batch ? part_of(p, seq_of(a, b), a.c.heads, tile_rows).units : 0u;
    return before + wave_scan(n);
}

// A piece in the workspace: 16 NQ x D fp32 sums, lane by lane as the accumulators hold them
// (for each 16 rows D/16 x 64 lanes x 4), then 16 NQ maxima and 16 NQ sums of p.
template <int D, int NQ>
struct Piece {
    static constexpr uint32_t SUMS = 16u * NQ * D;
    static constexpr uint32_t FLOATS = SUMS + 32u * NQ;
};

__device__ __forceinline__ float* pieces_of(const KvAttnArgs& a)
{
    return reinterpret_cast<float*>(static_cast<uint8_t*>(a.work) + meta_bytes(a.batch));
}

// sum and maximum over the four lanes n, 16 + n, 32 + n, 48 + n
__device__ __forceinline__ float over_groups_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float over_groups_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Finished rows: out = sums / l for 16 rows, lane 16 g + n having row n, elements
// (4 g + r) D/16 + j0 + 0..JW-1
template <int D, int JW>
__device__ __forceinline__ void store_rows(const KvAttnArgs& a, const AttnPlan& p, const Seq& s, uint32_t b, uint32_t hk,
                                           uint32_t row0, uint32_t j0, const f32x4 (&o)[JW], float m, float l)
{
    const uint32_t lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const uint32_t row = row0 + n;
    const uint32_t i = p.group_div.div(row);
    if (i >= s.fresh) return;
    const uint64_t at = ((uint64_t)b * a.nt + i) * a.q_heads + hk * p.group + (row - i * p.group);
    const bool some = l != 0.f;  // NaN stays NaN
    const float inv = some ? a.c.g[1] / l : 0.f;
    uint16_t* out = a.out + at * D + g * (D / 4) + j0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        uint32_t w[JW / 2];
#pragma unroll
        for (int j = 0; j < JW / 2; ++j)
            w[j] = some ? __builtin_bit_cast(uint32_t, bf16x2{(__bf16)(o[2 * j][r] * inv), (__bf16)(o[2 * j + 1][r] * inv)}) : 0u;
        uint32_t* q = reinterpret_cast<uint32_t*>(out + r * (D / 16));
        if constexpr (JW == 2) {
            *q = w[0];
        } else if constexpr (JW == 4) {
            *reinterpret_cast<u32x2*>(q) = u32x2{w[0], w[1]};
        } else {
#pragma unroll
            for (int j = 0; j < JW / 2; j += 4) *reinterpret_cast<u32x4*>(q + j) = u32x4{w[j], w[j + 1], w[j + 2], w[j + 3]};
        }
    }
    if (a.lse && g == 0 && j0 == 0) a.lse[at] = some ? m * LN2 + logf(l) : -INFINITY;
}

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

// The same value, which the compiler takes for a new one: what is computed from it stays where it is
// used, in place of a register held for it throughout the loop.
__device__ __forceinline__ uint32_t fresh(uint32_t v)
{
    asm volatile("" : "+v"(v));
    return v;
}

template <int N>
__device__ __forceinline__ void wait_loads()  // all but the N newest vector loads have arrived
{
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
    asm volatile("" ::: "memory");
}

// A wave's tile of 32 tokens in LDS: two halves of 16 rows of key codes, the same of value codes, then
// scale bytes.  It is brought there by asynchronous loads, several tiles ahead of the one that is
// worked on; only the wave that loaded a tile reads it, so that its own load counter is all the
// synchronization there is.
//  * Codes come in pieces of 16 bytes: piece c of row r stands in place c ^ swizzle(r) of the row, which
//    puts the pieces that 16 lanes read from their 16 rows at once into 16 distinct bank groups.
//  * Scales: (key half 0, key half 1, value half 0, value half 1) x 16 rows x bytes of a row.
// SPREAD: 0 where pages are whole numbers of 16 tokens, so that a half's rows are neighbours; 1 where rows are
// found one by one; 2 where moreover a row has one or two scale bytes, which are loaded one by one, four LDS
// bytes each.  200 rows x 8000 tokens of 128 FP8 elements under 16-element scales: 88 us with pages of 64, with
// pages of 100 98 us by words (byte by byte they took 1.7 times as long).
template <bool FP8, int D, int BS, int SPREAD>
struct Stage {
    static constexpr int RB = FP8 ? D : D / 2;        // bytes of a row
    static constexpr int CPR = RB / 16;               // its 16-byte pieces
    static constexpr int CODE_LOADS = RB / 32;        // loads of 64 pieces, for 32 rows
    static constexpr int MOST_SCALES = D / BS;        // scale bytes of a row at most
    static constexpr int SCALE_LOADS = SPREAD == 2 ? 2 : (MOST_SCALES < 4 ? 1 : MOST_SCALES / 4);
    static constexpr int LOADS = 2 * CODE_LOADS + SCALE_LOADS;
    static constexpr int VALUES = 32 * RB, SCALES = 64 * RB;  // offsets
    static constexpr int BYTES = SCALES + 256 * SCALE_LOADS;

    static __device__ __forceinline__ uint32_t swizzle(uint32_t row)
    {
        return (CPR >= 16 ? row : row / (16 / CPR)) & (CPR - 1);
    }
    static __device__ __forceinline__ uint32_t piece_at(uint32_t row, uint32_t c) { return (row * CPR + (c ^ swizzle(row))) * 16; }

    // The tile's rows row0 ... + 15 and row1 ... + 15, the same in all lanes: the codes' addresses are a
    // scalar base and an offset that a lane keeps.
    static __device__ __forceinline__ void issue_halves(const KvPool& c, const AttnPlan& p, uint8_t* at, uint64_t row0, uint64_t row1)
    {
        constexpr int PER_HALF = CODE_LOADS / 2;  // loads
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
            for (int i = 0; i < CODE_LOADS; ++i) {
                const rsrc_t from = make_rsrc(c.codes[kv] + (i < PER_HALF ? row0 : row1) * RB, 16 * RB);
                const uint32_t slot = 64 * (i % PER_HALF) + (threadIdx.x & 63), row = slot / CPR;
                const uint32_t off = row * RB + ((slot % CPR) ^ swizzle(row)) * 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void*)(at + (kv ? VALUES : 0) + 1024 * i), 16, off, 0, 0, 0);
            }
        }
        const uint32_t lane = fresh(threadIdx.x & 63);
#pragma unroll
        for (int i = 0; i < SCALE_LOADS; ++i) {
            const uint32_t slot = 64 * i + lane, sh = p.scale_shift;
            const uint32_t sel = slot >> (sh + 2), word = slot & ((4u << sh) - 1);  // places past the last one load a word again
            const uint8_t* k0 = c.scales[0] + (row0 << sh);
            const uint8_t* k1 = c.scales[0] + (row1 << sh);
            const uint8_t* v0 = c.scales[1] + (row0 << sh);
            const uint8_t* v1 = c.scales[1] + (row1 << sh);
            const uint8_t* from = (sel & 2 ? (sel & 1 ? v1 : v0) : (sel & 1 ? k1 : k0)) + 4 * word;
            __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)(at + SCALES + 256 * i), 4, 0, 0);
        }
    }

    // row_at(t) gives the pool row of the tile's token t (any lane may ask for any token)
    template <class R>
    static __device__ __forceinline__ void issue(const KvPool& c, const AttnPlan& p, uint8_t* at, R&& row_at)
    {
        const uint32_t lane = fresh(threadIdx.x & 63);
#pragma unroll
        for (int i = 0; i < CODE_LOADS; ++i) {
            const uint32_t slot = 64 * i + lane, row = slot / CPR, piece = (slot % CPR) ^ swizzle(row & 15);
            const uint64_t from = row_at(row) * RB + piece * 16;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv)
                __builtin_amdgcn_global_load_lds((global_void*)(c.codes[kv] + from), (lds_void*)(at + (kv ? VALUES : 0) + 1024 * i), 16, 0, 0);
        }
        const uint32_t sh = p.scale_shift;  // log2 of a row's scale bytes
#pragma unroll
        for (int i = 0; i < SCALE_LOADS; ++i) {
            const uint32_t slot = 64 * i + lane;
            if constexpr (SPREAD == 2) {
                const uint32_t sel = (slot >> sh) & 63;  // places past the last one load a byte again
                const uint8_t* from = (sel & 32 ? c.scales[1] : c.scales[0]) + (row_at(sel & 31) << sh) + (slot & ((1u << sh) - 1));
                __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)(at + SCALES + 256 * i), 1, 0, 0);
            } else if constexpr (SPREAD == 1) {
                const uint32_t sel = (slot >> (sh - 2)) & 63, word = slot & ((1u << (sh - 2)) - 1);  // as there
                const uint8_t* from = (sel & 32 ? c.scales[1] : c.scales[0]) + (row_at(sel & 31) << sh) + 4 * word;
                __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)(at + SCALES + 256 * i), 4, 0, 0);
            } else {
                const uint32_t sel = (slot >> (sh + 2)) & 3, word = slot & ((4u << sh) - 1);
                const uint8_t* from = (sel & 2 ? c.scales[1] : c.scales[0]) + (row_at(16 * (sel & 1)) << sh) + 4 * word;
                __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)(at + SCALES + 256 * i), 4, 0, 0);
            }
        }
    }

    // the key run of row `row` of half h that lane group g takes, RB / 4 bytes
    static __device__ __forceinline__ void key_run(const uint8_t* at, int h, uint32_t row, uint32_t g, uint32_t (&w)[RB / 16])
    {
        at += h * 16 * RB;
        if constexpr (CPR == 2) {
            const u32x2 x = *reinterpret_cast<const u32x2*>(at + piece_at(row, g >> 1) + 8 * (g & 1));
            w[0] = x.x;
            w[1] = x.y;
        } else {
#pragma unroll
            for (int i = 0; i < CPR / 4; ++i) {
                const u32x4 x = *reinterpret_cast<const u32x4*>(at + piece_at(row, g * (CPR / 4) + i));
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * i + j] = x[j];
            }
        }
    }
    // bytes n RB / 16 ... of the value of token 16 h + row
    static constexpr int VW = RB < 64 ? 1 : RB / 64;
    static __device__ __forceinline__ void value_run(const uint8_t* at, int h, uint32_t row, uint32_t n, uint32_t (&w)[VW])
    {
        const uint8_t* q = at + VALUES + h * 16 * RB + piece_at(row, n * (RB / 16) / 16) + (n * (RB / 16)) % 16;
        if constexpr (RB == 32) {
            w[0] = *reinterpret_cast<const uint16_t*>(q);
        } else if constexpr (RB == 64) {
            w[0] = *reinterpret_cast<const uint32_t*>(q);
        } else if constexpr (RB == 128) {
            const u32x2 x = *reinterpret_cast<const u32x2*>(q);
            w[0] = x.x;
            w[1] = x.y;
        } else {
            const u32x4 x = *reinterpret_cast<const u32x4*>(q);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = x[j];
        }
    }
    // scale byte of elements d ... of token t's key (kv 0) or value (kv 1)
    static __device__ __forceinline__ uint32_t scale(const AttnPlan& p, const uint8_t* at, int kv, uint32_t t, uint32_t d)
    {
        const uint32_t i = ((32 * kv + t) << p.scale_shift) + (d >> p.block_shift);
        return at[SCALES + (SPREAD == 2 ? 4 * i : i)];
    }
};

// 8 consecutive codes -> the 8 bf16 of an MFMA operand (exact: at most 8 significant bits)
template <bool FP8, bool POW2>
__device__ __forceinline__ bf16x8 decode_run(const uint32_t* w, float s)
{
    uint32_t d[4];
    if constexpr (POW2 && !FP8) {
        d[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], s, 0));
        d[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], s, 1));
        d[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], s, 2));
        d[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], s, 3));
    } else if constexpr (POW2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            d[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], s, false));
            d[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], s, true));
        }
    } else {
        f32x2 f[4];
        if constexpr (FP8) {
            f[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], 1.0f, false);
            f[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], 1.0f, true);
            f[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[1], 1.0f, false);
            f[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[1], 1.0f, true);
        } else {
            f[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 0);
            f[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 1);
            f[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 2);
            f[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 3);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)(f[i].x * s), (__bf16)(f[i].y * s)});
    }
    return __builtin_bit_cast(bf16x8, u32x4{d[0], d[1], d[2], d[3]});
}

// element pair J (elements 2 J, 2 J + 1) of a value run
template <bool FP8, int J>
__device__ __forceinline__ f32x2 pair_f32(const uint32_t* w)
{
    if constexpr (FP8) return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[J / 2], 1.0f, J % 2 != 0);
    else return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[J / 4], 1.0f, J % 4);
}
template <bool FP8, int J>
__device__ __forceinline__ uint32_t pair_bf16(const uint32_t* w, float s)
{
    if constexpr (FP8) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[J / 2], s, J % 2 != 0));
    else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[J / 4], s, J % 4));
}

// Elements 2 J and on of a value run with scale s, times p, to sums r of o, in rows that see the token
template <bool FP8, int J = 0, int VW, int NJ>
__device__ __forceinline__ void add_run(const uint32_t (&w)[VW], float s, float p, bool sees, f32x4 (&o)[NJ], int r)
{
    const f32x2 e = pair_f32<FP8, J>(w);
    o[2 * J][r] += sees ? e.x * s * p : 0.f;
    o[2 * J + 1][r] += sees ? e.y * s * p : 0.f;
    if constexpr (2 * J + 2 < NJ) add_run<FP8, J + 1>(w, s, p, sees, o, r);
}

// value operands of elements 2 J and 2 J + 1: 8 tokens each
template <bool FP8, bool POW2, int J, int VW>
__device__ __forceinline__ void value_pair(const uint32_t (&v)[8][VW], const float (&vs)[8], bf16x8& a0, bf16x8& a1)
{
    uint32_t d0[4], d1[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if constexpr (POW2) {
            const uint32_t x = pair_bf16<FP8, J>(v[2 * t], vs[2 * t]), y = pair_bf16<FP8, J>(v[2 * t + 1], vs[2 * t + 1]);
            d0[t] = __builtin_amdgcn_perm(y, x, 0x05040100u);
            d1[t] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        } else {
            const f32x2 x = pair_f32<FP8, J>(v[2 * t]), y = pair_f32<FP8, J>(v[2 * t + 1]);
            d0[t] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)(x.x * vs[2 * t]), (__bf16)(y.x * vs[2 * t + 1])});
            d1[t] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)(x.y * vs[2 * t]), (__bf16)(y.y * vs[2 * t + 1])});
        }
    }
    a0 = __builtin_bit_cast(bf16x8, u32x4{d0[0], d0[1], d0[2], d0[3]});
    a1 = __builtin_bit_cast(bf16x8, u32x4{d1[0], d1[1], d1[2], d1[3]});
}

// Whether a run of codes may stand for a value that is not finite in bf16: a NaN byte, or a power of two as its
// scale under which the format's largest magnitude, 6 or 448, reaches 2^128 -- bytes 253 (2^126) or 247 (2^120) and
// up, 255 (NaN) among them.  Under E4M3 and UE5M3 scales no value passes 2^26.
template <bool FP8, bool POW2, int VW>
__device__ __forceinline__ bool may_be_infinite(const uint32_t (&w)[VW], float s)
{
    bool yes = POW2 && f2u(s) >= (FP8 ? 247u : 253u) << 23;
    if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < VW; ++i) yes |= (((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
    }
    return yes;
}

// The lowest n bits
__device__ __forceinline__ uint32_t low_bits(uint32_t n) { return n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// Masks of up to MASK_BITS new tokens are packed in LDS when a piece begins; longer ones are read byte by
// byte, where a tile needs them.
constexpr uint32_t MASK_BITS = 256;

// Which of the 32 tokens from t0 on new token i sees: bit t for token t0 + t.  `valid` has the tokens
// that exist; `packed` is token i's mask row, or null: then of the new tokens only bits 16 s + 4 r + g are
// looked up, those that lane group g holds.
__device__ __forceinline__ uint32_t seen_bits(const KvAttnArgs& a, const Seq& s, uint32_t b, uint32_t i, uint32_t t0,
                                              uint32_t valid, uint32_t g, const uint32_t* packed)
{
    if (!a.mask) {
        const uint32_t end = i < s.fresh ? s.cached + i + 1 : 0u;
        return valid & low_bits(end > t0 ? end - t0 : 0u);
    }
    uint32_t bits = low_bits(s.cached > t0 ? s.cached - t0 : 0u);
    if (packed) {
        if (s.cached >= t0) {
            const uint32_t n = s.cached - t0;
            bits |= n < 32 ? packed[0] << n : 0u;
        } else {
            const uint32_t k = t0 - s.cached, w = k >> 5;
            const uint32_t lo = packed[w], hi = w + 1 < MASK_BITS / 32 ? packed[w + 1] : 0u;
            bits |= (uint32_t)((((uint64_t)hi << 32) | lo) >> (k & 31));
        }
    } else {
        const uint8_t* row = a.mask + b * a.ldm_b + (i < s.fresh ? i : 0u) * a.ldm_r;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t t = 16 * (k >> 2) + 4 * (k & 3) + g, j = t0 + t;
            const bool is_new = j >= s.cached && j < s.held;
            const uint32_t x = row[is_new ? j - s.cached : 0u];  // a byte of the row in any case
            bits |= (is_new && x != 0 ? 1u : 0u) << t;
        }
    }
    return i < s.fresh ? bits & valid : 0u;
}

template <bool POW2>
__device__ __forceinline__ float scale_f32(const AttnPlan& p, uint32_t byte)
{
    if constexpr (POW2) return u2f(byte << 23);  // the converter reads the exponent only
    else return u2f(((byte & p.s_bits) << 20) | ((byte & p.s_sign) << 24)) * p.s_mul;
}

// A scale as a factor: byte 0xFF, whose exponent the converters take for NaN, is NaN
template <bool POW2>
__device__ __forceinline__ float nan_scale(float s)
{
    return POW2 && s == INFINITY ? s - s : s;
}

// Workgroups of a CU (waves of a SIMD) that registers and LDS leave room for, and tiles that a wave's
// ring in LDS holds: 164 registers for 16 rows of 128 elements, 237 to 246 for 32.
constexpr int LDS_BYTES = 160 * 1024;
constexpr int least(int a, int b) { return a < b ? a : b; }
template <bool FP8, int D, int BS, int NQ, int SPREAD>
struct Room {
    using ST = Stage<FP8, D, BS, SPREAD>;
    static constexpr int OTHER = 1024 * (NQ < 2 ? 2 : NQ);  // what else the kernel has in LDS
    static constexpr int REGISTERS = NQ * D <= 64 ? 4 : (NQ * D <= 128 ? 3 : 2);
    static constexpr int LDS = LDS_BYTES / (8 * ST::BYTES + OTHER);  // with two tiles of each wave
    static constexpr int GROUPS = LDS < 1 ? 1 : least(LDS, REGISTERS);
    static constexpr int DEPTH = least(3, (LDS_BYTES / GROUPS - OTHER) / (4 * ST::BYTES));
    static constexpr int RING = 4 * DEPTH * ST::BYTES, JOIN = 4 * NQ * D * 64;
    static constexpr int DYNAMIC = RING > JOIN ? RING : JOIN;
    static_assert(GROUPS * (DYNAMIC + OTHER) <= LDS_BYTES);
};

// SPREAD: as for Stage.  The table's entries of a tile's tokens are then read a tile before they are needed and
// ahead of that tile's loads: loads arrive in order, and waiting for an entry must not wait for them.
template <bool FP8, bool POW2, int D, int BS, int NQ, int SPREAD>
__global__ __launch_bounds__(256, (Room<FP8, D, BS, NQ, SPREAD>::GROUPS)) void attn_tile_kernel(KvAttnArgs a, AttnPlan p)
{
    using ST = Stage<FP8, D, BS, SPREAD>;
    constexpr int NJ = D / 16, NS = D / 32, KS = (D / 4) / BS, ROWS = 16 * NQ;
    constexpr int DEPTH = Room<FP8, D, BS, NQ, SPREAD>::DEPTH;
    extern __shared__ __attribute__((aligned(16))) uint8_t ring[];
    __shared__ float wm[4][ROWS], wl[4][ROWS];
    __shared__ uint32_t masks[ROWS][MASK_BITS / 32];
    static_assert(sizeof(wm) + sizeof(wl) + sizeof(masks) <= (Room<FP8, D, BS, NQ, SPREAD>::OTHER));
    const uint32_t lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
    const uint32_t wave = uniform(threadIdx.x >> 6);

    if (a.n_new) fill_rest(a);

    // the list: for up to 64 sequences a lane keeps the end of one sequence's part
    uint32_t* meta = static_cast<uint32_t*>(a.work);
    uint32_t total, ends = 0;
    if (a.batch == 1) {
        total = part_of(p, seq_uniform(a, 0), a.c.heads, ROWS).units;
        if (blockIdx.x == 0 && threadIdx.x == 0) meta[1] = 0;
    } else {
        total = 0;
        for (uint32_t b0 = 0; b0 < a.batch; b0 += 64) {
            const uint32_t before = total;
            ends = scan_64(a, p, b0, before, ROWS);
            total = lane_value(ends, 63);
            if (blockIdx.x == 0 && wave == 0 && b0 + lane + 1 < a.batch) meta[2 + b0 + lane] = ends;
            if (blockIdx.x == 0 && threadIdx.x == 0 && b0 == 0) meta[1] = 0;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) meta[0] = total;
    const uint32_t teams = teams_for(p, total);
    const Cut cut{total / teams, total % teams};
    // Workgroups go to the 8 XCDs in turn: numbered so that those of an XCD, and with them those of a team, are
    // neighbours and find in its L2 what one of them has read: 8 x 16384 FP8 tokens with 192 rows for each of 8
    // heads take 210 us in place of 270, when next to no read of a second row tile is a hit.  Teams of one have
    // nothing to share and keep the turn (64 x up to 4096 FP4 tokens: 45.0 us, as neighbours 46.9).
    const uint32_t xcd = blockIdx.x & 7, each = gridDim.x >> 3, more = gridDim.x & 7;
    const uint32_t group = p.team == 1 ? blockIdx.x : xcd * each + (xcd < more ? xcd : more) + (blockIdx.x >> 3);
    const uint32_t team = group / p.team, member = group - team * p.team;
    uint32_t pos = team < teams ? cut.start(team) : total;
    const uint32_t stop = team < teams ? cut.start(team + 1) : total;

    while (pos < stop) {
        // the sequence that unit `pos` falls in, and the units before it
        uint32_t b = 0, before = 0;
        if (a.batch > 1) {
            uint32_t e = ends, b0 = 0, base = 0;
            if (a.batch > 64) e = scan_64(a, p, 0, 0, ROWS);
            for (;;) {
                const uint64_t past = __ballot(e > pos);
                if (past) {
                    const uint32_t at = (uint32_t)__builtin_ctzll(past);
                    b = b0 + at;
                    before = at ? lane_value(e, at - 1) : base;
                    break;
                }
                base = lane_value(e, 63);
                b0 += 64;
                e = scan_64(a, p, b0, base, ROWS);
            }
        }
        const Seq s = seq_uniform(a, b);
        const Part part = part_of(p, s, a.c.heads, ROWS);
        const uint32_t local = pos - before;
        const uint32_t steps = part.steps, seg = local / (steps + p.begin), unit = local - seg * (steps + p.begin);
        if (unit < p.begin) {
            pos += p.begin - unit;
            if (pos >= stop) break;
        }
        const uint32_t off = unit < p.begin ? 0u : unit - p.begin;
        const uint32_t count = steps - off < stop - pos ? steps - off : stop - pos;
        const uint32_t mine_of = seg * p.team + member;  // the row tile, of those of all heads
        const uint32_t hk = mine_of / part.tiles, row0 = (mine_of - hk * part.tiles) * ROWS;
        if (hk >= a.c.heads) {
            pos += count;
            continue;
        }
        const int32_t* table = a.table + b * a.ld_table;

        // Where a tile's tokens are.  Every row is one of the pool, whatever the tokens: one past the
        // sequence or on no page stands at another row, and its bit of `valid` is 0.
        struct Place {
            uint32_t valid;          // bit t: token t of the tile exists
            uint64_t row[2];         // the halves' first rows
            uint32_t low, high;      // SPREAD: the row of token `lane % 32`
        };
        auto token_of = [&](uint32_t t0) {  // SPREAD
            const uint32_t t = t0 + (lane & 31);
            return t < s.held ? t : s.held - 1;
        };
        auto entry_of = [&](uint32_t t0) -> uint32_t {
            if constexpr (SPREAD) return (uint32_t)table[p.page_div.div(token_of(t0))];
            else return 0u;
        };
        auto find = [&](uint32_t t0, uint32_t entry) {
            Place w{};
            w.valid = low_bits(s.held - t0);
            if constexpr (!SPREAD) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t t1 = t0 + 16 * h < s.held ? t0 + 16 * h : t0;
                    const uint32_t e = p.page_div.div(t1);
                    uint32_t page = (uint32_t)read_uniform(table, e);
                    if (page >= a.c.num_pages) {
                        w.valid &= h ? 0x0000FFFFu : 0xFFFF0000u;
                        page = 0;
                    }
                    w.row[h] = ((uint64_t)page * a.c.heads + hk) * a.c.page + (t1 - e * a.c.page);
                }
            } else {
                const uint32_t t1 = token_of(t0), e = p.page_div.div(t1);
                const bool good = entry < a.c.num_pages;
                w.valid &= (uint32_t)__ballot(good);
                const uint64_t row = ((uint64_t)(good ? entry : 0u) * a.c.heads + hk) * a.c.page + (t1 - e * a.c.page);
                w.low = (uint32_t)row;
                w.high = (uint32_t)(row >> 32);
            }
            return w;
        };
        uint8_t* mine = ring + wave * (DEPTH * ST::BYTES);
        auto issue = [&](const Place& w, uint32_t slot) {
            if constexpr (!SPREAD && ST::CPR >= 4) ST::issue_halves(a.c, p, mine + slot * ST::BYTES, w.row[0], w.row[1]);
            else ST::issue(a.c, p, mine + slot * ST::BYTES, [&](uint32_t t) -> uint64_t {
                if constexpr (SPREAD) {
                    return (uint64_t)(uint32_t)__shfl((int)w.high, (int)t) << 32 | (uint32_t)__shfl((int)w.low, (int)t);
                } else {
                    return (t & 16 ? w.row[1] : w.row[0]) + (t & 15);
                }
            });
        };

        // This wave's tiles of the piece, the first ones on their way
        const uint32_t end = (off + count) * STEP < s.held ? (off + count) * STEP : s.held;
        uint32_t t0 = off * STEP + 32 * wave;
        const uint32_t tiles = t0 < end && a.c.num_pages ? (end - t0 + STEP - 1) / STEP : 0u;
        uint32_t valid[DEPTH];
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) valid[i] = 0;
#pragma unroll
        for (int i = 0; i < DEPTH - 1; ++i) {
            if ((uint32_t)i < tiles) {
                const Place w = find(t0 + i * STEP, entry_of(t0 + i * STEP));
                valid[i] = w.valid;
                issue(w, i);
            }
        }

        // this lane's rows of Q
        bf16x8 q[NQ][NS];
        uint32_t tok[NQ];  // their new tokens
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const uint32_t row = row0 + 16 * i + n;
            tok[i] = p.group_div.div(row);
            const uint16_t* qp = a.q + b * a.ldq_b + tok[i] * a.ldq_t + (hk * p.group + row - tok[i] * p.group) * a.ldq_h + g * (D / 4);
#pragma unroll
            for (int st = 0; st < NS; ++st) {
                u32x4 w = {0u, 0u, 0u, 0u};
                if (tok[i] < s.fresh) {
                    if (a.q_aligned) {
                        w = *reinterpret_cast<const u32x4*>(qp + 8 * st);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = (uint32_t)qp[8 * st + 2 * j] | ((uint32_t)qp[8 * st + 2 * j + 1] << 16);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] ^= p.flip;
                }
                q[i][st] = __builtin_bit_cast(bf16x8, w);
            }
        }
        f32x4 o[NQ][NJ];
        float m[NQ], l[NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            m[i] = NO_MAX;
            l[i] = 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) o[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // the mask rows of this tile's tokens, where the piece reaches a new token
        const uint32_t tok0 = p.group_div.div(row0);
        const bool pack = a.mask && a.nt <= MASK_BITS && end > s.cached;
        if (pack) {
            const uint32_t last = p.group_div.div(row0 + ROWS - 1), ends = last < s.fresh ? last + 1 : s.fresh;
            for (uint32_t i = tok0 + wave; i < ends; i += 4) {
                const uint8_t* row = a.mask + b * a.ldm_b + i * a.ldm_r;
                for (uint32_t c = 0; c < a.nt; c += 64) {
                    const uint64_t bits = __ballot(c + lane < a.nt && row[c + lane] != 0);
                    if (lane < 2) masks[i - tok0][c / 32 + lane] = (uint32_t)(bits >> (32 * lane));
                }
            }
            __syncthreads();
        }

        uint32_t entry = tiles ? entry_of(t0 + (DEPTH - 1) * STEP) : 0u;
        uint32_t slot = 0;
        for (uint32_t k = 0; k < tiles; ++k, t0 += STEP) {
            // load the tile DEPTH - 1 ahead into the slot that was worked on last
            const uint32_t ahead = tiles - 1 - k;  // tiles after this one
            if (ahead >= DEPTH - 1) {
                const uint32_t next = entry_of(t0 + DEPTH * STEP);
                const Place w = find(t0 + (DEPTH - 1) * STEP, entry);
                entry = next;
                valid[DEPTH - 1] = w.valid;
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // its reads are done
                issue(w, slot == 0 ? DEPTH - 1 : slot - 1);
                wait_loads<(DEPTH - 1) * ST::LOADS>();
            } else if (DEPTH == 3 && ahead == 1) {
                wait_loads<ST::LOADS>();
            } else {
                wait_loads<0>();
            }
            // Of two workgroups of a CU the older is served first, and ends early: they take turns in front,
            // four tiles each (512 rows of a head over 131072 FP4 tokens: 485 to 462 us, FP8 495 to 490).  Fewer rows, which wait
            // for memory, gained nothing.
            if constexpr (NQ * D == 256) {
                if (((k >> 2) + (blockIdx.x >> 8)) & 1) __builtin_amdgcn_s_setprio(0);
                else __builtin_amdgcn_s_setprio(1);
            }
            const uint32_t here = valid[0];
            const uint8_t* at = mine + slot * ST::BYTES;
            const bool edge = here != 0xFFFFFFFFu || t0 + 32 > s.cached;
            f32x4 x[NQ][2];
#pragma unroll
            for (int i = 0; i < NQ; ++i) x[i][0] = x[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
            const uint32_t key = 4 * (n & 3) + (n >> 2);
            uint32_t kw[2][ST::RB / 16], v[8][ST::VW];
            float ks[2][KS], vs[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ST::key_run(at, h, key, g, kw[h]);
#pragma unroll
                for (int i = 0; i < KS; ++i) ks[h][i] = scale_f32<POW2>(p, ST::scale(p, at, 0, 16 * h + key, g * (D / 4) + i * BS));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                ST::value_run(at, k >> 2, 4 * (k & 3) + g, n, v[k]);
                vs[k] = scale_f32<POW2>(p, ST::scale(p, at, 1, 16 * (k >> 2) + 4 * (k & 3) + g, n * NJ));
            }
#pragma unroll
            for (int st = 0; st < NS; ++st)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bf16x8 kv = decode_run<FP8, POW2>(&kw[h][st * (FP8 ? 2 : 1)], ks[h][8 * st / BS]);
#pragma unroll
                    for (int i = 0; i < NQ; ++i) x[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kv, q[i][st], x[i][h], 0, 0, 0);
                }
            uint32_t apart = 0;  // tokens whose values are added to the rows that see them, and to no others
            uint32_t seen[NQ];  // bits of the tokens that a row sees, of the new ones those of the lane's group
            if (__builtin_expect(edge, 0)) {
                const uint32_t g = fresh(lane >> 4);
                bool hides = false;
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    seen[i] = seen_bits(a, s, b, tok[i], t0, here, g, pack ? masks[tok[i] < s.fresh ? tok[i] - tok0 : 0u] : nullptr);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t bit = 16 * (k >> 2) + 4 * (k & 3) + g;
                        if (!((seen[i] >> bit) & 1u)) x[i][k >> 2][k & 3] = -INFINITY;
                        hides |= tok[i] < s.fresh && (((here & ~seen[i]) >> bit) & 1u);
                    }
                }
                // What lies past the sequence may be anything, infinite or NaN too; so may what some rows do not
                // see, and 0 times that would be NaN in them.
                if (__ballot(hides)) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint64_t lanes = __ballot(may_be_infinite<FP8, POW2>(v[k], vs[k]));
#pragma unroll
                        for (int i = 0; i < 4; ++i) apart |= (lanes >> (16 * i)) & 0xFFFFu ? 1u << (16 * (k >> 2) + 4 * (k & 3) + i) : 0u;
                    }
                    apart &= here;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const bool taken = ((here & ~apart) >> (16 * (k >> 2) + 4 * (k & 3) + g)) & 1u;
                    vs[k] = taken ? vs[k] : 0.f;
#pragma unroll
                    for (int w = 0; w < ST::VW; ++w) v[k][w] = taken ? v[k][w] : 0u;
                }
            }
            bf16x8 pr[NQ], rest[NQ];  // p in two parts, bf16 each
            float top[NQ];
            bool raise = false;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                top[i] = x[i][0][0];
#pragma unroll
                for (int k = 1; k < 8; ++k) top[i] = fmaxf(top[i], x[i][k >> 2][k & 3]);
                top[i] *= p.c;
                raise |= top[i] > m[i] + RAISE;
            }
            if (__ballot(raise)) {
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    const float raised = fmaxf(m[i], over_groups_max(top[i]));
                    const float f = __builtin_amdgcn_exp2f(m[i] - raised);
                    m[i] = raised;
                    l[i] *= f;
#pragma unroll
                    for (int j = 0; j < NJ; ++j) o[i][j] *= f;
                }
            }
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                float e[8], sum = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    e[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i][k >> 2][k & 3], p.c, -m[i]));
                    sum += e[k];
                }
                l[i] += sum;
                u32x4 w, r;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    w[k] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)e[2 * k], (__bf16)e[2 * k + 1]});
                    const float r0 = e[2 * k] - u2f(w[k] << 16), r1 = e[2 * k + 1] - u2f(w[k] & 0xFFFF0000u);
                    r[k] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)r0, (__bf16)r1});
                }
                pr[i] = __builtin_bit_cast(bf16x8, w);
                rest[i] = __builtin_bit_cast(bf16x8, r);
            }
            for (uint32_t left = uniform(apart); left; left &= left - 1) {
                const uint32_t t = (uint32_t)__builtin_ctz(left), k = (t >> 4) * 4 + ((t >> 2) & 3);
                const uint32_t lane = fresh(threadIdx.x & 63), from = 16 * (t & 3) + (lane & 15);  // the lane with this row's p of t
                float pt[NQ];
                bool sees[NQ];  // not p != 0: of a token that is seen, NaN counts at any weight
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    sees[i] = ((uint32_t)__shfl((int)seen[i], (int)from) >> t) & 1u;
                    auto part = [&](const bf16x8& x) {
                        const u32x4 w = __builtin_bit_cast(u32x4, x);
                        const uint32_t both = k & 4 ? (k & 2 ? w[3] : w[2]) : (k & 2 ? w[1] : w[0]);
                        return u2f(k & 1 ? both & 0xFFFF0000u : both << 16);
                    };
                    pt[i] = __shfl(part(pr[i]) + part(rest[i]), (int)from);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    uint32_t run[ST::VW];
                    const uint32_t m = 4 * (lane >> 4) + r;
                    ST::value_run(at, t >> 4, t & 15, m, run);
                    const float f = nan_scale<POW2>(scale_f32<POW2>(p, ST::scale(p, at, 1, t, m * NJ)));
#pragma unroll
                    for (int i = 0; i < NQ; ++i) add_run<FP8>(run, f, pt[i], sees[i], o[i], r);
                }
            }
            __builtin_amdgcn_sched_barrier(0);  // the values are not decoded before their turn
            auto pv = [&](auto pair) {
                constexpr int J = decltype(pair)::value;
                bf16x8 a0, a1;
                value_pair<FP8, POW2, J>(v, vs, a0, a1);
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    o[i][2 * J] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, pr[i], o[i][2 * J], 0, 0, 0);
                    o[i][2 * J + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, pr[i], o[i][2 * J + 1], 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    o[i][2 * J] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a0, rest[i], o[i][2 * J], 0, 0, 0);
                    o[i][2 * J + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a1, rest[i], o[i][2 * J + 1], 0, 0, 0);
                }
            };
            pv(std::integral_constant<int, 0>{});
            pv(std::integral_constant<int, 1>{});
            if constexpr (NJ > 4) {
                pv(std::integral_constant<int, 2>{});
                pv(std::integral_constant<int, 3>{});
            }
            if constexpr (NJ > 8) {
                pv(std::integral_constant<int, 4>{});
                pv(std::integral_constant<int, 5>{});
                pv(std::integral_constant<int, 6>{});
                pv(std::integral_constant<int, 7>{});
            }
            slot = slot == DEPTH - 1 ? 0 : slot + 1;
#pragma unroll
            for (int i = 0; i + 1 < DEPTH; ++i) valid[i] = valid[i + 1];
        }

        // the four waves' sums together, in a fixed order
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            l[i] = over_groups_sum(l[i]);
            if (g == 0) {
                wm[wave][16 * i + n] = m[i];
                wl[wave][16 * i + n] = l[i];
            }
        }
        __syncthreads();  // every wave is done with its tiles, whose LDS the sums take
        f32x4(*sums)[NQ * NJ][64] = reinterpret_cast<f32x4(*)[NQ * NJ][64]>(ring);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            float top = wm[0][16 * i + n];
#pragma unroll
            for (int w = 1; w < 4; ++w) top = fmaxf(top, wm[w][16 * i + n]);
            l[i] = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) l[i] += wl[w][16 * i + n] * __builtin_amdgcn_exp2f(wm[w][16 * i + n] - top);
            const float f = __builtin_amdgcn_exp2f(m[i] - top);
            m[i] = top;
#pragma unroll
            for (int j = 0; j < NJ; ++j) sums[wave][i * NJ + j][lane] = o[i][j] * f;
        }
        __syncthreads();
        constexpr int JW = NQ * NJ / 4 < 2 ? 2 : NQ * NJ / 4;  // a wave adds up and stores JW of the NQ NJ accumulators
        const uint32_t mine0 = wave * JW, i = mine0 / NJ, j0 = mine0 % NJ;
        if (mine0 < NQ * NJ) {
            f32x4 x[JW];
#pragma unroll
            for (int j = 0; j < JW; ++j) {
                x[j] = sums[0][mine0 + j][lane];
#pragma unroll
                for (int w = 1; w < 4; ++w) x[j] += sums[w][mine0 + j][lane];
            }
            float mi = m[0], li = l[0];
#pragma unroll
            for (int k = 1; k < NQ; ++k) {
                mi = i == k ? m[k] : mi;
                li = i == k ? l[k] : li;
            }
            if (count == steps) {
                store_rows<D, JW>(a, p, s, b, hk, row0 + 16 * i, j0, x, mi, li);
            } else {
                float* piece = pieces_of(a) + (2 * (uint64_t)group + (off ? 0 : 1)) * Piece<D, NQ>::FLOATS;
#pragma unroll
                for (int j = 0; j < JW; ++j) reinterpret_cast<f32x4*>(piece)[(mine0 + j) * 64 + lane] = x[j];
                if (g == 0 && j0 == 0) {
                    piece[Piece<D, NQ>::SUMS + 16 * i + n] = mi;
                    piece[Piece<D, NQ>::SUMS + 16 * NQ + 16 * i + n] = li;
                }
            }
        }
        __syncthreads();  // the sums are read: the ring is free for the next piece
        pos += count;
    }
}

// Joins the pieces of the segments that were cut: a workgroup takes elements j0 ... j0 + JW - 1 of
// every run of D / 16 of 16 rows, its waves every WAVES-th piece, four at a time; all are added in
// an order that the lengths fix.  4 to 8 us, most of it the launch and three loads that wait for each other.
template <int D, int NQ, int WAVES, int JW>
__global__ __launch_bounds__(64 * WAVES) void attn_join_kernel(KvAttnArgs a, AttnPlan p)
{
    constexpr int NJ = D / 16, ROWS = 16 * NQ, AT_ONCE = 4;
    using P = Piece<D, NQ>;
    __shared__ f32x4 sums[WAVES - 1][JW][64];
    __shared__ float wm[WAVES][16], wl[WAVES][16];
    const uint32_t lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15, wave = threadIdx.x >> 6;
    const uint32_t j0 = blockIdx.x % (NJ / JW) * JW, rest = blockIdx.x / (NJ / JW);
    const uint32_t i = rest % NQ, tiles = rest / NQ, heads = tiles / p.row_tiles, tile = tiles - heads * p.row_tiles;
    const uint32_t b = heads / a.c.heads, hk = heads - b * a.c.heads;
    const uint32_t* meta = static_cast<const uint32_t*>(a.work);
    const uint32_t total = meta[0];
    const Seq s = seq_of(a, b);
    const Part part = part_of(p, s, a.c.heads, ROWS);
    const uint32_t teams = teams_for(p, total);
    const Cut cut{total / teams, total % teams};
    const uint32_t seg = (hk * part.tiles + tile) / p.team, member = hk * part.tiles + tile - seg * p.team;
    const uint32_t p0 = meta[1 + b] + seg * (part.steps + p.begin) + p.begin;  // its first step
    if (tile >= part.tiles) return;
    const uint32_t first = cut.owner(p0), last = cut.owner(p0 + part.steps - 1);
    if (first == last) return;
    const float* work = pieces_of(a);
    float m = NO_MAX, l = 0.f;
    f32x4 o[JW];
#pragma unroll
    for (int j = 0; j < JW; ++j) o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (uint32_t w0 = first + wave; w0 <= last; w0 += WAVES * AT_ONCE) {
        float pm[AT_ONCE], pl[AT_ONCE];
        f32x4 po[AT_ONCE][JW];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const bool there = w0 + k * WAVES <= last;
            const uint32_t w = there ? w0 + k * WAVES : w0;
            const float* q = work + (2 * ((uint64_t)w * p.team + member) + (w == first ? 1 : 0)) * P::FLOATS;
            pm[k] = there ? q[P::SUMS + 16 * i + n] : NO_MAX;
            pl[k] = there ? q[P::SUMS + ROWS + 16 * i + n] : 0.f;
#pragma unroll
            for (int j = 0; j < JW; ++j) {
                const f32x4 v = reinterpret_cast<const f32x4*>(q)[(i * NJ + j0 + j) * 64 + lane];
                po[k][j] = there ? v : f32x4{0.f, 0.f, 0.f, 0.f};
            }
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) top = fmaxf(top, pm[k]);
        const float f = __builtin_amdgcn_exp2f(m - top);
        m = top;
        l *= f;
#pragma unroll
        for (int j = 0; j < JW; ++j) o[j] *= f;
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const float e = __builtin_amdgcn_exp2f(pm[k] - top);
            l += e * pl[k];
#pragma unroll
            for (int j = 0; j < JW; ++j) o[j] += e * po[k][j];
        }
    }
    if (g == 0) {
        wm[wave][n] = m;
        wl[wave][n] = l;
    }
    __syncthreads();
    float top = wm[0][n];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) top = fmaxf(top, wm[w][n]);
    l = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) l += wl[w][n] * __builtin_amdgcn_exp2f(wm[w][n] - top);
    const float f = __builtin_amdgcn_exp2f(m - top);
#pragma unroll
    for (int j = 0; j < JW; ++j) {
        o[j] *= f;
        if (wave) sums[wave - 1][j][lane] = o[j];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int w = 0; w < WAVES - 1; ++w)
#pragma unroll
            for (int j = 0; j < JW; ++j) o[j] += sums[w][j][lane];
        store_rows<D, JW>(a, p, s, b, hk, tile * ROWS + 16 * i, j0, o, top, l);
    }
}

template <bool FP8, bool POW2, int D, int BS, int NQ, int SPREAD>
hipError_t launch_pieces(const KvAttnArgs& a, AttnPlan& p, hipStream_t st)
{
    using R = Room<FP8, D, BS, NQ, SPREAD>;
    static LdsLimit limit;
    const hipError_t e = limit.ensure((const void*)attn_tile_kernel<FP8, POW2, D, BS, NQ, SPREAD>, R::DYNAMIC, st);
    if (e != hipSuccess) return e;
    // as many workgroups as run at once, if there is a step for each team
    const uint32_t room = 256 * R::GROUPS / p.team;
    p.teams = p.most < room ? (uint32_t)p.most : room;
    hipLaunchKernelGGL((attn_tile_kernel<FP8, POW2, D, BS, NQ, SPREAD>), dim3(p.teams * p.team), dim3(256), R::DYNAMIC, st, a, p);
    return hipGetLastError();
}

template <bool FP8, bool POW2, int D, int BS, int NQ>
hipError_t launch_tiles(const KvAttnArgs& a, AttnPlan p, hipStream_t st)
{
    hipError_t e = hipErrorInvalidValue;
    if (a.c.page % 16 == 0) {
        e = launch_pieces<FP8, POW2, D, BS, NQ, 0>(a, p, st);
    } else if (p.scale_shift >= 2) {
        e = launch_pieces<FP8, POW2, D, BS, NQ, 1>(a, p, st);
    } else {
        if constexpr (BS > 16 || D == 64) e = launch_pieces<FP8, POW2, D, BS, NQ, 2>(a, p, st);
    }
    if (e == hipSuccess && p.teams > 1) {
        // Few segments are cut into many pieces each: more waves, and the elements shared out.
        const uint32_t rows = a.batch * a.c.heads * p.row_tiles * NQ;
        if (p.teams * p.team > 8 * a.batch * a.c.heads * p.row_tiles)
            hipLaunchKernelGGL((attn_join_kernel<D, NQ, 16, 2>), dim3(rows * (D / 32)), dim3(1024), 0, st, a, p);
        else
            hipLaunchKernelGGL((attn_join_kernel<D, NQ, 4, D / 16>), dim3(rows), dim3(256), 0, st, a, p);
        e = hipGetLastError();
    }
    return e;
}

template <int D, int BS, int NQ>
hipError_t launch_kind(const KvAttnArgs& a, const AttnPlan& p, hipStream_t st)
{
    const bool pow2 = a.c.fmt == FMT_E8M0;
    if (a.c.fp8) return pow2 ? launch_tiles<true, true, D, BS, NQ>(a, p, st) : launch_tiles<true, false, D, BS, NQ>(a, p, st);
    return pow2 ? launch_tiles<false, true, D, BS, NQ>(a, p, st) : launch_tiles<false, false, D, BS, NQ>(a, p, st);
}

}  // namespace kv

// one per head size; nq is 1, 2 or 4 for heads of 64, 1 or 2 for 128, 1 for 256
hipError_t launch_attn_64(const KvAttnArgs& a, const kv::AttnPlan& p, int nq, hipStream_t st);
hipError_t launch_attn_128(const KvAttnArgs& a, const kv::AttnPlan& p, int nq, hipStream_t st);
hipError_t launch_attn_256(const KvAttnArgs& a, const kv::AttnPlan& p, int nq, hipStream_t st);

}  // namespace mxk
