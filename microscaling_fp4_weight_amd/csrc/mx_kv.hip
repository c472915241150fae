// mx_kv.hip -- rotary positions, and the quantized write and read of the key/value cache.
//
// Rotation: the pair (a, b) of a head's elements becomes (a c - b s, b c + a s) with c, s the
// cosine and sine of position * frequency from a table; its transpose, the gradient, has -s.
// Products and sums are separate fp32 operations (no fused multiply-add), so that the value, and
// with it every code quantized from it, is the one that the formula gives in fp32, on every path.
//
// Write: per block of a head's key or value the scale and the codes of the block formats
// (nearest scale to absmax / (6 or 448) g, nearest element to |x| / (s g), exact decisions).
// Read: e * s * g rounded once to fp32, then to the output type.
//
// All of these move each byte once and do a few operations on it: HBM bounds the large calls (a copy reaches
// 5.2 TB/s here), the launch the small ones (2.1 us for a rotation of one token, 3.4 to 3.7 for a read or write).
// Times here are of calls back to back on three sets of inputs.  Rotations of whole chunks run at 5.8 to 6.0
// TB/s, reads at 5.7 to 6.0; writes at 4.7 (8192 x 8 heads of 128 to FP4) and 3.9 (FP8 under 16-element E4M3
// scales): 64- or 32-byte rows of codes and 4-byte rows of scales, scattered over the pool by slot, are what is
// left of their time.
#include "mx_device.h"
#include "mx_fp8_device.h"
#include "mx_kv_internal.h"

namespace mxk {
namespace kv {

constexpr int THREADS = 256;

// ---------------------------------------------------------------------------------------
// rotation
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void turn(float a, float b, float c, float s, float& u, float& w)
{
#pragma clang fp contract(off)
    const float ac = a * c, bs = b * s, bc = b * c, as = a * s;
    u = ac - bs;
    w = bc + as;
}

__device__ __forceinline__ const float* table_row(const RopePart& r, uint32_t token)
{
    int32_t p = r.positions[token];
    p = p < 0 ? 0 : p;
    const uint32_t q = (uint32_t)p < r.max_pos ? (uint32_t)p : r.max_pos - 1;
    return r.table + (int64_t)q * r.rot;
}

// A chunk is 16 bytes of a row: 8 bf16 or 4 fp32 elements, as fp32 here.
template <bool BF16>
struct Chunk {
    static constexpr int N = BF16 ? 8 : 4;
    float v[N];
};

template <bool BF16>
__device__ __forceinline__ Chunk<BF16> load_chunk(const void* p)
{
    Chunk<BF16> c;
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
    if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c.v[2 * j] = u2f(w[j] << 16);
            c.v[2 * j + 1] = u2f(w[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) c.v[j] = u2f(w[j]);
    }
    return c;
}

template <bool BF16>
__device__ __forceinline__ void store_chunk(void* p, const Chunk<BF16>& c)
{
    u32x4 w;
    if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)c.v[2 * j], (__bf16)c.v[2 * j + 1]});
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = f2u(c.v[j]);
    }
    *reinterpret_cast<u32x4*>(p) = w;
}

template <bool BF16>
__device__ __forceinline__ float load_elem(const void* base, int64_t i)
{
    if constexpr (BF16) return u2f((uint32_t)reinterpret_cast<const uint16_t*>(base)[i] << 16);
    else return reinterpret_cast<const float*>(base)[i];
}

template <bool BF16>
__device__ __forceinline__ void store_elem(void* base, int64_t i, float v)
{
    if constexpr (BF16) reinterpret_cast<__bf16*>(base)[i] = (__bf16)v;
    else reinterpret_cast<float*>(base)[i] = v;
}

template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[N])
{
    if constexpr (N == 2) {
        const f32x2 w = *reinterpret_cast<const f32x2*>(p);
        v[0] = w.x;
        v[1] = w.y;
        return;
    }
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(p + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j + i] = w[i];
    }
}

struct RopeGrid {
    FastDiv per_row_div, heads_div;
    uint32_t per_row, total;
    uint32_t rot_units;  // units of a row that rotate (half layout); the others are copied
};

// Rows whose pairs fall on whole chunks: a thread takes two chunks of a row, in the half layout
// a chunk and its partner, so that it reads and writes each element once.  8192 x 64 heads of 128, bf16: 47 us,
// 5.8 TB/s.
template <bool BF16, bool INTER>
__global__ __launch_bounds__(THREADS) void rope_kernel(RopeArgs a, RopeGrid g)
{
    constexpr int N = Chunk<BF16>::N;
    constexpr int ES = BF16 ? 2 : 4;
    const uint32_t id = blockIdx.x * THREADS + threadIdx.x;
    if (id >= g.total) return;
    const uint32_t row = g.per_row_div.div(id), u = id - row * g.per_row;
    const uint32_t token = g.heads_div.div(row), head = row - token * a.heads;
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + (token * a.ldx_t + head * a.ldx_h) * ES;
    uint8_t* y = static_cast<uint8_t*>(a.y) + (token * a.ldy_t + head * a.ldy_h) * ES;
    const uint32_t hr = a.r.rot / 2;
    const float sign = a.r.transpose ? -1.0f : 1.0f;
    uint32_t d0, d1;  // first elements of the two chunks
    if (INTER || u >= g.rot_units) {
        // the rest of the row in two halves, so that neighbouring threads read neighbouring chunks
        d0 = INTER ? N * u : a.r.rot + N * (u - g.rot_units);
        d1 = d0 + N * (g.per_row - (INTER ? 0 : g.rot_units));
    } else {
        d0 = N * u;
        d1 = d0 + hr;
    }
    const bool two = d1 < a.dim;
    Chunk<BF16> p = load_chunk<BF16>(x + d0 * ES);
    Chunk<BF16> q = p;
    if (two) q = load_chunk<BF16>(x + d1 * ES);
    if (d0 < a.r.rot) {
        const float* t = table_row(a.r, token);
        if constexpr (INTER) {
            float c[N / 2], s[N / 2];
            auto pairs = [&](Chunk<BF16>& k, uint32_t d) {
                load_floats(t + d / 2, c);
                load_floats(t + hr + d / 2, s);
#pragma unroll
                for (int j = 0; j < N / 2; ++j) turn(k.v[2 * j], k.v[2 * j + 1], c[j], s[j] * sign, k.v[2 * j], k.v[2 * j + 1]);
            };
            pairs(p, d0);
            if (two && d1 < a.r.rot) pairs(q, d1);
        } else {
            float c[N], s[N];
            load_floats(t + d0, c);
            load_floats(t + hr + d0, s);
#pragma unroll
            for (int j = 0; j < N; ++j) turn(p.v[j], q.v[j], c[j], s[j] * sign, p.v[j], q.v[j]);
        }
    }
    store_chunk<BF16>(y + d0 * ES, p);
    if (two) store_chunk<BF16>(y + d1 * ES, q);
}

// Any sizes and strides: a thread takes one pair, or one element that is copied.  What bounds it is the number of
// its 2- or 4-byte accesses: 24 of 96 elements, 8192 x 64 heads, bf16, take 150 us, 1.3 TB/s.
template <bool BF16>
__global__ __launch_bounds__(THREADS) void rope_any_kernel(RopeArgs a, RopeGrid g)
{
    const uint32_t id = blockIdx.x * THREADS + threadIdx.x;
    if (id >= g.total) return;
    const uint32_t row = g.per_row_div.div(id), u = id - row * g.per_row;
    const uint32_t token = g.heads_div.div(row), head = row - token * a.heads;
    const int64_t xo = token * a.ldx_t + head * a.ldx_h, yo = token * a.ldy_t + head * a.ldy_h;
    const uint32_t hr = a.r.rot / 2;
    if (u >= hr) {
        const uint32_t d = u + hr;
        store_elem<BF16>(a.y, yo + d, load_elem<BF16>(a.x, xo + d));
        return;
    }
    const uint32_t d0 = a.r.inter ? 2 * u : u, d1 = a.r.inter ? d0 + 1 : u + hr;
    const float* t = table_row(a.r, token);
    float p, q;
    turn(load_elem<BF16>(a.x, xo + d0), load_elem<BF16>(a.x, xo + d1), t[u], a.r.transpose ? -t[hr + u] : t[hr + u], p, q);
    store_elem<BF16>(a.y, yo + d0, p);
    store_elem<BF16>(a.y, yo + d1, q);
}

__global__ __launch_bounds__(THREADS) void rope_table_kernel(RopeTableArgs a)
{
    const uint32_t id = blockIdx.x * THREADS + threadIdx.x;
    if (id >= a.max_pos * a.half) return;
    const uint32_t p = id / a.half, i = id - p * a.half;
    const double R = 2.0 * a.half, PI = 3.14159265358979323846;
    const double base = a.scaling == 2 ? a.base * pow(a.factor, R / (R - 2.0)) : a.base;
    double f = pow(base, -2.0 * i / R);
    if (a.scaling == 1) f /= a.factor;
    if (a.scaling == 3) {
        const double w = fmin(fmax((a.original_len * f / (2.0 * PI) - a.low) / (a.high - a.low), 0.0), 1.0);
        f = f * w + f / a.factor * (1.0 - w);
    }
    double s, c;
    sincos((double)p * f, &s, &c);
    a.table[(int64_t)p * 2 * a.half + i] = (float)(c * a.magnitude);
    a.table[(int64_t)p * 2 * a.half + a.half + i] = (float)(s * a.magnitude);
}

// ---------------------------------------------------------------------------------------
// element codes of a thread's 8 elements
// ---------------------------------------------------------------------------------------

// Scale byte of a block of E4M3 elements from its absmax (fp32 bits), g = 1: the value nearest to
// a / 448.  448 = 7 * 2^6 and a midpoint m of the scale format has five significant bits, so an a that
// is not 448 m is at least one unit in its last place away from it, which in the quotient is at least 0.57
// of a unit: rounding fl64(a * fl64(1/448)) to fp32 gives m only for a = 448 m.  E8M0: with
// a = f 2^e the quotient reaches 1.5 * 2^k at a = 672 * 2^k = 1.3125 * 2^(k + 9), so the nearest power of
// two (ties up) has exponent e - 9 + [f >= 1.3125].
template <int FMT>
__device__ __forceinline__ uint32_t scale_code_fp8_g1(uint32_t abits)
{
    if constexpr (FMT == FMT_E8M0) {
        const int byte = (int)(abits >> 23) - 9 + ((abits & 0x7FFFFFu) >= 0x280000u ? 1 : 0);
        return byte < 0 ? 0u : (uint32_t)byte;
    } else {
        return fp8_code_f32<FMT>((float)((double)u2f(abits) * (1.0 / 448.0)));
    }
}

// Scale byte of a block from its absmax (fp32 bits) and g
template <bool FP8, int FMT, bool G1>
__device__ __forceinline__ uint32_t block_scale(uint32_t amax, double g)
{
    if constexpr (FP8 && G1) return scale_code_fp8_g1<FMT>(amax);
    else if constexpr (FP8) return scale_code_g<FMT>(amax, 448.0 * g);
    else if constexpr (G1) return scale_code_g1<FMT>(amax);
    else return scale_code_g<FMT>(amax, 6.0 * g);
}

// The codes of 8 elements (fp32 bits) under a scale byte: one word of E2M1 nibbles, or two
// words of E4M3 bytes.
template <bool FP8, int FMT, bool G1, bool BF16>
__device__ __forceinline__ u32x2 encode8(const uint32_t (&xb)[8], uint32_t sb, double g)
{
    u32x2 cw = {0u, 0u};
    if constexpr (!FP8 && G1) {
        const EncG1 p = enc_params_g1<FMT>(sb);
#pragma unroll
        for (int j = 0; j < 4; ++j) cw.x |= enc_pair_g1<FMT>(u2f(xb[2 * j]), u2f(xb[2 * j + 1]), p, 0u) << (8 * j);
    } else if constexpr (!FP8) {
        const EncG p = enc_params_g<FMT>(sb, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) cw.x |= enc_elem_g(xb[j], p) << (4 * j);
    } else if constexpr (G1 && BF16) {
        const EncG1 p = enc_params_g1<FMT>(sb);
        const float lim = 448.0f * p.pow2;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = (xb[2 * j] >> 16) | (xb[2 * j + 1] & 0xFFFF0000u);
        f8::i16x2 h0 = {0, 0}, h1 = {0, 0};
        h0 = f8::enc_fp8_pair<FMT, 0>(h0, w[0], p, lim);
        h0 = f8::enc_fp8_pair<FMT, 1>(h0, w[1], p, lim);
        h1 = f8::enc_fp8_pair<FMT, 0>(h1, w[2], p, lim);
        h1 = f8::enc_fp8_pair<FMT, 1>(h1, w[3], p, lim);
        cw = u32x2{__builtin_bit_cast(uint32_t, h0), __builtin_bit_cast(uint32_t, h1)};
    } else {
        const f8::Blk p = f8::block_params<FMT>(sb, G1 ? 1.0 : g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            cw.x |= f8::elem_byte(xb[j], p) << (8 * j);
            cw.y |= f8::elem_byte(xb[4 + j], p) << (8 * j);
        }
    }
    return cw;
}

// e * s * g of 8 codes, one fp32 rounding of the exact product
template <bool FP8, int FMT, bool G1>
__device__ __forceinline__ void decode8(const u32x2 cw, uint32_t sb, double g, float (&v)[8])
{
    f32x2 e[4];
    if constexpr (FP8) {
        e[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(cw.x, 1.0f, false);
        e[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(cw.x, 1.0f, true);
        e[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(cw.y, 1.0f, false);
        e[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(cw.y, 1.0f, true);
    } else {
        e[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw.x, 1.0f, 0);
        e[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw.x, 1.0f, 1);
        e[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw.x, 1.0f, 2);
        e[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cw.x, 1.0f, 3);
    }
    if constexpr (G1) {
        const float s = scale_value_f32<FMT>(sb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = e[j].x * s;
            v[2 * j + 1] = e[j].y * s;
        }
    } else {
        const double s = scale_value_f64<FMT>(sb) * g;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = (float)((double)e[j].x * s);
            v[2 * j + 1] = (float)((double)e[j].y * s);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, const float (&v)[8])
{
    u32x4* o = reinterpret_cast<u32x4*>(p);
    if constexpr (BF16) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * j], (__bf16)v[2 * j + 1]});
        o[0] = w;
    } else {
        o[0] = u32x4{f2u(v[0]), f2u(v[1]), f2u(v[2]), f2u(v[3])};
        o[1] = u32x4{f2u(v[4]), f2u(v[5]), f2u(v[6]), f2u(v[7])};
    }
}

struct KvGrid {
    FastDiv per_row_div, rows_div, page_div;
    uint32_t per_row, rows, total;  // threads of a row, rows of a token (2 x heads), threads in all
    uint32_t lanes;                 // threads of a block
    uint32_t rope;                  // 0: none, 1: pairs on whole units, 2: any
    uint32_t aligned;               // bit t: 16-byte rows of x[t]
    uint32_t block_shift;           // log2 of the block
    uint32_t token_shift;           // log2 of the tokens whose rows of one head are adjacent
    bool waves;                     // each wave's rows are of one token and tensor
    uint32_t row_shift;             // then: log2 of per_row; rows is then the waves of a token
};

// The token, tensor and head of row `row` of the grid.  Rows run over 2^token_shift tokens of one head, then
// over heads: neighbouring tokens' codes and scale bytes share lines of the pool, which one
// workgroup should touch, not eight on eight L2s.  E4M3 codes of 64-element heads under scales of 16 (4099 x 32
// heads, bf16): written in 21.9 us by four tokens, 22.7 one at a time, read in 11.5 by 32 against 14.0.  More
// tokens of a head at once read their rotation table rows from farther away (16: 17.8 against 17.1 us for 8192 x 8
// heads of 128 to FP4).
__device__ __forceinline__ void place_of(const KvGrid& g, uint32_t heads, uint32_t row, uint32_t& token, uint32_t& t, uint32_t& head)
{
    const uint32_t q = row >> g.token_shift, group = g.rows_div.div(q), th = q - group * g.rows;
    token = (group << g.token_shift) + (row & ((1u << g.token_shift) - 1));
    t = th >= heads ? 1u : 0u;
    head = th - t * heads;
}

// Where a thread works.  WAVES: a wave takes rows of one token and tensor only, so that everything but
// the head and the place in the row is computed once for the wave, on its scalar unit.
struct Spot {
    uint32_t token, t, head, u;
    bool act;
};

template <bool WAVES>
__device__ __forceinline__ Spot spot_of(const KvGrid& g, uint32_t heads, uint32_t tokens)
{
    Spot s;
    if constexpr (WAVES) {
        const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(blockIdx.x * (THREADS / 64) + (threadIdx.x >> 6)));
        const uint32_t lane = threadIdx.x & 63;
        const uint32_t q = wave >> g.token_shift, group = g.rows_div.div(q);
        s.token = (group << g.token_shift) + (wave & ((1u << g.token_shift) - 1));
        const uint32_t th = (q - group * g.rows) << (6 - g.row_shift);
        s.t = th >= heads ? 1u : 0u;
        s.head = th - s.t * heads + (lane >> g.row_shift);
        s.u = lane & ((1u << g.row_shift) - 1);
        s.act = s.token < tokens;
    } else {
        const uint32_t id = blockIdx.x * THREADS + threadIdx.x;
        const uint32_t row = id < g.total ? g.per_row_div.div(id) : 0u;
        s.u = id < g.total ? id - row * g.per_row : 0u;
        place_of(g, heads, row, s.token, s.t, s.head);
        s.act = id < g.total && s.token < tokens;
    }
    if (!s.act) s.token = tokens - 1;
    return s;
}

// index of the pool's row of (slot, head)
__device__ __forceinline__ uint64_t pool_row(const KvPool& c, const FastDiv& page_div, uint32_t slot, uint32_t head)
{
    const uint32_t page = page_div.div(slot);
    return ((uint64_t)page * c.heads + head) * c.page + (slot - page * c.page);
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t off, bool aligned, float (&v)[8])
{
    constexpr int ES = BF16 ? 2 : 4;
    constexpr int N = Chunk<BF16>::N;
    if (aligned) {
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) {
            const Chunk<BF16> c = load_chunk<BF16>(static_cast<const uint8_t*>(base) + (off + i * N) * ES);
#pragma unroll
            for (int j = 0; j < N; ++j) v[i * N + j] = c.v[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = load_elem<BF16>(base, off + j);
    }
}

// Elements of a row that a thread's chunks begin at.  Two chunks of a thread are half a row apart --
// of a rotated key half the rotated part, then half the rest, so that pairs meet in one thread -- and
// neighbouring threads have neighbouring chunks.
template <int CHUNKS>
__device__ __forceinline__ void chunks_of(uint32_t u, uint32_t dim, uint32_t rot, uint32_t (&d)[CHUNKS])
{
    if constexpr (CHUNKS == 1) {
        d[0] = 8 * u;
    } else {
        const bool first = 16 * u < rot;
        d[0] = first ? 8 * u : rot / 2 + 8 * u;
        d[1] = d[0] + (first ? rot / 2 : (dim - rot) / 2);
    }
}

// A thread takes CHUNKS times 8 consecutive elements of one head's key or value; a block's absmax
// comes together by lane shuffles (a block is 2 to 32 adjacent threads: chunks come in whole blocks, so that
// blocks never straddle a wave).  8192 x 8 heads of 128, bf16 to FP4 and the values back: 17.1 us, 4.7 TB/s.
template <bool FP8, int FMT, bool G1, bool BF16, int CHUNKS, bool WAVES>
__global__ __launch_bounds__(THREADS) void kv_write_kernel(KvWriteArgs a, KvGrid g)
{
    const Spot at = spot_of<WAVES>(g, a.c.heads, a.tokens);
    const uint32_t token = at.token, t = at.t, head = at.head, u = at.u;
    const int64_t xo = token * a.ld_t[t] + head * a.ld_h[t];
    const bool al = (g.aligned >> t) & 1u;
    const bool pairs = CHUNKS == 2 && g.rope == 1 && !a.r.inter && t == 0;
    uint32_t d0[CHUNKS];
    chunks_of<CHUNKS>(u, a.c.dim, pairs ? a.r.rot : 0u, d0);

    float v[CHUNKS][8];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) load8<BF16>(a.x[t], xo + d0[c], al, v[c]);
    const int32_t slot = a.slots[token];
    if (t == 0 && g.rope != 0) {
        const float* tr = table_row(a.r, token);
        const uint32_t hr = a.r.rot / 2;
        if (pairs) {
            if (d0[0] < hr) {
                float cs[8], sn[8];
                load_floats(tr + d0[0], cs);
                load_floats(tr + hr + d0[0], sn);
#pragma unroll
                for (int j = 0; j < 8; ++j) turn(v[0][j], v[CHUNKS - 1][j], cs[j], sn[j], v[0][j], v[CHUNKS - 1][j]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                if (d0[c] >= a.r.rot) continue;
                if (g.rope == 1 && a.r.inter) {
                    float cs[4], sn[4];
                    load_floats(tr + d0[c] / 2, cs);
                    load_floats(tr + hr + d0[c] / 2, sn);
#pragma unroll
                    for (int j = 0; j < 4; ++j) turn(v[c][2 * j], v[c][2 * j + 1], cs[j], sn[j], v[c][2 * j], v[c][2 * j + 1]);
                } else if (g.rope == 1) {  // the pairs' other elements are another thread's
                    const bool lo = d0[c] < hr;
                    float w[8], cs[8], sn[8], z;
                    load8<BF16>(a.x[0], xo + (lo ? d0[c] + hr : d0[c] - hr), al, w);
                    load_floats(tr + (lo ? d0[c] : d0[c] - hr), cs);
                    load_floats(tr + (lo ? d0[c] + hr : d0[c]), sn);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (lo) turn(v[c][j], w[j], cs[j], sn[j], v[c][j], z);
                        else turn(w[j], v[c][j], cs[j], sn[j], z, v[c][j]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t d = d0[c] + j;
                        if (d >= a.r.rot) continue;
                        const bool lo = a.r.inter ? !(d & 1u) : d < hr;
                        const uint32_t i = a.r.inter ? d / 2 : (lo ? d : d - hr);
                        const uint32_t other = a.r.inter ? d ^ 1u : (lo ? d + hr : d - hr);
                        const float w = load_elem<BF16>(a.x[0], xo + other);
                        float z;
                        if (lo) turn(v[c][j], w, tr[i], tr[hr + i], v[c][j], z);
                        else turn(w, v[c][j], tr[i], tr[hr + i], z, v[c][j]);
                    }
                }
            }
        }
    }
    uint32_t xb[CHUNKS][8], amax[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        amax[c] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // a rotated key has its input's type before it is quantized
            if constexpr (BF16) xb[c][j] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[c][j]) << 16;
            else xb[c][j] = f2u(v[c][j]);
            const uint32_t m = xb[c][j] & 0x7FFFFFFFu;
            amax[c] = m > amax[c] ? m : amax[c];
        }
    }
    for (uint32_t off = 1; off < g.lanes; off <<= 1) {
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const uint32_t o = (uint32_t)__shfl_xor((int)amax[c], (int)off);
            amax[c] = o > amax[c] ? o : amax[c];
        }
    }
    if (!at.act) return;
    const double gs = a.c.g[t];
    const bool stored = slot >= 0 && (uint32_t)slot < a.c.num_pages * a.c.page;
    const uint64_t r = stored ? pool_row(a.c, g.page_div, (uint32_t)slot, head) : 0;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const uint32_t sb = block_scale<FP8, FMT, G1>(amax[c], gs);
        const u32x2 cw = encode8<FP8, FMT, G1, BF16>(xb[c], sb, gs);
        if (stored) {
            if constexpr (FP8) *reinterpret_cast<u32x2*>(a.c.codes[t] + r * a.c.dim + d0[c]) = cw;
            else *reinterpret_cast<uint32_t*>(a.c.codes[t] + r * (a.c.dim / 2) + d0[c] / 2) = cw.x;
            if (((d0[c] / 8) & (g.lanes - 1)) == 0) a.c.scales[t][(r * a.c.dim + d0[c]) >> g.block_shift] = (uint8_t)sb;
        }
        if (a.hat[t]) {
            decode8<FP8, FMT, G1>(cw, sb, gs, v[c]);
            store8<BF16>(static_cast<uint8_t*>(a.hat[t]) + (((int64_t)token * a.c.heads + head) * a.c.dim + d0[c]) * (BF16 ? 2 : 4), v[c]);
        }
    }
}

// A thread takes two chunks of 8 elements, half a row apart; of 32 neighbouring tokens the rows of one head lie
// together.  16384 x 8 heads of 128 from FP4 to bf16: 15.0 us, 5.7 TB/s.
template <bool FP8, int FMT, bool G1, bool BF16>
__global__ __launch_bounds__(THREADS) void kv_read_kernel(KvReadArgs a, KvGrid g)
{
    const Spot at = spot_of<false>(g, a.c.heads, a.tokens);
    if (!at.act) return;
    const uint32_t token = at.token, t = at.t, head = at.head, u = at.u;
    uint32_t d0[2];
    chunks_of<2>(u, a.c.dim, 0u, d0);
    float v[2][8] = {};
    const int32_t slot = a.slots[token];
    if (slot >= 0 && (uint32_t)slot < a.c.num_pages * a.c.page) {
        const uint64_t r = pool_row(a.c, g.page_div, (uint32_t)slot, head);
        u32x2 cw[2];
        uint32_t sb[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if constexpr (FP8) cw[c] = *reinterpret_cast<const u32x2*>(a.c.codes[t] + r * a.c.dim + d0[c]);
            else cw[c] = u32x2{*reinterpret_cast<const uint32_t*>(a.c.codes[t] + r * (a.c.dim / 2) + d0[c] / 2), 0u};
            sb[c] = a.c.scales[t][(r * a.c.dim + d0[c]) >> g.block_shift];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) decode8<FP8, FMT, G1>(cw[c], sb[c], a.c.g[t], v[c]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
        store8<BF16>(static_cast<uint8_t*>(a.y[t]) + (((int64_t)token * a.c.heads + head) * a.c.dim + d0[c]) * (BF16 ? 2 : 4), v[c]);
}

KvGrid kv_grid(const KvPool& c, uint32_t tokens, uint32_t chunks, uint32_t token_shift, bool writes)
{
    KvGrid g{};
    g.per_row = c.dim / (8 * chunks);
    g.rows = 2 * c.heads;
    g.token_shift = tokens >= 64 ? token_shift : 0;
    g.total = ((((tokens - 1) >> g.token_shift) + 1) << g.token_shift) * g.rows * g.per_row;
    g.per_row_div = FastDiv::make(g.per_row);
    g.page_div = FastDiv::make(c.page);
    g.lanes = c.block / 8;
    while ((1u << g.block_shift) < c.block) ++g.block_shift;
    // A write with a power of two of threads a row, and heads in whole waves: a wave stays with one token, and its
    // slot, position and addresses are scalar: 17.1 us against 18.1 for 8192 x 8 heads of 128 (bf16 to FP4 and
    // back), 20.2 against 23.0 to FP8, 33.2 against 36.4 from fp32.  A read has too little of that to gain: 15.1 us
    // either way for twice the tokens, FP8 17.9 against 17.3.
    while (chunks == 2 && (1u << g.row_shift) < g.per_row) ++g.row_shift;
    g.waves = writes && chunks == 2 && (1u << g.row_shift) == g.per_row && g.per_row <= 64 && c.heads % (64 / g.per_row) == 0;
    if (g.waves) {
        g.rows = 2 * c.heads * g.per_row / 64;
        g.token_shift = tokens >= 64 ? 2 : 0;  // the waves of a workgroup: one token each, same heads
        g.total = ((((tokens - 1) >> g.token_shift) + 1) << g.token_shift) * g.rows * 64;
    }
    g.rows_div = FastDiv::make(g.rows);
    return g;
}

constexpr unsigned groups(uint32_t n) { return (n + THREADS - 1) / THREADS; }

}  // namespace kv

hipError_t launch_rope_table(const RopeTableArgs& a, hipStream_t st)
{
    hipLaunchKernelGGL(kv::rope_table_kernel, dim3(kv::groups(a.max_pos * a.half)), dim3(kv::THREADS), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs& a, hipStream_t st)
{
    const uint32_t n = a.bf16 ? 8 : 4, hr = a.r.rot / 2;
    const bool strides = a.ldx_t % n == 0 && a.ldx_h % n == 0 && a.ldy_t % n == 0 && a.ldy_h % n == 0;
    // Pairs on whole chunks: interleaved ones lie inside a chunk, halves are whole chunks apart.  8192 x 64 heads
    // of 128, bf16: 47 us against 104 pair by pair, half of each interleaved 45 against 176.
    const bool whole = strides && a.dim % n == 0 && (a.r.inter ? a.r.rot % n == 0 : hr % n == 0);
    kv::RopeGrid g{};
    g.rot_units = hr / n;
    if (!whole) g.per_row = hr + (a.dim - a.r.rot);
    else if (a.r.inter) g.per_row = (a.dim + 2 * n - 1) / (2 * n);
    else g.per_row = g.rot_units + (a.dim - a.r.rot + 2 * n - 1) / (2 * n);
    g.per_row_div = FastDiv::make(g.per_row);
    g.heads_div = FastDiv::make(a.heads);
    g.total = a.tokens * a.heads * g.per_row;
    const dim3 grid(kv::groups(g.total)), threads(kv::THREADS);
    if (!whole) {
        if (a.bf16) hipLaunchKernelGGL((kv::rope_any_kernel<true>), grid, threads, 0, st, a, g);
        else hipLaunchKernelGGL((kv::rope_any_kernel<false>), grid, threads, 0, st, a, g);
    } else if (a.bf16) {
        if (a.r.inter) hipLaunchKernelGGL((kv::rope_kernel<true, true>), grid, threads, 0, st, a, g);
        else hipLaunchKernelGGL((kv::rope_kernel<true, false>), grid, threads, 0, st, a, g);
    } else {
        if (a.r.inter) hipLaunchKernelGGL((kv::rope_kernel<false, true>), grid, threads, 0, st, a, g);
        else hipLaunchKernelGGL((kv::rope_kernel<false, false>), grid, threads, 0, st, a, g);
    }
    return hipGetLastError();
}

namespace {
template <bool FP8, int FMT, bool G1>
void write_fmt(const KvWriteArgs& a, const kv::KvGrid& g, hipStream_t st)
{
    const dim3 grid(kv::groups(g.total)), threads(kv::THREADS);
    const bool two = g.per_row * 16 == a.c.dim;
    if (a.bf16 && g.waves) hipLaunchKernelGGL((kv::kv_write_kernel<FP8, FMT, G1, true, 2, true>), grid, threads, 0, st, a, g);
    else if (a.bf16 && two) hipLaunchKernelGGL((kv::kv_write_kernel<FP8, FMT, G1, true, 2, false>), grid, threads, 0, st, a, g);
    else if (a.bf16) hipLaunchKernelGGL((kv::kv_write_kernel<FP8, FMT, G1, true, 1, false>), grid, threads, 0, st, a, g);
    else if (g.waves) hipLaunchKernelGGL((kv::kv_write_kernel<FP8, FMT, G1, false, 2, true>), grid, threads, 0, st, a, g);
    else if (two) hipLaunchKernelGGL((kv::kv_write_kernel<FP8, FMT, G1, false, 2, false>), grid, threads, 0, st, a, g);
    else hipLaunchKernelGGL((kv::kv_write_kernel<FP8, FMT, G1, false, 1, false>), grid, threads, 0, st, a, g);
}
template <bool FP8, int FMT, bool G1>
void read_fmt(const KvReadArgs& a, const kv::KvGrid& g, hipStream_t st)
{
    const dim3 grid(kv::groups(g.total)), threads(kv::THREADS);
    if (a.bf16) hipLaunchKernelGGL((kv::kv_read_kernel<FP8, FMT, G1, true>), grid, threads, 0, st, a, g);
    else hipLaunchKernelGGL((kv::kv_read_kernel<FP8, FMT, G1, false>), grid, threads, 0, st, a, g);
}
}  // namespace

// F(element is FP8, format, both per-tensor scales are 1)
#define MXKV_BY_FORMAT(c, F)                                             \
    do {                                                                 \
        const bool g1 = (c).g[0] == 1.0f && (c).g[1] == 1.0f;            \
        switch (((c).fp8 ? 6 : 0) + 2 * (c).fmt + (g1 ? 1 : 0)) {        \
            case 0: F(false, FMT_E4M3, false); break;                    \
            case 1: F(false, FMT_E4M3, true); break;                     \
            case 2: F(false, FMT_UE5M3, false); break;                   \
            case 3: F(false, FMT_UE5M3, true); break;                    \
            case 4: F(false, FMT_E8M0, false); break;                    \
            case 5: F(false, FMT_E8M0, true); break;                     \
            case 6: F(true, FMT_E4M3, false); break;                     \
            case 7: F(true, FMT_E4M3, true); break;                      \
            case 8: F(true, FMT_UE5M3, false); break;                    \
            case 9: F(true, FMT_UE5M3, true); break;                     \
            case 10: F(true, FMT_E8M0, false); break;                    \
            case 11: F(true, FMT_E8M0, true); break;                     \
            default: return hipErrorInvalidValue;                        \
        }                                                                \
    } while (0)

hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t st)
{
    const uint32_t rope = a.r.table && a.r.rot ? ((a.r.inter ? a.r.rot % 8 == 0 : a.r.rot % 16 == 0) ? 1u : 2u) : 0u;
    // Two chunks a thread where every half row is whole blocks; a rotated key's halves are those of its
    // rotated part and of the rest.  With one a pair's other half comes from another thread: 22.1 us against 17.1
    // for 8192 x 8 heads of 128, FP8 25.0 against 20.2.
    const uint32_t rot = rope == 1 && !a.r.inter ? a.r.rot : 0u;
    const bool two = a.c.dim / 2 % a.c.block == 0 && rot / 2 % a.c.block == 0 && (a.c.dim - rot) / 2 % a.c.block == 0;
    kv::KvGrid g = kv::kv_grid(a.c, a.tokens, two ? 2 : 1, 2, true);
    const int64_t n = a.bf16 ? 8 : 4;
    for (int t = 0; t < 2; ++t) g.aligned |= (a.ld_t[t] % n == 0 && a.ld_h[t] % n == 0) ? 1u << t : 0u;
    g.rope = rope;
#define F(E, FMT, G1) write_fmt<E, FMT, G1>(a, g, st)
    MXKV_BY_FORMAT(a.c, F);
#undef F
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t st)
{
    const kv::KvGrid g = kv::kv_grid(a.c, a.tokens, 2, 5, false);
#define F(E, FMT, G1) read_fmt<E, FMT, G1>(a, g, st)
    MXKV_BY_FORMAT(a.c, F);
#undef F
    return hipGetLastError();
}

}  // namespace mxk
