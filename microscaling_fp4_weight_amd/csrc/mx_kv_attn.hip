// mx_kv_attn.hip -- attention of new tokens over the quantized key/value cache.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q . k_j - max_j),   lse = max + log sum p
//
// over the keys a token sees: all cached ones, and the new ones that its mask row names.  Keys
// are visited once, with a running maximum m and sum l: on a larger maximum m' the sums so far
// are multiplied by exp(m - m').
#include <cmath>

#include "mx_kv_attn.h"

namespace mxk {
namespace kv {

// Whether new token i sees token j (j < held)
__device__ __forceinline__ bool sees(const KvAttnArgs& a, const Seq& s, uint32_t b, uint32_t i, uint32_t j)
{
    if (j < s.cached) return true;
    const uint32_t k = j - s.cached;
    return a.mask ? a.mask[b * a.ldm_b + i * a.ldm_r + k] != 0 : k <= i;
}

// Any head size up to 512: a workgroup takes one row (new token, query head), its four waves
// every fourth token, a lane the element pairs 2 lane + 128 i of the head.  Every row reads its tokens again, and
// six shuffles a token sum its score: what bounds it is that chain, not memory.  p stays in fp32.
template <bool FP8, int FMT>
__global__ __launch_bounds__(256) void attn_row_kernel(KvAttnArgs a, FastDiv page_div)
{
    constexpr int NP = 4;
    __shared__ float part[4][512];
    __shared__ float pm[4], pl[4];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t row = blockIdx.x;
    const uint32_t h = row % a.q_heads, bi = row / a.q_heads, i = bi % a.nt, b = bi / a.nt;
    const uint32_t hk = h / (a.q_heads / a.c.heads);
    const Seq s = seq_of(a, b);
    const uint16_t* qp = a.q + b * a.ldq_b + i * a.ldq_t + h * a.ldq_h;
    const float qs = a.scale * a.c.g[0] * LOG2E;  // scores in powers of two
    f32x2 q[NP], o[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const uint32_t d = 2 * lane + 128 * k;
        q[k] = o[k] = f32x2{0.f, 0.f};
        if (d < a.c.dim) q[k] = f32x2{u2f((uint32_t)qp[d] << 16) * qs, u2f((uint32_t)qp[d + 1] << 16) * qs};
    }
    auto pair = [&](int t, uint64_t r, int k) -> f32x2 {
        const uint32_t d = 2 * lane + 128 * k;
        if (d >= a.c.dim) return f32x2{0.f, 0.f};
        f32x2 e;
        if constexpr (FP8)
            e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(*reinterpret_cast<const uint16_t*>(a.c.codes[t] + r * a.c.dim + d), 1.0f, false);
        else
            e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(a.c.codes[t][r * (a.c.dim / 2) + d / 2], 1.0f, 0);
        const float f = nan_scale<FMT == FMT_E8M0>(scale_value_f32<FMT>(a.c.scales[t][r * (a.c.dim / a.c.block) + d / a.c.block]));
        return f32x2{e.x * f, e.y * f};
    };
    float m = -INFINITY, l = 0.f;
    const uint32_t held = i < s.fresh ? s.held : 0u;
    for (uint32_t j = wave; j < held; j += 4) {
        if (!sees(a, s, b, i, j)) continue;
        const uint32_t e = page_div.div(j);
        const int32_t page = a.table[b * a.ld_table + e];
        if (page < 0 || (uint32_t)page >= a.c.num_pages) continue;
        const uint64_t r = ((uint64_t)page * a.c.heads + hk) * a.c.page + (j - e * a.c.page);
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const f32x2 v = pair(0, r, k);
            x += q[k].x * v.x + q[k].y * v.y;
        }
        for (int off = 32; off; off >>= 1) x += __shfl_xor(x, off);
        // while no score is above -inf all weights are 0
        const float top = fmaxf(m, x), base = top == -INFINITY ? 0.f : top, f = exp2f(m - base), p = exp2f(x - base);
        m = top;
        l = l * f + p;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const f32x2 v = pair(1, r, k);
            o[k].x = o[k].x * f + p * v.x;
            o[k].y = o[k].y * f + p * v.y;
        }
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        part[wave][2 * lane + 128 * k] = o[k].x;
        part[wave][2 * lane + 128 * k + 1] = o[k].y;
    }
    if (lane == 0) {
        pm[wave] = m;
        pl[wave] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.f, f[4];
    for (int w = 0; w < 4; ++w) top = fmaxf(top, pm[w]);
    for (int w = 0; w < 4; ++w) {
        f[w] = pl[w] == 0.f ? 0.f : exp2f(pm[w] - top);  // a sum of NaN stays NaN
        sum += pl[w] * f[w];
    }
    const bool some = sum != 0.f;
    const float inv = some ? a.c.g[1] / sum : 0.f;
    for (uint32_t d = threadIdx.x; d < a.c.dim; d += 256) {
        float x = 0.f;
        for (int w = 0; w < 4; ++w) x += part[w][d] * f[w];  // NaN of a wave counts at any weight
        reinterpret_cast<__bf16*>(a.out)[(uint64_t)row * a.c.dim + d] = (__bf16)(some ? x * inv : 0.f);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = some ? top * LN2 + logf(sum) : -INFINITY;
}

}  // namespace kv

namespace {

// workgroups that run at once, at most; workgroups of a team
constexpr uint32_t MOST_GROUPS = 256 * 4, MOST_TEAM = 16;

bool on_matrix_cores(const KvPool& c) { return c.dim == 64 || c.dim == 128 || c.dim == 256; }

// 16-row tiles that a workgroup works on together: as many as the rows fill, since they share a token's decoded
// key and value, up to what the registers hold: 4096 sums of a wave's rows (8192 spill: 1209 us against 462 for
// 512 rows of a head of 128 over 131072 tokens)
int row_tile(const KvAttnArgs& a)
{
    const uint32_t rows = a.nt * (a.q_heads / a.c.heads);
    const int most = 256 / (int)a.c.dim;
    const int nq = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
    return nq < most ? nq : most;
}

kv::AttnPlan plan_of(const KvAttnArgs& a)
{
    kv::AttnPlan p{};
    const int nq = row_tile(a);
    p.group = a.q_heads / a.c.heads;
    p.row_tiles = (a.nt * p.group + 16 * nq - 1) / (16 * nq);
    // a head's tiles, or an equal part of them
    const uint32_t parts = (p.row_tiles + MOST_TEAM - 1) / MOST_TEAM;
    p.team = parts ? (p.row_tiles + parts - 1) / parts : 1;
    // What beginning and ending a segment costs, in steps.  64 sequences of up to 4096 FP4 tokens, one row tile: 47.1,
    // 45.0 and 46.0 us with 1, 2 and 3; 8 trees over up to 16384 FP8 tokens: 87, 81, 79 and 83 with 2, 3, 4 and 6.
    p.begin = nq == 1 ? 2 : 4;
    const uint64_t longest = ((uint64_t)a.max_pages * a.c.page + kv::STEP - 1) / kv::STEP;
    p.most = (uint64_t)a.batch * ((a.c.heads * p.row_tiles + p.team - 1) / p.team) * ((longest ? longest : 1) + p.begin);
    p.page_div = FastDiv::make(a.c.page);
    p.group_div = FastDiv::make(p.group);
    while ((1u << p.block_shift) < a.c.block) ++p.block_shift;
    while ((a.c.block << p.scale_shift) < a.c.dim) ++p.scale_shift;
    // not 0, so that a score of -inf (a key that is not seen) stays that; any other product counts, however small,
    // since keys may be as large as it is small
    p.c = fabsf(a.scale) * a.c.g[0] * kv::LOG2E;
    if (p.c == 0.f) p.c = 0x1p-149f;
    p.flip = a.scale < 0.f ? 0x80008000u : 0u;
    p.s_bits = a.c.fmt == FMT_E4M3 ? 0x7Fu : 0xFFu;
    p.s_sign = a.c.fmt == FMT_E4M3 ? 0x80u : 0u;
    p.s_mul = a.c.fmt == FMT_E4M3 ? 0x1p120f : 0x1p112f;
    return p;
}

}  // namespace

bool kv_attention_fits(const KvAttnArgs& a)
{
    if (!on_matrix_cores(a.c)) return true;
    const uint64_t longest = ((uint64_t)a.max_pages * a.c.page + kv::STEP - 1) / kv::STEP;
    const kv::AttnPlan p = plan_of(a);
    return (longest + p.begin + 1) * a.batch < (uint64_t(1) << 31) / (a.c.heads * p.row_tiles);
}

size_t kv_attention_work_bytes(const KvAttnArgs& a)
{
    if (!on_matrix_cores(a.c)) return 0;
    const size_t rows = 16 * (size_t)row_tile(a);
    const kv::AttnPlan p = plan_of(a);
    const uint64_t most = p.most * p.team, groups = most < MOST_GROUPS ? most : MOST_GROUPS;
    return kv::meta_bytes(a.batch) + 2 * groups * (rows * a.c.dim + 2 * rows) * sizeof(float);
}

hipError_t launch_kv_attention(const KvAttnArgs& args, hipStream_t st)
{
    KvAttnArgs a = args;
    if (on_matrix_cores(a.c)) {
        const kv::AttnPlan p = plan_of(a);
        a.q_aligned = a.ldq_b % 8 == 0 && a.ldq_t % 8 == 0 && a.ldq_h % 8 == 0;
        const int nq = row_tile(a);
        switch (a.c.dim) {
            case 64: return launch_attn_64(a, p, nq, st);
            case 128: return launch_attn_128(a, p, nq, st);
            default: return launch_attn_256(a, p, nq, st);
        }
    }
    const dim3 grid(a.batch * a.nt * a.q_heads), threads(256);
    const FastDiv pd = FastDiv::make(a.c.page);
    switch ((a.c.fp8 ? 3 : 0) + a.c.fmt) {
        case 0: hipLaunchKernelGGL((kv::attn_row_kernel<false, FMT_E4M3>), grid, threads, 0, st, a, pd); break;
        case 1: hipLaunchKernelGGL((kv::attn_row_kernel<false, FMT_UE5M3>), grid, threads, 0, st, a, pd); break;
        case 2: hipLaunchKernelGGL((kv::attn_row_kernel<false, FMT_E8M0>), grid, threads, 0, st, a, pd); break;
        case 3: hipLaunchKernelGGL((kv::attn_row_kernel<true, FMT_E4M3>), grid, threads, 0, st, a, pd); break;
        case 4: hipLaunchKernelGGL((kv::attn_row_kernel<true, FMT_UE5M3>), grid, threads, 0, st, a, pd); break;
        case 5: hipLaunchKernelGGL((kv::attn_row_kernel<true, FMT_E8M0>), grid, threads, 0, st, a, pd); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace mxk
