// The key/value-cache entry points of include/mx_kv.h on the host, over stand-ins for the device launchers:
// how a rotation is cut into launches.  The kernels divide the numbers of a launch's elements by
// multiplication (mxk::FastDiv, exact below 2^31), so no launch may have more of them.
#include <cstdio>
#include <vector>

#include "mx_kv.h"
#include "mx_kv_internal.h"

namespace {

std::vector<mxk::RopeArgs> launches;
int fail_at = -1;  // the launch that reports an error
int bad = 0, done = 0;

void expect(bool ok, const char* what, int64_t a = 0, int64_t b = 0)
{
    ++done;
    if (ok) return;
    ++bad;
    std::printf("FAILED: %s (%lld, %lld)\n", what, (long long)a, (long long)b);
}

uint8_t* const X = reinterpret_cast<uint8_t*>(uintptr_t(1) << 40);
uint8_t* const Y = reinterpret_cast<uint8_t*>(uintptr_t(1) << 44);
int32_t* const POS = reinterpret_cast<int32_t*>(uintptr_t(1) << 46);
float* const TABLE = reinterpret_cast<float*>(uintptr_t(1) << 47);

// One call; its launches together have to be every token and head once, at their places.
void call(mx_dtype type, int64_t tokens, int64_t heads, int64_t dim, int rot, int64_t gap, size_t most_launches)
{
    const int64_t es = type == MX_BF16 ? 2 : 4, lxh = dim + gap, lxt = heads * lxh, lyh = dim + 2 * gap, lyt = heads * lyh;
    launches.clear();
    const mx_status st = mxkv_rope(X, type, tokens, heads, dim, lxt, lxh, POS, TABLE, 100, rot, 1, 1, Y, lyt, lyh, nullptr);
    expect(st == MX_OK, "status", st);
    expect(!launches.empty() && launches.size() <= most_launches, "number of launches", (int64_t)launches.size(), (int64_t)most_launches);
    int64_t covered = 0;
    for (const mxk::RopeArgs& a : launches) {
        const int64_t units = (int64_t)a.tokens * a.heads * a.dim;  // no kernel has more units than elements
        expect(units > 0 && units < (int64_t(1) << 31), "elements of a launch", units);
        covered += units;
        const int64_t t0 = rot ? a.r.positions - POS : ((const uint8_t*)a.x - X) / es / lxt, at = ((const uint8_t*)a.x - X) / es;
        const int64_t h0 = (at - t0 * lxt) / lxh;
        expect(t0 >= 0 && t0 + a.tokens <= tokens && h0 >= 0 && h0 + a.heads <= heads, "part of the call", t0, h0);
        expect((uint8_t*)a.x == X + (t0 * lxt + h0 * lxh) * es, "x", t0, h0);
        expect((uint8_t*)a.y == Y + (t0 * lyt + h0 * lyh) * es, "y", t0, h0);
        expect(a.bf16 == (type == MX_BF16) && (int64_t)a.dim == dim && a.ldx_t == lxt && a.ldx_h == lxh && a.ldy_t == lyt && a.ldy_h == lyh,
               "sizes");
        expect(a.r.inter && a.r.transpose && a.r.max_pos == 100 && (int)a.r.rot == rot, "rotation");
        for (const mxk::RopeArgs& b : launches) {  // parts do not overlap
            if (&a == &b) break;
            const int64_t u0 = rot ? b.r.positions - POS : ((const uint8_t*)b.x - X) / es / lxt, g0 = (((const uint8_t*)b.x - X) / es - u0 * lxt) / lxh;
            const bool apart = t0 + a.tokens <= u0 || u0 + b.tokens <= t0 || h0 + a.heads <= g0 || g0 + b.heads <= h0;
            expect(apart, "overlap", t0, u0);
        }
    }
    expect(covered == tokens * heads * dim, "elements covered", covered, tokens * heads * dim);
}

}  // namespace

namespace mxk {
hipError_t launch_rope(const RopeArgs& a, hipStream_t)
{
    launches.push_back(a);
    return (int)launches.size() - 1 == fail_at ? hipErrorInvalidValue : hipSuccess;
}
hipError_t launch_rope_table(const RopeTableArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_kv_write(const KvWriteArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_kv_read(const KvReadArgs&, hipStream_t) { return hipSuccess; }
bool kv_attention_fits(const KvAttnArgs&) { return true; }
size_t kv_attention_work_bytes(const KvAttnArgs&) { return 0; }
hipError_t launch_kv_attention(const KvAttnArgs&, hipStream_t) { return hipSuccess; }
}  // namespace mxk

int main()
{
    // what FastDiv promises and no more: at the end of its range, and a number past it that it gets wrong
    for (uint32_t d : {1u, 2u, 7u, 65u, 74u, 84u, 96u, 148u, 512u}) {
        const mxk::FastDiv f = mxk::FastDiv::make(d);
        for (uint32_t u : {0u, 1u, d - 1, d, 0x7FFFFFFFu, 0x7FFFFFFEu, 0x7FFFFFFFu - d}) expect(f.div(u) == u / d, "division", u, d);
    }
    expect(mxk::FastDiv::make(84).div(2818572289u) != 2818572289u / 84, "division past its range");

    call(MX_BF16, 8192, 64, 128, 128, 0, 1);
    call(MX_BF16, 1, 1, 1, 0, 3, 1);
    call(MX_BF16, 524288, 64, 96, 24, 0, 2);             // 3.2e9 elements, 84 units a row pair by pair
    call(MX_BF16, 524288, 64, 96, 24, 4, 2);
    call(MX_F32, 838860, 64, 80, 12, 0, 3);              // 4 294 963 200 elements, 74 units a row
    call(MX_F32, (int64_t(1) << 26) - 1, 1, 64, 64, 0, 3);
    call(MX_BF16, 1032444, 64, 65, 0, 1, 3);             // nothing rotates: a unit for each element
    call(MX_BF16, 1, 66076419, 65, 0, 1, 3);             // one token of very many heads
    call(MX_BF16, 3, 22025473, 65, 2, 1, 6);
    call(MX_BF16, 3, 700000000, 2, 2, 0, 6);
    for (int64_t tokens : {(int64_t(1) << 25) - 1, int64_t(1) << 25, (int64_t(1) << 25) + 1}) call(MX_BF16, tokens, 1, 64, 64, 8, 2);

    fail_at = 1;
    launches.clear();
    expect(mxkv_rope(X, MX_BF16, 524288, 64, 96, 6144, 96, POS, TABLE, 100, 24, 0, 0, Y, 6144, 96, nullptr) == MX_ERR_HIP, "a failed part");
    expect(launches.size() == 2, "a failed part ends the call", (int64_t)launches.size());
    std::printf("%s%d checks passed\n", bad ? "not " : "all ", done - bad);
    return bad ? 1 : 0;
}
