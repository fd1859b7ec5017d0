// ffn_room_driver.cpp — the gated block's host side (csrc/ffn.hip) over many sizes,
// alignments and widths, without a GPU: every launch is caught and what it would
// read and write is checked against the workspace that ffn_workspace_bytes gives
// and against what the kernels ask of their operands. Built with the host side
// under AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_ffn_room.py.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "../../weight_only_quantized_qgemv_amd/csrc/ffn.hip"

namespace {

using addr = uintptr_t;
constexpr addr WS = addr(1) << 44, USER = addr(1) << 45;   // stand-ins, never dereferenced
size_t ws_bytes = 0;
int failures = 0, launches = 0;
qp::FfnArgs cur;
char what[256];

void fail(const char* why)
{
    if (++failures <= 20)
        std::fprintf(stderr, "FAIL %s: %s\n", what, why);
}
addr at(const void* p) { return reinterpret_cast<addr>(p); }
bool in_ws(const void* p) { return at(p) >= WS && at(p) < USER; }
// A range written (or read) by a launch: inside the workspace where it starts there.
void range(const void* p, size_t bytes, bool must, const char* why)
{
    if (must && !in_ws(p))
        return fail(why);
    if (in_ws(p) && (at(p) < WS || at(p) + bytes > WS + ws_bytes))
        fail(why);
}
size_t es() { return cur.dt == qp::DT_F32 ? 4 : 2; }

// gate_up.hip's own choice, by the operands that its kernels take.
hipError_t gate_up_stub(const qp::GateUpArgs& a, bool* done)
{
    ++launches;
    const int64_t G = int64_t(1) << 31;
    *done = false;
    if (a.dt == qp::DT_F32 || at(a.x) % 16 != 0 || a.N * (a.K * a.bits / 8) >= G || a.N * (a.K / a.gs) * 2 >= G - 4 ||
        a.M * a.N * 2 >= G || a.M * a.K * 2 >= G || a.K >= (1 << 30))
        return hipSuccess;
    if (a.M > 16 && (a.K % 64 != 0 || (at(a.gate.scales) | at(a.gate.biases) | at(a.up.scales) | at(a.up.biases)) % 4))
        return hipSuccess;
    *done = true;
    range(a.h, (size_t)a.M * a.N * 2, true, "h");
    range(a.x, (size_t)a.M * a.K * 2, false, "x");
    return hipSuccess;
}
hipError_t split_stub(const qp::FfnSplitArgs& a)
{
    ++launches;
    const qp::FfnSplit& p = a.plan;
    if (at(a.x) % 16 != 0 || a.K % 64 != 0 || (int64_t)p.splits * p.per_split * 64 < a.K || p.splits < 1)
        fail("split operands");
    if (a.M * a.K * 2 >= (int64_t(1) << 31) || a.N * (a.wk * a.bits / 8) >= (int64_t(1) << 31) ||
        a.M * a.N * 4 * a.nmat >= (int64_t(1) << 31))
        fail("split offsets");
    const bool ends = 4 * a.bits % (a.bits == 3 ? 12 : 16) == 0;
    if (a.wk != a.K && (a.wk + 32 != a.K || !ends))
        fail("codes end inside a piece");
    range(a.partial, (size_t)p.splits * a.nmat * a.M * a.N * 4, true, "split sums");
    range(a.x, (size_t)a.M * a.K * 2, a.wk != a.K, "split x");
    for (int t = 0; t < a.nmat; ++t) {
        if ((at(a.w[t].scales) | at(a.w[t].biases)) % 4 != 0)
            fail("split scales");
        range(a.w[t].scales, (size_t)a.N * (a.K / a.gs) * 2, false, "split scales");
        range(a.w[t].biases, (size_t)a.N * (a.K / a.gs) * 2, false, "split biases");
        range(a.w[t].wq, (size_t)a.N * (a.wk * a.bits / 8), false, "split codes");
        // Copies lie behind the sums.
        for (const void* q : {a.w[t].scales, a.w[t].biases, (const void*)a.w[t].wq})
            if (in_ws(q) && a.K != cur.D && a.K != cur.F &&
                at(q) < at(a.partial) + (size_t)p.splits * a.nmat * a.M * a.N * 4)
                fail("copies under the sums");
    }
    return hipSuccess;
}
hipError_t any_stub(const qp::FfnAnyArgs& a)
{
    ++launches;
    if (a.partial != nullptr)
        range(a.partial, ((size_t)(a.plan.splits - 1) * a.partial_stride + (size_t)a.M * a.N) * 4, true, "sums");
    else if (a.plan.splits != 1)
        fail("pieces without sums");
    else
        range(a.y, (size_t)a.M * a.N * es(), false, "product");
    return hipSuccess;
}
hipError_t product_stub(const qp::GemvArgs& a, bool tiles)
{
    ++launches;
    if (tiles && (a.K % 64 != 0 || (at(a.scales) | at(a.biases)) % 4 != 0 || a.M * a.K * 2 >= (int64_t(1) << 31) ||
                  a.M * a.N * 2 >= (int64_t(1) << 31) || a.N * (a.K * a.bits / 8) >= (int64_t(1) << 31)))
        fail("tile product operands");
    range(a.y, (size_t)a.M * a.N * es(), false, "product");
    range(a.x, (size_t)a.M * a.K * es(), false, "product x");
    return hipSuccess;
}

} // namespace

namespace qp {
#define STUBS(B)                                                                                            \
    hipError_t launch_gate_up_b##B(const GateUpArgs& a, hipStream_t, bool* d) { return gate_up_stub(a, d); } \
    hipError_t launch_ffn_split_b##B(const FfnSplitArgs& a, hipStream_t) { return split_stub(a); }           \
    hipError_t launch_ffn_any_b##B(const FfnAnyArgs& a, hipStream_t) { return any_stub(a); }
STUBS(2)
STUBS(3)
STUBS(4)
STUBS(6)
STUBS(8)
hipError_t launch_qgemv(const GemvArgs& a, hipStream_t) { return product_stub(a, false); }
hipError_t launch_qgemm(const GemvArgs& a, hipStream_t) { return product_stub(a, true); }
hipError_t launch_fill_zero(void*, int, int64_t, hipStream_t) { return ++launches, hipSuccess; }
} // namespace qp

// The launches of ffn.hip's own kernels end here.
extern "C" hipError_t hipLaunchKernel(const void* f, dim3, dim3, void** args, size_t, hipStream_t)
{
    ++launches;
    if (f == reinterpret_cast<const void*>(&qp::ffn_pad_kernel)) {
        const qp::PadArgs& p = *static_cast<const qp::PadArgs*>(args[0]);
        for (int i = 0; i < qp::PadArgs::MAX && p.in[i] != nullptr; ++i) {
            range(p.out[i], (size_t)p.rows[i] * p.pairs[i] * 4, true, "copy");
            if (at(p.out[i]) % 16 != 0 || p.rows[i] * p.pairs[i] >= (int64_t(1) << 30) || 2 * (int64_t)p.pairs[i] < p.cols[i])
                fail("copy shape");
        }
    } else if (f != reinterpret_cast<const void*>(&qp::ffn_gate_kernel)) {   // a join: partial, splits, total
        const void* partial = *static_cast<void**>(args[0]);
        const int splits = *static_cast<int*>(args[1]);
        const int64_t total = *static_cast<int64_t*>(args[2]);
        range(partial, (size_t)splits * total * 4, true, "joined sums");
    }
    return hipSuccess;
}
extern "C" hipError_t hipGetLastError() { return hipSuccess; }

int main()
{
    const int64_t ms[] = {1, 2, 3, 16, 17, 33, 64, 65, 128, 129, 257, 1000, 2048, 18689, 65280, 70000, 300000, 1 << 24};
    const int64_t dims[][2] = {{32, 32}, {32, 544}, {96, 160}, {256, 448}, {1120, 352}, {2080, 5600}, {4096, 14336},
                               {8256, 64}, {64, 16384}, {17408, 128}, {46336, 46304}, {46304, 46368}, {65536, 32768},
                               {131072, 65536}, {1 << 20, 64}, {2097184, 32}, {32, 4 << 20}, {67108832, 32}};
    for (int64_t m : ms)
        for (auto& df : dims)
            for (int dt : {qp::DT_F32, qp::DT_F16, qp::DT_BF16})
                for (int bits : {2, 3, 4, 6, 8})
                    for (int gs : {32, 64, 128})
                        for (int off = 0; off < 4; ++off) {
                            const int64_t d = df[0], f = df[1];
                            if (d % gs != 0 || f % gs != 0 || m * std::max(d, f) > (int64_t(1) << 34))
                                continue;
                            std::snprintf(what, sizeof what, "m=%lld d=%lld f=%lld dt=%d bits=%d gs=%d off=%d",
                                          (long long)m, (long long)d, (long long)f, dt, bits, gs, off);
                            ws_bytes = qp::ffn_workspace_bytes(m, d, f, dt);
                            qp::FfnArgs a{};
                            auto user = [&](int i, bool shifted) { return reinterpret_cast<void*>(USER + i * (addr(1) << 42) + (shifted ? 2 : 0)); };
                            a.x = user(0, off & 1);
                            a.dt = dt; a.act = 0; a.M = m; a.D = d; a.F = f;
                            auto w = [&](int i) {
                                return qp::QWeight{static_cast<const uint32_t*>(user(i, false)), user(i + 1, off & 2), user(i + 2, off & 2)};
                            };
                            a.gate = w(1); a.up = w(4); a.down = w(7);
                            a.bits = bits; a.gs = gs;
                            if (off == 1) {
                                a.saved[0] = user(10, false);
                                a.saved[1] = user(12, true);
                            }
                            a.y = user(14, off & 1);
                            a.workspace = reinterpret_cast<void*>(WS);
                            cur = a;
                            if (qp::launch_ffn(a, nullptr) != hipSuccess)
                                fail("status");
                        }
    // Sizes at the ends: no overflow on the way, where m d and m f stay below 2^57
    // (the entry refuses others).
    auto below = [](int64_t m, int64_t n) { return m == 0 || n <= INT64_MAX / 64 / m; };
    for (int64_t a : {int64_t(0), int64_t(1), int64_t(INT32_MAX), INT64_MAX / 64, INT64_MAX})
        for (int64_t b : {int64_t(0), int64_t(64), int64_t(INT32_MAX), INT64_MAX})
            for (int64_t c : {int64_t(0), int64_t(64), INT64_MAX / 4096, INT64_MAX})
                for (int dt : {qp::DT_F32, qp::DT_F16})
                    if (below(a, b) && below(a, c))
                        (void)qp::ffn_workspace_bytes(a, b, c, dt);
    std::printf("%d launches\n", launches);
    if (failures == 0)
        std::puts("all inside the workspace");
    return failures != 0;
}
