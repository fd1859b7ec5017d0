// ffn.hip — the dense gated feed-forward block over packed weights:
//   h = act(x Wg^T) * (x Wu^T),   y = h Wd^T
// (the block of qgemv_moe_ffn, ferrum-kernels src/stacked_expert.rs, with one
// set of weights for every row). h comes from the fp32 projections and is rounded
// once to the activations' type, because it is the down projection's operand on
// 16-bit instructions: with y's own rounding an error of 0.0023 of y's size in
// bf16 against 64 bits (one row), where one rounding gives 0.0016; the tile
// kernels' rounding of the weights makes it 0.0036.
#include <algorithm>

#include "act.hpp"
#include "common.hpp"
#include "model_ops.hpp"
#include "xgrad.hpp"

namespace qp {

namespace {

// fp32: h[i] = act(g[i]) u[i]; h may be g's own memory. (16-bit projections are
// closed from their sums, before any rounding.)
__global__ __launch_bounds__(256) void ffn_gate_kernel(const float* g, const float* u, int act, int64_t n, float* h)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        h[i] = act_f32(act, g[i]) * u[i];
}

hipError_t gate(const FfnArgs& a, const void* g, const void* u, void* h, hipStream_t st)
{
    const int64_t n = a.M * a.F;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 16384);
    hipLaunchKernelGGL(ffn_gate_kernel, dim3(blocks), dim3(256), 0, st, static_cast<const float*>(g),
                       static_cast<const float*>(u), a.act, n, static_cast<float*>(h));
    return hipGetLastError();
}

// The sums of a product in pieces: stored, or (gated) both products' sums
// closed into h, and kept where a backward pass follows. Partial sums
// [split][matrix][total].
template <int DT, bool GATED>
__global__ __launch_bounds__(256) void ffn_join_kernel(const float* __restrict__ partial, int splits, int64_t total,
                                                       int act, void* saved_g, void* saved_u, void* out)
{
    constexpr int NMAT = GATED ? 2 : 1;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const float v = sum_splits(partial, splits, NMAT * total, i);
        if constexpr (GATED) {
            const float u = sum_splits(partial + total, splits, NMAT * total, i);
            if (saved_g != nullptr) {
                store_elem<DT>(saved_g, i, v);
                store_elem<DT>(saved_u, i, u);
            }
            store_elem<DT>(out, i, act_f32(act, v) * u);
        } else {
            store_elem<DT>(out, i, v);
        }
    }
}

template <bool GATED>
hipError_t join(const FfnArgs& a, const float* partial, int splits, int64_t total, void* out, hipStream_t st)
{
    const unsigned blocks = (unsigned)std::min<int64_t>((total + 255) / 256, 16384);
    void* const sg = GATED ? a.saved[0] : nullptr;
    void* const su = GATED ? a.saved[1] : nullptr;
    if (!GATED && a.dt == DT_F32)
        hipLaunchKernelGGL((ffn_join_kernel<DT_F32, false>), dim3(blocks), dim3(256), 0, st, partial, splits, total,
                           a.act, sg, su, out);
    else if (a.dt == DT_F16)
        hipLaunchKernelGGL((ffn_join_kernel<DT_F16, GATED>), dim3(blocks), dim3(256), 0, st, partial, splits, total,
                           a.act, sg, su, out);
    else
        hipLaunchKernelGGL((ffn_join_kernel<DT_BF16, GATED>), dim3(blocks), dim3(256), 0, st, partial, splits, total,
                           a.act, sg, su, out);
    return hipGetLastError();
}

constexpr int64_t k2GB = int64_t(1) << 31;

// Whether the tile kernels' 32-bit offsets reach a weight [n, k]; and whether they
// might not, filled up or not, for the plans that know only the sizes (8-bit codes
// are the widest).
bool offsets_reach(int64_t n, int64_t k, int bits, int gs)
{
    return n * (k * bits / 8) < k2GB && n * (k / gs) * 2 < k2GB - 4;
}
bool huge_weight(int64_t n, int64_t k) { return k + 32 >= k2GB / (n + 32); }

// Whether ffn_any's kernel takes a product: the decode kernels, which qmatmul
// runs such shapes on, stream the weights once for every few rows (fp32, 4096 x
// 14336, 4-bit, the three products: 1 row 131 us against 152, 2 rows 227 against
// 152, 32 rows 3890 against 155).
bool any_product(const FfnArgs& a, int64_t k, const QWeight& w, int64_t n)
{
    if (a.dt == DT_F32)
        return a.M > 1;
    const uintptr_t sb = reinterpret_cast<uintptr_t>(w.scales) | reinterpret_cast<uintptr_t>(w.biases);
    return a.M > 16 && (k % 64 != 0 || sb % 4 != 0 || !offsets_reach(n, k, a.bits, a.gs));
}

// One product on ffn_any's kernel: its fp32 sums to partial, or (null) y.
hipError_t any_kernel(const FfnArgs& a, const void* x, int64_t k, const QWeight& w, int64_t n, const FfnSplit& plan,
                      float* partial, int64_t stride, void* y, hipStream_t st)
{
    FfnAnyArgs g{x, a.dt, a.M, k, n, w, a.gs, plan, partial, stride, y};
    switch (a.bits) {
    case 2: return launch_ffn_any_b2(g, st);
    case 3: return launch_ffn_any_b3(g, st);
    case 4: return launch_ffn_any_b4(g, st);
    case 6: return launch_ffn_any_b6(g, st);
    case 8: return launch_ffn_any_b8(g, st);
    }
    return hipErrorInvalidValue;
}

// y = x W^T: ffn_any's kernel, or qmatmul's.
hipError_t product(const FfnArgs& a, const void* x, int64_t k, const QWeight& w, int64_t n, float* partial, void* y,
                   hipStream_t st)
{
    if (any_product(a, k, w, n)) {
        const FfnSplit plan = ffn_any_plan(a.M, k, n);
        const bool parts = plan.splits > 1;
        if (hipError_t e = any_kernel(a, x, k, w, n, plan, parts ? partial : nullptr, a.M * n, y, st);
            e != hipSuccess || !parts)
            return e;
        return join<false>(a, partial, plan.splits, a.M * n, y, st);
    }
    GemvArgs g{x, a.dt, a.M, k, n, w.wq, w.scales, w.biases, a.bits, a.gs, y};
    return a.M <= 16 ? launch_qgemv(g, st) : launch_qgemm(g, st);
}

// The gate and up products of 16-bit operands on ffn_any's kernel, as fp32 sums
// closed into h: rounded nowhere before it, as in the fused kernels.
hipError_t any_gate_up(const FfnArgs& a, float* partial, void* h, hipStream_t st)
{
    const FfnSplit plan = ffn_any_plan(a.M, a.D, a.F);
    const int64_t total = a.M * a.F;
    if (hipError_t e = any_kernel(a, a.x, a.D, a.gate, a.F, plan, partial, 2 * total, nullptr, st); e != hipSuccess)
        return e;
    if (hipError_t e = any_kernel(a, a.x, a.D, a.up, a.F, plan, partial + total, 2 * total, nullptr, st); e != hipSuccess)
        return e;
    return join<true>(a, partial, plan.splits, total, h, st);
}
size_t any_gate_up_bytes(int64_t m, int64_t d, int64_t f)
{
    return (size_t)ffn_any_plan(m, d, f).splits * 2 * (size_t)m * (size_t)f * 4;
}

// Rows of 16-bit elements copied to longer rows, zeros behind: array blockIdx.y,
// two elements a thread.
struct PadArgs {
    static constexpr int MAX = 7;   // x, and two matrices' scales, biases and codes
    const uint16_t* in[MAX];
    uint32_t* out[MAX];
    int64_t rows[MAX];
    uint32_t cols[MAX], pairs[MAX];   // elements in a row, pairs in an output row
};
__global__ __launch_bounds__(256) void ffn_pad_kernel(PadArgs a)
{
    const int j = (int)blockIdx.y;
    const uint32_t pairs = a.pairs[j], cols = a.cols[j];
    const int64_t total = a.rows[j] * pairs;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const uint32_t r = (uint32_t)i / pairs, c = 2 * ((uint32_t)i - r * pairs);   // total is below 2^30
        const uint16_t* const p = a.in[j] + (int64_t)r * cols + c;
        const uint32_t lo = c < cols ? p[0] : 0u, hi = c + 1 < cols ? p[1] : 0u;
        a.out[j][i] = lo | (hi << 16);
    }
}

// Arrays copied side by side into a workspace, in one launch.
struct Copies {
    PadArgs pad{};
    char* to;
    int arrays = 0;
    int64_t most = 0;
    // rows of cols 16-bit elements to rows of cols_p (even); returns where they will be.
    const void* add(const void* from, int64_t rows, int64_t cols, int64_t cols_p)
    {
        pad.in[arrays] = static_cast<const uint16_t*>(from);
        pad.out[arrays] = reinterpret_cast<uint32_t*>(to);
        pad.rows[arrays] = rows;
        pad.cols[arrays] = (uint32_t)cols;
        pad.pairs[arrays++] = (uint32_t)(cols_p / 2);
        most = std::max(most, rows * (cols_p / 2));
        const void* const at = to;
        to += up16((size_t)rows * (size_t)cols_p * 2);
        return at;
    }
    hipError_t run(hipStream_t st) const
    {
        if (arrays == 0)
            return hipSuccess;
        hipLaunchKernelGGL(ffn_pad_kernel, dim3((unsigned)std::min<int64_t>((most + 255) / 256, 4096), (unsigned)arrays),
                           dim3(256), 0, st, pad);
        return hipGetLastError();
    }
};

// Whether a row of 64 n + 32 codes ends inside one of the pieces (16 bytes, at 3
// bits 12) that the tile kernel takes a step's codes in: at 2 and 6 bits.
constexpr bool ends_in_piece(int bits) { return 4 * bits % (bits == 3 ? 12 : 16) != 0; }

// A product in pieces where the plan allows it.
template <bool GATED>
hipError_t split_product(const FfnArgs& a, const void* x, int64_t k, const QWeight& w0, const QWeight& w1, int64_t n,
                         float* partial, void* out, hipStream_t st, bool* done)
{
    constexpr int NMAT = GATED ? 2 : 1;
    FfnSplitArgs s{x, a.dt, a.M, k, n, k, {w0, w1}, NMAT, a.bits, a.gs, ffn_split(a.M, k, n, NMAT, a.dt), partial};
    const FfnSplit& p = s.plan;
    const uintptr_t sb = reinterpret_cast<uintptr_t>(w0.scales) | reinterpret_cast<uintptr_t>(w0.biases) |
                         reinterpret_cast<uintptr_t>(w1.scales) | reinterpret_cast<uintptr_t>(w1.biases);
    if (p.per_split == 0 || (p.kp == 0 && sb % 4 != 0) || !offsets_reach(n, p.kp > 0 ? p.kp : k, a.bits, a.gs))
        return hipSuccess;
    if (p.kp > 0) {
        const int64_t kk = p.kp, groups = kk / a.gs;
        Copies c;
        c.to = reinterpret_cast<char*>(partial) + up16(p.partial_bytes);
        s.x = c.add(x, a.M, k, kk);
        s.K = kk;
        for (int t = 0; t < NMAT; ++t) {
            s.w[t].scales = c.add(s.w[t].scales, n, k / a.gs, groups);
            s.w[t].biases = c.add(s.w[t].biases, n, k / a.gs, groups);
            // Left where they lie, the last row's last piece would reach past
            // the codes' end. As 16-bit elements: 32 codes are 4, 12 of them.
            if (ends_in_piece(a.bits)) {
                s.w[t].wq = static_cast<const uint32_t*>(c.add(s.w[t].wq, n, k * a.bits / 16, kk * a.bits / 16));
                s.wk = kk;
            }
        }
        if (hipError_t e = c.run(st); e != hipSuccess)
            return e;
    }
    hipError_t e = hipErrorInvalidValue;
    switch (a.bits) {
    case 2: e = launch_ffn_split_b2(s, st); break;
    case 3: e = launch_ffn_split_b3(s, st); break;
    case 4: e = launch_ffn_split_b4(s, st); break;
    case 6: e = launch_ffn_split_b6(s, st); break;
    case 8: e = launch_ffn_split_b8(s, st); break;
    }
    if (e != hipSuccess)
        return e;
    *done = true;
    return join<GATED>(a, partial, p.splits, a.M * n, out, st);
}

// Scales and biases off a 4-byte address, for the tile kernels.
void align_scales(Copies& c, QWeight& w, int64_t count)
{
    auto move = [&](const void*& p) {
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0)
            p = c.add(p, 1, count, count + count % 2);
    };
    move(w.scales);
    move(w.biases);
}

hipError_t gate_up(const GateUpArgs& a, hipStream_t st, bool* done)
{
    switch (a.bits) {
    case 2: return launch_gate_up_b2(a, st, done);
    case 3: return launch_gate_up_b3(a, st, done);
    case 4: return launch_gate_up_b4(a, st, done);
    case 6: return launch_gate_up_b6(a, st, done);
    case 8: return launch_gate_up_b8(a, st, done);
    }
    return hipErrorInvalidValue;
}

} // namespace

// Tiles of 64 x 256 up to 128 rows, 256 x 128 beyond, and as many pieces as fill
// the 256 CUs once, at least four steps each. 4096 x 14336, 4-bit, the whole
// block, without pieces and with: 64 rows 254 and 70 us, 256 rows 277 and 124, 512
// rows 354 and 205. Filling the CUs twice: 64 rows 83 us.
// A contraction of whole 32-wide groups but not whole 64-wide steps (groups of 32
// then) is filled up with zeros: x, the scales and the biases in a copy, the codes
// where they lie, the next row's times zero, or (2 and 6 bits) in a copy too
// (5600 x 2080, 4-bit, bf16, 253 rows 222 us on ffn_any's kernel, 79 so; 2048 rows
// 1354 and 280; at 6 bits, with the codes' copy, 96 and 311). Below 64 the weights'
// roundings do not average out, and ffn_any's kernel takes the product. The room
// is for 6-bit codes: the sizes alone decide it.
FfnSplit ffn_split(int64_t m, int64_t k, int64_t n, int nmat, int dt)
{
    FfnSplit p{m <= 128 ? 64 : 256, 1, 0, 0, 0, 0};
    const bool pad = k % 64 == 32 && k > 64;
    if (dt == DT_F32 || m <= 16 || (k % 64 != 0 && !pad) || k == 0 || n == 0 || m * n * 4 * nmat >= k2GB ||
        m * (k + 32) * 2 >= k2GB)
        return p;
    const int64_t cols = p.tile == 64 ? 256 : 128;
    const int64_t tiles = ((m + p.tile - 1) / p.tile) * ((n * nmat + cols - 1) / cols), steps = (k + 63) / 64;
    const int64_t splits = std::min(256 / tiles, steps / 4);
    if (splits <= 1 && !pad)
        return p;
    p.per_split = (int)((steps + std::max<int64_t>(splits, 1) - 1) / std::max<int64_t>(splits, 1));
    p.splits = (int)((steps + p.per_split - 1) / p.per_split);
    p.partial_bytes = (size_t)p.splits * (size_t)nmat * (size_t)m * (size_t)n * 4;
    if (pad) {
        p.kp = k + 32;
        p.pad_bytes = up16((size_t)m * (size_t)p.kp * 2) +
                      (size_t)nmat * (2 * up16((size_t)n * (size_t)(p.kp / 32) * 2) + up16((size_t)n * (size_t)(p.kp / 4 * 3)));
    }
    return p;
}

FfnSplit ffn_any_plan(int64_t m, int64_t k, int64_t n)
{
    // The tile that the rows fit: 33 rows of 4096 x 14336, 4-bit, fp32, 256 us with
    // tiles of 64, 459 with tiles of 128. The pieces that an estimate, in us,
    // finds quickest: rounds of two blocks a CU (one alone takes about half the
    // time a step), the partial sums' way out and back, and a launch for their sum.
    FfnSplit p{m <= 32 ? 32 : m <= 64 ? 64 : 128, 1, (int)(k / 32), 0, 0, 0};
    if (m == 0 || n == 0 || k == 0)
        return p;
    const int64_t tiles = ((m + p.tile - 1) / p.tile) * ((n + 127) / 128), steps = k / 32;
    const double step_us = p.tile == 32 ? 1.5 : p.tile == 64 ? 2.4 : 4.4;
    double best = -1.0;
    for (int64_t want = 1; want <= 64 && (want == 1 || 2 * want <= steps); ++want) {
        const int64_t per = (steps + want - 1) / want, splits = (steps + per - 1) / per, blocks = tiles * splits;
        double us = (blocks <= 256 ? 0.55 : (double)((blocks + 511) / 512)) * (double)per * step_us;
        if (splits > 1)
            us += 4.0 + (double)splits * (double)m * (double)n * 8.0 / 8e6;
        if (best < 0.0 || us < best) {
            best = us;
            p.per_split = (int)per;
            p.splits = (int)splits;
        }
    }
    p.partial_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)n * 4 : 0;
    return p;
}

namespace {

// The rows of one pass, and what its workspace holds front to back: h, the up
// product (fp32, whose projections are separate launches), 16-bit operands in
// copies where they are not aligned, and one product's partial sums and
// filled-up operands. The 16-bit kernels reach 2 GB of an operand: x, h and y
// of more rows go in passes (70000 rows of d_ff 16384: two).
struct FfnRoom {   // (of sizes above zero)
    int64_t rows;
    size_t h, u, copies, partial;
};
FfnRoom ffn_room(int64_t m, int64_t d, int64_t f, int dt)
{
    const size_t es = elem_size(dt);
    FfnRoom r{m, 0, 0, 0, 0};
    // Filled-up contractions always go in pieces: 4 bytes for each of g and u.
    const int64_t bytes = d % 64 != 0 || f % 64 != 0 ? 8 : 2;
    if (dt != DT_F32) {
        const int64_t most = (k2GB - 1) / (bytes * std::max(d, f));
        r.rows = std::min(m, most >= 256 ? most / 256 * 256 : std::max<int64_t>(most, 1));
        r.copies = up16((size_t)r.rows * (size_t)d * 2);
        if (m > 16 && !huge_weight(d, f))
            r.copies += 4 * up16((size_t)f * (size_t)(d / 32) * 2 + 2);   // groups of 32 have most
    }
    r.h = up16((size_t)r.rows * (size_t)f * es);
    r.u = dt == DT_F32 ? r.h : 0;
    // The last pass may be shorter, and its plans others.
    for (const int64_t rows : {r.rows, m - (m - 1) / r.rows * r.rows}) {
        auto split = [](const FfnSplit& p) { return up16(p.partial_bytes) + p.pad_bytes; };
        size_t part = std::max(split(ffn_split(rows, d, f, 2, dt)), split(ffn_split(rows, f, d, 1, dt)));
        // ffn_any's products: every one of fp32; of 16 bits those that contract
        // over 32 and those past the other kernels' offsets.
        const bool far = dt != DT_F32 && (huge_weight(d, f) || rows * std::max(d, f) >= k2GB / bytes);
        if (dt == DT_F32)
            part = std::max(part, ffn_any_plan(rows, d, f).partial_bytes);
        else if (d < 64 || far)
            part = std::max(part, any_gate_up_bytes(rows, d, f));
        if (dt == DT_F32 || far)
            part = std::max(part, ffn_any_plan(rows, f, d).partial_bytes);
        r.partial = std::max(r.partial, part);
    }
    return r;
}

// One pass: a.M is at most room.rows.
hipError_t ffn_pass(FfnArgs a, const FfnRoom& room, hipStream_t st)
{
    char* const h = static_cast<char*>(a.workspace);
    char* const copies = h + room.h + room.u;
    float* const partial = reinterpret_cast<float*>(copies + room.copies);
    if (a.dt == DT_F32) {
        void* const g = a.saved[0] != nullptr ? a.saved[0] : h;
        void* const u = a.saved[1] != nullptr ? a.saved[1] : h + room.h;
        if (hipError_t e = product(a, a.x, a.D, a.gate, a.F, partial, g, st); e != hipSuccess)
            return e;
        if (hipError_t e = product(a, a.x, a.D, a.up, a.F, partial, u, st); e != hipSuccess)
            return e;
        if (hipError_t e = gate(a, g, u, h, st); e != hipSuccess)
            return e;
        return product(a, h, a.F, a.down, a.D, partial, a.y, st);
    }
    // What is not aligned is copied: one kernel for a shape, and one result.
    const bool tiles = a.M > 16 && !huge_weight(a.D, a.F);
    {
        Copies c;
        c.to = copies;
        if (!aligned16(a.x))
            a.x = c.add(a.x, 1, a.M * a.D, a.M * a.D);
        if (tiles) {
            align_scales(c, a.gate, a.F * (a.D / a.gs));
            align_scales(c, a.up, a.F * (a.D / a.gs));
        }
        if (hipError_t e = c.run(st); e != hipSuccess)
            return e;
    }
    bool done = false;
    if (hipError_t e = split_product<true>(a, a.x, a.D, a.gate, a.up, a.F, partial, h, st, &done); e != hipSuccess)
        return e;
    if (!done) {
        GateUpArgs k{a.x, a.dt, a.act, a.M, a.D, a.F, a.gate, a.up, a.bits, a.gs, h, {a.saved[0], a.saved[1]}};
        if (hipError_t e = gate_up(k, st, &done); e != hipSuccess)
            return e;
    }
    if (!done)
        if (hipError_t e = any_gate_up(a, partial, h, st); e != hipSuccess)
            return e;
    if (tiles) {   // over the first copies, which are read by now
        Copies c;
        c.to = copies;
        align_scales(c, a.down, a.D * (a.F / a.gs));
        if (hipError_t e = c.run(st); e != hipSuccess)
            return e;
    }
    done = false;
    if (hipError_t e = split_product<false>(a, h, a.F, a.down, a.down, a.D, partial, a.y, st, &done);
        e != hipSuccess || done)
        return e;
    return product(a, h, a.F, a.down, a.D, partial, a.y, st);
}

} // namespace

size_t ffn_workspace_bytes(int64_t m, int64_t d, int64_t f, int dt)
{
    if (m == 0 || d == 0 || f == 0)
        return 0;
    const FfnRoom r = ffn_room(m, d, f, dt);
    return r.h + r.u + r.copies + r.partial;
}

hipError_t launch_ffn(const FfnArgs& a, hipStream_t st)
{
    if (a.D == 0 || a.F == 0) {   // y = 0 (d_ff 0), or g = u = 0 (d_model 0)
        if (a.D > 0)
            return launch_fill_zero(a.y, a.dt, a.M * a.D, st);
        for (void* s : a.saved)
            if (s != nullptr && a.F > 0)
                if (hipError_t e = launch_fill_zero(s, a.dt, a.M * a.F, st); e != hipSuccess)
                    return e;
        return hipSuccess;
    }
    const FfnRoom room = ffn_room(a.M, a.D, a.F, a.dt);
    const int64_t es = (int64_t)elem_size(a.dt);
    for (int64_t m = 0; m < a.M; m += room.rows) {
        FfnArgs p = a;
        p.M = std::min(room.rows, a.M - m);
        p.x = static_cast<const char*>(a.x) + m * a.D * es;
        p.y = static_cast<char*>(a.y) + m * a.D * es;
        for (void*& s : p.saved)
            if (s != nullptr)
                s = static_cast<char*>(s) + m * a.F * es;
        if (hipError_t e = ffn_pass(p, room, st); e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace qp
