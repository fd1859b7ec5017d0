// loss.hip — softmax cross entropy over a packed head, without the logits:
//   z = x W^T (W [V, K] packed),  lse = log sum_v exp(z_v),  loss = lse - z_target
// and its gradients, with the rows' upstream gradients g:
//   dz = g (exp(z - lse) - [v = target]),  dx = dz W,  dW = dz^T x,
// of dW the sums that belong to the scales and biases (wgrad.hpp).
//
// The vocabulary goes in pieces: of each, the logits are formed in fp32 and
// reduced at once, to a maximum and a sum of exponentials for each row and part
// of the piece (forward), or to dz, the operand of the two gradient products
// (backward, where they are formed a second time: the price of not keeping them,
// 2 M K V of 6 M K V operations). The parts' pairs are joined in a fixed order.
#include <algorithm>

#include "common.hpp"
#include "loss_stat.hpp"
#include "train_ops.hpp"
#include "xgrad.hpp"

namespace qp {

namespace {

constexpr int kPart = 4096;   // logits of a part, in the kernels that read them

// The statistics of each row's part of z [M, N], and the target's logit where it
// is in it.
__global__ __launch_bounds__(256) void loss_parts_kernel(const float* __restrict__ z, int64_t m, int64_t n, int parts,
                                                         int64_t v0, const int32_t* __restrict__ targets,
                                                         Stat* __restrict__ stats, float* __restrict__ picked)
{
    __shared__ Stat room[4];
    const int64_t block = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    const int64_t row = block / parts, c0 = block % parts * kPart;
    if (row >= m)
        return;
    const float* const p = z + row * n;
    const int tid = (int)threadIdx.x;
    float v[kPart / 256];
    float top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kPart / 256; ++i) {
        const int64_t c = c0 + tid + 256 * i;
        v[i] = c < n ? p[c] : -__builtin_inff();
        top = fmaxf(top, v[i]);
    }
    Stat s{top, 0.0f};
    const float at = top == -__builtin_inff() ? 0.0f : top;   // nothing here: sums of 0
#pragma unroll
    for (int i = 0; i < kPart / 256; ++i)
        s.sum += expf(v[i] - at);
    s = wave_stat(s);
    if ((tid & 63) == 0)
        room[tid >> 6] = s;
    __syncthreads();
    if (tid != 0)
        return;
    for (int w = 1; w < 4; ++w)
        s = join_stats(s, room[w]);
    stats[(v0 + c0) / kPart * m + row] = s;
    const int64_t t = targets[row];
    if (t >= v0 + c0 && t < v0 + c0 + kPart && t < v0 + n)
        picked[row] = p[t - v0];
}

// The rows' losses from their parts: 16 rows a block, 64 threads a row, each a share of
// the parts, four of them on their way at a time.
__global__ __launch_bounds__(1024) void loss_finish_kernel(const Stat* __restrict__ stats, int64_t parts, int64_t m,
                                                           int64_t vocab, const int32_t* __restrict__ targets,
                                                           const float* __restrict__ picked, float* __restrict__ loss,
                                                           float* __restrict__ lse)
{
    __shared__ Stat room[16][64];
    const int tid = (int)threadIdx.x, share = tid >> 4;
    const int64_t row = (int64_t)blockIdx.x * 16 + (tid & 15), at = row < m ? row : m - 1;
    Stat s{-__builtin_inff(), 0.0f};
    for (int64_t i = share; i < parts; i += 256) {
        Stat p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t part = i + 64 * j;
            p[j] = stats[(part < parts ? part : i) * m + at];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + 64 * j < parts)
                s = join_stats(s, p[j]);
    }
    room[tid & 15][share] = s;
    __syncthreads();
    // A wave a row.
    const int64_t out = (int64_t)blockIdx.x * 16 + (tid >> 6);
    if (out >= m)
        return;
    s = wave_stat(room[tid >> 6][tid & 63]);
    const int32_t t = targets[out];
    const float l = s.top + logf(s.sum), z = picked[out];
    if ((tid & 63) == 0) {
        lse[out] = l;
        loss[out] = t >= 0 && t < vocab ? l - z : 0.0f;
    }
}

// The losses of few rows, a block each, from all their logits at once: 32 a thread at a
// time, the next 32 on their way.
__global__ __launch_bounds__(1024) void loss_rows_kernel(const float* __restrict__ z, int64_t vocab,
                                                         const int32_t* __restrict__ targets, float* __restrict__ loss,
                                                         float* __restrict__ lse)
{
    typedef f32x4_t Wide __attribute__((aligned(4)));
    constexpr int V = 8, STEP = 1024 * 4 * V;
    __shared__ Stat room[16];
    const int tid = (int)threadIdx.x;
    const int64_t row = blockIdx.x;
    const float* const p = z + row * vocab;
    const int32_t target = targets[row];
    const bool live = target >= 0 && target < vocab;
    f32x4_t v[2][V];
    auto fetch = [&](int64_t c0, f32x4_t (&to)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t c = c0 + 4 * (tid + 1024 * i);
            if (c + 4 <= vocab)
                to[i] = *reinterpret_cast<const Wide*>(p + c);
            else
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    to[i][j] = c + j < vocab ? p[c + j] : -__builtin_inff();
        }
    };
    Stat s{-__builtin_inff(), 0.0f};
    auto take = [&](const f32x4_t (&t)[V]) {
        float top = s.top;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = fmaxf(top, t[i][j]);
        // A thread without any logit keeps -infinity: the row's maximum is of logits alone.
        const float at = top == -__builtin_inff() ? 0.0f : top;   // nothing yet: sums of 0
        float sum = s.sum * expf(s.top - at);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sum += expf(t[i][j] - at);
        s = Stat{top, sum};
    };
    fetch(0, v[0]);
    const float picked = live ? p[target] : 0.0f;
    for (int64_t c = 0; c < vocab; c += 2 * STEP) {
        fetch(c + STEP, v[1]);
        take(v[0]);
        if (c + STEP >= vocab)
            break;
        fetch(c + 2 * STEP, v[0]);
        take(v[1]);
    }
    s = wave_stat(s);
    if ((tid & 63) == 0)
        room[tid >> 6] = s;
    __syncthreads();
    if (tid >= 64)
        return;
    s = wave_stat<16>(room[tid & 15]);
    const float l = s.top + logf(s.sum);
    if (tid == 0) {
        lse[row] = l;
        loss[row] = live ? l - picked : 0.0f;
    }
}

// No features: every logit is 0. No vocabulary: lse is log 0.
__global__ __launch_bounds__(256) void loss_even_kernel(int64_t m, int64_t vocab, const int32_t* __restrict__ targets,
                                                        float* __restrict__ loss, float* __restrict__ lse)
{
    const float l = logf((float)vocab);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < m; i += (int64_t)gridDim.x * 256) {
        lse[i] = l;
        loss[i] = targets[i] >= 0 && targets[i] < vocab ? l : 0.0f;
    }
}

// The factor of dz, for the logits that are formed in full (the tiles' is found as x is
// laid out).
__global__ __launch_bounds__(256) void loss_scale_kernel(const float* __restrict__ dloss, int64_t m,
                                                         const int32_t* __restrict__ targets, int64_t vocab,
                                                         float* __restrict__ scale)
{
    dz_factor(dloss, m, targets, vocab, scale);
}

// dz of a piece from its logits; columns up to the next multiple of 8 are zeros
// (the gradient products read 16-bit rows in 16-byte pieces). dz may be z (fp32).
template <int DT>
__global__ __launch_bounds__(256) void loss_dz_kernel(const float* z, int64_t m, int64_t n, int64_t v0, int64_t vocab,
                                                      const int32_t* __restrict__ targets, const float* __restrict__ lse,
                                                      const float* __restrict__ dloss, const float* __restrict__ scale,
                                                      void* dz, int64_t stride)
{
    const int64_t cols = DT == DT_F32 ? n : (n + 7) & ~(int64_t)7, total = m * cols;
    const float by = scale != nullptr ? *scale : 1.0f;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / cols, c = i - r * cols, t = targets[r];
        const float g = t >= 0 && t < vocab ? dloss[r] * by : 0.0f;
        float v = 0.0f;
        if (c < n && g != 0.0f)
            v = g * (expf(z[r * n + c] - lse[r]) - (t == v0 + c ? 1.0f : 0.0f));
        store_elem<DT>(dz, r * stride + c, v);
    }
}

// Vocabulary of a piece: logits of about 256 MB in fp32, whole parts, or all of it. (A part
// at the least: from 16384 rows on 16 KB a row, at 2^20 rows 17 GB.)
int64_t piece_of(int64_t m, int64_t v)
{
    const int64_t most = std::max<int64_t>((int64_t(1) << 26) / m / kPart * kPart, kPart);
    return std::min(most, v);
}

QWeight rows_from(const QWeight& w, int64_t v0, int64_t k, int bits, int gs, int dt)
{
    const int64_t es = (int64_t)elem_size(dt), groups = k / gs;
    return {w.wq + v0 * (k * bits / 32), static_cast<const char*>(w.scales) + v0 * groups * es,
            static_cast<const char*>(w.biases) + v0 * groups * es};
}

hipError_t any_product(int bits, const FfnAnyArgs& a, hipStream_t st)
{
    switch (bits) {
    case 2: return launch_ffn_any_b2(a, st);
    case 3: return launch_ffn_any_b3(a, st);
    case 4: return launch_ffn_any_b4(a, st);
    case 6: return launch_ffn_any_b6(a, st);
    case 8: return launch_ffn_any_b8(a, st);
    }
    return hipErrorInvalidValue;
}

// Whether the decode kernels take a product: up to 16 rows of 16 bits, the weights
// streamed once (1 row of 4096 x 32000, 4-bit: 15.6 us, 120 on ffn_any's kernel).
bool rows_product(int64_t m, int dt) { return dt != DT_F32 && m <= 16; }

// One piece's logits, from weight row v0 on, as fp32 [M, n].
hipError_t logits(const void* x, int dt, int64_t m, int64_t k, QWeight w, int bits, int gs, int64_t v0, int64_t n,
                  float* z, hipStream_t st)
{
    w = rows_from(w, v0, k, bits, gs, dt);
    if (rows_product(m, dt) && aligned16(x)) {
        const GemvArgs a{x, dt, m, k, n, w.wq, w.scales, w.biases, bits, gs, z};
        switch (bits) {
        case 2: return launch_loss_rows_b2(a, st);
        case 3: return launch_loss_rows_b3(a, st);
        case 4: return launch_loss_rows_b4(a, st);
        case 6: return launch_loss_rows_b6(a, st);
        case 8: return launch_loss_rows_b8(a, st);
        }
    }
    FfnSplit plan = ffn_any_plan(m, k, n);
    plan.splits = 1;   // the vocabulary fills the GPU
    plan.per_split = (int)(k / 32);
    return any_product(bits, FfnAnyArgs{x, dt, m, k, n, w, gs, plan, z, m * n, nullptr}, st);
}

unsigned grid_of(int64_t n) { return (unsigned)std::min<int64_t>((n + 255) / 256, 16384); }

// Whether the tile kernel takes a product (its last step holds a row's last 64 features;
// up to 16 rows the decode kernels stream the weights once).
bool tile_product(int64_t m, int64_t k, int dt) { return (dt == DT_F32 || m > 16) && k >= 64 && k <= (1 << 18); }

hipError_t tile_kernel(int bits, int dt, const LossTileArgs& a, hipStream_t st)
{
    switch (bits) {
    case 2: return launch_loss_tile_b2(dt, a, st);
    case 3: return launch_loss_tile_b3(dt, a, st);
    case 4: return launch_loss_tile_b4(dt, a, st);
    case 6: return launch_loss_tile_b6(dt, a, st);
    case 8: return launch_loss_tile_b8(dt, a, st);
    }
    return hipErrorInvalidValue;
}
hipError_t prep(int bits, int dt, const LossTileArgs& a, const LossPrepArgs& p, hipStream_t st)
{
    switch (bits) {
    case 2: return launch_loss_prep_b2(dt, a, p, st);
    case 3: return launch_loss_prep_b3(dt, a, p, st);
    case 4: return launch_loss_prep_b4(dt, a, p, st);
    case 6: return launch_loss_prep_b6(dt, a, p, st);
    case 8: return launch_loss_prep_b8(dt, a, p, st);
    }
    return hipErrorInvalidValue;
}

// What the tile kernel reads beside the codes, laid out once a call (x) or a piece (the
// weight's): sizes in bytes.
struct TileRoom {
    int64_t xn, gp;
    size_t xp, xs, st, bp;
    size_t all() const { return xp + xs + st + bp; }
};
TileRoom tile_room(int64_t m, int64_t k, int64_t piece, int gs, int dt)
{
    const bool f32 = dt == DT_F32;
    const size_t es = elem_size(dt);
    const int64_t fill = f32 ? 8 : 32, gp = (k / gs + fill - 1) / fill * fill, kp = (k + 63) / 64 * 64;
    const int64_t xn = f32 ? 3 * kp : 2 * gp + kp, np = (piece + LOSS_BN - 1) / LOSS_BN * LOSS_BN;
    return {xn, gp, up16((size_t)m * (size_t)xn * 2),
            f32 ? up16((size_t)m * (size_t)gp * 4) : dt == DT_F16 ? up16((size_t)m * 4) : 0,
            up16((size_t)(k / gs) * (size_t)np * es), up16((size_t)piece * (size_t)gp * es)};
}
// The kernel's arguments that all pieces share: x is laid out at `room`, the weight's
// follow it.
void tile_begin(LossTileArgs& t, const TileRoom& r, char* room, int64_t m, int64_t k, int gs, int64_t vocab,
                const int32_t* targets)
{
    t.xp = room;
    t.xs = room + r.xp;
    t.st = room + r.xp + r.xs;
    t.M = (int)m; t.K = (int)k; t.gs = gs;
    t.xn = (int)r.xn; t.gp = (int)r.gp;
    t.vocab = vocab;
    t.targets = targets;
    t.stat_rows = m;
}
// A piece: what it reads is laid out (x and the factor of dz with the first), then its tiles.
hipError_t tile_piece(LossTileArgs& t, const TileRoom& r, char* room, const void* x, float* scale, const QWeight& w,
                      int bits, int dt, int64_t v0, int64_t n, hipStream_t st)
{
    t.wq = w.wq;
    t.N = (int)n;
    t.np = (int)((n + LOSS_BN - 1) / LOSS_BN * LOSS_BN);
    t.v0 = v0;
    t.part0 = (int)(v0 / LOSS_BN);
    // The biases as they lie, where their rows are whole 16-byte pieces.
    const bool as_is = t.gp == t.K / t.gs && aligned16(w.biases);
    char* const bp = room + r.xp + r.xs + r.st;
    t.bp = as_is ? w.biases : bp;
    const LossPrepArgs p{v0 == 0 ? x : nullptr, w.scales, w.biases, as_is ? nullptr : bp, v0 == 0 ? scale : nullptr};
    if (hipError_t e = prep(bits, dt, t, p, st); e != hipSuccess)
        return e;
    return tile_kernel(bits, dt, t, st);
}
// Vocabulary of a piece: scales of up to 2^29 bytes, whole tiles, fewer than 2^31 threads
// (256 for 32 rows of 256 tokens at most), and (backward) dz of about 128 MB, but not
// less than 2048 tokens.
int64_t tile_piece_of(int64_t m, int64_t k, int64_t v, int gs, bool grad)
{
    int64_t most = std::min((int64_t(1) << 27) / (k / gs), (int64_t(1) << 36) / m);
    most = std::max<int64_t>(most / LOSS_BN * LOSS_BN, LOSS_BN);
    if (grad)
        most = std::min(most, std::max<int64_t>((int64_t(1) << 26) / m / LOSS_BN * LOSS_BN, 2048));
    return std::min(most, v);
}

// The workspace front to back: the parts' statistics, the targets' logits, and the
// logits of a piece (few rows: and a copy of x where it is not aligned) or what the tile
// kernel reads.
struct LossRoom {
    bool tiles;
    int64_t piece, parts;
    size_t stats, picked, z, x;
    TileRoom t;
    size_t all() const { return stats + picked + z + x + t.all(); }
};
LossRoom loss_room(int64_t m, int64_t k, int64_t v, int gs, int dt)
{
    LossRoom r{};
    r.tiles = tile_product(m, k, dt);
    r.piece = r.tiles ? tile_piece_of(m, k, v, gs, false) : piece_of(m, v);
    r.parts = r.tiles ? (v + LOSS_BN - 1) / LOSS_BN : (v + kPart - 1) / kPart;
    r.stats = up16((size_t)r.parts * (size_t)m * sizeof(Stat));
    r.picked = up16((size_t)m * 4);
    if (r.tiles)
        r.t = tile_room(m, k, r.piece, gs, dt);
    else
        r.z = up16((size_t)m * (size_t)r.piece * 4);
    if (rows_product(m, dt))
        r.x = piece_bytes(m, k);
    return r;
}

// The backward pass: the factor of dz (16 bits), the sums of dx over the pieces, a piece's
// logits (or what the tile kernel reads) and dz, a copy of x where it is not aligned, the
// products' partial sums.
struct LossGradRoom {
    bool tiles;
    int64_t piece, stride;
    size_t scale, sums, z, dz, x, partial;
    TileRoom t;
    size_t all() const { return scale + sums + z + t.all() + dz + x + partial; }
};
LossGradRoom loss_grad_room(int64_t m, int64_t k, int64_t v, int gs, int dt)
{
    LossGradRoom r{};
    r.tiles = tile_product(m, k, dt);
    r.piece = r.tiles ? tile_piece_of(m, k, v, gs, true) : piece_of(m, v);
    r.stride = dt == DT_F32 && !r.tiles ? r.piece : (r.piece + 7) & ~(int64_t)7;
    r.scale = 16;
    r.sums = r.piece < v ? up16((size_t)m * (size_t)k * 4) : 0;
    if (r.tiles)
        r.t = tile_room(m, k, r.piece, gs, dt);
    else
        r.z = up16((size_t)m * (size_t)r.piece * 4);
    r.dz = r.z != 0 && dt == DT_F32 ? 0 : up16((size_t)m * (size_t)r.stride * elem_size(dt));
    r.x = rows_product(m, dt) || grad_tile_sizes(r.piece, k, dt) ? piece_bytes(m, k) : 0;
    // The last piece may be shorter, and its plans others.
    for (const int64_t n : {r.piece, v - (v - 1) / r.piece * r.piece})
        for (const bool tiles : {false, true})
            r.partial = std::max(r.partial, up16(std::max(xgrad_plan(m, n, k, 1, tiles).partial_bytes,
                                                          wgrad_plan(m, n, k, 1, gs, tiles).partial_bytes)));
    return r;
}

// dz of a piece from its logits.
hipError_t dz_of(const LossGradArgs& a, const float* z, int64_t v0, int64_t n, const float* scale, void* dz,
                 int64_t stride, hipStream_t st)
{
    const dim3 grid(grid_of(a.M * n));
    switch (a.dt) {
    case DT_F32:
        hipLaunchKernelGGL(loss_dz_kernel<DT_F32>, grid, dim3(256), 0, st, z, a.M, n, v0, a.V, a.targets, a.lse,
                           a.dloss, scale, dz, stride);
        break;
    case DT_F16:
        hipLaunchKernelGGL(loss_dz_kernel<DT_F16>, grid, dim3(256), 0, st, z, a.M, n, v0, a.V, a.targets, a.lse,
                           a.dloss, scale, dz, stride);
        break;
    default:
        hipLaunchKernelGGL(loss_dz_kernel<DT_BF16>, grid, dim3(256), 0, st, z, a.M, n, v0, a.V, a.targets, a.lse,
                           a.dloss, scale, dz, stride);
    }
    return hipGetLastError();
}

} // namespace

size_t loss_workspace_bytes(int64_t m, int64_t k, int64_t v, int, int gs, int dt)
{
    return m == 0 || v == 0 || k == 0 ? 0 : loss_room(m, k, v, gs, dt).all();
}

hipError_t launch_loss(const LossArgs& a, hipStream_t st)
{
    if (a.V == 0 || a.K == 0) {
        hipLaunchKernelGGL(loss_even_kernel, dim3(grid_of(a.M)), dim3(256), 0, st, a.M, a.V, a.targets, a.loss, a.lse);
        return hipGetLastError();
    }
    const LossRoom r = loss_room(a.M, a.K, a.V, a.gs, a.dt);
    Stat* const stats = static_cast<Stat*>(a.workspace);
    float* const picked = reinterpret_cast<float*>(reinterpret_cast<char*>(stats) + r.stats);
    char* const room = reinterpret_cast<char*>(picked) + r.picked;
    float* const z = reinterpret_cast<float*>(room);
    LossTileArgs t{};
    if (r.tiles) {
        t.stats = stats;
        t.picked = picked;
        tile_begin(t, r.t, room, a.M, a.K, a.gs, a.V, a.targets);
    }
    // Few rows whose logits are one piece, of a vocabulary that a block reads in two steps,
    // need no parts: one row of 32000 6.7 us (in parts 3.9 and 3.8); 12 of 131071 18.9 (4.7 and
    // 4.5).
    const bool few = !r.tiles && a.M <= 16 && r.piece == a.V && a.V <= (1 << 16);
    const void* x = a.x;
    if (rows_product(a.M, a.dt)) {
        int64_t stride = a.K;   // whole pieces: it stays
        if (hipError_t e = pieces_of_rows(x, a.M, a.K, room + r.z, &stride, st); e != hipSuccess)
            return e;
    }
    for (int64_t v0 = 0; v0 < a.V; v0 += r.piece) {
        const int64_t n = std::min(r.piece, a.V - v0), parts = (n + kPart - 1) / kPart;
        if (r.tiles) {
            if (hipError_t e = tile_piece(t, r.t, room, a.x, nullptr, rows_from(a.w, v0, a.K, a.bits, a.gs, a.dt), a.bits,
                                          a.dt, v0, n, st);
                e != hipSuccess)
                return e;
            continue;
        }
        if (hipError_t e = logits(x, a.dt, a.M, a.K, a.w, a.bits, a.gs, v0, n, z, st); e != hipSuccess)
            return e;
        if (few) {
            hipLaunchKernelGGL(loss_rows_kernel, dim3((unsigned)a.M), dim3(1024), 0, st, z, a.V, a.targets, a.loss, a.lse);
            return hipGetLastError();
        }
        hipLaunchKernelGGL(loss_parts_kernel, wide_grid(a.M * parts, 256), dim3(256), 0, st, z, a.M, n, (int)parts, v0,
                           a.targets, stats, picked);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(loss_finish_kernel, dim3((unsigned)((a.M + 15) / 16)), dim3(1024), 0, st, stats, r.parts, a.M,
                       a.V, a.targets, picked, a.loss, a.lse);
    return hipGetLastError();
}

size_t loss_grad_workspace_bytes(int64_t m, int64_t k, int64_t v, int, int gs, int dt)
{
    return m == 0 || v == 0 || k == 0 ? 0 : loss_grad_room(m, k, v, gs, dt).all();
}

hipError_t launch_loss_grad(const LossGradArgs& a, hipStream_t st)
{
    if (a.M == 0 || a.V == 0 || a.K == 0) {   // nothing to sum over
        if (a.dx != nullptr && a.M * a.K > 0)
            if (hipError_t e = launch_fill_zero(a.dx, a.dt, a.M * a.K, st); e != hipSuccess)
                return e;
        if (a.dscales == nullptr || a.V * a.K == 0)
            return hipSuccess;
        if (hipError_t e = launch_fill_zero(a.dscales, a.dt, a.V * (a.K / a.gs), st); e != hipSuccess)
            return e;
        return launch_fill_zero(a.dbiases, a.dt, a.V * (a.K / a.gs), st);
    }
    const LossGradRoom r = loss_grad_room(a.M, a.K, a.V, a.gs, a.dt);
    char* at = static_cast<char*>(a.workspace);
    auto take = [&](size_t n) { return std::exchange(at, at + n); };
    float* const scale = reinterpret_cast<float*>(take(r.scale));
    float* const sums = reinterpret_cast<float*>(take(r.sums));
    float* const z = reinterpret_cast<float*>(take(r.z));
    char* const room = take(r.t.all());
    void* const dz = r.dz == 0 ? static_cast<void*>(z) : take(r.dz);   // (fp32: over the logits)
    char* const xcopy = take(r.x);
    float* const partial = reinterpret_cast<float*>(at);
    const bool half = a.dt != DT_F32, tiles = grad_tile_sizes(r.piece, a.K, a.dt);
    if (half && !r.tiles) {
        hipLaunchKernelGGL(loss_scale_kernel, dim3(1), dim3(256), 0, st, a.dloss, a.M, a.targets, a.V, scale);
        if (hipError_t e = hipGetLastError(); e != hipSuccess)
            return e;
    }
    const void* xs = a.x;
    if (rows_product(a.M, a.dt) || (tiles && a.dscales != nullptr)) {
        int64_t stride = a.K;   // whole pieces: it stays
        if (hipError_t e = pieces_of_rows(xs, a.M, a.K, xcopy, &stride, st); e != hipSuccess)
            return e;
    }
    LossTileArgs t{};
    if (r.tiles) {
        t.dz = dz;
        t.dz_stride = r.stride;
        t.lse = a.lse; t.dloss = a.dloss; t.scale = half ? scale : nullptr;
        tile_begin(t, r.t, room, a.M, a.K, a.gs, a.V, a.targets);
    }
    for (int64_t v0 = 0; v0 < a.V; v0 += r.piece) {
        const int64_t n = std::min(r.piece, a.V - v0), es = (int64_t)elem_size(a.dt);
        const QWeight w = rows_from(a.w, v0, a.K, a.bits, a.gs, a.dt);
        const int64_t stride = a.dt == DT_F32 && !r.tiles ? n : r.stride;
        if (r.tiles) {
            if (hipError_t e = tile_piece(t, r.t, room, a.x, half ? scale : nullptr, w, a.bits, a.dt, v0, n, st);
                e != hipSuccess)
                return e;
        } else {
            if (hipError_t e = logits(xs, a.dt, a.M, a.K, a.w, a.bits, a.gs, v0, n, z, st); e != hipSuccess)
                return e;
            if (hipError_t e = dz_of(a, z, v0, n, half ? scale : nullptr, dz, stride, st); e != hipSuccess)
                return e;
        }
        if (a.dscales != nullptr) {
            WgradArgs g{};
            g.x = xs;
            g.dy[0] = g.dy[1] = dz;
            g.dy_stride = stride;
            g.wq[0] = g.wq[1] = w.wq;
            g.nmat = 1;
            g.dt = a.dt;
            g.M = a.M; g.N = n; g.K = a.K;
            g.bits = a.bits; g.gs = a.gs;
            g.dscales[0] = static_cast<char*>(a.dscales) + v0 * (a.K / a.gs) * es;
            g.dbiases[0] = static_cast<char*>(a.dbiases) + v0 * (a.K / a.gs) * es;
            g.partial = partial;
            g.scale = half ? scale + 1 : nullptr;
            if (hipError_t e = launch_wgrad(g, wgrad_plan(a.M, n, a.K, 1, a.gs, tiles), st); e != hipSuccess)
                return e;
        }
        if (a.dx != nullptr) {
            XgradArgs g{};
            g.dy[0] = g.dy[1] = dz;
            g.dy_stride = stride;
            g.w[0] = g.w[1] = w;
            g.nmat = 1;
            g.dt = a.dt;
            g.M = a.M; g.N = n; g.K = a.K;
            g.bits = a.bits; g.gs = a.gs;
            g.out = a.dx;
            g.partial = partial;
            g.first = v0 == 0;
            g.last = v0 + n == a.V;
            g.sums = g.first && g.last && !half ? nullptr : g.first && g.last ? partial : sums;
            g.scale = half ? scale + 1 : nullptr;
            if (hipError_t e = launch_xgrad(g, xgrad_plan(a.M, n, a.K, 1, tiles && grad_averages(n)), st); e != hipSuccess)
                return e;
        }
    }
    return hipSuccess;
}

} // namespace qp
