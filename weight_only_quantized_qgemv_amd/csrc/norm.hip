// norm.hip — what stands between two blocks of a model, in one pass over a row:
//   t = y r(y) (post + offset),   r(v) = 1 / sqrt(mean(v^2) + eps)
//   s = x + factor gate t,        a = s r(s) (weight + offset)
// and its gradients, with G the whole gradient of s:
//   u = da (weight + offset),     G = ds + r(s) u - s r(s)^3 mean(u s),   dx = G
//   q = factor gate G,  v = q (post + offset),  dy = r(y) v - y r(y)^3 mean(v y)
//   dweight = sum da s r(s),  dpost = sum q y r(y),  dgate = sum factor t G.
// Everything is fp32 from the loads on and rounded once at each output; a is
// formed from s before its rounding (in bf16 0.0017 of its size off 64 bits, from
// the rounded s 0.0024). The backward pass reads s as it was written.
//
// A row's threads hold it in registers, eight consecutive elements a chunk,
// loaded as 16 bytes at any element's address, so that each array is read and
// written once; the statistics are sums over the row's threads in a fixed order.
#include <algorithm>

#include "common.hpp"
#include "train_ops.hpp"

namespace qp {

namespace {

// Sixteen bytes at any element's address (rows of an odd width).
typedef u32x4_t Wide16 __attribute__((aligned(2)));
typedef u32x4_t Wide32 __attribute__((aligned(4)));

// Eight elements as they are loaded: one 16-byte piece, or two (fp32).
template <int DT> struct Pack {
    static constexpr int N = DT == DT_F32 ? 2 : 1;
    u32x4_t w[N];
    __device__ __forceinline__ float operator[](int i) const
    {
        if constexpr (DT == DT_F32)
            return __uint_as_float(w[i / 4][i % 4]);
        else
            return Elem<DT>::to_f32((uint16_t)(w[0][i / 2] >> (16 * (i % 2))));
    }
};
template <int DT> using WideOf = std::conditional_t<DT == DT_F32, Wide32, Wide16>;

// Elements 8 c .. 8 c + 7 of a row of n at p; those past its end are zeros.
template <int DT>
__device__ __forceinline__ Pack<DT> load8(const void* p, int64_t at, int c, int n)
{
    const typename Elem<DT>::storage* const q = static_cast<const typename Elem<DT>::storage*>(p) + at + 8 * c;
    const int left = n - 8 * c;
    Pack<DT> v;
    if (left >= 8) {
#pragma unroll
        for (int i = 0; i < Pack<DT>::N; ++i)
            v.w[i] = *reinterpret_cast<const WideOf<DT>*>(q + 4 * i);
        return v;
    }
#pragma unroll
    for (int i = 0; i < Pack<DT>::N; ++i)
        v.w[i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) {
            if constexpr (DT == DT_F32)
                v.w[i / 4][i % 4] = __float_as_uint(q[i]);
            else
                v.w[0][i / 2] |= (uint32_t)q[i] << (16 * (i % 2));
        }
    return v;
}

template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t at, int c, int n, const float (&v)[8])
{
    using E = Elem<DT>;
    typename E::storage* const q = static_cast<typename E::storage*>(p) + at + 8 * c;
    const int left = n - 8 * c;
    if (left >= 8) {
#pragma unroll
        for (int i = 0; i < Pack<DT>::N; ++i) {
            u32x4_t a;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (DT == DT_F32)
                    a[j] = __float_as_uint(v[4 * i + j]);
                else
                    a[j] = (uint32_t)E::from_f32(v[2 * j]) | ((uint32_t)E::from_f32(v[2 * j + 1]) << 16);
            }
            *reinterpret_cast<WideOf<DT>*>(q + 4 * i) = a;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < left)
                q[i] = E::from_f32(v[i]);
    }
}

// N sums over a wave, in all its lanes: moves between lanes, no trips to LDS.
template <int N> __device__ __forceinline__ void wave_sums(float (&v)[N])
{
    reduce_slots<N, 16>(v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t t = __float_as_uint(v[i]);
        const auto x = __builtin_amdgcn_permlane16_swap(t, t, false, false);
        v[i] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t t = __float_as_uint(v[i]);
        const auto x = __builtin_amdgcn_permlane32_swap(t, t, false, false);
        v[i] = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    }
}

// N sums over the row's THREADS threads, the same in each of them. `room` is
// the block's; a call may follow another at once.
template <int N, int THREADS>
__device__ __forceinline__ void row_sums(float (&v)[N], float (&room)[2][3][16], int& turn)
{
    wave_sums<N>(v);
    if constexpr (THREADS > 64) {
        const int wave = (int)threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                room[turn][i][wave] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < THREADS / 64; ++w)
                t += room[turn][i][w];
            v[i] = t;
        }
        turn ^= 1;   // the next call's room is another: one barrier a call
    }
}

// A row's threads; rows of up to 64 x 8 C elements take a wave, four rows a block.
template <int ROWT> constexpr int kRowsPerBlock = ROWT == 64 ? 4 : 1;

template <int DT, int SDT, int ROWT, int C>
__global__ __launch_bounds__(ROWT * kRowsPerBlock<ROWT>) void norm_kernel(NormArgs a)
{
    constexpr int RPB = kRowsPerBlock<ROWT>;
    __shared__ float room[2][3][16];
    int turn = 0;
    const int n = (int)a.D, lane = (int)threadIdx.x % ROWT;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / ROWT;
    if (RPB > 1 && row >= a.M)
        return;
    const int64_t at = row * a.D;
    const bool block = a.y != nullptr, gated = a.gate != nullptr, last = a.weight == nullptr;
    // Everything whose address is known is asked for first.
    Pack<SDT> x[C];
    Pack<DT> y[C], post[C], gate[C], weight[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        x[c] = load8<SDT>(a.x, at, lane + c * ROWT, n);
        if (block)
            y[c] = load8<DT>(a.y, at, lane + c * ROWT, n);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (a.post != nullptr)
            post[c] = load8<DT>(a.post, 0, lane + c * ROWT, n);
        if (gated)
            gate[c] = load8<DT>(a.gate, row / (a.M / a.gates) * a.D, lane + c * ROWT, n);
        if (!last)
            weight[c] = load8<DT>(a.weight, 0, lane + c * ROWT, n);
    }
    float v[C][8];
    float q[1] = {0.0f};
    if (block) {
        float r = 1.0f;
        if (a.post != nullptr) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[0] = __builtin_fmaf(y[c][i], y[c][i], q[0]);
            row_sums<1, ROWT>(q, room, turn);
            r = 1.0f / sqrtf(q[0] / (float)n + a.eps);
        }
        q[0] = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float t = y[c][i];
                if (a.post != nullptr)
                    t = t * r * (post[c][i] + a.offset);
                if (gated)
                    t *= gate[c][i];
                v[c][i] = __builtin_fmaf(a.factor, t, x[c][i]);
                q[0] = __builtin_fmaf(v[c][i], v[c][i], q[0]);
            }
            store8<SDT>(a.s, at, lane + c * ROWT, n, v[c]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[c][i] = x[c][i];
                q[0] = __builtin_fmaf(v[c][i], v[c][i], q[0]);
            }
    }
    if (last)
        return;
    row_sums<1, ROWT>(q, room, turn);
    const float r = 1.0f / sqrtf(q[0] / (float)n + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[c][i] = v[c][i] * r * (weight[c][i] + a.offset);
        store8<DT>(a.a, at, lane + c * ROWT, n, v[c]);
    }
}

// The rows' shares of the backward pass. Gate row g's rows are those from g L on,
// L = M / gates; `groups` blocks side by side walk gate rows q, q + groups, ..,
// `parts` of them one gate row's rows p, p + parts, .. : with few gate rows
// several blocks to each (their sums of dgate are joined), with many one block,
// which writes dgate itself.
struct NormSplit {
    int64_t groups, parts;
};
// Threads of a row in the backward pass, and so many blocks as the GPU holds at once
// (two waves a SIMD): 8192 rows of 4096, bf16, 86 us, with half as many 148, with twice as
// many 92; 4096 rows of 2048 30.7 us on 512 blocks of 256 threads, 38.1 on 256, 31.2 on 768,
// 35.8 on 1024. Of as many rounds the fewest blocks, whose sums take the least room (600
// rows of 1027 17 us on 300 blocks as on 512).
int norm_threads(int64_t d) { return d <= 512 ? 64 : d <= 1024 ? 128 : d <= 2048 ? 256 : 512; }
NormSplit norm_split(int64_t m, int64_t d, int64_t gates)
{
    const int64_t blocks = 256 * (512 / norm_threads(d));
    auto even = [](int64_t n, int64_t most) {   // the fewest blocks that are as many rounds
        const int64_t rounds = (n + most - 1) / most;
        return (n + rounds - 1) / rounds;
    };
    const int64_t g = std::max<int64_t>(gates, 1), groups = even(g, std::min(g, blocks));
    const int64_t per = std::max<int64_t>(m / g, 1);
    return {groups, even(per, std::clamp<int64_t>(blocks / groups, 1, per))};
}

// r^3 mean(u v), of a row v and r = 1 / rms(v): from the mean on, which is of the row's own
// size, so that only powers that the squares' sums allow too are formed (r^3 alone is
// infinite for rows of 1e-13 and eps = 0, and subnormal for rows of 1e13).
__device__ __forceinline__ float thrice(float r, float mean) { return r * (r * (r * mean)); }

// Rows of up to 8192: the row, the weights and the block's column sums stay in
// registers. A row of one chunk a thread is loaded while the row before it is summed
// and closed.
template <int DT, int SDT, int ROWT, int C>
__global__ __launch_bounds__(ROWT, 2) void norm_grad_kernel(NormGradArgs a, int64_t groups, int64_t parts)
{
    __shared__ float room[2][3][16];
    int turn = 0;
    const int n = (int)a.D, lane = (int)threadIdx.x;
    const int64_t blocks = groups * parts, block = blockIdx.x, p = block % parts;
    const int64_t gates = a.gate != nullptr ? a.gates : 1, per = a.M / gates;
    const bool pre = a.weight != nullptr, post = a.post != nullptr, gated = a.gate != nullptr, whole = a.y != nullptr;
    float* const partial = static_cast<float*>(a.workspace);   // [3][blocks][D]: dweight, dpost, dgate
    float acc[3][C][8];
    auto clear = [&](int which) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[which][c][i] = 0.0f;
    };
    struct Row {
        Pack<SDT> ds[C], s[C];
        Pack<DT> da[C], y[C];
    };
    auto fetch = [&](int64_t row, Row& r) {
        const int64_t at = row * a.D;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (a.ds != nullptr)
                r.ds[c] = load8<SDT>(a.ds, at, lane + c * ROWT, n);
            if (pre) {
                r.s[c] = load8<SDT>(a.s, at, lane + c * ROWT, n);
                r.da[c] = load8<DT>(a.da, at, lane + c * ROWT, n);
            }
            if (whole)
                r.y[c] = load8<DT>(a.y, at, lane + c * ROWT, n);
        }
    };
    Row cur;
    fetch(block / parts * per + p, cur);
    Pack<DT> weight[C], postw[C], gate[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (pre)
            weight[c] = load8<DT>(a.weight, 0, lane + c * ROWT, n);
        if (post)
            postw[c] = load8<DT>(a.post, 0, lane + c * ROWT, n);
    }
    clear(0);
    clear(1);
    for (int64_t g = block / parts; g < gates; g += groups) {
        if (gated) {
            clear(2);
#pragma unroll
            for (int c = 0; c < C; ++c)
                gate[c] = load8<DT>(a.gate, g * a.D, lane + c * ROWT, n);
        }
        for (int64_t row = g * per + p; row < (g + 1) * per; row += parts) {
            const int64_t at = row * a.D;
            const int64_t after = row + parts < (g + 1) * per ? row + parts : g + groups < gates ? (g + groups) * per + p : -1;
            constexpr bool AHEAD = C == 1;
            Row next;
            if constexpr (AHEAD) {
                if (after >= 0)
                    fetch(after, next);
            }
            float q[3] = {0.0f, 0.0f, 0.0f};   // s s, u s, y y
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (pre) {
                        const float s = cur.s[c][i];
                        q[0] = __builtin_fmaf(s, s, q[0]);
                        q[1] = __builtin_fmaf(cur.da[c][i] * (weight[c][i] + a.offset), s, q[1]);
                    }
                    if (post)
                        q[2] = __builtin_fmaf(cur.y[c][i], cur.y[c][i], q[2]);
                }
            row_sums<3, ROWT>(q, room, turn);
            const float rs = pre ? 1.0f / sqrtf(q[0] / (float)n + a.eps) : 0.0f, ks = thrice(rs, q[1] / (float)n);
            const float ry = post ? 1.0f / sqrtf(q[2] / (float)n + a.eps) : 1.0f;
            float G[C][8], z[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    G[c][i] = a.ds != nullptr ? cur.ds[c][i] : 0.0f;
                if (pre) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float s = cur.s[c][i], u = cur.da[c][i];
                        acc[0][c][i] = __builtin_fmaf(u * s, rs, acc[0][c][i]);
                        G[c][i] += rs * (u * (weight[c][i] + a.offset)) - s * ks;
                    }
                }
                store8<SDT>(a.dx, at, lane + c * ROWT, n, G[c]);
                if (!whole)
                    continue;
                // G is now q, and then v: t is y r(y) (post + offset).
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    G[c][i] *= a.factor;
                if (gated) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float t = post ? cur.y[c][i] * (ry * (postw[c][i] + a.offset)) : cur.y[c][i];
                        acc[2][c][i] = __builtin_fmaf(t, G[c][i], acc[2][c][i]);
                        G[c][i] *= gate[c][i];
                    }
                }
                if (post) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        acc[1][c][i] = __builtin_fmaf(G[c][i] * cur.y[c][i], ry, acc[1][c][i]);
                        G[c][i] *= postw[c][i] + a.offset;
                        z[0] = __builtin_fmaf(G[c][i], cur.y[c][i], z[0]);
                    }
                }
            }
            if (whole) {
                float kz = 0.0f;
                if (post) {
                    row_sums<1, ROWT>(z, room, turn);
                    kz = thrice(ry, z[0] / (float)n);
                }
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (post) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            G[c][i] = ry * G[c][i] - cur.y[c][i] * kz;
                    }
                    store8<DT>(a.dy, at, lane + c * ROWT, n, G[c]);
                }
            }
            if constexpr (AHEAD)
                cur = next;
            else if (after >= 0)
                fetch(after, cur);
        }
        if (gated) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (parts == 1)
                    store8<DT>(a.dgate, g * a.D, lane + c * ROWT, n, acc[2][c]);
                else
                    store8<DT_F32>(partial, (2 * blocks + block) * a.D, lane + c * ROWT, n, acc[2][c]);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (pre)
            store8<DT_F32>(partial, block * a.D, lane + c * ROWT, n, acc[0][c]);
        if (post)
            store8<DT_F32>(partial, (blocks + block) * a.D, lane + c * ROWT, n, acc[1][c]);
    }
}

// Wider rows: read again for each of the three passes over a row (from L2), a chunk at
// a time, the column sums in the block's own part of the workspace, where each thread
// reads and writes the columns that are its own, once for three rows. 2048 rows of
// 16384, bf16, with a gate: 234 us; once for two rows 247; with every row, 0.8 GB of sums'
// way through the workspace, 309.
template <int DT, int SDT>
__global__ __launch_bounds__(512) void norm_grad_wide_kernel(NormGradArgs a, int64_t groups, int64_t parts)
{
    constexpr int T = 512, R = 3;
    __shared__ float room[2][3][16];
    int turn = 0;
    const int n = (int)a.D, lane = (int)threadIdx.x, chunks = (n + 7) / 8;
    const int64_t blocks = groups * parts, block = blockIdx.x, p = block % parts;
    const int64_t gates = a.gate != nullptr ? a.gates : 1, per = a.M / gates;
    const bool pre = a.weight != nullptr, post = a.post != nullptr, gated = a.gate != nullptr, whole = a.y != nullptr;
    float* const partial = static_cast<float*>(a.workspace);   // [3][blocks][D]: dweight, dpost, dgate
    bool first[3] = {true, true, true};   // of the sums: nothing to add to yet
    auto add = [&](int which, int c, const float (&v)[8]) {
        const int64_t at = (which * blocks + block) * a.D;
        float t[8];
        if (first[which]) {
            store8<DT_F32>(partial, at, c, n, v);
        } else {
            const Pack<DT_F32> old = load8<DT_F32>(partial, at, c, n);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                t[i] = old[i] + v[i];
            store8<DT_F32>(partial, at, c, n, t);
        }
    };
    for (int64_t g = block / parts; g < gates; g += groups) {
        first[2] = true;
        const int64_t end = (g + 1) * per;
        for (int64_t row = g * per + p; row < end; row += R * parts) {
            float rs[R], ks[R], ry[R], z[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                rs[r] = ks[r] = z[r] = 0.0f;
                ry[r] = 1.0f;
                const int64_t at = (row + r * parts) * a.D;
                if (row + r * parts >= end)   // (the same for the whole block)
                    continue;
                float q[3] = {0.0f, 0.0f, 0.0f};   // s s, u s, y y
                for (int c = lane; c < chunks; c += T) {
                    if (pre) {
                        const Pack<SDT> s = load8<SDT>(a.s, at, c, n);
                        const Pack<DT> da = load8<DT>(a.da, at, c, n), w = load8<DT>(a.weight, 0, c, n);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            q[0] = __builtin_fmaf(s[i], s[i], q[0]);
                            q[1] = __builtin_fmaf(da[i] * (w[i] + a.offset), s[i], q[1]);
                        }
                    }
                    if (post) {
                        const Pack<DT> y = load8<DT>(a.y, at, c, n);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            q[2] = __builtin_fmaf(y[i], y[i], q[2]);
                    }
                }
                row_sums<3, T>(q, room, turn);
                if (pre) {
                    rs[r] = 1.0f / sqrtf(q[0] / (float)n + a.eps);
                    ks[r] = thrice(rs[r], q[1] / (float)n);
                }
                if (post)
                    ry[r] = 1.0f / sqrtf(q[2] / (float)n + a.eps);
            }
            // v (or q) of row r's chunk c; with `sums`, what is summed on the way to it goes
            // to d. dx may be ds, and dy da or y: they are written when nothing of the chunk
            // is read any more.
            auto through = [&](int r, int c, bool sums, const Pack<DT>& y, float (&G)[8], float (&d)[3][8]) {
                const int64_t at = (row + r * parts) * a.D;
                if (a.ds != nullptr) {
                    const Pack<SDT> ds = load8<SDT>(a.ds, at, c, n);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        G[i] = ds[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        G[i] = 0.0f;
                }
                if (pre) {
                    const Pack<SDT> s = load8<SDT>(a.s, at, c, n);
                    const Pack<DT> da = load8<DT>(a.da, at, c, n), w = load8<DT>(a.weight, 0, c, n);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        d[0][i] = __builtin_fmaf(da[i] * s[i], rs[r], d[0][i]);
                        G[i] += rs[r] * (da[i] * (w[i] + a.offset)) - s[i] * ks[r];
                    }
                }
                if (!sums || !post)
                    store8<SDT>(a.dx, at, c, n, G);
                if (!whole)
                    return;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    G[i] *= a.factor;
                const Pack<DT> w = post ? load8<DT>(a.post, 0, c, n) : Pack<DT>{};
                if (gated) {
                    const Pack<DT> gate = load8<DT>(a.gate, g * a.D, c, n);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float t = post ? y[i] * (ry[r] * (w[i] + a.offset)) : y[i];
                        d[2][i] = __builtin_fmaf(t, G[i], d[2][i]);
                        G[i] *= gate[i];
                    }
                }
                if (post) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        d[1][i] = __builtin_fmaf(G[i] * y[i], ry[r], d[1][i]);
                        G[i] *= w[i] + a.offset;
                    }
                }
            };
            // A pass over the rows' chunks; the columns' sums of all R rows go out together.
            auto pass = [&](bool sums, auto close) {
                for (int c = lane; c < chunks; c += T) {
                    float d[3][8] = {};
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const int64_t at = (row + r * parts) * a.D;
                        if (row + r * parts >= end)
                            continue;
                        const Pack<DT> y = whole ? load8<DT>(a.y, at, c, n) : Pack<DT>{};
                        float G[8];
                        through(r, c, sums, y, G, d);
                        close(r, c, at, y, G);
                    }
                    if (sums) {
                        if (pre)
                            add(0, c, d[0]);
                        if (post)
                            add(1, c, d[1]);
                        if (gated)
                            add(2, c, d[2]);
                    }
                }
            };
            if (post) {
                pass(true, [&](int r, int, int64_t, const Pack<DT>& y, const float (&G)[8]) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        z[r] = __builtin_fmaf(G[i], y[i], z[r]);
                });
                row_sums<R, T>(z, room, turn);
            }
            pass(!post, [&](int r, int c, int64_t at, const Pack<DT>& y, float (&G)[8]) {
                if (!whole)
                    return;
                if (post) {
                    const float kz = thrice(ry[r], z[r] / (float)n);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        G[i] = ry[r] * G[i] - y[i] * kz;
                }
                store8<DT>(a.dy, at, c, n, G);
            });
            first[0] = first[1] = first[2] = false;
        }
        if (gated && parts == 1) {
            for (int c = lane; c < chunks; c += T) {
                const Pack<DT_F32> sum = load8<DT_F32>(partial, (2 * blocks + block) * a.D, c, n);
                float t[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    t[i] = sum[i];
                store8<DT>(a.dgate, g * a.D, c, n, t);
            }
        }
    }
}

// out[j][d] = the sum of `count` rows of `partial` from row j count on, in a fixed
// order: 16 columns a block, its 64 groups of 16 threads a share of the rows each.
struct NormJoin {
    const float* partial;
    void* out;
    int64_t count, rows;   // rows of a sum, sums
};
struct NormJoins {
    NormJoin j[3];
    int64_t D;
};
template <int DT>
__global__ __launch_bounds__(1024) void norm_join_kernel(NormJoins a)
{
    constexpr int COLS = 16, R = 1024 / COLS;
    __shared__ float room[R][COLS];
    const NormJoin& j = a.j[blockIdx.z];
    const int lane = (int)threadIdx.x % COLS, share = (int)threadIdx.x / COLS;
    const int64_t col = (int64_t)blockIdx.x * COLS + lane, sum = blockIdx.y;
    if (sum >= j.rows)   // uniform
        return;
    const float* const p = j.partial + sum * j.count * a.D + (col < a.D ? col : 0);
    float v = 0.0f;
    for (int64_t r = share; r < j.count; r += R * 8) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = r + R * i < j.count ? p[(r + R * i) * a.D] : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v += t[i];
    }
    room[share][lane] = v;
#pragma unroll
    for (int half = R / 2; half > 0; half /= 2) {
        __syncthreads();
        if (share < half)
            room[share][lane] += room[share + half][lane];
    }
    if (share == 0 && col < a.D)
        static_cast<typename Elem<DT>::storage*>(j.out)[sum * a.D + col] = Elem<DT>::from_f32(room[0][lane]);
}

template <int DT, int SDT, int ROWT, int C>
hipError_t run_fwd(const NormArgs& a, hipStream_t st)
{
    constexpr int RPB = kRowsPerBlock<ROWT>;
    const int64_t blocks = (a.M + RPB - 1) / RPB;
    if (!grid_fits(blocks, ROWT * RPB))
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((norm_kernel<DT, SDT, ROWT, C>), dim3((unsigned)blocks), dim3(ROWT * RPB), 0, st, a);
    return hipGetLastError();
}

template <int DT, int SDT>
hipError_t fwd(const NormArgs& a, hipStream_t st)
{
    if (a.D <= 512) return run_fwd<DT, SDT, 64, 1>(a, st);
    if (a.D <= 1024) return run_fwd<DT, SDT, 64, 2>(a, st);
    if (a.D <= 2048) return run_fwd<DT, SDT, 256, 1>(a, st);
    if (a.D <= 4096) return run_fwd<DT, SDT, 512, 1>(a, st);
    if (a.D <= 8192) return run_fwd<DT, SDT, 512, 2>(a, st);
    return run_fwd<DT, SDT, 512, 4>(a, st);
}

template <int DT, int SDT, int ROWT, int C>
hipError_t run_bwd(const NormGradArgs& a, hipStream_t st)
{
    const NormSplit p = norm_split(a.M, a.D, a.gate != nullptr ? a.gates : 1);
    const int64_t blocks = p.groups * p.parts;
    if constexpr (C > 0)
        hipLaunchKernelGGL((norm_grad_kernel<DT, SDT, ROWT, C>), dim3((unsigned)blocks), dim3(ROWT), 0, st, a, p.groups,
                           p.parts);
    else
        hipLaunchKernelGGL((norm_grad_wide_kernel<DT, SDT>), dim3((unsigned)blocks), dim3(ROWT), 0, st, a, p.groups,
                           p.parts);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    NormJoins j{};
    j.D = a.D;
    int n = 0;
    int64_t most = 1;
    const float* const partial = static_cast<const float*>(a.workspace);
    if (a.weight != nullptr)
        j.j[n++] = {partial, a.dweight, blocks, 1};
    if (a.post != nullptr)
        j.j[n++] = {partial + blocks * a.D, a.dpost, blocks, 1};
    if (a.gate != nullptr && p.parts > 1) {
        j.j[n++] = {partial + 2 * blocks * a.D, a.dgate, p.parts, a.gates};
        most = a.gates;
    }
    if (n == 0)
        return hipSuccess;
    hipLaunchKernelGGL((norm_join_kernel<DT>), dim3((unsigned)((a.D + 15) / 16), (unsigned)most, (unsigned)n),
                       dim3(1024), 0, st, j);
    return hipGetLastError();
}

template <int DT, int SDT>
hipError_t bwd(const NormGradArgs& a, hipStream_t st)
{
    if (a.D <= 512) return run_bwd<DT, SDT, 64, 1>(a, st);
    if (a.D <= 1024) return run_bwd<DT, SDT, 128, 1>(a, st);
    if (a.D <= 2048) return run_bwd<DT, SDT, 256, 1>(a, st);
    if (a.D <= 4096) return run_bwd<DT, SDT, 512, 1>(a, st);
    if (a.D <= 8192) return run_bwd<DT, SDT, 512, 2>(a, st);
    return run_bwd<DT, SDT, 512, 0>(a, st);
}

// f(types) for the block's type and the stream's.
template <class Args, class F>
hipError_t by_type(const Args& a, F&& f)
{
    using std::integral_constant;
    const bool same = a.sdt == a.dt;
    switch (a.dt) {
    case DT_F32: return f(integral_constant<int, DT_F32>{}, integral_constant<int, DT_F32>{});
    case DT_F16:
        return same ? f(integral_constant<int, DT_F16>{}, integral_constant<int, DT_F16>{})
                    : f(integral_constant<int, DT_F16>{}, integral_constant<int, DT_F32>{});
    case DT_BF16:
        return same ? f(integral_constant<int, DT_BF16>{}, integral_constant<int, DT_BF16>{})
                    : f(integral_constant<int, DT_BF16>{}, integral_constant<int, DT_F32>{});
    }
    return hipErrorInvalidValue;
}

} // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t st)
{
    return by_type(a, [&](auto T, auto S) { return fwd<decltype(T)::value, decltype(S)::value>(a, st); });
}

size_t norm_grad_workspace_bytes(int64_t m, int64_t d, int64_t gates)
{
    if (m == 0 || d == 0)
        return 0;
    const NormSplit p = norm_split(m, d, gates);
    return 3 * (size_t)(p.groups * p.parts) * (size_t)d * 4;
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st)
{
    if (a.M == 0) {   // no rows to sum over
        for (void* p : {a.dweight, a.dpost})
            if (p != nullptr)
                if (hipError_t e = launch_fill_zero(p, a.dt, a.D, st); e != hipSuccess)
                    return e;
        return a.dgate != nullptr ? launch_fill_zero(a.dgate, a.dt, a.gates * a.D, st) : hipSuccess;
    }
    return by_type(a, [&](auto T, auto S) { return bwd<decltype(T)::value, decltype(S)::value>(a, st); });
}

} // namespace qp
