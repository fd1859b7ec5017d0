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

// Elements 8 c .. 8 c + 7 of a row of n; those past its end are zeros.
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t at, int c, int n, float (&v)[8])
{
    using E = Elem<DT>;
    const typename E::storage* const q = static_cast<const typename E::storage*>(p) + at + 8 * c;
    const int left = n - 8 * c;
    if (left >= 8) {
        if constexpr (DT == DT_F32) {
            const u32x4_t a = *reinterpret_cast<const Wide32*>(q), b = *reinterpret_cast<const Wide32*>(q + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(a[i]);
                v[4 + i] = __uint_as_float(b[i]);
            }
        } else {
            const u32x4_t a = *reinterpret_cast<const Wide16*>(q);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = E::to_f32((uint16_t)(a[i / 2] >> (16 * (i % 2))));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = i < left ? E::to_f32(q[i]) : 0.0f;
    }
}

template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t at, int c, int n, const float (&v)[8])
{
    using E = Elem<DT>;
    typename E::storage* const q = static_cast<typename E::storage*>(p) + at + 8 * c;
    const int left = n - 8 * c;
    if (left >= 8) {
        if constexpr (DT == DT_F32) {
            u32x4_t a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = __float_as_uint(v[i]);
                b[i] = __float_as_uint(v[4 + i]);
            }
            *reinterpret_cast<Wide32*>(q) = a;
            *reinterpret_cast<Wide32*>(q + 4) = b;
        } else {
            u32x4_t a;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[i] = (uint32_t)E::from_f32(v[2 * i]) | ((uint32_t)E::from_f32(v[2 * i + 1]) << 16);
            *reinterpret_cast<Wide16*>(q) = a;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left)
                q[i] = E::from_f32(v[i]);
    }
}

// N sums over the row's THREADS threads, the same in each of them. `room` is
// the block's; a call may follow another at once.
template <int N, int THREADS>
__device__ __forceinline__ void row_sums(float (&v)[N], float (&room)[2][3][16], int& turn)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = segment_sum<64>(v[i]);
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
    float v[C][8], t[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
        load8<SDT>(a.x, at, lane + c * ROWT, n, v[c]);
    if (a.y != nullptr) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            load8<DT>(a.y, at, lane + c * ROWT, n, t[c]);
        if (a.post != nullptr) {
            float q[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[0] = __builtin_fmaf(t[c][i], t[c][i], q[0]);
            row_sums<1, ROWT>(q, room, turn);
            const float r = 1.0f / sqrtf(q[0] / (float)n + a.eps);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float w[8];
                load8<DT>(a.post, 0, lane + c * ROWT, n, w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    t[c][i] = t[c][i] * r * (w[i] + a.offset);
            }
        }
        if (a.gate != nullptr) {
            const int64_t g = row / (a.M / a.gates) * a.D;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float w[8];
                load8<DT>(a.gate, g, lane + c * ROWT, n, w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    t[c][i] *= w[i];
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[c][i] = __builtin_fmaf(a.factor, t[c][i], v[c][i]);
            store8<SDT>(a.s, at, lane + c * ROWT, n, v[c]);
        }
    }
    if (a.weight == nullptr)
        return;
    float q[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[0] = __builtin_fmaf(v[c][i], v[c][i], q[0]);
    row_sums<1, ROWT>(q, room, turn);
    const float r = 1.0f / sqrtf(q[0] / (float)n + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float w[8];
        load8<DT>(a.weight, 0, lane + c * ROWT, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = v[c][i] * r * (w[i] + a.offset);
        store8<DT>(a.a, at, lane + c * ROWT, n, w);
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
NormSplit norm_split(int64_t m, int64_t gates)
{
    constexpr int64_t kBlocks = 512;
    const int64_t g = std::max<int64_t>(gates, 1), groups = std::min(g, kBlocks);
    return {groups, std::clamp<int64_t>(kBlocks / groups, 1, std::max<int64_t>(m / g, 1))};
}

// The column sums of a block: in registers, or (rows of more than 8192) in the
// block's own part of the workspace, where each thread reads and writes the
// columns that are its own.
template <int DT, int SDT, int ROWT, int C, bool ACC_MEM>
__global__ __launch_bounds__(ROWT) void norm_grad_kernel(NormGradArgs a, int64_t groups, int64_t parts)
{
    __shared__ float room[2][3][16];
    int turn = 0;
    const int n = (int)a.D, lane = (int)threadIdx.x;
    const int64_t blocks = groups * parts, block = blockIdx.x, p = block % parts;
    const int64_t gates = a.gate != nullptr ? a.gates : 1, per = a.M / gates;
    float* const partial = static_cast<float*>(a.workspace);   // [3][blocks][D]: dweight, dpost, dgate
    float acc[ACC_MEM ? 1 : 3][C][8];
    auto clear = [&](int which) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float zero[8] = {};
            if constexpr (ACC_MEM)
                store8<DT_F32>(partial, (which * blocks + block) * a.D, lane + c * ROWT, n, zero);
            else
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[which][c][i] = 0.0f;
        }
    };
    auto add = [&](int which, int c, const float (&v)[8]) {
        if constexpr (ACC_MEM) {
            float t[8];
            load8<DT_F32>(partial, (which * blocks + block) * a.D, lane + c * ROWT, n, t);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                t[i] += v[i];
            store8<DT_F32>(partial, (which * blocks + block) * a.D, lane + c * ROWT, n, t);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[which][c][i] += v[i];
        }
    };
    if (!ACC_MEM || a.weight != nullptr)
        clear(0);
    if (!ACC_MEM || a.post != nullptr)
        clear(1);
    for (int64_t g = block / parts; g < gates; g += groups) {
        if (!ACC_MEM || a.gate != nullptr)
            clear(2);
        for (int64_t row = g * per + p; row < (g + 1) * per; row += parts) {
            const int64_t at = row * a.D;
            float G[C][8], v[C][8], u[C][8], y[C][8];
            float q[3] = {0.0f, 0.0f, 0.0f};   // s s, u s, y y
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (a.ds != nullptr) {
                    load8<SDT>(a.ds, at, lane + c * ROWT, n, G[c]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        G[c][i] = 0.0f;
                }
                if (a.weight != nullptr) {
                    load8<SDT>(a.s, at, lane + c * ROWT, n, v[c]);
                    load8<DT>(a.da, at, lane + c * ROWT, n, u[c]);
                    float w[8];
                    load8<DT>(a.weight, 0, lane + c * ROWT, n, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        q[0] = __builtin_fmaf(v[c][i], v[c][i], q[0]);
                        q[1] = __builtin_fmaf(u[c][i] * (w[i] + a.offset), v[c][i], q[1]);
                    }
                }
                if (a.y != nullptr) {
                    load8<DT>(a.y, at, lane + c * ROWT, n, y[c]);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        q[2] = __builtin_fmaf(y[c][i], y[c][i], q[2]);
                }
            }
            row_sums<3, ROWT>(q, room, turn);
            if (a.weight != nullptr) {
                const float r = 1.0f / sqrtf(q[0] / (float)n + a.eps);
                const float k = r * r * r * (q[1] / (float)n);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float w[8], d[8];
                    load8<DT>(a.weight, 0, lane + c * ROWT, n, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        d[i] = u[c][i] * v[c][i] * r;
                        G[c][i] += r * (u[c][i] * (w[i] + a.offset)) - v[c][i] * k;
                    }
                    add(0, c, d);
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                store8<SDT>(a.dx, at, lane + c * ROWT, n, G[c]);
            if (a.y == nullptr)
                continue;
            const float ry = 1.0f / sqrtf(q[2] / (float)n + a.eps);
            // t without the gate, then q and v over G and u.
            float z[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float w[8], t[8], d[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    t[i] = y[c][i];
                    G[c][i] *= a.factor;
                }
                if (a.post != nullptr) {
                    load8<DT>(a.post, 0, lane + c * ROWT, n, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        t[i] *= ry * (w[i] + a.offset);
                }
                if (a.gate != nullptr) {
                    float gt[8];
                    load8<DT>(a.gate, g * a.D, lane + c * ROWT, n, gt);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        d[i] = t[i] * G[c][i];
                        G[c][i] *= gt[i];
                    }
                    add(2, c, d);
                }
                if (a.post != nullptr) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        d[i] = G[c][i] * y[c][i] * ry;
                        G[c][i] *= w[i] + a.offset;
                        z[0] = __builtin_fmaf(G[c][i], y[c][i], z[0]);
                    }
                    add(1, c, d);
                }
            }
            if (a.post != nullptr) {
                row_sums<1, ROWT>(z, room, turn);
                const float k = ry * ry * ry * (z[0] / (float)n);
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        G[c][i] = ry * G[c][i] - y[c][i] * k;
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                store8<DT>(a.dy, at, lane + c * ROWT, n, G[c]);
        }
        if (a.gate != nullptr && (!ACC_MEM || parts == 1)) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float t[8];
                if constexpr (ACC_MEM)
                    load8<DT_F32>(partial, (2 * blocks + block) * a.D, lane + c * ROWT, n, t);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        t[i] = acc[2][c][i];
                if (parts == 1)
                    store8<DT>(a.dgate, g * a.D, lane + c * ROWT, n, t);
                else
                    store8<DT_F32>(partial, (2 * blocks + block) * a.D, lane + c * ROWT, n, t);
            }
        }
    }
    if constexpr (!ACC_MEM) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (a.weight != nullptr)
                store8<DT_F32>(partial, block * a.D, lane + c * ROWT, n, acc[0][c]);
            if (a.post != nullptr)
                store8<DT_F32>(partial, (blocks + block) * a.D, lane + c * ROWT, n, acc[1][c]);
        }
    }
}

// out[j][d] = the sum of `count` rows of `partial` from row j count on, in a fixed
// order: 64 columns a block, its 16 waves a share of the rows each.
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
    __shared__ float room[16][64];
    const NormJoin& j = a.j[blockIdx.z];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane, sum = blockIdx.y;
    if (sum >= j.rows)   // uniform
        return;
    const float* const p = j.partial + sum * j.count * a.D + (col < a.D ? col : 0);
    float v = 0.0f;
    for (int64_t r = wave; r < j.count; r += 16 * 8) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = r + 16 * i < j.count ? p[(r + 16 * i) * a.D] : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v += t[i];
    }
    room[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && col < a.D) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < 16; ++w)
            t += room[w][lane];
        static_cast<typename Elem<DT>::storage*>(j.out)[sum * a.D + col] = Elem<DT>::from_f32(t);
    }
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

template <int DT, int SDT, int ROWT, int C, bool ACC_MEM>
hipError_t run_bwd(const NormGradArgs& a, hipStream_t st)
{
    const NormSplit p = norm_split(a.M, a.gate != nullptr ? a.gates : 1);
    const int64_t blocks = p.groups * p.parts;
    hipLaunchKernelGGL((norm_grad_kernel<DT, SDT, ROWT, C, ACC_MEM>), dim3((unsigned)blocks), dim3(ROWT), 0, st, a,
                       p.groups, p.parts);
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
    hipLaunchKernelGGL((norm_join_kernel<DT>), dim3((unsigned)((a.D + 63) / 64), (unsigned)most, (unsigned)n),
                       dim3(1024), 0, st, j);
    return hipGetLastError();
}

template <int DT, int SDT>
hipError_t bwd(const NormGradArgs& a, hipStream_t st)
{
    if (a.D <= 512) return run_bwd<DT, SDT, 64, 1, false>(a, st);
    if (a.D <= 2048) return run_bwd<DT, SDT, 256, 1, false>(a, st);
    if (a.D <= 4096) return run_bwd<DT, SDT, 512, 1, false>(a, st);
    if (a.D <= 8192) return run_bwd<DT, SDT, 512, 2, false>(a, st);
    return run_bwd<DT, SDT, 512, 4, true>(a, st);
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
    const NormSplit p = norm_split(m, gates);
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
