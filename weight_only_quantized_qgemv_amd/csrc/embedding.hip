// embedding.hip — the packed embedding table: lookup with a factor,
//   out[t, k] = factor * (q[id, k] * s'[id, G] + b'[id, G]),   id = ids[t],
// and the gradient of its scales and biases,
//   dscales[v, G] = factor * sum_{t: ids[t] = v} sum_{k in G} q[v, k] dout[t, k],
//   dbiases[v, G] = factor * sum_{t: ids[t] = v} sum_{k in G} dout[t, k].
//
// The gradient sums a row's tokens in token order, by sorting: chunks of the
// ids are sorted by (id, token) in LDS, every token's place in the whole order
// is its place in its chunk plus the counts of smaller keys in the others,
// and a wave then sums one run of equal ids over 512 columns, in order, in
// fp32, before it meets the codes. Runs longer than kPiece tokens are cut into
// pieces whose sums are added in order by a last launch, so that a token that
// fills a tenth of a batch does not hold the rest up. No atomics: the result
// does not depend on the launch.
#include <algorithm>

#include "codes8.hpp"
#include "common.hpp"
#include "model_ops.hpp"
#include "xgrad.hpp"

namespace qp {

namespace {

// Eight consecutive elements, as one or two 16-byte accesses where the rows
// allow it.
template <int DT> __device__ __forceinline__ void load8(const void* p, int64_t i, bool vec, float (&v)[8])
{
    using St = typename Elem<DT>::storage;
    const St* s = static_cast<const St*>(p) + i;
    if (vec) {
        constexpr int NV = (int)sizeof(St) / 2;
        u32x4_t w[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            w[j] = reinterpret_cast<const u32x4_t*>(s)[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (DT == DT_F32)
                v[j] = __uint_as_float(w[j / 4][j % 4]);
            else
                v[j] = Elem<DT>::to_f32((uint16_t)(w[0][j / 2] >> (16 * (j % 2))));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = Elem<DT>::to_f32(s[j]);
    }
}
template <int DT> __device__ __forceinline__ void store8(void* p, int64_t i, bool vec, const float (&v)[8])
{
    using St = typename Elem<DT>::storage;
    St* s = static_cast<St*>(p) + i;
    if (vec) {
        if constexpr (DT == DT_F32) {
            reinterpret_cast<f32x4_t*>(s)[0] = f32x4_t{v[0], v[1], v[2], v[3]};
            reinterpret_cast<f32x4_t*>(s)[1] = f32x4_t{v[4], v[5], v[6], v[7]};
        } else {
            u32x4_t w;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = (uint32_t)Elem<DT>::from_f32(v[2 * j]) | ((uint32_t)Elem<DT>::from_f32(v[2 * j + 1]) << 16);
            *reinterpret_cast<u32x4_t*>(s) = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] = Elem<DT>::from_f32(v[j]);
    }
}

// blockDim.x lanes walk a token's octets, blockDim.y tokens a block.
template <int BITS, int DT>
__global__ __launch_bounds__(256) void embedding_kernel(EmbedArgs a, bool vec)
{
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= a.T)
        return;
    const int64_t id = a.ids[t];
    const bool live = id >= 0 && id < a.V;
    const int octets = (int)(a.K / 8);
    const int64_t groups = a.K / a.gs, row_words = a.K * BITS / 32;
    const int gs8 = a.gs / 8;
    for (int o = (int)threadIdx.x; o < octets; o += (int)blockDim.x) {
        float v[8] = {};
        if (live) {
            codes8_at<BITS>(a.table.wq + id * row_words, o, v);
            const int64_t gi = id * groups + o / gs8;
            const float s = load_elem<DT>(a.table.scales, gi), b = load_elem<DT>(a.table.biases, gi);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __builtin_fmaf(v[j], s, b) * a.factor;
        }
        store8<DT>(a.out, t * a.K + 8 * o, vec, v);
    }
}

// ---- gradient

constexpr int kChunk = 2048;   // ids sorted by one block
constexpr int kPiece = 32;     // tokens summed by one wave

struct GradTables {
    uint64_t* keys;       // [chunks * kChunk] (id, token in chunk), sorted by chunk
    int32_t* token;       // [T] tokens in the order of (id, token)
    int32_t* id;          // [T] their ids (-1: outside the table)
    int32_t* start;       // [T] first place of the id's run
    int32_t* longrun;     // [T / kPiece + 1] first place of a cut run in this window, or -1
    float* partial;       // [2 (T / kPiece + 1)][2 G]
};
size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }
size_t tables(int64_t t, int64_t groups, char* p, GradTables* out)
{
    const int64_t chunks = (t + kChunk - 1) / kChunk, windows = t / kPiece + 1;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += up16(n);
        return p + o;
    };
    GradTables g{};
    g.keys = reinterpret_cast<uint64_t*>(take((size_t)chunks * kChunk * 8));
    g.token = reinterpret_cast<int32_t*>(take((size_t)t * 4));
    g.id = reinterpret_cast<int32_t*>(take((size_t)t * 4));
    g.start = reinterpret_cast<int32_t*>(take((size_t)t * 4));
    g.longrun = reinterpret_cast<int32_t*>(take((size_t)windows * 4));
    g.partial = reinterpret_cast<float*>(take(t > kPiece ? (size_t)windows * 2 * 2 * (size_t)groups * 4 : 0));
    if (out != nullptr)
        *out = g;
    return at;
}

// Sorts chunk blockIdx.x by (id, token): a bitonic network over LDS. Ids
// outside the table and the places past T sort last.
__global__ __launch_bounds__(1024) void embed_sort_kernel(const int32_t* __restrict__ ids, int64_t T, int64_t V,
                                                          GradTables g)
{
    __shared__ uint64_t key[kChunk];
    const int tid = (int)threadIdx.x;
    const int64_t base = (int64_t)blockIdx.x * kChunk;
    for (int i = tid; i < kChunk; i += 1024) {
        const int64_t t = base + i;
        uint32_t id = 0xFFFFFFFFu;
        if (t < T) {
            const int32_t v = ids[t];
            id = v >= 0 && v < V ? (uint32_t)v : 0xFFFFFFFEu;
        }
        key[i] = ((uint64_t)id << 32) | (uint32_t)i;
    }
    for (int64_t w = (int64_t)blockIdx.x * 1024 + tid; w < T / kPiece + 1; w += (int64_t)gridDim.x * 1024)
        g.longrun[w] = -1;
    for (int size = 2; size <= kChunk; size <<= 1)
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
            __syncthreads();
            const int i = 2 * tid - (tid & (stride - 1)), j = i + stride;
            const uint64_t x = key[i], y = key[j];
            if ((x > y) == ((i & size) == 0)) {
                key[i] = y;
                key[j] = x;
            }
        }
    __syncthreads();
    for (int i = tid; i < kChunk; i += 1024)
        g.keys[base + i] = key[i];
}

// The place of every token in the whole order and the first place of its
// id's run: counts of smaller keys over all chunks, whose ids pass through LDS.
__global__ __launch_bounds__(1024) void embed_rank_kernel(int64_t T, int chunks, GradTables g)
{
    __shared__ uint32_t other[kChunk];
    const int tid = (int)threadIdx.x;
    const int c = (int)blockIdx.x;
    uint64_t key[2];
    int rank[2], start[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        key[e] = g.keys[(int64_t)c * kChunk + tid + 1024 * e];
        rank[e] = tid + 1024 * e;
        start[e] = 0;
    }
    for (int d = 0; d < chunks; ++d) {
        __syncthreads();
        for (int i = tid; i < kChunk; i += 1024)
            other[i] = (uint32_t)(g.keys[(int64_t)d * kChunk + i] >> 32);
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t id = (uint32_t)(key[e] >> 32);
            int lo = 0, up = 0;   // ids below this one, ids up to it
            for (int step = kChunk; step > 0; step >>= 1) {
                if (lo + step <= kChunk && other[lo + step - 1] < id)
                    lo += step;
                if (up + step <= kChunk && other[up + step - 1] <= id)
                    up += step;
            }
            start[e] += lo;
            rank[e] += d < c ? up : d > c ? lo : 0;
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t id = (uint32_t)(key[e] >> 32);
        if (id == 0xFFFFFFFFu)
            continue;   // past T
        g.token[rank[e]] = c * kChunk + (int)(uint32_t)key[e];
        g.id[rank[e]] = id == 0xFFFFFFFEu ? -1 : (int32_t)id;
        g.start[rank[e]] = start[e];
    }
}

// Slot of the piece at place p of a cut run: two pieces that start in one
// window of kPiece places are never both first or both later pieces (of one
// run they are kPiece apart, and a cut run is longer than that).
__device__ __forceinline__ int64_t piece_slot(int64_t p, bool first) { return 2 * (p / kPiece) + (first ? 1 : 0); }

// Wave: the piece that starts at place p (if one does), 512 columns.
template <int BITS, int DT>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedGradArgs a, GradTables g, bool vec)
{
    const int lane = (int)threadIdx.x & 63;
    const int64_t p = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (p >= a.T)
        return;
    const int32_t id = g.id[p];
    const int64_t first = g.start[p];
    if (id < 0 || (p - first) % kPiece != 0)
        return;
    const bool mine = p + lane < a.T && lane <= kPiece && g.id[p + lane] == id;
    const uint64_t run = __ballot(mine);
    const int len = (int)__builtin_ctzll(~run);            // up to kPiece + 1
    const int rows = len < kPiece ? len : kPiece;
    const bool cut = p != first || len > kPiece;
    const int token = lane < rows ? g.token[p + lane] : 0;
    const int o = (int)blockIdx.y * 64 + lane, octets = (int)(a.K / 8);
    const bool live = o < octets;
    const int oc = live ? o : 0;

    float acc[8] = {};
    int i = 0;
    for (; i + 4 <= rows; i += 4) {
        float v[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            load8<DT>(a.dout, (int64_t)__shfl(token, i + j, 64) * a.K + 8 * oc, vec, v[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                acc[k] += v[j][k];
    }
    for (; i < rows; ++i) {
        float v[8];
        load8<DT>(a.dout, (int64_t)__shfl(token, i, 64) * a.K + 8 * oc, vec, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            acc[k] += v[k];
    }
    float q[8];
    codes8_at<BITS>(a.wq + (int64_t)id * (a.K * BITS / 32), oc, q);
    float s = 0.0f, b = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        s = __builtin_fmaf(q[k], acc[k], s);
        b += acc[k];
    }
    const int seg = a.gs / 8;                              // lanes of a group: 4, 8 or 16
    s = segment_reduce(s, seg) * a.factor;
    b = segment_reduce(b, seg) * a.factor;
    if (!live || (lane & (seg - 1)) > 1)
        return;
    const bool bias = (lane & (seg - 1)) == 1;
    const int64_t groups = a.K / a.gs, gi = o / seg;
    if (cut) {
        if (lane == 0 && blockIdx.y == 0 && p == first)
            g.longrun[p / kPiece] = (int32_t)p;
        g.partial[(piece_slot(p, p == first) * 2 + (bias ? 1 : 0)) * groups + gi] = bias ? b : s;
    } else {
        store_elem<DT>(bias ? a.dbiases : a.dscales, (int64_t)id * groups + gi, bias ? b : s);
    }
}

// The cut run that starts in window blockIdx.x: its pieces' sums in order.
template <int DT>
__global__ __launch_bounds__(256) void embed_join_kernel(EmbedGradArgs a, GradTables g)
{
    const int64_t p = g.longrun[blockIdx.x];
    if (p < 0)
        return;
    const int32_t id = g.id[p];
    const int64_t groups = a.K / a.gs;
    for (int64_t i = threadIdx.x; i < 2 * groups; i += 256) {
        float v = 0.0f;
        for (int64_t at = p; at < a.T && g.id[at] == id; at += kPiece)
            v += g.partial[piece_slot(at, at == p) * 2 * groups + i];
        if (i < groups)
            store_elem<DT>(a.dscales, (int64_t)id * groups + i, v);
        else
            store_elem<DT>(a.dbiases, (int64_t)id * groups + i - groups, v);
    }
}

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int BITS, int DT> hipError_t lookup(const EmbedArgs& a, hipStream_t st)
{
    int tx = 16;
    while (tx < 256 && tx < a.K / 8)
        tx *= 2;
    const int ty = 256 / tx;
    hipLaunchKernelGGL((embedding_kernel<BITS, DT>), dim3((unsigned)((a.T + ty - 1) / ty)), dim3(tx, ty), 0, st, a,
                       aligned16(a.out));
    return hipGetLastError();
}

template <int BITS, int DT> hipError_t grad(const EmbedGradArgs& a, hipStream_t st)
{
    const int64_t groups = a.K / a.gs;
    if (hipError_t e = launch_fill_zero(a.dscales, DT, a.V * groups, st); e != hipSuccess)
        return e;
    if (hipError_t e = launch_fill_zero(a.dbiases, DT, a.V * groups, st); e != hipSuccess)
        return e;
    if (a.T == 0)
        return hipSuccess;
    GradTables g{};
    tables(a.T, groups, static_cast<char*>(a.workspace), &g);
    const int chunks = (int)((a.T + kChunk - 1) / kChunk);
    hipLaunchKernelGGL(embed_sort_kernel, dim3(chunks), dim3(1024), 0, st, a.ids, a.T, a.V, g);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    hipLaunchKernelGGL(embed_rank_kernel, dim3(chunks), dim3(1024), 0, st, a.T, chunks, g);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    hipLaunchKernelGGL((embed_sum_kernel<BITS, DT>),
                       dim3((unsigned)((a.T + 3) / 4), (unsigned)((a.K / 8 + 63) / 64)), dim3(256), 0, st, a, g,
                       aligned16(a.dout));
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return e;
    if (a.T > kPiece) {
        hipLaunchKernelGGL((embed_join_kernel<DT>), dim3((unsigned)(a.T / kPiece + 1)), dim3(256), 0, st, a, g);
        return hipGetLastError();
    }
    return hipSuccess;
}

template <class F> hipError_t by_type(int bits, int dt, F&& f)
{
    auto with_bits = [&](auto B) {
        switch (dt) {
        case DT_F32: return f(B, std::integral_constant<int, DT_F32>{});
        case DT_F16: return f(B, std::integral_constant<int, DT_F16>{});
        case DT_BF16: return f(B, std::integral_constant<int, DT_BF16>{});
        }
        return hipErrorInvalidValue;
    };
    switch (bits) {
    case 2: return with_bits(std::integral_constant<int, 2>{});
    case 3: return with_bits(std::integral_constant<int, 3>{});
    case 4: return with_bits(std::integral_constant<int, 4>{});
    case 6: return with_bits(std::integral_constant<int, 6>{});
    case 8: return with_bits(std::integral_constant<int, 8>{});
    }
    return hipErrorInvalidValue;
}

} // namespace

size_t embedding_grad_workspace_bytes(int64_t t, int64_t k, int gs)
{
    return t == 0 ? 0 : tables(t, k / gs, nullptr, nullptr);
}

hipError_t launch_embedding(const EmbedArgs& a, hipStream_t st)
{
    return by_type(a.bits, a.dt, [&](auto B, auto D) {
        return lookup<decltype(B)::value, decltype(D)::value>(a, st);
    });
}

hipError_t launch_embedding_grad(const EmbedGradArgs& a, hipStream_t st)
{
    return by_type(a.bits, a.dt, [&](auto B, auto D) {
        return grad<decltype(B)::value, decltype(D)::value>(a, st);
    });
}

} // namespace qp
