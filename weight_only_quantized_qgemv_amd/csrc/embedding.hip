// embedding.hip — the packed embedding table: lookup with a factor,
//   out[t, k] = factor * (q[id, k] * s'[id, G] + b'[id, G]),   id = ids[t],
// and the gradient of its scales and biases,
//   dscales[v, G] = factor * sum_{t: ids[t] = v} sum_{k in G} q[v, k] dout[t, k],
//   dbiases[v, G] = factor * sum_{t: ids[t] = v} sum_{k in G} dout[t, k].
//
// The gradient sums a row's tokens in token order, by sorting. Chunks of 2048
// ids are sorted by (id, token), each by one block (a bitonic network, eight
// keys a thread: strides below 8 in registers, below 512 across the lanes, the
// three others through LDS); a token's place in the whole order is its place
// in its chunk plus, for every other chunk, the count of smaller keys there, or
// (many chunks) comes from merging sorted runs in pairs.
// A wave then takes a window of kWindow places x 512 columns, whatever runs of
// equal ids lie in it, so all waves move the same bytes: it streams the rows,
// and where a run ends in its window it meets the codes and is stored. The
// sums of a run that crosses windows go to fp32 partial sums, which a last
// launch adds in order. No atomics: the result does not depend on the launch.
// 8192 tokens of 4096 columns, 4-bit, bf16, a table of 32000 rows: sort 11 us,
// places 5, sums 18 (5 TB/s), join 4. Windows of single tokens with atomics on
// the table would need the sums in fp32 tables of 2 V K / gs values first.
#include <algorithm>

#include "codes8.hpp"
#include "common.hpp"
#include "model_ops.hpp"
#include "xgrad.hpp"

namespace qp {

namespace {

// Eight consecutive elements as they lie in memory: one or two 16-byte loads
// where the rows allow it, element loads otherwise.
template <int DT> struct Raw8 {
    using St = typename Elem<DT>::storage;
    static constexpr int NV = (int)sizeof(St) / 2;
    u32x4_t w[NV];
    __device__ __forceinline__ void load(const void* p, int64_t i, bool vec)
    {
        const St* s = static_cast<const St*>(p) + i;
        if (vec) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                w[j] = reinterpret_cast<const u32x4_t*>(s)[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4 * NV; ++j) {
                if constexpr (DT == DT_F32)
                    w[j / 4][j % 4] = __float_as_uint(s[j]);
                else
                    w[0][j] = (uint32_t)s[2 * j] | ((uint32_t)s[2 * j + 1] << 16);
            }
        }
    }
    __device__ __forceinline__ float get(int j) const
    {
        if constexpr (DT == DT_F32)
            return __uint_as_float(w[j / 4][j % 4]);
        else
            return Elem<DT>::to_f32((uint16_t)(w[0][j / 2] >> (16 * (j % 2))));
    }
};
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

// blockDim.x lanes walk a token's octets, blockDim.y tokens a block. Bound by the
// output's writes: 16384 tokens of 2048, 8-bit, f16 18.9 us (5.6 TB/s); a few
// tokens take the launch, 3 us.
template <int BITS, int DT>
__global__ __launch_bounds__(256) void embedding_kernel(EmbedArgs a, bool vec)
{
    const int64_t t = (blockIdx.x + (int64_t)blockIdx.y * gridDim.x) * blockDim.y + threadIdx.y;
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

constexpr int kChunk = 2048;    // ids sorted by one block
constexpr int kSortThreads = kChunk / 8;
constexpr int kWindow = 16;     // places summed by one wave
constexpr int kFillBlocks = 512;

constexpr int64_t kMergeFrom = 112;   // chunks from which runs are merged

struct GradTables {
    void* keys;           // [chunks * kChunk] (id, token in chunk), sorted by chunk (two chunks or more)
    uint64_t* merged;     // [chunks * kChunk] the merges' other buffer (kMergeFrom chunks or more)
    int32_t* token;       // [T] tokens in the order of (id, token)
    int32_t* id;          // [T] their ids (-1: outside the table; these come last)
    float* partial;       // [2 windows][2 G]: of the run a window begins with, and of the one it ends with
};
int64_t window_count(int64_t t) { return (t + kWindow - 1) / kWindow; }
size_t tables(int64_t t, int64_t groups, char* p, GradTables* out)
{
    const int64_t chunks = (t + kChunk - 1) / kChunk;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += up16(n);
        return p + o;
    };
    GradTables g{};
    g.keys = take(chunks > 1 ? (size_t)chunks * kChunk * 8 : 0);
    g.merged = reinterpret_cast<uint64_t*>(take(chunks >= kMergeFrom ? (size_t)chunks * kChunk * 8 : 0));
    g.token = reinterpret_cast<int32_t*>(take((size_t)t * 4));
    g.id = reinterpret_cast<int32_t*>(take((size_t)t * 4));
    g.partial = reinterpret_cast<float*>(take(t > kWindow ? (size_t)window_count(t) * 4 * (size_t)groups * 4 : 0));
    if (out != nullptr)
        *out = g;
    return at;
}

// A key: the id above the token's place in its chunk. Ids of tables up to
// 2^21 - 2 rows fit 32 bits with it, which halves the exchanges.
template <class K> struct Key;
template <> struct Key<uint32_t> {
    static constexpr int SHIFT = 11;
    static constexpr uint32_t PAST = 0x1FFFFFu;
};
template <> struct Key<uint64_t> {
    static constexpr int SHIFT = 32;
    static constexpr uint32_t PAST = 0xFFFFFFFFu;
};
static_assert(kChunk == 1 << Key<uint32_t>::SHIFT, "a chunk's places fit beside the id");
// Ids outside the table take the value before PAST, that of places past T.
template <class K> constexpr uint32_t kOutside = Key<K>::PAST - 1;

// The middle one of three (one v_med3_u32).
__device__ __forceinline__ uint32_t median(uint32_t a, uint32_t b, uint32_t c)
{
    return max(min(a, b), min(max(a, b), c));
}
// v of lane (lane ^ MASK), without a trip through LDS: quad permutes and row
// mirrors (i -> 7 - i, 15 - i), and the row swaps for the two widest.
template <int CTRL> __device__ __forceinline__ uint32_t dpp_u32(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int MASK> __device__ __forceinline__ uint32_t lane_xor(uint32_t v)
{
    if constexpr (MASK == 1) {
        return dpp_u32<0xB1>(v);                  // quad_perm [1,0,3,2]
    } else if constexpr (MASK == 2) {
        return dpp_u32<0x4E>(v);                  // quad_perm [2,3,0,1]
    } else if constexpr (MASK == 4) {
        return dpp_u32<0x1B>(dpp_u32<0x141>(v));  // row_half_mirror (^ 7), quad_perm [3,2,1,0] (^ 3)
    } else if constexpr (MASK == 8) {
        return dpp_u32<0x141>(dpp_u32<0x140>(v)); // row_mirror (^ 15), row_half_mirror (^ 7)
    } else if constexpr (MASK == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);   // rows (0,0,2,2), (1,1,3,3)
        return (threadIdx.x & 16) ? r[0] : r[1];
    } else {
        static_assert(MASK == 32, "one bit of the lane");
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);   // rows (0,1,0,1), (2,3,2,3)
        return (threadIdx.x & 32) ? r[0] : r[1];
    }
}
template <int MASK> __device__ __forceinline__ uint64_t lane_xor(uint64_t v)
{
    return ((uint64_t)lane_xor<MASK>((uint32_t)(v >> 32)) << 32) | lane_xor<MASK>((uint32_t)v);
}

// Blocks 0 .. chunks - 1 sort a chunk each; the others write zeros to the
// outputs (rows without tokens keep them), which takes about as long.
template <class K>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(const int32_t* __restrict__ ids, int64_t T, int64_t V,
                                                                 int chunks, GradTables g, char* z0, char* z1,
                                                                 int64_t zbytes)
{
    __shared__ K key[kChunk];
    const int tid = (int)threadIdx.x;
    if ((int)blockIdx.x >= chunks) {
        const int64_t me = ((int64_t)blockIdx.x - chunks) * kSortThreads + tid;
        const int64_t step = ((int64_t)gridDim.x - chunks) * kSortThreads;
        for (int o = 0; o < 2; ++o) {
            char* const z = o ? z1 : z0;
            // Whole 16-byte pieces from the first aligned byte on, elements around them.
            const int64_t head = (int64_t)((16 - reinterpret_cast<uintptr_t>(z) % 16) % 16) < zbytes
                ? (int64_t)((16 - reinterpret_cast<uintptr_t>(z) % 16) % 16) : zbytes;
            const int64_t pieces = (zbytes - head) / 16;
            for (int64_t i = me; i < pieces; i += step)
                reinterpret_cast<u32x4_t*>(z + head)[i] = u32x4_t{0, 0, 0, 0};
            for (int64_t i = 2 * me; i < head; i += 2 * step)
                *reinterpret_cast<uint16_t*>(z + i) = 0;
            for (int64_t i = head + 16 * pieces + 2 * me; i < zbytes; i += 2 * step)
                *reinterpret_cast<uint16_t*>(z + i) = 0;
        }
        return;
    }
    const int64_t base = (int64_t)blockIdx.x * kChunk;
    constexpr int SHIFT = Key<K>::SHIFT;
    K k[8];   // keys 8 tid .. 8 tid + 7
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int64_t t = base + 8 * tid + e;
        uint32_t id = Key<K>::PAST;
        if (t < T) {
            const int32_t v = ids[t];
            id = v >= 0 && v < V ? (uint32_t)v : kOutside<K>;
        }
        k[e] = ((K)id << SHIFT) | (K)(8 * tid + e);
    }
    // Exchange at one stride: element i keeps the smaller of the pair where its
    // stride bit and its size bit agree.
    auto keep = [&](const K (&other)[8], int size, int stride) {
        const bool low = (((8 * tid) & stride) == 0) == (((8 * tid) & size) == 0);
        if constexpr (sizeof(K) == 4) {
            // The median of the pair and the end of the range is one of the pair.
            const uint32_t end = low ? 0u : ~0u;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                k[e] = median(k[e], other[e], end);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                k[e] = (k[e] < other[e]) == low ? k[e] : other[e];
        }
    };
    auto in_thread = [&](int size, auto STRIDE) {
        constexpr int stride = decltype(STRIDE)::value;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if ((e & stride) == 0) {
                const K x = k[e], y = k[e ^ stride];
                const bool up = ((8 * tid + e) & size) == 0;
                const bool swap = (x > y) == up;
                k[e] = swap ? y : x;
                k[e ^ stride] = swap ? x : y;
            }
    };
#pragma unroll 1
    for (int size = 2; size <= kChunk; size <<= 1) {
        int stride = size >> 1;
#pragma unroll 1
        for (; stride >= 512; stride >>= 1) {
            K other[8];
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e)
                key[e * kSortThreads + tid] = k[e];
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e)
                other[e] = key[e * kSortThreads + (tid ^ (stride / 8))];
            keep(other, size, stride);
        }
        static_for<6>([&](auto L) {
            constexpr int mask = 32 >> decltype(L)::value;
            if (8 * mask <= stride) {   // uniform
                K other[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    other[e] = lane_xor<mask>(k[e]);
                keep(other, size, 8 * mask);
            }
        });
        if (size >= 8)
            in_thread(size, std::integral_constant<int, 4>{});
        if (size >= 4)
            in_thread(size, std::integral_constant<int, 2>{});
        in_thread(size, std::integral_constant<int, 1>{});
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int place = 8 * tid + e;
        const uint32_t id = (uint32_t)(k[e] >> SHIFT);
        if (chunks >= kMergeFrom) {   // 64-bit keys: the token in the place of its chunk's one
            static_cast<K*>(g.keys)[base + place] = k[e] + (K)base;
        } else if (chunks > 1) {
            static_cast<K*>(g.keys)[base + place] = k[e];
        } else if (id != Key<K>::PAST) {
            g.token[place] = (int)((uint32_t)k[e] & (kChunk - 1));
            g.id[place] = id == kOutside<K> ? -1 : (int32_t)id;
        }
    }
}

// The place of every token in the whole order: its place in its chunk, and
// for every other chunk, whose ids pass through LDS, the ids up to this one
// (earlier chunks) or below it (later ones).
template <class K>
__global__ __launch_bounds__(256) void embed_rank_kernel(int chunks, GradTables g)
{
    __shared__ uint32_t other[kChunk];
    const int tid = (int)threadIdx.x;
    const int64_t at = (int64_t)blockIdx.x * 256 + tid;
    const int c = (int)(at / kChunk);
    const K* const keys = static_cast<const K*>(g.keys);
    const K key = keys[at];
    const uint32_t id = (uint32_t)(key >> Key<K>::SHIFT);
    int64_t rank = at - (int64_t)c * kChunk;
    for (int d = 0; d < chunks; ++d) {
        if (d == c)
            continue;   // the whole block is of one chunk
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kChunk / 256; ++i)
            other[tid + 256 * i] = (uint32_t)(keys[(int64_t)d * kChunk + tid + 256 * i] >> Key<K>::SHIFT);
        __syncthreads();
        const uint32_t below = d < c ? id + 1 : id;   // count the ids below this
        int n = 0;
#pragma unroll
        for (int step = kChunk; step > 0; step >>= 1)
            if (n + step <= kChunk && other[n + step - 1] < below)
                n += step;
        rank += n;
    }
    if (id == Key<K>::PAST)
        return;
    g.token[rank] = c * kChunk + (int)((uint32_t)key & (kChunk - 1));
    g.id[rank] = id == kOutside<K> ? -1 : (int32_t)id;
}

// One pass over sorted runs of `run` keys (whole chunks; the last may be shorter):
// runs 2 i and 2 i + 1 become one. All keys differ. A block makes one chunk of
// the result: how much of it comes from either run is found by bisection on the
// diagonal, those keys come to LDS, and each one's place there is its own plus
// the count of smaller keys of the other part. The last pass leaves the tokens
// and ids that the sums read. Ranking every key against every chunk takes time
// as the square of the chunks. The whole gradient of 64 columns: 2^17 tokens (64
// chunks) 111 us so, 143 by merging in six passes; 2^18 203 and 186; 2^20 1616 and
// 382; at 2^29, the most a call takes, a ranking would run for minutes.
template <bool LAST>
__global__ __launch_bounds__(256) void embed_merge_kernel(const uint64_t* __restrict__ in, uint64_t* __restrict__ out,
                                                          int64_t total, int64_t run, GradTables g)
{
    __shared__ uint64_t part[kChunk];
    const int tid = (int)threadIdx.x;
    const int64_t at = (int64_t)blockIdx.x * kChunk;          // the result's chunk
    const int64_t a0 = at / (2 * run) * (2 * run);            // the pair's runs: from a0 and b0, la and lb long
    const int64_t la = total - a0 < run ? total - a0 : run, b0 = a0 + la;
    const int64_t lb = total - b0 < run ? total - b0 : run;
    // Of the first d keys of the merged pair, those of its first run.
    auto taken = [&](int64_t d) {
        int64_t lo = d > lb ? d - lb : 0, hi = d < la ? d : la;
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (in[a0 + mid] < in[b0 + d - 1 - mid])
                lo = mid + 1;
            else
                hi = mid;
        }
        return lo;
    };
    const int64_t d0 = at - a0, i0 = taken(d0), i1 = taken(d0 + kChunk);
    const int na = (int)(i1 - i0);
    const int64_t j0 = d0 - i0;
#pragma unroll
    for (int e = 0; e < kChunk / 256; ++e) {
        const int x = tid + 256 * e;
        part[x] = x < na ? in[a0 + i0 + x] : in[b0 + j0 + (x - na)];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kChunk / 256; ++e) {
        const int x = tid + 256 * e;
        const uint64_t key = part[x];
        int lo = x < na ? na : 0;                             // count the other part's smaller keys
        const int from = lo;
        int hi = x < na ? kChunk : na;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (part[mid] < key)
                lo = mid + 1;
            else
                hi = mid;
        }
        const int64_t place = at + (x < na ? x : x - na) + (lo - from);
        if constexpr (LAST) {
            const uint32_t id = (uint32_t)(key >> Key<uint64_t>::SHIFT);
            if (id != Key<uint64_t>::PAST) {
                g.token[place] = (int32_t)(uint32_t)key;
                g.id[place] = id == kOutside<uint64_t> ? -1 : (int32_t)id;
            }
        } else {
            out[place] = key;
        }
    }
}

// Wave: the places of window w, 512 columns (lane l columns 8 l .. 8 l + 7 of
// them), rows in batches of RB with their codes beside them.
template <int BITS, int DT>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedGradArgs a, GradTables g, bool vec)
{
    using C8 = Codes8<BITS>;
    constexpr int RB = DT == DT_F32 ? 4 : 8;
    const int lane = (int)threadIdx.x & 63;
    const int64_t col_tiles = (a.K / 8 + 63) / 64;
    const int64_t item = (blockIdx.x + (int64_t)blockIdx.y * gridDim.x) * 4 + (threadIdx.x >> 6);
    const int64_t w = item / col_tiles, p0 = w * kWindow;
    if (p0 >= a.T)
        return;
    const int o = (int)(item % col_tiles) * 64 + lane, octets = (int)(a.K / 8);
    const bool live = o < octets;
    const int oc = live ? o : 0;
    // Lane i: the window's place i - 1 (lane 0: the place before it; lane
    // kWindow + 1: the one after).
    const int64_t pl = p0 - 1 + lane;
    const bool in = lane < kWindow + 2 && pl >= 0 && pl < a.T;
    const int my_id = in ? g.id[pl] : -1;
    const int my_token = in ? g.token[pl] : 0;
    const int count = (int)(a.T - p0 < kWindow ? a.T - p0 : kWindow);
    const int seg = a.gs / 8;                              // lanes of a group: 4, 8 or 16
    const int64_t groups = a.K / a.gs, row_words = a.K * BITS / 32;
    const int before = __shfl(my_id, 0, 64), after = __shfl(my_id, count + 1, 64);

    float acc[8] = {};
    int from = 0;   // first place of the run in progress
    for (int b0 = 0; b0 < count; b0 += RB) {
        Raw8<DT> v[RB];
        uint32_t cw[RB][C8::NW];
#pragma unroll
        for (int j = 0; j < RB; ++j) {
            // Places past the window's end repeat its last one, and places
            // outside the table read row 0: neither is used.
            const int i = b0 + j < count ? b0 + j : count - 1;
            const int t = __shfl(my_token, i + 1, 64);
            int id = __shfl(my_id, i + 1, 64);
            id = id < 0 ? 0 : id;
            v[j].load(a.dout, (int64_t)t * a.K + 8 * oc, vec);
            const uint32_t* row = a.wq + (int64_t)id * row_words;
            cw[j][0] = row[C8::word(oc)];
            if constexpr (C8::NW == 2)
                cw[j][1] = C8::need2(oc) ? row[C8::word(oc) + 1] : 0u;
        }
        __builtin_amdgcn_sched_barrier(0);   // the whole batch is asked for before any of it is used
#pragma unroll
        for (int j = 0; j < RB; ++j) {
            const int i = b0 + j;
            if (i >= count)
                break;
            const int id = __shfl(my_id, i + 1, 64), next = __shfl(my_id, i + 2, 64);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                acc[k] += v[j].get(k);
            if (i + 1 < count && next == id)
                continue;   // the run goes on in the window (uniform)
            if (id >= 0) {
                float q[8];
                C8::to_f32(cw[j], oc, q);
                float s = 0.0f, b = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s = __builtin_fmaf(q[k], acc[k], s);
                    b += acc[k];
                }
                s = segment_reduce(s, seg) * a.factor;
                b = segment_reduce(b, seg) * a.factor;
                const bool first = from == 0 && w > 0 && before == id;   // came from the window before
                const bool last = i + 1 == count && after == id && p0 + count < a.T;
                const int side = lane & (seg - 1);
                if (live && side < 2) {
                    const int64_t gi = o / seg;
                    const float r = side ? b : s;
                    if (first || last)
                        g.partial[((2 * w + (first ? 0 : 1)) * 2 + side) * groups + gi] = r;
                    else
                        store_elem<DT>(side ? a.dbiases : a.dscales, (int64_t)id * groups + gi, r);
                }
            }
            from = i + 1;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                acc[k] = 0.0f;
        }
    }
}

// The run that starts in window w, the block's, and crosses its end: its windows'
// sums (the first in the slot of a window's last run, the others in that of
// its first). 512 / (2 G) groups of threads take a contiguous share of the
// windows each, in order, and their sums are added in order: a run of
// thousands of tokens (padding, say) does not become one thread's chain.
constexpr int kJoinThreads = 512;
template <int DT>
__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(EmbedGradArgs a, GradTables g)
{
    __shared__ float part[kJoinThreads];
    __shared__ int s_len;
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int64_t w = blockIdx.x + (int64_t)blockIdx.y * gridDim.x, end = (w + 1) * kWindow;
    if (end >= a.T)
        return;
    const int32_t id = g.id[end];
    if (id < 0 || g.id[end - 1] != id)
        return;
    if (w > 0 && g.id[w * kWindow] == id && g.id[w * kWindow - 1] == id)
        return;   // came from an earlier window
    // Windows that the run reaches after this one: the first wave counts.
    if (tid < 64) {
        int len = 0;
        for (;; len += 64) {
            const int64_t at = (w + 1 + len + lane) * kWindow;
            const uint64_t same = __ballot(at < a.T && g.id[at < a.T ? at : 0] == id);
            if (same != ~0ull) {
                len += (int)__builtin_ctzll(~same);
                break;
            }
        }
        if (tid == 0)
            s_len = len;
    }
    __syncthreads();
    const int len = s_len;
    const int64_t groups = a.K / a.gs;
    const int values = (int)(2 * groups < kJoinThreads ? 2 * groups : kJoinThreads);
    const int shares = kJoinThreads / values, share = tid / values;
    const int per = (len + shares - 1) / shares;
    for (int64_t i0 = 0; i0 < 2 * groups; i0 += values) {
        const int64_t i = i0 + tid % values;
        float v = 0.0f;
        if (share < shares && i < 2 * groups) {
            const int lo = share * per, hi = lo + per < len ? lo + per : len;
            if (share == 0)
                v = g.partial[(2 * w + 1) * 2 * groups + i];
#pragma unroll 8
            for (int x = lo; x < hi; ++x)
                v += g.partial[2 * (w + 1 + x) * 2 * groups + i];
        }
        __syncthreads();
        part[tid] = v;
        __syncthreads();
        if (share == 0 && i < 2 * groups) {
            for (int x = 1; x < shares; ++x)
                v += part[x * values + tid];
            if (i < groups)
                store_elem<DT>(a.dscales, (int64_t)id * groups + i, v);
            else
                store_elem<DT>(a.dbiases, (int64_t)id * groups + i - groups, v);
        }
    }
}

template <int BITS, int DT> hipError_t lookup(const EmbedArgs& a, hipStream_t st)
{
    int tx = 16;
    while (tx < 256 && tx < a.K / 8)
        tx *= 2;
    const int ty = 256 / tx;
    hipLaunchKernelGGL((embedding_kernel<BITS, DT>), wide_grid((a.T + ty - 1) / ty, 256), dim3(tx, ty), 0, st, a,
                       aligned16(a.out));
    return hipGetLastError();
}

template <int BITS, int DT> hipError_t grad(const EmbedGradArgs& a, hipStream_t st)
{
    const int64_t groups = a.K / a.gs;
    GradTables g{};
    tables(a.T, groups, static_cast<char*>(a.workspace), &g);
    const int chunks = (int)((a.T + kChunk - 1) / kChunk);
    const int64_t zbytes = a.V * groups * (int64_t)sizeof(typename Elem<DT>::storage);
    const int fill = (int)std::min<int64_t>(zbytes / (16 * kSortThreads) + 1, kFillBlocks);
    auto order = [&](auto key) {
        using K = decltype(key);
        hipLaunchKernelGGL(embed_sort_kernel<K>, dim3(chunks + fill), dim3(kSortThreads), 0, st, a.ids, a.T, a.V, chunks,
                           g, static_cast<char*>(a.dscales), static_cast<char*>(a.dbiases), zbytes);
        if (hipError_t e = hipGetLastError(); e != hipSuccess || chunks <= 1)
            return e;
        if (chunks >= kMergeFrom) {
            const int64_t total = (int64_t)chunks * kChunk;
            uint64_t *in = static_cast<uint64_t*>(g.keys), *out = g.merged;
            for (int64_t run = kChunk; run < total; run *= 2) {
                if (2 * run < total)
                    hipLaunchKernelGGL(embed_merge_kernel<false>, dim3(chunks), dim3(256), 0, st, in, out, total, run, g);
                else
                    hipLaunchKernelGGL(embed_merge_kernel<true>, dim3(chunks), dim3(256), 0, st, in, out, total, run, g);
                if (hipError_t e = hipGetLastError(); e != hipSuccess)
                    return e;
                std::swap(in, out);
            }
            return hipSuccess;
        }
        hipLaunchKernelGGL(embed_rank_kernel<K>, dim3((unsigned)chunks * (kChunk / 256)), dim3(256), 0, st, chunks, g);
        return hipGetLastError();
    };
    const bool narrow = a.V < Key<uint32_t>::PAST && chunks < kMergeFrom;
    if (hipError_t e = narrow ? order(uint32_t{}) : order(uint64_t{}); e != hipSuccess || a.T == 0)
        return e;
    const int64_t windows = window_count(a.T), items = windows * ((a.K / 8 + 63) / 64);
    hipLaunchKernelGGL((embed_sum_kernel<BITS, DT>), wide_grid((items + 3) / 4, 256), dim3(256), 0, st, a, g,
                       aligned16(a.dout));
    if (hipError_t e = hipGetLastError(); e != hipSuccess || windows == 1)
        return e;
    hipLaunchKernelGGL((embed_join_kernel<DT>), wide_grid(windows - 1, kJoinThreads), dim3(kJoinThreads), 0, st, a, g);
    return hipGetLastError();
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
