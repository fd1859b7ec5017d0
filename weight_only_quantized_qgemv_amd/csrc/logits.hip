// logits.hip — the controls on a batch of logit rows before sampling. With
// row b's tokens so far (prompt, then made), z the fp32 logit of token v and
// c the times v was made:
//   v seen at all:  z = z > 0 ? z / repetition : z * repetition
//   then            z = z - frequency * c - presence * (c > 0) + bias(b, v)
//   v not allowed:  z = -inf
// rounded once to the logits' type.
//
// A block takes a tile of one row's vocabulary, 16 logits a thread in registers.
// It counts the row's tokens that fall into the tile in LDS (integer atomics:
// their order changes nothing), applies the penalties, then uses the same LDS
// for the last bias entry of each token. Bound by the read and write of the
// logits; the row's tokens are read once per tile, from L2. One word of LDS a
// token and 16 tokens a thread let 64 rows of 128K tokens be on the GPU at
// once; with a word each for counts and biases it takes two rounds. 64 rows of
// 131071 with 4000 tokens each, bf16: 14.4 us, 2.5 TB/s (with rows read twice and
// two words a token 40.7).
#include <algorithm>

#include "common.hpp"
#include "model_ops.hpp"
#include "span.hpp"

namespace qp {

namespace {

// Sixteen bytes at any element's address (rows of an odd vocabulary).
template <int DT> struct Wide;
template <> struct Wide<DT_F32> { typedef u32x4_t type __attribute__((aligned(4))); };
template <> struct Wide<DT_F16> { typedef u32x4_t type __attribute__((aligned(2))); };
template <> struct Wide<DT_BF16> { typedef u32x4_t type __attribute__((aligned(2))); };

constexpr int kThreads = 512, kSets = 2, kTile = kThreads * kSets * 8;

template <int DT>
__global__ __launch_bounds__(kThreads) void logits_kernel(LogitsArgs a, int tiles)
{
    using E = Elem<DT>;
    using St = typename E::storage;
    constexpr int NV = 8 * (int)sizeof(St) / 16;
    __shared__ __attribute__((aligned(16))) uint32_t slot[kTile];
    const int64_t block = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    const int64_t row = block / tiles;
    if (row >= a.rows)
        return;
    const int v0 = (int)(block % tiles) * kTile;
    const int n = (int)(a.vocab - v0 < kTile ? a.vocab - v0 : kTile);
    const int tid = (int)threadIdx.x;
    const bool hist = a.history != nullptr, bias = a.bias_ids != nullptr;

    // Everything whose address is known is asked for first: the tile's logits
    // (set s of a thread: eight from 8 (tid + s kThreads) on), the row's
    // parameters, the mask's byte of each set (a tile starts at a whole word,
    // and a word's bytes are in order), the ends of the row's tokens and
    // biases; then the first tokens. It arrives while the counts are cleared.
    const St* in = static_cast<const St*>(a.logits) + row * a.in_stride + v0;
    u32x4_t raw[kSets][NV];
    uint32_t allowed[kSets];
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
        const int i0 = 8 * (tid + s * kThreads);
        if (i0 + 8 <= n) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                raw[s][j] = *reinterpret_cast<const typename Wide<DT>::type*>(in + i0 + j * (16 / (int)sizeof(St)));
        }
        allowed[s] = 0xFFu;
        if (a.mask != nullptr && i0 < n)
            allowed[s] = a.mask[row * a.mask_stride + ((v0 + i0) >> 5)] >> (i0 & 31);
    }
    const float rep = a.repetition != nullptr ? a.repetition[row] : 1.0f;
    const float freq = a.frequency != nullptr ? a.frequency[row] : 0.0f;
    const float pres = a.presence != nullptr ? a.presence[row] : 0.0f;
    Span tokens{0, 0}, entries{0, 0};
    uint32_t made = 0;   // the first token that is not the prompt's
    if (hist) {
        tokens = held_span(a.offsets[row], a.offsets[row + 1], a.history_len);
        const int32_t prompt = a.prompt_lens != nullptr ? a.prompt_lens[row] : 0;
        made = prompt > 0 ? (uint32_t)prompt : 0u;
    }
    if (bias)
        entries = held_span(a.bias_offsets[row], a.bias_offsets[row + 1], a.bias_len);
    const int32_t* const history = a.history + tokens.first;   // all indices below count from the row's first
    const int32_t* const bias_ids = a.bias_ids + entries.first;
    constexpr uint32_t U = 4;
    int32_t t[U], tb = -1;
    auto fetch = [&](uint32_t i) {
#pragma unroll
        for (uint32_t j = 0; j < U; ++j)
            t[j] = i + j * kThreads < tokens.count ? history[i + j * kThreads] : -1;
    };
    fetch((uint32_t)tid);
    if ((uint32_t)tid < entries.count)
        tb = bias_ids[tid];
    auto clear = [&]() {
#pragma unroll
        for (int j = 0; j < 2 * kSets; ++j)
            reinterpret_cast<u32x4_t*>(slot)[tid + j * kThreads] = u32x4_t{0, 0, 0, 0};
    };
    auto slots = [&](int s, uint32_t (&c)[8]) {
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const u32x4_t w = *reinterpret_cast<const u32x4_t*>(slot + 8 * (tid + s * kThreads) + j);
            c[j] = w.x; c[j + 1] = w.y; c[j + 2] = w.z; c[j + 3] = w.w;
        }
    };
    // Slot: bit 0, in the prompt; the rest, times made.
    if (hist) {
        clear();
        __syncthreads();
        for (uint32_t i = (uint32_t)tid; i < tokens.count; i += U * kThreads) {
            if (i != (uint32_t)tid)
                fetch(i);
#pragma unroll
            for (uint32_t j = 0; j < U; ++j) {
                const uint32_t v = (uint32_t)t[j] - (uint32_t)v0;
                if (t[j] >= v0 && v < (uint32_t)n) {
                    if (i + j * kThreads >= made)
                        atomicAdd(&slot[v], 2u);
                    else
                        atomicOr(&slot[v], 1u);
                }
            }
        }
        __syncthreads();
    }
    float z[kSets][8];
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
        const int i0 = 8 * (tid + s * kThreads);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (i0 + 8 <= n) {
                if constexpr (DT == DT_F32)
                    z[s][j] = __uint_as_float(raw[s][j / 4][j % 4]);
                else
                    z[s][j] = E::to_f32((uint16_t)(raw[s][0][j / 2] >> (16 * (j % 2))));
            } else {
                z[s][j] = i0 + j < n ? E::to_f32(in[i0 + j]) : 0.0f;
            }
        }
        if (hist) {
            uint32_t c[8];
            slots(s, c);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c[j] != 0) {
                    z[s][j] = z[s][j] > 0.0f ? z[s][j] / rep : z[s][j] * rep;
                    if (c[j] > 1)
                        z[s][j] = z[s][j] - freq * (float)(c[j] >> 1) - pres;
                }
        }
    }
    // Slot: the token's last bias entry + 1.
    if (bias) {
        __syncthreads();   // the counts have been read
        clear();
        __syncthreads();
        for (uint32_t i = (uint32_t)tid; i < entries.count; i += kThreads) {
            if (i != (uint32_t)tid)
                tb = bias_ids[i];
            const uint32_t v = (uint32_t)tb - (uint32_t)v0;
            if (tb >= v0 && v < (uint32_t)n)
                atomicMax(&slot[v], i + 1u);
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            uint32_t e[8];
            slots(s, e);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (e[j] != 0)
                    z[s][j] += a.bias_values[entries.first + e[j] - 1];
        }
    }
    St* out = static_cast<St*>(a.out) + row * a.out_stride + v0;
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
        const int i0 = 8 * (tid + s * kThreads);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (((allowed[s] >> j) & 1u) == 0)
                z[s][j] = -__builtin_inff();
        if (i0 + 8 <= n) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                u32x4_t w;
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    if constexpr (DT == DT_F32)
                        w[l] = __float_as_uint(z[s][4 * j + l]);
                    else
                        w[l] = (uint32_t)E::from_f32(z[s][2 * l]) | ((uint32_t)E::from_f32(z[s][2 * l + 1]) << 16);
                }
                *reinterpret_cast<typename Wide<DT>::type*>(out + i0 + j * (16 / (int)sizeof(St))) = w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i0 + j < n)
                    out[i0 + j] = E::from_f32(z[s][j]);
        }
    }
}

template <int DT> hipError_t run(const LogitsArgs& a, hipStream_t st)
{
    const int64_t tiles = (a.vocab + kTile - 1) / kTile;
    hipLaunchKernelGGL((logits_kernel<DT>), wide_grid(tiles * a.rows, kThreads), dim3(kThreads), 0, st, a, (int)tiles);
    return hipGetLastError();
}

} // namespace

hipError_t launch_logits_adjust(const LogitsArgs& a, hipStream_t st)
{
    switch (a.dt) {
    case DT_F32: return run<DT_F32>(a, st);
    case DT_F16: return run<DT_F16>(a, st);
    case DT_BF16: return run<DT_BF16>(a, st);
    }
    return hipErrorInvalidValue;
}

} // namespace qp
