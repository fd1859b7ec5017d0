// logits.hip — the controls on a batch of logit rows before sampling. With
// row b's tokens so far (prompt, then made), z the fp32 logit of token v and
// c the times v was made:
//   v seen at all:  z = z > 0 ? z / repetition : z * repetition
//   then            z = z - frequency * c - presence * (c > 0) + bias(b, v)
//   v not allowed:  z = -inf
// rounded once to the logits' type.
//
// A block takes a tile of one row's vocabulary. It counts the row's tokens
// that fall into the tile in LDS (integer atomics: their order changes
// nothing) and notes the last bias entry of each token there, then streams
// the tile once. Bound by the read and write of the logits; the row's tokens
// are read once per tile, from L2.
#include <algorithm>

#include "common.hpp"
#include "model_ops.hpp"

namespace qp {

namespace {

template <int DT, int TILE>
__global__ __launch_bounds__(256) void logits_kernel(LogitsArgs a, int64_t tiles, bool vec)
{
    using E = Elem<DT>;
    using St = typename E::storage;
    constexpr int VN = 16 / (int)sizeof(St);
    __shared__ uint32_t count[TILE];   // bit 0: in the prompt; bits 1..: times made
    __shared__ uint32_t entry[TILE];   // last bias entry + 1
    const int64_t row = (int64_t)blockIdx.x / tiles;
    const int64_t v0 = ((int64_t)blockIdx.x % tiles) * TILE;
    const int n = (int)(a.vocab - v0 < TILE ? a.vocab - v0 : TILE);
    const int tid = (int)threadIdx.x;
    const bool hist = a.history != nullptr, bias = a.bias_ids != nullptr;
    if (hist || bias) {
        for (int i = tid; i < TILE; i += 256) {
            count[i] = 0;
            entry[i] = 0;
        }
        __syncthreads();
    }
    if (hist) {
        int64_t lo = a.offsets[row], hi = a.offsets[row + 1];
        lo = lo < 0 ? 0 : lo;
        hi = hi < a.history_len ? hi : a.history_len;
        const int64_t made = lo + (a.prompt_lens != nullptr ? a.prompt_lens[row] : 0);
        for (int64_t i = lo + tid; i < hi; i += 256) {
            const int64_t v = a.history[i] - v0;
            if (v >= 0 && v < n) {
                if (i >= made)
                    atomicAdd(&count[v], 2u);
                else
                    atomicOr(&count[v], 1u);
            }
        }
    }
    int64_t b0 = 0;
    if (bias) {
        int64_t hi = a.bias_offsets[row + 1];
        b0 = a.bias_offsets[row];
        b0 = b0 < 0 ? 0 : b0;
        hi = hi < a.bias_len ? hi : a.bias_len;
        for (int64_t i = b0 + tid; i < hi; i += 256) {
            const int64_t v = a.bias_ids[i] - v0;
            if (v >= 0 && v < n)
                atomicMax(&entry[v], (uint32_t)(i - b0) + 1u);
        }
    }
    if (hist || bias)
        __syncthreads();
    const float rep = a.repetition != nullptr ? a.repetition[row] : 1.0f;
    const float freq = a.frequency != nullptr ? a.frequency[row] : 0.0f;
    const float pres = a.presence != nullptr ? a.presence[row] : 0.0f;
    const uint32_t* mask = a.mask != nullptr ? a.mask + row * a.mask_stride : nullptr;
    const St* in = static_cast<const St*>(a.logits) + row * a.in_stride + v0;
    St* out = static_cast<St*>(a.out) + row * a.out_stride + v0;
    auto adjust = [&](int i, float z) {
        if (hist) {
            const uint32_t c = count[i];
            if (c != 0) {
                z = z > 0.0f ? z / rep : z * rep;
                if (c > 1)
                    z = z - freq * (float)(c >> 1) - pres;
            }
        }
        if (bias) {
            const uint32_t e = entry[i];
            if (e != 0)
                z += a.bias_values[b0 + (int64_t)e - 1];
        }
        if (mask != nullptr) {
            const int64_t v = v0 + i;
            if (((mask[v >> 5] >> (v & 31)) & 1u) == 0)
                z = -__builtin_inff();
        }
        return z;
    };
    int i = tid * VN;
    if (vec) {
        for (; i + VN <= n; i += 256 * VN) {
            u32x4_t w = *reinterpret_cast<const u32x4_t*>(in + i);
            float z[VN];
#pragma unroll
            for (int j = 0; j < VN; ++j) {
                if constexpr (DT == DT_F32)
                    z[j] = adjust(i + j, __uint_as_float(w[j]));
                else
                    z[j] = adjust(i + j, E::to_f32((uint16_t)(w[j / 2] >> (16 * (j % 2)))));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (DT == DT_F32)
                    w[j] = __float_as_uint(z[j]);
                else
                    w[j] = (uint32_t)E::from_f32(z[2 * j]) | ((uint32_t)E::from_f32(z[2 * j + 1]) << 16);
            }
            *reinterpret_cast<u32x4_t*>(out + i) = w;
        }
        for (int j = i; j < n && j < i + VN; ++j)
            out[j] = E::from_f32(adjust(j, E::to_f32(in[j])));
    } else {
        for (int j = tid; j < n; j += 256)
            out[j] = E::from_f32(adjust(j, E::to_f32(in[j])));
    }
}

template <int DT> hipError_t run(const LogitsArgs& a, hipStream_t st)
{
    constexpr int TILE = 4096;
    constexpr int64_t ES = DT == DT_F32 ? 4 : 2;
    const int64_t tiles = (a.vocab + TILE - 1) / TILE;
    auto rows16 = [&](const void* p, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.rows == 1 || (stride * ES) % 16 == 0);
    };
    const bool vec = rows16(a.logits, a.in_stride) && rows16(a.out, a.out_stride);
    hipLaunchKernelGGL((logits_kernel<DT, TILE>), dim3((unsigned)(tiles * a.rows)), dim3(256), 0, st, a, tiles, vec);
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
