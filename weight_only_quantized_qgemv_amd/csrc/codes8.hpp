// codes8.hpp — eight consecutive codes of a packed row, starting at a column
// that is a multiple of eight, as exact fp32 values. Their 8 * BITS bits start
// at a byte, but for 3- and 6-bit codes not at a word: those take the two
// words around them and a funnel shift. (Layout of emily
// lib/emily/quantization.ex, `dequantize_defn/1`: code i of a row at bit
// i * bits of its little-endian u32 stream.)
#pragma once

#include "codepair.hpp"
#include "common.hpp"

namespace qp {

template <int BITS> struct Codes8 {
    static constexpr int NW = (BITS == 2 || BITS == 4) ? 1 : 2;   // words held

    // Words of columns 8 * oct .. 8 * oct + 7 through ld(word index in the
    // row). The second word is needed, and so inside the row, only where the
    // codes reach it; need2() says so (3 bits; at 6 and 8 bits always).
    static __device__ __forceinline__ int word(int oct) { return (oct * BITS) >> 2; }
    static __device__ __forceinline__ bool need2(int oct)
    {
        return BITS == 3 ? ((oct * 3) & 3) > 1 : (BITS == 6 || BITS == 8);
    }

    // fp32 values of the eight codes.
    static __device__ __forceinline__ void to_f32(const uint32_t (&w)[NW], int oct, float (&q)[8])
    {
        if constexpr (BITS == 4 || BITS == 3) {
            uint32_t even, odd;   // codes 0, 2, 4, 6 and 1, 3, 5, 7, one per byte
            if constexpr (BITS == 4) {
                even = w[0] & 0x0F0F0F0Fu;
                odd = (w[0] >> 4) & 0x0F0F0F0Fu;
            } else {
                const uint32_t s = __builtin_amdgcn_alignbit(w[1], w[0], 8u * (uint32_t)((oct * 3) & 3));
                code_bytes3(s, 0u, even, odd);
            }
            const f32x2_t e01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.0f, false);
            const f32x2_t e23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(even, 512.0f, true);
            const f32x2_t o01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.0f, false);
            const f32x2_t o23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(odd, 512.0f, true);
            q[0] = e01.x; q[1] = o01.x; q[2] = e01.y; q[3] = o01.y;
            q[4] = e23.x; q[5] = o23.x; q[6] = e23.y; q[7] = o23.y;
        } else if constexpr (BITS == 2) {
            const uint32_t s = w[0] >> (16u * (uint32_t)(oct & 1));
            const uint32_t lo = s & 0x3333u, hi = (s >> 2) & 0x3333u;   // codes 0 2 4 6, 1 3 5 7
            const f32x2_t l0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 2.0f, 0);
            const f32x2_t l1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 2.0f, 1);
            const f32x2_t h0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(hi, 2.0f, 0);
            const f32x2_t h1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(hi, 2.0f, 1);
            q[0] = l0.x; q[1] = h0.x; q[2] = l0.y; q[3] = h0.y;
            q[4] = l1.x; q[5] = h1.x; q[6] = l1.y; q[7] = h1.y;
        } else if constexpr (BITS == 6) {
            const uint32_t sh = 16u * (uint32_t)(oct & 1);
            const uint32_t lo = __builtin_amdgcn_alignbit(w[1], w[0], sh);   // codes 0..3 in 24 bits
            const uint32_t a = code_bytes6(lo, 0u);
            // Codes 4..7: bits 24..47 of the piece.
            const uint32_t b = code_bytes6(__builtin_amdgcn_alignbit(w[1] >> sh, lo, 24u), 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[i] = (float)((a >> (8 * i)) & 0xFFu);
                q[4 + i] = (float)((b >> (8 * i)) & 0xFFu);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[i] = (float)((w[i / 4] >> (8 * (i % 4))) & 0xFFu);
        }
    }
};

// The eight codes of octet `oct` of a row of `words` words at `row`.
template <int BITS>
__device__ __forceinline__ void codes8_at(const uint32_t* __restrict__ row, int oct, float (&q)[8])
{
    using C = Codes8<BITS>;
    uint32_t w[C::NW];
    const int i = C::word(oct);
    w[0] = row[i];
    if constexpr (C::NW == 2)
        w[1] = C::need2(oct) ? row[i + 1] : 0u;
    C::to_f32(w, oct, q);
}

} // namespace qp
