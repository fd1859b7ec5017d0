// loss_tile.hpp — the matrix-core tile kernel of the cross entropy over a packed
// head (loss.hip): a block computes a tile of z = x W^T, 16-bit x, and closes it to
// each row's maximum and sum of exponentials, or to dz. The logits stay in registers.
//
// The logits are fp32 results (a loss of 15 is asked for to 1e-5 of itself), so the
// weights are not rounded to 16 bits as the other tile kernels round them (bf16: 2.6e-4
// of the loss). A row's group g of weights is q s + b:
//   z = sum_g s_g (sum_{k in g} q_k x_k) + sum_g b_g X_g,   X_g = sum_{k in g} x_k.
// The codes are exact 16-bit operands (codepair.hpp); a group's sum comes out of the
// matrix instructions in fp32 and is scaled and added by the vector units, 16 FMAs for
// each 4 (groups of 32: 2) of 32x32x16, beside the next tile's. The biases are a second,
// short contraction over the groups, with X in two 16-bit parts: exact to 2^-17 of X
// (bf16; fp16, where a power of two brings the row's largest |X| to 2^14 .. 2^15: 2^-22
// of X, and 2^-39 of the largest where that is more), G / 32 steps of 64 more.
//
// prep_x writes x once in the order that a unit's code pairs come in, rows filled
// up to whole 64-wide steps, and X; prep_w the scales transposed (a step's scales
// of a tile are then 512 bytes in a row) and the biases in rows of whole 16-byte
// pieces. Together a few microseconds beside the tiles.
//
// fp32 x is three steps of 16-bit parts, 24 bits together, so that its products are exact
// on the same instructions, 16 times as fast as the fp32 ones.
//
// 4096 rows of 4096 x 32000, 4-bit bf16: 1000 us with its layout and close, 1.07 PFLOP/s
// where a large library product of 16-bit weights reaches 1.36. It is bound by the vector
// units beside the matrix pipes, and by power: of 1.93 million cycles (1.74 GHz) the
// matrix pipes are busy in 55%, and 7 vector instructions stand beside each matrix
// instruction of 32 cycles, 4 of them the scaling.
//
// Waves of 32 FM rows x 64 columns, WMW x 4 of them; steps of 64 k; x in NA and codes
// and scales in NC stages of LDS, by DMA, with the swizzles of gemm_core.hpp.
#pragma once

#include "codepair.hpp"
#include "common.hpp"
#include "gemm_core.hpp"
#include "loss_stat.hpp"
#include "train_ops.hpp"

namespace qp {

namespace losstile {

using gemm::CodeLayout;
using gemm::CodeStage;
using gemm::MfmaTraits;
using gemm::code_swz;
using gemm::lds_off;
using gemm::rsrc;
using gemm::swz;
using gemm::waitcnt_vm_lgkm0;

constexpr uint32_t OOB = 0x80000000u;

// e^x for the closes: 2^-24 (1 + |x|) of itself, half the instructions of expf.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// The maximum and the sum over eight lanes in a row, in all of them.
__device__ __forceinline__ float max8(float v)
{
    v = fmaxf(v, dpp_f32<0xB1>(v));
    v = fmaxf(v, dpp_f32<0x4E>(v));
    return fmaxf(v, dpp_f32<0x141>(v));
}
__device__ __forceinline__ float sum8(float v)
{
    v += dpp_f32<0xB1>(v);
    v += dpp_f32<0x4E>(v);
    return v + dpp_f32<0x141>(v);
}

// fp32 x goes in three parts of 16 bits, each a step of its own.
template <int DT> constexpr int OPERAND = DT == DT_F32 ? DT_BF16 : DT;
template <int DT> constexpr int PARTS = DT == DT_F32 ? 3 : 1;

// A step's scales: 256 columns of one group (of 32: two) in pieces of 256 bytes, a piece a
// wave and instruction.
template <int DT, int WMW, bool G32> struct ScaleStage {
    static constexpr int PER_GROUP = DT == DT_F32 ? 4 : 2;
    static constexpr int PIECES = PER_GROUP * (G32 ? 2 : 1), WAVES = 4 * WMW;
    static constexpr int INSTR = (PIECES + WAVES - 1) / WAVES, STAGE = INSTR * WAVES * 256;
};

// Stages of x and of the codes and scales. Three of x, and four of the codes up to 4 bits;
// tiles of 32 and 64 rows, whose steps are short beside a memory latency, as many of both
// as leave room for two blocks a CU (24 rows of 4096 x 32000, 4-bit, 125 tiles: 0.64 us a
// step with three and four, 0.52 with six; 64-row tiles of 100 rows and 131072 tokens 184
// us and, with four of each, 171; with eight and one block a CU 214).
template <int BITS, int DT, int FM, int WMW, bool G32> struct Depth {
    static constexpr int A = 32 * FM * WMW * 128;
    static constexpr int C = CodeStage<BITS, LOSS_BN, 4 * WMW>::STAGE + ScaleStage<DT, WMW, G32>::STAGE;
    static constexpr int MOST = 80 * 1024 / (A + C), EVEN = MOST < 3 ? 3 : MOST > 8 ? 8 : MOST;
    static constexpr int NA = FM <= 2 ? EVEN : 3;
    static constexpr int NC = FM <= 2 ? EVEN : BITS >= 6 ? 3 : 4;
    static constexpr int BYTES = NA * A + NC * C;
};

// LDS of the products, and then of the close.
template <int BITS, int DT, int FM, int WMW, bool G32> constexpr int lds_bytes()
{
    constexpr int steps = Depth<BITS, DT, FM, WMW, G32>::BYTES;
    constexpr int close = 4 * WMW * 32 * 68 * 4 + 4 * 32 * FM * WMW * (int)sizeof(Stat);
    return steps > close ? steps : close;
}

// DMA of 16, 12 or 4 bytes a lane, from a lane's offset and a uniform one.
__device__ __forceinline__ void dma16_at(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void dma12_at(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 12, voff, soff, 0, 0);
}
__device__ __forceinline__ void dma4_at(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t voff, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 4, voff, soff, 0, 0);
}

template <int BITS, int DT, int FM, int WMW, bool G32>
__global__ __launch_bounds__(256 * WMW, 2) void loss_tile_kernel(LossTileArgs a)
{
    constexpr int OT = OPERAND<DT>, P3 = PARTS<DT>;
    using T = MfmaTraits<OT>;
    using St = typename Elem<DT>::storage;
    using SS = ScaleStage<DT, WMW, G32>;
    using frag_t = typename T::frag_t;
    using CL = CodeLayout<BITS>;
    constexpr int WAVES = 4 * WMW, WGN = 4, FN = 2, WN = 64, WM = 32 * FM, BM = WM * WMW, BN = LOSS_BN, BK = 64;
    constexpr int A_STAGE = BM * 128, A_INSTR = A_STAGE / 1024 / WAVES;
    static_assert(A_INSTR * 1024 * WAVES == A_STAGE, "whole DMA blocks");
    constexpr int C_INSTR = CodeStage<BITS, BN, WAVES>::INSTR, C_STAGE = CodeStage<BITS, BN, WAVES>::STAGE;
    constexpr int SB_STAGE = SS::STAGE, S_INSTR = SS::INSTR, ES = (int)sizeof(St);
    constexpr int NA = Depth<BITS, DT, FM, WMW, G32>::NA, NCS = Depth<BITS, DT, FM, WMW, G32>::NC;
    // Step kt + 1 reads the activations and codes of kt + 2 at its end, so those have
    // landed when step kt ends; what was issued for later steps may be in flight.
    constexpr int IN_FLIGHT = (NA - 3) * (A_INSTR + C_INSTR + S_INSTR) + (NCS > NA ? C_INSTR + S_INSTR : 0);
    static_assert(NA >= 3 && (NCS == NA || NCS == NA + 1) && IN_FLIGHT < 64, "prefetch depth");
    extern __shared__ __attribute__((aligned(16))) char lds[];
    char* const a_st = lds;
    char* const c_st = a_st + NA * A_STAGE;
    char* const sb_st = c_st + NCS * C_STAGE;

    const int xcd = blockIdx.x % 8, local = blockIdx.x / 8;
    const int tile = xcd * a.per_xcd + local;
    if (local >= a.per_xcd || tile >= a.tiles)
        return;
    const int tm = tile % a.tiles_m, tn = tile / a.tiles_m;
    const int m0 = tm * BM, n0 = tn * BN;

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, c32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WGN, wn = wave % WGN;
    const uint32_t xrow = (uint32_t)a.xn * 2, wrow = (uint32_t)a.K * BITS / 8;
    const int KT = (a.K + BK - 1) / BK * P3, BT = DT == DT_F32 ? 0 : a.gp / 32;   // steps of the codes, of the biases
    const int groups = a.K / a.gs, rows_left = a.M - m0;

    // A tile's own rows as resources: their offsets are below 2^31 whatever M and N are.
    const __amdgpu_buffer_rsrc_t rx = rsrc(static_cast<const char*>(a.xp) + (size_t)m0 * xrow,
                                           (uint32_t)(rows_left < BM ? rows_left : BM) * xrow);
    const int cols_left = a.N - n0;
    const __amdgpu_buffer_rsrc_t rw = rsrc(reinterpret_cast<const char*>(a.wq) + (size_t)n0 * wrow,
                                           (uint32_t)(cols_left < BN ? cols_left : BN) * wrow);
    const __amdgpu_buffer_rsrc_t rs = rsrc(static_cast<const char*>(a.st) + (size_t)n0 * ES,
                                           (uint32_t)(groups - 1) * (uint32_t)a.np * ES + ES * BN);

    // Instruction i's rows are 8 i on, where the swizzle has one bit the other way round.
    // (Past the tile's rows: past the range.)
    const int a_r = 8 * wave * A_INSTR + (lane >> 3);
    uint32_t a_goff = (uint32_t)a_r * xrow + (uint32_t)(((lane & 7) ^ swz(a_r)) * 16);
    // Codes: where an instruction's 64 chunks are whole rows, instruction i's rows are so many
    // rows on, with the same swizzle.
    constexpr bool WHOLE = 64 % CL::CPR == 0;
    uint32_t c_goff[WHOLE ? 1 : C_INSTR];
#pragma unroll
    for (int i = 0; i < (WHOLE ? 1 : C_INSTR); ++i) {
        const int q = 64 * (wave * C_INSTR + i) + lane;
        const int r = q / CL::CPR, part = (q % CL::CPR) ^ code_swz<BITS>(r);
        c_goff[i] = WHOLE || q < BN * CL::CPR ? (uint32_t)r * wrow + part * CL::CS : OOB;   // (past the tile: past the range)
    }
    // Scales: piece q is part q % PER_GROUP of group q / PER_GROUP of the step's; waves
    // without one read past the range, into spare room.
    const int gs_steps = a.gs == 128 ? 1 : 0;   // log2 of the steps of a group (of 64 and more)

    // DMA operation o of step kt's: A_INSTR of the activations, C_INSTR of the codes, the
    // scales. A row's place in the step goes into the scalar offset, which is not range
    // checked: rows past the tile are past the range by their own, and what is asked for
    // past the last step is the last step again.
    const int last_a = BT + KT - 1;
    auto dma_a = [&](int kt, int stage, int i) {
        dma16_at(rx, a_st + stage * A_STAGE + (wave * A_INSTR + i) * 1024, (a_goff ^ (i % 2 ? 64u : 0u)) + (uint32_t)(8 * i) * xrow,
                 (kt < last_a ? kt : last_a) * BK * 2);
    };
    auto dma_c = [&](int kt, int stage, int i) {
        // The last step of 64 n + 32 features holds the row's last two units; the biases'
        // steps, before step 0, have none of their own.
        const int k = (kt > 0 ? kt / P3 : 0) * CL::RB, last = (int)wrow - CL::RB, off = k < last ? k : last;
        char* const dst = c_st + stage * C_STAGE + (wave * C_INSTR + i) * 1024;
        const uint32_t at = WHOLE ? c_goff[0] + (uint32_t)(i * (64 / CL::CPR)) * wrow : c_goff[WHOLE ? 0 : i];
        if constexpr (CL::CS == 12)
            dma12_at(rw, dst, at, off);
        else
            dma16_at(rw, dst, at, off);
    };
    auto dma_s = [&](int kt, int stage, int i) {
        const int q = wave + WAVES * i;
        kt = kt > 0 ? kt / P3 : 0;
        int g = G32 ? 2 * kt : kt >> gs_steps;
        const int most = groups - (G32 ? 2 : 1);
        g = (g < most ? g : most) + (G32 ? q / SS::PER_GROUP % 2 : 0);
        dma4_at(rs, sb_st + stage * SB_STAGE + q * 256,
                q < SS::PIECES ? (uint32_t)(q % SS::PER_GROUP) * 256 + (uint32_t)lane * 4 : OOB, g * a.np * ES);
    };
    auto step_barrier = [&](auto VM) {
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(decltype(VM)::value));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    // Steps of the pipeline: BT of the biases, then KT of the codes.
#pragma unroll
    for (int s = 1 - NCS; s < 0; ++s) {
        if (s + NA - 1 >= 0)
            for (int i = 0; i < A_INSTR; ++i)
                dma_a(s + NA - 1, s + NA - 1, i);
        for (int i = 0; i < C_INSTR; ++i)
            dma_c(s + NCS - 1 - BT, s + NCS - 1, i);
        for (int i = 0; i < S_INSTR; ++i)
            dma_s(s + NCS - 1 - BT, s + NCS - 1, i);
    }
    f32x16_t total[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            total[i][j] = f32x16_t{};

    // Fragment kk of the rows of tile i. Groups of 32 (and X): an instruction's two halves
    // are 16 positions of one half of the step.
    auto a_frag = [&](int stage, int i, int kk) {
        const int chunk = G32 ? 4 * (kk >> 1) + (kk & 1) + 2 * half : kk + 4 * half;
        return *reinterpret_cast<const frag_t*>(a_st + stage * A_STAGE + lds_off(wm * WM + 32 * i + c32, chunk));
    };
    int a_cur = 0, c_cur = 0;
    // The biases: 32 groups a step, instructions 0 and 1 the high and the low part of X
    // times b of the first 16 groups, 2 and 3 of the others. b's fragments come from memory,
    // a step ahead. With fp32 x, X and b are fp32 too, eight groups at a time on the fp32
    // instruction.
    if constexpr (DT == DT_F32) {
        const uint32_t grow = (uint32_t)a.gp * 4;
        const __amdgpu_buffer_rsrc_t rb = rsrc(static_cast<const char*>(a.bp) + (size_t)n0 * grow,
                                               (uint32_t)(cols_left < BN ? cols_left : BN) * grow);
        const __amdgpu_buffer_rsrc_t rg = rsrc(static_cast<const char*>(a.xs) + (size_t)m0 * grow,
                                               (uint32_t)(rows_left < BM ? rows_left : BM) * grow);
        for (uint32_t g = 0; g < grow; g += 32) {
            f32x4_t bf[FN], xf[FM];
#pragma unroll
            for (int j = 0; j < FN; ++j)
                bf[j] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                    rb, (uint32_t)(wn * WN + 32 * j + c32) * grow + g + 16 * half, 0, 0));
#pragma unroll
            for (int i = 0; i < FM; ++i)
                xf[i] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                    rg, (uint32_t)(wm * WM + 32 * i + c32) * grow + g + 16 * half, 0, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        total[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(xf[i][e], bf[j][e], total[i][j], 0, 0, 0);
        }
        step_barrier(std::integral_constant<int, 0>{});
    } else {
        const uint32_t grow = (uint32_t)a.gp * 2;
        const __amdgpu_buffer_rsrc_t rb = rsrc(static_cast<const char*>(a.bp) + (size_t)n0 * grow,
                                               (uint32_t)(cols_left < BN ? cols_left : BN) * grow);
        frag_t bf[FN][2];
        auto load_b = [&](int bt) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    bf[j][h] = __builtin_bit_cast(frag_t, __builtin_amdgcn_raw_buffer_load_b128(
                        rb, (uint32_t)(wn * WN + 32 * j + c32) * grow + (uint32_t)bt * 64 + 32 * h + 16 * half, 0, 0));
        };
        load_b(0);
        step_barrier(std::integral_constant<int, 0>{});
        for (int bt = 0; bt < BT; ++bt) {
            const int a_new = a_cur == 0 ? NA - 1 : a_cur - 1, c_new = c_cur == 0 ? NCS - 1 : c_cur - 1;
            frag_t b0[FN][2];
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    b0[j][h] = bf[j][h];
            if (bt + 1 < BT)
                load_b(bt + 1);
#pragma unroll
            for (int i = 0; i < A_INSTR; ++i)
                dma_a(bt + NA - 1, a_new, i);
#pragma unroll
            for (int i = 0; i < C_INSTR; ++i)
                dma_c(bt + NCS - 1 - BT, c_new, i);
#pragma unroll
            for (int i = 0; i < S_INSTR; ++i)
                dma_s(bt + NCS - 1 - BT, c_new, i);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int kk = 3; kk >= 0; --kk) {   // (the low parts first)
                    const frag_t x = a_frag(a_cur, i, kk);
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        total[i][j] = T::mfma(x, b0[j][kk >> 1], total[i][j]);
                }
            step_barrier(std::integral_constant<int, IN_FLIGHT>{});
            a_cur = a_cur + 1 == NA ? 0 : a_cur + 1;
            c_cur = c_cur + 1 == NCS ? 0 : c_cur + 1;
        }
        if constexpr (DT == DT_F16) {   // each row's X was brought into fp16's range
            const __amdgpu_buffer_rsrc_t rf = rsrc(static_cast<const float*>(a.xs) + m0,
                                                   (uint32_t)((rows_left < BM ? rows_left : BM) + 3) / 4 * 16);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                f32x4_t f[4];   // registers 4 q .. 4 q + 3 are four rows
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    f[q] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                        rf, (uint32_t)(wm * WM + 32 * i + 8 * q + 4 * half) * 4, 0, 0));
#pragma unroll
                for (int r = 0; r < 16; ++r)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        total[i][j][r] *= f[r >> 2][r & 3];
                __builtin_amdgcn_sched_barrier(0);   // (no room for all of them at once)
            }
        }
    }

    // B fragments of column block j for a step: the unit `half` of its row as 16 code
    // pairs, four a matrix instruction; with groups of 32 the halves of the wave swap so
    // that an instruction's two halves are of one unit. Loaded, and converted in four
    // parts.
    uint32_t bq[FN][16], raw[FN][BITS];
    float sc[FN][G32 ? 2 : 1];
    St raws[FN][G32 ? 2 : 1];
    auto load_codes = [&](auto J, int stage) {
        constexpr int j = decltype(J)::value;
        const int r = wn * WN + 32 * j + c32;
        const char* const row = c_st + stage * C_STAGE + r * CL::SLOT_ROW;
        const int sw = code_swz<BITS>(r);
        uint32_t(&w)[BITS] = raw[j];
        if constexpr (BITS == 4 || BITS == 3) {
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(row + ((half ^ sw) << 4));
#pragma unroll
            for (int i = 0; i < BITS; ++i) w[i] = v[i];
        } else if constexpr (BITS == 8) {
            const u32x4_t v0 = *reinterpret_cast<const u32x4_t*>(row + (((2 * half) ^ sw) << 4));
            const u32x4_t v1 = *reinterpret_cast<const u32x4_t*>(row + (((2 * half + 1) ^ sw) << 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) { w[i] = v0[i]; w[4 + i] = v1[i]; }
        } else {
#pragma unroll
            for (int i = 0; i < BITS / 2; ++i) {
                const u32x2_t v = *reinterpret_cast<const u32x2_t*>(row + half * 4 * BITS + 8 * i);
                w[2 * i] = v[0];
                w[2 * i + 1] = v[1];
            }
        }
        const char* const sb = sb_st + stage * SB_STAGE + ES * r;
#pragma unroll
        for (int u = 0; u < (G32 ? 2 : 1); ++u)
            raws[j][u] = *reinterpret_cast<const St*>(sb + BN * ES * u);
    };
    auto convert = [&](auto J, auto P) {
        constexpr int j = decltype(J)::value, p = decltype(P)::value;
        uint32_t q[16];
        code_pairs<BITS, OT>(raw[j], 0u, q);   // (of which the rest is dropped)
        if constexpr (G32) {
#pragma unroll
            for (int i = 2 * p; i < 2 * p + 2; ++i) {
                const auto x = __builtin_amdgcn_permlane32_swap(q[i], q[8 + i], false, false);
                bq[j][i] = x[0];
                bq[j][8 + i] = x[1];
            }
        } else {
#pragma unroll
            for (int i = 4 * p; i < 4 * p + 4; ++i)
                bq[j][i] = q[i];
        }
    };
    auto take_scales = [&](auto J) {
#pragma unroll
        for (int u = 0; u < (G32 ? 2 : 1); ++u)
            sc[J][u] = Elem<DT>::to_f32(raws[J][u]);
    };
    auto b_frag = [&](int j, int kk) {
        return __builtin_bit_cast(frag_t, u32x4_t{bq[j][4 * kk], bq[j][4 * kk + 1], bq[j][4 * kk + 2], bq[j][4 * kk + 3]});
    };
    // A step is 2 FM chains of L = 4 matrix instructions (groups of 32: 4 FM of 2), each
    // into one of two accumulators, and every instruction has its share of the other work
    // beside it: the chain before is scaled and added once its result is there; the last
    // chains of a row block take the next one's fragments into the registers that they
    // have read; column block 0's codes of the next step are converted under the last
    // chain, block 1's under the next step's first; the DMA is spread over the first.
    constexpr int U = G32 ? 2 : 1, L = 4 / U, CHAINS = FM * FN * U, DMAS = A_INSTR + C_INSTR + S_INSTR;
    frag_t af[4];
    f32x16_t acc[2];
    auto scale_part = [&](auto C, auto R0, auto R1) {   // registers R0 .. R1 - 1 of chain C's sums
        constexpr int c = decltype(C)::value, i = c / (FN * U), j = c / U % FN, u = c % U;
#pragma unroll
        for (int r = decltype(R0)::value; r < decltype(R1)::value; ++r)
            total[i][j][r] = __builtin_fmaf(sc[j][u], acc[c & 1][r], total[i][j][r]);
    };
    static_for<FN>([&](auto J) {
        load_codes(J, c_cur);
        take_scales(J);
    });
    static_for<4>([&](auto P) { convert(std::integral_constant<int, 0>{}, P); });
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        af[kk] = a_frag(a_cur, 0, kk);
    acc[(CHAINS - 1) & 1] = f32x16_t{};   // before the first step: nothing to add
    for (int kt = 0; kt < KT; ++kt) {
        const int a_new = a_cur == 0 ? NA - 1 : a_cur - 1;
        const int c_new = c_cur == 0 ? NCS - 1 : c_cur - 1;
        const int a_nxt = a_cur + 1 == NA ? 0 : a_cur + 1;
        const int c_nxt = c_cur + 1 == NCS ? 0 : c_cur + 1;
        // Opaque, so that each instruction's offset is formed at its place and not kept in a
        // register of its own through the steps: there are none to spare.
        asm volatile("" : "+v"(a_goff), "+v"(c_goff[0]));
        static_for<CHAINS * L>([&](auto Q) {
            constexpr int q = decltype(Q)::value, c = q / L, l = q % L, i = c / (FN * U), j = c / U % FN, u = c % U;
            constexpr int kk = L * u + l, prev = (c + CHAINS - 1) % CHAINS;
            if constexpr (l == 0)
                acc[c & 1] = T::mfma(af[kk], b_frag(j, kk), f32x16_t{});
            else
                acc[c & 1] = T::mfma(af[kk], b_frag(j, kk), acc[c & 1]);
            if constexpr (j == FN - 1)
                af[kk] = i + 1 < FM ? a_frag(a_cur, i + 1, kk) : a_frag(a_nxt, 0, kk);
            if constexpr (q < DMAS) {
                if constexpr (q < A_INSTR)
                    dma_a(BT + kt + NA - 1, a_new, q);
                else if constexpr (q < A_INSTR + C_INSTR)
                    dma_c(kt + NCS - 1, c_new, q - A_INSTR);
                else
                    dma_s(kt + NCS - 1, c_new, q - A_INSTR - C_INSTR);
            }
            constexpr int R0 = L == 4 ? (l == 0 ? 0 : l == 1 ? 0 : l == 2 ? 6 : 11) : (l == 0 ? 0 : 4);
            constexpr int R1 = L == 4 ? (l == 0 ? 0 : l == 1 ? 6 : l == 2 ? 11 : 16) : (l == 0 ? 4 : 16);
            scale_part(std::integral_constant<int, prev>{}, std::integral_constant<int, R0>{}, std::integral_constant<int, R1>{});
            // Four slots each for the two conversions.
            if constexpr (q < 4)
                convert(std::integral_constant<int, 1>{}, std::integral_constant<int, q>{});
            if constexpr (q == CHAINS * L - 6)
                load_codes(std::integral_constant<int, 0>{}, c_nxt);
            if constexpr (q >= CHAINS * L - 4)
                convert(std::integral_constant<int, 0>{}, std::integral_constant<int, q - (CHAINS * L - 4)>{});
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (q == CHAINS * L - 1)
                take_scales(std::integral_constant<int, 0>{});
            if constexpr (c == 0 && l == L - 1)
                take_scales(std::integral_constant<int, 1>{});
        });
        load_codes(std::integral_constant<int, 1>{}, c_nxt);
        step_barrier(std::integral_constant<int, IN_FLIGHT>{});
        a_cur = a_nxt;
        c_cur = c_nxt;
    }
    scale_part(std::integral_constant<int, CHAINS - 1>{}, std::integral_constant<int, 0>{}, std::integral_constant<int, 16>{});
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    __builtin_amdgcn_s_barrier();   // the LDS is free
    // The lane's number anew, and opaque, so that neither it nor the close's addresses are
    // kept in registers through the steps.
    int l = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm volatile("" : "+v"(l));
    const int half2 = l >> 5, c = l & 31;

    // Each wave turns its totals in LDS of its own, 32 rows at a time: register r of a 32 x
    // 32 tile is row 8 (r / 4) + 4 half + r % 4, column c; read back, eight lanes hold a
    // row's 64 columns, eight each.
    constexpr int S = WN + 4;   // floats of a row there
    float* const turned = reinterpret_cast<float*>(lds) + wave * 32 * S;
    Stat* const stats = reinterpret_cast<Stat*>(lds + WAVES * 32 * S * 4);   // [WGN][BM]
    const int part = l & 7, col0 = wn * WN + 8 * part;   // the lane's first column in the tile
    const uint32_t drow = (uint32_t)a.dz_stride * ES;
    const __amdgpu_buffer_rsrc_t rd = rsrc(static_cast<char*>(a.dz) + (a.dz != nullptr ? (size_t)m0 * drow + (size_t)n0 * ES : 0),
                                           a.dz != nullptr ? (uint32_t)(rows_left < BM ? rows_left : BM) * drow - (uint32_t)n0 * ES : 0u);
    const float by = a.dz != nullptr && a.scale != nullptr ? a.scale[0] : 1.0f;
    static_for<FM>([&](auto I) {
        constexpr int i = decltype(I)::value;
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(63));   // the last rows have been read
        asm volatile("" ::: "memory");
        static_for<16>([&](auto R) {
            constexpr int r = decltype(R)::value;
#pragma unroll
            for (int j = 0; j < FN; ++j)
                turned[(8 * (r >> 2) + 4 * half2 + (r & 3)) * S + 32 * j + c] = total[i][j][r];
        });
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(63));
        asm volatile("" ::: "memory");
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int tr = 8 * it + (l >> 3), row = wm * WM + 32 * i + tr;
            const float* const p = turned + tr * S + 8 * part;
            const f32x4_t z0 = *reinterpret_cast<const f32x4_t*>(p), z1 = *reinterpret_cast<const f32x4_t*>(p + 4);
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                z[e] = e < 4 ? z0[e & 3] : z1[e & 3];
            const bool in = row < rows_left;
            const int32_t t = in ? a.targets[m0 + row] : -1;
            const bool live = t >= 0 && t < a.vocab;
            const int64_t at = (int64_t)t - a.v0 - n0 - col0;   // of the lane's eight
            if (a.dz != nullptr) {
                // dz, and zeros up to the next multiple of 8 columns. (A row without a target,
                // or of g = 0, is zeros whatever its logits are.)
                const float lse = in ? a.lse[m0 + row] : 0.0f, g = live ? a.dloss[m0 + row] * by : 0.0f;
                uint32_t w[2 * ES];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = g * (exp_fast(z[e] - lse) - (at == e ? 1.0f : 0.0f));
                    const bool keep = g != 0.0f && col0 + e < cols_left;
                    if constexpr (DT == DT_F32) {
                        w[e] = keep ? __float_as_uint(d) : 0u;
                    } else {
                        const uint32_t v = keep ? Elem<DT>::from_f32(d) : 0u;
                        w[e / 2] = e % 2 ? w[e / 2] | (v << 16) : v;
                    }
                }
#pragma unroll
                for (int e = 0; e < ES / 2; ++e)
                    __builtin_amdgcn_raw_buffer_store_b128(
                        u32x4_t{w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]}, rd,
                        in && col0 < cols_left ? (uint32_t)row * drow + (uint32_t)col0 * ES + 16 * e : OOB, 0, 0);
                continue;
            }
            if (live && at >= 0 && at < 8)
                a.picked[m0 + row] = p[at];
            float top = -__builtin_inff();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[e] = col0 + e < cols_left ? z[e] : -__builtin_inff();
                top = fmaxf(top, z[e]);
            }
            top = max8(top);
            const float from = top == -__builtin_inff() ? 0.0f : top;   // no column: sums of 0
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum += exp_fast(z[e] - from);
            sum = sum8(sum);
            if (part == 0)
                stats[wn * BM + row] = Stat{top, sum};
        }
    });
    if (a.dz != nullptr)
        return;
    __syncthreads();
    for (int r = wave * 64 + l; r < BM && r < rows_left; r += 64 * WAVES) {
        Stat s = stats[r];
#pragma unroll
        for (int w = 1; w < WGN; ++w)
            s = join_stats(s, stats[w * BM + r]);
        a.stats[(size_t)(a.part0 + tn) * (size_t)a.stat_rows + m0 + r] = s;
    }
}

// Waves of a row where x is laid out, 64 units each at a time. fp16 rows, whose largest |X|
// all of them need, stay in a block.
__host__ __device__ constexpr int prep_waves(int dt, int chunks) { return dt != DT_F16 ? chunks : chunks > 2 ? 4 : chunks; }

// x [M, K] as the tile kernel's steps take it, rows of xn: first the groups' sums X, 64
// values for 32 groups: their value in DT and what that leaves, in eights as the fragments
// take them; then x in the order of the code pairs: position 2 p (+ 1) of a unit of 32
// holds its code lo_code(p) (hi_code(p)). A row of 64 n + 32 features ends in a unit of
// zeros and then its last. fp16: X times a power of two that brings the row's largest to
// 2^14 .. 2^15 (128 values may sum to more than the range, and the part that is left of a
// small X would be subnormal: with 1 / 128 for all rows a loss of 6.2 from x of 1e-4 was 5e-4
// off); its inverse goes to xf.
template <int BITS, int DT>
__device__ __forceinline__ void prep_x(int64_t block, const uint16_t* __restrict__ x, int64_t m, int k, int gs, int xn,
                                       int gp, uint16_t* __restrict__ xp, float* __restrict__ xf)
{
    using Order = CodeOrder<BITS>;
    using E = Elem<DT>;
    typedef u32x4_t Wide __attribute__((aligned(2)));
    const int first = 2 * gp, units = (xn - first) / 32, chunks = (units + 63) / 64, lane = (int)threadIdx.x & 63;
    const int waves = prep_waves(DT, chunks), n = k / 32, per = gs / 32;
    const int64_t w = block * 4 + (threadIdx.x >> 6), row = w / waves;
    const int chunk0 = (int)(w % waves);
    uint16_t* const to = xp + row * xn;
    // Lane's unit of a chunk, and its group's sum.
    uint32_t e[16];
    int u = 0, src = -1;
    float sum = 0.0f;
    auto load = [&](int chunk) {
        u = chunk * 64 + lane;
        src = row >= m ? -1 : u < n - (n & 1) ? u : u == units - 1 ? n - 1 : -1;   // (n odd: the last step)
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            e[i] = 0u;
        if (src >= 0) {
            const uint16_t* const p = x + row * k + src * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4_t v = *reinterpret_cast<const Wide*>(p + 8 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    e[4 * i + j] = v[j];
                    sum += E::to_f32((uint16_t)v[j]) + E::to_f32((uint16_t)(v[j] >> 16));
                }
            }
        }
        for (int off = 1; off < per; off <<= 1)
            sum += __shfl_xor(sum, off, 64);
    };
    float by = 1.0f;
    if constexpr (DT == DT_F16) {
        __shared__ float room[4];
        float top = 0.0f;
        for (int chunk = chunk0; chunk < chunks; chunk += waves) {
            load(chunk);
            const float size = fabsf(sum);
            top = fmaxf(top, size < __builtin_inff() ? size : 0.0f);
        }
        top = wave_stat(Stat{top, 0.0f}).top;
        if (lane == 0)
            room[threadIdx.x >> 6] = top;
        __syncthreads();
        const int wave0 = (int)(threadIdx.x >> 6) - chunk0;   // the row's first
        for (int i = 0; i < waves; ++i)
            top = fmaxf(top, room[wave0 + i]);
        const int exponent = top > 0.0f ? (int)(__float_as_uint(top) >> 23) - 127 - 14 : 0;   // (top is normal)
        by = __uint_as_float((uint32_t)(127 - exponent) << 23);
        if (chunk0 == 0 && lane == 0 && row < m)
            xf[row] = __uint_as_float((uint32_t)(127 + exponent) << 23);
    }
    if (row >= m)
        return;
    // Group g of a step of 32: its 16 (g / 16 % 2) are instructions 2 i and 2 i + 1, their
    // halves of the wave eight each (a_frag's chunks, which differ with groups of 32).
    auto put = [&](int g, uint16_t hi, uint16_t lo) {
        const int i = g / 16 % 2, h = g / 8 % 2;
        uint16_t* const t = to + g / 32 * 64 + g % 8;
        const int c0 = gs == 32 ? 4 * i + 2 * h : 2 * i + 4 * h;   // the chunk of instruction 2 i
        t[8 * c0] = hi;
        t[8 * (c0 + 1)] = lo;
    };
    for (int chunk = chunk0; chunk < chunks; chunk += waves) {
        if (DT != DT_F16 || chunks > waves)   // (or it is there)
            load(chunk);
        if (u < units) {
            auto elem = [&](int i) { return (e[i / 2] >> (16 * (i % 2))) & 0xFFFFu; };
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u32x4_t v;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = elem(Order::lo_code(4 * i + j)) | (elem(Order::hi_code(4 * i + j)) << 16);
                *reinterpret_cast<u32x4_t*>(to + first + 32 * u + 8 * i) = v;
            }
        }
        if (src >= 0 && src % per == 0) {
            const float part = sum * by;
            const uint16_t hi = E::from_f32(part);
            put(src / per, hi, E::from_f32(part - E::to_f32(hi)));
        }
    }
    if (chunk0 == 0 && k / gs + lane < gp)   // fewer than 32 to fill up
        put(k / gs + lane, 0, 0);
}

// fp32 x: each 64 features are three steps, x in parts of 16 bits (what the parts before
// leave, which is exact: 24 bits in all); X in fp32, rows of gp.
template <int BITS>
__device__ __forceinline__ void prep_x32(int64_t block, const float* __restrict__ x, int64_t m, int k, int gs, int xn,
                                         int gp, uint16_t* __restrict__ xp, float* __restrict__ xs)
{
    using Order = CodeOrder<BITS>;
    using E = Elem<DT_BF16>;
    typedef f32x4_t Wide __attribute__((aligned(4)));
    const int units = xn / 96, chunks = (units + 63) / 64, lane = (int)threadIdx.x & 63;
    const int64_t w = block * 4 + (threadIdx.x >> 6), row = w / chunks;
    if (row >= m)
        return;
    const int chunk = (int)(w % chunks), u = chunk * 64 + lane, n = k / 32;
    const int src = u < n - (n & 1) ? u : u == units - 1 ? n - 1 : -1;   // (n odd: the last step)
    float e[32];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        e[i] = 0.0f;
    if (src >= 0) {
        const float* const p = x + row * k + src * 32;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const f32x4_t v = *reinterpret_cast<const Wide*>(p + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                e[4 * i + j] = v[j];
                sum += v[j];
            }
        }
    }
    if (u < units) {
        uint16_t* const to = xp + row * xn + u / 2 * 192 + u % 2 * 32;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            uint32_t h[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                h[i] = E::from_f32(e[i]);
                e[i] -= E::to_f32((uint16_t)h[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u32x4_t v;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = h[Order::lo_code(4 * i + j)] | (h[Order::hi_code(4 * i + j)] << 16);
                *reinterpret_cast<u32x4_t*>(to + 64 * part + 8 * i) = v;
            }
        }
    }
    const int per = gs / 32;
    for (int off = 1; off < per; off <<= 1)
        sum += __shfl_xor(sum, off, 64);
    if (src >= 0 && src % per == 0)
        xs[row * gp + src / per] = sum;
    if (chunk == 0 && k / gs + lane < gp)   // fewer than 8 to fill up
        xs[row * gp + k / gs + lane] = 0.0f;
}

// The scales [n, groups] transposed to [groups, np], zeros behind n, and the biases in
// rows of gp (null: they lie so already). Tiles of 64 x 64.
template <class E>
__device__ __forceinline__ void prep_w(int64_t block, const E* __restrict__ scales, const E* __restrict__ biases, int64_t n,
                                       int groups, int64_t np, int gp, E* __restrict__ st, E* __restrict__ bp)
{
    __shared__ E room[64][64 + 4 / sizeof(E)];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int tiles_g = (gp + 63) / 64;
    const int g0 = (int)(block % tiles_g) * 64;
    const int64_t v0 = block / tiles_g * 64;
    const int g = g0 + lane;
    // (All the loads first, with their indexes held inside and no branch around them.)
    E s[16], b[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t v = v0 + 4 * i + wave, at = (v < n ? v : n - 1) * groups + (g < groups ? g : groups - 1);
        s[i] = scales[at];
        b[i] = biases[at];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t v = v0 + 4 * i + wave;
        room[4 * i + wave][lane] = v < n && g < groups ? s[i] : (E)0;
        if (bp != nullptr && v < n && g < gp)
            bp[v * gp + g] = g < groups ? b[i] : (E)0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (g0 + 4 * i + wave < groups)
            st[(int64_t)(g0 + 4 * i + wave) * np + v0 + lane] = room[lane][4 * i + wave];
}

// What the tiles read, in one launch: blocks of the weight's, then of x's (with the first
// piece), then one for the factor of dz (where it has one). Three launches of a small call
// take 18 us (77 rows, 1024 x 50001), one 6.
template <int BITS, int DT>
__global__ __launch_bounds__(256) void loss_prep_kernel(LossTileArgs a, LossPrepArgs p, int64_t w_blocks, int64_t x_blocks)
{
    using E = typename Elem<DT>::storage;
    const int64_t block = blockIdx.x;
    uint16_t* const xp = static_cast<uint16_t*>(const_cast<void*>(a.xp));
    if (block < w_blocks)
        prep_w(block, static_cast<const E*>(p.scales), static_cast<const E*>(p.biases), (int64_t)a.N, a.K / a.gs,
               (int64_t)a.np, a.gp, static_cast<E*>(const_cast<void*>(a.st)), static_cast<E*>(p.bp));
    else if (block >= w_blocks + x_blocks)
        dz_factor(a.dloss, a.M, a.targets, a.vocab, p.factor);
    else if constexpr (DT == DT_F32)
        prep_x32<BITS>(block - w_blocks, static_cast<const float*>(p.x), a.M, a.K, a.gs, a.xn, a.gp, xp,
                       static_cast<float*>(const_cast<void*>(a.xs)));
    else
        prep_x<BITS, DT>(block - w_blocks, static_cast<const uint16_t*>(p.x), a.M, a.K, a.gs, a.xn, a.gp, xp,
                         static_cast<float*>(const_cast<void*>(a.xs)));
}

} // namespace losstile
} // namespace qp
