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
// (bf16; fp16 2^-22), G / 32 steps of 64 more.
//
// loss_prep_x writes x once in the order that a unit's code pairs come in, rows filled
// up to whole 64-wide steps, and X; loss_prep_w the scales transposed (a step's scales
// of a tile are then 512 bytes in a row) and the biases in rows of whole 16-byte
// pieces. Both are a few microseconds beside the tiles.
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
constexpr int NA = 3;
template <int BITS> constexpr int NC = BITS >= 6 ? 3 : 4;

// e^x for the closes: 2^-24 (1 + |x|) of itself, half the instructions of expf.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// The maximum and the sum over each half of a wave, in all its lanes.
__device__ __forceinline__ float max32(float v)
{
    v = fmaxf(v, dpp_f32<0xB1>(v));
    v = fmaxf(v, dpp_f32<0x4E>(v));
    v = fmaxf(v, dpp_f32<0x141>(v));
    v = fmaxf(v, dpp_f32<0x140>(v));
    const auto x = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)x[0]), __builtin_bit_cast(float, (uint32_t)x[1]));
}
__device__ __forceinline__ float sum32(float v)
{
    v += dpp_f32<0xB1>(v);
    v += dpp_f32<0x4E>(v);
    v += dpp_f32<0x141>(v);
    v += dpp_f32<0x140>(v);
    const auto x = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return __builtin_bit_cast(float, (uint32_t)x[0]) + __builtin_bit_cast(float, (uint32_t)x[1]);
}

template <int BITS, int FM, int WMW> constexpr int lds_bytes()
{
    return NA * 32 * FM * WMW * 128 + NC<BITS> * (CodeStage<BITS, LOSS_BN, 4 * WMW>::STAGE + 4 * WMW * 256);
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
    using T = MfmaTraits<DT>;
    using frag_t = typename T::frag_t;
    using CL = CodeLayout<BITS>;
    constexpr int WAVES = 4 * WMW, WGN = 4, FN = 2, WN = 64, WM = 32 * FM, BM = WM * WMW, BN = LOSS_BN, BK = 64;
    constexpr int A_STAGE = BM * 128, A_INSTR = A_STAGE / 1024 / WAVES;
    static_assert(A_INSTR * 1024 * WAVES == A_STAGE, "whole DMA blocks");
    constexpr int C_INSTR = CodeStage<BITS, BN, WAVES>::INSTR, C_STAGE = CodeStage<BITS, BN, WAVES>::STAGE;
    constexpr int SB_STAGE = WAVES * 256;
    constexpr int NCS = NC<BITS>;
    // As in gemm_core.hpp: step kt + 1 reads the activations and codes of kt + 2 at
    // its end; what was issued after them may be in flight when step kt ends.
    constexpr int IN_FLIGHT = NCS > NA ? C_INSTR + 1 : 0;
    static_assert(NA == 3 && (NCS == 3 || NCS == 4), "prefetch depth");
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
    const uint32_t xrow = (uint32_t)a.kp * 2, wrow = (uint32_t)a.K * BITS / 8;
    const int KT = a.kp / BK, groups = a.K / a.gs, rows_left = a.M - m0;

    // A tile's own rows as resources: their offsets are below 2^31 whatever M and N are.
    const __amdgpu_buffer_rsrc_t rx = rsrc(static_cast<const char*>(a.xp) + (size_t)m0 * xrow,
                                           (uint32_t)(rows_left < BM ? rows_left : BM) * xrow);
    const int cols_left = a.N - n0;
    const __amdgpu_buffer_rsrc_t rw = rsrc(reinterpret_cast<const char*>(a.wq) + (size_t)n0 * wrow,
                                           (uint32_t)(cols_left < BN ? cols_left : BN) * wrow);
    const __amdgpu_buffer_rsrc_t rs = rsrc(static_cast<const char*>(a.st) + (size_t)n0 * 2,
                                           (uint32_t)(groups - 1) * (uint32_t)a.np * 2 + 2 * BN);

    uint32_t a_goff[A_INSTR];
#pragma unroll
    for (int i = 0; i < A_INSTR; ++i) {
        const int r = 8 * (wave * A_INSTR + i) + (lane >> 3);
        a_goff[i] = r < rows_left ? (uint32_t)r * xrow + (uint32_t)(((lane & 7) ^ swz(r)) * 16) : OOB;
    }
    uint32_t c_goff[C_INSTR];
#pragma unroll
    for (int i = 0; i < C_INSTR; ++i) {
        const int q = 64 * (wave * C_INSTR + i) + lane;
        const int r = q / CL::CPR, part = (q % CL::CPR) ^ code_swz<BITS>(r);
        c_goff[i] = q < BN * CL::CPR && r < cols_left ? (uint32_t)r * wrow + part * CL::CS : OOB;
    }
    // Scales: wave w takes 128 columns of a group, w % 2 of the tile's two halves; groups
    // of 32 have two a step (waves 2, 3). The others' go to spare room.
    constexpr int SB_WAVES = G32 ? 4 : 2;
    const uint32_t s_goff = wave < SB_WAVES ? (uint32_t)(wave & 1) * 256 + (uint32_t)lane * 4 : OOB;
    const int gs_steps = a.gs == 128 ? 1 : 0;   // log2 of the steps of a group (of 64 and more)

    // DMA operation o of step kt's: A_INSTR of the activations, C_INSTR of the codes, the
    // scales. A row's place in the step goes into the scalar offset, which is not range
    // checked: rows past the tile are past the range by their own, and the activations'
    // last steps read on into the workspace behind them.
    auto dma_a = [&](int kt, int stage, int i) {
        dma16_at(rx, a_st + stage * A_STAGE + (wave * A_INSTR + i) * 1024, a_goff[i], kt * BK * 2);
    };
    auto dma_c = [&](int kt, int stage, int i) {
        // The last step of 64 n + 32 features holds the row's last two units.
        const int k = kt * CL::RB, last = (int)wrow - CL::RB, off = k < last ? k : last;
        char* const dst = c_st + stage * C_STAGE + (wave * C_INSTR + i) * 1024;
        if constexpr (CL::CS == 12)
            dma12_at(rw, dst, c_goff[i], off);
        else
            dma16_at(rw, dst, c_goff[i], off);
    };
    auto dma_s = [&](int kt, int stage) {
        int g = G32 ? 2 * kt : kt >> gs_steps;
        const int most = groups - (G32 ? 2 : 1);
        g = (g < most ? g : most) + (G32 ? wave >> 1 : 0);
        dma4_at(rs, sb_st + stage * SB_STAGE + wave * 256, s_goff, g * a.np * 2);
    };
    auto step_barrier = [&](auto VM) {
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(decltype(VM)::value));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

#pragma unroll
    for (int s = 1 - NCS; s < 0; ++s) {
        if (s + NA - 1 >= 0)
            for (int i = 0; i < A_INSTR; ++i)
                dma_a(s + NA - 1, s + NA - 1, i);
        for (int i = 0; i < C_INSTR; ++i)
            dma_c(s + NCS - 1, s + NCS - 1, i);
        dma_s(s + NCS - 1, s + NCS - 1);
    }

    // The biases: X (hi, lo) times b, 16 groups an instruction; they start the totals.
    f32x16_t total[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            total[i][j] = f32x16_t{};
    {
        const uint32_t grow = (uint32_t)a.gp * 2;
        const __amdgpu_buffer_rsrc_t rh = rsrc(static_cast<const char*>(a.xs) + (size_t)m0 * 2 * grow,
                                               (uint32_t)(rows_left < BM ? rows_left : BM) * 2 * grow);
        const __amdgpu_buffer_rsrc_t rb = rsrc(static_cast<const char*>(a.bp) + (size_t)n0 * grow,
                                               (uint32_t)(cols_left < BN ? cols_left : BN) * grow);
        for (uint32_t c = 0; c < grow; c += 32) {
            frag_t bf[FN], xh[FM], xl[FM];
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int col = wn * WN + 32 * j + c32;
                bf[j] = __builtin_bit_cast(frag_t, __builtin_amdgcn_raw_buffer_load_b128(
                    rb, col < cols_left ? (uint32_t)col * grow + c + 16 * half : OOB, 0, 0));
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int row = wm * WM + 32 * i + c32;
                const uint32_t at = row < rows_left ? (uint32_t)row * 2 * grow + c + 16 * half : OOB;
                xh[i] = __builtin_bit_cast(frag_t, __builtin_amdgcn_raw_buffer_load_b128(rh, at, 0, 0));
                xl[i] = __builtin_bit_cast(frag_t, __builtin_amdgcn_raw_buffer_load_b128(rh, at == OOB ? OOB : at + grow, 0, 0));
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    total[i][j] = T::mfma(xl[i], bf[j], total[i][j]);
                    total[i][j] = T::mfma(xh[i], bf[j], total[i][j]);
                }
        }
        if constexpr (DT == DT_F16) {   // X was divided by 128, which keeps it inside fp16's range
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    total[i][j] *= 128.0f;
        }
    }
    step_barrier(std::integral_constant<int, IN_FLIGHT>{});

    // B fragments of column block j for a step: the unit `half` of its row as 16 code
    // pairs, four a matrix instruction; with groups of 32 the halves of the wave swap so
    // that an instruction's two halves are of one unit. Loaded, and converted in four
    // parts (groups of 32: two).
    uint32_t bq[FN][16], raw[FN][BITS];
    float sc[FN][G32 ? 2 : 1];
    uint16_t raws[FN][G32 ? 2 : 1];
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
        const char* const sb = sb_st + stage * SB_STAGE + 2 * r;
#pragma unroll
        for (int u = 0; u < (G32 ? 2 : 1); ++u)
            raws[j][u] = *reinterpret_cast<const uint16_t*>(sb + 512 * u);
    };
    auto convert = [&](auto J, auto P) {
        constexpr int j = decltype(J)::value, p = decltype(P)::value;
        uint32_t q[16];
        code_pairs<BITS, DT>(raw[j], 0u, q);   // (of which the rest is dropped)
        if constexpr (G32) {
            if constexpr (p < 2) {
#pragma unroll
                for (int i = 4 * p; i < 4 * p + 4; ++i) {
                    const auto x = __builtin_amdgcn_permlane32_swap(q[i], q[8 + i], false, false);
                    bq[j][i] = x[0];
                    bq[j][8 + i] = x[1];
                }
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
    // Fragment kk of the rows of tile i.
    auto a_frag = [&](int stage, int i, int kk) {
        const int chunk = G32 ? 4 * (kk >> 1) + (kk & 1) + 2 * half : kk + 4 * half;
        return *reinterpret_cast<const frag_t*>(a_st + stage * A_STAGE + lds_off(wm * WM + 32 * i + c32, chunk));
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
    constexpr int U = G32 ? 2 : 1, L = 4 / U, CHAINS = FM * FN * U, DMAS = A_INSTR + C_INSTR + 1;
    frag_t af[4];
    f32x16_t acc[2];
    auto scale_part = [&](auto C, auto R0, auto R1) {   // registers R0 .. R1 - 1 of chain C's sums
        constexpr int c = decltype(C)::value, i = c / (FN * U), j = c / U % FN, u = c % U;
#pragma unroll
        for (int r = decltype(R0)::value; r < decltype(R1)::value; ++r)
            total[i][j][r] = __builtin_fmaf(sc[j][u], acc[c & 1][r], total[i][j][r]);
    };
    static_for<FN>([&](auto J) {
        load_codes(J, 0);
        take_scales(J);
    });
    static_for<4>([&](auto P) { convert(std::integral_constant<int, 0>{}, P); });
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        af[kk] = a_frag(0, 0, kk);
    acc[(CHAINS - 1) & 1] = f32x16_t{};   // before the first step: nothing to add
    int a_cur = 0, c_cur = 0;
    for (int kt = 0; kt < KT; ++kt) {
        const int a_new = a_cur == 0 ? NA - 1 : a_cur - 1;
        const int c_new = c_cur == 0 ? NCS - 1 : c_cur - 1;
        const int a_nxt = a_cur + 1 == NA ? 0 : a_cur + 1;
        const int c_nxt = c_cur + 1 == NCS ? 0 : c_cur + 1;
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
                    dma_a(kt + NA - 1, a_new, q);
                else if constexpr (q < A_INSTR + C_INSTR)
                    dma_c(kt + NCS - 1, c_new, q - A_INSTR);
                else
                    dma_s(kt + NCS - 1, c_new);
            }
            constexpr int R0 = L == 4 ? (l == 0 ? 0 : l == 1 ? 0 : l == 2 ? 6 : 11) : (l == 0 ? 0 : 4);
            constexpr int R1 = L == 4 ? (l == 0 ? 0 : l == 1 ? 6 : l == 2 ? 11 : 16) : (l == 0 ? 4 : 16);
            scale_part(std::integral_constant<int, prev>{}, std::integral_constant<int, R0>{}, std::integral_constant<int, R1>{});
            // Four slots each for the two conversions.
            if constexpr (q < 4)
                convert(std::integral_constant<int, 1>{}, std::integral_constant<int, q>{});
            if constexpr (q == CHAINS * L - 6)
                load_codes(std::integral_constant<int, 0>{}, c_nxt);
            if constexpr (q >= CHAINS * L - (G32 ? 2 : 4))
                convert(std::integral_constant<int, 0>{}, std::integral_constant<int, q - (CHAINS * L - (G32 ? 2 : 4))>{});
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
    // Opaque here, so that the close's addresses are formed now and not kept in
    // registers through the steps.
    int l = lane;
    asm volatile("" : "+v"(l));
    const int half2 = l >> 5, c = l & 31;

    // Register r of a 32 x 32 tile: row 8 (r / 4) + 4 half + r % 4, column c.
    struct Row {
        float lse, g;
        int32_t target;   // its column in the tile, or -1
    };
    Row* const rows = reinterpret_cast<Row*>(lds);
    for (int r = wave * 64 + l; r < BM; r += 64 * WAVES) {
        const bool in = r < rows_left;
        const int64_t t = in ? (int64_t)a.targets[m0 + r] : -1;
        const bool live = t >= 0 && t < a.vocab;
        const int64_t at = t - a.v0 - n0;
        Row p;
        p.target = live && at >= 0 && at < BN ? (int32_t)at : -1;
        p.lse = a.dz != nullptr && in ? a.lse[m0 + r] : 0.0f;
        p.g = a.dz != nullptr && live ? a.dloss[m0 + r] * a.scale[0] : 0.0f;
        rows[r] = p;
    }
    __syncthreads();
    const int col0 = wn * WN + c, row0 = wm * WM + 4 * half2;
    if (a.dz != nullptr) {
        // dz, and zeros up to the next multiple of 8 columns. (A row without a target, or
        // of g = 0, is zeros whatever its logits are.)
        const uint32_t drow = (uint32_t)a.dz_stride * 2;
        const __amdgpu_buffer_rsrc_t rd = rsrc(static_cast<char*>(a.dz) + (size_t)m0 * drow + (size_t)n0 * 2,
                                               (uint32_t)(rows_left < BM ? rows_left : BM) * drow - (uint32_t)n0 * 2);
        const int cols8 = (cols_left + 7) & ~7;
        static_for<FM>([&](auto I) {
            static_for<16>([&](auto R) {
                constexpr int i = decltype(I)::value, r = decltype(R)::value;
                const int row = row0 + 32 * i + 8 * (r >> 2) + (r & 3);
                const Row p = rows[row];
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const int col = col0 + 32 * j;
                    const float v = p.g * (exp_fast(total[i][j][r] - p.lse) - (p.target == col ? 1.0f : 0.0f));
                    const uint32_t keep = p.g != 0.0f && col < cols_left ? 0xFFFFu : 0u;
                    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(Elem<DT>::from_f32(v) & keep), rd,
                                                          col < cols8 && row < rows_left ? (uint32_t)row * drow + (uint32_t)col * 2 : OOB, 0, 0);
                }
            });
        });
        return;
    }
    // Statistics: of the lane's two columns, the half wave's 64, then the block's 256.
    Stat* const stats = reinterpret_cast<Stat*>(lds + BM * sizeof(Row));   // [WGN][BM]
    const float bar[FN] = {col0 < cols_left ? 0.0f : -__builtin_inff(), col0 + 32 < cols_left ? 0.0f : -__builtin_inff()};
    static_for<FM>([&](auto I) {
        static_for<16>([&](auto R) {
            constexpr int i = decltype(I)::value, r = decltype(R)::value;
            const int row = row0 + 32 * i + 8 * (r >> 2) + (r & 3);
            const float z0 = total[i][0][r] + bar[0], z1 = total[i][1][r] + bar[1];
            const int32_t t = rows[row].target - col0;
            if ((t & ~32) == 0)
                a.picked[m0 + row] = t == 0 ? z0 : z1;
            const float top = max32(fmaxf(z0, z1));
            const float at = top == -__builtin_inff() ? 0.0f : top;   // no column: sums of 0
            const float sum = sum32(exp_fast(z0 - at) + exp_fast(z1 - at));
            if (c == 0)
                stats[wn * BM + row] = Stat{top, sum};
        });
    });
    __syncthreads();
    for (int r = wave * 64 + l; r < BM && r < rows_left; r += 64 * WAVES) {
        Stat s = stats[r];
#pragma unroll
        for (int w = 1; w < WGN; ++w)
            s = join_stats(s, stats[w * BM + r]);
        a.stats[(size_t)(a.part0 + tn) * (size_t)a.stat_rows + m0 + r] = s;
    }
}

// x [M, K] in the order of the code pairs: position 2 p (+ 1) of a unit of 32 holds its
// code lo_code(p) (hi_code(p)). A row of 64 n + 32 features ends in a unit of zeros and
// then its last, as the tile kernel's last step takes them. And the groups' sums X (fp16:
// divided by 128), as their value in DT and what that leaves. A wave takes 64 units of
// a row.
template <int BITS, int DT>
__global__ __launch_bounds__(256) void loss_prep_x_kernel(const uint16_t* __restrict__ x, int64_t m, int k, int gs,
                                                          int kp, int gp, u32x4_t* __restrict__ xp,
                                                          uint16_t* __restrict__ xs)
{
    using Order = CodeOrder<BITS>;
    using E = Elem<DT>;
    typedef u32x4_t Wide __attribute__((aligned(2)));
    const int units = kp / 32, chunks = (units + 63) / 64, lane = (int)threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), row = w / chunks;
    if (row >= m)
        return;
    const int chunk = (int)(w % chunks), u = chunk * 64 + lane, n = k / 32;
    const int src = u < n - (n & 1) ? u : u == units - 1 ? n - 1 : -1;   // (n odd: the last step)
    uint32_t e[16];
    float sum = 0.0f;
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
    if (u < units) {
        auto elem = [&](int i) { return (e[i / 2] >> (16 * (i % 2))) & 0xFFFFu; };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u32x4_t v;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = elem(Order::lo_code(4 * i + j)) | (elem(Order::hi_code(4 * i + j)) << 16);
            xp[(row * units + u) * 4 + i] = v;
        }
    }
    const int per = gs / 32;
    for (int off = 1; off < per; off <<= 1)
        sum += __shfl_xor(sum, off, 64);
    const int g = src >= 0 && src % per == 0 ? src / per : -1;
    uint16_t* const hi = xs + row * 2 * gp;
    if (g >= 0) {
        if constexpr (DT == DT_F16)
            sum *= 1.0f / 128;
        hi[g] = E::from_f32(sum);
        hi[gp + g] = E::from_f32(sum - E::to_f32(hi[g]));
    }
    if (chunk == 0 && k / gs + lane < gp)   // fewer than 16 to fill up
        hi[k / gs + lane] = hi[gp + k / gs + lane] = 0;
}

} // namespace losstile
} // namespace qp
