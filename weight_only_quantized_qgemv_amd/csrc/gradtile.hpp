// gradtile.hpp — the matrix-core tile kernels of the gradient products, for
// 16-bit activations.
//
// Both products contract over an axis along which an operand is not
// contiguous: dx = dy W runs over the rows of the packed weight, dW = dy^T x
// over the rows of both activations. The 32x32x16 matrix instruction wants 8
// consecutive contraction elements per lane, so those operands are turned on
// their way to LDS: a thread loads a block of 4 contraction rows x 8 columns
// (8 codes, or 16 bytes of activations, a row), and writes each column's 4
// values as 8 bytes into the row that this column has in the LDS tile
// [column][64 contraction], where both operands then look alike. For the
// packed weight this is also where it is dequantized, once per block (q s' + b'
// in fp32, rounded to the activation type, as in the forward tile kernel of
// gemm_core.hpp).
//  - LDS rows are 128 bytes; the 16-byte chunk c of row r sits at
//    c ^ turn_swz(r), which spreads both the 16 consecutive rows of a fragment
//    read and the rows 8 o + j (o = 0..7, j fixed) of a turned write over all
//    banks; the two halves of a chunk are written by neighbouring lanes.
//  - steps of 64 contraction elements; two LDS stages of every turned operand,
//    whose raw loads run two steps ahead in registers; the activation operand
//    of dx, contiguous as it is, comes by DMA three stages deep.
#pragma once

#include "codes8.hpp"
#include "common.hpp"
#include "gemm_core.hpp"
#include "wgrad.hpp"
#include "xgrad.hpp"

namespace qp {
namespace gradtile {

using gemm::dma16;
using gemm::MfmaTraits;
using gemm::rsrc;
using gemm::waitcnt_vm_lgkm0;

constexpr int STEP = 64;
constexpr uint32_t OOB = 0x80000000u;

// Fragment reads take 16 lanes a cycle in groups of four consecutive rows (0-3,
// 12-15, 20-23, 24-27 and the rest): with (r >> 1) & 7 alone those hit 8
// chunks of both row parities, and the two bits of r >> 4, one value in each
// half of a 32-row tile, keep that while spreading rows 8 apart.
__device__ __forceinline__ int turn_swz(int r) { return ((r >> 1) & 7) ^ ((r >> 4) & 3); }

// Which 4 x 8 block a thread turns: octet o of the tile's columns, contraction
// rows 4 rq .. 4 rq + 3. Eight lanes walk octets, the next lane bit the two
// halves of a chunk (rq's low bit), so that 16 lanes fill 8 chunks.
template <int COLS> struct TurnMap {
    static constexpr int OCT = COLS / 8, HI = OCT / 8;
    int o, rq;
    uint32_t at[4];   // LDS byte offsets of columns 2 jj, jj = 0..3 (the next column is one row on)
    __device__ __forceinline__ TurnMap(int tid)
    {
        o = (tid & 7) | (((tid >> 4) & (HI - 1)) << 3);
        rq = ((tid >> 3) & 1) | ((tid >> (4 + __builtin_ctz(HI))) << 1);
        const int x = (rq >> 1) ^ (4 * (o & 1)) ^ ((o >> 1) & 3);   // chunk ^ turn_swz(8 o)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
            at[jj] = (uint32_t)((8 * o + 2 * jj) * 128 + ((x ^ jj) << 4) + 8 * (rq & 1));
    }
    // Column j's pairs (contraction rows 0, 1) and (2, 3).
    __device__ __forceinline__ void put(char* stage, int j, uint32_t p01, uint32_t p23) const
    {
        *reinterpret_cast<u32x2_t*>(stage + at[j >> 1] + 128 * (j & 1)) = u32x2_t{p01, p23};
    }
};

// Byte offsets of the fragments of LDS rows base + 32 J + lane % 32: chunk
// 2 kk + lane / 32 of tile J is at frag[kk ^ (J & 1)] + 4096 J, for base a
// multiple of 32 (32 rows on, the swizzle's bit 1 flips).
__device__ __forceinline__ void frag_offsets(int lane, int base, uint32_t (&f)[4])
{
    const int c = lane & 31, half = lane >> 5;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        f[kk] = (uint32_t)((base + c) * 128 + (((2 * kk + half) ^ turn_swz(base + c)) << 4));
}

// A step's end: at most `VM` of this wave's loads in flight, its LDS accesses
// done, then the block barrier (bare, with compiler fences around it).
template <int VM> __device__ __forceinline__ void step_barrier()
{
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(VM));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ------------------------------------------------------------------ dx = dy W

// A: dy [BM][64] by DMA; B: W [64][BN] turned and dequantized. Waves WMW x WNW.
template <int BM, int BN> constexpr int xgrad_lds() { return 3 * BM * 128 + 2 * BN * 128; }

template <int BITS, int DT, int BM, int BN, int WMW>
__global__ __launch_bounds__(2 * BN) void xgrad_tile_kernel(XgradArgs a, GradPlan plan, int tiles_k, int tiles,
                                                            int per_xcd)
{
    using T = MfmaTraits<DT>;
    using frag_t = typename T::frag_t;
    using C8 = Codes8<BITS>;
    constexpr int WAVES = BN / 32, WNW = WAVES / WMW, WM = BM / WMW, WN = BN / WNW, FM = WM / 32, FN = WN / 32;
    static_assert(FM * 32 * WMW == BM && FN * 32 * WNW == BN, "wave tiles");
    constexpr int A_STAGE = BM * 128, B_STAGE = BN * 128, A_INSTR = A_STAGE / 1024 / WAVES;
    static_assert(A_INSTR * 1024 * WAVES == A_STAGE, "activation stage in whole DMA blocks");
    constexpr int NW = C8::NW;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    char* const a_st = lds;
    char* const b_st = lds + 3 * A_STAGE;

    // Tiles XCD by XCD (block b runs on XCD b % 8), a contiguous run each.
    const int tile = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
    if ((int)(blockIdx.x / 8) >= per_xcd || tile >= tiles)
        return;
    const int64_t m0 = (int64_t)(tile / tiles_k) * BM, k0 = (int64_t)(tile % tiles_k) * BN;
    const int tid = (int)threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WNW, wn = wave % WNW;

    const int steps1 = (int)((a.N + STEP - 1) / STEP);      // of one pair
    const int lo = (int)blockIdx.y * (int)plan.per_split;
    int hi = lo + (int)plan.per_split;
    hi = hi < steps1 * a.nmat ? hi : steps1 * a.nmat;

    // Activation DMA: wave w's instruction i moves rows 8 g .. 8 g + 7 of the
    // tile, g = A_INSTR w + i; lane l lands in row 8 g + l / 8, slot l % 8.
    const uint32_t arow = (uint32_t)(a.dy_stride * 2);
    const int64_t rows_left = a.M - m0;
    const uint32_t a_rows = (uint32_t)(rows_left < BM ? rows_left : BM);
    uint32_t a_off[A_INSTR];
    int a_n[A_INSTR];
#pragma unroll
    for (int i = 0; i < A_INSTR; ++i) {
        const int r = 8 * (wave * A_INSTR + i) + (lane >> 3);
        a_n[i] = 8 * ((lane & 7) ^ turn_swz(r));
        a_off[i] = (uint32_t)r < a_rows ? (uint32_t)r * arow + (uint32_t)a_n[i] * 2 : OOB;
    }
    auto dma_a = [&](int step, int stage) {
        const int p = step >= steps1 ? 1 : 0;
        const int n0 = (step - p * steps1) * STEP;
        // The range ends after the last row's N values, in whole chunks.
        const __amdgpu_buffer_rsrc_t ra = rsrc(static_cast<const char*>(a.dy[p]) + m0 * a.dy_stride * 2,
                                               (a_rows - 1) * arow + ((uint32_t)a.N + 7) / 8 * 16);
#pragma unroll
        for (int i = 0; i < A_INSTR; ++i) {
            const uint32_t off = n0 + a_n[i] < (int)a.N && step < hi ? a_off[i] + (uint32_t)n0 * 2 : OOB;
            dma16(ra, a_st + stage * A_STAGE + (wave * A_INSTR + i) * 1024, off);
        }
    };

    // The weight block of this thread: rows 4 rq + i of the step, columns
    // k0 + 8 o .. k0 + 8 o + 7.
    const TurnMap<BN> turn(tid);
    const uint32_t wrow = (uint32_t)(a.K * BITS / 8), grow = (uint32_t)(a.K / a.gs) * 2;
    const int oct = (int)(k0 / 8) + turn.o;                 // octet in the row
    const bool live = 8 * (int64_t)oct < a.K;
    const uint32_t w_off = live ? (uint32_t)(4 * turn.rq) * wrow + 4u * (uint32_t)C8::word(oct) : OOB;
    const uint32_t g_off = live ? (uint32_t)(4 * turn.rq) * grow + 2u * (uint32_t)(8 * (int64_t)oct / a.gs) : OOB;
    struct Raw {
        uint32_t w[4][NW];
        uint16_t s[4], b[4];
    };
    Raw raw[2];
    auto load_w = [&](int step, Raw& r) {
        const int p = step >= steps1 ? 1 : 0;
        const int n0 = (step - p * steps1) * STEP;
        int64_t left = step < hi ? a.N - n0 : 0;             // rows past the step's read zeros
        const uint32_t rows = (uint32_t)(left < STEP ? left : STEP);
        const __amdgpu_buffer_rsrc_t rw =
            rsrc(reinterpret_cast<const char*>(a.w[p].wq) + (int64_t)n0 * wrow, rows * wrow);
        const __amdgpu_buffer_rsrc_t rs =
            rsrc(static_cast<const char*>(a.w[p].scales) + (int64_t)n0 * grow, rows * grow);
        const __amdgpu_buffer_rsrc_t rb =
            rsrc(static_cast<const char*>(a.w[p].biases) + (int64_t)n0 * grow, rows * grow);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.w[i][0] = __builtin_amdgcn_raw_buffer_load_b32(rw, w_off + (uint32_t)i * wrow, 0, 0);
            if constexpr (NW == 2)
                r.w[i][1] = __builtin_amdgcn_raw_buffer_load_b32(rw, C8::need2(oct) ? w_off + (uint32_t)i * wrow + 4 : OOB, 0, 0);
            r.s[i] = __builtin_amdgcn_raw_buffer_load_b16(rs, g_off + (uint32_t)i * grow, 0, 0);
            r.b[i] = __builtin_amdgcn_raw_buffer_load_b16(rb, g_off + (uint32_t)i * grow, 0, 0);
        }
    };
    // Rows 2 h and 2 h + 1 of the block, dequantized, as one pair per column.
    auto dequant2 = [&](const Raw& r, int h, uint32_t (&p)[8]) {
        float q0[8], q1[8];
        C8::to_f32(r.w[2 * h], oct, q0);
        C8::to_f32(r.w[2 * h + 1], oct, q1);
        const float s0 = Elem<DT>::to_f32(r.s[2 * h]), b0 = Elem<DT>::to_f32(r.b[2 * h]);
        const float s1 = Elem<DT>::to_f32(r.s[2 * h + 1]), b1 = Elem<DT>::to_f32(r.b[2 * h + 1]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p[j] = T::pack2(__builtin_fmaf(q0[j], s0, b0), __builtin_fmaf(q1[j], s1, b1));
    };

    f32x16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x16_t{};
    uint32_t fa[4], fb[4];
    frag_offsets(lane, wm * WM, fa);
    frag_offsets(lane, wn * WN, fb);

    load_w(lo, raw[0]);
    load_w(lo + 1, raw[1]);
    dma_a(lo, 0);
    dma_a(lo + 1, 1);
    {
        uint32_t p01[8], p23[8];
        dequant2(raw[0], 0, p01);
        dequant2(raw[0], 1, p23);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            turn.put(b_st, j, p01[j], p23[j]);
    }
    step_barrier<0>();

    // Step kt, in B stage P: its products, while the raw block of step kt + 1
    // is dequantized into the other stage and that of step kt + 2 is loaded.
    auto run_step = [&](int kt, int a_cur, auto PP) {
        constexpr int P = decltype(PP)::value;
        // The DMA last: the step's end leaves just these in flight.
        load_w(kt + 2, raw[P]);
        __builtin_amdgcn_sched_barrier(0);
        dma_a(kt + 2, a_cur + 2 >= 3 ? a_cur - 1 : a_cur + 2);
        __builtin_amdgcn_sched_barrier(0);
        const char* as = a_st + a_cur * A_STAGE;
        const char* bs = b_st + P * B_STAGE;
        char* bn = b_st + (1 - P) * B_STAGE;
        uint32_t p01[8], p23[8];
        static_for<4>([&](auto KK) {
            constexpr int kk = decltype(KK)::value;
            frag_t af[FM], bf[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i)
                af[i] = *reinterpret_cast<const frag_t*>(as + fa[kk ^ (i & 1)] + 4096 * i);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                bf[j] = *reinterpret_cast<const frag_t*>(bs + fb[kk ^ (j & 1)] + 4096 * j);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = T::mfma(af[i], bf[j], acc[i][j]);
            if constexpr (kk == 0)
                dequant2(raw[1 - P], 0, p01);
            if constexpr (kk == 1)
                dequant2(raw[1 - P], 1, p23);
            if constexpr (kk >= 2) {
#pragma unroll
                for (int j = 4 * (kk - 2); j < 4 * (kk - 2) + 4; ++j)
                    turn.put(bn, j, p01[j], p23[j]);
            }
        });
        step_barrier<A_INSTR>();
    };
    int a_cur = 0;
    for (int kt = lo; kt < hi; kt += 2) {
        run_step(kt, a_cur, std::integral_constant<int, 0>{});
        a_cur = a_cur == 2 ? 0 : a_cur + 1;
        if (kt + 1 < hi) {
            run_step(kt + 1, a_cur, std::integral_constant<int, 1>{});
            a_cur = a_cur == 2 ? 0 : a_cur + 1;
        }
    }
    // No DMA may still be writing the block's LDS when the block ends.
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));

    // Register r of a 32 x 32 tile: row 8 (r / 4) + 4 (lane / 32) + r % 4,
    // column lane % 32. Rows past M are past the resources' range.
    auto rows_of = [&](const void* p, int64_t row0, uint32_t es) {
        return rsrc(static_cast<const char*>(p) + row0 * a.K * es, a_rows * (uint32_t)a.K * es);
    };
    auto each_tile = [&](auto&& f) {
        static_for<FM>([&](auto I) {
            static_for<FN>([&](auto J) {
                const uint32_t row = (uint32_t)(wm * WM + 32 * decltype(I)::value + 4 * half);
                const uint32_t col = (uint32_t)(wn * WN + 32 * decltype(J)::value + (lane & 31));
                const int64_t k = k0 + col;
                // Element offset of register 0, and of register r from it.
                f(acc[I][J], k < a.K ? row * (uint32_t)a.K + (uint32_t)k : OOB);
            });
        });
    };
    auto reg_off = [&](int r) { return (uint32_t)(8 * (r >> 2) + (r & 3)) * (uint32_t)a.K; };
    if (plan.splits > 1) {
        const __amdgpu_buffer_rsrc_t ro = rows_of(a.partial, (int64_t)blockIdx.y * a.M + m0, 4);
        each_tile([&](const f32x16_t& v, uint32_t at) {
            static_for<16>([&](auto R) {
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (float)v[(int)R]), ro,
                                                      at == OOB ? OOB : 4 * (at + reg_off(R)), 0, 0);
            });
        });
    } else if (a.g == nullptr) {
        const __amdgpu_buffer_rsrc_t ro = rows_of(a.out, m0, 2);
        each_tile([&](const f32x16_t& v, uint32_t at) {
            static_for<16>([&](auto R) {
                __builtin_amdgcn_raw_buffer_store_b16(Elem<DT>::from_f32(v[(int)R]), ro,
                                                      at == OOB ? OOB : 2 * (at + reg_off(R)), 0, 0);
            });
        });
    } else {
        const __amdgpu_buffer_rsrc_t rg = rows_of(a.g, m0, 2), ru = rows_of(a.u, m0, 2);
        const __amdgpu_buffer_rsrc_t rdg = rows_of(a.dg, m0, 2), rdu = rows_of(a.du, m0, 2);
        // Without h its range is empty: the stores drop.
        const __amdgpu_buffer_rsrc_t rh =
            rsrc(static_cast<const char*>(a.h) + (a.h != nullptr ? m0 * a.K * 2 : 0),
                 a.h != nullptr ? a_rows * (uint32_t)a.K * 2 : 0u);
        auto close = [&](auto ACT) {
            each_tile([&](const f32x16_t& v, uint32_t at) {
                static_for<2>([&](auto H) {   // eight registers at a time
                    uint16_t g[8], u[8];
                    static_for<8>([&](auto R) {
                        const uint32_t off = at == OOB ? OOB : 2 * (at + reg_off(8 * H + R));
                        g[R] = __builtin_amdgcn_raw_buffer_load_b16(rg, off, 0, 0);
                        u[R] = __builtin_amdgcn_raw_buffer_load_b16(ru, off, 0, 0);
                    });
                    static_for<8>([&](auto R) {
                        const uint32_t off = at == OOB ? OOB : 2 * (at + reg_off(8 * H + R));
                        const float dh = v[8 * (int)H + (int)R], uf = Elem<DT>::to_f32(u[R]);
                        float act, dact;
                        act_grad_f32<decltype(ACT)::value>(Elem<DT>::to_f32(g[R]), act, dact);
                        __builtin_amdgcn_raw_buffer_store_b16(Elem<DT>::from_f32(dh * uf * dact), rdg, off, 0, 0);
                        __builtin_amdgcn_raw_buffer_store_b16(Elem<DT>::from_f32(dh * act), rdu, off, 0, 0);
                        __builtin_amdgcn_raw_buffer_store_b16(Elem<DT>::from_f32(act * uf), rh, off, 0, 0);
                    });
                });
            });
        };
        if (a.act == ACT_SILU)
            close(std::integral_constant<int, ACT_SILU>{});
        else
            close(std::integral_constant<int, ACT_GELU_TANH>{});
    }
}

// ------------------------------------------------------------------ dW = dy^T x

// A: x [64][BK] turned (its LDS rows are k), B: dy [64][BN] turned (n).
// WKW x WNW waves, each 128 k (every group closes inside a wave) x WN n.
template <int BK, int BN> constexpr int wgrad_lds() { return 2 * (BK + BN) * 128; }

template <int BITS, int DT, int BK, int BN>
__global__ __launch_bounds__(2 * BN) void wgrad_tile_kernel(WgradArgs a, GradPlan plan, int tiles_k, int tiles,
                                                            int per_xcd)
{
    using T = MfmaTraits<DT>;
    using frag_t = typename T::frag_t;
    static_assert(BK == BN && (BK == 256 || BK == 128), "one turned block of each operand per thread");
    constexpr int WAVES = BN / 32, WKW = BK / 128, WNW = WAVES / WKW, WN = BN / WNW, FM = 4, FN = WN / 32;
    constexpr int A_STAGE = BK * 128, B_STAGE = BN * 128;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    char* const a_st = lds;
    char* const b_st = lds + 2 * A_STAGE;

    const int item = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
    if ((int)(blockIdx.x / 8) >= per_xcd || item >= tiles * a.nmat)
        return;
    const int mat = item / tiles, tile = item % tiles;
    const int64_t n0 = (int64_t)(tile / tiles_k) * BN, k0 = (int64_t)(tile % tiles_k) * BK;
    const int tid = (int)threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave / WNW, wn = wave % WNW;
    const int lo = (int)blockIdx.y * (int)plan.per_split;
    int hi = lo + (int)plan.per_split;
    const int steps = (int)((a.M + STEP - 1) / STEP);
    hi = hi < steps ? hi : steps;

    // Raw blocks: rows 4 rq + i of the step, 16 bytes each of x and dy. K and
    // N are multiples of 8: an octet is inside a row or past it.
    const TurnMap<BN> turn(tid);
    const uint32_t xrow = (uint32_t)a.K * 2, yrow = (uint32_t)(a.dy_stride * 2);
    const uint32_t x_off = k0 + 8 * turn.o < a.K ? (uint32_t)(4 * turn.rq) * xrow + (uint32_t)(k0 + 8 * turn.o) * 2 : OOB;
    const uint32_t y_off = n0 + 8 * turn.o < a.N ? (uint32_t)(4 * turn.rq) * yrow + (uint32_t)(n0 + 8 * turn.o) * 2 : OOB;
    struct Raw {
        u32x4_t x[4], y[4];
    };
    Raw raw[2];
    auto load = [&](int step, Raw& r) {
        const int64_t m = (int64_t)step * STEP;
        const int64_t left = step < hi ? a.M - m : 0;
        const uint32_t rows = (uint32_t)(left < STEP ? left : STEP);
        const __amdgpu_buffer_rsrc_t rx = rsrc(static_cast<const char*>(a.x) + m * xrow, rows * xrow);
        const __amdgpu_buffer_rsrc_t ry = rsrc(static_cast<const char*>(a.dy[mat]) + m * yrow, rows * yrow);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.x[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rx, x_off + (uint32_t)i * xrow, 0, 0));
            r.y[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ry, y_off + (uint32_t)i * yrow, 0, 0));
        }
    };
    // Columns 2 d and 2 d + 1 of a raw block, turned.
    auto put2 = [&](char* stage, const u32x4_t (&v)[4], int d) {
        turn.put(stage, 2 * d, __builtin_amdgcn_perm(v[1][d], v[0][d], 0x05040100u),
                 __builtin_amdgcn_perm(v[3][d], v[2][d], 0x05040100u));
        turn.put(stage, 2 * d + 1, __builtin_amdgcn_perm(v[1][d], v[0][d], 0x07060302u),
                 __builtin_amdgcn_perm(v[3][d], v[2][d], 0x07060302u));
    };

    f32x16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x16_t{};
    uint32_t fa[4], fb[4];
    frag_offsets(lane, wk * 128, fa);
    frag_offsets(lane, wn * WN, fb);

    load(lo, raw[0]);
    load(lo + 1, raw[1]);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        put2(a_st, raw[0].x, d);
        put2(b_st, raw[0].y, d);
    }
    __syncthreads();

    auto run_step = [&](int kt, auto PP) {
        constexpr int P = decltype(PP)::value;
        load(kt + 2, raw[P]);
        __builtin_amdgcn_sched_barrier(0);   // issued now, not where the registers are next needed
        const char* as = a_st + P * A_STAGE;
        const char* bs = b_st + P * B_STAGE;
        char* an = a_st + (1 - P) * A_STAGE;
        char* bn = b_st + (1 - P) * B_STAGE;
        static_for<4>([&](auto KK) {
            constexpr int kk = decltype(KK)::value;
            frag_t af[FM], bf[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i)
                af[i] = *reinterpret_cast<const frag_t*>(as + fa[kk ^ (i & 1)] + 4096 * i);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                bf[j] = *reinterpret_cast<const frag_t*>(bs + fb[kk ^ (j & 1)] + 4096 * j);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = T::mfma(af[i], bf[j], acc[i][j]);
            put2(an, raw[1 - P].x, kk);
            put2(bn, raw[1 - P].y, kk);
        });
        // LDS only: the loads in flight belong to registers.
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    for (int kt = lo; kt < hi; kt += 2) {
        run_step(kt, std::integral_constant<int, 0>{});
        if (kt + 1 < hi)
            run_step(kt + 1, std::integral_constant<int, 1>{});
    }

    // Tile i, register r: k = k0 + 128 wk + 32 i + 8 (r / 4) + 4 half + r % 4
    // of weight row n: unit i of the wave's four.
    const int64_t row_words = a.K * BITS / 32;
    const int64_t kw = k0 + 128 * wk;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int64_t n = n0 + wn * WN + 32 * j + (lane & 31);
        float ps[4], pb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[BITS];
            const bool live = n < a.N && kw + 32 * i < a.K;
#pragma unroll
            for (int b = 0; b < BITS; ++b)
                w[b] = live ? a.wq[mat][n * row_words + (kw / 32 + i) * BITS + b] : 0u;
            float s = 0.0f, b = 0.0f;
            static_for<16>([&](auto R) {
                constexpr int r = decltype(R)::value, c = 8 * (r >> 2) + (r & 3);
                const uint32_t q = half ? unit_code<BITS, c + 4>(w) : unit_code<BITS, c>(w);
                s = __builtin_fmaf((float)q, acc[i][j][r], s);
                b += acc[i][j][r];
            });
            ps[i] = s + __shfl_xor(s, 32, 64);
            pb[i] = b + __shfl_xor(b, 32, 64);
        }
        if (n < a.N) {
            const int per = a.gs / 32;   // tiles of a group
            for (int i = 0; i < 4 && kw + 32 * i < a.K; i += per) {
                float v = 0.0f;
                static_for<4>([&](auto I) {
                    constexpr int ii = decltype(I)::value;
                    if (ii >= i && ii < i + per)
                        v += half ? pb[ii] : ps[ii];
                });
                wgrad_store<DT>(a, plan, mat, (int)blockIdx.y, n, (kw + 32 * i) / a.gs, half != 0, v);
            }
        }
    }
}

} // namespace gradtile
} // namespace qp
