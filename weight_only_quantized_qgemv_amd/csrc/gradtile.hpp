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
// Both are bound by the work beside the matrix instructions, which are busy 60
// to 62% of the time: a step of 256 x 256 outputs has 2048 cycles of them on
// each SIMD (and, with eight waves, as many of LDS reads and writes). 14336 x
// 4096, 4-bit, bf16, 2048 / 4096 / 8192 rows: dx 227 / 405 / 808 us, dW 225 / 425
// / 831 us (1058 to 1190 TFLOP/s; a library's product of dense operands 205 / 336
// / 685 us). The roundings of the weights here make dx 0.0023 of its size
// off 64 bits in bf16, where its own rounding alone makes it 0.0017.
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

// The accumulators of the four-wave tiles fill the accumulation registers, and
// are read from there one by one at a tile's end: left to itself the compiler
// copies them to vector registers by the tile, which pushes the pipeline's
// values out to scratch memory inside the steps. acc_settle() first: it lets
// the last matrix instructions finish (their results are not interlocked
// against the reads).
__device__ __forceinline__ void acc_settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }
__device__ __forceinline__ float acc_read(float v)
{
    float r;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(r) : "a"(v));
    return r;
}

// A resource from values that are the same in every lane, said so: kept in
// vector registers, each of its loads would be a loop over the lanes' values.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const char* p, uint32_t bytes)
{
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)u);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
    return rsrc(reinterpret_cast<const void*>(((uint64_t)hi << 32) | lo),
                (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes));
}

// A scheduling barrier's mask: everything but memory loads may cross it.
constexpr int kNotLoads = 0x38F;

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

// PIECES: a call of several over pieces of the contraction (XgradArgs::sums).
template <int BITS, int DT, int BM, int BN, int WMW, bool PIECES>
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
    // DMA instructions from .. to - 1 of a step's.
    auto dma_a = [&](int step, int stage, int from, int to) {
        const int p = step >= steps1 ? 1 : 0;
        const int n0 = (step - p * steps1) * STEP;
        // The range ends after the last row's N values, in whole chunks.
        const __amdgpu_buffer_rsrc_t ra = rsrc(static_cast<const char*>(a.dy[p]) + m0 * a.dy_stride * 2,
                                               (a_rows - 1) * arow + ((uint32_t)a.N + 7) / 8 * 16);
#pragma unroll
        for (int i = from; i < to; ++i) {
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
    // Loads a step, which its end counts: at 6 and 8 bits a row's two words,
    // which are always both needed, are one load by their form here, so that
    // no merging of the compiler's changes the count (at 3 bits the second has
    // an offset of its own, and two loads stay two).
    constexpr bool PAIR = BITS == 6 || BITS == 8;
    constexpr int W_LOADS = 4 * (PAIR ? 1 : NW) + 8;
    Raw raw[2];
    // Rows from .. to - 1 of a step's block.
    auto load_w = [&](int step, Raw& r, int from, int to) {
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
        for (int i = from; i < to; ++i) {
            if constexpr (PAIR) {
                const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(rw, w_off + (uint32_t)i * wrow, 0, 0));
                r.w[i][0] = v[0];
                r.w[i][1] = v[1];
            } else
                r.w[i][0] = __builtin_amdgcn_raw_buffer_load_b32(rw, w_off + (uint32_t)i * wrow, 0, 0);
            if constexpr (NW == 2 && !PAIR)
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

    load_w(lo, raw[0], 0, 4);
    load_w(lo + 1, raw[1], 0, 4);
    dma_a(lo, 0, 0, A_INSTR);
    dma_a(lo + 1, 1, 0, A_INSTR);
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
        const char* as = a_st + a_cur * A_STAGE;
        const char* bs = b_st + P * B_STAGE;
        char* bn = b_st + (1 - P) * B_STAGE;
        const int a_new = a_cur + 2 >= 3 ? a_cur - 1 : a_cur + 2;
        uint32_t p01[8], p23[8];
        static_for<4>([&](auto KK) {
            constexpr int kk = decltype(KK)::value;
            // The step's loads a share a kk (only loads are held there): all at
            // its start, they keep the matrix instructions waiting until the
            // address units have taken them (the backward pass of a 4096 x 14336
            // block at 2048 rows 1457 us, now 1416). The step's end leaves them in
            // flight, and no older ones: the DMA of step kt + 1 is there.
            // (Waiting for the weight loads too put a memory latency into every
            // step.)
            __builtin_amdgcn_sched_barrier(kNotLoads);
            if constexpr (kk < 2)
                load_w(kt + 2, raw[P], 2 * kk, 2 * kk + 2);
            else
                dma_a(kt + 2, a_new, (kk - 2) * A_INSTR / 2, (kk - 1) * A_INSTR / 2);
            __builtin_amdgcn_sched_barrier(kNotLoads);
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
        step_barrier<A_INSTR + W_LOADS>();
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
    } else if constexpr (PIECES) {   // (16 loads at a time)
        const __amdgpu_buffer_rsrc_t rs = rows_of(a.sums, m0, 4), ro = rows_of(a.out, m0, 2);
        const float scale = a.last && a.scale != nullptr ? *a.scale : 1.0f;
        each_tile([&](const f32x16_t& v, uint32_t at) {
            float t[16];
            static_for<16>([&](auto R) {
                t[R] = a.first ? 0.0f : __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                    rs, at == OOB ? OOB : 4 * (at + reg_off(R)), 0, 0));
            });
            static_for<16>([&](auto R) {
                const float w = v[(int)R] + t[R];
                if (a.last)
                    __builtin_amdgcn_raw_buffer_store_b16(Elem<DT>::from_f32(w * scale), ro,
                                                          at == OOB ? OOB : 2 * (at + reg_off(R)), 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, w), rs,
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

// The sums of a wave's 128 k (from kw on) x 32 FN weight rows (from nw on).
// Tile i, register r: k = kw + 32 i + 8 (r / 4) + 4 half + r % 4 of weight row
// nw + 32 j + lane % 32: unit i of the wave's four. All the codes are asked
// for before any is used; a unit is moved down by the half's four codes once.
// SCALED: the results are multiplied by `scale`.
template <int BITS, int DT, int FN, bool SCALED, bool WIDE = false>
__device__ __forceinline__ void wgrad_close(const WgradArgs& a, int splits, int mat, int split, int64_t kw,
                                            int64_t nw, int lane, float scale, const f32x16_t (&acc)[4][FN])
{
    // Opaque here, so that the addresses are formed at the tile's end and not
    // kept in registers through the steps.
    uint32_t row = (uint32_t)(a.K * BITS / 8);
    asm volatile("" : "+s"(row), "+v"(lane));
    const int half = lane >> 5;
    // Rows of the tile from nw on; units past K are past the row's codes.
    const int64_t left = a.N - nw;
    const uint32_t rows = left > 32 * FN ? 32 * FN : left > 0 ? (uint32_t)left : 0u;
    const __amdgpu_buffer_rsrc_t rw = rsrc(reinterpret_cast<const char*>(a.wq[mat]) + nw * row, rows * row);
    uint32_t w[FN][4][BITS];
    static_for<FN>([&](auto J) {
        static_for<4>([&](auto I) {
            constexpr int i = decltype(I)::value, j = decltype(J)::value;
            const uint32_t off = kw + 32 * i < a.K
                ? (uint32_t)(32 * j + (lane & 31)) * row + (uint32_t)(kw / 32 + i) * (4 * BITS) : OOB;
#pragma unroll
            for (int b = 0; b < BITS; ++b)
                w[j][i][b] = __builtin_amdgcn_raw_buffer_load_b32(rw, off + 4 * b, 0, 0);
        });
    });
    // Of unit i of row tile j: the scale's sum in lanes 0-31, the bias's in the
    // others. (No branch before the last of them: the accumulators would be
    // moved about.)
    float v[FN][4];
    static_for<FN>([&](auto J) {
        constexpr int j = decltype(J)::value;
        static_for<4>([&](auto I) {
            constexpr int i = decltype(I)::value;
            uint32_t u[BITS];   // the unit from code 4 half on
#pragma unroll
            for (int b = 0; b < BITS; ++b) {
                constexpr int WS = 4 * BITS / 32, SH = 4 * BITS % 32;   // four codes: whole words and bits
                const uint32_t lo = b + WS < BITS ? w[j][i][b + WS < BITS ? b + WS : 0] : 0u;
                const uint32_t hi = b + WS + 1 < BITS ? w[j][i][b + WS + 1 < BITS ? b + WS + 1 : 0] : 0u;
                const uint32_t moved = SH == 0 ? lo : __builtin_amdgcn_alignbit(hi, lo, SH);
                u[b] = half ? moved : w[j][i][b];
            }
            using CB = CodeBytes<BITS>;
            uint32_t bw[CB::NBW];
            CB::split(u, bw);
            float s = 0.0f, b = 0.0f;
            static_for<16>([&](auto R) {
                constexpr int r = decltype(R)::value, c = 8 * (r >> 2) + (r & 3);
                float d;
                if constexpr (WIDE)
                    d = acc_read(acc[i][j][r]);
                else
                    d = acc[i][j][r];
                s = __builtin_fmaf(CB::template code<c>(bw), d, s);
                b += d;
            });
            // The upper half of s for the lower half of b, then both halves' sum.
            const auto x = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, s),
                                                            __builtin_bit_cast(uint32_t, b), false, false);
            v[j][i] = __builtin_bit_cast(float, (uint32_t)x[0]) + __builtin_bit_cast(float, (uint32_t)x[1]);
            __builtin_amdgcn_sched_barrier(0);   // one tile's values at a time
        });
    });
    // Lanes 0-31 store the scales' sums, lanes 32-63 the biases'.
    using St = typename Elem<DT>::storage;
    const int64_t groups = a.K / a.gs, count = a.N * groups, at = (nw + (lane & 31)) * groups + kw / a.gs;
    const bool parts = splits > 1;
    float* const pd = parts ? a.partial + (((int64_t)split * a.nmat + mat) * 2 + half) * count + at : nullptr;
    St* const sd = parts ? nullptr : static_cast<St*>(half ? a.dbiases[mat] : a.dscales[mat]) + at;
    const int per = a.gs / 32;                                      // units of a group
    const int live = (int)((a.K - kw) / a.gs < 4 / per ? (a.K - kw) / a.gs : 4 / per);   // groups in range
    auto store = [&](int j, int g, float v) {
        if (nw + 32 * j + (lane & 31) < a.N && g < live) {
            const int64_t o = (int64_t)(32 * j) * groups + g;
            if (parts)
                pd[o] = v;
            else
                sd[o] = Elem<DT>::from_f32(SCALED ? v * scale : v);
        }
    };
    if (per == 1) {
        static_for<FN>([&](auto J) { static_for<4>([&](auto I) { store(J, I, v[J][I]); }); });
    } else if (per == 2) {
        static_for<FN>([&](auto J) {
            store(J, 0, v[J][0] + v[J][1]);
            store(J, 1, v[J][2] + v[J][3]);
        });
    } else {
        static_for<FN>([&](auto J) { store(J, 0, (v[J][0] + v[J][1]) + (v[J][2] + v[J][3])); });
    }
}

// A: x [64][BK] turned (its LDS rows are k), B: dy [64][BN] turned (n).
// WKW x WNW waves, each 128 k (every group closes inside a wave) x WN n.
template <int BK, int BN> constexpr int wgrad_lds() { return 2 * (BK + BN) * 128; }

// The factor of a call's results, read before the steps: at the tiles' ends it is waited
// for behind the codes (8 rows of 4096 x 32000 65.8 us, now 61).
template <bool SCALED> __device__ __forceinline__ float wgrad_factor(const WgradArgs& a)
{
    if constexpr (SCALED)
        return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, *a.scale)));
    else
        return 1.0f;
}

template <int BITS, int DT, int BK, int BN, bool SCALED>
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
    const float scale = wgrad_factor<SCALED>(a);
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

    wgrad_close<BITS, DT, FN, SCALED>(a, plan.splits, mat, (int)blockIdx.y, k0 + 128 * wk, n0 + wn * WN, lane, scale, acc);
}

// The same product with four waves of 128 k x 128 n, one on each SIMD: a
// fragment is read from LDS by half as many waves, and nothing but the step's
// own order has to hide the latencies. So the order is fixed: each kk's 16
// matrix instructions carry, between them, the reads of the next kk's
// fragments and a share of the turning of step kt + 1. The step's one barrier
// stands before its last kk: by then the next step's tile is written and this
// step's last fragments are in registers, and the last kk's instructions
// cover the first reads of the next step.
// The blocks are persistent (one a CU) and the pipeline runs on from one tile
// to the next: loads and turning are two steps and one step ahead of the
// products, in whatever tile that is, so only the sums at a tile's end stand
// still. There are tiles for every CU (wgrad_plan), so the contraction is whole.
struct WideItem {
    int mat, kt;   // weight, next step
    int64_t n0, k0;
};

// Tiles in the order in which an XCD's blocks share most: bands of 8 tiles of
// k, within a band row by row of n.
__device__ __forceinline__ void band_order(int tile, int tiles_n, int tiles_k, int& tn, int& tk)
{
    const int band = tile / (8 * tiles_n), in = tile % (8 * tiles_n);
    const int width = tiles_k - 8 * band < 8 ? tiles_k - 8 * band : 8;
    tn = in / width;
    tk = 8 * band + in % width;
}

template <int BITS, int DT, bool SCALED>
__global__ __launch_bounds__(256) void wgrad_wide_kernel(WgradArgs a, int tiles_n, int tiles_k)
{
    using T = MfmaTraits<DT>;
    using frag_t = typename T::frag_t;
    constexpr int BT = 256, STAGE = BT * 128;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    char* const a_st = lds;
    char* const b_st = lds + 2 * STAGE;

    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wk = wave >> 1, wn = wave & 1;
    const float scale = wgrad_factor<SCALED>(a);
    const int steps = (int)((a.M + STEP - 1) / STEP);
    // Items: tiles of every weight, XCD by XCD.
    const int tiles = tiles_n * tiles_k, items = tiles * a.nmat, per_xcd = (items + 7) / 8;
    const int local = (int)(blockIdx.x / 8), stride = (int)(gridDim.x / 8), first = (int)(blockIdx.x % 8) * per_xcd;
    auto item_at = [&](int round, WideItem& it) {
        const int l = local + round * stride;
        if (l >= per_xcd || first + l >= items)
            return false;
        const int i = first + l;
        it.mat = i / tiles;
        int tn, tk;
        band_order(i % tiles, tiles_n, tiles_k, tn, tk);
        it.n0 = (int64_t)tn * BT;
        it.k0 = (int64_t)tk * BT;
        it.kt = 0;
        return true;
    };
    WideItem cur, ahead;   // the item being multiplied, and that being loaded
    if (!item_at(0, cur))
        return;
    ahead = cur;

    // One 8 x 8 block of each operand a thread: contraction rows 8 ro .. 8 ro + 7
    // of the step, columns 8 o .. 8 o + 7 of the tile. A column's eight values are
    // one 16-byte chunk of its LDS row.
    const int o = tid & 31, ro = tid >> 5;
    const uint32_t xrow = (uint32_t)a.K * 2, yrow = (uint32_t)(a.dy_stride * 2);
    uint32_t off[2];   // of x and dy, in the item being loaded
    auto set_off = [&]() {
        const int64_t k = ahead.k0 + 8 * o, n = ahead.n0 + 8 * o;
        off[0] = k < a.K ? (uint32_t)(8 * ro) * xrow + (uint32_t)k * 2 : OOB;
        off[1] = n < a.N ? (uint32_t)(8 * ro) * yrow + (uint32_t)n * 2 : OOB;
    };
    // LDS offset of column 8 o + j: chunk ro of that row.
    uint32_t at[4];
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
        at[jj] = (uint32_t)((8 * o + 2 * jj) * 128 + ((ro ^ turn_swz(8 * o + 2 * jj)) << 4));
    // The step being loaded: its 64 rows of x and dy, kept as running pointers
    // and built into resources once a step (at each load, or from the item's
    // numbers at each step, that scalar work costs more than the loads).
    const char *xp, *yp;
    int64_t left;   // rows from the step's first on
    __amdgpu_buffer_rsrc_t rx, ry;
    auto set_rows = [&]() {
        const uint32_t rows = (uint32_t)(left < STEP ? left > 0 ? left : 0 : STEP);
        rx = uniform_rsrc(xp, rows * xrow);
        ry = uniform_rsrc(yp, rows * yrow);
    };
    auto set_item = [&]() {
        const bool any = ahead.kt < steps;
        const int64_t m = any ? (int64_t)ahead.kt * STEP : 0;
        left = any ? a.M - m : 0;
        xp = static_cast<const char*>(a.x) + m * xrow;
        yp = static_cast<const char*>(ahead.mat ? a.dy[1] : a.dy[0]) + m * yrow;
        set_off();
        set_rows();
    };
    set_item();
    int ahead_round = 0;
    auto advance = [&]() {   // the load cursor, one step on
        if (++ahead.kt < steps) {
            xp += (int64_t)STEP * xrow;
            yp += (int64_t)STEP * yrow;
            left -= STEP;
            set_rows();
        } else {
            if (!item_at(++ahead_round, ahead))
                ahead.kt = 0x3FFFFFFF;   // nothing left: loads read zeros
            set_item();
        }
    };
    u32x4_t raw[2][8];
    auto load = [&](auto G, auto I) {   // row i of operand g's block
        constexpr int g = decltype(G)::value, i = decltype(I)::value;
        // (The row goes into the offset that the range is checked with.)
        raw[g][i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
            g == 0 ? rx : ry, off[g] + (uint32_t)i * (g == 0 ? xrow : yrow), 0, 0));
    };
    // Column j of operand g's block, turned, into a stage.
    auto put = [&](int stage, auto G, auto J) {
        constexpr int g = decltype(G)::value, j = decltype(J)::value, d = j / 2;
        constexpr uint32_t sel = j % 2 ? 0x07060302u : 0x05040100u;
        const u32x4_t(&v)[8] = raw[g];
        *reinterpret_cast<u32x4_t*>((g == 0 ? a_st : b_st) + stage * STAGE + at[d] + 128 * (j & 1)) =
            u32x4_t{__builtin_amdgcn_perm(v[1][d], v[0][d], sel), __builtin_amdgcn_perm(v[3][d], v[2][d], sel),
                    __builtin_amdgcn_perm(v[5][d], v[4][d], sel), __builtin_amdgcn_perm(v[7][d], v[6][d], sel)};
    };

    uint32_t fa[4], fb[4];
    frag_offsets(lane, wk * 128, fa);
    frag_offsets(lane, wn * 128, fb);
    frag_t af[2][4], bf[2][4];
    // Fragment i (0..3: A, 4..7: B) of kk into buffer kk & 1.
    auto read = [&](int stage, auto KK, auto I) {
        constexpr int kk = decltype(KK)::value, i = decltype(I)::value;
        if constexpr (i < 4)
            af[kk & 1][i] = *reinterpret_cast<const frag_t*>(a_st + stage * STAGE + fa[kk ^ (i & 1)] + 4096 * i);
        else
            bf[kk & 1][i - 4] = *reinterpret_cast<const frag_t*>(b_st + stage * STAGE + fb[kk ^ (i & 1)] + 4096 * (i - 4));
    };

    static_for<2>([&](auto G) { static_for<8>([&](auto I) { load(G, I); }); });
    advance();
    static_for<2>([&](auto G) {
        static_for<8>([&](auto J) { put(0, G, J); });
        static_for<8>([&](auto I) { load(G, I); });
    });
    __syncthreads();
    static_for<8>([&](auto I) { read(0, std::integral_constant<int, 0>{}, I); });

    int stage = 0;
    for (int round = 0; item_at(round, cur); ++round) {
      f32x16_t acc[4][4];
      static_for<4>([&](auto I) { static_for<4>([&](auto J) { acc[I][J] = f32x16_t{}; }); });
#pragma unroll 1
      for (; cur.kt < steps; ++cur.kt) {
        advance();
        static_for<4>([&](auto KK) {
            constexpr int kk = decltype(KK)::value;
            if constexpr (kk == 3) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
            }
            static_for<16>([&](auto Q) {
                constexpr int q = decltype(Q)::value, i = q / 4, j = q % 4;
                acc[i][j] = T::mfma(af[kk & 1][i], bf[kk & 1][j], acc[i][j]);
                // The next fragments, one a matrix instruction.
                if constexpr (q < 8)
                    read(kk == 3 ? 1 - stage : stage, std::integral_constant<int, (kk + 1) & 3>{},
                         std::integral_constant<int, q>{});
                // Slot 16 g + 2 j + 1: column j of operand g is turned; slot 16 g +
                // 16 + 2 i: row i of its next block is loaded. One load every
                // other slot: four in one slot hold the wave up until the address
                // units have taken them (276 us, now 237, for 2048 rows of a
                // 14336 x 4096 weight, together with building the rows' resources
                // once a step).
                constexpr int slot = 16 * kk + q, h = slot / 2 % 8;
                if constexpr (slot % 2 == 1 && kk < 2)
                    put(1 - stage, std::integral_constant<int, kk>{}, std::integral_constant<int, h>{});
                if constexpr (slot % 2 == 0 && (kk == 1 || kk == 2))
                    load(std::integral_constant<int, kk - 1>{}, std::integral_constant<int, h>{});
                __builtin_amdgcn_sched_barrier(0);
            });
        });
        stage = 1 - stage;
      }
      acc_settle();
      wgrad_close<BITS, DT, 4, SCALED, true>(a, 1, cur.mat, 0, cur.k0 + 128 * wk, cur.n0 + 128 * wn, lane, scale, acc);
    }
}

} // namespace gradtile
} // namespace qp
