// model_ops.hpp — host-side launchers of the operators around the quantized
// products: the dense gated feed-forward block and its gradients, the
// gradients of a quantized linear layer, the packed embedding table and the
// adjustment of logits. Implemented by the kernel files, called by the C ABI
// layer (api_model.cpp), which validates the arguments; every launcher
// returns the hipError_t of its launches.
#pragma once

#include "launch.hpp"

namespace qp {

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
inline size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// One packed weight [N, K] with its scales and biases.
struct QWeight {
    const uint32_t* wq;     // [N, K*bits/32]
    const void* scales;     // [N, K/gs]
    const void* biases;
};

// Activations of the gated block, numbered as qp_act.
enum : int { ACT_SILU = 0, ACT_GELU_TANH = 1 };

// ---- the gated block, forward (ffn.hip)
struct FfnArgs {
    const void* x;          // [M, D] of dt
    int dt, act;
    int64_t M, D, F;
    QWeight gate, up, down; // [F, D], [F, D], [D, F]
    int bits, gs;
    void* saved[2];         // [M, F] of dt each (the gate's product, the up's), or null
    void* y;                // [M, D] of dt
    void* workspace;        // >= ffn_workspace_bytes, 16-byte aligned
};
size_t ffn_workspace_bytes(int64_t m, int64_t d, int64_t f, int dt);
hipError_t launch_ffn(const FfnArgs& a, hipStream_t stream);

// h = act(gate product) * (up product) in one launch, without or with storing
// the two products; false in *done where the shape is another path's.
struct GateUpArgs {
    const void* x;          // [M, K]
    int dt, act;
    int64_t M, K, N;        // N rows of each matrix
    QWeight gate, up;
    int bits, gs;
    void* h;                // [M, N]
    void* saved[2];         // [M, N] each, or null
};
// The block's products with the contraction in pieces, for batches whose tiles
// are too few to fill the GPU: x [M, K] times one or two matrices of N rows, as
// fp32 sums partial [splits][matrices][M][N] of per_split 64-wide steps each.
struct FfnSplit {
    int tile;               // activation rows of a tile
    int splits;             // 1: not in pieces
    int per_split;          // steps of a piece (ffn_split: 0 where the product is another path's)
    size_t partial_bytes;
    int64_t kp;             // ffn_split: the contraction filled up to whole 64-wide steps, 0: as it is
    size_t pad_bytes;       // and what the filled-up x, scales, biases and codes take
};
FfnSplit ffn_split(int64_t m, int64_t k, int64_t n, int nmat, int dt);
struct FfnSplitArgs {
    const void* x;
    int dt;
    int64_t M, K, N, wk;    // codes in a row of the weights: K, or less (gemm_core.hpp)
    QWeight w[2];
    int nmat, bits, gs;
    FfnSplit plan;
    float* partial;
};
// y = x W^T for any type, size and alignment (ffn_any.hip), in pieces of 32-wide
// steps where the plan asks for it: as fp32 sums to `partial` [splits], pieces
// partial_stride elements apart, or (null) as y.
FfnSplit ffn_any_plan(int64_t m, int64_t k, int64_t n);
struct FfnAnyArgs {
    const void* x;
    int dt;
    int64_t M, K, N;
    QWeight w;
    int gs;
    FfnSplit plan;
    float* partial;
    int64_t partial_stride;
    void* y;
};
#define QP_GATEUP_DECL(B) \
    hipError_t launch_ffn_any_b##B(const FfnAnyArgs& a, hipStream_t stream); \
    hipError_t launch_gate_up_b##B(const GateUpArgs& a, hipStream_t stream, bool* done); \
    hipError_t launch_ffn_split_b##B(const FfnSplitArgs& a, hipStream_t stream);
QP_GATEUP_DECL(2)
QP_GATEUP_DECL(3)
QP_GATEUP_DECL(4)
QP_GATEUP_DECL(6)
QP_GATEUP_DECL(8)
#undef QP_GATEUP_DECL

// ---- gradients (grad.hip, xgrad.hip, wgrad.hip)

// out[M, K] = sum over the nmat pairs of  dy[p] [M, N] @ dequant(W[p]) [N, K].
// With `g` set it is the gated block's down projection seen from behind: the
// product is dh, and dg = dh u act'(g), du = dh act(g), h = act(g) u are
// written instead of it.
struct XgradArgs {
    const void* dy[2];      // [M, N] of dt, rows dy_stride elements apart
    int64_t dy_stride;
    QWeight w[2];           // [N, K]
    int nmat, dt, act;
    int64_t M, N, K;
    int bits, gs;
    void* out;              // [M, K] of dt
    const void *g, *u;      // [M, K] of dt, or null
    void *dg, *du, *h;      // [M, K] of dt
    float* partial;         // fp32 partial sums of the splits (xgrad_plan)
};

// dscales[n, G] = sum_{k in G} q[n, k] dW[n, k], dbiases[n, G] = sum_{k in G} dW[n, k],
// dW = dy^T x, for one or two (dy, weight) pairs over one x.
struct WgradArgs {
    const void* x;          // [M, K] of dt
    const void* dy[2];      // [M, N] of dt, rows dy_stride elements apart
    int64_t dy_stride;
    const uint32_t* wq[2];  // [N, K*bits/32]
    int nmat, dt;
    int64_t M, N, K;
    int bits, gs;
    void* dscales[2];       // [N, K/gs] of dt
    void* dbiases[2];
    float* partial;         // fp32 partial sums of the splits (wgrad_plan)
};

// How a gradient product is cut: `tile` chooses the kernel and its tile,
// `splits` the pieces of the contraction (per_split steps of the kernel each),
// whose fp32 partial sums take partial_bytes.
struct GradPlan {
    int tile;               // 0: the fp32 kernel for every shape; else see gradtile.hpp
    int splits;
    int64_t per_split;
    size_t partial_bytes;
};
// The plan for these sizes: `tiles` asks for the matrix-core tile kernels
// (16-bit activations in rows of whole 16-byte pieces, 16-byte aligned).
GradPlan xgrad_plan(int64_t m, int64_t n, int64_t k, int nmat, bool tiles);
GradPlan wgrad_plan(int64_t m, int64_t n, int64_t k, int nmat, int gs, bool tiles);
#define QP_GRAD_DECL(B)                                                                        \
    hipError_t launch_xgrad_b##B(const XgradArgs& a, const GradPlan& p, hipStream_t stream);   \
    hipError_t launch_wgrad_b##B(const WgradArgs& a, const GradPlan& p, hipStream_t stream);
QP_GRAD_DECL(2)
QP_GRAD_DECL(3)
QP_GRAD_DECL(4)
QP_GRAD_DECL(6)
QP_GRAD_DECL(8)
#undef QP_GRAD_DECL

struct LinearGradArgs {
    const void *x, *dy;     // [M, K], [M, N] of dt
    int dt;
    int64_t M, K, N;
    QWeight w;
    int bits, gs;
    void* dx;               // [M, K] of dt, or null
    void *dscales, *dbiases;   // [N, K/gs] of dt, or both null
    void* workspace;        // >= linear_grad_workspace_bytes, 16-byte aligned
};
size_t linear_grad_workspace_bytes(int64_t m, int64_t k, int64_t n, int gs, int dt);
hipError_t launch_linear_grad(const LinearGradArgs& a, hipStream_t stream);

struct FfnGradArgs {
    const void *x, *dy;     // [M, D] of dt
    const void* saved;      // [2, M, F] of dt
    int dt, act;
    int64_t M, D, F;
    QWeight gate, up, down;
    int bits, gs;
    void* dx;               // [M, D] of dt, or null
    void *dgate[2], *dup[2], *ddown[2];   // scales, biases; null pairs are not computed
    void* workspace;        // >= ffn_grad_workspace_bytes, 16-byte aligned
};
size_t ffn_grad_workspace_bytes(int64_t m, int64_t d, int64_t f, int gs, int dt);
hipError_t launch_ffn_grad(const FfnGradArgs& a, hipStream_t stream);

// ---- the packed embedding table (embedding.hip)
struct EmbedArgs {
    const int32_t* ids;     // [T]
    int64_t T, V, K;
    QWeight table;          // [V, K]
    int dt, bits, gs;
    float factor;
    void* out;              // [T, K] of dt
};
hipError_t launch_embedding(const EmbedArgs& a, hipStream_t stream);

struct EmbedGradArgs {
    const int32_t* ids;     // [T]
    const void* dout;       // [T, K] of dt
    const uint32_t* wq;     // [V, K*bits/32]
    int64_t T, V, K;
    int dt, bits, gs;
    float factor;
    void *dscales, *dbiases;   // [V, K/gs] of dt
    void* workspace;        // >= embedding_grad_workspace_bytes, 16-byte aligned
};
size_t embedding_grad_workspace_bytes(int64_t t, int64_t k, int gs);
hipError_t launch_embedding_grad(const EmbedGradArgs& a, hipStream_t stream);

// ---- logits (logits.hip)
struct LogitsArgs {
    const void* logits;     // [rows, vocab] of dt, rows in_stride elements apart
    int dt;
    int64_t rows, vocab, in_stride;
    const int32_t* history; // tokens of all sequences (null: no penalties)
    int64_t history_len;
    const int32_t* offsets; // [rows + 1]
    const int32_t* prompt_lens;   // [rows], or null (no prompt tokens)
    const float *repetition, *frequency, *presence;   // [rows] each, or null
    const int32_t* bias_ids;      // sparse biases of all rows (null: none)
    const float* bias_values;
    int64_t bias_len;
    const int32_t* bias_offsets;  // [rows + 1]
    const uint32_t* mask;   // [rows, mask_stride] words, or null
    int64_t mask_stride;    // words between two rows (0: one row for all)
    void* out;              // [rows, vocab] of dt, rows out_stride elements apart
    int64_t out_stride;
};
hipError_t launch_logits_adjust(const LogitsArgs& a, hipStream_t stream);

} // namespace qp
