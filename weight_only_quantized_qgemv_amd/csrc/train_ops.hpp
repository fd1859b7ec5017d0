// train_ops.hpp — host-side launchers of the operators that train and score a
// model around the packed layers: the norms around a block and the cross entropy
// over a packed head, with their gradients. Implemented by the kernel files,
// called by the C ABI layer (api_train.cpp), which validates the arguments; every
// launcher returns the hipError_t of its launches.
#pragma once

#include "model_ops.hpp"

namespace qp {

// ---- norms around a block (norm.hip)
constexpr int64_t kNormMaxWidth = 16384, kNormMaxRows = int64_t(1) << 22;   // (rows of 512 threads: 2^31)

struct NormArgs {
    const void* x;           // [M, D] of sdt: the stream
    int sdt, dt;             // its type; the block's (sdt, or sdt is fp32)
    int64_t M, D;
    const void* y;           // [M, D] of dt: the block's output, or null
    const void *post, *weight;   // [D] of dt each: the norm after the block, before the next; or null
    const void* gate;        // [gates, D] of dt, or null
    int64_t gates;           // a divisor of M; gate row r / (M / gates) for row r
    float factor, offset, eps;
    void* s;                 // [M, D] of sdt: the new stream (with y)
    void* a;                 // [M, D] of dt (with weight)
};
hipError_t launch_norm(const NormArgs& a, hipStream_t stream);

struct NormGradArgs {
    const void* s;           // [M, D] of sdt (with weight)
    const void* da;          // [M, D] of dt (with weight)
    const void* ds;          // [M, D] of sdt, or null (zeros)
    const void* y;           // [M, D] of dt, or null
    int sdt, dt;
    int64_t M, D;
    const void *post, *weight, *gate;
    int64_t gates;
    float factor, offset, eps;
    void* dx;                // [M, D] of sdt
    void* dy;                // [M, D] of dt (with y)
    void *dweight, *dpost, *dgate;   // of dt, with what they are the gradients of
    void* workspace;         // >= norm_grad_workspace_bytes, 16-byte aligned
};
size_t norm_grad_workspace_bytes(int64_t m, int64_t d, int64_t gates);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t stream);

// ---- cross entropy over a packed head (loss.hip)
struct LossArgs {
    const void* x;           // [M, K] of dt
    int dt;
    int64_t M, K, V;
    const int32_t* targets;  // [M]; outside [0, V): no target
    QWeight w;               // [V, K]
    int bits, gs;
    float *loss, *lse;       // [M]
    void* workspace;         // >= loss_workspace_bytes, 16-byte aligned
};
size_t loss_workspace_bytes(int64_t m, int64_t k, int64_t v, int bits, int gs, int dt);
hipError_t launch_loss(const LossArgs& a, hipStream_t stream);

struct LossGradArgs {
    const void* x;
    int dt;
    int64_t M, K, V;
    const int32_t* targets;
    QWeight w;
    int bits, gs;
    const float *lse, *dloss;    // [M]
    void* dx;                // [M, K] of dt, or null
    void *dscales, *dbiases; // [V, K/gs] of dt, or both null
    void* workspace;         // >= loss_grad_workspace_bytes, 16-byte aligned
};
size_t loss_grad_workspace_bytes(int64_t m, int64_t k, int64_t v, int bits, int gs, int dt);
hipError_t launch_loss_grad(const LossGradArgs& a, hipStream_t stream);

// The tile kernel of the loss (loss_tile.hpp): rows of x times a piece of the
// vocabulary, closed to statistics or (dz) to the logits' gradient.
constexpr int LOSS_BN = 256;   // columns of a tile, and of a part of the statistics
struct Stat;
struct LossTileArgs {
    const void* xp;          // [M, xn] of 16 bits: the groups' sums of x, then x (fp32: x in three parts)
    const void* xs;          // [M, gp]: the groups' sums (fp32 x); [M] fp32: what takes the rows' factor
                             // out of the biases' products again (fp16 x)
    const uint32_t* wq;      // [N, K*bits/32]
    const void* st;          // [K/gs, np]: the scales, transposed (prep_w)
    const void* bp;          // [N, gp]: the biases
    int M, N, K, gs;
    int xn, gp, np;          // the groups filled up to 32 (fp32: 8), N to LOSS_BN; xn: 2 gp + K filled
                             // up to 64 (fp32: three times that K)
    int tiles_m, tiles, per_xcd;
    const int32_t* targets;  // [M]
    int64_t vocab, v0;       // the whole vocabulary; the piece's first token
    Stat* stats;             // [parts][stat_rows], from part part0 on
    float* picked;           // [M]: the targets' logits
    int64_t stat_rows;
    int part0;
    void* dz;                // [M, dz_stride], or null: statistics
    int64_t dz_stride;
    const float *lse, *dloss, *scale;   // [M], [M], and scale[0] a factor of dloss
};
// What is laid out before a piece's tiles, where they read it.
struct LossPrepArgs {
    const void* x;           // [M, K], or null: it has been
    const void *scales, *biases;
    void* bp;                // null: the biases are read as they lie
    float* factor;           // dz's factor and its inverse, or null
};
// Logits of up to 16 rows of 16-bit x (16-byte aligned) as fp32 y (loss_rows.hip).
#define QP_LOSS_DECL(B)                                                                                          \
    hipError_t launch_loss_prep_b##B(int dt, const LossTileArgs& a, const LossPrepArgs& p, hipStream_t stream); \
    hipError_t launch_loss_tile_b##B(int dt, LossTileArgs a, hipStream_t stream);                               \
    hipError_t launch_loss_rows_b##B(const GemvArgs& a, hipStream_t stream);
QP_LOSS_DECL(2)
QP_LOSS_DECL(3)
QP_LOSS_DECL(4)
QP_LOSS_DECL(6)
QP_LOSS_DECL(8)
#undef QP_LOSS_DECL

} // namespace qp
