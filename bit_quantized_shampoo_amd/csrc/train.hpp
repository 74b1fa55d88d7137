// Host-side launchers of the training operators (declared in shampoo4_train.h).  Every
// launcher enqueues on `stream` and returns the launch status; shapes, leading dimensions
// and workspace sizes have been checked by the caller.
#pragma once

#include "common.hpp"
#include "shampoo4_train.h"

namespace s4 {

// A checkpoint's buffers (codes [R, P], scales [R / 32, P]); codes NULL: none.
struct Act8Ptr {
    int8_t* codes;
    uint8_t* scales;
};
constexpr int64_t act8_rows(int64_t rows) { return (rows + 31) / 32 * 32; }
constexpr int64_t act8_pitch(int64_t cols) { return (cols + 15) / 16 * 16; }

// A wave's widest tile: ACT8_COLS columns of one block of 32 rows (the narrow one has a
// quarter of them).
constexpr int ACT8_COLS = 128;
constexpr int64_t act8_tiles(int64_t rows, int64_t cols) {
    return (rows + 31) / 32 * ((cols + ACT8_COLS - 1) / ACT8_COLS);
}
// 64 threads a tile: below 2^32 in a launch.  Loading to fp32 always takes the narrow tiles.
constexpr int64_t ACT8_MAX_TILES = (int64_t(1) << 26) - 8;
constexpr int64_t ACT8_MAX_TILES_F32_LOAD = (int64_t(1) << 24) - 8;

hipError_t launch_act8_store(shampoo4_dtype dtype, int64_t rows, int64_t cols, const void* x, int64_t ldx,
                             Act8Ptr out, hipStream_t stream);
hipError_t launch_act8_load(shampoo4_dtype dtype, int64_t rows, int64_t cols, Act8Ptr in, void* x, int64_t ldx,
                            hipStream_t stream);

struct ActForward {
    const void* gate;
    const void* up;           // NULL: not gated
    void* h;
    int64_t ldgate, ldup, ldh;
    Act8Ptr gate8, up8, h8;
    int64_t rows, cols;
};
hipError_t launch_activation_forward(int kind, shampoo4_dtype dtype, const ActForward& a, hipStream_t stream);

struct ActBackward {
    const void* dh;
    void* dgate;
    void* dup;                // NULL: not gated
    int64_t lddh, lddgate, lddup;
    Act8Ptr gate8, up8;
    int64_t rows, cols;
};
hipError_t launch_activation_backward(int kind, shampoo4_dtype dtype, const ActBackward& a, hipStream_t stream);

// Weight gradient G[n, cols] = alpha dY^T X^ + beta G.
struct WGrad {
    const void* dy;
    const int8_t* codes;
    const uint8_t* scales;
    float* g;
    float* parts;             // partial sums of the row ranges (splits > 1)
    int64_t rows, n, cols, lddy, ldg;
    float alpha, beta;
};
size_t wgrad_workspace_bytes(int64_t rows, int64_t n, int64_t cols);
hipError_t launch_wgrad(shampoo4_dtype dtype, const WGrad& w, hipStream_t stream);

struct Embed {
    const void* table;        // or dout
    const void* ids;
    void* out;
    int64_t tokens, vocab, dim, ldtable, ldout;
    float scale;
    int id64;
};
hipError_t launch_embedding(shampoo4_dtype dtype, const Embed& e, hipStream_t stream);

struct EmbedGrad {
    const void* dout;
    const void* ids;
    float* g;
    int64_t tokens, vocab, dim, lddout, ldg;
    float scale;
    int id64, accumulate;
};
size_t embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim);
hipError_t launch_embedding_grad(shampoo4_dtype dtype, const EmbedGrad& e, void* workspace, hipStream_t stream);

// Policy loss and token log-probabilities (train = 0: logp alone).
struct Policy {
    const void* logits;
    const void* targets;
    const float* old_logp;
    const float* ref_logp;
    const float* adv;
    const float* weights;
    float* loss;
    float* logp;
    void* dlogits;
    int64_t rows, vocab, ldz, ldd;
    float clip_low, clip_high, kl, grad_scale;
    int id64, train;
};
size_t policy_workspace_bytes(shampoo4_dtype dtype, int64_t rows, int64_t vocab, bool train);
hipError_t launch_policy(shampoo4_dtype dtype, const Policy& p, void* workspace, hipStream_t stream);

}  // namespace s4
