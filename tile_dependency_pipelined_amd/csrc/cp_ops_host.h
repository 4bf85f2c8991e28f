// cp_ops_host.h -- launchers the host side of the operators calls.  Internal.
#pragma once
#include <hip/hip_runtime.h>

#include "cp_ops_device.h"

namespace cpo {

// Which index of the operands is contiguous (see cp_ops_gemm.h).
enum Layout : int { kNN = 0, kNT = 1, kTN = 2 };  // A and B: KC/outer, KC/KC, outer/outer

constexpr int kGemvRows = 2;
constexpr int64_t kGemvColumnBytes = 64 << 20;  // weights stored [K][N] up to this size

// Tile configurations of the products; kGemv: no tiles, at most kGemvRows rows.
enum Config : int { kTile256, kTile128x256, kTile128, kTile64x128, kTile64, kTile16, kGemv, kConfigs };
struct ConfigShape {
    int bm, bn, threads;
};
constexpr ConfigShape kShapes[kConfigs] = {{256, 256, 512}, {128, 256, 512}, {128, 128, 256}, {64, 128, 256},
                                           {64, 64, 256},   {16, 128, 256},  {kGemvRows, 1, 0}};

// Blocks of `threads` threads that a dimension of a grid can hold.  It is counted
// in threads, in 32 bits: a launch of more wraps around without an error.
constexpr int64_t max_blocks(int threads) { return 0xFFFFFFFFll / threads; }
// A grid of at least `blocks` (> 0) blocks, over two dimensions if one does not
// hold them; kernels launched so take block_id() and leave alone what is past `blocks`.
inline dim3 grid_of(int64_t blocks, int threads) {
    const int64_t rows = (blocks + max_blocks(threads) - 1) / max_blocks(threads);
    return dim3((unsigned)((blocks + rows - 1) / rows), (unsigned)rows);
}

// Copies of up to three matrices (or stacks of `count`) with rows of whole
// 16-byte units, zero past the end.
struct PackArgs {
    struct One {
        const char *src;
        char *dst;
        int64_t ld, ldd;           // elements
        int64_t stride, stride_d;  // from one of `count` matrices to the next
        int32_t rows, cols, count;
    } one[3];
    int32_t n;
};
hipError_t launch_pack(int dtype, const PackArgs &a, hipStream_t s);

hipError_t launch_product_bf16(Layout l, Config c, bool direct, const GemmArgs &g, int grid, hipStream_t s);
hipError_t launch_product_f32(Layout l, Config c, bool direct, const GemmArgs &g, int grid, hipStream_t s);

// dX (x, nx workgroups), dW (w, nw) and bias sums (d, nd) of a layer with tiles of
// one configuration; x's A and w's operands as in Layout, lx is kNN or kNT.
hipError_t launch_gradients_bf16(Layout lx, Config c, const GemmArgs &x, int nx, const GemmArgs &w, int nw, const GradArgs &d,
                                 int nd, hipStream_t s);
hipError_t launch_gradients_f32(Layout lx, Config c, const GemmArgs &x, int nx, const GemmArgs &w, int nw, const GradArgs &d,
                                int nd, hipStream_t s);

// Products with at most kGemvRows rows; the weight's rows run along the
// contraction (w_rows) or along the output.
hipError_t launch_gemv(int dtype, bool w_rows, const GemmArgs &g, hipStream_t s);

// sums the partials of a split product and runs its epilogue
hipError_t launch_join(int dtype, const GemmArgs &g, hipStream_t s);

// dZ and the partial column sums, in the same launch the copies; then the bias
// gradient from those.
inline int grad_join_blocks(const GradArgs &a) { return a.groups * ((a.N + 63) / 64); }
hipError_t launch_grad(int dtype, const GradArgs &a, const PackArgs &packs, hipStream_t s);
hipError_t launch_grad_join(int dtype, const GradArgs &a, hipStream_t s);

struct NormArgs {
    const char *x, *dy, *w, *b;
    char *y, *dw, *db;     // y: output, or dX in the backward pass
    float *mean, *rstd;
    float *ws;             // backward: [2][blocks][N] partial sums
    int64_t ldx, ldd, ldy;
    int32_t M, N, blocks, vec;
    float eps;
};
hipError_t launch_norm(int dtype, const NormArgs &a, hipStream_t s);
constexpr int64_t kNormOneBlock = 8192;  // elements that one block takes on its own (such rows fit its registers)
int norm_backward_blocks(int64_t M, int64_t N);  // partial sums: one per block
hipError_t launch_norm_backward(int dtype, const NormArgs &a, hipStream_t s);

}  // namespace cpo
