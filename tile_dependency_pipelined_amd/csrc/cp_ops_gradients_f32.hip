// cp_ops_gradients_f32.hip -- a linear layer's fp32 gradients in one launch
// (gradients_kernel of cp_ops_gemm.h).
#include "cp_ops_gemm.h"

namespace cpo {

hipError_t launch_gradients_f32(Layout lx, Config c, const GemmArgs &x, int nx, const GemmArgs &w, int nw, const GradArgs &d,
                              int nd, hipStream_t s) {
    return lx == kNN ? launch_gradients_layout<float, false>(c, x, nx, w, nw, d, nd, s)
                     : launch_gradients_layout<float, true>(c, x, nx, w, nw, d, nd, s);
}

}  // namespace cpo
