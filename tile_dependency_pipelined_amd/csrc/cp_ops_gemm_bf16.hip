// cp_ops_gemm_bf16.hip -- the bf16 products of cp_ops_gemm.h.
#include "cp_ops_gemm.h"

namespace cpo {

hipError_t launch_product_bf16(Layout l, Config c, bool direct, const GemmArgs &g, int grid, hipStream_t s) {
    using T = __bf16;
    if (l == kNN) return launch_layout<T, true, false>(c, direct, g, grid, s);
    if (l == kNT) return launch_layout<T, true, true>(c, direct, g, grid, s);
    return launch_layout<T, false, false>(c, direct, g, grid, s);
}

}  // namespace cpo
