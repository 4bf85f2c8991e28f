// cp_ops_gemm_f32.hip -- the fp32 products of cp_ops_gemm.h.
#include "cp_ops_gemm.h"
#include "cp_ops_host.h"

namespace cpo {

namespace {

template <class P>
hipError_t launch(const GemmArgs &g, int grid, hipStream_t s) {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(product_kernel<P>), dim3(grid), dim3(P::NT), 0, s, g);
    return hipGetLastError();
}

template <bool AKC, bool BKC>
hipError_t launch_layout(Config c, bool direct, const GemmArgs &g, int grid, hipStream_t s) {
    using T = float;
    if constexpr (AKC)
        if (c == kTile16)
            return direct ? launch<Product<T, 16, 128, 1, 4, 4, AKC, BKC, true>>(g, grid, s)
                          : launch<Product<T, 16, 128, 1, 4, 2, AKC, BKC, false>>(g, grid, s);
    if (!direct) return hipErrorInvalidValue;  // the host packs their operands
    if (c == kTile128) return launch<Product<T, 128, 128, 2, 2, 2, AKC, BKC, true>>(g, grid, s);
    if (c == kTile64x128) return launch<Product<T, 64, 128, 2, 2, 3, AKC, BKC, true>>(g, grid, s);
    if (c == kTile64) return launch<Product<T, 64, 64, 2, 2, 4, AKC, BKC, true>>(g, grid, s);
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_product_f32(Layout l, Config c, bool direct, const GemmArgs &g, int grid, hipStream_t s) {
    if (l == kNN) return launch_layout<true, false>(c, direct, g, grid, s);
    if (l == kNT) return launch_layout<true, true>(c, direct, g, grid, s);
    return launch_layout<false, false>(c, direct, g, grid, s);
}

}  // namespace cpo
