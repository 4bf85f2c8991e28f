// Host model of the feed-forward operators' launches: cp_ops.cpp with launchers
// that print what they are asked for instead of launching.  Reads one call per
// line,
//   op dtype M K N E w_trans act parts aligned
// (op: forward | backward; dtype as in cp_chain.h; E = 0: dense; parts: bits 1
// dX or the residual, 2 dW, 4 db or the bias; aligned: 0 puts every matrix off 16
// bytes) and prints the launches of each in one line, ended by the status.  Or,
// with addresses of the caller's choice (0: NULL),
//   linear dtype M K N E w_trans X ldx W ldw stride_w bias offsets R ldr Y ldy pre ldp
//   norm dtype M N X ldx w b Y ldy
// Pointers are never followed on the host, so they are only plausible numbers.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../tile_dependency_pipelined_amd/csrc/cp_ops.cpp"

namespace {

const char *kNames[kConfigs] = {"256x256", "128x256", "128x128", "64x128", "64x64", "16x128", "gemv"};

int threads_of(Config c) { return c == kTile256 || c == kTile128x256 ? 512 : 256; }

hipError_t product(Layout l, Config c, bool direct, const GemmArgs &g, int grid) {
    printf("product:%s:layout=%d:split=%d:direct=%d:threads=%lld ", kNames[c], (int)l, g.nsplit, (int)direct,
           (long long)grid * threads_of(c));
    return hipSuccess;
}
hipError_t gradients(Config c, int nx, int nw, int nd) {
    printf("gradients:%s:nx=%d:nw=%d:nd=%d:threads=%lld ", kNames[c], nx, nw, nd,
           ((long long)nx + nw + nd) * threads_of(c));
    return hipSuccess;
}
hipError_t named(const char *what) {
    printf("%s ", what);
    return hipSuccess;
}

}  // namespace

namespace cpo {

hipError_t launch_pack(int, const PackArgs &, hipStream_t) { return named("pack"); }
hipError_t launch_product_bf16(Layout l, Config c, bool d, const GemmArgs &g, int n, hipStream_t) { return product(l, c, d, g, n); }
hipError_t launch_product_f32(Layout l, Config c, bool d, const GemmArgs &g, int n, hipStream_t) { return product(l, c, d, g, n); }
hipError_t launch_gradients_bf16(Layout, Config c, const GemmArgs &, int nx, const GemmArgs &, int nw, const GradArgs &, int nd,
                                 hipStream_t) {
    return gradients(c, nx, nw, nd);
}
hipError_t launch_gradients_f32(Layout, Config c, const GemmArgs &, int nx, const GemmArgs &, int nw, const GradArgs &, int nd,
                                hipStream_t) {
    return gradients(c, nx, nw, nd);
}
hipError_t launch_gemv(int, bool, const GemmArgs &, hipStream_t) { return named("gemv"); }
hipError_t launch_join(int, const GemmArgs &, hipStream_t) { return named("join"); }
hipError_t launch_grad(int, const GradArgs &, const PackArgs &, hipStream_t) { return named("grad"); }
hipError_t launch_grad_join(int, const GradArgs &, hipStream_t) { return named("grad_join"); }
hipError_t launch_norm(int, const NormArgs &, hipStream_t) { return named("norm"); }
int norm_backward_blocks(int64_t, int64_t) { return 1; }
hipError_t launch_norm_backward(int, const NormArgs &, hipStream_t) { return named("norm_backward"); }

}  // namespace cpo

int main() {
    char op[32];
    int dtype, E, wt, act, parts, aligned;
    long long M, K, N;
    while (scanf("%31s", op) == 1) {
        if (op[0] == 'l' || op[0] == 'n') {
            std::vector<long long> v(op[0] == 'l' ? 19 : 9);
            for (long long &x : v)
                if (scanf("%lld", &x) != 1) return 2;
            auto p = [&](int i) { return (void *)(uintptr_t)v[i]; };
            void *ws = (void *)(uintptr_t(1) << 54);
            const int64_t most = int64_t(1) << 53;
            int rc;
            if (op[0] == 'n')
                rc = cp_layer_norm((int)v[0], v[1], v[2], p(3), v[4], p(5), p(6), 1e-5f, p(7), v[8], nullptr, nullptr, nullptr);
            else if (v[4])
                rc = cp_grouped_linear((int)v[0], v[1], v[2], v[3], (int)v[4], p(6), v[7], p(8), v[9], v[10], (int)v[5],
                                       (const int32_t *)p(12), p(11), 0, p(15), v[16], p(17), v[18], ws, most, nullptr);
            else
                rc = cp_linear((int)v[0], v[1], v[2], v[3], p(6), v[7], p(8), v[9], (int)v[5], p(11), p(13), v[14], 0, p(15),
                               v[16], p(17), v[18], ws, most, nullptr);
            printf("status=%d %s\n", rc, cp_ops_last_error());
            continue;
        }
        if (scanf("%d %lld %lld %lld %d %d %d %d %d", &dtype, &M, &K, &N, &E, &wt, &act, &parts, &aligned) != 9) return 2;
        // each matrix in a space of its own
        const uintptr_t step = uintptr_t(1) << 54, off = aligned ? 0 : (dtype == CP_BF16 ? 2 : 4);
        auto at = [&](int i) { return (void *)(step * i + off); };
        const int64_t ldw = wt ? K : N, most = int64_t(1) << 53;
        int rc;
        if (op[0] == 'f' && E)
            rc = cp_grouped_linear(dtype, M, K, N, E, at(1), K, at(2), ldw, K * N, wt, (const int32_t *)(step * 3),
                                   parts & 4 ? at(4) : nullptr, act, at(5), N, nullptr, 0, (void *)(step * 6), most, nullptr);
        else if (op[0] == 'f')
            rc = cp_linear(dtype, M, K, N, at(1), K, at(2), ldw, wt, parts & 4 ? at(4) : nullptr, parts & 1 ? at(7) : nullptr, N,
                           act, at(5), N, nullptr, 0, (void *)(step * 6), most, nullptr);
        else if (E)
            rc = cp_grouped_linear_backward(dtype, M, K, N, E, at(1), N, at(2), K, at(3), ldw, K * N, wt,
                                            (const int32_t *)(step * 4), at(5), N, act, parts & 1 ? at(7) : nullptr, K,
                                            parts & 2 ? at(8) : nullptr, ldw, K * N, parts & 4 ? at(9) : nullptr,
                                            (void *)(step * 6), most, nullptr);
        else
            rc = cp_linear_backward(dtype, M, K, N, at(1), N, at(2), K, at(3), ldw, wt, at(5), N, act,
                                    parts & 1 ? at(7) : nullptr, K, parts & 2 ? at(8) : nullptr, ldw,
                                    parts & 4 ? at(9) : nullptr, (void *)(step * 6), most, nullptr);
        printf("status=%d\n", rc);
    }
    return 0;
}
