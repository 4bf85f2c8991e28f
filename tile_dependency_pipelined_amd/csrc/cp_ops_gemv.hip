// cp_ops_gemv.hip -- products of one or two rows (a decode step), bound by
// reading the weight once: no LDS tiles and no matrix instructions, every lane
// loads 16 bytes of the weight at a time, many loads in flight, and multiplies
// them with the rows in fp32.  One launch and no partial results in memory,
// where the 16-row tiles split the contraction and take a second launch to add
// it up: 1 x 4096 x 4096 (33.6 MB) 11.3 us, 4 of them the launch.
#include "cp_ops_host.h"

namespace cpo {

namespace {

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 15, 15, true));
}
// Sum over each 16 lanes, valid in the last of them.
__device__ __forceinline__ float sum16(float v) {
    v = dpp_add<0x111>(v);  // row_shr 1, 2, 4, 8
    v = dpp_add<0x112>(v);
    v = dpp_add<0x114>(v);
    return dpp_add<0x118>(v);
}

template <class T>
__device__ __forceinline__ void unpack(uint4 u, float (&v)[kUnit<T>]) {
    union {
        uint4 u;
        T e[kUnit<T>];
    } x;
    x.u = u;
#pragma unroll
    for (int i = 0; i < kUnit<T>; ++i) v[i] = to_f32(x.e[i]);
}

template <class T>
__device__ __forceinline__ void finish_one(const GemmArgs &g, int row, int col, float sum) {
    Raw<T, 1> b, r;
    float v[1][1] = {{sum}};
    if (g.bias) b.load(g.bias + (int64_t)col * sizeof(T));
    if (g.res) r.load(g.res + ((int64_t)row * g.ldr + col) * sizeof(T));
    finish<T, 1, 1>(g, g.C, row, 0, col, v, g.bias ? &b : nullptr, g.res ? &r : nullptr, false, true, true, 0);
}

// Weight stored [K][N].  A block takes L lanes x 16 bytes of columns and all of
// K: its 16 waves take 64 / L rows each in turn, so nothing has to be summed
// across blocks.  The columns per block are few enough for the blocks to fill
// the device; blocks next to each other share cache lines and an XCD.  Reading
// 32 or 64 bytes of a row at a time costs bandwidth, so this pays while the
// launch saved counts: bf16 1 x 4096 x 4096 11.4 us (16-row tiles 15.5), 1 x
// 8192 x 8192 33.9 (31.5), 1 x 28672 x 8192 128 (90).
template <class T, int MR, int L>
__global__ __launch_bounds__(1024) void gemv_columns_kernel(GemmArgs g) {
    constexpr int CE = kUnit<T>, W = 16, RPI = 64 / L, U = MR == 1 ? 8 : 4, O = MR * L * CE;
    __shared__ float part[W * 4][O + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane % L, r = wave * RPI + lane / L;
    const int tile = xcd_remap(blockIdx.x, gridDim.x), col = (tile * L + c) * CE;
    const bool whole = (tile + 1) * L * CE <= g.N;  // uniform
    const char *w = g.B + (int64_t)col * sizeof(T);
    const T *x = reinterpret_cast<const T *>(g.A);
    float acc[MR][CE];
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int i = 0; i < CE; ++i) acc[m][i] = 0.0f;
    for (int k0 = r; k0 - r < g.K; k0 += U * W * RPI) {
        uint4 wv[U];
        T xv[U][MR];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            int k = k0 + u * W * RPI;
            k = k < g.K ? k : g.K - 1;  // in range; not used beyond K
            const char *p = w + (int64_t)k * g.ldb * sizeof(T);
            if (whole) __builtin_memcpy(&wv[u], p, 16);
            else wv[u] = load_partial<T>(p, g.N - col);
#pragma unroll
            for (int m = 0; m < MR; ++m) xv[u][m] = x[(int64_t)(m < g.M ? m : g.M - 1) * g.lda + k];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = k0 + u * W * RPI < g.K;
            float f[CE];
            unpack<T>(wv[u], f);
#pragma unroll
            for (int i = 0; i < CE; ++i) f[i] = in ? f[i] : 0.0f;
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                const float xm = in ? to_f32(xv[u][m]) : 0.0f;
#pragma unroll
                for (int i = 0; i < CE; ++i) acc[m][i] = fmaf(xm, f[i], acc[m][i]);
            }
        }
    }
    // rows of a wave: lanes of each 16 with the same columns first
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int i = 0; i < CE; ++i) {
            float v = acc[m][i];
            if constexpr (L == 2) v = dpp_add<0x112>(v);
            if constexpr (L <= 4) v = dpp_add<0x114>(v);
            v = dpp_add<0x118>(v);
            if ((lane & 15) >= 16 - L) part[wave * 4 + (lane >> 4)][m * L * CE + c * CE + i] = v;
        }
    __syncthreads();
    const int s = threadIdx.x & 15;
    for (int o = threadIdx.x >> 4; o < O; o += 64) {
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < W * 4 / 16; ++j) v += part[s + 16 * j][o];
        v = sum16(v);
        const int m = o / (L * CE), n = tile * L * CE + o % (L * CE);
        if (s == 15 && m < g.M && n < g.N) finish_one<T>(g, m, n, v);
    }
}

// Weight stored [N][K]: `per` waves (1 or 4) to an output column, 64 lanes x 16
// bytes along K.  bf16 1 x 4096 x 4096 9.4 us, 1 x 8192 x 8192 27.0 (5.0 TB/s);
// with four rows 45 us there, as the rows are read again for every column,
// where the 16-row tiles take 28.
template <class T, int MR>
__global__ __launch_bounds__(256) void gemv_rows_kernel(GemmArgs g, int per) {
    constexpr int CE = kUnit<T>, U = 4;
    __shared__ float part[4][MR];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int b = xcd_remap(blockIdx.x, gridDim.x), n = b * (4 / per) + wave / per, slice = wave % per;
    float acc[MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) acc[m] = 0.0f;
    if (n < g.N) {
        const char *w = g.B + (int64_t)n * g.ldb * sizeof(T);
        for (int k0 = slice * 64 * CE; k0 < g.K; k0 += U * per * 64 * CE) {
            uint4 wv[U], xv[U][MR];
            if (k0 + ((U - 1) * per + 1) * 64 * CE <= g.K) {  // uniform
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t k = k0 + u * per * 64 * CE + lane * CE;
                    __builtin_memcpy(&wv[u], w + k * sizeof(T), 16);
#pragma unroll
                    for (int m = 0; m < MR; ++m)
                        __builtin_memcpy(&xv[u][m], g.A + ((m < g.M ? m : g.M - 1) * g.lda + k) * sizeof(T), 16);
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t k = k0 + u * per * 64 * CE + lane * CE;
                    const int left = (int)(g.K - k);
                    wv[u] = load_partial<T>(w + k * sizeof(T), left);
#pragma unroll
                    for (int m = 0; m < MR; ++m)
                        xv[u][m] = load_partial<T>(g.A + ((m < g.M ? m : g.M - 1) * g.lda + k) * sizeof(T), left);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[CE], x[CE];
                unpack<T>(wv[u], f);
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    unpack<T>(xv[u][m], x);
#pragma unroll
                    for (int i = 0; i < CE; ++i) acc[m] = fmaf(x[i], f[i], acc[m]);
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        const float v = sum16(acc[m]);
        auto at = [&](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l)); };
        acc[m] = (at(15) + at(31)) + (at(47) + at(63));
    }
    if (per > 1) {
        if (lane == 0)
#pragma unroll
            for (int m = 0; m < MR; ++m) part[wave][m] = acc[m];
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int m = 0; m < MR; ++m) acc[m] = (part[0][m] + part[1][m]) + (part[2][m] + part[3][m]);
    }
#pragma unroll
    for (int m = 0; m < MR; ++m)
        if (lane == m && m < g.M && n < g.N) finish_one<T>(g, m, n, acc[m]);
}

template <class T, int MR>
hipError_t gemv(bool w_rows, const GemmArgs &g, hipStream_t s) {
    constexpr int CE = kUnit<T>;
    if (w_rows) {
        // a wave per column; four where that leaves the device idle
        const int per = g.N < 2048 ? 4 : 1, cols = 4 / per;
        hipLaunchKernelGGL(HIP_KERNEL_NAME(gemv_rows_kernel<T, MR>), dim3((unsigned)((g.N + cols - 1) / cols)), dim3(256), 0,
                           s, g, per);
        return hipGetLastError();
    }
    auto blocks = [&](int l) { return (unsigned)((g.N + l * CE - 1) / (l * CE)); };
    if (blocks(8) >= 256)
        hipLaunchKernelGGL(HIP_KERNEL_NAME(gemv_columns_kernel<T, MR, 8>), dim3(blocks(8)), dim3(1024), 0, s, g);
    else if (blocks(4) >= 256)
        hipLaunchKernelGGL(HIP_KERNEL_NAME(gemv_columns_kernel<T, MR, 4>), dim3(blocks(4)), dim3(1024), 0, s, g);
    else
        hipLaunchKernelGGL(HIP_KERNEL_NAME(gemv_columns_kernel<T, MR, 2>), dim3(blocks(2)), dim3(1024), 0, s, g);
    return hipGetLastError();
}

template <class T>
hipError_t gemv_rows(bool w_rows, const GemmArgs &g, hipStream_t s) {
    return g.M == 1 ? gemv<T, 1>(w_rows, g, s) : gemv<T, 2>(w_rows, g, s);
}

}  // namespace

hipError_t launch_gemv(int dtype, bool w_rows, const GemmArgs &g, hipStream_t s) {
    return dtype == CP_BF16 ? gemv_rows<__bf16>(w_rows, g, s) : gemv_rows<float>(w_rows, g, s);
}

}  // namespace cpo
