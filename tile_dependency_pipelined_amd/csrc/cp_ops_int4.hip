// cp_ops_int4.hip -- linear layers with 4-bit weights, w_kn = s_gn (q_kn - z_gn),
// for a few rows at a time (decoding): bound by reading the codes, a quarter of
// the bf16 weight.
//
// The matrix cores multiply x with the codes as bf16, exactly: a code's four bits
// in bits 3 .. 6 of a bf16 pattern 0x4180 make it 16 + q, two codes with one shift
// and one and-or.  A product with ones gives sum x, and per group
//     s_n (sum x (16 + q) - (16 + z_n) sum x)
// joins the fp32 accumulator.  fp32 rows run as three bf16 parts that add up to
// them exactly.  The codes lie in memory as the instructions take them (Int4Layout),
// so a wave reads its operand with whole 16-byte loads and no LDS.
#include "cp_ops_experts.h"

namespace cpo {

namespace {

__device__ __forceinline__ bf16x8_t codes_bf16(uint32_t w) {
    union {
        uint32_t u[4];
        bf16x8_t v;
    } r;
    r.u[0] = ((w << 3) & 0x00780078u) | 0x41804180u;
    r.u[1] = ((w >> 1) & 0x00780078u) | 0x41804180u;
    r.u[2] = ((w >> 5) & 0x00780078u) | 0x41804180u;
    r.u[3] = ((w >> 9) & 0x00780078u) | 0x41804180u;
    return r.v;
}
__device__ __forceinline__ bf16x8_t ones_bf16() {
    union {
        uint32_t u[4];
        bf16x8_t v;
    } r;
    r.u[0] = r.u[1] = r.u[2] = r.u[3] = 0x3F803F80u;
    return r.v;
}

// Eight elements of x as XP bf16 parts.
template <class T>
struct Row8 {
    static constexpr int kUnits = 8 / kUnit<T>;
    uint4 u[kUnits];
    __device__ __forceinline__ void load(const char *p, int left) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) u[i] = load_partial<T>(p + i * 16, left - i * kUnit<T>);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
};
__device__ __forceinline__ void parts(const Row8<__bf16> &r, bf16x8_t (&p)[1]) { __builtin_memcpy(&p[0], &r.u[0], 16); }
__device__ __forceinline__ void parts(const Row8<float> &r, bf16x8_t (&p)[3]) {
    float x[8];
    __builtin_memcpy(x, r.u, 32);
    union {
        uint16_t h[8];
        bf16x8_t v;
    } a[3];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 3; ++j) {  // the leading 8 bits of what is left: each difference is exact
            const uint32_t top = __builtin_bit_cast(uint32_t, x[i]) & 0xFFFF0000u;
            a[j].h[i] = (uint16_t)(top >> 16);
            x[i] -= __builtin_bit_cast(float, top);
        }
#pragma unroll
    for (int j = 0; j < 3; ++j) p[j] = a[j].v;
}

// MT x 16 rows and NT x 16 columns to a block; its W waves take every W-th tile of
// the contraction and are added up in LDS.  SG: matrix instructions to a group.
template <class T, int MT, int NT, int W, int SG>
__global__ __launch_bounds__(W * 64) void int4_kernel(Int4Args g) {
    constexpr int XP = sizeof(T) == 2 ? 1 : 3, NG = 4 / SG, U = 2;
    __shared__ float red[W][MT * NT * 4][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n16 = lane & 15, quad = lane >> 4;
    const int b = xcd_remap(blockIdx.x, gridDim.x), rt = b % g.ntm, ct = b / g.ntm;
    int row0 = rt * 16 * MT, row_end = g.M, e = 0;
    if (g.experts) {
        GroupScan s;
        if (rt >= count_tiles(g.off, g.experts, g.M, 16 * MT, s)) return;
        const RowTile t = find_tile(g.off, g.experts, g.M, 16 * MT, rt, s);
        e = t.expert;
        row0 = t.row0 + (rt - t.before) * 16 * MT;
        row_end = t.end;
    }
    const bool none = g.experts && e >= g.experts;  // rows without an expert: zeros
    const int64_t es = none ? 0 : e;
    const char *codes = g.codes + es * g.sc;
    const T *scales = reinterpret_cast<const T *>(g.scales + es * g.ss);
    const uint8_t *zeros = g.zeros ? g.zeros + es * g.sz : nullptr;

    f32x4_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    if (!none)
        for (int kb0 = wave; kb0 < g.kblocks; kb0 += U * W) {
            uint4 wv[U][NT];
            T sv[U][NT][NG];
            uint8_t zv[U][NT][NG];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kb = kb0 + u * W < g.kblocks ? kb0 + u * W : kb0;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int tile = ct * NT + n < g.ntiles ? ct * NT + n : g.ntiles - 1;
                    wv[u][n] = *reinterpret_cast<const uint4 *>(codes + ((int64_t)tile * g.kblocks + kb) * kInt4TileBytes +
                                                                lane * 16);
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        int gr = SG == 4 ? kb * kInt4Depth / g.group : kb * NG + i;
                        gr = gr < g.ngroups ? gr : g.ngroups - 1;
                        const int64_t at = ((int64_t)tile * g.ngroups + gr) * kInt4Columns + n16;
                        sv[u][n][i] = scales[at];
                        zv[u][n][i] = zeros ? zeros[at] : (uint8_t)8;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kb = kb0 + u * W;
                if (kb >= g.kblocks) break;  // uniform
                Row8<T> xr[4][MT];
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const int row = row0 + m * 16 + n16, k = kb * kInt4Depth + s * 32 + quad * 8;
                        if (row < row_end && k < g.K) xr[s][m].load(g.x + ((int64_t)row * g.ldx + k) * (int64_t)sizeof(T), g.K - k);
                        else xr[s][m].zero();
                    }
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    f32x4_t p[MT][NT], xs[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        xs[m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int n = 0; n < NT; ++n) p[m][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                    }
#pragma unroll
                    for (int s = i * SG; s < i * SG + SG; ++s) {
                        bf16x8_t w[NT];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            w[n] = codes_bf16(s == 0 ? wv[u][n].x : s == 1 ? wv[u][n].y : s == 2 ? wv[u][n].z : wv[u][n].w);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            bf16x8_t x[XP];
                            parts(xr[s][m], x);
#pragma unroll
                            for (int j = 0; j < XP; ++j) {
                                xs[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j], ones_bf16(), xs[m], 0, 0, 0);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    p[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j], w[n], p[m][n], 0, 0, 0);
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float sc = to_f32(sv[u][n][i]), zp = -(float)(16 + (int)zv[u][n][i]);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                acc[m][n][r] = fmaf(sc, fmaf(zp, xs[m][r], p[m][n][r]), acc[m][n][r]);
                    }
                }
            }
        }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wave][(m * NT + n) * 4 + r][lane] = acc[m][n][r];
    __syncthreads();
    for (int o = tid; o < MT * NT * 256; o += W * 64) {
        const int c = o % (NT * 16), row = o / (NT * 16), m = row >> 4, q = (row >> 2) & 3, r = row & 3, n = c >> 4;
        const int gr = row0 + row, col = ct * NT * 16 + c;
        if (gr >= row_end || col >= g.N) continue;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += red[w][(m * NT + n) * 4 + r][q * 16 + (c & 15)];
        if (none) {
            v = 0.0f;
        } else {
            if (g.bias) v += to_f32(reinterpret_cast<const T *>(g.bias)[es * g.N + col]);
            v = act_apply(v, g.act);
        }
        if (g.res) v += to_f32(reinterpret_cast<const T *>(g.res)[(int64_t)gr * g.ldr + col]);
        reinterpret_cast<T *>(g.y)[(int64_t)gr * g.ldy + col] = from_f32<T>(v);
    }
}

// ------------------------------------------------- packing and quantisation

// A thread per word of the codes: eight k of a column.
__global__ __launch_bounds__(256) void int4_pack_codes_kernel(Int4PackArgs a) {
    const int64_t words = (int64_t)a.ntiles * a.kblocks * (kInt4TileBytes / 4), all = words * a.E;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        // neighbours in a wave take neighbouring columns
        const int64_t e = i / words, w = i % words;
        const int64_t cols = (int64_t)a.ntiles * kInt4Columns;
        const int64_t n = w % cols, k8 = w / cols, k0 = k8 * 8;
        uint32_t v = 0;
        if (n < a.N)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k0 + j < a.K)
                    v |= (uint32_t)(a.q[(e * a.K + k0 + j) * a.N + n] & 15) << (4 * (j / 2) + 16 * (j % 2));
        const int64_t tile = n / kInt4Columns, kb = k0 / kInt4Depth;
        const int lane = (int)(k8 % 4) * 16 + (int)(n % kInt4Columns), s = (int)(k0 % kInt4Depth) / 32;
        reinterpret_cast<uint32_t *>(a.codes)[e * words + (tile * a.kblocks + kb) * (kInt4TileBytes / 4) + lane * 4 + s] = v;
    }
}

__global__ __launch_bounds__(256) void int4_pack_scales_kernel(Int4PackArgs a) {
    const int64_t per = (int64_t)a.ntiles * a.ngroups * kInt4Columns, all = per * a.E;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t e = i / per, w = i % per, tile = w / ((int64_t)a.ngroups * kInt4Columns);
        const int64_t g = w / kInt4Columns % a.ngroups, n = tile * kInt4Columns + w % kInt4Columns;
        const int64_t from = (e * a.ngroups + g) * a.N + n;
        const bool in = n < a.N;
        if (a.scale_bytes == 2) reinterpret_cast<uint16_t *>(a.pscales)[i] = in ? reinterpret_cast<const uint16_t *>(a.scales)[from] : 0;
        else reinterpret_cast<uint32_t *>(a.pscales)[i] = in ? reinterpret_cast<const uint32_t *>(a.scales)[from] : 0;
        if (a.zeros) a.pzeros[i] = in ? a.zeros[from] & 15 : 0;
    }
}

// A thread per group and column.  With zero points the range is that of the values
// and 0, in 15 steps; without, 7 steps to either side.  The scale is rounded to its
// type first, codes and zero points belong to the rounded one.
template <class T>
__global__ __launch_bounds__(256) void int4_quantize_kernel(Int4QuantArgs a) {
    const int64_t per = (int64_t)a.ngroups * a.N, all = per * a.E;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t e = i / per, g = i % per / a.N, n = i % a.N;
        const int64_t k0 = g * a.group, k1 = k0 + a.group < a.K ? k0 + a.group : a.K;
        const T *w = reinterpret_cast<const T *>(a.w) + e * a.se + n * a.sn;
        float lo = 0.0f, hi = 0.0f;
        for (int64_t k = k0; k < k1; ++k) {
            const float v = to_f32(w[k * a.sk]);
            lo = fminf(lo, v);
            hi = fmaxf(hi, v);
        }
        // (halves first: the range of finite values may not be one)
        const T st = from_f32<T>(a.zeros ? 2.0f * ((0.5f * hi - 0.5f * lo) / 15.0f) : fmaxf(-lo, hi) / 7.0f);
        const float s = to_f32(st), z = a.zeros ? (s > 0.0f ? fminf(rintf(-lo / s), 15.0f) : 0.0f) : 8.0f;
        reinterpret_cast<T *>(a.scales)[i] = st;
        if (a.zeros) a.zeros[i] = (uint8_t)z;
        for (int64_t k = k0; k < k1; ++k) {
            const float q = s > 0.0f ? rintf(to_f32(w[k * a.sk]) / s) + z : z;
            a.q[(e * a.K + k) * a.N + n] = (uint8_t)fminf(fmaxf(q, 0.0f), 15.0f);
        }
    }
}

template <class T, int MT, int NT, int W>
hipError_t by_group(const Int4Args &a, unsigned blocks, hipStream_t s) {
    if (a.group == 32) hipLaunchKernelGGL(HIP_KERNEL_NAME(int4_kernel<T, MT, NT, W, 1>), dim3(blocks), dim3(W * 64), 0, s, a);
    else if (a.group == 64) hipLaunchKernelGGL(HIP_KERNEL_NAME(int4_kernel<T, MT, NT, W, 2>), dim3(blocks), dim3(W * 64), 0, s, a);
    else hipLaunchKernelGGL(HIP_KERNEL_NAME(int4_kernel<T, MT, NT, W, 4>), dim3(blocks), dim3(W * 64), 0, s, a);
    return hipGetLastError();
}

template <class T>
hipError_t int4(Int4Args a, hipStream_t s) {
    const Int4Tiles t = int4_tiles(a.experts, a.M, a.ntiles);
    a.ntm = t.ntm;
    a.ntn = t.ntn;
    const unsigned blocks = (unsigned)((int64_t)t.ntm * t.ntn);
    if (t.mt == 1 && t.nt == 1) return by_group<T, 1, 1, 8>(a, blocks, s);
    if (t.mt == 1) return by_group<T, 1, 2, 8>(a, blocks, s);
    return by_group<T, 4, 4, 4>(a, blocks, s);
}

}  // namespace

hipError_t launch_int4(int dtype, const Int4Args &a, hipStream_t s) {
    return dtype == CP_BF16 ? int4<__bf16>(a, s) : int4<float>(a, s);
}

hipError_t launch_int4_pack(const Int4PackArgs &a, hipStream_t s) {
    auto blocks = [](int64_t n) { return dim3((unsigned)((n + 255) / 256 < 16384 ? (n + 255) / 256 : 16384)); };
    const int64_t words = (int64_t)a.ntiles * a.kblocks * (kInt4TileBytes / 4) * a.E;
    const int64_t scales = (int64_t)a.ntiles * a.ngroups * kInt4Columns * a.E;
    if (words) hipLaunchKernelGGL(int4_pack_codes_kernel, blocks(words), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !scales) return e;
    hipLaunchKernelGGL(int4_pack_scales_kernel, blocks(scales), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_int4_quantize(int dtype, const Int4QuantArgs &a, hipStream_t s) {
    const int64_t n = (int64_t)a.ngroups * a.N * a.E;
    const dim3 blocks((unsigned)((n + 255) / 256 < 16384 ? (n + 255) / 256 : 16384));
    if (dtype == CP_BF16) hipLaunchKernelGGL(HIP_KERNEL_NAME(int4_quantize_kernel<__bf16>), blocks, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(HIP_KERNEL_NAME(int4_quantize_kernel<float>), blocks, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace cpo
