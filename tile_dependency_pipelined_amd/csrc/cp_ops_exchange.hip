// cp_ops_exchange.hip -- rows to their experts and back: out[rows_tj] = x_t, out_t
// = sum_j g_tj y[rows_tj] + r_t, and the gradients of the second.  No arithmetic
// worth the name: each kernel reads every row once and writes every row once, in
// 16-byte units at any alignment, token by token, so that a token's row is read
// once for all of its experts and no inverse of `rows` is needed.
#include "cp_ops_experts.h"
#include "cp_ops_units.h"

namespace cpo {

namespace {

// How a launch goes over tokens and the units of their rows: `lanes` lanes (a
// power of two, at most 64) side by side on a token, a wave on 64 / lanes tokens
// at a time, U units of a lane at a time; a token's row is `segs` such pieces.
struct Pieces {
    int32_t units, lanes, shift, segs;
    int64_t items;  // waves' worth of work
};
inline Pieces pieces(int64_t T, int D, int unit, int per_lane) {
    Pieces p;
    p.units = (D + unit - 1) / unit;
    p.shift = 0;
    while (p.shift < 6 && (1 << p.shift) * per_lane < p.units) ++p.shift;
    p.lanes = 1 << p.shift;
    p.segs = (p.units + p.lanes * per_lane - 1) / (p.lanes * per_lane);
    const int64_t tokens = 64 >> p.shift;
    p.items = (T + tokens - 1) / tokens * p.segs;
    if (p.items < 1) p.items = 1;  // (no tokens: rows of zeros may still be due)
    return p;
}

// Rows of y that belong to no slot: from *end on.
__device__ __forceinline__ int64_t first_free(const ExchangeArgs &a) {
    const int64_t e = *a.end;
    return e < 0 ? 0 : (e > a.R ? a.R : e);
}

// The wave's share of the zero rows: the same pieces, item after item.
template <class T, int U>
__device__ __forceinline__ void zero_rows(const ExchangeArgs &a, const Pieces &p, int64_t item, int64_t items, char *base,
                                          int64_t ld) {
    const int lane = threadIdx.x & 63;
    const int64_t from = first_free(a), n = a.R - from, per = 64 >> p.shift;
    for (int64_t i = item; i / p.segs * per < n; i += items) {
        const int64_t r = from + i / p.segs * per + (lane >> p.shift);
        if (r >= a.R) continue;
        const int u0 = (int)(i % p.segs) * p.lanes * U + (lane & (p.lanes - 1));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = u0 + u * p.lanes;
            if (at < p.units)
                store_partial<T>(base + (r * ld + (int64_t)at * kUnit<T>) * (int64_t)sizeof(T), make_uint4(0, 0, 0, 0),
                                 a.D - at * kUnit<T>);
        }
    }
}

// Four units of a lane at a time keep enough in flight; the rows of one token are written
// from the same registers.  8192 x 2 x 4096 bf16: 42.5 us, 4.7 TB/s.
constexpr int kDispatchUnits = 4;
template <class T>
__global__ __launch_bounds__(256) void dispatch_kernel(ExchangeArgs a, Pieces p) {
    constexpr int U = kDispatchUnits, CE = kUnit<T>;
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)block_id() * 4 + (threadIdx.x >> 6);
    if (item >= p.items) return;
    const int64_t t = item / p.segs * (64 >> p.shift) + (lane >> p.shift);
    const int u0 = (int)(item % p.segs) * p.lanes * U + (lane & (p.lanes - 1));
    if (t < a.T) {
        uint4 v[U];
        const char *x = a.x + t * a.ldx * (int64_t)sizeof(T);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = u0 + u * p.lanes;
            if (at < p.units) v[u] = load_partial<T>(x + (int64_t)at * 16, a.D - at * CE);
        }
        for (int j = 0; j < a.k; ++j) {
            const int64_t r = a.rows[t * a.k + j];
            if (r < 0 || r >= a.R) continue;
            char *o = a.out + r * a.ldo * (int64_t)sizeof(T);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = u0 + u * p.lanes;
                if (at < p.units) store_partial<T>(o + (int64_t)at * 16, v[u], a.D - at * CE);
            }
        }
    }
    zero_rows<T, U>(a, p, item, p.items, a.out, a.ldo);
}

// Slots C at a time, their rows requested together: of two slots one step of two (8192 x 2
// x 4096 bf16, a quarter of the tokens padding: 45.7 us, 5.1 TB/s), of more, steps of
// four.
template <class T, int U, int C>
__global__ __launch_bounds__(256) void combine_kernel(ExchangeArgs a, Pieces p) {
    constexpr int CE = kUnit<T>;
    const int lane = threadIdx.x & 63;
    const int64_t item = (int64_t)block_id() * 4 + (threadIdx.x >> 6);
    if (item >= p.items) return;
    const int64_t t = item / p.segs * (64 >> p.shift) + (lane >> p.shift);
    if (t >= a.T) return;
    const int u0 = (int)(item % p.segs) * p.lanes * U + (lane & (p.lanes - 1));
    float acc[U][CE];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < CE; ++i) acc[u][i] = 0.0f;
    uint4 res[U];
    if (a.res)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = u0 + u * p.lanes;
            if (at < p.units) res[u] = load_partial<T>(a.res + (t * a.ldr + (int64_t)at * CE) * (int64_t)sizeof(T), a.D - at * CE);
        }
    for (int j0 = 0; j0 < a.k; j0 += C) {
        int64_t r[C];
        float g[C];
        uint4 v[C][U];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            r[c] = j0 + c < a.k ? a.rows[t * a.k + j0 + c] : -1;
            g[c] = a.gates && j0 + c < a.k ? a.gates[t * a.k + j0 + c] : 1.0f;
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (r[c] >= 0 && r[c] < a.R)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int at = u0 + u * p.lanes;
                    if (at < p.units)
                        v[c][u] = load_partial<T>(a.y + (r[c] * a.ldy + (int64_t)at * CE) * (int64_t)sizeof(T), a.D - at * CE);
                }
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (r[c] >= 0 && r[c] < a.R)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[CE];
                    unpack_unit<T>(v[c][u], f);
#pragma unroll
                    for (int i = 0; i < CE; ++i) acc[u][i] = fmaf(g[c], f[i], acc[u][i]);
                }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = u0 + u * p.lanes;
        if (at >= p.units) continue;
        if (a.res) {
            float f[CE];
            unpack_unit<T>(res[u], f);
#pragma unroll
            for (int i = 0; i < CE; ++i) acc[u][i] += f[i];
        }
        store_partial<T>(a.out + (t * a.ldo + (int64_t)at * CE) * (int64_t)sizeof(T), pack_unit<T>(acc[u]), a.D - at * CE);
    }
}

// Sum over the `lanes` (a power of two) lanes of a token; every lane gets it.
__device__ __forceinline__ float sum_lanes(float v, int lanes) {
    for (int d = 1; d < lanes; d *= 2) v += __shfl_xor(v, d);
    return v;
}

// A token's whole row to the same lanes, as its gates' gradients are sums over it:
// C slots at a time, one unit of each requested together.  With `W` > 1 the waves
// of a block share a token and add up in LDS.  One pass gives both gradients: dout is
// read once for all slots, y and dy go by once.  4099 x 4 x 2048 bf16: 33.6 us, 4.5 TB/s.
template <class T, int C, int W>
__global__ __launch_bounds__(256) void combine_backward_kernel(ExchangeArgs a, Pieces p) {
    constexpr int CE = kUnit<T>;
    __shared__ float part[W][C];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t item = W > 1 ? (int64_t)block_id() : (int64_t)block_id() * 4 + wave;
    const int64_t t = item * (64 >> p.shift) + (lane >> p.shift);
    const int u0 = (W > 1 ? wave * p.lanes : 0) + (lane & (p.lanes - 1)), step = W * p.lanes;
    const bool in = t < a.T;
    for (int j0 = 0; j0 < a.k; j0 += C) {
        int64_t r[C];
        float g[C], dot[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const bool slot = in && j0 + c < a.k;
            r[c] = slot ? a.rows[t * a.k + j0 + c] : -1;
            if (r[c] >= a.R) r[c] = -1;
            g[c] = slot && a.gates ? a.gates[t * a.k + j0 + c] : 1.0f;
            dot[c] = 0.0f;
        }
        if (in)
            for (int at = u0; at < p.units; at += step) {
                const int left = a.D - at * CE;
                const uint4 du = load_partial<T>(a.x + (t * a.ldx + (int64_t)at * CE) * (int64_t)sizeof(T), left);
                uint4 yu[C];
                if (a.dgates)
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (r[c] >= 0)
                            yu[c] = load_partial<T>(a.y + (r[c] * a.ldy + (int64_t)at * CE) * (int64_t)sizeof(T), left);
                float d[CE];
                unpack_unit<T>(du, d);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (r[c] < 0) continue;
                    float f[CE];
                    if (a.dgates) {
                        unpack_unit<T>(yu[c], f);
#pragma unroll
                        for (int i = 0; i < CE; ++i) dot[c] = fmaf(d[i], f[i], dot[c]);
                    }
                    if (a.dy) {
#pragma unroll
                        for (int i = 0; i < CE; ++i) f[i] = g[c] * d[i];
                        store_partial<T>(a.dy + (r[c] * a.lddy + (int64_t)at * CE) * (int64_t)sizeof(T), pack_unit<T>(f), left);
                    }
                }
            }
        if (a.dgates) {
#pragma unroll
            for (int c = 0; c < C; ++c) dot[c] = sum_lanes(dot[c], p.lanes);
            if constexpr (W > 1) {
                __syncthreads();
                if (lane == 0)
#pragma unroll
                    for (int c = 0; c < C; ++c) part[wave][c] = dot[c];
                __syncthreads();
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    dot[c] = part[0][c];
#pragma unroll
                    for (int w = 1; w < W; ++w) dot[c] += part[w][c];
                }
            }
            if (in && (W == 1 || wave == 0) && (lane & (p.lanes - 1)) == 0)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (j0 + c < a.k) a.dgates[t * a.k + j0 + c] = r[c] < 0 ? 0.0f : dot[c];
        }
    }
    if (a.dy) {
        // whole rows are `segs` pieces of one unit per lane here
        const int64_t waves = (int64_t)gridDim.x * gridDim.y * 4;
        zero_rows<T, 1>(a, p, (int64_t)block_id() * 4 + wave, waves, a.dy, a.lddy);
    }
}

template <class T>
hipError_t dispatch(const ExchangeArgs &a, hipStream_t s) {
    const Pieces p = pieces(a.T, a.D, kUnit<T>, kDispatchUnits);
    hipLaunchKernelGGL(HIP_KERNEL_NAME(dispatch_kernel<T>), grid_of((p.items + 3) / 4, 256), dim3(256), 0, s, a, p);
    return hipGetLastError();
}

template <class T>
hipError_t combine(const ExchangeArgs &a, hipStream_t s) {
    const Pieces p = pieces(a.T, a.D, kUnit<T>, 2);
    const dim3 grid = grid_of((p.items + 3) / 4, 256);
    if (a.k <= 2) hipLaunchKernelGGL(HIP_KERNEL_NAME(combine_kernel<T, 2, 2>), grid, dim3(256), 0, s, a, p);
    else hipLaunchKernelGGL(HIP_KERNEL_NAME(combine_kernel<T, 2, 4>), grid, dim3(256), 0, s, a, p);
    return hipGetLastError();
}

template <class T>
hipError_t combine_backward(const ExchangeArgs &a, hipStream_t s) {
    const Pieces p = pieces(a.T, a.D, kUnit<T>, 1);
    const int64_t tokens = 64 >> p.shift, waves = a.T ? (a.T + tokens - 1) / tokens : 1;
    // Waves that share a token: where tokens are too few to fill the device with a wave to
    // each (256 x 4 x 4096 bf16 16.2 us against 7.7, 1024 x 4 x 8192 43 against 26), and where y and
    // dy are far from fitting the last cache of 256 MB, as fewer rows are then open at a time
    // (6000 x 4 x 6144 186 us against 138).  In between a wave to a token is faster: no
    // barriers (4096 x 4 x 4096 61 us against 67, 4096 x 4 x 1024 16 against 25).
    const int64_t bytes = a.T * a.k * a.D * (int64_t)sizeof(T);
    const bool shared = p.lanes == 64 && p.units > 64 && (a.T < 8 * kComputeUnits || bytes > (int64_t(160) << 20));
    if (shared)
        hipLaunchKernelGGL(HIP_KERNEL_NAME(combine_backward_kernel<T, 4, 4>), grid_of(waves, 256), dim3(256), 0, s, a, p);
    else
        hipLaunchKernelGGL(HIP_KERNEL_NAME(combine_backward_kernel<T, 4, 1>), grid_of((waves + 3) / 4, 256), dim3(256), 0, s,
                           a, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dispatch(int dtype, const ExchangeArgs &a, hipStream_t s) {
    return dtype == CP_BF16 ? dispatch<__bf16>(a, s) : dispatch<float>(a, s);
}
hipError_t launch_combine(int dtype, const ExchangeArgs &a, hipStream_t s) {
    return dtype == CP_BF16 ? combine<__bf16>(a, s) : combine<float>(a, s);
}
hipError_t launch_combine_backward(int dtype, const ExchangeArgs &a, hipStream_t s) {
    return dtype == CP_BF16 ? combine_backward<__bf16>(a, s) : combine_backward<float>(a, s);
}

}  // namespace cpo
