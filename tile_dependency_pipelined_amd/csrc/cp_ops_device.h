// cp_ops_device.h -- what the feed-forward operators' kernels share: launch
// arguments, element conversion, activations, the row spans of experts.
// Internal to the library (the C ABI is include/cp_ops.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "cp_ops.h"

namespace cpo {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) v4i16_t lds_v4i16_t;

// Elements of 16 bytes, the unit of all wide loads and stores.
template <class T>
constexpr int kUnit = 16 / (int)sizeof(T);

enum : int32_t { kDense = 0, kGroupRows = 1, kGroupSum = 2 };

// One product launch: C = epilogue(A . B) with A[m][k], B[k][n]; which of the
// two indices is contiguous in memory is a template argument of the kernel.
//   kDense      one product
//   kGroupRows  rows of A and C are sorted by expert; B (and bias) per expert
//   kGroupSum   the contraction runs over rows sorted by expert: one C per
//               expert
struct GemmArgs {
    const char *A, *B;
    char *C;
    const char *bias, *res;  // epilogue inputs or null
    char *pre;               // pre-activation output or null
    float *ws;               // nsplit > 1: fp32 partials [nsplit][M][ldws]
    int64_t lda, ldb, ldc, ldr, ldp;  // elements
    int64_t sb, sc;          // per-expert strides of B (kGroupRows) and C (kGroupSum)
    const int32_t *off;      // device: groups + 1 row offsets, or null
    int32_t groups, mode;
    int32_t M, N, K;         // rows and columns of C, contraction (kGroupRows: M = all rows; kGroupSum: K = all rows)
    int32_t act;
    int32_t nsplit;          // contraction ranges, each to its own partial
    int32_t ntm, ntn;        // tiles (kGroupRows: ntm is not used, the device counts)
    int32_t ldws;
    int32_t vec;             // C, R, pre and bias can be accessed 16 bytes at a time
};

// A block's number in a launch whose grid may have a second dimension (fewer
// than 2^31 blocks and those that fill its last row).
__device__ __forceinline__ unsigned block_id() { return blockIdx.y * gridDim.x + blockIdx.x; }

// ---------------------------------------------------------------- elements

template <class T>
__device__ __forceinline__ float to_f32(T v) {
    return (float)v;
}
// fp32 -> T: to nearest even, NaN stays NaN
template <class T>
__device__ __forceinline__ T from_f32(float v) {
    return (T)v;
}

template <class T>
__device__ __forceinline__ void load_unit(const void *p, float (&v)[kUnit<T>]) {  // 16-byte aligned
    union {
        uint4 u;
        T e[kUnit<T>];
    } x;
    x.u = *reinterpret_cast<const uint4 *>(p);
#pragma unroll
    for (int i = 0; i < kUnit<T>; ++i) v[i] = to_f32(x.e[i]);
}
template <class T>
__device__ __forceinline__ void store_unit(void *p, const float (&v)[kUnit<T>]) {
    union {
        uint4 u;
        T e[kUnit<T>];
    } x;
#pragma unroll
    for (int i = 0; i < kUnit<T>; ++i) x.e[i] = from_f32<T>(v[i]);
    *reinterpret_cast<uint4 *>(p) = x.u;
}

// 16 bytes of which only the first `n` elements (0 .. kUnit) may be read, the
// rest zero; any alignment.  A whole unit is one 16-byte load (global loads
// need no alignment on this target).
template <class T>
__device__ __forceinline__ uint4 load_partial(const char *p, int n) {
    union {
        uint4 u;
        T e[kUnit<T>];
    } x;
    if (n >= kUnit<T>) {
        __builtin_memcpy(&x.u, p, 16);
    } else {
        x.u = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kUnit<T> - 1; ++i)
            if (i < n) x.e[i] = reinterpret_cast<const T *>(p)[i];
    }
    return x.u;
}

// -------------------------------------------------------------- activations

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu0 = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGelu1 = 0.044715f;

// 1 / (1 + 2^t), two hardware approximations of 1 ulp
__device__ __forceinline__ float inv_1_exp2(float t) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}
__device__ __forceinline__ float sigmoid(float x) { return inv_1_exp2(-kLog2e * x); }
// sigmoid(2 u) of the tanh form of GeLU, u = sqrt(2/pi) (x + 0.044715 x^3):
// (1 + tanh u) / 2 without cancellation, and one product less
__device__ __forceinline__ float gelu_gate(float x) {
    constexpr float c = -2.0f * kLog2e * kGelu0;
    return inv_1_exp2(x * fmaf(c * kGelu1, x * x, c));
}

__device__ __forceinline__ float act_apply(float x, int act) {
    if (act == CP_ACT_GELU_TANH) return x * gelu_gate(x);
    if (act == CP_ACT_SILU) return x * sigmoid(x);
    if (act == CP_ACT_RELU) return x < 0.0f ? 0.0f : x;
    return x;
}

__device__ __forceinline__ float clamp_keep_nan(float x, float lim) { return fabsf(x) > lim ? copysignf(lim, x) : x; }

// Derivative.  Beyond the clamps it is 0 or 1 to fp32 precision; without them
// x^2 could overflow and 0 * inf give NaN for a finite x.
__device__ __forceinline__ float act_grad(float x, int act) {
    if (act == CP_ACT_GELU_TANH) {  // p + p (1 - p) 2 x u'(x), u' = sqrt(2/pi) (1 + 3 * 0.044715 x^2)
        x = clamp_keep_nan(x, 10.0f);
        const float p = gelu_gate(x);
        return p * fmaf(1.0f - p, x * fmaf(6.0f * kGelu0 * kGelu1, x * x, 2.0f * kGelu0), 1.0f);
    }
    if (act == CP_ACT_SILU) {
        x = clamp_keep_nan(x, 80.0f);
        const float p = sigmoid(x);
        return p * fmaf(1.0f - p, x, 1.0f);
    }
    if (act == CP_ACT_RELU) return x > 0.0f ? 1.0f : (x == x ? 0.0f : x);
    return 1.0f;
}

// ---------------------------------------------------------------- epilogue

// Epilogue of one run of CNT consecutive columns of a row (fp32 sums v): bias,
// pre-activation store, activation, residual, one rounding, store.  CNT is a
// unit (every pointer 16-byte aligned) or 1.  Bias and residual come in as
// loaded, so that a caller can request them early.
template <class T, int CNT>
struct Raw {
    std::conditional_t<CNT == 1, T, uint4> v;
    __device__ __forceinline__ void load(const char *p) {
        v = *reinterpret_cast<const std::conditional_t<CNT == 1, T, uint4> *>(p);
    }
    __device__ __forceinline__ void unpack(float (&x)[CNT]) const {
        if constexpr (CNT == 1) {
            x[0] = to_f32(v);
        } else {
            union {
                uint4 u;
                T e[CNT];
            } y;
            y.u = v;
#pragma unroll
            for (int i = 0; i < CNT; ++i) x[i] = to_f32(y.e[i]);
        }
    }
};

// NU runs at once, at rows row, row + step, ..: what the call asks for is
// branched on once for all of them.  Run i is stored if `inside` (uniform) or
// if the column is in range and its row is below row_end.
template <class T, int CNT, int NU>
__device__ __forceinline__ void finish(const GemmArgs &g, char *C, int row, int step, int col, float (&v)[NU][CNT],
                                       const Raw<T, CNT> *bias, const Raw<T, CNT> *res, bool zero, bool inside,
                                       bool col_in, int row_end) {
    static_assert(CNT == 1 || CNT == kUnit<T>, "columns per run");
    auto put = [&](char *base, int64_t ld) {
        char *p = base + ((int64_t)row * ld + col) * sizeof(T);
        auto one = [&](int i) {
            char *q = p + (int64_t)i * step * ld * sizeof(T);
            if constexpr (CNT > 1) store_unit<T>(q, v[i]);
            else *reinterpret_cast<T *>(q) = from_f32<T>(v[i][0]);
        };
        if (inside) {
#pragma unroll
            for (int i = 0; i < NU; ++i) one(i);
        } else if (col_in) {
#pragma unroll
            for (int i = 0; i < NU; ++i)
                if (row + i * step < row_end) one(i);
        }
    };
    auto each = [&](auto &&f) {
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[i][j] = f(v[i][j]);
    };
    if (bias) {
        float t[CNT];
        bias->unpack(t);
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[i][j] = zero ? 0.0f : v[i][j] + t[j];
    }
    if (g.pre) put(g.pre, g.ldp);
    if (g.act == CP_ACT_GELU_TANH) each([](float x) { return act_apply(x, CP_ACT_GELU_TANH); });
    else if (g.act == CP_ACT_SILU) each([](float x) { return act_apply(x, CP_ACT_SILU); });
    else if (g.act == CP_ACT_RELU) each([](float x) { return act_apply(x, CP_ACT_RELU); });
    if (res) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            float t[CNT];
            res[i].unpack(t);
#pragma unroll
            for (int j = 0; j < CNT; ++j) v[i][j] += t[j];
        }
    }
    put(C, g.ldc);
}

// ------------------------------------------------------------- expert spans

// Rows of one expert, as 64 lanes look at 64 experts at a time.  Lane l of a
// wave holds expert base + l; expert `groups` is the rest of the rows, which
// belong to none.  Offsets are taken as the running maximum of their values
// clamped to [0, rows], with the first one 0: any content stays in range.
struct GroupScan {
    int start, end;  // this lane's rows
    int tiles_end;   // tiles of `tile` rows up to and including this lane's expert
};

// Inclusive scan over the wave with cross-lane moves inside the vector unit (a
// scan by shuffles, twelve dependent LDS round trips, took longer than the
// offsets' loads).  The values are not negative: 0 is neutral.
template <class Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));  // row_shr 1, 2, 4, 8: within 16 lanes
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));  // lane 15 to the next 16, 47 likewise
    return op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));  // lane 31 to the upper half
}

__device__ __forceinline__ GroupScan scan_groups(const int32_t *off, int groups, int rows, int tile, int base,
                                                 int carry_end, int carry_tiles) {
    const int lane = threadIdx.x & 63, e = base + lane;
    int end = rows;
    if (e < groups) {
        end = off[e + 1];
        end = end < 0 ? 0 : (end > rows ? rows : end);
    }
    end = end > carry_end ? end : carry_end;
    end = wave_scan(end, [](int a, int b) { return a > b ? a : b; });
    int start = __shfl_up(end, 1);
    if (lane == 0) start = carry_end;
    int tiles = e <= groups ? (end - start + tile - 1) / tile : 0;
    tiles = wave_scan(tiles, [](int a, int b) { return a + b; });
    return {start, end, tiles + carry_tiles};
}

// All the row tiles of a launch (uniform over the wave).
__device__ __forceinline__ int count_tiles(const int32_t *off, int groups, int rows, int tile, GroupScan &s) {
    int carry_end = 0, carry_tiles = 0;
    for (int base = 0; base <= groups; base += 64) {
        s = scan_groups(off, groups, rows, tile, base, carry_end, carry_tiles);
        carry_end = __builtin_amdgcn_readlane(s.end, 63);
        carry_tiles = __builtin_amdgcn_readlane(s.tiles_end, 63);
    }
    return carry_tiles;
}

struct RowTile {
    int expert;      // == groups: rows without an expert
    int row0, end;   // the expert's rows
    int before;      // row tiles of the experts before it
};

// The expert whose rows row tile t (0 <= t < count_tiles) takes.  `s` is what
// count_tiles left: with fewer than 64 experts it is the only chunk.
__device__ __forceinline__ RowTile find_tile(const int32_t *off, int groups, int rows, int tile, int t, GroupScan s) {
    int carry_end = 0, carry_tiles = 0;
    for (int base = 0;; base += 64) {
        if (groups >= 64) s = scan_groups(off, groups, rows, tile, base, carry_end, carry_tiles);
        const uint64_t hit = __ballot(s.tiles_end > t);
        if (hit || base + 64 > groups) {
            const int l = hit ? __builtin_ctzll(hit) : 63;
            const int before = l ? __builtin_amdgcn_readlane(s.tiles_end, l - 1) : carry_tiles;
            const int start = __builtin_amdgcn_readlane(s.start, l);
            return {base + l, start, __builtin_amdgcn_readlane(s.end, l), before};
        }
        carry_end = __builtin_amdgcn_readlane(s.end, 63);
        carry_tiles = __builtin_amdgcn_readlane(s.tiles_end, 63);
    }
}

// The rows of expert e (uniform), by the same rule.
__device__ __forceinline__ RowTile expert_rows(const int32_t *off, int groups, int rows, int e) {
    int carry_end = 0;
    for (int base = 0;; base += 64) {
        const GroupScan s = scan_groups(off, groups, rows, 1, base, carry_end, 0);
        if (e < base + 64)
            return {e, __builtin_amdgcn_readlane(s.start, e - base), __builtin_amdgcn_readlane(s.end, e - base), 0};
        carry_end = __builtin_amdgcn_readlane(s.end, 63);
    }
}

// Workgroups go round-robin to the 8 XCDs, each with its own L2.  Of `n`
// items, give each XCD a contiguous range: item of workgroup b (b < n).
__device__ __forceinline__ int xcd_remap(int b, int n) {
    const int x = b & 7, q = n >> 3, r = n & 7;
    return x * q + (x < r ? x : r) + (b >> 3);
}

// Of `units` tiles of 256 x 256, how many are computed as two halves each: the
// last round's, if its halves fit the device.
constexpr int kComputeUnits = 256;
__host__ __device__ constexpr int halved_tiles(int units) {
    const int rest = units % kComputeUnits;
    return 2 * rest <= kComputeUnits ? rest : 0;
}

// dZ = dY act'(pre) and column sums of it per expert (dense: groups = 1, off null)
struct GradArgs {
    const char *dy, *pre;
    char *dz, *db;
    float *ws;             // [row tiles][N] partial column sums
    int64_t ldd, ldp, ldz;
    const int32_t *off;
    int32_t groups, M, N, act, tiles, vec;
    int32_t final;         // the only row tile: its sums are db
};
constexpr int kGradRows = 32;  // rows of a partial column sum

// db[e] = sum of its row tiles' partials (GradArgs): 64 columns x NT / 64
// ranges of tiles per block.
template <class T, int NT>
__device__ __forceinline__ void join_columns(const GradArgs &a, int b, float *part) {
    constexpr int R = NT / 64;
    const int col_blocks = (a.N + 63) / 64;
    const int e = b / col_blocks, t = threadIdx.x & 63, s = threadIdx.x >> 6;
    const int col = (b % col_blocks) * 64 + t;
    int from = 0, to = (a.M + kGradRows - 1) / kGradRows;
    if (a.off) {
        int carry_end = 0, carry_tiles = 0;
        for (int base = 0;; base += 64) {
            const GroupScan g = scan_groups(a.off, a.groups, a.M, kGradRows, base, carry_end, carry_tiles);
            if (e < base + 64) {
                const int l = e - base;
                from = l ? __builtin_amdgcn_readlane(g.tiles_end, l - 1) : carry_tiles;
                to = __builtin_amdgcn_readlane(g.tiles_end, l);
                break;
            }
            carry_end = __builtin_amdgcn_readlane(g.end, 63);
            carry_tiles = __builtin_amdgcn_readlane(g.tiles_end, 63);
        }
    }
    const int per = (to - from + R - 1) / R, p0 = from + s * per, p1 = p0 + per < to ? p0 + per : to;
    float v = 0.0f;
    if (col < a.N)
#pragma unroll 8
        for (int i = p0; i < p1; ++i) v += a.ws[(int64_t)i * a.N + col];
    part[s * 64 + t] = v;
    __syncthreads();
    if (s > 0 || col >= a.N) return;
#pragma unroll
    for (int i = 1; i < R; ++i) v += part[i * 64 + t];
    reinterpret_cast<T *>(a.db)[(int64_t)e * a.N + col] = from_f32<T>(v);
}

}  // namespace cpo
