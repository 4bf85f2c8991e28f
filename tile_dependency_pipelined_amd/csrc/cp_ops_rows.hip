// cp_ops_rows.hip -- the operators' row and column passes for gfx950: joining
// split products, activation gradients with bias sums, layer normalisation.
// All are bound by memory traffic: one pass over the data, 16 bytes per lane
// where the rows allow it, sums in fp32 in a fixed order.
#include "cp_ops_host.h"

namespace cpo {

namespace {

// ------------------------------------------------------------------- packing

// 64 units of 16 bytes x 4 rows per block; the source may lie anyhow.  777 x
// 1003 and 1003 x 2049 bf16 (5.7 MB each way) 7.6 us: the launch and the latency
// of one load and store.
struct PackGrid {
    int unit_blocks[3], end[3];  // of each copy: blocks along a row, last block + 1
};
template <class T>
__device__ __forceinline__ void pack_block(const PackArgs &a, const PackGrid &g, unsigned b) {
    constexpr int CE = kUnit<T>;
    if (b >= (unsigned)g.end[2]) return;
    int i = 0;
    while (i < 2 && b >= (unsigned)g.end[i]) ++i;
    if (i > 0) b -= g.end[i - 1];
    const PackArgs::One o = a.one[i];
    const int u = (b % g.unit_blocks[i]) * 64 + (threadIdx.x & 63);
    const int64_t r = (int64_t)(b / g.unit_blocks[i]) * 4 + (threadIdx.x >> 6);
    if (u * CE >= o.cols || r >= (int64_t)o.count * o.rows) return;
    const int m = (int)(r / o.rows), row = (int)(r - (int64_t)m * o.rows);
    const char *src = o.src + (m * o.stride + row * o.ld + u * CE) * (int64_t)sizeof(T);
    *reinterpret_cast<uint4 *>(o.dst + (m * o.stride_d + row * o.ldd + u * CE) * (int64_t)sizeof(T)) =
        load_partial<T>(src, o.cols - u * CE);
}

template <class T>
__global__ __launch_bounds__(256) void pack_kernel(PackArgs a, PackGrid g) {
    pack_block<T>(a, g, block_id());
}

// ------------------------------------------------------------------- joining

// Y = epilogue(sum over splits of partial); one block per row and 256 units.
// 4 x 515 x 2048 (17 MB, in the caches) 5.1 us, mostly the launch.
template <class T, int CNT>
__global__ __launch_bounds__(256) void join_kernel(GemmArgs g, int blocks_per_row) {
    const unsigned id = block_id();
    const int all = (int)(id / blocks_per_row);  // row of the partials
    if (all >= g.M * (g.mode == kGroupSum ? g.groups : 1)) return;
    const int expert = g.mode == kGroupSum ? all / g.M : 0, row = all - expert * g.M;
    const int col = (int)((id % blocks_per_row) * 256 + threadIdx.x) * CNT;
    char *C = g.C + (int64_t)expert * g.sc * sizeof(T);
    const char *bias = g.bias;
    bool zero = false;
    if (g.mode == kGroupRows && bias) {  // the row's expert
        int carry = 0, e = g.groups;
        for (int base = 0; base <= g.groups; base += 64) {
            const GroupScan s = scan_groups(g.off, g.groups, g.M, 1, base, carry, 0);
            const uint64_t hit = __ballot(s.end > row);
            if (hit) {
                e = base + __builtin_ctzll(hit);
                break;
            }
            carry = __builtin_amdgcn_readlane(s.end, 63);
        }
        zero = e >= g.groups;
        if (!zero) bias += (int64_t)e * g.N * sizeof(T);
    }
    if (col >= g.N) return;
    float v[1][CNT];
#pragma unroll
    for (int i = 0; i < CNT; ++i) v[0][i] = 0.0f;
    const float *p = g.ws + (int64_t)all * g.ldws + col;
    const int64_t step = (int64_t)g.M * g.ldws * (g.mode == kGroupSum ? g.groups : 1);
#pragma unroll 4
    for (int s = 0; s < g.nsplit; ++s) {
#pragma unroll
        for (int i = 0; i < CNT; ++i) v[0][i] += p[s * step + i];
    }
    Raw<T, CNT> b, r;
    if (bias) b.load(bias + (int64_t)col * sizeof(T));
    if (g.res) r.load(g.res + ((int64_t)row * g.ldr + col) * sizeof(T));
    finish<T, CNT, 1>(g, C, row, 0, col, v, bias ? &b : nullptr, g.res ? &r : nullptr, zero, true, true, 0);
}

// --------------------------------------------- activation gradient, bias sums

// 32 units of columns x 8 rows per pass; each block one row tile (kGradRows rows
// of one expert) and 32 units.  Rows that are not aligned are read by unaligned
// units (VEC false; only a row's last unit by elements), dZ's rows always are.
// Bound by its bytes: 2048 x 4096 bf16 with GELU (50 MB) 11.3 us, 4.5 TB/s.
// The blocks from `blocks` on make the copies that the products need, which
// saves a launch: 43 x 1059 x 696, rows off 16 bytes, 12.6 -> 10.2 us.
// dZ is rounded to the element type, being an operand of the products that follow:
// in bf16 that takes their results from 1.7e-3 to 2.3e-3 off (relative 2-norm),
// where a 32-bit dZ in halves would double the products.  The sums take it unrounded.
template <class T, int ACT, bool VEC>
__global__ __launch_bounds__(256) void grad_kernel(GradArgs a, int col_blocks, int blocks, PackArgs packs, PackGrid grid) {
    constexpr int CNT = kUnit<T>;
    __shared__ float part[8][32 * CNT];
    const unsigned id = block_id();
    if (id >= (unsigned)blocks) return pack_block<T>(packs, grid, id - blocks);
    const int ct = (int)(id % col_blocks), rt = (int)(id / col_blocks);
    int row0 = rt * kGradRows, end = a.M;
    if (a.off) {
        GroupScan s;
        if (rt >= count_tiles(a.off, a.groups, a.M, kGradRows, s)) return;
        const RowTile t = find_tile(a.off, a.groups, a.M, kGradRows, rt, s);
        if (t.expert == a.groups) return;  // their dZ is never read
        row0 = t.row0 + (rt - t.before) * kGradRows;
        end = t.end;
    }
    if (end > row0 + kGradRows) end = row0 + kGradRows;
    const int u = threadIdx.x & 31, r = threadIdx.x >> 5, col = (ct * 32 + u) * CNT;
    float sum[CNT];
#pragma unroll
    for (int i = 0; i < CNT; ++i) sum[i] = 0.0f;
    if (col < a.N) {
        // All rows are requested before the first one's dZ is stored, without
        // a branch in between (past the end the last row, again): with one
        // the compiler waited for each load.
        constexpr int R = kGradRows / 8;
        Raw<T, CNT> dy[R], z[R];
        auto request = [&](auto &&get) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int row = row0 + r + 8 * i < end ? row0 + r + 8 * i : end - 1;
                dy[i].v = get(a.dy + ((int64_t)row * a.ldd + col) * sizeof(T));
                if constexpr (ACT != CP_ACT_NONE) z[i].v = get(a.pre + ((int64_t)row * a.ldp + col) * sizeof(T));
            }
        };
        if constexpr (VEC)
            request([](const char *p) { return *reinterpret_cast<const uint4 *>(p); });
        else if (col + CNT <= a.N)
            request([](const char *p) {
                uint4 v;
                __builtin_memcpy(&v, p, 16);
                return v;
            });
        else
            request([&](const char *p) { return load_partial<T>(p, a.N - col); });
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = row0 + r + 8 * i;
            if (row >= end) break;
            float d[CNT];
            dy[i].unpack(d);
            if constexpr (ACT != CP_ACT_NONE) {
                float x[CNT];
                z[i].unpack(x);
                // (past the row's end dy is zero, so dZ's rows end in zeros)
#pragma unroll
                for (int j = 0; j < CNT; ++j) d[j] *= act_grad(x[j], ACT);
                store_unit<T>(a.dz + ((int64_t)row * a.ldz + col) * sizeof(T), d);
            }
#pragma unroll
            for (int j = 0; j < CNT; ++j) sum[j] += d[j];
        }
    }
    if (!a.db) return;
#pragma unroll
    for (int i = 0; i < CNT; ++i) part[r][u * CNT + i] = sum[i];
    __syncthreads();
    for (int c = threadIdx.x; c < 32 * CNT; c += 256) {
        const int gc = ct * 32 * CNT + c;
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += part[i][c];
        if (gc >= a.N) continue;
        if (a.final) reinterpret_cast<T *>(a.db)[gc] = from_f32<T>(v);
        else a.ws[(int64_t)rt * a.N + gc] = v;
    }
}

template <class T>
__global__ __launch_bounds__(256) void grad_join_kernel(GradArgs a) {
    __shared__ float part[256];
    const unsigned b = block_id();
    if (b < (unsigned)(a.groups * ((a.N + 63) / 64))) join_columns<T, 256>(a, (int)b, part);
}

// ------------------------------------------------------- layer normalisation

// Sum over a wave, the same value in every lane: cross-lane adds inside the
// vector unit (a shuffle through LDS takes several times as long).
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 15, 15, true));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0x111>(v);  // row_shr 1, 2, 4, 8: lane 15 of each 16 holds their sum
    v = dpp_add<0x112>(v);
    v = dpp_add<0x114>(v);
    v = dpp_add<0x118>(v);
    auto at = [&](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l)); };
    return (at(15) + at(31)) + (at(47) + at(63));
}

// Sum over the THREADS threads of a row: a wave, or a block through LDS
// (`sh`: one float per wave; two barriers, so it can be called again at once).
template <int THREADS>
__device__ __forceinline__ float row_sum(float v, float *sh) {
    v = wave_sum(v);
    if constexpr (THREADS > 64) {
        constexpr int W = THREADS / 64;
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) v += sh[i];
        __syncthreads();
    }
    return v;
}

// Column of element i of unit q of thread t: 16-byte units in turn, or single
// elements in turn where rows are not aligned (both read whole lines).
template <class T, int THREADS, bool VEC>
__device__ __forceinline__ int norm_col(int q, int i, int t) {
    return VEC ? (q * THREADS + t) * kUnit<T> + i : (q * kUnit<T> + i) * THREADS + t;
}

// The forward pass reads unaligned bf16 rows by 16-byte units as well: a row's
// last unit starts early enough to end with the row, and its thread leaves to
// the one before what they share.  (Single elements are as many loads as there
// are columns: 4477 x 9970 150 us, 36 with units; 4477 x 4097 73 and 29.  fp32
// gains nothing: 4096 x 9001 62 us, 76 with units.  Nor does the backward pass up
// to 8192 columns, where the masks cost more: 912 x 49 12 us, 22 with units, 4477 x
// 4097 45 and 53; beyond, little: 4477 x 9970 195 and 181.)
enum Access : int { kElements, kUnits, kShifted };

// First column of unit q, and whether its element i is this thread's.
template <class T, int THREADS>
__device__ __forceinline__ int shifted(int q, int t, int N) {
    const int c = (q * THREADS + t) * kUnit<T>;
    return c + kUnit<T> <= N ? c : N - kUnit<T>;
}
template <class T, int THREADS, Access A>
__device__ __forceinline__ bool norm_mine(int q, int i, int t, int N) {
    if constexpr (A == kShifted) {
        const int c = (q * THREADS + t) * kUnit<T>;
        return shifted<T, THREADS>(q, t, N) + i >= c && c < N;
    }
    return norm_col<T, THREADS, A == kUnits>(q, i, t) < N;
}

// (what is not this thread's: anything)
template <class T, int THREADS, int VPT, Access A>
__device__ __forceinline__ void norm_load(const char *row, int N, int t, float (&v)[VPT][kUnit<T>]) {
    if constexpr (A != kElements) {
        uint4 u[VPT];  // all requested before the first is used
#pragma unroll
        for (int q = 0; q < VPT; ++q) {
            u[q] = make_uint4(0, 0, 0, 0);
            if constexpr (A == kUnits) {
                const int c = norm_col<T, THREADS, A == kUnits>(q, 0, t);
                if (c < N) u[q] = *reinterpret_cast<const uint4 *>(row + (int64_t)c * sizeof(T));
            } else {
                __builtin_memcpy(&u[q], row + (int64_t)shifted<T, THREADS>(q, t, N) * sizeof(T), 16);
            }
        }
#pragma unroll
        for (int q = 0; q < VPT; ++q) load_unit<T>(&u[q], v[q]);
    } else {
#pragma unroll
        for (int q = 0; q < VPT; ++q)
#pragma unroll
            for (int i = 0; i < kUnit<T>; ++i) {
                const int c = norm_col<T, THREADS, A == kUnits>(q, i, t);
                v[q][i] = c < N ? to_f32(reinterpret_cast<const T *>(row)[c]) : 0.0f;
            }
    }
}

template <class T, int THREADS, int VPT, Access A>
__device__ __forceinline__ void norm_store(char *row, int N, int t, const float (&v)[VPT][kUnit<T>]) {
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        if constexpr (A == kUnits) {
            const int c = norm_col<T, THREADS, A == kUnits>(q, 0, t);
            if (c < N) store_unit<T>(row + (int64_t)c * sizeof(T), v[q]);
        } else if constexpr (A == kShifted) {
            const int c = (q * THREADS + t) * kUnit<T>;
            if (c + kUnit<T> <= N) {
                uint4 u;
                store_unit<T>(&u, v[q]);
                __builtin_memcpy(row + (int64_t)c * sizeof(T), &u, 16);
            } else if (c < N) {
#pragma unroll
                for (int i = 0; i < kUnit<T>; ++i) {
                    const int at = N - kUnit<T> + i;
                    if (at >= c) reinterpret_cast<T *>(row)[at] = from_f32<T>(v[q][i]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kUnit<T>; ++i) {
                const int c = norm_col<T, THREADS, A == kUnits>(q, i, t);
                if (c < N) reinterpret_cast<T *>(row)[c] = from_f32<T>(v[q][i]);
            }
        }
    }
}

// One row per THREADS threads, held in registers: the deviation is summed from
// the values themselves (no difference of large squares).  Bound by its bytes,
// read and written once: 4093 x 4099 fp32 (134 MB) 24.8 us, 5.4 TB/s; 16384 x
// 8192 bf16 (537 MB) 108 us, 5.0 TB/s.
template <class T, int THREADS, int VPT, Access A>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void norm_kernel(NormArgs a) {
    constexpr int BLOCK = THREADS < 256 ? 256 : THREADS, CE = kUnit<T>;
    __shared__ float sh[16];
    const int t = threadIdx.x % THREADS;
    const int row = blockIdx.x * (BLOCK / THREADS) + threadIdx.x / THREADS;
    if (row >= a.M) return;  // whole waves; with one row per block never taken
    float v[VPT][CE];
    norm_load<T, THREADS, VPT, A>(a.x + (int64_t)row * a.ldx * sizeof(T), a.N, t, v);
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < VPT; ++q)
#pragma unroll
        for (int i = 0; i < CE; ++i) s += norm_mine<T, THREADS, A>(q, i, t, a.N) ? v[q][i] : 0.0f;
    const float mean = row_sum<THREADS>(s, sh) / (float)a.N;
    float ss = 0.0f;
#pragma unroll
    for (int q = 0; q < VPT; ++q)
#pragma unroll
        for (int i = 0; i < CE; ++i) {
            v[q][i] = norm_mine<T, THREADS, A>(q, i, t, a.N) ? v[q][i] - mean : 0.0f;
            ss += v[q][i] * v[q][i];
        }
    const float rstd = 1.0f / sqrtf(row_sum<THREADS>(ss, sh) / (float)a.N + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int q = 0; q < VPT; ++q)
#pragma unroll
        for (int i = 0; i < CE; ++i) v[q][i] *= rstd;
    float p[VPT][CE];
    if (a.w) {
        norm_load<T, THREADS, VPT, A>(a.w, a.N, t, p);
#pragma unroll
        for (int q = 0; q < VPT; ++q)
#pragma unroll
            for (int i = 0; i < CE; ++i) v[q][i] *= p[q][i];
    }
    if (a.b) {
        norm_load<T, THREADS, VPT, A>(a.b, a.N, t, p);
#pragma unroll
        for (int q = 0; q < VPT; ++q)
#pragma unroll
            for (int i = 0; i < CE; ++i) v[q][i] += p[q][i];
    }
    norm_store<T, THREADS, VPT, A>(a.y + (int64_t)row * a.ldy * sizeof(T), a.N, t, v);
}

// Rows too long for registers: three passes over the row (the second and third
// mostly from the cache), element by element.
template <class T>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
    __shared__ float sh[16];
    const int row = blockIdx.x, t = threadIdx.x;
    const T *x = reinterpret_cast<const T *>(a.x) + (int64_t)row * a.ldx;
    const T *w = reinterpret_cast<const T *>(a.w), *b = reinterpret_cast<const T *>(a.b);
    T *y = reinterpret_cast<T *>(a.y) + (int64_t)row * a.ldy;
    float s = 0.0f;
    for (int c = t; c < a.N; c += 1024) s += to_f32(x[c]);
    const float mean = row_sum<1024>(s, sh) / (float)a.N;
    float ss = 0.0f;
    for (int c = t; c < a.N; c += 1024) {
        const float d = to_f32(x[c]) - mean;
        ss += d * d;
    }
    const float rstd = 1.0f / sqrtf(row_sum<1024>(ss, sh) / (float)a.N + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    for (int c = t; c < a.N; c += 1024) {
        float v = (to_f32(x[c]) - mean) * rstd;
        if (w) v *= to_f32(w[c]);
        if (b) v += to_f32(b[c]);
        y[c] = from_f32<T>(v);
    }
}

// A row (or parameter vector) as loaded, a thread's share of it.
template <class T, int THREADS, int VPT, bool VEC>
struct RowShare {
    static constexpr int CE = kUnit<T>;
    union {
        uint4 u[VPT];
        T e[VPT][CE];
    };
    __device__ __forceinline__ RowShare() {}
    __device__ __forceinline__ void load(const char *row, int N, int t) {
#pragma unroll
        for (int q = 0; q < VPT; ++q) {
            if constexpr (VEC) {
                const int c = norm_col<T, THREADS, VEC>(q, 0, t);
                u[q] = c < N ? *reinterpret_cast<const uint4 *>(row + (int64_t)c * sizeof(T)) : make_uint4(0, 0, 0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < CE; ++i) {
                    const int c = norm_col<T, THREADS, VEC>(q, i, t);
                    e[q][i] = c < N ? reinterpret_cast<const T *>(row)[c] : from_f32<T>(0.0f);
                }
            }
        }
    }
    __device__ __forceinline__ float at(int q, int i) const { return to_f32(e[q][i]); }
    // What was unpacked so far is not kept: the next use unpacks again.
    __device__ __forceinline__ void forget() {
        if constexpr (VEC && sizeof(T) == 2)
#pragma unroll
            for (int q = 0; q < VPT; ++q)
                asm volatile("" : "+v"(u[q].x), "+v"(u[q].y), "+v"(u[q].z), "+v"(u[q].w));
    }
};

// Backward: SUBS rows at a time per block, THREADS threads each.  A thread
// keeps its columns' weight and bias sums in registers over all its rows; the
// block adds its SUBS sums up in LDS and stores one partial, which
// norm_join_kernel adds up in block order.  The next rows are requested before
// the current ones are reduced, so that memory is read all the time: 16384 x
// 8192 bf16 (805 MB) 167 us with the join, 4.8 TB/s.
template <class T, int THREADS, int SUBS, int VPT, bool VEC>
__global__ __launch_bounds__(THREADS *SUBS) void norm_backward_kernel(NormArgs a) {
    constexpr int CE = kUnit<T>, W = THREADS / 64, COLS = THREADS * VPT * CE;
    __shared__ float2 sums[2][SUBS][W];
    __shared__ float total[SUBS > 1 ? COLS : 1];
    const int t = threadIdx.x % THREADS, sub = threadIdx.x / THREADS, wave = t >> 6;
    using Share = RowShare<T, THREADS, VPT, VEC>;
    float dw[VPT][CE], db[VPT][CE];
#pragma unroll
    for (int q = 0; q < VPT; ++q)
#pragma unroll
        for (int i = 0; i < CE; ++i) dw[q][i] = db[q][i] = 0.0f;
    struct Row {
        Share x, dy;
        float mean, rstd;
    } cur, next;
    Share w;
    if (a.w) w.load(a.w, a.N, t);
    const int step = a.blocks * SUBS;
    int row = blockIdx.x * SUBS + sub;
    auto request = [&](Row &to, int r) {
        to.x.load(a.x + (int64_t)r * a.ldx * sizeof(T), a.N, t);
        to.dy.load(a.dy + (int64_t)r * a.ldd * sizeof(T), a.N, t);
        to.mean = a.mean[r];
        to.rstd = a.rstd[r];
    };
    // past the row's end dy is zero, so x's value there does not count
    auto norm = [&](const Row &r, int q, int i) {
        return norm_col<T, THREADS, VEC>(q, i, t) < a.N ? (r.x.at(q, i) - r.mean) * r.rstd : 0.0f;
    };
    if (row < a.M) request(next, row);
    for (int base = blockIdx.x * SUBS, parity = 0; base < a.M; base += step, row += step, parity ^= 1) {
        const bool live = row < a.M;  // the same in a whole wave
        float s0 = 0.0f, s1 = 0.0f;
        if (live) {
            cur = next;
            if (row + step < a.M) request(next, row + step);
#pragma unroll
            for (int q = 0; q < VPT; ++q)
#pragma unroll
                for (int i = 0; i < CE; ++i) {
                    const float d = cur.dy.at(q, i), xh = norm(cur, q, i), g = a.w ? d * w.at(q, i) : d;
                    dw[q][i] += d * xh;
                    db[q][i] += d;
                    s0 += g;
                    s1 += g * xh;
                }
        }
        if (!a.y) continue;
        s0 = wave_sum(s0);
        s1 = wave_sum(s1);
        if constexpr (W > 1) {
            // the other parity's slots are written again only after the next barrier
            if ((t & 63) == 0) sums[parity][sub][wave] = make_float2(s0, s1);
            __syncthreads();
            s0 = s1 = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                s0 += sums[parity][sub][i].x;
                s1 += sums[parity][sub][i].y;
            }
        }
        if (live) {
            s0 /= (float)a.N;
            s1 /= (float)a.N;
            // xh and g are computed a second time: kept, they would take more
            // registers than there are
            cur.x.forget();
            cur.dy.forget();
            w.forget();
            char *out = a.y + (int64_t)row * a.ldy * sizeof(T);
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                float v[1][CE];
#pragma unroll
                for (int i = 0; i < CE; ++i) {
                    const float g = a.w ? cur.dy.at(q, i) * w.at(q, i) : cur.dy.at(q, i);
                    v[0][i] = cur.rstd * (g - s0 - norm(cur, q, i) * s1);
                }
                if constexpr (VEC) {
                    const int c = norm_col<T, THREADS, VEC>(q, 0, t);
                    if (c < a.N) store_unit<T>(out + (int64_t)c * sizeof(T), v[0]);
                } else {
#pragma unroll
                    for (int i = 0; i < CE; ++i) {
                        const int c = norm_col<T, THREADS, VEC>(q, i, t);
                        if (c < a.N) reinterpret_cast<T *>(out)[c] = from_f32<T>(v[0][i]);
                    }
                }
            }
        }
    }
    auto flush = [&](const float(&v)[VPT][CE], float *dst, char *out) {
#pragma unroll
        for (int s = 0; s < SUBS; ++s) {
            if (s > 0) __syncthreads();
            if (sub == s)
#pragma unroll
                for (int q = 0; q < VPT; ++q)
#pragma unroll
                    for (int i = 0; i < CE; ++i) {
                        const int c = norm_col<T, THREADS, VEC>(q, i, t);
                        float sum = v[q][i];
                        if constexpr (SUBS > 1)
                            if (s > 0) sum += total[c];
                        if (s + 1 == SUBS) {
                            if (c < a.N) {
                                if (a.blocks == 1) reinterpret_cast<T *>(out)[c] = from_f32<T>(sum);
                                else dst[c] = sum;
                            }
                        } else if constexpr (SUBS > 1) {
                            total[c] = sum;
                        }
                    }
        }
        if (SUBS > 1) __syncthreads();
    };
    float *pw = a.ws + (int64_t)blockIdx.x * a.N;
    if (a.dw) flush(dw, pw, a.dw);
    if (a.db) flush(db, pw + (int64_t)a.blocks * a.N, a.db);
}

// Rows too long for registers: dX by rows ...
template <class T>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(NormArgs a) {
    __shared__ float sh[16];
    const int row = blockIdx.x, t = threadIdx.x;
    const T *x = reinterpret_cast<const T *>(a.x) + (int64_t)row * a.ldx;
    const T *dy = reinterpret_cast<const T *>(a.dy) + (int64_t)row * a.ldd;
    const T *w = reinterpret_cast<const T *>(a.w);
    T *dx = reinterpret_cast<T *>(a.y) + (int64_t)row * a.ldy;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s0 = 0.0f, s1 = 0.0f;
    for (int c = t; c < a.N; c += 1024) {
        const float g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.0f);
        s0 += g;
        s1 += g * ((to_f32(x[c]) - mean) * rstd);
    }
    s0 = row_sum<1024>(s0, sh) / (float)a.N;
    s1 = row_sum<1024>(s1, sh) / (float)a.N;
    for (int c = t; c < a.N; c += 1024) {
        const float g = to_f32(dy[c]) * (w ? to_f32(w[c]) : 1.0f);
        dx[c] = from_f32<T>(rstd * (g - s0 - (to_f32(x[c]) - mean) * rstd * s1));
    }
}

// ... and the weight and bias sums by columns, before dX may overwrite dY or X.
template <class T>
__global__ __launch_bounds__(256) void norm_columns_kernel(NormArgs a, int col_blocks) {
    const int c = (blockIdx.x % col_blocks) * 256 + threadIdx.x, blk = blockIdx.x / col_blocks;
    if (c >= a.N) return;
    float dw = 0.0f, db = 0.0f;
    for (int row = blk; row < a.M; row += a.blocks) {
        const float d = to_f32(reinterpret_cast<const T *>(a.dy)[(int64_t)row * a.ldd + c]);
        const float x = to_f32(reinterpret_cast<const T *>(a.x)[(int64_t)row * a.ldx + c]);
        dw += d * ((x - a.mean[row]) * a.rstd[row]);
        db += d;
    }
    a.ws[(int64_t)blk * a.N + c] = dw;
    a.ws[(int64_t)(a.blocks + blk) * a.N + c] = db;
}

// dw and db from the blocks' partials: 64 columns x 16 ranges of blocks
template <class T>
__global__ __launch_bounds__(1024) void norm_join_kernel(NormArgs a, int col_blocks) {
    __shared__ float part[16][64];
    const int which = blockIdx.x / col_blocks;
    char *dst = which ? a.db : a.dw;
    if (!dst) return;  // whole blocks
    const int t = threadIdx.x & 63, s = threadIdx.x >> 6, c = (blockIdx.x % col_blocks) * 64 + t;
    const int per = (a.blocks + 15) / 16, to = (s + 1) * per < a.blocks ? (s + 1) * per : a.blocks;
    float v = 0.0f;
    if (c < a.N)
#pragma unroll 8
        for (int b = s * per; b < to; ++b) v += a.ws[((int64_t)which * a.blocks + b) * a.N + c];
    part[s][t] = v;
    __syncthreads();
    if (s > 0 || c >= a.N) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) v += part[i][t];
    reinterpret_cast<T *>(dst)[c] = from_f32<T>(v);
}

// ------------------------------------------------------------------ launchers

// The blocks of the copies; more than a grid can have: -1.
template <class T>
int64_t pack_grid(const PackArgs &a, PackGrid &g) {
    g = PackGrid{};
    int64_t blocks = 0;
    for (int i = 0; i < 3; ++i) {
        if (i < a.n) {
            g.unit_blocks[i] = (a.one[i].cols + 64 * kUnit<T> - 1) / (64 * kUnit<T>);
            blocks += ((int64_t)a.one[i].count * a.one[i].rows + 3) / 4 * g.unit_blocks[i];
            if (blocks > 0x7FFFFFFF) return -1;
        }
        g.end[i] = (int)blocks;
    }
    return blocks;
}

template <class T>
hipError_t pack(const PackArgs &a, hipStream_t s) {
    PackGrid g;
    const int64_t blocks = pack_grid<T>(a, g);
    if (blocks < 0) return hipErrorInvalidValue;
    hipLaunchKernelGGL(HIP_KERNEL_NAME(pack_kernel<T>), grid_of(blocks, 256), dim3(256), 0, s, a, g);
    return hipGetLastError();
}

template <class T>
hipError_t join(const GemmArgs &g, hipStream_t s) {
    const int unit = g.vec ? kUnit<T> : 1;
    const int per_row = (g.N + 256 * unit - 1) / (256 * unit);
    const dim3 grid = grid_of((int64_t)g.M * (g.mode == kGroupSum ? g.groups : 1) * per_row, 256);
    if (g.vec) hipLaunchKernelGGL(HIP_KERNEL_NAME(join_kernel<T, kUnit<T>>), grid, dim3(256), 0, s, g, per_row);
    else hipLaunchKernelGGL(HIP_KERNEL_NAME(join_kernel<T, 1>), grid, dim3(256), 0, s, g, per_row);
    return hipGetLastError();
}

template <class T>
hipError_t grad(const GradArgs &a, const PackArgs &packs, hipStream_t s) {
    const int cols = (a.N + 32 * kUnit<T> - 1) / (32 * kUnit<T>);
    PackGrid g;
    const int64_t blocks = (int64_t)a.tiles * cols, more = pack_grid<T>(packs, g);
    if (more < 0 || blocks + more > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (blocks + more > 0) {
        const dim3 grid = grid_of(blocks + more, 256);
        auto launch = [&](auto ACT) {
            constexpr int act = decltype(ACT)::value;
            if (a.vec)
                hipLaunchKernelGGL(HIP_KERNEL_NAME(grad_kernel<T, act, true>), grid, dim3(256), 0, s, a, cols, (int)blocks, packs, g);
            else
                hipLaunchKernelGGL(HIP_KERNEL_NAME(grad_kernel<T, act, false>), grid, dim3(256), 0, s, a, cols, (int)blocks, packs, g);
        };
        if (a.act == CP_ACT_NONE) launch(std::integral_constant<int, CP_ACT_NONE>{});
        else if (a.act == CP_ACT_GELU_TANH) launch(std::integral_constant<int, CP_ACT_GELU_TANH>{});
        else if (a.act == CP_ACT_SILU) launch(std::integral_constant<int, CP_ACT_SILU>{});
        else launch(std::integral_constant<int, CP_ACT_RELU>{});
    }
    return hipGetLastError();
}

template <class T>
hipError_t grad_join(const GradArgs &a, hipStream_t s) {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(grad_join_kernel<T>), grid_of(grad_join_blocks(a), 256), dim3(256), 0, s, a);
    return hipGetLastError();
}

// f(rows, blocks) for as many launches of `rows` rows to a block of `threads`
// as all rows take: one, unless a grid cannot hold that many threads.
template <class T, class F>
hipError_t by_rows(const NormArgs &a, int rows, int threads, F &&f) {
    const int64_t most = max_blocks(threads) * rows;
    for (int64_t row = 0; row < a.M; row += most) {
        NormArgs part = a;
        part.M = (int)(a.M - row < most ? a.M - row : most);
        if (a.x) part.x += row * a.ldx * (int64_t)sizeof(T);
        if (a.dy) part.dy += row * a.ldd * (int64_t)sizeof(T);
        if (a.y) part.y += row * a.ldy * (int64_t)sizeof(T);
        if (a.mean) part.mean += row;
        if (a.rstd) part.rstd += row;
        f(part, dim3((unsigned)((part.M + rows - 1) / rows)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T, int THREADS, int VPT, Access A>
hipError_t norm_rows(const NormArgs &a, hipStream_t s) {
    constexpr int BLOCK = THREADS < 256 ? 256 : THREADS;
    return by_rows<T>(a, BLOCK / THREADS, BLOCK, [&](const NormArgs &part, dim3 grid) {
        hipLaunchKernelGGL(HIP_KERNEL_NAME(norm_kernel<T, THREADS, VPT, A>), grid, dim3(BLOCK), 0, s, part);
    });
}

template <class T, Access A>
hipError_t norm_widths(const NormArgs &a, hipStream_t s) {
#define CPO_NORM(THREADS, VPT) \
    if (a.N <= THREADS * VPT * kUnit<T>) return norm_rows<T, THREADS, VPT, A>(a, s);
    CPO_NORM(64, 1)
    CPO_NORM(64, 2)
    CPO_NORM(256, 1)
    CPO_NORM(256, 2)
    CPO_NORM(256, 4)
    CPO_NORM(512, 3)
    CPO_NORM(512, 4)
    CPO_NORM(1024, 4)
#undef CPO_NORM
    return by_rows<T>(a, 1, 1024, [&](const NormArgs &part, dim3 grid) {
        hipLaunchKernelGGL(HIP_KERNEL_NAME(norm_long_kernel<T>), grid, dim3(1024), 0, s, part);
    });
}

template <class T>
hipError_t norm(const NormArgs &a, hipStream_t s) {
    if (a.vec) return norm_widths<T, kUnits>(a, s);
    if constexpr (sizeof(T) == 2)
        // a unit has to fit the row; narrower ones are a wave's single elements (as
        // rows too long for registers, a block each, 1048576 x 4 took 3279 us, 204 so)
        return a.N < kUnit<T> ? norm_rows<T, 64, 1, kElements>(a, s) : norm_widths<T, kShifted>(a, s);
    else
        return norm_widths<T, kElements>(a, s);
}

template <class T, bool VEC>
hipError_t norm_backward(const NormArgs &a, hipStream_t s) {
    // Threads of a row, rows at a time per block, units per thread: one block
    // per CU leaves the fewest partials, and the rows at a time make up the
    // waves that keep memory busy, as far as the registers go.
#define CPO_LAUNCH(THREADS, SUBS, VPT)                                                                              \
    if (a.N <= THREADS * VPT * kUnit<T>) {                                                                          \
        hipLaunchKernelGGL(HIP_KERNEL_NAME(norm_backward_kernel<T, THREADS, SUBS, VPT, VEC>), dim3((unsigned)a.blocks), \
                           dim3(THREADS * SUBS), 0, s, a);                                                          \
        return hipGetLastError();                                                                                   \
    }
    CPO_LAUNCH(64, 16, 1)
    CPO_LAUNCH(128, 8, 1)
    CPO_LAUNCH(256, 4, 1)
    if constexpr (VEC || sizeof(T) == 4) {
        CPO_LAUNCH(256, 4, 2)
        CPO_LAUNCH(512, 2, 2)
        CPO_LAUNCH(1024, 1, 2)
    } else {  // single bf16 elements take a register each
        CPO_LAUNCH(512, 2, 1)
        CPO_LAUNCH(1024, 1, 1)
    }
#undef CPO_LAUNCH
    const int cb = (a.N + 255) / 256;
    if (a.dw || a.db)
        hipLaunchKernelGGL(HIP_KERNEL_NAME(norm_columns_kernel<T>), dim3((unsigned)(a.blocks * cb)), dim3(256), 0, s, a, cb);
    if (a.y)
        return by_rows<T>(a, 1, 1024, [&](const NormArgs &part, dim3 grid) {
            hipLaunchKernelGGL(HIP_KERNEL_NAME(norm_backward_long_kernel<T>), grid, dim3(1024), 0, s, part);
        });
    return hipGetLastError();
}

template <class T>
hipError_t norm_backward_all(const NormArgs &a, hipStream_t s) {
    if (a.M > 0) {
        const hipError_t e = a.vec ? norm_backward<T, true>(a, s) : norm_backward<T, false>(a, s);
        if (e != hipSuccess) return e;
    }
    if ((a.dw || a.db) && a.blocks != 1) {
        const int cb = (a.N + 63) / 64;
        hipLaunchKernelGGL(HIP_KERNEL_NAME(norm_join_kernel<T>), dim3((unsigned)(2 * cb)), dim3(1024), 0, s, a, cb);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_pack(int dtype, const PackArgs &a, hipStream_t s) {
    return dtype == CP_BF16 ? pack<__bf16>(a, s) : pack<float>(a, s);
}

hipError_t launch_join(int dtype, const GemmArgs &g, hipStream_t s) {
    return dtype == CP_BF16 ? join<__bf16>(g, s) : join<float>(g, s);
}

hipError_t launch_grad(int dtype, const GradArgs &a, const PackArgs &packs, hipStream_t s) {
    return dtype == CP_BF16 ? grad<__bf16>(a, packs, s) : grad<float>(a, packs, s);
}

hipError_t launch_grad_join(int dtype, const GradArgs &a, hipStream_t s) {
    return dtype == CP_BF16 ? grad_join<__bf16>(a, s) : grad_join<float>(a, s);
}

hipError_t launch_norm(int dtype, const NormArgs &a, hipStream_t s) {
    return dtype == CP_BF16 ? norm<__bf16>(a, s) : norm<float>(a, s);
}

// One block, which stores the sums itself, where two launches would take longer
// than its rows; otherwise at least two.  A pass over 16 narrow rows takes 1.6
// us: 32 x 250 in one block 10.5 us; 64 x 26 in one 12.4, 71 x 26 in 71 11.3.
int norm_backward_blocks(int64_t M, int64_t N) {
    if (M == 0) return 0;
    if (M * N <= kNormOneBlock && M <= 32) return 1;
    return (int)(M < 2 ? 2 : M < 256 ? M : 256);
}

hipError_t launch_norm_backward(int dtype, const NormArgs &a, hipStream_t s) {
    return dtype == CP_BF16 ? norm_backward_all<__bf16>(a, s) : norm_backward_all<float>(a, s);
}

}  // namespace cpo
