// cp_ops_int4.hip -- linear layers with 4-bit weights, w_kn = s_gn (q_kn - z_gn).  For
// a few rows at a time (decoding) bound by reading the codes, a quarter of the bf16
// weight; for more rows by unpacking and scaling, which the vector unit does beside
// the matrix cores.
//
// The matrix cores multiply x with the codes as bf16, exactly: a code's four bits
// in bits 3 .. 6 of a bf16 pattern 0x4180 make it 16 + q, two codes with one shift
// and one and-or.  A product with ones gives sum x, and per group
//     s_n (sum x (16 + q) - (16 + z_n) sum x)
// joins the fp32 accumulator: of two sums up to four times as large as their difference
// can be, whose roundings, some 2^-24 of them, only a bf16 result near zero shows.
// fp32 rows run as three bf16 parts that add up to them exactly, and q - z is the other
// operand, as exact as 16 + q and more work to unpack: a result is as good as that of the
// weight in fp32 (K 4096, x of one sign: off by 1.3e-7 of its norm, by way of the
// two sums 1.8e-6), and weights of zero add nothing.  The codes lie in memory as the
// instructions take them (Int4Layout), so a wave reads its operand with whole 16-byte
// loads and no LDS.
#include "cp_ops_experts.h"
#include "cp_ops_units.h"

namespace cpo {

namespace {

// The constants in registers: an instruction with both takes them from nowhere else.
struct Spread {
    uint32_t mask = 0x00780078u, base = 0x41804180u;
    __device__ __forceinline__ Spread() { asm("" : "+v"(mask), "+v"(base)); }
    __device__ __forceinline__ bf16x8_t operator()(uint32_t w) const {
        union {
            uint32_t u[4];
            bf16x8_t v;
        } r;
        r.u[0] = (w & mask) | base;
        r.u[1] = ((w >> 4) & mask) | base;
        r.u[2] = ((w >> 8) & mask) | base;
        r.u[3] = (__builtin_amdgcn_alignbit(w, w, 12) & mask) | base;
        return r.v;
    }
};
// q - z, for the fp32 rows.  Four codes at a time in bytes: 0x80 + q - z borrows nothing from
// its neighbours, and without the 0x80 is signed.  20 instructions to eight codes, by way of
// fp32 differences of 16 + q 27; 16 + q itself is 7, which many experts of few rows feel
// (64 rows over 32 experts of 1024 x 4096 18.9 us, so 23.9).
__device__ __forceinline__ uint32_t centre_of(float zero) {  // zero: 16 + z
    return 0x80808080u - (uint32_t)((int)zero - 16) * 0x01010101u;
}
__device__ __forceinline__ bf16x8_t centred(uint32_t w, uint32_t centre) {
    auto bytes = [&](uint32_t q) { return ((q & 0x0F0F0F0Fu) + centre) ^ 0x80808080u; };
    auto pair = [](uint32_t d, int i) {  // bytes i and i + 2: whole numbers of up to 5 bits, the upper halves of their fp32
        const float lo = (float)(int)(int8_t)(d >> (8 * i)), hi = (float)(int)(int8_t)(d >> (8 * i + 16));
        return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
    };
    const uint32_t a = bytes(w >> 3), b = bytes(__builtin_amdgcn_alignbit(w, w, 7));
    union {
        uint32_t u[4];
        bf16x8_t v;
    } r;
    r.u[0] = pair(a, 0);
    r.u[1] = pair(b, 0);
    r.u[2] = pair(a, 1);
    r.u[3] = pair(b, 1);
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

// A group's scale and zero point for one column, as packed.
template <class T>
struct Meta;
template <>
struct Meta<__bf16> {
    uint32_t v;  // 16 + z over the scale, both bf16
    __device__ __forceinline__ float scale() const { return __builtin_bit_cast(float, v << 16); }
    __device__ __forceinline__ float zero() const { return __builtin_bit_cast(float, v & 0xFFFF0000u); }
    __device__ __forceinline__ void hold() { asm volatile("" : "+v"(v)); }
};
template <>
struct Meta<float> {
    float s, z;
    __device__ __forceinline__ float scale() const { return s; }
    __device__ __forceinline__ float zero() const { return z; }
    __device__ __forceinline__ void hold() { asm volatile("" : "+v"(s), "+v"(z)); }
};

// SG matrix instructions, 32 k each, to a group, as far as it lies in a tile.
template <int SG>
__device__ __forceinline__ int first_group(const Int4Args &g, int kb) {
    return SG < 4 ? kb * (4 / SG) : (g.group == kInt4Depth ? kb : kb / (g.group / kInt4Depth));
}
template <class T, int SG>
struct Tile {  // of codes, and its groups' scales
    static constexpr int NG = 4 / SG;
    uint4 w;
    Meta<T> m[NG];
    // gr: the tile's first group
    __device__ __forceinline__ void load(const Int4Args &g, const char *codes, const char *meta, int tile, int kb, int gr) {
        const int lane = threadIdx.x & 63;
        w = *reinterpret_cast<const uint4 *>(codes + ((int64_t)tile * g.kblocks + kb) * kInt4TileBytes + lane * 16);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int at = gr + i < g.ngroups ? gr + i : g.ngroups - 1;  // (past K: x is zero)
            m[i] = reinterpret_cast<const Meta<T> *>(meta)[((int64_t)tile * g.ngroups + at) * kInt4Columns + (lane & 15)];
        }
    }
    // Keeps what is computed from the tile behind this point: unpacked early it takes
    // several times the registers.
    __device__ __forceinline__ void hold() {
        asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
#pragma unroll
        for (int i = 0; i < NG; ++i) m[i].hold();
    }
    __device__ __forceinline__ uint32_t step(int s) const { return s == 0 ? w.x : s == 1 ? w.y : s == 2 ? w.z : w.w; }
};

// The rows of a block: a tile of `bm` rows, of one expert if there are experts.
struct BlockRows {
    int row0, end, expert;
    bool none;  // rows without an expert
};
__device__ __forceinline__ bool block_rows(const Int4Args &g, int bm, int rt, BlockRows &r) {
    r = {rt * bm, g.M, 0, false};
    if (g.experts) {
        GroupScan s;
        if (rt >= count_tiles(g.off, g.experts, g.M, bm, s)) return false;
        const RowTile t = find_tile(g.off, g.experts, g.M, bm, rt, s);
        r = {t.row0 + (rt - t.before) * bm, t.end, t.expert < g.experts ? t.expert : 0, t.expert >= g.experts};
    }
    return true;
}

template <class T>
__device__ __forceinline__ void finish_int4(const Int4Args &g, const BlockRows &b, int row, int col, float v) {
    if (row >= b.end || col >= g.N) return;
    if (g.bias) v += to_f32(reinterpret_cast<const T *>(g.bias)[(int64_t)b.expert * g.N + col]);
    v = b.none ? 0.0f : act_apply(v, g.act);
    if (g.res) v += to_f32(reinterpret_cast<const T *>(g.res)[(int64_t)row * g.ldr + col]);
    reinterpret_cast<T *>(g.y)[(int64_t)row * g.ldy + col] = from_f32<T>(v);
}

// Where a block writes: the result, or its part of the contraction's partial sums.
template <class T>
__device__ __forceinline__ void put_int4(const Int4Args &g, const BlockRows &b, int chunk, int row, int col, float v) {
    if (g.chunks == 1) return finish_int4<T>(g, b, row, col, v);
    if (row < b.end && col < g.N) g.ws[((int64_t)chunk * g.M + row) * g.ldws + col] = v;
}

template <class T>
__device__ __forceinline__ void put_int4_unit(const Int4Args &g, const BlockRows &b, int chunk, int row, int col, const float *v) {
    constexpr int CE = kUnit<T>;
    if (row >= b.end || col >= g.N) return;
    if (g.chunks > 1) {  // (rows of whole units: ldws)
        float *p = g.ws + ((int64_t)chunk * g.M + row) * g.ldws + col;
#pragma unroll
        for (int i = 0; i < CE; ++i) p[i] = v[i];
        return;
    }
    float f[CE];
#pragma unroll
    for (int i = 0; i < CE; ++i) f[i] = v[i];
    const int left = g.N - col;
    if (g.bias) {
        float t[CE];
        unpack_unit<T>(load_partial<T>(g.bias + ((int64_t)b.expert * g.N + col) * (int64_t)sizeof(T), left), t);
#pragma unroll
        for (int i = 0; i < CE; ++i) f[i] += t[i];
    }
#pragma unroll
    for (int i = 0; i < CE; ++i) f[i] = b.none ? 0.0f : act_apply(f[i], g.act);
    if (g.res) {
        float t[CE];
        unpack_unit<T>(load_partial<T>(g.res + ((int64_t)row * g.ldr + col) * (int64_t)sizeof(T), left), t);
#pragma unroll
        for (int i = 0; i < CE; ++i) f[i] += t[i];
    }
    store_partial<T>(g.y + ((int64_t)row * g.ldy + col) * (int64_t)sizeof(T), pack_unit<T>(f), left);
}

// Up to 16 rows (of an expert): a chunk of the contraction to a block, every W-th tile
// of it to each of its W waves, column tile after column tile.  A wave's part of x
// stays in its registers for all of them, so that the loop reads codes and scales
// alone, D column tiles ahead.  The loop has no branch around a load: the compiler
// could not tell how many are in flight behind it and would wait for all.  For the
// same reason the sums of a column tile go to LDS and are finished, with what bias and
// residual have to be read for it, some tiles at a time.
// 1 x 4096 x 4096 bf16 7.2 us (a launch and one trip to memory; 8.9 MB), 13 x 8192 x
// 28672 30.7 us (125 MB, 4.1 TB/s), 32 rows over 8 experts of 4096 x 4096 16.6 us (62 MB of
// the seven in use, 3.7 TB/s); half of the wave cycles wait for memory.
constexpr int kInt4Flush = 8;
template <class T, int W, int XK, int D, int SG>
__global__ __launch_bounds__(W * 64) void int4_stream_kernel(Int4Args g) {
    constexpr int XP = sizeof(T) == 2 ? 1 : 3, NG = 4 / SG;
    __shared__ f32x4_t red[2][W][64];
    __shared__ float done[kInt4Flush][256];
    __shared__ f32x4_t sums[XP == 1 ? W : 1][XK * NG][4];  // of x over the groups
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // An XCD has a range of the columns, for all row tiles: of those the last may not be
    // there, and would leave it idle were they all its own.
    const int per = g.ntn % 8 ? g.ntn : g.ntn / 8, b = g.ntn % 8 ? blockIdx.x : blockIdx.x / 8;
    const int cb = (g.ntn % 8 ? 0 : (blockIdx.x & 7) * per) + b % per, part = b / per, rt = part / g.chunks, chunk = part % g.chunks;
    BlockRows br;
    if (!block_rows(g, 16, rt, br)) return;
    const int t0 = (int)((int64_t)cb * g.ntiles / g.ntn), t1 = (int)((int64_t)(cb + 1) * g.ntiles / g.ntn), n = t1 - t0;
    if (br.none) {
        for (int i = tid; i < 16 * 16 * n; i += W * 64)
            put_int4<T>(g, br, chunk, br.row0 + i / (16 * n), t0 * 16 + i % (16 * n), 0.0f);
        return;
    }
    const char *codes = g.codes + (int64_t)br.expert * g.sc, *meta = g.meta + (int64_t)br.expert * g.sm;
    const Spread spread;

    // tiles of the contraction, past its end the last again, with x of zero
    const int kb_end = (chunk + 1) * g.kper < g.kblocks ? (chunk + 1) * g.kper : g.kblocks;
    int kb[XK], gr[XK];
    Tile<T, SG> w[D][XK];
#pragma unroll
    for (int i = 0; i < XK; ++i) {
        const int at = chunk * g.kper + i * W + wave;
        kb[i] = at < kb_end ? at : kb_end - 1;
        gr[i] = first_group<SG>(g, kb[i]);
    }
    auto load_one = [&](int d, int i, int t) { w[d][i].load(g, codes, meta, t0 + t, kb[i], gr[i]); };
    auto load = [&](int d, int t) {
#pragma unroll
        for (int i = 0; i < XK; ++i) load_one(d, i, t);
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < n) load(d, d);
    Row8<T> xr[XK][4];
    {
        const int row = br.row0 + (lane & 15) < br.end ? br.row0 + (lane & 15) : br.row0;  // (others' results are not used)
#pragma unroll
        for (int i = 0; i < XK; ++i) {
            const bool in = chunk * g.kper + i * W + wave < kb_end;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = kb[i] * kInt4Depth + s * 32 + (lane >> 4) * 8;
                if (in && k < g.K) xr[i][s].load(g.x + ((int64_t)row * g.ldx + k) * (int64_t)sizeof(T), g.K - k);
                else xr[i][s].zero();
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (XP == 1)
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    f32x4_t xs{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = j * SG; s < j * SG + SG; ++s) {
                        bf16x8_t x[XP];
                        parts(xr[i][s], x);
                        xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[0], ones_bf16(), xs, 0, 0, 0);
                    }
                    if ((lane & 15) == 0) sums[wave][i * NG + j][lane >> 4] = xs;
                }
        }
        if constexpr (XP == 1) __syncthreads();
    }
    auto column = [&](int d, int t) {
        f32x4_t acc{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < XK; ++i)
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const float sc = w[d][i].m[j].scale(), zero = w[d][i].m[j].zero();
                const uint32_t centre = XP > 1 ? centre_of(zero) : 0;
                f32x4_t xs{0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (XP == 1) xs = sums[wave][i * NG + j][lane >> 4];
                f32x4_t p{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = j * SG; s < j * SG + SG; ++s) {
                    const bf16x8_t c = XP == 1 ? spread(w[d][i].step(s)) : centred(w[d][i].step(s), centre);
                    bf16x8_t x[XP];
                    parts(xr[i][s], x);
#pragma unroll
                    for (int q = 0; q < XP; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[q], c, p, 0, 0, 0);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] = fmaf(sc, XP == 1 ? fmaf(-zero, xs[r], p[r]) : p[r], acc[r]);
                __builtin_amdgcn_sched_barrier(0);  // (one group's registers at a time)
                if (D == 1 && j == NG - 1) {  // the next tile's part as soon as its registers are free
                    asm volatile("" : "+v"(acc));
                    load_one(0, i, t + 1 < n ? t + 1 : t);
                }
            }
        // (one barrier to a tile: whoever writes a buffer again has passed the next one,
        // behind the sums that read it)
        red[t & 1][wave][lane] = acc;
    };
    auto sum = [&](int t) {
        __syncthreads();
        if (tid < 256) {  // element tid % 4 of lane tid / 4
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) v += reinterpret_cast<const float *>(&red[t & 1][i][0])[tid];
            done[t % kInt4Flush][tid] = v;
        }
        if ((t + 1) % kInt4Flush && t + 1 < n) return;
        __syncthreads();
        const int f0 = t / kInt4Flush * kInt4Flush, cols = (t + 1 - f0) * 16;
        for (int i = tid; i < 16 * cols; i += W * 64) {
            const int r = i / cols, c = i % cols;
            put_int4<T>(g, br, chunk, br.row0 + r, (t0 + f0) * 16 + c, done[c >> 4][((r >> 2) * 16 + (c & 15)) * 4 + (r & 3)]);
        }
        __syncthreads();
    };
    int t = 0;
    if constexpr (D == 1) {
        for (; t < n; ++t) {
            column(0, t);
            sum(t);
        }
        return;
    }
    for (; t + 2 * D <= n; t += D)
#pragma unroll
        for (int d = 0; d < D; ++d) {
            column(d, t + d);
            load(d, t + D + d);
            sum(t + d);
        }
    for (; t < n; t += D)  // the last, up to 2 D - 1 of them
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (t + d >= n) break;
            column(d, t + d);
            if (t + D + d < n) load(d, t + D + d);
            sum(t + d);
        }
}

// The sum of each 2 neighbouring lanes' values, in both (N = 1: the value).
template <int N>
__device__ __forceinline__ float sum_neighbours(float v) {
    static_assert(N == 1 || N == 2, "pieces of a group");
    if constexpr (N == 2)  // quad_perm 1 0 3 2
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xf, 0xf, true));
    return v;
}

// More rows: MT x 16 to a block, staged through LDS in the order the matrix
// instructions take them, while the codes go to the registers of the wave that needs
// them: wave wn of four has NT column tiles.  WK such quartets take a part of the
// contraction each.  A wave stages 32 or 64 k of 16 rows at a time and adds them up for
// each row; where the pieces do not go round, some are staged twice, alike.  x and
// codes are requested two tiles of the contraction ahead, x first: loads come back in
// order, and x is waited for first, to be staged one tile ahead.  (No branch around a
// load, as above: what lies past K comes last.)
// 300 x 8192 x 8191, groups of 64, bf16: 82 us, 490 TFLOP/s.  A wave has 46 matrix and
// 248 vector instructions to 128 k, 20 and 26 us of a SIMD's time for its two waves; the
// matrix cores are busy for 21% of the time, LDS for 28%.  The rest is waiting: one block
// fits a CU, and its waves meet at a barrier every 128 k.
template <class T, int MT, int NT, int WK, int SG>
__global__ __launch_bounds__(WK * 256) void int4_rows_kernel(Int4Args g) {
    constexpr int XP = sizeof(T) == 2 ? 1 : 3, NG = 4 / SG;
    constexpr int UF = SG < 2 ? SG : 2, UH = 4 / UF, PU = (MT * UH + 3) / 4;  // a unit's pieces of 32 k, units to a row tile, to a wave
    constexpr int CE = kUnit<T>, LD = NT * 16 + 4;  // columns and stride of a wave's results in LDS
    constexpr int kBuf = XP * 4 * MT * 1024, kJoin = (WK - 1) * MT * NT * 4096, kOut = 4 * MT * 16 * LD * 4;
    constexpr int kMost = kJoin > kOut ? kJoin : kOut;
    __shared__ __attribute__((aligned(16))) char stage[WK * 2 * kBuf > kMost ? WK * 2 * kBuf : kMost];
    __shared__ f32x4_t sums[XP == 1 ? WK : 1][2][UH][MT][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave & 3, wk = wave >> 2, n16 = lane & 15, quad = lane >> 4;
    const int b = xcd_remap(blockIdx.x, gridDim.x), part = b / g.ntm, rt = b % g.ntm, ct = part / g.chunks, chunk = part % g.chunks;
    BlockRows br;
    if (!block_rows(g, 16 * MT, rt, br)) return;
    const char *codes = g.codes + (int64_t)br.expert * g.sc, *meta = g.meta + (int64_t)br.expert * g.sm;
    const Spread spread;
    const int tile0 = (ct * 4 + wn) * NT;
    const int kb_end = br.none ? 0 : ((chunk + 1) * g.kper < g.kblocks ? (chunk + 1) * g.kper : g.kblocks);
    const int whole = g.K / kInt4Depth < kb_end ? g.K / kInt4Depth : kb_end;  // tiles without an end of K in them
    const int first = chunk * g.kper, per = whole > first ? (whole - first) / WK : 0, kb0 = first + wk * per;
    const char *xp[PU];
    int um[PU], uh[PU];
#pragma unroll
    for (int i = 0; i < PU; ++i) {
        const int u = wn + 4 * i < MT * UH ? wn + 4 * i : MT * UH - 1;
        um[i] = u / UH;
        uh[i] = u % UH;
        const int row = br.row0 + um[i] * 16 + n16;  // (rows past the end: their results are not used)
        xp[i] = g.x + ((int64_t)(row < br.end ? row : br.row0) * g.ldx + uh[i] * UF * 32 + quad * 8) * (int64_t)sizeof(T);
    }

    Row8<T> xr[PU][UF];
    Tile<T, SG> c[3][NT];  // in turn: copying one to the next would wait for it
    auto load_codes = [&](Tile<T, SG> (&to)[NT], int kb) {
        const int gr = first_group<SG>(g, kb);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            to[n].load(g, codes, meta, tile0 + n < g.ntiles ? tile0 + n : g.ntiles - 1, kb, gr);
    };
    auto at = [&](int it) { return kb0 + (it < per ? it : per - 1); };
    auto load_x = [&](int it) {
        const int64_t k = (int64_t)at(it) * kInt4Depth * (int64_t)sizeof(T);
#pragma unroll
        for (int u = 0; u < PU; ++u)
#pragma unroll
            for (int f = 0; f < UF; ++f)
#pragma unroll
                for (int i = 0; i < Row8<T>::kUnits; ++i)
                    __builtin_memcpy(&xr[u][f].u[i], xp[u] + k + f * 32 * sizeof(T) + i * 16, 16);
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int u = 0; u < PU; ++u) {
            f32x4_t xs{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int f = 0; f < UF; ++f) {
                bf16x8_t x[XP];
                parts(xr[u][f], x);
#pragma unroll
                for (int q = 0; q < XP; ++q) {
                    if constexpr (XP == 1) xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[q], ones_bf16(), xs, 0, 0, 0);
                    *reinterpret_cast<bf16x8_t *>(stage + (wk * 2 + buf) * kBuf + ((q * 4 + uh[u] * UF + f) * MT + um[u]) * 1024 +
                                                  lane * 16) = x[q];
                }
            }
            if constexpr (XP == 1)
                if (n16 == 0) sums[wk][buf][uh[u]][um[u]][quad] = xs;
        }
    };
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](Tile<T, SG> (&c0)[NT], int buf) {
#pragma unroll
        for (int n = 0; n < NT; ++n) c0[n].hold();
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            bf16x8_t w[SG][NT];
            uint32_t centre[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) centre[n] = XP > 1 ? centre_of(c0[n].m[j].zero()) : 0;
#pragma unroll
            for (int s = 0; s < SG; ++s)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    w[s][n] = XP == 1 ? spread(c0[n].step(j * SG + s)) : centred(c0[n].step(j * SG + s), centre[n]);
            // a row tile's operands are read while the one before is multiplied and the one
            // before that scaled
            bf16x8_t x[2][SG][XP];
            f32x4_t xs[2], ys[2];
            auto fetch = [&](int m) {
                if constexpr (XP == 1) xs[m & 1] = sums[wk][buf][SG > UF ? n16 % (SG / UF) : j][m][quad];
#pragma unroll
                for (int s = 0; s < SG; ++s)
#pragma unroll
                    for (int q = 0; q < XP; ++q)
                        x[m & 1][s][q] = *reinterpret_cast<const bf16x8_t *>(
                            stage + (wk * 2 + buf) * kBuf + ((q * 4 + j * SG + s) * MT + m) * 1024 + lane * 16);
            };
            f32x4_t p[2][NT];
            auto scale = [&](int m) {
                if constexpr (XP == 1)
#pragma unroll
                    for (int r = 0; r < 4; ++r) ys[m & 1][r] = sum_neighbours<SG / UF>(ys[m & 1][r]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float sc = c0[n].m[j].scale(), zero = c0[n].m[j].zero();
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float v = XP == 1 ? fmaf(-zero, ys[m & 1][r], p[m & 1][n][r]) : p[m & 1][n][r];
                        acc[m][n][r] = fmaf(sc, v, acc[m][n][r]);
                    }
                }
            };
            fetch(0);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (m + 1 < MT) fetch(m + 1);
                if constexpr (XP == 1) ys[m & 1] = xs[m & 1];
#pragma unroll
                for (int n = 0; n < NT; ++n) p[m & 1][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < SG; ++s)
#pragma unroll
                    for (int q = 0; q < XP; ++q)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            p[m & 1][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m & 1][s][q], w[s][n], p[m & 1][n], 0, 0, 0);
                if (m > 0) scale(m - 1);
            }
            scale(MT - 1);
            // (here and not where the sums are next used, blocks later, with all that they are made of)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) asm volatile("" : "+v"(acc[m][n]));
        }
    };
    auto step = [&](auto i, int it) {
        put(~it & 1);
        load_x(it + 2);
        load_codes(c[(i() + 2) % 3], at(it + 2));
        __builtin_amdgcn_sched_barrier(0);
        multiply(c[i()], it & 1);
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);  // (the next step's codes stay packed until then)
    };
    using std::integral_constant;
    if (per) {
        load_x(0);
        load_codes(c[0], at(0));
        put(0);
        load_x(1);
        load_codes(c[1], at(1));
        __syncthreads();
        int it = 0;
        for (; it + 3 <= per; it += 3) {
            step(integral_constant<int, 0>(), it);
            step(integral_constant<int, 1>(), it + 1);
            step(integral_constant<int, 2>(), it + 2);
        }
        if (it < per) step(integral_constant<int, 0>(), it);
        if (it + 1 < per) step(integral_constant<int, 1>(), it + 1);
    }
    if (first + per * WK < kb_end) {  // what the quartets have not shared out evenly, and a tile that K ends in: one each
        const int kb = first + per * WK + wk;
        load_codes(c[0], kb < kb_end ? kb : kb_end - 1);
#pragma unroll
        for (int u = 0; u < PU; ++u)
#pragma unroll
            for (int f = 0; f < UF; ++f) {
                const int k = kb * kInt4Depth + (uh[u] * UF + f) * 32 + quad * 8;
                if (kb < kb_end && k < g.K) xr[u][f].load(xp[u] + ((int64_t)kb * kInt4Depth + f * 32) * (int64_t)sizeof(T), g.K - k);
                else xr[u][f].zero();
            }
        put(per & 1);
        __syncthreads();
        multiply(c[0], per & 1);
    }
    __syncthreads();
    if constexpr (WK > 1) {
        f32x4_t *join = reinterpret_cast<f32x4_t *>(stage);
        if (wk > 0)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) join[(((wk - 1) * 4 + wn) * MT * NT + m * NT + n) * 64 + lane] = acc[m][n];
        __syncthreads();
        if (wk == 0)
#pragma unroll
            for (int w = 1; w < WK; ++w)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[m][n] += join[(((w - 1) * 4 + wn) * MT * NT + m * NT + n) * 64 + lane];
        __syncthreads();
        if (wk > 0) return;
    }
    // out by way of LDS, each wave its own part of it, in whole units of a row
    float *tile = reinterpret_cast<float *>(stage) + wn * MT * 16 * LD;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) tile[(m * 16 + quad * 4 + r) * LD + n * 16 + n16] = acc[m][n][r];
    settle_lds();
    for (int i = lane; i < MT * 16 * NT * 16 / CE; i += 64) {
        const int r = i / (NT * 16 / CE), c0 = i % (NT * 16 / CE) * CE;
        put_int4_unit<T>(g, br, chunk, br.row0 + r, tile0 * 16 + c0, tile + r * LD + c0);
    }
}

// ------------------------------------------------- packing and quantisation

// A thread per four columns and the four words that a lane of the layers' waves takes of
// each: it reads the columns' codes together and writes 64 bytes.  8192 x 28672 85 us with
// the scales, 4.2 TB/s.
__global__ __launch_bounds__(256) void int4_pack_codes_kernel(Int4PackArgs a) {
    constexpr int C = 4, kSets = kInt4Columns / C;
    const int64_t cols = (int64_t)a.ntiles * kSets, per = cols * 4 * a.kblocks, all = per * a.E;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        // neighbours in a wave take neighbouring columns
        const int64_t e = i / per, c = i % per % cols, kq = i % per / cols, kb = kq / 4, n = c * C;
        const int quad = (int)(kq % 4);
        uint32_t v[C][4] = {};
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t k = kb * kInt4Depth + s * 32 + quad * 8 + j;
                const uint8_t *q = a.q + (e * a.K + k) * a.N + n;
                uint32_t w = 0;
                if (k < a.K) {
                    if (n + C <= a.N) {
                        __builtin_memcpy(&w, q, sizeof w);
                    } else {
#pragma unroll
                        for (int u = 0; u < C; ++u)
                            if (n + u < a.N) w |= (uint32_t)q[u] << (8 * u);
                    }
                }
#pragma unroll
                for (int u = 0; u < C; ++u) v[u][s] |= (w >> (8 * u) & 15) << (4 * (j / 2) + 16 * (j % 2));
            }
        uint4 *to = reinterpret_cast<uint4 *>(a.codes + e * per * C * 16 + (c / kSets * a.kblocks + kb) * kInt4TileBytes) +
                    quad * kInt4Columns + c % kSets * C;
#pragma unroll
        for (int u = 0; u < C; ++u) {
#pragma unroll
            for (int s = 0; s < 4; ++s) v[u][s] = v[u][s] << 3 | v[u][s] >> 29;
            to[u] = make_uint4(v[u][0], v[u][1], v[u][2], v[u][3]);
        }
    }
}

template <class T>
__global__ __launch_bounds__(256) void int4_pack_scales_kernel(Int4PackArgs a) {
    const int64_t per = (int64_t)a.ntiles * a.ngroups * kInt4Columns, all = per * a.E;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t e = i / per, w = i % per, tile = w / ((int64_t)a.ngroups * kInt4Columns);
        const int64_t g = w / kInt4Columns % a.ngroups, n = tile * kInt4Columns + w % kInt4Columns;
        const int64_t from = (e * a.ngroups + g) * a.N + n;
        const bool in = n < a.N;
        const T s = in ? reinterpret_cast<const T *>(a.scales)[from] : from_f32<T>(0.0f);
        const T z = from_f32<T>(16.0f + (a.zeros && in ? a.zeros[from] & 15 : 8));
        reinterpret_cast<T *>(a.meta)[2 * i] = s;
        reinterpret_cast<T *>(a.meta)[2 * i + 1] = z;
    }
}

// A thread per group and column.  With zero points the range is that of the values
// and 0, in 15 steps; without, 7 steps to either side.  The scale is rounded to its
// type first, codes and zero points belong to the rounded one.  Eight values are
// requested together, with whole loads where they lie side by side (a weight stored
// [N][K]): one at a time, neighbouring threads' lines are fetched again for each.
// 8192 x 28672 bf16 297 us, stored [N][K] 1169 (one value at a time 484 and 5426).
template <class T>
__global__ __launch_bounds__(256) void int4_quantize_kernel(Int4QuantArgs a) {
    constexpr int C = 8;
    const int64_t per = (int64_t)a.ngroups * a.N, all = per * a.E;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t e = i / per, g = i % per / a.N, n = i % a.N;
        const int64_t k0 = g * a.group, k1 = k0 + a.group < a.K ? k0 + a.group : a.K;
        const T *w = reinterpret_cast<const T *>(a.w) + e * a.se + n * a.sn;
        auto load = [&](int64_t k, T (&v)[C]) {  // past the group: its first value again
            if (k + C <= k1 && a.sk == 1) {
                __builtin_memcpy(v, w + k, sizeof v);
            } else {
#pragma unroll
                for (int j = 0; j < C; ++j) v[j] = w[(k + j < k1 ? k + j : k0) * a.sk];
            }
        };
        float lo = 0.0f, hi = 0.0f;
        for (int64_t k = k0; k < k1; k += C) {
            T v[C];
            load(k, v);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                lo = fminf(lo, to_f32(v[j]));
                hi = fmaxf(hi, to_f32(v[j]));
            }
        }
        // (halves first: the range of finite values may not be one)
        const T st = from_f32<T>(a.zeros ? 2.0f * ((0.5f * hi - 0.5f * lo) / 15.0f) : fmaxf(-lo, hi) / 7.0f);
        const float s = to_f32(st), z = a.zeros ? (s > 0.0f ? fminf(rintf(-lo / s), 15.0f) : 0.0f) : 8.0f;
        reinterpret_cast<T *>(a.scales)[i] = st;
        if (a.zeros) a.zeros[i] = (uint8_t)z;
        for (int64_t k = k0; k < k1; k += C) {
            T v[C];
            load(k, v);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const float q = s > 0.0f ? rintf(to_f32(v[j]) / s) + z : z;
                if (k + j < k1) a.q[(e * a.K + k + j) * a.N + n] = (uint8_t)fminf(fmaxf(q, 0.0f), 15.0f);
            }
        }
    }
}

template <class F>
hipError_t by_group(int group, F &&f) {
    using std::integral_constant;
    if (group == 32) return f(integral_constant<int, 1>());
    if (group == 64) return f(integral_constant<int, 2>());
    return f(integral_constant<int, 4>());
}

// W waves, XK tiles of the contraction to each, D column tiles ahead (int4_tiles).
template <class T, int SG, int W, int XK, int D>
hipError_t stream_rows(const Int4Args &a, unsigned blocks, hipStream_t s) {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(int4_stream_kernel<T, W, XK, D, SG>), dim3(blocks), dim3(W * 64), 0, s, a);
    return hipGetLastError();
}
template <class T, int SG, int MT, int NT>
hipError_t many_rows(const Int4Args &a, unsigned blocks, hipStream_t s) {
    constexpr int WK = sizeof(T) == 2 ? 2 : 1;
    hipLaunchKernelGGL(HIP_KERNEL_NAME(int4_rows_kernel<T, MT, NT, WK, SG>), dim3(blocks), dim3(WK * 256), 0, s, a);
    return hipGetLastError();
}
template <class T>
hipError_t int4(const Int4Args &a, const Int4Tiles &t, hipStream_t s) {
    constexpr bool kWide = sizeof(T) == 4;
    const unsigned n = (unsigned)(t.ntm * t.ntn * t.chunks);
    if (!t.waves)
        return by_group(a.group, [&](auto sg) {
            constexpr int SG = sg();
            if constexpr (SG > 1) {
                if (t.mt == 2 && t.nt == 2) return many_rows<T, SG, 2, 2>(a, n, s);
                if constexpr (!kWide)
                    if (t.mt == 5) return many_rows<T, SG, 5, 2>(a, n, s);
            }
            return many_rows<T, SG, 2, 1>(a, n, s);
        });
    return by_group(a.group, [&](auto sg) {
        constexpr int SG = sg();
        // (fp32: as far ahead as leaves the registers for four waves to a SIMD.  13 x 512 x 28672
        // 4 ahead 8.8 us, 2 7.8; 13 x 1024 x 28672 4 ahead 10.4, 3 10.3, 2 10.9, with groups of 64 14.5, 10.8, 11.4)
        if (t.waves == 4) return stream_rows<T, SG, 4, 1, kWide ? 2 : 4>(a, n, s);
        if constexpr (kWide) {
            return t.waves == 8 ? stream_rows<T, SG, 8, 1, 3>(a, n, s) : stream_rows<T, SG, 16, 1, 2>(a, n, s);
        } else {
            if (t.kper <= 16) return stream_rows<T, SG, 16, 1, 4>(a, n, s);
            return t.kper <= 32 ? stream_rows<T, SG, 16, 2, (SG > 1 ? 2 : 1)>(a, n, s) : stream_rows<T, SG, 16, 4, 1>(a, n, s);
        }
    });
}

}  // namespace

hipError_t launch_int4(int dtype, const Int4Args &a, const Int4Tiles &t, hipStream_t s) {
    return dtype == CP_BF16 ? int4<__bf16>(a, t, s) : int4<float>(a, t, s);
}

hipError_t launch_int4_pack(int dtype, const Int4PackArgs &a, hipStream_t s) {
    auto blocks = [](int64_t n) { return dim3((unsigned)((n + 255) / 256 < 16384 ? (n + 255) / 256 : 16384)); };
    const int64_t lanes = (int64_t)a.ntiles * a.kblocks * (kInt4TileBytes / 64) * a.E;
    const int64_t scales = (int64_t)a.ntiles * a.ngroups * kInt4Columns * a.E;
    hipLaunchKernelGGL(int4_pack_codes_kernel, blocks(lanes), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (dtype == CP_BF16) hipLaunchKernelGGL(HIP_KERNEL_NAME(int4_pack_scales_kernel<__bf16>), blocks(scales), dim3(256), 0, s, a);
    else hipLaunchKernelGGL(HIP_KERNEL_NAME(int4_pack_scales_kernel<float>), blocks(scales), dim3(256), 0, s, a);
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
