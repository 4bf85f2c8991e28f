// cp_ops_experts.h -- launch arguments and launchers of the operators around a
// feed-forward block's products: router, exchange of rows with the experts,
// 4-bit linear layers, gradient norm and clipping.  Internal.
#pragma once
#include "cp_ops_host.h"

namespace cpo {

// ------------------------------------------------------------------- router

constexpr int kRouteTokens = 64;      // tokens of a chunk: one bit each of an expert's word
constexpr int kRouteBlocks = 256;     // blocks of a launch at most

struct RouteArgs {
    const char *logits;
    const uint8_t *valid;  // [T] or null
    int64_t ld;
    int32_t *experts, *rows, *counts, *offsets;
    float *gates, *loss, *slopes;
    int32_t *hist, *live;  // scratch: slots of each expert [blocks][stride] and tokens with an expert [blocks]
    float *psum;           // scratch: sums of probabilities [blocks][stride]
    int32_t T, E, k, normalize;
    int32_t blocks, chunks;  // chunks of kRouteTokens per block
    int32_t stride;          // E in whole 16 bytes
};
// A chunk to a block as long as the device has room.  Two chunks of few experts are
// faster in one block than in two with the launch that joins them: 128 tokens of 8
// experts 6.2 us against 7.5, of 32 9.9 against 10.3; of 64 it is 10.9 and 10.8, of 128
// 15.1 and 12.6, and three chunks of 8 take 8.1 against 7.7.
inline int route_chunks(int64_t T, int64_t E) {
    const int64_t chunks = (T + kRouteTokens - 1) / kRouteTokens;
    if (chunks == 2 && E <= 32) return 2;
    return chunks ? (int)((chunks + kRouteBlocks - 1) / kRouteBlocks) : 1;
}
inline int route_blocks(int64_t T, int64_t E) {
    const int64_t per = (int64_t)route_chunks(T, E) * kRouteTokens;
    return T ? (int)((T + per - 1) / per) : 1;
}
inline int64_t route_ws(int64_t T, int64_t E) {
    const int64_t blocks = route_blocks(T, E);
    return blocks > 1 ? (blocks * (2 * ((E + 3) / 4 * 4) + 1) * 4 + 255) / 256 * 256 : 0;
}
hipError_t launch_route(int dtype, const RouteArgs &a, hipStream_t s);

struct RouteGradArgs {
    const char *logits;
    const int32_t *experts;
    const float *dgates, *dloss, *slopes;  // dgates or dloss may be null
    char *dlogits;
    int64_t ld, ldd;
    int32_t T, E, k, normalize;
};
hipError_t launch_route_backward(int dtype, const RouteGradArgs &a, hipStream_t s);

// ----------------------------------------------------- rows to experts and back

// x [T][D] and y [R][D]; token t's slots are rows[t * k + j] of y (others than
// 0 .. R-1: no slot).  Which of the pointers are set depends on the operator.
struct ExchangeArgs {
    const char *x, *y, *res;
    char *out, *dy;
    const int32_t *rows, *end;  // *end: rows of y from there on belong to no slot
    const float *gates;
    float *dgates;
    int64_t ldx, ldy, ldr, ldo, lddy;
    int64_t T, R;
    int32_t k, D;
};
hipError_t launch_dispatch(int dtype, const ExchangeArgs &a, hipStream_t s);          // x -> out [R][D]
hipError_t launch_combine(int dtype, const ExchangeArgs &a, hipStream_t s);           // y, res -> out [T][D]
hipError_t launch_combine_backward(int dtype, const ExchangeArgs &a, hipStream_t s);  // x = dout, y -> dy, dgates

// ---------------------------------------------------------- 4-bit linear layers

// Codes as the matrix instructions take them: tiles of 16 columns x 128 of K,
// 1 KB each, a column's tiles one after another; lane l of a wave holds column
// l % 16 and four words, word s the k = 32 s + 8 (l / 16) .. + 7, whose codes i
// are at bits 4 (i / 2) + 16 (i % 2) + 3, modulo 32.  Behind them [column tile][group][16] pairs
// of the scale and 16 + zero point, both of the layer's type.
constexpr int kInt4Columns = 16, kInt4Depth = 128, kInt4TileBytes = 1024;

struct Int4Layout {
    int64_t ntiles, kblocks, ngroups;
    int64_t codes, meta;  // bytes per expert
    Int4Layout(int dtype, int64_t K, int64_t N, int64_t group)
        : ntiles((N + kInt4Columns - 1) / kInt4Columns),
          kblocks((K + kInt4Depth - 1) / kInt4Depth),
          ngroups((K + group - 1) / group),
          codes(ntiles * kblocks * kInt4TileBytes),
          meta(ntiles * ngroups * kInt4Columns * (dtype == CP_BF16 ? 4 : 8)) {}
    int64_t bytes(int64_t E) const { return E * (codes + meta); }
};

struct Int4Args {
    const char *x, *codes, *meta, *bias, *res;
    char *y;
    int64_t ldx, ldr, ldy;
    int64_t sc, sm;        // bytes from one expert to the next
    const int32_t *off;    // device: groups + 1 row offsets, or null
    int32_t experts;       // 0: dense
    int32_t M, K, N, act;
    int32_t ntiles, kblocks, ngroups, group;
    int32_t ntm, ntn;      // row tiles (at most) and column sets of the launch
    int32_t chunks, kper;  // parts of the contraction, each to its own partial sums, and tiles of one
    float *ws;             // chunks > 1: [chunks][M][ldws]
    int64_t ldws;
};
// Tiles of a launch: `waves` waves to a block that streams (16 rows, any number of
// column tiles), or 0: mt row tiles and 4 nt column tiles.
struct Int4Tiles {
    int32_t waves, mt, nt, ntm, ntn, chunks, kper;
};
inline Int4Tiles int4_tiles(int dtype, int experts, int64_t M, int64_t ntiles, int64_t kblocks, int64_t group) {
    Int4Tiles t{};
    const int64_t rows = experts ? (M + experts - 1) / experts : M;  // to an expert, on average
    const int64_t used = M < experts + 1 ? M : experts + 1;
    auto row_tiles = [&](int64_t bm) { return (int32_t)(experts ? (M + used * (bm - 1)) / bm : (M + bm - 1) / bm); };
    t.chunks = 1;
    if (rows <= 16) {
        t.ntm = row_tiles(16);
        const bool bf16 = dtype == CP_BF16;
        // (fp32 with more than 8 tiles of K: 16 waves of one tile each rather than 8 of two, whose
        // registers leave room for two waves to a SIMD: 13 x 8192 x 8192 25 us against 18)
        t.waves = kblocks <= 4 ? 4 : (bf16 || kblocks > 8 ? 16 : 8);
        const int64_t most = bf16 ? 64 : 16;  // tiles of x that a block's registers hold (fp32: three operands each)
        if (kblocks > most) t.chunks = (int32_t)((kblocks + most - 1) / most);
        // blocks that fill the device, shared out over the row tiles that are likely there
        const int64_t tiles = (experts ? (M < experts ? M : experts) : t.ntm) * t.chunks;
        int64_t blocks = kComputeUnits * (16 / t.waves) / (tiles ? tiles : 1);
        if (blocks >= 8) blocks = blocks / 8 * 8;  // (as many to each XCD)
        if (blocks < 1) blocks = 1;
        t.ntn = (int32_t)(blocks < ntiles ? blocks : ntiles);
    } else {
        // Tile and parts of the contraction by the rounds the device takes: microseconds
        // for 256 k of a block with a CU to itself, and of two that share one (of the
        // largest only one fits).  Whole calls with groups of 128 and 2x1 | 2x2 | 5x2 tiles:
        // 17 x 4096 x 4096 9.4 | 9.9 | 13.7, 64 x 8192 x 8192 28 | 24 | 28, 300 x 8192 x 8192
        // 103 | 78 | 74, 2048 x 8192 x 8192 616 | 434 | 509.
        constexpr struct {
            int mt, nt;
            double one, two;
        } kTiles[] = {{2, 1, 0.72, 1.0}, {2, 2, 0.9, 1.56}, {5, 2, 2.3, 0.0}};
        double least = 1e300;
        for (const auto &k : kTiles) {
            if (k.nt > 1 && group == 32) continue;        // (registers: small groups keep more scales,
            if (k.mt > 2 && dtype != CP_BF16) continue;   // and fp32 rows are three operands)
            const int64_t tm = row_tiles(16 * k.mt), tn = (ntiles + 4 * k.nt - 1) / (4 * k.nt);
            const int64_t likely = experts ? M / (16 * k.mt) + experts / 2 + 1 : tm;  // an expert's last is half empty
            for (int chunks = 1; chunks <= 8 && (chunks == 1 || kblocks >= 8 * chunks); chunks *= 2) {
                const int64_t blocks = likely * tn * chunks, per = k.two > 0.0 ? 2 * kComputeUnits : kComputeUnits;
                const int64_t rest = blocks % per;
                double us = (double)(blocks / per) * (k.two > 0.0 ? k.two : k.one);
                us += rest == 0 ? 0.0 : (rest <= kComputeUnits ? k.one : k.two);
                us *= (double)((kblocks + 2 * chunks - 1) / (2 * chunks)) * (dtype == CP_BF16 ? 1.0 : 2.5);
                if (chunks > 1) us += 3.0 + 3.0 * chunks * (double)M * (double)ntiles * 16.0 * 4.0 / 8e6;  // partials, a launch
                if (us >= least) continue;
                least = us;
                t.mt = k.mt;
                t.nt = k.nt;
                t.ntm = tm;
                t.ntn = (int32_t)tn;
                t.chunks = chunks;
            }
        }
    }
    t.kper = (int32_t)((kblocks + t.chunks - 1) / t.chunks);
    return t;
}
inline int64_t int4_ws(int dtype, int experts, int64_t M, int64_t K, int64_t N) {
    int64_t chunks = 1;  // (whatever the group)
    for (const int group : {32, 64, 128}) {
        const int64_t n = int4_tiles(dtype, experts, M, (N + 15) / 16, (K + 127) / 128, group).chunks;
        if (n > chunks) chunks = n;
    }
    return chunks > 1 ? (chunks * M * ((N + 7) / 8 * 8) * 4 + 255) / 256 * 256 : 0;
}
hipError_t launch_int4(int dtype, const Int4Args &a, const Int4Tiles &t, hipStream_t s);

struct Int4PackArgs {
    const uint8_t *q, *zeros;
    const char *scales;
    char *codes, *meta;
    int64_t K, N, E;
    int32_t ntiles, kblocks, ngroups;
};
hipError_t launch_int4_pack(int dtype, const Int4PackArgs &a, hipStream_t s);

struct Int4QuantArgs {
    const char *w;
    int64_t sk, sn, se;  // strides in elements
    uint8_t *q, *zeros;  // zeros null: symmetric
    char *scales;
    int64_t K, N, E;
    int32_t group, ngroups;
};
hipError_t launch_int4_quantize(int dtype, const Int4QuantArgs &a, hipStream_t s);

// ------------------------------------------------------ gradient norm, clipping

constexpr int kClipTensors = 160;   // of a launch, at most: its arguments, up to 4 KB, hold their addresses
constexpr int kClipFew = 8;         // of a launch with shorter arguments, which are quicker to hand over
constexpr int kClipBlocks = 1024;   // partial sums of a launch, at most

// Partial sums that every block of the scaling adds up itself.  More are added up once
// before, as their number and that of the blocks both grow with the tensors': bf16,
// 16000 tensors of 65536 by every block 4108 us, once 2267; 2560 of them 368 and 340.
// Up to here the launch costs more than it spares: 200 of 100000 36.3 us, with it 37.2,
// 300 of 1000 30.8 and 33.5.
constexpr int kClipPartials = 2048;

template <int N>
struct ClipArgs {
    const char *x[N];
    char *y[N];            // outputs, or null
    int32_t before[N];     // chunks of the tensors before it in this launch
    int32_t last[N];       // elements of its last chunk
    uint32_t bf16_in[(N + 31) / 32], bf16_out[(N + 31) / 32];
    int32_t n, blocks;
    int32_t chunk;         // elements of a chunk
    int32_t chunks;
    double *partial;       // this launch's
    const double *all;     // of all launches
    int32_t nall;
    float max_norm;
    float *norm;
};
static_assert(sizeof(ClipArgs<kClipTensors>) <= 4096, "arguments of a launch");
// Elements that a block takes at a time: few where there are few in all, for the
// blocks to fill the device.
inline int32_t clip_chunk(int64_t total) {
    const int64_t n = total / (2 * kClipBlocks) / 2048 * 2048;
    return (int32_t)(n < 2048 ? 2048 : (n > 16384 ? 16384 : n));
}
inline int64_t clip_ws(int64_t tensors) {  // partial sums of every launch
    return (tensors + kClipTensors - 1) / kClipTensors * kClipBlocks * (int64_t)sizeof(double);
}
hipError_t launch_norm_total(double *all, int n, hipStream_t s);  // all[0] = the sum of the n
// (N: kClipTensors or kClipFew)
template <int N>
hipError_t launch_norm_partials(const ClipArgs<N> &a, hipStream_t s);
template <int N>
hipError_t launch_clip(const ClipArgs<N> &a, hipStream_t s);

}  // namespace cpo
