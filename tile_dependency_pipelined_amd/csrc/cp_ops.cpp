// cp_ops.cpp -- host side of the feed-forward operators (include/cp_ops.h):
// argument checks, choice of tile and split, launches.  No allocation, no
// synchronisation; a thread keeps the choices of its recent shapes (choose).
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <numeric>

#include "cp_ops_host.h"

using namespace cpo;

namespace {

thread_local char g_error[512];

int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof g_error, fmt, ap);
    va_end(ap);
    return code;
}

int launched(hipError_t e, const char *what) {
    if (e == hipSuccess) return CP_OK;
    return fail(CP_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

constexpr int64_t kMaxRows = int64_t(1) << 30;

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int elem_size(int dtype) { return dtype == CP_BF16 ? 2 : 4; }

// ------------------------------------------------------------------- checks

struct Mat {
    const void *p;
    int64_t rows, cols, ld;
};

int check_dtype(int dtype) {
    if (dtype != CP_F32 && dtype != CP_BF16) return fail(CP_ERR_UNSUPPORTED, "dtype %d is not supported", dtype);
    return CP_OK;
}

int check_sizes(int64_t M, int64_t K, int64_t N) {
    if (M < 0 || K < 0 || N < 0)
        return fail(CP_ERR_SHAPE, "negative size (M=%lld K=%lld N=%lld)", (long long)M, (long long)K, (long long)N);
    if (M > kMaxRows || K > CP_OPS_MAX_WIDTH || N > CP_OPS_MAX_WIDTH)
        return fail(CP_ERR_SHAPE, "size too large (M=%lld K=%lld N=%lld; at most 2^30 rows, %d columns)", (long long)M,
                    (long long)K, (long long)N, CP_OPS_MAX_WIDTH);
    return CP_OK;
}

int check_act(int act) {
    if (act < CP_ACT_NONE || act > CP_ACT_SILU) return fail(CP_ERR_UNSUPPORTED, "activation %d is not supported", act);
    return CP_OK;
}

// A matrix that is read or written; its ld is set to something usable where
// there is at most one row.
int check_mat(Mat &m, int dtype, const char *name) {
    if (m.rows == 0 || m.cols == 0) {
        m.ld = up(m.cols, 8);
        return CP_OK;
    }
    if (!m.p) return fail(CP_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(m.p) % elem_size(dtype)) return fail(CP_ERR_INVALID_ARG, "%s is misaligned", name);
    if (m.rows == 1) {
        m.ld = up(m.cols, 8);
        return CP_OK;
    }
    if (m.ld < m.cols || m.ld > CP_OPS_MAX_WIDTH)
        return fail(CP_ERR_SHAPE, "%s: row stride %lld with rows of %lld (at least that, at most %d)", name,
                    (long long)m.ld, (long long)m.cols, CP_OPS_MAX_WIDTH);
    return CP_OK;
}

bool aligned16(const Mat &m, int dtype) {
    const int es = elem_size(dtype);
    return !m.p || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.ld * es % 16 == 0 && m.cols * es % 16 == 0);
}
bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Memory of a matrix, or of one in a stack of `count`: rows of `width` bytes, `ld` bytes apart.
struct Rows {
    uintptr_t p;
    int64_t rows, width, ld, count = 1, stride = 0;
    Rows(const void *at, int64_t n, int64_t bytes, int64_t step) : p((uintptr_t)at), rows(n), width(bytes), ld(step) {}
    Rows(const Mat &m, int dtype) : Rows(m.p, m.rows, m.cols * elem_size(dtype), m.ld * elem_size(dtype)) {}
    Rows(const void *at, int64_t bytes) : Rows(at, 1, bytes, bytes) {}
};

// Whether a and b share a byte.  Views of one buffer may interleave: of the rows
// of a that lie within b's extent, each is compared with b's rows, whose pattern
// is that of the row's offset modulo b's row stride and repeats.
bool overlap_one(const Rows &a, const Rows &b) {
    if (!a.p || !b.p || a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
    const int64_t d = (int64_t)(a.p - b.p), extent = (b.rows - 1) * b.ld + b.width;
    if (d >= extent || d + (a.rows - 1) * a.ld + a.width <= 0) return false;
    const int64_t from = d + a.width > 0 ? 0 : (-d - a.width) / a.ld + 1;
    int64_t to = (extent - 1 - d) / a.ld + 1;
    if (to > a.rows) to = a.rows;
    const int64_t period = b.ld / std::gcd(a.ld, b.ld);
    for (int64_t r = from; r < to && r < from + period; ++r) {
        const int64_t x = ((d + r * a.ld) % b.ld + b.ld) % b.ld;
        if (x < b.width || x + a.width > b.ld) return true;
    }
    return false;
}
bool overlap(const Rows &a, Rows b) {
    if (b.count > 1) {  // the usual case at once: apart from the whole stack
        const uintptr_t a_end = a.p + (a.rows - 1) * a.ld + a.width;
        const uintptr_t b_end = b.p + (b.count - 1) * b.stride + (b.rows - 1) * b.ld + b.width;
        if (a_end <= b.p || b_end <= a.p) return false;
    }
    for (int64_t i = 0; i < b.count; ++i, b.p += b.stride)
        if (overlap_one(a, b)) return true;
    return false;
}

// An output against an input, or the other output; `same`: it may be that very matrix.
int check_apart(const char *name, const Rows &out, const char *other, const Rows &in, bool same = false) {
    if (same && out.p == in.p && (out.ld == in.ld || out.rows <= 1)) return CP_OK;
    if (overlap(out, in)) return fail(CP_ERR_INVALID_ARG, "%s overlaps %s", name, other);
    return CP_OK;
}

#define CP_TRY(expr)                  \
    do {                              \
        const int rc_ = (expr);       \
        if (rc_ != CP_OK) return rc_; \
    } while (0)

// ------------------------------------------------------------ tile and split

// Products: what is to be computed, apart from where it lies.
struct Shape {
    int dtype;
    Layout layout;
    int mode;
    int64_t M, N, K;  // rows and columns of C, contraction; kGroupRows: M over all experts; kGroupSum: K over all
    int groups;
    bool operator==(const Shape &o) const {
        return dtype == o.dtype && layout == o.layout && mode == o.mode && M == o.M && N == o.N && K == o.K &&
               groups == o.groups;
    }
};

struct Choice {
    Config cfg;
    int nsplit;
};

// Row tiles of `bm` rows the launch can have at most.
int64_t max_row_tiles(const Shape &s, int bm) {
    if (s.mode != kGroupRows) return ceil_div(s.M, bm);
    const int64_t used = s.M < s.groups + 1 ? s.M : s.groups + 1;  // spans that hold a row
    return (s.M + used * (bm - 1)) / bm;
}

// Workgroups of a launch with tiles `c` and `n` splits, at most.
int64_t workgroups(const Shape &s, Config c, int n) {
    const int64_t tiles = max_row_tiles(s, kShapes[c].bm) * ceil_div(s.N, kShapes[c].bn) * n;
    return tiles * (s.mode == kGroupSum ? s.groups : 1) + (c == kTile256 ? kComputeUnits / 2 : 0);  // (halves: launch_args)
}
// The products' kernels count a launch's workgroups in one dimension of the grid.
bool fits_grid(int64_t n, Config c) { return n <= max_blocks(kShapes[c].threads); }

// Rows of all the results together.
int64_t result_rows(const Shape &s) { return s.M * (s.mode == kGroupSum ? s.groups : 1); }

int64_t slabs_of(const Shape &s) {
    return ceil_div(s.mode == kGroupSum ? ceil_div(s.K, s.groups) : s.K, 128 / elem_size(s.dtype));
}

// Few rows (per expert): 16-row tiles, whose time is that of reading B.  The
// split fills the device twice over, keeping four slabs of 64 (fp32: 32) to a
// split, so that the loads in flight are worth their latency.  Experts count by
// their mean, as the host does not know their rows: where one has most of them,
// its weight is read again by each of its tiles.  64 experts of 2048 x 4096, us
// with the rows even | half of them in one expert | nine tenths: 8 rows each 186 |
// 199 | 39, 16 each 190 | 232 | 285; 17 each, so with larger tiles, 192 | 192 | 198.
bool few_rows(const Shape &s) {
    return s.layout != kTN && (s.mode == kGroupRows ? ceil_div(s.M, s.groups) : s.M) <= 16;
}

// Tiles of an average launch: each expert's last row tile is half empty.
double average_tiles(const Shape &s, Config c) {
    const ConfigShape t = kShapes[c];
    const double tm = s.mode == kGroupRows ? (double)s.M / t.bm + 0.5 * s.groups : (double)ceil_div(s.M, t.bm);
    return tm * (double)ceil_div(s.N, t.bn) * (s.mode == kGroupSum ? s.groups : 1);
}

// Time in microseconds of one launch of `tiles` tiles with `slabs` slabs each
// (`halves`: with the last round of 256x256 tiles in halves where that fits),
// from the rounds the device takes: a time per slab, which grows with the share
// of the CUs that are busy (they share memory and power), and a fixed time.
// Fitted to bf16 products with the weights coming from memory (rows x columns x
// contraction, microseconds for 256x256 | 128x256 | 128x128 | 64x128 | 64x64 tiles):
//   512 x 2048 x 1024            | 14 | 9.4 | 7.5
//   256 x 4096 x 4096    83 | 51 | 42 | 24 | 17
//   512 x 4096 x 4096    83 | 50 | 42 | 25 | 28
//   1024 x 4096 x 4096   83 | 50 | 44     1024 x 8192 x 8192 176 | 118 | 137
//   2048 x 4096 x 4096   84 | 62 | 63     2048 x 8192 x 8192 213 | 248 | 268
//   4096 x 4096 x 4096  107 | 125 | 137   8192 x 4096 x 2048 114 | 130 | 130
// and to fp32: 512 x 2048 x 1024 64 us with 128x128, 36 with 64x128, 23 with 64x64.
double launch_time(Config c, int dtype, double tiles, double slabs, bool halves) {
    const double cus = tiles / kComputeUnits;  // tiles per CU
    const double busy = cus < 1.0 ? cus : 1.0;
    const double rounds = (double)(int64_t)(cus + 0.999);
    if (dtype == CP_F32)  // matrix-bound: several tiles on a CU take as many times as long
        return rounds * (c == kTile128 ? 1.9 : c == kTile64x128 ? 0.95 : 0.49) * slabs + 6.0;
    if (c == kTile256) {
        const double rest = tiles - kComputeUnits * (rounds - 1.0);
        if (halves && rounds > 1.0 && rest <= kComputeUnits / 2)
            return (rounds - 1.0) * (1.55 * slabs + 10.0) + launch_time(kTile128x256, dtype, 2.0 * rest, slabs, false);
        return rounds * ((1.12 + 0.43 * busy) * slabs + 10.0);
    }
    if (c == kTile128x256) return rounds * ((0.66 + 0.21 * busy) * slabs + 7.0);
    // two on a CU; a CU that is left with one runs it faster
    const double one = c == kTile128 ? 0.58 : c == kTile64x128 ? 0.31 : 0.19;
    const double two = c == kTile128 ? 0.97 : c == kTile64x128 ? 0.57 : 0.37;
    const double full = (double)(int64_t)(cus / 2.0), rest = cus - 2.0 * full;
    double t = full * (two * slabs + 4.0);
    if (rest > 0.0) t += (one + (rest > 1.0 ? (two - one) * (rest - 1.0) : 0.0)) * slabs + 5.0;
    return t;
}

// Time of a product with tiles `c` and `n` splits.
double product_time(const Shape &s, Config c, int n) {
    double us = launch_time(c, s.dtype, average_tiles(s, c) * n, (double)ceil_div(slabs_of(s), n), s.mode != kGroupSum);
    // Each expert's weights are read by few tiles: the smaller the
    // tile, the more of them wait for the same memory (8192 x 4096 x
    // 2048 over 16 experts: 178 us with 256x256 tiles, 169 with
    // 128x256, 183 with 128x128, which a single weight takes 130 us;
    // the smaller ones are taken to be like it).
    if (s.mode == kGroupRows && c >= kTile128) us *= 1.2;
    // A split writes and reads its partials, mostly in the caches, and
    // takes another launch.
    if (n > 1) us += 3.0 + 2.0 * n * (double)result_rows(s) * (double)s.N * 4.0 / 8e6;
    return us;
}

Choice choose_now(const Shape &s) {
    // (both sides measured: cp_ops_gemv.hip)
    if (few_rows(s) && s.mode == kDense && s.M <= kGemvRows &&
        (s.layout == kNT || s.K * s.N * elem_size(s.dtype) <= kGemvColumnBytes))
        return {kGemv, 1};
    if (few_rows(s)) {
        const int64_t tiles = max_row_tiles(s, 16) * ceil_div(s.N, 128);
        int64_t n = 2 * kComputeUnits / (tiles ? tiles : 1);
        if (n > slabs_of(s) / 4) n = slabs_of(s) / 4;
        if (n > 32) n = 32;
        return {kTile16, n < 1 ? 1 : (int)n};
    }
    const Config all[] = {kTile256, kTile128x256, kTile128, kTile64x128, kTile64};
    const int64_t slabs = slabs_of(s);
    Choice best{kTile128, 1};
    double least = 1e300;
    for (const Config c : all) {
        if (s.dtype == CP_F32 && c < kTile128) continue;
        for (int n = 1; n <= 16; ++n) {
            if ((n > 1 && slabs < 4 * n) || !fits_grid(workgroups(s, c, n), c)) break;
            const double us = product_time(s, c, n);
            if (us < least) {
                least = us;
                best = {c, n};
            }
        }
    }
    return best;
}

// The same for the shapes of this thread's recent calls: weighing all tiles and
// splits takes about a microsecond, several times in a call.
Choice choose(const Shape &s) {
    struct Entry {
        Shape s{-1, kNN, 0, 0, 0, 0, 0};
        Choice c{};
    };
    static thread_local Entry cache[64];
    uint64_t h = (uint64_t)s.M * 0x9E3779B97F4A7C15ull + (uint64_t)s.N;
    h = h * 0x9E3779B97F4A7C15ull + (uint64_t)s.K;
    h = h * 0x9E3779B97F4A7C15ull + (uint64_t)(s.layout * 64 + s.mode * 8 + s.dtype) + (uint64_t)s.groups * 1024;
    Entry &e = cache[(h * 0x9E3779B97F4A7C15ull) >> 58];
    if (!(e.s == s)) e = {s, choose_now(s)};
    return e.c;
}

// ------------------------------------------------------------------ products

struct Product {
    Shape s;
    Mat A, B, C;  // as stored
    int64_t sb = 0, sc = 0;
    const int32_t *off = nullptr;
    const void *bias = nullptr;
    Mat R{nullptr, 0, 0, 0}, P{nullptr, 0, 0, 0};
    int act = CP_ACT_NONE;
};

// Bytes of a packed copy of `count` matrices.
int64_t packed_bytes(int dtype, int64_t rows, int64_t cols, int64_t count) {
    return up(rows * up(cols, 8) * count * elem_size(dtype), 256);
}

// Scratch memory handed out front to back; with no base it only counts.
struct Arena {
    char *base;
    int64_t used = 0;
    char *take(int64_t bytes) {
        char *p = base ? base + used : nullptr;
        used += up(bytes, 256);
        return p;
    }
};

// Rows of whole 16-byte chunks, as the direct loads need them: the matrix
// itself if it has them, otherwise a copy, made by the launch that ends the
// list.  A copy moves the matrix twice; a kernel that read unaligned rows
// through registers instead took 200 us for 2048 x 4096 x 4096 with odd rows,
// where the aligned one takes 62 and the copies about 25.
struct Packs {
    PackArgs a{};
    int dtype;
    Arena &mem;

    void add(Mat &m, int64_t *stride, int count) {
        if (m.rows == 0 || m.cols == 0) return;
        if (aligned16(m, dtype) && (!stride || *stride * elem_size(dtype) % 16 == 0)) return;
        PackArgs::One &o = a.one[a.n++];
        o.src = (const char *)m.p;
        o.dst = mem.take(packed_bytes(dtype, m.rows, m.cols, count));
        o.ld = m.ld;
        o.ldd = up(m.cols, 8);
        o.stride = stride ? *stride : 0;
        o.stride_d = m.rows * o.ldd;
        o.rows = (int)m.rows;
        o.cols = (int)m.cols;
        o.count = count;
        m.p = o.dst;
        m.ld = o.ldd;
        if (stride) *stride = o.stride_d;
    }
    int launch(hipStream_t s) { return a.n ? launched(launch_pack(dtype, a, s), "pack") : CP_OK; }
};

int64_t split_bytes(const Shape &s) {
    if (s.M == 0 || s.N == 0) return 0;
    const Choice c = choose(s);
    return c.nsplit > 1 ? (int64_t)c.nsplit * result_rows(s) * up(s.N, 8) * 4 : 0;
}

// The launch of a product with this choice; its operands are aligned unless it
// is of few rows; `alone` in its launch.  Returns the number of workgroups, or
// an error.
int64_t launch_args(const Product &p, const Choice &c, void *split, GemmArgs &g, bool alone) {
    const Shape &s = p.s;
    const int es = elem_size(s.dtype);
    g = GemmArgs{};
    g.A = (const char *)p.A.p;
    g.B = (const char *)p.B.p;
    g.C = (char *)p.C.p;
    g.bias = (const char *)p.bias;
    g.res = (const char *)p.R.p;
    g.pre = (char *)p.P.p;
    g.ws = (float *)split;
    g.lda = p.A.ld;
    g.ldb = p.B.ld;
    g.ldc = p.C.ld;
    g.ldr = p.R.ld;
    g.ldp = p.P.ld;
    g.sb = p.sb;
    g.sc = p.sc;
    g.off = p.off;
    g.groups = s.groups;
    g.mode = s.mode;
    g.M = (int)s.M;
    g.N = (int)s.N;
    g.K = (int)s.K;
    g.act = p.act;
    g.nsplit = c.nsplit;
    g.ldws = (int)up(s.N, 8);
    g.vec = aligned16(p.C, s.dtype) && aligned16(p.R, s.dtype) && aligned16(p.P, s.dtype) && aligned16(p.bias) &&
            p.sc * es % 16 == 0;
    const ConfigShape t = kShapes[c.cfg];
    const int64_t ntm = max_row_tiles(s, t.bm), ntn = ceil_div(s.N, t.bn);
    const int64_t grid = ntm * ntn * c.nsplit * (s.mode == kGroupSum ? s.groups : 1);
    if (c.cfg != kGemv && !fits_grid(workgroups(s, c.cfg, c.nsplit), c.cfg))
        return fail(CP_ERR_SHAPE, "too many tiles of %d x %d (%lld)", t.bm, t.bn, (long long)grid);
    g.ntm = (int)ntm;
    g.ntn = (int)ntn;
    if (c.cfg == kTile256 && s.mode != kGroupSum && alone)  // (kGroupRows: any number of tiles up to `grid`)
        return grid + (s.mode == kGroupRows ? kComputeUnits / 2 : halved_tiles((int)grid));
    return grid;
}

// `split`: room for split_bytes().
int run_product(const Product &p, void *split, hipStream_t stream) {
    const Shape &s = p.s;
    if (s.M == 0 || s.N == 0) return CP_OK;
    const Choice c = choose(s);
    GemmArgs g;
    const int64_t grid = launch_args(p, c, split, g, true);
    if (grid < 0) return (int)grid;
    if (c.cfg == kGemv) return launched(launch_gemv(s.dtype, s.layout == kNT, g, stream), "product of few rows");
    const bool direct = c.cfg != kTile16 || (aligned16(p.A, s.dtype) && aligned16(p.B, s.dtype) &&
                                             p.sb * elem_size(s.dtype) % 16 == 0);
    CP_TRY(launched(s.dtype == CP_BF16 ? launch_product_bf16(s.layout, c.cfg, direct, g, (int)grid, stream)
                                       : launch_product_f32(s.layout, c.cfg, direct, g, (int)grid, stream),
                    "product"));
    if (c.nsplit > 1) CP_TRY(launched(launch_join(s.dtype, g, stream), "join"));
    return CP_OK;
}

// Time of dX's and dW's tiles in one launch: each slot of the device takes dX's
// first, then dW's as it comes free.
double gradients_time(const Shape &x, const Shape &w, Config c) {
    const int slots = kComputeUnits * (x.dtype == CP_BF16 && c >= kTile128 ? 2 : 1);
    const double penalty = x.mode == kGroupRows && c >= kTile128 ? 1.2 : 1.0;
    const int64_t nx = (int64_t)(average_tiles(x, c) + 0.5), nw = (int64_t)(average_tiles(w, c) + 0.5);
    const double busy = nx + nw < slots ? (double)(nx + nw) : (double)slots;
    const double tx = penalty * launch_time(c, x.dtype, busy, (double)slabs_of(x), false);
    const double tw = penalty * launch_time(c, w.dtype, busy, (double)slabs_of(w), false);
    const double t0 = (double)(nx / slots) * tx;  // most slots are done with dX
    const double late = (double)(nx % slots);     // these have one more of its tiles
    const double t1 = late > 0.0 ? t0 + tx : t0;
    // the earliest end by which all of dW's tiles fit; from a bound below it
    const double least = ((slots - late) * t0 + late * t1 + (double)nw * tw) / slots;
    double k0 = (double)(int64_t)((least - t0) / tw), k1 = (double)(int64_t)((least - t1) / tw);
    if (k0 < 1.0) k0 = 1.0;
    if (k1 < 1.0) k1 = 1.0;
    for (;;) {
        const double e0 = t0 + k0 * tw, e1 = t1 + k1 * tw, end = e0 < e1 ? e0 : e1;
        const double early = (double)(int64_t)((end - t0) / tw + 1e-6), after = (double)(int64_t)((end - t1) / tw + 1e-6);
        if ((slots - late) * early + late * (after > 0.0 ? after : 0.0) >= (double)nw) return end > t1 ? end : t1;
        (e0 < e1 ? k0 : k1) += 1.0;
    }
}

// Time of dX alone where it has few rows (its weights' bytes).
double few_rows_time(const Shape &x, const Choice &c) {
    const double experts = x.mode == kGroupRows ? (double)(x.M < x.groups ? x.M : x.groups) : 1.0;
    return 6.0 + experts * (double)x.N * (double)x.K * elem_size(x.dtype) / 4.8e6 + (c.nsplit > 1 ? 4.0 : 0.0);
}

// The configuration of one launch for both gradients, or kConfigs if two are
// better.  In two and in one, whole passes, bf16, microseconds: 140 x 200 x 1728
// 18.1 | 13.1 and 2048 x 512 x 512 20.3 | 15.7 (rather than split products); 4099 x
// 2048 x 4096 over 8 experts, the products 210 | 171.
Config choose_gradients(const Shape &x, const Shape &w) {
    const Choice cx = choose(x), cw = choose(w);
    const bool few = few_rows(x);
    double least = (few ? few_rows_time(x, cx) : product_time(x, cx.cfg, cx.nsplit)) + product_time(w, cw.cfg, cw.nsplit);
    Config best = kConfigs;
    for (const Config c : {kTile256, kTile128x256, kTile128, kTile64x128, kTile64}) {
        if (x.dtype == CP_F32 && c < kTile128) continue;
        const int64_t sums = ceil_div(x.K, 64) * (x.groups ? x.groups : 1);  // (the bias's)
        if (!fits_grid(workgroups(x, c, 1) + workgroups(w, c, 1) + sums, c)) continue;
        const double us = gradients_time(x, w, c) - 3.0;  // a launch less
        if (us < least) {
            least = us;
            best = c;
        }
    }
    return best;
}

// ------------------------------------------------- the linear layers, dense and
// grouped (groups == 0: dense)

Shape forward_shape(int dtype, int64_t M, int64_t K, int64_t N, int groups, bool wt) {
    return {dtype, wt ? kNT : kNN, groups ? kGroupRows : kDense, M, N, K, groups};
}
Shape dx_shape(int dtype, int64_t M, int64_t K, int64_t N, int groups, bool wt) {
    return {dtype, wt ? kNN : kNT, groups ? kGroupRows : kDense, M, K, N, groups};
}
Shape dw_shape(int dtype, int64_t M, int64_t K, int64_t N, int groups, bool wt) {
    return {dtype, kTN, groups ? kGroupSum : kDense, wt ? N : K, wt ? K : N, M, groups};
}

int64_t max64(int64_t a, int64_t b) { return a > b ? a : b; }

// Scratch memory of a forward pass: partials of a split, and with unaligned
// operands their copies.
int64_t forward_ws(int dtype, int64_t M, int64_t K, int64_t N, int E, bool aligned) {
    const Shape s = forward_shape(dtype, M, K, N, E, false);
    int64_t n = up(max64(split_bytes(s), split_bytes(forward_shape(dtype, M, K, N, E, true))), 256);
    if (!aligned && !few_rows(s))
        n += packed_bytes(dtype, M, K, 1) +
             max64(packed_bytes(dtype, K, N, E ? E : 1), packed_bytes(dtype, N, K, E ? E : 1));
    return n;
}

// Of a backward pass: partial column sums, dZ (or a copy of dY), partials of a
// split, copies of X and W.
int64_t sums_bytes(int dtype, int64_t M, int64_t N, int E) {
    const Shape rows{dtype, kNN, E ? kGroupRows : kDense, M, N, 0, E};
    return max_row_tiles(rows, kGradRows) * N * 4;
}
int64_t backward_split_bytes(int dtype, int64_t M, int64_t K, int64_t N, int E) {
    int64_t most = 0;
    for (int wt = 0; wt < 2; ++wt) {
        most = max64(most, split_bytes(dx_shape(dtype, M, K, N, E, wt)));
        most = max64(most, split_bytes(dw_shape(dtype, M, K, N, E, wt)));
    }
    return most;
}
int64_t backward_ws(int dtype, int64_t M, int64_t K, int64_t N, int E, bool aligned) {
    int64_t n = up(sums_bytes(dtype, M, N, E), 256) + packed_bytes(dtype, M, N, 1) +
                up(backward_split_bytes(dtype, M, K, N, E), 256);
    if (!aligned)
        n += packed_bytes(dtype, M, K, 1) +
             max64(packed_bytes(dtype, K, N, E ? E : 1), packed_bytes(dtype, N, K, E ? E : 1));
    return n;
}

// Partial sums of the norm's backward pass, unless one block has it all.
int64_t norm_ws(int64_t M, int64_t N) {
    const int blocks = norm_backward_blocks(M, N);
    return blocks > 1 ? (int64_t)blocks * N * 8 : 0;
}

int check_ws(const void *ws, int64_t have, int64_t need) {
    if (need == 0) return CP_OK;
    if (!ws || have < need)
        return fail(CP_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", ws ? (long long)have : 0, (long long)need);
    if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(CP_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    return CP_OK;
}

int check_groups(int E, const void *off, int64_t stride, const Mat &w, const char *name) {
    if (E < 1 || E > CP_OPS_MAX_GROUPS)
        return fail(CP_ERR_SHAPE, "%d experts (1 to %d)", E, CP_OPS_MAX_GROUPS);
    if (!off) return fail(CP_ERR_INVALID_ARG, "offsets is NULL");
    if (reinterpret_cast<uintptr_t>(off) % 4) return fail(CP_ERR_INVALID_ARG, "offsets is misaligned");
    const int64_t span = w.rows && w.cols ? (w.rows - 1) * w.ld + w.cols : 0;
    if (w.p && E > 1 && stride < (w.rows == 1 ? w.cols : span))
        return fail(CP_ERR_SHAPE, "%s: expert stride %lld, one expert spans %lld", name, (long long)stride,
                    (long long)span);
    return CP_OK;
}

int check_vector(const void *p, int dtype, const char *name) {
    if (reinterpret_cast<uintptr_t>(p) % elem_size(dtype)) return fail(CP_ERR_INVALID_ARG, "%s is misaligned", name);
    return CP_OK;
}

int forward(int dtype, int64_t M, int64_t K, int64_t N, int E, const void *X, int64_t ldx, const void *W, int64_t ldw,
            int64_t stride_w, bool wt, const int32_t *off, const void *bias, const void *R, int64_t ldr, int act, void *Y,
            int64_t ldy, void *pre, int64_t ldp, void *ws, int64_t ws_bytes, void *stream) {
    CP_TRY(check_dtype(dtype));
    CP_TRY(check_sizes(M, K, N));
    CP_TRY(check_act(act));
    Product p{};
    p.s = forward_shape(dtype, M, K, N, E, wt);
    p.A = {X, M, K, ldx};
    p.B = {W, wt ? N : K, wt ? K : N, ldw};
    p.C = {Y, M, N, ldy};
    CP_TRY(check_mat(p.A, dtype, "X"));
    CP_TRY(check_mat(p.B, dtype, "W"));
    CP_TRY(check_mat(p.C, dtype, "Y"));
    if (R) {
        p.R = {R, M, N, ldr};
        CP_TRY(check_mat(p.R, dtype, "R"));
    }
    if (pre) {
        p.P = {pre, M, N, ldp};
        CP_TRY(check_mat(p.P, dtype, "pre"));
    }
    CP_TRY(check_vector(bias, dtype, "bias"));
    if (E) CP_TRY(check_groups(E, off, stride_w, p.B, "W"));
    p.sb = E > 1 ? stride_w : 0;
    p.off = off;
    p.bias = bias;
    p.act = act;
    Rows w(p.B, dtype);
    w.count = E > 1 ? E : 1;
    w.stride = p.sb * elem_size(dtype);
    for (const Mat *m : {&p.C, &p.P}) {
        const char *name = m == &p.C ? "Y" : "pre";
        const Rows out(*m, dtype);
        CP_TRY(check_apart(name, out, "X", Rows(p.A, dtype)));
        CP_TRY(check_apart(name, out, "W", w));
        CP_TRY(check_apart(name, out, "bias", Rows(bias, (E ? E : 1) * N * elem_size(dtype))));
        CP_TRY(check_apart(name, out, "offsets", Rows(off, (E + 1) * 4)));
        CP_TRY(check_apart(name, out, "R", Rows(p.R, dtype), m == &p.C));
    }
    CP_TRY(check_apart("Y", Rows(p.C, dtype), "pre", Rows(p.P, dtype)));
    const bool aligned =
        aligned16(p.A, dtype) && aligned16(p.B, dtype) && p.sb * elem_size(dtype) % 16 == 0;
    CP_TRY(check_ws(ws, ws_bytes, forward_ws(dtype, M, K, N, E, aligned)));
    if (M == 0 || N == 0) return CP_OK;
    Arena mem{(char *)ws};
    void *split = mem.take(split_bytes(p.s));
    if (!few_rows(p.s)) {
        Packs packs{{}, dtype, mem};
        packs.add(p.A, nullptr, 1);
        packs.add(p.B, &p.sb, E ? E : 1);
        CP_TRY(packs.launch((hipStream_t)stream));
    }
    return run_product(p, split, (hipStream_t)stream);
}

// Of few rows, dX is worth a copy of an unaligned W, which lets it share dW's
// launch, up to this size: without and with the copy, whole passes, bf16, us,
// 8 x 513 x 497 17.7 | 10.4, 16 x 1001 x 1001 17.8 | 12.9, 16 x 2001 x 2001 (8
// MB) 20.8 | 19.8.
constexpr int64_t kCopyBytes = 8 << 20;

int backward(int dtype, int64_t M, int64_t K, int64_t N, int E, const void *dY, int64_t lddy, const void *X, int64_t ldx,
             const void *W, int64_t ldw, int64_t stride_w, bool wt, const int32_t *off, const void *pre, int64_t ldp,
             int act, void *dX, int64_t lddx, void *dW, int64_t lddw, int64_t stride_dw, void *db, void *ws,
             int64_t ws_bytes, void *stream) {
    CP_TRY(check_dtype(dtype));
    CP_TRY(check_sizes(M, K, N));
    CP_TRY(check_act(act));
    Mat dy{dY, M, N, lddy}, x{X, M, K, ldx}, w{W, wt ? N : K, wt ? K : N, ldw}, z{pre, M, N, ldp};
    Mat dx{dX, M, K, lddx}, dw{dW, w.rows, w.cols, lddw};
    if (dX || dW || db) CP_TRY(check_mat(dy, dtype, "dY"));
    if (act != CP_ACT_NONE) CP_TRY(check_mat(z, dtype, "pre"));
    if (dX) {
        CP_TRY(check_mat(w, dtype, "W"));
        CP_TRY(check_mat(dx, dtype, "dX"));
    }
    if (dW) {
        CP_TRY(check_mat(x, dtype, "X"));
        CP_TRY(check_mat(dw, dtype, "dW"));
    }
    CP_TRY(check_vector(db, dtype, "db"));
    if (E) {
        CP_TRY(check_groups(E, off, stride_w, dX ? w : Mat{nullptr, 0, 0, 0}, "W"));
        CP_TRY(check_groups(E, off, stride_dw, dW ? dw : Mat{nullptr, 0, 0, 0}, "dW"));
    }
    const int64_t es = elem_size(dtype);
    const bool aligned = (dy.p == nullptr || aligned16(dy, dtype)) && (!dW || aligned16(x, dtype)) &&
                         (!dX || (aligned16(w, dtype) && (E <= 1 || stride_w * es % 16 == 0)));
    CP_TRY(check_ws(ws, ws_bytes, backward_ws(dtype, M, K, N, E, aligned)));
    if (!dX && !dW && !db) return CP_OK;
    hipStream_t s = (hipStream_t)stream;
    Arena mem{(char *)ws};
    char *sums = mem.take(sums_bytes(dtype, M, N, E));
    void *split = mem.take(backward_split_bytes(dtype, M, K, N, E));
    Mat dz = dy;
    if (act != CP_ACT_NONE) dz = {mem.take(packed_bytes(dtype, M, N, 1)), M, N, up(N, 8)};
    const Shape sx = dx_shape(dtype, M, K, N, E, wt), sw = dw_shape(dtype, M, K, N, E, wt);
    int64_t sb = E > 1 ? stride_w : 0;
    Packs packs{{}, dtype, mem};
    // (with an activation, dZ is in aligned rows already, zero past their end)
    if (act == CP_ACT_NONE && (dW || (dX && !few_rows(sx)))) packs.add(dz, nullptr, 1);
    const bool w_ready = !few_rows(sx) || (aligned16(w, dtype) && sb * es % 16 == 0) ||
                         packed_bytes(dtype, w.rows, w.cols, E ? E : 1) <= kCopyBytes;
    const Config both = dX && dW && M > 0 && K > 0 && N > 0 && w_ready ? choose_gradients(sx, sw) : kConfigs;
    if (dX && (!few_rows(sx) || both != kConfigs)) packs.add(w, &sb, E ? E : 1);
    if (dW) packs.add(x, nullptr, 1);
    GradArgs a{};
    if (N > 0 && (act != CP_ACT_NONE || db)) {
        a.dy = (const char *)dy.p;
        a.ldd = dy.ld;
        if (act != CP_ACT_NONE) {
            a.pre = (const char *)z.p;
            a.ldp = z.ld;
            a.dz = (char *)const_cast<void *>(dz.p);
            a.ldz = dz.ld;
        }
        a.db = (char *)db;
        a.ws = (float *)sums;
        a.off = off;
        a.groups = E ? E : 1;
        a.M = (int)M;
        a.N = (int)N;
        a.act = act;
        const Shape rows{dtype, kNN, E ? kGroupRows : kDense, M, N, K, E};
        a.tiles = (int)max_row_tiles(rows, kGradRows);
        a.vec = aligned16(dy, dtype) && (act == CP_ACT_NONE || aligned16(z, dtype));
        a.final = !E && a.tiles == 1;
        CP_TRY(launched(launch_grad(dtype, a, packs.a, s), "activation gradient"));
    } else {
        CP_TRY(packs.launch(s));
    }
    Product px{}, pw{};
    px.s = sx;
    px.A = dz;
    px.B = w;
    px.C = dx;
    px.sb = sb;
    px.off = off;
    pw.s = sw;
    pw.A = wt ? dz : x;
    pw.B = wt ? x : dz;
    pw.C = dw;
    pw.sc = E > 1 ? stride_dw : 0;
    pw.off = off;
    if (both != kConfigs) {
        GemmArgs gx, gw;
        const int64_t nx = launch_args(px, {both, 1}, split, gx, false),
                      nw = launch_args(pw, {both, 1}, split, gw, false);
        if (nx < 0 || nw < 0) return (int)(nx < 0 ? nx : nw);
        const int nd = db && !a.final ? grad_join_blocks(a) : 0;
        return launched((dtype == CP_BF16 ? launch_gradients_bf16 : launch_gradients_f32)(sx.layout, both, gx, (int)nx, gw,
                                                                                         (int)nw, a, nd, s),
                        "gradients");
    }
    if (db && N > 0 && !a.final) CP_TRY(launched(launch_grad_join(dtype, a, s), "bias gradient"));
    if (dX) CP_TRY(run_product(px, split, s));
    if (dW) CP_TRY(run_product(pw, split, s));
    return CP_OK;
}

}  // namespace

extern "C" {

const char *cp_ops_last_error(void) { return g_error; }

int64_t cp_ops_workspace(int32_t op, int32_t dtype, int64_t M, int64_t K, int64_t N, int32_t E, int32_t aligned) {
    g_error[0] = 0;
    CP_TRY(check_dtype(dtype));
    CP_TRY(check_sizes(M, op == CP_OP_LAYER_NORM_BACKWARD ? 0 : K, N));
    const bool grouped = op == CP_OP_GROUPED_LINEAR || op == CP_OP_GROUPED_LINEAR_BACKWARD;
    if (grouped && (E < 1 || E > CP_OPS_MAX_GROUPS))
        return fail(CP_ERR_SHAPE, "%d experts (1 to %d)", E, CP_OPS_MAX_GROUPS);
    switch (op) {
        case CP_OP_LINEAR: return forward_ws(dtype, M, K, N, 0, aligned != 0);
        case CP_OP_GROUPED_LINEAR: return forward_ws(dtype, M, K, N, E, aligned != 0);
        case CP_OP_LINEAR_BACKWARD: return backward_ws(dtype, M, K, N, 0, aligned != 0);
        case CP_OP_GROUPED_LINEAR_BACKWARD: return backward_ws(dtype, M, K, N, E, aligned != 0);
        case CP_OP_LAYER_NORM_BACKWARD: return norm_ws(M, N);
    }
    return fail(CP_ERR_INVALID_ARG, "operator code %d", op);
}

int cp_linear(int32_t dtype, int64_t M, int64_t K, int64_t N, const void *X, int64_t ldx, const void *W, int64_t ldw,
              int32_t w_trans, const void *bias, const void *R, int64_t ldr, int32_t act, void *Y, int64_t ldy,
              void *pre, int64_t ldp, void *ws, int64_t ws_bytes, void *stream) {
    g_error[0] = 0;
    return forward(dtype, M, K, N, 0, X, ldx, W, ldw, 0, w_trans != 0, nullptr, bias, R, ldr, act, Y, ldy, pre, ldp, ws,
                   ws_bytes, stream);
}

int cp_linear_backward(int32_t dtype, int64_t M, int64_t K, int64_t N, const void *dY, int64_t lddy, const void *X,
                       int64_t ldx, const void *W, int64_t ldw, int32_t w_trans, const void *pre, int64_t ldp,
                       int32_t act, void *dX, int64_t lddx, void *dW, int64_t lddw, void *db, void *ws,
                       int64_t ws_bytes, void *stream) {
    g_error[0] = 0;
    return backward(dtype, M, K, N, 0, dY, lddy, X, ldx, W, ldw, 0, w_trans != 0, nullptr, pre, ldp, act, dX, lddx, dW,
                    lddw, 0, db, ws, ws_bytes, stream);
}

int cp_grouped_linear(int32_t dtype, int64_t T, int64_t K, int64_t N, int32_t E, const void *X, int64_t ldx,
                      const void *W, int64_t ldw, int64_t stride_w, int32_t w_trans, const int32_t *offsets,
                      const void *bias, int32_t act, void *Y, int64_t ldy, void *pre, int64_t ldp, void *ws,
                      int64_t ws_bytes, void *stream) {
    g_error[0] = 0;
    if (E < 1) return fail(CP_ERR_SHAPE, "%d experts (1 to %d)", E, CP_OPS_MAX_GROUPS);
    return forward(dtype, T, K, N, E, X, ldx, W, ldw, stride_w, w_trans != 0, offsets, bias, nullptr, 0, act, Y, ldy,
                   pre, ldp, ws, ws_bytes, stream);
}

int cp_grouped_linear_backward(int32_t dtype, int64_t T, int64_t K, int64_t N, int32_t E, const void *dY, int64_t lddy,
                               const void *X, int64_t ldx, const void *W, int64_t ldw, int64_t stride_w,
                               int32_t w_trans, const int32_t *offsets, const void *pre, int64_t ldp, int32_t act,
                               void *dX, int64_t lddx, void *dW, int64_t lddw, int64_t stride_dw, void *db, void *ws,
                               int64_t ws_bytes, void *stream) {
    g_error[0] = 0;
    if (E < 1) return fail(CP_ERR_SHAPE, "%d experts (1 to %d)", E, CP_OPS_MAX_GROUPS);
    return backward(dtype, T, K, N, E, dY, lddy, X, ldx, W, ldw, stride_w, w_trans != 0, offsets, pre, ldp, act, dX,
                    lddx, dW, lddw, stride_dw, db, ws, ws_bytes, stream);
}

int cp_layer_norm(int32_t dtype, int64_t M, int64_t N, const void *X, int64_t ldx, const void *w, const void *b,
                  float eps, void *Y, int64_t ldy, float *mean, float *rstd, void *stream) {
    g_error[0] = 0;
    CP_TRY(check_dtype(dtype));
    CP_TRY(check_sizes(M, 0, N));
    if (!(eps >= 0.0f)) return fail(CP_ERR_INVALID_ARG, "eps %g", (double)eps);
    if (M == 0) return CP_OK;
    if (N == 0) return fail(CP_ERR_SHAPE, "rows without elements have no mean");
    Mat x{X, M, N, ldx}, y{Y, M, N, ldy};
    CP_TRY(check_mat(x, dtype, "X"));
    CP_TRY(check_mat(y, dtype, "Y"));
    CP_TRY(check_vector(w, dtype, "w"));
    CP_TRY(check_vector(b, dtype, "b"));
    const Rows out(y, dtype);
    CP_TRY(check_apart("Y", out, "X", Rows(x, dtype), true));
    CP_TRY(check_apart("Y", out, "w", Rows(w, N * elem_size(dtype))));
    CP_TRY(check_apart("Y", out, "b", Rows(b, N * elem_size(dtype))));
    NormArgs a{};
    a.x = (const char *)X;
    a.w = (const char *)w;
    a.b = (const char *)b;
    a.y = (char *)Y;
    a.mean = mean;
    a.rstd = rstd;
    a.ldx = x.ld;
    a.ldy = y.ld;
    a.M = (int)M;
    a.N = (int)N;
    a.eps = eps;
    a.vec = aligned16(x, dtype) && aligned16(y, dtype) && aligned16(w) && aligned16(b);
    return launched(launch_norm(dtype, a, (hipStream_t)stream), "layer norm");
}

int cp_layer_norm_backward(int32_t dtype, int64_t M, int64_t N, const void *dY, int64_t lddy, const void *X,
                           int64_t ldx, const float *mean, const float *rstd, const void *w, void *dX, int64_t lddx,
                           void *dw, void *db, void *ws, int64_t ws_bytes, void *stream) {
    g_error[0] = 0;
    CP_TRY(check_dtype(dtype));
    CP_TRY(check_sizes(M, 0, N));
    if (N == 0 || (!dX && !dw && !db)) return CP_OK;
    Mat dy{dY, M, N, lddy}, x{X, M, N, ldx}, dx{dX, M, N, lddx};
    CP_TRY(check_mat(dy, dtype, "dY"));
    CP_TRY(check_mat(x, dtype, "X"));
    if (dX) CP_TRY(check_mat(dx, dtype, "dX"));
    if (M > 0 && (!mean || !rstd)) return fail(CP_ERR_INVALID_ARG, "mean or rstd is NULL");
    CP_TRY(check_vector(w, dtype, "w"));
    CP_TRY(check_vector(dw, dtype, "dw"));
    CP_TRY(check_vector(db, dtype, "db"));
    NormArgs a{};
    a.blocks = norm_backward_blocks(M, N);
    CP_TRY(check_ws(ws, ws_bytes, norm_ws(M, N)));
    a.x = (const char *)X;
    a.dy = (const char *)dY;
    a.w = (const char *)w;
    a.y = (char *)dX;
    a.dw = (char *)dw;
    a.db = (char *)db;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.ws = (float *)ws;
    a.ldx = x.ld;
    a.ldd = dy.ld;
    a.ldy = dx.ld;
    a.M = (int)M;
    a.N = (int)N;
    a.vec = aligned16(dy, dtype) && aligned16(x, dtype) && aligned16(dx, dtype) && aligned16(w);
    return launched(launch_norm_backward(dtype, a, (hipStream_t)stream), "layer norm backward");
}

}  // extern "C"
