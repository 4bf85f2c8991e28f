// cp_ops_experts.cpp -- host side of the operators around a feed-forward block's
// products (include/cp_ops.h): router, exchange of rows with the experts, 4-bit
// linear layers, gradient norm and clipping.  Argument checks and launches.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "cp_ops_check.h"
#include "cp_ops_experts.h"

using namespace cpo;

namespace {

int check_words(const void *p, int64_t n, const char *name) {
    if (n == 0) return CP_OK;
    if (!p) return fail(CP_ERR_INVALID_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % 4) return fail(CP_ERR_INVALID_ARG, "%s is misaligned", name);
    return CP_OK;
}

// Blocks of a launch in one dimension.
int check_grid(int64_t blocks, int threads) {
    if (blocks > max_blocks(threads) || blocks > INT32_MAX)
        return fail(CP_ERR_SHAPE, "too many workgroups (%lld)", (long long)blocks);
    return CP_OK;
}

// ------------------------------------------------------------------- router

int check_route(int dtype, int64_t T, int E, int k) {
    CP_TRY(check_dtype(dtype));
    if (E < 1 || E > CP_OPS_MAX_ROUTED) return fail(CP_ERR_SHAPE, "%d experts (1 to %d)", E, CP_OPS_MAX_ROUTED);
    if (k < 1 || k > E || k > CP_OPS_MAX_CHOSEN)
        return fail(CP_ERR_SHAPE, "%d of %d experts to a token (1 to %d)", k, E, E < CP_OPS_MAX_CHOSEN ? E : CP_OPS_MAX_CHOSEN);
    if (T < 0 || T > kMaxRows / k) return fail(CP_ERR_SHAPE, "%lld tokens of %d slots (at most 2^30 slots)", (long long)T, k);
    return CP_OK;
}

// ----------------------------------------------------------------- exchange

int check_exchange(int dtype, int64_t T, int k, int64_t R, int64_t D, const int32_t *rows) {
    CP_TRY(check_dtype(dtype));
    if (k < 1 || k > CP_OPS_MAX_CHOSEN) return fail(CP_ERR_SHAPE, "%d slots to a token (1 to %d)", k, CP_OPS_MAX_CHOSEN);
    if (T < 0 || R < 0 || D < 0 || T > kMaxRows / k || R > kMaxRows || D > CP_OPS_MAX_WIDTH)
        return fail(CP_ERR_SHAPE, "size out of range (T=%lld k=%d R=%lld D=%lld; at most 2^30 slots and rows, %d columns)",
                    (long long)T, k, (long long)R, (long long)D, CP_OPS_MAX_WIDTH);
    return check_words(rows, T * k, "rows");
}

// ------------------------------------------------------------- 4-bit weights

int check_int4(int dtype, int64_t K, int64_t N, int64_t E, int64_t group) {
    CP_TRY(check_dtype(dtype));
    CP_TRY(check_sizes(0, K, N));
    if (E < 1 || E > CP_OPS_MAX_GROUPS) return fail(CP_ERR_SHAPE, "%lld experts (1 to %d)", (long long)E, CP_OPS_MAX_GROUPS);
    if (group != 32 && group != 64 && (group < 128 || group % 128 || group > CP_OPS_MAX_WIDTH))
        return fail(CP_ERR_UNSUPPORTED, "groups of %lld (32, 64 or a multiple of 128)", (long long)group);
    return CP_OK;
}

int linear_int4(int dtype, int64_t M, int64_t K, int64_t N, int E, const void *X, int64_t ldx, const void *packed,
                int64_t group, const int32_t *off, const void *bias, const void *R, int64_t ldr, int act,
                void *Y, int64_t ldy, void *ws, int64_t ws_bytes, void *stream) {
    CP_TRY(check_int4(dtype, K, N, E ? E : 1, group));
    CP_TRY(check_sizes(M, K, N));
    CP_TRY(check_act(act));
    Mat x{X, M, K, ldx}, y{Y, M, N, ldy}, r{R, M, N, ldr};
    CP_TRY(check_mat(x, dtype, "X"));
    CP_TRY(check_mat(y, dtype, "Y"));
    if (R) CP_TRY(check_mat(r, dtype, "R"));
    CP_TRY(check_vector(bias, dtype, "bias"));
    if (E) CP_TRY(check_words(off, E + 1, "offsets"));
    const Int4Layout l(dtype, K, N, group);
    const int64_t experts = E ? E : 1;
    if (M && N && K) {
        if (!packed) return fail(CP_ERR_INVALID_ARG, "the packed weight is NULL");
        if (!aligned16(packed)) return fail(CP_ERR_INVALID_ARG, "the packed weight is not 16-byte aligned");
    }
    const Rows out(y, dtype);
    CP_TRY(check_apart("Y", out, "X", Rows(x, dtype)));
    CP_TRY(check_apart("Y", out, "the packed weight", Rows(packed, l.bytes(experts))));
    CP_TRY(check_apart("Y", out, "bias", Rows(bias, experts * N * elem_size(dtype))));
    CP_TRY(check_apart("Y", out, "offsets", Rows(off, (E + 1) * 4)));
    if (R) CP_TRY(check_apart("Y", out, "R", Rows(r, dtype), true));
    CP_TRY(check_ws(ws, ws_bytes, int4_ws(dtype, E, M, K, N)));
    if (M == 0 || N == 0) return CP_OK;
    Int4Args a{};
    a.x = (const char *)X;
    a.codes = (const char *)packed;
    a.meta = a.codes + experts * l.codes;
    a.bias = (const char *)bias;
    a.res = (const char *)R;
    a.y = (char *)Y;
    a.ldx = x.ld;
    a.ldr = r.ld;
    a.ldy = y.ld;
    a.sc = l.codes;
    a.sm = l.meta;
    a.off = off;
    a.experts = E;
    a.M = (int)M;
    a.K = (int)K;
    a.N = (int)N;
    a.act = act;
    a.ntiles = (int)l.ntiles;
    a.kblocks = (int)l.kblocks;
    a.ngroups = (int)l.ngroups;
    a.group = (int)group;
    const Int4Tiles t = int4_tiles(dtype, E, M, l.ntiles, l.kblocks, group);
    CP_TRY(check_grid((int64_t)t.ntm * t.ntn * t.chunks, 1024));
    a.ntm = t.ntm;
    a.ntn = t.ntn;
    a.chunks = t.chunks;
    a.kper = t.kper;
    a.ws = (float *)ws;
    a.ldws = up(N, 8);
    // (without a contraction the kernels would have no tile to read: the join's sum over no part is zero)
    if (K > 0) CP_TRY(launched(launch_int4(dtype, a, t, (hipStream_t)stream), "4-bit linear layer"));
    if (K > 0 && t.chunks == 1) return CP_OK;
    GemmArgs g{};
    g.C = a.y;
    g.bias = a.bias;
    g.res = a.res;
    g.ws = a.ws;
    g.ldc = a.ldy;
    g.ldr = a.ldr;
    g.off = off;
    g.groups = E;
    g.mode = E ? kGroupRows : kDense;
    g.M = a.M;
    g.N = a.N;
    g.act = act;
    g.nsplit = K > 0 ? t.chunks : 0;
    g.ldws = (int32_t)a.ldws;
    g.vec = aligned16(y, dtype) && (!R || aligned16(r, dtype)) && aligned16(bias);
    return launched(launch_join(dtype, g, (hipStream_t)stream), "join");
}

// ----------------------------------------------------------------- clipping

// Outputs against everything, except against their own input.
int check_clip_memory(int64_t n, const int32_t *dtypes, const void *const *grads, const int64_t *numels,
                      const int32_t *out_dtypes, void *const *outs) {
    struct Span {
        uintptr_t from, to;
        int64_t i;
        bool out;
    };
    std::vector<Span> spans;
    spans.reserve(2 * n);
    for (int64_t i = 0; i < n; ++i) {
        if (!numels[i]) continue;
        const uintptr_t x = (uintptr_t)grads[i], y = (uintptr_t)outs[i];
        const bool same = x == y && dtypes[i] == out_dtypes[i];
        spans.push_back({x, x + numels[i] * elem_size(dtypes[i]), i, same});
        if (!same) spans.push_back({y, y + numels[i] * elem_size(out_dtypes[i]), i, true});
    }
    auto before = [](const Span &a, const Span &b) { return a.from < b.from; };
    if (!std::is_sorted(spans.begin(), spans.end(), before)) std::sort(spans.begin(), spans.end(), before);
    uintptr_t all = 0, written = 0;  // ends so far
    for (const Span &s : spans) {
        if (s.from < (s.out ? all : written))
            return fail(CP_ERR_INVALID_ARG, "%s %lld shares memory with another tensor", s.out ? "output" : "gradient",
                        (long long)s.i);
        all = std::max(all, s.to);
        if (s.out) written = std::max(written, s.to);
    }
    return CP_OK;
}

// The launches for `total` elements, up to N tensors that are not empty to a launch.
template <int N>
int launch_clips(int64_t n, int64_t total, const int32_t *dtypes, const void *const *grads, const int64_t *numels,
                 float max_norm, const int32_t *out_dtypes, void *const *outs, float *norm, double *partial, hipStream_t s) {
    const int chunk = clip_chunk(total);
    auto fill = [&](int64_t *i) {  // from tensor *i on
        ClipArgs<N> a{};
        a.max_norm = max_norm;
        a.chunk = chunk;
        for (; *i < n && a.n < N; ++*i) {
            if (!numels[*i]) continue;
            const int64_t own = ceil_div(numels[*i], chunk);
            a.x[a.n] = (const char *)grads[*i];
            a.y[a.n] = outs ? (char *)outs[*i] : nullptr;
            a.before[a.n] = a.chunks;
            a.last[a.n] = (int32_t)(numels[*i] - (own - 1) * chunk);
            if (dtypes[*i] == CP_BF16) a.bf16_in[a.n >> 5] |= 1u << (a.n & 31);
            if (outs && out_dtypes[*i] == CP_BF16) a.bf16_out[a.n >> 5] |= 1u << (a.n & 31);
            a.chunks += (int32_t)own;
            ++a.n;
        }
        a.blocks = (int)std::min<int64_t>(a.chunks, kClipBlocks);
        return a;
    };
    int64_t i = 0;
    int nall = 0;
    while (i < n) {
        ClipArgs<N> a = fill(&i);
        if (!a.n) break;
        a.partial = partial + nall;
        nall += a.blocks;
        CP_TRY(launched(launch_norm_partials(a, s), "gradient norm"));
    }
    if (nall > kClipPartials) {
        CP_TRY(launched(launch_norm_total(partial, nall, s), "gradient norm"));
        nall = 1;
    }
    bool first = true;
    for (i = 0; first || (outs && i < n); first = false) {  // (one for the norm, also of nothing)
        ClipArgs<N> a = fill(&i);
        if (!a.n && !first) break;
        a.all = partial;
        a.nall = nall;
        a.norm = first ? norm : nullptr;
        a.blocks = outs && a.n ? (int)std::min<int64_t>(a.chunks, 2 * kClipBlocks) : 1;
        CP_TRY(launched(launch_clip(a, s), "gradient clipping"));
    }
    return CP_OK;
}

int clip(int64_t n, const int32_t *dtypes, const void *const *grads, const int64_t *numels, float max_norm,
         const int32_t *out_dtypes, void *const *outs, float *norm, void *ws, int64_t ws_bytes, hipStream_t s) {
    if (n < 0 || n > CP_OPS_MAX_TENSORS) return fail(CP_ERR_SHAPE, "%lld tensors (at most %d)", (long long)n, CP_OPS_MAX_TENSORS);
    if (n && (!dtypes || !grads || !numels || (outs && !out_dtypes)))
        return fail(CP_ERR_INVALID_ARG, "a list of tensors is NULL");
    if (!(max_norm >= 0.0f)) return fail(CP_ERR_INVALID_ARG, "max_norm %g", (double)max_norm);
    CP_TRY(check_words(norm, 1, "norm"));
    int64_t total = 0, used = 0;
    for (int64_t i = 0; i < n; ++i) {
        CP_TRY(check_dtype(dtypes[i]));
        if (outs) CP_TRY(check_dtype(out_dtypes[i]));
        // (chunks of 16384 are counted in 32 bits)
        if (numels[i] < 0 || numels[i] > (int64_t(1) << 44) - total)
            return fail(CP_ERR_SHAPE, "tensor %lld: %lld elements (at most 2^44 in all)", (long long)i, (long long)numels[i]);
        if (!numels[i]) continue;
        if (!grads[i] || (outs && !outs[i])) return fail(CP_ERR_INVALID_ARG, "tensor %lld is NULL", (long long)i);
        CP_TRY(check_vector(grads[i], dtypes[i], "a gradient"));
        if (outs) CP_TRY(check_vector(outs[i], out_dtypes[i], "an output"));
        CP_TRY(check_apart("norm", Rows(norm, 4), "a gradient", Rows(grads[i], numels[i] * elem_size(dtypes[i]))));
        if (outs) CP_TRY(check_apart("norm", Rows(norm, 4), "an output", Rows(outs[i], numels[i] * elem_size(out_dtypes[i]))));
        total += numels[i];
        ++used;
    }
    CP_TRY(check_ws(ws, ws_bytes, clip_ws(n)));
    if (outs) CP_TRY(check_clip_memory(n, dtypes, grads, numels, out_dtypes, outs));
    return (used <= kClipFew ? launch_clips<kClipFew> : launch_clips<kClipTensors>)(n, total, dtypes, grads, numels, max_norm,
                                                                                    out_dtypes, outs, norm, (double *)ws, s);
}

}  // namespace

extern "C" {

int cp_route(int32_t dtype, int64_t T, int32_t E, int32_t k, int32_t normalize, const void *logits, int64_t ld,
             const uint8_t *valid, int32_t *experts, float *gates, int32_t *rows, int32_t *counts, int32_t *offsets,
             float *loss, float *slopes, void *ws, int64_t ws_bytes, void *stream) {
    g_error[0] = 0;
    CP_TRY(check_route(dtype, T, E, k));
    Mat x{logits, T, E, ld};
    CP_TRY(check_mat(x, dtype, "logits"));
    CP_TRY(check_words(experts, T, "experts"));
    CP_TRY(check_words(gates, T, "gates"));
    CP_TRY(check_words(rows, T, "rows"));
    CP_TRY(check_words(counts, 1, "counts"));
    CP_TRY(check_words(offsets, 1, "offsets"));
    CP_TRY(check_words(loss, 1, "loss"));
    CP_TRY(check_words(slopes, 1, "slopes"));
    CP_TRY(check_ws(ws, ws_bytes, route_ws(T, E)));
    RouteArgs a{};
    a.logits = (const char *)logits;
    a.valid = valid;
    a.ld = x.ld;
    a.experts = experts;
    a.rows = rows;
    a.counts = counts;
    a.offsets = offsets;
    a.gates = gates;
    a.loss = loss;
    a.slopes = slopes;
    a.T = (int)T;
    a.E = E;
    a.k = k;
    a.normalize = normalize;
    a.blocks = route_blocks(T, E);
    a.chunks = route_chunks(T, E);
    a.hist = (int32_t *)ws;
    a.stride = (int)up(E, 4);
    a.psum = (float *)(a.hist + (int64_t)a.blocks * a.stride);
    a.live = (int32_t *)(a.psum + (int64_t)a.blocks * a.stride);
    return launched(launch_route(dtype, a, (hipStream_t)stream), "router");
}

int cp_route_backward(int32_t dtype, int64_t T, int32_t E, int32_t k, int32_t normalize, const float *dgates,
                      const float *dloss, const void *logits, int64_t ld, const int32_t *experts, const float *slopes,
                      void *dlogits, int64_t ldd, void *stream) {
    g_error[0] = 0;
    CP_TRY(check_route(dtype, T, E, k));
    Mat x{logits, T, E, ld}, d{dlogits, T, E, ldd};
    CP_TRY(check_mat(x, dtype, "logits"));
    CP_TRY(check_mat(d, dtype, "dlogits"));
    CP_TRY(check_words(experts, T, "experts"));
    CP_TRY(check_words(dgates, dgates ? 1 : 0, "dgates"));
    CP_TRY(check_words(dloss, dloss ? 1 : 0, "dloss"));
    CP_TRY(check_words(slopes, dloss ? 1 : 0, "slopes"));
    CP_TRY(check_apart("dlogits", Rows(d, dtype), "logits", Rows(x, dtype), true));
    if (T == 0) return CP_OK;
    RouteGradArgs a{};
    a.logits = (const char *)logits;
    a.experts = experts;
    a.dgates = dgates;
    a.dloss = dloss;
    a.slopes = slopes;
    a.dlogits = (char *)dlogits;
    a.ld = x.ld;
    a.ldd = d.ld;
    a.T = (int)T;
    a.E = E;
    a.k = k;
    a.normalize = normalize;
    return launched(launch_route_backward(dtype, a, (hipStream_t)stream), "router backward");
}

int cp_dispatch(int32_t dtype, int64_t T, int32_t k, int64_t R, int64_t D, const void *x, int64_t ldx,
                const int32_t *rows, const int32_t *end, void *out, int64_t ldo, void *stream) {
    g_error[0] = 0;
    CP_TRY(check_exchange(dtype, T, k, R, D, rows));
    Mat mx{x, T, D, ldx}, mo{out, R, D, ldo};
    CP_TRY(check_mat(mx, dtype, "x"));
    CP_TRY(check_mat(mo, dtype, "out"));
    CP_TRY(check_words(end, R, "end"));
    CP_TRY(check_apart("out", Rows(mo, dtype), "x", Rows(mx, dtype)));
    CP_TRY(check_apart("out", Rows(mo, dtype), "rows", Rows(rows, T * k * 4)));
    CP_TRY(check_apart("out", Rows(mo, dtype), "end", Rows(end, 4)));
    if (D == 0 || R == 0) return CP_OK;
    ExchangeArgs a{};
    a.x = (const char *)x;
    a.out = (char *)out;
    a.rows = rows;
    a.end = end;
    a.ldx = mx.ld;
    a.ldo = mo.ld;
    a.T = T;
    a.R = R;
    a.k = k;
    a.D = (int)D;
    return launched(launch_dispatch(dtype, a, (hipStream_t)stream), "dispatch");
}

int cp_combine(int32_t dtype, int64_t T, int32_t k, int64_t R, int64_t D, const void *y, int64_t ldy,
               const int32_t *rows, const float *gates, const void *res, int64_t ldr, void *out, int64_t ldo,
               void *stream) {
    g_error[0] = 0;
    CP_TRY(check_exchange(dtype, T, k, R, D, rows));
    Mat my{y, R, D, ldy}, mr{res, T, D, ldr}, mo{out, T, D, ldo};
    CP_TRY(check_mat(my, dtype, "y"));
    CP_TRY(check_mat(mo, dtype, "out"));
    if (res) CP_TRY(check_mat(mr, dtype, "res"));
    CP_TRY(check_words(gates, gates ? 1 : 0, "gates"));
    const Rows o(mo, dtype);
    CP_TRY(check_apart("out", o, "y", Rows(my, dtype)));
    CP_TRY(check_apart("out", o, "rows", Rows(rows, T * k * 4)));
    CP_TRY(check_apart("out", o, "gates", Rows(gates, T * k * 4)));
    if (res) CP_TRY(check_apart("out", o, "res", Rows(mr, dtype), true));
    if (D == 0 || T == 0) return CP_OK;
    ExchangeArgs a{};
    a.y = (const char *)y;
    a.res = (const char *)res;
    a.out = (char *)out;
    a.rows = rows;
    a.gates = gates;
    a.ldy = my.ld;
    a.ldr = mr.ld;
    a.ldo = mo.ld;
    a.T = T;
    a.R = R;
    a.k = k;
    a.D = (int)D;
    return launched(launch_combine(dtype, a, (hipStream_t)stream), "combine");
}

int cp_combine_backward(int32_t dtype, int64_t T, int32_t k, int64_t R, int64_t D, const void *dout, int64_t ldd,
                        const void *y, int64_t ldy, const int32_t *rows, const int32_t *end, const float *gates,
                        void *dy, int64_t lddy, float *dgates, void *stream) {
    g_error[0] = 0;
    CP_TRY(check_exchange(dtype, T, k, R, D, rows));
    Mat md{dout, T, D, ldd}, my{y, R, D, ldy}, mo{dy, R, D, lddy};
    CP_TRY(check_mat(md, dtype, "dout"));
    if (dgates) CP_TRY(check_mat(my, dtype, "y"));
    CP_TRY(check_words(gates, gates ? 1 : 0, "gates"));
    CP_TRY(check_words(dgates, dgates ? 1 : 0, "dgates"));
    const Rows in_rows(rows, T * k * 4), in_gates(gates, T * k * 4), in_end(dy ? end : nullptr, 4), slots(dgates, T * k * 4);
    if (dy) {
        CP_TRY(check_mat(mo, dtype, "dy"));
        CP_TRY(check_words(end, R, "end"));
        const Rows o(mo, dtype);
        CP_TRY(check_apart("dy", o, "dout", Rows(md, dtype)));
        if (dgates) CP_TRY(check_apart("dy", o, "y", Rows(my, dtype)));
        CP_TRY(check_apart("dy", o, "rows", in_rows));
        CP_TRY(check_apart("dy", o, "gates", in_gates));
        CP_TRY(check_apart("dy", o, "end", in_end));
        CP_TRY(check_apart("dgates", slots, "dy", o));
    }
    if (dgates) {
        CP_TRY(check_apart("dgates", slots, "dout", Rows(md, dtype)));
        CP_TRY(check_apart("dgates", slots, "y", Rows(my, dtype)));
        CP_TRY(check_apart("dgates", slots, "rows", in_rows));
        CP_TRY(check_apart("dgates", slots, "gates", in_gates));
        CP_TRY(check_apart("dgates", slots, "end", in_end));
    }
    if (!dy && !dgates) return CP_OK;
    if (T == 0 && (!dy || R == 0 || D == 0)) return CP_OK;
    ExchangeArgs a{};
    a.x = (const char *)dout;
    a.y = (const char *)y;
    a.dy = D && R ? (char *)dy : nullptr;
    a.rows = rows;
    a.end = end;
    a.gates = gates;
    a.dgates = dgates;
    a.ldx = md.ld;
    a.ldy = my.ld;
    a.lddy = mo.ld;
    a.T = T;
    a.R = R;
    a.k = k;
    a.D = (int)D;
    return launched(launch_combine_backward(dtype, a, (hipStream_t)stream), "combine backward");
}

int cp_int4_quantize(int32_t dtype, int64_t K, int64_t N, int32_t E, int64_t group, const void *W, int64_t stride_k,
                     int64_t stride_n, int64_t stride_e, uint8_t *codes, void *scales, uint8_t *zeros, void *stream) {
    g_error[0] = 0;
    CP_TRY(check_int4(dtype, K, N, E, group));
    if (K == 0 || N == 0) return CP_OK;
    if (!W || !codes || !scales) return fail(CP_ERR_INVALID_ARG, "W, codes or scales is NULL");
    CP_TRY(check_vector(W, dtype, "W"));
    CP_TRY(check_vector(scales, dtype, "scales"));
    if (stride_k < 0 || stride_n < 0 || stride_e < 0) return fail(CP_ERR_SHAPE, "negative stride");
    Int4QuantArgs a{};
    a.w = (const char *)W;
    a.sk = stride_k;
    a.sn = stride_n;
    a.se = stride_e;
    a.q = codes;
    a.zeros = zeros;
    a.scales = (char *)scales;
    a.K = K;
    a.N = N;
    a.E = E;
    a.group = (int)group;
    a.ngroups = (int)ceil_div(K, group);
    return launched(launch_int4_quantize(dtype, a, (hipStream_t)stream), "4-bit quantisation");
}

int64_t cp_int4_bytes(int32_t dtype, int64_t K, int64_t N, int32_t E, int64_t group) {
    g_error[0] = 0;
    CP_TRY(check_int4(dtype, K, N, E, group));
    return Int4Layout(dtype, K, N, group).bytes(E);
}

int cp_int4_pack(int32_t dtype, int64_t K, int64_t N, int32_t E, int64_t group, const uint8_t *codes,
                 const void *scales, const uint8_t *zeros, void *packed, void *stream) {
    g_error[0] = 0;
    CP_TRY(check_int4(dtype, K, N, E, group));
    if (K == 0 || N == 0) return CP_OK;
    if (!codes || !scales || !packed) return fail(CP_ERR_INVALID_ARG, "codes, scales or packed is NULL");
    CP_TRY(check_vector(scales, dtype, "scales"));
    if (!aligned16(packed)) return fail(CP_ERR_INVALID_ARG, "packed is not 16-byte aligned");
    const Int4Layout l(dtype, K, N, group);
    const Rows out(packed, l.bytes(E));
    CP_TRY(check_apart("packed", out, "codes", Rows(codes, E * K * N)));
    CP_TRY(check_apart("packed", out, "scales", Rows(scales, E * l.ngroups * N * elem_size(dtype))));
    CP_TRY(check_apart("packed", out, "zeros", Rows(zeros, E * l.ngroups * N)));
    Int4PackArgs a{};
    a.q = codes;
    a.zeros = zeros;
    a.scales = (const char *)scales;
    a.codes = (char *)packed;
    a.meta = a.codes + E * l.codes;
    a.K = K;
    a.N = N;
    a.E = E;
    a.ntiles = (int)l.ntiles;
    a.kblocks = (int)l.kblocks;
    a.ngroups = (int)l.ngroups;
    return launched(launch_int4_pack(dtype, a, (hipStream_t)stream), "4-bit packing");
}

int cp_linear_int4(int32_t dtype, int64_t M, int64_t K, int64_t N, const void *X, int64_t ldx, const void *packed,
                   int64_t group, const void *bias, const void *R, int64_t ldr, int32_t act,
                   void *Y, int64_t ldy, void *ws, int64_t ws_bytes, void *stream) {
    g_error[0] = 0;
    return linear_int4(dtype, M, K, N, 0, X, ldx, packed, group, nullptr, bias, R, ldr, act, Y, ldy, ws, ws_bytes, stream);
}

int cp_grouped_linear_int4(int32_t dtype, int64_t T, int64_t K, int64_t N, int32_t E, const void *X, int64_t ldx,
                           const void *packed, int64_t group, const int32_t *offsets,
                           const void *bias, int32_t act, void *Y, int64_t ldy, void *ws, int64_t ws_bytes,
                           void *stream) {
    g_error[0] = 0;
    if (E < 1) return fail(CP_ERR_SHAPE, "%d experts (1 to %d)", E, CP_OPS_MAX_GROUPS);
    return linear_int4(dtype, T, K, N, E, X, ldx, packed, group, offsets, bias, nullptr, 0, act, Y, ldy, ws, ws_bytes,
                       stream);
}

int cp_clip_grad_norm(int64_t n, const int32_t *dtypes, const void *const *grads, const int64_t *numels,
                      float max_norm, const int32_t *out_dtypes, void *const *outs, float *norm, void *ws,
                      int64_t ws_bytes, void *stream) {
    g_error[0] = 0;
    try {
        return clip(n, dtypes, grads, numels, max_norm, out_dtypes, outs, norm, ws, ws_bytes, (hipStream_t)stream);
    } catch (const std::bad_alloc &) {
        return fail(CP_ERR_OOM, "no memory for the lists of tensors");
    }
}

}  // extern "C"
