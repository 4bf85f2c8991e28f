// cp_ops_check.h -- argument checks that the host sides of the operators share,
// and the detail string of a thread's last failure.  Internal to the library.
#pragma once
#include <cstdarg>
#include <cstdio>
#include <numeric>

#include "cp_ops_host.h"

namespace cpo {

inline thread_local char g_error[512];

inline int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof g_error, fmt, ap);
    va_end(ap);
    return code;
}

inline int launched(hipError_t e, const char *what) {
    if (e == hipSuccess) return CP_OK;
    return fail(CP_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

constexpr int64_t kMaxRows = int64_t(1) << 30;

inline int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int elem_size(int dtype) { return dtype == CP_BF16 ? 2 : 4; }

// ------------------------------------------------------------------- checks

struct Mat {
    const void *p;
    int64_t rows, cols, ld;
};

inline int check_dtype(int dtype) {
    if (dtype != CP_F32 && dtype != CP_BF16) return fail(CP_ERR_UNSUPPORTED, "dtype %d is not supported", dtype);
    return CP_OK;
}

inline int check_sizes(int64_t M, int64_t K, int64_t N) {
    if (M < 0 || K < 0 || N < 0)
        return fail(CP_ERR_SHAPE, "negative size (M=%lld K=%lld N=%lld)", (long long)M, (long long)K, (long long)N);
    if (M > kMaxRows || K > CP_OPS_MAX_WIDTH || N > CP_OPS_MAX_WIDTH)
        return fail(CP_ERR_SHAPE, "size too large (M=%lld K=%lld N=%lld; at most 2^30 rows, %d columns)", (long long)M,
                    (long long)K, (long long)N, CP_OPS_MAX_WIDTH);
    return CP_OK;
}

inline int check_act(int act) {
    if (act < CP_ACT_NONE || act > CP_ACT_SILU) return fail(CP_ERR_UNSUPPORTED, "activation %d is not supported", act);
    return CP_OK;
}

// A matrix that is read or written; its ld is set to something usable where
// there is at most one row.
inline int check_mat(Mat &m, int dtype, const char *name) {
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

inline bool aligned16(const Mat &m, int dtype) {
    const int es = elem_size(dtype);
    return !m.p || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.ld * es % 16 == 0 && m.cols * es % 16 == 0);
}
inline bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

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
inline bool overlap_one(const Rows &a, const Rows &b) {
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
inline bool overlap(const Rows &a, Rows b) {
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
inline int check_apart(const char *name, const Rows &out, const char *other, const Rows &in, bool same = false) {
    if (same && out.p == in.p && (out.ld == in.ld || out.rows <= 1)) return CP_OK;
    if (overlap(out, in)) return fail(CP_ERR_INVALID_ARG, "%s overlaps %s", name, other);
    return CP_OK;
}

#define CP_TRY(expr)                  \
    do {                              \
        const int rc_ = (expr);       \
        if (rc_ != CP_OK) return rc_; \
    } while (0)

inline int check_ws(const void *ws, int64_t have, int64_t need) {
    if (need == 0) return CP_OK;
    if (!ws || have < need)
        return fail(CP_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", ws ? (long long)have : 0, (long long)need);
    if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(CP_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    return CP_OK;
}

inline int check_vector(const void *p, int dtype, const char *name) {
    if (reinterpret_cast<uintptr_t>(p) % elem_size(dtype)) return fail(CP_ERR_INVALID_ARG, "%s is misaligned", name);
    return CP_OK;
}

}  // namespace cpo
