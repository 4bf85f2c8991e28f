// cp_ops_clip.hip -- the norm over all the gradients of a model and their scaling:
// N = sqrt(sum x^2), x min(1, c / (N + 1e-6)).  Two passes over the tensors, a launch
// each for every 160 of them: the tensors are cut into chunks, numbered through, and
// their addresses ride in the launch's arguments.  Squares are added in 64 bits,
// which hold any fp32 value's square, and in an order that only the sizes set, so a
// norm does not depend on timing and no finite gradient overflows it.  Both
// passes are bound by memory, 64-bit sums run at the vector unit's full rate: 470 M
// elements bf16 to fp32 154 us for the norm (6.1 TB/s) and 542 to scale (5.2 TB/s).
// Of few elements each launch is its own latency: 2.1 M fp32 elements 10 to 11 us.
#include "cp_ops_experts.h"

namespace cpo {

namespace {

constexpr int kClipThreads = 256;

// The tensor that holds chunk c (uniform): the last that begins at or before it.  The
// arguments lie in the host's memory, so all are looked at at once: a search, step
// after step, waits for it each time.
template <class Args>
__device__ __forceinline__ int find_tensor(const Args &a, int c) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int base = 0; base < a.n; base += 64)
        n += __popcll(__ballot(base + lane < a.n && a.before[base + lane < a.n ? base + lane : 0] <= c));
    return n - 1;
}
__device__ __forceinline__ bool bit(const uint32_t *w, int i) { return w[i >> 5] >> (i & 31) & 1; }

// Sum over the block, every thread gets it; the order is fixed.
template <int NT>
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[NT / 64];
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) v += part[w];
    return v;
}

// Squares of n elements from p on.
template <class T, int NT>
__device__ __forceinline__ void add_squares(const char *p, int64_t n, double (&acc)[4]) {
    constexpr int CE = kUnit<T>, U = 4;
    int64_t i = (int64_t)threadIdx.x * CE;
    for (; i + (int64_t)(U - 1) * NT * CE + CE <= n; i += (int64_t)U * NT * CE) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) __builtin_memcpy(&v[u], p + (i + (int64_t)u * NT * CE) * (int64_t)sizeof(T), 16);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            T e[CE];
            __builtin_memcpy(e, &v[u], 16);
#pragma unroll
            for (int j = 0; j < CE; ++j) {
                const double d = (double)to_f32(e[j]);
                acc[j & 3] = fma(d, d, acc[j & 3]);
            }
        }
    }
    for (; i < n; i += (int64_t)NT * CE) {
        const uint4 v = load_partial<T>(p + i * (int64_t)sizeof(T), n - i < CE ? (int)(n - i) : CE);
        T e[CE];
        __builtin_memcpy(e, &v, 16);
#pragma unroll
        for (int j = 0; j < CE; ++j) {
            const double d = (double)to_f32(e[j]);
            acc[j & 3] = fma(d, d, acc[j & 3]);
        }
    }
}

// y = x f over n elements; x and y may be the same memory.  A lane takes 16 bytes of
// the wider type at a time, so that a wave stores whole lines, U such steps requested
// together.  Stores to 16-byte boundaries go past the caches, which keep more of the
// gradients for this second reading so: 134 M elements bf16 to bf16 148 -> 122 us.
template <class T, class O, int NT>
__device__ __forceinline__ void scale_to(const char *x, char *y, int64_t n, float f) {
    constexpr int CE = sizeof(T) == 4 || sizeof(O) == 4 ? 4 : 8, U = 32 / CE;
    typedef uint32_t word_t __attribute__((ext_vector_type(CE * sizeof(O) / 4)));
    const bool past = reinterpret_cast<uintptr_t>(y) % 16 == 0;
    T e[U][CE];
    auto load = [&](int u, int64_t i) { __builtin_memcpy(e[u], x + i * (int64_t)sizeof(T), sizeof e[u]); };
    auto store = [&](int u, int64_t i) {
        O o[CE];
#pragma unroll
        for (int j = 0; j < CE; ++j) o[j] = from_f32<O>(to_f32(e[u][j]) * f);
        word_t w;
        __builtin_memcpy(&w, o, sizeof o);
        char *to = y + i * (int64_t)sizeof(O);
        if (past) __builtin_nontemporal_store(w, reinterpret_cast<word_t *>(to));
        else __builtin_memcpy(to, &w, sizeof w);
    };
    int64_t i = (int64_t)threadIdx.x * CE;
    for (; i + (int64_t)(U - 1) * NT * CE + CE <= n; i += (int64_t)U * NT * CE) {
#pragma unroll
        for (int u = 0; u < U; ++u) load(u, i + (int64_t)u * NT * CE);
#pragma unroll
        for (int u = 0; u < U; ++u) store(u, i + (int64_t)u * NT * CE);
    }
    for (; i < n; i += (int64_t)NT * CE) {
        if (i + CE <= n) {
            load(0, i);
            store(0, i);
        } else {
            for (; i < n; ++i)
                reinterpret_cast<O *>(y)[i] = from_f32<O>(to_f32(reinterpret_cast<const T *>(x)[i]) * f);
        }
    }
}

// Where a block's chunk lies.
struct Piece {
    const char *x;
    char *y;
    int64_t n;
    bool bf16_in, bf16_out;
};
template <class Args>
__device__ __forceinline__ Piece piece_of(const Args &a, int c) {
    const int i = find_tensor(a, c), end = i + 1 < a.n ? a.before[i + 1] : a.chunks;
    const int64_t from = (int64_t)(c - a.before[i]) * a.chunk;
    const bool bi = bit(a.bf16_in, i), bo = bit(a.bf16_out, i);
    return {a.x[i] + from * (bi ? 2 : 4), a.y[i] + from * (bo ? 2 : 4), c + 1 < end ? a.chunk : a.last[i], bi, bo};
}

template <int NT, class Args>
__device__ __forceinline__ void square_chunk(const Args &a, int c, double (&acc)[4]) {
    const Piece p = piece_of(a, c);
    if (p.bf16_in) add_squares<__bf16, NT>(p.x, p.n, acc);
    else add_squares<float, NT>(p.x, p.n, acc);
}

template <int NT, class Args>
__device__ __forceinline__ void scale_chunk(const Args &a, int c, float f) {
    const Piece p = piece_of(a, c);
    if (f == 1.0f && p.y == p.x) return;  // in place, nothing to do
    if (p.bf16_in && p.bf16_out) scale_to<__bf16, __bf16, NT>(p.x, p.y, p.n, f);
    else if (p.bf16_in) scale_to<__bf16, float, NT>(p.x, p.y, p.n, f);
    else if (p.bf16_out) scale_to<float, __bf16, NT>(p.x, p.y, p.n, f);
    else scale_to<float, float, NT>(p.x, p.y, p.n, f);
}

__device__ __forceinline__ float clip_factor(double norm, float most) {
    const double f = (double)most / (norm + 1e-6);
    return f > 1.0 || most == __builtin_inff() ? 1.0f : (float)f;  // (a norm of NaN gives NaN)
}

template <int N>
__global__ __launch_bounds__(kClipThreads) void norm_partials_kernel(ClipArgs<N> a) {
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) square_chunk<kClipThreads>(a, c, acc);
    const double s = block_sum<kClipThreads>((acc[0] + acc[1]) + (acc[2] + acc[3]));
    if (threadIdx.x == 0) a.partial[blockIdx.x] = s;
}

// The sum of the partial sums: up to 8 of a thread requested together, in an order that
// their number alone sets.
__device__ __forceinline__ double sum_partials(const double *all, int n) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += 8 * kClipThreads) {
        double t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) t[u] = all[i + u * kClipThreads < n ? i + u * kClipThreads : i];
#pragma unroll
        for (int u = 0; u < 8; ++u) s += i + u * kClipThreads < n ? t[u] : 0.0;
    }
    return block_sum<kClipThreads>(s);
}

// One block: many launches' partial sums to their sum, in the place of the first.  (The
// sum's barriers lie between the last read and the write.)
__global__ __launch_bounds__(kClipThreads) void norm_total_kernel(double *all, int n) {
    const double s = sum_partials(all, n);
    if (threadIdx.x == 0) all[0] = s;
}

// Up to kClipPartials partial sums, 16 KB, are added up by every block, which spares a
// launch in between (norm_total_kernel); the chunks go last to first, as the last read
// are the ones that the caches still hold.  A block of one small chunk requests its
// elements before the partial sums, whose wait is as long.
template <int N>
__global__ __launch_bounds__(kClipThreads) void clip_kernel(ClipArgs<N> a) {
    const int c0 = a.chunks - 1 - (int)blockIdx.x;
    const bool single = a.y[0] && a.chunk == kClipThreads * 8 && c0 < (int)gridDim.x;  // (uniform)
    const int64_t at = (int64_t)threadIdx.x * 8;
    Piece p{};
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    bool whole = false;
    if (single) {
        p = piece_of(a, c0);
        whole = at + 8 <= p.n;
        if (whole) {  // (bf16: the same 16 bytes twice)
            const char *x = p.x + at * (p.bf16_in ? 2 : 4);
            __builtin_memcpy(&v0, x, 16);
            __builtin_memcpy(&v1, x + (p.bf16_in ? 0 : 16), 16);
        }
    }
    const double norm = sqrt(sum_partials(a.all, a.nall));
    if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
    const float f = clip_factor(norm, a.max_norm);
    if (!a.y[0]) return;  // (all have an output, or none)
    if (!single) {
        for (int c = c0; c >= 0; c -= (int)gridDim.x) scale_chunk<kClipThreads>(a, c, f);
        return;
    }
    if (f == 1.0f && p.x == p.y) return;
    float e[8];
    if (whole) {
        if (p.bf16_in) {
            __bf16 h[8];
            __builtin_memcpy(h, &v0, 16);
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = to_f32(h[j]) * f;
        } else {
            __builtin_memcpy(e, &v0, 16);
            __builtin_memcpy(e + 4, &v1, 16);
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] *= f;
        }
        if (p.bf16_out) {
            __bf16 h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = from_f32<__bf16>(e[j]);
            __builtin_memcpy(p.y + at * 2, h, 16);
        } else {
            __builtin_memcpy(p.y + at * 4, e, 32);
        }
        return;
    }
    for (int64_t i = at; i < p.n; ++i) {
        const float x = p.bf16_in ? to_f32(reinterpret_cast<const __bf16 *>(p.x)[i]) : reinterpret_cast<const float *>(p.x)[i];
        if (p.bf16_out) reinterpret_cast<__bf16 *>(p.y)[i] = from_f32<__bf16>(x * f);
        else reinterpret_cast<float *>(p.y)[i] = x * f;
    }
}

}  // namespace

hipError_t launch_norm_total(double *all, int n, hipStream_t s) {
    hipLaunchKernelGGL(norm_total_kernel, dim3(1), dim3(kClipThreads), 0, s, all, n);
    return hipGetLastError();
}
template <int N>
hipError_t launch_norm_partials(const ClipArgs<N> &a, hipStream_t s) {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(norm_partials_kernel<N>), dim3((unsigned)a.blocks), dim3(kClipThreads), 0, s, a);
    return hipGetLastError();
}
template <int N>
hipError_t launch_clip(const ClipArgs<N> &a, hipStream_t s) {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(clip_kernel<N>), dim3((unsigned)a.blocks), dim3(kClipThreads), 0, s, a);
    return hipGetLastError();
}
#define CP_CLIP(n)                                                            \
    template hipError_t launch_norm_partials<n>(const ClipArgs<n> &, hipStream_t); \
    template hipError_t launch_clip<n>(const ClipArgs<n> &, hipStream_t);
CP_CLIP(kClipFew)
CP_CLIP(kClipTensors)

}  // namespace cpo
