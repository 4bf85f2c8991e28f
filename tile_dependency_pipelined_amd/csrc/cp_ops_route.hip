// cp_ops_route.hip -- the router of an expert layer: softmax over a token's
// logits, the k largest, what each expert gets and the balance loss; and its
// gradient.
//
// A token's logits lie in the registers of LPR lanes, V consecutive ones each,
// so a wave works on 64 / LPR tokens at once and a reduction over the experts
// is V steps within a lane and a few cross-lane moves.  A token takes each
// expert at most once, so 64 tokens' choices of one expert are the bits of a
// word: a slot's place among its expert's is a count of the bits below its own,
// and does not depend on the order in which they were set.
#include "cp_ops_experts.h"

namespace cpo {

namespace {

// ------------------------------------------------- reductions over LPR lanes

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int l) { return __builtin_amdgcn_readlane(v, l); }

// Every lane gets its group's result.
template <int LPR, class Op>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, Op op) {
    static_assert(LPR == 4 || LPR == 8 || LPR == 16 || LPR == 64, "lanes per token");
    v = op(v, dpp<0xB1>(v));                             // quad_perm 1 0 3 2
    v = op(v, dpp<0x4E>(v));                             // quad_perm 2 3 0 1
    if constexpr (LPR >= 8) v = op(v, dpp<0x141>(v));    // row_half_mirror
    if constexpr (LPR >= 16) v = op(v, dpp<0x140>(v));   // row_mirror
    if constexpr (LPR == 64)
        v = op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
    return v;
}
template <int LPR>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    return group_reduce<LPR>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int LPR>
__device__ __forceinline__ float group_fmax(float v) {
    return __builtin_bit_cast(float, group_reduce<LPR>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
    }));
}
template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
    return __builtin_bit_cast(float, group_reduce<LPR>(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }));
}

// --------------------------------------------------------------- one token

// e^d for d <= 0 (or NaN): 2^t by the hardware with t = d log2(e) rounded, and
// what the rounding lost as a factor 1 + r ln 2.  Within about 2 ulp, where 2^t
// alone is off by |d| ulp.
__device__ __forceinline__ float exp_below_one(float d) {
    constexpr float hi = 1.44269502162933349609f, lo = 1.92596299112661746887e-8f;  // log2(e)
    d = d < -150.0f ? -150.0f : d;
    const float t = d * hi, r = fmaf(d, lo, fmaf(d, hi, -t));
    const float y = __builtin_amdgcn_exp2f(t);
    return fmaf(y * 0.693147180559945309f, r, y);
}

// A value's place in the order of choice: larger comes first, NaN before all,
// -inf and what is no expert: 0, never chosen.
__device__ __forceinline__ uint32_t order_key(float x) {
    x += 0.0f;  // -0 to 0: they tie
    const uint32_t b = __builtin_bit_cast(uint32_t, x), u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return x != x ? 0xFFFFFFFFu : (x == -__builtin_inff() ? 0u : u);
}

// V consecutive logits of a row from column c on; -inf past the last expert.
template <class T, int V>
__device__ __forceinline__ void load_logits(const char *row, int c, int E, float (&x)[V]) {
    const T *p = reinterpret_cast<const T *>(row) + c;
    if (c + V <= E) {
        T e[V];
        __builtin_memcpy(e, p, sizeof e);
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = to_f32(e[v]);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = c + v < E ? to_f32(p[v]) : -__builtin_inff();
    }
}

// Probabilities; all zero where every logit is -inf, all NaN with a NaN or inf
// among them.
template <int LPR, int V>
__device__ __forceinline__ void softmax(const float (&x)[V], float (&p)[V]) {
    float m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
    m = group_fmax<LPR>(m);
    m = m == -__builtin_inff() ? 0.0f : m;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        p[v] = exp_below_one(x[v] - m);
        p[v] = x[v] == -__builtin_inff() ? 0.0f * p[v] : p[v];
        sum += p[v];
    }
    sum = group_sum<LPR>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] *= inv;
}

// -------------------------------------------------- counts, offsets and loss

// Exclusive scan of cnt[E] into off[E + 1] (LDS), by the first wave.
__device__ __forceinline__ void scan_counts(const int32_t *cnt, int32_t *off, int E) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int base = 0; base < E; base += 64) {
        const int e = base + lane, c = e < E ? cnt[e] : 0;
        const int incl = wave_scan(c, [](int a, int b) { return a + b; }) + carry;
        if (e < E) off[e] = incl - c;
        carry = __builtin_amdgcn_readlane(incl, 63);
    }
    if (lane == 0) off[E] = carry;
}

// counts, offsets, slopes and loss from the totals (LDS), by the first wave.  n is
// at most 2^30, E counts at most 2^40: 64 bits hold what 32 would round.
__device__ __forceinline__ void write_totals(const RouteArgs &a, const int32_t *cnt, const int32_t *off, const float *psum,
                                             int live) {
    const int lane = threadIdx.x;
    const double n = live > 0 ? (double)live : 1.0, f = (double)a.E / ((double)a.k * n * n);
    double loss = 0.0;
    for (int e = lane; e < a.E; e += 64) {
        const double slope = f * (double)cnt[e];
        a.counts[e] = cnt[e];
        a.offsets[e] = off[e];
        a.slopes[e] = (float)slope;
        loss += slope * (double)psum[e];
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) loss += __shfl_xor(loss, d);
    if (lane == 0) {
        a.offsets[a.E] = off[a.E];
        a.loss[0] = (float)loss;
    }
}

// ------------------------------------------------------------------ forward

constexpr int kSumSlices = 4;  // waves that add their sums to LDS at a time

template <int LPR>
constexpr int kRouteThreads = 64 * LPR < 1024 ? 64 * LPR : 1024;

// LDS: a word per expert, its slots so far, offsets, sums of probabilities; then
// a chunk's slots.
inline size_t route_lds(int E, int k) {
    return (size_t)E * 8 + (size_t)(2 * E + 1) * 4 + (size_t)kSumSlices * E * 4 + (size_t)kRouteTokens * (8 * k + 4) + 16;
}

template <class T, int LPR, int V>
__global__ __launch_bounds__(kRouteThreads<LPR>) void route_kernel(RouteArgs a) {
    constexpr int NT = kRouteThreads<LPR>, RPW = 64 / LPR, PASSES = kRouteTokens * LPR / NT, W = NT / 64;
    extern __shared__ uint64_t lds[];
    uint64_t *mask = lds;
    float *part = reinterpret_cast<float *>(mask + a.E);                  // [kSumSlices][E]
    float *slot_p = part + kSumSlices * a.E;                              // [64][k]
    int32_t *slot_e = reinterpret_cast<int32_t *>(slot_p + kRouteTokens * a.k);
    float *chosen = reinterpret_cast<float *>(slot_e + kRouteTokens * a.k);  // [64]: sum over a token's slots
    int32_t *used = reinterpret_cast<int32_t *>(chosen + kRouteTokens);   // [E]
    int32_t *off = used + a.E;                                            // [E + 1]
    __shared__ int32_t live;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sub = lane % LPR, col = sub * V;
    const uint64_t group_lanes = (LPR == 64 ? ~0ull : ((1ull << LPR) - 1)) << (lane / LPR * LPR % 64);
    const uint64_t below = group_lanes & ((1ull << lane) - 1);
    for (int e = tid; e < a.E; e += NT) {
        mask[e] = 0;
        used[e] = 0;
    }
    if (tid == 0) live = 0;
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.0f;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.chunks * kRouteTokens;
    for (int c = 0; c < a.chunks; ++c) {
        const int64_t tc = t0 + c * kRouteTokens;
        if (tc >= a.T) break;  // uniform
#pragma unroll 1
        for (int pass = 0; pass < PASSES; ++pass) {
            const int row = (pass * W + wave) * RPW + lane / LPR;
            const int64_t t = tc + row;
            float x[V], p[V];
            if (t < a.T && (!a.valid || a.valid[t])) {
                load_logits<T, V>(a.logits + t * a.ld * (int64_t)sizeof(T), col, a.E, x);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) x[v] = -__builtin_inff();
            }
            softmax<LPR, V>(x, p);
            uint32_t key[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                acc[v] += p[v];
                key[v] = order_key(x[v]);
            }
            float mine = 0.0f;
            for (int j = 0; j < a.k; ++j) {
                uint32_t best = key[0];
#pragma unroll
                for (int v = 1; v < V; ++v) best = best > key[v] ? best : key[v];
                const uint32_t top = group_max<LPR>(best);
                // of equal logits the lowest index: the first lane that has one, its first
                const uint64_t owners = __ballot(best == top);
                if (best == top && !(owners & below)) {
                    int e = -1;
                    float pe = 0.0f;
                    if (top) {
#pragma unroll
                        for (int v = V - 1; v >= 0; --v)
                            if (key[v] == top) {
                                e = v;
                                pe = p[v];
                            }
#pragma unroll
                        for (int v = 0; v < V; ++v) key[v] = v == e ? 0u : key[v];
                        e += col;
                        atomicOr((unsigned long long *)&mask[e], 1ull << row);
                        mine += pe;
                    }
                    slot_e[row * a.k + j] = e;
                    slot_p[row * a.k + j] = pe;
                }
            }
            const float sum = group_sum<LPR>(mine);
            if (sub == 0) chosen[row] = sum;
        }
        __syncthreads();
        const int rows = a.T - tc < kRouteTokens ? (int)(a.T - tc) : kRouteTokens;
        for (int i = tid; i < rows * a.k; i += NT) {
            const int row = i / a.k, e = slot_e[i];
            const int64_t o = tc * a.k + i;
            a.experts[o] = e;
            a.gates[o] = e < 0 ? 0.0f : (a.normalize ? slot_p[i] / chosen[row] : slot_p[i]);
            a.rows[o] = e < 0 ? -1 : used[e] + __popcll(mask[e] & ((1ull << row) - 1));
        }
        if (wave == 0) {
            const uint64_t has = __ballot(lane < rows && slot_e[lane * a.k] >= 0);
            if (lane == 0) live += __popcll(has);
        }
        __syncthreads();
        for (int e = tid; e < a.E; e += NT) {
            used[e] += __popcll(mask[e]);
            mask[e] = 0;
        }
        __syncthreads();
    }
    // sums of probabilities: a wave's tokens, then the waves in order
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int d = LPR; d < 64; d *= 2) acc[v] += __shfl_xor(acc[v], d);
    for (int w0 = 0; w0 < W; w0 += kSumSlices) {
        if (wave >= w0 && wave < w0 + kSumSlices && lane < LPR)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (col + v < a.E) {
                    float *q = &part[(wave - w0) * a.E + col + v];
                    *q = w0 ? *q + acc[v] : acc[v];
                }
        __syncthreads();
    }
    for (int e = tid; e < a.E; e += NT) {
        float s = part[e];
#pragma unroll
        for (int i = 1; i < kSumSlices; ++i) s += part[i * a.E + e];
        part[e] = s;
        if (a.blocks > 1) {
            a.psum[(int64_t)blockIdx.x * a.E + e] = s;
            a.hist[(int64_t)blockIdx.x * a.E + e] = used[e];
        }
    }
    if (a.blocks > 1) {
        if (tid == 0) a.live[blockIdx.x] = live;
        return;
    }
    __syncthreads();
    if (wave == 0) scan_counts(used, off, a.E);
    __syncthreads();
    if (wave == 0) write_totals(a, used, off, part, live);
    // each thread on the slots it wrote above
    for (int64_t tc = 0; tc < a.T; tc += kRouteTokens) {
        const int rows = a.T - tc < kRouteTokens ? (int)(a.T - tc) : kRouteTokens;
        for (int i = tid; i < rows * a.k; i += NT) {
            const int64_t o = tc * a.k + i;
            const int e = a.experts[o];
            if (e >= 0) a.rows[o] += off[e];
        }
    }
}

// Places among all of an expert's slots: those of the blocks before, from their
// counts, and of the experts before.  Every block adds up the counts of all (at
// most 256 x E, from the L2), which costs less than a launch that does it once;
// the last block writes the totals.
constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void route_join_kernel(RouteArgs a) {
    extern __shared__ uint64_t lds[];
    int32_t *total = reinterpret_cast<int32_t *>(lds);  // [E]
    int32_t *base = total + a.E;                        // [E]
    int32_t *off = base + a.E;                          // [E + 1]
    int32_t *sum = off + a.E + 1;                       // [1024] and [1024]
    const int tid = threadIdx.x, b = blockIdx.x;
    const bool totals = b == a.blocks;
    const int per = a.E < kJoinThreads ? a.E : kJoinThreads, parts = kJoinThreads / per;
    const int e0 = tid % per, part = tid / per;
    for (int e = e0; e < a.E; e += per) {  // (E <= 1024: once)
        int all = 0, before = 0;
        if (part < parts)
#pragma unroll 8
            for (int i = part; i < a.blocks; i += parts) {
                const int h = a.hist[(int64_t)i * a.E + e];
                all += h;
                before += i < b ? h : 0;
            }
        sum[tid] = all;
        sum[kJoinThreads + tid] = before;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += kJoinThreads) {
        int all = 0, before = 0;
        for (int i = 0; i < parts; ++i) {
            all += sum[i * per + e];
            before += sum[kJoinThreads + i * per + e];
        }
        total[e] = all;
        base[e] = before;
    }
    __syncthreads();
    if (tid < 64) scan_counts(total, off, a.E);
    if (totals) {
        __syncthreads();
        float *p = reinterpret_cast<float *>(sum);
        float s = 0.0f;
        if (part < parts)
#pragma unroll 8
            for (int i = part; i < a.blocks; i += parts) s += a.psum[(int64_t)i * a.E + e0];
        p[tid] = s;
        __syncthreads();
        float *q = reinterpret_cast<float *>(base);
        for (int e = tid; e < a.E; e += kJoinThreads) {
            float v = 0.0f;
            for (int i = 0; i < parts; ++i) v += p[i * per + e];
            q[e] = v;
        }
        __syncthreads();
        if (tid >= 64) return;
        int live = 0;
        for (int i = tid; i < a.blocks; i += 64) live += a.live[i];
#pragma unroll
        for (int d = 32; d; d >>= 1) live += __shfl_xor(live, d);
        write_totals(a, total, off, q, live);
        return;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += kJoinThreads) base[e] += off[e];
    __syncthreads();
    const int64_t from = (int64_t)b * a.chunks * kRouteTokens * a.k, all = (int64_t)a.T * a.k;
    const int64_t to = from + (int64_t)a.chunks * kRouteTokens * a.k < all ? from + (int64_t)a.chunks * kRouteTokens * a.k : all;
    for (int64_t o = from + tid; o < to; o += kJoinThreads) {
        const int e = a.experts[o];
        if (e >= 0) a.rows[o] += base[e];
    }
}

// ----------------------------------------------------------------- backward

// With c_e = dloss slope_e, d_e the gate's gradient of a chosen expert and 0 for
// the others:
//   gates p_e:            dx = p (c + d - sum p (c + d))
//   gates p_e / P, P the sum over the chosen:  dx = p (c - sum p c) + g (d - sum g d)
// The probabilities are computed again from the logits, in registers: cheaper
// than to store and read them.
template <class T, int LPR, int V>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteGradArgs a) {
    constexpr int RPW = 64 / LPR;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LPR, col = sub * V;
    const float dloss = a.dloss ? *a.dloss : 0.0f;
    float c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = a.dloss && col + v < a.E ? dloss * a.slopes[col + v] : 0.0f;
    const int64_t step = (int64_t)gridDim.x * 4 * RPW;
    for (int64_t t = ((int64_t)blockIdx.x * 4 + wave) * RPW + lane / LPR; t - lane / LPR < a.T; t += step) {
        const bool in = t < a.T;
        const int32_t *ex = a.experts + (in ? t : 0) * a.k;
        const bool has = in && ex[0] >= 0 && ex[0] < a.E;
        float x[V], p[V], d[V], s[V];
        if (has) {
            load_logits<T, V>(a.logits + t * a.ld * (int64_t)sizeof(T), col, a.E, x);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = -__builtin_inff();
        }
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = s[v] = 0.0f;
        if (has && a.dgates)
            for (int j = 0; j < a.k; ++j) {
                const int e = ex[j] - col;
                const float g = a.dgates[t * a.k + j];
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (e == v) {
                        d[v] += g;
                        s[v] = 1.0f;
                    }
            }
        softmax<LPR, V>(x, p);
        float pc = 0.0f, pd = 0.0f, ps = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            pc = fmaf(p[v], c[v], pc);
            pd = fmaf(p[v], d[v], pd);
            ps = fmaf(p[v], s[v], ps);
        }
        pc = group_sum<LPR>(pc);
        pd = group_sum<LPR>(pd);
        if (a.normalize) {
            ps = group_sum<LPR>(ps);
            const float inv = ps == 0.0f ? 0.0f : 1.0f / ps;
            pd *= inv;
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = p[v] * (c[v] - pc) + p[v] * inv * s[v] * (d[v] - pd);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = p[v] * ((c[v] - pc) + (d[v] - pd));
        }
        if (!in || col >= a.E) continue;
        T *out = reinterpret_cast<T *>(a.dlogits) + t * a.ldd + col;
        T e[V];
#pragma unroll
        for (int v = 0; v < V; ++v) e[v] = from_f32<T>(has ? x[v] : 0.0f);
        if (col + V <= a.E) {
            __builtin_memcpy(out, e, sizeof e);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (col + v < a.E) out[v] = e[v];
        }
    }
}

// Lanes to a token and experts to a lane: the fewest lanes whose registers hold
// them, as more tokens to a wave share the steps across lanes.
template <class F>
hipError_t by_experts(int E, F &&f) {
    using std::integral_constant;
    if (E <= 16) return f(integral_constant<int, 4>(), integral_constant<int, 4>());
    if (E <= 64) return f(integral_constant<int, 8>(), integral_constant<int, 8>());
    if (E <= 128) return f(integral_constant<int, 16>(), integral_constant<int, 8>());
    if (E <= 256) return f(integral_constant<int, 16>(), integral_constant<int, 16>());
    if (E <= 512) return f(integral_constant<int, 64>(), integral_constant<int, 8>());
    return f(integral_constant<int, 64>(), integral_constant<int, 16>());
}

template <class T>
hipError_t route(const RouteArgs &a, hipStream_t s) {
    return by_experts(a.E, [&](auto lpr, auto v) {
        hipLaunchKernelGGL(HIP_KERNEL_NAME(route_kernel<T, lpr(), v()>), dim3((unsigned)a.blocks), dim3(kRouteThreads<lpr()>),
                           route_lds(a.E, a.k), s, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || a.blocks == 1) return e;
        hipLaunchKernelGGL(route_join_kernel, dim3((unsigned)a.blocks + 1), dim3(kJoinThreads),
                           (size_t)(3 * a.E + 1 + 2 * kJoinThreads) * 4, s, a);
        return hipGetLastError();
    });
}

template <class T>
hipError_t route_backward(const RouteGradArgs &a, hipStream_t s) {
    return by_experts(a.E, [&](auto lpr, auto v) {
        constexpr int per = 4 * 64 / lpr();  // tokens of a block
        const int64_t blocks = (a.T + per - 1) / per;
        hipLaunchKernelGGL(HIP_KERNEL_NAME(route_backward_kernel<T, lpr(), v()>),
                           dim3((unsigned)(blocks < 8 * kComputeUnits ? blocks : 8 * kComputeUnits)), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_route(int dtype, const RouteArgs &a, hipStream_t s) {
    return dtype == CP_BF16 ? route<__bf16>(a, s) : route<float>(a, s);
}
hipError_t launch_route_backward(int dtype, const RouteGradArgs &a, hipStream_t s) {
    return dtype == CP_BF16 ? route_backward<__bf16>(a, s) : route_backward<float>(a, s);
}

}  // namespace cpo
