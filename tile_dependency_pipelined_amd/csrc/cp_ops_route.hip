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
//
// The bytes are few (16384 x 128 fp32, k 8: 10 MB, 2 us).  What bounds the kernels is
// latency: the chain of k selections, each a maximum over the lanes, and then the
// launch that joins the blocks.  16 x 8 bf16 in one block 4.2 us; 16384 x 128 in 256
// blocks 11.1 and the join 8.2; backward 8191 x 60 4.9.
#include "cp_ops_experts.h"
#include "cp_ops_units.h"

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

// A value's place in the order of choice: larger comes first, NaN of either sign
// before all.  -inf, and what is no expert, has kNoKey: it is never chosen.
constexpr uint32_t kNoKey = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_key(float x) {  // (not for NaN)
    x += 0.0f;  // -0 to 0: they tie
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// The logit of a key (NaN for the largest).
__device__ __forceinline__ float key_value(uint32_t u) {
    return __builtin_bit_cast(float, u & 0x80000000u ? u ^ 0x80000000u : ~u);
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

// e^d for the sums: d log2(e) is rounded once more than above, which is |d| ulp of
// terms that count less the larger |d| is.
__device__ __forceinline__ float exp_term(float d) { return __builtin_amdgcn_exp2f(d * 1.44269504088896340736f); }

// Probabilities; all zero where every logit is -inf, all NaN with a NaN or inf
// among them.
struct Scale {  // p = e^(x - most) inv
    float most, inv;
};
template <int LPR, int V>
__device__ __forceinline__ Scale softmax(const float (&x)[V], float (&p)[V]) {
    float m = x[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
    m = group_fmax<LPR>(m);
    m = m == -__builtin_inff() ? 0.0f : m;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        p[v] = exp_term(x[v] - m);
        sum += p[v];
    }
    sum = group_sum<LPR>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] *= inv;
    return {m, inv};
}

// -------------------------------------------------- counts, offsets and loss

// Exclusive scan of the E counts cnt(e) into off[E + 1] (LDS), by the first wave.
template <class Counts>
__device__ __forceinline__ void scan_counts(Counts &&cnt, int32_t *off, int E) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int base = 0; base < E; base += 64) {
        const int e = base + lane, c = e < E ? cnt(e) : 0;
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

// A block takes 64 tokens at a time.  Selection writes the chosen logit's key to LDS, and
// each slot's gate is computed from it afterwards, once, by one thread, and not by all
// the lanes of a token in every step of the selection (16384 x 128 20.7 -> 18.7 us in all).

// Waves that add their sums to LDS at a time: all, unless the experts are many (and a
// token's lanes a wave, by_experts).
template <int LPR>
constexpr int kSumSlices = LPR < 64 ? 16 : 4;

template <int LPR>
constexpr int kRouteThreads = 64 * LPR < 1024 ? 64 * LPR : 1024;

// LDS: a word per expert, its slots so far, offsets, sums of probabilities; then
// a chunk's slots.
template <int LPR>
size_t route_lds(int E, int k) {
    return (size_t)E * 8 + (size_t)(2 * E + 1) * 4 + (size_t)kSumSlices<LPR> * E * 4 + (size_t)kRouteTokens * (8 * k + 8) + 16;
}

template <class T, int LPR, int V>
__global__ __launch_bounds__(kRouteThreads<LPR>) void route_kernel(RouteArgs a) {
    constexpr int NT = kRouteThreads<LPR>, RPW = 64 / LPR, PASSES = kRouteTokens * LPR / NT, W = NT / 64;
    extern __shared__ uint64_t lds[];
    uint64_t *mask = lds;
    constexpr int slices = kSumSlices<LPR>;
    float *part = reinterpret_cast<float *>(mask + a.E);                     // [slices][E]
    float *slot_p = part + slices * a.E;                                     // [64][k]: the logit's key, then p
    int32_t *slot_e = reinterpret_cast<int32_t *>(slot_p + kRouteTokens * a.k);
    Scale *scale = reinterpret_cast<Scale *>(slot_e + kRouteTokens * a.k);   // [64]
    int32_t *used = reinterpret_cast<int32_t *>(scale + kRouteTokens);       // [E]
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
    // One chunk is all there is: its offsets are known before its places are written.
    const bool single = a.blocks == 1 && a.T > 0 && a.T <= kRouteTokens;
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
            if (t - lane / LPR >= a.T) break;  // none of the wave's: nothing reads what it would leave
            float x[V], p[V];
            if (t < a.T && (!a.valid || a.valid[t])) {
                load_logits<T, V>(a.logits + t * a.ld * (int64_t)sizeof(T), col, a.E, x);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) x[v] = -__builtin_inff();
            }
            const Scale sc = softmax<LPR, V>(x, p);
            uint32_t key[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                acc[v] += p[v];
                key[v] = order_key(x[v]);
            }
            if (__any(sc.inv != sc.inv))  // NaN (or inf) among them
#pragma unroll
                for (int v = 0; v < V; ++v) key[v] = x[v] != x[v] ? 0xFFFFFFFFu : key[v];
            if (sub == 0) scale[row] = sc;
            for (int j = 0; j < a.k; ++j) {
                uint32_t best = key[0];
#pragma unroll
                for (int v = 1; v < V; ++v) best = best > key[v] ? best : key[v];
                const uint32_t top = group_max<LPR>(best);
                // of equal logits the lowest index: the first lane that has one, its first
                const uint64_t owners = __ballot(best == top);
                if (best == top && !(owners & below)) {
                    int e = -1;
                    if (top > kNoKey) {
                        bool seen = false;
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            const bool hit = key[v] == top && !seen;
                            seen |= hit;
                            e = hit ? v : e;
                            key[v] = hit ? 0u : key[v];
                        }
                        e += col;
                        atomicOr((unsigned long long *)&mask[e], 1ull << row);
                    }
                    slot_e[row * a.k + j] = e;
                    slot_p[row * a.k + j] = __builtin_bit_cast(float, top);
                }
            }
        }
        __syncthreads();
        const int rows = a.T - tc < kRouteTokens ? (int)(a.T - tc) : kRouteTokens;
        if (single && wave == 0) scan_counts([&](int e) { return __popcll(mask[e]); }, off, a.E);
        for (int i = tid; i < rows * a.k; i += NT) {
            const Scale sc = scale[i / a.k];
            const float x = key_value(__builtin_bit_cast(uint32_t, slot_p[i]));
            slot_p[i] = slot_e[i] < 0 ? 0.0f : exp_below_one(x - sc.most) * sc.inv;  // (with NaN, inv is)
        }
        __syncthreads();
        for (int i = tid; i < rows * a.k; i += NT) {
            const int row = i / a.k, e = slot_e[i];
            const int64_t o = tc * a.k + i;
            float sum = 1.0f;
            if (a.normalize) {
                sum = 0.0f;
                for (int j = 0; j < a.k; ++j) sum += slot_p[row * a.k + j];
            }
            a.experts[o] = e;
            a.gates[o] = e < 0 ? 0.0f : slot_p[i] / sum;
            a.rows[o] = e < 0 ? -1 : (single ? off[e] : used[e]) + __popcll(mask[e] & ((1ull << row) - 1));
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
    for (int w0 = 0; w0 < W; w0 += slices) {
        if (wave >= w0 && wave < w0 + slices && lane < LPR)
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
        for (int i = 1; i < (W < slices ? W : slices); ++i) s += part[i * a.E + e];
        part[e] = s;
        if (a.blocks > 1) {
            a.psum[(int64_t)blockIdx.x * a.stride + e] = s;
            a.hist[(int64_t)blockIdx.x * a.stride + e] = used[e];
        }
    }
    if (a.blocks > 1) {
        const int e = a.E + tid;  // the rest of the row's last 16 bytes
        if (e < a.stride) {
            a.psum[(int64_t)blockIdx.x * a.stride + e] = 0.0f;
            a.hist[(int64_t)blockIdx.x * a.stride + e] = 0;
        }
        if (tid == 0) a.live[blockIdx.x] = live;
        return;
    }
    __syncthreads();
    if (!single) {
        if (wave == 0) scan_counts([&](int e) { return used[e]; }, off, a.E);
        __syncthreads();
    }
    if (wave == 0) write_totals(a, used, off, part, live);
    if (single) return;
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
// counts, and of the experts before.  Every block adds up the counts of all, at most
// 256 x E from the caches, four experts to a thread and all its loads in flight at once,
// which spares another launch.  The last block writes the totals.
constexpr int kJoinThreads = 1024, kJoinParts = 64;
struct JoinShape {
    int quads, parts;  // 16 bytes of a row; ranges of the rows
    __host__ __device__ explicit JoinShape(int stride)
        : quads(stride / 4), parts(kJoinThreads / (stride / 4) < kJoinParts ? kJoinThreads / (stride / 4) : kJoinParts) {}
};
inline size_t join_lds(int E, int stride) { return ((size_t)2 * JoinShape(stride).parts * stride + 3 * (size_t)E + 1) * 4; }

// This thread's part of the rows' column sums: of all rows, and of those of the
// blocks before b.
template <class V>
__device__ __forceinline__ void column_sums(const RouteArgs &a, const JoinShape &j, const V *rows, int b, V (&s)[4], V (&t)[4]) {
    const int q = threadIdx.x % j.quads, part = threadIdx.x / j.quads;
#pragma unroll
    for (int c = 0; c < 4; ++c) s[c] = t[c] = V(0);
    if (part >= j.parts) return;
#pragma unroll 8
    for (int i = part; i < a.blocks; i += j.parts) {
        V v[4];
        __builtin_memcpy(v, __builtin_assume_aligned(rows + (int64_t)i * a.stride + q * 4, 16), 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            s[c] += v[c];
            t[c] += i < b ? v[c] : V(0);
        }
    }
}
template <class V>
__device__ __forceinline__ void put_sums(const RouteArgs &a, const JoinShape &j, V *to, const V (&s)[4]) {
    const int q = threadIdx.x % j.quads, part = threadIdx.x / j.quads;
    if (part < j.parts) __builtin_memcpy(__builtin_assume_aligned(to + part * a.stride + q * 4, 16), s, 16);
}
// Column e of what put_sums left, the parts in order.
template <class V>
__device__ __forceinline__ V total_of(const RouteArgs &a, const JoinShape &j, const V *from, int e) {
    V s = V(0);
#pragma unroll 8
    for (int i = 0; i < j.parts; ++i) s += from[i * a.stride + e];
    return s;
}

__global__ __launch_bounds__(kJoinThreads) void route_join_kernel(RouteArgs a) {
    extern __shared__ uint64_t lds[];
    const JoinShape j(a.stride);
    int32_t *all = reinterpret_cast<int32_t *>(lds), *before = all + j.parts * a.stride;  // [parts][stride]
    int32_t *total = before + j.parts * a.stride, *base = total + a.E, *off = base + a.E;  // [E], [E], [E + 1]
    const int tid = threadIdx.x, b = blockIdx.x;
    const bool totals = b == a.blocks;
    // the block's first slots, requested ahead; the last block's other inputs likewise
    const int64_t from = (int64_t)b * a.chunks * kRouteTokens * a.k, every = (int64_t)a.T * a.k;
    const int64_t to = from + (int64_t)a.chunks * kRouteTokens * a.k < every ? from + (int64_t)a.chunks * kRouteTokens * a.k : every;
    int e0 = -1, r0 = 0;
    if (from + tid < to) {
        e0 = a.experts[from + tid];
        r0 = a.rows[from + tid];
    }
    float ps[4], none[4];
    int live = 0;
    if (totals) {
        column_sums<float>(a, j, a.psum, 0, ps, none);
        if (tid < 64)
            for (int i = tid; i < a.blocks; i += 64) live += a.live[i];
    }
    int32_t s[4], t[4];
    column_sums<int32_t>(a, j, a.hist, b, s, t);
    put_sums(a, j, all, s);
    if (totals) put_sums(a, j, reinterpret_cast<float *>(before), ps);  // (it has no use for the others)
    else put_sums(a, j, before, t);
    __syncthreads();
    // one thread to a column, the counts' and the others' columns by different waves
    for (int e = tid; e < a.E; e += kJoinThreads / 2)
        if (tid < kJoinThreads / 2) total[e] = total_of(a, j, all, e);
    for (int e = tid - kJoinThreads / 2; e < a.E; e += kJoinThreads / 2)
        if (tid >= kJoinThreads / 2) {
            if (totals) reinterpret_cast<float *>(base)[e] = total_of(a, j, reinterpret_cast<const float *>(before), e);
            else base[e] = total_of(a, j, before, e);
        }
    __syncthreads();
    if (tid < 64) {
        scan_counts([&](int e) { return total[e]; }, off, a.E);
        if (totals) {
#pragma unroll
            for (int d = 32; d; d >>= 1) live += __shfl_xor(live, d);
            write_totals(a, total, off, reinterpret_cast<const float *>(base), live);
        }
    }
    if (totals) return;
    __syncthreads();
    if (e0 >= 0) a.rows[from + tid] = r0 + base[e0] + off[e0];
    for (int64_t o = from + tid + kJoinThreads; o < to; o += kJoinThreads) {
        const int e = a.experts[o];
        if (e >= 0) a.rows[o] += base[e] + off[e];
    }
}

// ----------------------------------------------------------------- backward

// With c_e = dloss slope_e, d_e the gate's gradient of a chosen expert and 0 for
// the others:
//   gates p_e:            dx = p (c + d - sum p (c + d))
//   gates p_e / P, P the sum over the chosen:  dx = p (c - sum p c) + g (d - sum g d)
// The probabilities are computed again from the logits, in registers: cheaper
// than to store and read them.
// The gates' gradients go to the lanes of their experts by way of LDS: compared with
// every logit's index in registers instead, they took most of the time (32768 x 512 bf16,
// k 8: 42 us, so 31).
template <class T, int LPR, int V>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteGradArgs a) {
    constexpr int RPW = 64 / LPR;
    constexpr uint32_t kNone = 0xFFFFFFFFu;  // no slot's: a NaN that no gradient is made of
    __shared__ __attribute__((aligned(16))) uint32_t spread[4][RPW][LPR * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane % LPR, col = sub * V;
    const float dloss = a.dloss ? *a.dloss : 0.0f;
    float c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = a.dloss && col + v < a.E ? dloss * a.slopes[col + v] : 0.0f;
    uint32_t *row_d = spread[wave][lane / LPR];
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
        uint32_t u[V];
#pragma unroll
        for (int v = 0; v < V; ++v) u[v] = kNone;
        if (a.dgates) {  // (a wave's own part of LDS)
            __builtin_memcpy(__builtin_assume_aligned(row_d + col, 16), u, sizeof u);
            settle_lds();
            for (int j = sub; j < a.k; j += LPR) {
                const int e = ex[j];
                if (has && e >= 0 && e < a.E) {
                    const float g = a.dgates[t * a.k + j];
                    row_d[e] = g != g ? 0x7FC00000u : __builtin_bit_cast(uint32_t, g);
                }
            }
            settle_lds();
            __builtin_memcpy(u, __builtin_assume_aligned(row_d + col, 16), sizeof u);
            settle_lds();
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = u[v] == kNone ? 0.0f : 1.0f;
            d[v] = u[v] == kNone ? 0.0f : __builtin_bit_cast(float, u[v]);
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
                           route_lds<lpr()>(a.E, a.k), s, a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || a.blocks == 1) return e;
        hipLaunchKernelGGL(route_join_kernel, dim3((unsigned)a.blocks + 1), dim3(kJoinThreads),
                           join_lds(a.E, a.stride), s, a);
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
