// cp_ops_gemm.h -- the products of the feed-forward operators for gfx950: one
// output tile per workgroup, operands through LDS, fp32 accumulation on the
// matrix cores, epilogue per wave.  Included by the files that instantiate it.
//
// C[M][N] = sum over k of A[m][k] B[k][n].  Each operand is either contiguous
// in k (KC: rows of k) or in its outer index (rows of m or n, one per k):
//   forward          A = X  KC     B = W   (KC if W is stored [N][K])
//   input gradient   A = dZ KC     B = W^t (KC if W is stored [K][N])
//   weight gradient  A = X^t, B = dZ, both contiguous in the outer index
//
// LDS tile of an operand with R outer indices (R x 128 bytes: 64 k of bf16,
// 32 k of fp32), filled by 16-byte loads that go straight to LDS (lane l of a
// load lands at base + 16 l, so the swizzle is in which chunk a lane fetches):
//   KC      [R][128 bytes], chunk c of row r at position c ^ swz_kc(r).  A
//           fragment (16 bytes of one row) is one ds_read_b128; 16 rows of a
//           block and the two chunks that lanes l and l + 32 read fall on
//           distinct 16-byte bank groups.
//   outer   [k][R elements], chunk c of row k at position c ^ swz_out(k).
//           bf16: a fragment is two ds_read_b64_tr_b16 (each transposes 4 k x
//           16 columns over 16 lanes); fp32: four 4-byte reads.
// MFMA v_mfma_f32_16x16x32_bf16 (32 k) or four v_mfma_f32_16x16x4_f32 (16 k:
// lane group g holds k 4 g + t of the block for product t; the sum does not
// care which k a lane holds as long as A and B agree).  B is the first operand,
// so a lane gets output row lane mod 16 and columns 4 (lane / 16) .. + 3.
#pragma once
#include <type_traits>

#include "cp_ops_host.h"

namespace cpo {

template <int U>
using ic = std::integral_constant<int, U>;

// wait until at most N vector-memory operations of this wave are in flight
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

constexpr int kRawBuffer = 0x00020000;       // word 3 of a raw (stride 0) buffer resource
constexpr uint32_t kOutside = 0xC0000000u;   // an offset past every resource made here (all < 2^31 bytes): reads zeros

// 16-byte direct load to LDS at `lds` + 16 lane (`lds` wave-uniform) in a form
// the compiler's wait insertion does not see: it would otherwise wait for all
// direct loads in flight before the next LDS read, whichever array that reads,
// and a pipeline of more than two stages would never have two slabs in flight.
// Every read of data loaded this way follows an explicit wait_vm and a barrier.
__device__ __forceinline__ void lds_load_untracked(__amdgpu_buffer_rsrc_t r, const void *lds, uint32_t voff) {
    const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_void_t *)lds);
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "buffer_load_dwordx4 %2, %3, 0 offen lds\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(m0), "v"(voff), "s"(r)
        : "memory");
}

// MFMAs spread evenly between LDS reads, and direct loads between both.
template <int I, int RD, int MF, int PER>
__device__ __forceinline__ void interleave() {
    if constexpr (I < RD) {
        constexpr int m = (I + 1) * MF / RD - I * MF / RD, p = (I + 1) * PER / RD - I * PER / RD;
        if constexpr (m > 0) __builtin_amdgcn_sched_group_barrier(0x008, m, 0);  // MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                       // LDS read
        if constexpr (p > 0) __builtin_amdgcn_sched_group_barrier(0x020, p, 0);  // vector memory read
        interleave<I + 1, RD, MF, PER>();
    }
}

// A value the compiler cannot tell from a new one: what is computed from it is
// computed where it is used, instead of once before the loop into registers
// that the accumulators and fragments need.
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}
__device__ __forceinline__ uint32_t fresh_uniform(uint32_t v) {
    asm volatile("" : "+s"(v));
    return v;
}

// One operand's tile of R outer indices.
template <class T, int R, bool KC, int NW, bool LEAN>
struct Operand {
    static constexpr int ES = sizeof(T), CE = 16 / ES, BK = 128 / ES;
    static constexpr bool BF = std::is_same<T, __bf16>::value;
    static constexpr int BYTES = R * 128;
    static constexpr int LOADS = BYTES / 1024;             // 1 KiB loads of a slab, over the waves
    static constexpr int PW = LOADS >= NW ? LOADS / NW : 1;  // per wave (fewer loads than waves: some repeat one)
    static constexpr int RB = R * ES;                      // bytes of an LDS row, outer-contiguous
    static constexpr int READS = KC ? 1 : (BF ? 2 : 4);    // LDS reads of a fragment
    // LDS rows from one load of a wave to its next.  Where that is a multiple
    // of 16 the swizzle is the same in all of them, and so is the step in memory.
    static constexpr int ROW_STEP = KC ? NW * 8 : NW * 1024 / RB;
    static constexpr bool EVEN = ROW_STEP % 16 == 0;
    // one offset register then serves all loads; a tile with registers to spare keeps one for each
    static constexpr int OFFS = EVEN && LEAN ? 1 : PW;
    static_assert(LOADS >= NW ? LOADS % NW == 0 : NW % LOADS == 0, "loads per wave");
    static_assert(KC || (R >= 64 && RB <= 1024), "bank swizzle");
    static_assert(!KC || EVEN, "loads of rows");

    // KC: rows r .. r + 15 of a block and chunks c, c + 2
    __device__ static int swz_kc(int r) { return ((r >> 1) & 1) | (((r >> 3) & 1) << 1) | (((r >> 2) & 1) << 2); }
    // outer: bf16 reads rows k .. k+3 and k+8 .. k+11 x 2 chunks per 32 lanes;
    // fp32 rows k, k+4, k+8, k+12 x 64 bytes per 64 lanes
    __device__ static int swz_out(int k) {
        if constexpr (!BF) return ((k >> 2) & 3) << 2;
        else if constexpr (R >= 128) return ((0xCA60 >> ((k & 3) * 4)) & 15) ^ (((k >> 3) & 1) << 1);
        else return ((k & 3) << 1) ^ ((k >> 3) & 1);
    }

    const char *base;   // KC: first outer row at the first contraction index; outer: first contraction row, first column
    int64_t ld;         // bytes
    int outer;          // valid outer indices (<= R)
    int klen;           // contraction length of this workgroup
    uint32_t off[OFFS]; // bytes from base of this lane's chunk in load q
    int kc;             // KC: this lane's first contraction index within a slab, the same in every load

    __device__ __forceinline__ static int load_id(int q, int wave) {
        return LOADS >= NW ? q * NW + wave : wave % LOADS;
    }

    // `again`: rows past the last one read that again (their results are not
    // stored) instead of zeros.
    __device__ __forceinline__ void init(const char *b, int64_t ld_elems, int outer_, int klen_, int wave, int lane,
                                         bool again) {
        base = b;
        ld = ld_elems * ES;
        outer = outer_ < R ? outer_ : R;
        klen = klen_;
#pragma unroll
        for (int q = 0; q < OFFS; ++q) {
            const int o = load_id(q, wave) * 1024 + lane * 16;
            if constexpr (KC) {
                const int r = o >> 7, c = ((o >> 4) & 7) ^ swz_kc(r);
                off[q] = (uint32_t)(again && r >= outer ? outer - 1 : r) * (uint32_t)ld + (uint32_t)c * 16u;
                kc = c * CE;
            } else {
                const int k = o / RB, c = ((o % RB) >> 4) ^ swz_out(k);
                off[q] = (uint32_t)k * (uint32_t)ld + (uint32_t)c * 16u;
            }
        }
    }

    // Request slab `s` into LDS `lds`.  Chunks past the contraction or the
    // outer range read zeros; past the last slab all of them do, without
    // touching memory, so that the number of loads in flight is constant.  A
    // row's last chunk is read whole: rows that are not whole chunks come only
    // from the host's packed copies, which end in zeros.
    template <bool TRACKED>
    __device__ __forceinline__ void issue(char *lds, int s, int wave) const {
        const int k0 = s * BK, left = klen - k0;  // uniform
        const char *p;
        int64_t bytes;
        if constexpr (KC) {
            p = base + (int64_t)k0 * ES;
            bytes = (int64_t)(outer - 1) * ld + (int64_t)((left + CE - 1) / CE * CE) * ES;
        } else {
            p = base + (int64_t)k0 * ld;
            bytes = (int64_t)((left < BK ? left : BK) - 1) * ld + (int64_t)((outer + CE - 1) / CE * CE) * ES;
        }
        if (left <= 0) bytes = 0;
        const __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), 0, (int)bytes, kRawBuffer);
        const uint32_t step = OFFS < PW ? fresh_uniform((uint32_t)ld * ROW_STEP) : 0;
        const bool past = KC && kc >= left;
#pragma unroll
        for (int q = 0; q < PW; ++q) {
            const uint32_t v = past ? kOutside : (OFFS < PW ? off[0] + q * step : off[OFFS < PW ? 0 : q]);
            char *dst = lds + load_id(q, wave) * 1024;
            if constexpr (TRACKED) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t *)dst, 16, v, 0, 0, 0);
            else lds_load_untracked(r, dst, v);
        }
    }

    // The same slab through registers, for rows that are not 16-byte aligned
    // or not a whole number of 16-byte chunks.  Unaligned 16-byte loads cost
    // little here (217 us aligned, 229 us with odd rows for 2048 x 4096 x 4096
    // before whole slabs had their own branch-free path); only chunks that
    // cross the end of a row or of the contraction are read by elements.
    __device__ __forceinline__ void fetch(uint4 (&v)[PW], int s, int wave, int lane) const {
        const int k0 = s * BK, left = klen - k0;
        const char *p = base + (KC ? (int64_t)k0 * ES : (int64_t)k0 * ld);
        if (left >= BK && (KC || outer == R)) {  // uniform
#pragma unroll
            for (int q = 0; q < PW; ++q) __builtin_memcpy(&v[q], p + off[q], 16);
            return;
        }
#pragma unroll
        for (int q = 0; q < PW; ++q) {
            const int o = load_id(q, wave) * 1024 + lane * 16;
            int n;
            if constexpr (KC) n = left - kc;
            else n = o / RB < left ? outer - (((o % RB) >> 4) ^ swz_out(o / RB)) * CE : 0;
            v[q] = load_partial<T>(p + off[q], n);
        }
    }
    __device__ __forceinline__ static void put(char *lds, const uint4 (&v)[PW], int wave, int lane) {
#pragma unroll
        for (int q = 0; q < PW; ++q)
            *reinterpret_cast<uint4 *>(lds + load_id(q, wave) * 1024 + lane * 16) = v[q];
    }

    // Where a lane reads its fragments, for the wave whose outer indices start
    // at o0.  Block f and step kk only flip bits that o0 leaves zero, or add a
    // constant: one register serves all of a slab's reads.
    __device__ __forceinline__ static uint32_t lane_base(int o0, int lane) {
        const int g = lane >> 4;
        if constexpr (KC) return (o0 + (lane & 15)) * 128 + ((g ^ swz_kc(lane & 15)) << 4);
        else if constexpr (BF) {
            const int k = 8 * g + ((lane & 15) >> 2);
            return k * RB + ((((o0 >> 3) + ((lane & 3) >> 1)) ^ swz_out(k)) << 4) + (lane & 1) * 8;
        } else {
            return 4 * g * RB + ((((o0 >> 2) + ((lane & 15) >> 2)) ^ swz_out(4 * g)) << 4) + (lane & 3) * 4;
        }
    }

    // Fragment of step kk (of two per slab), block f of 16 outer indices.
    __device__ __forceinline__ static uint4 frag(const char *lds, uint32_t lbase, int kk, int f) {
        if constexpr (KC) {
            return *reinterpret_cast<const uint4 *>(lds + (lbase ^ (kk << 6)) + f * 16 * 128);
        } else if constexpr (BF) {
            // the swizzle sees bits 0, 1 and 3 of k: the same for k + 4, and for either kk
            const char *p = lds + (lbase ^ (f << 5)) + kk * 32 * RB;
            const v4i16_t both[2] = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t *)p),
                                     __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t *)(p + 4 * RB))};
            return *reinterpret_cast<const uint4 *>(both);
        } else {
            const char *p = lds + (lbase ^ (f << 6)) + kk * 16 * RB;
            uint32_t e[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) e[t] = *reinterpret_cast<const uint32_t *>(p + t * RB);
            return make_uint4(e[0], e[1], e[2], e[3]);
        }
    }
};

// What the epilogue needs of the arguments at byte ARG of the kernel's, read
// again: kept in scalar registers over the main loop they would spill into the
// vector registers that the accumulators leave (the 256x256 gradients' kernel
// then spilled those too, 119 -> 174 us for 2048 x 4096 x 4096).
template <int ARG>
__device__ __forceinline__ GemmArgs epilogue_args() {
    typedef const __attribute__((address_space(4))) char *kernarg_t;
    typedef const __attribute__((address_space(4))) GemmArgs *args_t;
    kernarg_t p = (kernarg_t)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    const args_t g = (args_t)(p + ARG);
    GemmArgs e{};
    e.C = g->C;
    e.bias = g->bias;
    e.res = g->res;
    e.pre = g->pre;
    e.ws = g->ws;
    e.ldc = g->ldc;
    e.ldr = g->ldr;
    e.ldp = g->ldp;
    e.sc = g->sc;
    e.groups = g->groups;
    e.mode = g->mode;
    e.M = g->M;
    e.N = g->N;
    e.act = g->act;
    e.nsplit = g->nsplit;
    e.ldws = g->ldws;
    e.vec = g->vec;
    return e;
}

// Where a workgroup keeps its stages of A and B, and the rows of its epilogue.
struct Stages {
    char *a[4], *b[4], *rows;
};

// Which of a launch's tiles a workgroup computes: `unit` counts the tiles of
// split after split, for kGroupSum those of `expert`.
struct Place {
    int unit, expert;
    int ntm;         // row tiles
    GroupScan scan;  // kGroupRows
};

// A tile: from row0 and col0, rows up to row_end, over contraction indexes
// k_first .. k_first + klen - 1; zero: its rows belong to no expert.
struct Tile {
    int expert, split, row0, row_end, col0, k_first, klen;
    bool zero;
};

// What bounds it: a 256 x 256 tile takes 1.55 us per 64 k of bf16 with all CUs
// busy (1385 TFLOP/s; an 8192-cubed library product reaches 1430), reads from
// the L2 and the matrix cores together, and 8 to 12 us besides: 0.4 to find the
// tile, 2.5 to 4 for its first slab, 3.2 to store it (6.2 with bias and GELU, 13
// with a residual, whose 67 MB for all tiles then move at 5.1 TB/s) and 0.9 to
// the next workgroup's start.  2048 x 8192 x 8192 with GELU and residual: 215 us.
// 16-row tiles are bound by the weight's bytes: 13 x 8192 x 28672 in 90 us, 5.2
// TB/s; 16 rows over 8 experts of 4096 x 4096 in 39.
//
// Tile BM x BN, wave grid WGM x WGN, S LDS stages.  DIRECT: loads straight to
// LDS (16-byte aligned operands); otherwise through registers, two stages.
template <class T_, int BM_, int BN_, int WGM_, int WGN_, int S_, bool AKC_, bool BKC_, bool DIRECT_>
struct Product {
    using T = T_;
    static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, S = S_;
    static constexpr bool AKC = AKC_, BKC = BKC_, DIRECT = DIRECT_;
    static constexpr int NW = WGM * WGN, NT = 64 * NW;
    static constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
    static constexpr bool BF = std::is_same<T, __bf16>::value;
    // Accumulators that take half of a wave's registers or more: addresses are
    // recomputed rather than kept.
    static constexpr bool LEAN = DIRECT && (FM * FN * 4 > 128 || (FM * FN * 4 == 128 && !(AKC && BKC)));
    using OpA = Operand<T, BM, AKC, NW, LEAN>;
    using OpB = Operand<T, BN, BKC, NW, LEAN>;
    static constexpr int BK = OpA::BK;
    static constexpr int STAGE = OpA::BYTES + OpB::BYTES;
    static constexpr int PER = OpA::PW + OpB::PW;          // direct loads per wave and slab
    static constexpr int RD = FM * OpA::READS + FN * OpB::READS;
    static constexpr int MF = FM * FN * (BF ? 1 : 4);
    static constexpr int EPI_PITCH = WN + 4;               // floats of a staged output row
    static_assert(NW * 16 * EPI_PITCH * 4 <= STAGE, "epilogue staging");
    static_assert(S >= 2 && S <= 4 && (DIRECT || S == 2), "stages");
    static_assert(WN == 32 || WN == 64 || WN == 128, "epilogue layout");
    // waves per SIMD the registers are budgeted for: accumulators beyond half
    // of the 512 leave room for one
    static constexpr int WAVES = FM * FN * 4 > 128 ? 1 : 2;

    // Workgroup `b`'s place in a launch with one workgroup to a tile; false if it has none.
    __device__ __forceinline__ static bool place(const GemmArgs &g, int b, Place &p) {
        p.ntm = g.ntm;
        p.expert = 0;
        if (g.mode == kGroupRows) p.ntm = count_tiles(g.off, g.groups, g.M, BM, p.scan);
        const int units = p.ntm * g.ntn * g.nsplit;
        if (g.mode == kGroupSum) {  // experts one after the other, each spread over all XCDs
            p.expert = b / units;
            b -= p.expert * units;
        } else if (b >= units) {
            return false;  // the grid is sized for the most tiles there can be
        }
        p.unit = xcd_remap(b, units);
        return true;
    }

    // The tile at `at`, of BM rows and BN columns.
    __device__ __forceinline__ static Tile tile(const GemmArgs &g, const Place &at) {
        Tile t;
        int ntm = at.ntm, first = 0;  // first: rows before the expert's
        t.expert = at.expert;
        t.split = at.unit / (ntm * g.ntn);
        t.row_end = g.M;
        t.k_first = 0;
        t.klen = g.K;
        t.zero = false;
        int b = at.unit - t.split * ntm * g.ntn;
        if (g.mode == kGroupRows) {
            // expert by expert: its tiles are next to each other
            const RowTile r = find_tile(g.off, g.groups, g.M, BM, b / g.ntn, at.scan);
            t.expert = r.expert;
            first = r.row0;
            t.row_end = r.end;
            b -= r.before * g.ntn;
            ntm = (r.end - r.row0 + BM - 1) / BM;
            t.zero = r.expert == g.groups;  // rows without an expert
            if (t.zero) t.klen = 0;
        } else if (g.mode == kGroupSum) {
            const RowTile r = expert_rows(g.off, g.groups, g.K, t.expert);
            t.k_first = r.row0;
            t.klen = r.end - r.row0;
        }
        // Bands of 8 row tiles, row tiles fastest: the ~32 tiles an XCD works
        // on at a time form a near-square block, which reads least into its L2.
        constexpr int BAND = 8;
        const int band = b / (BAND * g.ntn), inband = b - band * BAND * g.ntn;
        const int left_rows = ntm - band * BAND, high = left_rows < BAND ? left_rows : BAND;
        const int nt = __builtin_amdgcn_readfirstlane(inband / high);
        const int mt = __builtin_amdgcn_readfirstlane(band * BAND + inband % high);
        t.col0 = nt * BN;
        t.row0 = first + mt * BM;
        if (g.nsplit > 1) {  // whole slabs per split
            const int slabs = (t.klen + BK - 1) / BK, per = (slabs + g.nsplit - 1) / g.nsplit;
            const int from = t.split * per * BK;
            t.k_first += from;
            t.klen = t.klen - from < per * BK ? t.klen - from : per * BK;
            if (t.klen < 0) t.klen = 0;
        }
        t.klen = __builtin_amdgcn_readfirstlane(t.klen);
        t.k_first = __builtin_amdgcn_readfirstlane(t.k_first);
        t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
        t.row_end = __builtin_amdgcn_readfirstlane(t.row_end);
        return t;
    }

    // `ARG`: where the kernel's arguments hold `g` (bytes).
    template <int ARG>
    __device__ __forceinline__ static void run(const GemmArgs &g, const Stages &st, const Tile &t) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave / WGN, wn = wave % WGN;
        const int expert = t.expert, split = t.split, row0 = t.row0, row_end = t.row_end, col0 = t.col0;
        const int k_first = t.k_first, klen = t.klen;
        const bool zero = t.zero;
        const char *A = g.A, *B = g.B;
        if (g.mode == kGroupRows && !zero) B += (int64_t)expert * g.sb * sizeof(T);

        f32x4_t acc[FM][FN];
#pragma unroll
        for (int fm = 0; fm < FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < FN; ++fn) acc[fm][fn] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

        const int nk = (klen + BK - 1) / BK;
        if (nk > 0) {
            OpA a;
            OpB w;
            a.init(A + ((AKC ? (int64_t)row0 * g.lda + k_first : (int64_t)k_first * g.lda + row0)) * (int64_t)sizeof(T),
                   g.lda, row_end - row0, klen, wave, lane, !DIRECT);
            w.init(B + ((BKC ? (int64_t)col0 * g.ldb + k_first : (int64_t)k_first * g.ldb + col0)) * (int64_t)sizeof(T),
                   g.ldb, g.N - col0, klen, wave, lane, !DIRECT);
            struct Frags {
                uint4 a[FM], b[FN];
            };
            const uint32_t abase = OpA::lane_base(wm * WM, lane), bbase = OpB::lane_base(wn * WN, lane);
            auto load = [&](int u, int kk, Frags &f) {
                const uint32_t ab = LEAN ? fresh(abase) : abase, bb = LEAN ? fresh(bbase) : bbase;
#pragma unroll
                for (int fn = 0; fn < FN; ++fn) f.b[fn] = OpB::frag(st.b[u], bb, kk, fn);
#pragma unroll
                for (int fm = 0; fm < FM; ++fm) f.a[fm] = OpA::frag(st.a[u], ab, kk, fm);
            };
            auto mma = [&](const Frags &f) {
#pragma unroll
                for (int fm = 0; fm < FM; ++fm)
#pragma unroll
                    for (int fn = 0; fn < FN; ++fn) {
                        if constexpr (BF) {
                            acc[fm][fn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8_t, f.b[fn]), __builtin_bit_cast(bf16x8_t, f.a[fm]),
                                acc[fm][fn], 0, 0, 0);
                        } else {
                            const f32x4_t x = __builtin_bit_cast(f32x4_t, f.b[fn]);
                            const f32x4_t y = __builtin_bit_cast(f32x4_t, f.a[fm]);
#pragma unroll
                            for (int t = 0; t < 4; ++t)
                                acc[fm][fn] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[t], y[t], acc[fm][fn], 0, 0, 0);
                        }
                    }
            };
            if constexpr (DIRECT) {
                // Slabs s+1 .. s+S-1 are in flight while slab s is multiplied.
                // The fragments of a step are read between the MFMAs of the
                // step before it, across slab boundaries: the barrier sits
                // before a slab's last step, when every wave holds all it
                // needs of that slab, so its stage can be refilled.
                constexpr bool TRACKED = S == 2;
                auto issue = [&](int u, int slab) {
                    a.template issue<TRACKED>(st.a[u], slab, wave);
                    w.template issue<TRACKED>(st.b[u], slab, wave);
                };
                Frags f0, f1;
                auto step = [&](auto U, int slab) {
                    constexpr int u = decltype(U)::value;
                    load(u, 1, f1);
                    mma(f0);
                    interleave<0, RD, MF, 0>();
                    wait_vm<(S - 2) * PER>();
                    __syncthreads();
                    issue(u, slab + S);
                    load((u + 1) % S, 0, f0);
                    mma(f1);
                    interleave<0, RD, MF, TRACKED ? PER : 0>();
                };
#pragma unroll
                for (int u = 0; u < S; ++u) issue(u, u);
                wait_vm<(S - 1) * PER>();
                __syncthreads();
                load(0, 0, f0);
                int slab = 0;
                for (; slab + S <= nk; slab += S) {
                    step(ic<0>{}, slab);
                    step(ic<1>{}, slab + 1);
                    if constexpr (S > 2) step(ic<2 % S>{}, slab + 2);
                    if constexpr (S > 3) step(ic<3 % S>{}, slab + 3);
                }
                if (slab < nk) step(ic<0>{}, slab++);
                if constexpr (S > 2)
                    if (slab < nk) step(ic<1>{}, slab++);
                if constexpr (S > 3)
                    if (slab < nk) step(ic<2>{}, slab++);
                wait_vm<0>();  // the trailing requests land before the LDS is reused
            } else {
                // Four slabs in registers on their way to two stages.
                uint4 ra[4][OpA::PW], rb[4][OpB::PW];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (u < nk) {
                        a.fetch(ra[u], u, wave, lane);
                        w.fetch(rb[u], u, wave, lane);
                    }
                auto step = [&](auto U, int slab) {
                    constexpr int u = decltype(U)::value;
                    OpA::put(st.a[u & 1], ra[u], wave, lane);
                    OpB::put(st.b[u & 1], rb[u], wave, lane);
                    __syncthreads();  // also: every wave is done with the other stage's previous slab
                    if (slab + 4 < nk) {
                        a.fetch(ra[u], slab + 4, wave, lane);
                        w.fetch(rb[u], slab + 4, wave, lane);
                    }
                    Frags f0;
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        load(u & 1, kk, f0);
                        mma(f0);
                    }
                };
                int slab = 0;
                for (; slab + 4 <= nk; slab += 4) {
                    step(ic<0>{}, slab);
                    step(ic<1>{}, slab + 1);
                    step(ic<2>{}, slab + 2);
                    step(ic<3>{}, slab + 3);
                }
                if (slab < nk) step(ic<0>{}, slab++);
                if (slab < nk) step(ic<1>{}, slab++);
                if (slab < nk) step(ic<2>{}, slab++);
            }
            __syncthreads();  // every wave is done with the stages
        }

        // ---- epilogue: 16 rows at a time through this wave's part of LDS, so
        // that memory is accessed in runs of whole rows of the wave's tile ----
        const GemmArgs e = epilogue_args<ARG>();
        const int wrow = row0 + wm * WM, wcol = col0 + wn * WN;
        char *C = e.C;
        const char *bias = e.bias;
        if (e.mode == kGroupSum) C += (int64_t)expert * e.sc * sizeof(T);
        if (e.mode == kGroupRows && bias && !zero) bias += (int64_t)expert * e.N * sizeof(T);
        if (e.nsplit > 1) {
            // (kGroupSum: the experts' rows one after the other)
            const int64_t above = e.mode == kGroupSum ? (int64_t)split * e.groups + expert : split;
            float *part = e.ws + above * e.M * e.ldws;
            constexpr int UPR = WN / 4;
            stage_rows(acc, st.rows, wave, lane, [&](int fm, const float *sh) {
#pragma unroll
                for (int i = 0; i < 16 * UPR / 64; ++i) {
                    const int u = i * 64 + lane, r = wrow + fm * 16 + u / UPR, c = (u % UPR) * 4;
                    if (r < row_end && wcol + c < e.ldws)  // ldws is a multiple of 4
                        *reinterpret_cast<f32x4_t *>(part + (int64_t)r * e.ldws + wcol + c) =
                            *reinterpret_cast<const f32x4_t *>(sh + u / UPR * EPI_PITCH + c);
                }
            });
        } else if (e.vec) {
            finish_tile<kUnit<T>>(e, acc, st.rows, C, bias, wrow, wcol, row_end, wave, lane, zero);
        } else {
            finish_tile<1>(e, acc, st.rows, C, bias, wrow, wcol, row_end, wave, lane, zero);
        }
    }

    // Epilogue and stores in runs of CNT columns.  A lane has the same columns
    // in all of its runs.  The residual is requested AHEAD blocks of 16 rows
    // early, so that its latency from memory is not paid for each of them.
    template <int CNT>
    __device__ __forceinline__ static void finish_tile(const GemmArgs &g, const f32x4_t (&acc)[FM][FN], char *lds, char *C,
                                                       const char *bias, int wrow, int wcol, int row_end, int wave,
                                                       int lane, bool zero) {
        constexpr int RUNS = WN / CNT;                        // of a row
        constexpr int STEP = RUNS < 64 ? 64 / RUNS : 1;       // rows between a lane's runs
        constexpr int COLS = RUNS < 64 ? 1 : RUNS / 64;       // runs of a row per lane
        constexpr int NU = 16 / STEP;
        constexpr int AHEAD = FM < (CNT > 1 ? 4 : 2) ? FM : (CNT > 1 ? 4 : 2);
        const int l0 = RUNS < 64 ? lane / RUNS : 0, r0 = wrow + l0;
        const int cl = (RUNS < 64 ? lane % RUNS : lane) * CNT;
        const bool inside = wrow + WM <= row_end && wcol + WN <= g.N;  // uniform
#pragma unroll
        for (int h = 0; h < COLS; ++h) {
            const int c = wcol + cl + h * 64 * CNT;
            const bool col_in = c < g.N;
            Raw<T, CNT> rb, rr[AHEAD][NU];
            if (bias && col_in) rb.load(bias + (int64_t)c * sizeof(T));
            auto request = [&](int fm) {
                if (!g.res) return;
                const char *p = g.res + ((int64_t)(r0 + fm * 16) * g.ldr + c) * sizeof(T);
                if (inside) {
#pragma unroll
                    for (int i = 0; i < NU; ++i) rr[fm % AHEAD][i].load(p + (int64_t)i * STEP * g.ldr * sizeof(T));
                } else if (col_in) {
#pragma unroll
                    for (int i = 0; i < NU; ++i)
                        if (r0 + fm * 16 + i * STEP < row_end)
                            rr[fm % AHEAD][i].load(p + (int64_t)i * STEP * g.ldr * sizeof(T));
                }
            };
#pragma unroll
            for (int fm = 0; fm < AHEAD; ++fm) request(fm);
            stage_rows(acc, lds, wave, lane, [&](int fm, const float *sh) {
                alignas(16) float v[NU][CNT];
#pragma unroll
                for (int i = 0; i < NU; ++i) {
                    const float *p = sh + (i * STEP + l0) * EPI_PITCH + cl + h * 64 * CNT;
                    if constexpr (CNT > 1) {
#pragma unroll
                        for (int e = 0; e < CNT; e += 4)
                            *reinterpret_cast<f32x4_t *>(v[i] + e) = *reinterpret_cast<const f32x4_t *>(p + e);
                    } else {
                        v[i][0] = *p;
                    }
                }
                finish<T, CNT, NU>(g, C, r0 + fm * 16, STEP, c, v, bias ? &rb : nullptr,
                                   g.res ? rr[fm % AHEAD] : nullptr, zero, inside, col_in, row_end);
                if (fm + AHEAD < FM) request(fm + AHEAD);
            });
        }
    }

    // Hands each block of 16 rows of the wave's tile to f(fm, rows in LDS).
    template <class F>
    __device__ __forceinline__ static void stage_rows(const f32x4_t (&acc)[FM][FN], char *lds, int wave, int lane, F &&f) {
        float *sh = reinterpret_cast<float *>(lds) + wave * 16 * EPI_PITCH;
        auto settle = [] {  // LDS accesses of this wave only: they execute in order, the compiler must keep it
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        };
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
                *reinterpret_cast<f32x4_t *>(sh + (lane & 15) * EPI_PITCH + fn * 16 + 4 * (lane >> 4)) = acc[fm][fn];
            settle();
            f(fm, sh);
            settle();
        }
    }
};

// The stages in LDS: one array each, as reads of one and direct loads into
// another do not alias.
#define CPO_STAGES(P)                                                                      \
    __shared__ __attribute__((aligned(1024))) char s0[P::STAGE];                           \
    __shared__ __attribute__((aligned(1024))) char s1[P::STAGE];                           \
    __shared__ __attribute__((aligned(1024))) char s2[P::S > 2 ? P::STAGE : 16];           \
    __shared__ __attribute__((aligned(1024))) char s3[P::S > 3 ? P::STAGE : 16];           \
    const Stages st = {{s0, s1, s2, s3},                                                   \
                       {s0 + P::OpA::BYTES, s1 + P::OpA::BYTES, s2 + P::OpA::BYTES, s3 + P::OpA::BYTES}, s0}

template <class P>
__global__ __launch_bounds__(P::NT, P::WAVES) void product_kernel(GemmArgs g) {
    CPO_STAGES(P);
    Place at;
    if (P::place(g, blockIdx.x, at)) P::template run<0>(g, st, P::tile(g, at));
}

// 256 x 256 tiles (P), one to a CU, and their halves by rows (H), with the
// stages of both in the same LDS: P's two of A and B, H's three of B and A.
template <class P, class H>
struct Halving {
    static_assert(P::NT == H::NT && 2 * H::BM == P::BM && H::BN == P::BN && P::S == 2 && H::S == 3, "halves");
    static constexpr int HA = H::OpA::BYTES, HB = H::OpB::BYTES;
    static_assert(P::STAGE == 2 * HB && P::STAGE == HB + 2 * HA, "stages");
    static constexpr int LAST = HA;

    template <int ARG>
    __device__ __forceinline__ static void run(const GemmArgs &g, char *s0, char *s1, char *s2, const Tile &t, bool half) {
        if (half)
            H::template run<ARG>(g, Stages{{s1 + HB, s1 + HB + HA, s2, s2}, {s0, s0 + HB, s1, s1}, s0}, t);
        else
            P::template run<ARG>(g, Stages{{s0, s1, s0, s1}, {s0 + P::OpA::BYTES, s1 + P::OpA::BYTES, s0, s1}, s0}, t);
    }
};
#define CPO_HALVING_STAGES(P, V)                                 \
    __shared__ __attribute__((aligned(1024))) char s0[P::STAGE]; \
    __shared__ __attribute__((aligned(1024))) char s1[P::STAGE]; \
    __shared__ __attribute__((aligned(1024))) char s2[V::LAST]

// A last round that is at most half full is computed as the halves of its
// tiles, a workgroup each: 8192 x 2048 x 4096 over 16 experts (2.5 rounds)
// 180 us with either tile alone, 163 with both; 2048 x 8192 x 10240 (1.25
// rounds) 375 -> 317 us.
template <class P, class H>
__global__ __launch_bounds__(P::NT, P::WAVES) void halving_kernel(GemmArgs g) {
    using V = Halving<P, H>;
    CPO_HALVING_STAGES(P, V);
    Place at{};
    at.ntm = g.mode == kGroupRows ? count_tiles(g.off, g.groups, g.M, P::BM, at.scan) : g.ntm;
    const int units = at.ntm * g.ntn * g.nsplit, halved = halved_tiles(units), whole = units - halved;
    const int b = blockIdx.x;
    int half = 0;
    if (b < whole) {
        at.unit = xcd_remap(b, whole);
    } else if (b < whole + 2 * halved) {
        const int h = xcd_remap(b - whole, 2 * halved);
        at.unit = whole + h / 2;
        half = h & 1;
    } else {
        return;
    }
    Tile t = P::tile(g, at);
    t.row0 += half * H::BM;
    if (t.row0 < t.row_end) V::template run<0>(g, s0, s1, s2, t, b >= whole);
}

// A layer's gradients in one launch: the tiles of dX (nx workgroups), of dW
// (nw), and the bias sums (the rest).  What one of them leaves of the device
// in its last round, the next one's tiles take.
static_assert(sizeof(GemmArgs) % 8 == 0, "the second argument follows the first");
template <class PX, class PW>
__global__ __launch_bounds__(PX::NT, PX::WAVES) void gradients_kernel(GemmArgs x, GemmArgs w, GradArgs d, int nx, int nw) {
    static_assert(PX::NT == PW::NT && PX::STAGE == PW::STAGE && PX::S == PW::S, "one shape of workgroup");
    CPO_STAGES(PX);
    const int b = blockIdx.x;
    Place at;
    if (b < nx) {
        if (PX::place(x, b, at)) PX::template run<0>(x, st, PX::tile(x, at));
    } else if (b < nx + nw) {
        if (PW::place(w, b - nx, at)) PW::template run<sizeof(GemmArgs)>(w, st, PW::tile(w, at));
    } else {
        join_columns<typename PX::T, PX::NT>(d, b - nx - nw, reinterpret_cast<float *>(s0));
    }
}

// The same for 256 x 256 tiles, dX's with at most half of their rows as halves:
// 4099 x 2048 x 4096 over 8 experts 180 -> 176 us.  (In the forward pass, where
// an expert's tiles keep step and share what they read, this lost: 161 -> 163.)
template <class PX, class HX, class PW>
__global__ __launch_bounds__(PX::NT, PX::WAVES) void halving_gradients_kernel(GemmArgs x, GemmArgs w, GradArgs d, int nx, int nw) {
    using V = Halving<PX, HX>;
    static_assert(PX::NT == PW::NT && PX::STAGE == PW::STAGE && PX::S == PW::S, "one shape of workgroup");
    CPO_HALVING_STAGES(PX, V);
    const int b = blockIdx.x;
    Place at;
    if (b < nx) {
        if (PX::place(x, b, at)) {
            const Tile t = PX::tile(x, at);
            V::template run<0>(x, s0, s1, s2, t, t.row_end - t.row0 <= HX::BM);
        }
    } else if (b < nx + nw) {
        if (PW::place(w, b - nx, at))
            PW::template run<sizeof(GemmArgs)>(
                w, Stages{{s0, s1, s0, s1}, {s0 + PW::OpA::BYTES, s1 + PW::OpA::BYTES, s0, s1}, s0}, PW::tile(w, at));
    } else {
        join_columns<typename PX::T, PX::NT>(d, b - nx - nw, reinterpret_cast<float *>(s0));
    }
}

// The tile configurations with direct loads, by type.
template <class T, bool AKC, bool BKC, int CFG>
struct TileOf;
template <class T, bool A, bool B> struct TileOf<T, A, B, kTile256> { using P = Product<T, 256, 256, 2, 4, 2, A, B, true>; };
template <class T, bool A, bool B> struct TileOf<T, A, B, kTile128x256> { using P = Product<T, 128, 256, 2, 4, 3, A, B, true>; };
template <class T, bool A, bool B> struct TileOf<T, A, B, kTile128> { using P = Product<T, 128, 128, 2, 2, 2, A, B, true>; };
template <class T, bool A, bool B> struct TileOf<T, A, B, kTile64x128> { using P = Product<T, 64, 128, 2, 2, 3, A, B, true>; };
template <class T, bool A, bool B> struct TileOf<T, A, B, kTile64> { using P = Product<T, 64, 64, 2, 2, 4, A, B, true>; };

// f(integral_constant) of a configuration that this type has
template <class T, class F>
hipError_t with_tile(Config c, F &&f) {
    if constexpr (sizeof(T) == 2) {
        if (c == kTile256) return f(ic<kTile256>{});
        if (c == kTile128x256) return f(ic<kTile128x256>{});
    }
    if (c == kTile128) return f(ic<kTile128>{});
    if (c == kTile64x128) return f(ic<kTile64x128>{});
    if (c == kTile64) return f(ic<kTile64>{});
    return hipErrorInvalidValue;
}

template <class T, bool AKC, bool BKC>
hipError_t launch_layout(Config c, bool direct, const GemmArgs &g, int grid, hipStream_t s) {
    auto launch = [&](auto P) {
        using K = typename decltype(P)::P;
        hipLaunchKernelGGL(HIP_KERNEL_NAME(product_kernel<K>), dim3(grid), dim3(K::NT), 0, s, g);
        return hipGetLastError();
    };
    if constexpr (AKC)
        if (c == kTile16) {
            struct Direct { using P = Product<T, 16, 128, 1, 4, 4, AKC, BKC, true>; };
            struct Staged { using P = Product<T, 16, 128, 1, 4, 2, AKC, BKC, false>; };
            static_assert(Direct::P::NT == kShapes[kTile16].threads && Staged::P::NT == Direct::P::NT, "threads");
            return direct ? launch(Direct{}) : launch(Staged{});
        }
    if (!direct) return hipErrorInvalidValue;  // the host packs their operands
    if constexpr (sizeof(T) == 2)
        if (c == kTile256 && (AKC || g.mode != kGroupSum)) {
            using P = typename TileOf<T, AKC, BKC, kTile256>::P;
            using H = typename TileOf<T, AKC, BKC, kTile128x256>::P;
            hipLaunchKernelGGL(HIP_KERNEL_NAME(halving_kernel<P, H>), dim3(grid), dim3(P::NT), 0, s, g);
            return hipGetLastError();
        }
    return with_tile<T>(c, [&](auto C) {
        if constexpr (AKC && C == kTile256) return hipErrorInvalidValue;  // (above)
        else return launch(TileOf<T, AKC, BKC, decltype(C)::value>{});
    });
}

template <class T, bool BKC>
hipError_t launch_gradients_layout(Config c, const GemmArgs &x, int nx, const GemmArgs &w, int nw, const GradArgs &d, int nd,
                                   hipStream_t s) {
    return with_tile<T>(c, [&](auto C) {
        using PX = typename TileOf<T, true, BKC, decltype(C)::value>::P;
        using PW = typename TileOf<T, false, false, decltype(C)::value>::P;
        static_assert(PX::NT == kShapes[decltype(C)::value].threads, "threads");
        const dim3 grid(nx + nw + nd), block(PX::NT);
        if constexpr (C == kTile256) {
            using HX = typename TileOf<T, true, BKC, kTile128x256>::P;
            hipLaunchKernelGGL(HIP_KERNEL_NAME(halving_gradients_kernel<PX, HX, PW>), grid, block, 0, s, x, w, d, nx, nw);
        } else {
            hipLaunchKernelGGL(HIP_KERNEL_NAME(gradients_kernel<PX, PW>), grid, block, 0, s, x, w, d, nx, nw);
        }
        return hipGetLastError();
    });
}

}  // namespace cpo
