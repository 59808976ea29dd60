// The gated feed-forward projections on scaled-FP4 matrix instructions.
//
//   forward   G = X Wg^T, U = X Wu^T, H = a(G) * U       a(g) = g s(z(g))
//   gradient  D = dY W^T, dU = D * a(G), dG = D * U * a'(G)
//
// (a in gated_act.h; few rows: gated_small.hip.)  Two forms of the K loop: where
// there are 256 x 256 tiles for every compute unit, that of gemm_core.h, eight
// waves of 128 x 64; where there are not, four waves on a tile of 256 or 128
// rows by 128 columns, with a shorter ring of its own (below), so that more
// compute units take part.
//
// Forward: the product's columns are G's and U's, half and half, interleaved
// in groups of 32 so that two neighbouring 32-column accumulator tiles of a
// wave are G and U of the same outputs.  The activation then needs no exchange
// between lanes: H is formed from the fp32 accumulators and only rounded
// results are written, instead of writing G and U, reading them back and
// writing H.
// Gradient: the plain tile, with the derivative applied to the fp32 tile in
// the epilogue; G and U are read ahead of their use there, so D is never
// written.
#include "gated_act.h"
#include "gemm_core.h"

namespace fp4q {

// 256 x 128 and 128 x 128 tiles, four waves of 128 x 64 or 64 x 64.
template <int ROWS>
struct MidLayout {
    static constexpr int WAVES = 4, WM = 2, WN = 2, TM = ROWS / 64, TN = 2;
    static constexpr int WROWS = 32 * TM, WCOLS = 32 * TN, BM = WM * WROWS, BN = WN * WCOLS;
    static constexpr int RA = BM / 16, RB = BN / 16;  // 1 KB code regions per step
    static constexpr int RPW_A = RA / WAVES, RPW_B = RB / WAVES;
    static constexpr int OFF_B = RA * REGION;
    static constexpr int SPW_A = BM / 128;            // 32-row scale pieces of A per wave
};
template <>
struct Layout<2> : MidLayout<256> {};
template <>
struct Layout<3> : MidLayout<128> {};

// LDS of the four-wave form: a ring of four K steps of codes and four groups
// of scales (8 bytes per row: two steps, or, where K % 128 == 64 and scale rows
// are only 2-byte aligned, one step whose two halves fill a dword each).
constexpr int MSTAGE = 24 * REGION, MSCALE = 384 * 8;
__shared__ __attribute__((aligned(16))) uint8_t mt0[MSTAGE];
__shared__ __attribute__((aligned(16))) uint8_t mt1[MSTAGE];
__shared__ __attribute__((aligned(16))) uint8_t mt2[MSTAGE];
__shared__ __attribute__((aligned(16))) uint8_t mt3[MSTAGE];
__shared__ __attribute__((aligned(16))) uint8_t ms0[MSCALE];
__shared__ __attribute__((aligned(16))) uint8_t ms1[MSCALE];
__shared__ __attribute__((aligned(16))) uint8_t ms2[MSCALE];
__shared__ __attribute__((aligned(16))) uint8_t ms3[MSCALE];

template <int CFG>
struct LaneMap {
    int lane, wave, wm, wn, half, l32;
    __device__ __forceinline__ static LaneMap make() {
        LaneMap m;
        m.lane = threadIdx.x & 63;
        m.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        m.wm = m.wave / Layout<CFG>::WN;
        m.wn = m.wave % Layout<CFG>::WN;
        m.half = m.lane >> 5;
        m.l32 = m.lane & 31;
        return m;
    }
};

#if defined(__HIP_DEVICE_COMPILE__)  // the host pass cannot instantiate buffer resources

// Load sources, as Src of gemm_core.h: resources that end at the operand's
// last row inside the tile, per-lane offsets, and the K step's scalar offset.
// PAIR: B's 32-row groups alternate between the two operands, so group 2w
// holds 32 rows of the first and group 2w + 1 the same rows of the second; a
// wave's code regions all belong to one of them (the parity of wave / 2), its
// scale rows to one (the parity of wave).
template <int CFG, int TAIL, int PAIR>
struct MidSrc {
    using G = Layout<CFG>;
    __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
    uint32_t va[G::RPW_A], vb[G::RPW_B], vsa[G::SPW_A], vsb;
    int soff;

    __device__ __forceinline__ void init(const GatedCall& o, int m0, int n0, const LaneMap<CFG>& l) {
        const int kbytes = o.K / 2, kscale = o.K / 32;
        const int rows_a = min(o.M - m0, G::BM), rows_b = min(o.F - n0, PAIR ? G::BN / 2 : G::BN);
        const uint8_t* bc = PAIR && ((l.wave >> 1) & 1) ? o.bc2 : o.bc;
        const uint8_t* bs = PAIR && (l.wave & 1) ? o.bs2 : o.bs;
        auto res = [](const uint8_t* p, int64_t first, int bytes) __attribute__((always_inline)) {
            return __builtin_amdgcn_make_buffer_rsrc((void*)(p + first), (short)0, bytes, BUF_FLAGS);
        };
        ra = res(o.ac, (int64_t)m0 * kbytes, rows_a * kbytes);
        rb = res(bc, (int64_t)n0 * kbytes, rows_b * kbytes);
        rsa = res(o.as, (int64_t)m0 * kscale, rows_a * kscale);
        rsb = res(bs, (int64_t)n0 * kscale, rows_b * kscale);
        // lane 4j + p of a region loads chunk p ^ ((j / 4) % 4) of row j
        const int j = l.lane >> 2, c = ((l.lane & 3) ^ ((j >> 2) & 3)) * 16;
#pragma unroll
        for (int q = 0; q < G::RPW_A; ++q)
            va[q] = (uint32_t)(((q * G::WAVES + l.wave) * 16 + j) * kbytes + c);
#pragma unroll
        for (int q = 0; q < G::RPW_B; ++q) {
            const int row = PAIR ? q * 32 + (l.wave & 1) * 16 : (q * G::WAVES + l.wave) * 16;
            vb[q] = (uint32_t)((row + j) * kbytes + c);
        }
        // a scale piece is 32 rows, two lanes each: pieces wave (and wave + 4) of
        // A's, and piece wave of B's four
        const int part = (l.lane & 1) * (TAIL ? 2 : 4), row = l.lane >> 1;
#pragma unroll
        for (int q = 0; q < G::SPW_A; ++q)
            vsa[q] = (uint32_t)(((q * 4 + l.wave) * 32 + row) * kscale + part);
        vsb = (uint32_t)(((PAIR ? l.wave >> 1 : l.wave) * 32 + row) * kscale + part);
        soff = 0;
    }
    // Direct-to-LDS loads of the K step the sources point at; they then advance
    // unless that was the last one (re-issued past the end of K, so that every
    // step issues the same number of loads).
    __device__ __forceinline__ void codes(uint8_t* stage, int wave, bool advance) {
#pragma unroll
        for (int q = 0; q < G::RPW_A; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra, (lds_ptr_t)(stage + (q * G::WAVES + wave) * REGION), 16, va[q], soff, 0, 0);
#pragma unroll
        for (int q = 0; q < G::RPW_B; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rb, (lds_ptr_t)(stage + G::OFF_B + (q * G::WAVES + wave) * REGION), 16, vb[q], soff, 0,
                0);
        soff += advance ? BKB : 0;
    }
    // Scales of group g: row R's 8 LDS bytes at 8 R.  The group's offset is part
    // of the lane's, so the range check covers it.
    __device__ __forceinline__ void scales(uint8_t* buf, int wave, int g) {
        uint32_t off = (uint32_t)g * (TAIL ? 4 : 8);
        asm volatile("" : "+s"(off));  // one scalar; no hoisted vector offsets
#pragma unroll
        for (int q = 0; q <= G::SPW_A; ++q) {
            const bool b = q == G::SPW_A;
            lds_ptr_t dst = (lds_ptr_t)(buf + (b ? G::BM / 32 + wave : q * 4 + wave) * 256);
            const uint32_t v = (b ? vsb : vsa[b ? 0 : q]) + off;
            if constexpr (TAIL)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(b ? rsb : rsa, dst, 2, v, 0, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(b ? rsb : rsa, dst, 4, v, 0, 0, 0);
        }
    }
};

// Scale words of step word w of a group for this lane's rows.
template <int CFG, int TAIL>
__device__ __forceinline__ void mid_scales(const uint8_t* buf, int w, const LaneMap<CFG>& l,
                                           uint32_t (&sa)[Layout<CFG>::TM],
                                           uint32_t (&sb)[Layout<CFG>::TN]) {
    using G = Layout<CFG>;
    auto word = [&](int row) __attribute__((always_inline)) -> uint32_t {
        if (TAIL) {
            const u32x2 d = *(const u32x2*)(buf + row * 8);
            return (d.x & 0xFFFFu) | (d.y << 16);
        }
        return *(const uint32_t*)(buf + row * 8 + w * 4);
    };
#pragma unroll
    for (int i = 0; i < G::TM; ++i) sa[i] = word(l.wm * G::WROWS + i * 32 + l.l32);
#pragma unroll
    for (int j = 0; j < G::TN; ++j) sb[j] = word(G::BM + l.wn * G::WCOLS + j * 32 + l.l32);
}

// The K loop of the four-wave form.  Step t multiplies two halves (64 elements
// each) of its stage; it issues the code loads of step t + 3 into the stage of
// step t - 1, which every wave finished reading before the last barrier, and,
// ahead of them, the scales of step t + 3 where that opens a group.  So what
// is behind the codes of step t + 1, which have to land before step t's
// barrier, is the codes of two steps and one group of scales (TAIL: two), the
// same in every step.  Order within a step, fenced against the compiler's
// scheduler: read the fragments of the second half, issue loads, multiply the
// first half; wait, barrier; read the scales and the first fragments of step
// t + 1, multiply the second half.  Eight steps are unrolled, so that every
// buffer is named at compile time (the compiler then sees that loads in flight
// and reads touch different LDS objects).
template <int CFG, int TAIL, int PAIR>
__device__ __forceinline__ void mid_kloop(v16f (&acc)[Layout<CFG>::TM][Layout<CFG>::TN],
                                          const GatedCall& o, int m0, int n0,
                                          const LaneMap<CFG>& l) {
    using G = Layout<CFG>;
    constexpr int SG = TAIL ? 1 : 2;
    constexpr int BEHIND = 2 * (G::RPW_A + G::RPW_B) + (TAIL ? 2 : 1) * (G::SPW_A + 1);
    const int ksteps = (o.K / 2 + BKB - 1) / BKB;
    const int off0 = (l.l32 >> 4) * REGION + region_slot(l.l32 & 15, l.half) * 16;
    const int off1 = (l.l32 >> 4) * REGION + region_slot(l.l32 & 15, 2 + l.half) * 16;
    MidSrc<CFG, TAIL, PAIR> src;
    src.init(o, m0, n0, l);
    Frags<CFG> FA, FB;
    uint32_t sa[G::TM], ra[G::TM], sb[G::TN], rb[G::TN];
    const int sh = 8 * l.half;
    src.scales(ms0, l.wave, 0);
    src.codes(mt0, l.wave, 1 < ksteps);
    if (TAIL) src.scales(ms1, l.wave, 1);
    src.codes(mt1, l.wave, 2 < ksteps);
    src.scales(TAIL ? ms2 : ms1, l.wave, TAIL ? 2 : 1);
    src.codes(mt2, l.wave, 3 < ksteps);
    FP4Q_WAIT_VMCNT(BEHIND);
    __builtin_amdgcn_s_barrier();
    mid_scales<CFG, TAIL>(ms0, 0, l, ra, rb);
    read_frags<CFG>(mt0, off0, l.wm, l.wn, FA);

#define FP4Q_SBUF(P) (((P) / SG) % 4 == 0 ? ms0 : ((P) / SG) % 4 == 1 ? ms1 : ((P) / SG) % 4 == 2 ? ms2 : ms3)
#define FP4Q_MSTEP(P, CUR, NEXT1, NEXTL)                                                \
    do {                                                                                \
        const int t_ = kt + (P);                                                        \
        __builtin_amdgcn_sched_barrier(0);                                              \
        shift_scales<CFG>(ra, rb, sh, sa, sb);                                          \
        read_frags<CFG>(CUR, off1, l.wm, l.wn, FB);                                     \
        if (((P) + 3) % SG == 0) src.scales(FP4Q_SBUF((P) + 3), l.wave, (t_ + 3) / SG); \
        src.codes(NEXTL, l.wave, t_ + 4 < ksteps);                                      \
        __builtin_amdgcn_sched_barrier(0);                                              \
        mfma_half<CFG, 0, 0>(FA, sa, sb, acc);                                          \
        __builtin_amdgcn_sched_barrier(0);                                              \
        FP4Q_WAIT_VMCNT(BEHIND);                                                        \
        __builtin_amdgcn_s_waitcnt(0xC07F);                                             \
        __builtin_amdgcn_s_barrier();                                                   \
        __builtin_amdgcn_sched_barrier(0);                                              \
        mid_scales<CFG, TAIL>(FP4Q_SBUF((P) + 1), ((P) + 1) % SG, l, ra, rb);           \
        read_frags<CFG>(NEXT1, off0, l.wm, l.wn, FA);                                   \
        if (!TAIL || t_ != ksteps - 1) mfma_half<CFG, 0, 1>(FB, sa, sb, acc);           \
    } while (0)
#define FP4Q_MTURN(O, GUARD)                                     \
    do {                                                         \
        if (GUARD(O + 0)) FP4Q_MSTEP(O + 0, mt0, mt1, mt3);      \
        if (GUARD(O + 1)) FP4Q_MSTEP(O + 1, mt1, mt2, mt0);      \
        if (GUARD(O + 2)) FP4Q_MSTEP(O + 2, mt2, mt3, mt1);      \
        if (GUARD(O + 3)) FP4Q_MSTEP(O + 3, mt3, mt0, mt2);      \
    } while (0)
#define FP4Q_ALL(P) true
#define FP4Q_EXISTS(P) (kt + (P) < ksteps)
    int kt = 0;
    for (; kt + 8 <= ksteps; kt += 8) {
        FP4Q_MTURN(0, FP4Q_ALL);
        FP4Q_MTURN(4, FP4Q_ALL);
    }
    if (kt < ksteps) {
        FP4Q_MTURN(0, FP4Q_EXISTS);
        FP4Q_MTURN(4, FP4Q_EXISTS);
    }
#undef FP4Q_MTURN
#undef FP4Q_MSTEP
#undef FP4Q_SBUF
#undef FP4Q_ALL
#undef FP4Q_EXISTS
    FP4Q_WAIT_VMCNT(0);  // the re-issued loads past the end of K have landed
}

// The tile's K loop in either form.
template <int CFG, int TAIL, int PAIR>
__device__ __forceinline__ void tile_kloop(v16f (&acc)[Layout<CFG>::TM][Layout<CFG>::TN],
                                           const GatedCall& o, int m0, int n0,
                                           const LaneMap<CFG>& l) {
#pragma unroll
    for (int i = 0; i < Layout<CFG>::TM; ++i)
#pragma unroll
        for (int j = 0; j < Layout<CFG>::TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    if constexpr (CFG == 0) {
        const int off0 = (l.l32 >> 4) * REGION + region_slot(l.l32 & 15, l.half) * 16;
        const int off1 = (l.l32 >> 4) * REGION + region_slot(l.l32 & 15, 2 + l.half) * 16;
        gemm_kloop<0, 0, TAIL, PAIR>(acc, o.ac, o.as, o.bc, o.bs, o.K, o.M, o.F, m0, n0, l.wave,
                                     l.lane, l.wm, l.wn, l.half, l.l32, off0, off1, (l.l32 >> 3) & 3,
                                     o.bc2, o.bs2);
    } else {
        mid_kloop<CFG, TAIL, PAIR>(acc, o, m0, n0, l);
    }
    __syncthreads();  // all waves are done with the operand stages
}

// This wave's private part of the operand stages, EREG bytes, free once the
// K loop's last barrier has passed.
template <int CFG, int EREG>
__device__ __forceinline__ uint8_t* wave_stage(int wave) {
    static_assert(EREG % 16 == 0 && 2 * EREG <= (CFG == 0 ? STAGE : MSTAGE), "two to a stage");
    const int s = wave >> 1;
    uint8_t* st;
    if constexpr (CFG == 0)
        st = s == 0 ? st0 : s == 1 ? st1 : s == 2 ? st2 : st3;
    else
        st = s == 0 ? mt0 : mt1;
    return st + (wave & 1) * EREG;
}
#endif

// Origin of tile number t, bm x bn outputs: XCD-contiguous, then grouped along M.
__device__ __forceinline__ void gated_origin(int t, int tiles_m, int tiles_n, int bm, int bn, int& m0,
                                             int& n0) {
    const int full = (tiles_m * tiles_n / 8) * 8;
    if (t < full) t = (t % 8) * (full / 8) + t / 8;
    const int per_group = GROUP_M * tiles_n;
    const int first = t / per_group * GROUP_M, in = t % per_group;
    const int gsize = min(GROUP_M, tiles_m - first);
    m0 = (first + in % gsize) * bm;
    n0 = in / gsize * bn;
}

// SAVE: G and U are written too (bf16, for the gradient).
template <int CFG, int GELU, int SAVE, int TAIL>
__global__ __launch_bounds__(64 * Layout<CFG>::WAVES, 1) void gemm_gated_kernel(const GatedCall o,
                                                                                int tiles_m,
                                                                                int tiles_n) {
#if defined(__HIP_DEVICE_COMPILE__)
    using G = Layout<CFG>;
    int m0, n0;
    gated_origin(blockIdx.x, tiles_m, tiles_n, G::BM, G::BN / 2, m0, n0);
    const LaneMap<CFG> l = LaneMap<CFG>::make();
    v16f acc[G::TM][G::TN];
    tile_kloop<CFG, TAIL, 1>(acc, o, m0, n0, l);

    constexpr int NOUT = SAVE ? 3 : 1;
    constexpr int PITCH = NOUT * 64 + 16;  // 32 bf16 of each output per row
    uint8_t* reg = wave_stage<CFG, 32 * PITCH>(l.wave);
    const int row0 = m0 + l.wm * G::WROWS;
    const int col = n0 + l.wn * 32 + (l.lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < G::TM; ++i) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float hv[4];
            const v16f &ga = acc[i][0], &ua = acc[i][1];
#pragma unroll
            for (int r = 0; r < 4; ++r) hv[r] = act_value<GELU>(ga[4 * g + r]) * ua[4 * g + r];
            uint8_t* dst = reg + l.l32 * PITCH + (8 * g + 4 * l.half) * 2;
            *(u32x2*)dst = (u32x2){pack_rne(hv[0], hv[1]), pack_rne(hv[2], hv[3])};
            if (SAVE) {
                *(u32x2*)(dst + 64) = (u32x2){pack_rne(ga[4 * g], ga[4 * g + 1]),
                                              pack_rne(ga[4 * g + 2], ga[4 * g + 3])};
                *(u32x2*)(dst + 128) = (u32x2){pack_rne(ua[4 * g], ua[4 * g + 1]),
                                               pack_rne(ua[4 * g + 2], ua[4 * g + 3])};
            }
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS writes done
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int out = 0; out < NOUT; ++out)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int rl = p * 16 + (l.lane >> 2);
                const u32x4 v = *(const u32x4*)(reg + rl * PITCH + out * 64 + (l.lane & 3) * 16);
                const int row = row0 + i * 32 + rl;
                if (row >= o.M) continue;
                uint16_t* base = out == 0 ? o.h : out == 1 ? o.gate : o.up;
                base += (int64_t)row * (out == 0 ? o.ldh : o.ldgu) + col;
                if (o.nt)
                    store8<1>(base, v, o.F - col);
                else
                    store8<0>(base, v, o.F - col);
            }
        __builtin_amdgcn_wave_barrier();
    }
#endif
}

template <int CFG, int GELU, int TAIL>
__global__ __launch_bounds__(64 * Layout<CFG>::WAVES, 1) void gemm_gated_grad_kernel(
    const GatedCall o, int tiles_m, int tiles_n) {
#if defined(__HIP_DEVICE_COMPILE__)
    using G = Layout<CFG>;
    int m0, n0;
    gated_origin(blockIdx.x, tiles_m, tiles_n, G::BM, G::BN, m0, n0);
    const LaneMap<CFG> l = LaneMap<CFG>::make();

    // In the epilogue a wave takes 32 rows of 64 columns at a time through LDS,
    // and a lane 8 consecutive columns of 4 rows.  G and U of that: four waves
    // have the registers to read all of it ahead of the K loop; eight read the
    // first two groups of rows before any is used, the others two groups ahead.
    constexpr int PITCH = 64 * 4 + 16, PASSES = 4;
    constexpr bool kEarly = CFG != 0;
    const int row0 = m0 + l.wm * G::WROWS + (l.lane >> 3);
    const int cl = (l.lane & 7) * 8;
    const int col = n0 + l.wn * G::WCOLS + cl;
    struct Pair {
        u32x4 g[PASSES], u[PASSES];
    };
    auto fetch = [&](int i, Pair& q) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int row = row0 + i * 32 + p * 8;
            q.g[p] = q.u[p] = (u32x4){0u, 0u, 0u, 0u};
            if (row >= o.M || col >= o.F) continue;
            const int64_t at = (int64_t)row * o.ldgu;
            q.g[p] = load8(o.gate + at, col, o.F);
            q.u[p] = load8(o.up + at, col, o.F);
        }
    };
    Pair in[kEarly ? G::TM : 2];
    if (kEarly) {
#pragma unroll
        for (int i = 0; i < G::TM; ++i) fetch(i, in[i]);
    }
    v16f acc[G::TM][G::TN];
    tile_kloop<CFG, TAIL, 0>(acc, o, m0, n0, l);

    uint8_t* reg = wave_stage<CFG, 32 * PITCH>(l.wave);
    if (!kEarly) {
        fetch(0, in[0]);
        fetch(1, in[1]);
    }
#pragma unroll
    for (int i = 0; i < G::TM; ++i) {
#pragma unroll
        for (int j = 0; j < G::TN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const v16f& a = acc[i][j];
                *(u32x4*)(reg + l.l32 * PITCH + (j * 32 + 8 * g + 4 * l.half) * 4) =
                    (u32x4){as_u32(a[4 * g]), as_u32(a[4 * g + 1]), as_u32(a[4 * g + 2]),
                            as_u32(a[4 * g + 3])};
            }
        __builtin_amdgcn_s_waitcnt(0xC07F);
        __builtin_amdgcn_wave_barrier();
        Pair& q = in[kEarly ? i : i & 1];
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const uint8_t* src = reg + (p * 8 + (l.lane >> 3)) * PITCH + cl * 4;
            const u32x4 d0 = *(const u32x4*)src, d1 = *(const u32x4*)(src + 16);
            const float d[8] = {as_f32(d0.x), as_f32(d0.y), as_f32(d0.z), as_f32(d0.w),
                                as_f32(d1.x), as_f32(d1.y), as_f32(d1.z), as_f32(d1.w)};
            u32x4 og, ou;
            gated_grad8<GELU>(d, settle8(q.g[p], col, o.F), settle8(q.u[p], col, o.F), og, ou);
            const int row = row0 + i * 32 + p * 8;
            if (row >= o.M) continue;
            const int64_t off = (int64_t)row * o.ldd + col;
            if (o.nt) {
                store8<1>(o.dgate + off, og, o.F - col);
                store8<1>(o.dup + off, ou, o.F - col);
            } else {
                store8<0>(o.dgate + off, og, o.F - col);
                store8<0>(o.dup + off, ou, o.F - col);
            }
        }
        __builtin_amdgcn_wave_barrier();
        if (!kEarly && i + 2 < G::TM) fetch(i + 2, q);
    }
#endif
}

template <int CFG, int GELU>
static hipError_t go_forward(const GatedCall& g, hipStream_t s) {
    using G = Layout<CFG>;
    const int tiles_m = (g.M + G::BM - 1) / G::BM, tiles_n = (g.F + G::BN / 2 - 1) / (G::BN / 2);
    const dim3 grid((unsigned)(tiles_m * tiles_n)), block(64 * G::WAVES);
#define FP4Q_GO(SAVE, TAIL)                                                                         \
    FP4Q_LAUNCH((gemm_gated_kernel<CFG, GELU, SAVE, TAIL>), grid, block, 0, s, g, tiles_m, tiles_n)
    if (g.gate) {
        if (g.K % 128) FP4Q_GO(1, 1); else FP4Q_GO(1, 0);
    } else {
        if (g.K % 128) FP4Q_GO(0, 1); else FP4Q_GO(0, 0);
    }
#undef FP4Q_GO
    return hipGetLastError();
}
// Outputs are stored non-temporally where their rows are whole cache lines: a
// line that two rows or tiles share would pass through memory in parts
// (gradient 4096 x 5601 x 2048 112 us, written back 82; at 5632 columns 70 and
// 68; forward 8192 x 5632 x 2048 120 and 124).
static bool lines(const void* p, int64_t ld) { return (uintptr_t)p % 128 == 0 && ld % 64 == 0; }

// Tiles of bm x bn outputs.
static int64_t tiles_of(const GatedCall& g, int bm, int bn) {
    return ((int64_t)g.M + bm - 1) / bm * ((g.F + bn - 1) / bn);
}

// The form is the one with the largest tiles that still finish in one round of
// the compute units, since larger tiles load less but a tile's K loop takes
// the same time on an idle chip.  Forward, us (small, 128-row, 256-row, 256 x 256):
//   M x F x K          64 x 1408 x 960    4.2   6.1   9.0  11.0
//                     512 x 1408 x 960    7.3   6.4   9.8  12.6
//                    2048 x 1408 x 960   20.6  13.3  10.8  13.3
//                    4096 x 1408 x 960   37.8  20.9  20.6  14.3
//                      1 x 5632 x 2048    7.1   7.3  11.5  14.5
//                    128 x 13824 x 5120   84.8  27.5  31.0  43.6
// and of the gradient:
//                     256 x 1408 x 960    4.7   9.2  15.7  23.1
//                    2048 x 1408 x 960   13.8  11.1  16.9  24.1
//                    1024 x 5632 x 2048  58.6  25.3  22.7  30.4
//                    2048 x 5632 x 2048   107  40.6  44.5  37.2
constexpr int64_t kOneRound = 256;

template <int GELU>
static hipError_t pick_forward(const GatedCall& g, hipStream_t s) {
    if (launch_gated_small(g, false, GELU, s)) return hipGetLastError();
    if (tiles_of(g, 128, 64) <= kOneRound) return go_forward<3, GELU>(g, s);
    if (tiles_of(g, 256, 64) <= kOneRound) return go_forward<2, GELU>(g, s);
    return go_forward<0, GELU>(g, s);
}

hipError_t launch_gemm_gated(int64_t M, int64_t F, int64_t K, const uint8_t* xc,
                             const uint8_t* xs, const uint8_t* gc, const uint8_t* gs,
                             const uint8_t* uc, const uint8_t* us, int act, uint16_t* h,
                             int64_t ldh, uint16_t* gate, uint16_t* up, int64_t ldgu,
                             hipStream_t s) {
    const GatedCall g{(int)M, (int)F, (int)K, xc, xs, gc, gs, uc, us, h, ldh, gate, up, ldgu,
                      nullptr, nullptr, 0,
                      lines(h, ldh) && (!gate || (lines(gate, ldgu) && lines(up, ldgu)))};
    return act ? pick_forward<1>(g, s) : pick_forward<0>(g, s);
}

template <int CFG, int GELU>
static hipError_t go_grad(const GatedCall& g, hipStream_t s) {
    using G = Layout<CFG>;
    const int tiles_m = (g.M + G::BM - 1) / G::BM, tiles_n = (g.F + G::BN - 1) / G::BN;
    const dim3 grid((unsigned)(tiles_m * tiles_n)), block(64 * G::WAVES);
    if (g.K % 128)
        FP4Q_LAUNCH((gemm_gated_grad_kernel<CFG, GELU, 1>), grid, block, 0, s, g, tiles_m, tiles_n);
    else
        FP4Q_LAUNCH((gemm_gated_grad_kernel<CFG, GELU, 0>), grid, block, 0, s, g, tiles_m, tiles_n);
    return hipGetLastError();
}
template <int GELU>
static hipError_t pick_grad(const GatedCall& g, hipStream_t s) {
    if (launch_gated_small(g, true, GELU, s)) return hipGetLastError();
    if (tiles_of(g, 128, 128) <= kOneRound) return go_grad<3, GELU>(g, s);
    if (tiles_of(g, 256, 128) <= kOneRound) return go_grad<2, GELU>(g, s);
    return go_grad<0, GELU>(g, s);
}

hipError_t launch_gemm_gated_grad(int64_t M, int64_t F, int64_t K, const uint8_t* yc,
                                  const uint8_t* ys, const uint8_t* wc, const uint8_t* ws,
                                  int act, const uint16_t* gate, const uint16_t* up,
                                  int64_t ldgu, uint16_t* dgate, uint16_t* dup, int64_t ldd,
                                  hipStream_t s) {
    const GatedCall g{(int)M, (int)F, (int)K, yc, ys, wc, ws, nullptr, nullptr, nullptr, 0,
                      (uint16_t*)gate, (uint16_t*)up, ldgu, dgate, dup, ldd,
                      lines(dgate, ldd) && lines(dup, ldd)};
    return act ? pick_grad<1>(g, s) : pick_grad<0>(g, s);
}

}  // namespace fp4q
