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

// 256 x 128 and 128 x 128 tiles, four waves of 128 x 64 or 64 x 64.  A K step is
// 256 elements, 128 bytes of each row: loads take whole cache lines (8 rows x
// 128 bytes each) and there is half as much waiting as with half the step.
template <int ROWS>
struct MidLayout {
    static constexpr int WAVES = 4, WM = 2, WN = 2, TM = ROWS / 64, TN = 2;
    static constexpr int WROWS = 32 * TM, WCOLS = 32 * TN, BM = WM * WROWS, BN = WN * WCOLS;
    static constexpr int RPW_A = BM / 32, RPW_B = BN / 32;  // 1 KB code regions per wave and step
    static constexpr int OFF_B = BM * 128;                  // B codes within a stage
    static constexpr int STAGES = ROWS == 128 ? 4 : 3;
};
template <>
struct Layout<2> : MidLayout<256> {};
template <>
struct Layout<3> : MidLayout<128> {};

// Their LDS: a ring of STAGES steps, codes and behind them scales.  A row's
// scales of a step are 8 bytes, or, where K % 128 == 64 (TAIL) and scale rows
// are only 2-byte aligned, four halves of a dword each.  At 256 rows TAIL has
// room for two steps of scales only, in buffers of their own.  Few objects, and
// each named at compile time: the compiler then tells reads from the loads in
// flight into other ones, and does not wait for those.
constexpr int MBK = 128;  // operand bytes per row per step
constexpr int MSTAGE3 = 256 * MBK, MSTAGE2 = 384 * MBK;
template <int CFG, int TAIL>
constexpr int scale_ring() { return CFG == 2 && TAIL ? 2 : Layout<CFG>::STAGES; }
__shared__ __attribute__((aligned(16))) uint8_t ma0[MSTAGE3 + 256 * 16];
__shared__ __attribute__((aligned(16))) uint8_t ma1[MSTAGE3 + 256 * 16];
__shared__ __attribute__((aligned(16))) uint8_t ma2[MSTAGE3 + 256 * 16];
__shared__ __attribute__((aligned(16))) uint8_t ma3[MSTAGE3 + 256 * 16];
__shared__ __attribute__((aligned(16))) uint8_t mb0[MSTAGE2 + 384 * 8];
__shared__ __attribute__((aligned(16))) uint8_t mb1[MSTAGE2 + 384 * 8];
__shared__ __attribute__((aligned(16))) uint8_t mb2[MSTAGE2 + 384 * 8];
__shared__ __attribute__((aligned(16))) uint8_t mc0[MSTAGE2];
__shared__ __attribute__((aligned(16))) uint8_t mc1[MSTAGE2];
__shared__ __attribute__((aligned(16))) uint8_t mc2[MSTAGE2];
__shared__ __attribute__((aligned(16))) uint8_t ms0[384 * 16];
__shared__ __attribute__((aligned(16))) uint8_t ms1[384 * 16];
// Stage and scale buffer of step number I.
template <int CFG, int TAIL, int I>
__device__ __forceinline__ uint8_t* mid_stage() {
    constexpr int i = I % Layout<CFG>::STAGES;
    if constexpr (CFG == 3)
        return i == 0 ? ma0 : i == 1 ? ma1 : i == 2 ? ma2 : ma3;
    else if constexpr (TAIL)
        return i == 0 ? mc0 : i == 1 ? mc1 : mc2;
    else
        return i == 0 ? mb0 : i == 1 ? mb1 : mb2;
}
template <int CFG, int TAIL, int I>
__device__ __forceinline__ uint8_t* mid_sbuf() {
    if constexpr (CFG == 2 && TAIL)
        return I % 2 ? ms1 : ms0;
    else
        return mid_stage<CFG, TAIL, I>() + (CFG == 3 ? MSTAGE3 : MSTAGE2);
}

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

// Load sources: buffer resources that end at the operand's last row inside the
// tile, and per-lane offsets that advance with K, so that the range check
// covers every byte (what lies past a row's end is the next row or zeros, and
// is not multiplied).  PAIR: B's 32-row groups alternate between the two
// operands, so group 2w holds 32 rows of the first and group 2w + 1 the same
// rows of the second.
//
// In LDS a region is 8 rows x 128 bytes; 16-byte chunk c of row j lies in slot
// 8 j + (c ^ j ^ (region's parity)), so that the 16 rows that are read together
// spread over all banks.
template <int CFG, int TAIL, int PAIR>
struct MidSrc {
    using G = Layout<CFG>;
    static constexpr int SROWS = TAIL ? 16 : 32;        // rows of a scale load, 64 / SROWS lanes each
    static constexpr int SPW_A = G::BM / SROWS / 4, SPW_B = G::BN / SROWS / 4;
    static constexpr int LC = G::RPW_A + G::RPW_B, LS = SPW_A + SPW_B;  // loads per wave and step
    __amdgpu_buffer_rsrc_t ra, rb, rb2, rsa, rsb;
    uint32_t va[G::RPW_A], vb[G::RPW_B], vsa[SPW_A], vsb[SPW_B];

    __device__ __forceinline__ void init(const GatedCall& o, int m0, int n0, const LaneMap<CFG>& l) {
        const int kbytes = o.K / 2, kscale = o.K / 32;
        const int rows_a = min(o.M - m0, G::BM), rows_b = min(o.F - n0, PAIR ? G::BN / 2 : G::BN);
        auto res = [](const uint8_t* p, int64_t first, int bytes) __attribute__((always_inline)) {
            return __builtin_amdgcn_make_buffer_rsrc((void*)(p + first), (short)0, bytes, BUF_FLAGS);
        };
        // scale loads of B: TAIL's are half a 32-row group, two of which a wave takes
        const bool second = PAIR && (TAIL ? (l.wave >> 1) & 1 : l.wave & 1);
        ra = res(o.ac, (int64_t)m0 * kbytes, rows_a * kbytes);
        rb = res(o.bc, (int64_t)n0 * kbytes, rows_b * kbytes);
        rb2 = PAIR ? res(o.bc2, (int64_t)n0 * kbytes, rows_b * kbytes) : rb;
        rsa = res(o.as, (int64_t)m0 * kscale, rows_a * kscale);
        rsb = res(second ? o.bs2 : o.bs, (int64_t)n0 * kscale, rows_b * kscale);
        const int j = l.lane >> 3, c = ((l.lane & 7) ^ j ^ (l.wave & 1)) * 16;
#pragma unroll
        for (int q = 0; q < G::RPW_A; ++q)
            va[q] = (uint32_t)(((q * 4 + l.wave) * 8 + j) * kbytes + c);
#pragma unroll
        for (int q = 0; q < G::RPW_B; ++q) {  // region 4 q + wave: group q
            const int row = (PAIR ? q >> 1 : q) * 32 + l.wave * 8;
            vb[q] = (uint32_t)((row + j) * kbytes + c);
        }
        const int srow = l.lane / (64 / SROWS), part = l.lane % (64 / SROWS) * (TAIL ? 2 : 4);
#pragma unroll
        for (int q = 0; q < SPW_A; ++q)
            vsa[q] = (uint32_t)(((q * 4 + l.wave) * SROWS + srow) * kscale + part);
#pragma unroll
        for (int q = 0; q < SPW_B; ++q) {
            const int row = !PAIR ? (q * 4 + l.wave) * SROWS
                            : TAIL ? q * 32 + (l.wave & 1) * 16 : (l.wave >> 1) * 32;
            vsb[q] = (uint32_t)((row + srow) * kscale + part);
        }
    }
    // Direct-to-LDS loads of the K step the sources point at; they then advance
    // unless that was the last one (re-issued past the end of K, so that every
    // step issues the same number of loads).
    __device__ __forceinline__ void codes(uint8_t* stage, int wave, bool advance) {
        const uint32_t by = advance ? MBK : 0;
#pragma unroll
        for (int q = 0; q < G::RPW_A; ++q) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra, (lds_ptr_t)(stage + (q * 4 + wave) * REGION), 16, va[q], 0, 0, 0);
            va[q] += by;
        }
#pragma unroll
        for (int q = 0; q < G::RPW_B; ++q) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                PAIR && (q & 1) ? rb2 : rb, (lds_ptr_t)(stage + G::OFF_B + (q * 4 + wave) * REGION), 16,
                vb[q], 0, 0, 0);
            vb[q] += by;
        }
    }
    // Scales of step t: row R's 8 (TAIL: 16) LDS bytes at that times R.
    __device__ __forceinline__ void scales(uint8_t* buf, int wave, int t) {
        uint32_t off = (uint32_t)t * 8;
        asm volatile("" : "+s"(off));  // one scalar; no hoisted vector offsets
#pragma unroll
        for (int q = 0; q < SPW_A + SPW_B; ++q) {
            const bool b = q >= SPW_A;
            lds_ptr_t dst = (lds_ptr_t)(buf + (q * 4 + wave) * 256);
            const uint32_t v = (b ? vsb[b ? q - SPW_A : 0] : vsa[b ? 0 : q]) + off;
            if constexpr (TAIL)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(b ? rsb : rsa, dst, 2, v, 0, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(b ? rsb : rsa, dst, 4, v, 0, 0, 0);
        }
    }
};

// The K loop of the four-wave form.  Step t multiplies four quarters (64
// elements each) of its stage; it issues the codes of the step one ring ahead
// into the stage of step t - 1, which every wave finished reading before the
// last barrier, and ahead of them that step's scales; so a count of the loads
// issued since tells that all of step t + 1 has landed.  A quarter's fragments
// are read while the one before is multiplied, the first quarter's of step t +
// 1 after the barrier, while the last of step t is.
template <int CFG, int TAIL, int PAIR>
struct MidLoop {
    using G = Layout<CFG>;
    using Src = MidSrc<CFG, TAIL, PAIR>;
    static constexpr int R = G::STAGES, SR = scale_ring<CFG, TAIL>(), D = R - 1, SD = SR - 1;
    static constexpr int UNROLL = R % SR == 0 ? R : R * SR;
    static constexpr int BEHIND = SD == D ? (D - 1) * (Src::LC + Src::LS) : (D - 1) * Src::LC;
    static_assert(SD == D || (D == 2 && SD == 1), "the order of loads that BEHIND counts");
    Src src;
    Frags<CFG> FA, FB;
    uint32_t ra[2][G::TM], rb[2][G::TN], sa[G::TM], sb[G::TN];  // scale words: raw, shifted
    int pa[4], pb[4];  // this lane's offsets of A's and B's quarters in a stage
    int sh, wm, wn, l32, wave, ksteps, quarters;

    // Fragments of quarter kk of a stage: row lane % 32 of each 32-row group,
    // chunk 2 kk + lane / 32.
    __device__ __forceinline__ void read(const uint8_t* stage, int kk, Frags<CFG>& f) {
#pragma unroll
        for (int i = 0; i < G::TM; ++i) f.a[i] = *(const u32x4*)&stage[pa[kk] + i * 4096];
#pragma unroll
        for (int j = 0; j < G::TN; ++j) f.b[j] = *(const u32x4*)&stage[pb[kk] + j * 4096];
    }
    __device__ __forceinline__ void read_scales(const uint8_t* buf) {
        auto words = [&](int row, uint32_t& w0, uint32_t& w1) __attribute__((always_inline)) {
            if (TAIL) {
                const u32x4 d = *(const u32x4*)(buf + row * 16);
                w0 = (d.x & 0xFFFFu) | (d.y << 16);
                w1 = (d.z & 0xFFFFu) | (d.w << 16);
            } else {
                const u32x2 d = *(const u32x2*)(buf + row * 8);
                w0 = d.x;
                w1 = d.y;
            }
        };
#pragma unroll
        for (int i = 0; i < G::TM; ++i) words(wm * G::WROWS + i * 32 + l32, ra[0][i], ra[1][i]);
#pragma unroll
        for (int j = 0; j < G::TN; ++j)
            words(G::BM + wn * G::WCOLS + j * 32 + l32, rb[0][j], rb[1][j]);
    }
    // ALL: not the last step.
    template <int P, bool ALL>
    __device__ __forceinline__ void step(int t, v16f (&acc)[G::TM][G::TN]) {
        uint8_t* cur = mid_stage<CFG, TAIL, P>();
        const bool last = !ALL && t == ksteps - 1;
        __builtin_amdgcn_sched_barrier(0);
        shift_scales<CFG>(ra[0], rb[0], sh, sa, sb);
        read(cur, 1, FB);
        __builtin_amdgcn_sched_barrier(0);
        mfma_half<CFG, 0, 0>(FA, sa, sb, acc);
        __builtin_amdgcn_sched_barrier(0);
        read(cur, 2, FA);
        if (!last || quarters > 1) mfma_half<CFG, 0, 1>(FB, sa, sb, acc);
        __builtin_amdgcn_sched_barrier(0);
        read(cur, 3, FB);
        src.scales(mid_sbuf<CFG, TAIL, P + SD>(), wave, t + SD);
        src.codes(mid_stage<CFG, TAIL, P + D>(), wave, t + D + 1 < ksteps);
        shift_scales<CFG>(ra[1], rb[1], sh, sa, sb);
        if (!last || quarters > 2) mfma_half<CFG, 0, 0>(FA, sa, sb, acc);
        __builtin_amdgcn_sched_barrier(0);
        FP4Q_WAIT_VMCNT(BEHIND);
        __builtin_amdgcn_s_waitcnt(0xC07F);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        read_scales(mid_sbuf<CFG, TAIL, P + 1>());
        read(mid_stage<CFG, TAIL, P + 1>(), 0, FA);
        if (!last || quarters > 3) mfma_half<CFG, 0, 1>(FB, sa, sb, acc);
    }
    template <int P, bool ALL>
    __device__ __forceinline__ void turn(int kt, v16f (&acc)[G::TM][G::TN]) {
        // each step inside the one before's condition: where paths with and without
        // a step's loads met again, the compiler would wait for all of them
        if (!ALL && kt + P >= ksteps) return;
        step<P, ALL>(kt + P, acc);
        if constexpr (P + 1 < UNROLL) turn<P + 1, ALL>(kt, acc);
    }
    __device__ __forceinline__ void run(v16f (&acc)[G::TM][G::TN], const GatedCall& o, int m0, int n0,
                                        const LaneMap<CFG>& l) {
        src.init(o, m0, n0, l);
        wm = l.wm;
        wn = l.wn;
        l32 = l.l32;
        wave = l.wave;
        sh = 8 * l.half;
        ksteps = (o.K + 255) / 256;
        quarters = (o.K / 64 - 1) % 4 + 1;  // of the last step
        const int j = l32 & 7, reg = l32 >> 3;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int p = reg * REGION + j * 128 + (((2 * kk + l.half) ^ j ^ (reg & 1)) * 16);
            pa[kk] = p + wm * G::TM * 4096;
            pb[kk] = p + wn * G::TN * 4096 + G::OFF_B;
            // opaque: rewritten as a longer chain of additions from the stage, a
            // read would lose the compiler's note of which LDS object it is of,
            // and wait for all loads in flight
            asm volatile("" : "+v"(pa[kk]), "+v"(pb[kk]));
        }
        src.scales(mid_sbuf<CFG, TAIL, 0>(), wave, 0);
        src.codes(mid_stage<CFG, TAIL, 0>(), wave, 1 < ksteps);
        if constexpr (SD > 1) src.scales(mid_sbuf<CFG, TAIL, 1>(), wave, 1);
        src.codes(mid_stage<CFG, TAIL, 1>(), wave, 2 < ksteps);
        if constexpr (D > 2) {
            src.scales(mid_sbuf<CFG, TAIL, 2>(), wave, 2);
            src.codes(mid_stage<CFG, TAIL, 2>(), wave, 3 < ksteps);
        }
        FP4Q_WAIT_VMCNT(BEHIND);
        __builtin_amdgcn_s_barrier();
        read_scales(mid_sbuf<CFG, TAIL, 0>());
        read(mid_stage<CFG, TAIL, 0>(), 0, FA);
        int kt = 0;
        const int whole = quarters == 4 ? ksteps : ksteps - 1;
        for (; kt + UNROLL <= whole; kt += UNROLL) turn<0, true>(kt, acc);
        turn<0, false>(kt, acc);
        FP4Q_WAIT_VMCNT(0);  // the re-issued loads past the end of K have landed
    }
};

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
        MidLoop<CFG, TAIL, PAIR> loop;
        loop.run(acc, o, m0, n0, l);
    }
    __syncthreads();  // all waves are done with the operand stages
}

// This wave's private part of the operand stages, EREG bytes, free once the
// K loop's last barrier has passed.
template <int CFG, int TAIL, int EREG>
__device__ __forceinline__ uint8_t* wave_stage(int wave) {
    static_assert(EREG % 16 == 0 && 2 * EREG <= STAGE, "two to a stage");
    const int s = wave >> 1;
    uint8_t* st;
    if constexpr (CFG == 0)
        st = s == 0 ? st0 : s == 1 ? st1 : s == 2 ? st2 : st3;
    else
        st = s == 0 ? mid_stage<CFG, TAIL, 0>() : mid_stage<CFG, TAIL, 1>();
    return st + (wave & 1) * EREG;
}
// Of EREG bytes for each pair of waves: a stage each.
template <int CFG, int TAIL, int EREG>
__device__ __forceinline__ uint8_t* pair_stage(int pair) {
    static_assert(EREG % 16 == 0 && EREG <= STAGE, "a pair to a stage");
    if constexpr (CFG == 0)
        return pair == 0 ? st0 : pair == 1 ? st1 : pair == 2 ? st2 : st3;
    else
        return pair == 0 ? mid_stage<CFG, TAIL, 0>() : mid_stage<CFG, TAIL, 1>();
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

    // Two neighbouring waves hold 64 columns of every output, whole cache lines.
    // They meet in LDS, 32 rows at a time (in two regions in turn, so one barrier
    // is enough), and each stores 16 of the rows.
    constexpr int NOUT = SAVE ? 3 : 1;
    constexpr int PITCH = NOUT * 128 + 16;
    uint8_t* reg = pair_stage<CFG, TAIL, 2 * 32 * PITCH>(l.wave >> 1);
    const int row0 = m0 + l.wm * G::WROWS + (l.wn & 1) * 16 + (l.lane >> 3);
    const int col = n0 + (l.wn >> 1) * 64 + (l.lane & 7) * 8;
#pragma unroll
    for (int i = 0; i < G::TM; ++i) {
        uint8_t* buf = reg + (i & 1) * 32 * PITCH;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float hv[4];
            const v16f &ga = acc[i][0], &ua = acc[i][1];
#pragma unroll
            for (int r = 0; r < 4; ++r) hv[r] = act_value<GELU>(ga[4 * g + r]) * ua[4 * g + r];
            uint8_t* dst = buf + l.l32 * PITCH + ((l.wn & 1) * 32 + 8 * g + 4 * l.half) * 2;
            *(u32x2*)dst = (u32x2){pack_rne(hv[0], hv[1]), pack_rne(hv[2], hv[3])};
            if (SAVE) {
                *(u32x2*)(dst + 128) = (u32x2){pack_rne(ga[4 * g], ga[4 * g + 1]),
                                               pack_rne(ga[4 * g + 2], ga[4 * g + 3])};
                *(u32x2*)(dst + 256) = (u32x2){pack_rne(ua[4 * g], ua[4 * g + 1]),
                                               pack_rne(ua[4 * g + 2], ua[4 * g + 3])};
            }
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS writes done
        __builtin_amdgcn_s_barrier();        // (stores stay in flight)
#pragma unroll
        for (int out = 0; out < NOUT; ++out)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int rl = (l.wn & 1) * 16 + p * 8 + (l.lane >> 3);
                const u32x4 v = *(const u32x4*)(buf + rl * PITCH + out * 128 + (l.lane & 7) * 16);
                const int row = row0 + i * 32 + p * 8;
                if (row >= o.M) continue;
                uint16_t* base = out == 0 ? o.h : out == 1 ? o.gate : o.up;
                base += (int64_t)row * (out == 0 ? o.ldh : o.ldgu) + col;
                if (o.nt)
                    store8<1>(base, v, o.F - col);
                else
                    store8<0>(base, v, o.F - col);
            }
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
        for (int p = 0; p < PASSES; ++p) {  // past M, the last row again: no load is conditional
            const int64_t at = (int64_t)min(row0 + i * 32 + p * 8, o.M - 1) * o.ldgu;
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

    uint8_t* reg = wave_stage<CFG, TAIL, 32 * PITCH>(l.wave);
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
// the same time on an idle chip.  Forward, us (128-row, 256-row, 256 x 256):
//   M x F x K         512 x 1408 x 960    6.7   9.8  12.6
//                    2048 x 1408 x 960   13.3  10.8  13.3
//                    4096 x 1408 x 960   20.9  20.6  14.3
//                     128 x 13824 x 5120 25.8  31.0  43.6
//                     256 x 13824 x 5120 50.6  33.2  50.3
// and of the gradient:
//                    2048 x 1408 x 960   11.3  16.9  24.1
//                    1024 x 5632 x 2048  25.3  23.6  30.4
//                    2048 x 5632 x 2048  40.6  44.5  35.2
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
