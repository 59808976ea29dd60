// The operand pipeline of the scaled-FP4 GEMMs: tile layouts, the direct-to-LDS
// load ring and the K loop that the kernels of gemm_fp4.hip (plain, DGE,
// quantising, hot-channel) and gated.hip (gated feed-forward) share.  The
// design is described at the head of gemm_fp4.hip.
#pragma once
#include <type_traits>

#include "fp4q_device.h"
#include "fp4q_internal.h"

namespace fp4q {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

static constexpr int BKB = 64;                  // operand bytes per row per K step
static constexpr int REGION = 1024;             // 16 rows x 64 bytes
static constexpr int STAGE = 32 * REGION;       // one K step of A and B codes
static constexpr int SROW = 32;                 // LDS bytes per scale row per group
static constexpr int SCALE_BUF = 512 * SROW;    // A rows, then B rows
// K steps per scale group: 8 (32 scale bytes per row) when every scale row
// starts on a 4-byte boundary (K % 128 == 0); 4 when K % 128 == 64, where the
// rows are only 2-byte aligned and are fetched with 2-byte loads, each of
// which fills a whole LDS dword (low half data, high half zero), so a group
// of 16 data bytes still takes 32 bytes of LDS per row.
template <int TAIL> struct Groups {
    static constexpr int SG = TAIL ? 4 : 8;
    static constexpr int SGB = 4 * SG;          // scale bytes per row per group in memory
};
static constexpr int GROUP_M = 4;
static constexpr int BUF_FLAGS = 0x00020000;    // buffer resource word 3: raw 32-bit data

// s_waitcnt with only the vector-memory counter constrained (gfx9 encoding:
// vmcnt in bits 3:0 and 15:14; expcnt 6:4 and lgkmcnt 11:8 at maximum).
#define FP4Q_WAIT_VMCNT(n) __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (((n) >> 4) << 14) | 0x0F70)

// Tile configurations: eight waves, two along M and four along N, each
// owning TM x TN MFMA tiles of 32 x 32.
//   CFG 0: 256 x 256 tile, 128 x 64 per wave (4 x 2 MFMA tiles);
//   CFG 1: 128 x 384 tile,  64 x 96 per wave (2 x 3 MFMA tiles), for shapes
//          whose 256 x 256 tiles would leave part of the chip idle in the
//          last round (three of its tiles cover the area of four of those).
// Both stage 512 operand rows (32 KB) per K step and 512 scale rows.
template <int CFG>
struct Layout {
    static constexpr int WAVES = 8, THREADS = 64 * WAVES;
    static constexpr int WM = 2, WN = 4;
    static constexpr int TM = CFG == 0 ? 4 : 2;  // 32-row MFMA tiles per wave
    static constexpr int TN = CFG == 0 ? 2 : 3;  // 32-column MFMA tiles per wave
    static constexpr int WROWS = 32 * TM, WCOLS = 32 * TN;
    static constexpr int BM = WM * WROWS, BN = WN * WCOLS;
    static constexpr int RA = BM / 16, RB = BN / 16;  // 1 KB code regions per step
    static constexpr int RPW_A = RA / WAVES, RPW_B = RB / WAVES;
    static constexpr int RPW = RPW_A > RPW_B ? RPW_A : RPW_B;
    static constexpr int OFF_B = RA * REGION;         // B codes within a stage
    static constexpr int SROWS = 512 / WAVES;         // scale rows fetched per wave
    static constexpr int SPIECES = SROWS / 8;         // 8-row scale pieces per wave per group
    static constexpr int A_SWAVES = BM / SROWS;       // waves fetching A scale rows
    static_assert(RA % WAVES == 0 && RB % WAVES == 0, "code regions divide among the waves");
    static_assert((RA + RB) * REGION == STAGE, "one 32 KB stage per K step");
    static_assert(BM + BN == WAVES * SROWS, "the waves fetch all scale rows");
    static_assert(SPIECES % 4 == 0, "scale pieces spread over four steps");
};

// 16-byte slot of chunk c (bytes 16c .. 16c+15 of the step) of row j within
// a 16-row region.
__device__ __forceinline__ int region_slot(int j, int c) { return 4 * j + (c ^ ((j >> 2) & 3)); }

// Load sources: buffer resources whose ranges end at the operand's last row
// inside this tile (rows past M or N read as zero), 32-bit per-lane offsets
// (they alone decide whether a row is in range), and the scalar byte offset
// of the current K step.
//
// GATED (256 x 256 tiles): B's 32-row groups alternate between two operands
// of the same size, so group 2w holds 32 rows of the first (the gate
// projection) and group 2w + 1 the same rows of the second (the up
// projection): wave column w then accumulates both products of the same 32
// output columns.  A wave's code regions all belong to one of the two (the
// group's parity is that of wave / 2), so only the row offsets differ from
// A's; its scale pieces 0..3 are of the first operand, 4..7 of the second.
template <int CFG, int GATED = 0>
struct Src {
    __amdgpu_buffer_rsrc_t ra, rb, rsc;  // rsc: scales of this wave's pieces (A or B)
    __amdgpu_buffer_rsrc_t rsc2;         // GATED: of its pieces 4..7
    uint32_t vrow[Layout<CFG>::RPW];     // region q of A and of B share the row offsets
    uint32_t vrow_b[Layout<CFG>::RPW];   // GATED: B's row offsets
    uint32_t vsc[4];  // scale piece offsets, by piece index % 4 (word swizzle)
    int srow;         // GATED: rows per scale piece index past the third (32, or 0 for B)
    int soff;
};

// Direct-to-LDS loads of the K step the sources point at into `stage`; the
// sources then advance to the next step if `advance` (past the end of K the
// last step is re-issued into a stage nobody reads again, so every step
// issues the same number of loads and the waits are compile-time).
template <int CFG, int BF16OPS, int GATED = 0>
__device__ __forceinline__ void issue_codes(Src<CFG, GATED>& src, uint8_t* stage, int wave,
                                            bool advance) {
    using L = Layout<CFG>;
#pragma unroll
    for (int q = 0; q < L::RPW; ++q) {
        const int rho = q * L::WAVES + wave;
        if (q < L::RPW_A)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(src.ra, (lds_ptr_t)(stage + rho * REGION), 16,
                                                     src.vrow[q], src.soff, 0, 0);
        if (q < L::RPW_B)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                src.rb, (lds_ptr_t)(stage + L::OFF_B + rho * REGION), 16,
                GATED ? src.vrow_b[q] : src.vrow[q], src.soff, 0, 0);
    }
    src.soff += advance ? BKB : 0;
}

// Scale piece P (0 .. SPIECES-1) of this wave for group g: combined rows
// wave*SROWS + P*8 .. +7 (A rows 0..BM-1, then B rows), 32 LDS bytes each.
// Whole words (TAIL = 0): lane 8j + pos loads word pos ^ (P % 4) of the
// piece's row j, so that in LDS word s of row R sits at R*32 + 4 (s ^ ((R / 8)
// % 4)) (SROWS / 8 is a multiple of 4).  Half words (TAIL = 1): lane 8j + pos
// loads half (pos % 2) of word (pos / 2) ^ (P % 4) into LDS dword pos of row
// j, so that word s of row R is the low halves of the dwords at R*32 +
// 8 (s ^ ((R / 8) % 4)) and the next one.  The group offset is part of the
// per-lane offset so the range check covers it.
template <int CFG, int P, int TAIL, int GATED = 0>
__device__ __forceinline__ void issue_scale_piece(const Src<CFG, GATED>& src, uint8_t* sbuf,
                                                  int wave, int kscale, int g) {
    // the uniform part as one scalar, so that the compiler does not keep a
    // hoisted per-piece vector offset live across the K loop
    const int row = GATED ? (P & 3) * 8 + (P > 3 ? src.srow : 0) : P * 8;
    uint32_t soff = (uint32_t)(row * kscale + g * Groups<TAIL>::SGB);
    asm volatile("" : "+s"(soff));
    const uint32_t voff = src.vsc[P & 3] + soff;
    lds_ptr_t dst = (lds_ptr_t)(sbuf + (wave * Layout<CFG>::SROWS + P * 8) * SROW);
    const __amdgpu_buffer_rsrc_t& rsc = GATED && P > 3 ? src.rsc2 : src.rsc;
    if constexpr (TAIL)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsc, dst, 2, voff, 0, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsc, dst, 4, voff, 0, 0, 0);
}

// Pieces P0 .. P0+N-1.
template <int CFG, int P0, int N, int TAIL, int GATED = 0>
__device__ __forceinline__ void issue_scale_pieces(const Src<CFG, GATED>& src, uint8_t* sbuf,
                                                   int wave, int kscale, int g) {
    if constexpr (N > 0) {
        issue_scale_piece<CFG, P0, TAIL, GATED>(src, sbuf, wave, kscale, g);
        issue_scale_pieces<CFG, P0 + 1, N - 1, TAIL, GATED>(src, sbuf, wave, kscale, g);
    }
}

template <int CFG>
struct Frags {
    u32x4 a[Layout<CFG>::TM], b[Layout<CFG>::TN];
};

// This wave's A and B fragments of one half of a staged step; `off` is this
// lane's offset within a 32-row group for that half (row lane % 32, chunk
// 2 kk + lane / 32).
template <int CFG>
__device__ __forceinline__ void read_frags(const uint8_t* base, int off, int wm, int wn,
                                           Frags<CFG>& F) {
    using L = Layout<CFG>;
#pragma unroll
    for (int i = 0; i < L::TM; ++i)
        F.a[i] = *(const u32x4*)(base + (wm * L::TM + i) * 2 * REGION + off);
#pragma unroll
    for (int j = 0; j < L::TN; ++j)
        F.b[j] = *(const u32x4*)(base + L::OFF_B + (wn * L::TN + j) * 2 * REGION + off);
}

// Scale words (4 K blocks of 32 elements each) of step word s of a group
// for this lane's MFMA rows (A) and columns (B); `sx` is this lane's
// swizzled byte offset of that word: 4 (s ^ ((lane % 32) / 8 % 4)) for whole
// words, 8 (s ^ ...) for the half-word layout (TAIL), whose two dwords carry
// the word's low and high halves.
template <int CFG, int TAIL>
__device__ __forceinline__ uint32_t scale_word(const uint8_t* p) {
    if constexpr (TAIL) {
        const uint2 d = *(const uint2*)p;
        return (d.x & 0xFFFFu) | (d.y << 16);
    } else {
        return *(const uint32_t*)p;
    }
}

template <int CFG, int TAIL>
__device__ __forceinline__ void read_scales(const uint8_t* sbuf, int sx, int wm, int wn, int lane,
                                            uint32_t (&sa)[Layout<CFG>::TM],
                                            uint32_t (&sb)[Layout<CFG>::TN]) {
    using L = Layout<CFG>;
    const int l32 = lane & 31;
#pragma unroll
    for (int i = 0; i < L::TM; ++i)
        sa[i] = scale_word<CFG, TAIL>(sbuf + (wm * L::WROWS + i * 32 + l32) * SROW + sx);
#pragma unroll
    for (int j = 0; j < L::TN; ++j)
        sb[j] = scale_word<CFG, TAIL>(sbuf + (L::BM + wn * L::WCOLS + j * 32 + l32) * SROW + sx);
}

// Shifts raw scale words so that byte 2 kk is the K block of half kk for
// this lane's 32-element K chunk (lanes 32..63 take the odd blocks).
template <int CFG>
__device__ __forceinline__ void shift_scales(const uint32_t (&ra)[Layout<CFG>::TM],
                                             const uint32_t (&rb)[Layout<CFG>::TN], int sh,
                                             uint32_t (&sa)[Layout<CFG>::TM],
                                             uint32_t (&sb)[Layout<CFG>::TN]) {
#pragma unroll
    for (int i = 0; i < Layout<CFG>::TM; ++i) sa[i] = ra[i] >> sh;
#pragma unroll
    for (int j = 0; j < Layout<CFG>::TN; ++j) sb[j] = rb[j] >> sh;
}

// The TM x TN MFMAs of this wave on half KK of a K step.  FP4: the scaled
// MFMA on E2M1 operands (64 K elements per half), its byte select picking
// byte 2 KK of the lane's (pre-shifted) scale words; BF16: plain bf16 MFMAs
// (16 K elements per half, the same 16 bytes per lane).  B is the MFMA's
// first operand, so each accumulator holds the transposed tile: register r
// of lane l is C[row l % 32][column 8 (r / 4) + 4 (l / 32) + r % 4], four
// consecutive columns per register group, which the epilogue stores whole.
template <int CFG, int BF16OPS, int KK>
__device__ __forceinline__ void mfma_half(const Frags<CFG>& F, const uint32_t (&sa)[Layout<CFG>::TM],
                                          const uint32_t (&sb)[Layout<CFG>::TN],
                                          v16f (&acc)[Layout<CFG>::TM][Layout<CFG>::TN]) {
    using L = Layout<CFG>;
    if (BF16OPS) {
#pragma unroll
        for (int i = 0; i < L::TM; ++i)
#pragma unroll
            for (int j = 0; j < L::TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    __builtin_bit_cast(bf16x8_t, F.b[j]), __builtin_bit_cast(bf16x8_t, F.a[i]),
                    acc[i][j], 0, 0, 0);
        return;
    }
#pragma unroll
    for (int i = 0; i < L::TM; ++i) {
        const v8i fa = (v8i){(int)F.a[i].x, (int)F.a[i].y, (int)F.a[i].z, (int)F.a[i].w, 0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < L::TN; ++j) {
            const v8i fb =
                (v8i){(int)F.b[j].x, (int)F.b[j].y, (int)F.b[j].z, (int)F.b[j].w, 0, 0, 0, 0};
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                fb, fa, acc[i][j], 4, 4, 2 * KK, (int)sb[j], 2 * KK, (int)sa[i]);
        }
    }
}

// The LDS ring stages and scale buffers: separate objects, so the compiler
// sees that loads in flight into one stage and reads of another do not
// alias; the epilogue reuses the stages.
__shared__ __attribute__((aligned(16))) uint8_t st0[STAGE];
__shared__ __attribute__((aligned(16))) uint8_t st1[STAGE];
__shared__ __attribute__((aligned(16))) uint8_t st2[STAGE];
__shared__ __attribute__((aligned(16))) uint8_t st3[STAGE];
__shared__ __attribute__((aligned(16))) uint8_t sc0[SCALE_BUF];
__shared__ __attribute__((aligned(16))) uint8_t sc1[SCALE_BUF];

// One K loop of the workgroup's tile over operands ac / bc (K-major rows, K
// elements deep; FP4 with scales as, bs, or bf16 without), accumulating into
// acc.  Leaves no loads in flight; the caller synchronises before the stages
// are reused.  TAIL (FP4 only, K % 128 == 64): the last K step holds one half
// (its second half's MFMAs are skipped; what its loads fetch past the row is
// never used) and the scale rows, only 2-byte aligned, go through the
// half-word layout in groups of 4 steps.  GATED: bc, bs are the first and
// bc2, bs2 the second of B's two operands (see Src), n0 and N count rows of
// one of them (128 of each per tile).
template <int CFG, int BF16OPS, int TAIL, int GATED = 0>
__device__ __forceinline__ void gemm_kloop(v16f (&acc)[Layout<CFG>::TM][Layout<CFG>::TN],
                                           const uint8_t* __restrict__ ac,
                                           const uint8_t* __restrict__ as,
                                           const uint8_t* __restrict__ bc,
                                           const uint8_t* __restrict__ bs, int K, int M, int N,
                                           int m0, int n0, int wave, int lane, int wm, int wn,
                                           int half, int l32, int off0, int off1, int sxor,
                                           const uint8_t* __restrict__ bc2 = nullptr,
                                           const uint8_t* __restrict__ bs2 = nullptr) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass cannot instantiate buffer resources
    using L = Layout<CFG>;
    constexpr int TM = L::TM, TN = L::TN;
    static_assert(!(TAIL && BF16OPS), "bf16 K loops are whole steps");
    constexpr int SG = Groups<TAIL>::SG;
    // bytes per operand row (< 2^23, checked by the caller); each K step
    // consumes 64 of them (the last one 32 with TAIL)
    const int kbytes = BF16OPS ? K * 2 : K / 2;
    const int kscale = K / 32;
    const int ksteps = (kbytes + BKB - 1) / BKB;

    static_assert(!GATED || (CFG == 0 && !BF16OPS), "gated tiles are FP4, 256 x 256");
    Src<CFG, GATED> src;
    {
        const int rows_a = min(M - m0, L::BM), rows_b = min(N - n0, GATED ? L::BN / 2 : L::BN);
        if (GATED && ((wave >> 1) & 1)) bc = bc2;
        src.ra = __builtin_amdgcn_make_buffer_rsrc((void*)(ac + (int64_t)m0 * kbytes), (short)0,
                                                   rows_a * kbytes, BUF_FLAGS);
        src.rb = __builtin_amdgcn_make_buffer_rsrc((void*)(bc + (int64_t)n0 * kbytes), (short)0,
                                                   rows_b * kbytes, BUF_FLAGS);
        // lane 4j + p of a region loads chunk p ^ ((j / 4) % 4) of row j
        const int j = lane >> 2;
        const int c = (lane & 3) ^ ((j >> 2) & 3);
#pragma unroll
        for (int q = 0; q < L::RPW; ++q)
            src.vrow[q] = (uint32_t)(((q * L::WAVES + wave) * 16 + j) * kbytes + c * 16);
        if (GATED) {
#pragma unroll
            for (int q = 0; q < L::RPW; ++q)
                src.vrow_b[q] = (uint32_t)((q * 64 + (wave >> 2) * 32 + (wave & 1) * 16 + j) *
                                               kbytes + c * 16);
        }
        // waves 0 .. A_SWAVES-1 fetch A scale rows, the others B
        constexpr int HW = L::A_SWAVES;
        src.rsc = wave < HW ? __builtin_amdgcn_make_buffer_rsrc((void*)(as + (int64_t)m0 * kscale),
                                                                (short)0, rows_a * kscale, BUF_FLAGS)
                            : __builtin_amdgcn_make_buffer_rsrc((void*)(bs + (int64_t)n0 * kscale),
                                                                (short)0, rows_b * kscale, BUF_FLAGS);
        int sbase = ((wave < HW ? wave : wave - HW) * L::SROWS + (lane >> 3)) * kscale;
        if (GATED) {
            src.rsc2 = wave < HW ? src.rsc
                                 : __builtin_amdgcn_make_buffer_rsrc(
                                       (void*)(bs2 + (int64_t)n0 * kscale), (short)0,
                                       rows_b * kscale, BUF_FLAGS);
            src.srow = wave < HW ? 32 : 0;
            if (wave >= HW) sbase = ((wave - HW) * 32 + (lane >> 3)) * kscale;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            src.vsc[q] = TAIL ? (uint32_t)(sbase + ((((lane & 7) >> 1) ^ q) << 2) + ((lane & 1) << 1))
                              : (uint32_t)(sbase + (((lane & 7) ^ q) << 2));
        src.soff = 0;
    }
    Frags<CFG> FA, FB;
    // sa/sb: shifted scale words of the step being computed; ra/rb: raw
    // words of the next step, read after the barrier that publishes it.
    uint32_t sa[TM], ra[TM], sb[TN], rb[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = ra[i] = 0;
#pragma unroll
    for (int j = 0; j < TN; ++j) sb[j] = rb[j] = 0;
    const int sh = 8 * half;

    // Software pipeline over K steps t with a 4-stage code ring: step t
    // issues the code loads of step t + 3 into the stage step t - 1 used
    // (every wave finished reading it before the previous barrier), and, in
    // the first half of each 8-step scale group, two scale pieces of the next
    // group into the other scale buffer (its previous group ended before);
    // with TAIL's 4-step groups, all eight pieces in the group's first step
    // (so that they have landed by the wait at the end of its last step).  Each
    // step computes two halves (K bytes 0..31 and 32..63 of the step); order
    // within a step, fenced against the compiler's scheduler:
    //   1. shift the step's scale words; read the fragments of (t, 1); issue
    //      loads;
    //   2. MFMAs of (t, 0), whose fragments were read during step t - 1;
    //   3. wait for this wave's loads of step t + 1 (later loads stay in
    //      flight) and its LDS reads, then one workgroup barrier;
    //   4. read the scales and (t + 1, 0) fragments; MFMAs of (t, 1).
    // The loop is unrolled by 16 steps (two or four scale groups, four turns
    // of the ring), so every load count, wait and LDS buffer is a
    // compile-time constant.
    constexpr int LC = L::RPW_A + L::RPW_B;  // code loads per wave per step
    // loads issued after the code loads of step t + 1, at the end of step t
    // with t % 8 == p: those of steps t - 1 and t plus the scale pieces
    // issued after the code loads in step t - 2
#define FP4Q_PIECES(p)                                                              \
    (BF16OPS ? 0 : TAIL ? ((((p) & 3) == 0) ? L::SPIECES : 0)                          \
                        : ((((p) & 7) >= 4) ? 0 : L::SPIECES / 4))
#define FP4Q_BEHIND(p) (FP4Q_PIECES((p) + 6) + LC + FP4Q_PIECES((p) + 7) + LC + FP4Q_PIECES(p))
    if (!BF16OPS) issue_scale_pieces<CFG, 0, L::SPIECES, TAIL, GATED>(src, sc0, wave, kscale, 0);
    issue_codes<CFG, BF16OPS, GATED>(src, st0, wave, 1 < ksteps);
    issue_codes<CFG, BF16OPS, GATED>(src, st1, wave, 2 < ksteps);
    issue_codes<CFG, BF16OPS, GATED>(src, st2, wave, 3 < ksteps);
    FP4Q_WAIT_VMCNT(2 * LC);
    __builtin_amdgcn_s_barrier();
    if (!BF16OPS) read_scales<CFG, TAIL>(sc0, TAIL ? sxor << 3 : sxor << 2, wm, wn, lane, ra, rb);
    read_frags<CFG>(st0, off0, wm, wn, FA);

// One K step t = kt + P (P = t % 16, compile-time; its position in its
// scale group is P % SG).  The scale buffer of step P's group and of the
// next group alternate with the group's parity.  The final step's reads of
// a next step are harmless (in-bounds, unused), so no step is special, except
// that with TAIL the last step's second half has no data.
#define FP4Q_SCUR(P) ((((P) / SG) & 1) ? sc1 : sc0)
#define FP4Q_SNXT(P) ((((P) / SG) & 1) ? sc0 : sc1)
#define FP4Q_GEMM_STEP(P, CUR, NEXT1, NEXTL)                                         \
    do {                                                                             \
        const int t_ = kt + (P);                                                     \
        __builtin_amdgcn_sched_barrier(0);                                           \
        if (!BF16OPS) shift_scales<CFG>(ra, rb, sh, sa, sb);                          \
        read_frags<CFG>(CUR, off1, wm, wn, FB);                                       \
        issue_codes<CFG, BF16OPS, GATED>(src, NEXTL, wave, t_ + 4 < ksteps);          \
        if (FP4Q_PIECES(P))                                                          \
            issue_scale_pieces<CFG, TAIL ? 0 : ((P) & 3) * (L::SPIECES / 4),             \
                               FP4Q_PIECES(P), TAIL, GATED>(src, FP4Q_SNXT(P), wave, kscale, \
                                                     t_ / SG + 1);                       \
        __builtin_amdgcn_sched_barrier(0);                                           \
        mfma_half<CFG, BF16OPS, 0>(FA, sa, sb, acc);                                  \
        __builtin_amdgcn_sched_barrier(0);                                           \
        FP4Q_WAIT_VMCNT(FP4Q_BEHIND(P));                                             \
        __builtin_amdgcn_s_waitcnt(0xC07F);                                          \
        __builtin_amdgcn_s_barrier();                                                \
        __builtin_amdgcn_sched_barrier(0);                                           \
        if (!BF16OPS)                                                                \
            read_scales<CFG, TAIL>(((P) % SG) == SG - 1 ? FP4Q_SNXT(P) : FP4Q_SCUR(P),       \
                                   TAIL ? (((P) + 1) & 3 ^ sxor) << 3                       \
                                        : (((P) + 1) & 7 ^ sxor) << 2,                      \
                                   wm, wn, lane, ra, rb);                                \
        read_frags<CFG>(NEXT1, off0, wm, wn, FA);                                     \
        if (!TAIL || t_ != ksteps - 1) mfma_half<CFG, BF16OPS, 1>(FB, sa, sb, acc);   \
    } while (0)

// Eight steps starting at t = kt + O (two turns of the code ring); GUARD(P)
// says whether step kt + P exists (compile-time true in full turns).
#define FP4Q_GEMM_GROUP(O, GUARD)                                                    \
    do {                                                                             \
        if (GUARD(O + 0)) FP4Q_GEMM_STEP(O + 0, st0, st1, st3);                       \
        if (GUARD(O + 1)) FP4Q_GEMM_STEP(O + 1, st1, st2, st0);                       \
        if (GUARD(O + 2)) FP4Q_GEMM_STEP(O + 2, st2, st3, st1);                       \
        if (GUARD(O + 3)) FP4Q_GEMM_STEP(O + 3, st3, st0, st2);                       \
        if (GUARD(O + 4)) FP4Q_GEMM_STEP(O + 4, st0, st1, st3);                       \
        if (GUARD(O + 5)) FP4Q_GEMM_STEP(O + 5, st1, st2, st0);                       \
        if (GUARD(O + 6)) FP4Q_GEMM_STEP(O + 6, st2, st3, st1);                       \
        if (GUARD(O + 7)) FP4Q_GEMM_STEP(O + 7, st3, st0, st2);                       \
    } while (0)
#define FP4Q_ALL(P) true
#define FP4Q_EXISTS(P) (kt + (P) < ksteps)

    // Step t uses code stage t % 4 and scale buffer (t / SG) % 2; a turn of
    // the loop covers 16 steps so every buffer is named at compile time (the
    // compiler then sees that scale reads and the loads in flight touch
    // different LDS objects).
    int kt = 0;
    for (; kt + 16 <= ksteps; kt += 16) {
        FP4Q_GEMM_GROUP(0, FP4Q_ALL);
        FP4Q_GEMM_GROUP(8, FP4Q_ALL);
    }
    if (kt < ksteps) {
        FP4Q_GEMM_GROUP(0, FP4Q_EXISTS);
        FP4Q_GEMM_GROUP(8, FP4Q_EXISTS);
    }
#undef FP4Q_GEMM_GROUP
#undef FP4Q_GEMM_STEP
#undef FP4Q_SCUR
#undef FP4Q_SNXT
#undef FP4Q_ALL
#undef FP4Q_EXISTS
#undef FP4Q_PIECES
#undef FP4Q_BEHIND
    FP4Q_WAIT_VMCNT(0);  // the re-issued loads past the end of K have landed
#endif
}

// Origin of tile number t of 256 x 256 tiles: XCD-contiguous, then grouped
// along M.
__device__ __forceinline__ void tile_origin(int t, int ntiles, int tiles_m, int tiles_n, int& m0,
                                            int& n0) {
    using L = Layout<0>;
    int wg = t;
    const int full = (ntiles / 8) * 8;
    if (wg < full) wg = (wg % 8) * (full / 8) + wg / 8;
    const int per_group = GROUP_M * tiles_n;
    const int grp = wg / per_group;
    const int first_m = grp * GROUP_M;
    const int gsize = min(GROUP_M, tiles_m - first_m);
    const int in_grp = wg - grp * per_group;
    m0 = (first_m + in_grp % gsize) * L::BM;
    n0 = (in_grp / gsize) * L::BN;
}

// Compute units of the current device (cached per device).
inline int device_cus() {
    static int cache[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (cache[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
            n <= 0)
            n = 256;
        cache[dev] = n;
    }
    return cache[dev];
}

}  // namespace fp4q
