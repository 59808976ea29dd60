// The gated feed-forward projections and their gradient where even the smaller
// tiles of gated.hip would leave most of the chip idle: few rows, or narrow
// blocks.
//
// A workgroup owns a small tile of outputs, 16 MT rows by 16 NT columns, and
// its KS waves split K: each wave multiplies the whole tile over its part of
// K, straight from memory into registers (an operand fragment is 16 rows x 64
// bytes, 16 bytes per lane; no wave shares operands with another, so LDS would
// only add a copy and a barrier), with the loads of the next steps in flight.
// The partial tiles then meet in LDS, where the sum, the activation and the
// rounding are done 8 columns per lane.  What bounds it at one token is the
// weights' way from memory, so every compute unit takes part of it, and K is
// split until each wave has only a few loads to wait for; the gradient's gate
// and up are fetched before K is walked.
//
// Rows past M and weight rows past F are read as the last one (their outputs
// are not written).  K % 128 == 64: in the last step the lanes of its missing
// half read the other half again, with A's codes and both scales set to zero.
#include "gated_act.h"
#include "fp4q_internal.h"

namespace fp4q {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// One 128-element K step of the tile's operands in this lane: row lane % 16
// of each fragment, elements 32 (lane / 16) .. + 31, and their scale.
template <int MT, int NB>
struct SmallStep {
    u32x4 a[MT], b[NB];
    uint32_t sa[MT], sb[NB];
};

template <int GELU, int GRAD, int SAVE, int MT, int NT, int KS>
__global__ __launch_bounds__(64 * KS) void gated_small_kernel(const GatedCall g,
                                                              int tiles_m) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int NB = GRAD ? NT : 2 * NT;       // B fragments: gate's, then up's
    constexpr int ROWS = 16 * MT, COLS = 16 * NT;
    constexpr int PITCH = 16 * NB + 4;
    constexpr int DEPTH = MT + NB <= 4 ? 4 : 2;  // steps in flight
    __shared__ __attribute__((aligned(16))) float part[KS][ROWS][PITCH];
    // workgroups of one XCD take neighbouring tiles, rows fastest: they share
    // the weights in its L2
    int tile = blockIdx.x;
    const int full = (int)(gridDim.x / 8) * 8;
    if (tile < full) tile = (tile % 8) * (full / 8) + tile / 8;
    const int m0 = tile % tiles_m * ROWS, n0 = tile / tiles_m * COLS;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, q = lane >> 4;
    const uint32_t kbytes = (uint32_t)g.K / 2, kscale = (uint32_t)g.K / 32;

    // 8 columns of a row per lane in the epilogue
    constexpr int GROUPS = ROWS * 2 * NT, PER = (GROUPS + 64 * KS - 1) / (64 * KS);
    u32x4 gin[GRAD ? PER : 1], uin[GRAD ? PER : 1];
    if (GRAD) {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int i = p * 64 * KS + threadIdx.x;
            const int row = m0 + i / (2 * NT), col = n0 + i % (2 * NT) * 8;
            if (i < GROUPS && row < g.M && col < g.F) {
                const uint16_t *gr = g.gate + row * g.ldgu, *ur = g.up + row * g.ldgu;
                gin[p] = g.F >= 8 ? load8(gr, col, g.F) : load_short(gr, col, g.F);
                uin[p] = g.F >= 8 ? load8(ur, col, g.F) : load_short(ur, col, g.F);
            }
        }
    }

    uint32_t arow[MT], brow[NT];  // row of each fragment within the tile
#pragma unroll
    for (int i = 0; i < MT; ++i) arow[i] = (uint32_t)min(i * 16 + l16, g.M - 1 - m0);
#pragma unroll
    for (int j = 0; j < NT; ++j) brow[j] = (uint32_t)min(j * 16 + l16, g.F - 1 - n0);
    const uint8_t* ac = g.ac + (int64_t)m0 * kbytes;
    const uint8_t* as = g.as + (int64_t)m0 * kscale;
    const uint8_t* bc[2] = {g.bc + (int64_t)n0 * kbytes, g.bc2 + (int64_t)n0 * kbytes};
    const uint8_t* bs[2] = {g.bs + (int64_t)n0 * kscale, g.bs2 + (int64_t)n0 * kscale};

    const int steps = (g.K + 127) / 128, each = (steps + KS - 1) / KS;
    const int s0 = wave * each, s1 = min(s0 + each, steps);
    auto load = [&](SmallStep<MT, NB>& t, int s) __attribute__((always_inline)) {
        const bool half = (s + 1) * 128 > g.K;  // the last step of K % 128 == 64
        const uint32_t qq = half ? q & 1 : q;
        const uint32_t oc = s * 64 + qq * 16, os = s * 4 + qq;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            t.a[i] = *(const u32x4*)(ac + (arow[i] * kbytes + oc));
            t.sa[i] = as[arow[i] * kscale + os];
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int o = j / NT;
            t.b[j] = *(const u32x4*)(bc[o] + (brow[j % NT] * kbytes + oc));
            t.sb[j] = bs[o][brow[j % NT] * kscale + os];
        }
    };
    v4f acc[MT][NB];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](SmallStep<MT, NB>& t, int s) __attribute__((always_inline)) {
        if ((s + 1) * 128 > g.K && q > 1) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                t.a[i] = (u32x4){0u, 0u, 0u, 0u};
                t.sa[i] = 0;
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) t.sb[j] = 0;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const v8i fa = {(int)t.a[i].x, (int)t.a[i].y, (int)t.a[i].z, (int)t.a[i].w, 0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const v8i fb = {(int)t.b[j].x, (int)t.b[j].y, (int)t.b[j].z, (int)t.b[j].w, 0, 0, 0, 0};
                // B first: register r of a lane is row lane % 16, column 4 (lane / 16) + r
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    fb, fa, acc[i][j], 4, 4, 0, (int)t.sb[j], 0, (int)t.sa[i]);
            }
        }
    };
    SmallStep<MT, NB> st[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (s0 + d < s1) load(st[d], s0 + d);
    for (int s = s0; s < s1; s += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (s + d < s1) {
                multiply(st[d], s + d);
                if (s + d + DEPTH < s1) load(st[d], s + d + DEPTH);
            }
        }
    }

#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *(v4f*)&part[wave][i * 16 + l16][j * 16 + q * 4] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int i = p * 64 * KS + threadIdx.x;
        const int r = i / (2 * NT), c = i % (2 * NT) * 8;
        const int row = m0 + r, col = n0 + c, n = g.F - col;
        if (i >= GROUPS || row >= g.M || n <= 0) continue;
        float v[2][8] = {};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int o = 0; o < (GRAD ? 1 : 2); ++o)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const v4f x = *(const v4f*)&part[k][r][o * COLS + c + 4 * h];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[o][4 * h + e] += x[e];
                }
        if (GRAD) {
            u32x4 dg, du;
            gated_grad8<GELU>(v[0], settle8(gin[p], col, g.F), settle8(uin[p], col, g.F), dg,
                              du);
            store8<0>(g.dgate + row * g.ldd + col, dg, n);
            store8<0>(g.dup + row * g.ldd + col, du, n);
        } else {
            u32x4 hv, gv, uv;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hv[e] = pack_rne(act_value<GELU>(v[0][2 * e]) * v[1][2 * e],
                                 act_value<GELU>(v[0][2 * e + 1]) * v[1][2 * e + 1]);
                gv[e] = pack_rne(v[0][2 * e], v[0][2 * e + 1]);
                uv[e] = pack_rne(v[1][2 * e], v[1][2 * e + 1]);
            }
            store8<0>(g.h + row * g.ldh + col, hv, n);
            if (SAVE) {
                store8<0>(g.gate + row * g.ldgu + col, gv, n);
                store8<0>(g.up + row * g.ldgu + col, uv, n);
            }
        }
    }
#endif
}

template <int GELU, int GRAD, int SAVE, int MT, int NT, int KS>
static void go(const GatedCall& g, hipStream_t s) {
    const int tiles_m = (g.M + 16 * MT - 1) / (16 * MT), tiles_n = (g.F + 16 * NT - 1) / (16 * NT);
    FP4Q_LAUNCH((gated_small_kernel<GELU, GRAD, SAVE, MT, NT, KS>), dim3((unsigned)(tiles_m * tiles_n)),
                dim3(64 * KS), 0, s, g, tiles_m);
}

// The smallest tiles first: each is taken while its workgroups are one round of
// the 256 compute units, where it takes about 2.5 us and 1.4 ns an element of K
// (32 rows: 1.9 ns, 32 x 32: 2.9 ns; gradient 1.4, 1.9 and 2.9), against 4 us and
// 2.2 ns (gradient 6 and 2.6) of the LDS tiles of gated.hip.  Around the limits,
// us, small tiles in the order below and LDS tiles (groups of the first):
//   forward   M x F x K    64 x 704 x 5120   (176)   9.6, 11.9, 16.1; 14.6
//                         128 x 704 x 5120   (352)  16.3, 12.1, 16.2; 15.7
//                          64 x 1408 x 960   (352)   4.2,  4.7,  4.2;  6.1
//                         128 x 1408 x 960   (704)   5.0,  5.9,  4.2;  6.1
//                         256 x 704 x 2048   (704)  10.9, 10.8,  8.4;  8.2
//                           1 x 6660 x 4032  (417)   9.7, 10.4, 10.4; 14.4
//                          16 x 5632 x 2048  (352)   8.6,  8.9,  7.8;  7.8
//   gradient              128 x 704 x 5120   (176)   9.8, 12.0, 16.8; 18.2
//                         128 x 1408 x 4096  (352)  14.0, 10.6, 14.4; 16.9
//                         256 x 1408 x 4096  (704)  19.7, 18.0, 14.9; 17.0
//                         512 x 1408 x 960  (1408)   9.1,  6.4,  6.1;  9.5
//                         512 x 1408 x 2048 (1408)  20.8, 14.7, 14.8; 12.1
// Up to 16 rows a second round is taken too, since what larger tiles would share
// are rows of A: 5632 x 2048 (352 groups) with 1, 4, 8 and 16 rows 7.1, 7.5, 7.8
// and 8.5 us, 32 x 32 tiles 7.3, 7.5, 7.7 and 7.9, LDS tiles 7.8 to 8.0; so at 16
// rows the rule gives away 0.5 us there, and at 6660 x 4032 (417) 0.6 of 14.4.  At
// short K a second round is taken too, where the LDS tiles' start counts for more.
// The gradient's 32 x 64 tiles past one round: where groups and K together stay
// below what 352 groups take at K = 1024 (512 x 1408: 6.0 us against 9.2 of the LDS
// tiles at K = 960, 8.8 and 9.1 at 1024; at 1088, past the limit, 6.6 and 9.8, but
// 2000 x 2000 x 192, as much in more groups, 14.8 and 11.3).
bool launch_gated_small(const GatedCall& g, bool grad, int gelu, hipStream_t s) {
    auto groups = [&](int64_t bm, int64_t bn) { return (g.M + bm - 1) / bm * ((g.F + bn - 1) / bn); };
    const int64_t K = g.K;
#define FP4Q_GO(GRAD, SAVE, MT, NT, KS) \
    (gelu ? go<1, GRAD, SAVE, MT, NT, KS>(g, s) : go<0, GRAD, SAVE, MT, NT, KS>(g, s))
    if (grad) {
        if (groups(16, 32) <= 256) return FP4Q_GO(1, 0, 1, 2, 8), true;
        if (groups(32, 32) <= 256) return FP4Q_GO(1, 0, 2, 2, 4), true;
        // (rows below 8 elements are this form's alone)
        if (groups(32, 64) <= 256 || groups(32, 64) * K <= 365000 || g.F < 8)
            return FP4Q_GO(1, 0, 2, 4, 4), true;
        return false;
    }
    if (groups(16, 16) <= 256 || (groups(16, 16) <= 512 && (g.M <= 16 || K <= 1024)))
        return g.gate ? FP4Q_GO(0, 1, 1, 1, 4) : FP4Q_GO(0, 0, 1, 1, 4), true;
    if (groups(32, 16) <= 256)
        return g.gate ? FP4Q_GO(0, 1, 2, 1, 8) : FP4Q_GO(0, 0, 2, 1, 8), true;
    if (groups(32, 32) <= 256 && K <= 1536)
        return g.gate ? FP4Q_GO(0, 1, 2, 2, 4) : FP4Q_GO(0, 0, 2, 2, 4), true;
#undef FP4Q_GO
    return false;
}

}  // namespace fp4q
