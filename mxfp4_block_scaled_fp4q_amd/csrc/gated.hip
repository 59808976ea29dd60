// The gated feed-forward projections on the scaled-FP4 GEMM pipeline.
//
//   forward   G = X Wg^T, U = X Wu^T, H = a(G) * U       a(g) = g s(z(g))
//   gradient  D = dY W^T, dU = D * a(G), dG = D * U * a'(G)
//
// with s(z) = 1 / (1 + exp(-z)), z(g) = g for SiLU and z(g) = 2 sqrt(2 / pi)
// (g + 0.044715 g^3) for the tanh form of GELU (0.5 (1 + tanh(z / 2)) = s(z)),
// and a'(g) = s + g s (1 - s) z'(g).
//
// Forward: one 256 x 256 tile of the product holds 128 columns of G and the
// same 128 columns of U, interleaved in groups of 32 so that each wave's two
// 32-column accumulator tiles are G and U of the same outputs (Src in
// gemm_core.h).  The activation then needs no exchange between lanes: H is
// formed from the fp32 accumulators and only rounded results are written,
// instead of writing G and U, reading them back and writing H.
// Gradient: the plain tile, with the derivative applied to the fp32 tile in
// the epilogue; G and U are read ahead of their use there, so D is never
// written.
#include "gemm_core.h"

namespace fp4q {

// z = c0 g + c1 g^3: c0 = 1, c1 = 0 (SiLU) or the tanh GELU's pair; t0, t1 are
// those times log2(e), so that the exponent is rounded three times only.  With
// e = exp(-|z|), s is 1 / (1 + e) or, below zero, e / (1 + e), and 1 - s the
// other of the two: neither cancels, and s keeps its relative error (that of
// e, 4 |z| half steps, and the hardware exp2's and reciprocal's ulp) down to
// the subnormals.  exp2's results below 2^-126 would be flushed, so far
// arguments are shifted by 64 and the result scaled back.  g^2 is held below
// 1e30 so that c1 = 0 never meets an infinity, and so that z' stays finite
// where s (1 - s) is zero.
struct Act {
    float c0, c1, t0, t1;
};
struct Sigma {
    float s, c, g2;  // s, 1 - s, g^2
};
__device__ __forceinline__ Sigma act_sigma(float g, Act a) {
    Sigma o;
    o.g2 = fminf(g * g, 1e30f);
    const float z = g * (a.t0 + a.t1 * o.g2);
    const float t = -fabsf(z);
    const bool far = t < -64.0f;
    const float e = __builtin_amdgcn_exp2f(far ? t + 64.0f : t) * (far ? 0x1p-64f : 1.0f);
    const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
    o.s = z < 0.0f ? er : r;
    o.c = z < 0.0f ? r : er;
    return o;
}
__device__ __forceinline__ float act_value(float g, Act a) { return g * act_sigma(g, a).s; }

__device__ __forceinline__ uint32_t pack_rne(float lo, float hi) {
    const bf16x2_t p = {(__bf16)lo, (__bf16)hi};  // v_cvt_pk_bf16_f32
    return __builtin_bit_cast(uint32_t, p);
}

// 8 bf16 of a row at p: one 16-byte access where `vec`, else the first n of
// them one by one (n may be below 1).
__device__ __forceinline__ void store8(uint16_t* p, u32x4 v, bool vec, int n) {
    if (vec && n >= 8) {
        __builtin_nontemporal_store(v, (u32x4*)p);
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
}
__device__ __forceinline__ u32x4 load8(const uint16_t* p, bool vec, int n) {
    if (vec && n >= 8) return __builtin_nontemporal_load((const u32x4*)p);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    return (u32x4){w[0], w[1], w[2], w[3]};
}

struct LaneMap {
    int lane, wave, wm, wn, half, l32, off0, off1, sxor;
};
__device__ __forceinline__ LaneMap lane_map() {
    using L = Layout<0>;
    LaneMap m;
    m.lane = threadIdx.x & 63;
    m.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    m.wm = m.wave / L::WN;
    m.wn = m.wave % L::WN;
    m.half = m.lane >> 5;
    m.l32 = m.lane & 31;
    m.off0 = (m.l32 >> 4) * REGION + region_slot(m.l32 & 15, m.half) * 16;
    m.off1 = (m.l32 >> 4) * REGION + region_slot(m.l32 & 15, 2 + m.half) * 16;
    m.sxor = (m.l32 >> 3) & 3;
    return m;
}

// This wave's private part of the operand stages, EREG bytes, free once the
// K loop's last barrier has passed.
template <int EREG>
__device__ __forceinline__ uint8_t* wave_stage(int wave) {
    constexpr int PER = STAGE / EREG;
    static_assert(PER * 4 >= Layout<0>::WAVES, "epilogue regions fit in the four stages");
    uint8_t* st = wave / PER == 0 ? st0 : wave / PER == 1 ? st1 : wave / PER == 2 ? st2 : st3;
    return st + (wave % PER) * EREG;
}

// SAVE: G and U are written too (bf16, for the gradient).
template <int SAVE, int TAIL>
__global__ __launch_bounds__(512, 1) void gemm_gated_kernel(
    int M, int F, int K, const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
    const uint8_t* __restrict__ gc, const uint8_t* __restrict__ gs,
    const uint8_t* __restrict__ uc, const uint8_t* __restrict__ us, Act act,
    uint16_t* __restrict__ h, int64_t ldh, uint16_t* __restrict__ gate,
    uint16_t* __restrict__ up, int64_t ldgu, int vec, int tiles_m, int tiles_n) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass cannot instantiate buffer resources
    using L = Layout<0>;
    int m0, n0;
    tile_origin(blockIdx.x, gridDim.x, tiles_m, tiles_n, m0, n0);
    n0 >>= 1;  // 128 output columns per tile
    const LaneMap lm = lane_map();
    v16f acc[L::TM][L::TN];
#pragma unroll
    for (int i = 0; i < L::TM; ++i)
#pragma unroll
        for (int j = 0; j < L::TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    gemm_kloop<0, 0, TAIL, 1>(acc, xc, xs, gc, gs, K, M, F, m0, n0, lm.wave, lm.lane, lm.wm, lm.wn,
                              lm.half, lm.l32, lm.off0, lm.off1, lm.sxor, uc, us);
    __syncthreads();  // all waves are done with the operand stages

    constexpr int NOUT = SAVE ? 3 : 1;
    constexpr int PITCH = NOUT * 64 + 16;  // 32 bf16 of each output per row
    uint8_t* reg = wave_stage<32 * PITCH>(lm.wave);
    const int row0 = m0 + lm.wm * L::WROWS;
    const int col = n0 + lm.wn * 32 + (lm.lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < L::TM; ++i) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float hv[4];
            const v16f &ga = acc[i][0], &ua = acc[i][1];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                hv[r] = act_value(ga[4 * g + r], act) * ua[4 * g + r];
            uint8_t* dst = reg + lm.l32 * PITCH + (8 * g + 4 * lm.half) * 2;
            *(uint2*)dst = make_uint2(pack_rne(hv[0], hv[1]), pack_rne(hv[2], hv[3]));
            if (SAVE) {
                *(uint2*)(dst + 64) = make_uint2(pack_rne(ga[4 * g], ga[4 * g + 1]),
                                                 pack_rne(ga[4 * g + 2], ga[4 * g + 3]));
                *(uint2*)(dst + 128) = make_uint2(pack_rne(ua[4 * g], ua[4 * g + 1]),
                                                  pack_rne(ua[4 * g + 2], ua[4 * g + 3]));
            }
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's LDS writes done
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int o = 0; o < NOUT; ++o)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int rl = p * 16 + (lm.lane >> 2);
                const u32x4 v = *(const u32x4*)(reg + rl * PITCH + o * 64 + (lm.lane & 3) * 16);
                const int row = row0 + i * 32 + rl;
                if (row >= M) continue;
                uint16_t* base = o == 0 ? h : o == 1 ? gate : up;
                store8(base + (int64_t)row * (o == 0 ? ldh : ldgu) + col, v, vec, F - col);
            }
        __builtin_amdgcn_wave_barrier();
    }
#endif
}

template <int TAIL>
__global__ __launch_bounds__(512, 1) void gemm_gated_grad_kernel(
    int M, int F, int K, const uint8_t* __restrict__ yc, const uint8_t* __restrict__ ys,
    const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws, Act act,
    const uint16_t* __restrict__ gate, const uint16_t* __restrict__ up, int64_t ldgu,
    uint16_t* __restrict__ dgate, uint16_t* __restrict__ dup, int64_t ldd, int vec, int tiles_m,
    int tiles_n) {
#if defined(__HIP_DEVICE_COMPILE__)
    using L = Layout<0>;
    int m0, n0;
    tile_origin(blockIdx.x, gridDim.x, tiles_m, tiles_n, m0, n0);
    const LaneMap lm = lane_map();
    v16f acc[L::TM][L::TN];
#pragma unroll
    for (int i = 0; i < L::TM; ++i)
#pragma unroll
        for (int j = 0; j < L::TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    gemm_kloop<0, 0, TAIL>(acc, yc, ys, wc, ws, K, M, F, m0, n0, lm.wave, lm.lane, lm.wm, lm.wn,
                           lm.half, lm.l32, lm.off0, lm.off1, lm.sxor);
    __syncthreads();

    // 32 rows of 64 fp32 per wave at a time; a lane then owns 8 consecutive
    // columns of 4 rows.  G and U of the first two 32-row groups are read
    // before any is used, those of the others two groups ahead.
    constexpr int PITCH = 64 * 4 + 16, PASSES = 4;
    uint8_t* reg = wave_stage<32 * PITCH>(lm.wave);
    const int row0 = m0 + lm.wm * L::WROWS + (lm.lane >> 3);
    const int cl = (lm.lane & 7) * 8;
    const int col = n0 + lm.wn * L::WCOLS + cl;
    struct Pair {
        u32x4 g[PASSES], u[PASSES];
    };
    auto fetch = [&](int i, Pair& q) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int row = row0 + i * 32 + p * 8;
            q.g[p] = q.u[p] = (u32x4){0u, 0u, 0u, 0u};
            if (row < M) {
                q.g[p] = load8(gate + (int64_t)row * ldgu + col, vec, F - col);
                q.u[p] = load8(up + (int64_t)row * ldgu + col, vec, F - col);
            }
        }
    };
    auto group = [&](const int i, const Pair& in) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < L::TN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const v16f& a = acc[i][j];
                *(u32x4*)(reg + lm.l32 * PITCH + (j * 32 + 8 * g + 4 * lm.half) * 4) =
                    (u32x4){as_u32(a[4 * g]), as_u32(a[4 * g + 1]), as_u32(a[4 * g + 2]),
                            as_u32(a[4 * g + 3])};
            }
        __builtin_amdgcn_s_waitcnt(0xC07F);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const uint8_t* src = reg + (p * 8 + (lm.lane >> 3)) * PITCH + cl * 4;
            const u32x4 d0 = *(const u32x4*)src, d1 = *(const u32x4*)(src + 16);
            const uint32_t d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
            const uint32_t gw[4] = {in.g[p].x, in.g[p].y, in.g[p].z, in.g[p].w};
            const uint32_t uw[4] = {in.u[p].x, in.u[p].y, in.u[p].z, in.u[p].w};
            float og[8], ou[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gv = (e & 1) ? bf16_hi(gw[e >> 1]) : bf16_lo(gw[e >> 1]);
                const float uv = (e & 1) ? bf16_hi(uw[e >> 1]) : bf16_lo(uw[e >> 1]);
                const Sigma q = act_sigma(gv, act);
                const float slope = q.s + gv * (q.s * q.c) * (act.c0 + 3.0f * act.c1 * q.g2);
                const float dv = as_f32(d[e]);
                og[e] = dv * uv * slope;
                ou[e] = dv * (gv * q.s);
            }
            const int row = row0 + i * 32 + p * 8;
            if (row >= M) continue;
            const int64_t off = (int64_t)row * ldd + col;
            store8(dgate + off, (u32x4){pack_rne(og[0], og[1]), pack_rne(og[2], og[3]),
                                        pack_rne(og[4], og[5]), pack_rne(og[6], og[7])},
                   vec, F - col);
            store8(dup + off, (u32x4){pack_rne(ou[0], ou[1]), pack_rne(ou[2], ou[3]),
                                      pack_rne(ou[4], ou[5]), pack_rne(ou[6], ou[7])},
                   vec, F - col);
        }
        __builtin_amdgcn_wave_barrier();
    };
    Pair qa, qb;
    fetch(0, qa);
    fetch(1, qb);
    group(0, qa);
    fetch(2, qa);
    group(1, qb);
    fetch(3, qb);
    group(2, qa);
    group(3, qb);
#endif
}

static Act make_act(int act) {
    constexpr double kLog2e = 1.4426950408889634;
    const double c0 = act == 0 ? 1.0 : 1.5957691216057308;  // 2 sqrt(2 / pi)
    const double c1 = act == 0 ? 0.0 : c0 * 0.044715;
    return Act{(float)c0, (float)c1, (float)(c0 * kLog2e), (float)(c1 * kLog2e)};
}
static bool vec16(const void* p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && ld % 8 == 0; }

hipError_t launch_gemm_gated(int64_t M, int64_t F, int64_t K, const uint8_t* xc,
                             const uint8_t* xs, const uint8_t* gc, const uint8_t* gs,
                             const uint8_t* uc, const uint8_t* us, int act, uint16_t* h,
                             int64_t ldh, uint16_t* gate, uint16_t* up, int64_t ldgu,
                             hipStream_t s) {
    const int tiles_m = (int)((M + 255) / 256), tiles_n = (int)((F + 127) / 128);
    const dim3 grid((unsigned)(tiles_m * tiles_n));
    const Act a = make_act(act);
    const int vec = vec16(h, ldh) && (!gate || (vec16(gate, ldgu) && vec16(up, ldgu)));
#define FP4Q_GO(SAVE, TAIL)                                                                   \
    FP4Q_LAUNCH((gemm_gated_kernel<SAVE, TAIL>), grid, dim3(512), 0, s, (int)M, (int)F, (int)K, \
                xc, xs, gc, gs, uc, us, a, h, ldh, gate, up, ldgu, vec, tiles_m, tiles_n)
    if (gate) {
        if (K % 128) FP4Q_GO(1, 1); else FP4Q_GO(1, 0);
    } else {
        if (K % 128) FP4Q_GO(0, 1); else FP4Q_GO(0, 0);
    }
#undef FP4Q_GO
    return hipGetLastError();
}

hipError_t launch_gemm_gated_grad(int64_t M, int64_t F, int64_t K, const uint8_t* yc,
                                  const uint8_t* ys, const uint8_t* wc, const uint8_t* ws,
                                  int act, const uint16_t* gate, const uint16_t* up,
                                  int64_t ldgu, uint16_t* dgate, uint16_t* dup, int64_t ldd,
                                  hipStream_t s) {
    const int tiles_m = (int)((M + 255) / 256), tiles_n = (int)((F + 255) / 256);
    const dim3 grid((unsigned)(tiles_m * tiles_n));
    const Act a = make_act(act);
    const int vec = vec16(gate, ldgu) && vec16(up, ldgu) && vec16(dgate, ldd) && vec16(dup, ldd);
    if (K % 128)
        FP4Q_LAUNCH((gemm_gated_grad_kernel<1>), grid, dim3(512), 0, s, (int)M, (int)F, (int)K, yc,
                    ys, wc, ws, a, gate, up, ldgu, dgate, dup, ldd, vec, tiles_m, tiles_n);
    else
        FP4Q_LAUNCH((gemm_gated_grad_kernel<0>), grid, dim3(512), 0, s, (int)M, (int)F, (int)K, yc,
                    ys, wc, ws, a, gate, up, ldgu, dgate, dup, ldd, vec, tiles_m, tiles_n);
    return hipGetLastError();
}

}  // namespace fp4q
