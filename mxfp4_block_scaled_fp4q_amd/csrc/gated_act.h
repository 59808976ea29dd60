// The activation of the gated feed-forward kernels, and their row accesses.
#pragma once
#include "fp4q_device.h"

namespace fp4q {

// The activation a(g) = g s(z(g)), s(z) = 1 / (1 + exp(-z)): z = g (SiLU) or
// 2 sqrt(2 / pi) (g + 0.044715 g^3) (GELU = 1, the tanh form).
//
// s is 2^-24 / (2^-24 + e) with e = exp2(-z log2(e) - 24): the reciprocal then
// stays in the normal range (its subnormal results would be flushed) down to
// s = 2^-150, and the last product rounds into the subnormals; no case has to
// be told from another.  The shift costs accuracy near z = 0: the exponent's
// sum has 2^-20 for a half step, so s is off by up to 11 half steps of fp32
// there, and by about 4 |z| far out.  Formed in the fewest operations: where
// 256 x 256 outputs of a compute unit meet their activation, these decide how
// long it takes (exp2 and reciprocal count four each).
constexpr float kLog2e = 1.44269504f, kGeluA = 1.59576912f, kGeluB = 0.044715f;
template <int GELU>
__device__ __forceinline__ float act_sigma(float g) {
    const float w =
        GELU ? __builtin_fmaf(kGeluA * kGeluB * kLog2e, g * g, kGeluA * kLog2e) : kLog2e;
    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(-g, w, -24.0f));
    return __builtin_amdgcn_rcpf(e + 0x1p-24f) * 0x1p-24f;
}
template <int GELU>
__device__ __forceinline__ float act_value(float g) {
    return g * act_sigma<GELU>(g);
}

__device__ __forceinline__ uint32_t pack_rne(float lo, float hi) {
    const bf16x2_t p = {(__bf16)lo, (__bf16)hi};  // v_cvt_pk_bf16_f32
    return __builtin_bit_cast(uint32_t, p);
}

// A call of the gated kernels: A with M rows, B with F rows, K-major, and in the
// forward pass B2, the up projection; what they write and, in the gradient,
// read (gate and up).
struct GatedCall {
    int M, F, K;
    const uint8_t *ac, *as, *bc, *bs, *bc2, *bs2;
    uint16_t* h;                 // forward
    int64_t ldh;
    uint16_t *gate, *up;         // forward: written (or null); gradient: read
    int64_t ldgu;
    uint16_t *dgate, *dup;       // gradient
    int64_t ldd;
    int nt;                      // outputs are stored non-temporally
};

// Launches the small-tile form (gated_small.hip) and says so, where it is the
// one to take.
bool launch_gated_small(const GatedCall& g, bool grad, int gelu, hipStream_t s);

template <int NT>
__device__ __forceinline__ void put16(uint16_t* p, u32x4 v) {
    if (NT)
        __builtin_nontemporal_store(v, (u32x4_a2*)p);
    else
        *(u32x4_a2*)p = v;
}

// 8 bf16 at p, of which the row still holds n.
template <int NT>
__device__ __forceinline__ void store8(uint16_t* p, u32x4 v, int n) {
    typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
    typedef uint32_t u32_a2 __attribute__((aligned(2)));
    if (n >= 8) {
        put16<NT>(p, v);
    } else if (n > 0) {
        uint32_t w = v.x;
        if (n & 4) {
            *(u32x2_a2*)p = (u32x2){v.x, v.y};
            w = v.z;
        }
        uint16_t* q = p + (n & 4);
        if (n & 2) *(u32_a2*)q = w;
        if (n & 1) q[n & 2] = (uint16_t)((n & 2) ? ((n & 4) ? v.w : v.y) : w);
    }
}
// Elements col .. col + 7 of a row of F >= 8, in two steps, so that no lane waits
// for its data where it loads them: the row's last ones come from F - 8 and are
// shifted into place at their use.  They are read once: non-temporal (gradient
// 4096 x 5632 x 2048 68 us, 81 without).
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int col, int F) {
    return __builtin_nontemporal_load((const u32x4_a2*)(row + min(col, F - 8)));
}
// The same of a shorter row, one by one and in place.
__device__ __forceinline__ u32x4 load_short(const uint16_t* row, int col, int F) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col + e < F) w[e >> 1] |= (uint32_t)row[col + e] << (16 * (e & 1));
    return (u32x4){w[0], w[1], w[2], w[3]};
}
__device__ __forceinline__ u32x4 settle8(u32x4 v, int col, int F) {
    const int n = F - col;
    if (n >= 8 || n <= 0 || F < 8) return v;
    uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
    const int s = 16 * (8 - n);
    if (s >= 64) {
        lo = hi >> (s - 64);
        hi = 0;
    } else {
        lo = lo >> s | hi << (64 - s);
        hi >>= s;
    }
    return (u32x4){(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Of 8 elements with gradients d, gate g and up u (bf16 pairs), the gradients
// of gate and up: a'(g) = s + g s (1 - s) z'(g).  g^2 is held below 1e30 so
// that z' stays finite where s (1 - s) is zero.
template <int GELU>
__device__ __forceinline__ void gated_grad8(const float (&d)[8], u32x4 g, u32x4 u, u32x4& dg,
                                            u32x4& du) {
    float og[8], ou[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float gv = (e & 1) ? bf16_hi(g[e >> 1]) : bf16_lo(g[e >> 1]);
        const float uv = (e & 1) ? bf16_hi(u[e >> 1]) : bf16_lo(u[e >> 1]);
        const float s = act_sigma<GELU>(gv), a = gv * s;
        float rest = 1.0f - s;
        if (GELU) rest *= __builtin_fmaf(3.0f * kGeluA * kGeluB, fminf(gv * gv, 1e30f), kGeluA);
        og[e] = d[e] * uv * __builtin_fmaf(a, rest, s);
        ou[e] = d[e] * a;
    }
    dg = (u32x4){pack_rne(og[0], og[1]), pack_rne(og[2], og[3]), pack_rne(og[4], og[5]),
                 pack_rne(og[6], og[7])};
    du = (u32x4){pack_rne(ou[0], ou[1]), pack_rne(ou[2], ou[3]), pack_rne(ou[4], ou[5]),
                 pack_rne(ou[6], ou[7])};
}

}  // namespace fp4q
