// One AdamW step over many tensors, with the two moments in 32 bits or in 8.
//
//   g = grad * grad_scale
//   m' = b1 m + (1 - b1) g            v' = b2 v + (1 - b2) g^2
//   p' = p (1 - lr wd) - lr (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps)
//
// 8-bit moments: m and r = sqrt(v) as E4M3 values (4 exponent bits, 3
// mantissa bits, +-448) with one E8M0 scale byte per 32 consecutive elements
// of a tensor, 2^(byte-127) = 2^(floor(log2 amax) - 7), so that a block's
// largest magnitude lands in [128, 256) and rounds to at most 256: nothing
// saturates.  r and not v is stored because its exponents span half as much.
// Rounding is stochastic: an average that moves by 1 - b2 of itself per step
// moves by far less than half of E4M3's step (1/8 to 1/16), so rounding to
// nearest would leave it where it is, while the stochastic one moves it by
// the right amount on average.  The random bits are Philox4x32-10 with the
// seed as key, counter (position / 4, 0, step, 0), one 32-bit word per
// element: the low half rounds m, the high half r.  An element's position is
// its index plus the rounded-up-to-32 sizes of the tensors before it.
//
// The tensors' descriptors travel in the kernel arguments, kTensors to a
// launch, so a call copies nothing to the device and can be captured.
#include <cmath>

#include "../../include/libfp4q.h"
#include "fp4q_device.h"
#include "fp4q_internal.h"

// Products and sums below are rounded one by one, as written: the states are
// then the same whichever way the compiler arranges the code.
#pragma clang fp contract(off)

namespace fp4q {

constexpr int kTensors = 44;     // descriptors per launch: 4 KB of kernel arguments
constexpr int kChunk = 4096;     // elements per workgroup

struct AdamwArg {
    float* p;
    const void* g;
    void *m, *v;
    uint8_t *ms, *vs;
    uint16_t* copy;
    int64_t n;
    uint64_t base;   // position of element 0
    float decay;     // 1 - lr * weight decay
    uint32_t first;  // first workgroup
};
struct AdamwArgs {
    AdamwArg t[kTensors];
    const float* grad_scale;
    uint64_t seed;
    uint32_t step;
    int count;
    float b1, a1, b2, a2, lr, rc2, eps;  // a = 1 - b, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
};
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");

// Magnitude y (finite, below 256 + a step) to E4M3 with 16 random bits u: up
// iff u + floor(fraction 2^16) >= 2^16, the fraction taken of the step
// between E4M3 neighbours.
__device__ __forceinline__ float sr_e4m3(float y, uint32_t u) {
    if (y >= 0.015625f) return as_f32((as_u32(y) + (u << 4)) & ~0xFFFFFu);
    const float q = y * 512.0f, low = floorf(q);  // subnormals: multiples of 2^-9
    const float up = (uint32_t)((q - low) * 65536.0f) + u >= 65536u ? 1.0f : 0.0f;
    return (low + up) * 0.001953125f;
}

// The update of one element; v is v or (8-bit) r squared.
__device__ __forceinline__ float adamw_one(const AdamwArgs& a, float p, float g, float m, float v,
                                           float decay, float& m1, float& v1, float& r1) {
    m1 = a.b1 * m + a.a1 * g;
    v1 = a.b2 * v + a.a2 * g * g;
    r1 = sqrtf(v1);
    return p * decay - a.lr * m1 / (r1 * a.rc2 + a.eps);
}

template <int GB, int BITS>
__global__ __launch_bounds__(256) void adamw_kernel(const AdamwArgs a) {
    int t = 0;
    while (t + 1 < a.count && blockIdx.x >= a.t[t + 1].first) ++t;
    const AdamwArg d = a.t[t];
    const float gscale = a.grad_scale ? *a.grad_scale : 1.0f;
    const int64_t i0 = (int64_t)(blockIdx.x - d.first) * kChunk;
    for (int k = 0; k < kChunk / 1024; ++k) {
        const int64_t i = i0 + k * 1024 + threadIdx.x * 4;
        // a block of 32 is held by 8 lanes; its lanes past the end hold zeros
        float m1[4], r1[4];
        for (int e = 0; e < 4; ++e) {
            m1[e] = r1[e] = 0.0f;
            if (i + e >= d.n) continue;
            float g = GB ? as_f32((uint32_t)((const uint16_t*)d.g)[i + e] << 16)
                         : ((const float*)d.g)[i + e];
            g *= gscale;
            float m, v;
            if (BITS == 8) {
                const float sm = e8m0_scale_f32(d.ms[(i + e) >> 5]);
                const float sv = e8m0_scale_f32(d.vs[(i + e) >> 5]);
                m = __builtin_amdgcn_cvt_f32_fp8(((const uint8_t*)d.m)[i + e], 0) * sm;
                v = __builtin_amdgcn_cvt_f32_fp8(((const uint8_t*)d.v)[i + e], 0) * sv;
                v *= v;
            } else {
                m = ((const float*)d.m)[i + e];
                v = ((const float*)d.v)[i + e];
            }
            float v1;
            const float p = adamw_one(a, d.p[i + e], g, m, v, d.decay, m1[e], v1, r1[e]);
            d.p[i + e] = p;
            if (d.copy) d.copy[i + e] = (uint16_t)f32_to_bf16_bits(p);
            if (BITS == 32) {
                ((float*)d.m)[i + e] = m1[e];
                ((float*)d.v)[i + e] = v1;
            }
        }
        if (BITS == 8) {
            uint32_t mm = 0, mr = 0;
            for (int e = 0; e < 4; ++e) {
                mm = max(mm, as_u32(m1[e]) & 0x7FFFFFFFu);
                mr = max(mr, as_u32(r1[e]) & 0x7FFFFFFFu);
            }
            mm = group_max_u32<8>(mm);
            mr = group_max_u32<8>(mr);
            const bool badm = mm >= 0x7F800000u, badr = mr >= 0x7F800000u;
            const uint32_t bm = badm ? 0xFFu : (uint32_t)max((int)(mm >> 23) - 7, 0);
            const uint32_t br = badr ? 0xFFu : (uint32_t)max((int)(mr >> 23) - 7, 0);
            const float im = e8m0_inv_scale_f32(badm ? 0u : bm);
            const float ir = e8m0_inv_scale_f32(badr ? 0u : br);
            const uint64_t n = (d.base + i) >> 2;
            const Philox4 w = philox4x32_10((uint32_t)n, (uint32_t)(n >> 32), a.step, 0u,
                                            (uint32_t)a.seed, (uint32_t)(a.seed >> 32));
            for (int e = 0; e < 4; ++e) {
                if (i + e >= d.n) continue;
                const float qm = copysignf(sr_e4m3(fabsf(m1[e]) * im, w.v[e] & 0xFFFFu), m1[e]);
                const float qr = sr_e4m3(r1[e] * ir, w.v[e] >> 16);
                const uint32_t c = __builtin_amdgcn_cvt_pk_fp8_f32(qm, qr, 0, false);
                ((uint8_t*)d.m)[i + e] = badm ? 0 : (uint8_t)c;
                ((uint8_t*)d.v)[i + e] = badr ? 0 : (uint8_t)(c >> 8);
            }
            if ((threadIdx.x & 7) == 0 && i < d.n) {
                d.ms[i >> 5] = (uint8_t)bm;
                d.vs[i >> 5] = (uint8_t)br;
            }
        }
    }
}

hipError_t launch_adamw(const fp4q_adamw_tensor_t* t, int n, int bits, int gdtype, double lr,
                        double beta1, double beta2, double eps, int64_t step, uint64_t seed,
                        const float* grad_scale, hipStream_t s) {
    AdamwArgs a;
    a.grad_scale = grad_scale;
    a.seed = seed;
    a.step = (uint32_t)step;
    a.b1 = (float)beta1;
    a.a1 = (float)(1.0 - beta1);
    a.b2 = (float)beta2;
    a.a2 = (float)(1.0 - beta2);
    a.lr = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
    a.rc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
    a.eps = (float)eps;
    uint64_t base = 0;
    for (int i = 0; i < n;) {
        uint64_t groups = 0;
        a.count = 0;
        for (; i < n && a.count < kTensors; ++i) {
            const uint64_t need = (uint64_t)((t[i].numel + kChunk - 1) / kChunk);
            if (t[i].numel == 0) continue;
            if (groups + need > 0x7FFFFFFFu) break;
            AdamwArg& d = a.t[a.count++];
            d.p = t[i].param;
            d.g = t[i].grad;
            d.m = t[i].exp_avg;
            d.v = t[i].exp_avg_sq;
            d.ms = t[i].exp_avg_scales;
            d.vs = t[i].exp_avg_sq_scales;
            d.copy = t[i].copy;
            d.n = t[i].numel;
            d.base = base;
            d.decay = (float)(1.0 - lr * (double)t[i].weight_decay);
            d.first = (uint32_t)groups;
            groups += need;
            base += (uint64_t)((t[i].numel + 31) / 32) * 32;
        }
        if (a.count == 0) break;
        const dim3 grid((unsigned)groups);
        if (bits == 8) {
            if (gdtype == BF16)
                FP4Q_LAUNCH((adamw_kernel<1, 8>), grid, dim3(256), 0, s, a);
            else
                FP4Q_LAUNCH((adamw_kernel<0, 8>), grid, dim3(256), 0, s, a);
        } else {
            if (gdtype == BF16)
                FP4Q_LAUNCH((adamw_kernel<1, 32>), grid, dim3(256), 0, s, a);
            else
                FP4Q_LAUNCH((adamw_kernel<0, 32>), grid, dim3(256), 0, s, a);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace fp4q
