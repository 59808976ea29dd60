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
// seed as key, counter (low and high word of position / 4, step, 0), one
// 32-bit word per element: the low half rounds m, the high half r.  An element's position is
// its index plus the rounded-up-to-32 sizes of the tensors before it.
//
// Bound by memory: param, gradient and moments are read once and written once
// (30 bytes an element with 32-bit moments, fp32 gradients and the bf16 copy,
// 14 with 8-bit moments and bf16 gradients and no copy).  A workgroup owns a
// chunk of 4096 elements of one tensor; a whole chunk's loads are issued ahead
// of its arithmetic, 16 bytes per lane (8-bit moments: 8 bytes of codes, for 8
// elements per lane, so that 4 lanes hold a block of 32).  A tensor's last
// chunk takes its last elements, fewer than a vector, one by one.  173M
// elements with 32-bit moments and the copy 937 us (5.5 TB/s), 212M with 8-bit
// ones 531 us (5.7): loads and stores are non-temporal (neither so 965 and 539
// us, the loads alone 954 and 550, the stores alone 979 and 538); chunks of
// 8192 elements 980 and 557 us.
//
// Up to kTensors descriptors travel in the kernel arguments, so that such a
// call copies nothing to the device.  More come in a table in device memory
// that the caller has made and copied there once (adamw_table), with the
// tensor of every chunk, so that any number of tensors is one launch.
#include <cmath>
#include <cstring>

#include "../../include/libfp4q.h"
#include "fp4q_device.h"
#include "fp4q_internal.h"

// Products and sums below are rounded one by one, as written: the states are
// then the same whichever way the compiler arranges the code.
#pragma clang fp contract(off)

namespace fp4q {

// Pointers that come from memory are generic to the compiler, and generic
// accesses wait on the LDS counter too: global<T>(p) is p in global memory.
template <class T>
using Global = T __attribute__((address_space(1))) *;
template <class T>
__device__ __forceinline__ Global<T> global(const void* p) {
    return (Global<T>)p;
}

constexpr int kTensors = 44;     // descriptors per launch: 4 KB of kernel arguments
constexpr int kChunk = 4096;     // elements per workgroup
// Threads of a workgroup.  With 8-bit moments a lane has one set of 8 elements
// (of 16 with 256 threads): its random numbers and roundings are a long chain,
// which is all that a few small tensors wait for (4191 elements 6.7 and 5.2 us).
constexpr int group_threads(int bits) { return bits == 8 ? 512 : 256; }
constexpr int kMaxGroups = 1 << 22;  // workgroups per launch: 2^31 threads

struct AdamwArg {
    float* p;
    const void* g;
    void *m, *v;
    uint8_t *ms, *vs;
    uint16_t* copy;
    int64_t n;
    uint64_t base;   // position of element 0
    double decay;    // weight decay
    uint32_t first;  // first workgroup
    uint32_t unused;
};
struct AdamwScalars {
    const float* grad_scale;
    uint64_t seed;
    double lr_wd;                        // lr, of the decay
    uint32_t step;
    float b1, a1, b2, a2, lr, rc2, eps;  // a = 1 - b, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
};
struct AdamwArgs {
    AdamwArg t[kTensors];
    AdamwScalars h;
    int count;
};
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");

// E4M3 code of the magnitude y (finite, below 256 + a step) rounded with 16
// random bits u: up iff u + floor(fraction 2^16) >= 2^16, the fraction taken
// of the step between E4M3 neighbours.  Codes count the values in order, so a
// carry out of the mantissa is the next code.
__device__ __forceinline__ uint32_t sr_e4m3(float y, uint32_t u) {
    const uint32_t normal = ((as_u32(y) + (u << 4)) >> 20) - (120u << 3);
    const uint32_t sub = ((uint32_t)(y * 33554432.0f) + u) >> 16;  // multiples of 2^-9
    return y >= 0.015625f ? normal : sub;
}

// The update of one element with 32-bit moments.
__device__ __forceinline__ float adamw_one(const AdamwScalars& a, float p, float g, float m, float v,
                                           float decay, float& m1, float& v1) {
    m1 = a.b1 * m + a.a1 * g;
    v1 = a.b2 * v + a.a2 * g * g;
    return p * decay - a.lr * m1 / (sqrtf(v1) * a.rc2 + a.eps);
}

// Roots of 8 values that are not negative (or NaN), rounded to nearest: a root
// that is a unit off lets a stochastic rounding now and then take the other
// code, and where r is small the next step moves the parameter by that much.
// y ~ 1/sqrt(x) is within a unit, s = x y within two, so that x - s^2 is exact
// in an fma and one Newton step s + (x - s^2) y / 2 is off by 2^-45 of s before
// its rounding.  Values outside [2^-96, infinity), where a step of that could
// leave the normal numbers, take sqrtf; one test for the wave's 8 x 64.
__device__ __forceinline__ void roots8(const float (&x)[8], float (&r)[8]) {
    uint32_t lo = as_u32(x[0]), hi = lo;
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        lo = min(lo, as_u32(x[e]));
        hi = max(hi, as_u32(x[e]));
    }
    if (__any(lo < (31u << 23) || hi >= 0x7F800000u)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = sqrtf(x[e]);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = __builtin_amdgcn_rsqf(x[e]);
        const float s = x[e] * y;
        r[e] = __builtin_fmaf(__builtin_fmaf(-s, s, x[e]), 0.5f * y, s);
    }
}

// Scale bytes of the block of 32 whose magnitudes this lane and its three
// neighbours hold, and this lane's 8 codes of m and of r.
__device__ __forceinline__ void encode8(const float (&m1)[8], const float (&r1)[8], uint64_t pos,
                                        const AdamwScalars& a, uint32_t& bm, uint32_t& br,
                                        u32x2& cm, u32x2& cr) {
    uint32_t mm = 0, mr = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        mm = max(mm, as_u32(m1[e]) & 0x7FFFFFFFu);
        mr = max(mr, as_u32(r1[e]) & 0x7FFFFFFFu);
    }
    mm = group_max_u32<4>(mm);
    mr = group_max_u32<4>(mr);
    const bool badm = mm >= 0x7F800000u, badr = mr >= 0x7F800000u;
    bm = (uint32_t)max((int)(mm >> 23) - 7, 0);
    br = (uint32_t)max((int)(mr >> 23) - 7, 0);
    const float im = e8m0_inv_scale_f32(badm ? 0u : bm), ir = e8m0_inv_scale_f32(badr ? 0u : br);
    cm = cr = (u32x2){0u, 0u};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint64_t n = (pos >> 2) + q;
        const Philox4 w = philox4x32_10((uint32_t)n, (uint32_t)(n >> 32), a.step, 0u,
                                        (uint32_t)a.seed, (uint32_t)(a.seed >> 32));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = m1[4 * q + e];
            const uint32_t c = sr_e4m3(fabsf(x) * im, w.v[e] & 0xFFFFu) | ((as_u32(x) >> 24) & 0x80u);
            cm[q] |= c << (8 * e);
            cr[q] |= sr_e4m3(r1[4 * q + e] * ir, w.v[e] >> 16) << (8 * e);
        }
    }
    if (badm) bm = 0xFFu, cm = (u32x2){0u, 0u};
    if (badr) br = 0xFFu, cr = (u32x2){0u, 0u};
}

template <int GB>
__device__ __forceinline__ float grad1(const void* g, int64_t i) {
    return GB ? as_f32((uint32_t)global<const uint16_t>(g)[i] << 16) : global<const float>(g)[i];
}
__device__ __forceinline__ uint32_t pack_copy(float lo, float hi) {
    const bf16x2_t q = {(__bf16)lo, (__bf16)hi};  // v_cvt_pk_bf16_f32
    return __builtin_bit_cast(uint32_t, q);
}

// Four elements of a lane as they lie in memory.
template <int GB>
struct Grad4 {
    u32x4 w;
    __device__ __forceinline__ void load(const void* g, int64_t i) {
        if (GB) {
            const u32x2 v = __builtin_nontemporal_load(global<const u32x2>((const uint16_t*)g + i));
            w.x = v.x;
            w.y = v.y;
        } else {
            w = __builtin_nontemporal_load(global<const u32x4>((const float*)g + i));
        }
    }
    __device__ __forceinline__ float at(int e) const {
        if (GB) return (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
        return as_f32(w[e]);
    }
};

// Elements i0 .. of one tensor with 32-bit moments: 1024 at a time.
template <int GB>
__device__ __forceinline__ void chunk32(const AdamwScalars& a, const AdamwArg& d, int64_t i0,
                                        float gscale, float decay) {
    constexpr int U = kChunk / 1024;
    const Global<float> dp = global<float>(d.p), dm = global<float>(d.m), dv = global<float>(d.v);
    const Global<uint16_t> dc = global<uint16_t>(d.copy);
    const int64_t i = i0 + threadIdx.x * 4;
    const bool whole = i0 + kChunk <= d.n;
    u32x4 p[U], m[U], v[U];
    Grad4<GB> g[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t j = i + k * 1024;
        if (!whole && j + 4 > d.n) continue;
        p[k] = __builtin_nontemporal_load((Global<const u32x4>)(dp + j));
        g[k].load(d.g, j);
        m[k] = __builtin_nontemporal_load((Global<const u32x4>)(dm + j));
        v[k] = __builtin_nontemporal_load((Global<const u32x4>)(dv + j));
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t j = i + k * 1024;
        if (!whole && j + 4 > d.n) continue;
        float p1[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float m1, v1;
            p1[e] = adamw_one(a, as_f32(p[k][e]), g[k].at(e) * gscale, as_f32(m[k][e]),
                              as_f32(v[k][e]), decay, m1, v1);
            p[k][e] = as_u32(p1[e]);
            m[k][e] = as_u32(m1);
            v[k][e] = as_u32(v1);
        }
        __builtin_nontemporal_store(p[k], (Global<u32x4>)(dp + j));
        __builtin_nontemporal_store(m[k], (Global<u32x4>)(dm + j));
        __builtin_nontemporal_store(v[k], (Global<u32x4>)(dv + j));
        if (dc)
            *(Global<u32x2>)(dc + j) = (u32x2){pack_copy(p1[0], p1[1]), pack_copy(p1[2], p1[3])};
    }
    const int64_t j = (d.n & ~(int64_t)3) + threadIdx.x;  // what is left past the vectors
    if (whole || j >= d.n) return;
    float m1, v1;
    const float p1 = adamw_one(a, dp[j], grad1<GB>(d.g, j) * gscale, dm[j], dv[j], decay, m1, v1);
    dp[j] = p1;
    dm[j] = m1;
    dv[j] = v1;
    if (dc) dc[j] = (uint16_t)f32_to_bf16_bits(p1);
}

// The same with 8-bit moments: 8 elements per lane, the whole chunk at a time.
template <int GB>
__device__ __forceinline__ void chunk8(const AdamwScalars& a, const AdamwArg& d, int64_t i0,
                                       float gscale, float decay) {
    constexpr int SPAN = 8 * group_threads(8), U = kChunk / SPAN;
    const int64_t i = i0 + threadIdx.x * 8;
    const Global<float> dp = global<float>(d.p);
    const Global<uint8_t> dm = global<uint8_t>(d.m), dv = global<uint8_t>(d.v);
    const Global<uint8_t> dms = global<uint8_t>(d.ms), dvs = global<uint8_t>(d.vs);
    const Global<uint16_t> dc = global<uint16_t>(d.copy);
    const bool whole = i0 + kChunk <= d.n;
    u32x4 p[U][2];
    Grad4<GB> g[U][2];
    u32x2 m[U], v[U];
    float sm[U], sv[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t j = i + k * SPAN;
        if (whole || j + 8 <= d.n) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                p[k][q] = __builtin_nontemporal_load((Global<const u32x4>)(dp + j + 4 * q));
                g[k][q].load(d.g, j + 4 * q);
            }
            m[k] = __builtin_nontemporal_load((Global<const u32x2>)(dm + j));
            v[k] = __builtin_nontemporal_load((Global<const u32x2>)(dv + j));
        } else {  // past the end: zeros, which leave zero moments
            p[k][0] = p[k][1] = g[k][0].w = g[k][1].w = (u32x4){0u, 0u, 0u, 0u};
            m[k] = v[k] = (u32x2){0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (j + e >= d.n) continue;
                p[k][e >> 2][e & 3] = as_u32(dp[j + e]);
                if (GB)
                    g[k][e >> 2].w[(e >> 1) & 1] |= (uint32_t)global<const uint16_t>(d.g)[j + e]
                                                    << (16 * (e & 1));
                else
                    g[k][e >> 2].w[e & 3] = global<const uint32_t>(d.g)[j + e];
                m[k][e >> 2] |= (uint32_t)dm[j + e] << (8 * (e & 3));
                v[k][e >> 2] |= (uint32_t)dv[j + e] << (8 * (e & 3));
            }
        }
        const bool any = whole || j < d.n;
        sm[k] = any ? e8m0_scale_f32(dms[j >> 5]) : 0.0f;
        sv[k] = any ? e8m0_scale_f32(dvs[j >> 5]) : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t j = i + k * SPAN;
        float m1[8], v1[8], r1[8], p1[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t wm = m[k][e >> 2], wv = v[k][e >> 2];
            const int b = e & 3;
            const float mf = b == 0   ? __builtin_amdgcn_cvt_f32_fp8(wm, 0)
                             : b == 1 ? __builtin_amdgcn_cvt_f32_fp8(wm, 1)
                             : b == 2 ? __builtin_amdgcn_cvt_f32_fp8(wm, 2)
                                      : __builtin_amdgcn_cvt_f32_fp8(wm, 3);
            const float vf = b == 0   ? __builtin_amdgcn_cvt_f32_fp8(wv, 0)
                             : b == 1 ? __builtin_amdgcn_cvt_f32_fp8(wv, 1)
                             : b == 2 ? __builtin_amdgcn_cvt_f32_fp8(wv, 2)
                                      : __builtin_amdgcn_cvt_f32_fp8(wv, 3);
            const float r = vf * sv[k], gr = g[k][e >> 2].at(b) * gscale;
            m1[e] = a.b1 * (mf * sm[k]) + a.a1 * gr;
            v1[e] = a.b2 * (r * r) + a.a2 * gr * gr;
        }
        roots8(v1, r1);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // the quotient is the hardware's, a unit off at most: it leaves in p only
            p1[e] = as_f32(p[k][e >> 2][e & 3]) * decay -
                    a.lr * m1[e] * __builtin_amdgcn_rcpf(r1[e] * a.rc2 + a.eps);
            if (!whole && j + e >= d.n) m1[e] = r1[e] = 0.0f;
        }
        uint32_t bm, br;
        u32x2 cm, cr;
        encode8(m1, r1, d.base + j, a, bm, br, cm, cr);
        if (whole || j + 8 <= d.n) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                __builtin_nontemporal_store(
                    (u32x4){as_u32(p1[4 * q]), as_u32(p1[4 * q + 1]), as_u32(p1[4 * q + 2]),
                            as_u32(p1[4 * q + 3])},
                    (Global<u32x4>)(dp + j + 4 * q));
            __builtin_nontemporal_store(cm, (Global<u32x2>)(dm + j));
            __builtin_nontemporal_store(cr, (Global<u32x2>)(dv + j));
            if (dc)
                *(Global<u32x4>)(dc + j) = (u32x4){pack_copy(p1[0], p1[1]), pack_copy(p1[2], p1[3]),
                                                pack_copy(p1[4], p1[5]), pack_copy(p1[6], p1[7])};
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (j + e >= d.n) continue;
                dp[j + e] = p1[e];
                dm[j + e] = (uint8_t)(cm[e >> 2] >> (8 * (e & 3)));
                dv[j + e] = (uint8_t)(cr[e >> 2] >> (8 * (e & 3)));
                if (dc) dc[j + e] = (uint16_t)f32_to_bf16_bits(p1[e]);
            }
        }
        if ((threadIdx.x & 3) == 0 && (whole || j < d.n)) {
            dms[j >> 5] = (uint8_t)bm;
            dvs[j >> 5] = (uint8_t)br;
        }
    }
}

template <int GB, int BITS>
__device__ __forceinline__ void adamw_group(const AdamwScalars& h, const AdamwArg& d, uint32_t group) {
    const float gscale = h.grad_scale ? *h.grad_scale : 1.0f;
    const float decay = (float)(1.0 - h.lr_wd * d.decay);
    const int64_t i0 = (int64_t)(group - d.first) * kChunk;
    if (BITS == 32)
        chunk32<GB>(h, d, i0, gscale, decay);
    else
        chunk8<GB>(h, d, i0, gscale, decay);
}

template <int GB, int BITS>
__global__ __launch_bounds__(group_threads(BITS)) void adamw_kernel(const AdamwArgs a) {
    // the group's tensor: the last that starts at or before it, found by all
    // lanes at once
    const int l = threadIdx.x & 63;
    const bool below = l < a.count && (l == 0 || a.t[l].first <= blockIdx.x);
    const int t = __popcll(__ballot(below)) - 1;
    adamw_group<GB, BITS>(a.h, a.t[t], blockIdx.x);
}
template <int GB, int BITS>
__global__ __launch_bounds__(group_threads(BITS)) void adamw_table_kernel(const AdamwArg* __restrict__ table,
                                                          const uint32_t* __restrict__ owner,
                                                          uint32_t group0, const AdamwScalars h) {
    const uint32_t group = group0 + blockIdx.x;
    adamw_group<GB, BITS>(h, table[owner[group]], group);
}

static AdamwScalars scalars(double lr, double beta1, double beta2, double eps, int64_t step,
                            uint64_t seed, const float* grad_scale) {
    AdamwScalars a;
    a.grad_scale = grad_scale;
    a.seed = seed;
    a.lr_wd = lr;
    a.step = (uint32_t)step;
    a.b1 = (float)beta1;
    a.a1 = (float)(1.0 - beta1);
    a.b2 = (float)beta2;
    a.a2 = (float)(1.0 - beta2);
    a.lr = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
    a.rc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
    a.eps = (float)eps;
    return a;
}

static int64_t groups_of(const fp4q_adamw_tensor_t& t) { return (t.numel + kChunk - 1) / kChunk; }

static AdamwArg describe(const fp4q_adamw_tensor_t& t, uint64_t base, uint64_t first) {
    AdamwArg d;
    d.p = t.param;
    d.g = t.grad;
    d.m = t.exp_avg;
    d.v = t.exp_avg_sq;
    d.ms = t.exp_avg_scales;
    d.vs = t.exp_avg_sq_scales;
    d.copy = t.copy;
    d.n = t.numel;
    d.base = base;
    d.decay = t.weight_decay;
    d.first = (uint32_t)first;
    d.unused = 0;
    return d;
}
static uint64_t rounded(int64_t n) { return (uint64_t)((n + 31) / 32) * 32; }

#define FP4Q_ADAMW(KERNEL, ...)                                                   \
    do {                                                                          \
        if (bits == 8) {                                                          \
            if (gdtype == BF16)                                                   \
                FP4Q_LAUNCH((KERNEL<1, 8>), grid, dim3(group_threads(8)), 0, s, __VA_ARGS__);  \
            else                                                                  \
                FP4Q_LAUNCH((KERNEL<0, 8>), grid, dim3(group_threads(8)), 0, s, __VA_ARGS__);  \
        } else {                                                                  \
            if (gdtype == BF16)                                                   \
                FP4Q_LAUNCH((KERNEL<1, 32>), grid, dim3(group_threads(32)), 0, s, __VA_ARGS__); \
            else                                                                  \
                FP4Q_LAUNCH((KERNEL<0, 32>), grid, dim3(group_threads(32)), 0, s, __VA_ARGS__); \
        }                                                                         \
        const hipError_t e_ = hipGetLastError();                                  \
        if (e_ != hipSuccess) return e_;                                          \
    } while (0)

hipError_t launch_adamw(const fp4q_adamw_tensor_t* t, int n, int bits, int gdtype, double lr,
                        double beta1, double beta2, double eps, int64_t step, uint64_t seed,
                        const float* grad_scale, hipStream_t s) {
    AdamwArgs a;
    a.h = scalars(lr, beta1, beta2, eps, step, seed, grad_scale);
    uint64_t base = 0;
    int64_t done = 0;  // chunks of tensor i that earlier launches took
    for (int i = 0; i < n;) {
        int64_t groups = 0;
        a.count = 0;
        while (i < n && a.count < kTensors && groups < kMaxGroups) {
            const int64_t left = groups_of(t[i]) - done;
            if (left > 0) {
                const int64_t take = left < kMaxGroups - groups ? left : kMaxGroups - groups;
                // of a tensor that an earlier launch began, `first` wraps below zero;
                // group - first is the chunk all the same
                a.t[a.count++] = describe(t[i], base, (uint64_t)(groups - done));
                groups += take;
                done += take;
                if (take < left) break;
            }
            base += rounded(t[i++].numel);
            done = 0;
        }
        if (a.count == 0) break;
        const dim3 grid((unsigned)groups);
        FP4Q_ADAMW(adamw_kernel, a);
    }
    return hipSuccess;
}

size_t adamw_table_bytes(const fp4q_adamw_tensor_t* t, int n, int64_t* groups) {
    *groups = 0;
    for (int i = 0; i < n; ++i) *groups += groups_of(t[i]);
    return (size_t)n * sizeof(AdamwArg) + (size_t)*groups * 4;
}

void adamw_table(const fp4q_adamw_tensor_t* t, int n, void* table) {
    AdamwArg* d = (AdamwArg*)table;
    uint32_t* owner = (uint32_t*)(d + n);
    uint64_t base = 0, groups = 0;
    for (int i = 0; i < n; ++i) {
        d[i] = describe(t[i], base, groups);
        base += rounded(t[i].numel);
        for (int64_t k = groups_of(t[i]); k > 0; --k) owner[groups++] = (uint32_t)i;
    }
}

hipError_t launch_adamw_table(const void* table, int n, int64_t groups, int bits, int gdtype,
                              double lr, double beta1, double beta2, double eps, int64_t step,
                              uint64_t seed, const float* grad_scale, hipStream_t s) {
    const AdamwScalars h = scalars(lr, beta1, beta2, eps, step, seed, grad_scale);
    const AdamwArg* d = (const AdamwArg*)table;
    const uint32_t* owner = (const uint32_t*)(d + n);
    for (int64_t g = 0; g < groups; g += kMaxGroups) {
        const int64_t now = groups - g < kMaxGroups ? groups - g : kMaxGroups;
        const dim3 grid((unsigned)now);
        FP4Q_ADAMW(adamw_table_kernel, d, owner, (uint32_t)g, h);
    }
    return hipSuccess;
}
#undef FP4Q_ADAMW

}  // namespace fp4q
