// The norms behind and in front of a block, fused with the block's gate and the
// residual sum between them, forward and backward.
//
//   n  = (b - mb) rb wp + bp   (the norm behind the block; n = b without it)
//   x' = xs x + bs g n         y = (x' - m) r w + c
//
// with the statistics of the rows of b and of x'.  Backward, from dy and the
// gradient dx' that arrives at x' along the residual stream:
//
//   xh = (x' - m) r    t = dy w    D = dx' + r (t - mean_c(t) [layer] - xh mean_c(t xh))
//   nh = (b - mb) rb   u = bs g D wp
//   dx = xs D          db = rb (u - mean_c(u) [layer] - nh mean_c(u nh))
//   dw = sum_r dy xh   dc = sum_r dy
// and with S1 = sum D nh, S2 = sum D over the rows that share a gate
//   dg = bs (wp S1 + bp S2)    dwp = sum_groups bs g S1    dbp = sum_groups bs g S2
//
// The forward pass (here) is bound by memory: x and b are read once, x' and y
// written once.  So a row stays in registers from its load to its last use, held
// by one wave or by all waves of a workgroup, 8 elements per lane and chunk, as
// in norm.hip; each norm costs the waves one barrier; y is formed from x' before
// it is rounded, and where a quantised y is asked for, its codes leave instead of
// y (0.53 bytes an element for 2; 8192 x 2048 19.9 us, y and its codes in a launch
// of their own 32.8).  The factors bs g wp and bs g bp, w and c stay
// in registers over a workgroup's rows; rows of gates that come with the rows are
// loaded with them.  8192 x 2048 bf16 24.7 us and 16384 x 5120 with an fp32 stream
// 178 us: 5.4 and 5.6 TB/s; 8 rows take 3.8 us, and the host 10.
#include <algorithm>

#include "residual_norm.h"
#include "row_norm.h"

namespace fp4q {

constexpr int64_t kAnyGrid = 1 << 16;

// Codes of 8 values of a block of 32 that four neighbouring lanes hold, as
// fp4q_quantize gives them, and its scale byte.
__device__ __forceinline__ uint32_t quantise8(const float (&f)[8], uint32_t& byte) {
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max(amax, as_u32(f[e]) & 0x7FFFFFFFu);
    amax = group_max_u32<4>(amax);
    const bool finite = amax < 0x7F800000u;
    byte = finite ? e8m0_from_amax(amax) : 0xFFu;
    const float sc = e8m0_scale_f32(byte);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[0], f[1], sc, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[2], f[3], sc, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[4], f[5], sc, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[6], f[7], sc, 3);
    return finite ? q : 0u;
}

// ---- any width: a workgroup per row, the row read once per sum ----

__global__ __launch_bounds__(256) void residual_norm_any_kernel(const ResidualNorm a) {
    __shared__ float red[4];
    const float n = (float)a.cols;
    const bool post = a.post != kPostNone;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t g0 = r / a.gate_rows * a.ldg;
        float pm = 0.0f, pr = 1.0f, m = 0.0f, sum = 0.0f, mid = 0.0f;
        // sums of the branch's elements and of their squares around `mid`
        auto of_branch = [&](int64_t c, auto full, int left) __attribute__((always_inline)) {
            constexpr int FULL = decltype(full)::value;
            float b[8];
            load8_as<FULL>(a.b, a.b_bf16, r * a.ldb + c, left, 0.0f, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += FULL || e < left ? b[e] : 0.0f;
        };
        auto of_branch2 = [&](int64_t c, auto full, int left) __attribute__((always_inline)) {
            constexpr int FULL = decltype(full)::value;
            float b[8];
            load8_as<FULL>(a.b, a.b_bf16, r * a.ldb + c, left, 0.0f, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += FULL || e < left ? (b[e] - mid) * (b[e] - mid) : 0.0f;
        };
        if (post) {
            if (a.post == 0) {
                over8(a.cols, of_branch);
                pm = block_sum(sum, red) / n;
            }
            sum = 0.0f;
            mid = pm;
            over8(a.cols, of_branch2);
            pr = 1.0f / sqrtf(block_sum(sum, red) / n + a.eps);
        }
        // x' of 8 elements
        auto stream = [&](int64_t c, auto full, int left, float(&x)[8]) __attribute__((always_inline)) {
            constexpr int FULL = decltype(full)::value;
            float b[8], w[8], v[8];
            load8_as<FULL>(a.b, a.b_bf16, r * a.ldb + c, left, 0.0f, b);
            load8_as<FULL>(a.x, a.x_bf16, r * a.ldx + c, left, 0.0f, x);
            load8_as<FULL>(a.post_weight, a.w_bf16, c, left, 1.0f, w);
            load8_as<FULL>(a.post_bias, a.w_bf16, c, left, 0.0f, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = (b[e] - pm) * pr * w[e] + v[e];
            load8_as<FULL>(a.gate, a.gate_bf16, g0 + c, left, 1.0f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = a.x_scale * x[e] + a.branch_scale * (b[e] * w[e]);
        };
        auto of_stream = [&](int64_t c, auto full, int left) __attribute__((always_inline)) {
            float x[8];
            stream(c, full, left, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += decltype(full)::value || e < left ? x[e] : 0.0f;
        };
        auto of_stream2 = [&](int64_t c, auto full, int left) __attribute__((always_inline)) {
            float x[8];
            stream(c, full, left, x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum += decltype(full)::value || e < left ? (x[e] - mid) * (x[e] - mid) : 0.0f;
        };
        sum = 0.0f;
        if (!a.rms) {
            over8(a.cols, of_stream);
            m = block_sum(sum, red) / n;
        }
        sum = 0.0f;
        mid = m;
        over8(a.cols, of_stream2);
        const float rs = 1.0f / sqrtf(block_sum(sum, red) / n + a.eps);
        // (each lane reads what it then writes: x_out may be x)
        auto write = [&](int64_t c, auto full, int left) __attribute__((always_inline)) {
            constexpr int FULL = decltype(full)::value;
            float x[8], f[8], v[8];
            stream(c, full, left, x);
            load8_as<FULL>(a.weight, a.w_bf16, c, left, 1.0f, f);
            load8_as<FULL>(a.bias, a.w_bf16, c, left, 0.0f, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = (x[e] - m) * rs * f[e] + v[e];
            store8_as<FULL>(a.xo, a.x_bf16, r * a.ldxo + c, left, x);
            if (a.codes) {  // cols is a multiple of 32: whole groups of four lanes
                uint32_t byte;
                const uint32_t q = quantise8(f, byte);
                *(uint32_t*)(a.codes + r * (a.cols / 2) + c / 2) = q;
                a.scales[r * (a.cols / 32) + c / 32] = (uint8_t)byte;
            } else {
                store8_as<FULL>(a.y, a.y_bf16, r * a.ldy + c, left, f);
            }
        };
        over8(a.cols, write);
        if (threadIdx.x == 0) {
            if (a.post_mean && a.post == 0) a.post_mean[r] = pm;
            if (a.post_rstd && post) a.post_rstd[r] = pr;
            if (a.mean && !a.rms) a.mean[r] = m;
            if (a.rstd) a.rstd[r] = rs;
        }
    }
}

// ---- rows in registers ----

// Mean and mean square around it (RMS norm: around 0) of the row that the lanes
// hold, with one barrier where waves share it: each wave sums its squares around
// its own mean, and the sums are moved to the row's mean,
//   sum (v - m)^2 = sum_waves [sum (v - m_w)^2 + n_w (m_w - m)^2].
template <int MULTI, int NV>
struct Moments {
    float* red;  // two sets of 2 * 16 floats that take turns, as in row_sums
    float n, mine, theirs;  // elements of the row, of this wave, of wave threadIdx.x % 16
    int turn;
    __device__ __forceinline__ static float owned(const Place<NV>& pl, int cols, int wave) {
        int c = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) c += min(max(cols - k * pl.step - wave * 512, 0), 512);
        return (float)c;
    }
    __device__ __forceinline__ Moments(const Place<NV>& pl, int cols, float* red)
        : red(red), n((float)cols), turn(0) {
        const int l = threadIdx.x & 15;
        mine = MULTI ? owned(pl, cols, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) : n;
        theirs = MULTI && l < pl.W ? owned(pl, cols, l) : 0.0f;
    }
    __device__ __forceinline__ void of(const Place<NV>& pl, const float (&v)[NV][8], bool layer,
                                       float& mean, float& var) {
        float s = 0.0f, q = 0.0f, m = 0.0f;
        if (layer) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float p = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) p += pl.owns(k, e) ? v[k][e] : 0.0f;
                s += p;
            }
            s = wave_sum(s);
            m = s / mine;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float p = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = v[k][e] - m;
                p += pl.owns(k, e) ? d * d : 0.0f;
            }
            q += p;
        }
        q = wave_sum(q);
        if (!MULTI) {
            mean = m;
            var = q / n;
            return;
        }
        float* r = red + turn * 32;
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) {
            r[threadIdx.x >> 6] = q;
            if (layer) r[16 + (threadIdx.x >> 6)] = s;
        }
        __syncthreads();
        const int l = threadIdx.x & 15;
        q = l < pl.W ? r[l] : 0.0f;
        mean = 0.0f;
        if (layer) {
            s = l < pl.W ? r[16 + l] : 0.0f;
            mean = sum16(s) / n;
            const float d = l < pl.W ? s / theirs - mean : 0.0f;
            q += theirs * (d * d);
        }
        var = sum16(q) / n;
    }
};

// OUT: y in fp32 (0), in bf16 (1), its codes (2).  GATE: one row of gates for
// all rows, or none (0), a row of gates read with every row, fp32 (1), bf16 (2).
template <int XB, int BB, int OUT, int GATE, int MULTI, int NV>
__global__ __launch_bounds__(MULTI ? 1024 : 256) void residual_norm_kernel(const ResidualNorm a,
                                                                           const FastDiv div) {
    // two chunks leave 1024 threads no registers for the vectors of the norm
    // behind the block, which then lie in LDS, 16 floats per lane each
    constexpr bool kLds = MULTI && NV == 2;
    // nor, where gates come with the rows, for the next row (2000 x 13824 fp32 150
    // us with spills, 91 without the next row)
    constexpr bool kAhead = !kLds || !GATE;
    __shared__ float red[MULTI ? 2 * 32 : 1];
    __shared__ u32x4 vectors[kLds ? 2 * 2 * NV * 1024 : 1];
    const int cols = (int)a.cols;
    Place<NV> pl = Place<NV>::template make<MULTI>(cols);
    // a lane past the row's end holds its place in the last block of 32 again,
    // so that four lanes hold a block there too
    if (OUT == 2 && pl.skip == 8) pl.tail = cols - 32 + (pl.t & 31);
    const int64_t step = MULTI ? gridDim.x : gridDim.x * 4;
    int64_t r = first_row<MULTI>();
    if (r >= a.rows) return;  // whole waves, and whole workgroups where they share a row
    Moments<MULTI, NV> moments(pl, cols, red);
    struct Row {
        Chunk<XB> x[NV];
        Chunk<BB> b[NV];
        Chunk<GATE == 2> g[GATE ? NV : 1];
    };
    Row in;
    auto fetch = [&](int64_t row) __attribute__((always_inline)) {
        row = min(row, a.rows - 1);
        const int64_t g = GATE ? (int64_t)fastdiv((uint32_t)row, div) * a.ldg : 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            in.b[k].load_row(a.b, row * a.ldb, pl.start(k));
            in.x[k].load_row(a.x, row * a.ldx, pl.start(k));
            if (GATE) in.g[k].load_row(a.gate, g, pl.start(k));
        }
    };
    if (kAhead) fetch(r);
    // half h of this lane's chunk k of the weight (o = 0) or the bias
    auto slot = [&](int o, int k, int h) __attribute__((always_inline)) -> u32x4& {
        return vectors[((o * NV + k) * 2 + h) * 1024 + threadIdx.x];
    };
    auto words = [](const float(&v)[8], int h) __attribute__((always_inline)) {
        return (u32x4){as_u32(v[4 * h]), as_u32(v[4 * h + 1]), as_u32(v[4 * h + 2]), as_u32(v[4 * h + 3])};
    };
    float pw[NV][8], pc[NV][8], w[NV][8], c[NV][8];
    const bool post = a.post != kPostNone, post_layer = a.post == 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_vec8(a.post_weight, a.w_bf16, pl.start(k), 1.0f, pw[k]);
        load_vec8(a.post_bias, a.w_bf16, pl.start(k), 0.0f, pc[k]);
        load_vec8(a.weight, a.w_bf16, pl.start(k), 1.0f, w[k]);
        load_vec8(a.bias, a.w_bf16, pl.start(k), 0.0f, c[k]);
        float g[8];
        load_vec8(GATE ? nullptr : a.gate, a.gate_bf16, pl.start(k), 1.0f, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            pw[k][e] *= a.branch_scale * g[e];
            pc[k][e] *= a.branch_scale * g[e];
        }
        if (kLds) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                slot(0, k, h) = words(pw[k], h);
                slot(1, k, h) = words(pc[k], h);
            }
        }
    }
    float pm = 0.0f, pr = 1.0f, m = 0.0f, rs = 0.0f;
    // the statistics of a row are stored ahead of the next row's loads
    auto stats = [&](int64_t row) __attribute__((always_inline)) {
        if (pl.t) return;
        if (a.post_mean && post_layer) a.post_mean[row] = pm;
        if (a.post_rstd && post) a.post_rstd[row] = pr;
        if (a.mean && !a.rms) a.mean[row] = m;
        if (a.rstd) a.rstd[row] = rs;
    };
    int64_t last = -1;
    for (; r < a.rows; r += step) {
        float v[NV][8], n[NV][8], g[NV][8];
        if (!kAhead) fetch(r);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[k][e] = in.b[k].at(e);
                v[k][e] = in.x[k].at(e);
                if (GATE) g[k][e] = in.g[k].at(e);
            }
        // x' may lie on x, whose last elements two waves hold: all of a row has
        // arrived before the barrier that its stores come after
#pragma unroll
        for (int k = 0; MULTI && k < NV; ++k) in.x[k].arrived();
        if (last >= 0) stats(last);
        last = r;
        if (kAhead) fetch(r + step);
        if (post) {
            float var;
            moments.of(pl, n, post_layer, pm, var);
            pr = 1.0f / sqrtf(var + a.eps);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (kLds) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 vw = slot(0, k, h), vc = slot(1, k, h);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pw[k][4 * h + e] = as_f32(vw[e]);
                        pc[k][4 * h + e] = as_f32(vc[e]);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float t = (n[k][e] - pm) * pr * pw[k][e] + pc[k][e];
                if (GATE) t *= g[k][e];
                // not a contraction of either product: two waves may hold the element
                v[k][e] = __builtin_fmaf(a.x_scale, v[k][e], t);
            }
        }
        float var;
        moments.of(pl, v, !a.rms, m, var);
        rs = 1.0f / sqrtf(var + a.eps);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c0 = pl.start(k);
            store_row<XB>(a.xo, r * a.ldxo, pl.start(k), v[k]);
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = ((v[k][e] - m) * rs) * w[k][e] + c[k][e];
            if (OUT == 2) {
                uint32_t byte;
                const uint32_t q = quantise8(f, byte);
                *(uint32_t*)(a.codes + r * (cols / 2) + c0 / 2) = q;
                a.scales[r * (cols / 32) + c0 / 32] = (uint8_t)byte;
            } else {
                store_row<OUT>(a.y, r * a.ldy, pl.start(k), f);
            }
        }
    }
    stats(last);
}

// Waves per compute unit by the bytes that a lane loads for an element: up to 4
// leave registers for more of them.  16, 20, 24 and 32 waves: 8192 x 2048 bf16
// 26.3, 25.6, 24.7, 25.7 us, 16384 x 5120 158, 139, 139, 140; with an fp32 stream
// 34.4, 34.6, 35.6, 36.9 and 178, 190, 190, 192; 4000 x 1111 fp32 with a gate per
// sequence 13.3, 13.6, 14.7, 14.3.
constexpr int kWavesLight = 24, kWavesHeavy = 16;

template <int XB, int BB, int OUT, int GATE>
static void go_rows(const NormShape sh, const ResidualNorm& a, hipStream_t s) {
    const FastDiv div = make_fastdiv((uint32_t)a.gate_rows);
    const int loaded = (XB ? 2 : 4) + (BB ? 2 : 4) + (GATE == 0 ? 0 : GATE == 2 ? 2 : 4);
    const unsigned groups = (unsigned)norm_groups(sh, a.rows, loaded <= 4 ? kWavesLight : kWavesHeavy, 1);
#define FP4Q_GO(MULTI, NV)                                                                      \
    if (sh.multi == (bool)MULTI && sh.nv == NV)                                                 \
    FP4Q_LAUNCH((residual_norm_kernel<XB, BB, OUT, GATE, MULTI, NV>), dim3(groups),             \
                dim3((unsigned)sh.threads), 0, s, a, div)
    FP4Q_GO(0, 1);
    FP4Q_GO(0, 2);
    FP4Q_GO(1, 1);
    FP4Q_GO(1, 2);
#undef FP4Q_GO
}
template <int XB, int BB, int OUT>
static void go_gate(const NormShape sh, const ResidualNorm& a, hipStream_t s) {
    if (!a.gate || a.gate_rows >= a.rows)
        go_rows<XB, BB, OUT, 0>(sh, a, s);
    else if (!a.gate_bf16)
        go_rows<XB, BB, OUT, 1>(sh, a, s);
    else
        go_rows<XB, BB, OUT, 2>(sh, a, s);
}
template <int XB, int BB>
static void go_out(const NormShape sh, const ResidualNorm& a, hipStream_t s) {
    if (a.codes)
        go_gate<XB, BB, 2>(sh, a, s);
    else if (a.y_bf16)
        go_gate<XB, BB, 1>(sh, a, s);
    else
        go_gate<XB, BB, 0>(sh, a, s);
}

hipError_t launch_residual_norm(const ResidualNorm& a, hipStream_t s) {
    const NormShape sh = norm_shape(a.rows, a.cols);
    if (sh.nv == 0)
        FP4Q_LAUNCH(residual_norm_any_kernel, dim3((unsigned)std::min(a.rows, kAnyGrid)), dim3(256), 0,
                    s, a);
    else if (a.x_bf16)
        a.b_bf16 ? go_out<1, 1>(sh, a, s) : go_out<1, 0>(sh, a, s);
    else
        a.b_bf16 ? go_out<0, 1>(sh, a, s) : go_out<0, 0>(sh, a, s);
    return hipGetLastError();
}

}  // namespace fp4q
