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
#include <algorithm>

#include "residual_norm.h"
#include "row_norm.h"

namespace fp4q {

__device__ __forceinline__ float load_as(const void* p, int bf16, int64_t i) {
    return bf16 ? load1<1>(p, i) : load1<0>(p, i);
}
__device__ __forceinline__ void store_as(void* p, int bf16, int64_t i, float v) {
    if (bf16)
        store1<1>(p, i, v);
    else
        store1<0>(p, i, v);
}

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
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t g0 = r / a.gate_rows * a.ldg;
        float pm = 0.0f, pr = 1.0f, m = 0.0f;
        if (a.post != kPostNone) {
            if (a.post == 0) {
                float s = 0.0f;
                for (int64_t c = threadIdx.x; c < a.cols; c += 256)
                    s += load_as(a.b, a.b_bf16, r * a.ldb + c);
                pm = block_sum(s, red) / n;
            }
            float q = 0.0f;
            for (int64_t c = threadIdx.x; c < a.cols; c += 256) {
                const float d = load_as(a.b, a.b_bf16, r * a.ldb + c) - pm;
                q += d * d;
            }
            pr = 1.0f / sqrtf(block_sum(q, red) / n + a.eps);
        }
        auto sum_at = [&](int64_t c) __attribute__((always_inline)) {
            float v = load_as(a.b, a.b_bf16, r * a.ldb + c);
            if (a.post != kPostNone)
                v = (v - pm) * pr * vec1(a.post_weight, a.w_bf16, c, 1.0f) +
                    vec1(a.post_bias, a.w_bf16, c, 0.0f);
            if (a.gate) v *= load_as(a.gate, a.gate_bf16, g0 + c);
            return a.x_scale * load_as(a.x, a.x_bf16, r * a.ldx + c) + a.branch_scale * v;
        };
        if (!a.rms) {
            float s = 0.0f;
            for (int64_t c = threadIdx.x; c < a.cols; c += 256) s += sum_at(c);
            m = block_sum(s, red) / n;
        }
        float q = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += 256) {
            const float d = sum_at(c) - m;
            q += d * d;
        }
        const float rs = 1.0f / sqrtf(block_sum(q, red) / n + a.eps);
        if (a.codes) {  // cols is a multiple of 32: whole groups of four lanes
            for (int64_t c = threadIdx.x * 8; c < a.cols; c += 2048) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = sum_at(c + e);
                    store_as(a.xo, a.x_bf16, r * a.ldxo + c + e, v);
                    f[e] = (v - m) * rs * vec1(a.weight, a.w_bf16, c + e, 1.0f) +
                           vec1(a.bias, a.w_bf16, c + e, 0.0f);
                }
                uint32_t byte;
                const uint32_t q8 = quantise8(f, byte);
                *(uint32_t*)(a.codes + r * (a.cols / 2) + c / 2) = q8;
                a.scales[r * (a.cols / 32) + c / 32] = (uint8_t)byte;
            }
        } else {
            for (int64_t c = threadIdx.x; c < a.cols; c += 256) {
                const float v = sum_at(c);
                store_as(a.xo, a.x_bf16, r * a.ldxo + c, v);
                store_as(a.y, a.y_bf16, r * a.ldy + c,
                         (v - m) * rs * vec1(a.weight, a.w_bf16, c, 1.0f) +
                             vec1(a.bias, a.w_bf16, c, 0.0f));
            }
        }
        if (threadIdx.x == 0) {
            if (a.post_mean && a.post == 0) a.post_mean[r] = pm;
            if (a.post_rstd && a.post != kPostNone) a.post_rstd[r] = pr;
            if (a.mean && !a.rms) a.mean[r] = m;
            if (a.rstd) a.rstd[r] = rs;
        }
    }
}

// ---- the gradient ----

// Slabs of rows that each leave one row of partial column sums.  A slab holds
// whole groups of rows that share a gate, or, where a group is longer than a
// slab, one of the k even parts of one group.
struct Slabs {
    int64_t count, rows, group;  // group: rows of a group
    int64_t k;                   // slabs of a group, 0 with whole groups
    int64_t groups;              // groups of a slab, with whole groups
    __host__ __device__ void bounds(int64_t i, int64_t& r0, int64_t& r1) const {
        if (k) {
            const int64_t g = i / k, j = i % k, base = g * group;
            const int64_t n = rows - base < group ? rows - base : group;
            r0 = base + n * j / k;
            r1 = base + n * (j + 1) / k;
        } else {
            r0 = i * groups * group;
            r1 = rows - r0 < groups * group ? rows : r0 + groups * group;
        }
    }
    __host__ __device__ int64_t group_of(int64_t i) const { return i / k; }  // with parts
};
static Slabs make_slabs(int64_t rows, int64_t gate_rows, int64_t want) {
    Slabs s;
    s.rows = rows;
    s.group = std::min(gate_rows, rows);
    const int64_t all = (rows + s.group - 1) / s.group;
    const int64_t each = (rows + want - 1) / want;
    if (s.group > each) {
        s.k = (s.group + each - 1) / each;
        s.groups = 0;
        s.count = all * s.k;
    } else {
        s.k = 0;
        s.groups = each / s.group;
        s.count = (all + s.groups - 1) / s.groups;
    }
    return s;
}

// Sums of row r: mean_c(t xh), mean_c(t), mean_c(u nh), mean_c(u).
struct RowMeans {
    float txh, t, unh, u;
};
struct RowStats {
    float m, r, pm, pr;
    __device__ __forceinline__ static RowStats of(const ResidualNormGrad& a, int64_t r) {
        RowStats s = {0.0f, a.rstd[r], 0.0f, 1.0f};
        if (!a.rms) s.m = a.mean[r];
        if (a.post != kPostNone) s.pr = a.post_rstd[r];
        if (a.post == 0) s.pm = a.post_mean[r];
        return s;
    }
};
struct RowPoint {
    const ResidualNormGrad& a;
    int64_t r, g0;
    RowStats s;
    __device__ __forceinline__ RowPoint(const ResidualNormGrad& a, int64_t r)
        : a(a), r(r), g0(r / a.gate_rows * a.ldg), s(RowStats::of(a, r)) {}
    __device__ __forceinline__ float dy(int64_t c) const {
        return load_as(a.dy, a.dy_bf16, r * a.lddy + c);
    }
    __device__ __forceinline__ float xh(int64_t c) const {
        return (load_as(a.xo, a.x_bf16, r * a.ldxo + c) - s.m) * s.r;
    }
    __device__ __forceinline__ float nh(int64_t c) const {
        return a.b ? (load_as(a.b, a.b_bf16, r * a.ldb + c) - s.pm) * s.pr : 0.0f;
    }
    __device__ __forceinline__ float D(int64_t c, const RowMeans& k) const {
        const float t = dy(c) * vec1(a.weight, a.w_bf16, c, 1.0f);
        const float d = s.r * (t - k.t - xh(c) * k.txh);
        return a.dxo ? load_as(a.dxo, a.x_bf16, r * a.lddxo + c) + d : d;
    }
    __device__ __forceinline__ float u(int64_t c, float d) const {
        d *= a.branch_scale * vec1(a.post_weight, a.w_bf16, c, 1.0f);
        return a.gate ? d * load_as(a.gate, a.gate_bf16, g0 + c) : d;
    }
};

__global__ __launch_bounds__(256) void residual_grad_rows_kernel(const ResidualNormGrad a,
                                                                 RowMeans* __restrict__ means) {
    __shared__ float red[4];
    const float n = (float)a.cols;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const RowPoint p(a, r);
        RowMeans k = {0.0f, 0.0f, 0.0f, 0.0f};
        float s0 = 0.0f, s1 = 0.0f;
        for (int64_t c = threadIdx.x; c < a.cols; c += 256) {
            const float t = p.dy(c) * vec1(a.weight, a.w_bf16, c, 1.0f);
            s0 += t * p.xh(c);
            s1 += t;
        }
        k.txh = block_sum(s0, red) / n;
        if (!a.rms) k.t = block_sum(s1, red) / n;
        if (a.post != kPostNone) {
            s0 = s1 = 0.0f;
            for (int64_t c = threadIdx.x; c < a.cols; c += 256) {
                const float u = p.u(c, p.D(c, k));
                s0 += u * p.nh(c);
                s1 += u;
            }
            k.unh = block_sum(s0, red) / n;
            if (a.post == 0) k.u = block_sum(s1, red) / n;
        }
        if (threadIdx.x == 0) means[r] = k;
    }
}

// Column sums of a slab, four rows of `cols` floats of the partial sums: dw,
// dc, and S1, S2 of the slab's group, or with whole groups dwp, dbp (the
// groups' dg is then written at once).
__global__ __launch_bounds__(256) void residual_grad_cols_kernel(const ResidualNormGrad a,
                                                                 const RowMeans* __restrict__ means,
                                                                 const Slabs sl,
                                                                 float* __restrict__ part) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= a.cols) return;
    const float wp = vec1(a.post_weight, a.w_bf16, c, 1.0f), bp = vec1(a.post_bias, a.w_bf16, c, 0.0f);
    for (int64_t i = blockIdx.y; i < sl.count; i += gridDim.y) {
        int64_t r0, r1;
        sl.bounds(i, r0, r1);
        float dw = 0.0f, dc = 0.0f, s1 = 0.0f, s2 = 0.0f, dwp = 0.0f, dbp = 0.0f;
        for (int64_t r = r0; r < r1; ++r) {
            const RowPoint p(a, r);
            const float dy = p.dy(c), d = p.D(c, means[r]);
            dw += dy * p.xh(c);
            dc += dy;
            s1 += d * p.nh(c);
            s2 += d;
            if (!sl.k && ((r + 1) % sl.group == 0 || r + 1 == r1)) {
                const int64_t g = r / sl.group;
                const float f = a.branch_scale * (a.gate ? load_as(a.gate, a.gate_bf16, g * a.ldg + c) : 1.0f);
                if (a.dgate) a.dgate[g * a.cols + c] = a.branch_scale * (wp * s1 + bp * s2);
                dwp += f * s1;
                dbp += f * s2;
                s1 = s2 = 0.0f;
            }
        }
        float* o = part + i * 4 * a.cols + c;
        o[0] = dw;
        o[a.cols] = dc;
        o[2 * a.cols] = sl.k ? s1 : dwp;
        o[3 * a.cols] = sl.k ? s2 : dbp;
    }
}

__global__ __launch_bounds__(256) void residual_grad_any_kernel(const ResidualNormGrad a,
                                                                const RowMeans* __restrict__ means) {
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const RowPoint p(a, r);
        const RowMeans k = means[r];
        for (int64_t c = threadIdx.x; c < a.cols; c += 256) {
            const float d = p.D(c, k), u = p.u(c, d);
            const float v = a.post == kPostNone ? u : p.s.pr * (u - k.u - p.nh(c) * k.unh);
            store_as(a.dx, a.x_bf16, r * a.lddx + c, a.x_scale * d);
            store_as(a.db, a.b_bf16, r * a.lddb + c, v);
        }
    }
}

// Adds up the rows of partial sums: 16 columns per workgroup, 64 groups of 16
// lanes over the slabs, so that few loads follow each other.  blockIdx.y: dw,
// dc, dwp, dbp, then the gate's groups, grid_y apart.
constexpr int64_t kJoinGroups = 1 << 21;
__device__ __forceinline__ float join16(float s, float (*red)[16]) {
    const int l = threadIdx.x & 15, wave = threadIdx.x >> 6;
    s = rows_sum(s);
    __syncthreads();
    if ((threadIdx.x & 63) < 16) red[wave][l] = s;
    __syncthreads();
    const int r = (threadIdx.x & 63) >> 4;
    return rows_sum((red[r][l] + red[4 + r][l]) + (red[8 + r][l] + red[12 + r][l]));
}
__global__ __launch_bounds__(1024) void residual_grad_join_kernel(const ResidualNormGrad a,
                                                                  const float* __restrict__ part,
                                                                  const Slabs sl, int64_t group0) {
    __shared__ float red[16][16];
    const int64_t c = (group0 + blockIdx.x) * 16 + (threadIdx.x & 15);
    const bool in = c < a.cols;
    const int first = threadIdx.x >> 4;
    const float* p = part + c;
    if (blockIdx.y < 4) {
        const int y = blockIdx.y;
        float* out = y == 0 ? a.dweight : y == 1 ? a.dbias : y == 2 ? a.dpost_weight : a.dpost_bias;
        if (!out) return;
        const bool scaled = y >= 2 && sl.k;
        float s = 0.0f;
        if (in) {
            for (int64_t i = first; i < sl.count; i += 64) {
                float v = p[(i * 4 + y) * a.cols];
                if (scaled) {
                    v *= a.branch_scale;
                    if (a.gate) v *= load_as(a.gate, a.gate_bf16, sl.group_of(i) * a.ldg + c);
                }
                s += v;
            }
        }
        s = join16(s, red);
        if (threadIdx.x < 16 && in) out[c] = s;
        return;
    }
    const float wp = in ? vec1(a.post_weight, a.w_bf16, c, 1.0f) : 0.0f;
    const float bp = in ? vec1(a.post_bias, a.w_bf16, c, 0.0f) : 0.0f;
    const int64_t groups = sl.count / sl.k;
    for (int64_t g = blockIdx.y - 4; g < groups; g += gridDim.y - 4) {
        float s1 = 0.0f, s2 = 0.0f;
        if (in) {
            for (int64_t i = first; i < sl.k; i += 64) {
                s1 += p[((g * sl.k + i) * 4 + 2) * a.cols];
                s2 += p[((g * sl.k + i) * 4 + 3) * a.cols];
            }
        }
        s1 = join16(s1, red);
        s2 = join16(s2, red);
        if (threadIdx.x < 16 && in) a.dgate[g * a.cols + c] = a.branch_scale * (wp * s1 + bp * s2);
    }
}

constexpr int64_t kAnyGrid = 1 << 16;
constexpr int64_t kGridY = 1 << 15;

static bool any_sums(const ResidualNormGrad& a) {
    return a.dweight || a.dbias || a.dpost_weight || a.dpost_bias || a.dgate;
}

static Slabs grad_slabs(int64_t rows, int64_t cols, int64_t gate_rows) {
    return make_slabs(rows, gate_rows, std::min<int64_t>(256, (rows + 15) / 16));
}

size_t residual_norm_grad_workspace_bytes(int64_t rows, int64_t cols, int64_t gate_rows) {
    const Slabs sl = grad_slabs(rows, cols, gate_rows);
    return (size_t)rows * sizeof(RowMeans) + (size_t)sl.count * 4 * (size_t)cols * sizeof(float);
}

hipError_t launch_residual_norm(const ResidualNorm& a, hipStream_t s) {
    FP4Q_LAUNCH(residual_norm_any_kernel, dim3((unsigned)std::min(a.rows, kAnyGrid)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_residual_norm_grad(const ResidualNormGrad& a, void* ws, hipStream_t s) {
    const Slabs sl = grad_slabs(a.rows, a.cols, a.gate_rows);
    RowMeans* means = (RowMeans*)ws;
    float* part = (float*)(means + a.rows);
    const unsigned rows = (unsigned)std::min(a.rows, kAnyGrid);
    FP4Q_LAUNCH(residual_grad_rows_kernel, dim3(rows), dim3(256), 0, s, a, means);
    if (any_sums(a))  // before dx and db, which may lie on dxo and b
        FP4Q_LAUNCH(residual_grad_cols_kernel,
                    dim3((unsigned)((a.cols + 255) / 256), (unsigned)std::min(sl.count, kGridY)),
                    dim3(256), 0, s, a, means, sl, part);
    FP4Q_LAUNCH(residual_grad_any_kernel, dim3(rows), dim3(256), 0, s, a, means);
    if (any_sums(a)) {
        const int64_t gates = a.dgate && sl.k ? std::min(sl.count / sl.k, kGridY) : 0;
        const int64_t groups = (a.cols + 15) / 16;
        for (int64_t g = 0; g < groups; g += kJoinGroups)
            FP4Q_LAUNCH(residual_grad_join_kernel,
                        dim3((unsigned)std::min(groups - g, kJoinGroups), (unsigned)(4 + gates)),
                        dim3(1024), 0, s, a, part, sl, g);
    }
    return hipGetLastError();
}

}  // namespace fp4q
