// The backward pass of the residual norms (the formulas stand at the head of
// residual_norm.hip).
#include <algorithm>

#include "residual_norm.h"
#include "row_norm.h"

namespace fp4q {

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
