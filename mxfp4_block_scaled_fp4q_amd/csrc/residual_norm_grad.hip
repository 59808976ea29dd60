// The backward pass of the residual norms (the formulas stand at the head of
// residual_norm.hip).
//
// Bound by memory: dy, dx', x' and b are read once, dx and db written once, and
// the rows stay in registers between the two row sums that the two norms need.
// The column sums go along in registers too (dw, dc, S1, S2), and each workgroup
// leaves one row of partial sums, which a second, small kernel adds up: no
// atomics, the order of every sum is fixed by the sizes.  Four streams, their next
// row and the sums take 140 to 165 registers, so a compute unit holds 12 waves.
// These are one workgroup of teams of waves, a row to a team, so that they leave
// one row of partial sums together: 8192 x 2048 bf16 44 to 49 us a call (36 to 39
// and the join's 4.0 to 4.7; 5.2 TB/s) against 55 with a workgroup to each team,
// whose partial sums were a quarter of the data.  16384 x 5120 with an fp32 stream
// 305 + 7.7 us (5.0 TB/s), 1999 x 1111 fp32 with gates per sequence 16.3 + 4.8
// (three rows to a team one after another, and two launches).
#include <algorithm>
#include <type_traits>

#include "residual_norm.h"
#include "row_norm.h"

// A product and a sum become one operation where they stand in one expression,
// and nowhere else.  Elements that two waves hold have different places in their
// lanes, and left to itself the compiler contracts a b + c d one way for one place
// and the other way for another: their bits differed, and the last store won.
#pragma clang fp contract(on)

namespace fp4q {

// Slabs of rows that each leave one row of partial column sums.  A slab holds
// whole groups of rows that share a gate, or, where a group is longer than a
// slab or the only one, one of the k parts of one group (the last may be short,
// or empty in a short group).
struct Slabs {
    int64_t count, rows, group;  // group: rows of a group
    int64_t k;                   // slabs of a group, 0 with whole groups
    int64_t each;                // rows of a slab
    FastDiv div;                 // by k
    __device__ __forceinline__ void bounds(uint32_t i, int64_t& r0, int64_t& r1) const {
        if (k) {
            const uint32_t g = fastdiv(i, div);
            r0 = g * group + (i - g * (uint32_t)k) * each;
            r1 = min(min(r0 + each, (g + 1) * group), rows);
        } else {
            r0 = i * each;
            r1 = min(r0 + each, rows);
        }
    }
    __device__ __forceinline__ int64_t group_of(uint32_t i) const { return fastdiv(i, div); }  // of parts
};
// `groups` whole groups to a slab.
static Slabs whole_slabs(int64_t rows, int64_t group, int64_t groups) {
    Slabs s = {};
    s.rows = rows;
    s.group = group;
    s.each = groups * group;
    s.count = (rows + s.each - 1) / s.each;
    s.div = make_fastdiv(1);
    return s;
}
// Parts of groups, of about `each` rows: at most `most` slabs, or one to a group.
static Slabs part_slabs(int64_t rows, int64_t group, int64_t most, int64_t each) {
    Slabs s = {};
    s.rows = rows;
    s.group = group;
    const int64_t all = (rows + group - 1) / group;
    const int64_t k = std::max<int64_t>(1, std::min((group + each - 1) / each, most / all));
    s.each = (group + k - 1) / k;
    s.k = (group + s.each - 1) / s.each;
    s.count = all * s.k;
    s.div = make_fastdiv((uint32_t)s.k);
    return s;
}

// Which of the four column sums anybody asks for, a bit each.
__host__ __device__ inline int wanted_sums(const ResidualNormGrad& a) {
    return (a.dweight ? 1 : 0) | (a.dbias ? 2 : 0) | (a.dpost_weight || a.dgate ? 4 : 0) |
           (a.dpost_bias || (a.dgate && a.post_bias) ? 8 : 0);
}

// Sums of row r: mean_c(t xh), mean_c(t), mean_c(u nh), mean_c(u).
struct RowMeans {
    float txh, t, unh, u;
};
struct RowStats {
    float m, r, pm, pr;
    // Every row reads four numbers, those that are not there from rstd: a load
    // under a condition would have the compiler wait for more than it needs.
    __device__ __forceinline__ static RowStats of(const ResidualNormGrad& a, int64_t r) {
        const float* m = a.rms ? a.rstd : a.mean;
        const float* pm = a.post == 0 ? a.post_mean : a.rstd;
        const float* pr = a.post != kPostNone ? a.post_rstd : a.rstd;
        const RowStats s = {m[r], a.rstd[r], pm[r], pr[r]};
        return {a.rms ? 0.0f : s.m, s.r, a.post == 0 ? s.pm : 0.0f, a.post != kPostNone ? s.pr : 1.0f};
    }
};
__global__ __launch_bounds__(256) void residual_grad_rows_kernel(const ResidualNormGrad a,
                                                                 RowMeans* __restrict__ means) {
    __shared__ float red[4];
    const float n = (float)a.cols;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const RowStats st = RowStats::of(a, r);
        const int64_t g0 = r / a.gate_rows * a.ldg;
        RowMeans k = {0.0f, 0.0f, 0.0f, 0.0f};
        float s0 = 0.0f, s1 = 0.0f;
        auto first = [&](int64_t c, auto full, int left) __attribute__((always_inline)) {
            constexpr int FULL = decltype(full)::value;
            float x[8], t[8], w[8];
            load8_as<FULL>(a.xo, a.x_bf16, r * a.ldxo + c, left, 0.0f, x);
            load8_as<FULL>(a.dy, a.dy_bf16, r * a.lddy + c, left, 0.0f, t);
            load8_as<FULL>(a.weight, a.w_bf16, c, left, 1.0f, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[e] *= w[e];  // 0 past the row's end
                s0 += t[e] * ((x[e] - st.m) * st.r);
                s1 += t[e];
            }
        };
        over8(a.cols, first);
        k.txh = block_sum(s0, red) / n;
        if (!a.rms) k.t = block_sum(s1, red) / n;
        if (a.post != kPostNone) {
            s0 = s1 = 0.0f;
            auto second = [&](int64_t c, auto full, int left) __attribute__((always_inline)) {
                constexpr int FULL = decltype(full)::value;
                float x[8], t[8], w[8], s[8], b[8], p[8], g[8];
                load8_as<FULL>(a.xo, a.x_bf16, r * a.ldxo + c, left, 0.0f, x);
                load8_as<FULL>(a.dy, a.dy_bf16, r * a.lddy + c, left, 0.0f, t);
                load8_as<FULL>(a.dxo, a.x_bf16, r * a.lddxo + c, left, 0.0f, s);
                load8_as<FULL>(a.b, a.b_bf16, r * a.ldb + c, left, 0.0f, b);
                load8_as<FULL>(a.weight, a.w_bf16, c, left, 1.0f, w);
                load8_as<FULL>(a.post_weight, a.w_bf16, c, left, 1.0f, p);
                load8_as<FULL>(a.gate, a.gate_bf16, g0 + c, left, 1.0f, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = s[e] + st.r * (t[e] * w[e] - k.t - (x[e] - st.m) * st.r * k.txh);
                    const float u = FULL || e < left ? d * (a.branch_scale * p[e] * g[e]) : 0.0f;
                    s0 += u * ((b[e] - st.pm) * st.pr);
                    s1 += u;
                }
            };
            over8(a.cols, second);
            k.unh = block_sum(s0, red) / n;
            if (a.post == 0) k.u = block_sum(s1, red) / n;
        }
        if (threadIdx.x == 0) means[r] = k;
    }
}

// The same with the row in registers, two chunks of 8 elements to a lane (8 to
// 16384 columns).
template <int XB, int BB, int DB>
__global__ __launch_bounds__(1024) void residual_grad_means_kernel(const ResidualNormGrad a,
                                                                   RowMeans* __restrict__ means) {
    __shared__ float red[4 * 16];
    const int cols = (int)a.cols;
    const Place<2> pl = Place<2>::template make<1>(cols);
    int turn = 0;
    const float rn = 1.0f / (float)cols;
    const void* dxo = a.dxo ? a.dxo : a.xo;
    const int64_t lddxo = a.dxo ? a.lddxo : a.ldxo;
    const bool post = a.post != kPostNone;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const RowStats st = RowStats::of(a, r);
        Chunk<XB> x[2], sx[2];
        Chunk<DB> dy[2];
        Chunk<BB> b[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            x[k].load(a.xo, r * a.ldxo + pl.start(k));
            dy[k].load(a.dy, r * a.lddy + pl.start(k));
        }
        if (post) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                sx[k].load(dxo, r * lddxo + pl.start(k));
                b[k].load(a.b, r * a.ldb + pl.start(k));
            }
        }
        float xh[2][8], t[2][8], s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            load_vec8(a.weight, a.w_bf16, pl.start(k), 1.0f, t[k]);
            float p0 = 0.0f, p1 = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[k][e] = (x[k].at(e) - st.m) * st.r;
                t[k][e] *= dy[k].at(e);
                const float o = pl.owns(k, e) ? t[k][e] : 0.0f;
                p0 += o * xh[k][e];
                p1 += o;
            }
            s[0] += p0;
            s[1] += p1;
        }
        row_sums<1>(s, red, pl.W, turn);
        RowMeans m = {s[0] * rn, a.rms ? 0.0f : s[1] * rn, 0.0f, 0.0f};
        if (post) {
            const int64_t g0 = r / a.gate_rows * a.ldg;
            s[0] = s[1] = 0.0f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float wp[8], g[8], p0 = 0.0f, p1 = 0.0f;
                load_vec8(a.post_weight, a.w_bf16, pl.start(k), 1.0f, wp);
                load_vec8(a.gate, a.gate_bf16, g0 + pl.start(k), 1.0f, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = (a.dxo ? sx[k].at(e) : 0.0f) + st.r * (t[k][e] - m.t - xh[k][e] * m.txh);
                    const float o = pl.owns(k, e) ? d * (a.branch_scale * wp[e] * g[e]) : 0.0f;
                    p0 += o * ((b[k].at(e) - st.pm) * st.pr);
                    p1 += o;
                }
                s[0] += p0;
                s[1] += p1;
            }
            row_sums<1>(s, red, pl.W, turn);
            m.unh = s[0] * rn;
            if (a.post == 0) m.u = s[1] * rn;
        }
        if (threadIdx.x == 0) means[r] = m;
    }
}

// Outputs and column sums where the rows' means are known (rows too long for the
// registers next to their column sums, which are read twice: 4096 x 13824 with an
// fp32 stream 170 us for the means, 203 here, 14 for the join): 8 columns to a lane,
// 2048 to a workgroup, over the rows of a slab.  The sums are four rows of
// `cols` floats: dw, dc, and S1, S2 of the slab's group, or with whole groups
// dwp, dbp (the groups' dg is then written at once).  Each element is read and
// written by one lane, so that dx and db may lie on dxo and b.
template <int XB, int BB, int DB, int FULL>
__device__ __forceinline__ void tile(const ResidualNormGrad& a, const RowMeans* __restrict__ means,
                                     const Slabs& sl, float* part, int64_t c, int left) {
    float w[8], wp[8], bp[8];
    load8_as<FULL>(a.weight, a.w_bf16, c, left, 1.0f, w);
    load8_as<FULL>(a.post_weight, a.w_bf16, c, left, 1.0f, wp);
    load8_as<FULL>(a.post_bias, a.w_bf16, c, left, 0.0f, bp);
    const bool post = a.post != kPostNone;
    // operands that are not there are read where others are, and not used
    const void* dxo = a.dxo ? a.dxo : a.xo;
    const int64_t lddxo = a.dxo ? a.lddxo : a.ldxo;
    const void* b = a.b ? a.b : a.db;
    const int64_t ldb = a.b ? a.ldb : a.lddb;
    for (int64_t i = blockIdx.y; i < sl.count; i += gridDim.y) {
        int64_t r0, r1;
        sl.bounds(i, r0, r1);
        float dw[8] = {}, dc[8] = {}, s1[8] = {}, s2[8] = {}, dwp[8] = {}, dbp[8] = {};
        for (int64_t g = r0 / sl.group, r = r0; r < r1; ++g) {
            const int64_t end = min((g + 1) * sl.group, r1);
            float gate[8];
            load8_as<FULL>(a.gate, a.gate_bf16, g * a.ldg + c, left, 1.0f, gate);
#pragma unroll
            for (int e = 0; e < 8; ++e) gate[e] *= a.branch_scale;
#pragma unroll 2
            for (; r < end; ++r) {
                const RowStats st = RowStats::of(a, r);
                const RowMeans k = means[r];
                float x[8], d[8], s[8], h[8], f[8];
                load8<XB, FULL>(a.xo, r * a.ldxo + c, left, x);
                load8<DB, FULL>(a.dy, r * a.lddy + c, left, d);
                load8<BB, FULL>(b, r * ldb + c, left, h);
                load8<XB, FULL>(dxo, r * lddxo + c, left, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xh = (x[e] - st.m) * st.r;
                    dw[e] += d[e] * xh;
                    dc[e] += d[e];
                    d[e] = (a.dxo ? s[e] : 0.0f) + st.r * (d[e] * w[e] - k.t - xh * k.txh);
                    h[e] = a.b ? (h[e] - st.pm) * st.pr : 0.0f;
                    s1[e] += d[e] * h[e];
                    s2[e] += d[e];
                    f[e] = a.x_scale * d[e];
                }
                store8<XB, FULL>(a.dx, r * a.lddx + c, left, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = d[e] * (gate[e] * wp[e]);
                    f[e] = post ? st.pr * (u - k.u - h[e] * k.unh) : u;
                }
                store8<BB, FULL>(a.db, r * a.lddb + c, left, f);
            }
            if (sl.k) continue;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = a.branch_scale * (wp[e] * s1[e] + bp[e] * s2[e]);
                dwp[e] += gate[e] * s1[e];
                dbp[e] += gate[e] * s2[e];
                s1[e] = s2[e] = 0.0f;
            }
            if (a.dgate) store8<0, FULL>(a.dgate, g * a.cols + c, left, f);
        }
        if (!part) continue;
        const int64_t o = i * 4 * a.cols + c;
        store8<0, FULL>(part, o, left, dw);
        store8<0, FULL>(part, o + a.cols, left, dc);
        store8<0, FULL>(part, o + 2 * a.cols, left, sl.k ? s1 : dwp);
        store8<0, FULL>(part, o + 3 * a.cols, left, sl.k ? s2 : dbp);
    }
}
template <int XB, int BB, int DB>
__global__ __launch_bounds__(256) void residual_grad_tile_kernel(const ResidualNormGrad a,
                                                                 const RowMeans* __restrict__ means,
                                                                 const Slabs sl, float* part) {
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (c + 8 <= a.cols)
        tile<XB, BB, DB, 1>(a, means, sl, part, c, 8);
    else if (c < a.cols)
        tile<XB, BB, DB, 0>(a, means, sl, part, c, (int)(a.cols - c));
}

// Adds up the rows of partial sums: 64 columns per workgroup, one to a lane, 16
// waves over the slabs.  blockIdx.y: dw, dc, dwp, dbp, then the gate's groups:
// one at a time, gridDim.y - 4 apart, or 16 at a time where a wave adds up the
// few parts of one (kFewParts).  group0: the first workgroup's number, since a
// launch holds below 2^32 threads a side.
constexpr int64_t kJoinThreads = 1024, kJoinGroups = 1 << 21;
static_assert(kJoinGroups * kJoinThreads < (int64_t)1 << 32, "threads of a launch");
constexpr int kFewParts = 16;
// factor(i): of slab i's row
template <class F>
__device__ __forceinline__ float slab_sum(const float* p, int64_t stride, int first, int step,
                                          int64_t count, F factor) {
    float s = 0.0f;
#pragma unroll 8
    for (int64_t i = first; i < count; i += step) s += p[i * stride] * factor(i);
    return s;
}
__device__ __forceinline__ float slab_sum(const float* p, int64_t stride, int first, int step,
                                          int64_t count) {
    float s = 0.0f;
#pragma unroll 8
    for (int64_t i = first; i < count; i += step) s += p[i * stride];
    return s;
}
__global__ __launch_bounds__(kJoinThreads) void residual_grad_join_kernel(
    const ResidualNormGrad a, const float* __restrict__ part, const Slabs sl, int64_t group0) {
    __shared__ float red[2][16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t at = (group0 + blockIdx.x) * 64 + lane, c = min(at, a.cols - 1);
    const int64_t stride = 4 * a.cols;
    const float* p = part + c;
    // of all waves, in the first
    auto all16 = [&](float v, int n) __attribute__((always_inline)) {
        red[n][wave][lane] = v;
        __syncthreads();
        float s = 0.0f;
        if (wave == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s += red[n][i][lane];
        }
        return s;
    };
    if (blockIdx.y < 4) {
        const int y = blockIdx.y;
        float* out = y == 0 ? a.dweight : y == 1 ? a.dbias : y == 2 ? a.dpost_weight : a.dpost_bias;
        if (!out) return;
        p += y * a.cols;
        const bool gates = y >= 2 && sl.k && a.gate;
        float s;
        if (!gates)
            s = slab_sum(p, stride, wave, 16, sl.count);
        else if (a.gate_bf16)
            s = slab_sum(p, stride, wave, 16, sl.count,
                         [&](int64_t i) { return load1<1>(a.gate, sl.group_of(i) * a.ldg + c); });
        else
            s = slab_sum(p, stride, wave, 16, sl.count,
                         [&](int64_t i) { return load1<0>(a.gate, sl.group_of(i) * a.ldg + c); });
        s = all16(s, 0);
        if (y >= 2 && sl.k) s *= a.branch_scale;
        if (wave == 0 && at < a.cols) out[c] = s;
        return;
    }
    const float wp = a.branch_scale * vec1(a.post_weight, a.w_bf16, c, 1.0f);
    const float bp = a.branch_scale * vec1(a.post_bias, a.w_bf16, c, 0.0f);
    const int64_t groups = sl.count / sl.k;
    const bool few = sl.k <= kFewParts;
    const int64_t step = (gridDim.y - 4) * (few ? 16 : 1);
    for (int64_t g = (blockIdx.y - 4) * (few ? 16 : 1) + (few ? wave : 0); g < groups; g += step) {
        const float* q = p + (g * sl.k * 4 + 2) * a.cols;
        float s1 = slab_sum(q, stride, few ? 0 : wave, few ? 1 : 16, sl.k);
        float s2 = a.post_bias ? slab_sum(q + a.cols, stride, few ? 0 : wave, few ? 1 : 16, sl.k) : 0.0f;
        if (!few) {
            __syncthreads();
            s1 = all16(s1, 0);
            s2 = all16(s2, 1);
        }
        if ((few || wave == 0) && at < a.cols) a.dgate[g * a.cols + c] = wp * s1 + bp * s2;
    }
}

// ---- rows in registers ----

// A row is held by a team of W waves, NV chunks of 8 elements per lane, and a
// workgroup has P teams (waves of their own where W = 1 and T = 0), which take
// the slab's rows, or with whole groups its groups, in turn.
template <int GATE>
struct Walk {
    int64_t r, gend;
    bool in;
    __device__ __forceinline__ void begin(const Slabs& sl, int64_t r0, int64_t r1, int first) {
        r = r0 + (GATE ? first * sl.group : first);
        gend = GATE ? min(r + sl.group, r1) : r1;
        in = r < r1;
    }
    __device__ __forceinline__ bool last_of_group() const { return r + 1 == gend; }
    __device__ __forceinline__ void next(const Slabs& sl, int64_t r1, int step) {
        if (!GATE) {
            r += step;
        } else if (++r >= gend) {
            r += (step - 1) * sl.group;
            gend = min(r + sl.group, r1);
        }
        in = r < r1;
    }
};
// Sums of N values over the waves of a team, in every lane (row_sums of
// row_norm.h for a workgroup of several teams).
template <int MULTI, int N>
__device__ __forceinline__ void team_sums(float (&v)[N], float* red, int W, int wave0, int& turn) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
    if (!MULTI) return;
    float* r = red + turn * (N * 16);
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) r[n * 16 + (threadIdx.x >> 6)] = v[n];
    }
    __syncthreads();
    const int l = threadIdx.x & 15;
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = sum16(l < W ? r[n * 16 + wave0 + l] : 0.0f);
}

// Operands that are not there: a row of zeros, read with a row stride of 0.
__device__ const float zeros[8192] = {};

// GATE 0: the slab's rows share one row of gates, or have none; its partial
// sums are dw, dc, S1, S2.  GATE 1, 2: whole groups with a row of gates each,
// fp32 or bf16; dg is written group by group, and the partial sums are dw, dc,
// dwp, dbp (part is null where none are wanted).
template <int XB, int BB, int DB, int GATE, int T, int NV>
__global__ __launch_bounds__(T ? T : 256) void residual_grad_kernel(
    const ResidualNormGrad a, const Slabs sl, const int W, float* __restrict__ part) {
    constexpr int MULTI = T != 0;
    __shared__ __attribute__((aligned(16))) float red[4 * 16];
    __shared__ u32x4 sums[NV == 1 ? 8 * (T ? T : 256) : 1];
    const int cols = (int)a.cols;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int P = MULTI ? (int)(blockDim.x >> 6) / W : 4, team = MULTI ? wave / W : wave;
    const int wave0 = MULTI ? team * W : wave;
    const Place<NV> pl = Place<NV>::of_team(cols, MULTI ? W : 1, threadIdx.x - wave0 * 64);
    int64_t r0, r1;
    sl.bounds(blockIdx.x, r0, r1);
    // The teams meet at the row sums' barriers: all go as often as the first, the
    // last of them perhaps without a row.
    Walk<GATE> at, lead, trail;
    at.begin(sl, r0, r1, team);
    lead.begin(sl, r0, r1, 0);
    trail.begin(sl, r0, r1, P - 1);
    int turn = 0;
    const bool post = a.post != kPostNone, post_layer = a.post == 0;
    struct Row {
        Chunk<XB> x[NV], s[NV];
        Chunk<DB> d[NV];
        Chunk<BB> b[NV];
        Chunk<GATE == 2> g[GATE ? NV : 1];
        RowStats st;
    };
    Row in;
    const void* dxo = a.dxo ? a.dxo : zeros;
    const int64_t lddxo = a.dxo ? a.lddxo : 0;
    const void* b = a.b ? a.b : zeros;
    const int64_t ldb = a.b ? a.ldb : 0;
    const int64_t group0 = GATE ? r0 / sl.group : 0;
    auto gate_row = [&](int64_t row) __attribute__((always_inline)) {
        return group0 + (uint32_t)(row - r0) / (uint32_t)sl.group;
    };
    auto fetch = [&]() __attribute__((always_inline)) {
        const int64_t row = at.in ? at.r : r1 - 1;
        in.st = RowStats::of(a, row);
        const int64_t g = GATE ? gate_row(row) * a.ldg : 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            in.x[k].load_row(a.xo, row * a.ldxo, pl.start(k));
            in.d[k].load_row(a.dy, row * a.lddy, pl.start(k));
            in.s[k].load_row(dxo, row * lddxo, pl.start(k));
            in.b[k].load_row(b, row * ldb, pl.start(k));
            if (GATE) in.g[k].load_row(a.gate, g, pl.start(k));
        }
    };
    fetch();
    float w[NV][8], u[NV][8];
    float dw[NV][8] = {}, dc[NV][8] = {}, s1[NV][8] = {}, s2[NV][8] = {};
    float dpw[GATE ? NV : 1][8] = {}, dpc[GATE ? NV : 1][8] = {};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_vec8(a.weight, a.w_bf16, pl.start(k), 1.0f, w[k]);
        load_vec8(a.post_weight, a.w_bf16, pl.start(k), 1.0f, u[k]);
        if (GATE || !a.gate) {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[k][e] *= a.branch_scale;
        } else {
            float g[8];
            load_vec8(a.gate, a.gate_bf16, sl.group_of(blockIdx.x) * a.ldg + pl.start(k), 1.0f, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[k][e] *= a.branch_scale * g[e];
        }
    }
    const float rn = 1.0f / (float)cols;
    // One row of each team; `all`: every team has one.  (A store under a condition
    // leaves the compiler not knowing how many are in flight, and it would wait
    // for them with the next row's loads.)
    auto one = [&](auto all) __attribute__((always_inline)) {
        const RowStats st = in.st;
        const bool on = decltype(all)::value || at.in;
        const bool flush = GATE && on && at.last_of_group();
        const int64_t r = at.r;
        float xh[NV][8], d[NV][8], sx[NV][8], h[NV][8], g[GATE ? NV : 1][8];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[k][e] = (in.x[k].at(e) - st.m) * st.r;
                d[k][e] = in.d[k].at(e);
                sx[k][e] = in.s[k].at(e);
                h[k][e] = (in.b[k].at(e) - st.pm) * st.pr;
                if (GATE) g[k][e] = in.g[k].at(e);
            }
        // dx and db may lie on dxo, b and dy, whose last elements two waves hold:
        // all of a row has arrived before the barrier that its stores come after
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            in.d[k].arrived();
            in.s[k].arrived();
            in.b[k].arrived();
        }
        at.next(sl, r1, P);
        if (MULTI) {
            lead.next(sl, r1, P);
            trail.next(sl, r1, P);
        }
        fetch();
        float s[2] = {0.0f, 0.0f};  // of t xh, and of t
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float p0 = 0.0f, p1 = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (on) {
                    dw[k][e] += d[k][e] * xh[k][e];
                    dc[k][e] += d[k][e];
                }
                d[k][e] *= w[k][e];
                const float o = pl.owns(k, e) ? d[k][e] : 0.0f;
                p0 += o * xh[k][e];
                p1 += o;
            }
            s[0] += p0;
            s[1] += p1;
        }
        team_sums<MULTI>(s, red, W, wave0, turn);
        const float mx = s[0] * rn, mt = a.rms ? 0.0f : s[1] * rn;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) d[k][e] = sx[k][e] + st.r * (d[k][e] - mt - xh[k][e] * mx);
        if (on) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s1[k][e] += d[k][e] * h[k][e];
                    s2[k][e] += d[k][e];
                    f[e] = a.x_scale * d[k][e];
                }
                store_row<XB>(a.dx, r * a.lddx, pl.start(k), f);
            }
        }
        if (flush) {
            const int64_t at_g = gate_row(r) * a.cols;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float f[8], pc[8];
                load_vec8(a.post_bias, a.w_bf16, pl.start(k), 0.0f, pc);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[e] = u[k][e] * s1[k][e] + a.branch_scale * pc[e] * s2[k][e];  // u = bs wp here
                    dpw[k][e] += a.branch_scale * g[k][e] * s1[k][e];
                    dpc[k][e] += a.branch_scale * g[k][e] * s2[k][e];
                    s1[k][e] = s2[k][e] = 0.0f;
                }
                if (a.dgate) store_chunk<0>(a.dgate, at_g + pl.start(k), f);
            }
        }
        float mh = 0.0f, mu = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                d[k][e] *= u[k][e];
                if (GATE) d[k][e] *= g[k][e];
            }
        if (post) {
            s[0] = s[1] = 0.0f;  // of u nh, and of u
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float p0 = 0.0f, p1 = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float t = pl.owns(k, e) ? d[k][e] : 0.0f;
                    p0 += t * h[k][e];
                    p1 += t;
                }
                s[0] += p0;
                s[1] += p1;
            }
            team_sums<MULTI>(s, red, W, wave0, turn);
            mh = s[0] * rn;
            mu = post_layer ? s[1] * rn : 0.0f;
        }
        if (on) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = post ? st.pr * (d[k][e] - mu - h[k][e] * mh) : d[k][e];
                store_row<BB>(a.db, r * a.lddb, pl.start(k), f);
            }
        }
    };
    while (MULTI ? trail.in : at.in) one(std::true_type{});
    if (MULTI)
        while (lead.in) one(std::false_type{});
    if (!part) return;
    float* out = part + (int64_t)blockIdx.x * 4 * cols;
    auto sums_of = [&](int o, int k) __attribute__((always_inline)) -> float(&)[8] {
        return o == 0 ? dw[k] : o == 1 ? dc[k] : o == 2 ? (GATE ? dpw[k] : s1[k]) : (GATE ? dpc[k] : s2[k]);
    };
    const int wanted = wanted_sums(a);
    // (where two lanes hold an element, their sums of it are the same bits)
    if (NV != 1 || P == 1) {
#pragma unroll
        for (int o = 0; o < 4; ++o) {
            if (!(wanted >> o & 1)) continue;
#pragma unroll
            for (int k = 0; k < NV; ++k) store_row<0>(out, o * cols, pl.start(k), sums_of(o, k));
        }
    } else {
        // The teams' sums of the same columns are added up through LDS, four of a
        // lane's columns at a time: part j of a lane's eight is added by team j % P.
        const int threads = blockDim.x;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float* v = sums_of(j >> 1, 0) + 4 * (j & 1);
            sums[(NV == 1 ? j : 0) * threads + threadIdx.x] =
                (u32x4){as_u32(v[0]), as_u32(v[1]), as_u32(v[2]), as_u32(v[3])};
        }
        __syncthreads();
        const int lane = threadIdx.x - wave0 * 64, waves = MULTI ? W * 64 : 64;
        for (int j = team; j < 8; j += P) {
            if (!(wanted >> (j >> 1) & 1)) continue;
            float v[4] = {};
#pragma unroll 4
            for (int q = 0; q < P; ++q) {
                const u32x4 t = sums[j * threads + q * waves + lane];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += as_f32(t[e]);
            }
            *(u32x4_a4*)(out + (j >> 1) * cols + pl.start(0) + 4 * (j & 1)) =
                (u32x4){as_u32(v[0]), as_u32(v[1]), as_u32(v[2]), as_u32(v[3])};
        }
    }
    if (sl.count > 1) return;
    // the only slab: what the join kernel does
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
        float s1c = out[2 * cols + c], s2c = wanted & 8 ? out[3 * cols + c] : 0.0f;
        if (a.dweight) a.dweight[c] = out[c];
        if (a.dbias) a.dbias[c] = out[cols + c];
        if (!GATE) {
            s1c *= a.branch_scale;
            s2c *= a.branch_scale;
            if (a.dgate)
                a.dgate[c] = vec1(a.post_weight, a.w_bf16, c, 1.0f) * s1c +
                             vec1(a.post_bias, a.w_bf16, c, 0.0f) * s2c;
            if (a.gate) {
                const float g = load_as(a.gate, a.gate_bf16, c);
                s1c *= g;
                s2c *= g;
            }
        }
        if (a.dpost_weight) a.dpost_weight[c] = s1c;
        if (a.dpost_bias) a.dpost_bias[c] = s2c;
    }
}

constexpr int64_t kAnyGrid = 1 << 16;
constexpr int64_t kGridY = 1 << 15;

// How rows are held: by waves of their own (T = 0) or by teams of W waves in a
// workgroup of at most T threads, nv chunks per lane; nv = 0: the rows' means
// first, then tiles.  whole: slabs of whole groups of a gate's rows.
struct GradShape {
    int T, nv, W, threads;
};
static GradShape grad_shape(int64_t cols, bool whole) {
    const int waves = (int)((cols + 511) / 512);
    if (cols < 8 || cols > 8192 || (whole && cols > 6144)) return {0, 0, 0, 256};
    if (cols <= 512) return {0, 1, 1, 256};
    if (cols > 6144) return {512, 2, (waves + 1) / 2, 64 * ((waves + 1) / 2)};
    const int T = whole && waves <= 8 ? 512 : 768;
    return {T, 1, waves, 64 * waves * (T / 64 / waves)};
}
// As many slabs as 256 compute units hold workgroups of (12 waves to a unit, 8
// where a row of gates comes with every row), of a few rows and more: 4 and 8
// rows take 7.4 and 9.9 us at 256 x 1112 fp32 (32 and 64 workgroups), 20.4 and
// 18.9 with the join at 1000 x 2048 bf16, where the partial sums count.  Up to 4
// rows to a team are one slab, which needs no join.
//
// Groups that are shorter than such a slab lie in slabs of whole groups, a group
// to a team.  Where that leaves a quarter of the teams and more without a group,
// the groups may be slabs of their own, whose rows all teams share: whichever has
// the fewer rows one after another, a slab's beginning and end counted as 3 of
// them (4 with waves on their own).  16384 x 1024 bf16 with 8, 12, 24, 32, 40 and
// 64 rows to a group: whole 53, 62, 59, 65, 79 and 117 us, on their own 87, 68, 52,
// 49, 50 and 44; 49152 x 512 with 16, 24, 32, 40 and 64: 72, 65, 66, 77, 106 and
// 88, 78, 71, 74, 65.
static Slabs grad_slabs(int64_t rows, int64_t cols, int64_t gate_rows) {
    struct Limits {
        int64_t teams, most, each;  // teams of a workgroup, slabs, rows of a slab
        bool one;                   // one slab for all rows
    };
    const auto limits = [&](const GradShape& sh, int waves) {
        Limits l;
        l.teams = sh.nv ? sh.threads / 64 / sh.W : 1;
        l.most = sh.nv ? 256 * std::max(1, waves * 64 / sh.threads) : 256;
        l.each = std::max<int64_t>(sh.nv && sh.T ? (rows <= 512 ? 4 : 8) : 16, (rows + l.most - 1) / l.most);
        l.one = sh.nv && rows <= 4 * l.teams;
        return l;
    };
    const Limits p = limits(grad_shape(cols, false), 12);
    if (gate_rows >= rows) return part_slabs(rows, rows, p.one ? 1 : p.most, p.one ? rows : p.each);
    const GradShape sh = grad_shape(cols, true);
    const Limits w = limits(sh, 8);
    const int64_t all = (rows + gate_rows - 1) / gate_rows;
    if (w.one) return whole_slabs(rows, gate_rows, all);
    const Slabs parts = part_slabs(rows, gate_rows, p.most, p.each);
    if (gate_rows > p.each) return parts;
    const int64_t fit = w.each < rows ? w.each / gate_rows : all;
    if (sh.nv == 0) return whole_slabs(rows, gate_rows, fit);
    const int64_t groups = std::max(fit, (all + w.most - 1) / w.most);
    const int64_t turns = (groups + w.teams - 1) / w.teams;
    const int64_t shared = (parts.count + p.most - 1) / p.most *
                           ((gate_rows + p.teams - 1) / p.teams + (sh.T ? 3 : 4));
    const bool idle = 4 * groups <= 3 * turns * w.teams;
    return idle && shared < turns * gate_rows ? parts : whole_slabs(rows, gate_rows, groups);
}

size_t residual_norm_grad_workspace_bytes(int64_t rows, int64_t cols, int64_t gate_rows) {
    const Slabs sl = grad_slabs(rows, cols, gate_rows);
    const bool whole = gate_rows < rows && !sl.k;
    const size_t means = grad_shape(cols, whole).nv == 0 ? (size_t)rows * sizeof(RowMeans) : 0;
    return means + (size_t)sl.count * 4 * (size_t)cols * sizeof(float);
}

template <int XB, int BB, int DB, int GATE>
static void go_rows(const GradShape sh, const ResidualNormGrad& a, const Slabs& sl, float* part,
                    hipStream_t s) {
#define FP4Q_GO(T_, NV_)                                                                        \
    if (sh.T == T_ && sh.nv == NV_)                                                             \
    FP4Q_LAUNCH((residual_grad_kernel<XB, BB, DB, GATE, T_, NV_>), dim3((unsigned)sl.count),    \
                dim3((unsigned)sh.threads), 0, s, a, sl, sh.W, part)
    FP4Q_GO(0, 1);
    FP4Q_GO(768, 1);
    if constexpr (GATE == 0) {
        FP4Q_GO(512, 2);
    } else {
        FP4Q_GO(512, 1);
    }
#undef FP4Q_GO
}
template <int XB, int BB, int DB>
static void go_gate(const GradShape sh, const ResidualNormGrad& a, const Slabs& sl, RowMeans* means,
                    float* part, hipStream_t s) {
    if (sh.nv == 0) {
        if (a.cols >= 8 && a.cols <= 16384)
            FP4Q_LAUNCH((residual_grad_means_kernel<XB, BB, DB>),
                        dim3((unsigned)std::min<int64_t>(a.rows, 1024)),
                        dim3(64 * (unsigned)((a.cols + 1023) / 1024)), 0, s, a, means);
        else
            FP4Q_LAUNCH(residual_grad_rows_kernel, dim3((unsigned)std::min(a.rows, kAnyGrid)), dim3(256), 0,
                        s, a, means);
        const int64_t tiles = (a.cols + 2047) / 2048;
        FP4Q_LAUNCH((residual_grad_tile_kernel<XB, BB, DB>),
                    dim3((unsigned)tiles, (unsigned)std::min(sl.count, kGridY)), dim3(256), 0, s, a,
                    means, sl, part);
    } else if (sl.k) {
        go_rows<XB, BB, DB, 0>(sh, a, sl, part, s);
    } else if (!a.gate_bf16) {
        go_rows<XB, BB, DB, 1>(sh, a, sl, part, s);
    } else {
        go_rows<XB, BB, DB, 2>(sh, a, sl, part, s);
    }
}
template <int XB, int BB>
static void go_dy(const GradShape sh, const ResidualNormGrad& a, const Slabs& sl, RowMeans* means,
                  float* part, hipStream_t s) {
    a.dy_bf16 ? go_gate<XB, BB, 1>(sh, a, sl, means, part, s)
              : go_gate<XB, BB, 0>(sh, a, sl, means, part, s);
}

hipError_t launch_residual_norm_grad(const ResidualNormGrad& a, void* ws, hipStream_t s) {
    const Slabs sl = grad_slabs(a.rows, a.cols, a.gate_rows);
    const GradShape sh = grad_shape(a.cols, a.gate_rows < a.rows && !sl.k);
    const bool sums = wanted_sums(a) != 0;
    RowMeans* means = (RowMeans*)ws;
    float* part = sh.nv == 0 ? (float*)(means + a.rows) : (float*)ws;
    float* p = sums ? part : nullptr;
    if (a.x_bf16)
        a.b_bf16 ? go_dy<1, 1>(sh, a, sl, means, p, s) : go_dy<1, 0>(sh, a, sl, means, p, s);
    else
        a.b_bf16 ? go_dy<0, 1>(sh, a, sl, means, p, s) : go_dy<0, 0>(sh, a, sl, means, p, s);
    hipError_t e = hipGetLastError();
    if (sums && (sh.nv == 0 || sl.count > 1)) {
        int64_t gates = a.dgate && sl.k ? sl.count / sl.k : 0;
        if (sl.k <= kFewParts) gates = (gates + 15) / 16;
        gates = std::min(gates, kGridY);
        const int64_t groups = (a.cols + 63) / 64;
        for (int64_t g = 0; g < groups && e == hipSuccess; g += kJoinGroups) {
            FP4Q_LAUNCH(residual_grad_join_kernel,
                        dim3((unsigned)std::min(groups - g, kJoinGroups), (unsigned)(4 + gates)),
                        dim3((unsigned)kJoinThreads), 0, s, a, part, sl, g);
            e = hipGetLastError();
        }
    }
    return e;
}

}  // namespace fp4q
