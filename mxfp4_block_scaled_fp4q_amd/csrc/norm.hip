// Layer norm and RMS norm of the rows of a matrix, forward and backward.
//
//   mean_r = sum_c x / C (0 for RMS)      rstd_r = (sum_c (x - mean)^2 / C + eps)^-1/2
//   xh = (x - mean) rstd                  y = xh w + b
//   t = dy w      dx = rstd (t - mean_c(t) [layer norm only] - xh mean_c(t xh))
//   dw = sum_r dy xh                      db = sum_r dy
//
// Both directions are bound by memory: the forward pass reads x and writes y,
// the backward pass reads x and dy and writes dx, each once.  So a row stays
// in registers from its load to its last use, in chunks of 8 elements per
// lane; the sums run over lanes, and over waves through LDS, in fp32, and the
// squares are summed around the mean that is already known.  A workgroup
// walks over rows and loads the next row (short rows: the next two) before it
// works on the present one; the weight and bias stay in registers, and in the
// backward pass the lane's partial column sums do too, so dw and db cost no
// second read of x and dy: each workgroup leaves one row of partial sums,
// which a second, small kernel adds up.  No atomics: the order of every sum is
// fixed by the sizes.
//
// A row's last chunk, where 8 does not divide C, is read 8 elements wide from
// C - 8; its first elements belong to the chunk before it and are left out of
// the sums.  Vector accesses need only the elements' alignment.
#include <algorithm>

#include "fp4q_device.h"
#include "fp4q_internal.h"

namespace fp4q {

template <int BF16T>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    if (BF16T) return as_f32((uint32_t)((const uint16_t*)p)[i] << 16);
    return ((const float*)p)[i];
}
template <int BF16T>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
    if (BF16T)
        ((uint16_t*)p)[i] = (uint16_t)f32_to_bf16_bits(v);
    else
        ((float*)p)[i] = v;
}
// A weight or bias element; `none` where the caller passed no vector.
__device__ __forceinline__ float vec1(const void* p, int bf16, int64_t i, float none) {
    if (!p) return none;
    return bf16 ? load1<1>(p, i) : load1<0>(p, i);
}

// 8 consecutive elements as they lie in memory.
template <int BF16T>
struct Chunk {
    u32x4 v[BF16T ? 1 : 2];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        if (BF16T) {
            v[0] = *(const u32x4_a2*)((const uint16_t*)p + i);
        } else {
            v[0] = *(const u32x4_a4*)((const float*)p + i);
            v[BF16T ? 0 : 1] = *(const u32x4_a4*)((const float*)p + i + 4);
        }
    }
    __device__ __forceinline__ float at(int e) const {
        if (BF16T) {
            const uint32_t w = v[0][e >> 1];
            return (e & 1) ? bf16_hi(w) : bf16_lo(w);
        }
        return as_f32(v[BF16T ? 0 : e >> 2][e & 3]);
    }
};
template <int BF16T>
__device__ __forceinline__ void store_chunk(void* p, int64_t i, const float (&f)[8]) {
    if (BF16T) {
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bf16x2_t q = {(__bf16)f[2 * e], (__bf16)f[2 * e + 1]};  // v_cvt_pk_bf16_f32
            v[e] = __builtin_bit_cast(uint32_t, q);
        }
        *(u32x4_a2*)((uint16_t*)p + i) = v;
    } else {
        float* q = (float*)p + i;
        *(u32x4_a4*)q = (u32x4){as_u32(f[0]), as_u32(f[1]), as_u32(f[2]), as_u32(f[3])};
        *(u32x4_a4*)(q + 4) = (u32x4){as_u32(f[4]), as_u32(f[5]), as_u32(f[6]), as_u32(f[7])};
    }
}
// All of them, or elements skip .. 7.
template <int BF16T>
__device__ __forceinline__ void store_own(void* p, int64_t i, const float (&f)[8], int skip) {
    if (skip == 0) {
        store_chunk<BF16T>(p, i, f);
    } else {
#pragma unroll
        for (int e = 1; e < 8; ++e)
            if (e >= skip) store1<BF16T>(p, i + e, f[e]);
    }
}
__device__ __forceinline__ void load_vec8(const void* p, int bf16, int64_t i, float none,
                                          float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = none;
    } else if (bf16) {
        Chunk<1> c;
        c.load(p, i);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = c.at(e);
    } else {
        Chunk<0> c;
        c.load(p, i);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = c.at(e);
    }
}

// Sums over 16 lanes (DPP steps, as in group_max_u32) and over the wave (then
// the four rows of 16 by gfx950's lane swaps), in every lane.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + as_f32((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_u32(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float sum16(float v) {
    return dpp_add<0x140>(dpp_add<0x141>(dpp_add<0x4E>(dpp_add<0xB1>(v))));
}
__device__ __forceinline__ float rows_sum(float v) {  // over the four rows, lane by lane
    const auto a = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
    v = as_f32(a[0]) + as_f32(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
    return as_f32(b[0]) + as_f32(b[1]);
}
__device__ __forceinline__ float wave_sum(float v) { return rows_sum(sum16(v)); }

// Sums of N values over the waves that share a row (W of them, at most 16), in
// every lane.  `red` holds two sets of N * 16 floats that take turns, so one
// barrier is enough: a set is written again only after the next sum's barrier.
template <int MULTI, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int W, int& turn) {
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
    for (int n = 0; n < N; ++n) v[n] = sum16(l < W ? r[n * 16 + l] : 0.0f);
}

// A row is held by one wave (MULTI = 0; 256 threads work on four rows) or by
// all W waves of its workgroup, NV chunks per lane.  The last chunk begins at
// `tail` in this lane and its first `skip` elements are another lane's; a lane
// past the row's end holds that row's last chunk again, with skip = 8.
//
// Every lane loads and stores all its chunks, and past the last row loads that
// row again: a load or store under a condition would leave the compiler not
// knowing how many are in flight, and it would wait for the rows ahead too.
// Elements that two lanes hold are stored by both, with the same bits.
template <int NV>
struct Place {
    int W, t, step, tail, skip;
    template <int MULTI>
    __device__ __forceinline__ static Place make(int cols) {
        Place p;
        p.W = MULTI ? (int)(blockDim.x >> 6) : 1;
        p.t = (MULTI ? (int)threadIdx.x : (int)(threadIdx.x & 63)) * 8;
        p.step = p.W * 512;
        const int c0 = (NV - 1) * p.step + p.t;
        p.tail = min(c0, cols - 8);
        p.skip = c0 < cols ? c0 - p.tail : 8;
        return p;
    }
    __device__ __forceinline__ int start(int k) const { return k < NV - 1 ? k * step + t : tail; }
    __device__ __forceinline__ bool owns(int k, int e) const { return k < NV - 1 || e >= skip; }
};

// First row of this wave's (or workgroup's) walk, a scalar.
template <int MULTI>
__device__ __forceinline__ int64_t first_row() {
    if (MULTI) return blockIdx.x;
    return (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
}

template <int XB, int YB, int MULTI, int NV>
__global__ __launch_bounds__(MULTI ? 1024 : 256) void norm_kernel(
    const void* __restrict__ x, int64_t rows, int cols, int64_t ldx, const void* __restrict__ w,
    const void* __restrict__ b, int wb, float eps, int rms, void* __restrict__ y, int64_t ldy,
    float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float red[MULTI ? 2 * 16 : 1];
    const Place<NV> pl = Place<NV>::template make<MULTI>(cols);
    const int64_t step = MULTI ? gridDim.x : gridDim.x * 4;
    int64_t r = first_row<MULTI>();
    if (r >= rows) return;  // whole waves, and whole workgroups where they share a row
    int turn = 0;
    constexpr int AHEAD = NV == 1 ? 2 : 1;  // rows in flight
    Chunk<XB> xr[AHEAD][NV];
    auto fetch = [&](int64_t row, Chunk<XB>(&xn)[NV]) __attribute__((always_inline)) {
        row = min(row, rows - 1);
#pragma unroll
        for (int k = 0; k < NV; ++k) xn[k].load(x, row * ldx + pl.start(k));
    };
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) fetch(r + a * step, xr[a]);
    float wv[NV][8], bv[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        load_vec8(w, wb, pl.start(k), 1.0f, wv[k]);
        load_vec8(b, wb, pl.start(k), 0.0f, bv[k]);
    }
    const float n = (float)cols;
    float mu = 0.0f, rs = 0.0f;
    // the statistics of a row are stored ahead of the next row's loads
    auto stats = [&](int64_t row) __attribute__((always_inline)) {
        if (pl.t) return;
        if (mean && !rms) mean[row] = mu;
        if (rstd) rstd[row] = rs;
    };
    int64_t last = -1;
    auto one = [&](int64_t r, Chunk<XB>(&xn)[NV]) __attribute__((always_inline)) {
        float xf[NV][8];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) xf[k][e] = xn[k].at(e);
        if (last >= 0) stats(last);
        last = r;
        fetch(r + AHEAD * step, xn);
        if (!rms) {
            float s[1] = {0.0f};
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float p = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) p += pl.owns(k, e) ? xf[k][e] : 0.0f;
                s[0] += p;
            }
            row_sums<MULTI>(s, red, pl.W, turn);
            mu = s[0] / n;
        }
        float q[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float p = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = xf[k][e] -= mu;
                p += pl.owns(k, e) ? d * d : 0.0f;
            }
            q[0] += p;
        }
        row_sums<MULTI>(q, red, pl.W, turn);
        rs = 1.0f / sqrtf(q[0] / n + eps);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = (xf[k][e] * rs) * wv[k][e] + bv[k][e];
            store_chunk<YB>(y, r * ldy + pl.start(k), f);
        }
    };
    for (; r < rows; r += AHEAD * step) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
            if (a == 0 || r + a * step < rows) one(r + a * step, xr[a]);
    }
    stats(last);
}

// dw and db (or either, or neither, null) get this workgroup's column sums:
// row blockIdx.x, part_stride floats long, of the partial sums.
template <int XB, int DB, int MULTI, int NV>
__global__ __launch_bounds__(MULTI ? 1024 : 256) void norm_grad_kernel(
    const void* dy, int64_t lddy, const void* x, int64_t rows, int cols, int64_t ldx,
    const void* __restrict__ w, int wb, const float* __restrict__ mean,
    const float* __restrict__ rstd, int rms, void* dx, int64_t lddx, float* __restrict__ dw,
    float* __restrict__ db, int64_t part_stride) {
    // two chunks leave 1024 threads no registers for the column sums, which
    // then lie in LDS, 16 floats per lane
    constexpr bool kLds = MULTI && NV == 2;
    __shared__ __attribute__((aligned(16))) float red[MULTI ? 4 * 16 : 4 * 512];
    __shared__ u32x4 sums[kLds ? 2 * 2 * NV * 1024 : 1];
    const Place<NV> pl = Place<NV>::template make<MULTI>(cols);
    const int64_t step = MULTI ? gridDim.x : gridDim.x * 4;
    int64_t r = first_row<MULTI>();
    int turn = 0;
    constexpr int AHEAD = NV == 1 ? 2 : 1;
    struct Row {
        Chunk<XB> x[NV];
        Chunk<DB> d[NV];
        float mu, rs;
    };
    Row in[AHEAD];
    float wv[NV][8], aw[NV][8] = {}, ab[NV][8] = {};
    // this lane's sums of chunk k in LDS, half h of dw's (o = 0) or db's eight
    auto slot = [&](int o, int k, int h) __attribute__((always_inline)) -> u32x4& {
        return sums[((o * NV + k) * 2 + h) * 1024 + threadIdx.x];
    };
    if (kLds) {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) slot(i >> 2, (i >> 1) & 1, i & 1) = (u32x4){0u, 0u, 0u, 0u};
    }
    auto fetch = [&](int64_t row, Row& n) __attribute__((always_inline)) {
        row = min(row, rows - 1);
        n.mu = rms ? 0.0f : mean[row];
        n.rs = rstd[row];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            n.x[k].load(x, row * ldx + pl.start(k));
            n.d[k].load(dy, row * lddy + pl.start(k));
        }
    };
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) fetch(r + a * step, in[a]);
#pragma unroll
    for (int k = 0; k < NV; ++k)
        load_vec8(w, wb, pl.start(k), 1.0f, wv[k]);
    const float n = (float)cols;
    auto one = [&](int64_t r, Row& now) __attribute__((always_inline)) {
        const float mu = now.mu, rs = now.rs;
        float xh[NV][8], d[NV][8];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[k][e] = (now.x[k].at(e) - mu) * rs;
                d[k][e] = now.d[k].at(e);
            }
        fetch(r + AHEAD * step, now);
        float s[2] = {0.0f, 0.0f};  // of t xh, and of t
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float p0 = 0.0f, p1 = 0.0f;
            float own[8];  // zero for elements that are another lane's: no sum holds them twice
#pragma unroll
            for (int e = 0; e < 8; ++e) own[e] = pl.owns(k, e) ? d[k][e] : 0.0f;
            if (kLds) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    u32x4 vw = slot(0, k, h), vb = slot(1, k, h);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        vw[i] = as_u32(as_f32(vw[i]) + own[4 * h + i] * xh[k][4 * h + i]);
                        vb[i] = as_u32(as_f32(vb[i]) + own[4 * h + i]);
                    }
                    slot(0, k, h) = vw;
                    slot(1, k, h) = vb;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!kLds) {
                    aw[k][e] += own[e] * xh[k][e];
                    ab[k][e] += own[e];
                }
                own[e] *= wv[k][e];
                p0 += own[e] * xh[k][e];
                p1 += own[e];
                d[k][e] *= wv[k][e];
            }
            s[0] += p0;
            s[1] += p1;
        }
        row_sums<MULTI>(s, red, pl.W, turn);
        const float mx = s[0] / n, mt = rms ? 0.0f : s[1] / n;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = rs * (d[k][e] - mt - xh[k][e] * mx);
            store_chunk<XB>(dx, r * lddx + pl.start(k), f);
        }
    };
    for (; r < rows; r += AHEAD * step) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
            if (a == 0 || r + a * step < rows) one(r + a * step, in[a]);
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        float* out = o == 0 ? dw : db;
        if (!out) continue;
        out += blockIdx.x * part_stride;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float(&a)[8] = o == 0 ? aw[k] : ab[k];
            if (kLds) {
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = as_f32(slot(o, k, e >> 2)[e & 3]);
            }
            const int skip = k < NV - 1 ? 0 : pl.skip, c = pl.start(k);
            if (MULTI) {
                store_own<0>(out, c, a, skip);
                continue;
            }
            // the four waves hold the same 512 columns of different rows
            __syncthreads();
            float* mine = red + (threadIdx.x >> 6) * 512;
            if (skip == 0) {
                *(u32x4*)(mine + pl.t) =
                    (u32x4){as_u32(a[0]), as_u32(a[1]), as_u32(a[2]), as_u32(a[3])};
                *(u32x4*)(mine + pl.t + 4) =
                    (u32x4){as_u32(a[4]), as_u32(a[5]), as_u32(a[6]), as_u32(a[7])};
            } else {
#pragma unroll
                for (int e = 1; e < 8; ++e)
                    if (e >= skip) mine[c - k * 512 + e] = a[e];
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = h * 256 + threadIdx.x;
                if (k * 512 + i < cols)
                    out[k * 512 + i] = (red[i] + red[512 + i]) + (red[1024 + i] + red[1536 + i]);
            }
        }
    }
}

// Adds up the rows of partial sums: 16 columns per workgroup, 64 groups of 16
// lanes over the rows, so that few loads follow each other.  group0: the first
// workgroup's number, since a launch holds below 2^32 threads.
constexpr int64_t kJoinGroups = 1 << 21;
__global__ __launch_bounds__(1024) void norm_grad_join_kernel(const float* __restrict__ part,
                                                              int64_t cols, int slabs,
                                                              float* __restrict__ dw,
                                                              float* __restrict__ db,
                                                              int64_t group0) {
    __shared__ float red[16][16];
    float* out = blockIdx.y == 0 ? dw : db;
    if (!out) return;
    const int l = threadIdx.x & 15, wave = threadIdx.x >> 6;
    const int64_t c = (group0 + blockIdx.x) * 16 + l;
    float s = 0.0f;
    if (c < cols) {
        const float* p = part + blockIdx.y * cols + c;
#pragma unroll 8
        for (int i = threadIdx.x >> 4; i < slabs; i += 64) s += p[(int64_t)i * 2 * cols];
    }
    s = rows_sum(s);
    if ((threadIdx.x & 63) < 16) red[wave][l] = s;
    __syncthreads();
    if (wave) return;
    const int r = threadIdx.x >> 4;
    s = rows_sum((red[r][l] + red[4 + r][l]) + (red[8 + r][l] + red[12 + r][l]));
    if (threadIdx.x < 16 && c < cols) out[c] = s;
}

// Rows below 8 columns, or too long for the registers: 256 threads walk over
// the row once per sum, element by element.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

template <int XB, int YB>
__global__ __launch_bounds__(256) void norm_any_kernel(
    const void* __restrict__ x, int64_t rows, int64_t cols, int64_t ldx, const void* __restrict__ w,
    const void* __restrict__ b, int wb, float eps, int rms, void* __restrict__ y, int64_t ldy,
    float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float red[4];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        float mu = 0.0f;
        if (!rms) {
            float s = 0.0f;
            for (int64_t c = threadIdx.x; c < cols; c += 256) s += load1<XB>(x, r * ldx + c);
            mu = block_sum(s, red) / (float)cols;
        }
        float q = 0.0f;
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            const float d = load1<XB>(x, r * ldx + c) - mu;
            q += d * d;
        }
        const float rs = 1.0f / sqrtf(block_sum(q, red) / (float)cols + eps);
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            const float xh = (load1<XB>(x, r * ldx + c) - mu) * rs;
            store1<YB>(y, r * ldy + c, xh * vec1(w, wb, c, 1.0f) + vec1(b, wb, c, 0.0f));
        }
        if (threadIdx.x == 0) {
            if (mean && !rms) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

template <int XB, int DB>
__global__ __launch_bounds__(256) void norm_grad_any_kernel(
    const void* dy, int64_t lddy, const void* x, int64_t rows, int64_t cols, int64_t ldx,
    const void* __restrict__ w, int wb, const float* __restrict__ mean,
    const float* __restrict__ rstd, int rms, void* dx, int64_t lddx) {
    __shared__ float red[4];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const float mu = rms ? 0.0f : mean[r], rs = rstd[r];
        float st = 0.0f, sx = 0.0f;
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            const float t = load1<DB>(dy, r * lddy + c) * vec1(w, wb, c, 1.0f);
            st += t;
            sx += t * ((load1<XB>(x, r * ldx + c) - mu) * rs);
        }
        const float mx = block_sum(sx, red) / (float)cols;
        const float mt = rms ? 0.0f : block_sum(st, red) / (float)cols;
        for (int64_t c = threadIdx.x; c < cols; c += 256) {
            const float t = load1<DB>(dy, r * lddy + c) * vec1(w, wb, c, 1.0f);
            const float xh = (load1<XB>(x, r * ldx + c) - mu) * rs;
            store1<XB>(dx, r * lddx + c, rs * (t - mt - xh * mx));
        }
    }
}

// Column sums over a slab of rows each (before dx is written, which may lie
// on x or dy).
template <int XB, int DB>
__global__ __launch_bounds__(256) void norm_grad_cols_kernel(
    const void* __restrict__ dy, int64_t lddy, const void* __restrict__ x, int64_t rows,
    int64_t cols, int64_t ldx, const float* __restrict__ mean, const float* __restrict__ rstd,
    int rms, int64_t slab, float* __restrict__ part) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= cols) return;
    const int64_t r0 = (int64_t)blockIdx.y * slab, r1 = min(r0 + slab, rows);
    float sw = 0.0f, sb = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float d = load1<DB>(dy, r * lddy + c);
        sb += d;
        sw += d * ((load1<XB>(x, r * ldx + c) - (rms ? 0.0f : mean[r])) * rstd[r]);
    }
    part[((int64_t)blockIdx.y * 2) * cols + c] = sw;
    part[((int64_t)blockIdx.y * 2 + 1) * cols + c] = sb;
}

// How rows of `cols` elements are held: by one wave or by all waves of their
// workgroup, in nv chunks per lane (nv = 0: not in registers).  One wave needs
// no barrier, but has only enough loads in flight where there are rows for all
// of them.
struct NormShape {
    bool multi;
    int nv, threads;
};
static NormShape norm_shape(int64_t rows, int64_t cols) {
    if (cols < 8 || cols > 16384) return {false, 0, 256};
    if (cols <= 512) return {false, 1, 256};
    if (cols <= 1024 && rows > 1024) return {false, 2, 256};
    const int nv = cols <= 8192 ? 1 : 2;
    return {true, nv, 64 * (int)((cols + nv * 512 - 1) / (nv * 512))};
}
constexpr int64_t kAnyGrid = 1 << 16;

// Workgroups of a walk over the rows: what 256 compute units hold of them at
// `waves` waves each, and at least `min_rows` rows to a workgroup (or to each
// of its four waves).  Forward, 16, 24 and 32 waves: 16384 x 5120 bf16 77, 66
// and 72 us (ten waves per row: 16 is one workgroup), fp32 125, 129 and 151,
// 16384 x 8192 bf16 101, 98 and 96, 8192 x 2048 15.8, 14.8 and 14.7.  Backward:
// 16384 x 5120 bf16 98, 105 and 112, fp32 184, 195 and 203, 16384 x 8192 152,
// 153 and 164.  There a walk costs a latency per row and each workgroup a row
// of partial sums to write and join: 2, 4, 8, 16 rows take 7.3, 7.2, 8.9, 13.3
// us at 400 x 1024, 18.0, 15.3, 13.6, 17.8 at 1999 x 1111 fp32, 9.8, 8.6, 9.3,
// 12.2 at 4000 x 300 fp32 (four rows at a time) and 26.3, 26.2, 26.2, 25.3 at
// 8192 x 2048.  The width hardly moves the best: 19.0, 18.9, 18.4, 23.7 at
// 1024 x 5120, 19.3, 19.2, 18.7, 24.1 with a row more, 21.9, 21.7, 21.7, 25.5 at
// 2040 x 5120, 30.3 to 30.6 at 4096 x 5120 and 19.6, 18.4, 19.5, 28.2 at 500 x
// 8192, so the rule asks for the rows alone (its step past 1024 rows, 256 to 129
// workgroups at 5120 columns, costs nothing).
constexpr int kNormWaves = 24, kGradWaves = 16;
static int norm_groups(const NormShape& sh, int64_t rows, int waves, int min_rows) {
    const int64_t per = (int64_t)min_rows * (sh.multi ? 1 : 4);
    return (int)std::min<int64_t>(256 * (waves * 64 / sh.threads), (rows + per - 1) / per);
}
static int norm_slabs(int64_t rows, int64_t cols) {
    const NormShape sh = norm_shape(rows, cols);
    if (sh.nv == 0) return (int)std::min<int64_t>(128, (rows + 63) / 64);
    const int min_rows = rows <= 1024 ? 2 : sh.multi ? (rows <= 4096 ? 8 : 16) : rows <= 12000 ? 4 : 8;
    return norm_groups(sh, rows, kGradWaves, min_rows);
}

size_t norm_grad_workspace_bytes(int64_t rows, int64_t cols) {
    return (size_t)norm_slabs(rows, cols) * 2 * (size_t)cols * 4;
}

template <int XB, int YB>
static void go_norm(const NormShape sh, const void* x, int64_t rows, int64_t cols, int64_t ldx,
                    const void* w, const void* b, int wb, float eps, int rms, void* y, int64_t ldy,
                    float* mean, float* rstd, hipStream_t s) {
#define FP4Q_GO(MULTI, NV)                                                                        \
    if (sh.multi == (bool)MULTI && sh.nv == NV)                                                   \
    FP4Q_LAUNCH((norm_kernel<XB, YB, MULTI, NV>), dim3((unsigned)norm_groups(sh, rows, kNormWaves, 1)),   \
                dim3((unsigned)sh.threads), 0, s, x, rows, (int)cols, ldx, w, b, wb, eps, rms, y, \
                ldy, mean, rstd)
    FP4Q_GO(0, 1);
    FP4Q_GO(0, 2);
    FP4Q_GO(1, 1);
    FP4Q_GO(1, 2);
#undef FP4Q_GO
    if (sh.nv == 0)
        FP4Q_LAUNCH((norm_any_kernel<XB, YB>), dim3((unsigned)std::min(rows, kAnyGrid)), dim3(256), 0,
                    s, x, rows, cols, ldx, w, b, wb, eps, rms, y, ldy, mean, rstd);
}

hipError_t launch_norm(const void* x, int xdtype, int64_t rows, int64_t cols, int64_t ldx,
                       const void* w, const void* b, int wdtype, float eps, bool rms, void* y,
                       int ydtype, int64_t ldy, float* mean, float* rstd, hipStream_t s) {
    const NormShape sh = norm_shape(rows, cols);
#define FP4Q_GO(XB, YB) \
    go_norm<XB, YB>(sh, x, rows, cols, ldx, w, b, wdtype, eps, (int)rms, y, ldy, mean, rstd, s)
    if (xdtype == BF16) {
        if (ydtype == BF16) FP4Q_GO(1, 1); else FP4Q_GO(1, 0);
    } else {
        if (ydtype == BF16) FP4Q_GO(0, 1); else FP4Q_GO(0, 0);
    }
#undef FP4Q_GO
    return hipGetLastError();
}

template <int XB, int DB>
static void go_grad(const NormShape sh, const void* dy, int64_t lddy, const void* x, int64_t rows,
                    int64_t cols, int64_t ldx, const void* w, int wb, const float* mean,
                    const float* rstd, int rms, void* dx, int64_t lddx, float* dw, float* db,
                    void* ws, hipStream_t s) {
    const int slabs = norm_slabs(rows, cols);
    float* part = (float*)ws;
    if (sh.nv == 0) {
        const int64_t slab = (rows + slabs - 1) / slabs;
        if (dw || db)
            FP4Q_LAUNCH((norm_grad_cols_kernel<XB, DB>),
                        dim3((unsigned)((cols + 255) / 256), (unsigned)slabs), dim3(256), 0, s, dy,
                        lddy, x, rows, cols, ldx, mean, rstd, rms, slab, part);
        FP4Q_LAUNCH((norm_grad_any_kernel<XB, DB>), dim3((unsigned)std::min(rows, kAnyGrid)),
                    dim3(256), 0, s, dy, lddy, x, rows, cols, ldx, w, wb, mean, rstd, rms, dx, lddx);
    } else {
        // one workgroup's sums are the result; otherwise they are joined below
        float* pw = !dw ? nullptr : slabs == 1 ? dw : part;
        float* pb = !db ? nullptr : slabs == 1 ? db : part + cols;
#define FP4Q_GO(MULTI, NV)                                                                       \
    if (sh.multi == (bool)MULTI && sh.nv == NV)                                                  \
    FP4Q_LAUNCH((norm_grad_kernel<XB, DB, MULTI, NV>), dim3((unsigned)slabs),                    \
                dim3((unsigned)sh.threads), 0, s, dy, lddy, x, rows, (int)cols, ldx, w, wb, mean, \
                rstd, rms, dx, lddx, pw, pb, 2 * cols)
        FP4Q_GO(0, 1);
        FP4Q_GO(0, 2);
        FP4Q_GO(1, 1);
        FP4Q_GO(1, 2);
#undef FP4Q_GO
        if (slabs == 1) return;
    }
    const int64_t groups = dw || db ? (cols + 15) / 16 : 0;
    for (int64_t g = 0; g < groups; g += kJoinGroups)
        FP4Q_LAUNCH(norm_grad_join_kernel, dim3((unsigned)std::min(groups - g, kJoinGroups), 2),
                    dim3(1024), 0, s, part, cols, slabs, dw, db, g);
}

hipError_t launch_norm_grad(const void* dy, int dydtype, int64_t lddy, const void* x, int xdtype,
                            int64_t rows, int64_t cols, int64_t ldx, const void* w, int wdtype,
                            const float* mean, const float* rstd, bool rms, void* dx, int64_t lddx,
                            float* dw, float* db, void* ws, hipStream_t s) {
    const NormShape sh = norm_shape(rows, cols);
#define FP4Q_GO(XB, DB)                                                                       \
    go_grad<XB, DB>(sh, dy, lddy, x, rows, cols, ldx, w, wdtype, mean, rstd, (int)rms, dx, lddx, \
                    dw, db, ws, s)
    if (xdtype == BF16) {
        if (dydtype == BF16) FP4Q_GO(1, 1); else FP4Q_GO(1, 0);
    } else {
        if (dydtype == BF16) FP4Q_GO(0, 1); else FP4Q_GO(0, 0);
    }
#undef FP4Q_GO
    return hipGetLastError();
}

}  // namespace fp4q
