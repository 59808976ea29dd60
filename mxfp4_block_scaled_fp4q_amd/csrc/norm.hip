// Layer norm and RMS norm of the rows of a matrix, forward and backward.
//
//   mean_r = sum_c x / C (0 for RMS)      rstd_r = (sum_c (x - mean)^2 / C + eps)^-1/2
//   xh = (x - mean) rstd                  y = xh w + b
//   t = dy w      dx = rstd (t - mean_c(t) [layer norm only] - xh mean_c(t xh))
//   dw = sum_r dy xh                      db = sum_r dy
//
// All sums are held in fp32 in a fixed order: no atomics, so results do not
// change from run to run.
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

// Sum over the 256 threads of the workgroup, in every thread.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

template <int XB, int YB>
__global__ __launch_bounds__(256) void norm_kernel(const void* __restrict__ x, int64_t cols,
                                                   int64_t ldx, const void* __restrict__ w,
                                                   const void* __restrict__ b, int wb, float eps,
                                                   int rms, void* __restrict__ y, int64_t ldy,
                                                   float* __restrict__ mean,
                                                   float* __restrict__ rstd) {
    __shared__ float red[4];
    const int64_t r = blockIdx.x;
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

template <int XB, int DB>
__global__ __launch_bounds__(256) void norm_grad_kernel(
    const void* __restrict__ dy, int64_t lddy, const void* __restrict__ x, int64_t cols,
    int64_t ldx, const void* __restrict__ w, int wb, const float* __restrict__ mean,
    const float* __restrict__ rstd, int rms, void* __restrict__ dx, int64_t lddx) {
    __shared__ float red[4];
    const int64_t r = blockIdx.x;
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

// Column sums over a slab of rows each, then over the slabs.
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

__global__ __launch_bounds__(256) void norm_grad_join_kernel(const float* __restrict__ part,
                                                             int64_t cols, int slabs,
                                                             float* __restrict__ dw,
                                                             float* __restrict__ db) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= cols) return;
    float sw = 0.0f, sb = 0.0f;
    for (int i = 0; i < slabs; ++i) {
        sw += part[((int64_t)i * 2) * cols + c];
        sb += part[((int64_t)i * 2 + 1) * cols + c];
    }
    if (dw) dw[c] = sw;
    if (db) db[c] = sb;
}

static int norm_slabs(int64_t rows) { return (int)std::min<int64_t>(128, (rows + 63) / 64); }

size_t norm_grad_workspace_bytes(int64_t rows, int64_t cols) {
    return (size_t)norm_slabs(rows) * 2 * (size_t)cols * 4;
}

hipError_t launch_norm(const void* x, int xdtype, int64_t rows, int64_t cols, int64_t ldx,
                       const void* w, const void* b, int wdtype, float eps, bool rms, void* y,
                       int ydtype, int64_t ldy, float* mean, float* rstd, hipStream_t s) {
#define FP4Q_GO(XB, YB)                                                                      \
    FP4Q_LAUNCH((norm_kernel<XB, YB>), dim3((unsigned)rows), dim3(256), 0, s, x, cols, ldx, w, b, \
                wdtype, eps, (int)rms, y, ldy, mean, rstd)
    if (xdtype == BF16) {
        if (ydtype == BF16) FP4Q_GO(1, 1); else FP4Q_GO(1, 0);
    } else {
        if (ydtype == BF16) FP4Q_GO(0, 1); else FP4Q_GO(0, 0);
    }
#undef FP4Q_GO
    return hipGetLastError();
}

hipError_t launch_norm_grad(const void* dy, int dydtype, int64_t lddy, const void* x, int xdtype,
                            int64_t rows, int64_t cols, int64_t ldx, const void* w, int wdtype,
                            const float* mean, const float* rstd, bool rms, void* dx, int64_t lddx,
                            float* dw, float* db, void* ws, hipStream_t s) {
    const int slabs = norm_slabs(rows);
    const int64_t slab = (rows + slabs - 1) / slabs;
    const unsigned cb = (unsigned)((cols + 255) / 256);
#define FP4Q_GO(XB, DB)                                                                       \
    do {                                                                                      \
        if (dw || db)                                                                         \
            FP4Q_LAUNCH((norm_grad_cols_kernel<XB, DB>), dim3(cb, (unsigned)slabs), dim3(256), 0, \
                        s, dy, lddy, x, rows, cols, ldx, mean, rstd, (int)rms, slab, (float*)ws); \
        FP4Q_LAUNCH((norm_grad_kernel<XB, DB>), dim3((unsigned)rows), dim3(256), 0, s, dy, lddy, x, \
                    cols, ldx, w, wdtype, mean, rstd, (int)rms, dx, lddx);                    \
    } while (0)
    if (xdtype == BF16) {
        if (dydtype == BF16) FP4Q_GO(1, 1); else FP4Q_GO(1, 0);
    } else {
        if (dydtype == BF16) FP4Q_GO(0, 1); else FP4Q_GO(0, 0);
    }
#undef FP4Q_GO
    if (dw || db)
        FP4Q_LAUNCH(norm_grad_join_kernel, dim3(cb), dim3(256), 0, s, (const float*)ws, cols, slabs,
                    dw, db);
    return hipGetLastError();
}

}  // namespace fp4q
