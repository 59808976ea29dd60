// The norm of many gradients taken as one vector, the factor that clips it, and
// the clipping.
//
//   norm = sqrt(sum g^2), or max |g|       scale = min(1, max_norm / (norm + eps))
//   g = g scale
//
// Squares and their sums are in 64 bits: the square of an fp32 value is exact
// there and neither overflows nor underflows, so the norm is the exact one
// rounded to fp32 (off by at most one step), whatever the order of the sum.
#include <algorithm>
#include <cmath>

#include "../../include/libfp4q.h"
#include "fp4q_device.h"
#include "fp4q_internal.h"

namespace fp4q {

constexpr int kTensors = 192;            // descriptors per launch: 4 KB of kernel arguments
constexpr int64_t kChunk = 16384;        // elements per workgroup
constexpr int64_t kMaxGroups = 1 << 22;  // workgroups per launch: 2^30 threads

struct Tensors {
    void* p[kTensors];
    int64_t n[kTensors];        // elements; the top bit: bf16
    uint32_t first[kTensors];   // first workgroup
    int count;
};
static_assert(sizeof(Tensors) <= 4096 - 64, "kernel arguments");
constexpr int64_t kBf16Bit = (int64_t)1 << 62;

// The workgroup's tensor (the last that starts at or before it, found by all
// lanes at once) and its elements [i0, i1).
struct Piece {
    void* p;
    int64_t i0, i1;
    bool bf16;
};
__device__ __forceinline__ Piece piece_of(const Tensors& t, uint32_t group) {
    const int l = threadIdx.x & 63;
    int k = 0;
#pragma unroll
    for (int j = 0; j < kTensors; j += 64) {
        const int i = j + l;
        const bool below = i < t.count && (i == 0 || t.first[i] <= group);
        k += __popcll(__ballot(below));
    }
    k -= 1;
    Piece q;
    const int64_t n = t.n[k];
    q.p = t.p[k];
    q.bf16 = (n & kBf16Bit) != 0;
    q.i0 = (int64_t)(group - t.first[k]) * kChunk;
    q.i1 = min(q.i0 + kChunk, n & ~kBf16Bit);
    return q;
}
__device__ __forceinline__ float element(const Piece& q, int64_t i) {
    return q.bf16 ? as_f32((uint32_t)((const uint16_t*)q.p)[i] << 16) : ((const float*)q.p)[i];
}

__global__ __launch_bounds__(256) void grad_norm_kernel(const Tensors t, int largest,
                                                        double* __restrict__ part) {
    __shared__ double red[256];
    const Piece q = piece_of(t, blockIdx.x);
    double s = 0.0;
    uint32_t top = 0;
    for (int64_t i = q.i0 + threadIdx.x; i < q.i1; i += 256) {
        const float g = element(q, i);
        top = max(top, as_u32(g) & 0x7FFFFFFFu);
        s += (double)g * (double)g;
    }
    red[threadIdx.x] = largest ? (double)top : s;
    __syncthreads();
    for (int k = 128; k; k >>= 1) {
        if ((int)threadIdx.x < k)
            red[threadIdx.x] = largest ? fmax(red[threadIdx.x], red[threadIdx.x + k])
                                       : red[threadIdx.x] + red[threadIdx.x + k];
        __syncthreads();
    }
    if (threadIdx.x == 0) part[blockIdx.x] = red[0];
}

__global__ __launch_bounds__(1024) void grad_norm_join_kernel(const double* __restrict__ part,
                                                              int64_t n, int largest,
                                                              double max_norm, double eps,
                                                              float* __restrict__ norm,
                                                              float* __restrict__ scale) {
    __shared__ double red[1024];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 1024) s = largest ? fmax(s, part[i]) : s + part[i];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int k = 512; k; k >>= 1) {
        if ((int)threadIdx.x < k)
            red[threadIdx.x] = largest ? fmax(red[threadIdx.x], red[threadIdx.x + k])
                                       : red[threadIdx.x] + red[threadIdx.x + k];
        __syncthreads();
    }
    if (threadIdx.x) return;
    // the largest magnitude's bits, which order magnitudes as whole numbers do,
    // infinity above the finite ones and NaN above it
    const double v = largest ? (double)as_f32((uint32_t)red[0]) : sqrt(red[0]);
    if (norm) *norm = (float)v;
    if (scale) {
        const double d = v + eps, c = max_norm / d;
        *scale = c >= 1.0 || d == 0.0 ? 1.0f : (float)c;  // a NaN stays one
    }
}

__global__ __launch_bounds__(256) void grad_scale_kernel(const Tensors t,
                                                         const float* __restrict__ scale) {
    const Piece q = piece_of(t, blockIdx.x);
    const float f = *scale;
    for (int64_t i = q.i0 + threadIdx.x; i < q.i1; i += 256) {
        const float g = element(q, i) * f;
        if (q.bf16)
            ((uint16_t*)q.p)[i] = (uint16_t)f32_to_bf16_bits(g);
        else
            ((float*)q.p)[i] = g;
    }
}

static int64_t groups_of(const fp4q_tensor_t& t) { return (t.numel + kChunk - 1) / kChunk; }

// Calls launch(tensors, groups, groups of earlier launches) until all are done.
template <class F>
static hipError_t for_tensors(const fp4q_tensor_t* t, int n, F launch) {
    Tensors a;
    int64_t done = 0, before = 0;  // chunks of tensor i that earlier launches took; of all
    for (int i = 0; i < n;) {
        int64_t groups = 0;
        a.count = 0;
        while (i < n && a.count < kTensors && groups < kMaxGroups) {
            const int64_t left = groups_of(t[i]) - done;
            if (left > 0) {
                const int64_t take = std::min(left, kMaxGroups - groups);
                a.p[a.count] = t[i].data;
                a.n[a.count] = t[i].numel | (t[i].dtype == FP4Q_BF16 ? kBf16Bit : 0);
                // of a tensor that an earlier launch began, `first` wraps below
                // zero; group - first is the chunk all the same
                a.first[a.count++] = (uint32_t)(uint64_t)(groups - done);
                groups += take;
                done += take;
                if (take < left) break;
            }
            ++i;
            done = 0;
        }
        if (a.count == 0) break;
        launch(a, groups, before);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        before += groups;
    }
    return hipSuccess;
}

size_t grad_norm_workspace_bytes(const fp4q_tensor_t* t, int n) {
    int64_t groups = 0;
    for (int i = 0; i < n; ++i) groups += groups_of(t[i]);
    return (size_t)std::max<int64_t>(groups, 2) * sizeof(double);
}

hipError_t launch_grad_norm(const fp4q_tensor_t* t, int n, bool largest, double max_norm, double eps,
                            float* norm, float* scale, void* ws, hipStream_t s) {
    double* part = (double*)ws;
    int64_t groups = 0;
    const hipError_t e = for_tensors(t, n, [&](const Tensors& a, int64_t now, int64_t before) {
        FP4Q_LAUNCH(grad_norm_kernel, dim3((unsigned)now), dim3(256), 0, s, a, (int)largest, part + before);
        groups = before + now;
    });
    if (e != hipSuccess) return e;
    FP4Q_LAUNCH(grad_norm_join_kernel, dim3(1), dim3(1024), 0, s, part, groups, (int)largest, max_norm,
                eps, norm, scale);
    return hipGetLastError();
}

hipError_t launch_grad_scale(const fp4q_tensor_t* t, int n, const float* scale, hipStream_t s) {
    return for_tensors(t, n, [&](const Tensors& a, int64_t now, int64_t) {
        FP4Q_LAUNCH(grad_scale_kernel, dim3((unsigned)now), dim3(256), 0, s, a, scale);
    });
}

}  // namespace fp4q
