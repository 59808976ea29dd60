// The norm of many gradients taken as one vector, the factor that clips it, and
// the clipping.
//
//   norm = sqrt(sum g^2), or max |g|       scale = min(1, max_norm / (norm + eps))
//   g = g scale
//
// Squares and their sums are in 64 bits: the square of an fp32 value is exact
// there and neither overflows nor underflows.  An element's way into the sum has 26
// additions in its workgroup, 23 in the join and one more for every 4096 partial
// sums, so with p of them the norm is within (50 + p / 4096) 2^-54 of itself (212M
// elements 2^-48, 2^44, the most that a call takes, 2^-36) before it is rounded to
// fp32.  That costs no time: the gradients are read at 5.8 TB/s in fp32 (173M
// elements 119 us) and 5.7 in bf16 (212M 75 us), as the largest magnitude, which
// needs no 64-bit arithmetic, is (75).
//
// A workgroup takes 16384 elements, 8 loads of 16 bytes per lane in flight (4 of
// them 118 and 74 us; chunks of 32768 elements 118 and 76), and leaves one partial
// sum, which a second kernel joins, or, in the clipping, every workgroup where
// they are few.  The clipping reads and writes the gradients once more: 212M
// mostly bf16 elements 250 us (116 + 5 + 125), 5.1 TB/s over the three passes;
// the last elements first, which the norm has left in the caches, 245, but 28.6
// for 28.0 where all of them are there.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/libfp4q.h"
#include "fp4q_device.h"
#include "fp4q_internal.h"

namespace fp4q {

constexpr int64_t kChunk = 16384;        // elements per workgroup
constexpr int64_t kMaxGroups = 1 << 22;  // workgroups per launch: 2^30 threads

// Where a launch's tensors stand: in the kernel arguments, up to N of them, or in
// device memory, with the tensor of every chunk (40, 150, 300 and 1000 tensors of
// up to 9000 elements: 8.6, 8.9, 13.5 and 32 us a norm against 7.4, 7.5, 7.6 and
// 8.5).
constexpr int64_t kBf16Bit = (int64_t)1 << 62;  // in a number of elements: they are bf16
template <int N>
struct Tensors {
    void* p[N];
    int64_t n[N];
    uint32_t first[N];  // first workgroup
    int count;
};
constexpr int kFew = 64, kMany = 192;
static_assert(sizeof(Tensors<kMany>) <= 4096 - 64, "kernel arguments");
struct Desc {
    void* p;
    int64_t n;
    uint64_t first;
};
struct Table {
    const Desc* d;
    const uint32_t* owner;
    uint32_t group0;  // of the launch's first workgroup
};

// A workgroup's (or wave's) part of a tensor: elements [i0, i1).
struct Piece {
    void* p;
    int64_t i0, i1;
    bool bf16;
};
__device__ __forceinline__ Piece make_piece(void* p, int64_t n, int64_t i0, int64_t chunk) {
    return {p, i0, min(i0 + chunk, n & ~kBf16Bit), (n & kBf16Bit) != 0};
}
// The tensor of `group`: the last that starts at or before it, found by all lanes
// at once.
template <int64_t CHUNK, int N>
__device__ __forceinline__ Piece piece_of(const Tensors<N>& t, uint32_t group) {
    const int l = threadIdx.x & 63;
    int k = -1;
#pragma unroll
    for (int j = 0; j < N; j += 64) {
        const int i = j + l;
        const bool below = i < t.count && (i == 0 || t.first[i] <= group);
        k += __popcll(__ballot(below));
    }
    return make_piece(t.p[k], t.n[k], (int64_t)(group - t.first[k]) * CHUNK, CHUNK);
}
template <int64_t CHUNK>
__device__ __forceinline__ Piece piece_of(const Table& t, uint32_t group) {
    group += t.group0;
    const Desc d = t.d[t.owner[group]];
    return make_piece(d.p, d.n, (int64_t)(group - (uint32_t)d.first) * CHUNK, CHUNK);
}
// 16 bytes of a gradient at any element, and its values.
template <int B16>
struct Vec {
    static constexpr int N = B16 ? 8 : 4;
    u32x4 w;
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        w = B16 ? *global<const u32x4_a2>((const uint16_t*)p + i)
                : *global<const u32x4_a4>((const float*)p + i);
    }
    __device__ __forceinline__ void store(void* p, int64_t i) const {
        if (B16)
            *global<u32x4_a2>((uint16_t*)p + i) = w;
        else
            *global<u32x4_a4>((float*)p + i) = w;
    }
    __device__ __forceinline__ float at(int e) const {
        if (B16) return (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
        return as_f32(w[e & 3]);
    }
};
template <int B16>
__device__ __forceinline__ float element(const void* p, int64_t i) {
    return B16 ? as_f32((uint32_t)global<const uint16_t>(p)[i] << 16) : global<const float>(p)[i];
}

// Sums of squares, or the bits of the largest magnitude, which order
// magnitudes as whole numbers do, infinity above the finite ones and NaN above
// it.  Four sums take turns, so that few additions follow each other.
template <int MAX>
struct Total {
    double s[4];
    uint32_t top;
    __device__ __forceinline__ Total() : s{0.0, 0.0, 0.0, 0.0}, top(0) {}
    __device__ __forceinline__ void add(float g, int k) {
        if (MAX)
            top = max(top, as_u32(g) & 0x7FFFFFFFu);
        else
            s[k & 3] = __builtin_fma((double)g, (double)g, s[k & 3]);
    }
};

// Of all lanes of a workgroup, in thread 0.
template <int MAX>
__device__ __forceinline__ double total_of(double v, double* red) {
#pragma unroll
    for (int k = 32; k; k >>= 1) {
        const double o = __shfl_xor(v, k);
        v = MAX ? fmax(v, o) : v + o;
    }
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x) return 0.0;
    v = red[0];
    for (int k = 1; k < (int)(blockDim.x >> 6); ++k) v = MAX ? fmax(v, red[k]) : v + red[k];
    return v;
}

constexpr int kThreads = 256, kAhead = 8;  // loads of a lane in flight

// f(vector, its first element) over the whole vectors of a piece that T lanes
// share, kAhead of a lane's at a time, f1(element's place) over the rest.
template <int T, int B16, class F, class F1>
__device__ __forceinline__ void over(const Piece& q, F f, F1 f1) {
    constexpr int N = Vec<B16>::N, SPAN = T * N;
    const int n = (int)(q.i1 - q.i0), t = threadIdx.x & (T - 1);
    int i = t * N;
    for (; i - t * N + kAhead * SPAN <= n; i += kAhead * SPAN) {
        Vec<B16> v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) v[k].load(q.p, q.i0 + i + k * SPAN);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) f(v[k], q.i0 + i + k * SPAN);
    }
    if (i + N <= n) {
        Vec<B16> v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k * SPAN + N <= n) v[k].load(q.p, q.i0 + i + k * SPAN);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k * SPAN + N <= n) f(v[k], q.i0 + i + k * SPAN);
    }
    const int rest = (n & ~(N - 1)) + t;
    if (rest < n) f1(q.i0 + rest);
}

template <int T, int MAX, int B16>
__device__ __forceinline__ void add_piece(const Piece& q, Total<MAX>& t) {
    over<T, B16>(
        q,
        [&](const Vec<B16>& v, int64_t) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < Vec<B16>::N; ++e) t.add(v.at(e), e);
        },
        [&](int64_t i) __attribute__((always_inline)) { t.add(element<B16>(q.p, i), 0); });
}
template <int MAX>
__device__ __forceinline__ double value_of(const Total<MAX>& t) {
    return MAX ? (double)t.top : (t.s[0] + t.s[1]) + (t.s[2] + t.s[3]);
}

template <int MAX, class SOURCE>
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const SOURCE t, double* __restrict__ part) {
    __shared__ double red[kThreads / 64];
    const Piece q = piece_of<kChunk>(t, blockIdx.x);
    Total<MAX> t0;
    q.bf16 ? add_piece<kThreads, MAX, 1>(q, t0) : add_piece<kThreads, MAX, 0>(q, t0);
    const double v = total_of<MAX>(value_of(t0), red);
    if (threadIdx.x == 0) part[blockIdx.x] = v;
}

struct Clip {
    double max_norm, eps;
    float *norm, *scale;
};
// The factor for a sum of squares (or the bits of the largest magnitude), and
// with `write` what the caller wants of both.
template <int MAX>
__device__ __forceinline__ float finish(double all, const Clip& c, bool write) {
    const double v = MAX ? (double)as_f32((uint32_t)all) : sqrt(all);
    const double d = v + c.eps, q = c.max_norm / d;
    const float f = q >= 1.0 || d == 0.0 ? 1.0f : (float)q;  // a NaN stays one
    if (write) {
        if (c.norm) *c.norm = (float)v;
        if (c.scale) *c.scale = f;
    }
    return f;
}

template <int MAX>
__global__ __launch_bounds__(1024) void grad_norm_join_kernel(const double* __restrict__ part, int64_t n,
                                                              const Clip c) {
    __shared__ double red[16];
    double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 2
    for (int64_t i = threadIdx.x; i < n; i += 4096) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const double v = i + k * 1024 < n ? part[i + k * 1024] : 0.0;
            s[k] = MAX ? fmax(s[k], v) : s[k] + v;
        }
    }
    const double all = total_of<MAX>(MAX ? fmax(fmax(s[0], s[1]), fmax(s[2], s[3]))
                                         : (s[0] + s[1]) + (s[2] + s[3]), red);
    if (threadIdx.x == 0) finish<MAX>(all, c, true);
}

template <int T, int B16>
__device__ __forceinline__ void scale_piece(const Piece& q, float f) {
    over<T, B16>(
        q,
        [&](Vec<B16> v, int64_t i) __attribute__((always_inline)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (B16) {
                    const bf16x2_t p = {(__bf16)(v.at(2 * k) * f), (__bf16)(v.at(2 * k + 1) * f)};
                    v.w[k] = __builtin_bit_cast(uint32_t, p);
                } else {
                    v.w[k] = as_u32(v.at(k) * f);
                }
            }
            v.store(q.p, i);
        },
        [&](int64_t i) __attribute__((always_inline)) {
            const float g = element<B16>(q.p, i) * f;
            if (B16)
                global<uint16_t>(q.p)[i] = (uint16_t)f32_to_bf16_bits(g);
            else
                global<float>(q.p)[i] = g;
        });
}
template <class SOURCE>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const SOURCE t,
                                                              const float* __restrict__ scale) {
    const float f = *scale;
    if (f == 1.0f) return;
    const Piece q = piece_of<kChunk>(t, blockIdx.x);
    q.bf16 ? scale_piece<kThreads, 1>(q, f) : scale_piece<kThreads, 0>(q, f);
}

// The same where the factor is still to be made of up to kFewParts partial sums:
// every workgroup adds them up, in the join kernel's order, which costs a launch
// less (40 tensors of up to 5000 elements 16.5 -> 10.5 us a call).
constexpr int kFewParts = 1024;
template <int MAX, class SOURCE>
__global__ __launch_bounds__(kThreads) void grad_clip_kernel(const SOURCE t,
                                                             const double* __restrict__ part, int n,
                                                             const Clip c) {
    __shared__ double red[16];
    double v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = k * kThreads + threadIdx.x;
        v[k] = i < n ? part[i] : 0.0;
    }
#pragma unroll
    for (int m = 32; m; m >>= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const double o = __shfl_xor(v[k], m);
            v[k] = MAX ? fmax(v[k], o) : v[k] + o;
        }
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) red[4 * k + (threadIdx.x >> 6)] = v[k];
    }
    __syncthreads();
    double all = red[0];
#pragma unroll
    for (int k = 1; k < 16; ++k) all = MAX ? fmax(all, red[k]) : all + red[k];
    const float f = finish<MAX>(all, c, blockIdx.x == 0 && threadIdx.x == 0);
    if (f == 1.0f) return;
    const Piece q = piece_of<kChunk>(t, blockIdx.x);
    q.bf16 ? scale_piece<kThreads, 1>(q, f) : scale_piece<kThreads, 0>(q, f);
}

// Norm, factor and clipping of a few small tensors in one launch: the waves of one
// workgroup take pieces of 1024 elements in turn.  30 tensors of up to 1000
// elements 9.3 -> 6.8 us a call, clipped 9.0 -> 7.0; at 64 pieces the norm takes
// as long, the clipping, which goes over them twice, 9.6 (one limit for both, so
// that both make the same norm).
constexpr int64_t kSmallChunk = 1024, kSmallPieces = 64;
template <int MAX, int CLIP>
__global__ __launch_bounds__(1024) void grad_small_kernel(const Tensors<kFew> t, int pieces,
                                                          const Clip c) {
    __shared__ double red[16];
    __shared__ float factor;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Total<MAX> sum;
    for (int i = wave; i < pieces; i += 16) {
        const Piece q = piece_of<kSmallChunk>(t, i);
        q.bf16 ? add_piece<64, MAX, 1>(q, sum) : add_piece<64, MAX, 0>(q, sum);
    }
    const double all = total_of<MAX>(value_of(sum), red);
    if (threadIdx.x == 0) factor = finish<MAX>(all, c, true);
    if (!CLIP) return;
    __syncthreads();
    const float f = factor;
    if (f == 1.0f) return;
    for (int i = wave; i < pieces; i += 16) {
        const Piece q = piece_of<kSmallChunk>(t, i);
        q.bf16 ? scale_piece<64, 1>(q, f) : scale_piece<64, 0>(q, f);
    }
}

static int64_t groups_of(const fp4q_tensor_t& t, int64_t chunk = kChunk) {
    return (t.numel + chunk - 1) / chunk;
}
static bool is_small(const fp4q_tensor_t* t, int n) {
    int64_t pieces = 0;
    for (int i = 0; i < n && pieces <= kSmallPieces; ++i) pieces += groups_of(t[i], kSmallChunk);
    return pieces <= kSmallPieces;
}

// Calls launch(tensors, groups, groups of earlier launches) until all are done.
template <int N, class F>
static hipError_t for_args(const fp4q_tensor_t* t, int n, F launch, int64_t chunk = kChunk) {
    Tensors<N> a;
    int64_t done = 0, before = 0;  // chunks of tensor i that earlier launches took; of all
    for (int i = 0; i < n;) {
        int64_t groups = 0;
        a.count = 0;
        while (i < n && a.count < N && groups < kMaxGroups) {
            const int64_t left = groups_of(t[i], chunk) - done;
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
static int64_t all_groups(const fp4q_tensor_t* t, int n) {
    int64_t groups = 0;
    for (int i = 0; i < n; ++i) groups += groups_of(t[i]);
    return groups;
}
template <class F>
static hipError_t for_tensors(const fp4q_tensor_t* t, int n, const void* table, F launch) {
    if (!table) return n <= kFew ? for_args<kFew>(t, n, launch) : for_args<kMany>(t, n, launch);
    const int64_t groups = all_groups(t, n);
    for (int64_t g = 0; g < groups; g += kMaxGroups) {
        const Table a = {(const Desc*)table, (const uint32_t*)((const Desc*)table + n), (uint32_t)g};
        launch(a, std::min(groups - g, kMaxGroups), g);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

size_t grad_table_bytes(const fp4q_tensor_t* t, int n) {
    return (size_t)n * sizeof(Desc) + (size_t)all_groups(t, n) * 4;
}
void grad_table(const fp4q_tensor_t* t, int n, void* table) {
    Desc* d = (Desc*)table;
    uint32_t* owner = (uint32_t*)(d + n);
    uint64_t groups = 0;
    for (int i = 0; i < n; ++i) {
        d[i] = {t[i].data, t[i].numel | (t[i].dtype == FP4Q_BF16 ? kBf16Bit : 0), groups};
        for (int64_t k = groups_of(t[i]); k > 0; --k) owner[groups++] = (uint32_t)i;
    }
}

size_t grad_norm_workspace_bytes(const fp4q_tensor_t* t, int n) {
    return (size_t)(all_groups(t, n) + 2) * sizeof(double);  // a factor, and partial sums
}

// Partial sums of all tensors; their number in *groups.
static hipError_t launch_parts(const fp4q_tensor_t* t, int n, const void* table, bool largest,
                               double* part, int64_t* groups, hipStream_t s) {
    *groups = 0;
    return for_tensors(t, n, table, [&](const auto& a, int64_t now, int64_t before) {
        using S = std::decay_t<decltype(a)>;
        const dim3 grid((unsigned)now), block(kThreads);
        if (largest)
            FP4Q_LAUNCH((grad_norm_kernel<1, S>), grid, block, 0, s, a, part + before);
        else
            FP4Q_LAUNCH((grad_norm_kernel<0, S>), grid, block, 0, s, a, part + before);
        *groups = before + now;
    });
}
static hipError_t launch_join(const double* part, int64_t groups, bool largest, const Clip& c,
                              hipStream_t s) {
    if (largest)
        FP4Q_LAUNCH(grad_norm_join_kernel<1>, dim3(1), dim3(1024), 0, s, part, groups, c);
    else
        FP4Q_LAUNCH(grad_norm_join_kernel<0>, dim3(1), dim3(1024), 0, s, part, groups, c);
    return hipGetLastError();
}

static hipError_t launch_small(const fp4q_tensor_t* t, int n, bool largest, bool clip, const Clip& c,
                               hipStream_t s) {
    bool done = false;
    const auto go = [&](const Tensors<kFew>& a, int64_t now, int64_t) {
        done = true;
        if (largest && clip)
            FP4Q_LAUNCH((grad_small_kernel<1, 1>), dim3(1), dim3(1024), 0, s, a, (int)now, c);
        else if (largest)
            FP4Q_LAUNCH((grad_small_kernel<1, 0>), dim3(1), dim3(1024), 0, s, a, (int)now, c);
        else if (clip)
            FP4Q_LAUNCH((grad_small_kernel<0, 1>), dim3(1), dim3(1024), 0, s, a, (int)now, c);
        else
            FP4Q_LAUNCH((grad_small_kernel<0, 0>), dim3(1), dim3(1024), 0, s, a, (int)now, c);
    };
    static_assert(kSmallPieces <= kFew, "each piece may be a tensor");
    const hipError_t e = for_args<kFew>(t, n, go, kSmallChunk);
    return e != hipSuccess || done ? e : launch_join(nullptr, 0, largest, c, s);  // nothing: norm 0
}

hipError_t launch_grad_norm(const fp4q_tensor_t* t, int n, const void* table, bool largest,
                            double max_norm, double eps, float* norm, float* scale, void* ws,
                            hipStream_t s) {
    const Clip c = {max_norm, eps, norm, scale};
    if (is_small(t, n)) return launch_small(t, n, largest, false, c, s);
    int64_t groups;
    const hipError_t e = launch_parts(t, n, table, largest, (double*)ws, &groups, s);
    return e != hipSuccess ? e : launch_join((double*)ws, groups, largest, c, s);
}

hipError_t launch_grad_scale(const fp4q_tensor_t* t, int n, const void* table, const float* scale,
                             hipStream_t s) {
    return for_tensors(t, n, table, [&](const auto& a, int64_t now, int64_t) {
        using S = std::decay_t<decltype(a)>;
        FP4Q_LAUNCH(grad_scale_kernel<S>, dim3((unsigned)now), dim3(kThreads), 0, s, a, scale);
    });
}

hipError_t launch_grad_clip(const fp4q_tensor_t* t, int n, const void* table, bool largest,
                            double max_norm, double eps, float* norm, void* ws, hipStream_t s) {
    if (is_small(t, n))
        return launch_small(t, n, largest, true, {max_norm, eps, norm, nullptr}, s);
    double* part = (double*)ws + 2;  // behind the factor
    float* scale = (float*)ws;
    int64_t groups;
    hipError_t e = launch_parts(t, n, table, largest, part, &groups, s);
    if (e != hipSuccess) return e;
    if (groups > kFewParts) {
        e = launch_join(part, groups, largest, {max_norm, eps, norm, scale}, s);
        return e != hipSuccess ? e : launch_grad_scale(t, n, table, scale, s);
    }
    // (only the first launch writes the norm)
    return for_tensors(t, n, table, [&](const auto& a, int64_t now, int64_t before) {
        using S = std::decay_t<decltype(a)>;
        const dim3 grid((unsigned)now), block(kThreads);
        const Clip c = {max_norm, eps, before ? nullptr : norm, nullptr};
        if (largest)
            FP4Q_LAUNCH((grad_clip_kernel<1, S>), grid, block, 0, s, a, part, (int)groups, c);
        else
            FP4Q_LAUNCH((grad_clip_kernel<0, S>), grid, block, 0, s, a, part, (int)groups, c);
    });
}

}  // namespace fp4q
