// Pieces that the row norms share (norm.hip, residual_norm.hip): vector accesses
// of a row's elements, sums over its lanes and waves, and where a row's elements
// lie in the registers of the lanes that hold it.
#pragma once
#include <type_traits>

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

// The same where the type is known at run time only.
__device__ __forceinline__ float load_as(const void* p, int bf16, int64_t i) {
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
    // From element `first` of p, the same for the wave, and this lane's `c`: an
    // address of a scalar and a 32-bit part.
    __device__ __forceinline__ void load_row(const void* p, int64_t first, int c) {
        const char* q = (const char*)p + first * (BF16T ? 2 : 4) + (uint32_t)c * (BF16T ? 2u : 4u);
        load(q, 0);
    }
    // Waits here for the load.
    __device__ __forceinline__ void arrived() const {
        asm volatile("" ::"v"(v[0][0]));
        if (!BF16T) asm volatile("" ::"v"(v[BF16T ? 0 : 1][0]));
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
// From element `first` of p, the same for the wave, and this lane's `c`.
template <int BF16T>
__device__ __forceinline__ void store_row(void* p, int64_t first, int c, const float (&f)[8]) {
    store_chunk<BF16T>((char*)p + first * (BF16T ? 2 : 4) + (uint32_t)c * (BF16T ? 2u : 4u), 0, f);
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

// Any width: a lane takes 8 elements at a time.  FULL: all 8 are there, otherwise
// the first `left`.
template <int B16, int FULL>
__device__ __forceinline__ void load8(const void* p, int64_t i, int left, float (&f)[8]) {
    if (FULL) {
        Chunk<B16> c;
        c.load(p, i);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = c.at(e);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = e < left ? load1<B16>(p, i + e) : 0.0f;
    }
}
template <int B16, int FULL>
__device__ __forceinline__ void store8(void* p, int64_t i, int left, const float (&f)[8]) {
    if (FULL) {
        store_chunk<B16>(p, i, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) store1<B16>(p, i + e, f[e]);
    }
}
template <int FULL>
__device__ __forceinline__ void load8_as(const void* p, int bf16, int64_t i, int left, float none,
                                         float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = none;
    } else if (bf16) {
        load8<1, FULL>(p, i, left, f);
    } else {
        load8<0, FULL>(p, i, left, f);
    }
}
template <int FULL>
__device__ __forceinline__ void store8_as(void* p, int bf16, int64_t i, int left, const float (&f)[8]) {
    if (bf16)
        store8<1, FULL>(p, i, left, f);
    else
        store8<0, FULL>(p, i, left, f);
}
// f(first element, whether 8 are left (std::true_type or false_type), how many)
// over a row that 256 threads share.
template <class F>
__device__ __forceinline__ void over8(int64_t cols, F f) {
    for (int64_t c = threadIdx.x * 8; c < cols; c += 2048) {
        if (c + 8 <= cols)
            f(c, std::true_type{}, 8);
        else
            f(c, std::false_type{}, (int)(cols - c));
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
        return of_team(cols, MULTI ? (int)(blockDim.x >> 6) : 1,
                       MULTI ? (int)threadIdx.x : (int)(threadIdx.x & 63));
    }
    // The same for `waves` waves, this lane the `lane`-th of theirs.
    __device__ __forceinline__ static Place of_team(int cols, int waves, int lane) {
        Place p;
        p.W = waves;
        p.t = lane * 8;
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

// Sum over a workgroup of 256 threads, in every lane.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// How rows of `cols` elements are held: by one wave or by all waves of their
// workgroup, in nv chunks per lane (nv = 0: not in registers).  One wave needs
// no barrier, but has only enough loads in flight where there are rows for all
// of them.
struct NormShape {
    bool multi;
    int nv, threads;
};
inline NormShape norm_shape(int64_t rows, int64_t cols) {
    if (cols < 8 || cols > 16384) return {false, 0, 256};
    if (cols <= 512) return {false, 1, 256};
    if (cols <= 1024 && rows > 1024) return {false, 2, 256};
    const int nv = cols <= 8192 ? 1 : 2;
    return {true, nv, 64 * (int)((cols + nv * 512 - 1) / (nv * 512))};
}
// Workgroups of a walk over the rows: what 256 compute units hold of them at
// `waves` waves each, and at least `min_rows` rows to a workgroup (or to each
// of its four waves).
inline int norm_groups(const NormShape& sh, int64_t rows, int waves, int min_rows) {
    const int64_t per = (int64_t)min_rows * (sh.multi ? 1 : 4);
    return (int)std::min<int64_t>(256 * (waves * 64 / sh.threads), (rows + per - 1) / per);
}

}  // namespace fp4q
