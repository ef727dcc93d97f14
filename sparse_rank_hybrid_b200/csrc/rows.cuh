// Helpers of the row kernels (residual_norm.cu, qk_rope.cu): typed vectors of eight elements, each
// thread's own ring of asynchronous loads, and sums over the threads that share a row.
#pragma once

#include "common.cuh"

namespace slra {

// Element types of the tensors, as the values of slra_dtype.
constexpr int kBf16 = 0, kF32 = 1, kF16 = 2;

// Eight elements of a tensor: one 16-byte unit of a 16-bit type, two of fp32.
template <typename T>
constexpr int kUnits = sizeof(T) / 2;

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 (&u)[kUnits<T>], float (&f)[8]);
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(const uint4 (&u)[1], float (&f)[8]) {
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // bf16 is the upper half of fp32
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <>
__device__ __forceinline__ void unpack8<__half>(const uint4 (&u)[1], float (&f)[8]) {
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
        f[2 * i] = __low2float(h);
        f[2 * i + 1] = __high2float(h);
    }
}
template <>
__device__ __forceinline__ void unpack8<float>(const uint4 (&u)[2], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(u[i].x);
        f[4 * i + 1] = __uint_as_float(u[i].y);
        f[4 * i + 2] = __uint_as_float(u[i].z);
        f[4 * i + 3] = __uint_as_float(u[i].w);
    }
}

// Rounded to nearest even, once, on the way to memory.
template <typename T>
__device__ __forceinline__ void pack8(const float (&f)[8], uint4 (&u)[kUnits<T>]);
template <>
__device__ __forceinline__ void pack8<__nv_bfloat16>(const float (&f)[8], uint4 (&u)[1]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    u[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void pack8<__half>(const float (&f)[8], uint4 (&u)[1]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    u[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void pack8<float>(const float (&f)[8], uint4 (&u)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        u[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
    uint4 u[kUnits<T>];
#pragma unroll
    for (int i = 0; i < kUnits<T>; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    unpack8<T>(u, f);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
    uint4 u[kUnits<T>];
    pack8<T>(f, u);
#pragma unroll
    for (int i = 0; i < kUnits<T>; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
}

// Eight elements of a vector whose type is known at run time (weights, modulation rows), or `fill`
// where there is no such vector.
__device__ __forceinline__ void load8_any(const void* base, long long at, int dtype, float fill, float (&f)[8]) {
    if (!base) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fill;
    } else if (dtype == kF32) {
        load8(static_cast<const float*>(base) + at, f);
    } else if (dtype == kBf16) {
        load8(static_cast<const __nv_bfloat16*>(base) + at, f);
    } else {
        load8(static_cast<const __half*>(base) + at, f);
    }
}

// Asynchronous copies global -> shared.  Every thread reads back only what it copied itself, so its own
// wait orders the data and no barrier is needed.
__device__ __forceinline__ void async_copy16(void* smem, const void* gmem) {
    const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
}
__device__ __forceinline__ void async_copy8(void* smem, const void* gmem) {
    const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(s), "l"(gmem) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A team of threads shares a row: `size` threads, a power of two up to 32 (several teams in a block) or
// the whole block of `size` = blockDim.x threads, a multiple of 32.
constexpr int kTeamScratch = 2 * 4 * 32;  // floats of shared memory for a block-wide team's sums

struct Team {
    int size;
    float* scratch;  // kTeamScratch floats (block-wide teams)
    int turn;        // which half of the scratch the next sum uses

    // Every value summed over the team, in a fixed order; each thread gets the sums.  Consecutive sums use
    // the scratch's halves in turn: before a thread can write a half again, every thread has passed the
    // other half's barrier and so has read this one.
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N]) {
        static_assert(N <= 4, "scratch holds four values a warp");
        if (size <= 32) {
            for (int o = size >> 1; o > 0; o >>= 1)
#pragma unroll
                for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
            return;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = size >> 5;
        float* s = scratch + turn * (4 * 32);
        turn ^= 1;
        if (lane == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) s[n * 32 + warp] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = lane < warps ? s[n * 32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    }
    __device__ __forceinline__ void sync() const {
        if (size <= 32) __syncwarp();
        else __syncthreads();
    }
};

// Rows [lo, hi) of worker w among `workers` workers sharing n rows; the worker that has row r.
__host__ __device__ inline long long worker_lo(long long n, int workers, int w) { return n * w / workers; }
__host__ __device__ inline int worker_of(long long n, int workers, long long r) {
    return static_cast<int>(((r + 1) * workers - 1) / n);
}

}  // namespace slra
