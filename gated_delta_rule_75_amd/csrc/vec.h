// Rows of elements in 16-byte pieces, or one element at a time where a row's
// length or address allows no more (gfx950 only).
#pragma once

#include "common.h"

namespace kda {

template <typename T> constexpr int kVec16 = 16 / (int)sizeof(T);

template <typename T, int N> struct VecOf { typedef T type __attribute__((ext_vector_type(N))); };
template <typename T> struct VecOf<T, 1> { typedef T type; };

template <typename T, int N>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[N]) {
    if constexpr (N == 1) {
        x[0] = to_f32(*p);
    } else {
        const auto v = *reinterpret_cast<const typename VecOf<T, N>::type*>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = to_f32((T)v[i]);
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[N]) {
    if constexpr (N == 1) {
        *p = from_f32<T>(x[0]);
    } else {
        typename VecOf<T, N>::type v;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = from_f32<T>(x[i]);
        *reinterpret_cast<typename VecOf<T, N>::type*>(p) = v;
    }
}

// Runs of N elements at any element address (the hardware takes 16 bytes at
// element alignment), of which the first n exist; the others read as zeros.
template <typename T, int N> struct LooseVec { typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T)))); };
template <typename T, int N>
__device__ __forceinline__ typename VecOf<T, N>::type load_raw(const T* p, int n) {
    typename VecOf<T, N>::type v;
    if (n >= N) {
        v = *reinterpret_cast<const typename LooseVec<T, N>::type*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < n ? p[i] : from_f32<T>(0.f);
    }
    return v;
}
template <typename T, int N>
__device__ __forceinline__ void load_run(const T* p, int n, float (&x)[N]) {
    const auto v = load_raw<T, N>(p, n);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32((T)v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_run(T* p, int n, const float (&x)[N]) {
    if (n >= N) {
        typename LooseVec<T, N>::type v;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = from_f32<T>(x[i]);
        *reinterpret_cast<typename LooseVec<T, N>::type*>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = from_f32<T>(x[i]);
    }
}

// n workgroups as a grid: an axis of a launch holds less than 2^32 threads, so
// many small rows take a second axis, whose last line may reach past n.
inline dim3 folded_grid(int64_t n) {
    constexpr int64_t line = 1 << 20;
    return n <= line ? dim3((unsigned)n) : dim3((unsigned)line, (unsigned)((n + line - 1) / line));
}

// Sum over LANES consecutive threads of a workgroup, the same bits in each of
// them.  Up to a wave: DPP adds over 16 lanes, then two permutes.  More: the
// waves' sums through LDS (`part`, one float a wave; the caller's barriers keep
// two uses of one buffer apart).
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x, float* part) {
    static_assert(LANES == 16 || LANES == 64 || LANES % 64 == 0, "lanes");
    x = row16_sum(x);
    if constexpr (LANES >= 64) {
        x += __shfl_xor(x, 16);
        x += __shfl_xor(x, 32);
    }
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int w = 0; w < LANES / 64; ++w) x += part[w];
    }
    return x;
}

// Two sums at once: one barrier.
template <int LANES>
__device__ __forceinline__ void lanes_sum2(float& x, float& y, float* part) {
    x = row16_sum(x);
    y = row16_sum(y);
    if constexpr (LANES >= 64) {
        x += __shfl_xor(x, 16);
        y += __shfl_xor(y, 16);
        x += __shfl_xor(x, 32);
        y += __shfl_xor(y, 32);
    }
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0) {
            part[threadIdx.x >> 6] = x;
            part[LANES / 64 + (threadIdx.x >> 6)] = y;
        }
        __syncthreads();
        x = y = 0.f;
#pragma unroll
        for (int w = 0; w < LANES / 64; ++w) {
            x += part[w];
            y += part[LANES / 64 + w];
        }
    }
}

}  // namespace kda
