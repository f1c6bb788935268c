// Norm of a mixer's output rows with the output gate, and its gradient.
//
// Row r = (token t, head h), D elements, weight and bias of the row's head:
//   m = mean(x) (layer) or 0 (rms);  rstd = (mean((x - m)^2) + eps)^-1/2
//   h = (x - m) rstd;  n = h w + b;  y = n sigmoid(z)
// and with d = dy sigmoid(z):
//   dw = sum_t d h;  db = sum_t d;  dz = dy n sigmoid(z) (1 - sigmoid(z))
//   e = d w;  dx = rstd (e - h mean(e h) - [layer: mean(e)])
// All of it in fp32 from the stored values, one rounding at each output.
//
// Both passes are bound by memory: a row stays in the registers of LANES
// threads (16, 64, 256 or 1024, so that a thread holds 16 elements at most),
// which read it once; the centred sum of squares is a second pass over
// registers, so no cancellation.  The gradient's workgroups walk rows s, s + S,
// s + 2S, ... (S a multiple of H: the head, and with it a thread's weight
// columns, never change), keep dw and db in registers, and write one partial
// row each; a second kernel adds the partials in a fixed order.
//
// Measured: 8192 x 96 heads of 128 with the gate (bf16, 607 MB) 105 us, 5.8 TB/s
// (a large copy reaches 6.2); its gradient for 4096 x 32 heads (168 MB) 38 us a
// call, 29 and 4 in the two kernels; for 4099 rows of 2047 (fp32, layer, 101 MB)
// 30, 21 and 6 in the kernels.
#include "launch.h"
#include "vec.h"

namespace kda {

namespace {

// sigmoid(z), and sigmoid(-z), which is 1 - sigmoid(z) without cancellation.  fp32:
// from the accurate exponential of -|z|, which does not overflow.  bf16: the fast
// exponential (off by up to 5e-6 of the value at |z| = 80) is far below the
// output's rounding.
template <typename T>
__device__ __forceinline__ float gate(float z) {
    if constexpr (sizeof(T) == 2) return sigmoid(z);
    const float t = expf(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.f + t);
    return z < 0.f ? t * r : r;
}
template <typename T>
__device__ __forceinline__ void gate(float z, float& s, float& c) {
    const float t = sizeof(T) == 2 ? __expf(-fabsf(z)) : expf(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.f + t);
    s = z < 0.f ? t * r : r;
    c = z < 0.f ? r : t * r;
}

// A thread's NV runs of VEC columns of a row of D: columns (j LANES + lane) VEC.
// TAIL: the last run may be cut.
template <int VEC, int LANES, int NV, bool TAIL>
struct Cols {
    int lane, D;
    __device__ __forceinline__ int at(int j) const { return (j * LANES + lane) * VEC; }
    __device__ __forceinline__ bool in(int j) const { return at(j) < D; }
    __device__ __forceinline__ int left(int j) const { return TAIL ? D - at(j) : VEC; }   // elements of the run, >= VEC: all
};

// y may be x or z: a thread reads all of its elements before it writes them.
template <typename T, int VEC, int LANES, int NV, bool TAIL>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void norm_fwd_kernel(
    int64_t rows, int H, int D, float eps, int rms, const T* x, const float* __restrict__ w,
    const float* __restrict__ b, const T* z, T* y, float* __restrict__ mean, float* __restrict__ rstd) {
    constexpr int RPB = LANES < 256 ? 256 / LANES : 1;   // rows of a workgroup
    __shared__ float part[2][LANES > 64 ? LANES / 64 : 1];
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RPB + threadIdx.x / LANES;
    if (row >= rows) return;                             // LANES > 64: a whole workgroup
    const Cols<VEC, LANES, NV, TAIL> c{(int)(threadIdx.x % LANES), D};
    const int64_t base = row * D, wb = (int64_t)(row % H) * D;
    float v[NV][VEC];
    typename VecOf<T, VEC>::type zv[NV];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (c.in(j)) {
            load_run<T, VEC>(x + base + c.at(j), c.left(j), v[j]);
            if (z) zv[j] = load_raw<T, VEC>(z + base + c.at(j), c.left(j));
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += v[j][i];
    }
    float m = 0.f;
    if (!rms) m = lanes_sum<LANES>(s, part[0]) / (float)D;
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (c.in(j)) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) q += i < c.left(j) ? (v[j][i] - m) * (v[j][i] - m) : 0.f;
        }
    q = lanes_sum<LANES>(q, part[1]);
    const float r = 1.f / sqrtf(q / (float)D + eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!c.in(j)) continue;
        float wv[VEC], o[VEC];
        load_run<float, VEC>(w + wb + c.at(j), c.left(j), wv);
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = (v[j][i] - m) * r * wv[i];
        if (b) {
            float bv[VEC];
            load_run<float, VEC>(b + wb + c.at(j), c.left(j), bv);
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] += bv[i];
        }
        if (z) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] *= gate<T>(to_f32((T)zv[j][i]));
        }
        store_run<T, VEC>(y + base + c.at(j), c.left(j), o);
    }
    if (c.lane == 0) {
        if (mean) mean[row] = m;
        if (rstd) rstd[row] = r;
    }
}

template <typename T, int VEC, int LANES, int NV, bool TAIL>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void norm_bwd_kernel(
    int64_t rows, int64_t S, int H, int D, const T* __restrict__ x, const float* __restrict__ w,
    const float* __restrict__ b, const T* __restrict__ z, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* __restrict__ dy, T* __restrict__ dx, T* __restrict__ dz,
    float* __restrict__ dwp, float* __restrict__ dbp) {
    constexpr int RPB = LANES < 256 ? 256 / LANES : 1;
    __shared__ float part[2][LANES > 64 ? LANES / 32 : 1];
    const int64_t slot = (int64_t)blockIdx.x * RPB + threadIdx.x / LANES;
    if (slot >= S) return;   // whole lane groups (a whole workgroup where LANES > 64)
    const Cols<VEC, LANES, NV, TAIL> c{(int)(threadIdx.x % LANES), D};
    const int64_t wb = (int64_t)(slot % H) * D;
    float wv[NV][VEC], bv[NV][VEC], aw[NV][VEC], ab[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) wv[j][i] = bv[j][i] = aw[j][i] = ab[j][i] = 0.f;
        if (c.in(j)) {
            load_run<float, VEC>(w + wb + c.at(j), c.left(j), wv[j]);
            if (b) load_run<float, VEC>(b + wb + c.at(j), c.left(j), bv[j]);
        }
    }
    // a row's values are loaded while the row before is summed (not where 16
    // elements a thread of 1024 leave no registers for it)
    constexpr bool kAhead = LANES < 1024 || NV * VEC < 16;
    typename VecOf<T, VEC>::type xn[NV], dn[NV], zn[NV];
    float mn = 0.f, rn = 0.f;
    auto fetch = [&](int64_t row) {
        const int64_t base = row * D;
        mn = mean ? mean[row] : 0.f;
        rn = rstd[row];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!c.in(j)) continue;
            xn[j] = load_raw<T, VEC>(x + base + c.at(j), c.left(j));
            dn[j] = load_raw<T, VEC>(dy + base + c.at(j), c.left(j));
            if (z) zn[j] = load_raw<T, VEC>(z + base + c.at(j), c.left(j));
        }
    };
    if (kAhead && slot < rows) fetch(slot);
    int par = 0;
    for (int64_t row = slot; row < rows; row += S, par ^= 1) {
        if (!kAhead) fetch(row);
        const int64_t base = row * D;
        const float m = mn, r = rn;
        float h[NV][VEC], d[NV][VEC];
        float se = 0.f, seh = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const bool in = TAIL ? c.at(j) + i < D : c.in(j);
                h[j][i] = in ? (to_f32((T)xn[j][i]) - m) * r : 0.f;
                d[j][i] = in ? to_f32((T)dn[j][i]) : 0.f;
            }
            if (!c.in(j)) continue;
            if (z) {
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float s, rest;
                    gate<T>(to_f32((T)zn[j][i]), s, rest);
                    d[j][i] *= s;
                    o[i] = d[j][i] * (h[j][i] * wv[j][i] + bv[j][i]) * rest;
                }
                store_run<T, VEC>(dz + base + c.at(j), c.left(j), o);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                aw[j][i] += d[j][i] * h[j][i];
                ab[j][i] += d[j][i];
                d[j][i] *= wv[j][i];
                se += d[j][i];
                seh += d[j][i] * h[j][i];
            }
        }
        if (kAhead && row + S < rows) fetch(row + S);
        // two buffers in turn: a row's sums are read before the barrier of the next row's
        lanes_sum2<LANES>(se, seh, part[par]);
        seh /= (float)D;
        se = mean ? se / (float)D : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!c.in(j)) continue;
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = r * (d[j][i] - h[j][i] * seh - se);
            store_run<T, VEC>(dx + base + c.at(j), c.left(j), o);
        }
    }
    const int64_t pb = slot * D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (!c.in(j)) continue;
        store_run<float, VEC>(dwp + pb + c.at(j), c.left(j), aw[j]);
        if (dbp) store_run<float, VEC>(dbp + pb + c.at(j), c.left(j), ab[j]);
    }
}

// dw[c] = sum over P partial rows of HD columns, in a fixed order: 32 threads
// take every 32nd partial of a column, then their sums are added.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(int64_t P, int64_t HD, const float* __restrict__ dwp,
                                                           const float* __restrict__ dbp, float* __restrict__ dw,
                                                           float* __restrict__ db) {
    __shared__ float s[32][33];
    const float* src = blockIdx.y ? dbp : dwp;
    float* dst = blockIdx.y ? db : dw;
    const int cx = threadIdx.x & 31, py = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + cx;
    float a = 0.f;
    if (col < HD) {
#pragma unroll 4
        for (int64_t p = py; p < P; p += 32) a += src[p * HD + col];
    }
    s[py][cx] = a;
    __syncthreads();
    // thread (py, cx) adds column py's 32 sums with its half wave
    a = s[cx][py];
    a = row16_sum(a);
    a += __shfl_xor(a, 16);
    const int64_t c2 = (int64_t)blockIdx.x * 32 + py;
    if (cx == 0 && c2 < HD) dst[c2] = a;
}

template <typename T, int VEC, int LANES, int NV, bool TAIL>
hipError_t launch_t(const NormArgs& a) {
    constexpr int RPB = LANES < 256 ? 256 / LANES : 1, NT = LANES < 256 ? 256 : LANES;
    const int64_t rows = a.T * a.H;
    if (!a.dy) {
        hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, LANES, NV, TAIL>), folded_grid((rows + RPB - 1) / RPB), dim3(NT), 0,
                           (hipStream_t)a.stream, rows, a.H, a.D, a.eps, a.rms, (const T*)a.x, a.weight, a.bias,
                           (const T*)a.z, (T*)a.y, a.mean, a.rstd);
    } else {
        hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, LANES, NV, TAIL>), dim3((unsigned)((a.slots + RPB - 1) / RPB)), dim3(NT),
                           0, (hipStream_t)a.stream, rows, a.slots, a.H, a.D, (const T*)a.x, a.weight, a.bias,
                           (const T*)a.z, a.mean, a.rstd, (const T*)a.dy, (T*)a.dx, (T*)a.dz, a.dwp, a.dbp);
    }
    return hipGetLastError();
}

// The narrowest lane group that holds a row with at most 16 elements a thread.
template <typename T, bool TAIL>
hipError_t launch_r(const NormArgs& a) {
    constexpr int VEC = kVec16<T>;
    const int n = (a.D + VEC - 1) / VEC;   // runs of a row
    if (n <= 16) return launch_t<T, VEC, 16, 1, TAIL>(a);
    if (n <= 64) return launch_t<T, VEC, 64, 1, TAIL>(a);
    if (n <= 128) return launch_t<T, VEC, 64, 2, TAIL>(a);
    if constexpr (VEC == 4) {
        if (n <= 256) return launch_t<T, VEC, 64, 4, TAIL>(a);
        if (n <= 512) return launch_t<T, VEC, 256, 2, TAIL>(a);
        if (n <= 1024) return launch_t<T, VEC, 256, 4, TAIL>(a);
        if (n <= 2048) return launch_t<T, VEC, 1024, 2, TAIL>(a);
        return launch_t<T, VEC, 1024, 4, TAIL>(a);
    } else {
        if (n <= 256) return launch_t<T, VEC, 256, 1, TAIL>(a);
        if (n <= 512) return launch_t<T, VEC, 256, 2, TAIL>(a);
        if (n <= 1024) return launch_t<T, VEC, 1024, 1, TAIL>(a);
        return launch_t<T, VEC, 1024, 2, TAIL>(a);
    }
}

template <typename T>
hipError_t launch_d(const NormArgs& a) {
    return a.D % kVec16<T> ? launch_r<T, true>(a) : launch_r<T, false>(a);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a) {
    if (a.T > 0) {
        const hipError_t e = a.dtype == 0 ? launch_d<__bf16>(a) : launch_d<float>(a);
        if (e != hipSuccess) return e;
    }
    if (a.dweight) {
        const int64_t HD = (int64_t)a.H * a.D;
        hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((HD + 31) / 32), a.dbias ? 2 : 1), dim3(1024), 0,
                           (hipStream_t)a.stream, a.T > 0 ? a.slots / a.H : 0, HD, a.dwp, a.dbp, a.dweight, a.dbias);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace kda
