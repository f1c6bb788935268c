// Rotary positions: each token's first `rot` channels of every query and key
// head are turned in pairs by the angle position x frequency,
//   (a, b) -> m (a cos - b sin,  b cos + a sin),
// with b's sign of the sine reversed for the inverse (the gradient: the turn's
// matrix is orthogonal up to m).  Pairs are (i, i + rot/2) or (2i, 2i + 1).
//
// The angle of a far position needs more than fp32 (at 10^6 positions an fp32
// angle is off by 0.06): the product is taken in fp64 in turns (radians / 2 pi),
// its fraction is exact, and only that goes to fp32.  A workgroup's tokens share
// their cosines and sines among all heads through LDS, one sincospi for each
// (token, pair).  The rest is a copy at memory speed in 16-byte pieces: 8192 x
// 192 heads of 128 in bf16 (806 MB) take 150 us, 5.4 TB/s, where a large copy
// reaches 6.2.
#include "launch.h"
#include "vec.h"

namespace kda {

namespace {

constexpr double kInv2Pi = 0.15915494309189533576888376337251;

template <typename T, int VEC, bool HALF>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int tpb) {
    extern __shared__ float cs[];   // cos [tpb][n], then sin [tpb][n]
    const int n = a.rot / 2;
    const int64_t t0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * tpb;
    if (t0 >= a.T) return;
    const int nt = (int)(a.T - t0 < tpb ? a.T - t0 : tpb);
    float* sn = cs + tpb * n;
    for (int i = threadIdx.x; i < nt * n; i += 256) {
        const double turns = (double)a.positions[t0 + i / n] * (a.inv_freq[i % n] * kInv2Pi);
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        cs[i] = a.mscale * c;
        sn[i] = a.mscale * (a.inverse ? -s : s);
    }
    __syncthreads();
    // a head's units, two runs of VEC channels each: the two runs of VEC pairs,
    // or two neighbouring runs that are copied (none where the output is the
    // input); a thread has two units in flight
    const int pairs = HALF ? n / VEC : a.rot / (2 * VEC);
    const int rest = (a.d - a.rot) / VEC;
    const int heads = a.Hq + a.Hk;
    const int per = pairs + (rest + 1) / 2;
    const int total = nt * heads * per;
    struct Unit {
        const T* src;
        T* dst;
        int c0, c1, cs;       // channels of the runs (c1 < 0: one run); cosines, or -1: a copy
        float x[VEC], w[VEC];
    };
    auto fetch = [&](Unit& m, int i) {
        const int u = i % per, th = i / per, hd = th % heads, t = th / heads;
        const bool isq = hd < a.Hq;
        const int hh = isq ? hd : hd - a.Hq;
        m.src = (const T*)(isq ? a.q : a.k) + (t0 + t) * (isq ? a.q_stride : a.k_stride) + (int64_t)hh * a.d;
        m.dst = (T*)(isq ? a.q_out : a.k_out) + (t0 + t) * (isq ? a.qo_stride : a.ko_stride) + (int64_t)hh * a.d;
        if (u < pairs) {
            m.cs = t * n + u * VEC;
            m.c0 = HALF ? u * VEC : 2 * u * VEC;
            m.c1 = HALF ? n + u * VEC : 2 * u * VEC + VEC;
        } else {
            m.cs = -1;
            m.c0 = a.rot + 2 * (u - pairs) * VEC;
            m.c1 = 2 * (u - pairs) + 1 < rest ? m.c0 + VEC : -1;
            if (m.src == m.dst) return;
        }
        load_vec<T, VEC>(m.src + m.c0, m.x);
        if (m.c1 >= 0) load_vec<T, VEC>(m.src + m.c1, m.w);
    };
    auto put = [&](Unit& m) {
        if (m.cs < 0) {
            if (m.src == m.dst) return;
            store_vec<T, VEC>(m.dst + m.c0, m.x);
            if (m.c1 >= 0) store_vec<T, VEC>(m.dst + m.c1, m.w);
            return;
        }
        const float* co = cs + m.cs;
        const float* si = sn + m.cs;
        float p[VEC], r[VEC];
        if constexpr (HALF) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                p[j] = m.x[j] * co[j] - m.w[j] * si[j];
                r[j] = m.w[j] * co[j] + m.x[j] * si[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float e = 2 * j < VEC ? m.x[(2 * j) % VEC] : m.w[(2 * j) % VEC];
                const float f = 2 * j + 1 < VEC ? m.x[(2 * j + 1) % VEC] : m.w[(2 * j + 1) % VEC];
                const float pe = e * co[j] - f * si[j], pf = f * co[j] + e * si[j];
                if (2 * j < VEC) p[(2 * j) % VEC] = pe;
                else r[(2 * j) % VEC] = pe;
                if (2 * j + 1 < VEC) p[(2 * j + 1) % VEC] = pf;
                else r[(2 * j + 1) % VEC] = pf;
            }
        }
        store_vec<T, VEC>(m.dst + m.c0, p);
        store_vec<T, VEC>(m.dst + m.c1, r);
    };
    for (int i = threadIdx.x; i < total; i += 512) {
        Unit m, o;
        fetch(m, i);
        const bool two = i + 256 < total;
        if (two) fetch(o, i + 256);
        put(m);
        if (two) put(o);
    }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T>
hipError_t launch_t(const RopeArgs& a) {
    constexpr int V = kVec16<T>;
    const int n = a.rot / 2;
    const bool vec = n % V == 0 && a.d % V == 0 && a.q_stride % V == 0 && a.k_stride % V == 0 &&
                     a.qo_stride % V == 0 && a.ko_stride % V == 0 && al16(a.q) && al16(a.k) && al16(a.q_out) &&
                     al16(a.k_out);
    const int w = vec ? V : 1;
    const int per = (n + (a.d - a.rot) / 2) / w * (a.Hq + a.Hk);
    // tokens of a workgroup: about 8 units a thread, while the launch still has
    // workgroups for every CU and the table fits 16 KiB
    int tpb = 1;
    while (tpb < 16 && tpb * 2 * per <= 2048 && tpb * 2 * n <= 2048 && a.T / (tpb * 2) >= 2048) tpb *= 2;
    const dim3 grid = folded_grid((a.T + tpb - 1) / tpb);
    const size_t lds = (size_t)tpb * n * 2 * sizeof(float);
    if (vec) {
        if (a.half) hipLaunchKernelGGL((rope_kernel<T, V, true>), grid, dim3(256), lds, (hipStream_t)a.stream, a, tpb);
        else hipLaunchKernelGGL((rope_kernel<T, V, false>), grid, dim3(256), lds, (hipStream_t)a.stream, a, tpb);
    } else {
        if (a.half) hipLaunchKernelGGL((rope_kernel<T, 1, true>), grid, dim3(256), lds, (hipStream_t)a.stream, a, tpb);
        else hipLaunchKernelGGL((rope_kernel<T, 1, false>), grid, dim3(256), lds, (hipStream_t)a.stream, a, tpb);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a) {
    if (a.T == 0) return hipSuccess;
    return a.dtype == 0 ? launch_t<__bf16>(a) : launch_t<float>(a);
}

}  // namespace kda
