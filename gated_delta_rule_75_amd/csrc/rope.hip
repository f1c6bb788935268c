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
// (token, pair).  The rest is a copy at memory speed in 16-byte pieces.
#include "launch.h"
#include "vec.h"

namespace kda {

namespace {

constexpr double kInv2Pi = 0.15915494309189533576888376337251;

template <typename T, int VEC, bool HALF>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int tpb) {
    extern __shared__ float cs[];   // cos [tpb][n], then sin [tpb][n]
    const int n = a.rot / 2;
    const int64_t t0 = (int64_t)blockIdx.x * tpb;
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
    // a head's units: `pairs` runs of VEC pairs, then runs of VEC channels that
    // are copied (none where the output is the input)
    const int pairs = HALF ? n / VEC : a.rot / (2 * VEC);
    const int rest = (a.d - a.rot) / VEC;
    const int heads = a.Hq + a.Hk;
    const int per = pairs + rest;
    const int total = nt * heads * per;
    for (int i = threadIdx.x; i < total; i += 256) {
        const int u = i % per, th = i / per, hd = th % heads, t = th / heads;
        const bool isq = hd < a.Hq;
        const int hh = isq ? hd : hd - a.Hq;
        const T* src = (const T*)(isq ? a.q : a.k) + (t0 + t) * (isq ? a.q_stride : a.k_stride) + (int64_t)hh * a.d;
        T* dst = (T*)(isq ? a.q_out : a.k_out) + (t0 + t) * (isq ? a.qo_stride : a.ko_stride) + (int64_t)hh * a.d;
        if (u >= pairs) {
            if (src == dst) continue;
            const int c = a.rot + (u - pairs) * VEC;
            float x[VEC];
            load_vec<T, VEC>(src + c, x);
            store_vec<T, VEC>(dst + c, x);
            continue;
        }
        const float* co = cs + t * n + u * VEC;
        const float* si = sn + t * n + u * VEC;
        float x[VEC], w[VEC], p[VEC], r[VEC];
        if constexpr (HALF) {
            load_vec<T, VEC>(src + u * VEC, x);
            load_vec<T, VEC>(src + n + u * VEC, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                p[j] = x[j] * co[j] - w[j] * si[j];
                r[j] = w[j] * co[j] + x[j] * si[j];
            }
            store_vec<T, VEC>(dst + u * VEC, p);
            store_vec<T, VEC>(dst + n + u * VEC, r);
        } else {
            // channels 2 VEC u .. 2 VEC u + 2 VEC - 1 as two runs
            load_vec<T, VEC>(src + 2 * u * VEC, x);
            load_vec<T, VEC>(src + 2 * u * VEC + VEC, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float e = 2 * j < VEC ? x[(2 * j) % VEC] : w[(2 * j) % VEC];
                const float f = 2 * j + 1 < VEC ? x[(2 * j + 1) % VEC] : w[(2 * j + 1) % VEC];
                const float pe = e * co[j] - f * si[j], pf = f * co[j] + e * si[j];
                if (2 * j < VEC) p[(2 * j) % VEC] = pe;
                else r[(2 * j) % VEC] = pe;
                if (2 * j + 1 < VEC) p[(2 * j + 1) % VEC] = pf;
                else r[(2 * j + 1) % VEC] = pf;
            }
            store_vec<T, VEC>(dst + 2 * u * VEC, p);
            store_vec<T, VEC>(dst + 2 * u * VEC + VEC, r);
        }
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
    const int per = (n + (a.d - a.rot)) / w * (a.Hq + a.Hk);
    // tokens of a workgroup: about 8 units a thread, while the launch still has
    // workgroups for every CU and the table fits 16 KiB
    int tpb = 1;
    while (tpb < 16 && tpb * 2 * per <= 2048 && tpb * 2 * n <= 2048 && a.T / (tpb * 2) >= 2048) tpb *= 2;
    const dim3 grid((unsigned)((a.T + tpb - 1) / tpb));
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
