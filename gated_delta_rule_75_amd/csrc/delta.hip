// The gated delta rule with a decay for each head, by chunks of 64 tokens.
//
// Per sequence and value head, from token to token:
//   u = exp(g) S,   e = v - u^T k,   S <- u + beta k e^T,   y = scale S^T q
// For a chunk, with G the sum of g inside it, D_ij = exp(G_i - G_j) for j <= i
// and S the state that enters:
//   M = strictly lower part of (K K^T . D),   X = (I + M diag(beta))^-1
//   E = X (V - exp(G) K S)                    errors of prediction
//   y = P diag(beta) E + scale exp(G) Q S,    P = scale Q K^T . D
//   S <- exp(G_63) S + K^T diag(exp(G_63 - G) beta) E
// and for the gradient, with R that of the state behind the chunk:
//   Z = (I + M^T diag(beta))^-1,  U = Z (P^T dY + exp(G_63 - G) K R),  dV = diag(beta) U
//   R <- exp(G_63) R + scale Q^T diag(exp(G)) dY - K^T diag(exp(G)) dV
//   W = scale dY E^T . D,   Y = -(strictly lower part of dV E^T . D)
//   dQ = W diag(beta) K + scale exp(G) dY S^T
//   dK = Y diag(beta) K - exp(G) dV S^T + diag(beta) (W^T Q + Y^T K + exp(G_63 - G) E R^T)
//   dbeta_t = e_t.u_t
// and the decay's gradient as the sum of all that crosses token t, from what entered the
// state before it to what reads it from t on:
//   dg_t = sum_{j >= t > i} N_ji + sum_{j >= t} a_j + sum_{i < t} b_i + exp(G_63) <S, R>
//   N = (W . Q K^T + Y . K K^T) diag(beta)      pairs of the chunk, j behind i
//   a_j = exp(G_j) (scale q_j.S dy_j - k_j.S dv_j)   of the state that enters
//   b_i = exp(G_63 - G_i) beta_i k_i.R e_i           into the state behind the chunk
// Each of these holds the decay of t as a factor, so that dg keeps its digits where
// decays are strong, and is 0 where one is 0 and at a first token without a state.  (As
// the sum over s >= t of q.dq - v.dv it would be a small difference of large terms:
// 1 % off at g = -10, all of it at -20.)
//
// A first kernel makes what does not involve the state (X, Z, P and P^T as operands,
// the tables of decays) for all chunks at once.  A second walks a sequence's chunks
// with the state in its accumulators, a workgroup for 64 value columns of a head.
// The gradient walks twice, forwards (keeping each chunk's state and E) and
// backwards (its R and U); then a kernel makes dQ, dK, dV, dbeta and dg for all chunks
// at once.
//
// bf16 inputs enter products as they are.  What is computed enters as a sum of
// bf16 values: of three, 24 bits, on the way to fp32 outputs (states, E, U, X, Z,
// the gates' gradients), of two, 16 bits, on the way to an output in bf16 alone, whose
// own rounding is then the one that shows: y is off by 1.66e-3 of its norm either way,
// and 0.5 % of its values are the neighbour of the exact value's rounding.  With three parts
// 0.02 % are, and the prompt takes 587 us for 537 (8192 tokens of 96 heads).
#include "tiles.h"

namespace kda {

namespace {

// Parts of a computed operand: for outputs in T, and for fp32 ones.
template <typename T> constexpr int kTwo = sizeof(T) == 2 ? 2 : 1;
template <typename T> constexpr int kThree = sizeof(T) == 2 ? 3 : 1;

// c += a b for operands in parts, the smallest products first (those beyond the
// finer operand's own bits are left out).
template <typename T, int NA, int NB>
__device__ __forceinline__ f32x4_t mma_parts(const Frag8<T> (&a)[NA], const Frag8<T> (&b)[NB], f32x4_t c) {
#pragma unroll
    for (int s = NA + NB - 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB && s < (NA > NB ? NA : NB)) c = mma(a[i], b[s - i], c);
    return c;
}

// Operand tiles of a lower triangle (rows i, contraction j <= i) and of its
// transpose, in the order in which lanes read them: 6 pieces of 16 rows x 32 that
// are not all zeros, each lane's 8 values in runs of 16 bytes (bf16: a run a part;
// fp32: two halves), a run of all lanes side by side.
__device__ __forceinline__ constexpr int tri_piece(int t, int s) { return t < 2 ? t : 2 * (t - 1) + s; }
__device__ __forceinline__ constexpr int tri_piece_t(int t, int s) { return t < 2 ? 2 * t + s : t + 2; }
template <typename T, int N> constexpr int kRuns = sizeof(T) == 2 ? N : 2;
template <typename T, int N> constexpr int kTri = 6 * 1024 * kRuns<T, N>;   // bytes
static_assert(kTri<__bf16, 3> <= kTriBytes && kTri<float, 1> <= kTriBytes, "workspace");

template <typename T, int N>
__device__ __forceinline__ void put_operand(char* base, int piece, int lane, const float (&x)[8]) {
    Frag8<T> f[N];
    split(x, f);
    u32x4_t* const at = reinterpret_cast<u32x4_t*>(base) + piece * 64 * kRuns<T, N> + lane;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int p = 0; p < N; ++p) at[64 * p] = __builtin_bit_cast(u32x4_t, f[p].v);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x4_t u;
#pragma unroll
            for (int r = 0; r < 4; ++r) u[r] = f[0].v[4 * h + r];
            at[64 * h] = __builtin_bit_cast(u32x4_t, u);
        }
    }
}
// Half of one in two parts: contraction 4 g + (0..3) of the first (0) or second (1) 16.
template <typename T>
__device__ __forceinline__ void put_half(char* base, int piece, int half, int lane, const f32x4_t& x) {
    char* const at = base + piece * 2048 + lane * 16;
    if constexpr (sizeof(T) == 2) {
        store4<T>(reinterpret_cast<T*>(at + 8 * half), x);
        f32x4_t rest;
#pragma unroll
        for (int r = 0; r < 4; ++r) rest[r] = x[r] - (float)(__bf16)x[r];
        store4<T>(reinterpret_cast<T*>(at + 1024 + 8 * half), rest);
    } else {
        *reinterpret_cast<f32x4_t*>(at + 1024 * half) = x;
    }
}
template <typename T, int N>
__device__ __forceinline__ void get_operand(const char* base, int piece, int lane, Frag8<T> (&f)[N]) {
    const u32x4_t* const at = reinterpret_cast<const u32x4_t*>(base) + piece * 64 * kRuns<T, N> + lane;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int p = 0; p < N; ++p) f[p].v = __builtin_bit_cast(bf16x8_t, at[64 * p]);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4_t u = __builtin_bit_cast(f32x4_t, at[64 * h]);
#pragma unroll
            for (int r = 0; r < 4; ++r) f[0].v[4 * h + r] = u[r];
        }
    }
}

// Eight consecutive elements as an operand of type T, from global memory.
__device__ __forceinline__ Frag8<__bf16> frag_at(const __bf16* p) {
    Frag8<__bf16> f;
    f.v = *reinterpret_cast<const bf16x8_t*>(p);
    return f;
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p), b = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        x[r] = a[r];
        x[4 + r] = b[r];
    }
}
__device__ __forceinline__ Frag8<float> frag_at(const float* p) {
    Frag8<float> f;
    load8(p, f.v);
    return f;
}

// The state's rows in a wave's accumulators: tile 2 s + h, row 4 g + r holds
// channel 32 s + 8 g + 4 h + r, so that two tiles are an operand whose contraction
// runs over 8 consecutive channels a lane.  cols8: the operand whose rows are a
// tile's channels, contraction over tokens 32 s2 + {0, 16} + 4 g + (0..3).
template <typename T, int D>
__device__ __forceinline__ Frag8<T> cols8(const T* t, int s, int h, int s2, int lane) {
    Frag8<T> f;
    if constexpr (sizeof(T) == 2) {
        const int row = 32 * s2 + 4 * (lane >> 4) + ((lane & 15) >> 2), col = 32 * s + 8 * (lane & 3) + 4 * h;
        const bf16x4_t x = __builtin_bit_cast(bf16x4_t, lds_tr(t + Tile<T, D>::off(row, col)));
        const bf16x4_t y = __builtin_bit_cast(bf16x4_t, lds_tr(t + Tile<T, D>::off(row + 16, col)));
        f.v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        const int m = lane & 15, row = 32 * s2 + 4 * (lane >> 4), col = 32 * s + 8 * (m >> 2) + 4 * h + (m & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f.v[i] = t[Tile<T, D>::off(row + i, col)];
            f.v[4 + i] = t[Tile<T, D>::off(row + 16 + i, col)];
        }
    }
    return f;
}

// 2^(difference of two sums), each as integer and fraction.
typedef int i32x4_t __attribute__((ext_vector_type(4)));
struct __attribute__((aligned(16))) Sums {
    float frac[C];
    int whole[C];
    __device__ __forceinline__ void set(int lane, double G, bool valid) {
        const double w = floor(G);
        frac[lane] = (float)(G - w);
        whole[lane] = valid ? (int)w : -(1 << 20);   // a row without a token reads nothing
    }
    // rows i against j .. j + 3, those behind i and (strict) i itself 0; and rows i .. i + 3
    // against j
    __device__ __forceinline__ f32x4_t before(int i, int j, bool strict) const {
        const f32x4_t f = *reinterpret_cast<const f32x4_t*>(frac + j);
        const i32x4_t w = *reinterpret_cast<const i32x4_t*>(whole + j);
        const float fi = frac[i];
        const int wi = whole[i];
        f32x4_t d;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            d[r] = __builtin_amdgcn_ldexpf(exp2_fast(fi - f[r]), wi - w[r]);
            d[r] = j + r < i + !strict ? d[r] : 0.f;
        }
        return d;
    }
    __device__ __forceinline__ f32x4_t behind(int i, int j, bool strict) const {
        const f32x4_t f = *reinterpret_cast<const f32x4_t*>(frac + i);
        const i32x4_t w = *reinterpret_cast<const i32x4_t*>(whole + i);
        const float fj = frac[j];
        const int wj = whole[j];
        f32x4_t d;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            d[r] = __builtin_amdgcn_ldexpf(exp2_fast(f[r] - fj), w[r] - wj);
            d[r] = j < i + r + !strict ? d[r] : 0.f;
        }
        return d;
    }
};

__device__ __forceinline__ f32x4_t mma16(const f32x4_t& a, const f32x4_t& b, f32x4_t c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

constexpr int kLd = C + 4;   // pitch of a 64 x 64 matrix in LDS

// The inverse of I + A, in place in LDS, A strictly lower: the four 16 x 16 blocks on
// the diagonal by forward substitution, a column a lane, then block column by
// block column X_ij = -X_ii sum_k A_ik X_kj with fp32 products.  (As a product of
// powers, (I - A)(I + A^2)..., a chunk of equal keys would lose four digits.)  A
// wave has a block and a block column; what lies above the diagonal blocks is
// neither read nor written.
__device__ __forceinline__ void invert(float* sx, int wave, int lane) {
    const int lr = lane & 15, lg = lane >> 4;
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    {
        float x[16];
        const float* const m = sx + 16 * wave * (kLd + 1);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float d = i == lr ? 1.f : 0.f;
#pragma unroll
            for (int j4 = 0; j4 < i; j4 += 4) {
                const f32x4_t v = *reinterpret_cast<const f32x4_t*>(m + i * kLd + j4);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (j4 + r < i) d -= v[r] * x[j4 + r];
            }
            x[i] = d;
        }
        if (lg == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sx[(16 * wave + i) * kLd + 16 * wave + lr] = x[i];
        }
    }
    __syncthreads();
    f32x4_t col[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i < wave) continue;
        if (i == wave) {
#pragma unroll
            for (int r = 0; r < 4; ++r) col[i][r] = sx[(16 * i + 4 * lg + r) * kLd + 16 * i + lr];
            continue;
        }
        f32x4_t s = zero;
#pragma unroll
        for (int k = 0; k < i; ++k)
            if (k >= wave) s = mma16(*reinterpret_cast<const f32x4_t*>(sx + (16 * i + lr) * kLd + 16 * k + 4 * lg), col[k], s);
        col[i] = -mma16(*reinterpret_cast<const f32x4_t*>(sx + (16 * i + lr) * kLd + 16 * i + 4 * lg), s, zero);
    }
    __syncthreads();
#pragma unroll
    for (int i = 1; i < 4; ++i)
        if (i > wave) {
#pragma unroll
            for (int r = 0; r < 4; ++r) sx[(16 * i + 4 * lg + r) * kLd + 16 * wave + lr] = col[i][r];
        }
    __syncthreads();
}

// Tables, scores and inverse of a (chunk, head).  GRAD: X, Z and P^T.
// LDS: the rows of k (GRAD: and q), then the matrices in their place.  For a chunk of
// its own, since nothing here waits for the state: it fills the card where the walk
// cannot.  A workgroup asks for all that it reads at once, and the matrices take the
// rows' place in LDS (8192 tokens of 96 heads: 246 -> 158 us).  Bound by the
// chain of the 16 x 16 substitutions and by what it writes, 396 MB of operands, 3.9
// TB/s with what it reads.
template <typename T, int DK, bool GRAD> constexpr int prep_bytes() {
    constexpr int rows = C * DK * (int)sizeof(T) * (GRAD ? 2 : 1), m = C * kLd * 4 * (GRAD ? 2 : 1);
    return rows > m ? rows : m;
}

template <typename T, int DK, bool GRAD>
__global__ __launch_bounds__(256) void gdr_prep_kernel(GdrArgs a) {
    typedef Tile<T, DK> TK;
    constexpr int SN = DK / 32, EP = 16 / (int)sizeof(T), NR = C * DK / EP / 256;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    T* const sk = reinterpret_cast<T*>(smem);
    T* const sq = sk + C * DK;
    float* const sx = reinterpret_cast<float*>(smem);
    float* const sz = sx + C * kLd;
    __shared__ Sums sums;
    __shared__ __attribute__((aligned(16))) float s_beta[C];
    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), lr = lane & 15, lg = lane >> 4;
    const int H = a.at.H, b = uni(blockIdx.x / H), h = blockIdx.x - b * H;
    if (a.at.clear) {
        if constexpr (GRAD) {
            LinArgs shared = a.at;
            shared.H = H / a.k.share;
            if (h < shared.H) {
                clear_rest<T, DK>(shared, (T*)a.dq, b, h);
                clear_rest<T, DK>(shared, (T*)a.dk, b, h);
            }
            if (a.dg) clear_rest<float, 1>(a.at, a.dg, b, h);
            clear_rest<float, 1>(a.at, a.dbeta, b, h);
        }
        T* const out = (T*)(GRAD ? a.dv_out : a.y);
        if (a.head_v == 64) clear_rest<T, 64>(a.at, out, b, h);
        else clear_rest<T, 128>(a.at, out, b, h);
    }
    const Block bl = find_block(a.at, b);
    if (bl.n < 0 || bl.cnt == 0) return;
    const int cnt = uni(bl.cnt);
    const int64_t start = uni64(bl.start), slot = (int64_t)b * H + h;
    // all of the chunk's reads at once; rows without a token: the last one's
    const T* const k = (const T*)a.k.p + start * a.k.stride + (int64_t)(h / a.k.share) * DK;
    const T* const q = (const T*)a.q.p + start * a.q.stride + (int64_t)(h / a.q.share) * DK;
    const int own = GRAD ? wave : 3 - wave;   // rows i (GRAD: j) of the scores that the wave makes: as many tiles as of M in all
    u32x4_t rk[NR], rq[GRAD ? NR : 1];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int u = i * 256 + tid, row = u / (DK / EP), col = u % (DK / EP) * EP;
        const int64_t tok = row < cnt ? row : cnt - 1;
        rk[i] = *reinterpret_cast<const u32x4_t*>(k + tok * a.k.stride + col);
        if constexpr (GRAD) rq[i] = *reinterpret_cast<const u32x4_t*>(q + tok * a.q.stride + col);
    }
    Frag8<T> mine[SN];
    if constexpr (!GRAD) {
        const int row = 16 * own + lr < cnt ? 16 * own + lr : cnt - 1;
#pragma unroll
        for (int s = 0; s < SN; ++s) mine[s] = frag_at(q + row * a.q.stride + 32 * s + 8 * lg);
    }
    if (wave == 0) {
        const bool valid = lane < cnt;
        const int64_t at = (start + lane) * H + h;
        const float beta = valid ? a.beta[at] : 0.f;
        const double G = decay_scan(valid && a.g ? a.g[at] : 0.f), end = lane_d(G, 63);
        sums.set(lane, G, valid);
        s_beta[lane] = beta;
        float* const tab = a.tab + slot * kGdrTab;
        tab[lane] = valid ? exp2_fast((float)G) : 0.f;
        tab[C + lane] = valid ? exp2_fast((float)(end - G)) : 0.f;
        tab[2 * C + lane] = beta;
        tab[3 * C + lane] = exp2_fast((float)end);
        tab[4 * C + lane] = sums.frac[lane];
        tab[5 * C + lane] = __int_as_float(sums.whole[lane]);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int u = i * 256 + tid, at = TK::off(u / (DK / EP), u % (DK / EP) * EP);
        *reinterpret_cast<u32x4_t*>(sk + at) = rk[i];
        if constexpr (GRAD) *reinterpret_cast<u32x4_t*>(sq + at) = rq[i];
    }
    __syncthreads();
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    auto product = [&](const T* rows, int t, const Frag8<T> (&f)[SN]) {
        f32x4_t d = zero;
#pragma unroll
        for (int s = 0; s < SN; ++s) d = mma(TK::rows8(rows, 16 * t, s, lane), f[s], d);
        return d;
    };
    // scores, as operands: the wave's rows i, or (transposed) its rows j
    char* const p = a.p + slot * kTriBytes;
    if constexpr (GRAD) {
#pragma unroll
        for (int s = 0; s < SN; ++s) mine[s] = TK::rows8(sk, 16 * own, s, lane);
    }
#pragma unroll
    for (int s2 = 0; s2 < 2; ++s2) {
        if (GRAD ? 2 * s2 + 1 < own : 2 * s2 > own) continue;
        float x[8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = 2 * s2 + half;
            f32x4_t d = zero;
            if (GRAD ? t >= own : t <= own) {
                const int c = 16 * t + 4 * lg, w = 16 * own + lr;
                d = product(GRAD ? sq : sk, t, mine) * (GRAD ? sums.behind(c, w, false) : sums.before(w, c, false)) * a.scale;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) x[4 * half + r] = d[r];
        }
        put_operand<T, GRAD ? kThree<T> : kTwo<T>>(p, GRAD ? tri_piece_t(own, s2) : tri_piece(own, s2), lane, x);
    }
    // keys of the wave's rows against all before: M
    if constexpr (!GRAD) {
#pragma unroll
        for (int s = 0; s < SN; ++s) mine[s] = TK::rows8(sk, 16 * wave, s, lane);
    }
    f32x4_t m[4];
#pragma unroll
    for (int tj = 0; tj < 4; ++tj)
        if (tj <= wave) m[tj] = product(sk, tj, mine) * sums.before(16 * wave + lr, 16 * tj + 4 * lg, true);
    __syncthreads();
#pragma unroll
    for (int tj = 0; tj < 4; ++tj) {
        if (tj > wave) continue;
        const int i = 16 * wave + lr, j = 16 * tj + 4 * lg;
        *reinterpret_cast<f32x4_t*>(sx + i * kLd + j) = m[tj] * *reinterpret_cast<const f32x4_t*>(s_beta + j);
        if constexpr (GRAD) *reinterpret_cast<f32x4_t*>(sz + i * kLd + j) = m[tj] * s_beta[i];
    }
    __syncthreads();
    invert(sx, wave, lane);
    if constexpr (GRAD) invert(sz, wave, lane);
    char* const xo = a.x + slot * kTriBytes;
#pragma unroll
    for (int s2 = 0; s2 < 2; ++s2) {
        float x[8];
        if (2 * s2 <= wave) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const f32x4_t v = *reinterpret_cast<const f32x4_t*>(sx + (16 * wave + lr) * kLd + 32 * s2 + 16 * half + 4 * lg);
#pragma unroll
                for (int r = 0; r < 4; ++r) x[4 * half + r] = 2 * s2 + half <= wave ? v[r] : 0.f;
            }
            put_operand<T, kThree<T>>(xo, tri_piece(wave, s2), lane, x);
        }
        if constexpr (GRAD) {
            if (2 * s2 + 1 >= wave) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = 2 * s2 + (e >> 2);
                    x[e] = t >= wave ? sz[(16 * t + 4 * lg + (e & 3)) * kLd + 16 * wave + lr] : 0.f;
                }
                put_operand<T, kThree<T>>(a.z + slot * kTriBytes, tri_piece_t(wave, s2), lane, x);
            }
        }
    }
}

// Walks: outputs, or (for the gradient) states and errors; backwards; and forwards
// and backwards over the segments of cut sequences, from zero (or, forwards, from the
// unit matrix), for what a segment does to a state alone.
enum : int { kGdrOut = 0, kGdrStates = 1, kGdrBack = 2, kGdrSeg = 3, kGdrBackSeg = 4 };
constexpr bool back_mode(int m) { return m == kGdrBack || m == kGdrBackSeg; }
constexpr bool reads_q(int m) { return m == kGdrOut || back_mode(m); }

// LDS of the walks: rows of k and q, 64 columns of v or dy, operand tiles of the
// inverse and the scores, the tables; twice where two fit (the next chunk's are
// then copied while this one is worked on).
template <typename T, int DK, int MODE> constexpr int walk_bytes() {
    return C * DK * (int)sizeof(T) * (reads_q(MODE) ? 2 : 1) + C * 64 * (int)sizeof(T) + kTri<T, kThree<T>> +
           (!reads_q(MODE) ? 0 : MODE == kGdrOut ? kTri<T, kTwo<T>> : kTri<T, kThree<T>>) + 1024;
}
template <typename T, int DK, int MODE> constexpr int walk_bufs() { return 2 * walk_bytes<T, DK, MODE>() <= 160 * 1024 ? 2 : 1; }

template <typename T, int DK> constexpr int walk_threads(int m) { return m == kGdrOut || (sizeof(T) == 4 && DK == 128) ? 512 : 256; }

template <int BYTES>
__device__ __forceinline__ void copy_flat(char* lds, const char* src, int wave, int lane) {
    static_assert(BYTES % 1024 == 0, "whole copies");
#pragma unroll
    for (int i = 0; i < (BYTES + 4095) / 4096; ++i)
        if ((i + 1) * 4096 <= BYTES || wave * 1024 + i * 4096 < BYTES)
            copy16(uni(lds_addr(lds) + wave * 1024 + i * 4096), src, (unsigned)(wave * 1024 + i * 4096 + lane * 16));
}

// A walk over a sequence's chunks: a workgroup has 64 value columns of a head, each of
// four waves 16 of them, the state (or its gradient) in its accumulators.  The walk
// that writes outputs has four more waves, which copy the next chunk's rows and
// operands to LDS: a wave stalls on a copy while the memory pipe is full.  It then
// reads operands where they are multiplied, for two waves of a SIMD have half the
// registers each (8192 tokens of 96 heads: 587 -> 492 us).  The others wait for their
// stores as well; there the four waves copy themselves, and read ahead (4 x 2048 tokens
// of 32 heads, with waves that copy: states 148 -> 165 us, backwards 210 -> 229),
// unless what they read ahead overfills the registers, in fp32 with 128 channels (the
// gradient of the same sizes: 3225 -> 1658 us, with all that came later 1606).
//
// What bounds it: a chunk's products follow one another (K S, E, the state), 182 of
// them a wave in 16 cycles each beside 580 other vector operations, most to split
// operands, in 6800 cycles: 3.4 us at 2 GHz.  Copies cost nothing of that any more.
// Those that keep states take 4.2 us a chunk, backwards 6.4, where they write 411 MB
// at 3.0 and 2.0 TB/s, half of what memory takes and less: the chain again.
template <typename T, int DK, int MODE>
__global__ __launch_bounds__((walk_threads<T, DK>(MODE)), (walk_threads<T, DK>(MODE) / 256)) void gdr_walk_kernel(GdrArgs a) {
    constexpr int SN = DK / 32, KT = DK / 16, N3 = kThree<T>, NPP = MODE == kGdrOut ? kTwo<T> : N3, NB = walk_bufs<T, DK, MODE>(), SZ = (int)sizeof(T);
    constexpr bool kBack = back_mode(MODE), kQ = reads_q(MODE), kKeep = MODE == kGdrStates || MODE == kGdrBack;
    constexpr bool kCopiers = walk_threads<T, DK>(MODE) == 512;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int lane0 = threadIdx.x & 63, wave = uni(threadIdx.x >> 6) & 3;
    int lane = lane0, lr = lane & 15, lg = lane >> 4;
    const int H = a.at.H, DV = a.head_v, slices = DV / 64 + (MODE == kGdrSeg ? DK / 64 : 0);
    constexpr bool kSeg = MODE == kGdrSeg || MODE == kGdrBackSeg;   // of the cut sequences alone
    const int chains = (kSeg ? a.cuts : a.seg.nblocks) * H;
    // the slices of a head read the same rows: 8 heads apart in the launch, so
    // that they run on one XCD
    const int wg = uni((int)(blockIdx.y * gridDim.x + blockIdx.x));
    if (wg >= chains * slices) return;
    const int group = uni(wg / (8 * slices)), rem = wg - group * 8 * slices;
    const int width = chains - group * 8 < 8 ? chains - group * 8 : 8;
    const int slice = uni(rem / width), chain = group * 8 + rem - slice * width;
    int sgm = uni(chain / H);
    const int h = chain - sgm * H;
    const Block sb = find_block<kGdrLeastSegments, kSeg>(a.seg, sgm);
    if (sb.n < 0) return;
    if constexpr (kSeg) {
        sgm = uni(first_block<kGdrLeastSegments>(a.seg, sb.n) + sb.j);
        if (sgm >= a.seg.nblocks) return;   // offsets out of order: stay inside the arrays
    }
    const bool first = sb.j == 0, last = sb.j == sb.nb - 1;
    const bool unit = MODE == kGdrSeg && slice * 64 >= DV;   // columns of the transition, not of values
    if (MODE == kGdrSeg && last && !(unit && a.seg_mt)) return;
    if (MODE == kGdrBackSeg && first) return;
    // (uni: else the compiler takes addresses for different in each lane)
    const int n = uni(sb.n), cnt = uni(sb.cnt);
    const int64_t begin = uni64(sb.start);
    const int fb = uni(first_block(a.at, n) + sb.j * (int)(a.seg.L / C));
    int nch = (cnt + C - 1) / C;
    nch = uni(nch < a.at.nblocks - fb ? nch : a.at.nblocks - fb);   // offsets out of order: stay inside the workspace
    const Rows rows{cnt, nch * C, false};
    const int col0 = unit ? slice * 64 - DV : slice * 64, wcol = 16 * wave;
    const int64_t DKV = (int64_t)DK * DV;

    Src xk, xq, xv, xo;
    xk.set((const T*)a.k.p, begin * a.k.stride + (int64_t)(h / a.k.share) * DK, a.k.stride);
    xq.set((const T*)a.q.p, begin * a.q.stride + (int64_t)(h / a.q.share) * DK, a.q.stride);
    if constexpr (kBack) xv.set((const T*)a.dy, (begin * H + h) * DV + col0, (int64_t)H * DV);
    else xv.set((const T*)a.v.p, begin * a.v.stride + (int64_t)h * DV + (unit ? 0 : col0), a.v.stride);
    if constexpr (MODE == kGdrOut) xo.set((const T*)a.y, (begin * H + h) * DV + col0, (int64_t)H * DV);
    const float scale = pin(a.scale);

    struct Buf {
        T *k, *q, *v;
        char *x, *p;
        float* tab;
    };
    auto buf = [&](int c) {
        char* at = smem + (NB == 2 ? (c & 1) * walk_bytes<T, DK, MODE>() : 0);
        Buf f;
        f.k = reinterpret_cast<T*>(at);
        at += C * DK * SZ;
        f.q = reinterpret_cast<T*>(at);
        if (kQ) at += C * DK * SZ;
        f.v = reinterpret_cast<T*>(at);
        at += C * 64 * SZ;
        f.x = at;
        at += kTri<T, N3>;
        f.p = at;
        if (kQ) at += kTri<T, NPP>;
        f.tab = reinterpret_cast<float*>(at);
        return f;
    };
    auto fetch = [&](int c) {
        const Buf f = buf(c);
        const int m0 = c * C;
        const int64_t slot = (int64_t)(fb + c) * H + h;
        copy_tile<T, DK>(f.k, xk, rows, m0, wave, lane);
        copy_tile<T, 64>(f.v, xv, rows, m0, wave, lane);
        copy_flat<kTri<T, N3>>(f.x, (kBack ? a.z : a.x) + slot * kTriBytes, wave, lane);
        if constexpr (kQ) {
            copy_tile<T, DK>(f.q, xq, rows, m0, wave, lane);
            copy_flat<kTri<T, NPP>>(f.p, a.p + slot * kTriBytes, wave, lane);
        }
        if (wave == 3) copy16(uni(lds_addr(f.tab)), a.tab + slot * kGdrTab, (unsigned)lane * 16);
    };
    auto chunk_at = [&](int step) { return kBack ? nch - 1 - step : step; };
    if (kCopiers && threadIdx.x >= 256) {
        for (int step = 0; step < nch; ++step) {
            if (NB == 1 || step == 0) fetch(chunk_at(step));
            wait_vmcnt<0>();
            barrier_keep_loads();                   // the chunk is there (two buffers: and the one before read)
            if (NB == 2 && step + 1 < nch) fetch(chunk_at(step + 1));
            if (NB == 1) barrier_keep_loads();      // it is read
        }
        return;
    }
    // channel of the state's tile i, row r of this lane
    auto channel = [&](int i, int r) { return 32 * (i >> 1) + 8 * lg + 4 * (i & 1) + r; };

    f32x4_t S[KT];
    {
        const float* s0 = nullptr;
        if (!kSeg) {
            s0 = sb.nb == 1 ? nullptr : kBack ? a.seg_r : a.seg_s;
            if (s0) s0 += ((int64_t)sgm * H + h) * DKV;
            else if ((s0 = kBack ? a.d_final : a.initial)) s0 += ((int64_t)n * H + h) * DKV;
            if (s0) s0 += col0 + wcol + lr;
        }
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S[i][r] = s0 ? s0[(int64_t)channel(i, r) * DV] : unit && channel(i, r) == col0 + wcol + lr ? 1.f : 0.f;
    }
    // Without copiers a chunk's operands are read from LDS a phase before they are
    // multiplied: a wave has its SIMD to itself, and nothing else hides the reads.  All of them are in
    // registers when the chunk's barrier comes, so that its buffer takes the copies of
    // the chunk after the next behind it, and the next one's rows of k are read.
    Frag8<T> kr[4][SN];
    auto read_k = [&](const Buf& f) {
#pragma unroll
        for (int s = 0; s < SN; ++s)
#pragma unroll
            for (int t = 0; t < 4; ++t) kr[t][s] = Tile<T, DK>::rows8(f.k, 16 * t, s, lane);
    };
    // stores between the copies of a chunk and the wait for them
    constexpr int NST = kKeep ? KT * 4 + 16 : 0;
    static_assert(NST < 64, "vmcnt");
    static_assert(kCopiers || NB == 2, "without copiers the chunk after the next needs a buffer");
    if (!kCopiers && nch > 0) {
        fetch(chunk_at(0));
        wait_vmcnt<0>();
        barrier_keep_loads();
        read_k(buf(chunk_at(0)));
        if (nch > 1) fetch(chunk_at(1));
    }
    for (int step = 0; step < nch; ++step) {
        const int c = chunk_at(step), m0 = c * C;
        const Buf f = buf(c);
        if constexpr (kCopiers) {
            barrier_keep_loads();
            // LDS addresses are formed anew in each chunk: kept across the loop they spill
            lane = lane0;
            asm volatile("" : "+v"(lane));
            lr = lane & 15;
            lg = lane >> 4;
        }
        const int64_t slot = (int64_t)(fb + c) * H + h;
        const float end = unif(f.tab[3 * C]);
        const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
        unsigned long long lost = 0;   // columns of a state that is not finite and that a decay of 0 ends here
        if (MODE == kGdrOut && end == 0.f) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) m += S[i][r] * 0.f;
            m += __shfl_xor(m, 16);
            m += __shfl_xor(m, 32);
            lost = __ballot(!(m == 0.f));
            if (!(m == 0.f)) {
#pragma unroll
                for (int i = 0; i < KT; ++i) S[i] = zero;
            }
        }
        if constexpr (kKeep) {
            // the state before the chunk, or the gradient behind it
            float* const dst = (kBack ? a.rstates : a.states) + slot * DKV + col0 + wcol;
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(dst, 0, (unsigned)(DKV * 4), 0x00027000);
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][r]), rsrc,
                                                          (unsigned)((channel(i, r) * DV + lr) * 4), 0, 0);
        }
        // A: K S (or K R), a lane 4 tokens of a column; X (Z), P^T, the tables and v (dy) come
        Frag8<T> fx[6][N3], fp[6][NPP], fs[SN][N3];
        auto read_x = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 6; ++i) get_operand<T, N3>(f.x, i, lane, fx[i]);
        };
        if constexpr (!kCopiers) read_x();
        if constexpr (kBack) {
#pragma unroll
            for (int i = 0; i < 6; ++i) get_operand<T, NPP>(f.p, i, lane, fp[i]);
        }
        f32x4_t in[4], out[4], beta[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            in[t] = *reinterpret_cast<const f32x4_t*>(f.tab + 16 * t + 4 * lg);
            out[t] = *reinterpret_cast<const f32x4_t*>(f.tab + C + 16 * t + 4 * lg);
            beta[t] = *reinterpret_cast<const f32x4_t*>(f.tab + 2 * C + 16 * t + 4 * lg);
        }
        // the wave's columns of v (or dy), a lane 4 tokens of each tile
        Frag8<T> fv[2] = {Tile<T, 64>::cols(f.v, wcol, 0, lane), Tile<T, 64>::cols(f.v, wcol, 1, lane)};
        if (unit) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                fv[0].set(j, 0.f);
                fv[1].set(j, 0.f);
            }
        }
        f32x4_t ks[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int s = 0; s < SN; ++s) {
            float x[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[r] = S[2 * s][r];
                x[4 + r] = S[2 * s + 1][r];
            }
            if constexpr (kCopiers) {
#pragma unroll
                for (int t = 0; t < 4; ++t) kr[t][s] = Tile<T, DK>::rows8(f.k, 16 * t, s, lane);
            }
            split(x, fs[s]);
#pragma unroll
            for (int p = N3 - 1; p >= 0; --p)
#pragma unroll
                for (int t = 0; t < 4; ++t) ks[t] = mma(kr[t][s], fs[s][p], ks[t]);
        }
        if (end == 0.f) {
#pragma unroll
            for (int i = 0; i < KT; ++i) S[i] = zero;
        } else {
#pragma unroll
            for (int i = 0; i < KT; ++i) S[i] *= end;
        }
        if constexpr (!kCopiers) __builtin_amdgcn_sched_barrier(0);
        // B: V - exp(G) K S, or P^T dY + exp(G_63 - G) K R; rows of q come (backwards: its columns)
        Frag8<T> fq[kBack ? KT : 4][kBack ? 2 : SN];
        if constexpr (kBack) {
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
                for (int i = 0; i < KT; ++i) fq[i][s2] = cols8<T, DK>(f.q, i >> 1, i & 1, s2, lane);
        }
        // two 16-token tiles as an operand in parts
        auto operand = [&](const f32x4_t& lo, const f32x4_t& hi, auto& o) {
            float x[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[r] = lo[r];
                x[4 + r] = hi[r];
            }
            split(x, o);
        };
        f32x4_t e[4];
        Frag8<T> fe[2][N3];
        if constexpr (!kBack) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) e[t][r] = fv[t >> 1].get(4 * (t & 1) + r) - in[t][r] * ks[t][r];
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) e[t] = out[t] * ks[t];
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
                for (int p = NPP - 1; p >= 0; --p)
#pragma unroll
                    for (int t = 0; t < 2 * s2 + 2; ++t) e[t] = mma(fp[tri_piece_t(t, s2)][p], fv[s2], e[t]);
        }
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) operand(e[2 * s2], e[2 * s2 + 1], fe[s2]);
        if constexpr (!kCopiers) __builtin_amdgcn_sched_barrier(0);
        // C: E (or U); the columns of k come.  Beside it what does not wait for E: y's part of
        // the entering state, transposed tiles, a lane 4 columns of token 16 t + l % 16; or dY's
        // part of R
        Frag8<T> fk[KT][2];
        auto read_cols = [&](int s2) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < KT; ++i) fk[i][s2] = cols8<T, DK>(f.k, i >> 1, i & 1, s2, lane);
        };
        if constexpr (kCopiers) {
            read_x();
        } else {
            read_cols(0);
            read_cols(1);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) e[t] = zero;
#pragma unroll
        for (int s = N3 - 1; s >= 0; --s)
#pragma unroll
            for (int i = 0; i <= s; ++i)
#pragma unroll
                for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        if (kBack ? 2 * s2 + 1 >= t : 2 * s2 <= t)
                            e[t] = mma(fx[kBack ? tri_piece_t(t, s2) : tri_piece(t, s2)][i], fe[s2][s - i], e[t]);
        f32x4_t y[4] = {zero, zero, zero, zero};
        float into[4];
        if constexpr (MODE == kGdrOut) {
#pragma unroll
            for (int t = 0; t < 4; ++t) into[t] = f.tab[16 * t + lr];
            // the state's leading 16 bits
#pragma unroll
            for (int s = 0; s < SN; ++s) {
#pragma unroll
                for (int t = 0; t < 4; ++t) fq[t][s] = Tile<T, DK>::rows8(f.q, 16 * t, s, lane);
#pragma unroll
                for (int p = NPP - 1; p >= 0; --p)
#pragma unroll
                    for (int t = 0; t < 4; ++t) y[t] = mma(fs[s][p], fq[t][s], y[t]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) y[t] *= into[t] * scale;
        } else if constexpr (kBack) {
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2) {
                Frag8<T> u[N3];
                f32x4_t d[2];
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int r = 0; r < 4; ++r) d[half][r] = fv[s2].get(4 * half + r) * (in[2 * s2 + half][r] * scale);
                operand(d[0], d[1], u);
#pragma unroll
                for (int p = N3 - 1; p >= 0; --p)
#pragma unroll
                    for (int i = 0; i < KT; ++i) S[i] = mma(fq[i][s2], u[p], S[i]);
            }
        }
        if constexpr (kKeep) {
            float* const dst = (kBack ? a.u : a.errors) + slot * C * DV + col0 + wcol;
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(dst, 0, (unsigned)(C * DV * 4), 0x00027000);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(e[t][r]), rsrc,
                                                          (unsigned)(((16 * t + 4 * lg + r) * DV + lr) * 4), 0, 0);
        }
        if constexpr (!kCopiers) {
            // the next chunk's copies are there, this one's operands in registers
            wait_vmcnt<NST>();
            barrier_keep_loads();
            if (step + 2 < nch) fetch(chunk_at(step + 2));
            if (step + 1 < nch) read_k(buf(chunk_at(step + 1)));
        }
        // D: the chunk's own part of y, and of the state behind it (or of the gradient before it)
#pragma unroll
        for (int t = 0; t < 4; ++t) e[t] *= beta[t];
        if constexpr (MODE == kGdrOut) {
            Frag8<T> fb[2][NPP];
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2) operand(e[2 * s2], e[2 * s2 + 1], fb[s2]);
#pragma unroll
            for (int i = 0; i < 6; ++i) get_operand<T, NPP>(f.p, i, lane, fp[i]);
#pragma unroll
            for (int s = NPP - 1; s >= 0; --s)
#pragma unroll
                for (int i = 0; i <= s; ++i)
#pragma unroll
                    for (int s2 = 0; s2 < 2; ++s2)
#pragma unroll
                        for (int t = 2 * s2; t < 4; ++t) y[t] = mma(fb[s2][i], fp[tri_piece(t, s2)][s - i], y[t]);
        }
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) {
            Frag8<T> u[N3];
            if constexpr (kCopiers) read_cols(s2);
            if constexpr (!kBack) operand(out[2 * s2] * e[2 * s2], out[2 * s2 + 1] * e[2 * s2 + 1], u);
            else operand(-(in[2 * s2] * e[2 * s2]), -(in[2 * s2 + 1] * e[2 * s2 + 1]), u);
#pragma unroll
            for (int p = N3 - 1; p >= 0; --p)
#pragma unroll
                for (int i = 0; i < KT; ++i) S[i] = mma(fk[i][s2], u[p], S[i]);
        }
        if constexpr (MODE == kGdrOut) {
            // rows without a token lie behind the bound and are dropped
            const unsigned step_o = xo.step;
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(xo.token(m0)), 0,
                                                                uni((unsigned)(rows.tokens(m0) - 1) * step_o + 64 * SZ), 0x00027000);
            auto store = [&](int t, const f32x4_t& v) {
                const unsigned at = (unsigned)(16 * t + lr) * step_o + (unsigned)((wcol + 4 * lg) * SZ);
                if constexpr (SZ == 4) {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rsrc, at, 0, 0);
                } else {
                    const u32x2_t o = {cvt2(v[0], v[1]), cvt2(v[2], v[3])};
                    __builtin_amdgcn_raw_buffer_store_b64(o, rsrc, at, 0, 0);
                }
            };
#pragma unroll
            for (int t = 0; t < 4; ++t) store(t, y[t]);
            if (lost) {   // once more, with what the lost state has made of the tokens before its end
#pragma unroll
                for (int t = 0; t < 4; ++t) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if ((lost >> (4 * lg + r) & 1) && into[t] != 0.f) y[t][r] = __builtin_nanf("");
                    store(t, y[t]);
                }
            }
        }
        if (kCopiers && NB == 1) barrier_keep_loads();
    }
    if (unit) {
        const int col = col0 + wcol + lr;
        const int64_t at = ((int64_t)sgm * H + h) * DK * DK;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) a.seg_m[at + channel(i, r) * DK + col] = S[i][r];
            if (a.seg_mt) *reinterpret_cast<f32x4_t*>(a.seg_mt + at + col * DK + channel(i, 0)) = S[i];
        }
        return;
    }
    float* dst = nullptr;
    if (kSeg) dst = (kBack ? a.seg_r : a.seg_s) + ((int64_t)sgm * H + h) * DKV;
    else if (kBack ? first : last) dst = kBack ? a.d_initial : a.final;
    if (dst) {
        if (!kSeg) dst += ((int64_t)n * H + h) * DKV;
        dst += col0 + wcol + lr;
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) dst[(int64_t)channel(i, r) * DV] = S[i][r];
    }
}

// The states that enter the segments of a (sequence, head), 64 columns, in place of
// the segments' own ones: S_{j+1} = M_j S_j + own_j from the sequence's initial state
// (backwards R_{j-1} = M_j^T R_j + own_j).  A wave has 16 columns; matrices and
// states enter the products with 24 bits.  A segment takes 13 us with 128 channels, 8
// with 64: latency, since each wave reads the segment's matrix as it multiplies.
template <int DK>
__global__ __launch_bounds__(256, 1) void gdr_join_kernel(GdrArgs a, int backwards) {
    constexpr int SN = DK / 32, KT = DK / 16;
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), lr = lane & 15, lg = lane >> 4;
    const int H = a.at.H, DV = a.head_v, n = uni(blockIdx.x / H), h = blockIdx.x - n * H;
    const int64_t DKV = (int64_t)DK * DV;
    const int col = blockIdx.y * 64 + 16 * wave + lr;
    int nb = uni(blocks_of<kGdrLeastSegments>(a.seg, seq_at(a.seg, n + 1) - seq_at(a.seg, n)));
    if (nb == 1) return;   // not cut: the walk begins with the sequence's own state
    const int b0 = uni(first_block<kGdrLeastSegments>(a.seg, n));
    nb = nb < a.seg.nblocks - b0 ? nb : a.seg.nblocks - b0;   // offsets out of order: stay inside the arrays
    const float* const m = backwards ? a.seg_mt : a.seg_m;
    float* const own = backwards ? a.seg_r : a.seg_s;
    auto channel = [&](int i, int r) { return 32 * (i >> 1) + 8 * lg + 4 * (i & 1) + r; };
    f32x4_t S[KT];
    const float* s0 = backwards ? a.d_final : a.initial;
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[i][r] = s0 ? s0[((int64_t)n * H + h) * DKV + (int64_t)channel(i, r) * DV + col] : 0.f;
    for (int step = 0; step < nb; ++step) {
        const int64_t slot = (int64_t)(b0 + (backwards ? nb - 1 - step : step)) * H + h;
        const bool more = step + 1 < nb;
        float* const p = own + slot * DKV + col;
        f32x4_t next[KT];
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t at = (int64_t)channel(i, r) * DV;
                next[i][r] = more ? p[at] : 0.f;
                p[at] = S[i][r];
            }
        if (!more) break;
        float sick = 0.f;
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) sick += S[i][r] * 0.f;
        if (__any(!(sick == 0.f))) {
            // a state that is not finite ends where a decay of 0 made the segment's matrix zero
            unsigned bits = 0;
            for (int e = 4 * lane; e < DK * DK; e += 256) {
                const u32x4_t v = *reinterpret_cast<const u32x4_t*>(m + slot * DK * DK + e);
                bits |= (v[0] | v[1] | v[2] | v[3]) << 1;
            }
            if (!__any(bits != 0)) {
#pragma unroll
                for (int i = 0; i < KT; ++i) S[i] = next[i];
                continue;
            }
        }
        Frag8<__bf16> fs[SN][3];
#pragma unroll
        for (int s = 0; s < SN; ++s) {
            float x[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[r] = S[2 * s][r];
                x[4 + r] = S[2 * s + 1][r];
            }
            split(x, fs[s]);
        }
        // a tile's rows are its channels
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int row = 32 * (i >> 1) + 8 * (lr >> 2) + 4 * (i & 1) + (lr & 3);
#pragma unroll
            for (int s = 0; s < SN; ++s) {
                float x[8];
                load8(m + slot * DK * DK + row * DK + 32 * s + 8 * lg, x);
                Frag8<__bf16> f[3];
                split(x, f);
                next[i] = mma_parts(f, fs[s], next[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < KT; ++i) S[i] = next[i];
    }
}

// dQ, dK, dV in the inputs' type (dQ and dK of shared key heads: each value head's
// part in fp32), dbeta and dg of a (chunk, head).
//
// 64 value columns at a time the rows of E, dV = beta U and dY are laid out in LDS as
// operands in parts; each wave adds to its tiles of W and Y (rows i = its own against
// all before, and all behind against its own as j) and, for its DK / 4 channels, to
// the states' parts, whose rows are operands as they lie in memory.  W and Y then
// take the rows' place, and q that of k.  In bf16 two workgroups share a CU: one
// loads while the other multiplies (4 x 2048 tokens of 32 heads: 430 us with all value
// columns at once and one workgroup a CU, 295 so; with dg made here, which needs 24 bits
// in E, dV, S and R, 341, and a kernel of 35 for dg less).  It moves 726 MB, 2.1 TB/s, with
// matrix instructions 27 % and vector ones 42 % of the time, and waits for 53 % of it:
// states are asked for right before they are multiplied.
template <typename T, int DK>
struct GradLds {
    static constexpr int SZ = (int)sizeof(T), N2 = kTwo<T>, N3 = kThree<T>, TRI = kTri<T, N2>, ROWS = C * 64 * SZ;
    static constexpr int k = 0, rest = C * DK * SZ;
    static constexpr int e = rest, x = e + N3 * ROWS, y = x + N3 * ROWS, first = y + ROWS;
    static constexpr int w = rest, second = w + 4 * TRI;                              // over the rows, once they are read
    static constexpr int dq = rest, dk = dq + C * DK * SZ, third = dk + C * DK * SZ;   // over those, at the end
    static constexpr int most = first > second ? first : second, bytes = most > third ? most : third;
};

template <typename T, int DK, int DV>
__global__ __launch_bounds__(256, sizeof(T) == 2 || DK == 64 ? 2 : 1) void gdr_grad_kernel(GdrArgs a) {
    typedef GradLds<T, DK> Lds;
    typedef Tile<T, 64> TV;
    typedef Tile<T, DK> TK;
    constexpr int SK = DK / 32, NT = DK / 64, N2 = kTwo<T>, N3 = kThree<T>, EP = 16 / (int)sizeof(T), TRI = kTri<T, N2>;
    constexpr int NQ = C * DK / EP / 256;               // runs of 16 bytes of a thread, of k and of q
    extern __shared__ __attribute__((aligned(16))) char smem[];
    T* const sk = reinterpret_cast<T*>(smem + Lds::k);
    T* const se = reinterpret_cast<T*>(smem + Lds::e);
    T* const sx = reinterpret_cast<T*>(smem + Lds::x);
    T* const sy = reinterpret_cast<T*>(smem + Lds::y);
    char* const wy = smem + Lds::w;                     // W beta and Y beta, rows i, then rows j
    __shared__ Sums sums;
    __shared__ __attribute__((aligned(16))) float tab[3 * C];
    __shared__ float part_q[4][C], part_k[4][C], part_b[4][C], part_n[4][C];   // of a wave: q.S dy, k.S dv, k.R e; pairs
    __shared__ double part_c[4];                                                // <S, R>
    int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
    const int wave = uni(tid >> 6);
    // LDS addresses are formed anew in each part: kept from part to part they spill
    auto anew = [&] {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" : "+v"(tid));
        lane = tid & 63;
        lr = lane & 15;
        lg = lane >> 4;
    };
    const int H = a.at.H, r_heads = a.k.share, b = uni(blockIdx.x / H), h = blockIdx.x - b * H, hk = uni(h / r_heads);
    const Block bl = find_block(a.at, b);
    if (bl.n < 0 || bl.cnt == 0) return;
    const int cnt = uni(bl.cnt);
    const int64_t start = uni64(bl.start), slot = (int64_t)b * H + h;
    const T* const gk = (const T*)a.k.p + start * a.k.stride + (int64_t)hk * DK;
    const T* const gq = (const T*)a.q.p + start * a.q.stride + (int64_t)hk * DK;
    auto row_of = [&](int row) { return row < cnt ? row : cnt - 1; };   // rows without a token: the last one's
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int u = i * 256 + tid, row = u / (DK / EP), col = u % (DK / EP) * EP;
        *reinterpret_cast<u32x4_t*>(sk + TK::off(row, col)) =
            *reinterpret_cast<const u32x4_t*>(gk + (int64_t)row_of(row) * a.k.stride + col);
    }
    const float* const gtab = a.tab + slot * kGdrTab;
    if (tid < 3 * C) tab[tid] = gtab[tid];
    if (tid < C) {
        sums.frac[tid] = gtab[4 * C + tid];
        sums.whole[tid] = __float_as_int(gtab[5 * C + tid]);
    }
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    // tiles of W and Y: wave + 1 with its rows as i, 4 - wave with them as j
    f32x4_t w[5], y[5];
#pragma unroll
    for (int m = 0; m < 5; ++m) w[m] = y[m] = zero;
    f32x4_t ps[4][NT], pa[4][NT], pb[4][NT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) ps[t][n] = pa[t][n] = pb[t][n] = zero;
    const int ch0 = wave * (DK / 4);
    float eu[2] = {0.f, 0.f};
    double across = 0.0;
    auto rows_of = [&](const T* base, int t, int s, auto& f) {   // 8 consecutive columns a lane, in parts
        constexpr int N = sizeof(f) / sizeof(f[0]);
#pragma unroll
        for (int p = 0; p < N; ++p) f[p] = TV::rows8(base + p * C * 64, 16 * t, s, lane);
    };
    // (a loop also where it runs once: unrolled, all of its loads are asked for at the start, and spill)
    int columns = DV;
    if constexpr (DV == 64) asm volatile("" : "+s"(columns));
#pragma unroll 1
    for (int v0 = 0; v0 < columns; v0 += 64) {
        if (v0 > 0) __syncthreads();
        anew();
        // rows to LDS, and dv; e.u by tokens
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int u = i * 256 + tid, row = u / 8, lc = u % 8 * 8, col = v0 + lc;
            const int64_t tok = start + row_of(row), at = slot * C * DV + row * DV + col;
            float e[8], x[8];
            load8(a.errors + at, e);
            load8(a.u + at, x);
            const T* const py = (const T*)a.dy + (tok * H + h) * DV + col;
            const float be = gtab[2 * C + row];
#pragma unroll
            for (int c = 0; c < 8; c += EP)
                *reinterpret_cast<u32x4_t*>(sy + TV::off(row, lc + c)) = *reinterpret_cast<const u32x4_t*>(py + c);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                eu[i] += e[j] * x[j];
                x[j] *= be;
            }
            if constexpr (sizeof(T) == 2) {
                Frag8<T> fe[N3], fx[N3];
                split(e, fe);
                split(x, fx);
#pragma unroll
                for (int p = 0; p < N3; ++p) {
                    *reinterpret_cast<bf16x8_t*>(se + p * C * 64 + TV::off(row, lc)) = fe[p].v;
                    *reinterpret_cast<bf16x8_t*>(sx + p * C * 64 + TV::off(row, lc)) = fx[p].v;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 8; c += 4) {
                    *reinterpret_cast<f32x4_t*>(se + TV::off(row, lc + c)) = f32x4_t{e[c], e[c + 1], e[c + 2], e[c + 3]};
                    *reinterpret_cast<f32x4_t*>(sx + TV::off(row, lc + c)) = f32x4_t{x[c], x[c + 1], x[c + 2], x[c + 3]};
                }
            }
            if (row < cnt) {
                T* const o = (T*)a.dv_out + (tok * H + h) * DV + col;
#pragma unroll
                for (int c = 0; c < 8; c += EP) {
                    float f[EP];
#pragma unroll
                    for (int j = 0; j < EP; ++j) f[j] = x[c + j];
                    store_vec<T, EP>(o + c, f);
                }
            }
        }
        __syncthreads();
        anew();
        {
            // the wave's rows, as i (these make dg's pairs too, an fp32 output's) and as j
            Frag8<T> fy[2][1], fx[2][N3], fe[2][N2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                rows_of(sy, wave, s, fy[s]);
                rows_of(sx, wave, s, fx[s]);
                rows_of(se, wave, s, fe[s]);
            }
#pragma unroll
            for (int m = 0; m < 5; ++m) {
                if (m <= wave) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        Frag8<T> e3[N3];
                        rows_of(se, m, s, e3);
                        w[m] = mma_parts(e3, fy[s], w[m]);
                        y[m] = mma_parts(e3, fx[s], y[m]);
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        Frag8<T> y1[1], x2[N2];
                        rows_of(sy, m - 1, s, y1);
                        rows_of(sx, m - 1, s, x2);
                        w[m] = mma_parts(y1, fe[s], w[m]);
                        y[m] = mma_parts(x2, fe[s], y[m]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // the states' parts, the wave's channels
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            anew();
            float z[NT][8];
            Frag8<T> f[NT][N3];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int64_t at = slot * DK * DV + (int64_t)(ch0 + 16 * n + lr) * DV + v0 + 32 * s + 8 * lg;
                float x[8];
                load8(a.states + at, x);
                load8(a.rstates + at, z[n]);
#pragma unroll
                for (int j = 0; j < 8; ++j) across += (double)x[j] * (double)z[n][j];
                split(x, f[n]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                Frag8<T> fy[1], fx[N3];
                rows_of(sy, t, s, fy);
                rows_of(sx, t, s, fx);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    ps[t][n] = mma_parts(fy, f[n], ps[t][n]);
                    pa[t][n] = mma_parts(fx, f[n], pa[t][n]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) split(z[n], f[n]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                Frag8<T> fe[N3];
                rows_of(se, t, s, fe);
#pragma unroll
                for (int n = 0; n < NT; ++n) pb[t][n] = mma_parts(fe, f[n], pb[t][n]);
            }
        }
    }
    anew();
    // W and Y: decays, beta; what the pairs of the wave's rows j carry across each token t: the
    // sums of N_ji over i < t, for t <= j, then over the rows.  Sums only ever grow towards
    // the nearer, larger pairs: nothing is taken away again
    {
        const int own = 16 * wave + lr;
        float before = 0.f;
        Frag8<T> fq[SK], fo[SK];
#pragma unroll
        for (int s = 0; s < SK; ++s) {
            fq[s] = frag_at(gq + (int64_t)row_of(own) * a.q.stride + 32 * s + 8 * lg);
            fo[s] = TK::rows8(sk, 16 * wave, s, lane);
        }
#pragma unroll
        for (int m = 0; m < 5; ++m) {
            if (m <= wave) {
                const int j = 16 * m + 4 * lg;
                const f32x4_t be = *reinterpret_cast<const f32x4_t*>(tab + 2 * C + j);
                f32x4_t qk = zero, kk = zero;
#pragma unroll
                for (int s = 0; s < SK; ++s) {
                    const Frag8<T> f = TK::rows8(sk, 16 * m, s, lane);
                    qk = mma(f, fq[s], qk);
                    kk = mma(f, fo[s], kk);
                }
                w[m] *= sums.before(own, j, false) * be * a.scale;
                y[m] *= sums.before(own, j, true) * -be;
                const f32x4_t n = w[m] * qk + y[m] * kk;
                // of the lane groups before this one, and of all four
                float upto = (n[0] + n[1]) + (n[2] + n[3]);
                float x = __shfl_up(upto, 16);
                upto += lg >= 1 ? x : 0.f;
                x = __shfl_up(upto, 32);
                upto += lg >= 2 ? x : 0.f;
                x = __shfl_up(upto, 16);
                f32x4_t p;
                p[0] = before + (lg >= 1 ? x : 0.f);
#pragma unroll
                for (int r = 1; r < 4; ++r) p[r] = p[r - 1] + n[r - 1];
                before += __shfl(upto, 48 + lr);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float u = row16_sum(j + r <= own ? p[r] : 0.f);
                    if (lr == 0) part_n[wave][j + r] = u;
                }
            } else {
                const float be = tab[2 * C + own];
                w[m] *= sums.behind(16 * (m - 1) + 4 * lg, own, false) * (be * a.scale);
                y[m] *= sums.behind(16 * (m - 1) + 4 * lg, own, true) * -be;
            }
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) across += shfl_d(across, lane ^ d);
    if (lane == 0) part_c[wave] = across * (double)gtab[3 * C];
    // over the 8 threads of a row
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = (i * 256 + tid) / 8;
        eu[i] += dpp_mov<0xB1>(eu[i]);
        eu[i] += dpp_mov<0x4E>(eu[i]);
        eu[i] += dpp_mov<0x141>(eu[i]);
        if (tid % 8 == 0 && row < cnt) a.dbeta[(start + row) * H + h] = eu[i];
    }
    anew();
    u32x4_t rq[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int u = i * 256 + tid, row = u / (DK / EP), col = u % (DK / EP) * EP;
        rq[i] = *reinterpret_cast<const u32x4_t*>(gq + (int64_t)row_of(row) * a.q.stride + col);
    }
    __syncthreads();
    // W and Y over the rows, each piece's other half zeros where it lies beyond the diagonal
#pragma unroll
    for (int m = 0; m < 5; ++m) {
        const bool before = m <= wave;
        char* const at = wy + (before ? 0 : 2 * TRI);
        const int t = before ? m : m - 1, piece = before ? tri_piece(wave, t >> 1) : tri_piece_t(wave, t >> 1);
        put_half<T>(at, piece, t & 1, lane, w[m]);
        put_half<T>(at + TRI, piece, t & 1, lane, y[m]);
    }
    {
        char* const at = wy + (wave & 1 ? 2 * TRI : 0);
        const int piece = wave & 1 ? tri_piece_t(wave, wave >> 1) : tri_piece(wave, wave >> 1);
        put_half<T>(at, piece, !(wave & 1), lane, zero);
        put_half<T>(at + TRI, piece, !(wave & 1), lane, zero);
    }
    Frag8<T> fk[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) fk[n][s2] = TK::cols(sk, ch0 + 16 * n, s2, lane);
    __syncthreads();
    // q over k
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int u = i * 256 + tid;
        *reinterpret_cast<u32x4_t*>(sk + TK::off(u / (DK / EP), u % (DK / EP) * EP)) = rq[i];
    }
    anew();
    f32x4_t dk[4][NT];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const f32x4_t in = *reinterpret_cast<const f32x4_t*>(tab + 16 * t + 4 * lg);
        const f32x4_t out = *reinterpret_cast<const f32x4_t*>(tab + C + 16 * t + 4 * lg);
        const f32x4_t beta = *reinterpret_cast<const f32x4_t*>(tab + 2 * C + 16 * t + 4 * lg);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            ps[t][n] *= in * a.scale;
            pa[t][n] *= in;
            pb[t][n] *= out * beta;
            dk[t][n] = pb[t][n] - pa[t][n];
        }
        // k . (state's parts of dk)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float u = 0.f, v = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float f = fk[n][t >> 1].get(4 * (t & 1) + r);
                u += f * pa[t][n][r];
                v += f * pb[t][n][r];
            }
            u = row16_sum(u);
            v = row16_sum(v);
            if (lr == 0) {
                part_k[wave][16 * t + 4 * lg + r] = u;
                part_b[wave][16 * t + 4 * lg + r] = v;
            }
        }
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) {
            Frag8<T> f[N2];
            if (2 * s2 <= t) {
                get_operand<T, N2>(wy + TRI, tri_piece(t, s2), lane, f);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const Frag8<T> bk[1] = {fk[n][s2]};
                    dk[t][n] = mma_parts(f, bk, dk[t][n]);
                }
            }
            if (2 * s2 + 1 >= t) {
                get_operand<T, N2>(wy + 3 * TRI, tri_piece_t(t, s2), lane, f);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const Frag8<T> bk[1] = {fk[n][s2]};
                    dk[t][n] = mma_parts(f, bk, dk[t][n]);
                }
            }
        }
    }
    __syncthreads();
    Frag8<T> fq[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) fq[n][s2] = TK::cols(sk, ch0 + 16 * n, s2, lane);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        // q . (state's part of dq)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float u = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) u += fq[n][t >> 1].get(4 * (t & 1) + r) * ps[t][n][r];
            u = row16_sum(u);
            if (lr == 0) part_q[wave][16 * t + 4 * lg + r] = u;
        }
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) {
            Frag8<T> f[N2];
            if (2 * s2 <= t) {
                get_operand<T, N2>(wy, tri_piece(t, s2), lane, f);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const Frag8<T> bk[1] = {fk[n][s2]};
                    ps[t][n] = mma_parts(f, bk, ps[t][n]);
                }
            }
            if (2 * s2 + 1 >= t) {
                get_operand<T, N2>(wy + 2 * TRI, tri_piece_t(t, s2), lane, f);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const Frag8<T> bq[1] = {fq[n][s2]};
                    dk[t][n] = mma_parts(f, bq, dk[t][n]);
                }
            }
        }
    }
    __syncthreads();
    if (wave == 0 && a.dg) {
        // a token a lane: what enters with the state and is read from here on, what was written before
        // and goes on behind the chunk, the pairs, and what passes the whole chunk
        const int t = lane;
        double from = 0.0, until = 0.0, n = 0.0;
#pragma unroll
        for (int w4 = 0; w4 < 4; ++w4) {
            from += (double)part_q[w4][t] - (double)part_k[w4][t];
            until += (double)part_b[w4][t];
            if (16 * w4 + 15 >= t) n += (double)part_n[w4][t];
        }
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const double x = shfl_d(from, t + d < kWave ? t + d : t), y = shfl_d(until, t >= d ? t - d : t);
            if (t + d < kWave) from += x;
            if (t >= d) until += y;
        }
        until = shfl_d(until, t > 0 ? t - 1 : 0);
        if (t == 0) until = 0.0;
        const double all = (part_c[0] + part_c[1]) + (part_c[2] + part_c[3]);
        if (t < cnt) a.dg[(start + t) * H + h] = (float)((n + from) + (until + all));
    }
    if (a.parts) {
        // shared key heads: each value head's part
        const int64_t all = a.at.T_total * H * DK;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * t + 4 * lg + r;
                if (row >= cnt) continue;
                float* const at = a.parts + ((start + row) * H + h) * DK + ch0 + lr;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    at[16 * n] = ps[t][n][r];
                    at[all + 16 * n] = dk[t][n][r];
                }
            }
        return;
    }
    // whole rows of dq and dk through LDS
    T* const oq = reinterpret_cast<T*>(smem + Lds::dq);
    T* const ok = reinterpret_cast<T*>(smem + Lds::dk);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int at = TK::off(16 * t + 4 * lg + r, ch0 + 16 * n + lr);
                oq[at] = from_f32<T>(ps[t][n][r]);
                ok[at] = from_f32<T>(dk[t][n][r]);
            }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int u = i * 256 + tid, row = u / (DK / EP), col = u % (DK / EP) * EP;
        if (row >= cnt) continue;
        const int64_t at = ((start + row) * H + h) * DK + col;
        *reinterpret_cast<u32x4_t*>((T*)a.dq + at) = *reinterpret_cast<const u32x4_t*>(oq + TK::off(row, col));
        *reinterpret_cast<u32x4_t*>((T*)a.dk + at) = *reinterpret_cast<const u32x4_t*>(ok + TK::off(row, col));
    }
}

// dq and dk of key heads that value heads share: the sums of these heads' parts.
template <typename T>
__global__ __launch_bounds__(256) void gdr_share_kernel(GdrArgs a, int D) {
    const int r = a.k.share, Hk = a.at.H / r, per = Hk * (D / 4);   // runs of 4 of a token
    const int64_t t0 = seq_at(a.at, 0), t1 = seq_at(a.at, a.at.num_seqs), n4 = a.at.T_total * per, all = a.at.T_total * a.at.H * D;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < 2 * n4; u += (int64_t)gridDim.x * 256) {
        const int64_t i = u < n4 ? u : u - n4, tok = i / per;
        if (tok < t0 || tok >= t1) continue;
        const float* const p = a.parts + (u < n4 ? 0 : all) + (i / (D / 4)) * r * D + i % (D / 4) * 4;
        f32x4_t s = *reinterpret_cast<const f32x4_t*>(p);
        for (int j = 1; j < r; ++j) s += *reinterpret_cast<const f32x4_t*>(p + (int64_t)j * D);
        const float o[4] = {s[0], s[1], s[2], s[3]};
        store_vec<T, 4>((T*)(u < n4 ? a.dq : a.dk) + i * 4, o);
    }
}

template <typename T, int DK, bool GRAD>
hipError_t prep_t(const GdrArgs& a) {
    if (a.at.T_total == 0) return hipSuccess;
    constexpr int lds = prep_bytes<T, DK, GRAD>();
    const void* kern = reinterpret_cast<const void*>(&gdr_prep_kernel<T, DK, GRAD>);
    const hipError_t e = ensure_lds_limit(kern, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gdr_prep_kernel<T, DK, GRAD>), dim3((unsigned)((int64_t)a.at.nblocks * a.at.H)), dim3(256), lds,
                       (hipStream_t)a.at.stream, a);
    return hipGetLastError();
}

template <typename T, int DK, int MODE>
hipError_t walk_t(const GdrArgs& a) {
    constexpr int lds = walk_bytes<T, DK, MODE>() * walk_bufs<T, DK, MODE>();
    static_assert(lds <= 160 * 1024, "LDS");
    const void* kern = reinterpret_cast<const void*>(&gdr_walk_kernel<T, DK, MODE>);
    const hipError_t e = ensure_lds_limit(kern, lds);
    if (e != hipSuccess) return e;
    const int64_t groups = (int64_t)(MODE == kGdrSeg || MODE == kGdrBackSeg ? a.cuts : a.seg.nblocks) * a.at.H *
                           (a.head_v / 64 + (MODE == kGdrSeg ? DK / 64 : 0));
    hipLaunchKernelGGL((gdr_walk_kernel<T, DK, MODE>), folded_grid(groups), dim3((walk_threads<T, DK>(MODE))), lds,
                       (hipStream_t)a.at.stream, a);
    return hipGetLastError();
}

template <int DK>
hipError_t join(const GdrArgs& a, int backwards) {
    hipLaunchKernelGGL((gdr_join_kernel<DK>), dim3((unsigned)(a.at.num_seqs * a.at.H), (unsigned)(a.head_v / 64)), dim3(256),
                       0, (hipStream_t)a.at.stream, a, backwards);
    return hipGetLastError();
}

template <typename T, int DK, int DV>
hipError_t grad_t(const GdrArgs& a) {
    if (a.at.T_total == 0) return hipSuccess;
    constexpr int lds = GradLds<T, DK>::bytes;
    static_assert(lds <= 152 * 1024, "LDS");
    const void* kern = reinterpret_cast<const void*>(&gdr_grad_kernel<T, DK, DV>);
    const hipError_t e = ensure_lds_limit(kern, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gdr_grad_kernel<T, DK, DV>), dim3((unsigned)((int64_t)a.at.nblocks * a.at.H)), dim3(256), lds,
                       (hipStream_t)a.at.stream, a);
    hipError_t st = hipGetLastError();
    if (st != hipSuccess || !a.parts) return st;
    const int64_t runs = a.at.T_total * (a.at.H / a.k.share) * (DK / 2), groups = (runs + 1023) / 1024;   // four a thread
    hipLaunchKernelGGL((gdr_share_kernel<T>), dim3((unsigned)(groups < 65536 ? groups : 65536)), dim3(256), 0,
                       (hipStream_t)a.at.stream, a, DK);
    return hipGetLastError();
}

template <typename T, int DK>
hipError_t fwd_t(const GdrArgs& a) {
    hipError_t e = prep_t<T, DK, false>(a);
    if (e != hipSuccess) return e;
    if (a.seg_s) {
        if ((e = walk_t<T, DK, kGdrSeg>(a)) != hipSuccess) return e;
        if ((e = join<DK>(a, 0)) != hipSuccess) return e;
    }
    return walk_t<T, DK, kGdrOut>(a);
}

template <typename T, int DK>
hipError_t bwd_t(const GdrArgs& a) {
    hipError_t e = prep_t<T, DK, true>(a);
    if (e != hipSuccess) return e;
    if (a.seg_s) {
        if ((e = walk_t<T, DK, kGdrSeg>(a)) != hipSuccess) return e;
        if ((e = walk_t<T, DK, kGdrBackSeg>(a)) != hipSuccess) return e;
        if ((e = join<DK>(a, 0)) != hipSuccess) return e;
        if ((e = join<DK>(a, 1)) != hipSuccess) return e;
    }
    if (a.at.T_total > 0 && (e = walk_t<T, DK, kGdrStates>(a)) != hipSuccess) return e;
    if ((a.at.T_total > 0 || a.d_initial) && (e = walk_t<T, DK, kGdrBack>(a)) != hipSuccess) return e;
    return a.head_v == 64 ? grad_t<T, DK, 64>(a) : grad_t<T, DK, 128>(a);
}

}  // namespace

hipError_t launch_gdr_fwd(const GdrArgs& a) {
    const hipError_t e = launch_block_plan(a.at);
    if (e != hipSuccess) return e;
    if (a.dtype == 0) return a.head_k == 64 ? fwd_t<__bf16, 64>(a) : fwd_t<__bf16, 128>(a);
    return a.head_k == 64 ? fwd_t<float, 64>(a) : fwd_t<float, 128>(a);
}

hipError_t launch_gdr_bwd(const GdrArgs& a) {
    const hipError_t e = launch_block_plan(a.at);
    if (e != hipSuccess) return e;
    if (a.dtype == 0) return a.head_k == 64 ? bwd_t<__bf16, 64>(a) : bwd_t<__bf16, 128>(a);
    return a.head_k == 64 ? bwd_t<float, 64>(a) : bwd_t<float, 128>(a);
}

// One token a request against the resident fp32 state [N, H, dk, dv], updated in
// place.  A workgroup takes a state whole: in slices of 16 columns, to spread few
// states over the CUs, 16 states of 128 x 128 take 4.3 us against 4.0, and 256 take
// 13.4 against 6.3.  S^T k and S^T q are summed in one pass over the state in
// registers (S'^T q = exp(g) S^T q + beta (k.q) e), so it crosses memory once each
// way, which bounds the step: 128 requests of 96 heads (1.62 GB) 274 us, 5.9 TB/s.
namespace {

template <typename T, int DK, int DV>
__global__ __launch_bounds__(256) void gdr_decode_kernel(GdrDecodeArgs a) {
    constexpr int CG = DV / 4, RG = 256 / CG, RPT = DK / RG;
    static_assert(RG * CG == 256 && RPT * RG == DK, "decode tiling");
    __shared__ float s_k[DK], s_q[DK], s_e[DV], s_kq[RG];
    __shared__ float s_p[RG][DV + 4], s_o[RG][DV + 4];
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
    // each XCD takes states in runs of two (workgroups i, i + 8, ... share one), as
    // the KDA decode step does
    int nh = blockIdx.x;
    if (gridDim.x % 16 == 0) nh = nh / 16 * 16 + nh % 8 * 2 + nh / 8 % 2;
    const int n = nh / a.H, h = nh % a.H;
    float* st = a.state + (int64_t)nh * DK * DV + 4 * cg;
    f32x4_t S[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) S[r] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(st + (int64_t)(r * RG + rg) * DV));
    const T* q = (const T*)a.q.p + (int64_t)n * a.q.stride + (int64_t)(h / a.q.share) * DK;
    const T* k = (const T*)a.k.p + (int64_t)n * a.k.stride + (int64_t)(h / a.k.share) * DK;
    const T* v = (const T*)a.v.p + (int64_t)n * a.v.stride + (int64_t)h * DV;
    for (int c = tid; c < DK; c += 256) {
        s_k[c] = gload(k + c);
        s_q[c] = gload(q + c);
    }
    const float vt = tid < DV ? gload(v + tid) : 0.f;
    const float decay = a.g ? expf(a.g[nh]) : 1.f, beta = a.beta[nh];
    if (decay == 0.f) {   // anew, whatever the state holds
#pragma unroll
        for (int r = 0; r < RPT; ++r) S[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    __syncthreads();
    f32x4_t p = {0.f, 0.f, 0.f, 0.f}, o = p;
    float kq = 0.f;
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int row = r * RG + rg;
        S[r] *= decay;
        p += s_k[row] * S[r];
        o += s_q[row] * S[r];
        kq += s_k[row] * s_q[row];
    }
    if (cg == 0) s_kq[rg] = kq;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s_p[rg][4 * cg + i] = p[i];
        s_o[rg][4 * cg + i] = o[i];
    }
    __syncthreads();
    if (tid < DV) {
        float x = 0.f, y = 0.f, z = 0.f;
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            x += s_p[r][tid];
            y += s_o[r][tid];
            z += s_kq[r];
        }
        const float e = beta * (vt - x);
        s_e[tid] = e;
        gstore((T*)a.y + (int64_t)nh * DV + tid, a.scale * (y + z * e));
    }
    __syncthreads();
    const f32x4_t e = {s_e[4 * cg], s_e[4 * cg + 1], s_e[4 * cg + 2], s_e[4 * cg + 3]};
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int row = r * RG + rg;
        __builtin_nontemporal_store(S[r] + s_k[row] * e, reinterpret_cast<f32x4_t*>(st + (int64_t)row * DV));
    }
}

template <typename T, int DK, int DV>
hipError_t decode_t(const GdrDecodeArgs& a) {
    hipLaunchKernelGGL((gdr_decode_kernel<T, DK, DV>), dim3((unsigned)((int64_t)a.N * a.H)), dim3(256), 0,
                       (hipStream_t)a.stream, a);
    return hipGetLastError();
}

template <typename T, int DK>
hipError_t decode_c(const GdrDecodeArgs& a) {
    return a.dv == 64 ? decode_t<T, DK, 64>(a) : decode_t<T, DK, 128>(a);
}

}  // namespace

hipError_t launch_gdr_decode(const GdrDecodeArgs& a) {
    if (a.N == 0) return hipSuccess;
    if (a.dtype == 0) return a.dk == 64 ? decode_c<__bf16, 64>(a) : decode_c<__bf16, 128>(a);
    return a.dk == 64 ? decode_c<float, 64>(a) : decode_c<float, 128>(a);
}

}  // namespace kda
