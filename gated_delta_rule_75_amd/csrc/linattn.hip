// Linear attention with a decay for each head, by chunks of 64 tokens.
//
// One kernel computes, for operand rows q_i, k_i (DK channels), v_i (DV) and
// log-decays g_i, the causal form of
//   S_i = exp(g_i) S_{i-1} + u k_i v_i^T,       o_i = S_i^T q_i
// and, with G the sum of g inside the chunk, does so chunk by chunk:
//   P_ij = p exp(G_i - G_j) q_i.k_j  (j <= i, else 0)
//   O    = P V + s exp(G_i) Q S_in
//   S    = exp(G_63) S_in + u sum_j exp(G_63 - G_j) k_j v_j^T
// The prompt is (p, s, u) = (scale, scale, 1) on (q, k, v).  Its gradient is
// three more runs of the same form:
//   dq: rows (dy, v, k), state S^T, first token to last
//   dv: rows (k, q, dy), state R,   last to first
//   dk: rows (v, dy, q), state R^T, last to first
// where R is the gradient of the state.  Run backwards, the decay between a
// token and the one handled before it is the later token's, so the local
// decays are g shifted by one.
//
// Every exponent is a difference of sums that is at most 0: sums are kept in
// fp64 (one wave, a scan over lanes) and enter as a quotient against the start
// of a 16-token tile, or inside a tile as integer and fraction, so that a decay
// of any strength leaves the small ones behind it exact.
//
// A workgroup of four waves owns a (block of tokens, head); each wave owns
// DV / 4 columns of the fp32 state in its MFMA accumulators.  The accumulator
// layout (lane l: rows 4 (l / 16) + r of column l % 16) is a B operand as it
// stands when the contraction runs in the order 16a + 4g + r, 16(a + 1) + 4g + r,
// so the state never leaves the registers; the other operand is read from LDS
// in that order, and the token-contracted operands by transposing LDS reads.
// Rows are kept in LDS in 16-byte pieces, piece index xor row, against bank
// conflicts.
//
// Sequences are cut into blocks that run side by side: a first pass leaves each
// block's own state from zero (kState), a small kernel chains them, a second
// pass makes the outputs (kOut, kGrad) from the states that enter.
//
// What bounds it (d = 128, bf16): instructions.  With the update's operand in
// three parts, P and the entering state in two, 8192 tokens x 96 heads are 219
// GFLOP in the two passes, 170 us at the 1.29 PFLOP/s that a large bf16 product
// reaches here; their 815 MB need 131 us at a copy's 6.2 TB/s.  The call takes 326
// to 341 us: about 107 the state pass, 11 the chain, 215 the output pass.  (With
// the entering state in one part, 309 to 322.  Of that output pass its loads and
// stores alone took 183, its products alone 182.)  By counters its SIMDs are busy
// 49 % with vector and 30 % with matrix instructions (operands are split and
// decayed on the way), and 25 % of the waves' time is waiting, with two workgroups
// a CU (190 to 250 registers a thread).  Under load without pauses the clock
// falls, and a call takes 397 us at the median.
// Measured and not kept: eight waves a workgroup (276 against 258 us, the pass
// alone), half a head's columns a workgroup (457 the call), nontemporal output
// stores (80 more), placement of a head's blocks on one XCD (no change).
// The gradient, 4 x 2048 tokens x 32 heads (215 GFLOP; 497 MB, of which its
// passes read most more than once, 1.4 GB in all): 367 to 377 us.
#include <type_traits>

#include "launch.h"
#include "vec.h"

namespace kda {

namespace {

constexpr int C = 64;               // tokens of a chunk
constexpr float kFloor = -200.f;    // exp(-200) is 0 in fp32 with room for any factor: g is held above it

typedef short s16x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ s16x4_t lds_tr(const __bf16* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p);
}

// Eight consecutive contraction steps of a lane and the product of a 16 x 32
// by a 32 x 16 tile.  fp32: eight 16x16x4 products, step e of every lane group
// at a time.
template <typename T> struct Frag8;
template <> struct Frag8<__bf16> {
    bf16x8_t v;
    __device__ __forceinline__ float get(int i) const { return (float)v[i]; }
    __device__ __forceinline__ void set(int i, float x) { v[i] = (__bf16)x; }
};
template <> struct Frag8<float> {
    float v[8];
    __device__ __forceinline__ float get(int i) const { return v[i]; }
    __device__ __forceinline__ void set(int i, float x) { v[i] = x; }
};
__device__ __forceinline__ f32x4_t mma(const Frag8<__bf16>& a, const Frag8<__bf16>& b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma(const Frag8<float>& a, const Frag8<float>& b, f32x4_t c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
}

// A tile of rows of D elements in LDS, 16-byte pieces swizzled by the row.
template <typename T, int D>
struct Tile {
    static constexpr int EP = 16 / (int)sizeof(T);        // elements of a piece
    static constexpr int PIECES = D / EP;
    // Which piece xor: 16 rows of one piece, and the rows and 16 columns of a
    // transposing (bf16) or plain (fp32) column read, then each touch every bank
    // once.  (bf16 rows of 128 bytes share a line of banks in twos.)
    static __device__ __forceinline__ int swz(int row) {
        if constexpr (sizeof(T) == 4) return row & 15;
        if constexpr (PIECES == 16) return ((row << 1) | ((row >> 3) & 1)) & 15;
        return (row & 6) | ((row >> 3) & 1);   // rows in twos: bits 3 2 1 turned to 2 1 3
    }
    static __device__ __forceinline__ int off(int row, int col) {
        return row * D + (((col / EP) ^ swz(row)) * EP) + col % EP;
    }
    // rows row0 + l % 16, contraction 32 s + {0, 16} + 4 g + (0..3)
    static __device__ __forceinline__ Frag8<T> rows(const T* t, int row0, int s, int lane) {
        const int row = row0 + (lane & 15), k = 32 * s + 4 * (lane >> 4);
        Frag8<T> f;
        if constexpr (sizeof(T) == 2) {
            const bf16x4_t a = *reinterpret_cast<const bf16x4_t*>(t + off(row, k));
            const bf16x4_t b = *reinterpret_cast<const bf16x4_t*>(t + off(row, k + 16));
            f.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const f32x4_t a = *reinterpret_cast<const f32x4_t*>(t + off(row, k));
            const f32x4_t b = *reinterpret_cast<const f32x4_t*>(t + off(row, k + 16));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f.v[i] = a[i];
                f.v[4 + i] = b[i];
            }
        }
        return f;
    }
    // rows row0 + l % 16, contraction 32 s + 8 g + (0..7): for products of two
    // operands that are both read by rows
    static __device__ __forceinline__ Frag8<T> rows8(const T* t, int row0, int s, int lane) {
        const int row = row0 + (lane & 15), k = 32 * s + 8 * (lane >> 4);
        Frag8<T> f;
        if constexpr (sizeof(T) == 2) {
            f.v = *reinterpret_cast<const bf16x8_t*>(t + off(row, k));
        } else {
            const f32x4_t a = *reinterpret_cast<const f32x4_t*>(t + off(row, k));
            const f32x4_t b = *reinterpret_cast<const f32x4_t*>(t + off(row, k + 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f.v[i] = a[i];
                f.v[4 + i] = b[i];
            }
        }
        return f;
    }
    // columns col0 + l % 16, contraction over rows 32 s + {0, 16} + 4 g + (0..3)
    static __device__ __forceinline__ Frag8<T> cols(const T* t, int col0, int s, int lane) {
        Frag8<T> f;
        if constexpr (sizeof(T) == 2) {
            // a transposing read takes 4 rows x 16 columns from 16 lanes: lane
            // i of them points at row i / 4, columns 4 (i % 4)
            const int row = 32 * s + 4 * (lane >> 4) + ((lane & 15) >> 2), col = col0 + 4 * (lane & 3);
            const s16x4_t a = lds_tr(t + off(row, col));
            const s16x4_t b = lds_tr(t + off(row + 16, col));
            const bf16x4_t x = __builtin_bit_cast(bf16x4_t, a), y = __builtin_bit_cast(bf16x4_t, b);
            f.v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const int row = 32 * s + 4 * (lane >> 4), col = col0 + (lane & 15);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f.v[i] = t[off(row + i, col)];
                f.v[4 + i] = t[off(row + 16 + i, col)];
            }
        }
        return f;
    }
};

// The same value in every lane, as a scalar.
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ float unif(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}
__device__ __forceinline__ int64_t uni64(int64_t x) {
    return ((int64_t)uni((int)(x >> 32)) << 32) | (uint32_t)uni((int)x);
}

// The block of tokens of a workgroup: block j of sequence n.  A sequence has
// max(1, ceil(len / L)) blocks, numbered across the sequences in order.
struct Block {
    int n, j;            // sequence, block in it (n < 0: no such block)
    int nb;              // blocks of the sequence
    int64_t begin;       // the sequence's first token
    int64_t start;       // the block's first token
    int cnt;             // tokens of the block
};

__device__ __forceinline__ int64_t seq_at(const LinArgs& a, int n) {
    if (!a.cu_seqlens) return n == 0 ? 0 : a.T_total;
    int64_t x = a.cu_seqlens[n];
    return x < 0 ? 0 : x > a.T_total ? a.T_total : x;
}

// At most the bound on all blocks: offsets out of order stay inside the arrays.
__device__ __forceinline__ int blocks_of(const LinArgs& a, int64_t len) {
    const int64_t nb = len <= a.L ? 1 : (len + a.L - 1) / a.L;
    return nb < a.nblocks ? (int)nb : a.nblocks;
}

__device__ __forceinline__ int wave_incl_sum(int x, int lane) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    return x;
}

__device__ __forceinline__ int64_t shfl_i64(int64_t x, int src) {
    return ((int64_t)__shfl((int)(x >> 32), src) << 32) | (uint32_t)__shfl((int)x, src);
}

// Every wave finds the block itself.  Uncut sequences are their blocks.  Else by
// the sequences' first blocks, a 64th of what is left at a step; for up to
// kPlanSeqs sequences, which have no such table, by counting, 64 at a time.
__device__ __forceinline__ Block find_block(const LinArgs& a, int b) {
    const int lane = threadIdx.x & 63;
    Block r;
    r.n = -1;
    r.j = 0;
    r.nb = 1;
    int64_t s = 0, e = 0;
    if (a.L >= a.T_total) {
        if (b < a.num_seqs) r.n = b;
    } else if (a.first) {
        if (b < a.first[a.num_seqs]) {
            int lo = 0, span = a.num_seqs;   // it is one of [lo, lo + span)
            while (span > 1) {
                const int step = (span + kWave - 1) / kWave, at = lane * step;
                const int k = __popcll(__ballot(at < span && a.first[lo + (at < span ? at : 0)] <= b)) - 1;
                lo += k * step;
                span = span - k * step < step ? span - k * step : step;
            }
            r.n = lo;
            r.j = b - a.first[lo];
            r.nb = a.first[lo + 1] - a.first[lo];
        }
    } else {
        int before = 0;
        for (int n0 = 0; n0 < a.num_seqs; n0 += kWave) {
            const int n = n0 + lane;
            int nb = 0;
            if (n < a.num_seqs) {
                s = seq_at(a, n);
                e = seq_at(a, n + 1);
                nb = blocks_of(a, e - s);
            }
            const int incl = wave_incl_sum(nb, lane);
            const int total = __shfl(incl, kWave - 1);
            if (b < before + total) {
                const uint64_t m = __ballot(before + incl > b);
                const int src = __ffsll((unsigned long long)m) - 1;
                r.n = n0 + src;
                r.nb = __shfl(nb, src);
                r.j = b - before - (__shfl(incl, src) - r.nb);
                s = shfl_i64(s, src);
                e = shfl_i64(e, src);
                break;
            }
            before += total;
        }
    }
    r.n = uni(r.n);
    if (r.n < 0) return r;
    r.j = uni(r.j);
    r.nb = uni(r.nb);
    if (a.L >= a.T_total || a.first) {
        s = seq_at(a, r.n);
        e = seq_at(a, r.n + 1);
    }
    r.begin = uni64(s);
    r.start = r.begin + (int64_t)r.j * a.L;
    const int64_t left = uni64(e) - r.start;
    r.cnt = uni((int)(left < 0 ? 0 : left < a.L ? left : a.L));
    return r;
}

// Index of sequence n's first block.
__device__ __forceinline__ int first_block(const LinArgs& a, int n) {
    if (a.L >= a.T_total) return n;
    if (a.first) return a.first[n];
    const int lane = threadIdx.x & 63;
    int sum = 0;
    for (int m = lane; m < n; m += kWave) sum += blocks_of(a, seq_at(a, m + 1) - seq_at(a, m));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    return sum;
}

// The sequences' first blocks, and behind them their number, none above the
// bound: one workgroup, 4096 sequences a step.
__global__ __launch_bounds__(1024) void linattn_plan_kernel(LinArgs a) {
    __shared__ int part[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int before = 0;   // of the steps done
    for (int64_t n0 = 0; n0 < a.num_seqs; n0 += 4096) {
        int nb[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = n0 + 4 * tid + i;
            nb[i] = n < a.num_seqs ? blocks_of(a, seq_at(a, (int)n + 1) - seq_at(a, (int)n)) : 0;
            sum += nb[i];
        }
        // more than the bound only where the offsets are out of order: held there
        // (it is below 2^22, so no sum of these overflows)
        sum = sum < a.nblocks ? sum : a.nblocks;
        int incl = sum;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int y = __shfl_up(incl, d);
            if (lane >= d) incl += y;
            incl = incl < a.nblocks ? incl : a.nblocks;
        }
        if (lane == kWave - 1) part[wave] = incl;
        __syncthreads();
        int at = before + (incl - sum);
        for (int w = 0; w < wave; ++w) at += part[w];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = n0 + 4 * tid + i;
            if (n < a.num_seqs) a.first[n] = at < a.nblocks ? at : a.nblocks;
            at += nb[i];
        }
        for (int w = 0; w < 16; ++w) before += part[w];
        before = before < a.nblocks ? before : a.nblocks;
        __syncthreads();
    }
    if (tid == 0) a.first[a.num_seqs] = before;
}

// Decay tables of a chunk, one token a lane.
struct __attribute__((aligned(16))) Tables {
    float frac[C];      // log2 sum G = whole + frac
    int whole[C];
    float tile[C];      // exp2(G_i - G at the start of i's 16-token tile)
    float upto[96];     // exp2(G at the start of tile t - G_j), j before it: at 8 t (t - 1) + j
    float in[C];        // exp2(G_i)
    float out[C];       // exp2(G_63 - G_j)
    float total;
};
// beside the two tables: log-decays of two chunks, and partial sums of the
// waves for the decay's gradient
struct __attribute__((aligned(16))) Scratch {
    float g[2][C];
    float row[4][C];
};

__device__ __forceinline__ double shfl_d(double x, int src) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __shfl((int)(uint32_t)u, src), hi = __shfl((int)(uint32_t)(u >> 32), src);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// x moved by a DPP pattern, zero where it has no source.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_d(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, ROWS, 0xF, ROWS == 0xF);
    const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, ROWS, 0xF, ROWS == 0xF);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double lane_d(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const unsigned lo = __builtin_amdgcn_readlane((int)(unsigned)u, lane);
    const unsigned hi = __builtin_amdgcn_readlane((int)(unsigned)(u >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Inclusive sum over the wave: shifts within rows of 16 lanes, then the last
// lane of a row into the rows behind it.
__device__ __forceinline__ double decay_scan(float g) {
    double x = (double)(g < kFloor ? kFloor : g) * 1.4426950408889634074;
    x += dpp_d<0x111, 0xF>(x);
    x += dpp_d<0x112, 0xF>(x);
    x += dpp_d<0x114, 0xF>(x);
    x += dpp_d<0x118, 0xF>(x);
    x += dpp_d<0x142, 0xA>(x);
    x += dpp_d<0x143, 0xC>(x);
    return x;
}

// valid: the lane has a token.  The others, behind the last token or (backwards)
// before the first one, get weight 0 in every product that is kept.
__device__ __forceinline__ void write_tables(Tables* t, double G, int lane, bool valid, bool rev) {
    const double w = floor(G);
    t->frac[lane] = (float)(G - w);
    t->whole[lane] = valid ? (int)w : rev ? 1 << 20 : -(1 << 20);
    const double r1 = lane_d(G, 15), r2 = lane_d(G, 31), r3 = lane_d(G, 47), end = lane_d(G, 63);
    const double mine = lane < 16 ? 0.0 : lane < 32 ? r1 : lane < 48 ? r2 : r3;
    t->tile[lane] = valid ? exp2_fast((float)(G - mine)) : 0.f;
    if (lane < 16) t->upto[lane] = valid ? exp2_fast((float)(r1 - G)) : 0.f;
    if (lane < 32) t->upto[16 + lane] = valid ? exp2_fast((float)(r2 - G)) : 0.f;
    if (lane < 48) t->upto[48 + lane] = valid ? exp2_fast((float)(r3 - G)) : 0.f;
    t->in[lane] = exp2_fast((float)G);
    t->out[lane] = valid ? exp2_fast((float)(end - G)) : 0.f;
    if (lane == 0) t->total = exp2_fast((float)end);
}

// Zeros into the rows of no sequence of out [T, H, D], of head h: the block b of
// the launch's takes its share of them.
template <typename T, int D>
__device__ __forceinline__ void clear_rest(const LinArgs& a, T* out, int b, int h) {
    constexpr int EP = 16 / (int)sizeof(T) < D ? 16 / (int)sizeof(T) : D, P = D / EP, RPW = 256 / P;
    const int64_t t0 = seq_at(a, 0), end = seq_at(a, a.num_seqs), t1 = end < t0 ? t0 : end;
    for (int64_t r = (int64_t)b * RPW + threadIdx.x / P; r < t0 + (a.T_total - t1); r += (int64_t)a.nblocks * RPW) {
        const int64_t tok = r < t0 ? r : t1 + (r - t0);
        const float zero[EP] = {};
        store_vec<T, EP>(out + (tok * a.H + h) * D + threadIdx.x % P * EP, zero);
    }
}

enum : int { kOut = 0, kState = 1, kGrad = 2 };

// Tokens of a block in the order they are handled: chunk boundaries lie at the
// same tokens in both directions, so backwards the first rows may be empty.
struct Rows {
    int cnt, rows;   // tokens; rows, a multiple of 64
    bool rev;
    __device__ __forceinline__ bool has(int m) const { return rev ? m >= rows - cnt : m < cnt; }
    // token of row m, counted from the block's first
    __device__ __forceinline__ int token(int m) const { return rev ? rows - 1 - m : m; }
    // lowest token of the chunk of rows m0 .. m0 + 63, and its tokens
    __device__ __forceinline__ int low(int m0) const { return rev ? rows - C - m0 : m0; }
    __device__ __forceinline__ int tokens(int m0) const { return cnt - low(m0) < C ? cnt - low(m0) : C; }
};

typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));

// An operand's rows of one head from the block's first token on: address and
// bytes from token to token, pinned to scalar registers (left to itself the
// compiler reads them from the kernel's arguments again in every chunk, and each
// such read waits for all LDS reads in flight).
struct Src {
    int64_t at;
    unsigned step;
    template <typename T>
    __device__ __forceinline__ void set(const T* p, int64_t offset, int64_t stride) {
        at = uni64(reinterpret_cast<int64_t>(p + offset));
        step = uni((unsigned)stride * (unsigned)sizeof(T));
        asm volatile("" : "+s"(at), "+s"(step));
    }
    __device__ __forceinline__ int64_t token(int t) const { return uni64(at + (int64_t)(uint64_t)((uint64_t)(unsigned)t * step)); }
};
__device__ __forceinline__ float pin(float x) {
    int y = uni(__builtin_bit_cast(int, x));
    asm volatile("" : "+s"(y));
    return __builtin_bit_cast(float, y);
}

// 16 (or 4) bytes a lane from global memory straight to LDS address lds + 16
// (4) lane.  As assembly: the compiler makes every later LDS read of the wave
// wait for a copy that it knows of, and here the copy is for the next chunk;
// the waits are the kernel's own.  (No register is written; the first s_nop
// covers scalars that a vector instruction has just produced.)
__device__ __forceinline__ unsigned lds_addr(const void* p) {
    return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}
// (m0 is no register that a statement can name as changed: it is put back.)
__device__ __forceinline__ void copy16(unsigned lds, const void* base, unsigned off) {
    unsigned old;
    asm volatile("s_mov_b32 %0, m0\n\ts_nop 4\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
                 : "=&s"(old) : "s"(uni(lds)), "v"(off), "s"(uni64(reinterpret_cast<int64_t>(base))) : "memory");
}
__device__ __forceinline__ void copy4(unsigned lds, const void* addr) {
    unsigned old;
    asm volatile("s_mov_b32 %0, m0\n\ts_nop 4\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %2, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(old) : "s"(uni(lds)), "v"(addr) : "memory");
}

// The copy of a chunk's rows into a tile by the workgroup's four waves.  A
// wave's copy is 1 KiB of LDS in order, so the swizzle is on the source side.
// Rows without a token take the last token's: the tables give them no weight.
template <typename T, int D> constexpr int kCopies = C * D * (int)sizeof(T) / 4096;   // of a wave
template <typename T, int D>
__device__ __forceinline__ void copy_part(T* t, const Src& x, const Rows& rows, int m0, int wave, int lane, int i) {
    constexpr int PIECES = Tile<T, D>::PIECES, RPW = 64 / PIECES, N = kCopies<T, D>;
    const int top = rows.tokens(m0) - 1;
    const int row0 = wave * RPW + lane / PIECES, row = 4 * RPW * i + row0;
    const unsigned lds = uni(lds_addr(t) + wave * 1024) + i * 4096;
    const unsigned piece = (unsigned)((lane % PIECES) ^ Tile<T, D>::swz(row)) * 16u;
    const int64_t base = x.token(rows.low(m0));
    if (top == C - 1) {
        const int64_t at = base + (int64_t)((rows.rev ? N - 1 - i : i) * 4 * RPW) * x.step;
        copy16(lds, reinterpret_cast<const void*>(at), (unsigned)(rows.rev ? 4 * RPW - 1 - row0 : row0) * x.step + piece);
    } else {
        const int tok = rows.rev ? C - 1 - row : row;
        copy16(lds, reinterpret_cast<const void*>(base), (unsigned)(tok < top ? tok : top) * x.step + piece);
    }
}
template <typename T, int D>
__device__ __forceinline__ void copy_tile(T* t, const Src& x, const Rows& rows, int m0, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < kCopies<T, D>; ++i) copy_part<T, D>(t, x, rows, m0, wave, lane, i);
}

// A wave's columns of the v rows (SW of them): to registers a chunk ahead, then
// 32 tokens at a time through LDS of the wave's own, where the transposing reads
// take them.  No other wave waits for them, and P's tiles of the wave take their
// place once they are read.
template <typename T, int SW>
struct Slice {
    static constexpr int EP = 16 / (int)sizeof(T), PIECES = SW / EP, RPI = 64 / PIECES, N = C / RPI, HALF = N / 2;
    static constexpr int SIZE = 32 * SW > 3 * 256 ? 32 * SW : 3 * 256;   // elements: half the rows, or three tiles of P
    static_assert(N % 2 == 0, "two halves");
    u32x4_t r[N];
    static __device__ __forceinline__ int off(int row, int col) {
        // conflict-free for SW = 32 in bf16: rows r and r + 4 in different pieces
        const int x = PIECES >= 4 ? ((row >> 2) & 1) * (PIECES / 2) : 0;
        return row * SW + (((col / EP) ^ x) * EP) + col % EP;
    }
    __device__ __forceinline__ void load(const Src& x, int col0, const Rows& rows, int m0, int lane) {
        const unsigned step = x.step;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
            reinterpret_cast<void*>(x.token(rows.low(m0)) + col0 * (int)sizeof(T)), 0,
            uni((unsigned)(rows.tokens(m0) - 1) * step + SW * (unsigned)sizeof(T)), 0x00027000);
        const int row = lane / PIECES;
        const unsigned at = (unsigned)(rows.rev ? RPI - 1 - row : row) * step + (lane % PIECES) * 16u;
#pragma unroll
        for (int i = 0; i < N; ++i)
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, (unsigned)((rows.rev ? N - 1 - i : i) * RPI) * step, 0);
    }
    // tokens 32 s .. of the wave's columns as operands
    template <int NT>
    __device__ __forceinline__ void cols(T* t, int s, int lane, Frag8<T> (&f)[NT]) const {
#pragma unroll
        for (int i = 0; i < HALF; ++i)
            *reinterpret_cast<u32x4_t*>(t + off(i * RPI + lane / PIECES, (lane % PIECES) * EP)) = r[s * HALF + i];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (sizeof(T) == 2) {
                const int row = 4 * (lane >> 4) + ((lane & 15) >> 2), col = 16 * n + 4 * (lane & 3);
                const bf16x4_t x = __builtin_bit_cast(bf16x4_t, lds_tr(t + off(row, col)));
                const bf16x4_t y = __builtin_bit_cast(bf16x4_t, lds_tr(t + off(row + 16, col)));
                f[n].v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
            } else {
                const int row = 4 * (lane >> 4), col = 16 * n + (lane & 15);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[n].v[i] = t[off(row + i, col)];
                    f[n].v[4 + i] = t[off(row + 16 + i, col)];
                }
            }
        }
    }
};

// P as 16 x 16 tiles of their own (rows of 16 elements, 4 at a time), of bf16 in
// two parts: value and remainder, since with few tokens its rounding would not
// average out of a row.  Only tiles on and below the diagonal; the two above it
// that are read, (0, 1) and (2, 3), are one tile of zeros.
template <typename T> constexpr int kParts = sizeof(T) == 2 ? 2 : 1;
constexpr int tri(int ti, int tj) { return ti * (ti + 1) / 2 + tj; }

// Where a tile lies, in elements.  Gradient runs: an array of their own.
template <typename T> constexpr int p_tiles() { return 10 * kParts<T> + 1; }
template <typename T>
__device__ __forceinline__ constexpr int p_at_own(int ti, int tj, int part) {
    return 256 * (tj > ti ? 10 * kParts<T> : 10 * part + tri(ti, tj));
}
// Else the tiles of a wave lie in its slice of v (SIZE elements), where each
// wave may write once it has read its own v, and what does not fit behind the
// slices.  Waves hold (0,0) (1,0) (1,1); (2,*); (3,0) (3,1) and the zeros; (3,2) (3,3).
template <int SIZE>
__device__ __forceinline__ constexpr int p_at(int ti, int tj, int part) {
    const int w = ti < 2 ? 0 : ti == 2 ? 1 : tj < 2 ? 2 : 3;
    if (tj > ti) return 2 * SIZE + 512;
    if (part == 0) return w * SIZE + 256 * (ti < 2 ? tri(ti, tj) : ti == 2 ? tj : tj & 1);
    const int t = tri(ti, tj);   // remainders of (0,0) .. (3,3)
    if (SIZE >= 1024) {
        if (t == 0) return 0 * SIZE + 768;
        if (t == 3) return 1 * SIZE + 768;
        if (t == 6) return 2 * SIZE + 768;
        if (t >= 8) return 3 * SIZE + 512 + 256 * (t - 8);
        return 4 * SIZE + 256 * (t == 1 ? 0 : t == 2 ? 1 : t == 4 ? 2 : t == 5 ? 3 : 4);
    }
    if (t == 8) return 3 * SIZE + 512;
    return 4 * SIZE + 256 * (t < 8 ? t : 8);
}
template <typename T, int SIZE> constexpr int p_extra() { return sizeof(T) == 4 ? 0 : SIZE >= 1024 ? 5 * 256 : 9 * 256; }
template <typename T>
__device__ __forceinline__ int p_off(int i, int j4) {   // row, run of 4 columns
    return i * 16 + (sizeof(T) == 2 ? (j4 ^ ((i >> 2) & 2)) : (j4 ^ ((i >> 2) & 3))) * 4;
}

// LDS.  Prompt and state pass: k and q rows twice (the copy of the next chunk's
// runs through a whole chunk), the waves' slices of v, which P takes over, and
// the tables twice: two workgroups a CU in bf16.  Gradient runs: rows k, v, q, x
// once, P, the tables twice.
template <typename T, int DK, int DV, int MODE>
constexpr int lds_bytes() {
    const int sz = (int)sizeof(T), tables = 2 * (int)sizeof(Tables) + (MODE == kGrad ? (int)sizeof(Scratch) : (int)sizeof(float[2][C]));
    if (MODE == kGrad) return (C * (2 * DK + 2 * DV) + 256 * p_tiles<T>()) * sz + tables;
    constexpr int SL = Slice<T, DV / 4>::SIZE;
    return (2 * C * DK * (MODE == kState ? 1 : 2) + 4 * SL + (MODE == kState ? 0 : p_extra<T, SL>())) * sz + tables;
}

// Eight values as a sum of NS operands of type T.  One: rounded to nearest.
// Two bf16: value and remainder, each rounded to nearest.  Three bf16: the leading 8 bits, the next 8 and the rest, by cutting; exact.
__device__ __forceinline__ unsigned cvt2(float a, float b) {
    return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}
template <int NS>
__device__ __forceinline__ void split(const float (&x)[8], Frag8<__bf16> (&f)[NS]) {
    static_assert(NS >= 1 && NS <= 3, "parts");
    u32x4_t p[NS];
    if constexpr (NS < 3) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[0][i] = cvt2(x[2 * i], x[2 * i + 1]);
        if constexpr (NS == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                p[1][i] = cvt2(x[2 * i] - __builtin_bit_cast(float, p[0][i] << 16),
                               x[2 * i + 1] - __builtin_bit_cast(float, p[0][i] & 0xffff0000u));
        }
    } else {
        unsigned y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __builtin_bit_cast(unsigned, x[i]);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[s][i] = __builtin_amdgcn_perm(y[2 * i + 1], y[2 * i], 0x07060302);
            if (s + 1 < NS) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i] = __builtin_bit_cast(unsigned, __builtin_bit_cast(float, y[i]) -
                                                            __builtin_bit_cast(float, y[i] & 0xffff0000u));
            }
        }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) f[s].v = __builtin_bit_cast(bf16x8_t, p[s]);
}
__device__ __forceinline__ void split(const float (&x)[8], Frag8<float> (&f)[1]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[0].v[i] = x[i];
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const f32x4_t& x) {
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2*>(p) = make_uint2(cvt2(x[0], x[1]), cvt2(x[2], x[3]));
    else
        *reinterpret_cast<f32x4_t*>(p) = x;
}
__device__ __forceinline__ f32x4_t load4(const __bf16* p) {
    const bf16x4_t v = *reinterpret_cast<const bf16x4_t*>(p);
    return f32x4_t{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
__device__ __forceinline__ f32x4_t load4(const float* p) { return *reinterpret_cast<const f32x4_t*>(p); }

// MODE kState: the block's own state from zero (a.states) and its decay
// (a.decays); kOut: outputs, from the entering state; kGrad: outputs, and for
// the decay's gradient the products of extra rows x_i with the part of o_i that
// comes from the entering state, plus (a.pairs) those of pairs inside a chunk.
//
// Roundings of bf16 inputs: as operands P and the state that enters the chunk are
// sums of two bf16 values, 16 bits, whatever the cut into blocks: the output's own
// rounding to 8 bits is the one that shows.  (The state as one bf16 value made the
// error of y 2.1e-3 where that rounding alone is 1.66e-3.)  As three in kGrad,
// whose sums are fp32 outputs; the update's exp(G_63 - G_j) v_j enters as a sum of
// three too, so that the state keeps its 24 bits.
template <typename T, int DK, int DV, int MODE>
__device__ __forceinline__ void linattn_body(const LinArgs& a) {
    constexpr bool kBf = sizeof(T) == 2;
    constexpr int NT = DV / 64;             // 16-column tiles of a wave
    constexpr int KT = DK / 16;             // 16-row tiles of the state
    constexpr int NU = kBf ? 3 : 1;         // parts of an update operand
    constexpr int NS = !kBf ? 1 : MODE == kGrad ? 3 : 2;   // parts of the state as an operand
    extern __shared__ __attribute__((aligned(16))) char smem[];
    constexpr bool kPair = MODE != kGrad;               // two buffers of k and q
    T* const skb = reinterpret_cast<T*>(smem);          // [2 or 1][C][DK]
    T* const sqb = skb + (kPair ? 2 : 1) * C * DK;      // [2 or 1][C][DK]
    T* const sv = sqb + (MODE == kState ? 0 : kPair ? 2 : 1) * C * DK;   // slices, or [C][DV]
    constexpr int SL = Slice<T, DV / 4>::SIZE;
    constexpr int NP = kParts<T>;
    T* const sx = sv + (kPair ? 4 * SL : C * DV);       // [C][DV]
    T* const sp = sx + (kPair ? 0 : C * DV);            // P's tiles, or those behind the slices
    Tables* const tbb = reinterpret_cast<Tables*>(
        sp + (!kPair ? 256 * p_tiles<T>() : MODE == kState ? 0 : p_extra<T, SL>()));
    Scratch* const scr = reinterpret_cast<Scratch*>(tbb + 2);

    const int tid = threadIdx.x, lane0 = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = lane0, lr = lane & 15, lg = lane >> 4;
    // divisions run on the vector unit; their results are the same in every lane
    const int b = uni(blockIdx.x / a.H), h = blockIdx.x - b * a.H;
    const int hq = MODE == kState ? 0 : uni(h / a.q.share), hk = uni(h / a.k.share), hv = uni(h / a.v.share);
    const int hx = MODE == kGrad ? uni(h / a.x.share) : 0;
    if (MODE != kState && a.clear && !a.out_f32) clear_rest<T, DV>(a, (T*)a.out, b, h);
    const Block bl = find_block(a, b);
    if (bl.n < 0) return;
    const bool rev = a.reverse;
    const bool first = rev ? bl.j == bl.nb - 1 : bl.j == 0;         // no block is handled before it
    const bool last = rev ? bl.j == 0 : bl.j == bl.nb - 1;
    if (MODE == kState && last && !a.last_state) return;
    const int cnt = bl.cnt;
    const Rows rows{cnt, (cnt + C - 1) / C * C, rev};
    Src xk, xv, xq, xx, xo, xg;
    xk.set((const T*)a.k.p, bl.start * a.k.stride + (int64_t)hk * DK, a.k.stride);
    xv.set((const T*)a.v.p, bl.start * a.v.stride + (int64_t)hv * DV, a.v.stride);
    if constexpr (MODE != kState) xq.set((const T*)a.q.p, bl.start * a.q.stride + (int64_t)hq * DK, a.q.stride);
    if constexpr (MODE == kGrad) xx.set((const T*)a.x.p, bl.start * a.x.stride + (int64_t)hx * DV, a.x.stride);
    const bool wide = MODE == kGrad && a.out_f32;
    if (wide) xo.set((const float*)a.out, (bl.start * a.H + h) * DV, (int64_t)a.H * DV);
    else xo.set((const T*)a.out, (bl.start * a.H + h) * DV, (int64_t)a.H * DV);
    xg.set(a.g, a.g_per_token ? bl.start * a.H + h : h, a.g_per_token ? a.H : 0);
    // tokens from the block's first to the end of everything, for the decays
    const int64_t left = a.T_total - 1 - bl.start;
    const int glast = uni(left < INT32_MAX ? (int)left : INT32_MAX);
    const float p_scale = pin(a.p_scale), s_scale = pin(a.s_scale), u_scale = pin(a.u_scale);
    const bool pairs = MODE == kGrad && uni(a.pairs) != 0;
    const int wcol = wave * (DV / 4);

    f32x4_t S[KT][NT];
    {
        const float* s0 = nullptr;
        if (MODE != kState) {
            if (a.states) s0 = a.states + ((int64_t)b * a.H + h) * DK * DV;
            else if (a.initial) s0 = a.initial + ((int64_t)bl.n * a.H + h) * DK * DV;
        }
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                f32x4_t x = {0.f, 0.f, 0.f, 0.f};
                if (s0) {
                    const int row = 16 * i + 4 * lg, col = wcol + 16 * n + lr;
                    if (a.transposed) {
                        x = *reinterpret_cast<const f32x4_t*>(s0 + (int64_t)col * DK + row);
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] = s0[(int64_t)(row + r) * DV + col];
                    }
                }
                S[i][n] = x;
            }
    }

    // The state is c S: a chunk's decay multiplies c, and S (with the update
    // divided by c) only once c gets small, 64 multiplications a chunk less.
    float c = 1.f;
    double sum_total = 0.0;
    constexpr int kTab = 3;    // the wave that makes the tables: one with two tiles of P
    // The log-decay of local row m goes to LDS, two chunks ahead.
    auto fetch_g = [&](int m0) {
        int tok = rows.token(m0 + lane) + (rev ? 1 : 0);   // backwards: the token after it
        tok = tok < 0 ? 0 : tok > glast ? glast : tok;
        copy4(uni(lds_addr(scr->g[(m0 / C) & 1])), reinterpret_cast<const void*>(xg.at + (int64_t)((uint64_t)(unsigned)tok * xg.step)));
    };
    Slice<T, DV / 4> rv;
    // A wave stalls on a copy while the memory pipe is full (about 100 cycles
    // each when they come at once), so the copies of the next chunk are spread
    // over the work on this one.
    constexpr int NC = kCopies<T, DK>;
    auto part_k = [&](int m0, int i) {
        copy_part<T, DK>(skb + ((m0 / C) & 1) * C * DK, xk, rows, m0, wave, lane, i);
    };
    auto part_q = [&](int m0, int i) {
        copy_part<T, DK>(sqb + ((m0 / C) & 1) * C * DK, xq, rows, m0, wave, lane, i);
    };
    auto fetch_k = [&](int m0) {
        copy_tile<T, DK>(skb + (kPair ? ((m0 / C) & 1) * C * DK : 0), xk, rows, m0, wave, lane);
    };
    auto fetch_q = [&](int m0) {
        if constexpr (MODE == kOut) copy_tile<T, DK>(sqb + ((m0 / C) & 1) * C * DK, xq, rows, m0, wave, lane);
    };
    auto fetch_v = [&](int m0) {
        if constexpr (kPair) {
            rv.load(xv, wcol, rows, m0, lane);
        } else {
            copy_tile<T, DV>(sv, xv, rows, m0, wave, lane);
            copy_tile<T, DK>(sqb, xq, rows, m0, wave, lane);
            copy_tile<T, DV>(sx, xx, rows, m0, wave, lane);
        }
    };
    auto tables = [&](int m0) {
        const int m = m0 + lane;
        const bool valid = rows.has(m);
        // backwards nothing decays before the sequence's last token
        const float g = valid && !(rev && first && rows.token(m) == cnt - 1) ? scr->g[(m0 / C) & 1][lane] : 0.f;
        const double G = decay_scan(g);
        write_tables(tbb + ((m0 / C) & 1), G, lane, valid, rev);
        if (MODE == kState) sum_total += lane_d(G, 63);
    };
    // Outputs in whole rows: through the chunk's own q rows once they are read,
    // stored by all waves in the next chunk (a wave's own 8-byte pieces, 32 bytes
    // of a row side by side, made the pass 25 % slower).  Where the q rows are
    // too short for it, pieces; those stores are then the youngest of a wave's
    // memory operations where the copies are waited for.
    constexpr bool kRows = MODE == kOut && DK >= DV;
    constexpr int NST = MODE == kOut && !kRows ? 4 * NT : 0;
    auto store_rows = [&](int m0) {
        typedef Tile<T, DV> O;
        constexpr int RPW = 64 / O::PIECES, N = C / (4 * RPW);
        const T* o = sqb + ((m0 / C) & 1) * C * DK;
        const unsigned step = xo.step;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
            reinterpret_cast<void*>(xo.token(rows.low(m0))), 0,
            uni((unsigned)(rows.tokens(m0) - 1) * step + DV * (unsigned)sizeof(T)), 0x00027000);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = (i * 4 + wave) * RPW + lane / O::PIECES, piece = lane % O::PIECES;
            __builtin_amdgcn_raw_buffer_store_b128(
                *reinterpret_cast<const u32x4_t*>(o + O::off(row, piece * O::EP)), rsrc,
                (unsigned)(rev ? C - 1 - row : row) * step + piece * 16u, 0, 0);
        }
    };
    if (cnt > 0) {
        if (wave == kTab) {
            fetch_g(0);
            if (C < rows.rows) fetch_g(C);
        }
        fetch_k(0);
        fetch_q(0);
        fetch_v(0);
    }
    // on every path: else the compiler still has the state's first loads to wait
    // for inside the loop, and that wait takes the next chunk's copies with it
    wait_vmcnt<0>();
    if (cnt > 0 && wave == kTab) tables(0);
    for (int m0 = 0; m0 < rows.rows; m0 += C) {
        // LDS addresses are formed anew in each chunk (a few dozen operations):
        // kept across the loop they cost registers that spill
        lane = lane0;
        asm volatile("" : "+v"(lane));
        lr = lane & 15;
        lg = lane >> 4;
        // A: this chunk's copies and tables are there; the chunk before is read
        if (m0 > 0) wait_vmcnt<NST>();
        barrier_keep_loads();
        const T* const sk = skb + (kPair ? ((m0 / C) & 1) * C * DK : 0);
        const T* const sq = sqb + (kPair ? ((m0 / C) & 1) * C * DK : 0);
        const Tables* const tb = tbb + ((m0 / C) & 1);
        const bool more = m0 + C < rows.rows;
        // v's columns of this wave, before v is overwritten
        Frag8<T> fv[2][NT];
        T* const slice = sv + wave * SL;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if constexpr (kPair) {
                rv.cols(slice, s, lane, fv[s]);
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n) fv[s][n] = Tile<T, DV>::cols(sv, wcol + 16 * n, s, lane);
            }
        }
        if (wave == kTab && m0 + 2 * C < rows.rows) fetch_g(m0 + 2 * C);
        if (kPair && more) {
            if (MODE == kState) fetch_k(m0 + C);
            fetch_v(m0 + C);
        }
        if (MODE == kOut && !kRows && more) fetch_q(m0 + C);

        const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
        // outputs, transposed tiles: a lane holds 4 consecutive columns of row
        // 16 t + l % 16
        f32x4_t acc[4][NT];
        Frag8<T> fk[KT];      // k's columns, tokens 0 to 31, then 32 to 63
        if constexpr (MODE != kState) {
            // P, transposed tiles (rows j, columns i): a lane holds 4 consecutive
            // j of one i.  Waves take 3, 3, 2 and 2 of the 10 tiles on or below
            // the diagonal.
            auto put_p = [&](int ti, int tj, const f32x4_t& p) {
                f32x4_t rest = p;
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    T* const at = (kPair ? sv + p_at<SL>(ti, tj, k) : sp + p_at_own<T>(ti, tj, k)) + p_off<T>(lr, lg);
                    store4<T>(at, rest);
                    if constexpr (kBf) {
                        if (k + 1 < NP) {
#pragma unroll
                            for (int r = 0; r < 4; ++r) rest[r] -= (float)(__bf16)rest[r];
                        }
                    }
                }
            };
            auto ptile = [&](int ti, int tj, const f32x4_t& x) {
                const int i = 16 * ti + lr, j = 16 * tj + 4 * lg;
                f32x4_t w;
                if (ti == tj) {
                    const float fi = tb->frac[i];
                    const int wi = tb->whole[i];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float e = exp2_fast(fi - tb->frac[j + r]);
                        w[r] = __builtin_amdgcn_ldexpf(e, wi - tb->whole[j + r]);
                    }
                } else {
                    w = *reinterpret_cast<const f32x4_t*>(&tb->upto[8 * ti * (ti - 1) + j]) * tb->tile[i];
                }
                f32x4_t p;
#pragma unroll
                for (int r = 0; r < 4; ++r) p[r] = ti != tj || j + r <= i ? x[r] * w[r] * p_scale : 0.f;
                put_p(ti, tj, p);
                if constexpr (MODE == kGrad) {
                    if (pairs) {
                        // weight of each pair i > j in the decay's gradient
                        f32x4_t d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int s = 0; s < DV / 32; ++s)
                            d = mma(Tile<T, DV>::rows8(sv, 16 * tj, s, lane), Tile<T, DV>::rows8(sx, 16 * ti, s, lane), d);
                        float sum = 0.f;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float e = j + r < i ? p[r] * d[r] : 0.f;
                            sum += e;
                            const float col = row16_sum(e);
                            if (lr == 0) atomicAdd(&scr->row[wave][j + r], -col);
                        }
                        sum += __shfl_xor(sum, 16);
                        sum += __shfl_xor(sum, 32);
                        if (lg == 0) atomicAdd(&scr->row[wave][i], sum);
                    }
                }
            };
            auto pzero = [&] {
                store4<T>((kPair ? sv + p_at<SL>(0, 1, 0) : sp + p_at_own<T>(0, 1, 0)) + p_off<T>(lr, lg),
                          f32x4_t{0.f, 0.f, 0.f, 0.f});
            };
            if constexpr (MODE == kGrad) scr->row[wave][lane] = 0.f;
            // all operands of a wave's tiles are read before the first product
            constexpr int SN = DK / 32;
            auto read = [&](Frag8<T> (&f)[SN], const T* rows0, int tile) {
#pragma unroll
                for (int s = 0; s < SN; ++s) f[s] = Tile<T, DK>::rows8(rows0, 16 * tile, s, lane);
            };
            if (wave == 0) {
                Frag8<T> k0[SN], k1[SN], q0[SN], q1[SN];
                read(k0, sk, 0);
                read(q0, sq, 0);
                read(q1, sq, 1);
                read(k1, sk, 1);
                __builtin_amdgcn_sched_barrier(0);
                f32x4_t x = zero, y = zero, z = zero;
#pragma unroll
                for (int s = 0; s < SN; ++s) {
                    x = mma(k0[s], q0[s], x);
                    y = mma(k0[s], q1[s], y);
                    z = mma(k1[s], q1[s], z);
                }
                ptile(0, 0, x);
                ptile(1, 0, y);
                ptile(1, 1, z);
            } else if (wave == 1) {
                Frag8<T> k0[SN], k1[SN], k2[SN], q2[SN];
                read(q2, sq, 2);
                read(k0, sk, 0);
                read(k1, sk, 1);
                read(k2, sk, 2);
                __builtin_amdgcn_sched_barrier(0);
                f32x4_t x = zero, y = zero, z = zero;
#pragma unroll
                for (int s = 0; s < SN; ++s) {
                    x = mma(k0[s], q2[s], x);
                    y = mma(k1[s], q2[s], y);
                    z = mma(k2[s], q2[s], z);
                }
                ptile(2, 0, x);
                ptile(2, 1, y);
                ptile(2, 2, z);
            } else {
                const int tj = wave == 2 ? 0 : 2;
                Frag8<T> k0[SN], k1[SN], q3[SN];
                read(q3, sq, 3);
                read(k0, sk, tj);
                read(k1, sk, tj + 1);
                __builtin_amdgcn_sched_barrier(0);
                f32x4_t x = zero, y = zero;
#pragma unroll
                for (int s = 0; s < SN; ++s) {
                    x = mma(k0[s], q3[s], x);
                    y = mma(k1[s], q3[s], y);
                }
                if (wave == 2) {
                    ptile(3, 0, x);
                    ptile(3, 1, y);
                    pzero();
                } else {
                    ptile(3, 2, x);
                    ptile(3, 3, y);
                }
            }
            if (kRows && m0 > 0) store_rows(m0 - C);
            // the entering state's part, this wave's columns
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[t][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            Frag8<T> fq[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) fq[t] = Tile<T, DK>::rows(sq, 16 * t, 0, lane);
#pragma unroll
            for (int s = 0; s < SN; ++s) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    Frag8<T> fs[NS];
                    float x[8];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        x[r] = S[2 * s][n][r];
                        x[4 + r] = S[2 * s + 1][n][r];
                    }
                    split(x, fs);
#pragma unroll
                    for (int p = NS - 1; p >= 0; --p)
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            acc[t][n] = mma(fs[p], fq[t], acc[t][n]);
                            if (p == 0 && n == NT - 1 && s + 1 < SN) fq[t] = Tile<T, DK>::rows(sq, 16 * t, s + 1, lane);
                        }
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (MODE == kOut && more) {
#pragma unroll
                    for (int i = s * NC / SN; i < (s + 1) * NC / SN; ++i) part_k(m0 + C, i);
                }
            }
            float in[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) in[t] = tb->in[16 * t + lr];
            if (__any(in[3] == 0.f)) {
                // a decay of 0 in the chunk (its last row has it too): behind it a
                // state that is not finite ends
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n) acc[t][n] = in[t] == 0.f ? zero : acc[t][n];
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int i = 16 * t + lr;
                const float e = in[t] * (s_scale * c);
                float dot = 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[t][n] *= e;
                    if constexpr (MODE == kGrad) {
                        const f32x4_t x = load4(sx + Tile<T, DV>::off(i, wcol + 16 * n + 4 * lg));
#pragma unroll
                        for (int r = 0; r < 4; ++r) dot += acc[t][n][r] * x[r];
                    }
                }
                if constexpr (MODE == kGrad) {
                    dot += __shfl_xor(dot, 16);
                    dot += __shfl_xor(dot, 32);
                    if (lg == 0) atomicAdd(&scr->row[wave][i], dot);
                }
            }
#pragma unroll
            for (int i = 0; i < KT; ++i) fk[i] = Tile<T, DK>::cols(sk, 16 * i, 0, lane);
            // the next chunk's tables: its decays came with this chunk's copies
            if (kPair && wave == kTab && more) tables(m0 + C);
            // B: P is whole; v, q and x are read
            barrier_keep_loads();
            if constexpr (MODE == kGrad) {
                if (tid < C && rows.has(m0 + tid)) {
                    a.sums[(int64_t)h * a.T_total + bl.start + rows.token(m0 + tid)] =
                        (scr->row[0][tid] + scr->row[1][tid]) + (scr->row[2][tid] + scr->row[3][tid]);
                }
            }
        }
        if constexpr (MODE == kState) {
#pragma unroll
            for (int i = 0; i < KT; ++i) fk[i] = Tile<T, DK>::cols(sk, 16 * i, 0, lane);
            if (wave == kTab && more) tables(m0 + C);
        }
        if (!kPair && more) fetch_v(m0 + C);
        if (kRows && more) part_q(m0 + C, 0);
        c = unif(c * tb->total);
        if (c < 1.f / 4096.f) {
            const bool off = c == 0.f;
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) S[i][n] = off ? zero : S[i][n] * c;
            c = 1.f;
        }
        const float u = u_scale / c;
        auto get_p = [&](int t, int s, int k) {
            Frag8<T> f;
            const T* x = (kPair ? sv + p_at<SL>(t, 2 * s, k) : sp + p_at_own<T>(t, 2 * s, k)) + p_off<T>(lr, lg);
            const T* y = (kPair ? sv + p_at<SL>(t, 2 * s + 1, k) : sp + p_at_own<T>(t, 2 * s + 1, k)) + p_off<T>(lr, lg);
            if constexpr (kBf) {
                f.v = __builtin_shufflevector(*reinterpret_cast<const bf16x4_t*>(x), *reinterpret_cast<const bf16x4_t*>(y),
                                              0, 1, 2, 3, 4, 5, 6, 7);
            } else {
                const f32x4_t u = load4(x), w = load4(y);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    f.v[r] = u[r];
                    f.v[4 + r] = w[r];
                }
            }
            return f;
        };
#pragma unroll
        for (int s = 0; s < C / 32; ++s) {
            Frag8<T> fu[NT][NU];
            const f32x4_t e0 = *reinterpret_cast<const f32x4_t*>(&tb->out[32 * s + 4 * lg]) * u;
            const f32x4_t e1 = *reinterpret_cast<const f32x4_t*>(&tb->out[32 * s + 16 + 4 * lg]) * u;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float x[8];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[r] = fv[s][n].get(r) * e0[r];
                    x[4 + r] = fv[s][n].get(4 + r) * e1[r];
                }
                split(x, fu[n]);
            }
            auto rest_q = [&](int from, int to) {   // the first half's three places for the other copies
                if (kRows && more && s == 0) {
#pragma unroll
                    for (int i = from; i < to; ++i) part_q(m0 + C, i);
                }
            };
            rest_q(1, 1 + (NC - 1 + 2) / 3);
            if constexpr (MODE != kState) {
#pragma unroll
                for (int t = 2 * s; t < 4; ++t) {
#pragma unroll
                    for (int k = NP - 1; k >= 0; --k) {
                        const Frag8<T> fp = get_p(t, s, k);
#pragma unroll
                        for (int n = 0; n < NT; ++n) acc[t][n] = mma(fv[s][n], fp, acc[t][n]);
                    }
                }
            }
            rest_q(1 + (NC - 1 + 2) / 3, 1 + (2 * (NC - 1) + 2) / 3);
            // one part for all of the state's tiles, then the next: a product on
            // the accumulator of the one before it would wait for that
#pragma unroll
            for (int p = NU - 1; p >= 0; --p) {
                if (p == 0) rest_q(1 + (2 * (NC - 1) + 2) / 3, NC);
#pragma unroll
                for (int i = 0; i < KT; ++i) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) S[i][n] = mma(fk[i], fu[n][p], S[i][n]);
                    if (s == 0 && p == 0) fk[i] = Tile<T, DK>::cols(sk, 16 * i, 1, lane);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if constexpr (kRows) {
            T* const o = sqb + ((m0 / C) & 1) * C * DK;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    store4<T>(o + Tile<T, DV>::off(16 * t + lr, wcol + 16 * n + 4 * lg), acc[t][n]);
        } else if constexpr (MODE != kState) {
            // buffer stores: the same number in every chunk, rows without a
            // token lie behind the bound and are dropped
            const int es = wide ? 4 : (int)sizeof(T);
            const unsigned step = xo.step;
            const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(
                reinterpret_cast<void*>(xo.token(rows.low(m0))), 0,
                uni((unsigned)(rows.tokens(m0) - 1) * step + DV * es), 0x00027000);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int row = 16 * t + lr;
                const unsigned at = (unsigned)(rev ? C - 1 - row : row) * step + (unsigned)((wcol + 4 * lg) * es);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (sizeof(T) == 4 || wide) {
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[t][n]), rsrc, at + 16 * n * 4, 0, 0);
                    } else {
                        const u32x2_t p = {cvt2(acc[t][n][0], acc[t][n][1]), cvt2(acc[t][n][2], acc[t][n][3])};
                        __builtin_amdgcn_raw_buffer_store_b64(p, rsrc, at + 16 * n * 2, 0, 0);
                    }
                }
            }
        }
        if (!kPair && more) {
            if (wave == kTab) tables(m0 + C);
            barrier_keep_loads();   // k is read
            fetch_k(m0 + C);
        }
    }
    if (kRows && cnt > 0) {
        barrier_keep_loads();
        store_rows(rows.rows - C);
    }

    float* dst = nullptr;
    float f = 1.f;
    if (MODE == kState) {
        dst = a.states + ((int64_t)b * a.H + h) * DK * DV;
        if (tid == 64 * kTab) a.decays[(int64_t)b * a.H + h] = exp2_fast((float)sum_total);
    } else if (last && a.final) {
        dst = a.final + ((int64_t)bl.n * a.H + h) * DK * DV;
        // backwards: the first token's own decay is still to come
        if (rev && cnt > 0) {
            const float g = a.g[a.g_per_token ? bl.begin * a.H + h : h];
            f = expf(g < kFloor ? kFloor : g);
        }
    }
    if (dst) {
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    dst[(int64_t)(16 * i + 4 * lg + r) * DV + wcol + 16 * n + lr] = S[i][n][r] * (f * c);
    }
}

// Entering states of every block from the blocks' own ones, in place:
// S_{j+1} = decay_j S_j + U_j, S_0 the sequence's (or 0); backwards from the
// last block for the state's gradient.  blockIdx.z: which of the two arrays.
// after (one state a sequence and head) gets the state behind the last block.
__global__ __launch_bounds__(256) void linattn_carry_kernel(LinArgs a, LinCarry c0, LinCarry c1) {
    const LinCarry c = blockIdx.z ? c1 : c0;
    const int n = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int b0 = first_block(a, n);
    int nb = blocks_of(a, seq_at(a, n + 1) - seq_at(a, n));
    if (nb > a.nblocks - b0) nb = a.nblocks - b0;   // offsets out of order: stay inside the arrays
    const int64_t e = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4, size = (int64_t)gridDim.y * 1024;
    f32x4_t s = {0.f, 0.f, 0.f, 0.f};
    if (c.initial) s = *reinterpret_cast<const f32x4_t*>(c.initial + ((int64_t)n * a.H + h) * size + e);
    // the blocks' own states and decays are read four ahead of the chain (16384
    // tokens of one head, d = 128, 256 blocks: the call 112 us with one ahead, 69
    // with four, 61 with eight, which many short chains pay for: 4 x 2048 tokens x
    // 32 heads, gradient, 370 against 377)
    constexpr int A = 4;
    auto index = [&](int i) { return (int64_t)(b0 + (c.reverse ? nb - 1 - i : i)) * a.H + h; };
    auto own = [&](int i) { return i + 1 < nb || (c.after && i < nb); };   // built by the state pass
    f32x4_t u[A], next[A];
    float d[A], dn[A];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int m = 0; m < A; ++m) {
            if (!own(i0 + m)) continue;
            next[m] = *reinterpret_cast<const f32x4_t*>(c.states + index(i0 + m) * size + e);
            dn[m] = c.decays[index(i0 + m)];
        }
    };
    fetch(0);
    for (int i0 = 0; i0 < nb; i0 += A) {
#pragma unroll
        for (int m = 0; m < A; ++m) {
            u[m] = next[m];
            d[m] = dn[m];
        }
        fetch(i0 + A);
#pragma unroll
        for (int m = 0; m < A; ++m) {
            if (i0 + m >= nb) break;
            *reinterpret_cast<f32x4_t*>(c.states + index(i0 + m) * size + e) = s;
            if (own(i0 + m)) s = d[m] == 0.f ? u[m] : s * d[m] + u[m];
        }
    }
    if (c.after) *reinterpret_cast<f32x4_t*>(c.after + ((int64_t)n * a.H + h) * size + e) = s;
}

template <typename T, int DK, int DV, int MODE>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void linattn_kernel(LinPair pair) {
    linattn_body<T, DK, DV, MODE>(pair.a[blockIdx.y]);
}

// The decay's gradient of a (block, head): dg_t = sum_{s >= t} (A_s - B_s) + E,
// A and B the two kGrad runs' sums of the block's tokens, E what crosses the
// block's end: the product of the state there with its gradient.
__device__ __forceinline__ void decay_gradient(const LinArgs& a, const LinTail& x, int size) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    double* const part = reinterpret_cast<double*>(smem);   // [4], of the waves
    double& carry = part[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
    if (a.clear) clear_rest<float, 1>(a, x.dg, b, h);
    const Block bl = find_block(a, b);
    if (bl.n < 0) return;
    const bool last = bl.j == bl.nb - 1 || b + 1 >= a.nblocks;
    const float *S = nullptr, *R = nullptr;
    if (!last) {
        S = x.states + ((int64_t)(b + 1) * a.H + h) * size;
        R = x.rstates + ((int64_t)b * a.H + h) * size;
    } else if (x.r_end) {
        S = x.s_end + ((int64_t)bl.n * a.H + h) * size;
        R = x.r_end + ((int64_t)bl.n * a.H + h) * size;
    }
    double e = 0.0;
    if (S) {
        // in fp64: under strong decays the tokens next to the block's end take
        // nearly all of it away again
#pragma unroll 8
        for (int i = tid * 4; i < size; i += 1024) {
            const f32x4_t u = *reinterpret_cast<const f32x4_t*>(S + i), v = *reinterpret_cast<const f32x4_t*>(R + i);
#pragma unroll
            for (int r = 0; r < 4; ++r) e += (double)u[r] * (double)v[r];
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) e += shfl_d(e, lane ^ d);
    }
    if (lane == 0) part[wave] = e;
    __syncthreads();
    if (tid == 0) {
        double s = (part[0] + part[1]) + (part[2] + part[3]);
        if (!last) {
            const float g = a.g[a.g_per_token ? (bl.start + bl.cnt) * a.H + h : h];
            s *= exp((double)(g < kFloor ? kFloor : g));
        }
        carry = s;
    }
    __syncthreads();
    // from the block's end, 256 tokens at a time
    for (int m0 = 0; m0 < bl.cnt; m0 += 256) {
        const int m = m0 + tid;
        const int64_t tok = bl.start + bl.cnt - 1 - m, at = (int64_t)h * a.T_total + tok;
        double d = m < bl.cnt ? (double)x.sums_a[at] - (double)x.sums_b[at] : 0.0;
#pragma unroll
        for (int k = 1; k < kWave; k <<= 1) {
            const double o = shfl_d(d, lane - k < 0 ? 0 : lane - k);
            if (lane >= k) d += o;
        }
        if (lane == 63) part[wave] = d;
        __syncthreads();
        double before = carry;
        for (int w = 0; w < wave; ++w) before += part[w];
        const double v = before + d;
        __syncthreads();
        if (tid == 255) carry = v;
        if (m < bl.cnt) x.dg[tok * a.H + h] = (float)v;
        __syncthreads();
    }
}

// Sums over the value heads that share a key head, fp32 [T, H, D] to
// [T, H / r, D], of dq's and dk's parts: runs of 4 elements, four a thread in
// flight.
template <typename T, int D>
__device__ __forceinline__ void share_sums(const LinArgs& a, const LinTail& x) {
    const int r = x.share;
    const int64_t n4 = a.T_total * (a.H / r) * (D / 4), all = 2 * n4, step = (int64_t)gridDim.x * 256;
    const int64_t t0 = seq_at(a, 0), t1 = seq_at(a, a.num_seqs);
    const int per = a.H / r * (D / 4);   // runs of a token
    for (int64_t u0 = (int64_t)blockIdx.x * 256 + threadIdx.x; u0 < all; u0 += 4 * step) {
        const float* p[4];
        f32x4_t s[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int64_t u = u0 + m * step < all ? u0 + m * step : u0;
            p[m] = x.parts + (u / (D / 4)) * r * D + u % (D / 4) * 4;
            s[m] = *reinterpret_cast<const f32x4_t*>(p[m]);
        }
        for (int j = 1; j < r; ++j)
#pragma unroll
            for (int m = 0; m < 4; ++m) s[m] += *reinterpret_cast<const f32x4_t*>(p[m] + (int64_t)j * D);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int64_t u = u0 + m * step, i = u < n4 ? u : u - n4;
            const int64_t tok = i / per;
            const bool outside = tok < t0 || tok >= t1;
            if (u >= all || (outside && !a.clear)) continue;
            if (outside) s[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            const float o[4] = {s[m][0], s[m][1], s[m][2], s[m][3]};
            store_vec<T, 4>((T*)(u < n4 ? x.dq : x.dk) + i * 4, o);
        }
    }
}

// The gradient's last run, for dv, and beside it what waits for the runs before
// only (dv's workgroups leave CUs half empty).  1531 ragged tokens of 8 heads in
// fp32: the gradient 49 us, 59 with a launch each for these; 8192 tokens x 32
// heads on 8 key heads 390 and 420.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void linattn_last_kernel(LinArgs a, LinTail x) {
    if (blockIdx.y == 0) linattn_body<T, DK, DV, kOut>(a);
    else if (blockIdx.y == 1) decay_gradient(a, x, DK * DV);
    else share_sums<T, DK>(a, x);
}

// dg of a decay that all tokens of a head share: the sum over tokens, one
// workgroup a head, in a fixed order.
__global__ __launch_bounds__(256) void linattn_dg_sum_kernel(LinArgs a, const float* dg, float* out) {
    __shared__ double part[256];
    const int h = blockIdx.x, tid = threadIdx.x;
    const int64_t end = seq_at(a, a.num_seqs);
    double s = 0.0;
    for (int64_t t = seq_at(a, 0) + tid; t < end; t += 256) s += (double)dg[t * a.H + h];
    part[tid] = s;
    __syncthreads();
    for (int d = 128; d > 0; d >>= 1) {
        if (tid < d) part[tid] += part[tid + d];
        __syncthreads();
    }
    if (tid == 0) out[h] = (float)part[0];
}

template <typename T, int DK, int DV, int MODE>
hipError_t launch_t(const LinArgs* a, int n) {
    constexpr int lds = lds_bytes<T, DK, DV, MODE>();
    static_assert(lds <= 160 * 1024, "LDS");
    const void* kern = reinterpret_cast<const void*>(&linattn_kernel<T, DK, DV, MODE>);
    hipError_t e = ensure_lds_limit(kern, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((linattn_kernel<T, DK, DV, MODE>), dim3((unsigned)(a->nblocks * a->H), n), dim3(256), lds,
                       (hipStream_t)a->stream, LinPair{{a[0], a[n - 1]}});
    return hipGetLastError();
}

template <typename T, int DK, int DV>
hipError_t launch_last_t(const LinArgs& a, const LinTail& x) {
    constexpr int lds = lds_bytes<T, DK, DV, kOut>();
    const void* kern = reinterpret_cast<const void*>(&linattn_last_kernel<T, DK, DV>);
    hipError_t e = ensure_lds_limit(kern, lds);
    if (e != hipSuccess) return e;
    const unsigned parts = !x.dg ? 1 : x.share > 1 ? 3 : 2;
    hipLaunchKernelGGL((linattn_last_kernel<T, DK, DV>), dim3((unsigned)(a.nblocks * a.H), parts), dim3(256), lds,
                       (hipStream_t)a.stream, a, x);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_last(const LinArgs& a, const LinTail& x, int dk, int dv) {
    if (dk == 64) return dv == 64 ? launch_last_t<T, 64, 64>(a, x) : launch_last_t<T, 64, 128>(a, x);
    return dv == 64 ? launch_last_t<T, 128, 64>(a, x) : launch_last_t<T, 128, 128>(a, x);
}

template <typename T, int MODE>
hipError_t launch_m(const LinArgs* a, int n, int dk, int dv) {
    if (dk == 64) return dv == 64 ? launch_t<T, 64, 64, MODE>(a, n) : launch_t<T, 64, 128, MODE>(a, n);
    return dv == 64 ? launch_t<T, 128, 64, MODE>(a, n) : launch_t<T, 128, 128, MODE>(a, n);
}

template <typename T>
hipError_t launch_k(const LinArgs* a, int n, int dk, int dv, int mode) {
    if (mode == kState) return launch_m<T, kState>(a, n, dk, dv);
    return mode == kOut ? launch_m<T, kOut>(a, n, dk, dv) : launch_m<T, kGrad>(a, n, dk, dv);
}

// One or two runs of the same kernel, side by side in one launch.
hipError_t launch_core(const LinArgs* a, int n, int dtype, int dk, int dv, int mode) {
    return dtype == 0 ? launch_k<__bf16>(a, n, dk, dv, mode) : launch_k<float>(a, n, dk, dv, mode);
}

hipError_t launch_plan(const LinArgs& a) {
    if (!a.first) return hipSuccess;
    hipLaunchKernelGGL(linattn_plan_kernel, dim3(1), dim3(1024), 0, (hipStream_t)a.stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linattn_fwd(const LinCall& c) {
    LinArgs a = c.args;
    const hipError_t planned = launch_plan(a);
    if (planned != hipSuccess) return planned;
    a.q = c.q;
    a.k = c.k;
    a.v = c.v;
    a.p_scale = a.s_scale = c.scale;
    a.u_scale = 1.f;
    if (c.states) {
        // several blocks a sequence: their own states, the carry, then all outputs at once
        LinArgs s = a;
        s.states = c.states;
        s.decays = c.decays;
        hipError_t e = launch_core(&s, 1, c.dtype, c.dk, c.dv, kState);
        if (e != hipSuccess) return e;
        const LinCarry f{c.states, c.decays, c.initial_state, nullptr, 0};
        hipLaunchKernelGGL(linattn_carry_kernel, dim3((unsigned)(a.num_seqs * a.H), (unsigned)(c.dk * c.dv / 1024), 1),
                           dim3(256), 0, (hipStream_t)a.stream, a, f, f);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.states = c.states;
    } else {
        a.initial = c.initial_state;
    }
    a.final = c.final_state;
    a.out = c.y;
    return launch_core(&a, 1, c.dtype, c.dk, c.dv, kOut);
}

hipError_t launch_linattn_bwd(const LinCall& c) {
    LinArgs a = c.args;
    a.p_scale = c.scale;
    hipError_t e = launch_plan(a);
    if (e != hipSuccess) return e;
    // the blocks' own states, of the recurrence and of its gradient
    LinArgs s[2] = {a, a};
    s[0].k = c.k;
    s[0].v = c.v;
    s[0].u_scale = 1.f;
    s[0].states = c.states;
    s[0].decays = c.decays;
    s[0].last_state = c.d_final_state != nullptr;
    s[1].k = c.q;
    s[1].v = c.dy;
    s[1].u_scale = c.scale;
    s[1].states = c.rstates;
    s[1].decays = c.rdecays;
    s[1].reverse = true;
    if ((e = launch_core(s, 2, c.dtype, c.dk, c.dv, kState)) != hipSuccess) return e;
    const LinCarry f{c.states, c.decays, c.initial_state, c.d_final_state ? c.s_end : nullptr, 0};
    const LinCarry r{c.rstates, c.rdecays, c.d_final_state, nullptr, 1};
    hipLaunchKernelGGL(linattn_carry_kernel, dim3((unsigned)(a.num_seqs * a.H), (unsigned)(c.dk * c.dv / 1024), 2),
                       dim3(256), 0, (hipStream_t)a.stream, a, f, r);
    if ((e = hipGetLastError()) != hipSuccess) return e;

    // dq with the pairs' and the entering state's part of dg, and dk
    const bool shared = c.k.share > 1;
    LinArgs x[2] = {a, a};
    x[0].q = c.dy;
    x[0].k = c.v;
    x[0].v = c.k;
    x[0].x = c.q;
    x[0].s_scale = c.scale;
    x[0].u_scale = 1.f;
    x[0].states = c.states;
    x[0].transposed = true;
    x[0].pairs = true;
    x[0].sums = c.sums_a;
    x[0].out = shared ? c.share_buf : c.dq;
    x[0].out_f32 = shared;
    x[1] = x[0];
    x[1].q = c.v;
    x[1].k = c.dy;
    x[1].v = c.q;
    x[1].x = c.k;
    x[1].s_scale = 1.f;
    x[1].u_scale = c.scale;
    x[1].states = c.rstates;
    x[1].pairs = false;
    x[1].reverse = true;
    x[1].sums = c.sums_b;
    x[1].out = shared ? static_cast<float*>(c.share_buf) + a.T_total * a.H * c.dk : c.dk_out;
    if ((e = launch_core(x, 2, c.dtype, c.dv, c.dk, kGrad)) != hipSuccess) return e;
    // dv and the gradient of the initial state
    LinArgs d = a;
    d.q = c.k;
    d.k = c.q;
    d.v = c.dy;
    d.s_scale = 1.f;
    d.u_scale = c.scale;
    d.states = c.rstates;
    d.reverse = true;
    d.final = c.d_initial_state;
    d.out = c.dv_out;
    // beside it dg, and dq and dk of shared heads
    LinTail t{};
    t.states = c.states;
    t.rstates = c.rstates;
    t.s_end = c.s_end;
    t.r_end = c.d_final_state;
    t.sums_a = c.sums_a;
    t.sums_b = c.sums_b;
    t.dg = c.dg && !a.g_per_token ? c.dg_tokens : c.dg;
    t.share = c.k.share;
    t.parts = (const float*)c.share_buf;
    t.dq = c.dq;
    t.dk = c.dk_out;
    e = c.dtype == 0 ? launch_last<__bf16>(d, t, c.dk, c.dv) : launch_last<float>(d, t, c.dk, c.dv);
    if (e != hipSuccess) return e;
    if (c.dg && !a.g_per_token) {
        hipLaunchKernelGGL(linattn_dg_sum_kernel, dim3((unsigned)a.H), dim3(256), 0, (hipStream_t)a.stream, a,
                           c.dg_tokens, c.dg);
        return hipGetLastError();
    }
    return hipSuccess;
}

// One token a request against the resident fp32 state [N, H, dk, dv], updated
// in place: S <- exp(g) S + k v^T, y = scale S^T q.  Unlike the delta rule,
// columns are independent, so a workgroup takes COLS columns of a (request,
// head): all of them, or narrow slices to spread few states over the CUs.  Bound
// by the state's two crossings of memory; both nontemporal, and the writes
// behind all of a workgroup's reads (128 x 96 states of 128 x 128: 302 us with
// each piece written at once, 292 behind, 272 with nontemporal reads).
namespace {

template <typename T, int DK, int COLS>
__global__ __launch_bounds__(256) void linattn_decode_kernel(LinDecodeArgs a) {
    constexpr int CG = COLS / 4, RG = 256 / CG, RPT = DK / RG;
    static_assert(RG * CG == 256 && RPT * RG == DK, "decode tiling");
    __shared__ float s_k[DK], s_q[DK];
    __shared__ float s_o[RG][COLS + 4];
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
    const int slices = a.dv / COLS;
    // whole states: each XCD takes them in runs of two (workgroups i, i + 8,
    // ... share one), as the KDA decode step does
    int id = blockIdx.x;
    if (slices == 1 && gridDim.x % 16 == 0) id = id / 16 * 16 + id % 8 * 2 + id / 8 % 2;
    const int nh = id / slices, col0 = (id % slices) * COLS;
    const int n = nh / a.H, h = nh % a.H;
    float* st = a.state + (int64_t)nh * DK * a.dv + col0 + 4 * cg;
    f32x4_t S[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) S[r] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(st + (int64_t)(r * RG + rg) * a.dv));
    const T* q = (const T*)a.q.p + (int64_t)n * a.q.stride + (int64_t)(h / a.q.share) * DK;
    const T* k = (const T*)a.k.p + (int64_t)n * a.k.stride + (int64_t)(h / a.k.share) * DK;
    const T* v = (const T*)a.v.p + (int64_t)n * a.v.stride + (int64_t)h * a.dv + col0 + 4 * cg;
    for (int c = tid; c < DK; c += 256) {
        s_k[c] = gload(k + c);
        s_q[c] = gload(q + c);
    }
    float vv[4];
    load_vec<T, 4>(v, vv);
    const f32x4_t v4 = {vv[0], vv[1], vv[2], vv[3]};
    const float decay = expf(a.g[a.g_per_token ? nh : h]);
    if (decay == 0.f) {   // anew, whatever the state holds
#pragma unroll
        for (int r = 0; r < RPT; ++r) S[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    __syncthreads();
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int row = r * RG + rg;
        S[r] = S[r] * decay + s_k[row] * v4;
        o += s_q[row] * S[r];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s_o[rg][4 * cg + i] = o[i];
    __syncthreads();
    if (tid < COLS) {
        float x = 0.f;
#pragma unroll
        for (int r = 0; r < RG; ++r) x += s_o[r][tid];
        gstore((T*)a.y + (int64_t)nh * a.dv + col0 + tid, a.scale * x);
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) __builtin_nontemporal_store(S[r], reinterpret_cast<f32x4_t*>(st + (int64_t)(r * RG + rg) * a.dv));
}

template <typename T, int DK, int COLS>
hipError_t decode_t(const LinDecodeArgs& a) {
    hipLaunchKernelGGL((linattn_decode_kernel<T, DK, COLS>), dim3((unsigned)((int64_t)a.N * a.H * (a.dv / COLS))),
                       dim3(256), 0, (hipStream_t)a.stream, a);
    return hipGetLastError();
}

template <typename T, int DK>
hipError_t decode_c(const LinDecodeArgs& a) {
    if (a.N * (int64_t)a.H < 512) return decode_t<T, DK, 16>(a);
    return a.dv == 64 ? decode_t<T, DK, 64>(a) : decode_t<T, DK, 128>(a);
}

}  // namespace

hipError_t launch_linattn_decode(const LinDecodeArgs& a) {
    if (a.N == 0) return hipSuccess;
    if (a.dtype == 0) return a.dk == 64 ? decode_c<__bf16, 64>(a) : decode_c<__bf16, 128>(a);
    return a.dk == 64 ? decode_c<float, 64>(a) : decode_c<float, 128>(a);
}

}  // namespace kda
