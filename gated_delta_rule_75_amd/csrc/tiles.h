// Tiles, operands, copies and blocks of tokens shared by the kernels that work by
// chunks of 64 tokens (gfx950 only).
#pragma once

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
// max(1, ceil(len / L)) blocks, numbered across the sequences in order; with LEAST one
// of fewer than LEAST blocks stays whole, as one block of any length, and with CUT such
// sequences are passed over in the numbering.
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
template <int LEAST = 1>
__device__ __forceinline__ int blocks_of(const LinArgs& a, int64_t len) {
    const int64_t nb = len <= (LEAST > 1 ? (LEAST - 1) * a.L : a.L) ? 1 : (len + a.L - 1) / a.L;
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
template <int LEAST = 1, bool CUT = false>
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
                nb = blocks_of<LEAST>(a, e - s);
                if (CUT && nb == 1) nb = 0;
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
    r.cnt = uni((int)(left < 0 ? 0 : left < a.L || (LEAST > 1 && r.nb == 1) ? left : a.L));
    return r;
}

// Index of sequence n's first block.
template <int LEAST = 1>
__device__ __forceinline__ int first_block(const LinArgs& a, int n) {
    if (a.L >= a.T_total) return n;
    if (a.first) return a.first[n];
    const int lane = threadIdx.x & 63;
    int sum = 0;
    for (int m = lane; m < n; m += kWave) sum += blocks_of<LEAST>(a, seq_at(a, m + 1) - seq_at(a, m));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    return sum;
}

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

}  // namespace

}  // namespace kda
