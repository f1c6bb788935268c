// C ABI of the layer operators around the KDA recurrence: linear attention with
// a decay for each head, rotary positions, the gated norm.  Every check runs
// before anything is enqueued.
#include "../../include/kda.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "launch.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(kda_dtype dt) { return dt == KDA_BF16 || dt == KDA_F32; }
size_t elt(kda_dtype dt) { return dt == KDA_BF16 ? 2 : 4; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Nothing is thrown across the ABI (the launchers keep a locked set).
template <typename F>
kda_status launched(F f) {
    try {
        return f() == hipSuccess ? KDA_OK : KDA_ERR_HIP;
    } catch (...) {
        return KDA_ERR_HIP;
    }
}

bool head_ok(int d) { return d == 64 || d == 128; }

// A chunk of 64 tokens is addressed with 32 bits.
constexpr int64_t kMaxStride = int64_t(1) << 23;

// Rows of heads x d elements at a token stride, moved in 16-byte pieces.
bool rows_ok(kda_dtype dt, const void* p, int64_t stride, int heads, int d) {
    return aligned(p, 16) && stride >= (int64_t)heads * d && stride <= kMaxStride && stride % (int64_t)(16 / elt(dt)) == 0;
}

// Tokens of a block.  Sequences longer than a block are cut, and their blocks
// run side by side from states that a first pass over k and v builds (about half
// the call's reads again): worth it where uncut sequences leave CUs without
// work.  In bf16 512 workgroups (two a CU) run at once, and the ones behind them
// would take a second round: so the blocks of one long sequence are as many as
// that holds (`groups` workgroups), and no shorter than `least`.  The rule is of
// tokens and heads alone.  In fp32 with d = 128 a CU holds one workgroup, so the
// blocks take two rounds; and in a batch of sequences that are all shorter than a
// block, each still gets an entering state in the workspace.
int64_t block_len(int H, int64_t T, int groups, int64_t least, int64_t most) {
    const int64_t n = H < groups ? groups / H : 1;
    int64_t L = ((T + n - 1) / n + 63) / 64 * 64;
    if (L < least) L = least;
    if (L > most) L = most;
    const int64_t all = T < 64 ? 64 : (T + 63) / 64 * 64;
    return L < all ? L : all;
}

// One chunk at least: for few tokens the chain of chunks is what takes the time
// (1531 ragged tokens of 8 heads, gradient: 105 us with blocks of 256 tokens or
// more, 72 with 128, 67 with 64).  The gradient re-anchors its decay sums at
// block ends, at most 1024 tokens apart, and runs two passes side by side: half
// as many blocks (8192 tokens x 32 heads, d = 128: 379 us, 405 with twice as many).
int64_t fwd_block(int H, int64_t T) { return block_len(H, T, 512, 64, INT64_MAX); }
int64_t bwd_block(int H, int64_t T) { return block_len(H, T, 256, 64, 1024); }

// (block, head) pairs of a call: an axis of a launch holds less than 2^32
// threads, 256 a pair; well inside that, as blocks shorter than 1024 tokens add
// at most 512 pairs or one block a head.
constexpr int64_t kMaxBlocks = (int64_t(1) << 22) - 1024;

bool sizes_ok(kda_dtype dt, int H, int Hk, int dk, int dv, int num_seqs, int64_t T) {
    return dtype_ok(dt) && H > 0 && Hk > 0 && H % Hk == 0 && num_seqs > 0 && T >= 0 && T <= INT32_MAX - 64 &&
           head_ok(dk) && head_ok(dv) && (T / 1024 + num_seqs) * (int64_t)H < kMaxBlocks;
}

// Parts of a workspace, each 256-byte aligned.
struct Parts {
    size_t at = 0;
    size_t take(size_t bytes) {
        const size_t p = at;
        at += round_up(bytes, 256);
        return p;
    }
};

// Above this many sequences, cut ones get a table of their first blocks: a
// workgroup finds its block by counting otherwise, 64 sequences at a step, which
// with N sequences is N^2 / 64 steps in all.
constexpr int kPlanSeqs = 256;
size_t plan_bytes(int num_seqs) { return num_seqs > kPlanSeqs ? ((size_t)num_seqs + 1) * 4 : 0; }

struct FwdLayout { size_t states, decays, plan, total; int64_t L, nblocks; };
FwdLayout fwd_layout(int H, int dk, int dv, int num_seqs, int64_t T) {
    FwdLayout l{};
    l.L = fwd_block(H, T);
    const bool cut = l.L < T;
    l.nblocks = cut ? T / l.L + num_seqs : num_seqs;
    Parts p;
    if (cut) {
        l.states = p.take((size_t)l.nblocks * H * dk * dv * 4);
        l.decays = p.take((size_t)l.nblocks * H * 4);
        l.plan = p.take(plan_bytes(num_seqs));
    }
    l.total = p.at;
    return l;
}

struct BwdLayout { size_t states, decays, rstates, rdecays, s_end, sums_a, sums_b, dg, share, plan, total; int64_t L, nblocks; };
BwdLayout bwd_layout(int H, int Hk, int dk, int dv, int num_seqs, int64_t T) {
    BwdLayout l{};
    l.L = bwd_block(H, T);
    l.nblocks = l.L < T ? T / l.L + num_seqs : num_seqs;
    const size_t state = (size_t)H * dk * dv * 4, th = (size_t)T * H * 4;
    Parts p;
    l.states = p.take(l.nblocks * state);
    l.rstates = p.take(l.nblocks * state);
    l.decays = p.take((size_t)l.nblocks * H * 4);
    l.rdecays = p.take((size_t)l.nblocks * H * 4);
    l.s_end = p.take(num_seqs * state);
    l.sums_a = p.take(th);
    l.sums_b = p.take(th);
    l.dg = p.take(th);
    l.share = p.take(Hk < H ? 2 * th * dk : 0);
    l.plan = p.take(l.L < T ? plan_bytes(num_seqs) : 0);
    l.total = p.at;
    return l;
}

template <typename P> P* part(void* ws, size_t at) { return reinterpret_cast<P*>(static_cast<char*>(ws) + at); }

kda::LinRows rows(const void* p, int64_t stride, int share) { return kda::LinRows{p, stride, share}; }

kda_status rope_call(kda_dtype dt, int64_t T, int Hq, int Hk, int d, int rot, kda_rope_layout layout, int inverse,
                     float mscale, int axes, const int32_t* positions, const uint8_t* pair_axis, const double* inv_freq, const void* q, int64_t q_stride,
                     const void* k, int64_t k_stride, void* q_out, int64_t q_out_stride, void* k_out,
                     int64_t k_out_stride, void* stream) {
    if (!dtype_ok(dt) || T < 0 || T > INT32_MAX || Hq <= 0 || Hk < 0 || d <= 0) return KDA_ERR_INVALID_ARGUMENT;
    if (layout != KDA_ROPE_HALF && layout != KDA_ROPE_INTERLEAVED) return KDA_ERR_INVALID_ARGUMENT;
    if (rot <= 0 || rot % 2 != 0 || rot > d) return KDA_ERR_INVALID_ARGUMENT;
    if (d > 1024 || (int64_t)(Hq + (int64_t)Hk) * d > 1 << 24) return KDA_ERR_UNSUPPORTED;
    if (T > 0 && (!positions || !inv_freq || !q || !q_out || (Hk > 0 && (!k || !k_out)))) return KDA_ERR_INVALID_ARGUMENT;
    if (q_stride < (int64_t)Hq * d || q_out_stride < (int64_t)Hq * d || k_stride < (int64_t)Hk * d ||
        k_out_stride < (int64_t)Hk * d)
        return KDA_ERR_INVALID_ARGUMENT;
    if ((q == q_out && q_stride != q_out_stride) || (Hk > 0 && k == k_out && k_stride != k_out_stride))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t e = elt(dt);
    if (!aligned(q, e) || !aligned(k, e) || !aligned(q_out, e) || !aligned(k_out, e) || !aligned(positions, 4) ||
        !aligned(inv_freq, 8))
        return KDA_ERR_INVALID_ARGUMENT;
    kda::RopeArgs a{};
    a.dtype = (int)dt;
    a.T = T;
    a.Hq = Hq;
    a.Hk = Hk;
    a.d = d;
    a.rot = rot;
    a.half = layout == KDA_ROPE_HALF;
    a.inverse = inverse != 0;
    a.mscale = mscale;
    a.positions = positions;
    a.pair_axis = pair_axis;
    a.axes = axes;
    a.inv_freq = inv_freq;
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_out = q_out;
    a.k_out = k_out;
    a.qo_stride = q_out_stride;
    a.ko_stride = k_out_stride;
    a.stream = stream;
    return launched([&] { return kda::launch_rope(a); });
}

// clear: rows of no sequence of the outputs become zeros.
kda_status linattn_fwd(bool clear, kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs,
                       int64_t T_total, const int32_t* cu_seqlens, const void* q, int64_t q_stride, const void* k,
                       int64_t k_stride, const void* v, int64_t v_stride, const float* g, int g_per_token,
                       const float* initial_state, float* final_state, void* y, void* workspace,
                       size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return KDA_ERR_INVALID_ARGUMENT;
    if (!cu_seqlens && num_seqs != 1) return KDA_ERR_INVALID_ARGUMENT;
    if (H > 0 && Hk > 0 && (!head_ok(dk) || !head_ok(dv))) return KDA_ERR_UNSUPPORTED;
    if (!sizes_ok(dt, H, Hk, dk, dv, num_seqs, T_total)) return KDA_ERR_INVALID_ARGUMENT;
    if (T_total > 0 && (!q || !k || !v || !g || !y)) return KDA_ERR_INVALID_ARGUMENT;
    if (!rows_ok(dt, q, q_stride, Hk, dk) || !rows_ok(dt, k, k_stride, Hk, dk) || !rows_ok(dt, v, v_stride, H, dv) ||
        !aligned(y, 16) || !aligned(g, 4) || !aligned(cu_seqlens, 4) || !aligned(initial_state, 16) ||
        !aligned(final_state, 16) || !aligned(workspace, 256))
        return KDA_ERR_INVALID_ARGUMENT;
    const FwdLayout l = fwd_layout(H, dk, dv, num_seqs, T_total);
    if (l.total && !workspace) return KDA_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < l.total) return KDA_ERR_WORKSPACE_TOO_SMALL;
    kda::LinCall c{};
    c.args.H = H;
    c.args.num_seqs = num_seqs;
    c.args.T_total = T_total;
    c.args.cu_seqlens = cu_seqlens;
    c.args.L = l.L;
    c.args.nblocks = (int)l.nblocks;
    c.args.g = g;
    c.args.g_per_token = g_per_token != 0;
    c.args.clear = clear;
    c.args.stream = stream;
    c.dtype = (int)dt;
    c.dk = dk;
    c.dv = dv;
    c.scale = scale;
    c.q = rows(q, q_stride, H / Hk);
    c.k = rows(k, k_stride, H / Hk);
    c.v = rows(v, v_stride, 1);
    c.initial_state = initial_state;
    c.final_state = final_state;
    c.y = y;
    if (l.total) {
        c.states = part<float>(workspace, l.states);
        c.decays = part<float>(workspace, l.decays);
        if (num_seqs > kPlanSeqs) c.args.first = part<int32_t>(workspace, l.plan);
    }
    return launched([&] { return kda::launch_linattn_fwd(c); });
}

kda_status linattn_bwd(bool clear, kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs,
                       int64_t T_total, const int32_t* cu_seqlens, const void* q, int64_t q_stride, const void* k,
                       int64_t k_stride, const void* v, int64_t v_stride, const float* g, int g_per_token,
                       const float* initial_state, const void* dy, const float* d_final_state, void* dq,
                       void* dk_out, void* dv_out, float* dg, float* d_initial_state, void* workspace,
                       size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return KDA_ERR_INVALID_ARGUMENT;
    if (!cu_seqlens && num_seqs != 1) return KDA_ERR_INVALID_ARGUMENT;
    if (H > 0 && Hk > 0 && (!head_ok(dk) || !head_ok(dv))) return KDA_ERR_UNSUPPORTED;
    if (!sizes_ok(dt, H, Hk, dk, dv, num_seqs, T_total)) return KDA_ERR_INVALID_ARGUMENT;
    if (T_total > 0 && (!q || !k || !v || !g || !dy || !dq || !dk_out || !dv_out)) return KDA_ERR_INVALID_ARGUMENT;
    if ((!dg && (T_total > 0 || !g_per_token)) || !workspace) return KDA_ERR_INVALID_ARGUMENT;
    if (!rows_ok(dt, q, q_stride, Hk, dk) || !rows_ok(dt, k, k_stride, Hk, dk) || !rows_ok(dt, v, v_stride, H, dv) ||
        !aligned(dy, 16) || !aligned(dq, 16) || !aligned(dk_out, 16) || !aligned(dv_out, 16) || !aligned(g, 4) ||
        !aligned(dg, 4) || !aligned(cu_seqlens, 4) || !aligned(initial_state, 16) || !aligned(d_final_state, 16) ||
        !aligned(d_initial_state, 16) || !aligned(workspace, 256))
        return KDA_ERR_INVALID_ARGUMENT;
    const BwdLayout l = bwd_layout(H, Hk, dk, dv, num_seqs, T_total);
    if (workspace_bytes < l.total) return KDA_ERR_WORKSPACE_TOO_SMALL;
    kda::LinCall c{};
    c.args.H = H;
    c.args.num_seqs = num_seqs;
    c.args.T_total = T_total;
    c.args.cu_seqlens = cu_seqlens;
    c.args.L = l.L;
    c.args.nblocks = (int)l.nblocks;
    c.args.g = g;
    c.args.g_per_token = g_per_token != 0;
    c.args.clear = clear;
    c.args.stream = stream;
    c.dtype = (int)dt;
    c.dk = dk;
    c.dv = dv;
    c.scale = scale;
    c.q = rows(q, q_stride, H / Hk);
    c.k = rows(k, k_stride, H / Hk);
    c.v = rows(v, v_stride, 1);
    c.dy = rows(dy, (int64_t)H * dv, 1);
    c.initial_state = initial_state;
    c.d_final_state = d_final_state;
    c.d_initial_state = d_initial_state;
    c.dq = dq;
    c.dk_out = dk_out;
    c.dv_out = dv_out;
    c.dg = dg;
    c.states = part<float>(workspace, l.states);
    c.rstates = part<float>(workspace, l.rstates);
    c.decays = part<float>(workspace, l.decays);
    c.rdecays = part<float>(workspace, l.rdecays);
    c.s_end = part<float>(workspace, l.s_end);
    c.sums_a = part<float>(workspace, l.sums_a);
    c.sums_b = part<float>(workspace, l.sums_b);
    c.dg_tokens = part<float>(workspace, l.dg);
    c.share_buf = part<void>(workspace, l.share);
    if (num_seqs > kPlanSeqs && l.L < T_total) c.args.first = part<int32_t>(workspace, l.plan);
    return launched([&] { return kda::launch_linattn_bwd(c); });
}

}  // namespace

extern "C" {

size_t kda_linattn_fwd_workspace_size(kda_dtype dt, int H, int Hk, int dk, int dv, int num_seqs, int64_t T_total) {
    if (!sizes_ok(dt, H, Hk, dk, dv, num_seqs, T_total)) return 0;
    const size_t n = fwd_layout(H, dk, dv, num_seqs, T_total).total;
    return n ? n : 256;
}

kda_status kda_linattn_fwd(kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs, int64_t T_total,
                           const int32_t* cu_seqlens, const void* q, int64_t q_stride, const void* k,
                           int64_t k_stride, const void* v, int64_t v_stride, const float* g, int g_per_token,
                           const float* initial_state, float* final_state, void* y, void* workspace,
                           size_t workspace_bytes, void* stream) {
    return linattn_fwd(false, dt, H, Hk, dk, dv, scale, num_seqs, T_total, cu_seqlens, q, q_stride, k,
                       k_stride, v, v_stride, g, g_per_token, initial_state, final_state, y, workspace,
                       workspace_bytes, stream);
}

kda_status kda_linattn_fwd_padded(kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs,
                                  int64_t T_total, const int32_t* cu_seqlens, const void* q, int64_t q_stride,
                                  const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* g, int g_per_token,
                                  const float* initial_state, float* final_state, void* y, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    return linattn_fwd(true, dt, H, Hk, dk, dv, scale, num_seqs, T_total, cu_seqlens, q, q_stride, k,
                       k_stride, v, v_stride, g, g_per_token, initial_state, final_state, y, workspace,
                       workspace_bytes, stream);
}

size_t kda_linattn_bwd_workspace_size(kda_dtype dt, int H, int Hk, int dk, int dv, int num_seqs, int64_t T_total) {
    if (!sizes_ok(dt, H, Hk, dk, dv, num_seqs, T_total)) return 0;
    return bwd_layout(H, Hk, dk, dv, num_seqs, T_total).total;
}

kda_status kda_linattn_bwd(kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs, int64_t T_total,
                           const int32_t* cu_seqlens, const void* q, int64_t q_stride, const void* k,
                           int64_t k_stride, const void* v, int64_t v_stride, const float* g, int g_per_token,
                           const float* initial_state, const void* dy, const float* d_final_state, void* dq,
                           void* dk_out, void* dv_out, float* dg, float* d_initial_state, void* workspace,
                           size_t workspace_bytes, void* stream) {
    return linattn_bwd(false, dt, H, Hk, dk, dv, scale, num_seqs, T_total, cu_seqlens, q, q_stride, k,
                       k_stride, v, v_stride, g, g_per_token, initial_state, dy, d_final_state, dq, dk_out,
                       dv_out, dg, d_initial_state, workspace, workspace_bytes, stream);
}

kda_status kda_linattn_bwd_padded(kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs,
                                  int64_t T_total, const int32_t* cu_seqlens, const void* q, int64_t q_stride,
                                  const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* g, int g_per_token,
                                  const float* initial_state, const void* dy, const float* d_final_state, void* dq,
                                  void* dk_out, void* dv_out, float* dg, float* d_initial_state, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    return linattn_bwd(true, dt, H, Hk, dk, dv, scale, num_seqs, T_total, cu_seqlens, q, q_stride, k,
                       k_stride, v, v_stride, g, g_per_token, initial_state, dy, d_final_state, dq, dk_out,
                       dv_out, dg, d_initial_state, workspace, workspace_bytes, stream);
}

kda_status kda_linattn_decode_step(kda_dtype dt, int N, int H, int Hk, int dk, int dv, float scale, const void* q,
                                   int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                   int64_t v_stride, const float* g, int g_per_token, float* state, void* y,
                                   void* stream) {
    if (!dtype_ok(dt) || N < 0 || H <= 0 || Hk <= 0 || H % Hk != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (!head_ok(dk) || !head_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)N * H >= (int64_t)1 << 24) return KDA_ERR_INVALID_ARGUMENT;
    if (N > 0 && (!q || !k || !v || !g || !state || !y)) return KDA_ERR_INVALID_ARGUMENT;
    if (!rows_ok(dt, q, q_stride, Hk, dk) || !rows_ok(dt, k, k_stride, Hk, dk) || !rows_ok(dt, v, v_stride, H, dv) ||
        !aligned(y, 16) || !aligned(g, 4) || !aligned(state, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    kda::LinDecodeArgs a{};
    a.dtype = (int)dt;
    a.N = N;
    a.H = H;
    a.dk = dk;
    a.dv = dv;
    a.scale = scale;
    a.q = rows(q, q_stride, H / Hk);
    a.k = rows(k, k_stride, H / Hk);
    a.v = rows(v, v_stride, 1);
    a.g = g;
    a.g_per_token = g_per_token != 0;
    a.state = state;
    a.y = y;
    a.stream = stream;
    return launched([&] { return kda::launch_linattn_decode(a); });
}

kda_status kda_rope_frequencies(int rot, double base, kda_rope_scaling scaling, double factor, double trained_len,
                                double beta_fast, double beta_slow, double* inv_freq, float* mscale) {
    if (rot <= 0 || rot % 2 != 0 || !inv_freq || !mscale || !(base > 1.0) || !std::isfinite(base))
        return KDA_ERR_INVALID_ARGUMENT;
    if (scaling != KDA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return KDA_ERR_INVALID_ARGUMENT;
    if (scaling == KDA_ROPE_YARN && (!(trained_len > 0.0) || !(beta_fast > 0.0) || !(beta_slow > 0.0)))
        return KDA_ERR_INVALID_ARGUMENT;
    const int n = rot / 2;
    *mscale = 1.f;
    switch (scaling) {
        case KDA_ROPE_PLAIN:
            for (int i = 0; i < n; ++i) inv_freq[i] = std::pow(base, -2.0 * i / rot);
            return KDA_OK;
        case KDA_ROPE_LINEAR:
            for (int i = 0; i < n; ++i) inv_freq[i] = std::pow(base, -2.0 * i / rot) / factor;
            return KDA_OK;
        case KDA_ROPE_NTK: {
            if (rot <= 2) return KDA_ERR_INVALID_ARGUMENT;
            const double b = base * std::pow(factor, (double)rot / (rot - 2));
            for (int i = 0; i < n; ++i) inv_freq[i] = std::pow(b, -2.0 * i / rot);
            return KDA_OK;
        }
        case KDA_ROPE_YARN: {
            // pairs that turn more than beta_fast times over the trained length
            // keep their frequency, those below beta_slow turns are stretched,
            // a ramp between
            const double two_pi = 6.283185307179586476925;
            auto pair = [&](double turns) { return rot * std::log(trained_len / (turns * two_pi)) / (2 * std::log(base)); };
            const double lo = std::fmax(std::floor(pair(beta_fast)), 0.0);
            const double hi = std::fmin(std::ceil(pair(beta_slow)), rot - 1.0);
            const double width = std::fmax(hi - lo, 0.001);
            for (int i = 0; i < n; ++i) {
                const double f = std::pow(base, -2.0 * i / rot);
                const double r = std::fmin(std::fmax((i - lo) / width, 0.0), 1.0);
                inv_freq[i] = f / factor * r + f * (1.0 - r);
            }
            *mscale = (float)(0.1 * std::log(factor) + 1.0);
            return KDA_OK;
        }
    }
    return KDA_ERR_INVALID_ARGUMENT;
}

kda_status kda_rope_pair_axes(int axes, const int32_t* sections, kda_rope_order order, uint8_t* pair_axis) {
    if (axes <= 0 || axes > 255 || !sections || !pair_axis) return KDA_ERR_INVALID_ARGUMENT;
    if (order != KDA_ROPE_RUNS && order != KDA_ROPE_TURNS) return KDA_ERR_INVALID_ARGUMENT;
    int64_t pairs = 0;
    for (int x = 0; x < axes; ++x) {
        if (sections[x] < 0) return KDA_ERR_INVALID_ARGUMENT;
        pairs += sections[x];
    }
    if (pairs == 0 || pairs > 512) return KDA_ERR_INVALID_ARGUMENT;   // a head has 1024 channels at most
    // turn n takes a pair of every axis that has more than n; runs: an axis's all at once
    if (order == KDA_ROPE_RUNS) {
        for (int x = 0; x < axes; ++x)
            for (int n = 0; n < sections[x]; ++n) *pair_axis++ = (uint8_t)x;
    } else {
        for (int n = 0; n < 512; ++n)
            for (int x = 0; x < axes; ++x)
                if (sections[x] > n) *pair_axis++ = (uint8_t)x;
    }
    return KDA_OK;
}

kda_status kda_rope(kda_dtype dt, int64_t T, int Hq, int Hk, int d, int rot, kda_rope_layout layout, int inverse,
                    float mscale, const int32_t* positions, const double* inv_freq, const void* q, int64_t q_stride,
                    const void* k, int64_t k_stride, void* q_out, int64_t q_out_stride, void* k_out,
                    int64_t k_out_stride, void* stream) {
    return rope_call(dt, T, Hq, Hk, d, rot, layout, inverse, mscale, 1, positions, nullptr, inv_freq, q, q_stride, k,
                     k_stride, q_out, q_out_stride, k_out, k_out_stride, stream);
}

kda_status kda_rope_axes(kda_dtype dt, int64_t T, int Hq, int Hk, int d, int rot, kda_rope_layout layout, int inverse,
                         float mscale, int axes, const int32_t* positions, const uint8_t* pair_axis,
                         const double* inv_freq, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                         void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
    if (axes <= 0 || axes > 255 || (T > 0 && !pair_axis)) return KDA_ERR_INVALID_ARGUMENT;
    return rope_call(dt, T, Hq, Hk, d, rot, layout, inverse, mscale, axes, positions, pair_axis, inv_freq, q, q_stride, k,
                     k_stride, q_out, q_out_stride, k_out, k_out_stride, stream);
}

}  // extern "C"

namespace {

// Chunks of 64 tokens: (chunk, head) pairs as workgroups of 256 threads on an axis of
// less than 2^32 threads.  (The walks, of up to 512 threads and two a head of a sequence
// or more, fold their grid.)
constexpr int64_t kMaxChunks = int64_t(1) << 23;

bool gdr_sizes_ok(kda_dtype dt, int H, int Hk, int dk, int dv, int num_seqs, int64_t T) {
    return dtype_ok(dt) && H > 0 && Hk > 0 && H % Hk == 0 && num_seqs > 0 && T >= 0 && T <= INT32_MAX - 64 &&
           head_ok(dk) && head_ok(dv) && (T / 64 + num_seqs) * (int64_t)H < kMaxChunks;
}

// Tokens of a segment.  A walk takes about 4 us a chunk and a CU has one workgroup of
// it, so long sequences of few heads are cut: the segments' own effects side by side
// (value columns and the columns of their transitions, about what 256 CUs hold at
// once), a product of matrices a segment to join them (13 us with 128 channels, 8 with
// 64), then the walk over all segments at once.  As the joins are a chain too, a segment
// has sqrt(chunks / 2) chunks at least.  Times uncut and cut, d = 128, bf16 prompt, its gradient, and the
// same in fp32 (us):
//   8192 tokens x 12 heads        394  238   1051  706   1427 550   2803 1500
//   6000 + 15 x 146 tokens x 8    295  188    799  534   1051 398   2082 1069
//   2 x 4096 x 12                 211  198    623  624    737 510   1598 1421
//   3 x 2730 x 8 (3 segments)     148  150    447  474    500 358   1114 1031
//   4 x 2048 x 8 (2 segments)     116  136    345  409    378 344    863  923
//   6 x 1365 x 8 (2 segments)      89  138    314  412    276 348    734  909
// so a sequence of fewer than three segments stays whole; which ones these are the
// kernels see, the host knows the tokens of all alone.  What is cut nowhere
// pays for two launches that find nothing to do, and for finding so (16 x 512 x 8: 52 and
// 58, gradient 207 and 218; 128 x 64 x 12: 139 and 159, 412 and 458).  A few chunks
// gain nothing (1277 ragged tokens of 8 heads, fp32 gradient: 148 uncut, 164 in segments
// of 256).  The rule is of tokens and head sizes alone.
int64_t gdr_segment(int H, int dk, int dv, int num_seqs, int64_t T) {
    const int64_t all = T < 64 ? 64 : (T + 63) / 64 * 64, chunks = all / 64;
    int64_t m = (chunks * H * ((dk + dv) / 64) + 255) / 256;
    const int64_t least = (int64_t)std::ceil(std::sqrt(chunks / 2.0));
    if (m < least) m = least;
    if (m < 4) m = 4;
    return kda::kGdrLeastSegments * m > chunks || chunks < 32 || num_seqs > kPlanSeqs ? all : 64 * m;
}

struct GdrLayout {
    size_t x, p, z, tab, states, rstates, errors, u, share, plan, seg_m, seg_mt, seg_s, seg_r, total;
    int64_t chunks, L, segments;
};
GdrLayout gdr_layout(bool grad, int H, int Hk, int dk, int dv, int num_seqs, int64_t T) {
    GdrLayout l{};
    l.chunks = T > 64 ? T / 64 + num_seqs : num_seqs;
    l.L = gdr_segment(H, dk, dv, num_seqs, T);
    l.segments = l.L < T ? T / l.L + num_seqs : num_seqs;
    Parts p;
    if (T > 0) {
        const size_t n = (size_t)l.chunks * H;
        l.x = p.take(n * kda::kTriBytes);
        l.p = p.take(n * kda::kTriBytes);
        l.tab = p.take(n * kda::kGdrTab * 4);
        if (grad) {
            l.z = p.take(n * kda::kTriBytes);
            l.states = p.take(n * dk * dv * 4);
            l.rstates = p.take(n * dk * dv * 4);
            l.errors = p.take(n * 64 * dv * 4);
            l.u = p.take(n * 64 * dv * 4);
            l.share = p.take(Hk < H ? 2 * (size_t)T * H * dk * 4 : 0);
        }
        l.plan = p.take(T > 64 ? plan_bytes(num_seqs) : 0);
        if (l.L < T) {
            const size_t m = (size_t)l.segments * H;
            l.seg_m = p.take(m * dk * dk * 4);
            l.seg_mt = p.take(grad ? m * dk * dk * 4 : 0);
            l.seg_s = p.take(m * dk * dv * 4);
            l.seg_r = p.take(grad ? m * dk * dv * 4 : 0);
        }
    }
    l.total = p.at ? p.at : 256;
    return l;
}

// What both directions check and hand on.
kda_status gdr_args(bool grad, kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs, int64_t T_total,
                    const int32_t* cu_seqlens, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                    const void* v, int64_t v_stride, const float* g, const float* beta, const float* initial_state,
                    void* workspace, size_t workspace_bytes, void* stream, kda::GdrArgs& a) {
    if (!dtype_ok(dt)) return KDA_ERR_INVALID_ARGUMENT;
    if (!cu_seqlens && num_seqs != 1) return KDA_ERR_INVALID_ARGUMENT;
    if (H > 0 && Hk > 0 && (!head_ok(dk) || !head_ok(dv))) return KDA_ERR_UNSUPPORTED;
    if (!gdr_sizes_ok(dt, H, Hk, dk, dv, num_seqs, T_total)) return KDA_ERR_INVALID_ARGUMENT;
    if (T_total > 0 && (!q || !k || !v || !beta)) return KDA_ERR_INVALID_ARGUMENT;
    if (!rows_ok(dt, q, q_stride, Hk, dk) || !rows_ok(dt, k, k_stride, Hk, dk) || !rows_ok(dt, v, v_stride, H, dv) ||
        (int64_t)H * dv > kMaxStride || !aligned(g, 4) || !aligned(beta, 4) || !aligned(cu_seqlens, 4) ||
        !aligned(initial_state, 16) || !aligned(workspace, 256) || !workspace)
        return KDA_ERR_INVALID_ARGUMENT;
    const GdrLayout l = gdr_layout(grad, H, Hk, dk, dv, num_seqs, T_total);
    if (workspace_bytes < l.total) return KDA_ERR_WORKSPACE_TOO_SMALL;
    a.at.H = H;
    a.at.num_seqs = num_seqs;
    a.at.T_total = T_total;
    a.at.cu_seqlens = cu_seqlens;
    a.at.L = 64;
    a.at.nblocks = (int)l.chunks;
    a.at.stream = stream;
    if (num_seqs > kPlanSeqs && T_total > 64) a.at.first = part<int32_t>(workspace, l.plan);
    a.seg = a.at;
    a.seg.L = l.L;
    a.seg.nblocks = (int)l.segments;
    a.seg.first = nullptr;
    if (l.L < T_total) {
        // (more than two segments long: at most half as many again as fit)
        a.cuts = (int)(3 * T_total / (2 * l.L));
        a.seg_m = part<float>(workspace, l.seg_m);
        a.seg_s = part<float>(workspace, l.seg_s);
        if (grad) {
            a.seg_mt = part<float>(workspace, l.seg_mt);
            a.seg_r = part<float>(workspace, l.seg_r);
        }
    }
    a.q = rows(q, q_stride, H / Hk);
    a.k = rows(k, k_stride, H / Hk);
    a.v = rows(v, v_stride, 1);
    a.g = g;
    a.beta = beta;
    a.scale = scale;
    a.x = part<char>(workspace, l.x);
    a.p = part<char>(workspace, l.p);
    a.tab = part<float>(workspace, l.tab);
    a.initial = initial_state;
    if (grad) {
        a.z = part<char>(workspace, l.z);
        a.states = part<float>(workspace, l.states);
        a.rstates = part<float>(workspace, l.rstates);
        a.errors = part<float>(workspace, l.errors);
        a.u = part<float>(workspace, l.u);
        if (Hk < H) a.parts = part<float>(workspace, l.share);
    }
    a.dtype = (int)dt;
    a.head_k = dk;
    a.head_v = dv;
    return KDA_OK;
}

// clear: rows of no sequence of the outputs become zeros.
kda_status gdr_fwd(bool clear, kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs, int64_t T_total,
                   const int32_t* cu_seqlens, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                   const void* v, int64_t v_stride, const float* g, const float* beta, const float* initial_state,
                   float* final_state, void* y, void* workspace, size_t workspace_bytes, void* stream) {
    kda::GdrArgs a{};
    if ((T_total > 0 && !y) || !aligned(y, 16) || !aligned(final_state, 16)) return KDA_ERR_INVALID_ARGUMENT;
    const kda_status st = gdr_args(false, dt, H, Hk, dk, dv, scale, num_seqs, T_total, cu_seqlens, q, q_stride, k, k_stride,
                                   v, v_stride, g, beta, initial_state, workspace, workspace_bytes, stream, a);
    if (st != KDA_OK) return st;
    a.at.clear = clear;
    a.final = final_state;
    a.y = y;
    return launched([&] { return kda::launch_gdr_fwd(a); });
}

kda_status gdr_bwd(bool clear, kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs, int64_t T_total,
                   const int32_t* cu_seqlens, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                   const void* v, int64_t v_stride, const float* g, const float* beta, const float* initial_state,
                   const void* dy, const float* d_final_state, void* dq, void* dk_out, void* dv_out, float* dg,
                   float* dbeta, float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
    kda::GdrArgs a{};
    if (T_total > 0 && (!dy || !dq || !dk_out || !dv_out || !dbeta || (g != nullptr) != (dg != nullptr)))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!aligned(dy, 16) || !aligned(dq, 16) || !aligned(dk_out, 16) || !aligned(dv_out, 16) || !aligned(dg, 4) ||
        !aligned(dbeta, 4) || !aligned(d_final_state, 16) || !aligned(d_initial_state, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    const kda_status st = gdr_args(true, dt, H, Hk, dk, dv, scale, num_seqs, T_total, cu_seqlens, q, q_stride, k, k_stride,
                                   v, v_stride, g, beta, initial_state, workspace, workspace_bytes, stream, a);
    if (st != KDA_OK) return st;
    a.at.clear = clear;
    a.dy = dy;
    a.d_final = d_final_state;
    a.d_initial = d_initial_state;
    a.dq = dq;
    a.dk = dk_out;
    a.dv_out = dv_out;
    a.dg = dg;
    a.dbeta = dbeta;
    return launched([&] { return kda::launch_gdr_bwd(a); });
}

}  // namespace

extern "C" {

size_t kda_gdr_fwd_workspace_size(kda_dtype dt, int H, int Hk, int dk, int dv, int num_seqs, int64_t T_total) {
    return gdr_sizes_ok(dt, H, Hk, dk, dv, num_seqs, T_total) ? gdr_layout(false, H, Hk, dk, dv, num_seqs, T_total).total : 0;
}

size_t kda_gdr_bwd_workspace_size(kda_dtype dt, int H, int Hk, int dk, int dv, int num_seqs, int64_t T_total) {
    return gdr_sizes_ok(dt, H, Hk, dk, dv, num_seqs, T_total) ? gdr_layout(true, H, Hk, dk, dv, num_seqs, T_total).total : 0;
}

kda_status kda_gdr_fwd(kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs, int64_t T_total,
                       const int32_t* cu_seqlens, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, const float* g, const float* beta,
                       const float* initial_state, float* final_state, void* y, void* workspace,
                       size_t workspace_bytes, void* stream) {
    return gdr_fwd(false, dt, H, Hk, dk, dv, scale, num_seqs, T_total, cu_seqlens, q, q_stride, k, k_stride, v, v_stride, g,
                   beta, initial_state, final_state, y, workspace, workspace_bytes, stream);
}

kda_status kda_gdr_fwd_padded(kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs,
                              int64_t T_total, const int32_t* cu_seqlens, const void* q, int64_t q_stride,
                              const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* g,
                              const float* beta, const float* initial_state, float* final_state, void* y,
                              void* workspace, size_t workspace_bytes, void* stream) {
    return gdr_fwd(true, dt, H, Hk, dk, dv, scale, num_seqs, T_total, cu_seqlens, q, q_stride, k, k_stride, v, v_stride, g,
                   beta, initial_state, final_state, y, workspace, workspace_bytes, stream);
}

kda_status kda_gdr_bwd(kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs, int64_t T_total,
                       const int32_t* cu_seqlens, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, const float* g, const float* beta,
                       const float* initial_state, const void* dy, const float* d_final_state, void* dq, void* dk_out,
                       void* dv_out, float* dg, float* dbeta, float* d_initial_state, void* workspace,
                       size_t workspace_bytes, void* stream) {
    return gdr_bwd(false, dt, H, Hk, dk, dv, scale, num_seqs, T_total, cu_seqlens, q, q_stride, k, k_stride, v, v_stride, g,
                   beta, initial_state, dy, d_final_state, dq, dk_out, dv_out, dg, dbeta, d_initial_state, workspace,
                   workspace_bytes, stream);
}

kda_status kda_gdr_bwd_padded(kda_dtype dt, int H, int Hk, int dk, int dv, float scale, int num_seqs,
                              int64_t T_total, const int32_t* cu_seqlens, const void* q, int64_t q_stride,
                              const void* k, int64_t k_stride, const void* v, int64_t v_stride, const float* g,
                              const float* beta, const float* initial_state, const void* dy,
                              const float* d_final_state, void* dq, void* dk_out, void* dv_out, float* dg,
                              float* dbeta, float* d_initial_state, void* workspace, size_t workspace_bytes,
                              void* stream) {
    return gdr_bwd(true, dt, H, Hk, dk, dv, scale, num_seqs, T_total, cu_seqlens, q, q_stride, k, k_stride, v, v_stride, g,
                   beta, initial_state, dy, d_final_state, dq, dk_out, dv_out, dg, dbeta, d_initial_state, workspace,
                   workspace_bytes, stream);
}

kda_status kda_gdr_decode_step(kda_dtype dt, int N, int H, int Hk, int dk, int dv, float scale, const void* q,
                               int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               const float* g, const float* beta, float* state, void* y, void* stream) {
    if (!dtype_ok(dt) || N < 0 || H <= 0 || Hk <= 0 || H % Hk != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (!head_ok(dk) || !head_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)N * H >= (int64_t)1 << 24) return KDA_ERR_INVALID_ARGUMENT;
    if (N > 0 && (!q || !k || !v || !beta || !state || !y)) return KDA_ERR_INVALID_ARGUMENT;
    if (!rows_ok(dt, q, q_stride, Hk, dk) || !rows_ok(dt, k, k_stride, Hk, dk) || !rows_ok(dt, v, v_stride, H, dv) ||
        !aligned(y, 16) || !aligned(g, 4) || !aligned(beta, 4) || !aligned(state, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    kda::GdrDecodeArgs a{};
    a.dtype = (int)dt;
    a.N = N;
    a.H = H;
    a.dk = dk;
    a.dv = dv;
    a.scale = scale;
    a.q = rows(q, q_stride, H / Hk);
    a.k = rows(k, k_stride, H / Hk);
    a.v = rows(v, v_stride, 1);
    a.g = g;
    a.beta = beta;
    a.state = state;
    a.y = y;
    a.stream = stream;
    return launched([&] { return kda::launch_gdr_decode(a); });
}

}  // extern "C"

namespace {

// Rows walked side by side by the norm's gradient: a multiple of H, at most all
// rows, and about what fills the CUs with three workgroups each (two of 1024
// threads); each adds a partial row of the weight's gradient.  Rounded down:
// a few workgroups more than run at once take a second round (8192 x 96 rows of
// 128, bf16, gate: 235 us with 1026 workgroups, 202 with 768; 4096 x 32 rows
// 34.3 and 32.8).
int64_t norm_slots(kda_dtype dt, int64_t T, int H, int D) {
    const int vec = dt == KDA_BF16 ? 8 : 4, n = (D + vec - 1) / vec;
    const int64_t want = n <= 16 ? 768 * 16 : n <= 1024 / vec ? 768 * 4 : n <= 4096 / vec ? 768 : 512;
    int64_t p = want / H;
    if (p > T) p = T;
    return (p < 1 ? 1 : p) * (int64_t)H;
}

bool norm_sizes_ok(kda_dtype dt, int64_t T, int H, int D) {
    return dtype_ok(dt) && T >= 0 && H > 0 && D > 0 && T <= ((int64_t)1 << 31) / H - 1 && (int64_t)H * D <= 1 << 26;
}

bool kind_ok(kda_norm_kind kind) { return kind == KDA_NORM_LAYER || kind == KDA_NORM_RMS; }

// x and z in 8 bits: values and, for each 128 of a row, the power of two.
struct Kept {
    uint8_t *x8, *xe, *z8, *ze;
};

kda_status norm_fwd(kda_dtype dt, kda_norm_kind kind, int64_t T, int H, int D, float eps, const void* x,
                    const float* weight, const float* bias, const void* z, void* y, float* mean, float* rstd,
                    const Kept& kept, void* stream) {
    if (!norm_sizes_ok(dt, T, H, D) || !kind_ok(kind) || !(eps >= 0.f)) return KDA_ERR_INVALID_ARGUMENT;
    if (D > 16384) return KDA_ERR_UNSUPPORTED;
    if (!weight || (T > 0 && (!x || !y))) return KDA_ERR_INVALID_ARGUMENT;
    if (kind == KDA_NORM_RMS && mean) return KDA_ERR_INVALID_ARGUMENT;
    const size_t e = elt(dt);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(z, e) || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    kda::NormArgs a{};
    a.dtype = (int)dt;
    a.T = T;
    a.H = H;
    a.D = D;
    a.eps = eps;
    a.rms = kind == KDA_NORM_RMS;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.z = z;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.x8 = kept.x8;
    a.xe = kept.xe;
    a.z8 = kept.z8;
    a.ze = kept.ze;
    a.stream = stream;
    return launched([&] { return kda::launch_norm(a); });
}

kda_status norm_bwd(kda_dtype dt, kda_norm_kind kind, int64_t T, int H, int D, const void* x, const float* weight,
                    const float* bias, const void* z, const float* mean, const float* rstd, const void* dy,
                    void* dx, float* dweight, float* dbias, void* dz, void* workspace, size_t workspace_bytes,
                    const Kept& kept, void* stream) {
    if (!norm_sizes_ok(dt, T, H, D) || !kind_ok(kind)) return KDA_ERR_INVALID_ARGUMENT;
    if (D > 16384) return KDA_ERR_UNSUPPORTED;
    if (!weight || !dweight || !workspace) return KDA_ERR_INVALID_ARGUMENT;
    if (T > 0 && ((!x && !kept.x8) || !rstd || !dy || !dx || (kind == KDA_NORM_LAYER && !mean))) return KDA_ERR_INVALID_ARGUMENT;
    if (kind == KDA_NORM_RMS && mean) return KDA_ERR_INVALID_ARGUMENT;
    if ((z != nullptr || kept.z8 != nullptr) != (dz != nullptr) && T > 0) return KDA_ERR_INVALID_ARGUMENT;
    const size_t e = elt(dt);
    if (!aligned(x, e) || !aligned(dy, e) || !aligned(dx, e) || !aligned(z, e) || !aligned(dz, e) ||
        !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) ||
        !aligned(dbias, 4) || !aligned(workspace, 256))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t half = round_up((size_t)norm_slots(dt, T, H, D) * D * 4, 256);
    if (workspace_bytes < 2 * half) return KDA_ERR_WORKSPACE_TOO_SMALL;
    kda::NormArgs a{};
    a.dtype = (int)dt;
    a.T = T;
    a.H = H;
    a.D = D;
    a.rms = kind == KDA_NORM_RMS;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.z = z;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.dx = dx;
    a.dz = dz;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dwp = part<float>(workspace, 0);
    a.dbp = dbias ? part<float>(workspace, half) : nullptr;
    a.slots = norm_slots(dt, T, H, D);
    a.x8 = kept.x8;
    a.xe = kept.xe;
    a.z8 = kept.z8;
    a.ze = kept.ze;
    a.stream = stream;
    return launched([&] { return kda::launch_norm(a); });
}

}  // namespace

extern "C" {

kda_status kda_norm_fwd(kda_dtype dt, kda_norm_kind kind, int64_t T, int H, int D, float eps, const void* x,
                        const float* weight, const float* bias, const void* z, void* y, float* mean, float* rstd,
                        void* stream) {
    return norm_fwd(dt, kind, T, H, D, eps, x, weight, bias, z, y, mean, rstd, Kept{}, stream);
}

kda_status kda_norm_fwd_kept(kda_dtype dt, kda_norm_kind kind, int64_t T, int H, int D, float eps, const void* x,
                             const float* weight, const float* bias, const void* z, void* y, float* mean, float* rstd,
                             void* x8, uint8_t* x_exp, void* z8, uint8_t* z_exp, void* stream) {
    if (T > 0 && (!x8 || !x_exp || (z != nullptr) != (z8 != nullptr) || (z != nullptr) != (z_exp != nullptr)))
        return KDA_ERR_INVALID_ARGUMENT;
    return norm_fwd(dt, kind, T, H, D, eps, x, weight, bias, z, y, mean, rstd,
                    Kept{(uint8_t*)x8, x_exp, (uint8_t*)z8, z_exp}, stream);
}

size_t kda_norm_bwd_workspace_size(kda_dtype dt, int64_t T, int H, int D) {
    if (!norm_sizes_ok(dt, T, H, D) || D > 16384) return 0;
    return 2 * round_up((size_t)norm_slots(dt, T, H, D) * D * 4, 256);
}

kda_status kda_norm_bwd(kda_dtype dt, kda_norm_kind kind, int64_t T, int H, int D, const void* x, const float* weight,
                        const float* bias, const void* z, const float* mean, const float* rstd, const void* dy,
                        void* dx, float* dweight, float* dbias, void* dz, void* workspace, size_t workspace_bytes,
                        void* stream) {
    return norm_bwd(dt, kind, T, H, D, x, weight, bias, z, mean, rstd, dy, dx, dweight, dbias, dz, workspace,
                    workspace_bytes, Kept{}, stream);
}

kda_status kda_norm_bwd_kept(kda_dtype dt, kda_norm_kind kind, int64_t T, int H, int D, const void* x8,
                             const uint8_t* x_exp, const float* weight, const float* bias, const void* z8,
                             const uint8_t* z_exp, const float* mean, const float* rstd, const void* dy, void* dx,
                             float* dweight, float* dbias, void* dz, void* workspace, size_t workspace_bytes,
                             void* stream) {
    if (T > 0 && (!x8 || !x_exp || (z8 != nullptr) != (z_exp != nullptr))) return KDA_ERR_INVALID_ARGUMENT;
    return norm_bwd(dt, kind, T, H, D, nullptr, weight, bias, nullptr, mean, rstd, dy, dx, dweight, dbias, dz, workspace,
                    workspace_bytes,
                    Kept{(uint8_t*)x8, const_cast<uint8_t*>(x_exp), (uint8_t*)z8, const_cast<uint8_t*>(z_exp)}, stream);
}

}  // extern "C"
