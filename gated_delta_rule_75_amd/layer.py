"""The operators around the recurrence: linear attention with a decay for each
head (prompt, gradient, single token), rotary positions, and the norm of a
mixer's output with its gate.  The same kind of binding as the recurrence's:
checks on the host, outputs from torch, everything else in libkda.so.

Rows q, k, v of linear attention and of rotary positions may be slices of one
projection's output: [T, heads, d] views whose heads are contiguous within a
token (any stride from token to token).  A call runs on its tensors' device, on
that device's current stream.

Nothing here is recorded for autograd, also where an input requires a gradient:
a training step calls the gradients itself (linattn_bwd, norm_bwd, rope with
inverse), as from the two halves of a torch.autograd.Function.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import KDAError, _check, _dt, _need, _need_workspace, lib

_LAYOUT = {"half": 0, "interleaved": 1}
_SCALING = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
_KIND = {"layer": 0, "rms": 1}


def _p(t):
    return None if t is None else t.data_ptr()


def _device(*ts):
    """The device that every given tensor lives on."""
    dev = ts[0].device
    if dev.type != "cuda":
        raise ValueError("libkda tensors must live on the GPU")
    i = dev.index
    for t in ts:
        if t is not None and t.get_device() != i:
            raise ValueError("libkda tensors must share one device")
    return dev


def _contiguous(**ts):
    for name, t in ts.items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _buf(name: str, t, shape, dtype) -> None:
    """A contiguous tensor of this shape and dtype, or None."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape:
        _need(name, t, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _call(dev, fn, name: str, *args) -> None:
    """The C call on the device's current stream, with that device current (a HIP
    launch needs its stream's)."""
    i = dev.index
    stream = _raw_stream(i)
    if _current_device() == i:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(i):
            st = fn(*args, stream)
    if st != 0:
        raise KDAError(name, st)


def _raw_stream(i: int) -> int:
    return torch._C._cuda_getCurrentRawStream(i)


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _rows(name: str, t: torch.Tensor) -> int:
    """The token stride of [T, heads, d] rows whose heads are contiguous."""
    T, heads, d = t.shape
    if t.is_contiguous():
        return heads * d
    st = t.stride()
    if T == 0:
        return heads * d
    if (st[2] != 1 and d > 1) or (st[1] != d and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if T == 1:
        return heads * d
    if st[0] < heads * d:
        raise ValueError(f"{name}: tokens must not overlap")
    return st[0]


def _qkv(q, k, v, g) -> Tuple[int, int, int, int, int, int, int]:
    """(dtype, T, H, Hk, dk, dv, g per token) of q, k [T, Hk, dk], v [T, H, dv],
    g [T, H] or [H]."""
    dt = _dt(q)
    if q.dim() != 3 or v.dim() != 3 or k.shape != q.shape:
        raise ValueError("q, k must be [T, Hk, dk] and v [T, H, dv]")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError(f"k and v must have q's dtype {q.dtype}")
    T, Hk, dk = q.shape
    Tv, H, dv = v.shape
    if Tv != T or Hk == 0 or H % Hk != 0:
        raise ValueError("v must have q's tokens, and a multiple of its heads")
    if g.dtype != torch.float32:
        raise TypeError("g must be float32")
    if g.shape != (T, H) and g.shape != (H,):
        raise ValueError("g must be [T, H] or [H]")
    return dt, T, H, Hk, dk, dv, g.dim() - 1


def _seqs(cu_seqlens) -> int:
    if cu_seqlens is None:
        return 1
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be 1-D with at least two offsets")
    return cu_seqlens.numel() - 1


def _workspace(fn, need, workspace, dev):
    if need == 0:
        raise KDAError(fn + " workspace size query", 2)
    return torch.empty(need, dtype=torch.uint8, device=dev) if workspace is None else workspace


def linattn_fwd_workspace_size(dtype: int, H: int, Hk: int, dk: int, dv: int, num_seqs: int, T_total: int) -> int:
    """Bytes of workspace that linattn_fwd needs for these sizes (0: not supported)."""
    return int(lib().kda_linattn_fwd_workspace_size(dtype, H, Hk, dk, dv, num_seqs, T_total))


def linattn_bwd_workspace_size(dtype: int, H: int, Hk: int, dk: int, dv: int, num_seqs: int, T_total: int) -> int:
    """Bytes of workspace that linattn_bwd needs for these sizes (0: not supported)."""
    return int(lib().kda_linattn_bwd_workspace_size(dtype, H, Hk, dk, dv, num_seqs, T_total))


def linattn_fwd(q, k, v, g, cu_seqlens: Optional[torch.Tensor] = None, initial_state=None,
                output_final_state: bool = True, scale: float = 1.0, y: Optional[torch.Tensor] = None,
                final_state: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Linear attention with a decay for each head over packed sequences:
    S_t = exp(g_t) S_{t-1} + k_t v_t^T, y_t = scale S_t^T q_t.

    q, k [T, Hk, dk] and v [T, H, dv] (bf16 or fp32; H / Hk value heads share a
    key head), all finite; g fp32 [T, H] or, one decay for all tokens, [H], never
    above 0 (-inf starts the state anew, whatever it held).  cu_seqlens may begin
    after 0 or end before T: rows of no sequence are not read; they are zeros in a
    y made here, and left as they are in one that is given.  Returns (y,
    final_state or None)."""
    dt, T, H, Hk, dk, dv, per_token = _qkv(q, k, v, g)
    N = _seqs(cu_seqlens)
    _need("initial_state", initial_state, (N, H, dk, dv), torch.float32)
    _need("final_state", final_state, (N, H, dk, dv), torch.float32)
    _need("y", y, (T, H, dv), q.dtype)
    _need_workspace(workspace)
    qs, ks, vs = _rows("q", q), _rows("k", k), _rows("v", v)
    _contiguous(g=g, cu_seqlens=cu_seqlens, initial_state=initial_state, final_state=final_state, y=y,
                workspace=workspace)
    dev = _device(q, k, v, g, cu_seqlens, initial_state, final_state, y, workspace)
    L = lib()
    fn = L.kda_linattn_fwd
    if y is None:
        y = torch.empty(T, H, dv, dtype=q.dtype, device=dev)
        fn = L.kda_linattn_fwd_padded
    if final_state is None and output_final_state:
        final_state = torch.empty(N, H, dk, dv, dtype=torch.float32, device=dev)
    workspace = _workspace("kda_linattn_fwd", L.kda_linattn_fwd_workspace_size(dt, H, Hk, dk, dv, N, T), workspace,
                           dev)
    _call(dev, fn, "kda_linattn_fwd", dt, H, Hk, dk, dv, scale, N, T, _p(cu_seqlens), _p(q), qs,
          _p(k), ks, _p(v), vs, _p(g), per_token, _p(initial_state), _p(final_state), _p(y), _p(workspace),
          workspace.numel())
    return y, final_state


def linattn_bwd(q, k, v, g, dy, cu_seqlens: Optional[torch.Tensor] = None, initial_state=None, d_final_state=None,
                scale: float = 1.0, workspace: Optional[torch.Tensor] = None):
    """The gradient of linattn_fwd for the gradients dy [T, H, dv] of y and
    (optional) d_final_state of the final state.  Returns (dq, dk, dv, dg,
    d_initial_state): dq, dk [T, Hk, dk] summed over the value heads that share
    a key head, dg shaped like g (one decay for all tokens: summed over them);
    zeros in rows of no sequence."""
    dt, T, H, Hk, dk, dv, per_token = _qkv(q, k, v, g)
    N = _seqs(cu_seqlens)
    _need("dy", dy, (T, H, dv), q.dtype)
    _need("initial_state", initial_state, (N, H, dk, dv), torch.float32)
    _need("d_final_state", d_final_state, (N, H, dk, dv), torch.float32)
    _need_workspace(workspace)
    qs, ks, vs = _rows("q", q), _rows("k", k), _rows("v", v)
    _contiguous(g=g, dy=dy, cu_seqlens=cu_seqlens, initial_state=initial_state, d_final_state=d_final_state,
                workspace=workspace)
    dev = _device(q, k, v, g, dy, cu_seqlens, initial_state, d_final_state, workspace)
    L = lib()
    dq = torch.empty(T, Hk, dk, dtype=q.dtype, device=dev)
    dk_out = torch.empty_like(dq)
    dv_out = torch.empty(T, H, dv, dtype=q.dtype, device=dev)
    dg = torch.empty(g.shape, dtype=torch.float32, device=dev)
    ds0 = torch.empty(N, H, dk, dv, dtype=torch.float32, device=dev)
    workspace = _workspace("kda_linattn_bwd", L.kda_linattn_bwd_workspace_size(dt, H, Hk, dk, dv, N, T), workspace,
                           dev)
    _call(dev, L.kda_linattn_bwd_padded, "kda_linattn_bwd", dt, H, Hk, dk, dv, scale, N, T, _p(cu_seqlens), _p(q), qs,
          _p(k), ks, _p(v), vs, _p(g), per_token, _p(initial_state), _p(dy), _p(d_final_state), _p(dq),
          _p(dk_out), _p(dv_out), _p(dg), _p(ds0), _p(workspace), workspace.numel())
    return dq, dk_out, dv_out, dg, ds0


def linattn_decode_step(q, k, v, g, state, scale: float = 1.0, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for each of N requests: q, k [N, Hk, dk], v [N, H, dv], g [N, H]
    or [H] as in linattn_fwd, state fp32 [N, H, dk, dv] updated in place.  Returns y [N, H, dv]."""
    dt, N, H, Hk, dk, dv, per_token = _qkv(q, k, v, g)
    if state is None:
        raise ValueError("state is required")
    _buf("state", state, (N, H, dk, dv), torch.float32)
    _buf("y", y, (N, H, dv), q.dtype)
    _buf("g", g, g.shape, torch.float32)
    qs, ks, vs = _rows("q", q), _rows("k", k), _rows("v", v)
    dev = _device(q, k, v, g, state, y)
    if y is None:
        y = torch.empty(N, H, dv, dtype=q.dtype, device=dev)
    _call(dev, lib().kda_linattn_decode_step, "kda_linattn_decode_step", dt, N, H, Hk, dk, dv, scale, _p(q), qs,
          _p(k), ks, _p(v), vs, _p(g), per_token, _p(state), _p(y))
    return y


def rope_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     trained_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """The rot / 2 angles a position as a float64 CPU tensor, and the factor on
    cosines and sines, for scaling None, "linear", "ntk" or "yarn" by `factor`."""
    if scaling not in _SCALING:
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    freq = torch.empty(max(rot, 0) // 2, dtype=torch.float64)
    m = ctypes.c_float()
    st = lib().kda_rope_frequencies(rot, base, _SCALING[scaling], factor, float(trained_len), beta_fast, beta_slow,
                                    _p(freq), ctypes.byref(m))
    _check("kda_rope_frequencies", st)
    return freq, m.value


def rope(q, k, positions, inv_freq, layout: str = "half", inverse: bool = False, mscale: float = 1.0,
         q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Turns the first 2 * len(inv_freq) channels of every head of q [T, Hq, d]
    and k [T, Hk, d] (or None) by positions (int32 [T]) times inv_freq (float64,
    on the device); inverse turns back, which is the gradient.  layout "half"
    pairs channels (i, i + rot/2), "interleaved" (2i, 2i + 1).  Outputs may be
    the inputs.  Returns (q_out, k_out)."""
    dt = _dt(q)
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, d]")
    T, Hq, d = q.shape
    Hk = 0
    if k is not None:
        if k.dtype != q.dtype:
            raise TypeError(f"k must have q's dtype {q.dtype}")
        if k.dim() != 3 or k.shape[0] != T or k.shape[2] != d:
            raise ValueError("k must be [T, Hk, d] with q's T and d")
        Hk = k.shape[1]
    elif k_out is not None:
        raise ValueError("k_out given without k")
    if layout not in _LAYOUT:
        raise ValueError("layout must be 'half' or 'interleaved'")
    _buf("positions", positions, (T,), torch.int32)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be 1-D")
    _buf("inv_freq", inv_freq, inv_freq.shape, torch.float64)
    _need("q_out", q_out, q.shape, q.dtype)
    _need("k_out", k_out, None if k is None else k.shape, q.dtype)
    dev = _device(q, k, positions, inv_freq, q_out, k_out)
    if q_out is None:
        q_out = torch.empty(T, Hq, d, dtype=q.dtype, device=dev)
    if k is not None and k_out is None:
        k_out = torch.empty(T, Hk, d, dtype=q.dtype, device=dev)
    ks, kos = (_rows("k", k), _rows("k_out", k_out)) if k is not None else (0, 0)
    _call(dev, lib().kda_rope, "kda_rope", dt, T, Hq, Hk, d, 2 * inv_freq.shape[0], _LAYOUT[layout], int(inverse),
          mscale, _p(positions), _p(inv_freq), _p(q), _rows("q", q), _p(k), ks, _p(q_out), _rows("q_out", q_out),
          _p(k_out), kos)
    return q_out, k_out


def _norm_args(x, weight, bias, z, kind):
    dt = _dt(x)
    if kind not in _KIND:
        raise ValueError("kind must be 'layer' or 'rms'")
    if x.dim() != 3:
        raise ValueError("x must be [T, H, D]")
    T, H, D = x.shape
    if weight is None:
        raise ValueError("weight is required")
    _buf("weight", weight, (H, D), torch.float32)
    _buf("bias", bias, (H, D), torch.float32)
    _buf("z", z, x.shape, x.dtype)
    _buf("x", x, x.shape, x.dtype)
    return dt, T, H, D


def norm_fwd(x, weight, bias=None, z=None, eps: float = 1e-5, kind: str = "layer", stats: bool = True,
             y: Optional[torch.Tensor] = None):
    """Norm of each row of x [T, H, D] with weight (and bias) fp32 [H, D], times
    sigmoid(z) where z is given.  kind "layer" takes mean and variance, "rms"
    the mean square.  Returns (y, mean, rstd): fp32 [T, H], what norm_bwd needs
    (mean None for "rms", both None without stats)."""
    dt, T, H, D = _norm_args(x, weight, bias, z, kind)
    _buf("y", y, x.shape, x.dtype)
    dev = _device(x, weight, bias, z, y)
    if y is None:
        y = torch.empty_like(x)
    mean = rstd = None
    if stats:
        rstd = torch.empty(T, H, dtype=torch.float32, device=dev)
        if kind == "layer":
            mean = torch.empty_like(rstd)
    _call(dev, lib().kda_norm_fwd, "kda_norm_fwd", dt, _KIND[kind], T, H, D, eps, _p(x), _p(weight), _p(bias),
          _p(z), _p(y), _p(mean), _p(rstd))
    return y, mean, rstd


def norm_bwd_workspace_size(dtype: int, T: int, H: int, D: int) -> int:
    """Bytes of workspace that norm_bwd needs for these sizes (0: not supported)."""
    return int(lib().kda_norm_bwd_workspace_size(dtype, T, H, D))


def norm_bwd(dy, x, weight, mean, rstd, bias=None, z=None, kind: str = "layer",
             workspace: Optional[torch.Tensor] = None):
    """The gradient of norm_fwd with the mean and rstd it returned.  Returns
    (dx, dweight, dbias, dz); dbias and dz are None where bias and z are."""
    dt, T, H, D = _norm_args(x, weight, bias, z, kind)
    _buf("dy", dy, x.shape, x.dtype)
    if rstd is None or (mean is None) != (kind == "rms"):
        raise ValueError("rstd is required, and mean exactly for kind 'layer'")
    _buf("mean", mean, (T, H), torch.float32)
    _buf("rstd", rstd, (T, H), torch.float32)
    _need_workspace(workspace)
    _contiguous(workspace=workspace)
    dev = _device(x, dy, weight, mean, rstd, bias, z, workspace)
    L = lib()
    dx = torch.empty_like(x)
    dz = None if z is None else torch.empty_like(z)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    workspace = _workspace("kda_norm_bwd", L.kda_norm_bwd_workspace_size(dt, T, H, D), workspace, dev)
    _call(dev, L.kda_norm_bwd, "kda_norm_bwd", dt, _KIND[kind], T, H, D, _p(x), _p(weight), _p(bias), _p(z),
          _p(mean), _p(rstd), _p(dy), _p(dx), _p(dw), _p(db), _p(dz), _p(workspace), workspace.numel())
    return dx, dw, db, dz
