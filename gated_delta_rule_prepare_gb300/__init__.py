"""Python binding of libkda, the GB300 (sm_103a) KDA core library.

Argument marshalling only: every function here checks tensor dtypes, shapes
and devices, then calls the C ABI declared in ``include/kda.h`` with raw
device pointers and the current CUDA stream.  All arithmetic runs in the
library's CUDA kernels; there is no fallback.  Importing this package on a
machine without the built library raises immediately.

Entry points (same names as the C ABI): ``kda_decode``, ``kda_decode_k``,
``kda_prefill``, ``kda_prefill_gated``, ``kda_prefill_o_norm``, ``kda_conv_silu_l2``,
``kda_conv_silu_l2_k``,
``kda_gate``, ``kda_o_norm_gated``, ``kda_prefill_workspace_size``, ``kda_sync_status``.
Full attention: ``kda_attn_prefill`` over packed prompts, and the paged 4-bit cache's
``kda_attn_kv4_append``, ``kda_attn_kv4_read`` and ``kda_attn_kv4_decode`` (``kv4_cache``
allocates one).
Their rows' positions: ``kda_attn_rope``; the cache's pages: ``kda_attn_kv4_resize``,
``kda_attn_kv4_fork``, ``kda_attn_kv4_compact`` and ``kda_attn_kv4_copy``.
Linear attention with a decay for each head: ``kda_lin_prefill``, ``kda_lin_decode``.
``kda_prefill_static_ws`` is reached through ``LIB`` (its callers hold raw pointers).
"""

from __future__ import annotations

import ctypes
import importlib.util
import operator
import os

import torch

from . import build as _build

HEAD_DIM = 128
Q_SCALE = 0.08838834764831845
MAX_K = 8
F32, BF16, F16 = 0, 1, 2
KV4_TOKEN_BYTES = 144
KV4_PAGES = (16, 32, 64, 128, 256)
KV4_MAX_CACHES = 128

_c = ctypes
_vp, _i, _u64, _i64, _f, _sz = _c.c_void_p, _c.c_int, _c.c_uint64, _c.c_int64, _c.c_float, _c.c_size_t


class KdaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("kda status %d: %s" % (status, message))
        self.status = status


def _load():
    path = _build.LIB
    if not os.path.exists(path):
        raise ImportError("libkda.so is not built (%s); run __graft_entry__.build() first" % path)
    lib = _c.CDLL(path)
    sig = {
        "kda_decode": [_vp] * 7 + [_i] * 3 + [_u64],
        "kda_decode_k": [_vp] * 7 + [_i] * 4 + [_vp, _i, _u64],
        "kda_prefill": [_vp] * 7 + [_i, _i, _i, _f, _i, _i, _i, _i64, _vp, _i, _vp, _sz, _u64],
        "kda_conv_silu_l2": [_vp] * 4 + [_i, _i, _vp, _i, _f, _i, _i, _u64],
        "kda_sync_status": [_u64],
        "kda_o_norm_gated": [_vp] * 4 + [_i64, _i, _i, _f, _u64],
        "kda_gate": [_vp, _i64, _vp, _vp, _f, _vp, _i64, _vp, _vp, _i, _i64, _i, _i, _u64],
        "kda_prefill_gated": [_vp] * 5 + [_i64, _vp, _vp, _f, _vp, _i64, _vp, _i, _i, _i, _i,
                                          _i64, _vp, _i, _vp, _sz, _u64],
        "kda_conv_silu_l2_k": [_vp] * 4 + [_i, _i, _i, _f, _i, _i, _vp, _i, _u64],
        "kda_prefill_o_norm": [_vp] * 7 + [_i64, _vp, _f, _vp, _i64, _i, _i, _i, _i, _i, _i,
                                           _i64, _vp, _i, _vp, _sz, _u64],
    }
    sig.update({
        "kda_attn_prefill": [_vp] * 5 + [_i, _i, _vp, _vp] + [_i] * 5 + [_i64] * 4
                            + [_i, _f, _vp, _sz, _u64],
        "kda_attn_kv4_append": [_vp, _vp, _i64, _i64, _i, _vp, _i, _i, _i, _i, _vp, _i64, _i, _vp,
                                _i, _vp, _u64],
        "kda_attn_kv4_decode": [_vp, _vp, _i64, _i, _vp, _i, _vp, _vp, _vp] + [_i] * 7
                               + [_f, _vp, _sz, _u64],
    })
    sig["kda_attn_kv4_read"] = sig["kda_attn_kv4_append"]
    sig.update({
        "kda_lin_prefill": [_vp] * 7 + [_i, _i, _vp] + [_i] * 5 + [_i64] * 5 + [_f, _vp, _sz, _u64],
        "kda_lin_decode": [_vp] * 7 + [_i] * 6 + [_i64] * 5 + [_f, _vp, _i, _u64],
        "kda_attn_rope": [_vp] * 4 + [_i64] + [_i] * 4 + [_i64] * 4
                         + [_vp, _i, _vp, _i, _vp, _i, _f, _u64],
        "kda_attn_kv4_resize": [_vp] * 3 + [_i, _i, _i64, _i, _vp, _sz, _u64],
        "kda_attn_kv4_fork": [_vp] * 10 + [_i, _i, _i64, _i, _vp, _sz, _u64],
        "kda_attn_kv4_compact": [_vp] * 7 + [_i, _i, _i64, _vp, _sz, _u64],
        "kda_attn_kv4_copy": [_vp, _i, _i64, _i, _i, _vp, _vp, _vp, _i, _u64],
    })
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = _i
    lib.kda_prefill_workspace_size.argtypes = [_i64, _i, _i, _i, _i, _i]
    lib.kda_prefill_workspace_size.restype = _sz
    lib.kda_attn_prefill_workspace_size.argtypes = [_i64, _i, _i, _i]
    lib.kda_attn_prefill_workspace_size.restype = _sz
    lib.kda_attn_kv4_workspace_size.argtypes = [_i] * 4
    lib.kda_attn_kv4_workspace_size.restype = _sz
    lib.kda_lin_prefill_workspace_size.argtypes = [_i64, _i, _i]
    lib.kda_lin_prefill_workspace_size.restype = _sz
    lib.kda_attn_kv4_pages_workspace_size.argtypes = [_i64, _i, _i]
    lib.kda_attn_kv4_pages_workspace_size.restype = _sz
    lib.kda_last_error.argtypes = []
    lib.kda_last_error.restype = _c.c_char_p
    lib.kda_version.argtypes = []
    lib.kda_version.restype = _c.c_char_p
    return lib


LIB = _load()


def _check(status: int):
    if status != 0:
        raise KdaError(status, LIB.kda_last_error().decode())


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t.data_ptr()


def _contig(t, name):
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def version() -> str:
    return LIB.kda_version().decode()


def kda_decode(state, q, k, v, g, beta, o):
    """One token per sequence: state [N,H,128,128] FP32 in place; q, k, v, g, o
    [N,H,128] FP32; beta [N,H] FP32."""
    N, H = state.shape[0], state.shape[1]
    for n_, t in (("state", state), ("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta),
                  ("o", o)):
        _contig(t, n_)
    if q.shape != (N, H, HEAD_DIM) or beta.shape != (N, H):
        raise ValueError("kda_decode: shape mismatch")
    f = torch.float32
    _check(LIB.kda_decode(_ptr(state, f, "state"), _ptr(q, f, "q"), _ptr(k, f, "k"),
                          _ptr(v, f, "v"), _ptr(g, f, "g"), _ptr(beta, f, "beta"),
                          _ptr(o, f, "o"), N, H, state.shape[-1], _stream(state)))


def kda_decode_k(state, q, k, v, g, beta, o, snapshots=()):
    """k rows per sequence walked in order: q, k, v, g, o [N,k,H,128]; beta
    [N,k,H]; snapshots: up to k tensors [N,H,128,128], snapshots[t] = state
    after row t."""
    N, krows, H = q.shape[0], q.shape[1], q.shape[2]
    for n_, t in (("state", state), ("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta),
                  ("o", o)):
        _contig(t, n_)
    if beta.shape != (N, krows, H) or state.shape[:2] != (N, H):
        raise ValueError("kda_decode_k: shape mismatch")
    f = torch.float32
    snaps = list(snapshots)
    for s in snaps:
        _contig(s, "snapshot")
        if s.shape != state.shape or s.dtype != f:
            raise ValueError("kda_decode_k: snapshot shape/dtype mismatch")
    arr = (_c.c_void_p * max(1, len(snaps)))(*[s.data_ptr() for s in snaps])
    _check(LIB.kda_decode_k(_ptr(state, f, "state"), _ptr(q, f, "q"), _ptr(k, f, "k"),
                            _ptr(v, f, "v"), _ptr(g, f, "g"), _ptr(beta, f, "beta"),
                            _ptr(o, f, "o"), N, krows, H, state.shape[-1],
                            _c.cast(arr, _c.c_void_p) if snaps else None, len(snaps),
                            _stream(state)))


def kda_prefill_workspace_size(rows, n_seqs, chunk, heads, dtype=torch.bfloat16):
    """Workspace bytes kda_prefill needs for `rows` token rows in total."""
    in_dtype = BF16 if dtype == torch.bfloat16 else F32
    return int(LIB.kda_prefill_workspace_size(int(rows), n_seqs, chunk, heads, HEAD_DIM, in_dtype))


def kda_prefill(state, q, k, v, g, beta, o, t, chunk, pad_fill=0.0, cu_seqlens=None,
                workspace=None):
    """Chunked prefill.  Without cu_seqlens: q, k, v, g [N, T_pad, H, 128]
    (or [T_pad, H, 128] for one sequence), beta [N, T_pad, H], t valid tokens
    per sequence; rows [t, T_pad) are the caller's padded tail (pad_fill),
    neither read into arithmetic nor written.  With
    cu_seqlens (device int32 [N+1]): packed rows [T, H, 128] and t = T.
    q, k and v may be strided views whose token rows are ``q.stride(-3)``
    elements apart (e.g. slices of one [T, 3*H*128] buffer)."""
    dt = q.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError("kda_prefill: inputs must be float32 or bfloat16")
    in_dtype = BF16 if dt == torch.bfloat16 else F32
    H = q.shape[-2]
    if q.shape[-1] != HEAD_DIM:
        raise ValueError("kda_prefill: head_dim must be 128")
    for n_, t_ in (("q", q), ("k", k), ("v", v)):
        if t_.dtype != dt or t_.stride(-1) != 1 or t_.stride(-2) != HEAD_DIM:
            raise ValueError("kda_prefill: %s must have unit channel stride and heads packed" % n_)
    stride = q.stride(-3)
    if k.stride(-3) != stride or v.stride(-3) != stride:
        raise ValueError("kda_prefill: q, k, v must share one token-row stride")
    for n_, t_ in (("g", g), ("beta", beta), ("o", o), ("state", state)):
        _contig(t_, n_)
    if g.dtype != dt or beta.dtype != dt:
        raise TypeError("kda_prefill: g and beta must have the inputs' dtype")
    if cu_seqlens is not None:
        n_seqs = cu_seqlens.numel() - 1
        t_pad = t
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
            raise TypeError("kda_prefill: cu_seqlens must be a CUDA int32 tensor")
        rows = q.shape[0]
    else:
        if q.dim() == 3:
            n_seqs, t_pad = 1, q.shape[0]
        else:
            n_seqs, t_pad = q.shape[0], q.shape[1]
            if q.dim() == 4 and q.stride(0) != t_pad * stride:
                raise ValueError("kda_prefill: sequences must be consecutive row blocks")
        rows = n_seqs * t_pad
    if g.numel() != rows * H * HEAD_DIM or beta.numel() != rows * H or o.numel() != rows * H * HEAD_DIM:
        raise ValueError("kda_prefill: g/beta/o sizes do not match the token rows")
    if state.numel() != n_seqs * H * HEAD_DIM * HEAD_DIM or state.dtype != torch.float32:
        raise ValueError("kda_prefill: state must be FP32 [N, H, 128, 128]")
    ws_need = kda_prefill_workspace_size(rows, n_seqs, chunk, H, dt)
    if ws_need and workspace is None:
        # The caller gave none: allocate one here, outside the library (which
        # never allocates).  Timed callers pass a preallocated buffer.
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(LIB.kda_prefill(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                           _ptr(o, torch.float32, "o"), int(t), int(t_pad), int(chunk),
                           float(pad_fill), H, HEAD_DIM, in_dtype, int(stride),
                           _ptr(cu_seqlens), n_seqs, ws_ptr, ws_bytes, _stream(state)))


def _row_view(x, rows, hd, name):
    """(pointer, token-row stride) of a BF16 [rows, >= hd] view with unit
    channel stride, or of any contiguous tensor of rows x hd values."""
    if x.dtype != torch.bfloat16 or not x.is_cuda:
        raise TypeError("%s must be a CUDA bfloat16 tensor" % name)
    if x.is_contiguous() and x.numel() == rows * hd:
        return x.data_ptr(), hd
    if x.dim() == 2 and x.shape[0] == rows and x.shape[1] >= hd and x.stride(1) == 1:
        return x.data_ptr(), x.stride(0)
    raise ValueError("%s must hold rows x heads*128 values (contiguous, or a 2-D row view)" % name)


def kda_prefill_o_norm(state, q, k, v, g, beta, gate, w, out, t, chunk=64, eps=1e-6,
                       cu_seqlens=None, workspace=None):
    """kda_prefill with the sigmoid-gated RMSNorm fused into its epilogue (BF16
    inputs, tensor-core path): writes out BF16 [rows, H*128] =
    rmsnorm(o) * w * sigmoid(gate) instead of the FP32 core output o.  gate
    and out: BF16 with rows x H*128 values (contiguous, or 2-D row views);
    w: BF16 [128].  The other arguments are kda_prefill's."""
    if q.dtype != torch.bfloat16:
        raise TypeError("kda_prefill_o_norm: inputs must be bfloat16")
    H = q.shape[-2]
    if q.shape[-1] != HEAD_DIM:
        raise ValueError("kda_prefill_o_norm: head_dim must be 128")
    for n_, t_ in (("q", q), ("k", k), ("v", v)):
        if t_.dtype != q.dtype or t_.stride(-1) != 1 or t_.stride(-2) != HEAD_DIM:
            raise ValueError("kda_prefill_o_norm: %s must have unit channel stride and heads "
                             "packed" % n_)
    stride = q.stride(-3)
    if k.stride(-3) != stride or v.stride(-3) != stride:
        raise ValueError("kda_prefill_o_norm: q, k, v must share one token-row stride")
    for n_, t_ in (("g", g), ("beta", beta), ("state", state), ("w", w)):
        _contig(t_, n_)
    if g.dtype != q.dtype or beta.dtype != q.dtype:
        raise TypeError("kda_prefill_o_norm: g and beta must have the inputs' dtype")
    if cu_seqlens is not None:
        n_seqs = cu_seqlens.numel() - 1
        t_pad = t
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
            raise TypeError("kda_prefill_o_norm: cu_seqlens must be a CUDA int32 tensor")
    else:
        if q.dim() == 3:
            n_seqs, t_pad = 1, q.shape[0]
        else:
            n_seqs, t_pad = q.shape[0], q.shape[1]
            if q.dim() == 4 and q.stride(0) != t_pad * stride:
                raise ValueError("kda_prefill_o_norm: sequences must be consecutive row blocks")
    rows = t if cu_seqlens is not None else n_seqs * t_pad
    if g.numel() != rows * H * HEAD_DIM or beta.numel() != rows * H:
        raise ValueError("kda_prefill_o_norm: g/beta sizes do not match the token rows")
    if state.numel() != n_seqs * H * HEAD_DIM * HEAD_DIM or state.dtype != torch.float32:
        raise ValueError("kda_prefill_o_norm: state must be FP32 [N, H, 128, 128]")
    if w.numel() != HEAD_DIM or w.dtype != torch.bfloat16:
        raise ValueError("kda_prefill_o_norm: w must be BF16 [128]")
    g_ptr, g_stride = _row_view(gate, rows, H * HEAD_DIM, "gate")
    o_ptr, o_stride = _row_view(out, rows, H * HEAD_DIM, "out")
    ws_need = kda_prefill_workspace_size(rows, n_seqs, chunk, H, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(ws_need, 1), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(LIB.kda_prefill_o_norm(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  g_ptr, int(g_stride), _ptr(w), float(eps), o_ptr,
                                  int(o_stride), int(t), int(t_pad), int(chunk), H, HEAD_DIM,
                                  BF16, int(stride), _ptr(cu_seqlens), n_seqs,
                                  workspace.data_ptr(), ws_bytes, _stream(state)))


def kda_prefill_gated(state, q, k, v, g_raw, dt_bias, a_log, b_raw, o, t, gate_lower_bound,
                      cu_seqlens=None, workspace=None):
    """Tensor-core prefill (BF16 q, k, v; chunk 64) with the forget gate and
    beta formed in the prepare kernel from g_raw BF16 [rows, >= H*128],
    dt_bias FP32 [H*128], a_log FP32 [H] and b_raw BF16 [rows, >= H].
    Without cu_seqlens: q, k, v [N, T_pad, H, 128] (or [T_pad, H, 128]), t
    valid tokens per sequence, rows [t, T_pad) left as they are and never
    used.  With cu_seqlens (device int32 [N+1]): packed rows and t = T."""
    b16 = torch.bfloat16
    H = q.shape[-2]
    if q.shape[-1] != HEAD_DIM:
        raise ValueError("kda_prefill_gated: head_dim must be 128")
    for n_, t_ in (("q", q), ("k", k), ("v", v)):
        if t_.dtype != b16 or t_.stride(-1) != 1 or t_.stride(-2) != HEAD_DIM:
            raise ValueError("kda_prefill_gated: %s must be bfloat16 with unit channel stride "
                             "and heads packed" % n_)
    stride = q.stride(-3)
    if k.stride(-3) != stride or v.stride(-3) != stride:
        raise ValueError("kda_prefill_gated: q, k, v must share one token-row stride")
    for n_, t_ in (("dt_bias", dt_bias), ("a_log", a_log), ("o", o), ("state", state)):
        _contig(t_, n_)
    if g_raw.dim() != 2 or g_raw.stride(1) != 1 or b_raw.dim() != 2 or b_raw.stride(1) != 1:
        raise ValueError("kda_prefill_gated: g_raw and b_raw must be 2-D with unit channel stride")
    if cu_seqlens is not None:
        n_seqs = cu_seqlens.numel() - 1
        t_pad = t
        if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
            raise TypeError("kda_prefill_gated: cu_seqlens must be a CUDA int32 tensor")
    elif q.dim() == 3:
        n_seqs, t_pad = 1, q.shape[0]
    else:
        n_seqs, t_pad = q.shape[0], q.shape[1]
        if q.stride(0) != t_pad * stride:
            raise ValueError("kda_prefill_gated: sequences must be consecutive row blocks")
    rows = t if cu_seqlens is not None else n_seqs * t_pad
    if (g_raw.shape[0] != rows or b_raw.shape[0] != rows or g_raw.shape[1] < H * HEAD_DIM
            or b_raw.shape[1] < H or dt_bias.numel() != H * HEAD_DIM or a_log.numel() != H
            or o.numel() != rows * H * HEAD_DIM):
        raise ValueError("kda_prefill_gated: shape mismatch")
    if state.numel() != n_seqs * H * HEAD_DIM * HEAD_DIM or state.dtype != torch.float32:
        raise ValueError("kda_prefill_gated: state must be FP32 [N, H, 128, 128]")
    if workspace is None:
        need = kda_prefill_workspace_size(rows, n_seqs, 64, H, b16)
        if need == 0:  # KDA_PREFILL_IMPL=simt makes the size query answer for the SIMT kernel
            raise KdaError(3, "kda_prefill_gated runs only on the tensor-core "
                           "kernels: unset KDA_PREFILL_IMPL=simt or pass a workspace")
        # allocated here, outside the library (which never allocates)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(LIB.kda_prefill_gated(
        _ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(g_raw, b16, "g_raw"), int(g_raw.stride(0)),
        _ptr(dt_bias, torch.float32, "dt_bias"), _ptr(a_log, torch.float32, "a_log"),
        float(gate_lower_bound), _ptr(b_raw, b16, "b_raw"), int(b_raw.stride(0)),
        _ptr(o, torch.float32, "o"), int(t), int(t_pad), H, HEAD_DIM, int(stride),
        _ptr(cu_seqlens), n_seqs, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(state)))


def kda_conv_silu_l2(conv_state, x, w, out, cu_seqlens=None, n_seqs=None, l2_eps=1e-6):
    """Depthwise causal conv + SiLU + L2(q, k).  x, out BF16 [tokens, 3*H*128];
    w BF16 [3*H*128, K]; conv_state FP32 [N, 3*H*128, K] in place.  Without
    cu_seqlens x holds N sequences of tokens/N tokens each."""
    for n_, t_ in (("conv_state", conv_state), ("x", x), ("w", w), ("out", out)):
        _contig(t_, n_)
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
        raise TypeError("kda_conv_silu_l2: x, w, out must be bfloat16")
    conv_dim = x.shape[-1]
    if conv_dim % (3 * HEAD_DIM):
        raise ValueError("kda_conv_silu_l2: channels must be 3 * heads * 128")
    H = conv_dim // (3 * HEAD_DIM)
    K = w.shape[1]
    tokens = x.numel() // conv_dim
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        t = tokens
    else:
        N = conv_state.shape[0] if n_seqs is None else n_seqs
        if tokens % N:
            raise ValueError("kda_conv_silu_l2: tokens not divisible by n_seqs")
        t = tokens // N
    if conv_state.shape != (N, conv_dim, K):
        raise ValueError("kda_conv_silu_l2: conv_state must be [N, conv_dim, K]")
    _check(LIB.kda_conv_silu_l2(_ptr(conv_state, torch.float32, "conv_state"), _ptr(x), _ptr(w),
                                _ptr(out), t, N, _ptr(cu_seqlens), K, float(l2_eps), H,
                                HEAD_DIM, _stream(x)))


def kda_conv_silu_l2_k(conv_state, x, w, out, snapshots=(), l2_eps=1e-6):
    """k rows per sequence through the conv front end: x, out BF16 [N, k,
    3*H*128]; conv_state FP32 [N, 3*H*128, K] in place; snapshots: up to k
    FP32 tensors shaped like conv_state, snapshots[t] = conv state after row t."""
    for n_, t_ in (("conv_state", conv_state), ("x", x), ("w", w), ("out", out)):
        _contig(t_, n_)
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16 or out.dtype != torch.bfloat16:
        raise TypeError("kda_conv_silu_l2_k: x, w, out must be bfloat16")
    N, krows, conv_dim = x.shape
    if conv_dim % (3 * HEAD_DIM) or conv_state.shape != (N, conv_dim, w.shape[1]):
        raise ValueError("kda_conv_silu_l2_k: shape mismatch")
    snaps = list(snapshots)
    for s_ in snaps:
        _contig(s_, "snapshot")
        if s_.shape != conv_state.shape or s_.dtype != torch.float32:
            raise ValueError("kda_conv_silu_l2_k: snapshot shape/dtype mismatch")
    arr = (_c.c_void_p * max(1, len(snaps)))(*[s_.data_ptr() for s_ in snaps])
    _check(LIB.kda_conv_silu_l2_k(_ptr(conv_state, torch.float32, "conv_state"), _ptr(x),
                                  _ptr(w), _ptr(out), N, krows, w.shape[1], float(l2_eps),
                                  conv_dim // (3 * HEAD_DIM), HEAD_DIM,
                                  _c.cast(arr, _c.c_void_p) if snaps else None, len(snaps),
                                  _stream(x)))


def kda_o_norm_gated(core, gate, w, out, eps=1e-6):
    """Sigmoid-gated RMSNorm: core FP32 [rows, H, 128] (or [rows, H*128]),
    gate and out BF16 [rows, H*128], w BF16 [128]."""
    for n_, t_ in (("core", core), ("gate", gate), ("w", w), ("out", out)):
        _contig(t_, n_)
    rows = core.shape[0]
    hd = core.numel() // max(rows, 1) if rows else gate.shape[-1]
    if hd % HEAD_DIM or gate.numel() != core.numel() or out.numel() != core.numel():
        raise ValueError("kda_o_norm_gated: core, gate and out must hold rows x H x 128 values")
    if w.numel() != HEAD_DIM:
        raise ValueError("kda_o_norm_gated: w must hold 128 values")
    b16 = torch.bfloat16
    _check(LIB.kda_o_norm_gated(_ptr(core, torch.float32, "core"), _ptr(gate, b16, "gate"),
                                _ptr(w, b16, "w"), _ptr(out, b16, "out"), int(rows),
                                hd // HEAD_DIM, HEAD_DIM, float(eps), _stream(core)))


def kda_gate(g_raw, dt_bias, a_log, b_raw, g_out, beta_out, gate_lower_bound):
    """Forget gate and beta: g_raw BF16 [rows, >= H*128] (row pitch a multiple
    of 8 channels), dt_bias FP32 [H*128], a_log FP32 [H], b_raw BF16
    [rows, >= H]; g_out [rows, H, 128] and beta_out [rows, H] in FP32 or BF16
    (both the same dtype)."""
    for n_, t_ in (("dt_bias", dt_bias), ("a_log", a_log), ("g_out", g_out),
                   ("beta_out", beta_out)):
        _contig(t_, n_)
    if g_raw.dim() != 2 or g_raw.stride(1) != 1 or b_raw.dim() != 2 or b_raw.stride(1) != 1:
        raise ValueError("kda_gate: g_raw and b_raw must be 2-D with unit channel stride")
    rows, H = g_out.shape[0], a_log.numel()
    if (g_out.numel() != rows * H * HEAD_DIM or beta_out.numel() != rows * H
            or dt_bias.numel() != H * HEAD_DIM or g_raw.shape[0] != rows
            or b_raw.shape[0] != rows or g_raw.shape[1] < H * HEAD_DIM or b_raw.shape[1] < H):
        raise ValueError("kda_gate: shape mismatch")
    if g_out.dtype != beta_out.dtype or g_out.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("kda_gate: g_out and beta_out must both be FP32 or both BF16")
    b16 = torch.bfloat16
    _check(LIB.kda_gate(_ptr(g_raw, b16, "g_raw"), int(g_raw.stride(0)),
                        _ptr(dt_bias, torch.float32, "dt_bias"), _ptr(a_log, torch.float32, "a_log"),
                        float(gate_lower_bound), _ptr(b_raw, b16, "b_raw"), int(b_raw.stride(0)),
                        _ptr(g_out), _ptr(beta_out), BF16 if g_out.dtype == b16 else F32,
                        int(rows), H, HEAD_DIM, _stream(g_out)))


# ---------------------------------------------------------------- full attention

# These calls are short, and a decode step makes them once a layer: arguments are
# checked with few attribute reads, and a tensor's device by its index (-1: none).

_ATTN_TYPES = {torch.bfloat16: BF16, torch.float16: F16}
_raw_stream = torch._C._cuda_getCurrentRawStream


def _attn_type(t, name):
    dt = _ATTN_TYPES.get(t.dtype)
    if dt is None:
        raise TypeError("%s must be bfloat16 or float16" % name)
    dev = t.get_device()
    if dev < 0:
        raise TypeError("%s must be a CUDA tensor" % name)
    return dt, dev


def _at(t, dtype, dev, name):
    """Pointer of a tensor of the given type on device `dev`."""
    if t.dtype != dtype or t.get_device() != dev:
        raise TypeError("%s must be a %s tensor on the call's CUDA device" % (name, dtype))
    return t.data_ptr()


def _packed(t, dtype, dev, name):
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return _at(t, dtype, dev, name)


def _rows(t, dtype, dev, name):
    """(pointer, token-row stride) of a [..., rows, heads, 128] tensor with its
    heads packed; a leading sequence dimension must be consecutive row blocks."""
    ptr, shape = _at(t, dtype, dev, name), t.shape
    if len(shape) not in (3, 4) or shape[-1] != HEAD_DIM:
        raise ValueError("%s must be [rows, heads, 128]" % name)
    if t.is_contiguous():
        return ptr, shape[-2] * HEAD_DIM
    stride = t.stride()
    if stride[-1] != 1 or (stride[-2] != HEAD_DIM and shape[-2] > 1):
        raise ValueError("%s must have unit channel stride and heads packed" % name)
    row = stride[-3] if shape[-3] > 1 else shape[-2] * HEAD_DIM
    if len(shape) == 4 and shape[0] > 1:
        if shape[1] == 1:
            row = stride[0]
        elif stride[0] != shape[1] * row:
            raise ValueError("%s: sequences must be consecutive row blocks" % name)
    return ptr, row


def _window(window):
    """In the C type's range: no position passes its end, and below 0 the call refuses."""
    return window if 0 <= window <= 0x7fffffff else -1 if window < 0 else 0x7fffffff


def _scratch(workspace, need, dev):
    """(tensor, pointer, bytes) of the caller's workspace, or of one allocated
    here (the library itself never allocates)."""
    if workspace is None:
        workspace = torch.empty(need(), dtype=torch.uint8, device="cuda:%d" % dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on the call's device")
    return workspace, workspace.data_ptr(), workspace.nbytes


def kda_attn_prefill_workspace(rows, n_seqs, heads, kv_heads, device="cuda"):
    """Workspace for kda_attn_prefill over `rows` query rows in total."""
    need = LIB.kda_attn_prefill_workspace_size(int(rows), n_seqs, heads, kv_heads)
    return torch.empty(int(need), dtype=torch.uint8, device=device)


def kda_attn_prefill(q, k, v, out, lse=None, cu_seqlens=None, cu_seqlens_k=None, window=0,
                     scale=Q_SCALE, workspace=None):
    """Causal attention with grouped heads.  BF16 or FP16 q, out
    [rows, heads, 128] and k, v [key rows, kv_heads, 128], which may be strided
    views of wider rows; lse FP32 [rows, heads] or None.  cu_seqlens and
    cu_seqlens_k (device int32 [N+1]; the keys' default to the queries') give
    packed sequences; without them, tensors of four dimensions
    [N, T, heads, 128] hold N sequences and of three one.  A sequence's queries
    are its last positions; window > 0 limits each to the last `window` keys."""
    in_dtype, dev = _attn_type(q, "q")
    dt, q_shape, k_shape = q.dtype, q.shape, k.shape
    q_ptr, q_row = _rows(q, dt, dev, "q")
    k_ptr, k_row = _rows(k, dt, dev, "k")
    v_ptr, v_row = _rows(v, dt, dev, "v")
    o_ptr, o_row = _rows(out, dt, dev, "out")
    heads, kv_heads = q_shape[-2], k_shape[-2]
    if out.shape != q_shape or v.shape != k_shape or len(q_shape) != len(k_shape):
        raise ValueError("kda_attn_prefill: out must have q's shape, v k's, and k q's dimensions")
    cu_q = cu_k = None
    t_q, t_k, n_seqs = q_shape[-3], k_shape[-3], 1
    if cu_seqlens is not None:
        if len(q_shape) != 3:
            raise ValueError("kda_attn_prefill: packed rows have three dimensions")
        n_seqs = cu_seqlens.numel() - 1
        cu_q = cu_k = _packed(cu_seqlens, torch.int32, dev, "cu_seqlens")
        if cu_seqlens_k is not None:
            cu_k = _packed(cu_seqlens_k, torch.int32, dev, "cu_seqlens_k")
            if cu_seqlens_k.numel() != n_seqs + 1:
                raise ValueError("kda_attn_prefill: cu_seqlens_k must be as long as cu_seqlens")
    elif cu_seqlens_k is not None:
        raise ValueError("kda_attn_prefill: cu_seqlens_k needs cu_seqlens")
    elif len(q_shape) == 4:
        n_seqs = q_shape[0]
        if k_shape[0] != n_seqs:
            raise ValueError("kda_attn_prefill: q and k hold different numbers of sequences")
    lse_ptr = None
    if lse is not None:
        if lse.shape != q_shape[:-1]:
            raise ValueError("kda_attn_prefill: lse must be [rows, heads]")
        lse_ptr = _packed(lse, torch.float32, dev, "lse")
    rows = t_q if cu_q else t_q * n_seqs
    workspace, ws_ptr, ws_bytes = _scratch(
        workspace,
        lambda: LIB.kda_attn_prefill_workspace_size(rows, n_seqs, heads, kv_heads), dev)
    _check(LIB.kda_attn_prefill(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, t_q, t_k, cu_q, cu_k, n_seqs,
                                heads, kv_heads, HEAD_DIM, in_dtype, q_row, k_row, v_row, o_row,
                                _window(window), scale, ws_ptr, ws_bytes, _raw_stream(dev)))


def kv4_cache(n_pages, kv_heads, page=64, device="cuda"):
    """A 4-bit cache of n_pages pages: uint8 [n_pages, kv_heads, page * 144]."""
    if page not in KV4_PAGES:
        raise ValueError("page must be one of %s" % (KV4_PAGES,))
    return torch.zeros((n_pages, kv_heads, page * KV4_TOKEN_BYTES), dtype=torch.uint8,
                       device=device)


def _kv4(cache, page_table, lens, dev):
    """The cache arguments: (pointer, pages, tokens a page, table, width, lens)."""
    ptr, shape, table = _packed(cache, torch.uint8, dev, "cache"), cache.shape, page_table.shape
    if len(shape) != 3 or shape[2] % KV4_TOKEN_BYTES or shape[2] // KV4_TOKEN_BYTES not in KV4_PAGES:
        raise ValueError("the cache must be [pages, kv_heads, page * 144], page one of %s"
                         % (KV4_PAGES,))
    if len(table) != 2 or table[0] != lens.numel():
        raise ValueError("page_table must be [sequences, pages], lens [sequences]")
    return (ptr, shape[0], shape[2] // KV4_TOKEN_BYTES,
            _packed(page_table, torch.int32, dev, "page_table"), table[1],
            _packed(lens, torch.int32, dev, "lens"))


def _kv4_rows(name, fn, k, v, cache, page_table, lens, cu_seqlens):
    in_dtype, dev = _attn_type(k, "k")
    k_ptr, k_row = _rows(k, k.dtype, dev, "k")
    v_ptr, v_row = _rows(v, k.dtype, dev, "v")
    cache_args = _kv4(cache, page_table, lens, dev)
    shape, n_seqs, kv_heads = k.shape, page_table.shape[0], cache.shape[1]
    if v.shape != shape or shape[-2] != kv_heads:
        raise ValueError("%s: k and v must be [rows, kv_heads, 128] of the cache's kv_heads" % name)
    cu = None
    if cu_seqlens is not None:
        if len(shape) != 3 or cu_seqlens.numel() != n_seqs + 1:
            raise ValueError("%s: packed rows have three dimensions, and one offset more than "
                             "sequences" % name)
        cu, t = _packed(cu_seqlens, torch.int32, dev, "cu_seqlens"), shape[0]
    else:
        rows = shape[0] * (shape[1] if len(shape) == 4 else 1)
        t = rows // n_seqs if n_seqs else 0   # (without sequences the call refuses)
        if rows != t * n_seqs or (len(shape) == 4 and shape[0] != n_seqs):
            raise ValueError("%s: the rows do not divide over the sequences" % name)
    _check(fn(k_ptr, v_ptr, k_row, v_row, t, cu, n_seqs, kv_heads, HEAD_DIM, in_dtype, *cache_args,
              _raw_stream(dev)))


def kda_attn_kv4_append(k, v, cache, page_table, lens, cu_seqlens=None):
    """Writes rows into the 4-bit cache: BF16 or FP16 k, v [rows, kv_heads, 128]
    become the last positions of their sequences, lens (device int32 [N]) counting
    them already.  page_table: device int32 [N, pages].  cu_seqlens: offsets of
    packed rows; without it each sequence has rows / N (also [N, k, kv_heads, 128])."""
    _kv4_rows("kda_attn_kv4_append", LIB.kda_attn_kv4_append, k, v, cache, page_table, lens,
              cu_seqlens)


def kda_attn_kv4_read(k, v, cache, page_table, lens, cu_seqlens=None):
    """The last rows of each sequence out of the 4-bit cache into k and v, which
    are laid out as kda_attn_kv4_append's."""
    _kv4_rows("kda_attn_kv4_read", LIB.kda_attn_kv4_read, k, v, cache, page_table, lens,
              cu_seqlens)


def kda_attn_kv4_workspace(n_seqs, krows, heads, kv_heads, device="cuda"):
    """Workspace for kda_attn_kv4_decode."""
    need = LIB.kda_attn_kv4_workspace_size(n_seqs, krows, heads, kv_heads)
    return torch.empty(int(need), dtype=torch.uint8, device=device)


def kda_attn_kv4_decode(q, cache, page_table, lens, out, lse=None, window=0, scale=Q_SCALE,
                        workspace=None):
    """k query rows of each sequence over the 4-bit cache: q, out BF16 or FP16
    [N, k, heads, 128] (or [N, heads, 128]), the last k of lens[n] positions; lse
    FP32 [N, k, heads] or None."""
    in_dtype, dev = _attn_type(q, "q")
    shape = q.shape
    if len(shape) not in (3, 4) or shape[-1] != HEAD_DIM or out.shape != shape:
        raise ValueError("kda_attn_kv4_decode: q and out must be [N, k, heads, 128]")
    q_ptr, o_ptr = _packed(q, q.dtype, dev, "q"), _packed(out, q.dtype, dev, "out")
    c_ptr, n_pages, page, table, width, lens_ptr = _kv4(cache, page_table, lens, dev)
    n_seqs, heads, kv_heads = shape[0], shape[-2], cache.shape[1]
    krows = shape[1] if len(shape) == 4 else 1
    if page_table.shape[0] != n_seqs:
        raise ValueError("kda_attn_kv4_decode: page_table and lens must have q's sequences")
    lse_ptr = None
    if lse is not None:
        if lse.shape != shape[:-1]:
            raise ValueError("kda_attn_kv4_decode: lse must be [N, k, heads]")
        lse_ptr = _packed(lse, torch.float32, dev, "lse")
    workspace, ws_ptr, ws_bytes = _scratch(
        workspace, lambda: LIB.kda_attn_kv4_workspace_size(n_seqs, krows, heads, kv_heads), dev)
    _check(LIB.kda_attn_kv4_decode(q_ptr, c_ptr, n_pages, page, table, width, lens_ptr, o_ptr,
                                   lse_ptr, n_seqs, krows, heads, kv_heads, HEAD_DIM, in_dtype,
                                   _window(window), scale, ws_ptr, ws_bytes, _raw_stream(dev)))


# ---------------------------------------------------------------- rotary positions, pages

_device = torch._C._cuda_getDevice
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


class _Slow:
    """In the extension's place."""

    def __getattr__(self, name):
        return lambda *args: -1


def _load_fast():
    """The calls below in C, for arguments that are as they should be; for others each
    returns -1 and calls nothing, and the Python code says what is wrong.  Where the
    extension is not built, Python does all of it."""
    if not os.path.exists(_build.FAST):
        return _Slow()
    spec = importlib.util.spec_from_file_location("fast_calls", _build.FAST)
    fast = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fast)
    names = ("kda_lin_prefill", "kda_lin_decode", "kda_attn_rope", "kda_attn_kv4_resize",
             "kda_attn_kv4_fork", "kda_attn_kv4_compact", "kda_attn_kv4_copy")
    fast.setup(tuple(_c.cast(getattr(LIB, name), _vp).value for name in names),
               (torch.bfloat16, torch.float16, _F32, _I32, _U8), _raw_stream, _device)
    return fast


_fast = _load_fast()


def _call(dev, fn, *args):
    """`fn` on device `dev`'s current stream."""
    if _device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status:
        _check(status)


def _array(t, dtype, dev, shape, name):
    """Pointer of a contiguous array of the given type and shape."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError("%s must be %s" % (name, list(shape)))
    return _packed(t, dtype, dev, name)


def _space(workspace, dev, size, *args):
    """(tensor, pointer, bytes): the caller's workspace, or one of size(*args) bytes."""
    if workspace is None:
        workspace = torch.empty(size(*args), dtype=_U8, device="cuda:%d" % dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on the call's device")
    return workspace, workspace.data_ptr(), workspace.nbytes


def kda_attn_rope(q, k, positions, inv_freq, q_out=None, k_out=None, pair_axis=None,
                  interleaved=False, factor=1.0):
    """Rotary positions: BF16 or FP16 q [rows, heads, 128] and k [rows, kv_heads, 128]
    (or None), which may be strided views, into q_out and k_out (default: in place).
    positions: device int32 [rows] or [rows, axes]; inv_freq: device FP32 [pairs];
    pair_axis: the axis of each pair (a sequence of pairs numbers), needed with
    several axes.  interleaved: a pair is two neighbours, else channels p and
    p + pairs; channels behind the pairs stay."""
    status = _fast.rope(q, k, positions, inv_freq, q_out, k_out, pair_axis, interleaved, factor)
    if status >= 0:
        return _check(status)
    in_dtype, dev = _attn_type(q, "q")
    dt, shape = q.dtype, q.shape
    q_ptr, q_row = _rows(q, dt, dev, "q")
    qo_ptr, qo_row = (q_ptr, q_row) if q_out is None else _rows(q_out, dt, dev, "q_out")
    if q_out is not None and q_out.shape != shape:
        raise ValueError("kda_attn_rope: q_out must have q's shape")
    k_ptr = ko_ptr = None
    k_row = ko_row = kv_heads = 0
    lead = shape[:-2]
    if k is not None:
        k_shape = k.shape
        k_ptr, k_row = _rows(k, dt, dev, "k")
        ko_ptr, ko_row = (k_ptr, k_row) if k_out is None else _rows(k_out, dt, dev, "k_out")
        kv_heads = k_shape[-2]
        if k_shape[:-2] != lead or (k_out is not None and k_out.shape != k_shape):
            raise ValueError("kda_attn_rope: k_out must have k's shape, and k q's rows")
    elif k_out is not None:
        raise ValueError("kda_attn_rope: k_out without k")
    rows = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    pos_shape = positions.shape
    axes = 1 if pos_shape == lead else pos_shape[-1] if pos_shape[:-1] == lead else 0
    if not axes:
        raise ValueError("kda_attn_rope: positions must be [rows] or [rows, axes]")
    pairs = inv_freq.shape[0] if inv_freq.dim() == 1 else 0
    table = None
    if pair_axis is not None:
        table = bytes([operator.index(a) for a in pair_axis])
        if len(table) != pairs or max(table, default=0) >= axes:
            raise ValueError("kda_attn_rope: pair_axis must hold an axis below %d for each pair"
                             % axes)
    elif axes > 1:
        raise ValueError("kda_attn_rope: several axes need pair_axis")
    _call(dev, LIB.kda_attn_rope, q_ptr, k_ptr, qo_ptr, ko_ptr, rows, shape[-2], kv_heads,
          HEAD_DIM, in_dtype, q_row, k_row, qo_row, ko_row,
          _array(positions, _I32, dev, pos_shape, "positions"), axes,
          _array(inv_freq, _F32, dev, (pairs,), "inv_freq"), pairs, table, bool(interleaved),
          factor)


def kda_attn_kv4_pages_workspace(n_pages, n_seqs, max_pages, device="cuda"):
    """Workspace for kda_attn_kv4_resize, kda_attn_kv4_fork and kda_attn_kv4_compact."""
    need = LIB.kda_attn_kv4_pages_workspace_size(int(n_pages), n_seqs, max_pages)
    return torch.empty(int(need), dtype=torch.uint8, device=device)


def _pages(page_table, refs, workspace):
    """(table pointer, its shape, refs pointer, shape, device, workspace, pointer, bytes)"""
    dev, shape, n = page_table.get_device(), page_table.shape, refs.shape
    if dev < 0:
        raise TypeError("page_table must be a CUDA tensor")
    if len(shape) != 2 or len(n) != 1:
        raise ValueError("page_table must be [sequences, pages], refs [pages of the cache]")
    return (_array(page_table, _I32, dev, shape, "page_table"), shape,
            _array(refs, _I32, dev, n, "refs"), n, dev,
            *_space(workspace, dev, LIB.kda_attn_kv4_pages_workspace_size, n[0], *shape))


def kda_attn_kv4_resize(page_table, lens, refs, page=64, workspace=None):
    """Gives and frees pages in place, so that each sequence has those of its lens
    positions: page_table device int32 [N, max_pages] (-1: none), lens [N], refs
    [pages of the cache], how often each page is named (0: free)."""
    status = _fast.resize(page_table, lens, refs, page, workspace)
    if status >= 0:
        return _check(status)
    table, shape, refs_ptr, n, dev, workspace, ws, ws_bytes = _pages(page_table, refs, workspace)
    _call(dev, LIB.kda_attn_kv4_resize, table, _array(lens, _I32, dev, shape[:1], "lens"), refs_ptr,
          shape[0], shape[1], n[0], page, ws, ws_bytes)


def _lists(src, dst, count, n, dev):
    def new(t, size):
        return torch.empty(size, dtype=_I32, device="cuda:%d" % dev) if t is None else t
    return new(src, n), new(dst, n), new(count, 1)


def kda_attn_kv4_fork(page_table, lens, refs, parent, page_table_out=None, lens_out=None,
                      refs_out=None, src=None, dst=None, count=None, page=64, workspace=None):
    """Sequence n goes on from sequence parent[n] (device int32 [N]; -1: it ends).
    The outputs default to being in place.  Returns (src, dst, count), the pages for
    kda_attn_kv4_copy: device int32 [N], [N] and [1], allocated where not given."""
    status = _fast.fork(page_table, lens, refs, parent, page_table_out, lens_out, refs_out, src, dst,
                        count, page, workspace)
    if status >= 0:
        _check(status)
        return src, dst, count
    table, shape, refs_ptr, n, dev, workspace, ws, ws_bytes = _pages(page_table, refs, workspace)
    rows = shape[:1]
    src, dst, count = _lists(src, dst, count, rows[0], dev)
    lens_ptr = _array(lens, _I32, dev, rows, "lens")
    _call(dev, LIB.kda_attn_kv4_fork, table, lens_ptr, refs_ptr,
          _array(parent, _I32, dev, rows, "parent"),
          table if page_table_out is None
          else _array(page_table_out, _I32, dev, shape, "page_table_out"),
          lens_ptr if lens_out is None else _array(lens_out, _I32, dev, rows, "lens_out"),
          refs_ptr if refs_out is None else _array(refs_out, _I32, dev, n, "refs_out"),
          _array(src, _I32, dev, rows, "src"), _array(dst, _I32, dev, rows, "dst"),
          _array(count, _I32, dev, (1,), "count"), rows[0], shape[1], n[0], page, ws, ws_bytes)
    return src, dst, count


def kda_attn_kv4_compact(page_table, refs, page_table_out=None, refs_out=None, src=None, dst=None,
                         count=None, workspace=None):
    """Makes the pages in use the lowest-numbered ones.  The outputs default to being
    in place.  Returns (src, dst, count), the moves for kda_attn_kv4_copy: device
    int32 [pages // 2] twice and [1], allocated where not given."""
    status = _fast.compact(page_table, refs, page_table_out, refs_out, src, dst, count, workspace)
    if status >= 0:
        _check(status)
        return src, dst, count
    table, shape, refs_ptr, n, dev, workspace, ws, ws_bytes = _pages(page_table, refs, workspace)
    half = (n[0] // 2,)
    src, dst, count = _lists(src, dst, count, half[0], dev)
    _call(dev, LIB.kda_attn_kv4_compact, table, refs_ptr,
          table if page_table_out is None
          else _array(page_table_out, _I32, dev, shape, "page_table_out"),
          refs_ptr if refs_out is None else _array(refs_out, _I32, dev, n, "refs_out"),
          _array(src, _I32, dev, half, "src"), _array(dst, _I32, dev, half, "dst"),
          _array(count, _I32, dev, (1,), "count"), shape[0], shape[1], n[0], ws, ws_bytes)
    return src, dst, count


def kda_attn_kv4_copy(caches, src, dst, count):
    """Copies pages src[i] to dst[i], i < count, in each of `caches` (one 4-bit cache, or a
    list of them, one for each layer, all of one shape); src and dst device int32
    [n], count [1]."""
    status = _fast.copy(caches, src, dst, count)
    if status >= 0:
        return _check(status)
    caches = [caches] if isinstance(caches, torch.Tensor) else list(caches)
    if not 1 <= len(caches) <= KV4_MAX_CACHES:
        raise ValueError("kda_attn_kv4_copy: 1 to %d caches" % KV4_MAX_CACHES)
    dev, shape = caches[0].get_device(), caches[0].shape
    if dev < 0:
        raise TypeError("the caches must be CUDA tensors")
    if len(shape) != 3 or shape[2] % KV4_TOKEN_BYTES or shape[2] // KV4_TOKEN_BYTES not in KV4_PAGES:
        raise ValueError("a cache must be [pages, kv_heads, page * 144], page one of %s"
                         % (KV4_PAGES,))
    rows = src.shape
    if len(rows) != 1:
        raise ValueError("kda_attn_kv4_copy: src must be [n]")
    array = (_c.c_void_p * len(caches))(*[_array(c, _U8, dev, shape, "cache") for c in caches])
    _call(dev, LIB.kda_attn_kv4_copy, array, len(caches), shape[0], shape[2] // KV4_TOKEN_BYTES,
          shape[1], _array(src, _I32, dev, rows, "src"), _array(dst, _I32, dev, rows, "dst"),
          _array(count, _I32, dev, (1,), "count"), rows[0])


# ---------------------------------------------------------------- linear attention

def _decays(g, lead, heads, dev):
    """(pointer, token-row stride) of g: [heads], or [.., rows, heads] in rows."""
    shape = g.shape
    if len(shape) == 1:
        return _array(g, _F32, dev, (heads,), "g"), 0
    if shape[:-1] != lead or shape[-1] != heads:
        raise ValueError("g must be [rows, heads] or [heads]")
    ptr = _at(g, _F32, dev, "g")
    if g.is_contiguous():
        return ptr, heads
    stride = g.stride()
    row = stride[-2] if lead[-1] > 1 else heads
    if stride[-1] != 1 and heads > 1:
        raise ValueError("g must have unit head stride")
    if len(lead) == 2 and lead[0] > 1:
        if lead[1] == 1:
            row = stride[0]
        elif stride[0] != lead[1] * row:
            raise ValueError("g: sequences must be consecutive row blocks")
    if row < heads:
        raise ValueError("g: rows must not overlap")
    return ptr, row


def _lin_rows(name, q, k, v, g, out):
    """What both calls take of their rows: (type, device, pointers, strides, lead, heads)."""
    in_dtype, dev = _attn_type(q, "q")
    dt, shape, v_shape = q.dtype, q.shape, v.shape
    q_ptr, q_row = _rows(q, dt, dev, "q")
    k_ptr, k_row = _rows(k, dt, dev, "k")
    v_ptr, v_row = _rows(v, dt, dev, "v")
    o_ptr, o_row = _rows(out, dt, dev, "out")
    lead, heads = shape[:-2], v_shape[-2]
    if k.shape != shape or v_shape[:-2] != lead or out.shape != v_shape:
        raise ValueError("%s: k must have q's shape, out v's, and v q's rows" % name)
    g_ptr, g_row = _decays(g, lead, heads, dev)
    return (in_dtype, dev, (q_ptr, k_ptr, v_ptr, g_ptr, o_ptr),
            (q_row, k_row, v_row, g_row, o_row), lead, heads, shape[-2])


def kda_lin_prefill_workspace(rows, n_seqs, heads, device="cuda"):
    """Workspace for kda_lin_prefill over `rows` token rows in total."""
    need = LIB.kda_lin_prefill_workspace_size(int(rows), n_seqs, heads)
    return torch.empty(int(need), dtype=torch.uint8, device=device)


def kda_lin_prefill(q, k, v, g, out, state_in=None, state_out=None, t=None, cu_seqlens=None,
                    scale=Q_SCALE, workspace=None):
    """Linear attention with a decay for each head over prompts.  BF16 or FP16 q, k
    [rows, qk_heads, 128] and v, out [rows, heads, 128], which may be strided views;
    g FP32 [rows, heads] or [heads]; state_in and state_out FP32 [N, heads, 128, 128],
    None for states of zero, or states that are not wanted; they may be one.
    cu_seqlens (device int32 [N+1]) gives packed sequences; without it, four
    dimensions [N, T, heads, 128] hold N sequences and three one, of t tokens each
    (default: all) with the rows behind them left alone."""
    status = _fast.lin_prefill(q, k, v, g, out, state_in, state_out, t, cu_seqlens, scale, workspace)
    if status >= 0:
        return _check(status)
    in_dtype, dev, ptrs, strides, lead, heads, qk_heads = _lin_rows("kda_lin_prefill", q, k, v, g,
                                                                    out)
    cu = None
    if cu_seqlens is not None:
        if len(lead) != 1 or t not in (None, lead[0]):
            raise ValueError("kda_lin_prefill: packed rows have three dimensions, and t is all "
                             "of them")
        cu = _packed(cu_seqlens, _I32, dev, "cu_seqlens")
        n_seqs, t_pad = cu_seqlens.numel() - 1, lead[0]
    else:
        n_seqs, t_pad = (1, lead[0]) if len(lead) == 1 else lead
    want = (n_seqs, heads, HEAD_DIM, HEAD_DIM)
    rows = t_pad if cu else t_pad * n_seqs
    workspace, ws, ws_bytes = _space(workspace, dev, LIB.kda_lin_prefill_workspace_size, rows,
                                     n_seqs, heads)
    _call(dev, LIB.kda_lin_prefill,
          None if state_in is None else _array(state_in, _F32, dev, want, "state_in"),
          None if state_out is None else _array(state_out, _F32, dev, want, "state_out"), *ptrs,
          t_pad if t is None else t, t_pad, cu, n_seqs, heads, qk_heads, HEAD_DIM, in_dtype,
          *strides, scale, ws, ws_bytes)


def kda_lin_decode(q, k, v, g, out, state_in=None, state_out=None, snapshots=(), scale=Q_SCALE):
    """Up to 8 tokens of each sequence: q, k [N, k, qk_heads, 128] and v, out
    [N, k, heads, 128] (or without k: one token), g FP32 [N, k, heads] or [heads];
    states as kda_lin_prefill's; snapshots: up to k tensors like the states,
    snapshots[t] = state after row t."""
    status = _fast.lin_decode(q, k, v, g, out, state_in, state_out, snapshots, scale)
    if status >= 0:
        return _check(status)
    in_dtype, dev, ptrs, strides, lead, heads, qk_heads = _lin_rows("kda_lin_decode", q, k, v, g,
                                                                    out)
    n_seqs, krows = lead if len(lead) == 2 else (lead[0], 1)
    want = (n_seqs, heads, HEAD_DIM, HEAD_DIM)
    array, n_snap = None, len(snapshots)
    if n_snap:
        array = (_c.c_void_p * n_snap)(*[_array(s, _F32, dev, want, "snapshot")
                                         for s in snapshots])
    _call(dev, LIB.kda_lin_decode,
          None if state_in is None else _array(state_in, _F32, dev, want, "state_in"),
          None if state_out is None else _array(state_out, _F32, dev, want, "state_out"), *ptrs,
          n_seqs, krows, heads, qk_heads, HEAD_DIM, in_dtype, *strides, scale, array, n_snap)


def kda_sync_status(device=None):
    """Synchronise the current stream and raise if a device-side check failed."""
    s = torch.cuda.current_stream(device).cuda_stream
    _check(LIB.kda_sync_status(s))
