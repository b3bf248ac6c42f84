"""From a projection to the attention: per-head RMS norm and position rotation
in one pass, token-major in and head-major out, and its gradients.

Marshalling only; contracts are in ``include/bsa.h`` and the kernels in
``csrc/bsa_rope.cu``.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._binding import (_NormRopeArgs, _NormRopeGrads, _RopeSpec, _Stride3, _addr, _check, _same_device, _scope,
                       _stream, lib)

_SCALING = {None: 0, "linear": 1, "base": 2, "by_parts": 3}


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                  original_length: float = 0.0, low: float = 1.0, high: float = 32.0, device="cuda") -> torch.Tensor:
    """Frequencies (radians per position) of the rotary pairs, float64 [rotary_dim / 2].

    scaling None: base^(-2i / rotary_dim); "linear": divided by factor;
    "base": the base times factor^(rotary_dim / (rotary_dim - 2));
    "by_parts": pairs that turn fewer than `low` times over original_length
    positions are divided by factor, those of more than `high` turns kept, a
    linear ramp between."""
    if scaling not in _SCALING:
        raise ValueError("scaling: None, 'linear', 'base' or 'by_parts'")
    spec = _RopeSpec(int(rotary_dim), _SCALING[scaling], float(base), float(factor), float(original_length),
                     float(low), float(high))
    out = torch.empty(max(0, int(rotary_dim)) // 2, dtype=torch.float64)
    _check("bsa_rope_inv_freq", lib().bsa_rope_inv_freq(ctypes.byref(spec), ctypes.c_void_p(out.data_ptr())))
    return out.to(device)


def _row_stride(t: torch.Tensor, what: str):
    """(batch, token, head) strides in elements of a token-major bf16 tensor."""
    if t.dtype != torch.bfloat16 or (t.stride(-1) != 1 and t.numel() > 0):
        raise ValueError("%s: expected bf16 with contiguous head rows" % what)
    # a dimension of one element has no stride worth checking
    return [s if n > 1 else 0 for s, n in zip(t.stride()[:-1], t.shape[:-1])]


def _side_args(q, k, v, inv_freq, positions, q_weight, k_weight, eps, gain, interleaved, kv_repeat, tokens_dims):
    """Checks and C arguments shared by the forward, its gradients and the
    cache append (tokens_dims: 2 for [B, N, H, D], 1 for [tokens, H, D])."""
    nd = tokens_dims + 2
    if q.dim() != nd or k.dim() != nd or (v is not None and v.shape != k.shape) \
            or q.shape[:tokens_dims] != k.shape[:tokens_dims] or q.shape[-1] != k.shape[-1]:
        raise ValueError("expected q, k, v with one shape up to their number of heads (k, v alike)")
    device = _same_device(q, k, v, inv_freq, positions, q_weight, k_weight)
    Hq, D = q.shape[-2:]
    B, N = q.shape[:2] if tokens_dims == 2 else (1, q.shape[0])
    rd = 0
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq: contiguous float64 [rotary_dim / 2] (rope_inv_freq)")
        rd = 2 * inv_freq.numel()
    pos_stride = 0
    if positions is not None:
        if positions.dtype != torch.int32 or (N > 1 and positions.stride(-1) != 1) or \
                positions.shape[-1] != N or positions.dim() > tokens_dims or \
                (positions.dim() == 2 and positions.shape[0] != B):
            raise ValueError("positions: int32 [N] or [B, N], one per token")
        pos_stride = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype != torch.float32 or w.shape != (D,) or not w.is_contiguous()):
            raise ValueError("norm weights: contiguous float32 [D]")
    pad = [0] * (2 - tokens_dims)
    st = [_Stride3(*(pad + _row_stride(t, n))) if t is not None else _Stride3() for t, n in
          ((q, "q"), (k, "k"), (v, "v"))]
    a = _NormRopeArgs(B, N, Hq, k.shape[-2], D, rd, int(kv_repeat), int(bool(interleaved)), float(eps), float(gain),
                      _addr(q), _addr(k), _addr(v), st[0], st[1], st[2], _addr(inv_freq), _addr(positions),
                      pos_stride, _addr(q_weight), _addr(k_weight))
    return a, device, B, N, Hq, k.shape[-2], D


def _outputs(given, shapes, like):
    """Contiguous bf16 tensors of `shapes`: the given ones, checked, or new ones."""
    if given is None:
        return [None if s is None else torch.empty(s, dtype=torch.bfloat16, device=like.device) for s in shapes]
    if len(given) != len(shapes):
        raise ValueError("out: %d tensors" % len(shapes))
    for t, s in zip(given, shapes):
        if (t is None) != (s is None) or (t is not None and (t.shape != s or t.dtype != torch.bfloat16
                                                             or not t.is_contiguous() or t.device != like.device)):
            raise ValueError("out: contiguous bf16 tensors of shapes %s on %s" % (shapes, like.device))
    return list(given)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor] = None,
                 inv_freq: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 gain: float = 1.0, interleaved: bool = False, kv_repeat: int = 1, out=None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """RMS norm of the heads (where a weight is given) and rotation of the
    first 2 * len(inv_freq) values, from token-major q [B,N,Hq,D] and k, v
    [B,N,Hkv,D] (bf16, any strides with contiguous head rows, such as slices of
    a fused projection) to what `forward` takes: (q [B,Hq,N,D], k and v
    [B,Hkv*kv_repeat,N,D]), head h of k and v written at h*kv_repeat and on.

    positions: int32 [N] or [B,N] (default 0..N-1).  inv_freq None: no
    rotation.  gain multiplies the rotated values.  out: (q, k, v) to write."""
    a, device, B, N, Hq, Hkv, D = _side_args(q, k, v, inv_freq, positions, q_weight, k_weight, eps, gain,
                                             interleaved, kv_repeat, 2)
    kv = (B, Hkv * int(kv_repeat), N, D)
    with _scope(device, stream):
        oq, ok, ov = _outputs(out, [(B, Hq, N, D), kv, None if v is None else kv], q)
        _check("bsa_qk_norm_rope", lib().bsa_qk_norm_rope(ctypes.byref(a), _addr(oq), _addr(ok), _addr(ov),
                                                          _stream(None)))
    return oq, ok, ov


def qk_norm_rope_backward(dq: torch.Tensor, dk: torch.Tensor, dv: Optional[torch.Tensor], q: torch.Tensor,
                          k: torch.Tensor, inv_freq: Optional[torch.Tensor] = None,
                          positions: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                          k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, gain: float = 1.0,
                          interleaved: bool = False, kv_repeat: int = 1, out=None, stream=None):
    """Gradients of `qk_norm_rope` for head-major dq [B,Hq,N,D] and dk, dv
    [B,Hkv*kv_repeat,N,D] (contiguous bf16, what `backward` returns; dv may be
    None); q, k and the options as in the forward.

    Returns (q, k, v gradients, token-major bf16; q_weight, k_weight gradients,
    float32 or None).  out: the three token-major tensors to write, with any
    strides (slices of one gradient of a fused projection)."""
    a, device, B, N, Hq, Hkv, D = _side_args(q, k, None, inv_freq, positions, q_weight, k_weight, eps, gain,
                                             interleaved, kv_repeat, 2)
    kv = (B, Hkv * int(kv_repeat), N, D)
    _same_device(q, dq, dk, dv)
    for t, s in ((dq, (B, Hq, N, D)), (dk, kv), (dv, kv)):
        if t is not None and (t.shape != s or t.dtype != torch.bfloat16 or not t.is_contiguous()):
            raise ValueError("dq, dk, dv: contiguous bf16 tensors of the forward's output shapes")
    shapes = [(B, N, Hq, D), (B, N, Hkv, D), None if dv is None else (B, N, Hkv, D)]
    with _scope(device, stream):
        if out is None:
            gq, gk, gv = (None if s is None else torch.empty(s, dtype=torch.bfloat16, device=device) for s in shapes)
        else:
            gq, gk, gv = out
            _same_device(q, gq, gk, gv)
            for t, s in zip((gq, gk, gv), shapes):
                if (t is None) != (s is None) or (t is not None and t.shape != s):
                    raise ValueError("out: token-major tensors of shapes %s" % (shapes,))
        st = [_Stride3(*_row_stride(t, "out")) if t is not None else _Stride3() for t in (gq, gk, gv)]
        gqw = torch.empty(D, dtype=torch.float32, device=device) if q_weight is not None else None
        gkw = torch.empty(D, dtype=torch.float32, device=device) if k_weight is not None else None
        n = int(lib().bsa_qk_norm_rope_backward_workspace(D)) if gqw is not None or gkw is not None else 0
        ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None
        g = _NormRopeGrads(_addr(dq), _addr(dk), _addr(dv), _addr(gq), _addr(gk), _addr(gv), st[0], st[1], st[2],
                           _addr(gqw), _addr(gkw))
        _check("bsa_qk_norm_rope_backward", lib().bsa_qk_norm_rope_backward(
            ctypes.byref(a), ctypes.byref(g), _addr(ws), n, _stream(None)))
    return gq, gk, gv, gqw, gkw
