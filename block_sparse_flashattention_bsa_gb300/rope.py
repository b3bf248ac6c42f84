"""From a projection to the attention: per-head RMS norm and position rotation
in one pass, token-major in and head-major out, and its gradients.

Marshalling only; contracts are in ``include/bsa.h`` and the kernels in
``csrc/bsa_rope.cu``.
"""

from __future__ import annotations

import struct
from typing import Optional, Tuple

import torch

from ._binding import _addr, _check, _raw_stream, _same_device, _scope, lib

_SCALING = {None: 0, "linear": 1, "base": 2, "by_parts": 3}
_BF16, _F32, _F64, _I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
_SPEC = struct.Struct("@2i5d")              # bsa_rope_spec
_ARGS = struct.Struct("@8i2f3P9qPPq2P")     # bsa_norm_rope_args
_GRADS = struct.Struct("@6P9q2P")           # bsa_norm_rope_grads


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
    spec = _SPEC.pack(int(rotary_dim), _SCALING[scaling], float(base), float(factor), float(original_length),
                      float(low), float(high))
    out = torch.empty(max(0, int(rotary_dim)) // 2, dtype=_F64)
    _check("bsa_rope_inv_freq", lib().bsa_rope_inv_freq(spec, out.data_ptr() or None))
    return out.to(device)


def _row_stride(t: torch.Tensor, what: str):
    """(batch, token, head) strides in elements of a token-major bf16 tensor
    ([tokens, heads, D]: batch 0).  An extent of one has no stride worth checking."""
    if t.dtype is not _BF16:
        raise ValueError("%s: expected bf16" % what)
    if t.dim() == 4:
        (b, n, h, _), (sb, sn, sh, sd) = t.shape, t.stride()
    else:
        (n, h, _), (sn, sh, sd) = t.shape, t.stride()
        b, sb = 1, 0
    if sd != 1:
        raise ValueError("%s: head rows must be contiguous" % what)
    return sb if b > 1 else 0, sn if n > 1 else 0, sh if h > 1 else 0


def _side_args(q, k, v, inv_freq, positions, q_weight, k_weight, eps, gain, interleaved, kv_repeat, batched):
    """Checks and packed C arguments shared by the forward, its gradients and
    the cache append (batched: [B, N, H, D], else [tokens, H, D])."""
    qs, ks = q.shape, k.shape
    if len(qs) != (4 if batched else 3) or len(ks) != len(qs) or qs[:-2] != ks[:-2] or qs[-1] != ks[-1] \
            or (v is not None and v.shape != ks):
        raise ValueError("expected q, k, v with one shape up to their number of heads (k, v alike)")
    index = _same_device(q, k, v, inv_freq, positions, q_weight, k_weight)
    if batched:
        B, N, Hq, D = qs
    else:
        B, (N, Hq, D) = 1, qs
    rd = 0
    if inv_freq is not None:
        if inv_freq.dtype is not _F64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq: contiguous float64 [rotary_dim / 2] (rope_inv_freq)")
        rd = 2 * inv_freq.numel()
    pos_stride = 0
    if positions is not None:
        ps = positions.shape
        if positions.dtype is not _I32 or not (ps == (N,) or (batched and ps == (B, N))) \
                or (N > 1 and positions.stride(-1) != 1):
            raise ValueError("positions: int32 [N] or [B, N], one per token")
        pos_stride = positions.stride(0) if len(ps) == 2 and B > 1 else 0
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype is not _F32 or w.shape != (D,) or not w.is_contiguous()):
            raise ValueError("norm weights: contiguous float32 [D]")
    a = _ARGS.pack(B, N, Hq, ks[-2], D, rd, kv_repeat, 1 if interleaved else 0, eps, gain, q.data_ptr(),
                   k.data_ptr(), _addr(v), *_row_stride(q, "q"), *_row_stride(k, "k"),
                   *((0, 0, 0) if v is None else _row_stride(v, "v")), _addr(inv_freq), _addr(positions), pos_stride,
                   _addr(q_weight), _addr(k_weight))
    return a, index, B, N, Hq, ks[-2], D


def _output(given, shape, like):
    """A contiguous bf16 tensor of `shape`: the given one, checked, or a new one."""
    if given is None:
        return torch.empty(shape, dtype=_BF16, device=like.device)
    if given.shape != shape or given.dtype is not _BF16 or not given.is_contiguous() or given.device != like.device:
        raise ValueError("out: contiguous bf16 %s on %s" % (tuple(shape), like.device))
    return given


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
    a, index, B, N, Hq, Hkv, D = _side_args(q, k, v, inv_freq, positions, q_weight, k_weight, eps, gain,
                                            interleaved, kv_repeat, True)
    kv = (B, Hkv * kv_repeat, N, D)
    oq, ok, ov = (None, None, None) if out is None else out
    if v is None and ov is not None:
        raise ValueError("out: no v to write")
    with _scope(index, stream):
        oq, ok = _output(oq, (B, Hq, N, D), q), _output(ok, kv, q)
        ov = None if v is None else _output(ov, kv, q)
        st = lib().bsa_qk_norm_rope(a, oq.data_ptr(), ok.data_ptr(), _addr(ov), _raw_stream(index))
    if st:
        _check("bsa_qk_norm_rope", st)
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
    a, index, B, N, Hq, Hkv, D = _side_args(q, k, None, inv_freq, positions, q_weight, k_weight, eps, gain,
                                            interleaved, kv_repeat, True)
    kv = (B, Hkv * kv_repeat, N, D)
    _same_device(q, dq, dk, dv)
    for t, s in ((dq, (B, Hq, N, D)), (dk, kv), (dv, kv)):
        if t is not None and (t.shape != s or t.dtype is not _BF16 or not t.is_contiguous()):
            raise ValueError("dq, dk, dv: contiguous bf16 tensors of the forward's output shapes")
    device = q.device
    sq, sk = (B, N, Hq, D), (B, N, Hkv, D)
    with _scope(index, stream):
        if out is None:
            gq = torch.empty(sq, dtype=_BF16, device=device)
            gk = torch.empty(sk, dtype=_BF16, device=device)
            gv = None if dv is None else torch.empty(sk, dtype=_BF16, device=device)
        else:
            gq, gk, gv = out
            _same_device(q, gq, gk, gv)
            if gq.shape != sq or gk.shape != sk or (gv is None) != (dv is None) or (gv is not None
                                                                                    and gv.shape != sk):
                raise ValueError("out: token-major tensors of shapes %s, %s, %s" % (sq, sk, sk))
        gqw = torch.empty(D, dtype=_F32, device=device) if q_weight is not None else None
        gkw = torch.empty(D, dtype=_F32, device=device) if k_weight is not None else None
        L = lib()
        n = int(L.bsa_qk_norm_rope_backward_workspace(D)) if gqw is not None or gkw is not None else 0
        ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None
        g = _GRADS.pack(dq.data_ptr(), dk.data_ptr(), _addr(dv), gq.data_ptr(), gk.data_ptr(), _addr(gv),
                        *_row_stride(gq, "out"), *_row_stride(gk, "out"),
                        *((0, 0, 0) if gv is None else _row_stride(gv, "out")), _addr(gqw), _addr(gkw))
        st = L.bsa_qk_norm_rope_backward(a, g, _addr(ws), n, _raw_stream(index))
    if st:
        _check("bsa_qk_norm_rope_backward", st)
    return gq, gk, gv, gqw, gkw
