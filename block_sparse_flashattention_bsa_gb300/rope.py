"""From a projection to the attention: per-head RMS norm and position rotation
in one pass, token-major in and head-major out, and its gradients.

Marshalling only (``csrc/bsa_torch.cpp``); contracts are in ``include/bsa.h``
and the kernels in ``csrc/bsa_rope.cu``.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._binding import _RopeSpec, _call, _check, compiled, lib

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
    _check("bsa_rope_inv_freq", lib().bsa_rope_inv_freq(ctypes.byref(spec), out.data_ptr() or None))
    return out.to(device)


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
    oq, ok, ov = (None, None, None) if out is None else out
    return _call(compiled().qk_norm_rope, "bsa_qk_norm_rope", stream, q, k, v, inv_freq, positions, q_weight,
                 k_weight, eps, gain, interleaved, kv_repeat, oq, ok, ov)


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
    oq, ok, ov = (None, None, None) if out is None else out
    return _call(compiled().qk_norm_rope_backward, "bsa_qk_norm_rope_backward", stream, q, k, None, inv_freq,
                 positions, q_weight, k_weight, eps, gain, interleaved, kv_repeat, dq, dk, dv,
                 None if out is None else True, oq, ok, ov)
