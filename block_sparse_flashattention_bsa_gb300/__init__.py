"""Block-sparse FlashAttention forward for GB300 (sm_103a).

A thin ctypes binding over ``libbsa.so`` (declared in ``include/bsa.h``).
Every step of the computation runs in the library's CUDA kernels; this module
only marshals torch tensors (device memory) and the current CUDA stream into
the C ABI and turns status codes into exceptions (for the projection and
paged-cache calls, whose kernels can be shorter than that in Python, compiled:
``csrc/bsa_torch.cpp``).  There is no fallback: if the library is missing or
the device is not sm_103, calls raise.

Entry points (same names as the C ABI, minus the ``bsa_`` prefix):

* :func:`build_mask_csr`  pattern (window / globals / causal) -> block CSR
* :func:`build_mask_csr_heads`  per-head patterns (:class:`PatternEx`: dilated
  windows, stride, globals, causal) -> block CSR
* :func:`topk_blocks`     content-based block CSR (pooled Q.K top-k + diagonal)
* :func:`forward`         block-sparse attention forward -> (O bf16, LSE fp32)
* :func:`forward_ex`      the same with key blocks apart from the query blocks
  (sequence shards), a query offset and per-row causal flags
  (:func:`pattern_row_flags`: global query rows of a causal model)
* :func:`forward_fp8`     the same with FP8 scores (e4m3 Q and K, per-tensor
  descale factors); :func:`quantize_e4m3` makes the e4m3 inputs;
  :func:`forward_fp8_blocks` / :func:`quantize_e4m3_blocks` take one
  descale factor per (head, block)
* :func:`backward`        its gradients (dQ, dK, dV) through the same mask
* :func:`forward_noalloc`  the forward with no allocation by the library
* :func:`validate_csr`, :func:`device_error`, :func:`pattern_nnz`
* :func:`set_wait_limit` (hang detection), :func:`debug_stall_next_forward`
  (its test hook)
* :func:`block_sparse_attention`  convenience: mask + forward in one call
* :func:`qk_norm_rope`, :func:`qk_norm_rope_backward`  norm of query and key
  heads and position rotation on the way from a projection to the attention,
  and its gradients; :func:`rope_inv_freq` makes the frequencies
* :func:`cache_append`, :func:`tree_attention`, :func:`cache_accept`  serving
  over a paged cache: write new tokens, attend with one or a tree of drafted
  tokens per sequence, keep the accepted ones
* :func:`chunk_attention`  attention of chunks of new tokens (or one token a
  sequence) over a paged cache, over all slots or a sliding window with sinks
* :func:`cache_resize`, :func:`cache_fork`, :func:`cache_compact`  its pages
* :func:`cache_read`  ranges of a cache back as what :func:`forward` takes; the
  cache calls, `chunk_attention` and this one also take caches of 8-bit rows
  (e4m3 codes, a power of two per row)
"""

from ._binding import (  # noqa: F401
    BsaError,
    Pattern,
    PatternEx,
    backward,
    block_sparse_attention,
    build_mask_csr,
    build_mask_csr_heads,
    debug_stall_next_forward,
    device_error,
    forward,
    forward_ex,
    forward_fp8,
    forward_fp8_blocks,
    forward_noalloc,
    get_wait_limit,
    lib,
    lib_path,
    mask_heads_nnz,
    pattern_nnz,
    pattern_row_flags,
    quantize_e4m3,
    quantize_e4m3_blocks,
    release_workspace,
    set_wait_limit,
    topk_blocks,
    validate_csr,
)
from .paged import (  # noqa: F401
    cache_accept,
    cache_append,
    cache_compact,
    cache_fork,
    cache_read,
    cache_resize,
    chunk_attention,
    tree_attention,
)
from .rope import (  # noqa: F401
    qk_norm_rope,
    qk_norm_rope_backward,
    rope_inv_freq,
)
