"""Operators around the layer: norms of queries and keys with the position
rotation (and its gradients), and a paged cache of keys and values with the
attention of new tokens over it.

Like GSALayer these pass torch tensors' pointers to the C entry points
(include/gsa.h, "operators around the layer"); all arithmetic runs in the CUDA
kernels.  Calls go to the current stream of the tensors' device, or to `stream`
(a raw handle).  Outputs and workspaces are allocated for that stream, one per
call, so that calls in flight and captured graphs share none.  There is no
autograd: gradients are calls of their own, which record none themselves.  In grad
mode a result of inputs that require a gradient raises when one is asked of it, and
values that require one are not written to `out` or into a cache (GSAError: use
torch.no_grad() or detached tensors).  What the device finds wrong
(a page outside the pool, a place without a page) is reported by
operator_status().
"""
from __future__ import annotations

import ctypes

import torch

from . import GSAError, LIB_PATH, load_library

HEAD_DIM = 64
NORMS = {"none": 0, "layer": 1, "rms": 2}
_ENTRIES = ("gsa_qk_norm_rope", "gsa_qk_norm_rope_backward", "gsa_qk_norm_rope_workspace_bytes", "gsa_cache_append",
            "gsa_cache_attention", "gsa_cache_attention_workspace_bytes", "gsa_strerror")


def _bind():
    lib = load_library()
    try:
        from . import _torch_binding as b
    except ImportError as e:
        raise ImportError(f"the torch binding is not built beside {LIB_PATH} "
                          f"(run `python -m sparse_global_attention_b200.build`): {e}") from e
    b.bind(GSAError, *[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _ENTRIES])
    return b


_b = _bind()


def _norm(norm):
    n = NORMS.get(norm)
    if n is None:
        raise GSAError(f"norm must be one of {sorted(NORMS)}, got {norm!r}")
    return n


def qk_norm_rope(q, k=None, v=None, *, norm="layer", eps=1e-5, q_weight=None, q_bias=None, k_weight=None,
                 k_bias=None, positions=None, rope_base=100.0, head_major=False, out=None, stream=None):
    """Norm of queries and keys per head, then the position rotation, in one pass; values carried along.

    q, k, v: [outer, tokens, heads, 64] (outer: frames or batch; any strides, channels contiguous), bf16 or fp32, each
    may be None.  norm: "layer" (weight, optional bias), "rms" (weight) or "none".  positions: int32 [tokens, axes] or
    [outer, tokens, axes]; one axis turns channels (i, i + 32), two turn the halves by a coordinate each; None: no
    rotation.  head_major: outputs are [heads, outer, tokens, 64], the layer's layout.  out: tensors of the output
    shapes to write (q, k, v), which may be the inputs themselves.  Returns (q, k, v), None where there was none.  Outputs
    of up to 256 KB together share one allocation: one that is kept (or saved) keeps all; clone it to keep it alone."""
    return _b.norm_rope(q, k, v, _norm(norm), eps, q_weight, q_bias, k_weight, k_bias, positions, rope_base, head_major, out,
                        stream)


def qk_norm_rope_backward(q, k, dq, dk, dv=None, *, norm="layer", eps=1e-5, q_weight=None, q_bias=None, k_weight=None,
                          k_bias=None, positions=None, rope_base=100.0, head_major=False, out=None, stream=None):
    """Gradients of qk_norm_rope(q, k, v, ...) from its outputs' gradients dq, dk, dv (each may be None; shaped like the
    outputs, float32 as the layer's backward gives them, or bfloat16 with bfloat16 inputs).

    Returns {"dq", "dk", "dv"} of the gradients' type, shaped like the inputs [outer, tokens, heads, 64] (or written
    to `out`), and float32 {"dq_weight", "dq_bias", "dk_weight", "dk_bias"}; None where there is none (a bias has a
    gradient when it is given).  q and k may be None with norm "none".  dq, dk and dv of up to 256 KB together share one
    allocation, and so do the four gradients of weights and biases."""
    return _b.norm_rope_backward(q, k, dq, dk, dv, _norm(norm), eps, q_weight, q_bias, k_weight, k_bias, positions, rope_base,
                                 head_major, out, stream)


def operator_status(device=None, stream=None) -> int:
    """Device status of the operators (synchronises the stream, returns the code and clears it): 0,
    GSA_ERR_DEVICE_BOUNDS (7) or GSA_ERR_DEVICE_TIMEOUT (6)."""
    with torch.cuda.device(device):
        st = torch.cuda.current_stream().cuda_stream if stream is None else stream
        fn = load_library().gsa_operator_status
        fn.argtypes, fn.restype = [ctypes.c_void_p], ctypes.c_int
        return fn(st or None)


class KVCache:
    """Pools of pages [num_pages, heads, page_size, 64] for keys and values.

    Which pages hold which sequence is the caller's block table, int32 [batch, max_pages]: token t of sequence b is row
    t % page_size of page block_table[b, t // page_size].  New tokens are packed, sequence after sequence:
    cu_tokens, int32 [batch + 1], has the first row of each (and the end)."""

    def __init__(self, num_pages, page_size, num_heads, dtype=torch.bfloat16, device="cuda"):
        shape = (num_pages, num_heads, page_size, HEAD_DIM)
        self._take(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device))

    @classmethod
    def from_pages(cls, k_pages, v_pages):
        """A cache over existing pools (shared, not copied)."""
        self = cls.__new__(cls)
        self._take(k_pages, v_pages)
        return self

    def _take(self, k_pages, v_pages):
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if (not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in (torch.bfloat16, torch.float32)
                    or t.dim() != 4 or t.shape[3] != HEAD_DIM or not t.is_contiguous()):
                raise GSAError(f"{name} must be a contiguous CUDA tensor [pages, heads, page_size, 64], bfloat16 or float32")
        if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype or k_pages.device != v_pages.device:
            raise GSAError("k_pages and v_pages must agree in shape, type and device")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.num_pages, self.num_heads, self.page_size = k_pages.shape[:3]
        self.dtype, self.device = k_pages.dtype, k_pages.device

    def append(self, k, v, block_table, start, cu_tokens, *, norm="none", eps=1e-5, k_weight=None, k_bias=None,
               positions=None, rope_axes=0, rope_base=10000.0, stream=None):
        """Write new tokens: k (normed and rotated on the way) and v, [tokens, heads, 64].  The first new token of
        sequence b becomes its token start[b].  positions: int32 [tokens, rope_axes]; None with one axis: a token's own
        place in its sequence.  Rows from cu_tokens[-1] on are not used."""
        _b.append(self.k_pages, self.v_pages, k, v, block_table, start, cu_tokens, _norm(norm), eps, k_weight, k_bias, positions,
                  rope_axes, rope_base, stream)

    def attention(self, q, block_table, lengths, cu_tokens, max_new, *, max_len=None, causal=True, softmax_scale=0.0,
                  return_lse=False, out=None, stream=None):
        """Attention of new tokens q [tokens, query heads, 64] over the cache: those of sequence b see its cached tokens
        0 .. lengths[b] - 1, or with `causal` (they are then its last ones) up to their own.  Query heads are a multiple
        of the cache's heads.  max_new: at least the most new tokens of a sequence.  max_len: about the longest of
        `lengths` (default: what the block table can hold); it only sets how the work is split.  softmax_scale 0: 1 / 8.
        Returns out (rows from cu_tokens[-1] on untouched), with return_lse also float32 [query heads, tokens] (columns
        from cu_tokens[-1] on not written)."""
        return _b.attention(self.k_pages, self.v_pages, q, block_table, lengths, cu_tokens, max_new, max_len, causal,
                            softmax_scale, return_lse, out, stream)
