"""Operators around the layer: norms of queries and keys with the position
rotation (and its gradients), and a paged cache of keys and values with the
attention of new tokens over it.

Like GSALayer these pass torch tensors' pointers to the C entry points
(include/gsa.h, "operators around the layer"); all arithmetic runs in the CUDA
kernels.  Calls go to the current stream of the tensors' device, or to `stream`
(a raw handle).  Outputs and workspaces are allocated for that stream, one per
call, so that calls in flight and captured graphs share none.  There is no
autograd: gradients are calls of their own.  What the device finds wrong
(a page outside the pool, a place without a page) is reported by
operator_status().
"""
from __future__ import annotations

import ctypes
import struct

import torch

HEAD_DIM = 64
NORMS = {"none": 0, "layer": 1, "rms": 2}
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}

# the argument structures of include/gsa.h, packed with native alignment
_rows = struct.Struct("@Piqqq").pack        # gsa_rows
_op = struct.Struct("@iifid").pack          # gsa_norm_rope
_cache = struct.Struct("@PPiiiiPiiq").pack  # gsa_kv_cache

_fns = None


def _lib():
    global _fns
    if _fns is None:
        from . import load_library
        lib = load_library()
        p, i, q = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        sig = {"gsa_qk_norm_rope": (i, [p, q, q] + [p] * 6 + [p] * 4 + [p, q, p]),
               "gsa_qk_norm_rope_backward": (i, [p, i, q, q] + [p] * 8 + [p] * 2 + [p, q] + [p] * 4 + [p, q, p]),
               "gsa_qk_norm_rope_workspace_bytes": (ctypes.c_size_t, []),
               "gsa_cache_append": (i, [p, p, q, p, p, p, p, p, p, p, p]),
               "gsa_cache_attention": (i, [p, q, p, p, p, p, i, q, i, ctypes.c_float, p, p, q, p]),
               "gsa_cache_attention_workspace_bytes": (ctypes.c_size_t, [p, q, i, i, q]),
               "gsa_operator_status": (i, [p])}
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _fns = lib
    return _fns


def _fail(msg):
    from . import GSAError
    raise GSAError(msg)


def _check(rc, what):
    if rc:
        from . import _check as check
        check(rc, what)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _same(t, name, dtype, device):
    if t.dtype != dtype or t.device != device:
        _fail(f"{name} must be {dtype} on {device}, got {t.dtype} on {t.device}")


class _On:
    """The device and stream of one call: makes them current while outputs and
    workspaces are allocated and the kernels launched."""

    def __init__(self, device, stream):
        self.inner = []
        if torch.cuda.current_device() != device.index:
            self.inner.append(torch.cuda.device(device))
        self.device, self.stream = device, stream

    def __enter__(self):
        for c in self.inner:
            c.__enter__()
        now = torch.cuda.current_stream(self.device).cuda_stream
        if self.stream is not None and self.stream != now:
            s = torch.cuda.stream(torch.cuda.ExternalStream(self.stream, device=self.device))
            s.__enter__()
            self.inner.append(s)
            now = self.stream
        return now or None

    def __exit__(self, *exc):
        for c in reversed(self.inner):
            c.__exit__(*exc)
        return False


def _first(*tensors):
    for t in tensors:
        if t is not None:
            return t
    _fail("nothing to do: every tensor is None")


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _fail(f"{name} must be a CUDA tensor")


def _rows4(t, name, dtype, device, shape, head_major):
    """gsa_rows of [outer][tokens][heads][64] (or [heads][outer][tokens][64])."""
    _same(t, name, dtype, device)
    if tuple(t.shape) != shape:
        _fail(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    s = t.stride()
    if s[3] != 1:
        _fail(f"{name}: the 64 channels must be contiguous")
    if head_major:
        return _rows(t.data_ptr(), shape[0], s[1], s[2], s[0])
    return _rows(t.data_ptr(), shape[2], s[0], s[1], s[2])


def _affine(t, name, dtype, device):
    if t is None:
        return None
    _same(t, name, dtype, device)
    if t.shape != (HEAD_DIM,) or not t.is_contiguous():
        _fail(f"{name} must be contiguous with shape ({HEAD_DIM},)")
    return t.data_ptr()


def _positions(t, outer, tokens, device):
    """(pointer, stride of outer, axes) of int32 [tokens][axes] or [outer][tokens][axes]."""
    if t is None:
        return None, 0, 0
    _same(t, "positions", torch.int32, device)
    shape, s = tuple(t.shape), t.stride()
    if len(shape) == 2:
        shape, s = (outer,) + shape, (0,) + s
    if len(shape) != 3 or shape[:2] != (outer, tokens) or shape[2] not in (1, 2):
        _fail(f"positions must be [tokens, axes] or [outer, tokens, axes] with 1 or 2 axes, got {tuple(t.shape)}")
    axes = shape[2]
    if (axes > 1 and s[2] != 1) or (tokens > 1 and s[1] != axes):
        _fail("positions: the tokens' coordinates must be contiguous")
    return t.data_ptr(), s[0], axes


def _norm_op(norm, eps, axes, base, dtype):
    if norm not in NORMS:
        _fail(f"norm must be one of {sorted(NORMS)}, got {norm!r}")
    return _op(dtype, NORMS[norm], eps, axes, base)


def _shape4(t, name, head_major=False):
    _cuda(t, name)
    if t.dim() != 4 or t.shape[3] != HEAD_DIM:
        _fail(f"{name} must have four dimensions, the last of {HEAD_DIM}, got {tuple(t.shape)}")
    return tuple(t.shape)


def qk_norm_rope(q, k=None, v=None, *, norm="layer", eps=1e-5, q_weight=None, q_bias=None, k_weight=None,
                 k_bias=None, positions=None, rope_base=100.0, head_major=False, out=None, stream=None):
    """Norm of queries and keys per head, then the position rotation, in one pass; values carried along.

    q, k, v: [outer, tokens, heads, 64] (outer: frames or batch; any strides, channels contiguous), bf16 or fp32, each
    may be None.  norm: "layer" (weight, optional bias), "rms" (weight) or "none".  positions: int32 [tokens, axes] or
    [outer, tokens, axes]; one axis turns channels (i, i + 32), two turn the halves by a coordinate each; None: no
    rotation.  head_major: outputs are [heads, outer, tokens, 64], the layer's layout.  out: tensors of the output
    shapes to write (q, k, v), which may be the inputs themselves.  Returns (q, k, v), None where there was none."""
    first = _first(q, k, v)
    outer, tokens = _shape4(first, "q, k, v")[:2]
    dtype, device = first.dtype, first.device
    if dtype not in _DTYPES:
        _fail(f"q, k, v must be bfloat16 or float32, got {dtype}")
    op_in, op_out, res = [None] * 3, [None] * 3, [None] * 3
    pos, pos_so, axes = _positions(positions, outer, tokens, device)
    op = _norm_op(norm, eps, axes, rope_base, _DTYPES[dtype])
    with _On(device, stream) as st:
        for i, t in enumerate((q, k, v)):
            if t is None:
                continue
            name = "qkv"[i]
            heads = _shape4(t, name)[2]
            op_in[i] = _rows4(t, name, dtype, device, (outer, tokens, heads, HEAD_DIM), False)
            shape = (heads, outer, tokens, HEAD_DIM) if head_major else (outer, tokens, heads, HEAD_DIM)
            o = out[i] if out is not None and out[i] is not None else torch.empty(shape, dtype=dtype, device=device)
            op_out[i] = _rows4(o, name + " output", dtype, device, shape, head_major)
            res[i] = o
        _check(_lib().gsa_qk_norm_rope(op, outer, tokens, *op_in, *op_out, _affine(q_weight, "q_weight", dtype, device),
                                       _affine(q_bias, "q_bias", dtype, device), _affine(k_weight, "k_weight", dtype, device),
                                       _affine(k_bias, "k_bias", dtype, device), pos, pos_so, st), "gsa_qk_norm_rope")
    return tuple(res)


def qk_norm_rope_backward(q, k, dq, dk, dv=None, *, norm="layer", eps=1e-5, q_weight=None, q_bias=None, k_weight=None,
                          k_bias=None, positions=None, rope_base=100.0, head_major=False, out=None, stream=None):
    """Gradients of qk_norm_rope(q, k, v, ...) from its outputs' gradients dq, dk, dv (each may be None; shaped like the
    outputs, float32 as the layer's backward gives them, or bfloat16 with bfloat16 inputs).

    Returns {"dq", "dk", "dv"} of the gradients' type, shaped like the inputs [outer, tokens, heads, 64] (or written
    to `out`), and float32 {"dq_weight", "dq_bias", "dk_weight", "dk_bias"}; None where there is none (a bias has a
    gradient when it is given).  q and k may be None with norm "none"."""
    first = _first(dq, dk, dv)
    shape = _shape4(first, "dq, dk, dv")
    outer, tokens = shape[1:3] if head_major else shape[:2]
    gtype, device = first.dtype, first.device
    x = [None if dq is None else q, None if dk is None else k]
    dtype = next((t.dtype for t in x if t is not None), gtype)
    if gtype not in _DTYPES or dtype not in _DTYPES:
        _fail(f"inputs and gradients must be bfloat16 or float32, got {dtype} and {gtype}")
    pos, pos_so, axes = _positions(positions, outer, tokens, device)
    op = _norm_op(norm, eps, axes, rope_base, _DTYPES[dtype])
    rows_x, rows_go, rows_gi = [None] * 2, [None] * 3, [None] * 3
    names = ("dq", "dk", "dv")
    res = dict.fromkeys(names + ("dq_weight", "dq_bias", "dk_weight", "dk_bias"))
    with _On(device, stream) as st:
        for i, t in enumerate((dq, dk, dv)):
            if t is None:
                continue
            s = _shape4(t, names[i])
            heads = s[0] if head_major else s[2]
            like = (outer, tokens, heads, HEAD_DIM)
            rows_go[i] = _rows4(t, names[i], gtype, device, (heads, outer, tokens, HEAD_DIM) if head_major else like, head_major)
            if i < 2 and norm != "none":
                if x[i] is None:
                    _fail(f"{names[i]} needs its input {names[i][1]}")
                _cuda(x[i], names[i][1])
                rows_x[i] = _rows4(x[i], names[i][1], dtype, device, like, False)
            o = out[i] if out is not None and out[i] is not None else torch.empty(like, dtype=gtype, device=device)
            rows_gi[i] = _rows4(o, names[i] + " output", gtype, device, like, False)
            res[names[i]] = o
        if norm != "none":
            sums = torch.empty(4, HEAD_DIM, dtype=torch.float32, device=device)
            wanted = (dq is not None, dq is not None and q_bias is not None, dk is not None,
                      dk is not None and k_bias is not None)
            for i, name in enumerate(("dq_weight", "dq_bias", "dk_weight", "dk_bias")):
                if wanted[i]:
                    res[name] = sums[i]
        nbytes = _lib().gsa_qk_norm_rope_workspace_bytes() if norm != "none" else 0
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _check(_lib().gsa_qk_norm_rope_backward(
            op, _DTYPES[gtype], outer, tokens, *rows_x, *rows_go, *rows_gi, _affine(q_weight, "q_weight", dtype, device),
            _affine(k_weight, "k_weight", dtype, device), pos, pos_so, _ptr(res["dq_weight"]), _ptr(res["dq_bias"]),
            _ptr(res["dk_weight"]), _ptr(res["dk_bias"]), ws.data_ptr() or None, nbytes, st), "gsa_qk_norm_rope_backward")
    return res


def operator_status(device=None, stream=None) -> int:
    """Device status of the operators (synchronises the stream, returns the code and clears it): 0,
    GSA_ERR_DEVICE_BOUNDS (7) or GSA_ERR_DEVICE_TIMEOUT (6)."""
    with torch.cuda.device(device):
        st = torch.cuda.current_stream().cuda_stream if stream is None else stream
        return _lib().gsa_operator_status(st or None)


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
            _shape4(t, name)
            if t.dtype not in _DTYPES or not t.is_contiguous():
                _fail(f"{name} must be contiguous, bfloat16 or float32")
        if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype or k_pages.device != v_pages.device:
            _fail("k_pages and v_pages must agree in shape, type and device")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.num_pages, self.num_heads, self.page_size = k_pages.shape[:3]
        self.dtype, self.device = k_pages.dtype, k_pages.device

    def _struct(self, block_table):
        _same(block_table, "block_table", torch.int32, self.device)
        if block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
            _fail("block_table must be [batch, max_pages] with contiguous rows")
        batch, most = block_table.shape
        return _cache(self.k_pages.data_ptr(), self.v_pages.data_ptr(), _DTYPES[self.dtype], self.num_pages, self.page_size,
                      self.num_heads, block_table.data_ptr(), batch, most, block_table.stride(0)), batch

    def _ints(self, t, name, n):
        _same(t, name, torch.int32, self.device)
        if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
            _fail(f"{name} must be contiguous int32 [{n}]")
        return t.data_ptr()

    def _rows3(self, t, name, tokens=None, heads=None):
        _cuda(t, name)
        _same(t, name, self.dtype, self.device)
        shape, s = t.shape, t.stride()
        if len(shape) != 3 or shape[2] != HEAD_DIM or (shape[1] > 0 and s[2] != 1):
            _fail(f"{name} must be [tokens, heads, {HEAD_DIM}] with contiguous channels, got {tuple(shape)}")
        if (tokens is not None and shape[0] != tokens) or (heads is not None and shape[1] != heads):
            _fail(f"{name} must be [{tokens}, {heads}, {HEAD_DIM}], got {tuple(shape)}")
        return _rows(t.data_ptr(), shape[1], 0, s[0], s[1])

    def append(self, k, v, block_table, start, cu_tokens, *, norm="none", eps=1e-5, k_weight=None, k_bias=None,
               positions=None, rope_axes=0, rope_base=10000.0, stream=None):
        """Write new tokens: k (normed and rotated on the way) and v, [tokens, heads, 64].  The first new token of
        sequence b becomes its token start[b].  positions: int32 [tokens, rope_axes]; None with one axis: a token's own
        place in its sequence.  Rows from cu_tokens[-1] on are not used."""
        cache, batch = self._struct(block_table)
        rk = self._rows3(k, "k")
        tokens, heads = k.shape[:2]
        rv = self._rows3(v, "v", tokens, heads)
        pos, _, axes = _positions(positions, 1, tokens, self.device)
        if pos is not None and axes != rope_axes:
            _fail(f"positions have {axes} axes, rope_axes is {rope_axes}")
        op = _norm_op(norm, eps, rope_axes, rope_base, _DTYPES[self.dtype])
        with _On(self.device, stream) as st:
            _check(_lib().gsa_cache_append(cache, op, tokens, rk, rv, self._ints(cu_tokens, "cu_tokens", batch + 1),
                                           self._ints(start, "start", batch), _affine(k_weight, "k_weight", self.dtype, self.device),
                                           _affine(k_bias, "k_bias", self.dtype, self.device), pos, st), "gsa_cache_append")

    def attention(self, q, block_table, lengths, cu_tokens, max_new, *, max_len=None, causal=True, softmax_scale=0.0,
                  return_lse=False, out=None, stream=None):
        """Attention of new tokens q [tokens, query heads, 64] over the cache: those of sequence b see its cached tokens
        0 .. lengths[b] - 1, or with `causal` (they are then its last ones) up to their own.  Query heads are a multiple
        of the cache's heads.  max_new: at least the most new tokens of a sequence.  max_len: about the longest of
        `lengths` (default: what the block table can hold); it only sets how the work is split.  softmax_scale 0: 1 / 8.
        Returns out (rows from cu_tokens[-1] on untouched), with return_lse also float32 [query heads, tokens]."""
        cache, batch = self._struct(block_table)
        rq = self._rows3(q, "q")
        tokens, heads = q.shape[:2]
        if max_len is None:
            max_len = block_table.shape[1] * self.page_size
        with _On(self.device, stream) as st:
            if out is None:
                out = torch.empty((tokens, heads, HEAD_DIM), dtype=self.dtype, device=self.device)
            ro = self._rows3(out, "out", tokens, heads)
            lse = torch.empty((heads, tokens), dtype=torch.float32, device=self.device) if return_lse else None
            lib = _lib()
            nbytes = lib.gsa_cache_attention_workspace_bytes(cache, tokens, heads, max_new, max_len)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None
            _check(lib.gsa_cache_attention(cache, tokens, rq, ro, self._ints(cu_tokens, "cu_tokens", batch + 1),
                                           self._ints(lengths, "lengths", batch), max_new, max_len, int(bool(causal)),
                                           softmax_scale, _ptr(lse), _ptr(ws), nbytes, st), "gsa_cache_attention")
        return (out, lse) if return_lse else out
