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

# A call of a few microseconds of GPU time is bounded by this file: the checks read each attribute once, the stream
# and device come as plain numbers, and a call on another device or stream takes a path of its own.
_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream

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


def _failed(rc, what):
    from . import _check
    _check(rc, what)


def _elsewhere(dev, stream, fn, *args, **kw):
    """The call with its device and stream current, so that what it allocates belongs to them."""
    with torch.cuda.device(dev):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(torch.cuda.ExternalStream(stream)):
            return fn(*args, **kw)


def _cuda_device(t, name):
    """Device number of a CUDA tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _fail(f"{name} must be a CUDA tensor")
    return t.get_device()


def _expect(t, name, dtype, dev):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.get_device() != dev:
        _fail(f"{name} must be a {dtype} tensor on cuda:{dev}, got "
              + (f"{t.dtype} on {t.device}" if isinstance(t, torch.Tensor) else repr(t)))


def _rows4(t, name, dtype, dev, shape=None, head_major=False):
    """gsa_rows of [outer, tokens, heads, 64] (head_major: [heads, outer, tokens, 64]), of that shape if given."""
    if t.dtype != dtype or t.get_device() != dev:
        _expect(t, name, dtype, dev)
    size = t.shape
    if len(size) != 4 or size[3] != HEAD_DIM or (shape is not None and size != shape):
        _fail(f"{name} must have shape {tuple(shape) if shape is not None else '[outer, tokens, heads, 64]'}, got {tuple(size)}")
    a, b, c, d = t.stride()
    if d != 1:
        _fail(f"{name}: the 64 channels must be contiguous")
    if head_major:
        return _rows(t.data_ptr(), size[0], b, c, a)
    return _rows(t.data_ptr(), size[2], a, b, c)


def _affine(t, name, dtype, dev):
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != dev:
        _expect(t, name, dtype, dev)
    if t.dim() != 1 or t.numel() != HEAD_DIM or not t.is_contiguous():
        _fail(f"{name} must be contiguous with shape ({HEAD_DIM},)")
    return t.data_ptr()


def _positions(t, outer, tokens, dev):
    """(pointer, stride of outer, axes) of int32 [tokens, axes] or [outer, tokens, axes]."""
    if t is None:
        return None, 0, 0
    _expect(t, "positions", torch.int32, dev)
    size, s = t.shape, t.stride()
    if len(size) == 2:
        n, axes = size
        sn, sa = s
        so = 0
    elif len(size) == 3:
        o, n, axes = size
        so, sn, sa = s
        if o != outer:
            n = -1
    else:
        n = axes = -1
    if n != tokens or axes not in (1, 2):
        _fail(f"positions must be [{tokens}, axes] or [{outer}, {tokens}, axes] with 1 or 2 axes, got {tuple(size)}")
    if (axes > 1 and sa != 1) or (n > 1 and sn != axes):
        _fail("positions: the tokens' coordinates must be contiguous")
    return t.data_ptr(), so, axes


def _norm_op(norm, eps, axes, base, dtype):
    if norm not in NORMS:
        _fail(f"norm must be one of {sorted(NORMS)}, got {norm!r}")
    return _op(dtype, NORMS[norm], eps, axes, base)


def qk_norm_rope(q, k=None, v=None, *, norm="layer", eps=1e-5, q_weight=None, q_bias=None, k_weight=None,
                 k_bias=None, positions=None, rope_base=100.0, head_major=False, out=None, stream=None):
    """Norm of queries and keys per head, then the position rotation, in one pass; values carried along.

    q, k, v: [outer, tokens, heads, 64] (outer: frames or batch; any strides, channels contiguous), bf16 or fp32, each
    may be None.  norm: "layer" (weight, optional bias), "rms" (weight) or "none".  positions: int32 [tokens, axes] or
    [outer, tokens, axes]; one axis turns channels (i, i + 32), two turn the halves by a coordinate each; None: no
    rotation.  head_major: outputs are [heads, outer, tokens, 64], the layer's layout.  out: tensors of the output
    shapes to write (q, k, v), which may be the inputs themselves.  Returns (q, k, v), None where there was none."""
    first = q if q is not None else k if k is not None else v
    dev = _cuda_device(first, "q, k, v")
    if stream is not None or _device() != dev:
        return _elsewhere(dev, stream, qk_norm_rope, q, k, v, norm=norm, eps=eps, q_weight=q_weight, q_bias=q_bias,
                          k_weight=k_weight, k_bias=k_bias, positions=positions, rope_base=rope_base,
                          head_major=head_major, out=out)
    dtype = first.dtype
    if dtype not in _DTYPES or first.dim() != 4:
        _fail(f"q, k, v must be bfloat16 or float32 [outer, tokens, heads, 64], got {dtype} {tuple(first.shape)}")
    outer, tokens = first.shape[:2]
    pos, pos_so, axes = _positions(positions, outer, tokens, dev)
    op = _norm_op(norm, eps, axes, rope_base, _DTYPES[dtype])
    rows_in, rows_out, res = [None] * 3, [None] * 3, [None] * 3
    for i, t in enumerate((q, k, v)):
        if t is None:
            continue
        rows_in[i] = _rows4(t, "qkv"[i], dtype, dev)
        o, n, heads, _ = t.shape
        if o != outer or n != tokens:
            _fail(f"{'qkv'[i]} must have {outer} x {tokens} tokens, got {o} x {n}")
        shape = (heads, outer, tokens, HEAD_DIM) if head_major else (outer, tokens, heads, HEAD_DIM)
        y = out[i] if out is not None else None
        if y is None:
            y = t.new_empty(shape)
            rows_out[i] = _rows(y.data_ptr(), heads, tokens * HEAD_DIM, HEAD_DIM, outer * tokens * HEAD_DIM) if head_major \
                else _rows(y.data_ptr(), heads, tokens * heads * HEAD_DIM, heads * HEAD_DIM, HEAD_DIM)
        else:
            rows_out[i] = _rows4(y, "qkv"[i] + " output", dtype, dev, shape, head_major)
        res[i] = y
    rc = _lib().gsa_qk_norm_rope(op, outer, tokens, *rows_in, *rows_out, _affine(q_weight, "q_weight", dtype, dev),
                                 _affine(q_bias, "q_bias", dtype, dev), _affine(k_weight, "k_weight", dtype, dev),
                                 _affine(k_bias, "k_bias", dtype, dev), pos, pos_so, _current_stream(dev))
    if rc:
        _failed(rc, "gsa_qk_norm_rope")
    return tuple(res)


_bwd_bytes = None


def qk_norm_rope_backward(q, k, dq, dk, dv=None, *, norm="layer", eps=1e-5, q_weight=None, q_bias=None, k_weight=None,
                          k_bias=None, positions=None, rope_base=100.0, head_major=False, out=None, stream=None):
    """Gradients of qk_norm_rope(q, k, v, ...) from its outputs' gradients dq, dk, dv (each may be None; shaped like the
    outputs, float32 as the layer's backward gives them, or bfloat16 with bfloat16 inputs).

    Returns {"dq", "dk", "dv"} of the gradients' type, shaped like the inputs [outer, tokens, heads, 64] (or written
    to `out`), and float32 {"dq_weight", "dq_bias", "dk_weight", "dk_bias"}; None where there is none (a bias has a
    gradient when it is given).  q and k may be None with norm "none"."""
    global _bwd_bytes
    first = dq if dq is not None else dk if dk is not None else dv
    dev = _cuda_device(first, "dq, dk, dv")
    if stream is not None or _device() != dev:
        return _elsewhere(dev, stream, qk_norm_rope_backward, q, k, dq, dk, dv, norm=norm, eps=eps, q_weight=q_weight,
                          q_bias=q_bias, k_weight=k_weight, k_bias=k_bias, positions=positions, rope_base=rope_base,
                          head_major=head_major, out=out)
    gtype = first.dtype
    x = (None if dq is None else q, None if dk is None else k)
    dtype = x[0].dtype if x[0] is not None else x[1].dtype if x[1] is not None else gtype
    if gtype not in _DTYPES or dtype not in _DTYPES or first.dim() != 4:
        _fail(f"inputs and gradients must be bfloat16 or float32 with four dimensions, got {dtype}, {gtype} {tuple(first.shape)}")
    outer, tokens = first.shape[1:3] if head_major else first.shape[:2]
    normed = norm != "none"
    pos, pos_so, axes = _positions(positions, outer, tokens, dev)
    op = _norm_op(norm, eps, axes, rope_base, _DTYPES[dtype])
    rows_x, rows_go, rows_gi = [None] * 2, [None] * 3, [None] * 3
    names = ("dq", "dk", "dv")
    res = {}
    for i, t in enumerate((dq, dk, dv)):
        res[names[i]] = None
        if t is None:
            continue
        rows_go[i] = _rows4(t, names[i], gtype, dev, None, head_major)
        size = t.shape
        heads = size[0] if head_major else size[2]
        if (size[1:3] if head_major else size[:2]) != (outer, tokens):
            _fail(f"{names[i]} must be of {outer} x {tokens} tokens, got {tuple(size)}")
        like = (outer, tokens, heads, HEAD_DIM)
        if i < 2 and normed:
            if x[i] is None:
                _fail(f"{names[i]} needs its input {names[i][1]}")
            rows_x[i] = _rows4(x[i], names[i][1], dtype, dev, like)
        y = out[i] if out is not None else None
        if y is None:
            y = t.new_empty(like)
            rows_gi[i] = _rows(y.data_ptr(), heads, tokens * heads * HEAD_DIM, heads * HEAD_DIM, HEAD_DIM)
        else:
            rows_gi[i] = _rows4(y, names[i] + " output", gtype, dev, like)
        res[names[i]] = y
    sums, nbytes, ws = [None] * 4, 0, None
    if normed:
        wanted = (dq is not None, dq is not None and q_bias is not None, dk is not None, dk is not None and k_bias is not None)
        sums = [torch.empty(HEAD_DIM, dtype=torch.float32, device=first.device) if n else None for n in wanted]
        if _bwd_bytes is None:
            _bwd_bytes = _lib().gsa_qk_norm_rope_workspace_bytes()
        nbytes = _bwd_bytes
        ws = torch.empty(nbytes, dtype=torch.uint8, device=first.device)
    res["dq_weight"], res["dq_bias"], res["dk_weight"], res["dk_bias"] = sums
    rc = _lib().gsa_qk_norm_rope_backward(
        op, _DTYPES[gtype], outer, tokens, *rows_x, *rows_go, *rows_gi, _affine(q_weight, "q_weight", dtype, dev),
        _affine(k_weight, "k_weight", dtype, dev), pos, pos_so, *[t.data_ptr() if t is not None else None for t in sums],
        ws.data_ptr() if ws is not None else None, nbytes, _current_stream(dev))
    if rc:
        _failed(rc, "gsa_qk_norm_rope_backward")
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
            _cuda_device(t, name)
            if t.dtype not in _DTYPES or t.dim() != 4 or t.shape[3] != HEAD_DIM or not t.is_contiguous():
                _fail(f"{name} must be contiguous [pages, heads, page_size, 64], bfloat16 or float32, got {t.dtype} {tuple(t.shape)}")
        if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype or k_pages.device != v_pages.device:
            _fail("k_pages and v_pages must agree in shape, type and device")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.num_pages, self.num_heads, self.page_size = k_pages.shape[:3]
        self.dtype, self.device = k_pages.dtype, k_pages.device
        self._dev = k_pages.get_device()

    def _struct(self, table):
        _expect(table, "block_table", torch.int32, self._dev)
        size = table.shape
        if len(size) != 2 or (size[1] > 1 and table.stride(1) != 1):
            _fail("block_table must be [batch, max_pages] with contiguous rows")
        batch, most = size
        return _cache(self.k_pages.data_ptr(), self.v_pages.data_ptr(), _DTYPES[self.dtype], self.num_pages, self.page_size,
                      self.num_heads, table.data_ptr(), batch, most, table.stride(0)), batch, most

    def _ints(self, t, name, n):
        _expect(t, name, torch.int32, self._dev)
        if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
            _fail(f"{name} must be contiguous int32 [{n}]")
        return t.data_ptr()

    def _rows3(self, t, name, shape=None):
        _expect(t, name, self.dtype, self._dev)
        size = t.shape
        if len(size) != 3 or size[2] != HEAD_DIM or (shape is not None and size != shape):
            _fail(f"{name} must have shape {shape if shape is not None else '[tokens, heads, 64]'}, got {tuple(size)}")
        a, b, c = t.stride()
        if c != 1:
            _fail(f"{name}: the 64 channels must be contiguous")
        return _rows(t.data_ptr(), size[1], 0, a, b)

    def append(self, k, v, block_table, start, cu_tokens, *, norm="none", eps=1e-5, k_weight=None, k_bias=None,
               positions=None, rope_axes=0, rope_base=10000.0, stream=None):
        """Write new tokens: k (normed and rotated on the way) and v, [tokens, heads, 64].  The first new token of
        sequence b becomes its token start[b].  positions: int32 [tokens, rope_axes]; None with one axis: a token's own
        place in its sequence.  Rows from cu_tokens[-1] on are not used."""
        dev = self._dev
        if stream is not None or _device() != dev:
            return _elsewhere(dev, stream, self.append, k, v, block_table, start, cu_tokens, norm=norm, eps=eps,
                              k_weight=k_weight, k_bias=k_bias, positions=positions, rope_axes=rope_axes, rope_base=rope_base)
        cache, batch, _ = self._struct(block_table)
        rk = self._rows3(k, "k")
        rv = self._rows3(v, "v", k.shape)
        tokens = k.shape[0]
        pos, _, axes = _positions(positions, 1, tokens, dev)
        if pos is not None and axes != rope_axes:
            _fail(f"positions have {axes} axes, rope_axes is {rope_axes}")
        rc = _lib().gsa_cache_append(cache, _norm_op(norm, eps, rope_axes, rope_base, _DTYPES[self.dtype]), tokens, rk, rv,
                                     self._ints(cu_tokens, "cu_tokens", batch + 1), self._ints(start, "start", batch),
                                     _affine(k_weight, "k_weight", self.dtype, dev), _affine(k_bias, "k_bias", self.dtype, dev),
                                     pos, _current_stream(dev))
        if rc:
            _failed(rc, "gsa_cache_append")

    def attention(self, q, block_table, lengths, cu_tokens, max_new, *, max_len=None, causal=True, softmax_scale=0.0,
                  return_lse=False, out=None, stream=None):
        """Attention of new tokens q [tokens, query heads, 64] over the cache: those of sequence b see its cached tokens
        0 .. lengths[b] - 1, or with `causal` (they are then its last ones) up to their own.  Query heads are a multiple
        of the cache's heads.  max_new: at least the most new tokens of a sequence.  max_len: about the longest of
        `lengths` (default: what the block table can hold); it only sets how the work is split.  softmax_scale 0: 1 / 8.
        Returns out (rows from cu_tokens[-1] on untouched), with return_lse also float32 [query heads, tokens]."""
        dev = self._dev
        if stream is not None or _device() != dev:
            return _elsewhere(dev, stream, self.attention, q, block_table, lengths, cu_tokens, max_new, max_len=max_len,
                              causal=causal, softmax_scale=softmax_scale, return_lse=return_lse, out=out)
        cache, batch, most = self._struct(block_table)
        rq = self._rows3(q, "q")
        tokens, heads, _ = q.shape
        if max_len is None:
            max_len = most * self.page_size
        if out is None:
            out = q.new_empty((tokens, heads, HEAD_DIM))
            ro = _rows(out.data_ptr(), heads, 0, heads * HEAD_DIM, HEAD_DIM)
        else:
            ro = self._rows3(out, "out", q.shape)
        lse = torch.empty((heads, tokens), dtype=torch.float32, device=self.device) if return_lse else None
        lib = _lib()
        nbytes = lib.gsa_cache_attention_workspace_bytes(cache, tokens, heads, max_new, max_len)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None
        rc = lib.gsa_cache_attention(cache, tokens, rq, ro, self._ints(cu_tokens, "cu_tokens", batch + 1),
                                     self._ints(lengths, "lengths", batch), max_new, max_len, int(bool(causal)),
                                     softmax_scale, lse.data_ptr() if return_lse else None,
                                     ws.data_ptr() if nbytes else None, nbytes, _current_stream(dev))
        if rc:
            _failed(rc, "gsa_cache_attention")
        return (out, lse) if return_lse else out
