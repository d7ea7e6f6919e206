"""The operators around the layer without a GPU: the oracle's gradients against
differences, and the refusals of the C entry points (all on the host, before any
CUDA call)."""
import ctypes
import struct

import numpy as np
import pytest

import sparse_global_attention_b200 as gsa
from oracle import operators_oracle as oo

P = 0x7f0000001000            # an aligned address; never read: every call here is refused


def _rows(ptr=P, heads=2, so=64 * 2 * 8, st=128, sh=64):
    return struct.pack("@Piqqq", ptr, heads, so, st, sh)


def _op(dtype=0, norm=1, eps=1e-5, axes=1, base=100.0):
    return struct.pack("@iifid", dtype, norm, eps, axes, base)


def _cache(k=P, v=P, dtype=0, pages=8, page=16, heads=2, table=P, batch=3, most=4, stride=4):
    return struct.pack("@PPiiiiPiiq", k, v, dtype, pages, page, heads, table, batch, most, stride)


def _fn(name, *args):
    fn = getattr(gsa.load_library(), name)
    p, q = ctypes.c_void_p, ctypes.c_int64
    fn.argtypes = {"gsa_qk_norm_rope": [p, q, q] + [p] * 11 + [q, p],
                   "gsa_qk_norm_rope_backward": [p, ctypes.c_int, q, q] + [p] * 11 + [q] + [p] * 5 + [q, p],
                   "gsa_cache_append": [p, p, q] + [p] * 8,
                   "gsa_cache_attention": [p, q, p, p, p, p, ctypes.c_int, q, ctypes.c_int, ctypes.c_float, p, p, q, p],
                   "gsa_cache_attention_workspace_bytes": [p, q, ctypes.c_int, ctypes.c_int, q]}[name]
    fn.restype = ctypes.c_size_t if name.endswith("bytes") else ctypes.c_int
    return fn(*args)


def _norm_rope(op=None, outer=2, tokens=8, q=_rows(), k=None, v=None, qo=_rows(), ko=None, vo=None, qw=P, qb=None,
               kw=None, kb=None, pos=P, pso=8):
    return _fn("gsa_qk_norm_rope", _op() if op is None else op, outer, tokens, q, k, v, qo, ko, vo, qw, qb, kw, kb, pos, pso, None)


@pytest.mark.parametrize("kw,code", [
    (dict(op=_op(dtype=2)), 1), (dict(op=_op(norm=3)), 1), (dict(op=_op(norm=-1)), 1), (dict(op=_op(eps=-1.0)), 1),
    (dict(op=_op(eps=float("nan"))), 1), (dict(op=_op(axes=3)), 1), (dict(op=_op(base=0.0)), 1),
    (dict(op=_op(base=float("inf"))), 1),
    (dict(q=None, qo=None), 1),                       # nothing to do
    (dict(qo=None), 1), (dict(k=_rows()), 1),         # an input without its output
    (dict(qw=None), 1), (dict(qw=P + 2), 1),          # the norm's weight is missing, not aligned
    (dict(op=_op(norm=2), qb=P), 1),                  # RMS has no bias
    (dict(pos=None), 1), (dict(pos=P + 2), 1), (dict(pso=-1), 1),
    (dict(op=_op(axes=0)), 1),                        # positions without a rotation
    (dict(q=_rows(P + 8)), 1), (dict(q=_rows(0)), 1), (dict(q=_rows(st=68)), 1), (dict(q=_rows(sh=-64)), 1),
    (dict(q=_rows(heads=0)), 1),
    (dict(qo=_rows(st=0)), 1), (dict(qo=_rows(so=0)), 1), (dict(qo=_rows(sh=0)), 1),   # rows written over one another
    (dict(qo=_rows(heads=3)), 2),
    (dict(outer=-1), 1), (dict(tokens=1 << 31), 1),
])
def test_norm_rope_refusals(kw, code):
    assert _norm_rope(**kw) == code


def test_empty_calls_do_nothing():
    assert _norm_rope(outer=0) == 0 and _norm_rope(tokens=0, q=_rows(0), qo=_rows(0)) == 0
    rows = _rows(0)
    assert _fn("gsa_cache_append", _cache(), _op(axes=0, norm=0), 0, rows, rows, None, None, None, None, None, None) == 0
    assert _fn("gsa_cache_append", _cache(batch=0), _op(axes=0, norm=0), 5, _rows(), _rows(), None, None, None, None, None, None) == 0
    assert _attention(tokens=0, q=rows, out=rows) == 0 and _attention(cache=_cache(batch=0)) == 0


def _backward(op=None, gdtype=1, outer=2, tokens=8, q=_rows(), k=None, go=(_rows(), None, None), gi=(_rows(), None, None),
              qw=P, kw=None, pos=P, pso=8, sums=(P, P, None, None), ws=P, nbytes=1 << 30):
    return _fn("gsa_qk_norm_rope_backward", _op() if op is None else op, gdtype, outer, tokens, q, k, *go, *gi, qw, kw, pos,
               pso, *sums, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(gdtype=2), 1), (dict(op=_op(dtype=1), gdtype=0), 1),      # bf16 gradients of fp32 inputs
    (dict(go=(None,) * 3, gi=(None,) * 3), 1), (dict(gi=(None,) * 3), 1),
    (dict(q=None), 1),                                              # the norm needs its input
    (dict(ws=None), 1), (dict(nbytes=100), 1), (dict(ws=P + 4), 1),
    (dict(sums=(None, None, P, None)), 1),                          # sums of a tensor that is not there
    (dict(op=_op(norm=0)), 1),                                      # sums without a norm
    (dict(op=_op(norm=2)), 1),                                      # a bias sum of RMS
    (dict(qw=None), 1), (dict(pos=None), 1),
    (dict(q=_rows(heads=3)), 2), (dict(gi=(_rows(heads=3), None, None)), 2),
    (dict(gi=(_rows(st=0), None, None)), 1),
])
def test_norm_rope_backward_refusals(kw, code):
    assert _backward(**kw) == code


def _append(cache=None, op=None, tokens=5, k=_rows(), v=_rows(), cu=P, start=P, w=P, b=None, pos=None):
    return _fn("gsa_cache_append", _cache() if cache is None else cache, _op() if op is None else op, tokens, k, v, cu, start, w,
               b, pos, None)


@pytest.mark.parametrize("kw,code", [
    (dict(cache=_cache(page=8)), 3), (dict(cache=_cache(page=48)), 3), (dict(cache=_cache(page=512)), 3),
    (dict(cache=_cache(pages=0)), 1), (dict(cache=_cache(heads=0)), 1), (dict(cache=_cache(k=0)), 1),
    (dict(cache=_cache(v=P + 4)), 1), (dict(cache=_cache(table=0)), 1), (dict(cache=_cache(stride=3)), 1),
    (dict(cache=_cache(dtype=1)), 1),                        # another type than the rows'
    (dict(cache=_cache(pages=1 << 30, page=256)), 3),
    (dict(k=None), 1), (dict(v=None), 1), (dict(cu=None), 1), (dict(start=None), 1), (dict(w=None), 1),
    (dict(k=_rows(heads=3)), 2), (dict(op=_op(axes=2)), 1),  # two axes need positions
    (dict(op=_op(axes=0), pos=P), 1), (dict(tokens=-1), 1),
])
def test_append_refusals(kw, code):
    assert _append(**kw) == code


def _attention(cache=None, tokens=5, q=_rows(heads=4), out=_rows(heads=4), cu=P, lens=P, most=5, length=64, causal=1,
               scale=0.0, lse=None, ws=None, nbytes=0):
    return _fn("gsa_cache_attention", _cache() if cache is None else cache, tokens, q, out, cu, lens, most, length, causal, scale,
               lse, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(cache=_cache(page=8)), 3), (dict(q=None), 1), (dict(out=None), 1), (dict(cu=None), 1), (dict(lens=None), 1),
    (dict(q=_rows(heads=3), out=_rows(heads=3)), 2), (dict(out=_rows(heads=2)), 2),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(most=-1), 1),
    (dict(length=-1), 1), (dict(out=_rows(heads=4, st=0)), 1), (dict(q=_rows(P + 2, heads=4)), 1),
    (dict(length=100000), 1),                                # split over keys without a workspace
    (dict(cache=_cache(batch=1 << 20), most=1 << 26, tokens=1 << 26), 3),
])
def test_attention_refusals(kw, code):
    assert _attention(**kw) == code


def test_attention_workspace_bytes():
    size = lambda cache, *a: _fn("gsa_cache_attention_workspace_bytes", cache, *a)
    assert size(_cache(), 3, 4, 1, 64) == 0                  # short: one part
    one = size(_cache(batch=1), 1, 4, 1, 100000)             # one token, a long cache: parts of 66 floats per head
    assert one > 0 and one % (4 * 66 * 4) == 0
    assert size(_cache(page=8), 1, 4, 1, 100000) == 0        # refused sizes
    assert size(_cache(batch=64), 64 * 2000, 4, 2000, 2000) == 0    # enough rows


def test_lengths_and_places_beyond_32_bits():
    size = lambda cache, *a: _fn("gsa_cache_attention_workspace_bytes", cache, *a)
    for batch in (1, 3):                                     # a length is never longer than 2^31 - 1
        assert size(_cache(batch=batch), batch, 4, 1, (1 << 63) - 1) == size(_cache(batch=batch), batch, 4, 1, (1 << 31) - 1) > 0
    wide = _cache(page=256, most=(1 << 23) - 1, stride=1 << 23)      # places up to 2^31 - 256 are one tile too many
    assert _append(cache=wide) == 3 and _attention(cache=wide) == 3


@pytest.mark.parametrize("call", [
    lambda: _append(cu=P + 2), lambda: _append(start=P + 1), lambda: _append(cache=_cache(table=P + 2)),
    lambda: _attention(cu=P + 2), lambda: _attention(lens=P + 2), lambda: _attention(lse=P + 2),
    lambda: _backward(sums=(P + 2, None, None, None)), lambda: _backward(sums=(P, P + 1, None, None))])
def test_arrays_of_32_bits_are_aligned(call):
    assert call() == 1


def test_softmax_scale_in_units_of_log2():
    """The kernels take the scale times log2(e), in 32 bits."""
    none = dict(tokens=0, q=_rows(0, heads=4), out=_rows(0, heads=4))
    assert _attention(scale=2.4e38, **none) == 1 and _attention(scale=3.4e38, **none) == 1
    assert _attention(scale=2.3e38, **none) == 0


@pytest.mark.parametrize("norm", ["none", "layer", "rms"])
@pytest.mark.parametrize("axes", [0, 1, 2])
def test_oracle_gradients_against_differences(norm, axes):
    rng = np.random.default_rng(axes)
    x, dy = rng.normal(size=(2, 3, 2, 64)) + 0.3, rng.normal(size=(2, 3, 2, 64))
    w, b = 1 + 0.2 * rng.normal(size=64), 0.1 * rng.normal(size=64)
    if norm == "none":
        w = b = None
    if norm == "rms":
        b = None
    pos = rng.integers(-5, 900, size=(2, 3, max(axes, 1)))
    f = lambda x, w, b: float((oo.norm_rope(x, norm, 1e-5, w, b, pos, axes, 50.0) * dy).sum())
    dx, dw, db = oo.norm_rope_backward(x, dy, norm, 1e-5, w, pos, axes, 50.0)
    h = 1e-5
    # central differences: truncation h^2 ~ 1e-10, rounding 1e-16 * |f| / h ~ 1e-9
    for at in [(0, 0, 0, 0), (1, 2, 1, 37), (0, 1, 1, 63), (1, 0, 0, 16)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w, b) - f(x - e, w, b)) / (2 * h) - dx[at]) < 1e-7
    for i in (0, 17, 63):
        e = np.zeros(64)
        e[i] = h
        if w is not None:
            assert abs((f(x, w + e, b) - f(x, w - e, b)) / (2 * h) - dw[i]) < 1e-7
        if b is not None:
            assert abs((f(x, w, b + e) - f(x, w, b - e)) / (2 * h) - db[i]) < 1e-7


def test_oracle_rotation_keeps_relative_positions():
    """Scores of rotated rows depend on the difference of the positions only."""
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(2, 64))
    for axes in (1, 2):
        turn = lambda x, p: oo.rotate(x, oo.rotation_angles(np.array(p)[:axes], axes, 100.0), axes)
        a = turn(q, [7, 3]) @ turn(k, [2, 9])
        b = turn(q, [1007, 503]) @ turn(k, [1002, 509])
        assert abs(a - b) < 1e-10
        assert abs(np.linalg.norm(turn(q, [12, 5])) - np.linalg.norm(q)) < 1e-12


def test_oracle_attention_over_pages_is_attention():
    rng = np.random.default_rng(1)
    n, length, size = 3, 21, 16
    k, v, q = rng.normal(size=(length, 1, 64)), rng.normal(size=(length, 1, 64)), rng.normal(size=(n, 2, 64))
    table = np.array([[2, 0]])
    kp, _ = oo.cache_append(np.full((3, 1, size, 64), np.nan), k, table, [0], [0, length])
    vp, left = oo.cache_append(np.full((3, 1, size, 64), np.nan), v, table, [0], [0, length])
    assert not left
    out, lse, _ = oo.cache_attention(q, kp, vp, table, [length], [0, n], True)
    for h in range(2):
        for i in range(n):
            s = k[:length - n + i + 1, 0] @ q[i, h] / 8
            p = np.exp(s - s.max())
            assert np.allclose(out[i, h], p @ v[:len(p), 0] / p.sum(), atol=1e-12)
            assert abs(lse[h, i] - (s.max() + np.log(p.sum()))) < 1e-12
