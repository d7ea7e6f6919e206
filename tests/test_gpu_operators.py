"""The operators around the layer on the GPU against the float64 oracle.

Tolerances (u = 2^-24, half a step of fp32; r = half a step of the output type,
finfo.eps / 2: 2^-8 for bf16, u for fp32):
  * norm and rotation: every intermediate is fp32.  A row's mean and variance
    are sums of 64 terms in chains of 8 + 3 additions; with |mean| <= 4 times the
    row's deviation (the inputs here) the centred values are off by at most
    11 u * 5 + u of a deviation, the factor by 20 u, weight, bias and the
    rotation's products by 8 u, cos and sin by 2^-22 = 4 u: under 128 u of the
    largest value that a row can hold, M = sqrt(64) max|w| + max|b| (no norm: the
    row's largest |x|), times sqrt 2 for the pair.  Bound: 256 u M + r |want|.
  * its gradients: the same count on g, u = g w and the two means, each taken
    with absolute values: 512 u s (|u| + mean|u| + |h| mean|u h|) + r |want|
    (the normalised row's own error of 100 u enters twice).  Weight sums of N rows:
    chains of at most N additions of terms that are off by 200 u:
    (256 + N) u sum|term|.
  * attention: a score is a sum of 64 products, off by 64 u A with A the largest
    sum|q k| scale; the exponential by 2^-22 + u (1 + |score|); so weights by
    (128 (1 + A)) u relative, bf16 weights by 2^-8 more (they are rounded for the
    product; the sum is not), and a sum over n keys in fp32 by n u at the most:
    bound (128 (1 + A) u + n u [+ 2^-8]) * sum p|v| / sum p + r |want|.
    lse: (128 (1 + A) + n) u + 4 u |lse|.
"""
import numpy as np
import pytest
import torch

import oracle
import sparse_global_attention_b200 as gsa
from gsa_inputs import GSAConfig, make_inputs
from oracle import operators_oracle as oo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def clean():
    assert gsa.operator_status() == 0


def assert_within(name, got, want, tol):
    err = np.abs(got - want)
    bad = ~(err <= tol) & ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} values off, worst {np.max(err[bad])} "
                           f"against {np.broadcast_to(tol, err.shape)[bad].flat[0]}")


# ---- norm and rotation ------------------------------------------------------------------
def norm_inputs(g, outer, tokens, hq, hk, dtype, norm, axes, far=False):
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = {"q": (rand(outer, tokens, hq, 64) * 1.5 + 0.3).to(dtype), "k": (rand(outer, tokens, hk, 64) - 0.2).to(dtype),
         "v": rand(outer, tokens, hk, 64).to(dtype)}
    w = {}
    if norm != "none":
        w = {n: (1 + 0.3 * rand(64)).to(dtype) for n in ("q_weight", "k_weight")}
    if norm == "layer":
        w.update({n: (0.2 * rand(64)).to(dtype) for n in ("q_bias", "k_bias")})
    pos = None
    if axes:
        lo, hi = (-2 ** 31, 2 ** 31) if far else (-3, 4000)
        pos = torch.randint(lo, hi, (outer, tokens, axes), generator=g, device="cuda").to(torch.int32)
    return x, w, pos


def check_norm_rope(x, w, pos, norm, axes, base, got, dtype, eps):
    for a in ("q", "k"):
        if x.get(a) is None:
            continue
        xa, wa, ba = f64(x[a]), f64(w.get(a + "_weight")), f64(w.get(a + "_bias"))
        want = oo.norm_rope(xa, norm, eps, wa, ba, f64(pos), axes, base)
        big = (8 * np.abs(wa).max() + (0 if ba is None else np.abs(ba).max())) if norm != "none" \
            else np.abs(xa).max(-1, keepdims=True)
        assert_within(a, f64(got[a]), want, 256 * U * big + half_step(dtype) * np.abs(want))
    if x.get("v") is not None:
        assert torch.equal(got["v"], x["v"])


@pytest.mark.parametrize("axes", [0, 1, 2])
@pytest.mark.parametrize("norm", ["none", "layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("outer,tokens,hq,hk", [(1, 1, 1, 1), (2, 37, 6, 2), (3, 9, 21, 7)])
def test_norm_rope(outer, tokens, hq, hk, dtype, norm, axes):
    g = torch.Generator(device="cuda").manual_seed(outer * 100 + tokens)
    dt = TYPES[dtype]
    x, w, pos = norm_inputs(g, outer, tokens, hq, hk, dt, norm, axes)
    for head_major in (False, True):
        q, k, v = gsa.qk_norm_rope(x["q"], x["k"], x["v"], norm=norm, eps=1e-5, positions=pos, rope_base=100.0,
                                   head_major=head_major, **w)
        back = (lambda t: t.permute(1, 2, 0, 3)) if head_major else (lambda t: t)
        assert q.is_contiguous()
        check_norm_rope(x, w, pos, norm, axes, 100.0, {"q": back(q), "k": back(k), "v": back(v)}, dt, 1e-5)
    clean()


@pytest.mark.parametrize("norm,axes", [("none", 2), ("layer", 2), ("rms", 1), ("layer", 0), ("rms", 2), ("layer", 1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (6, 2), (21, 7)])
def test_norm_rope_of_many_tokens(hq, hk, dtype, norm, axes):
    """More tokens than warps: every group of lanes has a token of its own; a count that no four divide."""
    test_norm_rope(3, 1201, hq, hk, dtype, norm, axes)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_rope_of_many_tokens_in_place_and_with_strides(dtype):
    g = torch.Generator(device="cuda").manual_seed(9)
    dt, n = TYPES[dtype], 2501
    y = torch.randn(2, n, 7, 64, generator=g, device="cuda").to(dt)
    w = {a: (1 + 0.2 * torch.randn(64, generator=g, device="cuda")).to(dt) for a in ("q_weight", "k_weight")}
    pos = torch.randint(0, 40, (n, 2), generator=g, device="cuda", dtype=torch.int32)
    x = y.clone()
    gsa.qk_norm_rope(y[:, :, :5], y[:, :, 5:6], norm="rms", positions=pos, out=(y[:, :, :5], y[:, :, 5:6], None), **w)
    check_norm_rope({"q": x[:, :, :5], "k": x[:, :, 5:6]}, w, pos[None].expand(2, n, 2), "rms", 2, 100.0,
                    {"q": y[:, :, :5], "k": y[:, :, 5:6]}, dt, 1e-5)
    assert torch.equal(y[:, :, 6], x[:, :, 6])
    clean()


@pytest.mark.parametrize("axes", [1, 2])
def test_positions_at_the_ends_of_their_range(axes):
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w, pos = norm_inputs(g, 2, 64, 2, 2, torch.float32, "rms", axes, far=True)
    pos.view(-1)[0], pos.view(-1)[-1] = -2 ** 31, 2 ** 31 - 1
    q, k, v = gsa.qk_norm_rope(x["q"], x["k"], norm="rms", eps=1e-6, positions=pos, rope_base=10000.0, **w)
    assert v is None
    # angles of 2^31 positions are off by 2^31 * 2^-53 * 2 pi at the most: below 2^-19; the oracle's own by as much
    want = oo.norm_rope(f64(x["q"]), "rms", 1e-6, f64(w["q_weight"]), None, f64(pos), axes, 10000.0)
    big = 8 * float(w["q_weight"].abs().max())
    assert_within("q", f64(q), want, (256 * U + 2.0 ** -18) * big)


@pytest.mark.parametrize("axes", [1, 2])
@pytest.mark.parametrize("base", [1.0, 0.01, 1e-4])
def test_norm_rope_with_a_base_of_one_or_less(base, axes):
    """Pairs that turn by up to 1 / base a position: the oracle's own angles, 4000 / base at the most, are off by 2^-53 of
    that, 2^-27; the kernel's by 95 roundings of 2^-64 of it.  Both below 2^-22, an eighth of the bound's 2^-19."""
    g = torch.Generator(device="cuda").manual_seed(8)
    x, w, pos = norm_inputs(g, 2, 70, 3, 1, torch.float32, "rms", axes)
    q, k, _ = gsa.qk_norm_rope(x["q"], x["k"], norm="rms", eps=1e-5, positions=pos, rope_base=base, **w)
    check_norm_rope({"q": x["q"], "k": x["k"]}, w, pos, "rms", axes, base, {"q": q, "k": k}, torch.float32, 1e-5)
    clean()


def test_norm_rope_strides_shared_positions_and_parts():
    """A fused projection's views, one set of positions for all frames, outputs into a larger buffer, parts left out."""
    g = torch.Generator(device="cuda").manual_seed(6)
    qkv = torch.randn(3, 11, 3, 4, 64, generator=g, device="cuda", dtype=torch.bfloat16)
    w = {n: (1 + 0.2 * torch.randn(64, generator=g, device="cuda")).bfloat16() for n in ("q_weight", "k_weight")}
    pos = torch.randint(0, 40, (11, 2), generator=g, device="cuda", dtype=torch.int32)
    full = pos[None].expand(3, 11, 2)
    x = {a: qkv[:, :, i] for i, a in enumerate("qkv")}
    room = torch.full((4, 3, 16, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    out = (room[:, :, 2:13], None, None)
    q, k, v = gsa.qk_norm_rope(x["q"], x["k"], x["v"], norm="rms", positions=pos, head_major=True, out=out, **w)
    got = {"q": room[:, :, 2:13].permute(1, 2, 0, 3), "k": k.permute(1, 2, 0, 3), "v": v.permute(1, 2, 0, 3)}
    check_norm_rope(x, w, full, "rms", 2, 100.0, got, torch.bfloat16, 1e-5)
    assert (room[:, :, :2] == 7).all() and (room[:, :, 13:] == 7).all()
    only = gsa.qk_norm_rope(None, x["k"], norm="rms", positions=pos, k_weight=w["k_weight"])
    assert only[0] is None and only[2] is None and torch.equal(only[1], got["k"])
    # head-first strides of the inputs too
    turned = qkv.permute(3, 2, 0, 1, 4).contiguous()
    again = gsa.qk_norm_rope(turned[:, 0].permute(1, 2, 0, 3), norm="rms", positions=pos, q_weight=w["q_weight"])[0]
    assert torch.equal(again, got["q"])
    # in place
    y = qkv.clone()
    gsa.qk_norm_rope(y[:, :, 0], y[:, :, 1], norm="rms", positions=pos, out=(y[:, :, 0], y[:, :, 1], None), **w)
    assert torch.equal(y[:, :, 0], got["q"]) and torch.equal(y[:, :, 1], got["k"]) and torch.equal(y[:, :, 2], qkv[:, :, 2])
    assert gsa.qk_norm_rope(x["q"][:0], norm="rms", q_weight=w["q_weight"], positions=pos)[0].shape == (0, 11, 4, 64)


def test_norm_rope_special_values():
    """A constant row, NaN and infinity stay in their rows."""
    x = torch.randn(1, 5, 2, 64, device="cuda")
    x[0, 1] = 3.0
    x[0, 2, 0, 5] = float("nan")
    x[0, 3, 1, 9] = float("inf")
    w = torch.ones(64, device="cuda")
    y = gsa.qk_norm_rope(x, norm="layer", q_weight=w, positions=None)[0]
    assert (y[0, 1] == 0).all()
    assert y[0, 2, 0].isnan().all() and y[0, 2, 1].isfinite().all()
    assert not y[0, 3, 1].isfinite().all() and y[0, 3, 0].isfinite().all()
    assert y[0, 0].isfinite().all() and y[0, 4].isfinite().all()


@pytest.mark.parametrize("axes", [0, 1, 2])
@pytest.mark.parametrize("norm", ["none", "layer", "rms"])
@pytest.mark.parametrize("dtype,gdtype", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("outer,tokens,hq,hk", [(1, 1, 1, 1), (2, 83, 6, 2), (3, 9, 21, 7)])
def test_norm_rope_backward(outer, tokens, hq, hk, dtype, gdtype, norm, axes):
    g = torch.Generator(device="cuda").manual_seed(outer * 10 + tokens)
    dt, gt = TYPES[dtype], TYPES[gdtype]
    x, w, pos = norm_inputs(g, outer, tokens, hq, hk, dt, norm, axes)
    head_major = tokens % 2 == 1
    d = {}
    for a, h in (("q", hq), ("k", hk), ("v", hk)):
        shape = (h, outer, tokens, 64) if head_major else (outer, tokens, h, 64)
        d[a] = torch.randn(shape, generator=g, device="cuda").to(gt)
    r = gsa.qk_norm_rope_backward(x["q"], x["k"], d["q"], d["k"], d["v"], norm=norm, eps=1e-5, positions=pos,
                                  rope_base=100.0, head_major=head_major, **w)
    back = (lambda t: t.permute(1, 2, 0, 3)) if head_major else (lambda t: t)
    assert torch.equal(r["dv"], back(d["v"]))
    for a in ("q", "k"):
        dy, xa, wa = f64(back(d[a])), f64(x[a]), f64(w.get(a + "_weight"))
        want, dw, db = oo.norm_rope_backward(xa, dy, norm, 1e-5, wa, f64(pos), axes, 100.0)
        gy = oo.norm_rope_backward(xa, dy, "none", 1e-5, None, f64(pos), axes, 100.0)[0]
        h, s = oo.normed(xa, norm, 1e-5)
        # a pair's turned values are as large as the two together
        i, j = oo._pairs(max(axes, 1))
        mag = np.abs(dy).copy()
        mag[..., i] += np.abs(dy[..., j])
        mag[..., j] += np.abs(dy[..., i])
        uu = mag * (1.0 if wa is None else np.abs(wa))
        bound = uu if norm == "none" else s * (uu + uu.mean(-1, keepdims=True) + np.abs(h) * (uu * np.abs(h)).mean(-1, keepdims=True))
        got = r["d" + a]
        assert got.dtype == gt and got.shape == x[a].shape
        assert_within("d" + a, f64(got), want, 512 * U * bound + half_step(gt) * np.abs(want))
        n = outer * tokens * x[a].shape[2]
        if norm == "none":
            assert r[f"d{a}_weight"] is None and r[f"d{a}_bias"] is None
            continue
        terms = (mag * np.abs(h)).sum((0, 1, 2))
        assert_within("dw", f64(r[f"d{a}_weight"]), dw, (256 + n) * U * terms)
        if norm == "layer":
            assert_within("db", f64(r[f"d{a}_bias"]), db, (256 + n) * U * mag.sum((0, 1, 2)))
        else:
            assert r[f"d{a}_bias"] is None
    again = gsa.qk_norm_rope_backward(x["q"], x["k"], d["q"], d["k"], d["v"], norm=norm, eps=1e-5, positions=pos,
                                      rope_base=100.0, head_major=head_major, **w)
    assert all(r[n] is None or torch.equal(r[n], again[n]) for n in r)       # a fixed order of sums
    clean()


@pytest.mark.parametrize("norm,axes", [("none", 2), ("layer", 2), ("rms", 1), ("layer", 0)])
@pytest.mark.parametrize("dtype,gdtype", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("outer,tokens,hq,hk", [(3, 1201, 1, 1), (2, 1802, 6, 2), (1, 3603, 21, 7)])
def test_norm_rope_backward_of_many_tokens(outer, tokens, hq, hk, dtype, gdtype, norm, axes):
    """More tokens than warps: every group of lanes has a token of its own; counts that no four divide."""
    test_norm_rope_backward(outer, tokens, hq, hk, dtype, gdtype, norm, axes)


def test_norm_rope_backward_against_differences():
    """The kernel's gradient against central differences of the kernel's forward, fp32, step h = 2^-6: an output is off
    by 2^-14 of its size at the most (256 u M, M ~ 9), a sum of 64 of them by sqrt-free 64 * 2^-14 * |dy| = 2^-8 in the
    worst case, over 2 h: 0.125; the truncation is h^2 / 6 times the third derivative, below 2^-12 * 8.  Measured
    against values of up to about 1, with the errors' signs mixed, far below; the bound is the worst case's."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w, pos = norm_inputs(g, 1, 4, 2, 2, torch.float32, "layer", 2)
    dy = torch.randn(1, 4, 2, 64, generator=g, device="cuda")
    run = lambda q: gsa.qk_norm_rope(q, norm="layer", positions=pos, q_weight=w["q_weight"], q_bias=w["q_bias"])[0]
    r = gsa.qk_norm_rope_backward(x["q"], None, dy, None, norm="layer", positions=pos, q_weight=w["q_weight"],
                                  q_bias=w["q_bias"])
    h = 2.0 ** -6
    for at in [(0, 0, 0, 0), (0, 1, 1, 31), (0, 3, 0, 47), (0, 2, 1, 63)]:
        up, down = x["q"].clone(), x["q"].clone()
        up[at] += h
        down[at] -= h
        diff = float(((run(up).double() - run(down).double()) * dy.double()).sum()) / float(up[at].double() - down[at].double())
        assert abs(diff - float(r["dq"][at])) < 0.125 + 2.0 ** -9


def test_norm_rope_backward_parts_places_and_many_rows():
    g = torch.Generator(device="cuda").manual_seed(9)
    x, w, pos = norm_inputs(g, 2, 3000, 2, 1, torch.bfloat16, "layer", 2)
    d = {a: torch.randn(2, 3000, h, 64, generator=g, device="cuda") for a, h in (("q", 2), ("k", 1), ("v", 1))}
    full = gsa.qk_norm_rope_backward(x["q"], x["k"], d["q"], d["k"], d["v"], positions=pos, **w)
    want = oo.norm_rope_backward(f64(x["q"]), f64(d["q"]), "layer", 1e-5, f64(w["q_weight"]), f64(pos), 2, 100.0)
    h, _ = oo.normed(f64(x["q"]), "layer", 1e-5)
    terms = (2 * np.abs(f64(d["q"])).max(-1, keepdims=True) * np.abs(h)).sum((0, 1, 2))
    assert_within("dw", f64(full["dq_weight"]), want[1], (256 + 12000) * U * terms)
    part = gsa.qk_norm_rope_backward(None, x["k"], None, d["k"], None, positions=pos, k_weight=w["k_weight"])
    assert part["dq"] is None and part["dq_weight"] is None and part["dk_bias"] is None
    assert torch.equal(part["dk"], full["dk"])
    # the blocks of the sums depend on the tensors of the call: another order of the same 6,000 terms,
    # each result within (256 + N) u sum|term| of the exact sum, the two within twice that
    hk, _ = oo.normed(f64(x["k"]), "layer", 1e-5)
    terms = (2 * np.abs(f64(d["k"])).max(-1, keepdims=True) * np.abs(hk)).sum((0, 1, 2))
    assert_within("dk_weight", f64(part["dk_weight"]), f64(full["dk_weight"]), 2 * (256 + 6000) * U * terms)
    # over the output gradients themselves
    dq = d["q"].clone()
    over = gsa.qk_norm_rope_backward(x["q"], None, dq, None, positions=pos, out=(dq, None, None), q_weight=w["q_weight"],
                                     q_bias=w["q_bias"])
    assert over["dq"] is dq and torch.equal(dq, full["dq"])
    none = gsa.qk_norm_rope_backward(x["q"][:0], None, d["q"][:0], None, positions=pos[:0], q_weight=w["q_weight"],
                                     q_bias=w["q_bias"])
    assert none["dq"].numel() == 0 and (none["dq_weight"] == 0).all() and (none["dq_bias"] == 0).all()


@pytest.mark.parametrize("change", [
    dict(q_weight=None), dict(q_weight=torch.ones(64)), dict(norm="batch"), dict(positions=torch.zeros(2, 5, 3, dtype=torch.int32)),
    dict(q=torch.zeros(2, 5, 3, 32)), dict(q=torch.zeros(2, 5, 64)), dict(q="half"), dict(q="cpu"), dict(q="odd")])
def test_norm_rope_python_refusals(change):
    q = torch.zeros(2, 5, 3, 64, device="cuda")
    kw = dict(norm="layer", q_weight=torch.ones(64, device="cuda"), positions=torch.zeros(5, 2, dtype=torch.int32, device="cuda"))
    change = {n: (t.cuda() if isinstance(t, torch.Tensor) and n != "q_weight" else t) for n, t in change.items()}
    q = {"half": q.half(), "cpu": q.cpu(), "odd": torch.zeros(2, 5, 3, 128, device="cuda")[..., ::2]}.get(change.get("q"), q) \
        if not isinstance(change.get("q"), torch.Tensor) else change["q"]
    change.pop("q", None)
    with pytest.raises(gsa.GSAError):
        gsa.qk_norm_rope(q, **{**kw, **change})


# ---- the cache ---------------------------------------------------------------------------
class Streams:
    """Sequences in a paged cache: `old` tokens before the new ones, unused memory NaN."""

    def __init__(self, new, old, page, hk, dtype, seed=0, spare=2, fill=float("nan"), width=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.new, self.old, self.page, self.hk, self.dtype = new, old, page, hk, dtype
        total = [n + o for n, o in zip(new, old)]
        need = [max(0, -(-t // page)) for t in total]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=self.g, device="cuda").to(torch.int32)
        width = max(width, max(need), 1)
        table = torch.full((len(new), width), -99, dtype=torch.int32, device="cuda")     # never to be read
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table, self.total = table, total
        self.cache = gsa.KVCache(pages, page, hk, dtype)
        self.cache.k_pages.fill_(fill)
        self.cache.v_pages.fill_(fill)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.cu_list, self.cu, self.start, self.lengths = cu, i32(cu), i32(old), i32(total)
        if sum(max(o, 0) for o in old):     # the older tokens, as they are
            cu_old = np.concatenate([[0], np.cumsum([max(o, 0) for o in old])]).tolist()
            k, v = (self.rand(cu_old[-1], hk) for _ in range(2))
            self.cache.append(k, v, table, i32([0] * len(old)), i32(cu_old))

    def rand(self, tokens, heads, scale=1.0):
        return (torch.randn(tokens, heads, 64, generator=self.g, device="cuda") * scale).to(self.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("norm,axes", [("none", 0), ("rms", 1), ("layer", 2), ("none", 1)])
@pytest.mark.parametrize("new,old,page,hk", [
    ([1], [0], 16, 1), ([1, 1, 1], [15, 16, 300], 16, 4), ([0, 40, 0, 0, 17, 1, 0], [3, 0, 0, 9, 64, 31, 5], 32, 3),
    ([130, 5], [100, 250], 256, 2), ([3] * 70, list(range(70)), 64, 2)])
def test_append(new, old, page, hk, dtype, norm, axes):
    dt = TYPES[dtype]
    s = Streams(new, old, page, hk, dt)
    tokens = sum(new)
    extra = 3                                   # rows behind the last sequence: not used
    k, v = s.rand(tokens + extra, hk), s.rand(tokens + extra, hk)
    w = (1 + 0.3 * torch.randn(64, generator=s.g, device="cuda")).to(dt) if norm != "none" else None
    b = (0.2 * torch.randn(64, generator=s.g, device="cuda")).to(dt) if norm == "layer" else None
    pos = torch.randint(0, 5000, (tokens + extra, axes), generator=s.g, device="cuda").to(torch.int32) if axes == 2 else None
    before = s.cache.k_pages.clone(), s.cache.v_pages.clone()
    s.cache.append(k, v, s.table, s.start, s.cu, norm=norm, k_weight=w, k_bias=b, positions=pos, rope_axes=axes)
    clean()
    table, own = s.table.cpu().numpy(), np.concatenate([o + np.arange(n) for n, o in zip(new, old)])[:, None]
    p = f64(pos[:tokens]) if pos is not None else own
    rows = oo.norm_rope(f64(k[:tokens]), norm, 1e-5, f64(w), f64(b), p, axes, 10000.0)
    want, left = oo.cache_append(f64(before[0]), rows, table, old, s.cu_list)
    assert not left
    big = (8 * float(w.abs().max()) + (0 if b is None else float(b.abs().max()))) if w is not None else float(k.abs().max())
    assert_within("k", f64(s.cache.k_pages), want, 256 * U * big + half_step(dt) * np.abs(np.nan_to_num(want)))
    untouched = np.isnan(want)
    assert np.array_equal(np.isnan(f64(s.cache.k_pages)), untouched)
    want, _ = oo.cache_append(f64(before[1]), f64(v[:tokens]), table, old, s.cu_list)
    assert np.array_equal(f64(s.cache.v_pages), want, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("norm,axes", [("none", 0), ("rms", 1), ("layer", 2)])
@pytest.mark.parametrize("new,old,page,hk", [([0, 900, 0, 1100, 1, 0], [4, 100, 0, 0, 63, 9], 16, 3), ([2, 1902], [0, 30], 128, 8)])
def test_append_of_many_tokens(new, old, page, hk, dtype, norm, axes):
    test_append(new, old, page, hk, dtype, norm, axes)


def test_append_of_many_tokens_leaves_out_what_has_no_page():
    s = Streams([1000, 1000], [10, 10], 16, 2, torch.bfloat16)
    s.table[0, 3], s.table[1, 5] = s.cache.num_pages, -1
    k, v = s.rand(2000, 2), s.rand(2000, 2)
    before = f64(s.cache.v_pages)
    s.cache.append(k, v, s.table, s.start, s.cu, norm="none", rope_axes=1)
    assert gsa.operator_status() == 7
    clean()
    want, left = oo.cache_append(before, f64(v), s.table.cpu().numpy(), [10] * 2, s.cu_list)
    assert len(left) == 32 and np.array_equal(f64(s.cache.v_pages), want, equal_nan=True)


def test_append_leaves_out_what_has_no_page():
    s = Streams([4, 4, 4], [14, 14, 14], 16, 2, torch.bfloat16)
    s.table[1, 1] = s.cache.num_pages           # one page behind the pool
    s.table[2, 1] = -1
    start = s.start.clone()
    k, v = s.rand(12, 2), s.rand(12, 2)
    before = f64(s.cache.k_pages)
    s.cache.append(k, v, s.table, start, s.cu)
    assert gsa.operator_status() == 7           # GSA_ERR_DEVICE_BOUNDS, and cleared by the read
    clean()
    want, left = oo.cache_append(before, f64(k), s.table.cpu().numpy(), [14] * 3, s.cu_list)
    assert len(left) == 4 and np.array_equal(f64(s.cache.k_pages), want, equal_nan=True)
    # places outside the table: before its first token, behind its last page
    start[0], start[1], start[2] = -1, 32, 0
    before = f64(s.cache.k_pages)
    s.cache.append(k, v, s.table, start, s.cu)
    assert gsa.operator_status() == 7
    want, left = oo.cache_append(before, f64(k), s.table.cpu().numpy(), [-10 ** 6, 32, 0], s.cu_list)
    assert len(left) == 8 and np.array_equal(f64(s.cache.k_pages), want, equal_nan=True)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("place,value", [(3, 99), (3, 9000), (0, -2), (2, 1), (1, -5), (4, 0)])
def test_append_records_wrong_sequences(place, value, many):
    """cu_tokens that end behind the rows, start before them or decrease: recorded, and no row outside the sequences'
    own pages is touched."""
    per = 800 if many else 3
    s = Streams([per] * 4, [5] * 4, 16, 2, torch.bfloat16)
    cu = s.cu.clone()
    cu[place] = value if value != 99 else 4 * per + 1
    k, v = s.rand(4 * per, 2), s.rand(4 * per, 2)
    before = s.cache.k_pages.clone()
    clean()
    s.cache.append(k, v, s.table, s.start, cu)
    assert gsa.operator_status() == 7
    spare = torch.ones(s.cache.num_pages, dtype=torch.bool, device="cuda")
    spare[s.table[s.table >= 0].long()] = False
    assert spare.any() and torch.equal(s.cache.k_pages[spare].nan_to_num(7.0), before[spare].nan_to_num(7.0))
    # rows behind the last sequence are no mistake
    s.cache.append(s.rand(4 * per + 7, 2), s.rand(4 * per + 7, 2), s.table, s.start, s.cu)
    clean()


# ---- attention over the cache ----------------------------------------------------------------
def check_attention(s, q, out, lse, causal, scale=0.125, table=None, lengths=None, cu=None):
    table = s.table.cpu().numpy() if table is None else table
    lengths = s.total if lengths is None else lengths
    cu = s.cu_list if cu is None else cu
    qd, kp, vp = f64(q), f64(s.cache.k_pages), f64(s.cache.v_pages)
    want, wlse, mag = oo.cache_attention(qd, kp, vp, table, lengths, cu, causal, scale)
    t = slice(cu[0], cu[-1])
    group = q.shape[1] // s.hk
    big_k = np.abs(kp[np.isfinite(kp)]).max(initial=0.0)
    a = np.abs(qd[t]).sum(-1).max() * big_k * scale          # at least the largest sum|q k| scale
    n = max(max(lengths), 1)
    weight = 128 * (1 + a) * U + n * U + (2.0 ** -8 if s.dtype == torch.bfloat16 else 0)
    assert group >= 1
    assert_within("out", f64(out)[t], want[t], weight * mag[t] + half_step(s.dtype) * np.abs(want[t]))
    if lse is not None:
        w = wlse[:, t]
        fine = np.isfinite(w)
        assert np.array_equal(f64(lse)[:, t][~fine], w[~fine])
        assert_within("lse", f64(lse)[:, t][fine], w[fine], (128 * (1 + a) + n) * U + 4 * U * np.abs(w[fine]))


ATTEND = [
    # new, old, page, hk, group
    ([1], [0], 16, 1, 1),
    ([1, 1, 1, 1], [0, 15, 16, 127], 16, 2, 1),
    ([1, 1, 1], [128, 700, 2049], 16, 2, 4),
    ([1, 1], [1000, 31], 64, 1, 48),                           # more rows than a quarter holds
    ([1], [5000], 32, 1, 12),                                  # split over keys
    ([5, 0, 3, 1], [300, 77, 0, 1], 32, 2, 3),
    ([17, 31, 32], [0, 100, 257], 128, 1, 1),
    ([40, 7], [200, 1200], 256, 3, 2),
    ([128], [128], 64, 1, 1),
    ([129, 1, 64], [0, 300, 63], 16, 2, 1),
    ([300, 0, 257], [0, 50, 500], 64, 1, 2),
    ([70], [3000], 128, 1, 5),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new,old,page,hk,group", ATTEND)
def test_attention(new, old, page, hk, group, dtype, causal):
    s = Streams(new, old, page, hk, TYPES[dtype], seed=len(new) + page)
    tokens = sum(new)
    s.cache.append(s.rand(tokens, hk), s.rand(tokens, hk), s.table, s.start, s.cu)
    q = s.rand(tokens + 2, hk * group, 1.5)
    room = torch.full_like(q, 5.0)
    out, lse = s.cache.attention(q, s.table, s.lengths, s.cu, max(new), causal=causal, return_lse=True, out=room)
    clean()
    check_attention(s, q, out, lse, causal)
    assert (out[tokens:] == 5).all()                           # rows behind the last sequence stay as they are
    again = s.cache.attention(q, s.table, s.lengths, s.cu, max(new), causal=causal)
    assert torch.equal(out[:tokens], again[:tokens])
    # another way to split the keys: the same within the same bounds
    for max_len in (1, 200000):
        other, olse = s.cache.attention(q, s.table, s.lengths, s.cu, max(new) + 200 * (max_len > 1), max_len=max_len,
                                        causal=causal, return_lse=True)
        check_attention(s, q, other, olse, causal)
    clean()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_rows_without_keys(dtype):
    """Empty caches, and causal queries ahead of every key: 0 and -inf, whatever the memory holds."""
    for new, lengths in (([3, 2], [0, 0]), ([6, 3], [2, 1]), ([40, 35], [7, 0]), ([200, 150], [3, 130])):
        s = Streams(new, [0] * len(new), 16, 2, TYPES[dtype])
        if any(lengths):
            cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
            s.cache.append(s.rand(int(cu[-1]), 2), s.rand(int(cu[-1]), 2), s.table, s.start, cu)
        q = s.rand(sum(new), 4)
        ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        for max_len in (None, 100000):
            out, lse = s.cache.attention(q, s.table, ln, s.cu, max(new), max_len=max_len, causal=True, return_lse=True)
            check_attention(s, q, out, lse, True, lengths=lengths)
            none = lengths[0] - new[0] + 1 + np.arange(new[0]) <= 0
            assert none.any() and (out[:new[0]][torch.from_numpy(none)] == 0).all()
    clean()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("group,n", [(1, 1), (4, 20), (2, 150)])
def test_attention_leaves_out_bad_pages(dtype, group, n):
    s = Streams([n, n], [250, 90], 32, 2, TYPES[dtype], fill=0.0)
    s.cache.append(s.rand(2 * n, 2), s.rand(2 * n, 2), s.table, s.start, s.cu)
    clean()
    s.table[0, 2], s.table[0, 5], s.table[1, 0] = s.cache.num_pages, -7, 2 ** 30
    q = s.rand(2 * n, 2 * group)
    out, lse = s.cache.attention(q, s.table, s.lengths, s.cu, n, return_lse=True, max_len=128)
    assert gsa.operator_status() == 7
    clean()
    check_attention(s, q, out, lse, True)


def test_attention_refuses_bad_sequences_on_the_device():
    """Lengths that do not fit: the sequence is left out (its rows untouched), the others are computed."""
    s = Streams([4, 6, 5], [20, 30, 40], 16, 1, torch.bfloat16)
    s.cache.append(s.rand(15, 1), s.rand(15, 1), s.table, s.start, s.cu)
    q = s.rand(15, 2)
    clean()
    good = s.cache.attention(q, s.table, s.lengths, s.cu, 6)
    for max_len in (None, 100000):
        out = torch.full_like(q, 3.0)
        s.cache.attention(q, s.table, s.lengths, s.cu, 5, out=out, max_len=max_len)      # the second has six new tokens
        assert gsa.operator_status() == 7
        assert (out[4:10] == 3).all()
        keep = torch.cat([out[:4], out[10:]]).float()
        assert (keep - torch.cat([good[:4], good[10:]]).float()).abs().max() < 2 ** -5
    bad = s.lengths.clone()
    bad[1] = -1
    out = torch.full_like(q, 3.0)
    s.cache.attention(q, s.table, bad, s.cu, 6, out=out)
    assert gsa.operator_status() == 7 and (out[4:10] == 3).all() and torch.equal(out[:4], good[:4])
    cu = s.cu.clone()
    cu[3] = 99                                       # behind the queries
    out = torch.full_like(q, 3.0)
    s.cache.attention(q, s.table, s.lengths, cu, 100, out=out)
    assert gsa.operator_status() == 7 and (out[10:] == 3).all()
    cu[3] = 7                                        # decreasing
    s.cache.attention(q, s.table, s.lengths, cu, 100, out=out)
    assert gsa.operator_status() == 7 and (out[10:] == 3).all()
    long = s.lengths.clone()
    long[0] = 10 ** 6                                # more than the table holds: what it holds is read
    s.cache.attention(q, s.table, long, s.cu, 6, causal=False)
    assert gsa.operator_status() == 7
    clean()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_of_no_new_tokens_at_most(dtype):
    """max_new 0: sequences that have new tokens are left out and recorded, as with any other max_new that is too small."""
    s = Streams([2, 0, 1], [20, 30, 0], 16, 2, TYPES[dtype], width=3000)
    q = s.rand(3, 2)
    clean()
    for max_len in (None, 0):
        out = torch.full_like(q, 3.0)
        s.cache.attention(q, s.table, s.lengths, s.cu, 0, out=out, max_len=max_len, return_lse=True)
        assert gsa.operator_status() == 7 and (out == 3).all()
        s.cache.attention(q, s.table, s.lengths, torch.zeros_like(s.cu), 0, out=out, max_len=max_len)
        clean()
        assert (out == 3).all()


def test_attention_values_of_special_size():
    """Large scores; infinities and NaN in real keys reach the sequence's outputs, and no other's."""
    s = Streams([1, 1, 1], [200, 200, 200], 16, 1, torch.bfloat16)
    k, v = s.rand(3, 1), s.rand(3, 1)
    s.cache.append(k, v, s.table, s.start, s.cu)
    q = s.rand(3, 1, 60.0)                            # one key takes nearly all the weight
    out, lse = s.cache.attention(q, s.table, s.lengths, s.cu, 1, return_lse=True)
    check_attention(s, q, out, lse, True)
    page = int(s.table[1, 3])
    s.cache.k_pages[page, 0, 5, 3] = float("nan")     # in sequence 1 only
    page = int(s.table[2, 3])
    s.cache.v_pages[page, 0, 5, 3] = float("inf")     # in sequence 2, channel 3
    q = s.rand(3, 1)
    out = s.cache.attention(q, s.table, s.lengths, s.cu, 1)
    assert out[0].isfinite().all() and out[1].isnan().all()
    assert not out[2, 0, 3].isfinite() and out[2, 0, [i for i in range(64) if i != 3]].isfinite().all()
    clean()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 50, 300])
def test_attention_strides_scale_and_table_width(dtype, n):
    """Queries inside a fused projection, outputs head by head, a scale, a table wider than a sequence needs."""
    s = Streams([n, n], [33, 64], 16, 2, TYPES[dtype], width=40)
    s.cache.append(s.rand(2 * n, 2), s.rand(2 * n, 2), s.table, s.start, s.cu)
    q = s.rand(2 * n, 12).view(2 * n, 3, 4, 64)[:, 1]
    room = torch.zeros(4, 2 * n, 64, device="cuda", dtype=TYPES[dtype])
    out, lse = s.cache.attention(q, s.table[:, :30], s.lengths, s.cu, n, softmax_scale=0.3, return_lse=True,
                                 out=room.transpose(0, 1))
    check_attention(s, q, room.transpose(0, 1), lse, True, scale=0.3)
    clean()


def test_attention_python_refusals():
    s = Streams([2, 2], [5, 6], 16, 2, torch.bfloat16)
    q = s.rand(4, 4)
    ok = dict(q=q, block_table=s.table, lengths=s.lengths, cu_tokens=s.cu, max_new=2)
    for change in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[..., :32]), dict(q=s.rand(4, 3)), dict(block_table=s.table.long()),
                   dict(block_table=s.table.t()), dict(lengths=s.lengths[:1]), dict(cu_tokens=s.cu[:2]),
                   dict(lengths=s.lengths.float()), dict(max_new=-1), dict(softmax_scale=-1.0),
                   dict(out=torch.empty(3, 4, 64, device="cuda", dtype=torch.bfloat16))):
        with pytest.raises(gsa.GSAError):
            s.cache.attention(**{**ok, **change})
    with pytest.raises(gsa.GSAError):
        gsa.KVCache(4, 24, 2).append(s.rand(4, 2), s.rand(4, 2), s.table, s.start, s.cu)     # such pages there are not
    with pytest.raises(gsa.GSAError):
        s.cache.append(s.rand(4, 3), s.rand(4, 3), s.table, s.start, s.cu)
    with pytest.raises(gsa.GSAError):
        s.cache.append(s.rand(4, 2), s.rand(3, 2), s.table, s.start, s.cu)
    with pytest.raises(gsa.GSAError):
        s.cache.append(s.rand(4, 2), s.rand(4, 2), s.table, s.start, s.cu, rope_axes=2)
    with pytest.raises(gsa.GSAError):
        gsa.KVCache.from_pages(s.cache.k_pages, s.cache.v_pages[:-1])
    clean()


# ---- together -------------------------------------------------------------------------------
def test_frames_arriving_one_by_one():
    """Frames of two streams: keys normed and rotated into the cache, queries likewise, every token attends to its
    stream's frames so far; against attention over all tokens from the formulas."""
    g = torch.Generator(device="cuda").manual_seed(0)
    dt, frames, grid, heads, page = torch.bfloat16, 4, 6, 3, 16
    n = grid * grid + 2
    w = {a: (1 + 0.2 * torch.randn(64, generator=g, device="cuda")).to(dt) for a in ("q_weight", "k_weight")}
    b = {a: (0.1 * torch.randn(64, generator=g, device="cuda")).to(dt) for a in ("q_bias", "k_bias")}
    at = torch.arange(grid * grid, device="cuda", dtype=torch.int32)
    pos = torch.cat([torch.zeros(2, 2, device="cuda", dtype=torch.int32), torch.stack([at // grid + 1, at % grid + 1], 1).int()])
    pages = -(-frames * n // page)
    cache = gsa.KVCache(2 * pages, page, heads, dt)
    table = torch.arange(2 * pages, device="cuda", dtype=torch.int32).view(pages, 2).t().contiguous()
    cu = torch.tensor([0, n, 2 * n], device="cuda", dtype=torch.int32)
    ks, vs = [], []
    for f in range(frames):
        qkv = torch.randn(2, n, 3, heads, 64, generator=g, device="cuda").to(dt)
        start = torch.full((2,), f * n, device="cuda", dtype=torch.int32)
        flat = qkv.view(2 * n, 3, heads, 64)
        cache.append(flat[:, 1], flat[:, 2], table, start, cu, norm="layer", k_weight=w["k_weight"], k_bias=b["k_bias"],
                     positions=pos.repeat(2, 1), rope_axes=2, rope_base=100.0)
        q = gsa.qk_norm_rope(qkv[:, :, 0], norm="layer", q_weight=w["q_weight"], q_bias=b["q_bias"], positions=pos)[0]
        out = cache.attention(q.view(2 * n, heads, 64), table, start + n, cu, n, causal=False)
        k = oo.norm_rope(f64(qkv[:, :, 1]), "layer", 1e-5, f64(w["k_weight"]), f64(b["k_bias"]), f64(pos), 2, 100.0)
        ks.append(k)
        vs.append(f64(qkv[:, :, 2]))
        qw = oo.norm_rope(f64(qkv[:, :, 0]), "layer", 1e-5, f64(w["q_weight"]), f64(b["q_bias"]), f64(pos), 2, 100.0)
        kk, vv = np.concatenate(ks, 1), np.concatenate(vs, 1)
        sc = np.einsum("bihd,bjhd->bhij", qw, kk) / 8
        p = np.exp(sc - sc.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        want = np.einsum("bhij,bjhd->bihd", p, vv)
        # q and k are rounded to bf16 on the way: a score moves by 2 * 2^-8 sum|q k| / 8, a weight by twice that
        shift = 4 * 2.0 ** -8 * np.einsum("bihd,bjhd->bhij", np.abs(qw), np.abs(kk)).max() / 8
        mag = np.einsum("bhij,bjhd->bihd", p, np.abs(vv))
        assert_within(f"frame {f}", f64(out).reshape(want.shape), want, (np.expm1(shift) + 2.0 ** -7) * mag + 2.0 ** -8 * np.abs(want))
    clean()


SMALL = GSAConfig("ops_small", 3, 12, 12, 12, 12, 2, 2, 64, 4, 6, "bf16")
PADDED = GSAConfig("ops_padded", 3, 10, 11, 12, 12, 3, 2, 64, 4, 6, "bf16")
NO_SPEC = GSAConfig("ops_nospec", 2, 8, 8, 8, 8, 0, 2, 64, 4, 4, "bf16")
FP32 = GSAConfig("ops_fp32", 2, 8, 8, 8, 8, 1, 2, 64, 4, 4, "fp32")


@pytest.mark.parametrize("cfg", [SMALL, PADDED, NO_SPEC, FP32], ids=lambda c: c.name)
def test_layer_inputs_from_a_projection(cfg):
    """split_qkv gives the layer's inputs; the layer runs on them; split_qkv_backward takes the layer's gradients."""
    g = torch.Generator(device="cuda").manual_seed(1)
    dt = TYPES[cfg.dtype]
    F, H, ns, per = cfg.num_frames, cfg.num_heads, cfg.num_special, cfg.pad_h * cfg.pad_w
    qkv = torch.randn(F, ns + per, 3, H, 64, generator=g, device="cuda").to(dt)
    w = {n: (1 + 0.2 * torch.randn(64, generator=g, device="cuda")).to(dt) for n in ("q_weight", "k_weight")}
    w.update({n: (0.1 * torch.randn(64, generator=g, device="cuda")).to(dt) for n in ("q_bias", "k_bias")})
    w_g = (torch.randn(H, 64, 64, generator=g, device="cuda") / 8).to(dt)
    layer = gsa.GSALayer.from_workload(cfg)
    try:
        x = layer.split_qkv(qkv, w_g, **w)
        y, xx = np.meshgrid(np.arange(cfg.pad_h) + 1, np.arange(cfg.pad_w) + 1, indexing="ij")
        pos = np.concatenate([np.zeros((ns, 2)), np.stack([y.ravel(), xx.ravel()], 1)])
        for i, a in enumerate("qkv"):
            want = f64(qkv[:, :, i])
            if a != "v":
                want = oo.norm_rope(want, "layer", 1e-5, f64(w[a + "_weight"]), f64(w[a + "_bias"]), pos, 2, 100.0)
            want = want.transpose(2, 0, 1, 3)
            got = np.concatenate([f64(x[a + "_spec"]), f64(x[a + "_img"]).reshape(H, F, per, 64)], 2)
            tol = 0 if a == "v" else 256 * U * 17 + half_step(dt) * np.abs(want)
            assert_within(a, got, want, tol)
        out = layer.forward(x)
        assert layer.status() == 0 and out["o_img"].isfinite().all()
        if cfg.dtype != "bf16":
            return
        grads = layer.backward(x, out, {"o_img": torch.randn(x["q_img"].shape, generator=g, device="cuda").to(dt),
                                        "o_spec": torch.randn(x["q_spec"].shape, generator=g, device="cuda").to(dt)})
        r = layer.split_qkv_backward(qkv, grads, **w)
        assert layer.status() == 0
        for i, a in enumerate("qk"):
            dy = np.concatenate([f64(grads[f"d{a}_spec"]), f64(grads[f"d{a}_img"]).reshape(H, F, per, 64)], 2).transpose(1, 2, 0, 3)
            want, dw, db = oo.norm_rope_backward(f64(qkv[:, :, i]), dy, "layer", 1e-5, f64(w[a + "_weight"]), pos, 2, 100.0)
            h, s = oo.normed(f64(qkv[:, :, i]), "layer", 1e-5)
            big = 2 * np.abs(dy).max(-1, keepdims=True) * float(w[a + "_weight"].abs().max())
            assert_within("d" + a, f64(r["dqkv"][:, :, i]), want, 512 * U * s * big * (2 + np.abs(h)) + U * np.abs(want))
            n = F * (ns + per) * H
            assert_within("dw", f64(r[f"d{a}_weight"]), dw, (256 + n) * U * (big * np.abs(h)).sum((0, 1, 2)))
            assert_within("db", f64(r[f"d{a}_bias"]), db, (256 + n) * U * big.sum() * np.ones(64))
        dv = np.concatenate([f64(grads["dv_spec"]), f64(grads["dv_img"]).reshape(H, F, per, 64)], 2).transpose(1, 2, 0, 3)
        assert np.array_equal(f64(r["dqkv"][:, :, 2]), dv)
        with pytest.raises(gsa.GSAError):
            layer.split_qkv(qkv[:, 1:], w_g, **w)
        with pytest.raises(gsa.GSAError):
            layer.split_qkv(qkv.float(), w_g, **w)
    finally:
        layer.close()


def test_default_positions_are_made_outside_a_capture():
    cfg = SMALL
    qkv = torch.randn(cfg.num_frames, cfg.num_special + cfg.pad_h * cfg.pad_w, 3, cfg.num_heads, 64, device="cuda")
    qkv = qkv.to(TYPES[cfg.dtype])
    layer = gsa.GSALayer.from_workload(cfg)
    try:
        one = torch.ones(3, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            two = one + 1
            with pytest.raises(gsa.GSAError, match="capture"):
                layer.split_qkv(qkv, None, norm="none")
        graph.replay()
        assert (two == 2).all()
        want = layer.split_qkv(qkv, None, norm="none")
        with torch.cuda.graph(graph2 := torch.cuda.CUDAGraph()):
            got = layer.split_qkv(qkv, None, norm="none")
        graph2.replay()
        assert all(torch.equal(got[n], want[n]) for n in want if n != "w_g")
    finally:
        layer.close()


def test_outputs_from_a_sequence_that_makes_its_items():
    """`out` may be any sequence of three, also one whose items nothing else holds."""
    class Parts:
        def __init__(self, whole):
            self.whole = whole

        def __len__(self):
            return len(self.whole)

        def __getitem__(self, i):
            return self.whole[i]

    g = torch.Generator(device="cuda").manual_seed(3)
    x = [torch.randn(2, 9, 4, 64, generator=g, device="cuda") for _ in range(3)]
    pos = torch.arange(9, dtype=torch.int32, device="cuda")[:, None]
    want = gsa.qk_norm_rope(*x, norm="none", positions=pos)
    room = torch.zeros(3, 2, 9, 4, 64, device="cuda")
    got = gsa.qk_norm_rope(*x, norm="none", positions=pos, out=Parts(room))
    assert all(torch.equal(a, b) and torch.equal(a, r) for a, b, r in zip(got, want, room))
    back = torch.zeros_like(room)
    r = gsa.qk_norm_rope_backward(None, None, *want, norm="none", positions=pos, out=Parts(back))
    again = gsa.qk_norm_rope_backward(None, None, *want, norm="none", positions=pos)
    assert all(torch.equal(r[n], again[n]) and torch.equal(r[n], b) for n, b in zip(("dq", "dk", "dv"), back))
    for bad in (room, Parts(room[:2]), "abc", 3, [1, 2, 3]):
        with pytest.raises(gsa.GSAError):
            gsa.qk_norm_rope(*x, norm="none", positions=pos, out=bad)


def test_arguments_that_are_no_truth_values_or_streams():
    x = torch.randn(2, 9, 4, 64, device="cuda")
    for kw in (dict(head_major=torch.zeros(2)), dict(stream=1), dict(stream=2), dict(stream="a")):
        with pytest.raises(gsa.GSAError):
            gsa.qk_norm_rope(x, norm="none", **kw)
    s = Streams([1], [3], 16, 1, torch.float32)
    q = s.rand(1, 1)
    for kw in (dict(causal=torch.zeros(2)), dict(return_lse=torch.zeros(2))):
        with pytest.raises(gsa.GSAError):
            s.cache.attention(q, s.table, s.lengths, s.cu, 1, **kw)
    clean()


# ---- streams and graphs ------------------------------------------------------------------------
def test_two_streams_at_once():
    """The same calls on two streams at the same time: no workspace is shared."""
    a = Streams([1] * 3, [9000, 4000, 100], 64, 2, torch.bfloat16, seed=1)
    b = Streams([1] * 3, [300, 8000, 7000], 64, 2, torch.bfloat16, seed=2)
    for s in (a, b):
        s.cache.append(s.rand(3, 2), s.rand(3, 2), s.table, s.start, s.cu)
    qa, qb = a.rand(3, 8), b.rand(3, 8)
    call = lambda s, q: s.cache.attention(q, s.table, s.lengths, s.cu, 1)
    wa, wb = call(a, qa), call(b, qb)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(sa):
            x = call(a, qa)
        y = b.cache.attention(qb, b.table, b.lengths, b.cu, 1, stream=sb.cuda_stream)     # by its handle
        got.append((x, y))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in got)
    clean()


def test_captured_decoding_step():
    """A step captured once and replayed as the lengths grow on the device, two such graphs in turn."""
    s = Streams([1, 1], [0, 0], 16, 2, torch.bfloat16, width=20, spare=40)
    s.table.copy_(torch.arange(40, device="cuda", dtype=torch.int32).view(2, 20))
    k, v, q = s.rand(2, 2), s.rand(2, 2), s.rand(2, 4)
    start = torch.zeros(2, device="cuda", dtype=torch.int32)

    def step():
        s.cache.append(k, v, s.table, start, s.cu, rope_axes=1)
        r = gsa.qk_norm_rope(q[:, None], norm="none", positions=start.view(2, 1, 1), rope_base=10000.0)[0]
        out = s.cache.attention(r[:, 0], s.table, start + 1, s.cu, 1, max_len=20000, return_lse=True)
        start.add_(1)
        return out
    step()
    start.zero_()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for i in range(45):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=s.g, device="cuda"))
        graph, (out, lse) = graphs[i % 2]
        graph.replay()
        assert int(start[0]) == i + 1
        qr = oo.norm_rope(f64(q), "none", 0.0, None, None, np.full((2, 1), i), 1, 10000.0)
        qr = torch.from_numpy(qr).to(torch.bfloat16).cuda()
        if i % 9 == 0 or i == 44:
            want, wlse, mag = oo.cache_attention(f64(qr), f64(s.cache.k_pages), f64(s.cache.v_pages), s.table.cpu().numpy(),
                                                 [i + 1] * 2, [0, 1, 2], True)
            # a rotated query may round to the neighbour: 2^-7 of a score's terms
            a = np.abs(f64(qr)).sum(-1).max() * np.nanmax(np.abs(f64(s.cache.k_pages))) / 8
            assert_within("out", f64(out), want, (2.0 ** -8 * 3 + np.expm1(2.0 ** -13 * (1 + a)) + 2.0 ** -6) * mag + 2.0 ** -8 * np.abs(want))
    clean()


def test_captured_norm_and_gradients():
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w, pos = norm_inputs(g, 2, 50, 4, 2, torch.bfloat16, "layer", 2)
    d = {a: torch.randn(2, 50, h, 64, generator=g, device="cuda") for a, h in (("q", 4), ("k", 2))}

    def both():
        return gsa.qk_norm_rope(x["q"], x["k"], positions=pos, **w), \
            gsa.qk_norm_rope_backward(x["q"], x["k"], d["q"], d["k"], positions=pos, **w)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, grads = both()
    x["q"].normal_(generator=g)
    d["q"].normal_(generator=g)
    graph.replay()
    torch.cuda.synchronize()
    eager, egrads = both()
    assert torch.equal(out[0], eager[0]) and torch.equal(grads["dq"], egrads["dq"])
    assert torch.equal(grads["dq_weight"], egrads["dq_weight"]) and torch.equal(grads["dk_bias"], egrads["dk_bias"])
    clean()


def test_a_timeout_of_the_other_calls_does_not_show_here():
    """The operators' status words are their own."""
    gsa.gsa_debug_expire_wait(None, 1000, torch.cuda.current_stream().cuda_stream)
    clean()
    assert gsa.gsa_special_attention_noalloc_status(torch.cuda.current_stream().cuda_stream) == 6


# ---- offsets beyond 32 bits ----------------------------------------------------------------------
def test_pages_beyond_32_bit_offsets():
    """A pool of more than 2^31 elements: the sequence's pages lie at its end."""
    page, hk, pages = 256, 16, 8400
    assert pages * hk * page * 64 > 2 ** 31
    cache = gsa.KVCache(pages, page, hk)
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda t, h: torch.randn(t, h, 64, generator=g, device="cuda").bfloat16()
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    n = 600
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    k, v = rand(n, hk), rand(n, hk)
    cache.append(k, v, table, i32([0]), i32([0, n]))
    assert torch.equal(cache.k_pages[pages - 1], k[:256].transpose(0, 1))
    assert torch.equal(cache.v_pages[pages - 2, :, :88], v[512:].transpose(0, 1))
    for new, group in ((1, 1), (70, 1), (200, 1)):
        q = rand(new, hk * group)
        out = cache.attention(q, table, i32([n]), i32([0, new]), new)
        seen = np.arange(n)[None] <= np.arange(n - new, n)[:, None]
        for h in (0, hk - 1):
            kd, vd, qd = f64(k[:, h]), f64(v[:, h]), f64(q[:, h])
            s = np.where(seen, qd @ kd.T / 8, -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            a = np.abs(qd).sum(-1).max() * np.abs(kd).max() / 8
            assert_within("out", f64(out[:, h]), p @ vd, (128 * (1 + a) * U + n * U + 2.0 ** -8) * (p @ np.abs(vd)) + 2.0 ** -8 * np.abs(p @ vd))
    clean()


def test_rows_beyond_32_bit_offsets():
    tokens, heads = (1 << 21) + 5, 16
    assert tokens * heads * 64 > 2 ** 31
    x = torch.empty(1, tokens, heads, 64, dtype=torch.bfloat16, device="cuda")
    x[:, -7:] = torch.randn(1, 7, heads, 64, device="cuda")
    x[:, :3] = torch.randn(1, 3, heads, 64, device="cuda")
    w = torch.randn(64, device="cuda").bfloat16()
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda").unsqueeze(-1)
    for head_major in (False, True):
        y = gsa.qk_norm_rope(x, norm="rms", q_weight=w, positions=pos, rope_base=10000.0, head_major=head_major)[0]
        y = y.permute(1, 2, 0, 3) if head_major else y
        for part in (slice(0, 3), slice(-7, None)):
            check_norm_rope({"q": x[:, part]}, {"q_weight": w}, pos[None, part], "rms", 1, 10000.0, {"q": y[:, part]},
                            torch.bfloat16, 1e-5)
        del y
    clean()
