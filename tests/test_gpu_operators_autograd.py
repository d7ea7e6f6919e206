"""What autograd learns of the operators around the layer."""
import pytest
import torch

import sparse_global_attention_b200 as gsa
from test_gpu_operators import Streams, clean

pytestmark = pytest.mark.gpu


def rows(*shape):
    return torch.randn(*shape, 64, device="cuda")


@pytest.mark.parametrize("inference", [False, True])
def test_written_tensors_have_a_new_version(inference):
    """Tensors of the caller's that a call writes: a product that was saved from them cannot be differentiated any more
    (in inference mode tensors have no version, and the calls write them as well)."""
    with torch.inference_mode(inference):
        version = (lambda t: 0) if inference else (lambda t: t._version)
        step = 0 if inference else 1
        q, k, out = rows(2, 9, 4), rows(2, 9, 2), [rows(2, 9, 4), rows(2, 9, 2), None]
        was = [version(t) for t in (*out[:2], q, k)]
        gsa.qk_norm_rope(q, k, norm="none", out=out)
        assert [version(t) for t in (*out[:2], q, k)] == [was[0] + step, was[1] + step, was[2], was[3]]
        assert torch.equal(out[0], q) and torch.equal(out[1], k)
        room = rows(3, 2, 9, 4)
        was = version(room)
        gsa.qk_norm_rope_backward(None, None, q, None, q, norm="none", out=(room[0], None, room[1]))
        assert version(room) == was + 2 * step and torch.equal(room[0], q) and torch.equal(room[1], q)
        s = Streams([3], [5], 16, 2, torch.float32)
        was = version(s.cache.k_pages), version(s.cache.v_pages)
        s.cache.append(rows(3, 2), rows(3, 2), s.table, s.start, s.cu)
        assert (version(s.cache.k_pages), version(s.cache.v_pages)) == (was[0] + step, was[1] + step)
        x, out = rows(3, 4), rows(3, 4)
        was = version(out), version(x), version(s.cache.k_pages)
        s.cache.attention(x, s.table, s.lengths, s.cu, 3, out=out)
        assert (version(out), version(x), version(s.cache.k_pages)) == (was[0] + step, was[1], was[2])
    # written outside the mode
    gsa.qk_norm_rope(q, norm="none", out=(room[2], None, None))
    assert torch.equal(room[2], q)
    clean()


def test_saved_tensors_that_a_call_overwrote():
    w = rows(2, 9, 4).requires_grad_()
    x = rows(2, 9, 4)
    y = (w * x).sum()
    with torch.no_grad():
        gsa.qk_norm_rope(rows(2, 9, 4), norm="none", out=(x, None, None))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_results_of_inputs_that_require_a_gradient():
    """No gradient is recorded: asking for one raises, at the results that depend on such an input and at no other."""
    q, k, v = rows(2, 9, 4), rows(2, 9, 2), rows(2, 9, 2)
    w = torch.ones(64, device="cuda")
    call = lambda **kw: gsa.qk_norm_rope(kw.pop("q", q), k, kw.pop("v", v), norm="layer", **{**dict(q_weight=w, k_weight=w), **kw})
    want = call()
    assert not any(t.requires_grad for t in want)
    leaf = lambda t: t.clone().requires_grad_()
    for kw, depends in ((dict(q=leaf(q)), (1, 0, 0)), (dict(v=leaf(v)), (0, 0, 1)), (dict(k_weight=leaf(w)), (0, 1, 0)),
                        (dict(q_bias=leaf(0 * w), k_weight=leaf(w)), (1, 1, 0))):
        got = call(**kw)
        assert [t.requires_grad for t in got] == [bool(d) for d in depends]
        assert all(torch.equal(a.detach(), b) for a, b in zip(got, want))
        for t, d in zip(got, depends):
            if d:
                with pytest.raises(RuntimeError, match="qk_norm_rope_backward"):
                    t.square().sum().backward()
        assert all(t.grad is None for t in kw.values())
        with torch.no_grad():
            assert not any(t.requires_grad for t in call(**kw))
        with torch.inference_mode():
            assert not any(t.requires_grad for t in call(**kw))
    # weights that a call without a norm does not read
    out = rows(2, 9, 4)
    got = gsa.qk_norm_rope(q, k, norm="none", q_weight=leaf(w), k_weight=leaf(w), out=(out, None, None))
    assert got[0] is out and not got[1].requires_grad and torch.equal(out, q)
    s = Streams([3], [5], 16, 2, torch.float32)
    s.cache.append(rows(3, 2), rows(3, 2), s.table, s.start, s.cu, norm="none", k_weight=leaf(w))
    # the gradients' call takes such tensors and records nothing itself
    r = gsa.qk_norm_rope_backward(leaf(q), None, rows(2, 9, 4), None, norm="rms", q_weight=leaf(w))
    assert not r["dq"].requires_grad and not r["dq_weight"].requires_grad


def test_memory_of_the_caller_takes_no_values_that_require_a_gradient():
    q, k = rows(2, 9, 4), rows(2, 9, 2)
    out = rows(2, 9, 4)
    was = out.clone()
    leaf = lambda t: t.clone().requires_grad_()
    for kw in (dict(q=leaf(q), out=(out, None, None)), dict(q=q, out=(leaf(out), None, None))):
        with pytest.raises(gsa.GSAError, match="no_grad"):
            gsa.qk_norm_rope(kw["q"], norm="none", out=kw["out"])
    assert torch.equal(out, was)
    # the other tensors' outputs may be given
    got = gsa.qk_norm_rope(leaf(q), k, norm="none", out=(None, rows(2, 9, 2), None))
    assert got[0].requires_grad and not got[1].requires_grad
    with torch.no_grad():
        gsa.qk_norm_rope(leaf(q), norm="none", out=(out, None, None))
    assert torch.equal(out, q)
    s = Streams([3], [5], 16, 2, torch.float32)
    k, v, x, w = rows(3, 2), rows(3, 2), rows(3, 4), torch.ones(64, device="cuda")
    pages = s.cache.k_pages.clone()
    for kw in (dict(k=leaf(k), v=v), dict(k=k, v=leaf(v)), dict(k=k, v=v, norm="rms", k_weight=leaf(w))):
        with pytest.raises(gsa.GSAError, match="no_grad"):
            s.cache.append(block_table=s.table, start=s.start, cu_tokens=s.cu, **kw)
    assert torch.equal(s.cache.k_pages.nan_to_num(), pages.nan_to_num())
    with torch.no_grad():
        s.cache.append(leaf(k), leaf(v), s.table, s.start, s.cu)
    want = s.cache.attention(x, s.table, s.lengths, s.cu, 3)
    out, lse = s.cache.attention(leaf(x), s.table, s.lengths, s.cu, 3, return_lse=True)
    assert torch.equal(out.detach(), want) and not want.requires_grad
    for t in (out, lse):
        with pytest.raises(RuntimeError, match="no gradient"):
            t.sum().backward()
    with pytest.raises(gsa.GSAError, match="no_grad"):
        s.cache.attention(leaf(x), s.table, s.lengths, s.cu, 3, out=rows(3, 4))
    with torch.no_grad():
        assert torch.equal(s.cache.attention(leaf(x), s.table, s.lengths, s.cu, 3, out=rows(3, 4)), want)
    clean()


def test_layer_inputs_of_a_projection_that_requires_a_gradient():
    """The way back by the calls of its own, next to autograd's part."""
    from gsa_inputs import GSAConfig
    cfg = GSAConfig("autograd_small", 2, 8, 8, 8, 8, 1, 2, 64, 4, 4, "bf16")
    layer = gsa.GSALayer.from_workload(cfg)
    try:
        g = torch.Generator(device="cuda").manual_seed(0)
        src = torch.randn(2, 65, 3, 2, 64, generator=g, device="cuda").requires_grad_()
        w_g = (torch.randn(2, 64, 64, generator=g, device="cuda") / 8).bfloat16()
        w = torch.ones(64, device="cuda", dtype=torch.bfloat16).requires_grad_()
        d = {n: torch.randn(2, 2, *s, 64, generator=g, device="cuda").bfloat16() for n, s in (("o_img", (8, 8)), ("o_spec", (1,)))}
        res, grads = [], None
        for grad in (True, False):
            with torch.set_grad_enabled(grad):
                qkv = src.bfloat16()
                kw = dict(norm="rms", q_weight=w, k_weight=w)
                x = layer.split_qkv(qkv, w_g, **kw)
                assert x["q_img"].requires_grad == grad
                out = layer.forward(x)
                grads = grads or layer.backward(x, out, d)
                r = layer.split_qkv_backward(qkv, grads, **kw)
                assert not any(t is not None and t.requires_grad for t in r.values())
                res.append((out, r))
                if grad:
                    qkv.backward(r["dqkv"].bfloat16())
                    assert torch.equal(src.grad, r["dqkv"].bfloat16().float())
        assert layer.status() == 0
        for a, b in zip(*res):
            assert all(torch.equal(a[n], b[n]) for n in a if a[n] is not None)
    finally:
        layer.close()
    clean()
