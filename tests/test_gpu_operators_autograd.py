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
