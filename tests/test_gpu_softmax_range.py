"""Online softmax over scores whose running maximum moves far: between two key tiles
the factor that brings the sums so far to the new maximum, 2^((old - new) log2 e scale),
can underflow to zero, and the output so far has to be multiplied by that zero as the
sum of the weights is.

Keys lie along (1, .., 1) at a level of their own group of places, so a group's scaled
scores are 8 * level * query, and each group's values have a mean of their own: a group
that stays in the output although its weight is gone moves it by the means' distance.
Tolerances: those of test_gpu_operators (attention over the cache) and of gpu_helpers (the layer)."""
import pytest
import torch

import oracle
import sparse_global_attention_b200 as gsa
from gpu_helpers import assert_close, compare_head, run_gpu
from gsa_inputs import GSAConfig, make_inputs, to_f64_numpy
from test_gpu_operators import TYPES, Streams, check_attention, clean

pytestmark = pytest.mark.gpu

# (places up to which a level holds, as parts of the length; levels in 32nds, a quarter of which is a unit query's scaled score)
RISING = ((0.31, 0.72, 1.0), (-800, -100, 400))         # -200, -25, 100
FALLING = ((0.31, 0.72, 1.0), (400, -100, -800))
JUST = ((0.31, 0.72, 1.0), (-200, 0, 240))              # -50, 0, 60: factors of 2^-72 and 2^-87, no underflow
LATE = ((0.93, 1.0), (-480, 480))                       # -120, 120: 2^-346


def levels(length, steps, device="cuda"):
    at = torch.arange(length, device=device)
    ends, values = steps
    k = torch.full((length,), values[-1] / 32.0, device=device)
    for e, v in reversed(list(zip(ends, values))):
        k[at < round(e * length)] = v / 32.0
    return k


def keys_and_values(g, length, heads, steps, dtype):
    """Keys at their levels, and values 5, 1, -3 (by the group of places) with noise."""
    k = levels(length, steps)
    mean = torch.full((length,), 5.0, device="cuda")
    for i, e in enumerate(steps[0][:-1]):
        mean[torch.arange(length, device="cuda") >= round(e * length)] = 1.0 - 4.0 * i
    noise = torch.randn(length, heads, 64, generator=g, device="cuda")
    near = torch.randn(length, heads, 64, generator=g, device="cuda") / 16       # scores of a group spread by 1/16
    return (k[:, None, None] + near).to(dtype), (mean[:, None, None] + 0.5 * noise).to(dtype)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("steps", [RISING, FALLING, JUST, LATE], ids=["rising", "falling", "just", "late"])
@pytest.mark.parametrize("rows", ["same", "mixed"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,hk,group", [(1, 2, 1), (1, 2, 4), (5, 1, 3), (50, 2, 1), (300, 1, 1), (100, 1, 5)])
def test_cache_attention_when_the_maximum_moves_far(n, hk, group, dtype, rows, steps, causal):
    dt, lengths = TYPES[dtype], [1100, 777]
    s = Streams([n, n], [t - n for t in lengths], 16, hk, dt, seed=n + group)
    parts = [keys_and_values(s.g, t, hk, steps, dt) for t in lengths]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    s.cache.append(torch.cat([k for k, _ in parts]), torch.cat([v for _, v in parts]), s.table, i32([0, 0]),
                   i32([0, lengths[0], sum(lengths)]))
    q = torch.ones(2 * n, hk * group, 64, device="cuda")
    if rows == "mixed":      # in one warp rows whose maximum rises, falls and stays
        q *= torch.tensor([1.0, -1.0, 0.25, 0.0], device="cuda")[torch.arange(q.shape[0] * q.shape[1], device="cuda") % 4].view(
            q.shape[0], -1, 1)
    q = q.to(dt)
    for max_len in (1, 300, 200000):           # one part, and several
        out, lse = s.cache.attention(q, s.table, s.lengths, s.cu, n, max_len=max_len, causal=causal, return_lse=True)
        check_attention(s, q, out, lse, causal)
    clean()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,group", [(1, 1), (9, 2), (50, 1), (300, 1)])
def test_cache_attention_weights_that_are_zero(n, group, dtype):
    """Scores of -inf throughout a sequence: 0 and -inf, as for a query without a key.  Keys whose weight underflows
    (2^-432 of the largest) add nothing, however large their values are: 2^126, of which 2^-126 would be one a key."""
    dt, lengths = TYPES[dtype], [900, 700]
    s = Streams([n, n], [t - n for t in lengths], 64, 1, dt, seed=n)
    k0, v0 = keys_and_values(s.g, lengths[0], 1, FALLING, dt)
    k0[:, 0, 0] = float("-inf")
    k1, v1 = keys_and_values(s.g, lengths[1], 1, ((0.5, 1.0), (400, -800)), dt)
    v1[350:] = 2.0 ** 126
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    s.cache.append(torch.cat([k0, k1]), torch.cat([v0, v1]), s.table, i32([0, 0]), i32([0, lengths[0], sum(lengths)]))
    q = torch.ones(2 * n, group, 64, device="cuda", dtype=dt)
    out, lse = s.cache.attention(q, s.table, s.lengths, s.cu, n, max_len=1, causal=False, return_lse=True)
    check_attention(s, q, out, lse, False)
    assert (out[:n] == 0).all() and (lse[:, :n] == float("-inf")).all()
    clean()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 50, 300])
def test_cache_attention_with_scales_at_the_ends(n, dtype):
    """A scale so small that all keys weigh the same, and one that 32 bits would hold as 0, which stands for 1 / 8."""
    s = Streams([n], [700 - n], 16, 1, TYPES[dtype], seed=n)
    s.cache.append(s.rand(n, 1), s.rand(n, 1), s.table, s.start, s.cu)
    q = s.rand(n, 1)
    for scale in (1e-40, 1e-30):
        out, lse = s.cache.attention(q, s.table, s.lengths, s.cu, n, softmax_scale=scale, return_lse=True)
        check_attention(s, q, out, lse, True, scale=scale)
    for scale in (1e-60, 2.4e38, 1e39, float("nan")):
        with pytest.raises(gsa.GSAError):
            s.cache.attention(q, s.table, s.lengths, s.cu, n, softmax_scale=scale)
    clean()


# ---- the layer's kernels --------------------------------------------------------------------
WIDE = GSAConfig("wide_bf16", 6, 24, 24, 24, 24, 5, 2, 64, 4, 32, "bf16")      # R = 216 regions: two key tiles
FIXED = GSAConfig("wide_fixed_bf16", 6, 24, 24, 24, 24, 5, 2, 64, 4, 16, "bf16", (0, 4))


def layer_inputs(cfg, low, high, value):
    """Queries near one; keys at `low` in the first frames and at `high` in the last ones (`value` the frame and the
    region row that they begin at), values 1 and -1 with noise (small: the bar on the outputs is absolute)."""
    frame, rows = value
    x = {k: v.float() for k, v in make_inputs(cfg, seed=2).items()}
    g = torch.Generator().manual_seed(5)
    late = torch.zeros(cfg.num_frames, cfg.pad_h, 1, 1)
    late[frame + 1:] = 1
    late[frame, 4 * rows:] = 1
    spec = torch.zeros(cfg.num_frames, 1, 1)
    spec[frame:] = 1
    for part, at in (("img", late), ("spec", spec)):
        noise = lambda: torch.randn(x["q_" + part].shape, generator=g)
        x["q_" + part] = 1 + noise() / 8
        x["k_" + part] = low + (high - low) * at + noise() / 8
        x["v_" + part] = 1 - 2 * at + noise() / 8
    return {k: v.bfloat16().cuda() for k, v in x.items()}


JUMPS = [(-25.0, 12.5, (4, 0)),       # scores -200 and 100, from region 144 on: inside the second tile
         (-25.0, 12.5, (5, 2)),       # from region 192 on: the second half of that tile
         (-6.25, 7.5, (4, 0)),        # -50 and 60: 2^-159
         (-4.0, 4.0, (4, 0)),         # -32 and 32: 2^-92, no underflow
         (12.5, -25.0, (4, 0))]       # falling


@pytest.mark.parametrize("low,high,value", JUMPS)
@pytest.mark.parametrize("cfg", [WIDE, FIXED], ids=lambda c: c.name)
def test_layer_when_the_maximum_moves_far(cfg, low, high, value):
    """Compressed attention, special tokens and (FIXED) the fixed context."""
    x = layer_inputs(cfg, low, high, value)
    res = run_gpu(cfg, x)
    for h in range(cfg.num_heads):
        compare_head(cfg, x, res, h)


@pytest.mark.parametrize("low,high,value", JUMPS)
def test_dense_attention_when_the_maximum_moves_far(low, high, value):
    cfg = WIDE
    H, F, d = cfg.num_heads, cfg.num_frames, 64
    x = layer_inputs(cfg, low, high, value)
    q, k, v = (torch.cat([x[n + "_spec"], x[n + "_img"].reshape(H, F, -1, d)], dim=2).reshape(H, -1, d).contiguous()
               for n in "qkv")
    layer = gsa.GSALayer.from_workload(cfg)
    o = layer.dense(q, k, v)
    torch.cuda.synchronize()
    status = layer.status()
    layer.close()
    assert status == 0
    for h in range(H):
        want = oracle.dense_attention(to_f64_numpy(q[h]), to_f64_numpy(k[h]), to_f64_numpy(v[h]))
        assert_close("dense", o[h].float().cpu().numpy(), want, cfg)
