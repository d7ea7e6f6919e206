"""Timed cases of the operators around the attention layer.

norm_rope   per-head norm of queries and keys with the position rotation in the same pass, values carried along
            (forward and backward): how the layer's inputs are made from a projection.
append      keys and values of new tokens into a paged cache, keys normed and rotated on the way.
attend      a chunk of new tokens of each sequence over its pages of the cache.

`own` false runs plain torch in 32 bits (angles in 64), `own` true the framework's entry points.
"""
import math
import random

import torch

own = False
D = 64      # head dimension of the layer
EPS = 1e-6


def listed():
    return [
        # the tokens of one incoming frame (5 special tokens and a 36 x 36 grid): latency counts
        dict(name="norm_frame", op="norm_rope", back=False, dtype="bf16", norm="layer", axes=2, outer=1, tokens=1301,
             q_heads=16, kv_heads=16, wide=37),
        # the layer's inputs of a whole clip: 128 frames of the 36 x 36 grid
        dict(name="norm_clip", op="norm_rope", back=False, dtype="bf16", norm="layer", axes=2, outer=128, tokens=1296,
             q_heads=16, kv_heads=16, wide=36),
        # token sequences far into a stream, fewer key heads, 32-bit
        dict(name="norm_text_fp32", op="norm_rope", back=False, dtype="fp32", norm="rms", axes=1, outer=2, tokens=1777,
             q_heads=12, kv_heads=4, wide=0),
        # training: gradients of a 32-frame clip on their way back from the layer (which gives them in 32 bits)
        dict(name="norm_back_clip", op="norm_rope", back=True, dtype="bf16", norm="layer", axes=2, outer=32, tokens=1296,
             q_heads=16, kv_heads=16, wide=36),
        # a small ragged training batch in 32 bits
        dict(name="norm_back_fp32", op="norm_rope", back=True, dtype="fp32", norm="rms", axes=1, outer=3, tokens=517,
             q_heads=6, kv_heads=2, wide=0),
        # one new token of each of 48 sequences
        dict(name="append_token", op="append", dtype="bf16", norm="rms", axes=1, batch=48, new_min=1, new_max=1, old_min=100,
             old_max=8000, page=16, kv_heads=4, wide=0),
        # one new frame of each of 8 streams
        dict(name="append_frames", op="append", dtype="bf16", norm="layer", axes=2, batch=8, new_min=1301, new_max=1301,
             old_min=0, old_max=13010, page=64, kv_heads=16, wide=37),
        # a decoding step: one token of each of 48 sequences, ragged lengths, shared key heads, small pages
        dict(name="attend_token", op="attend", dtype="bf16", batch=48, new_min=1, new_max=1, old_min=100, old_max=8000,
             page=16, q_heads=16, kv_heads=4, causal=True, lse=False),
        # one token over a single stream of 200 cached frames
        dict(name="attend_token_long", op="attend", dtype="bf16", batch=1, new_min=1, new_max=1, old_min=260199, old_max=260199,
             page=64, q_heads=16, kv_heads=16, causal=True, lse=False),
        # a new frame over 63 cached ones: every token of it sees the whole frame
        dict(name="attend_frame", op="attend", dtype="bf16", batch=1, new_min=1301, new_max=1301, old_min=81963, old_max=81963,
             page=64, q_heads=16, kv_heads=16, causal=False, lse=False),
        # ragged prompts, some with a cached beginning, causal
        dict(name="attend_prompts", op="attend", dtype="bf16", batch=6, new_min=200, new_max=2000, old_min=0, old_max=3000,
             page=16, q_heads=16, kv_heads=4, causal=True, lse=True),
        # small ragged chunks in 32 bits
        dict(name="attend_fp32", op="attend", dtype="fp32", batch=3, new_min=1, new_max=70, old_min=0, old_max=700, page=32,
             q_heads=4, kv_heads=2, causal=True, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend"])
    kv = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    heads = kv * rng.choice([1, 1, 2, 3, 4])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    while op == "norm_rope":
        axes = rng.choice([1, 2])
        c = dict(op=op, back=rng.random() < 0.4, dtype=dtype, norm=rng.choice(["layer", "rms", "none"]), axes=axes,
                 outer=_log(rng, 1, 128), tokens=_log(rng, 1, 6000), q_heads=heads, kv_heads=kv, wide=rng.randint(1, 48))
        big = listed()[3 if c["back"] else 1]
        if work(c)["bytes"] <= work(big)["bytes"]:
            return c
    while op == "append":
        top = _log(rng, 1, 4000)
        old = _log(rng, 1, 20000)
        c = dict(op=op, dtype=dtype, norm=rng.choice(["layer", "rms", "none"]), axes=rng.choice([1, 2]), batch=_log(rng, 1, 64),
                 new_min=rng.randint(0, top), new_max=top, old_min=rng.randint(0, old), old_max=old,
                 page=rng.choice([16, 32, 64, 128]), kv_heads=kv, wide=rng.randint(1, 48))
        if 0 < work(c)["bytes"] <= work(listed()[6])["bytes"] and sum(_lengths(c)[1]) * kv <= 2500000:
            return c
    while True:
        few = rng.random() < 0.5
        top = rng.randint(1, 6) if few else _log(rng, 7, 2500)
        old = _log(rng, 10, 270000 if few else 90000)
        c = dict(op=op, dtype=dtype, batch=_log(rng, 1, 64), new_min=rng.randint(1, top), new_max=top,
                 old_min=rng.randint(0, old), old_max=old, page=rng.choice([16, 32, 64, 128]), q_heads=heads, kv_heads=kv,
                 causal=rng.random() < 0.7, lse=rng.random() < 0.5)
        new, total = _lengths(c)
        w = work(c)
        share = 16 if dtype == "fp32" else 1      # 32-bit products cost more
        if (w["flops"] * share <= work(listed()[9])["flops"] and w["bytes"] <= work(listed()[8])["bytes"]
                and len(new) * max(total) * kv <= 4500000 and len(new) * heads * max(new) * max(total) <= 1700000000):
            return c


def _lengths(c):
    """New tokens of each sequence, and its cached length with them: the same for every seed, so that work() knows them."""
    r = random.Random(c["batch"] * 7919 + c["new_max"] * 31 + c["old_max"])
    new = [r.randint(c["new_min"], c["new_max"]) for _ in range(c["batch"])]
    old = [r.randint(c["old_min"], c["old_max"]) for _ in range(c["batch"])]
    return new, [n + o for n, o in zip(new, old)]


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm_rope":
        t, hq, hk = c["outer"] * c["tokens"], c["q_heads"], c["kv_heads"]
        if c["back"]:      # queries and keys again, three gradients in and out in 32 bits
            return {"bytes": t * D * ((hq + hk) * e + 8 * (hq + 2 * hk)), "flops": t * D * (hq + hk) * 20}
        return {"bytes": 2 * t * D * (hq + 2 * hk) * e, "flops": t * D * (hq + hk) * 12}
    new, total = _lengths(c)
    if c["op"] == "append":
        return {"bytes": 4 * sum(new) * c["kv_heads"] * D * e, "flops": sum(new) * c["kv_heads"] * D * 12}
    pairs = sum(n * (l - n) + n * (n + 1) // 2 if c["causal"] else n * l for n, l in zip(new, total))
    return {"bytes": 2 * sum(new) * c["q_heads"] * D * e + 2 * sum(total) * c["kv_heads"] * D * e,
            "flops": 4 * D * c["q_heads"] * pairs}


def _weights(c, g, dt):
    """Norm weights near one and small biases, as a trained model has them."""
    w = {}
    if c["norm"] != "none":
        w = {"q_weight": 1 + 0.2 * torch.randn(D, generator=g, device="cuda"), "k_weight": 1 + 0.2 * torch.randn(D, generator=g, device="cuda")}
    if c["norm"] == "layer":
        w["q_bias"] = 0.1 * torch.randn(D, generator=g, device="cuda")
        w["k_bias"] = 0.1 * torch.randn(D, generator=g, device="cuda")
    return {k: v.to(dt) for k, v in w.items()}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    s = {"case": c}
    if c["op"] == "norm_rope":
        n, t, hq, hk = c["outer"], c["tokens"], c["q_heads"], c["kv_heads"]
        s["w"] = _weights(c, g, dt)
        s["q"], s["k"], s["v"] = (rand(n, t, hq, D) * 1.5 + 0.2).to(dt), (rand(n, t, hk, D) * 1.5 - 0.1).to(dt), rand(n, t, hk, D).to(dt)
        at = torch.arange(t, device="cuda", dtype=torch.int32)
        if c["axes"] == 2:      # the patch grid, the same for every frame
            s["positions"] = torch.stack([at // c["wide"] + 1, at % c["wide"] + 1], dim=1).to(torch.int32).contiguous()
            s["base"] = 100.0
        else:                   # far into a stream
            far = torch.randint(0, 1000000, (n, 1), generator=g, device="cuda", dtype=torch.int32)
            s["positions"] = (far + at[None]).to(torch.int32).unsqueeze(-1).contiguous()
            s["base"] = 10000.0
        if c["back"]:           # gradients in the layer's layout [heads][frames][tokens][64]
            s["dq"], s["dk"], s["dv"] = rand(hq, n, t, D), rand(hk, n, t, D), rand(hk, n, t, D)
        return s
    new, total = _lengths(c)
    hk, page = c["kv_heads"], c["page"]
    need = [(l + page - 1) // page for l in total]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda", dtype=torch.int64)
    wide = max(max(need), 1)
    slot = first[:, None] + torch.arange(wide, device="cuda")[None]
    s["table"] = order[slot.clamp(max=pages - 1)].contiguous()
    s["k_pages"] = rand(pages, hk, page, D).to(dt)
    s["v_pages"] = rand(pages, hk, page, D).to(dt)
    i32 = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"], s["total"], s["old"] = i32(cu), i32(total), i32([l - n for n, l in zip(new, total)])
    s["tokens"], s["most_new"], s["most"] = cu[-1], max(new), max(total)
    if c["op"] == "append":
        s["w"] = {k: v for k, v in _weights(c, g, dt).items() if k[0] == "k"}
        s["k"], s["v"] = (rand(cu[-1], hk, D) * 1.5 - 0.1).to(dt), rand(cu[-1], hk, D).to(dt)
        if c["axes"] == 2:
            at = torch.arange(cu[-1], device="cuda")
            s["positions"] = torch.stack([at // c["wide"] % 40 + 1, at % c["wide"] + 1], dim=1).to(torch.int32).contiguous()
            s["base"] = 100.0
        else:
            s["positions"], s["base"] = None, 10000.0      # a token's place in its sequence
    else:
        s["q"] = (rand(cu[-1], c["q_heads"], D) * 1.5).to(dt)
    return s


# ---- the framework's calls -------------------------------------------------------------
def _run_own(s):
    import sparse_global_attention_b200 as gsa
    c = s["case"]
    if c["op"] == "norm_rope":
        if c["back"]:
            return gsa.qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], s["dv"], norm=c["norm"], eps=EPS,
                                             positions=s["positions"], rope_base=s["base"], head_major=True, **s["w"])
        return gsa.qk_norm_rope(s["q"], s["k"], s["v"], norm=c["norm"], eps=EPS, positions=s["positions"],
                                rope_base=s["base"], head_major=True, **s["w"])
    cache = s.get("cache")
    if cache is None:      # a program keeps the handle of its cache
        cache = s["cache"] = gsa.KVCache.from_pages(s["k_pages"], s["v_pages"])
    if c["op"] == "append":
        cache.append(s["k"], s["v"], s["table"], s["old"], s["cu"], norm=c["norm"], eps=EPS, positions=s["positions"],
                     rope_axes=c["axes"], rope_base=s["base"], **s["w"])
        return s["k_pages"], s["v_pages"]
    return cache.attention(s["q"], s["table"], s["total"], s["cu"], s["most_new"], max_len=s["most"], causal=c["causal"],
                           return_lse=c["lse"])


# ---- the plain form -------------------------------------------------------------------
def _norm(x, norm, weight, bias):
    if norm == "none":
        return x
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight.float()
    return x + bias.float() if bias is not None else x


def _angles(positions, axes, base):
    """cos and sin [..., axes, 1, 32 / axes] of positions [..., axes], from angles in 64 bits."""
    half = D // 2 // axes
    f = torch.pow(torch.tensor(base, device=positions.device, dtype=torch.float64),
                  -torch.arange(half, device=positions.device, dtype=torch.float64) / half)
    a = positions.double().unsqueeze(-1) * f
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, axes):
    """x [..., heads, 64] by cos, sin [..., axes, 32 / axes]: each axis turns its own 64 / axes dimensions."""
    y = x.unflatten(-1, (axes, 2, D // 2 // axes))
    c, s = cos.unsqueeze(-3), sin.unsqueeze(-3)
    a, b = y[..., 0, :], y[..., 1, :]
    return torch.stack([a * c - b * s, b * c + a * s], dim=-2).flatten(-3)


def _plain_norm_rope(s):
    c = s["case"]
    cos, sin = _angles(s["positions"], c["axes"], s["base"])
    out = []
    for x, w, b in ((s["q"], "q_weight", "q_bias"), (s["k"], "k_weight", "k_bias")):
        y = _rotate(_norm(x.float(), c["norm"], s["w"].get(w), s["w"].get(b)), cos, sin, c["axes"])
        out.append(y.to(x.dtype).permute(2, 0, 1, 3).contiguous())
    return out[0], out[1], s["v"].permute(2, 0, 1, 3).contiguous()


def _plain_back_one(x, dy, norm, weight, cos, sin, axes):
    """Gradients of one tensor, its weight and its bias."""
    g = _rotate(dy.permute(1, 2, 0, 3), cos, -sin, axes)
    if norm == "none":
        return g.contiguous(), None, None
    x = x.float()
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    h = x * r
    u = g * weight.float()
    dx = u - h * (u * h).mean(-1, keepdim=True)
    if norm == "layer":
        dx = dx - u.mean(-1, keepdim=True)
    dw = (g * h).sum((0, 1, 2))
    return (dx * r).contiguous(), dw, g.sum((0, 1, 2)) if norm == "layer" else None


def _plain_back(s):
    c = s["case"]
    cos, sin = _angles(s["positions"], c["axes"], s["base"])
    dq, dqw, dqb = _plain_back_one(s["q"], s["dq"], c["norm"], s["w"].get("q_weight"), cos, sin, c["axes"])
    dk, dkw, dkb = _plain_back_one(s["k"], s["dk"], c["norm"], s["w"].get("k_weight"), cos, sin, c["axes"])
    return {"dq": dq, "dk": dk, "dv": s["dv"].permute(1, 2, 0, 3).contiguous(), "dq_weight": dqw, "dq_bias": dqb,
            "dk_weight": dkw, "dk_bias": dkb}


def _plain_append(s):
    c = s["case"]
    at = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].contiguous(), at.to(torch.int32), right=True)
    place = at - s["cu"][seq] + s["old"][seq]
    pos = s["positions"] if s["positions"] is not None else place.unsqueeze(-1)
    cos, sin = _angles(pos, c["axes"], s["base"])
    k = _rotate(_norm(s["k"].float(), c["norm"], s["w"].get("k_weight"), s["w"].get("k_bias")), cos, sin, c["axes"])
    page, row = s["table"][seq, place // c["page"]].long(), place % c["page"]
    s["k_pages"][page, :, row] = k.to(s["k_pages"].dtype)
    s["v_pages"][page, :, row] = s["v"]
    return s["k_pages"], s["v_pages"]


def _plain_attend(s):
    c = s["case"]
    hq, hk, dev = c["q_heads"], c["kv_heads"], "cuda"
    n, l = s["cu"].diff(), s["total"]
    i = torch.arange(s["most_new"], device=dev)
    j = torch.arange(s["most"], device=dev)
    real = i[None] < n[:, None]
    token = (s["cu"][:-1, None] + i[None]).clamp(max=s["tokens"] - 1)
    q = s["q"][token].float().unflatten(2, (hk, hq // hk)).permute(0, 2, 1, 3, 4).flatten(2, 3) * D ** -0.5
    used = s["table"][:, :-(-s["most"] // c["page"])].long()
    k, v = (p[used].float().transpose(1, 2).flatten(2, 3)[:, :, :s["most"]] for p in (s["k_pages"], s["v_pages"]))
    score = q @ k.transpose(-1, -2)                                  # [batch, kv heads, new * shared, keys]
    end = (l - n)[:, None] + i[None] + 1 if c["causal"] else l[:, None].expand(-1, s["most_new"])
    end = end.repeat_interleave(hq // hk, 1)
    score.masked_fill_((j[None, None] >= end[:, :, None])[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    weight = score.sum(-1, keepdim=True)
    o = (score @ v) / weight.masked_fill(weight == 0, 1.0)
    lse = (top + weight.log()).squeeze(-1)
    unpack = lambda x: x.unflatten(2, (s["most_new"], hq // hk)).transpose(1, 2).flatten(2, 3)[real]
    out = unpack(o).to(s["q"].dtype)
    return (out, unpack(lse).T.contiguous()) if c["lse"] else out


def run(state):
    c = state["case"]
    if own:
        return _run_own(state)
    if c["op"] == "norm_rope":
        return _plain_back(state) if c["back"] else _plain_norm_rope(state)
    return _plain_append(state) if c["op"] == "append" else _plain_attend(state)


# ---- the definition, in 64 bits ---------------------------------------------------------
def _exact_matrix(pos, axes, base):
    """Rotation matrices [n, 64, 64] of n positions [n, axes]."""
    r = torch.zeros(pos.shape[0], D, D, dtype=torch.float64, device=pos.device)
    span = D // axes
    for a in range(axes):
        for f in range(span // 2):
            t = pos[:, a].double() * base ** (-2.0 * f / span)
            x, y = a * span + f, a * span + f + span // 2
            r[:, x, x] = t.cos()
            r[:, y, y] = t.cos()
            r[:, x, y] = -t.sin()
            r[:, y, x] = t.sin()
    return r


def _exact_hat(x, norm):
    """Normed rows without weight, and the factor of each row."""
    x = x.double()
    if norm == "none":
        return x, torch.ones_like(x[..., :1])
    mid = x.mean(-1, keepdim=True) if norm == "layer" else torch.zeros_like(x[..., :1])
    inv = 1.0 / torch.sqrt(((x - mid) ** 2).mean(-1, keepdim=True) + EPS)
    return (x - mid) * inv, inv


def _exact_normed(x, norm, w, b):
    y, _ = _exact_hat(x, norm)
    if w is not None:
        y = y * w.double()
    return y if b is None else y + b.double()


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    w = s.get("w", {})
    if c["op"] == "norm_rope":
        if c["outer"] * c["tokens"] * (c["q_heads"] + 2 * c["kv_heads"]) > 9000000:
            return None                                             # over 20 GB in 64 bits
        n, t = c["outer"], c["tokens"]
        pos = s["positions"].expand(n, t, c["axes"]) if s["positions"].dim() == 2 else s["positions"]
        grid = _exact_matrix(pos[0], 2, s["base"]) if c["axes"] == 2 else None      # one grid for all frames
        turn = lambda o: grid if grid is not None else _exact_matrix(pos[o], 1, s["base"])
        if not c["back"]:
            res = []
            for x, a in ((s["q"], "q"), (s["k"], "k")):
                y = [torch.einsum("tij,thj->hti", turn(o), _exact_normed(x[o], c["norm"], w.get(a + "_weight"), w.get(a + "_bias")))
                     for o in range(n)]
                res.append(torch.stack(y, 1))
            return res[0], res[1], s["v"].double().permute(2, 0, 1, 3).contiguous()
        out = {"dv": s["dv"].double().permute(1, 2, 0, 3).contiguous()}
        for a in ("q", "k"):
            dx, dw, db = [], 0, 0
            for o in range(n):
                g = torch.einsum("tij,hti->thj", turn(o), s["d" + a][:, o].double())
                hat, inv = _exact_hat(s[a][o], c["norm"])
                if c["norm"] == "none":
                    dx.append(g)
                    continue
                dw, db = dw + (g * hat).sum((0, 1)), db + g.sum((0, 1))
                u = g * w[a + "_weight"].double()
                d = u - hat * (u * hat).mean(-1, keepdim=True)
                dx.append(inv * (d - u.mean(-1, keepdim=True) if c["norm"] == "layer" else d))
            out["d" + a] = torch.stack(dx)
            out["d%s_weight" % a] = dw if c["norm"] != "none" else None
            out["d%s_bias" % a] = db if c["norm"] == "layer" else None
        return out
    new, total = _lengths(c)
    cu = s["cu"].tolist()
    if c["op"] == "append":
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        for b, (n, l) in enumerate(zip(new, total)):
            if not n:
                continue
            place = torch.arange(l - n, l, device="cuda")
            at = slice(cu[b], cu[b + 1])
            pos = s["positions"][at] if s["positions"] is not None else place[:, None]
            k = torch.einsum("tij,thj->thi", _exact_matrix(pos, c["axes"], s["base"]),
                             _exact_normed(s["k"][at], c["norm"], w.get("k_weight"), w.get("k_bias")))
            page = s["table"][b][place // c["page"]].long()
            k_pages[page, :, place % c["page"]] = k
            v_pages[page, :, place % c["page"]] = s["v"][at].double()
        return k_pages, v_pages
    out = torch.zeros(cu[-1], c["q_heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["q_heads"], cu[-1], dtype=torch.float64, device="cuda")
    share = c["q_heads"] // c["kv_heads"]
    for b, (n, l) in enumerate(zip(new, total)):
        pages = s["table"][b, :-(-l // c["page"])].long()
        for h in range(c["q_heads"]):
            k, v = (p[pages, h // share].reshape(-1, D)[:l].double() for p in (s["k_pages"], s["v_pages"]))
            x = s["q"][cu[b]:cu[b + 1], h].double() @ k.T / math.sqrt(D)
            if c["causal"]:
                ahead = torch.arange(l, device="cuda")[None] > torch.arange(l - n, l, device="cuda")[:, None]
                x = x.masked_fill(ahead, -math.inf)
            lse[h, cu[b]:cu[b + 1]] = torch.logsumexp(x, -1)
            out[cu[b]:cu[b + 1], h] = torch.softmax(x, -1) @ v
    return (out, lse) if c["lse"] else out
