"""Cases that measure the linear layer, the cross attention and the 1-D rotary
embedding, with a plain form of each in elementary torch operations.

``listed()`` gives the fixed cases, ``draw(rng)`` more of the same ranges,
``prepare(case, seed)`` a case's inputs on the GPU, ``run(state)`` one pass:
in plain form while ``own`` is false, through the library's entry points while
it is true. ``work(case)`` counts the bytes and operations a pass cannot do
without, ``exact(case, seed)`` is the definition in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- the cases

def _rope(tokens, heads, kv_heads, head_dim, rot_dim, layout, scaling, dtype, first, fused, **kw):
    return dict(kw, op="rope", tokens=tokens, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                rot_dim=rot_dim, layout=layout, scaling=scaling, dtype=dtype, first=first,
                fused=fused)


def _linear(rows, features, inputs, act, gated, bias, residual, dtype, **kw):
    return dict(kw, op="linear", rows=rows, features=features, inputs=inputs, act=act,
                gated=gated, bias=bias, residual=residual, dtype=dtype)


def _cross(queries, keys, heads, kv_heads, head_dim, masked, lse, dtype, **kw):
    """``queries`` and ``keys``: the segments' lengths, "a,b,c"."""
    return dict(kw, op="cross", queries=queries, keys=keys, heads=heads, kv_heads=kv_heads,
                head_dim=head_dim, masked=masked, lse=lse, dtype=dtype)


def listed():
    return [
        # one token a sequence at far positions, 64 query and 8 key heads: a decoding step
        _rope(4, 64, 8, 128, 128, "half", "yarn", "bf16", 120000, False, name="rope_step"),
        # odd length, a head of 80 of which 40 channels rotate, 32-bit values
        _rope(777, 12, 12, 80, 40, "interleaved", "none", "fp32", 0, False, name="rope_odd"),
        # a batch of prompts, half of the head, read out of the fused projection's output
        _rope(8320, 64, 8, 128, 64, "interleaved", "linear", "fp16", 0, True, name="rope_prompt"),
        # one very long context
        _rope(131072, 64, 8, 128, 128, "half", "yarn", "bf16", 0, False, name="rope_long"),
        # the modulation of one timestep: a weight read once for two rows
        _linear(2, 6 * 5376, 5376, "none", False, True, False, "bf16", name="linear_modulation"),
        # odd sizes, a tanh GELU
        _linear(1001, 1003, 1000, "gelu_tanh", False, True, True, "fp16", name="linear_odd"),
        # attention output projection of one clip, added to the residual stream
        _linear(8320, 5376, 7168, "none", False, True, True, "bf16", name="linear_out"),
        # gated feed-forward of one clip, gate and up in one product
        _linear(8320, 14336, 5376, "silu", True, False, False, "bf16", name="linear_gated"),
        # one token of each of eight sequences attends to its encoder states
        _cross("1,1,1,1,1,1,1,1", "8192,517,4096,1,2048,7000,33,1024", 64, 8, 128, False, True,
               "fp16", name="cross_step"),
        # learned queries that read a long clip, part of it masked out
        _cross("64", "33280", 24, 24, 64, True, False, "bf16", name="cross_reader"),
        # one clip attends to 512 states of its text
        _cross("8320", "512", 56, 56, 128, False, False, "bf16", name="cross_clip"),
        # four packed clips, four texts of their own lengths
        _cross("5120,12288,20480,33024", "77,300,512,1021", 40, 40, 128, False, False, "bf16",
               name="cross_packed"),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over their logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("rope", "linear", "cross"))
    if op == "rope":
        head_dim = rng.choice((64, 80, 96, 128, 256))
        kv_heads = rng.choice((1, 2, 5, 8, 12))
        heads = kv_heads * rng.choice((1, 2, 4, 8))
        layout = rng.choice(("interleaved", "half"))
        rot_dim = rng.choice((head_dim, head_dim // 2, 2 * (head_dim // 5)))
        dtype = rng.choice(("bf16", "fp16", "fp32"))
        most = 131072 * 72 * 128 // ((heads + kv_heads) * head_dim * (2 if dtype == "fp32" else 1))
        return _rope(_spread(rng, 1, min(131072, most)), heads, kv_heads, head_dim, rot_dim,
                     layout, rng.choice(("none", "linear", "ntk", "turns", "yarn")), dtype,
                     rng.choice((0, 0, rng.randrange(1 << 20))), rng.random() < 0.5)
    if op == "linear":
        inputs = _spread(rng, 40, 14336)
        features = _spread(rng, 17, 14336)
        gated = rng.random() < 0.3
        most = 8320 * 14336 * 2 * 5376 // (inputs * features * (2 if gated else 1))
        rows = _spread(rng, 1, max(1, min(33280, most)))
        return _linear(rows, features, inputs,
                       rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")), gated,
                       rng.random() < 0.6, rng.random() < 0.5, rng.choice(("bf16", "fp16")))
    kv_heads = rng.choice((1, 4, 8, 12, 24))
    heads = kv_heads * rng.choice((1, 1, 2, 3, 8))
    heads = kv_heads if heads > 64 else heads
    segments = rng.choice((1, 2, 3, 8))
    if rng.random() < 0.5:  # few queries, many keys
        queries = [_spread(rng, 1, 128) for _ in range(segments)]
        keys = [_spread(rng, 1, 16384) for _ in range(segments)]
    else:
        queries = [_spread(rng, 64, 8192) for _ in range(segments)]
        keys = [_spread(rng, 1, 1024) for _ in range(segments)]
    text = lambda v: ",".join(str(x) for x in v)  # noqa: E731
    return _cross(text(queries), text(keys), heads, kv_heads, rng.choice((64, 128)),
                  rng.random() < 0.3, rng.random() < 0.3, rng.choice(("bf16", "fp16")))


def _lengths(text):
    return [int(x) for x in text.split(",")]


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rope":
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["head_dim"]
        turned = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["rot_dim"]
        return {"bytes": 2 * size * values + 4 * case["tokens"], "flops": 3 * turned}
    if case["op"] == "linear":
        m, n, k = case["rows"], case["features"], case["inputs"]
        rows_w = 2 * n if case["gated"] else n
        values = m * k + rows_w * k + m * n * (2 if case["residual"] else 1)
        values += rows_w if case["bias"] else 0
        return {"bytes": size * values, "flops": 2 * m * rows_w * k}
    q, k = _lengths(case["queries"]), _lengths(case["keys"])
    values = 2 * sum(q) * case["heads"] * case["head_dim"]
    values += 2 * sum(k) * case["kv_heads"] * case["head_dim"]
    more = 4 * sum(q) * case["heads"] if case["lse"] else 0
    more += sum(k) if case["masked"] else 0
    return {"bytes": size * values + more,
            "flops": 4 * sum(a * b for a, b in zip(q, k)) * case["heads"] * case["head_dim"]}


# ------------------------------------------------------------------ the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)

    state = dict(case)
    if case["op"] == "rope":
        n, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
        if case["fused"]:  # q and k are views of one projection's rows, v behind them
            qkv = normal(n, (h + 2 * hk) * d)
            state["q"] = qkv[:, :h * d].view(n, h, d)
            state["k"] = qkv[:, h * d:(h + hk) * d].view(n, hk, d)
        else:
            state["q"], state["k"] = normal(n, h, d), normal(n, hk, d)
        start = case["first"] + int(torch.randint(0, 64, (1,), generator=gen, device="cuda"))
        state["positions"] = torch.arange(start, start + n, device="cuda", dtype=torch.int32)
    elif case["op"] == "linear":
        m, n, k = case["rows"], case["features"], case["inputs"]
        rows_w = 2 * n if case["gated"] else n
        ld = (k + 7) // 8 * 8  # rows of inputs and weights start on 16 bytes
        state["x"] = normal(m, ld)[:, :k]
        state["w"] = normal(rows_w, ld, scale=k ** -0.5)[:, :k]
        state["bias"] = normal(rows_w, scale=0.1) if case["bias"] else None
        state["residual"] = normal(m, n) if case["residual"] else None
        state["workspace"] = _workspace_linear(case) if own else None
    else:
        q, k = _lengths(case["queries"]), _lengths(case["keys"])
        d, hk = case["head_dim"], case["kv_heads"]
        state["q"] = normal(sum(q), case["heads"], d)
        kv = normal(sum(k), 2 * hk * d)  # one projection of the states gives both
        state["k"] = kv[:, :hk * d].view(sum(k), hk, d)
        state["v"] = kv[:, hk * d:].view(sum(k), hk, d)
        state["mask"] = None
        if case["masked"]:
            state["mask"] = torch.rand(sum(k), generator=gen, device="cuda") < 0.8
        for name, lengths in (("cu_q", q), ("cu_k", k)):
            cu = torch.tensor([0] + lengths).cumsum(0)
            state[name] = cu.to(device="cuda", dtype=torch.int32)
        state["max_q"], state["max_k"] = max(q), max(k)
        state["workspace"] = _workspace_cross(case) if own else None
    return state


def _workspace_linear(case):
    import audio_diffusion_transformer_h3_b200 as h3
    return h3.linear_workspace_for(case["rows"], case["features"], case["inputs"],
                                   case["gated"], device="cuda")


def _workspace_cross(case):
    import audio_diffusion_transformer_h3_b200 as h3
    q, k = _lengths(case["queries"]), _lengths(case["keys"])
    return h3.cross_workspace_for(sum(q), case["heads"], case["kv_heads"], case["head_dim"],
                                  len(q), max(q), max(k), device="cuda")


# -------------------------------------------------------------------- one pass

SCALINGS = {
    "none": {},
    "linear": {"kind": "linear", "factor": 4.0},
    "ntk": {"kind": "ntk", "factor": 4.0},
    "turns": {"kind": "turns", "factor": 8.0, "original_len": 8192, "beta_fast": 4.0,
              "beta_slow": 1.0},
    "yarn": {"kind": "yarn", "factor": 4.0, "original_len": 32768, "beta_fast": 32.0,
             "beta_slow": 1.0, "attn_factor": 0.1 * math.log(4.0) + 1.0},
}
THETA = 1000000.0


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "linear": _plain_linear, "cross": _plain_cross}[state["op"]](state)


def _run_own(state):
    import audio_diffusion_transformer_h3_b200 as h3
    if state["op"] == "rope":
        return h3.rope_qk_t(state["q"], state["k"], state["positions"], rot_dim=state["rot_dim"],
                            theta=THETA, layout=state["layout"],
                            scaling=SCALINGS[state["scaling"]] or None)
    if state["op"] == "linear":
        return h3.linear_t(state["x"], state["w"], bias=state["bias"], act=state["act"],
                           gated=state["gated"], residual=state["residual"],
                           workspace=state["workspace"])
    return h3.cross_attn_fwd_t(state["q"], state["k"], state["v"], state["cu_q"], state["cu_k"],
                               state["max_q"], state["max_k"], key_mask=state["mask"],
                               return_lse=state["lse"], workspace=state["workspace"])


def _frequencies(rot_dim, scaling, device):
    """(angle per position of each pair in 64 bits, factor of cos and sin)."""
    s = SCALINGS[scaling]
    kind, factor = s.get("kind", "none"), s.get("factor", 1.0)
    theta = THETA
    if kind == "ntk":
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    j = torch.arange(rot_dim // 2, device=device, dtype=torch.float64)
    f = theta ** (-2.0 * j / rot_dim)
    if kind == "linear":
        f = f / factor
    elif kind == "turns":  # pairs that make few turns over the original length are stretched
        turns = s["original_len"] * f / (2 * math.pi)
        keep = ((turns - s["beta_slow"]) / (s["beta_fast"] - s["beta_slow"])).clamp(0, 1)
        f = keep * f + (1 - keep) * f / factor
    elif kind == "yarn":  # the same, even over the pairs' numbers
        at = lambda b: rot_dim * math.log(s["original_len"] / (2 * math.pi * b)) / (2 * math.log(theta))  # noqa: E731
        low = max(math.floor(at(s["beta_fast"])), 0)
        high = min(math.ceil(at(s["beta_slow"])), rot_dim - 1)
        keep = 1 - ((j - low) / max(high - low, 0.001)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / factor
    return f, s.get("attn_factor", 1.0)


def _plain_rope(state):
    r = state["rot_dim"]
    f, factor = _frequencies(r, state["scaling"], state["q"].device)
    angle = state["positions"].double()[:, None] * f  # far positions: 64 bits
    cos = (angle.cos() * factor).float()[:, None, :]
    sin = (angle.sin() * factor).float()[:, None, :]

    def turn(x):
        t = x[..., :r].float()
        if state["layout"] == "half":
            a, b = t[..., :r // 2], t[..., r // 2:]
            t = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
        else:
            a, b = t[..., 0::2], t[..., 1::2]
            t = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
        return torch.cat((t.to(x.dtype), x[..., r:]), dim=-1)

    return turn(state["q"]), turn(state["k"])


def _activate(x, act):
    if act == "relu":
        return x.clamp_min(0)
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh((2 / math.pi) ** 0.5 * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return x


def _plain_linear(state):
    y = state["x"].float() @ state["w"].float().t()
    if state["bias"] is not None:
        y = y + state["bias"].float()
    if state["gated"]:
        n = state["features"]
        y = _activate(y[:, :n], state["act"]) * y[:, n:]
    else:
        y = _activate(y, state["act"])
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return y.to(state["x"].dtype)


def _plain_cross(state):
    """All segments at once, padded to the longest; keys that are not there count as masked."""
    q, k, v, cu_q, cu_k = (state[x] for x in ("q", "k", "v", "cu_q", "cu_k"))
    heads, hk, d = state["heads"], state["kv_heads"], state["head_dim"]

    def padded(cu, most):
        at = torch.arange(most, device=cu.device)
        there = at < (cu[1:] - cu[:-1])[:, None]
        return there, torch.where(there, cu[:-1, None] + at, 0)

    there_q, at_q = padded(cu_q, state["max_q"])
    there_k, at_k = padded(cu_k, state["max_k"])
    if state["mask"] is not None:
        there_k = there_k & state["mask"][at_k]
    rows = q[at_q].float().unflatten(2, (hk, heads // hk)).permute(0, 2, 3, 1, 4)  # s hk g i d
    keys = k[at_k].float().permute(0, 2, 3, 1)[:, :, None]                         # s hk 1 d j
    values = v[at_k].float().masked_fill(~there_k[:, :, None, None], 0)
    values = values.permute(0, 2, 1, 3)[:, :, None]                                # s hk 1 j d
    scores = (rows * d ** -0.5) @ keys
    scores.masked_fill_(~there_k[:, None, None, None, :], -math.inf)
    most = scores.amax(-1, keepdim=True)
    most = torch.where(most == -math.inf, 0, most)
    weights = scores.sub_(most).exp_()
    total = weights.sum(-1, keepdim=True)
    out = (weights @ values) / torch.where(total == 0, 1, total)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[there_q].to(q.dtype)
    if not state["lse"]:
        return out
    lse = (most + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[there_q]
    return out, lse.t().contiguous()


# --------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return {"rope": _exact_rope, "linear": _exact_linear, "cross": _exact_cross}[case["op"]](state)


def _exact_rope(state):
    """Each pair as a complex number times attn_factor * exp(i angle), a block of tokens at a time."""
    r = state["rot_dim"]
    f, factor = _frequencies(r, state["scaling"], "cpu")
    f = f.to("cuda")

    def turn(x):
        # results go into 32 bits where 64 of the whole tensor would not fit beside the state
        out = torch.empty(x.shape, device="cuda", dtype=torch.float64 if x.numel() < 1 << 28 else torch.float32)
        for at in range(0, len(x), 8192):
            here = x[at:at + 8192].double()
            angle = state["positions"][at:at + 8192].double()[:, None, None] * f
            spin = torch.polar(torch.full_like(angle, factor), angle)
            if state["layout"] == "half":
                z = torch.complex(here[..., :r // 2], here[..., r // 2:r]) * spin
                here[..., :r // 2], here[..., r // 2:r] = z.real, z.imag
            else:
                z = torch.complex(here[..., 0:r:2], here[..., 1:r:2]) * spin
                here[..., 0:r:2], here[..., 1:r:2] = z.real, z.imag
            out[at:at + 8192] = here
        return out

    return turn(state["q"]), turn(state["k"])


def _exact_linear(state):
    x, w, n = state["x"], state["w"].double(), state["features"]
    out = torch.empty((len(x), n), device="cuda", dtype=torch.float64)
    for at in range(0, len(x), 2048):
        y = torch.mm(x[at:at + 2048].double(), w.t())
        if state["bias"] is not None:
            y += state["bias"].double()
        g = y[:, :n]
        if state["act"] == "relu":
            g = torch.where(g > 0, g, 0.0)
        elif state["act"] == "gelu":
            g = g * torch.special.ndtr(g)
        elif state["act"] == "gelu_tanh":
            g = g * torch.sigmoid(math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3))
        elif state["act"] == "silu":
            g = g * torch.sigmoid(g)
        if state["gated"]:
            g = g * y[:, n:]
        if state["residual"] is not None:
            g = g + state["residual"][at:at + 2048].double()
        out[at:at + 2048] = g
    return out


def _exact_cross(state):
    q, k, v = state["q"], state["k"], state["v"]
    group = state["heads"] // state["kv_heads"]
    out = torch.zeros(q.shape, device="cuda", dtype=torch.float64)
    lse = torch.full((q.shape[1], len(q)), -math.inf, device="cuda", dtype=torch.float64)
    cu_q, cu_k = state["cu_q"].tolist(), state["cu_k"].tolist()
    for a, b, c, d in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        keep = torch.arange(c, d, device="cuda")
        if state["mask"] is not None:
            keep = keep[state["mask"][c:d]]
        if len(keep) == 0 or b == a:
            continue
        for h in range(q.shape[1]):
            s = q[a:b, h].double() @ k[keep, h // group].double().t() / math.sqrt(q.shape[2])
            lse[h, a:b] = torch.logsumexp(s, 1)
            out[a:b, h] = torch.softmax(s, 1) @ v[keep, h // group].double()
    return (out, lse) if state["lse"] else out
