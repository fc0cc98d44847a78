"""The layers around the attention on the GPU: waits, values, streams and sizes
at their ends, against float64 references (oracle/layers.py) within the error
bounds that test_layers_gpu.py derives."""

import fractions
import math

import numpy as np
import pytest

from test_layers_gpu import (_check_cross, _check_linear, _cross_case, _cu, _draw, _dtype, _f64,
                             _h3, _linear_case, _run_cross, _u, _within)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ cross attention

@pytest.mark.parametrize("lq,lk", [([300], [6401]), ([40, 130], [3333, 4100]), ([1], [20001]),
                                   ([128] * 6, [1025, 1, 900, 2049, 127, 1300])])
@pytest.mark.parametrize("Hq,Hk,D,dtype", [(4, 4, 128, "bf16"), (8, 2, 64, "fp16")])
def test_cross_long_unmasked_segments_that_end_inside_a_tile(lq, lk, Hq, Hk, D, dtype):
    """Many value tiles that need nothing, then one whose last rows must not count:
    the warp that writes zeros there is at that tile and no other."""
    import torch
    q, k, v, cu_q, cu_k = _cross_case(lq + [0], lk + [200], Hq, Hk, D, dtype)
    cu_q, cu_k = cu_q[:-1].contiguous(), cu_k[:-1].contiguous()
    n = sum(lk)
    k[n:], v[n:] = math.nan, math.inf
    first = None
    for _ in range(10):
        o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
        if first is None:
            first = o
            _check_cross(q, k[:n], v[:n], cu_q, cu_k, o, lse, D ** -0.5, None, "o")
        assert torch.equal(o, first)


def _low_scores(q, k, at, channel=3):
    """Keys `at` score -infinity with every query: q is positive in a channel where
    they are -infinity."""
    q[:, :, channel] = q[:, :, channel].abs().clamp_min(0.25)
    k[at, :, channel] = -math.inf


# the kept keys that score -infinity, and whether the others are masked
@pytest.mark.parametrize("case", ["first tile", "only kept key of the first tile", "a tile between",
                                  "all but the last key", "single keys"])
@pytest.mark.parametrize("lq,lk", [([300], [700]), ([1], [9000]), ([40, 3], [2000, 700])])
@pytest.mark.parametrize("Hq,Hk,D,dtype", [(4, 4, 128, "bf16"), (16, 2, 64, "fp16")])
def test_cross_keys_that_score_minus_infinity(case, lq, lk, Hq, Hk, D, dtype):
    """Such keys weigh nothing, wherever they lie and whether or not the keys are
    split over blocks: the result is that of the other keys alone."""
    import torch
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, Hq, Hk, D, dtype)
    n = sum(lk)
    low, mask = torch.zeros(n, dtype=torch.bool), torch.ones(n, dtype=torch.bool)
    for a, b in zip(np.cumsum([0] + lk), np.cumsum(lk)):
        a, b = int(a), int(b)
        if case == "first tile":
            low[a:a + 128] = True
        elif case == "only kept key of the first tile":
            mask[a:a + 128] = False
            mask[a + 5] = low[a + 5] = True
        elif case == "a tile between":
            low[a + 256:a + 384] = True
        elif case == "all but the last key":
            low[a:b - 1] = True
        else:
            low[a], low[a + 130], low[b - 1] = True, True, True
    _low_scores(q, k, low.cuda())
    for m in ([mask] if not mask.all() else [None, mask]):
        o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk, key_mask=None if m is None else m.cuda())
        kept = (~low if m is None else m & ~low).cuda()
        _check_cross(q, torch.where(low.cuda()[:, None, None], 0, k), v, cu_q, cu_k, o, lse, D ** -0.5,
                     kept, case)


@pytest.mark.parametrize("lq,lk", [([300], [700]), ([1], [9000]), ([2], [1])])
def test_cross_rows_whose_every_key_scores_minus_infinity(lq, lk):
    """No key has weight: 0 and -infinity, as where there is no key."""
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, 4, 2, 128, "bf16")
    _low_scores(q, k, slice(None))
    o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("lq,lk", [([300], [700]), ([3], [9000]), ([1, 70], [900, 100])])
@pytest.mark.parametrize("Hq,Hk,D,dtype", [(4, 4, 128, "bf16"), (16, 2, 64, "fp16")])
def test_cross_nan_shows_in_the_result_and_in_the_lse(lq, lk, Hq, Hk, D, dtype):
    """A NaN in a query or in a key that counts makes its rows NaN, the LSE too: it
    does not read as a row without keys. Other rows are as they were."""
    import torch
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, Hq, Hk, D, dtype)
    clean, lse0 = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
    bad = q.clone()
    bad[0, 1, 7] = math.nan
    o, lse = _run_cross(bad, k, v, cu_q, cu_k, lq, lk)
    there = torch.zeros(Hq, sum(lq), dtype=torch.bool, device="cuda")
    there[1, 0] = True
    assert torch.isnan(lse[there]).all() and torch.isnan(o[there.t()]).all()
    assert torch.equal(lse[~there], lse0[~there]) and torch.equal(o[~there.t()], clean[~there.t()])
    bad = k.clone()
    bad[lk[0] - 1, Hk - 1, 0] = math.nan      # the first segment's last key, the last group's heads
    o, lse = _run_cross(q, bad, v, cu_q, cu_k, lq, lk)
    there[:] = False
    there[-(Hq // Hk):, :lq[0]] = True
    assert torch.isnan(lse[there]).all() and torch.isnan(o[there.t()]).all()
    assert torch.equal(lse[~there], lse0[~there]) and torch.equal(o[~there.t()], clean[~there.t()])
    # every key that counts is NaN
    mask = torch.zeros(sum(lk), dtype=torch.bool, device="cuda")
    mask[:lk[0]:3] = True
    bad = k.clone()
    bad[:lk[0]] = math.nan
    o, lse = _run_cross(q, bad, v, cu_q, cu_k, lq, lk, key_mask=mask)
    assert torch.isnan(lse[:, :lq[0]]).all() and torch.isnan(o[:lq[0]]).all()
    assert (lse[:, lq[0]:] == -math.inf).all() and (o[lq[0]:] == 0).all()


def test_cross_as_many_segments_as_are_allowed():
    """65535 segments, many of them empty on one side or both."""
    rng = np.random.default_rng(8)
    lq, lk = (rng.integers(0, 3, 65535).tolist() for _ in range(2))
    lq[40000], lk[40000], lk[40001] = 300, 500, 0
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, 1, 1, 64, "bf16")
    o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
    _check_cross(q, k, v, cu_q, cu_k, o, lse, 0.125, None, "o")


@pytest.mark.parametrize("lq,lk", [([200], [500]), ([2], [3000])])
@pytest.mark.parametrize("scale", [0.0, 1e-38, 1e-42])
def test_cross_small_scales_of_large_scores(lq, lk, scale):
    """Scores near fp32's largest times a scale near its smallest, and times 0 (the mean
    of the values). 1e-42 is subnormal: 2^-11 of it is its last place."""
    import torch
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, 2, 2, 64, "bf16")
    q.mul_(2e18), k.mul_(2e18)
    o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk, softmax_scale=scale)
    exact = scale if scale != 1e-42 else float(np.float32(1e-42))
    if scale != 1e-42:
        _check_cross(q, k, v, cu_q, cu_k, o, lse, exact, None, f"scale {scale}")
    else:   # no score is above 2e-3: the mean, to that much
        mean = v.double().mean(0).expand(o.shape)
        assert torch.all((o.double() - mean).abs() <= 2.0 ** -8 * mean.abs() + 5e-3 * v.double().abs().mean(0))


# --------------------------------------------------------------------- linear

@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,dtype", [(4, "bf16"), (4, "fp16"), (200, "bf16"), (200, "fp16")])
def test_linear_activations_keep_their_tails(act, M, dtype):
    """Relative accuracy where an activation is small. Pre-activations are exact (one
    product with 1 each), -9 to 9, so that 1 + exp(-2u) stays below 2^126.
    Bound, relative, in units of 2^-23, t the exponent's argument: 1.2 |t| + 2 for
    exp, 2 |t| for t's three roundings, 8 for what is left. GELU by erfc: 4 for erfc,
    and 2 (x^2 / 2 + 1) for its argument's two roundings (|z erfc'(z) / erfc(z)| is
    at most 2 z^2 + 1)."""
    import torch
    h3 = _h3()
    d = _dtype(dtype)
    x = torch.zeros(M, 8, dtype=d, device="cuda")
    x[:, 0] = torch.linspace(-9, 9, M).to(d)
    w = torch.zeros(136, 8, dtype=d, device="cuda")
    w[:, 0] = torch.tensor([1.0, 0.5, 0.75, -1.0], dtype=d).repeat(34)
    z = (x[:, :1].double() * w[:, 0].double()).cpu()
    got = _f64(h3.linear_t(x, w, act=act))
    zz = z.numpy()
    if act == "gelu":
        want = 0.5 * zz * np.vectorize(math.erfc)(-zz / math.sqrt(2))
        rel = 12 + 2 * (zz ** 2 / 2 + 1)
    else:
        t = zz if act == "silu" else math.sqrt(8 / math.pi) * (zz + 0.044715 * zz ** 3)
        want = zz / (1 + np.exp(-t))
        rel = 10 + 3.2 * np.abs(t)
    least = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134
    bound = (_u(d) + rel * 2.0 ** -23) * np.abs(want) + least
    _within(got, want, bound, act)


@pytest.mark.parametrize("M,N,K,gated,act", [
    # on 148 SMs, tile columns / parts of the last round's tiles:
    (2690, 1999, 200, False, "gelu_tanh"),   # 256 / 4, 22 row tiles (a partial last group), 8 column tiles
    (3000, 2000, 136, False, "none"),        # 256 / 2
    (2600, 4001, 72, False, "silu"),         # 192 / 1, three tiles a CTA
    (6000, 900, 72, False, "relu"),          # 160 / 1, 47 row tiles
    (4100, 2333, 72, True, "silu"),          # 128 / 4, gate and up
    (2690, 1999, 136, True, "gelu_tanh"),    # 128 / 2
    (2600, 4001, 72, True, "none"),          # 96 / 1, six tiles a CTA
])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_linear_many_tiles(M, N, K, gated, act, dtype):
    """Every output of layers that take several tiles a CTA, of several column tiles and
    more row tiles than sweep the columns together, the last ones in parts."""
    h3 = _h3()
    x, w, b, r = _linear_case(M, N, K, act, gated, True, True, dtype)
    _check_linear(x, w, b, act, gated, r, h3.linear_t(x, w, b, act, gated, r), "y")


@pytest.mark.parametrize("M,N,K", [(1, 300, 14336), (2, 5376, 5376), (17, 260, 14336), (96, 200, 8200),
                                   (128, 300, 14336), (300, 513, 14336), (130, 1100, 4104),
                                   (2690, 1999, 1000)])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_whole_numbers_are_exact(M, N, K, gated):
    """Inputs of -1, 0 and 1: sums of at most 14337 and the products of the gate stay
    whole numbers below 2^24 (a sum is about 80, a product beyond 2^24 takes sums of 50
    times that), exact in fp32 in any order, so y is the definition's value rounded
    once. A K step that is lost or taken twice shows."""
    import torch
    h3 = _h3()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M + N + K)

    def draw(*shape):
        return torch.randint(-1, 2, shape, generator=gen, device="cuda").to(torch.bfloat16)

    W = 2 * N if gated else N
    x, w, b, r = draw(M, K), draw(W, K), draw(W), draw(M, N)
    z = x.double() @ w.double().t() + b.double()
    want = (z[:, :N].clamp_min(0) * z[:, N:] if gated else z.clamp_min(0)) + r.double()
    assert want.abs().max() < 2 ** 24
    y = h3.linear_t(x, w, b, "relu", gated, r)
    assert torch.equal(y, want.to(torch.bfloat16))


# --------------------------------------------------------------------- rotary

# pi to 60 places
PI = fractions.Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


@pytest.mark.parametrize("layout,scaling", [
    ("half", None), ("interleaved", dict(kind="linear", factor=7.0)),
    ("half", dict(kind="yarn", factor=4.0, original_len=32768, beta_fast=32.0, beta_slow=1.0))])
def test_rope_angles_at_every_position(layout, scaling):
    """cos and sin of position * f_j, for the f_j that h3_rope_qk_freqs gives, anywhere
    in int32: off by 2^-26 + 2^-32 + 2^-34 turns (the fraction of a turn in fp32, its
    bits that are left out, the phase's own rounding) and 2 units of fp32 for sincospi.
    The reference reduces the angle in exact fractions."""
    import torch
    h3 = _h3()
    rot, theta = 64, 1e6
    rng = np.random.default_rng(21)
    positions = np.unique(np.concatenate([
        rng.integers(-2 ** 31, 2 ** 31, 150), rng.integers(0, 1 << 18, 150), 2 ** np.arange(31),
        [0, -1, 2 ** 31 - 1, -2 ** 31]])).astype(np.int32)
    freqs = [fractions.Fraction(float(f)) for f in
             h3.h3_rope_qk_freqs(h3.rope_qk_cfg(rot, theta, layout, scaling))]
    turns = np.array([[float((int(p) * f / (2 * PI)) % 1) for f in freqs] for p in positions])
    x = torch.zeros(len(positions), 1, rot, device="cuda")
    first, second = ((slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half"
                     else (slice(0, rot, 2), slice(1, rot, 2)))
    x[..., first] = 1.0
    y, _ = h3.rope_qk_t(x, None, torch.from_numpy(positions).cuda(), rot, theta, layout, scaling)
    bound = 2 * math.pi * (2.0 ** -26 + 2.0 ** -32 + 2.0 ** -34) + 2.0 ** -23 + 1e-15
    _within(_f64(y)[:, 0, first], np.cos(2 * math.pi * turns), bound, "cos")
    _within(_f64(y)[:, 0, second], np.sin(2 * math.pi * turns), bound, "sin")


def test_rope_configuration_by_value():
    """A configuration is what its numbers are at the call: objects that hold them may
    change between calls."""
    import torch
    h3 = _h3()
    q = _draw(np.random.default_rng(4), (40, 2, 64), torch.float32)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    factor, theta = torch.tensor(2.0), torch.tensor(1e4)

    def run(f, t):
        return h3.rope_qk_t(q, None, pos, 64, t, "half", dict(kind="linear", factor=f))[0]

    for f, t in ((2.0, 1e4), (5.0, 1e4), (5.0, 500.0)):
        factor.fill_(f), theta.fill_(t)
        assert torch.equal(run(factor, theta), run(f, t)), (f, t)


# ------------------------------------------------------- streams, autograd, memory

def _calls(h3):
    """Each helper as (name of the entry point, call with keywords)."""
    import torch
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(16, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    a, b = x.view(4, 1, 64), w.view(16, 1, 64)
    cu_q, cu_k = _cu([4]), _cu([16])
    return [("h3_linear_fwd", lambda **kw: h3.linear_t(x, w, **kw)),
            ("h3_rope_qk_apply", lambda **kw: h3.rope_qk_t(a, None, pos, **kw)),
            ("h3_cross_attn_fwd", lambda **kw: h3.cross_attn_fwd_t(a, b, b, cu_q, cu_k, 4, 16, **kw))]


def test_stream_handles_are_taken_as_they_are(monkeypatch):
    """A raw handle names that stream, 0 the device's default stream."""
    import torch
    h3 = _h3()
    side = torch.cuda.Stream()
    seen = []
    for name, call in _calls(h3):
        entry = getattr(h3, name)
        monkeypatch.setattr(h3, name, lambda *a, entry=entry: (seen.append(a[-1]), entry(*a))[1])
        for stream, handle in ((0, 0), (None, 0), (side.cuda_stream, side.cuda_stream),
                               (side, side.cuda_stream), (torch.cuda.default_stream(), 0)):
            call(stream=stream)
            assert seen[-1] == handle, (name, stream)
        with torch.cuda.stream(side):
            call(stream=0)
            assert seen[-1] == 0, name
            call()
            assert seen[-1] == side.cuda_stream, name
    torch.cuda.synchronize()


def test_inputs_of_a_call_on_another_stream_are_kept_until_it_is_done():
    """Inputs that are dropped after a call on another stream: their memory is not
    given out again before that stream has come to the call. (Nothing is written into
    what is given out.)"""
    import torch
    h3 = _h3()
    side = torch.cuda.Stream()
    rows, n = 2048, 2048

    def inputs():
        x = torch.ones(rows, n, dtype=torch.bfloat16, device="cuda")
        w = torch.ones(n, n, dtype=torch.bfloat16, device="cuda")
        pos = torch.arange(rows, dtype=torch.int32, device="cuda")
        return x, w, pos, _cu([rows])

    def linear(x, w, pos, cu):
        return h3.linear_t(x, w, residual=x, stream=side)

    def rope(x, w, pos, cu):
        return h3.rope_qk_t(x.view(rows, 32, 64), w.view(n, 32, 64), pos, stream=side)

    def cross(x, w, pos, cu):
        return h3.cross_attn_fwd_t(x.view(rows, 32, 64), w.view(n, 32, 64), w.view(n, 32, 64), cu, cu,
                                   rows, rows, stream=side)

    for call in (linear, rope, cross):
        call(*inputs())
        torch.cuda.synchronize()
        tensors = inputs()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(400_000_000)   # about 0.2 s
        kept = call(*tensors)
        old = {t.data_ptr() for t in tensors}
        del tensors
        new = [torch.empty(rows, n, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        busy = not side.query()
        assert busy and not old & {t.data_ptr() for t in new}, call.__name__
        del new, kept
        torch.cuda.synchronize()


def test_a_raw_stream_may_end_before_its_tensors():
    """A stream that is given by its handle belongs to the caller, who may destroy it
    once it is done; tensors of calls on it are freed later."""
    import ctypes

    import torch
    cudart = torch.cuda.cudart()
    h3 = _h3()
    handle = ctypes.c_void_p()
    cudart.cudaStreamCreate(ctypes.addressof(handle))
    x = torch.ones(256, 512, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(512, 512, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    y = h3.linear_t(x, w, stream=handle.value)
    z = h3.linear_t(x, w, stream=torch.cuda.ExternalStream(handle.value))
    torch.cuda.synchronize()
    assert torch.equal(y, z) and (y == 512).all()
    cudart.cudaStreamDestroy(handle.value)
    del x, w
    torch.cuda.synchronize()


def test_tangents_are_refused():
    """Forward only: a forward-mode tangent would be lost, so the call is refused."""
    import torch
    import torch.autograd.forward_ad as fwd
    h3 = _h3()
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(16, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    with fwd.dual_level():
        dx, dw = (fwd.make_dual(t, torch.ones_like(t)) for t in (x, w))
        a, b, c = dx.view(4, 1, 64), dw.view(16, 1, 64), w.view(16, 1, 64)
        for call in (lambda: h3.linear_t(dx, w), lambda: h3.linear_t(x, dw),
                     lambda: h3.linear_t(x, w, bias=dw[:, 0].contiguous()),
                     lambda: h3.rope_qk_t(a, None, pos), lambda: h3.rope_qk_t(c[:4], a, pos),
                     lambda: h3.cross_attn_fwd_t(x.view(4, 1, 64), c, b, _cu([4]), _cu([16]), 4, 16)):
            with pytest.raises(ValueError), torch.no_grad():
                call()
        h3.linear_t(x, w)   # neither has a tangent


def test_writing_into_a_given_tensor_counts_as_a_change():
    """Autograd keeps tensors for the backward pass and notices when one is written
    over; so it does where a call writes into ``out``."""
    import torch
    h3 = _h3()
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(16, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    a, b = torch.ones(4, 1, 64, device="cuda"), torch.ones(4, 2, 64, device="cuda")
    o = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.ones(4, 16, dtype=torch.bfloat16, device="cuda")
    c = w.view(16, 1, 64)
    for call, outs in (
            (lambda: h3.linear_t(x, w, out=y), [y]),
            (lambda: h3.linear_t(x, w, residual=y, out=y), [y]),
            (lambda: h3.rope_qk_t(a, b, pos, out=(a, b)), [a, b]),
            (lambda: h3.rope_qk_t(a, None, pos, out=(a, None)), [a]),
            (lambda: h3.cross_attn_fwd_t(x.view(4, 1, 64), c, c, _cu([4]), _cu([16]), 4, 16, out=o), [o])):
        for out in outs:
            leaf = torch.ones_like(out, requires_grad=True)
            loss = (leaf * out).sum()   # keeps out
            call()
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()
    with torch.inference_mode():   # such tensors have no count of changes
        h3.linear_t(x, w, out=torch.empty(4, 16, dtype=torch.bfloat16, device="cuda"))


def test_a_workspace_is_as_large_as_its_memory():
    """The count of bytes that goes with the pointer is that of memory behind it: a
    view that says more elements than it has is refused, a wider type counts whole."""
    import torch
    h3 = _h3()
    size = 1 << 12
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for name, call in _calls(h3):
        if name == "h3_rope_qk_apply":   # has none
            continue
        want = call(workspace=ws)
        assert torch.equal(call(workspace=torch.empty(64, dtype=torch.float32, device="cuda")), want)
        for bad in (ws[:1].expand(size), ws[::2]):
            with pytest.raises(ValueError):
                call(workspace=bad)
        with pytest.raises(h3.H3Error):   # 252 bytes
            call(workspace=torch.empty(63, dtype=torch.float32, device="cuda"))
