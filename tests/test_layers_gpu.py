"""The layers around the attention on the GPU against their float64
references (oracle/layers.py).

Error bounds, with u = half a step of the type (torch.finfo.eps / 2):
  rotary  u |y| for the rounding; 2^-20 a (|x0| + |x1|) for the angle (2^-33
          turns and its fp32 form, 2e-7 radians), sincospi (2 ulp) and two
          fp32 operations.
  linear  u |y|; (K + 8) 2^-23 times the spread (sum of |x w| through the
          activation's slope) for K fp32 additions that may truncate;
          2^-18 (|y| + 1) for the activation in fp32.
  cross   u |O|; u A for P's rounding (A: weighted |v|); a score is off by
          d = D 2^-23 S (S: scale sum |q k|), an exponential by another 8e-5
          at most, so numerator and sum move the result by 2 (d + 8e-5) A;
          fp16 P below 2^-20 of the largest is subnormal: n 2^-31 max|v|.
          LSE: d + 8e-5 + 2^-21 |LSE|.
Values below fp16's normal range add 2^-25.
"""

import math

import numpy as np
import pytest

from oracle import layers as ref

pytestmark = pytest.mark.gpu


def _h3():
    import audio_diffusion_transformer_h3_b200 as h3
    return h3


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _u(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


def _draw(rng, shape, dtype, scale=1.0):
    """A device tensor of the type (contiguous)."""
    import torch
    x = rng.standard_normal(shape, dtype=np.float32) * np.float32(scale)
    return torch.from_numpy(x).cuda().to(dtype)


def _f64(t):
    return t.double().cpu().numpy()


def _strided(t, extra):
    """The same values with `extra` more elements between rows, NaN in the gaps."""
    import torch
    n = t[0].numel() if t.shape[0] else int(np.prod(t.shape[1:]))
    wide = torch.full((t.shape[0], n + extra), math.nan, dtype=t.dtype, device=t.device)
    wide[:, :n] = t.reshape(t.shape[0], n)
    return wide[:, :n].unflatten(1, t.shape[1:]) if t.dim() > 2 else wide[:, :n]


def _within(got, want, bound, what):
    err = np.abs(got - want)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.argwhere(err > bound)
    assert over.size == 0, (f"{what}: {len(over)} of {err.size} outside, first {over[:3].tolist()}, "
                            f"largest {float((err / bound).max()):.3g} times the bound")


# --------------------------------------------------------------------- rotary

YARN = dict(kind="yarn", factor=4.0, original_len=32768, beta_fast=32.0, beta_slow=1.0,
            attn_factor=1.1386)


def _check_rope(x, y, positions, rot, layout, theta, scaling, what):
    s = dict(scaling or {})
    a = s.get("attn_factor", 1.0)
    want = ref.rope_qk_ref(_f64(x), positions, rot, ref.rope_freqs_ref(rot, theta, **s), layout, a)
    ax = np.abs(_f64(x))
    h = rot // 2
    pair = np.zeros_like(ax)
    one, two = ((slice(0, h), slice(h, rot)) if layout == "half"
                else (slice(0, rot, 2), slice(1, rot, 2)))
    pair[..., one] = pair[..., two] = ax[..., one] + ax[..., two]
    bound = _u(y.dtype) * np.abs(want) + 2.0 ** -20 * abs(a) * pair + 2.0 ** -25
    _within(_f64(y), want, bound, what)
    assert np.array_equal(_f64(y)[..., rot:], _f64(x)[..., rot:]), what


@pytest.mark.parametrize("N,Hq,Hk,D,rot,layout,dtype,scaling,extra", [
    (1, 64, 8, 128, 128, "half", "bf16", YARN, 0),
    (5, 1, 0, 64, 64, "interleaved", "bf16", None, 0),          # q alone
    (33, 3, 1, 80, 40, "interleaved", "fp32", None, 0),         # 20 pairs
    (33, 3, 1, 80, 40, "half", "fp16", None, 8),                # halves of 20 channels: scalar
    (130, 2, 2, 128, 64, "interleaved", "fp16", dict(kind="linear", factor=4.0), 256),
    (130, 2, 2, 128, 64, "half", "bf16", dict(kind="ntk", factor=4.0), 3),   # odd stride
    (17, 5, 5, 7, 4, "half", "bf16", None, 0),                  # odd head dim
    (17, 5, 5, 7, 4, "interleaved", "fp32", None, 1),
    (9, 2, 1, 512, 512, "half", "fp16", None, 0),
    (9, 2, 1, 256, 2, "interleaved", "bf16", None, 0),
    (1000, 12, 4, 96, 96, "half", "bf16",
     dict(kind="turns", factor=8.0, original_len=8192, beta_fast=4.0, beta_slow=1.0), 0),
    (2049, 8, 1, 128, 128, "interleaved", "fp32", YARN, 0),
])
def test_rope(N, Hq, Hk, D, rot, layout, dtype, scaling, extra):
    import torch
    h3 = _h3()
    rng = np.random.default_rng(N + D + rot)
    q = _strided(_draw(rng, (N, Hq, D), _dtype(dtype)), extra)
    k = _strided(_draw(rng, (N, Hk, D), _dtype(dtype)), extra) if Hk else None
    positions = rng.integers(-3, 200000, N).astype(np.int32)
    positions[0] = 131071
    pos = torch.from_numpy(positions).cuda()
    for theta in (1e4, 1e6):
        qo, ko = h3.rope_qk_t(q, k, pos, rot, theta, layout, scaling)
        _check_rope(q, qo, positions, rot, layout, theta, scaling, "q")
        if Hk:
            _check_rope(k, ko, positions, rot, layout, theta, scaling, "k")
        else:
            assert ko is None


def test_rope_positions_at_the_ends_of_int32():
    import torch
    h3 = _h3()
    rng = np.random.default_rng(5)
    positions = np.array([0, -1, 1, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1, 2 ** 30 + 1], np.int32)
    q = _draw(rng, (7, 2, 64), torch.float32)
    qo, _ = h3.rope_qk_t(q, None, torch.from_numpy(positions).cuda(), 64, 1e4, "half")
    # the reference's own angle in double is off by 2^31 2^-53 = 2^-22 at most
    want = ref.rope_qk_ref(_f64(q), positions, 64, ref.rope_freqs_ref(64, 1e4), "half")
    ax = np.abs(_f64(q))
    pair = np.concatenate([ax[..., :32] + ax[..., 32:]] * 2, axis=-1)
    _within(_f64(qo), want, 2.0 ** -24 * np.abs(want) + (2.0 ** -20 + 2.0 ** -21) * pair, "ends")


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype,D,rot", [("bf16", 128, 64), ("fp32", 20, 12), ("fp16", 64, 64)])
def test_rope_in_place_equals_out_of_place_and_keeps_the_gaps(layout, dtype, D, rot):
    import torch
    h3 = _h3()
    rng = np.random.default_rng(6)
    q, k = (_draw(rng, (300, h, D), _dtype(dtype)) for h in (6, 2))
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    want = h3.rope_qk_t(q, k, pos, rot, 1e4, layout)
    wide = torch.full((300, 8 * D + 16), 7.0, dtype=q.dtype, device="cuda")
    a, b = wide[:, :6 * D].view(300, 6, D), wide[:, 6 * D:8 * D].view(300, 2, D)
    a.copy_(q), b.copy_(k)
    got = h3.rope_qk_t(a, b, pos, rot, 1e4, layout, out=(a, b))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.all(wide[:, 8 * D:] == 7.0)


def test_rope_gradient_is_the_negated_position():
    # y is linear in x: <g, J dx> = <J^T g, dx>; J dx by a difference, J^T g by
    # the call with negated positions, both in fp32 (2^-20 a value, 64 values)
    import torch
    h3 = _h3()
    rng = np.random.default_rng(7)
    pos = torch.arange(1000, 1050, dtype=torch.int32, device="cuda")
    x, dx, g = (_draw(rng, (50, 3, 64), torch.float32) for _ in range(3))
    f = lambda t, p: h3.rope_qk_t(t, None, p, 48, 1e4, "half", YARN)[0].double()  # noqa: E731
    lhs = (g.double() * (f(x + dx, pos) - f(x, pos))).sum((1, 2))
    rhs = (f(g, -pos) * dx.double()).sum((1, 2))
    size = (g.double().abs().sum((1, 2)) * dx.abs().amax((1, 2)).double()).clamp_min(1)
    assert torch.all((lhs - rhs).abs() <= 2.0 ** -18 * size)


def test_rope_empty():
    import torch
    h3 = _h3()
    q = torch.empty(0, 4, 64, device="cuda")
    out, none = h3.rope_qk_t(q, None, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64) and none is None


# --------------------------------------------------------------------- linear

def _check_linear(x, w, bias, act, gated, residual, y, what):
    want, spread = ref.linear_ref(_f64(x), _f64(w), None if bias is None else _f64(bias), act, gated,
                                  None if residual is None else _f64(residual))
    bound = (_u(y.dtype) * np.abs(want) + (x.shape[1] + 8) * 2.0 ** -23 * spread
             + 2.0 ** -18 * (np.abs(want) + 1) + 2.0 ** -25)
    _within(_f64(y), want, bound, what)


def _linear_case(M, N, K, act, gated, bias, residual, dtype, seed=0, extra=0):
    """x and w with rows padded to 16 bytes (NaN behind them)."""
    rng = np.random.default_rng(1000 * M + 10 * N + K + seed)
    d = _dtype(dtype)
    W = 2 * N if gated else N
    pad = -K % 8 + 8 * extra
    x, w = _strided(_draw(rng, (M, K), d), pad), _strided(_draw(rng, (W, K), d, K ** -0.5), pad)
    if M == 1:
        x = x[:, :K]
    b = _draw(rng, (W,), d, 0.5) if bias else None
    r = _draw(rng, (M, N), d) if residual else None
    return x, w, b, r


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 8, 8), (1, 300, 5376), (2, 1003, 1000), (3, 256, 14336), (7, 17, 63),
    (16, 129, 65), (17, 128, 64), (33, 500, 640), (64, 1024, 200), (65, 96, 4097), (127, 255, 127),
    (128, 256, 128), (129, 257, 129), (300, 513, 1000), (1001, 1003, 1000),
])
@pytest.mark.parametrize("act,gated,bias,residual,dtype", [
    ("none", False, False, False, "bf16"), ("gelu_tanh", False, True, True, "fp16"),
    ("silu", True, True, True, "bf16"),
])
def test_linear(M, N, K, act, gated, bias, residual, dtype):
    h3 = _h3()
    x, w, b, r = _linear_case(M, N, K, act, gated, bias, residual, dtype)
    _check_linear(x, w, b, act, gated, r, h3.linear_t(x, w, b, act, gated, r), "y")


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,dtype", [(5, "bf16"), (200, "fp16"), (5, "fp16"), (200, "bf16")])
def test_linear_activations(act, gated, M, dtype):
    h3 = _h3()
    x, w, b, r = _linear_case(M, 96, 320, act, gated, True, False, dtype, seed=3)
    x *= 4  # reaches both tails of the activations
    _check_linear(x, w, b, act, gated, r, h3.linear_t(x, w, b, act, gated, r), act)


@pytest.mark.parametrize("M", [4, 20, 50, 140, 700])
@pytest.mark.parametrize("gap", [1, 8, 13])
def test_linear_strides_and_in_place_residual(M, gap):
    """Rows of y and residual at any stride and element alignment; what lies
    between the rows stays as it was; y over its own residual."""
    import torch
    h3 = _h3()
    N, K = 200, 520
    x, w, b, r = _linear_case(M, N, K, "gelu", False, True, True, "bf16", extra=gap)
    wide = torch.full((M, N + 2 * gap), 7.0, dtype=torch.bfloat16, device="cuda")
    y = wide[:, gap:gap + N]
    y.copy_(r)
    out = h3.linear_t(x, w, b, "gelu", False, y, out=y)
    _check_linear(x, w, b, "gelu", False, r, out, "in place")
    assert torch.all(wide[:, :gap] == 7.0) and torch.all(wide[:, gap + N:] == 7.0)


def test_linear_infinities_stay_in_their_row_and_column():
    import torch
    h3 = _h3()
    for M in (3, 150):
        x, w, b, _ = _linear_case(M, 140, 136, "none", False, True, False, "bf16")
        clean = h3.linear_t(x, w, b)
        x2, w2 = x.clone(), w.clone()
        x2 = torch.cat([x2, x2[:, :0]], 1)
        x2[1, 5], w2[7, 9] = math.nan, math.inf
        y = h3.linear_t(x2, w2, b)
        keep = torch.ones_like(y, dtype=torch.bool)
        keep[1], keep[:, 7] = False, False
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[:, 7]).any()
        assert torch.equal(y[keep], clean[keep])


def test_linear_no_rows():
    import torch
    h3 = _h3()
    y = h3.linear_t(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                    torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda"))
    assert y.shape == (0, 32)


@pytest.mark.parametrize("M,N,K", [(1, 5376, 5376), (40, 700, 8192), (1500, 2000, 520)])
def test_linear_is_deterministic(M, N, K):
    import torch
    h3 = _h3()
    x, w, b, r = _linear_case(M, N, K, "silu", True, True, True, "bf16")
    first = h3.linear_t(x, w, b, "silu", True, r)
    for _ in range(5):
        assert torch.equal(h3.linear_t(x, w, b, "silu", True, r), first)


# ------------------------------------------------------------ cross attention

def _cu(lengths):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).cuda()


def _check_cross(q, k, v, cu_q, cu_k, o, lse, scale, mask, what):
    Q, K, V = _f64(q), _f64(k), _f64(v)
    cq, ck = cu_q.cpu().numpy(), cu_k.cpu().numpy()
    m = None if mask is None else mask.cpu().numpy()
    O, L, A, S = ref.cross_attention_ref(Q, K, V, cq, ck, scale, m)
    n = int(cq[-1])
    D, u = q.shape[2], _u(q.dtype)
    d = D * 2.0 ** -23 * S[..., None] + 8e-5
    kept = np.isfinite(V) if m is None else np.isfinite(V) & (m != 0)[:, None, None]
    vmax = np.abs(V[kept]).max() if kept.any() else 0.0
    most = int((ck[1:] - ck[:-1]).max()) if len(ck) > 1 else 0
    bound = u * np.abs(O) + (u + 2 * d) * A + most * 2.0 ** -31 * vmax + 2.0 ** -25
    _within(_f64(o)[:n], O[:n], bound[:n], what)
    if lse is not None:
        got, want = _f64(lse)[:, :n], L[:, :n]
        none = np.isinf(want)
        assert np.array_equal(np.isneginf(got), none), f"{what}: rows without keys"
        lb = d[..., 0].T[:, :n] + 2.0 ** -21 * np.abs(np.where(none, 0, want)) + 1e-30
        _within(np.where(none, 0, got), np.where(none, 0, want), lb, f"{what} lse")


def _cross_case(lq, lk, Hq, Hk, D, dtype, seed=0, std=1.0):
    rng = np.random.default_rng(seed + sum(lq) + 7 * sum(lk) + Hq)
    d = _dtype(dtype)
    return (_draw(rng, (sum(lq), Hq, D), d, std), _draw(rng, (sum(lk), Hk, D), d, std),
            _draw(rng, (sum(lk), Hk, D), d), _cu(lq), _cu(lk))


def _run_cross(q, k, v, cu_q, cu_k, lq, lk, **kw):
    import torch
    h3 = _h3()
    ws = h3.cross_workspace_for(q.shape[0], q.shape[1], k.shape[1], q.shape[2], len(lq), max(lq),
                                max(lk))
    ws.fill_(0xA5)   # nothing may rely on what the workspace held
    o, lse = h3.cross_attn_fwd_t(q, k, v, cu_q, cu_k, max(lq), max(lk), return_lse=True,
                                 workspace=ws, **kw)
    torch.cuda.synchronize()
    assert h3.device_status_t(ws) == h3.H3_OK
    return o, lse


CROSS_LENGTHS = [
    ([1], [1]), ([1], [128]), ([1], [129]), ([128], [128]), ([129], [127]), ([300], [77]),
    ([257], [1]), ([5], [3000]), ([1, 1, 1], [700, 1, 33]), ([64], [5000]),
    ([0, 70, 0, 1, 300, 0], [40, 0, 0, 5, 260, 9]), ([200, 100], [0, 0]), ([513], [384]),
]


@pytest.mark.parametrize("lq,lk", CROSS_LENGTHS)
@pytest.mark.parametrize("Hq,Hk,D,dtype", [(2, 2, 128, "bf16"), (6, 2, 64, "fp16"),
                                           (8, 1, 128, "fp16"), (7, 7, 64, "bf16")])
def test_cross(lq, lk, Hq, Hk, D, dtype):
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, Hq, Hk, D, dtype)
    o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
    _check_cross(q, k, v, cu_q, cu_k, o, lse, D ** -0.5, None, "o")


@pytest.mark.parametrize("lq", [[1], [1, 300, 2], [400]])
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp16"), (128, "fp16")])
def test_cross_single_key_is_exact(lq, D, dtype):
    """One key has the weight 1, whatever its score: O is v, bit for bit (P and the
    sum are the same power of two). A reference maximum other than the row's own
    shows here."""
    import torch
    lk = [1] * len(lq)
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, 16, 8, D, dtype)
    o, _ = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
    want = torch.cat([v[s].repeat_interleave(2, 0).expand(n, 16, D) for s, n in enumerate(lq)])
    assert torch.equal(o, want)


@pytest.mark.parametrize("lk", [40, 128, 200, 300])
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "fp16")])
def test_cross_many_items_a_cta(lk, D, dtype):
    """Several times as many items as SMs, with one to three key tiles each."""
    lq = [3700, 1, 200]
    q, k, v, cu_q, cu_k = _cross_case(lq, [lk, lk, 1], 48, 48, D, dtype)
    o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, [lk, lk, 1])
    _check_cross(q, k, v, cu_q, cu_k, o, lse, D ** -0.5, None, "o")


@pytest.mark.parametrize("group", [3, 5, 7, 16, 56, 100, 130])
@pytest.mark.parametrize("lq,lk", [([1, 1], [900, 3]), ([90, 33], [70, 300])])
def test_cross_group_sizes(group, lq, lk):
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, 2 * group, 2, 64, "bf16")
    o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
    _check_cross(q, k, v, cu_q, cu_k, o, lse, 0.125, None, f"group {group}")


@pytest.mark.parametrize("lq,lk", [([300, 40, 7], [500, 129, 64]), ([1, 2], [4000, 900]),
                                   ([130], [257])])
@pytest.mark.parametrize("Hq,Hk,D,dtype", [(2, 2, 128, "bf16"), (8, 2, 64, "fp16")])
@pytest.mark.parametrize("kind", ["random", "first tiles gone", "one key", "none"])
def test_cross_masks(lq, lk, Hq, Hk, D, dtype, kind):
    """What lies in masked places, NaN and infinities too, has no influence."""
    import torch
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, Hq, Hk, D, dtype)
    rng = np.random.default_rng(3)
    mask = rng.random(sum(lk)) < 0.5
    if kind == "first tiles gone":
        mask[:] = False
        mask[np.cumsum(lk) - 1] = True
        mask[np.cumsum(lk)[0] - 5:np.cumsum(lk)[0]] = True
    elif kind == "one key":
        mask[:] = False
        mask[sum(lk) // 2] = True
    elif kind == "none":
        mask[:] = False
    m = torch.from_numpy(mask).cuda()
    gone = ~m
    bad = torch.tensor([math.nan, math.inf, -math.inf, 60000.0], device="cuda").to(q.dtype)
    k[gone] = bad[torch.arange(int(gone.sum()), device="cuda") % 4][:, None, None]
    v[gone] = bad[torch.arange(int(gone.sum()), device="cuda") % 3][:, None, None]
    for mm in (m, m.to(torch.uint8) * 255):
        o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk, key_mask=mm)
        _check_cross(q, torch.where(m[:, None, None], k, 0), torch.where(m[:, None, None], v, 0),
                     cu_q, cu_k, o, lse, D ** -0.5, m, kind)


@pytest.mark.parametrize("lq,lk,Hq,Hk", [([100, 50], [200, 90], 2, 2), ([1, 1], [900, 1500], 8, 2)])
def test_cross_neighbours_and_rows_behind_the_last_sequence(lq, lk, Hq, Hk):
    """Keys of other segments and behind the last one may hold NaN; rows of o
    and lse behind the last query are left as they were."""
    import torch
    h3 = _h3()
    D = 128
    q, k, v, cu_q, cu_k = _cross_case(lq + [30], lk + [70], Hq, Hk, D, "bf16")
    cu_q, cu_k = cu_q[:-1].contiguous(), cu_k[:-1].contiguous()
    nq, nk = sum(lq), sum(lk)
    q[nq:], k[nk:], v[nk:] = math.nan, math.nan, math.inf
    alone = []
    for s in range(2):   # the other segment's keys are NaN: this one's rows must not see it
        kk, vv = k.clone(), v.clone()
        a, b = int(cu_k[1 - s]), int(cu_k[2 - s])
        kk[a:b], vv[a:b] = math.nan, math.nan
        o = torch.full_like(q, 7.0)
        lse = torch.full((Hq, q.shape[0]), 7.0, device="cuda")
        st = h3.h3_cross_attn_fwd(
            q.data_ptr(), Hq * D, kk.data_ptr(), Hk * D, vv.data_ptr(), Hk * D, o.data_ptr(), Hq * D,
            lse.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(), 2, max(lq), max(lk), 0, q.shape[0],
            k.shape[0], Hq, Hk, D, D ** -0.5, h3.H3_BF16,
            (ws := h3.cross_workspace_for(q.shape[0], Hq, Hk, D, 2, max(lq), max(lk))).data_ptr(),
            ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert st == h3.H3_OK
        torch.cuda.synchronize()
        assert torch.all(o[nq:] == 7.0) and torch.all(lse[:, nq:] == 7.0)
        a, b = int(cu_q[s]), int(cu_q[s + 1])
        alone.append((o[a:b].clone(), lse[:, a:b].clone()))
    o = torch.cat([x[0] for x in alone])
    lse = torch.cat([x[1] for x in alone], 1)
    _check_cross(q[:nq], k[:nk], v[:nk], cu_q, cu_k, o, lse, D ** -0.5, None, "alone")


@pytest.mark.parametrize("nseg", [300, 2500])
def test_cross_many_segments(nseg):
    rng = np.random.default_rng(nseg)
    lq, lk = (rng.integers(0, 4, nseg).tolist() for _ in range(2))
    lq[nseg // 2], lk[nseg // 2] = 150, 400
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, 4, 2, 64, "bf16")
    o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
    _check_cross(q, k, v, cu_q, cu_k, o, lse, 0.125, None, "o")


@pytest.mark.parametrize("lq,lk", [([150], [300]), ([2], [2000])])
def test_cross_strided_views_of_one_projection(lq, lk):
    import torch
    h3 = _h3()
    Hq, Hk, D = 4, 2, 64
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, Hq, Hk, D, "fp16")
    kv = torch.cat([k.flatten(1), v.flatten(1)], 1)
    wide = torch.full((sum(lq), Hq * D + 8), 7.0, dtype=q.dtype, device="cuda")
    out = wide[:, :Hq * D].view(-1, Hq, D)
    o = h3.cross_attn_fwd_t(_strided(q, 24), kv[:, :Hk * D].view(-1, Hk, D),
                            kv[:, Hk * D:].view(-1, Hk, D), cu_q, cu_k, max(lq), max(lk), out=out)
    want = h3.cross_attn_fwd_t(q, k, v, cu_q, cu_k, max(lq), max(lk))
    assert torch.equal(o, want) and torch.all(wide[:, Hq * D:] == 7.0)


@pytest.mark.parametrize("scale,std", [(0.0, 1.0), (0.5, 3.0), (1e-3, 1.0)])
@pytest.mark.parametrize("lq,lk,dtype", [([200], [700], "bf16"), ([3], [2500], "fp16")])
def test_cross_scales(scale, std, lq, lk, dtype):
    """scale 0 is the mean of the values; large scores leave one key a row."""
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, 3, 3, 128, dtype, std=std)
    o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk, softmax_scale=scale)
    _check_cross(q, k, v, cu_q, cu_k, o, lse, scale, None, f"scale {scale}")


def test_cross_growing_scores():
    """Every key tile raises the running maximum by more than the slack that
    lets the accumulator keep its scale."""
    import torch
    lq, lk, D = [140], [1000], 64
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, 2, 2, D, "bf16")
    q[:] = 1.0
    k[:] = (torch.arange(1000, device="cuda") / 64).to(q.dtype)[:, None, None]
    o, lse = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
    _check_cross(q, k, v, cu_q, cu_k, o, lse, D ** -0.5, None, "growing")


@pytest.mark.parametrize("cu_q,cu_k", [
    ([0, 60, 101], [0, 20, 70]), ([0, 70, 60], [0, 20, 70]), ([1, 60, 100], [0, 20, 70]),
    ([0, 60, 100], [0, 20, 71]), ([0, 60, 100], [0, 50, 40]), ([0, 60, 100], [5, 20, 70]),
    ([0, 80, 100], [0, 20, 70]), ([0, 60, 100], [0, 8, 70]),
])
def test_cross_bad_lengths_are_reported_and_nothing_is_written(cu_q, cu_k):
    import torch
    h3 = _h3()
    q, k, v, _, _ = _cross_case([100], [70], 2, 2, 64, "bf16")
    a, b = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_k))
    ws = h3.cross_workspace_for(100, 2, 2, 64, 2, 60, 60)
    out = torch.full_like(q, 7.0)
    h3.cross_attn_fwd_t(q, k, v, a, b, 60, 60, out=out, workspace=ws)
    assert h3.device_status_t(ws) == h3.H3_ERR_BAD_SEQLENS
    assert torch.all(out == 7.0)
    good = [torch.tensor(c, dtype=torch.int32, device="cuda") for c in ([0, 60, 100], [0, 20, 70])]
    h3.cross_attn_fwd_t(q, k, v, *good, 60, 60, out=out, workspace=ws)
    assert h3.device_status_t(ws) == h3.H3_OK


@pytest.mark.parametrize("lq,lk", [([1], [9000]), ([700, 300], [300, 77])])
def test_cross_is_deterministic(lq, lk):
    import torch
    q, k, v, cu_q, cu_k = _cross_case(lq, lk, 8, 2, 128, "bf16")
    first = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
    for _ in range(5):
        again = _run_cross(q, k, v, cu_q, cu_k, lq, lk)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------- together

def _block(h3, t, stream=None):
    """A conditioned block's second half as a user runs it: rotated queries and
    keys, cross attention, output projection on the residual stream, gated
    feed-forward on it."""
    lq, lk, H, Hk, D = t["lq"], t["lk"], 8, 2, 64
    q = h3.linear_t(t["x"], t["wq"], t["bq"], stream=stream).view(-1, H, D)
    kv = h3.linear_t(t["states"], t["wkv"], stream=stream)
    k, v = kv[:, :Hk * D].view(-1, Hk, D), kv[:, Hk * D:].view(-1, Hk, D)
    q, _ = h3.rope_qk_t(q, None, t["pos_q"], layout="half", out=(q, None), stream=stream)
    k, _ = h3.rope_qk_t(k, None, t["pos_k"], layout="half", stream=stream)
    o = h3.cross_attn_fwd_t(q, k, v, t["cu_q"], t["cu_k"], max(lq), max(lk), key_mask=t["mask"],
                            stream=stream)
    y = h3.linear_t(o.flatten(1), t["wo"], t["bo"], residual=t["x"], stream=stream)
    g = h3.linear_t(y, t["wg"], act="silu", gated=True, stream=stream)
    return h3.linear_t(g, t["wd"], residual=y, stream=stream)


def _block_inputs(dtype="bf16"):
    import torch
    rng = np.random.default_rng(77)
    d = _dtype(dtype)
    lq, lk, E = [200, 1, 90], [33, 140, 7], 256
    t = dict(lq=lq, lk=lk, cu_q=_cu(lq), cu_k=_cu(lk))
    t["x"], t["states"] = _draw(rng, (sum(lq), E), d), _draw(rng, (sum(lk), E), d)
    t["wq"], t["bq"] = _draw(rng, (512, E), d, E ** -0.5), _draw(rng, (512,), d, 0.1)
    t["wkv"], t["wo"] = _draw(rng, (256, E), d, E ** -0.5), _draw(rng, (E, 512), d, 512 ** -0.5)
    t["bo"], t["wg"] = _draw(rng, (E,), d, 0.1), _draw(rng, (1344, E), d, E ** -0.5)
    t["wd"] = _draw(rng, (E, 672), d, 672 ** -0.5)
    for n, l in (("pos_q", lq), ("pos_k", lk)):
        t[n] = torch.cat([torch.arange(i, dtype=torch.int32) for i in l]).cuda()
    t["mask"] = torch.from_numpy(rng.random(sum(lk)) < 0.8).cuda()
    return t


def _block_ref(t):
    f = {n: _f64(x) for n, x in t.items() if hasattr(x, "cpu")}
    fr = ref.rope_freqs_ref(64, 1e4)
    q = (f["x"] @ f["wq"].T + f["bq"]).reshape(-1, 8, 64)
    kv = f["states"] @ f["wkv"].T
    k, v = kv[:, :128].reshape(-1, 2, 64), kv[:, 128:].reshape(-1, 2, 64)
    q = ref.rope_qk_ref(q, f["pos_q"], 64, fr, "half")
    k = ref.rope_qk_ref(k, f["pos_k"], 64, fr, "half")
    o = ref.cross_attention_ref(q, k, v, t["cu_q"].cpu().numpy(), t["cu_k"].cpu().numpy(), 0.125,
                                f["mask"])[0]
    y = ref.linear_ref(o.reshape(-1, 512), f["wo"], f["bo"], residual=f["x"])[0]
    g = ref.linear_ref(y, f["wg"], None, "silu", True)[0]
    return ref.linear_ref(g, f["wd"], residual=y)[0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_block(dtype):
    # eight roundings of values of about 1 to 2, each at most u (2-norm: well
    # below u / sqrt 3 a step); 8 u relative in the 2-norm bounds the chain
    h3 = _h3()
    t = _block_inputs(dtype)
    got, want = _f64(_block(h3, t)), _block_ref(t)
    assert np.linalg.norm(got - want) <= 8 * _u(_dtype(dtype)) * np.linalg.norm(want)


def test_block_on_another_stream_and_captured():
    import torch
    h3 = _h3()
    t = _block_inputs()
    want = _block(h3, t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):   # a stream object, a raw handle
        got = _block(h3, t, stream)
        side.synchronize()
        assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _block(h3, t)
    for factor in (1.0, -0.5):
        t["x"].mul_(factor)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, _block(h3, t))


def test_short_calls_captured_and_replayed():
    """One graph with the forms for few rows: the sum over K shared by a cluster,
    the keys split and joined, one token rotated; replayed on changed inputs."""
    import torch
    h3 = _h3()
    x, w, b, _ = _linear_case(3, 512, 4096, "silu", False, True, False, "bf16")
    q0, k, v, cu_q, cu_k = _cross_case([1, 2], [5000, 300], 8, 2, 64, "bf16")
    pos = torch.tensor([7, 100000, -5], dtype=torch.int32, device="cuda")

    def run():
        y = h3.linear_t(x, w, b, "silu")
        q, _ = h3.rope_qk_t(y.view(3, 8, 64), None, pos, layout="half")
        return h3.cross_attn_fwd_t(q, k, v, cu_q, cu_k, 2, 5000, return_lse=True)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for factor in (1.0, 0.5, -2.0):
        x.mul_(factor)
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_same_buffer_twice():
    """One tensor as several inputs: keys as values, the input as the residual, q as k."""
    import torch
    h3 = _h3()
    q, k, _, cu_q, cu_k = _cross_case([70, 1], [200, 900], 4, 2, 64, "bf16")
    o, lse = _run_cross(q, k, k, cu_q, cu_k, [70, 1], [200, 900])
    _check_cross(q, k, k, cu_q, cu_k, o, lse, 0.125, None, "k as v")
    x, w, b, _ = _linear_case(150, 256, 256, "none", False, True, False, "bf16")
    _check_linear(x, w, b, "none", False, x, h3.linear_t(x, w, b, residual=x), "x as residual")
    pos = torch.arange(71, dtype=torch.int32, device="cuda")
    a, c = h3.rope_qk_t(q, q, pos)
    assert torch.equal(a, c)


def test_offsets_beyond_32_bits():
    """Rows that begin more than 2^31 elements into their tensor (5 GB views of one
    buffer): the last ones are right."""
    import torch
    h3 = _h3()
    rows, ld, tail = 150000, 16384, 300
    wide = torch.zeros(rows, ld, dtype=torch.bfloat16, device="cuda")
    assert (rows - tail) * ld > 2 ** 31
    wide[-tail:, :1024] = _draw(np.random.default_rng(9), (tail, 1024), torch.bfloat16)
    # rotary: q and k read and written in place of the wide rows' first 384 channels
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    q, k = wide[:, :256].view(rows, 4, 64), wide[:, 256:384].view(rows, 2, 64)
    want = h3.rope_qk_t(q[-tail:].contiguous(), k[-tail:].contiguous(), pos[-tail:])
    h3.rope_qk_t(q, k, pos, out=(q, k))
    assert torch.equal(q[-tail:], want[0]) and torch.equal(k[-tail:], want[1])
    # linear: x, residual and y in the wide rows
    w = _draw(np.random.default_rng(10), (96, 256), torch.bfloat16, 1 / 16)
    x, r, y = wide[:, :256], wide[:, 256:352], wide[:, 2048:2144]
    h3.linear_t(x, w, residual=r, out=y)
    _check_linear(x[-tail:], w, None, "none", False, r[-tail:], y[-tail:], "linear")
    # cross attention: the second of two segments, queries and keys at the end
    cu_q = torch.tensor([0, 10, 10 + tail], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, rows - tail, rows], dtype=torch.int32, device="cuda")
    v, qq = wide[:, 512:640].view(rows, 2, 64), q[-tail - 10:]
    mask = torch.ones(rows, dtype=torch.bool, device="cuda")
    mask[-1] = False
    o, lse = h3.cross_attn_fwd_t(qq, k, v, cu_q, cu, tail, rows, key_mask=mask, return_lse=True)
    near = torch.tensor([0, tail], dtype=torch.int32, device="cuda")
    _check_cross(qq[10:], k[-tail:], v[-tail:], near, near, o[10:], lse[:, 10:], 0.125, mask[-tail:],
                 "cross")


def test_two_calls_at_once():
    """Calls on two streams with workspaces of their own do not disturb each other."""
    import torch
    h3 = _h3()
    cases = [_cross_case([1], [20000], 8, 2, 128, "bf16", seed=s) for s in range(2)]
    lin = [_linear_case(2, 4000, 4096, "none", False, True, False, "bf16", seed=s) for s in range(2)]
    want = [h3.cross_attn_fwd_t(*c, 1, 20000) for c in cases]
    wantl = [h3.linear_t(x, w, b) for x, w, b, _ in lin]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append((h3.cross_attn_fwd_t(*cases[i], 1, 20000, stream=s),
                           h3.linear_t(*lin[i][:3], stream=s)))
    torch.cuda.synchronize()
    for i in range(2):
        for o, y in got[i]:
            assert torch.equal(o, want[i]) and torch.equal(y, wantl[i])


def test_helpers_refuse():
    import torch
    h3 = _h3()
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda")
    for call in (
        lambda: h3.linear_t(x.float(), w.float()), lambda: h3.linear_t(x, w.half()),
        lambda: h3.linear_t(x, w[:, :32]), lambda: h3.linear_t(x, w.cpu()),
        lambda: h3.linear_t(x, w, act="tanh"), lambda: h3.linear_t(x, w[:15], gated=True),
        lambda: h3.linear_t(x, w, bias=x[0]), lambda: h3.linear_t(x, w, residual=x),
        lambda: h3.linear_t(x.t(), w), lambda: h3.linear_t(x, w, out=x),
        lambda: h3.linear_t(x.clone().requires_grad_(), w),
        lambda: h3.rope_qk_t(x.view(4, 1, 64), None, torch.arange(4, device="cuda")),
        lambda: h3.rope_qk_t(x.view(4, 1, 64), w.view(16, 1, 64),
                             torch.zeros(4, dtype=torch.int32, device="cuda")),
        lambda: h3.cross_attn_fwd_t(x.view(4, 1, 64), w.view(16, 1, 64), w.view(16, 1, 64)[:3],
                                    _cu([4]), _cu([16]), 4, 16),
        lambda: h3.cross_attn_fwd_t(x.view(4, 1, 64), w.view(16, 1, 64), w.view(16, 1, 64),
                                    _cu([4]), _cu([16]), 4, 16,
                                    key_mask=torch.zeros(15, dtype=torch.bool, device="cuda")),
    ):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(h3.H3Error):   # rows of x not on 16 bytes
        h3.linear_t(torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")[:, :64], w)
