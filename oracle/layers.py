"""Float64 references of the layers around the attention: 1-D rotary
positions, linear layer with epilogue, cross attention. Inputs are float64
arrays that hold the device values exactly; each function also returns what
the tests' error bounds are made of.
"""

from __future__ import annotations

import math

import numpy as np


def rope_freqs_ref(rot_dim, theta, kind="none", factor=1.0, original_len=0.0, beta_fast=0.0,
                   beta_slow=0.0, attn_factor=1.0):
    """Angle per position of each pair, one at a time in Python floats."""
    out = []
    for j in range(rot_dim // 2):
        base = theta
        if kind == "ntk":
            base = theta * factor ** (rot_dim / (rot_dim - 2))
        f = base ** (-2.0 * j / rot_dim)
        if kind == "linear":
            f = f / factor
        if kind in ("turns", "yarn"):
            if kind == "turns":
                turns = original_len * f / (2 * math.pi)
                g = (turns - beta_slow) / (beta_fast - beta_slow)
            else:
                # the pair number at which a pair makes `b` turns over the original length
                number = [rot_dim / 2 * math.log(original_len / (2 * math.pi * b), theta)
                          for b in (beta_fast, beta_slow)]
                lo = max(math.floor(number[0]), 0)
                hi = min(math.ceil(number[1]), rot_dim - 1)
                g = 1 - (j - lo) / max(hi - lo, 0.001)
            g = min(1.0, max(0.0, g))
            f = g * f + (1 - g) * f / factor
        out.append(f)
    return np.array(out)


def rope_qk_ref(x, positions, rot_dim, freqs, layout, attn_factor=1.0):
    """x [N, H, D] rotated as complex numbers."""
    z = np.exp(1j * positions.astype(np.float64)[:, None] * freqs) * attn_factor
    y = np.array(x, dtype=np.float64)
    h = rot_dim // 2
    a, b = ((slice(0, h), slice(h, rot_dim)) if layout == "half"
            else (slice(0, rot_dim, 2), slice(1, rot_dim, 2)))
    t = (y[..., a] + 1j * y[..., b]) * z[:, None, :]
    y[..., a], y[..., b] = t.real, t.imag
    return y


_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation_ref(x, act):
    if act == "relu":
        return np.where(x < 0, 0.0, x)
    if act == "gelu":
        return 0.5 * x * (1 + _erf(x / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + np.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    if act == "silu":
        return x / (1 + np.exp(-x))
    assert act == "none"
    return x


def linear_ref(x, w, bias=None, act="none", gated=False, residual=None):
    """(y, spread): spread bounds |dy| per unit of relative error in every
    product x_i w_i (sum of |x_i w_i| and |bias|, through the activation, whose
    slope is at most 1.13, and the gate product)."""
    z = x @ w.T
    s = np.abs(x) @ np.abs(w).T
    if bias is not None:
        z = z + bias
        s = s + np.abs(bias)
    if gated:
        n = w.shape[0] // 2
        g = activation_ref(z[:, :n], act)
        y = g * z[:, n:]
        s = 1.13 * s[:, :n] * np.abs(z[:, n:]) + np.abs(g) * s[:, n:]
    else:
        y = activation_ref(z, act)
        s = 1.13 * s
    if residual is not None:
        y = y + residual
        s = s + np.abs(residual)
    return y, s


def cross_attention_ref(q, k, v, cu_q, cu_k, scale, mask=None):
    """(O, LSE, A, S): A = softmax-weighted |v| and S = largest scale * sum
    |q_i k_i| of a row over its kept keys, for error bounds."""
    Nq, Hq, D = q.shape
    G = Hq // k.shape[1]
    O, A = np.zeros((Nq, Hq, D)), np.zeros((Nq, Hq, D))
    lse, S = np.full((Hq, Nq), -np.inf), np.zeros((Nq, Hq))
    for s in range(len(cu_q) - 1):
        a, b = int(cu_q[s]), int(cu_q[s + 1])
        keys = np.arange(int(cu_k[s]), int(cu_k[s + 1]))
        if mask is not None:
            keys = keys[mask[keys] != 0]
        if b == a or keys.size == 0:
            continue
        for h in range(Hq):
            kk, vv = k[keys, h // G], v[keys, h // G]
            x = scale * (q[a:b, h] @ kk.T)
            m = x.max(axis=1, keepdims=True)
            p = np.exp(x - m)
            l = p.sum(axis=1, keepdims=True)
            O[a:b, h] = p @ vv / l
            A[a:b, h] = p @ np.abs(vv) / l
            lse[h, a:b] = (m + np.log(l))[:, 0]
            S[a:b, h] = scale * (np.abs(q[a:b, h]) @ np.abs(kk).T).max(axis=1)
    return O, lse, A, S
