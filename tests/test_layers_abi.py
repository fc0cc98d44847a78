"""The layers around the attention, without a GPU: refusals before any CUDA
call, workspace sizes, and the rotary frequencies against the reference."""

import ctypes
import math

import numpy as np
import pytest

import audio_diffusion_transformer_h3_b200 as h3
from oracle import layers as ref

YARN = dict(kind="yarn", factor=4.0, original_len=32768, beta_fast=32.0, beta_slow=1.0)


@pytest.mark.parametrize("scaling", [
    None,
    dict(kind="linear", factor=2.5),
    dict(kind="ntk", factor=4.0),
    dict(kind="turns", factor=8.0, original_len=8192, beta_fast=4.0, beta_slow=1.0),
    YARN,
    dict(YARN, original_len=100, factor=40.0),      # every pair below beta_slow at the end
    dict(YARN, original_len=1e9),                   # no pair is stretched
])
@pytest.mark.parametrize("rot_dim,theta", [(128, 1e6), (40, 1e4), (4, 500.0), (512, 1e4)])
def test_rope_frequencies(scaling, rot_dim, theta):
    got = h3.h3_rope_qk_freqs(h3.rope_qk_cfg(rot_dim, theta, "half", scaling))
    want = ref.rope_freqs_ref(rot_dim, theta, **(scaling or {}))
    # a few roundings of double in pow and log; the YARN ramp divides by hi - lo
    assert np.all(np.abs(got - want) <= 1e-12 * np.abs(want))


def _cfg(**over):
    c = h3.rope_qk_cfg(64, 1e4, "half", YARN)
    for name, value in over.items():
        setattr(c, name, value)
    return c


def _rope(cfg=None, **over):
    a = dict(q=0x10000, ldq=1024, q_out=0x20000, ldq_out=1024, k=0x30000, ldk=256, k_out=0x40000,
             ldk_out=256, positions=0x50000, cfg=cfg or _cfg(), N=100, Hq=8, Hk=2, D=128, dtype=0,
             stream=0)
    a.update(over)
    return h3.h3_rope_qk_apply(**a)


def test_rope_refusals():
    for bad in (dict(rot_dim=0), dict(rot_dim=63), dict(rot_dim=130), dict(rot_dim=-2),
                dict(layout=2), dict(scaling=5), dict(scaling=-1), dict(reserved=1),
                dict(theta=0.0), dict(theta=math.nan), dict(theta=0.9), dict(factor=0.0),
                dict(factor=math.inf), dict(original_len=0.0), dict(beta_slow=32.0),
                dict(attn_factor=math.nan)):
        assert _rope(_cfg(**bad)) == h3.H3_ERR_INVALID_ARG, bad
    for bad in (dict(N=-1), dict(Hq=0), dict(Hq=65536), dict(Hk=-1), dict(ldq=1023),
                dict(ldk_out=255), dict(q=0), dict(k=0), dict(k_out=0), dict(positions=0),
                dict(ldq=1 << 46), dict(N=(1 << 30) + 1), dict(q_out=0x10000, ldq_out=1032)):
        assert _rope(**bad) == h3.H3_ERR_INVALID_ARG, bad
    for bad in (dict(D=513), dict(D=1), dict(dtype=3), dict(dtype=-1)):
        assert _rope(**bad) == h3.H3_ERR_UNSUPPORTED, bad
    for bad in (dict(q=0x10001), dict(k_out=0x40001), dict(positions=0x50002),
                dict(dtype=2, q=0x10002)):
        assert _rope(**bad) == h3.H3_ERR_MISALIGNED, bad
    assert _rope(_cfg(scaling=h3.ROPE_SCALINGS["ntk"], rot_dim=2)) == h3.H3_ERR_INVALID_ARG
    # nothing to do: succeeds without a device
    assert _rope(N=0, q=0, q_out=0, k=0, k_out=0, positions=0) == h3.H3_OK
    assert h3._lib.h3_rope_qk_freqs(None, None) == h3.H3_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        h3.rope_qk_cfg(64, 1e4, "halves")
    with pytest.raises(ValueError):
        h3.rope_qk_cfg(64, 1e4, "half", dict(kind="spline"))
    with pytest.raises(ValueError):
        h3.rope_qk_cfg(64, 1e4, "half", dict(kind="yarn", beta=3))


def _linear(**over):
    a = dict(x=0x10000, ldx=104, w=0x20000, ldw=104, bias=0x30000, residual=0x40000, ldr=50,
             y=0x50000, ldy=50, M=33, N=50, K=100, act=1, dtype=0, workspace=0x60000,
             workspace_bytes=1 << 30, stream=0)
    a.update(over)
    return h3.h3_linear_fwd(**a)


def test_linear_refusals():
    for bad in (dict(M=-1), dict(M=2 ** 31 - 256), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0),
                dict(K=(1 << 20) + 1), dict(act=5), dict(act=-1), dict(act=512),
                dict(act=256 + 5), dict(ldx=96), dict(ldw=96), dict(ldy=49), dict(ldr=49),
                dict(x=0), dict(w=0), dict(y=0), dict(y=0x10000), dict(y=0x20000),
                dict(y=0x40000, ldy=51), dict(ldx=1 << 40), dict(ldy=1 << 32)):
        assert _linear(**bad) == h3.H3_ERR_INVALID_ARG, bad
    for bad in (dict(dtype=2), dict(dtype=-1)):
        assert _linear(**bad) == h3.H3_ERR_UNSUPPORTED, bad
    for bad in (dict(x=0x10008), dict(w=0x20008), dict(ldx=100), dict(ldw=102), dict(bias=0x30001),
                dict(residual=0x40001), dict(y=0x50001)):
        assert _linear(**bad) == h3.H3_ERR_MISALIGNED, bad
    for bad in (dict(workspace=0), dict(workspace=0x60010), dict(workspace_bytes=255)):
        assert _linear(**bad) == h3.H3_ERR_WORKSPACE, bad
    # one byte less than the size asked for is too little, for few rows too
    need = h3.h3_linear_workspace_size(2, 5376, 5376, 0)
    assert need >= 256
    assert _linear(M=2, N=5376, K=5376, ldx=5376, ldw=5376, ldr=5376, ldy=5376,
                   workspace_bytes=need - 1) == h3.H3_ERR_WORKSPACE
    assert h3.h3_linear_workspace_size(-1, 5, 5, 0) == 0
    assert h3.h3_linear_workspace_size(5, 5, 5, 7) == 0


def _cross(**over):
    a = dict(q=0x10000, ldq=512, k=0x20000, ldk=256, v=0x30000, ldv=256, o=0x40000, ldo=512, lse=0,
             cu_q=0x50000, cu_k=0x60000, nseg=2, max_q=60, max_k=40, key_mask=0, Nq=100, Nk=70,
             Hq=4, Hk=2, D=128, softmax_scale=0.1, dtype=0, workspace=0x70000,
             workspace_bytes=1 << 30, stream=0)
    a.update(over)
    return h3.h3_cross_attn_fwd(**a)


def test_cross_refusals():
    for bad in (dict(Nq=-1), dict(Nq=2 ** 31), dict(Nk=-1), dict(Hq=3), dict(Hk=0),
                dict(Hq=65536), dict(Hq=1), dict(nseg=0), dict(nseg=65536), dict(max_q=0),
                dict(max_q=101), dict(max_k=-1), dict(max_k=71), dict(q=0), dict(o=0), dict(k=0),
                dict(v=0), dict(cu_q=0), dict(cu_k=0), dict(softmax_scale=math.inf),
                dict(softmax_scale=-1.0), dict(softmax_scale=3e38), dict(ldq=504), dict(ldv=248), dict(ldo=504),
                dict(o=0x10000), dict(o=0x30000), dict(ldk=1 << 32)):
        assert _cross(**bad) == h3.H3_ERR_INVALID_ARG, bad
    for bad in (dict(D=96), dict(dtype=2), dict(dtype=-1)):
        assert _cross(**bad) == h3.H3_ERR_UNSUPPORTED, bad
    for bad in (dict(q=0x10008), dict(k=0x20002), dict(ldq=516), dict(ldk=260), dict(lse=0x90002),
                dict(cu_k=0x60002)):
        assert _cross(**bad) == h3.H3_ERR_MISALIGNED, bad
    for bad in (dict(workspace=0), dict(workspace=0x70010), dict(workspace_bytes=255)):
        assert _cross(**bad) == h3.H3_ERR_WORKSPACE, bad
    need = h3.h3_cross_workspace_size(1, 8, 8, 64, 1, 1, 60000)
    assert _cross(Nq=1, Nk=60000, Hq=8, Hk=8, D=64, nseg=1, max_q=1, max_k=60000, ldk=512, ldv=512,
                  workspace_bytes=need - 1) == h3.H3_ERR_WORKSPACE
    assert h3.h3_cross_workspace_size(10, 3, 2, 64, 1, 10, 10) == 0
    assert h3.h3_cross_workspace_size(10, 4, 2, 80, 1, 10, 10) == 0


def test_helpers_refuse_host_tensors():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        h3.linear_t(x, x)
    with pytest.raises(ValueError):
        h3.rope_qk_t(x.view(4, 1, 8), None, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        h3.cross_attn_fwd_t(x, x, x, x, x, 1, 1)


def test_struct_matches_the_header():
    assert ctypes.sizeof(h3.h3_rope_qk_cfg) == 64
