"""Calls of the layers around the attention that are refused before any CUDA
call: sizes and factors beyond their types, outputs that overlap."""

import pytest

import audio_diffusion_transformer_h3_b200 as h3
from test_layers_abi import _cfg, _cross, _linear, _rope

WRAP = 1 << 32   # what a 32-bit size loses


def test_sizes_beyond_32_bits_do_not_come_round():
    for call, sizes in ((_linear, dict(N=50, K=100, act=1, dtype=0)),
                        (_rope, dict(Hq=8, Hk=2, D=128, dtype=0)),
                        (_cross, dict(nseg=2, max_q=60, max_k=40, Hq=4, Hk=2, D=128, dtype=0))):
        for name, value in sizes.items():
            for far in (value + WRAP, value + (1 << 40), value - WRAP):
                assert call(**{name: far}) == h3.H3_ERR_INVALID_ARG, (call.__name__, name, far)
    for far in (WRAP, -WRAP):
        assert h3.h3_linear_workspace_size(5, 5 + far, 5, 0) == 0
        assert h3.h3_linear_workspace_size(5, 5, 5 + far, 0) == 0
        assert h3.h3_linear_workspace_size(5, 5, 5, far) == 0
        good = (10, 4, 2, 64, 1, 10, 10)
        assert h3.h3_cross_workspace_size(*good) > 0
        for i in range(1, 7):
            assert h3.h3_cross_workspace_size(*good[:i], good[i] + far, *good[i + 1:]) == 0
    for far in (WRAP, -WRAP):
        with pytest.raises(ValueError):
            h3.rope_qk_cfg(64 + far, 1e4)


def test_rope_factors_beyond_fp32():
    """cos and sin are multiplied in fp32: a factor that is infinite there turns zeros into NaN."""
    for bad in (1e39, -1e39, 1.7e308):
        assert _rope(_cfg(attn_factor=bad)) == h3.H3_ERR_INVALID_ARG
        with pytest.raises(h3.H3Error):
            h3.h3_rope_qk_freqs(_cfg(attn_factor=bad))
    assert len(h3.h3_rope_qk_freqs(_cfg(attn_factor=3.4e38))) == 32


def test_rope_outputs_that_are_other_operands():
    """Blocks of q and k run in no order: an output that is the other's input or
    output would be read and written at once."""
    for bad in (dict(k_out=0x20000, ldk_out=1024), dict(q_out=0x30000), dict(k_out=0x10000),
                dict(q_out=0x10000, k_out=0x10000), dict(q=0x10000, k=0x10000, q_out=0x10000),
                dict(q=0x10000, k=0x10000, q_out=0x10000, k_out=0x10000)):
        a = dict(Hq=2, Hk=2, ldq=1024, ldk=1024, ldq_out=1024, ldk_out=1024)
        a.update(bad)
        assert _rope(**a) == h3.H3_ERR_INVALID_ARG, bad
