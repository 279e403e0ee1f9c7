"""Sizes beyond what the kernels count in are refused: by the binding where an int does not hold them, by the library above its own limits."""
import pytest
import torch

from gated_linear_attention_fwd_b200 import dig

BIG = (1 << 32) + 8     # its low 32 bits are 8


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_the_binding_refuses_what_an_int_does_not_hold():
    g = _meta(1, dtype=torch.float32)
    ws = _meta(4096, dtype=torch.uint8)
    x = _meta(1, BIG)
    row = _meta(1, dtype=torch.float32)
    calls = [
        lambda: dig.dig_layer_norm_fwd(x, x),
        lambda: dig.dig_layer_norm_bwd(x, x, row, row, x),
        lambda: dig.new_layer_norm_workspace(1, BIG),
        lambda: dig.new_decay_attn_workspace(1, 1, BIG, 4, 4),
        lambda: dig.dig_decay_attn_step(*[_meta(BIG, 1, 4)] * 3, g, _meta(8, 1, 4, 4, dtype=torch.float32), _meta(BIG, 1, 4)),
        lambda: dig.dig_decay_attn_step(*[_meta(8, 1, 4)] * 3, g, _meta(BIG, 1, 4, 4, dtype=torch.float32), _meta(8, 1, 4)),
    ]
    for lead, cu in (((1, BIG), None), ((BIG, 8), None), ((BIG,), _meta(2, dtype=torch.int32))):
        t = _meta(*lead, 1, 4)
        calls += [lambda t=t, cu=cu: dig.dig_decay_attn_fwd(t, t, t, g, t, ws, cu_seqlens=cu),
                  lambda t=t, cu=cu: dig.dig_decay_attn_bwd(t, t, t, g, t, t, t, t, ws, cu_seqlens=cu)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="more than the library takes"):
            call()


def test_layer_norm_refuses_widths_past_its_counters():
    D = (1 << 30) + 1
    assert dig.lib.dig_layer_norm_fwd(1024, D, None, None, 1e-5, 1024, None, None, 1, D, 1, 1, None) == dig.DIG_ERR_INVALID_ARGUMENT
    assert dig.lib.dig_layer_norm_bwd(1024, D, None, 1024, 1024, 1024, 1024, None, None, 1, D, 1, 1, None, 0, None) == \
        dig.DIG_ERR_INVALID_ARGUMENT
