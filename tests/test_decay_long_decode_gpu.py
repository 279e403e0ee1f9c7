"""Thousands of single tokens at decays near 1: the states follow the recurrence to the roundings of the states themselves."""
import numpy as np
import pytest
import torch

from tests import decay_reference as ref

pytestmark = pytest.mark.gpu
N, H, D = 4096, 4, 64


def _decays():
    """Log decays whose exp, rounded to fp32, is nearly half a step off: the two furthest above and the two furthest below."""
    g = -(np.arange(1, 2000) * 1e-6).astype(np.float32)
    off = np.exp(g.astype(np.float64)).astype(np.float32).astype(np.float64) / np.exp(g.astype(np.float64)) - 1
    order = np.argsort(off)
    g = g[[order[0], order[1], order[-1], order[-2]]]
    assert np.abs(off[order[[0, 1, -1, -2]]]).min() > 0.9 * ref.U32 / 2
    return torch.from_numpy(g).cuda()


def _check(got, want, size):
    """A state is rounded three times a token, by at most U32 of it each (once where nothing is added): the roundings go
    either way, so that after N tokens they leave sqrt(N) of that, in the 2-norm over the head's values."""
    for h in range(H):
        off = (got[:, h].double() - want[:, h]).norm() / size[:, h].norm()
        assert off <= np.sqrt(3 * N) * ref.U32, (h, off.item())


def test_states_decay_as_given():
    from gated_linear_attention_fwd_b200 import dig
    g = _decays()
    gen = torch.Generator().manual_seed(1)
    S = torch.randn(1, H, D, D, generator=gen).cuda()
    want = S.double() * torch.exp(g.double() * N)[:, None, None]
    zero, o = torch.zeros(1, H, D, device="cuda"), torch.empty(1, H, D, device="cuda")
    for _ in range(N):
        dig.dig_decay_attn_step(zero, zero, zero, g, S, o)
    _check(S, want, want)


def test_tokens_one_by_one_end_where_the_prompt_form_does():
    from gated_linear_attention_fwd_b200 import dig
    g = _decays()
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(1, N, H, D, generator=gen).cuda() for _ in range(3))
    S, o = torch.zeros(1, H, D, D, device="cuda"), torch.empty(1, H, D, device="cuda")
    want, lam = S.double(), torch.exp(g.double())[:, None, None]
    for t in range(N):
        dig.dig_decay_attn_step(q[:, t], k[:, t], v[:, t], g, S, o)
        want = lam * want + k[:, t].double()[..., None] * v[:, t].double()[..., None, :]
    prompt, out = torch.empty_like(S), torch.empty_like(q)
    dig.dig_decay_attn_fwd(q, k, v, g, out, dig.new_decay_attn_workspace(1, H, N, D, D, dtype=torch.float32), S_final=prompt)
    _check(S, want, want)
    _check(prompt, want, want)
    last = torch.einsum("bhk,bhkv->bhv", q[:, -1].double(), want)
    for h in range(H):   # a sum over D channels of values that are off by as much
        for got in (o[:, h], out[:, -1, h]):
            assert (got.double() - last[:, h]).norm() <= np.sqrt(3 * N + D) * ref.U32 * q[:, -1, h].norm() * want[:, h].norm()
