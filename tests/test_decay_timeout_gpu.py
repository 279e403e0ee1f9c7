"""Waits of the head-decay attention's tensor-core kernel that run out: the call returns with a status, nothing is left in
flight, and flags and counters are fit for the next call.

A limit of less than a microsecond in DIG_DEVICE_WAIT_LIMIT_NS, i ns, shortens the waits to some 0.1 ms and lets the v tile
of chunk i - 1 of each block come only after the others have given up, or after a millisecond."""
import pytest
import torch

from tests.test_decay_attn_gpu import Case, _dig
from tests.test_timeout_gpu import wait_bound_ns

pytestmark = pytest.mark.gpu

CASES = [
    dict(B=3, H=2, dk=32, dv=64, L=2),                                       # a chunk a block
    dict(B=5, H=70, dk=32, dv=8, L=600),                                     # states handed on, whole rows
    dict(B=5, H=40, dk=72, dv=8, L=600, mode=1),                             # the same at D = 128, chunks of two and three terms
    dict(B=5, H=70, dk=32, dv=8, grid=(16, 38), mode=3),                     # column runs
    dict(B=4, H=50, dk=8, dv=72, grid=(32, 19), mode=2),
    dict(B=1, H=2, dk=32, dv=16, L=4100), dict(B=1, H=1, dk=72, dv=8, L=4200),   # a first pass and a kernel that joins
    dict(B=1, H=2, dk=36, dv=12, L=2500), dict(B=2, H=2, dk=20, dv=68, grid=(19, 70), mode=2),   # token by token
    dict(B=4, H=2, dk=32, dv=64, lens=[3000, 5, 0, 900], tail=7),            # packed, chunks that end inside their tiles
    dict(B=3, H=3, dk=128, dv=40, lens=[129, 1500, 640], tail=1, mode=1),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_expiry_is_reported_and_the_workspace_is_fit_for_the_next_call(i, backward):
    dig = _dig()
    c = Case(dtype="bf16", seed=i, states=True, **CASES[i])
    S0, dSf, g = c.S0.cuda(), c.dSf.cuda(), c.g.cuda()
    ws = c.workspace(backward=backward)

    def run():
        if backward:
            out = [torch.zeros_like(x) for x in (c.q, c.k, c.v, S0)]
            dig.dig_decay_attn_bwd(c.q, c.k, c.v, g, c.dO, *out[:3], ws, S0=S0, dS_final=dSf, dS0=out[3], **c.call())
        else:
            out = [torch.zeros_like(c.v), torch.zeros_like(S0)]
            dig.dig_decay_attn_fwd(c.q, c.k, c.v, g, out[0], ws, S0=S0, S_final=out[1], **c.call())
        return out

    want = run()
    assert dig.dig_read_status(ws) == dig.DIG_OK
    for limit in (1, 2, 4):
        with wait_bound_ns(limit):
            got = run()
            torch.cuda.synchronize()  # no CUDA error: the blocks drained and left
        status = dig.dig_read_status(ws)
        # a block of fewer chunks has none that could be late
        assert status == dig.DIG_ERR_DEVICE_TIMEOUT if limit == 1 else status in (dig.DIG_OK, dig.DIG_ERR_DEVICE_TIMEOUT)
        if status == dig.DIG_OK:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert not ws[:2048].any()    # status read and cleared, counters and flags left zero
        ws.zero_()
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
        assert dig.dig_read_status(ws) == dig.DIG_OK
