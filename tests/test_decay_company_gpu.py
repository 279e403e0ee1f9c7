"""The same sequence alone and in different company: where it is cut among blocks may change, and so its roundings, no more;
the same call again gives the same bits."""
import numpy as np
import pytest
import torch

from tests import decay_reference as ref
from tests.test_decay_attn_gpu import Case, _close, _np

pytestmark = pytest.mark.gpu


def _run(c):
    """Outputs and final states of the call, twice, which have to be the same bits."""
    res = []
    for _ in range(2):
        Sf = torch.zeros(c.B, c.H, c.dk, c.dv, device="cuda")
        o, _ = c.fwd(S0=c.S0.cuda(), Sf=Sf)
        res.append((o, Sf))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    return res[0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H, dk, dv, lens", [(2, 64, 64, [300, 1100, 500]), (6, 32, 64, [4000, 1500, 3]), (3, 128, 72, [129, 2000, 64]),
                                             (2, 36, 72, [700, 900, 100])])
def test_a_packed_sequence_alone_and_among_others(H, dk, dv, lens, dtype):
    many = Case(B=3, H=H, dk=dk, dv=dv, dtype=dtype, lens=lens, states=True, seed=1)
    first, n = many.seqs[1]
    one = Case(B=1, H=H, dk=dk, dv=dv, dtype=dtype, L=n, states=True, seed=2)
    one.g, one.S0 = many.g, many.S0[1:2]
    one.q, one.k, one.v, one.dO = (x[first:first + n][None].contiguous() for x in (many.q, many.k, many.v, many.dO))
    one.host = [x[first:first + n] for x in many.host]
    o, Sf = _run(many)
    o1, Sf1 = _run(one)
    want, S, size, Ssize = one.reference()
    tol = ref.attn_bound(size, n, dk, dv, one.bf16)
    for got, state in ((o[first:first + n], Sf[1:2]), (o1[0], Sf1)):
        _close(got, want, tol, one.out_dtype, "o")
        _close(state, S, ref.attn_bound(Ssize, n, dk, dv, False), torch.float32, "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_whole_sequences_in_smaller_and_larger_batches(dtype):
    """256 tokens, 6 heads of 64/64: several segments a sequence among 8 sequences, one among 64."""
    big = Case(B=64, H=6, dk=64, dv=64, dtype=dtype, L=256, states=True, seed=3)
    o, Sf = _run(big)
    small = Case(B=8, H=6, dk=64, dv=64, dtype=dtype, L=256, states=True, seed=4)
    small.g, small.S0 = big.g, big.S0[:8]
    small.q, small.k, small.v = (x[:8].contiguous() for x in (big.q, big.k, big.v))
    o8, Sf8 = _run(small)
    # each is off its value by attn_bound at most (test_forward_whole_sequences), the two by twice that and both roundings
    size = [np.abs(x) for x in big.host[:3]]
    S = np.abs(_np(big.S0[:8]))
    ob, Sb = ref.attn(*[x[:8 * 256] for x in size], big.g.numpy(), big.seqs[:8], S0=S)
    tol = 2 * ref.attn_bound(ob, 256, 64, 64, small.bf16) + 2 * (ref.UBF if small.bf16 else ref.U32) * np.abs(_np(o8)).reshape(ob.shape) * 1.01
    assert (np.abs(_np(o[:8]) - _np(o8)).reshape(ob.shape) <= tol).all()
    assert (np.abs(_np(Sf[:8]) - _np(Sf8)) <= 2 * ref.attn_bound(Sb, 256, 64, 64, False)).all()
