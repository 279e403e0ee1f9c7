"""Head-decay linear attention on the GPU where the work is cut across blocks: states handed from block to block, or formed
by a first pass and joined; tiles fetched as rows, column runs or token by token."""
import pytest
import torch

from tests import decay_reference as ref
from tests.test_decay_attn_gpu import Case, _close, _dig

pytestmark = pytest.mark.gpu

# more units (sequences x heads) than blocks run at once, each shorter than a block's share: handed over
HANDED = [
    dict(B=5, H=70, dk=32, dv=8, L=600), dict(B=5, H=70, dk=32, dv=8, grid=(16, 38), mode=3),
    dict(B=5, H=40, dk=72, dv=8, L=600, mode=1), dict(B=4, H=50, dk=8, dv=72, grid=(32, 19), mode=2),
]
# few units, each over several blocks, or over 32 and more
JOINED = [
    dict(B=1, H=2, dk=32, dv=16, L=4001), dict(B=2, H=1, dk=16, dv=64, grid=(16, 150), mode=3),
    dict(B=1, H=2, dk=72, dv=8, L=3000, mode=1), dict(B=1, H=1, dk=128, dv=128, L=700),
    dict(B=1, H=2, dk=36, dv=12, L=2500), dict(B=1, H=1, dk=72, dv=8, L=4200), dict(B=3, H=20, dk=72, dv=8, L=1100, mode=1), dict(B=1, H=2, dk=20, dv=68, grid=(19, 70), mode=2),
]
PACKED = [
    dict(B=4, H=2, dk=32, dv=64, lens=[3000, 5, 0, 900], tail=7), dict(B=4, H=2, dk=32, dv=64, lens=[3000, 5, 0, 900], tail=7, mode=1),
    dict(B=3, H=3, dk=128, dv=40, lens=[129, 1500, 640], tail=1), dict(B=3, H=2, dk=68, dv=12, lens=[1, 2000, 257], mode=1),
]


@pytest.mark.parametrize("i", range(len(HANDED)))
def test_states_handed_from_block_to_block(i):
    Case(dtype="bf16", seed=i, states=i != 1, **HANDED[i]).check_fwd()
    Case(dtype="bf16", seed=20 + i, states=i != 2, **HANDED[i]).check_bwd()


@pytest.mark.parametrize("i", range(len(JOINED)))
def test_states_joined(i):
    Case(dtype="bf16", seed=40 + i, states=True, **JOINED[i]).check_fwd()
    Case(dtype="bf16", seed=60 + i, states=i % 2 == 0, **JOINED[i]).check_bwd()


@pytest.mark.parametrize("i", range(len(PACKED)))
def test_long_packed_sequences(i):
    Case(dtype="bf16", seed=80 + i, states=True, **PACKED[i]).check_fwd()
    Case(dtype="bf16", seed=90 + i, states=True, **PACKED[i]).check_bwd()


def test_initial_states_continued_in_place():
    """S_final over S0 where one block reads a state and another writes it."""
    for kw in (dict(B=1, H=2, dk=32, dv=16, L=2000), dict(B=5, H=40, dk=72, dv=8, L=600), dict(B=2, H=2, dk=64, dv=64, lens=[1400, 600])):
        c = Case(dtype="bf16", seed=7, states=True, **kw)
        P = c.S0.cuda()
        o, ws = c.fwd(S0=P, Sf=P)
        assert _dig().dig_read_status(ws) == _dig().DIG_OK
        want, S, size, Ssize = c.reference()
        _close(o.reshape(-1, c.H, c.dv), want, ref.attn_bound(size, c.longest, c.dk, c.dv, True), c.out_dtype, "o")
        _close(P, S, ref.attn_bound(Ssize, c.longest, c.dk, c.dv, False), torch.float32, "state")


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("dk, dv", [(64, 64), (128, 72), (36, 36)])
def test_nothing_crosses_between_packed_sequences(dk, dv, mode):
    """NaN and infinities of one sequence stay in it, forward and backward, where tiles reach over its ends."""
    dig = _dig()
    lens = [70, 300, 45]
    c = Case(B=3, H=2, dk=dk, dv=dv, dtype="bf16", lens=lens, mode=mode, seed=3)
    grads = lambda: [torch.zeros_like(x) for x in (c.q, c.k, c.v)]
    ws = c.workspace(backward=True)

    def run():
        o, _ = c.fwd()
        g = grads()
        dig.dig_decay_attn_bwd(c.q, c.k, c.v, c.g.cuda(), c.dO, *g, ws, **c.call())
        return [o, *g]

    before = run()
    for x in (c.q, c.k, c.v, c.dO):
        x[70:370] = float("nan")
    c.v[100:200] = float("inf")
    for a, b in zip(before, run()):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[370:], b[370:])


def test_one_workspace_for_calls_of_different_shapes():
    """A workspace large enough for several calls serves them in turn; each leaves it fit for the next."""
    cases = [Case(dtype="bf16", seed=11 + i, **kw) for i, kw in enumerate((HANDED[0], JOINED[0], HANDED[2], JOINED[3], PACKED[0]))]
    shared = torch.zeros(max(c.workspace().numel() for c in cases), dtype=torch.uint8, device="cuda")
    fresh = [c.fwd()[0] for c in cases]
    for _ in range(2):
        for c, want in zip(cases, fresh):
            assert torch.equal(c.fwd(ws=shared)[0], want)
    assert _dig().dig_read_status(shared) == _dig().DIG_OK


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, where blocks wait for blocks of their own call."""
    cases = [Case(dtype="bf16", seed=30 + i, **HANDED[i]) for i in (0, 2)]
    want = [c.fwd()[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [c.workspace() for c in cases]
    outs = [[torch.zeros_like(w) for _ in range(5)] for w in want]
    gs = [c.g.cuda() for c in cases]
    torch.cuda.synchronize()
    for n in range(5):
        for c, s, w, o, g in zip(cases, streams, ws, outs, gs):
            _dig().dig_decay_attn_fwd(c.q, c.k, c.v, g, o[n], w, stream=s, **c.call())
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, w) for x in o)


def test_captured_and_replayed_backward():
    for kw in (HANDED[2], JOINED[0]):
        c = Case(dtype="bf16", seed=50, states=True, **kw)
        dig = _dig()
        S0, dSf, g = c.S0.cuda(), c.dSf.cuda(), c.g.cuda()
        ws = c.workspace(backward=True)
        outs = [torch.empty_like(x) for x in (c.q, c.k, c.v)]
        dS0 = torch.empty_like(S0)
        call = lambda: dig.dig_decay_attn_bwd(c.q, c.k, c.v, g, c.dO, *outs, ws, S0=S0, dS_final=dSf, dS0=dS0, **c.call())
        call()
        want = [x.clone() for x in (*outs, dS0)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for _ in range(3):
            for x in (*outs, dS0):
                x.zero_()
            graph.replay()
            assert all(torch.equal(x, w) for x, w in zip((*outs, dS0), want))


def test_training_step_of_norm_and_attention():
    """Layer norm -> fused q, k, v slices -> attention, and back through both, against automatic differentiation in 64 bits."""
    dig = _dig()
    B, L, H, dk, dv = 2, 150, 3, 32, 64
    D = H * (2 * dk + dv)
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(B, L, D, generator=gen)
    w, b = 0.2 + 0.05 * torch.randn(D, generator=gen), 0.05 * torch.randn(D, generator=gen)
    g = -torch.exp2(-2.0 * torch.arange(1, H + 1))
    dO = torch.randn(B, L, H, dv, generator=gen)

    xr, wr, br = (t.double().requires_grad_() for t in (x, w, b))
    q, k, v = torch.nn.functional.layer_norm(xr, (D,), wr, br, 1e-5).split([H * dk, H * dk, H * dv], -1)
    q, k, v = q.unflatten(-1, (H, dk)), k.unflatten(-1, (H, dk)), v.unflatten(-1, (H, dv))
    S, outs = torch.zeros(B, H, dk, dv, dtype=torch.float64), []
    for t in range(L):
        S = torch.exp(g.double())[:, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        outs.append(torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    want_o = torch.stack(outs, 1)
    (want_o * dO.double()).sum().backward()

    xd, wd, bd, gd, dOd = (t.cuda() for t in (x, w, b, g, dO))
    y, mean, rstd = torch.empty_like(xd), torch.empty(B * L, device="cuda"), torch.empty(B * L, device="cuda")
    dig.dig_layer_norm_fwd(xd, y, weight=wd, bias=bd, mean=mean, rstd=rstd)
    sizes = [H * dk, H * dk, H * dv]
    qkv = [p.unflatten(-1, (H, d)) for p, d in zip(y.split(sizes, -1), (dk, dk, dv))]
    o = torch.empty(B, L, H, dv, device="cuda")
    ws = dig.new_decay_attn_workspace(B, H, L, dk, dv, dtype=torch.float32)
    dig.dig_decay_attn_fwd(*qkv, gd, o, ws)
    grads = [torch.empty(B, L, H, d, device="cuda") for d in (dk, dk, dv)]
    wsb = dig.new_decay_attn_workspace(B, H, L, dk, dv, dtype=torch.float32, backward=True)
    dig.dig_decay_attn_bwd(*qkv, gd, dOd, *grads, wsb)
    dy = torch.cat([t.flatten(-2) for t in grads], -1)
    dx, dw, db = torch.empty_like(xd), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    dig.dig_layer_norm_bwd(xd, dy, mean, rstd, dx, weight=wd, dw=dw, db=db, workspace=dig.new_layer_norm_workspace(B * L, D))
    # chains of at most dk + dv + L + D additions of fp32 values, whose roundings add up like random numbers do: the root of
    # their number times 2^-24, times four for the four operators in a row
    bound = 4 * (dk + dv + L + D) ** 0.5 * 2.0 ** -24
    for got, want in ((o, want_o), (dx, xr.grad), (dw, wr.grad), (db, br.grad)):
        want = want.detach()
        assert (got.double().cpu() - want).norm() <= bound * want.norm()
