"""Head-decay linear attention on the GPU (prompt form, backward, single tokens) against the 64-bit recurrence."""
import numpy as np
import pytest
import torch

from tests import decay_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _dig():
    from gated_linear_attention_fwd_b200 import dig
    return dig


def _rand(gen, *shape, dt, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dt)


def _np(t):
    return t.double().cpu().numpy()


def _decays(H, gen, kind):
    if kind == "edge":  # no decay, total decay, almost none, strong, ...
        return torch.tensor([0.0, -float("inf"), -1e-4, -3.0, -0.05, -40.0])[:H].clone()
    return -torch.exp2(-8 * torch.arange(1, H + 1) / H) * (1 + 0.1 * torch.rand(H, generator=gen))


def _close(got, want, bound, out_dtype, what):
    """Every element within its bound, and half a step more where the output is rounded to bf16."""
    got, want = _np(got), np.asarray(want)
    tol = bound + np.abs(want) * (ref.U32 if out_dtype == torch.float32 else ref.UBF * (1 + ref.UBF)) + bound * ref.UBF
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - want)[bad] / (tol[bad] + 1e-300)))
    # the roundings are independent of one another, so in the 2-norm, where random terms add up like their roundings,
    # two of at most UBF each (the output's and the state's) leave sqrt(2) UBF
    size = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= (ref.U32 * 128 if out_dtype == torch.float32 else 1.5 * ref.UBF) * size + 1e-30, what


class Case:
    """Inputs of one call: B sequences, whole (lens None) or packed."""

    def __init__(self, B, H, dk, dv, dtype, L=None, grid=None, lens=None, tail=0, mode=0, scale=1.0, states=False,
                 decays="slopes", fused=False, out_dtype=None, seed=0):
        gen = torch.Generator().manual_seed(seed)
        dt = DT[dtype]
        self.__dict__.update(B=B, H=H, dk=dk, dv=dv, dtype=dt, bf16=dtype == "bf16" and out_dtype != "f32", grid=grid, mode=mode, scale=scale,
                             out_dtype=DT[out_dtype] if out_dtype else dt, packed=lens is not None)
        if lens is not None:
            self.L = sum(lens) + tail
            first = np.concatenate([[0], np.cumsum(lens)])
            self.seqs = list(zip(first[:-1].tolist(), lens))
            self.cu = torch.tensor(first, dtype=torch.int32, device="cuda")
            lead = (self.L,)
        else:
            self.L = L if grid is None else grid[0] * grid[1]
            self.seqs = [(b * self.L, self.L) for b in range(B)]
            self.cu, lead = None, (B, self.L)
        self.longest = max([n for _, n in self.seqs] + [1])
        q, k = (_rand(gen, *lead, H, dk, dt=dt, scale=dk ** -0.5) for _ in range(2))
        v, dO = (_rand(gen, *lead, H, dv, dt=dt) for _ in range(2))
        if tail:  # what stands behind the last sequence is never read
            for x in (q, k, v, dO):
                x[-tail:] = float("nan")
        self.g = _decays(H, gen, decays)
        self.S0 = _rand(gen, B, H, dk, dv, dt=torch.float32) if states else None
        self.dSf = _rand(gen, B, H, dk, dv, dt=torch.float32) if states else None
        self.host = [_np(x).reshape(-1, H, x.shape[-1]) for x in (q, k, v, dO)]
        if fused:  # token slices of one projection with a few columns more
            big = torch.full((*lead, H * (2 * dk + dv) + 8), float("nan"), dtype=dt, device="cuda")
            parts, at = [], 0
            for x, d in ((q, dk), (k, dk), (v, dv)):
                piece = big[..., at:at + H * d].unflatten(-1, (H, d))
                piece.copy_(x)
                parts.append(piece)
                at += H * d
            self.q, self.k, self.v = parts
        else:
            self.q, self.k, self.v = q.cuda(), k.cuda(), v.cuda()
        self.dO = dO.cuda()
        self.rows = np.concatenate([np.arange(f, f + n) for f, n in self.seqs]) if self.seqs else np.zeros(0, int)

    def call(self):
        kw = dict(scan_mode=self.mode, cu_seqlens=self.cu, scale=self.scale)
        if self.grid:
            kw.update(grid_h=self.grid[0], grid_w=self.grid[1])
        return kw

    def workspace(self, backward=False):
        return _dig().new_decay_attn_workspace(self.B, self.H, self.L, self.dk, self.dv, dtype=self.dtype, packed=self.packed,
                                               backward=backward)

    def fwd(self, o=None, S0=None, Sf=None, ws=None, **kw):
        o = torch.full(self.v.shape, 77.0, dtype=self.out_dtype, device="cuda") if o is None else o
        ws = self.workspace() if ws is None else ws
        _dig().dig_decay_attn_fwd(self.q, self.k, self.v, self.g.cuda(), o, ws, S0=S0, S_final=Sf, **self.call(), **kw)
        return o, ws

    def reference(self):
        q, k, v, _ = self.host
        S0 = None if self.S0 is None else _np(self.S0)
        args = (self.seqs, self.mode, self.grid, self.scale)
        o, S = ref.attn(q, k, v, self.g.numpy(), *args, S0)
        ob, Sb = ref.attn(np.abs(q), np.abs(k), np.abs(v), self.g.numpy(), *args[:3], abs(self.scale),
                          None if S0 is None else np.abs(S0))
        return o, S, ob, Sb

    def check_fwd(self):
        S0 = None if self.S0 is None else self.S0.cuda()
        Sf = torch.full((self.B, self.H, self.dk, self.dv), 55.0, device="cuda")
        o, ws = self.fwd(S0=S0, Sf=Sf)
        assert _dig().dig_read_status(ws) == _dig().DIG_OK
        want, S, size, Ssize = self.reference()
        o = o.reshape(-1, self.H, self.dv)
        r = self.rows
        _close(o[r], want[r], ref.attn_bound(size[r], self.longest, self.dk, self.dv, self.bf16), self.out_dtype, "o")
        # the state's products are exact to fp32 for every input type
        _close(Sf, S, ref.attn_bound(Ssize, self.longest, self.dk, self.dv, False), torch.float32, "S_final")
        rest = np.setdiff1d(np.arange(o.shape[0]), r)
        assert (o[rest] == 77.0).all()

    def check_bwd(self):
        out = self.out_dtype
        H = self.H
        dq, dk, dv = (torch.full(x.shape, 77.0, dtype=out, device="cuda") for x in (self.q, self.k, self.v))
        S0 = None if self.S0 is None else self.S0.cuda()
        dSf = None if self.dSf is None else self.dSf.cuda()
        dS0 = torch.full((self.B, H, self.dk, self.dv), 55.0, device="cuda")
        ws = self.workspace(backward=True)
        _dig().dig_decay_attn_bwd(self.q, self.k, self.v, self.g.cuda(), self.dO, dq, dk, dv, ws, S0=S0, dS_final=dSf, dS0=dS0,
                                  **self.call())
        assert _dig().dig_read_status(ws) == _dig().DIG_OK
        n = lambda x: None if x is None else _np(x)
        a = lambda x: None if x is None else np.abs(x)
        q, k, v, dO = self.host
        args = (self.seqs, self.mode, self.grid, self.scale, n(self.S0), n(self.dSf))
        want = ref.attn_bwd(q, k, v, self.g.numpy(), dO, *args)
        size = ref.attn_bwd(a(q), a(k), a(v), self.g.numpy(), a(dO), *args[:3], abs(self.scale), a(args[4]),
                            a(args[5]))
        r = self.rows
        for name, got, w, s in zip(("dq", "dk", "dv"), (dq, dk, dv), want, size):
            got = got.reshape(-1, H, got.shape[-1])
            _close(got[r], w[r], ref.attn_bound(s[r], self.longest, self.dk, self.dv, self.bf16), out, name)
            rest = np.setdiff1d(np.arange(got.shape[0]), r)
            assert (got[rest] == 77.0).all()
        _close(dS0, want[3], ref.attn_bound(size[3], self.longest, self.dk, self.dv, False), torch.float32, "dS0")


WHOLE = [
    dict(B=1, H=1, dk=64, dv=64, L=1), dict(B=3, H=2, dk=32, dv=64, L=2, states=True),
    dict(B=2, H=3, dk=36, dv=72, L=31), dict(B=2, H=2, dk=128, dv=128, L=127, states=True),
    dict(B=1, H=6, dk=128, dv=128, L=128, decays="edge", states=True), dict(B=2, H=6, dk=64, dv=64, L=129, decays="edge", mode=1),
    dict(B=1, H=2, dk=128, dv=128, L=1000, states=True), dict(B=1, H=6, dk=32, dv=64, L=700, decays="edge", states=True, mode=1),
    dict(B=2, H=2, dk=32, dv=64, grid=(13, 29), mode=2, states=True), dict(B=2, H=2, dk=36, dv=72, grid=(16, 17), mode=3, scale=0.3),
    dict(B=2, H=2, dk=4, dv=128, L=200, states=True, scale=-1.5), dict(B=2, H=1, dk=128, dv=4, L=257, states=True),
    dict(B=2, H=3, dk=100, dv=44, L=300, fused=True, states=True), dict(B=2, H=3, dk=64, dv=32, L=140, fused=True, mode=1),
    dict(B=2, H=2, dk=0x40, dv=64, L=0, states=True),
]
PACKED = [
    dict(B=1, H=2, dk=64, dv=64, lens=[1]), dict(B=5, H=2, dk=128, dv=128, lens=[130, 0, 1, 300, 64], tail=9, states=True),
    dict(B=4, H=3, dk=36, dv=72, lens=[0, 33, 0, 129], tail=3, mode=1, states=True),
    dict(B=3, H=6, dk=32, dv=64, lens=[5, 517, 128], decays="edge", states=True, fused=True),
    dict(B=40, H=1, dk=64, dv=64, lens=[(7 * i) % 50 for i in range(40)], tail=200, states=True),
    dict(B=2, H=1, dk=128, dv=128, lens=[0, 0], tail=5, states=True),
    dict(B=2, H=1, dk=128, dv=64, lens=[1100, 900], states=True, scale=0.5),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(WHOLE)))
def test_forward_whole_sequences(i, dtype):
    Case(dtype=dtype, seed=i, **WHOLE[i]).check_fwd()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(PACKED)))
def test_forward_packed_sequences(i, dtype):
    Case(dtype=dtype, seed=100 + i, **PACKED[i]).check_fwd()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(WHOLE)))
def test_backward_whole_sequences(i, dtype):
    Case(dtype=dtype, seed=200 + i, **WHOLE[i]).check_bwd()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(PACKED)))
def test_backward_packed_sequences(i, dtype):
    Case(dtype=dtype, seed=300 + i, **PACKED[i]).check_bwd()


@pytest.mark.parametrize("dtype, out", [("bf16", "f32"), ("f32", "bf16")])
def test_other_output_types(dtype, out):
    for kw in (dict(B=2, H=2, dk=32, dv=64, L=150), dict(B=1, H=2, dk=128, dv=96, L=200, states=True)):
        Case(dtype=dtype, out_dtype=out, seed=7, **kw).check_fwd()
        Case(dtype=dtype, out_dtype=out, seed=8, **kw).check_bwd()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_states_in_a_pool(dtype):
    """Sequences continue states of a pool in place; negative slots start from zero and leave nothing; a slot that does
    not exist or that an earlier sequence has is reported and taken as negative."""
    dig = _dig()
    lens = [200, 3, 0, 500, 17]
    c = Case(B=5, H=2, dk=64, dv=128, dtype=dtype, lens=lens, tail=2, seed=4)
    gen = torch.Generator().manual_seed(9)
    pool = torch.randn(9, 2, 64, 128, generator=gen)
    for slots, status in (([7, -1, 0, 3, 8], dig.DIG_OK), ([7, -3, 9, 3, 7], dig.DIG_ERR_INVALID_ARGUMENT)):
        kept, seen = [], set()
        for s in slots:
            kept.append(s if 0 <= s < 9 and s not in seen else -1)
            seen.add(s)
        c.S0 = torch.stack([pool[s] if s >= 0 else torch.zeros(2, 64, 128) for s in kept])
        P = pool.cuda()
        o, ws = c.fwd(S0=P, Sf=P, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        assert dig.dig_read_status(ws) == status
        want, S, size, Ssize = c.reference()
        r = c.rows
        _close(o[r], want[r], ref.attn_bound(size[r], c.longest, 64, 128, c.bf16), c.out_dtype, "o")
        for s in range(9):
            if s in kept:
                b = kept.index(s)
                _close(P[s], S[b], ref.attn_bound(Ssize[b], c.longest, 64, 128, False), torch.float32, "state %d" % s)
            else:
                assert torch.equal(P[s].cpu(), pool[s])


def test_bad_offsets_are_reported_and_stay_in_range():
    """Offsets outside the rows or descending: a status, nothing outside the tensors (checked on the CPU: every row comes
    from bounds clamped to 0 .. L and every segment beyond the grid is dropped)."""
    dig = _dig()
    c = Case(B=3, H=2, dk=64, dv=64, dtype="bf16", lens=[40, 50, 60], seed=2)
    for cu in ([0, 40, 30, 150], [-5, 40, 90, 150], [0, 40, 90, 4000]):
        c.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        _, ws = c.fwd()
        assert dig.dig_read_status(ws) == dig.DIG_ERR_INVALID_ARGUMENT
        assert dig.dig_read_status(ws) == dig.DIG_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segment_by_segment_equals_whole(dtype):
    """A sequence cut in two, the second half started from the first's state in place, against one call."""
    c = Case(B=1, H=3, dk=64, dv=64, dtype=dtype, L=333, states=True, out_dtype="f32", seed=21)
    want, S, size, Ssize = c.reference()
    P = c.S0.cuda()
    outs = []
    for a, b in ((0, 150), (150, 333)):
        half = Case(B=1, H=3, dk=64, dv=64, dtype=dtype, L=b - a, out_dtype="f32")
        half.g = c.g
        half.q, half.k, half.v = (x[:, a:b] for x in (c.q, c.k, c.v))
        outs.append(half.fwd(S0=P, Sf=P)[0])
    o = torch.cat(outs, 1).reshape(-1, 3, 64)
    _close(o, want, ref.attn_bound(size, 333, 64, 64, c.bf16), torch.float32, "o")
    _close(P, S, ref.attn_bound(Ssize, 333, 64, 64, False), torch.float32, "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_sequence_does_not_see_its_neighbours(dtype):
    """NaN and infinities in one sequence stay there, also where tiles cross the border between sequences."""
    lens = [70, 45, 200]
    c = Case(B=3, H=2, dk=64, dv=64, dtype=dtype, lens=lens, seed=31)
    o1, _ = c.fwd()
    bad = c.k.clone()
    c.k = bad
    c.v = c.v.clone()
    bad[70:115] = float("nan")
    c.v[70:115] = float("inf")
    o2, _ = c.fwd()
    assert torch.equal(o1[:70], o2[:70]) and torch.equal(o1[115:], o2[115:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_again_on_a_stream_and_in_a_graph(dtype):
    c = Case(B=2, H=3, dk=64, dv=64, dtype=dtype, L=900, states=True, seed=41)
    S0 = c.S0.cuda()
    Sf = torch.empty_like(S0)
    o, ws = c.fwd(S0=S0, Sf=Sf)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Sf2 = torch.empty_like(Sf)
    o2 = torch.empty_like(o)
    g, ws2 = c.g.cuda(), c.workspace()
    torch.cuda.synchronize()
    _dig().dig_decay_attn_fwd(c.q, c.k, c.v, g, o2, ws2, S0=S0, S_final=Sf2, stream=side, **c.call())
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(Sf, Sf2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _dig().dig_decay_attn_fwd(c.q, c.k, c.v, g, o2, ws2, S0=S0, S_final=Sf2, **c.call())
    for _ in range(3):
        o2.zero_()
        Sf2.zero_()
        graph.replay()
        assert torch.equal(o, o2) and torch.equal(Sf, Sf2)


# ------------------------------------------------------------------ single tokens
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B, H, dk, dv, fused", [(1, 1, 64, 64, False), (3, 6, 32, 64, True), (5, 4, 36, 72, False), (7, 2, 128, 128, True),
                                                 (2, 2, 256, 256, False), (2, 3, 4, 12, False), (300, 2, 8, 4, False), (3, 1, 252, 20, True)])
def test_single_tokens(B, H, dk, dv, fused, dtype):
    c = Case(B=B, H=H, dk=min(dk, 128), dv=min(dv, 128), dtype="f32", L=1, decays="edge" if H == 6 else "slopes")
    gen = torch.Generator().manual_seed(B)
    dt = DT[dtype]
    q, k, v = (_rand(gen, B, H, d, dt=dt) for d in (dk, dk, dv))
    S = torch.randn(B + 2, H, dk, dv, generator=gen)
    slots = torch.randperm(B + 2, generator=gen)[:B].to(torch.int32)
    if B > 2:
        slots[1] = -1                       # a padding row
    args = [x.cuda() for x in (q, k, v)]
    if fused:
        big = torch.zeros(B, H * (2 * dk + dv) + 4, dtype=dt, device="cuda")
        at, parts = 0, []
        for x, d in zip(args, (dk, dk, dv)):
            parts.append(big[:, at:at + H * d].unflatten(-1, (H, d)))
            parts[-1].copy_(x)
            at += H * d
        args = parts
    P = S.cuda()
    o = torch.full((B, H, dv), 77.0, dtype=dt, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _dig().dig_decay_attn_step(*args, c.g.cuda(), P, o, slots=slots.cuda(), scale=0.5, device_status=status)
    assert status.item() == 0
    lam = np.exp(c.g.double().numpy())[:, None, None]
    touched = set()
    for b in range(B):
        s = int(slots[b])
        if s < 0:
            assert (o[b] == 77.0).all()
            continue
        touched.add(s)
        kn, vn, qn = (_np(x[b]) for x in (k, v, q))
        kv = kn[:, :, None] * vn[:, None, :]
        want = lam * _np(S[s]) + kv
        size = lam * np.abs(_np(S[s])) + np.abs(kv)
        _close(P[s], want, 4 * ref.U32 * size, torch.float32, "state")   # lambda, two products, one sum
        ow = 0.5 * np.einsum("hk,hkv->hv", qn, want)
        ob = 0.5 * np.einsum("hk,hkv->hv", np.abs(qn), size)
        _close(o[b], ow, (dk + 8) * ref.U32 * ob, dt, "o")
    for s in set(range(B + 2)) - touched:
        assert torch.equal(P[s].cpu(), S[s])


def test_single_tokens_with_bad_slots():
    """A slot twice belongs to its first row; one that does not exist is left out; both are reported."""
    dig = _dig()
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(4, 2, 16, generator=gen).cuda() for _ in range(3))
    S = torch.randn(3, 2, 16, 16, generator=gen).cuda()
    g = torch.tensor([-0.1, -0.2]).cuda()
    want_S, want_o = S.clone(), torch.zeros(4, 2, 16, device="cuda")
    dig.dig_decay_attn_step(q[:1], k[:1], v[:1], g, want_S, want_o[:1], slots=torch.tensor([2], dtype=torch.int32, device="cuda"))
    o = torch.zeros(4, 2, 16, device="cuda")
    for slots in ([2, 2, -1, -1], [2, 3, -1, -1]):
        P = S.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        dig.dig_decay_attn_step(q, k, v, g, P, o, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"), device_status=status)
        assert status.item() == dig.DIG_ERR_INVALID_ARGUMENT
        assert torch.equal(P, want_S) and torch.equal(o, want_o)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_prompt_and_decoding_run_together(dtype):
    """Layer norm, prompt, then single tokens on the states that the prompt left, against the 64-bit recurrence over it all."""
    dig = _dig()
    dt = DT[dtype]
    lens, new, H, d = [130, 1, 57], 4, 2, 64
    gen = torch.Generator().manual_seed(77)
    B, L = len(lens), sum(lens)
    x = torch.randn(L + B * new, H * d, generator=gen).to(dt).cuda()
    y = torch.empty_like(x)
    dig.dig_layer_norm_fwd(x, y)
    qkv = y.view(-1, H, d)
    g = torch.tensor([-0.05, -0.4]).cuda()
    pool = torch.zeros(B + 1, H, d, d, device="cuda")
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 130, 131, 188], dtype=torch.int32, device="cuda")
    prompt = qkv[:L]
    o = torch.empty(L, H, d, dtype=dt, device="cuda")
    ws = dig.new_decay_attn_workspace(B, H, L, d, d, dtype=dt, packed=True)
    dig.dig_decay_attn_fwd(prompt, prompt, prompt, g, o, ws, cu_seqlens=cu, scale=d ** -0.5, S_final=pool, slots=slots)
    steps = []
    for t in range(new):
        z = qkv[L + t * B:L + (t + 1) * B].contiguous()
        ot = torch.empty(B, H, d, dtype=dt, device="cuda")
        dig.dig_decay_attn_step(z, z, z, g, pool, ot, slots=slots, scale=d ** -0.5)
        steps.append(ot)
    yn = _np(qkv)
    for b, (first, n) in enumerate(zip([0, 130, 131], lens)):
        rows = np.concatenate([yn[first:first + n], yn[L + b:L + B * new:B]])
        want, S = ref.attn(rows, rows, rows, _np(g), [(0, n + new)], scale=d ** -0.5)
        size, Ssize = ref.attn(abs(rows), abs(rows), abs(rows), _np(g), [(0, n + new)], scale=d ** -0.5)
        got = torch.cat([o[first:first + n]] + [s[b:b + 1] for s in steps])
        _close(got, want, ref.attn_bound(size, n + new, d, d, dtype == "bf16"), dt, "o")
        _close(pool[int(slots[b])], S[0], ref.attn_bound(Ssize[0], n + new, d, d, False), torch.float32, "state")
