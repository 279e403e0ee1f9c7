"""Offsets of packed sequences that do not ascend, on the FP32 pipes: every access stays inside the workspace.

The kernels' index arithmetic is restated here (how long segments are, which slot of the workspace a segment's state
takes) and pinned to the library by the size of the workspace it asks for."""
import random

import pytest
import torch

from gated_linear_attention_fwd_b200 import dig

SMS, CHUNK, STATES_AT = 148, 32, 2048


def cut(B, H, L, dk, dv, nprob):
    """(tokens of a segment, segment slots, segment states, padded head dim) of a packed call."""
    D = 128 if max(dk, dv) > 64 else 64
    share = L * H * nprob // (2 * SMS * (2 if D == 128 else 3))
    seg = -(-min(max(share, 1), 1 << 30) // CHUNK) * CHUNK
    return seg, B + L // seg, min(B + L // seg, 2 * (L // seg)), D


def units(cu, L, seg, total):
    """(segment, first slot, first state, segments of its sequence) of each block's unit, over all slots."""
    base = states = 0
    for b in range(len(cu) - 1):
        lo = min(max(cu[b], 0), L)
        n = min(max(cu[b + 1], lo), L) - lo
        nseg = max(1, -(-n // seg))
        for i in range(nseg):
            if base + i < total:
                yield i, base, states, nseg
        base += nseg
        states += nseg if nseg > 1 else 0


def states_used(cu, L, seg, total, keep):
    """Segment states that some block writes or reads; keep(first slot, first state, nseg): whether a sequence is computed."""
    for i, first, state, nseg in units(cu, L, seg, total):
        if nseg > 1 and keep(first, state, nseg):
            yield state + nseg - 1        # the copy of S0
            yield from range(state, state + i)
            if i < nseg - 1:
                yield state + i


SHAPES = [(3, 2, 150, 64, 64), (256, 16, 16384, 128, 128), (40, 3, 2000, 64, 64), (3, 16, 16384, 128, 128), (4, 6, 3000, 32, 64), (9, 1, 5000, 100, 8)]


def offsets(B, L, rng):
    yield [0] + [L if b % 2 == 0 else 0 for b in range(B)]              # there and back again
    yield [L] * B + [0]
    yield [0] * B + [L]
    for _ in range(200):
        yield [rng.randint(-L // 4, L + L // 4) for _ in range(B + 1)]
    for _ in range(50):
        yield sorted(rng.randint(0, L) for _ in range(B + 1))
    for step in range(1, min(L, 1200)):    # alike lengths, just past a segment among them
        yield [min(b * step, L) for b in range(B + 1)]


@pytest.mark.parametrize("nprob", [1, 3])
@pytest.mark.parametrize("B, H, L, dk, dv", SHAPES)
def test_segment_states_stay_in_the_workspace(B, H, L, dk, dv, nprob):
    seg, total, kept, D = cut(B, H, L, dk, dv, nprob)
    floats = nprob * kept * H * D * D if L > seg else 0
    assert dig.lib.dig_decay_attn_workspace_bytes(B, H, L, dk, dv, dig.DIG_F32, 1, nprob == 3) == STATES_AT + 4 * floats
    fits = lambda first, state, nseg: first + nseg <= total and (nseg == 1 or state + nseg <= kept)
    past = False
    for cu in offsets(B, L, random.Random(B * L)):
        assert all(s < kept for s in states_used(cu, L, seg, total, fits))
        past |= any(s >= kept for s in states_used(cu, L, seg, total, lambda *_: True))
        if all(0 <= a <= b <= L for a, b in zip(cu, cu[1:])):           # nothing of a valid call is left out
            got = list(units(cu, L, seg, total))
            assert all(fits(*u[1:]) for u in got)
            assert len(got) == sum(max(1, -(-(b - a) // seg)) for a, b in zip(cu, cu[1:]))
    assert past    # without that rule some of these offsets do leave the workspace


@pytest.mark.gpu
@pytest.mark.parametrize("dtype, out", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("B, H, L, dk, dv", [(3, 2, 150, 64, 64), (4, 6, 3000, 32, 64), (3, 2, 700, 128, 72)])
def test_nothing_behind_the_workspace_is_written(B, H, L, dk, dv, dtype, out):
    """Both directions with offsets that descend: a status, and the bytes behind the workspace as they were."""
    DT = {"f32": torch.float32, "bf16": torch.bfloat16}
    gen = torch.Generator().manual_seed(L)
    rand = lambda *shape, dt=DT[dtype]: torch.randn(*shape, generator=gen).to("cuda", dt)
    q, k, v, dO = rand(L, H, dk), rand(L, H, dk), rand(L, H, dv), rand(L, H, dv)
    S0, dSf = rand(B, H, dk, dv, dt=torch.float32), rand(B, H, dk, dv, dt=torch.float32)
    g = torch.full((H,), -0.1, device="cuda")
    guard = 1 << 23
    for cu in ([0] + [L if b % 2 == 0 else 0 for b in range(B)], [0, L // 3, L // 4] + [L] * (B - 2), [L] * B + [0]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for backward in (False, True):
            n = dig.decay_attn_workspace_bytes(B, H, L, dk, dv, DT[dtype], True, backward)
            buf = torch.full((n + guard,), 0x5A, dtype=torch.uint8, device="cuda")
            ws = buf[:n].zero_()
            new = lambda x: torch.empty_like(x, dtype=DT[out])
            if backward:
                dig.dig_decay_attn_bwd(q, k, v, g, dO, new(q), new(k), new(v), ws, cu_seqlens=cu, S0=S0, dS_final=dSf,
                                       dS0=torch.empty_like(S0))
            else:
                dig.dig_decay_attn_fwd(q, k, v, g, new(v), ws, cu_seqlens=cu, S0=S0, S_final=torch.empty_like(S0))
            assert dig.dig_read_status(ws) == dig.DIG_ERR_INVALID_ARGUMENT
            assert (buf[n:] == 0x5A).all()


def test_many_short_sequences_do_not_pay_for_states():
    """256 sequences in 16384 rows, 16 heads of 128/128, bf16 in: 75 MB a problem at most, not one state each (306 MB)."""
    W = dig.lib.dig_decay_attn_workspace_bytes
    assert W(256, 16, 16384, 128, 128, dig.DIG_BF16, 1, 0) < 76e6
    assert W(1 << 16, 16, 1 << 16, 128, 128, dig.DIG_BF16, 1, 0) < 76e6
