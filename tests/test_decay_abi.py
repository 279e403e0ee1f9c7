"""Host-side refusals of the head-decay attention and layer norm entry points (no GPU)."""
import pytest
import torch

from gated_linear_attention_fwd_b200 import dig

N = None
INV, UNS, MIS, SMALL = (dig.DIG_ERR_INVALID_ARGUMENT, dig.DIG_ERR_UNSUPPORTED, dig.DIG_ERR_MISALIGNED,
                        dig.DIG_ERR_WORKSPACE_TOO_SMALL)


def _fwd(**kw):
    a = dict(q=1024, k=1024, v=1024, qs=64, ks=64, vs=128, g=1024, scale=1.0, cu=N, S0=N, Sf=N, slots=N, n=0, o=1024,
             B=1, H=2, L=12, dk=32, dv=64, gh=3, gw=4, mode=0, dt=1, odt=1, ws=4096, wsb=1 << 30, st=N)
    a.update(kw)
    return dig.lib.dig_decay_attn_fwd(*a.values())


def _bwd(**kw):
    a = dict(q=1024, k=1024, v=1024, qs=64, ks=64, vs=128, g=1024, scale=1.0, cu=N, S0=N, dO=1024, dSf=N, dq=1024,
             dk_=1024, dv_=1024, dS0=N, B=1, H=2, L=12, dk=32, dv=64, gh=3, gw=4, mode=0, dt=1, odt=1, ws=4096,
             wsb=1 << 30, st=N)
    a.update(kw)
    return dig.lib.dig_decay_attn_bwd(*a.values())


COMMON = [
    (dict(L=13), INV), (dict(B=-1), INV), (dict(H=0), INV), (dict(dk=0), INV), (dict(mode=4), INV), (dict(mode=-1), INV),
    (dict(cu=1024, mode=2), INV),                       # packed sequences are lines
    (dict(dt=2), INV), (dict(odt=-1), INV), (dict(dk=30), UNS), (dict(dv=132, vs=264), UNS),
    (dict(qs=60), INV), (dict(vs=64), INV), (dict(ks=66), UNS), (dict(g=N), INV), (dict(ws=N), INV), (dict(q=N), INV),
    (dict(q=1028), MIS), (dict(q=1032, dt=0), MIS), (dict(ws=4100), MIS), (dict(wsb=16), SMALL), (dict(S0=1028), MIS),
    (dict(B=1 << 20, L=1 << 20, gh=1 << 10, gw=1 << 10), INV), (dict(H=70000, qs=70000 * 32, ks=70000 * 32, vs=70000 * 64), INV),
]


@pytest.mark.parametrize("kw, code", COMMON)
def test_both_directions_refuse(kw, code):
    assert _fwd(**kw) == code and dig.lib.dig_last_error()
    assert _bwd(**kw) == code and dig.lib.dig_last_error()


def test_each_direction_refuses():
    assert _fwd(o=N) == INV
    assert _fwd(o=1028) == MIS
    assert _fwd(slots=1024, n=-1) == INV
    for name in ("dO", "dq", "dk_", "dv_"):
        assert _bwd(**{name: N}) == INV
        assert _bwd(**{name: 1028}) == MIS
    assert _bwd(dS0=1032) == MIS
    assert _fwd(B=0) == dig.DIG_OK and _bwd(B=0) == dig.DIG_OK


def test_step_refuses():
    def step(**kw):
        a = dict(q=1024, k=1024, v=1024, qs=64, ks=64, vs=128, g=1024, scale=1.0, S=1024, slots=N, n=3, o=1024, B=3, H=2,
                 dk=32, dv=64, dt=1, odt=1, status=N, st=N)
        a.update(kw)
        return dig.lib.dig_decay_attn_step(*a.values())
    assert step(B=0) == dig.DIG_OK
    for kw, code in [(dict(B=-1), INV), (dict(H=0), INV), (dict(dk=34), UNS), (dict(dv=260, vs=520), UNS), (dict(dt=5), INV),
                     (dict(qs=32), INV), (dict(vs=130), UNS), (dict(n=2), INV), (dict(S=N), INV), (dict(o=N), INV),
                     (dict(k=1028), MIS), (dict(k=1032, dt=0), MIS), (dict(S=1032), MIS), (dict(o=1032), MIS), (dict(g=N), INV), (dict(n=-1, slots=1024), INV)]:
        assert step(**kw) == code, kw


def test_layer_norm_refuses():
    def fwd(**kw):
        a = dict(x=1024, xs=64, w=N, b=N, eps=1e-5, y=1024, mean=N, rstd=N, rows=4, D=64, dt=1, odt=1, st=N)
        a.update(kw)
        return dig.lib.dig_layer_norm_fwd(*a.values())

    def bwd(**kw):
        a = dict(x=1024, xs=64, w=N, mean=1024, rstd=1024, dy=1024, dx=1024, dw=N, db=N, rows=4, D=64, dt=1, odt=1, ws=N,
                 wsb=0, st=N)
        a.update(kw)
        return dig.lib.dig_layer_norm_bwd(*a.values())
    for f in (fwd, bwd):
        for kw, code in [(dict(rows=-1), INV), (dict(D=0), INV), (dict(xs=63), INV), (dict(dt=3), INV), (dict(odt=2), INV),
                         (dict(x=N), INV), (dict(x=1032), MIS), (dict(w=1028), MIS), (dict(rows=1 << 40), INV)]:
            assert f(**kw) == code, kw
    assert fwd(eps=-1.0) == INV and fwd(eps=float("nan")) == INV and fwd(y=N) == INV
    assert fwd(rows=0) == dig.DIG_OK
    assert bwd(dw=1024) == INV                               # no workspace
    assert bwd(db=1024, ws=1024, wsb=64) == SMALL
    assert bwd(mean=N) == INV and bwd(dx=N) == INV and bwd(ws=1028, dw=1024, wsb=1 << 30) == MIS


def test_workspace_bytes():
    W = dig.lib.dig_decay_attn_workspace_bytes
    assert W(1, 2, 12, 32, 64, 1, 0, 0) >= 256
    assert W(1, 1, 1 << 16, 128, 128, 1, 0, 1) >= W(1, 1, 1 << 16, 128, 128, 1, 0, 0) > 256   # segments
    assert W(0, 1, 0, 4, 4, 0, 1, 0) >= 256
    for bad in [(1, 0, 1, 32, 64, 1, 0, 0), (1, 1, 1, 33, 64, 1, 0, 0), (1, 1, 1, 32, 64, 7, 0, 0), (1, 1, 1, 32, 64, 1, 0, 2)]:
        assert W(*bad) == 0
    assert dig.lib.dig_layer_norm_workspace_bytes(10, 64) == 10 * 64 * 8
    assert dig.lib.dig_layer_norm_workspace_bytes(-1, 64) == 0


def test_binding_refuses_tensors_of_the_wrong_form():
    x = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):        # not on a GPU
        dig.dig_decay_attn_step(x, x, x, torch.zeros(2), torch.zeros(4, 2, 8, 8), torch.zeros(4, 2, 8))
    with pytest.raises(ValueError):        # k of another shape
        dig.dig_decay_attn_step(x, x[:3], x, torch.zeros(2), torch.zeros(4, 2, 8, 8), torch.zeros(4, 2, 8))
    with pytest.raises(ValueError):        # packed tensors have no batch dimension
        dig.dig_decay_attn_fwd(x[None], x[None], x[None], torch.zeros(2), x[None], torch.zeros(256, dtype=torch.uint8),
                               cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        dig.dig_layer_norm_fwd(torch.zeros(3, 8), torch.zeros(3, 8))
    assert dig._tokens(torch.zeros(5, 3, 2, 8)[:, :, :], "q", 2, 8) == 16
    fused = torch.zeros(5, 3, 6, 8)
    assert dig._tokens(fused[:, :, 2:4], "k", 2, 8) == 48
    with pytest.raises(ValueError):        # heads of one token are not dense
        dig._tokens(fused[:, :, ::2][:, :, :2], "k", 2, 8)
    with pytest.raises(ValueError):        # rows are not one stride apart
        dig._tokens(torch.zeros(5, 4, 2, 8)[:, :3], "q", 2, 8)
