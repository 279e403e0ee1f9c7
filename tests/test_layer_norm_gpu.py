"""Layer norm forward and backward on the GPU against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from tests import decay_reference as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.double().cpu().numpy()


def _inputs(rows, D, dtype, affine, seed=0, strided=0):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, D + strided, generator=gen) * 1.5 + torch.randn(rows, 1, generator=gen)).to(DT[dtype]).cuda()
    x = x[:, :D] if strided else x
    dy = torch.randn(rows, D, generator=gen).to(DT[dtype]).cuda()
    w = (1 + 0.2 * torch.randn(D, generator=gen)).cuda() if affine else None
    b = (0.2 * torch.randn(D, generator=gen)).cuda() if affine else None
    return x, dy, w, b


def _close(got, want, tol, what):
    got = _np(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d, worst %.3g of its bound" % (
        what, bad.sum(), bad.size, np.nanmax((np.abs(got - want) / (tol + 1e-300))[bad]))


SHAPES = [(1, 1), (3, 2), (5, 37), (2, 256), (9, 257), (7, 384), (33, 510), (4, 1024), (5, 1025), (6, 1152), (3, 2048), (2, 2056),
          (3, 4096), (2, 5000), (2, 8192), (3, 8193), (2, 10000), (700, 64), (1300, 384), (300, 2050)]


def _fwd(x, w, b, out, eps=1e-5):
    from gated_linear_attention_fwd_b200 import dig
    rows = x.shape[0]
    y = torch.full(x.shape, 77.0, dtype=out, device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dig.dig_layer_norm_fwd(x, y, weight=w, bias=b, eps=eps, mean=mean, rstd=rstd)
    return y, mean, rstd


@pytest.mark.parametrize("dtype, out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows, D", SHAPES)
def test_forward(rows, D, dtype, out):
    affine = (rows + D) % 3 != 0
    x, _, w, b = _inputs(rows, D, dtype, affine, seed=D, strided=8 if D % 5 == 0 else 0)
    y, mean, rstd = _fwd(x, w, b, DT[out])
    xn = _np(x)
    n = lambda t: None if t is None else _np(t)
    want, m, r = ref.layer_norm(xn, n(w), n(b), 1e-5)
    # sums of D fp32 terms: a chain of D roundings at most
    em = (D + 2) * ref.U32 * np.abs(xn).mean(1)
    _close(mean, m, em, "mean")
    # d = x - mean is off by em and a rounding; var by 2 |d| em on average (which sums to em^2 as sum(d) = 0, bounded here
    # without that) and by D + 4 roundings; rstd = var^-1/2 by half the relative error of var, and rsqrt by 2 steps
    dev = np.abs(xn - m[:, None])
    ed = em[:, None] + 2 * ref.U32 * dev
    evar = (2 * dev * ed + ed * ed).mean(1) + (D + 4) * ref.U32 / r ** 2
    er = np.minimum(0.5 * evar * r ** 3, r) + 4 * ref.U32 * r
    er = er * np.where(evar * r ** 2 < 0.25, 1.5, np.inf)   # the expansion holds for small relative errors only
    _close(rstd, r, er, "rstd")
    wn = 1.0 if w is None else np.abs(_np(w))
    tol = (ed * r[:, None] + dev * er[:, None]) * wn + 4 * ref.U32 * (np.abs(want) + (0 if b is None else np.abs(_np(b))) + dev * r[:, None] * wn)
    tol = tol + np.abs(want) * ref.UBF * 1.01 + 0.01 * tol if out == "bf16" else tol
    _close(y, want, tol, "y")


@pytest.mark.parametrize("dtype, out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows, D", SHAPES)
def test_backward(rows, D, dtype, out):
    from gated_linear_attention_fwd_b200 import dig
    affine = (rows + D) % 3 != 0
    x, dy, w, b = _inputs(rows, D, dtype, affine, seed=D + 1, strided=8 if D % 5 == 0 else 0)
    _, mean, rstd = _fwd(x, w, b, DT[out])
    dx = torch.full(x.shape, 77.0, dtype=DT[out], device="cuda")
    dw, db = torch.full((D,), 55.0, device="cuda"), torch.full((D,), 55.0, device="cuda")
    dig.dig_layer_norm_bwd(x, dy, mean, rstd, dx, weight=w, dw=dw, db=db, workspace=dig.new_layer_norm_workspace(rows, D))
    n = lambda t: None if t is None else _np(t)
    # the formulas on the same mean and rstd
    want, wdw, wdb = ref.layer_norm_bwd(_np(x), n(w), _np(mean), _np(rstd), _np(dy))
    r = _np(rstd)[:, None]
    xh = np.abs(_np(x) - _np(mean)[:, None]) * r
    a = np.abs(_np(dy)) * (1.0 if w is None else np.abs(_np(w)))
    size = r * (a + a.mean(1, keepdims=True) + xh * (a * xh).mean(1, keepdims=True))
    tol = (D + 8) * ref.U32 * size
    tol = tol + np.abs(want) * ref.UBF * 1.01 + 0.01 * tol if out == "bf16" else tol
    _close(dx, want, tol, "dx")
    _close(dw, wdw, (rows + 4) * ref.U32 * (np.abs(_np(dy)) * xh).sum(0), "dw")
    _close(db, wdb, (rows + 4) * ref.U32 * np.abs(_np(dy)).sum(0), "db")
    # the same bits again, and each of the gradients alone
    again, dx2 = torch.empty_like(dw), torch.empty_like(dx)
    ws = dig.new_layer_norm_workspace(rows, D).fill_(255)
    dig.dig_layer_norm_bwd(x, dy, mean, rstd, dx2, weight=w, dw=again, workspace=ws)
    assert torch.equal(dw, again) and torch.equal(dx, dx2)
    dig.dig_layer_norm_bwd(x, dy, mean, rstd, dx2, weight=w, db=again, workspace=ws)
    assert torch.equal(db, again)
    dx2.zero_()
    dig.dig_layer_norm_bwd(x, dy, mean, rstd, dx2, weight=w)
    assert torch.equal(dx, dx2)


def test_no_rows():
    from gated_linear_attention_fwd_b200 import dig
    x = torch.empty(0, 64, device="cuda")
    e = torch.empty(0, device="cuda")
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    dig.dig_layer_norm_fwd(x, torch.empty_like(x), mean=e, rstd=e)
    dig.dig_layer_norm_bwd(x, x, e, e, torch.empty_like(x), dw=dw, db=db, workspace=dig.new_layer_norm_workspace(0, 64))
    assert (dw == 0).all() and (db == 0).all()


def test_values_far_from_zero():
    """A large common offset: the variance is taken about the mean, so nothing is lost to cancellation."""
    gen = torch.Generator().manual_seed(0)
    x = (1000 + torch.randn(4, 512, generator=gen)).cuda()
    y, mean, rstd = _fwd(x, None, None, torch.float32)
    want, m, r = ref.layer_norm(_np(x), None, None, 1e-5)
    # x - mean: the mean is off by half a step of 1000 (2^-15) and less than 4 more from its sum; relative to a deviation of 1
    assert np.abs(_np(y) - want).max() < 2.0 ** -12
    assert np.abs(_np(rstd) / r - 1).max() < 2.0 ** -15


def test_captured_backward_is_replayed_with_new_inputs():
    from gated_linear_attention_fwd_b200 import dig
    x, dy, w, b = _inputs(600, 384, "bf16", True)
    _, mean, rstd = _fwd(x, w, b, torch.bfloat16)
    dx, dw, db = torch.empty_like(x), torch.empty(384, device="cuda"), torch.empty(384, device="cuda")
    ws = dig.new_layer_norm_workspace(600, 384)
    run = lambda: dig.dig_layer_norm_bwd(x, dy, mean, rstd, dx, weight=w, dw=dw, db=db, workspace=ws)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (3, 4):
        dy.copy_(_inputs(600, 384, "bf16", True, seed=seed)[1])
        run()
        want = [t.clone() for t in (dx, dw, db)]
        for t in (dx, dw, db):
            t.zero_()
        graph.replay()
        assert all(torch.equal(s, t) for s, t in zip(want, (dx, dw, db)))
