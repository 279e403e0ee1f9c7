"""Layer norm backward on rows of one large value: what stands past the row's width takes no part in its sums."""
import numpy as np
import pytest
import torch

from tests import decay_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [1, 4, 16, 32, 64, 384, 1152, 3000, 5000, 5001, 8184])
def test_rows_of_one_large_value(D, dtype):
    """All values are 2^112, so that their sum (at most 2^125) and mean are exact (D times the rounded 1 / D is 1 in fp32
    for these D), x - mean is 0 and rstd eps^-1/2 = 2^20; mean times rstd is past fp32's range."""
    big, eps = 2.0 ** 112, 2.0 ** -40
    assert np.float32(D) * (np.float32(1) / np.float32(D)) == 1
    from gated_linear_attention_fwd_b200 import dig
    rows = 5
    gen = torch.Generator().manual_seed(D)
    x = torch.randn(rows, D, generator=gen)
    x[1:4] = big
    x, dy = x.to("cuda", dtype), torch.randn(rows, D, generator=gen).to("cuda", dtype)
    w = (1 + 0.2 * torch.randn(D, generator=gen)).cuda()
    y, dx = torch.empty(rows, D, device="cuda"), torch.empty(rows, D, device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    dig.dig_layer_norm_fwd(x, y, weight=w, eps=eps, mean=mean, rstd=rstd)
    assert (y[1:4] == 0).all() and (mean[1:4] == big).all()
    dig.dig_layer_norm_bwd(x, dy, mean, rstd, dx, weight=w, dw=dw, db=db, workspace=dig.new_layer_norm_workspace(rows, D))
    n = lambda t: t.double().cpu().numpy()
    want = ref.layer_norm_bwd(n(x), n(w), n(mean), n(rstd), n(dy))
    r = n(rstd)[:, None]
    xh = np.abs(n(x) - n(mean)[:, None]) * r
    a = np.abs(n(dy) * n(w))
    size = (r * (a + a.mean(1, keepdims=True) + xh * (a * xh).mean(1, keepdims=True)), (np.abs(n(dy)) * xh).sum(0),
            np.abs(n(dy)).sum(0))
    for got, v, s, terms in zip((dx, dw, db), want, size, (D + 8, rows + 4, rows + 4)):   # chains of that many roundings
        assert (np.abs(n(got) - v) <= terms * ref.U32 * s).all()
