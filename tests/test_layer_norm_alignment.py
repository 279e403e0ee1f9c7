"""Layer norm on tensors that start where they happen to: refused only where rows are taken in 16-byte pieces."""
import pytest
import torch

from gated_linear_attention_fwd_b200 import dig

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def test_half_elements_are_refused():
    ok = dict(x=1024, xs=63, w=1024, b=1024, eps=1e-5, y=1024, mean=1024, rstd=1024, rows=4, D=63, dt=1, odt=0, st=None)
    for name, at in (("x", 1025), ("y", 1026), ("w", 1026), ("b", 1025), ("mean", 1026), ("rstd", 1027)):
        assert dig.lib.dig_layer_norm_fwd(*{**ok, name: at}.values()) == dig.DIG_ERR_MISALIGNED, name
    ok = dict(x=1024, xs=63, w=1024, mean=1024, rstd=1024, dy=1024, dx=1024, dw=1024, db=1024, rows=4, D=63, dt=1, odt=0,
              ws=1024, wsb=1 << 20, st=None)
    for name, at in (("x", 1025), ("dy", 1027), ("dx", 1026), ("w", 1026), ("mean", 1026), ("rstd", 1027), ("dw", 1026),
                     ("db", 1025), ("ws", 1028)):
        assert dig.lib.dig_layer_norm_bwd(*{**ok, name: at}.values()) == dig.DIG_ERR_MISALIGNED, name


def _off(t, by=1):
    """A copy of t that starts `by` elements into its storage."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    v = buf[by:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.gpu
@pytest.mark.parametrize("dtype, out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows, D", [(3, 1), (61, 37), (7, 1153), (5, 8198), (3, 10000)])
def test_tensors_that_start_anywhere(rows, D, dtype, out):
    """The same bits as of aligned tensors, forward and backward, with mean and rstd the halves of one tensor."""
    gen = torch.Generator().manual_seed(D)
    x, dy = (torch.randn(rows, D, generator=gen).to("cuda", DT[dtype]) for _ in range(2))
    w, b = (torch.randn(D, generator=gen).cuda() for _ in range(2))

    def run(put, stats):
        xs, dys, ws_, bs = put(x), put(dy), put(w), put(b)
        y, dx = (put(torch.zeros(rows, D, dtype=DT[out], device="cuda")) for _ in range(2))
        dw, db = (put(torch.zeros(D, device="cuda")) for _ in range(2))
        mean, rstd = stats[:rows], stats[rows:2 * rows]
        dig.dig_layer_norm_fwd(xs, y, weight=ws_, bias=bs, mean=mean, rstd=rstd)
        dig.dig_layer_norm_bwd(xs, dys, mean, rstd, dx, weight=ws_, dw=dw, db=db, workspace=dig.new_layer_norm_workspace(rows, D))
        return y, mean, rstd, dx, dw, db

    want = run(lambda t: t, torch.zeros(2 * rows, device="cuda"))
    for by in (1, 3):
        got = run(lambda t: _off(t, by), _off(torch.zeros(2 * rows, device="cuda"), by))
        assert all(torch.equal(a, c) for a, c in zip(got, want))


@pytest.mark.gpu
def test_statistics_and_weight_gradients_start_anywhere_at_full_vectors_too():
    rows, D = 61, 384
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(rows, D, generator=gen).cuda().bfloat16() for _ in range(2))
    res = []
    for by in (0, 1):
        stats = _off(torch.zeros(2 * rows, device="cuda"), by)
        grads = _off(torch.zeros(2 * D, device="cuda"), by)
        y, dx = torch.empty_like(x), torch.empty_like(x)
        dig.dig_layer_norm_fwd(x, y, mean=stats[:rows], rstd=stats[rows:])
        dig.dig_layer_norm_bwd(x, dy, stats[:rows], stats[rows:], dx, dw=grads[:D], db=grads[D:],
                               workspace=dig.new_layer_norm_workspace(rows, D))
        res.append((y, dx, stats.clone(), grads.clone()))
    assert all(torch.equal(a, c) for a, c in zip(*res))
    with pytest.raises(dig.DigError):
        dig.dig_layer_norm_fwd(_off(x), y)
