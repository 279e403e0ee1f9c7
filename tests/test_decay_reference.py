"""The 64-bit references against the quadratic form and against differences."""
import numpy as np

from tests import decay_reference as ref


def _case(seed=3, B=2, n=9, H=2, dk=3, dv=4):
    r = np.random.default_rng(seed)
    q, k = r.standard_normal((2, B * n, H, dk))
    v, dO = r.standard_normal((2, B * n, H, dv))
    g = -np.abs(r.standard_normal(H))
    S0, dSf = r.standard_normal((2, B, H, dk, dv))
    return q, k, v, dO, g, S0, dSf, [(b * n, n) for b in range(B)]


def test_forward_is_the_masked_product():
    q, k, v, _, g, S0, _, seqs = _case()
    for mode, grid in ((0, None), (1, None), (2, (3, 3)), (3, (3, 3))):
        o, S = ref.attn(q, k, v, g, seqs, mode, grid, 0.5, S0)
        for b, (first, n) in enumerate(seqs):
            rows = first + ref.order(n, grid, mode)
            t = np.arange(n)
            D = np.where(t[:, None] >= t, np.exp(g[:, None, None] * (t[:, None] - t)), 0.0)
            P = np.einsum("thc,shc->hts", q[rows], k[rows]) * D
            want = np.einsum("hts,shj->thj", P, v[rows]) + np.einsum(
                "thc,hcj,th->thj", q[rows], S0[b], np.exp(g * (t[:, None] + 1)))
            np.testing.assert_allclose(o[rows], 0.5 * want, rtol=1e-11, atol=1e-11)


def test_backward_against_differences():
    q, k, v, dO, g, S0, dSf, seqs = _case(n=6)
    mode, grid, scale = 3, (2, 3), 0.7
    grads = ref.attn_bwd(q, k, v, g, dO, seqs, mode, grid, scale, S0, dSf)

    def loss():
        o, S = ref.attn(q, k, v, g, seqs, mode, grid, scale, S0)
        return (o * dO).sum() + (S * dSf).sum()
    for x, d in zip((q, k, v, S0), grads):
        for i in np.random.default_rng(1).integers(0, x.size, 12):
            e = 1e-5
            x.flat[i] += e
            up = loss()
            x.flat[i] -= 2 * e
            down = loss()
            x.flat[i] += e
            # the loss is linear in each input, so the difference is exact but for 64-bit rounding over 2e-5
            assert abs((up - down) / (2 * e) - d.flat[i]) < 1e-8 * max(1, abs(d.flat[i]))


def test_layer_norm_backward_against_differences():
    r = np.random.default_rng(5)
    x, dy = r.standard_normal((2, 4, 7))
    w, b = r.standard_normal((2, 7))
    _, mean, rstd = ref.layer_norm(x, w, b, 1e-3)
    dx, dw, db = ref.layer_norm_bwd(x, w, mean, rstd, dy)
    loss = lambda: (ref.layer_norm(x, w, b, 1e-3)[0] * dy).sum()
    for a, d in ((x, dx), (w, dw), (b, db)):
        for i in range(a.size):
            e = 1e-5
            a.flat[i] += e
            up = loss()
            a.flat[i] -= 2 * e
            down = loss()
            a.flat[i] += e
            # central differences: third-derivative term e^2 and 64-bit rounding over 2e, both below 1e-8 here
            assert abs((up - down) / (2 * e) - d.flat[i]) < 1e-7
