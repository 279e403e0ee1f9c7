"""Plain 64-bit references of the head-decay linear attention and of layer norm,
token by token from the definitions, with the bounds that rounding allows."""
import numpy as np

U32 = 2.0 ** -24   # half a step of fp32, relative
UBF = 2.0 ** -8    # half a step of bf16, relative


def order(n, grid, mode):
    """Rows of a sequence's scan positions."""
    if grid is None:
        r = np.arange(n)
    else:
        r = np.arange(n).reshape(grid)
        r = (r.T if mode & 2 else r).reshape(-1)
    return r[::-1] if mode & 1 else r


def attn(q, k, v, g, seqs, mode=0, grid=None, scale=1.0, S0=None):
    """q, k [rows, H, dk], v [rows, H, dv] float64; seqs: (first row, length) of each sequence; S0 [B, H, dk, dv].
    Returns o (NaN on rows of no sequence) and the final states."""
    H, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    lam = np.exp(np.asarray(g, np.float64))[:, None, None]
    o = np.full(v.shape, np.nan)
    states = np.zeros((len(seqs), H, dk, dv))
    for b, (first, n) in enumerate(seqs):
        S = np.zeros((H, dk, dv)) if S0 is None else S0[b].copy()
        for t in order(n, grid, mode):
            S = lam * S + k[first + t][:, :, None] * v[first + t][:, None, :]
            o[first + t] = scale * np.einsum("hk,hkv->hv", q[first + t], S)
        states[b] = S
    return o, states


def attn_bwd(q, k, v, g, dO, seqs, mode=0, grid=None, scale=1.0, S0=None, dSf=None):
    """Gradients (dq, dk, dv, dS0) of sum(o dO) + sum(S_final dSf)."""
    H, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    lam = np.exp(np.asarray(g, np.float64))[:, None, None]
    dq, dk_, dv_ = (np.full(x.shape, np.nan) for x in (q, k, v))
    dS0 = np.zeros((len(seqs), H, dk, dv))
    for b, (first, n) in enumerate(seqs):
        S = np.zeros((H, dk, dv)) if S0 is None else S0[b].copy()
        G = np.zeros((H, dk, dv)) if dSf is None else dSf[b].copy()
        seq = order(n, grid, mode)
        for t in seq:
            S = lam * S + k[first + t][:, :, None] * v[first + t][:, None, :]
            dq[first + t] = scale * np.einsum("hkv,hv->hk", S, dO[first + t])
        for t in seq[::-1]:
            G = G + scale * q[first + t][:, :, None] * dO[first + t][:, None, :]
            dk_[first + t] = np.einsum("hkv,hv->hk", G, v[first + t])
            dv_[first + t] = np.einsum("hk,hkv->hv", k[first + t], G)
            G = lam * G
        dS0[b] = G
    return dq, dk_, dv_, dS0


def attn_bound(size, longest, dk, dv, bf16):
    """Largest error of a sum that has sum(|terms|) = `size` (the reference run on absolute values).

    Every output is a sum of products q k v lambda^n.  A chain of at most dk + dv + 2 longest + 64 roundings of
    2^-23 at most (a tensor-core addition may cut instead of rounding; the decays cost a few more) leads to it.
    With bf16 inputs and outputs the state enters its product with q rounded to bf16, the way the output leaves: off by
    at most UBF.  The masked products and the decayed keys enter theirs as two bf16 terms, off by at most UBF^2 each."""
    c = (dk + dv + 2 * longest + 64) * 2 * U32
    return (c + (UBF + 3 * UBF * UBF if bf16 else 0.0)) * size


def layer_norm(x, w, b, eps):
    mean = x.mean(-1)
    var = ((x - mean[:, None]) ** 2).mean(-1)
    rstd = 1 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean, rstd


def layer_norm_bwd(x, w, mean, rstd, dy):
    xh = (x - mean[:, None]) * rstd[:, None]
    a = dy if w is None else dy * w
    dx = rstd[:, None] * (a - a.mean(-1, keepdims=True) - xh * (a * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
