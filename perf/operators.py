"""Measured cases of the head-decay linear attention (prompt form, single-token
form, backward) and of layer norm (forward, backward).

`run` computes an operator either in its plain form (elementary torch operations
in 32 bits) or, with `own` set, by the library's entry points.  Sizes are those of
the DiG workloads (DiG-S/2: 6 heads of 32/64, D = 384; DiG-XL/2: 16 heads of 36/72,
D = 1152) and generic language-model ones (16 heads of 128/128).
"""
import math

import torch

own = False

DEV = "cuda"

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 64


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a DiG-S/2 layer at 1792^2 (112 x 112 tokens), scanned down the columns
        dict(name="attn_fwd_dig_s2_1792", op="attn_fwd", B=2, H=6, grid_h=112, grid_w=112, mode=2, dk=32, dv=64,
             dtype="bf16", packed=False, tail=0, pool=0),
        # prompts of different lengths packed together, each continuing the state in its slot of a pool
        dict(name="attn_fwd_prompts", op="attn_fwd", B=7, H=16, grid_h=1, grid_w=16411, mode=0, dk=128, dv=128,
             dtype="bf16", packed=True, tail=29, pool=12),
        # the fp32 path at the 64/64 head dims of the smallest workload
        dict(name="attn_fwd_fp32", op="attn_fwd", B=8, H=6, grid_h=16, grid_w=16, mode=1, dk=64, dv=64, dtype="f32",
             packed=False, tail=0, pool=0),
        # one sequence decoding on its own: latency
        dict(name="attn_step_one", op="attn_step", B=1, H=6, dk=32, dv=64, dtype="bf16", pool=0),
        # a large decoding batch over a pool of states
        dict(name="attn_step_batch", op="attn_step", B=253, H=16, dk=128, dv=128, dtype="bf16", pool=256),
        # training a DiG-S/2 layer at 1024^2
        dict(name="attn_bwd_dig_s2_1024", op="attn_bwd", B=4, H=6, grid_h=64, grid_w=64, mode=3, dk=32, dv=64,
             dtype="bf16", states=False),
        # training on long segments with the state carried from segment to segment
        dict(name="attn_bwd_long", op="attn_bwd", B=4, H=16, grid_h=1, grid_w=4096, mode=0, dk=128, dv=128,
             dtype="bf16", states=True),
        # norms of a DiG-S/2 block at 1792^2
        dict(name="ln_fwd_dig_s2_1792", op="ln_fwd", rows=25088, D=384, dtype="bf16", affine=True),
        # a few rows of a decoding step
        dict(name="ln_fwd_rows_fp32", op="ln_fwd", rows=61, D=1152, dtype="f32", affine=True),
        # a long wide batch
        dict(name="ln_fwd_wide", op="ln_fwd", rows=16384, D=4096, dtype="bf16", affine=True),
        dict(name="ln_bwd_dig_s2_1792", op="ln_bwd", rows=25088, D=384, dtype="bf16", affine=True),
        dict(name="ln_bwd_wide_fp32", op="ln_bwd", rows=8191, D=4096, dtype="f32", affine=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_step", "attn_bwd", "attn_bwd", "ln_fwd", "ln_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("ln_fwd", "ln_bwd"):
        D = _log_int(rng, 33, 8192) if rng.random() < 0.5 else 8 * _log_int(rng, 8, 1024)
        return dict(op=op, rows=_log_int(rng, 1, (32 << 20) // D), D=D, dtype=dtype, affine=rng.random() < 0.8)
    dk, dv = rng.choice([(32, 64), (36, 72), (64, 64), (128, 128), (128, 128), (96, 80), (4 * rng.randint(4, 32), 4 * rng.randint(4, 32))])
    H = rng.choice([1, 3, 6, 8, 16])
    if op == "attn_step":
        B = _log_int(rng, 1, 256)
        return dict(op=op, B=B, H=H, dk=dk, dv=dv, dtype=dtype, pool=rng.choice([0, B, B + rng.randint(1, 9)]))
    top = (16384 if op == "attn_fwd" else 8192) // (1 if dtype == "bf16" else 4)  # tokens of the whole call at 16 heads
    tokens = _log_int(rng, 1, top * 16 // H if H > 4 else top * 4)
    B = rng.randint(1, max(1, min(8, tokens // 16)))
    if op == "attn_fwd" and rng.random() < 0.5:
        T = max(B, tokens)
        tail = rng.choice([0, rng.randint(1, 40)])
        return dict(op=op, B=B, H=H, grid_h=1, grid_w=T + tail, mode=rng.choice([0, 0, 1]), dk=dk, dv=dv, dtype=dtype,
                    packed=True, tail=tail, pool=rng.choice([0, B, B + rng.randint(1, 9)]))
    L = max(1, tokens // B)
    grid_h = rng.randint(1, max(1, int(math.isqrt(L))))
    c = dict(op=op, B=B, H=H, grid_h=grid_h, grid_w=max(1, L // grid_h), mode=rng.randint(0, 3), dk=dk, dv=dv, dtype=dtype)
    c.update(dict(packed=False, tail=0, pool=0) if op == "attn_fwd" else dict(states=rng.random() < 0.5))
    return c


# ------------------------------------------------------------------ inputs
def _lengths(c):
    """Lengths of a packed call's sequences: uneven, summing to the rows before the tail."""
    T, B = c["grid_w"] - c["tail"], c["B"]
    w = [1 + (i * 7 + 3) % 11 for i in range(B)]
    n = [T * x // sum(w) for x in w]
    n[-1] += T - sum(n)
    return n


def _decays(H, gen):
    """Log decays from about -0.7 to -0.004, as slopes halving over the heads, with a little of the seed in them."""
    h = torch.arange(1, H + 1, dtype=torch.float32, device=DEV)
    jitter = 1 + 0.1 * torch.rand(H, device=DEV, generator=gen)
    return -torch.exp2(-8 * h / H) * jitter


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DT[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, device=DEV, generator=gen) * scale).to(dtype)

    if c["op"] in ("ln_fwd", "ln_bwd"):
        R, D = c["rows"], c["D"]
        x = torch.randn(R, D, device=DEV, generator=gen)
        x = (x * (0.5 + torch.rand(R, 1, device=DEV, generator=gen)) + torch.randn(R, 1, device=DEV, generator=gen)).to(dt)
        s = dict(c, x=x, eps=1e-5, w=None, b=None)
        if c["affine"]:
            s["w"] = 1 + 0.1 * torch.randn(D, device=DEV, generator=gen)
            s["b"] = 0.1 * torch.randn(D, device=DEV, generator=gen)
        if c["op"] == "ln_fwd":
            s.update(y=torch.empty_like(x), mean=torch.empty(R, device=DEV), rstd=torch.empty(R, device=DEV))
        else:
            xf = x.double()
            mean = xf.mean(1)
            rstd = torch.rsqrt(xf.var(1, unbiased=False) + s["eps"])
            s.update(dy=normal(R, D), mean=mean.float(), rstd=rstd.float(), dx=torch.empty_like(x),
                     dw=torch.empty(D, device=DEV), db=torch.empty(D, device=DEV))
            if own:
                from gated_linear_attention_fwd_b200 import dig
                s["ws"] = dig.new_layer_norm_workspace(R, D)
        return s

    B, H, dk, dv = c["B"], c["H"], c["dk"], c["dv"]
    if c["op"] == "attn_step":
        s = dict(c, q=normal(B, H, dk, scale=dk ** -0.5), k=normal(B, H, dk, scale=dk ** -0.5), v=normal(B, H, dv),
                 g=_decays(H, gen), o=torch.empty(B, H, dv, device=DEV, dtype=dt), slots=None)
        s["S"] = torch.randn(c["pool"] or B, H, dk, dv, device=DEV, generator=gen)
        if c["pool"]:
            s["slots"] = torch.randperm(c["pool"], device=DEV, generator=gen)[:B].to(torch.int32)
        return s

    L = c["grid_h"] * c["grid_w"]
    lead = (L,) if c.get("packed") else (B, L)
    s = dict(c, q=normal(*lead, H, dk, scale=dk ** -0.5), k=normal(*lead, H, dk, scale=dk ** -0.5), v=normal(*lead, H, dv),
             g=_decays(H, gen), S0=None, Sf=None, slots=None, cu=None)
    if c["op"] == "attn_fwd":
        s["o"] = torch.zeros(*lead, H, dv, device=DEV, dtype=dt)
        s["lens"] = _lengths(c) if c["packed"] else [L] * B
        if c["packed"]:
            ends = torch.tensor([0] + s["lens"]).cumsum(0)
            s["cu"] = ends.to(DEV, torch.int32)
        if c["pool"]:  # the states are continued in place
            s["S0"] = s["Sf"] = torch.randn(c["pool"], H, dk, dv, device=DEV, generator=gen)
            s["slots"] = torch.randperm(c["pool"], device=DEV, generator=gen)[:B].to(torch.int32)
    else:
        s["dO"] = normal(*lead, H, dv)
        s.update(dq=torch.empty_like(s["q"]), dk_=torch.empty_like(s["k"]), dv_=torch.empty_like(s["v"]), dSf=None, dS0=None)
        if c["states"]:
            s["S0"] = torch.randn(B, H, dk, dv, device=DEV, generator=gen)
            s["dSf"] = torch.randn(B, H, dk, dv, device=DEV, generator=gen)
            s["dS0"] = torch.empty(B, H, dk, dv, device=DEV)
    if own:
        from gated_linear_attention_fwd_b200 import dig
        s["ws"] = dig.new_decay_attn_workspace(B, H, L, dk, dv, dtype=dt, packed=bool(c.get("packed")),
                                               backward=c["op"] == "attn_bwd")
    return s


# ------------------------------------------------------------------ plain forms
def _rows(s, mode):
    """[B, longest] token row of each scan position of each sequence, and whether the position is in the sequence."""
    dev = s["q"].device
    if s.get("packed"):
        n = (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
        t = torch.arange(max(s["lens"]), device=dev)[None, :]
        inside = t < n
        at = torch.where(inside, n - 1 - t, t) if mode & 1 else t
        return torch.where(inside, s["cu"][:-1].long()[:, None] + at, 0), inside
    Hg, Wg = s["grid_h"], s["grid_w"]
    L = Hg * Wg
    t = torch.arange(L, device=dev)
    t = L - 1 - t if mode & 1 else t
    t = (t % Hg) * Wg + t // Hg if mode & 2 else t
    rows = torch.arange(s["B"], device=dev)[:, None] * L + t[None, :]
    return rows, torch.ones_like(rows, dtype=torch.bool)


def _scan(q, k, v, g, inside, S0, lag, want_state):
    """o_t = lambda^(t+1-lag) q_t S0 + sum_{s<=t} lambda^(t-s) (q_t . k_s) v_s over positions [B, n, H, d] (chunked), and the
    state after each sequence's last position times lambda^lag."""
    B, n, H, dk = q.shape
    dv = v.shape[3]
    C = CHUNK
    nc = -(-n // C)
    inside = inside[:, :, None, None]
    pad = (0, 0, 0, 0, 0, nc * C - n)
    zero = torch.zeros((), device=q.device)

    def chunks(x):
        x = torch.nn.functional.pad(torch.where(inside, x.float(), zero), pad)
        return x.view(B, nc, C, H, x.shape[3]).permute(0, 3, 1, 2, 4)  # [B, H, nc, C, d]

    qc, kc, vc = chunks(q), chunks(k), chunks(v)
    gd = g.double()
    i = torch.arange(C, device=q.device)
    d = (i[:, None] - i[None, :]).double()
    D = torch.where(d >= 0, torch.exp(d.clamp(min=0) * gd[:, None, None]), 0.0).float()  # [H, C, C]
    o = (torch.matmul(qc, kc.transpose(-1, -2)) * D[None, :, None]) @ vc
    dS = (kc * torch.exp((C - 1 - i).double() * gd[:, None]).float()[None, :, None, :, None]).transpose(-1, -2) @ vc
    m = torch.arange(nc, device=q.device)
    e = (m[:, None] - 1 - m[None, :]).double() * C  # chunk m' enters chunk m
    E = torch.where(e >= 0, torch.exp(e.clamp(min=0) * gd[:, None, None]), 0.0).float()  # [H, nc, nc]
    S = (E[None] @ dS.reshape(B, H, nc, dk * dv)).view(B, H, nc, dk, dv)
    qd = qc * torch.exp((i + 1).double() * gd[:, None]).float()[None, :, None, :, None]
    o = o + qd @ S
    if S0 is not None:
        t = (torch.arange(nc * C, device=q.device) + 1 - lag).double()
        w = torch.exp(t * gd[:, None]).float().view(1, H, nc, C, 1)
        o = o + (qc * w) @ S0[:, :, None]
    o = o.permute(0, 2, 3, 1, 4).reshape(B, nc * C, H, dv)[:, :n]
    if not want_state:
        return o, None
    count = inside[..., 0, 0].sum(1)
    left = (count[:, None] - 1 - torch.arange(n, device=q.device)[None, :] + lag).clamp(min=0).double()
    w = torch.exp(left[:, :, None] * gd[None, None, :]).float()[..., None]
    kw = torch.where(inside, k.float() * w, zero)
    St = torch.einsum("bnhk,bnhv->bhkv", kw, torch.where(inside, v.float(), zero))
    if S0 is not None:
        St = St + torch.exp(count[:, None].double() * gd[None, :]).float()[..., None, None] * S0
    return o, St


def _plain_attn_fwd(s):
    rows, inside = _rows(s, s["mode"])
    q, k, v = (s[n].reshape(-1, s["H"], s[n].shape[-1])[rows] for n in ("q", "k", "v"))
    slots = s["slots"].long() if s["slots"] is not None else None
    S0 = s["S0"][slots] if slots is not None else None
    o, S = _scan(q, k, v, s["g"], inside, S0, 0, slots is not None)
    out = s["o"].view(-1, s["H"], s["dv"])
    out[rows[inside]] = o[inside].to(out.dtype)
    if slots is not None:
        s["Sf"][slots] = S
        return {"o": s["o"], "state": s["Sf"]}
    return {"o": s["o"]}


def _plain_attn_bwd(s):
    H = s["H"]
    names = ("q", "k", "v", "dO")
    rows, inside = _rows(s, s["mode"])
    q, k, v, dO = (s[n].reshape(-1, H, s[n].shape[-1])[rows] for n in names)
    S0t = s["S0"].transpose(-1, -2) if s["states"] else None
    dq, _ = _scan(dO, v, k, s["g"], inside, S0t, 0, False)
    back, inside_b = _rows(s, s["mode"] ^ 1)
    qb, kb, vb, dOb = (s[n].reshape(-1, H, s[n].shape[-1])[back] for n in names)
    Sf = s["dSf"]
    dv, dS0 = _scan(kb, qb, dOb, s["g"], inside_b, Sf, 1, s["states"])
    dk, _ = _scan(vb, dOb, qb, s["g"], inside_b, Sf.transpose(-1, -2) if s["states"] else None, 1, False)
    out = {}
    for name, x, r in (("dq", dq, rows), ("dk", dk, back), ("dv", dv, back)):
        y = torch.empty(r.numel(), H, x.shape[-1], device=x.device, dtype=s["q"].dtype)
        y[r.reshape(-1)] = x.reshape(r.numel(), H, -1).to(y.dtype)
        out[name] = y
    if s["states"]:
        out["dS0"] = dS0
    return out


def _plain_attn_step(s):
    slots = s["slots"].long() if s["slots"] is not None else torch.arange(s["B"], device=s["q"].device)
    lam = torch.exp(s["g"])[None, :, None, None]
    S = lam * s["S"][slots] + s["k"].float()[..., :, None] * s["v"].float()[..., None, :]
    s["S"][slots] = S
    o = (s["q"].float()[..., None, :] @ S)[..., 0, :]
    return {"o": o.to(s["q"].dtype), "state": s["S"]}


def _plain_ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + s["eps"])
    y = xc * rstd
    if s["affine"]:
        y = y * s["w"] + s["b"]
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_ln_bwd(s):
    dy = s["dy"].float()
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    a = dy * s["w"] if s["affine"] else dy
    dx = s["rstd"][:, None] * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    out = {"dx": dx.to(s["x"].dtype)}
    if s["affine"]:
        out.update(dw=(dy * xh).sum(0), db=dy.sum(0))
    return out


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["op"]
    if not own:
        return {"attn_fwd": _plain_attn_fwd, "attn_bwd": _plain_attn_bwd, "attn_step": _plain_attn_step,
                "ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd}[op](s)
    from gated_linear_attention_fwd_b200 import dig
    if op == "attn_fwd":
        dig.dig_decay_attn_fwd(s["q"], s["k"], s["v"], s["g"], s["o"], s["ws"], grid_h=s["grid_h"], grid_w=s["grid_w"],
                               scan_mode=s["mode"], cu_seqlens=s["cu"], S0=s["S0"], S_final=s["Sf"], slots=s["slots"])
        return {"o": s["o"], "state": s["Sf"]} if s["slots"] is not None else {"o": s["o"]}
    if op == "attn_step":
        dig.dig_decay_attn_step(s["q"], s["k"], s["v"], s["g"], s["S"], s["o"], slots=s["slots"])
        return {"o": s["o"], "state": s["S"]}
    if op == "attn_bwd":
        dig.dig_decay_attn_bwd(s["q"], s["k"], s["v"], s["g"], s["dO"], s["dq"], s["dk_"], s["dv_"], s["ws"],
                               grid_h=s["grid_h"], grid_w=s["grid_w"], scan_mode=s["mode"], S0=s["S0"],
                               dS_final=s["dSf"], dS0=s["dS0"])
        H = s["H"]
        out = {"dq": s["dq"].view(-1, H, s["dk"]), "dk": s["dk_"].view(-1, H, s["dk"]), "dv": s["dv_"].view(-1, H, s["dv"])}
        if s["states"]:
            out["dS0"] = s["dS0"]
        return out
    if op == "ln_fwd":
        dig.dig_layer_norm_fwd(s["x"], s["y"], weight=s["w"], bias=s["b"], eps=s["eps"], mean=s["mean"], rstd=s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    affine = s["affine"]
    dig.dig_layer_norm_bwd(s["x"], s["dy"], s["mean"], s["rstd"], s["dx"], weight=s["w"], dw=s["dw"] if affine else None,
                           db=s["db"] if affine else None, workspace=s["ws"])
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]} if affine else {"dx": s["dx"]}


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("ln_fwd", "ln_bwd"):
        n = c["rows"] * c["D"]
        par = 8 * c["D"] if c["affine"] else 0
        if c["op"] == "ln_fwd":
            return {"bytes": 2 * n * es + 8 * c["rows"] + par, "flops": 8 * n}
        return {"bytes": 3 * n * es + 8 * c["rows"] + par * 3 // 2, "flops": 14 * n}
    dk, dv, H, B = c["dk"], c["dv"], c["H"], c["B"]
    state = 4 * dk * dv * H * B
    if c["op"] == "attn_step":
        return {"bytes": 2 * state + B * H * (2 * dk + 2 * dv) * es, "flops": 5 * B * H * dk * dv}
    tokens = c["grid_w"] - c["tail"] if c.get("packed") else B * c["grid_h"] * c["grid_w"]
    if c["op"] == "attn_fwd":
        return {"bytes": tokens * H * (2 * dk + 2 * dv) * es + (2 * state if c["pool"] else 0), "flops": 4 * tokens * H * dk * dv}
    return {"bytes": tokens * H * (4 * dk + 3 * dv) * es + (3 * state if c["states"] else 0), "flops": 10 * tokens * H * dk * dv}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("ln_fwd", "ln_bwd"):
        x, D = s["x"].double(), s["D"]
        w = s["w"].double() if s["affine"] else torch.ones(D, device=DEV, dtype=torch.float64)
        if op == "ln_fwd":
            mu = x.sum(1) / D
            var = (x * x).sum(1) / D - mu * mu
            r = 1 / torch.sqrt(var + s["eps"])
            y = (x - mu[:, None]) / torch.sqrt(var + s["eps"])[:, None] * w
            return {"y": y + s["b"].double() if s["affine"] else y, "mean": mu, "rstd": r}
        dy, mu, r = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
        p = dy * w
        c1 = p.sum(1, keepdim=True)
        c2 = (p * (x - mu)).sum(1, keepdim=True)
        out = {"dx": r * p - r / D * c1 - r ** 3 / D * (x - mu) * c2}
        if s["affine"]:
            out["dw"] = ((x - mu) * r * dy).sum(0)
            out["db"] = dy.sum(0)
        return out
    H, dk, dv = s["H"], s["dk"], s["dv"]
    lam = torch.exp(s["g"].double())[:, None, None]
    if op == "attn_step":
        S = s["S"].double()
        o = torch.empty(s["B"], H, dv, device=DEV, dtype=torch.float64)
        where = s["slots"].tolist() if s["slots"] is not None else range(s["B"])
        for n, j in enumerate(where):
            S[j] = lam * S[j] + torch.einsum("hk,hv->hkv", s["k"][n].double(), s["v"][n].double())
            o[n] = torch.einsum("hk,hkv->hv", s["q"][n].double(), S[j])
        return {"o": o, "state": S}

    def order(n, first):
        """Token rows of a sequence of n tokens in its scan order."""
        if s.get("packed"):
            r = list(range(first, first + n))
        else:
            Hg, Wg = s["grid_h"], s["grid_w"]
            r = [i * Wg + j for i in range(Hg) for j in range(Wg)] if s["mode"] < 2 else [i * Wg + j for j in range(Wg) for i in range(Hg)]
        return r[::-1] if s["mode"] & 1 else r

    if op == "attn_fwd":
        o = s["o"].double()
        state = s["Sf"].double() if s["slots"] is not None else None
        first = 0
        flat = [s[n].double() for n in ("q", "k", "v")]
        if s["packed"]:
            for b, n in enumerate(s["lens"]):
                j = int(s["slots"][b]) if s["slots"] is not None else None
                S = state[j].clone() if j is not None else torch.zeros(H, dk, dv, device=DEV, dtype=torch.float64)
                for t in order(n, first):
                    S.mul_(lam).add_(flat[1][t][:, :, None] * flat[2][t][:, None, :])
                    o[t] = torch.matmul(flat[0][t][:, None, :], S)[:, 0]
                if j is not None:
                    state[j] = S
                first += n
        else:
            S = torch.zeros(s["B"], H, dk, dv, device=DEV, dtype=torch.float64)
            for t in order(s["grid_h"] * s["grid_w"], 0):
                S.mul_(lam).add_(flat[1][:, t, :, :, None] * flat[2][:, t, :, None, :])
                o[:, t] = torch.matmul(flat[0][:, t, :, None, :], S)[:, :, 0]
        return {"o": o, "state": state} if state is not None else {"o": o}
    q, k, v, dO = (s[n].double() for n in ("q", "k", "v", "dO"))
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    zero = torch.zeros(s["B"], H, dk, dv, device=DEV, dtype=torch.float64)
    S = s["S0"].double() if s["states"] else zero.clone()
    G = s["dSf"].double() if s["states"] else zero.clone()
    seq = order(s["grid_h"] * s["grid_w"], 0)
    for t in seq:
        S = lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = torch.matmul(S, dO[:, t, :, :, None])[..., 0]
    for t in reversed(seq):
        G = G + q[:, t, :, :, None] * dO[:, t, :, None, :]
        dk_[:, t] = torch.matmul(G, v[:, t, :, :, None])[..., 0]
        dv_[:, t] = torch.matmul(k[:, t, :, None, :], G)[:, :, 0]
        G = lam * G
    out = {"dq": dq.view(-1, H, dk), "dk": dk_.view(-1, H, dk), "dv": dv_.view(-1, H, dv)}
    if s["states"]:
        out["dS0"] = G
    return out
