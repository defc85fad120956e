"""Measured cases of the training operators: layer norm forward and backward,
the global gradient norm with clipping, and PatchGroupNorm's backward pass.

``own`` false: plain torch, in 32 bits, rounded once at the end.  ``own``
true: the calls a user makes of ``patch_groupnorm_gb300.tileblend``.

A case's ``op`` is one of

* ``ln_fwd``   y = LN(h) * gamma + beta, h = x or (residual) x + residual
* ``ln_bwd``   dx, dgamma, dbeta of the same (residual: the gradient that
               reaches h past the norm is added to dx)
* ``clip``     every gradient times min(1, max_norm / (norm + 1e-6)), into the
               flat buffers an optimizer reads
* ``gn_bwd``   dx, dgamma, dbeta of a GroupNorm (+ SiLU) over patches
"""
import math

import torch

own = False

EPS = 1e-6
PARTS = 8          # statistics records per (patch, sample, group)
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _lib():
    from patch_groupnorm_gb300 import tileblend
    return tileblend


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode loop: a residual stream of 4096, weights in 32 bits
        dict(name="ln_fwd_token", op="ln_fwd", rows=1, cols=4096, dtype="bf16", wdtype="f32", residual=True),
        # a ragged batch with an odd width: no row but the first is aligned
        dict(name="ln_fwd_odd", op="ln_fwd", rows=4099, cols=1111, dtype="f16", wdtype="f16", residual=False),
        # the positions of a 512 x 256 x 256 decoder activation, as tokens of an attention block
        dict(name="ln_fwd_tokens", op="ln_fwd", rows=65536, cols=512, dtype="bf16", wdtype="bf16", residual=False),
        # a long prompt, or a training batch, of a residual stream of 4096
        dict(name="ln_fwd_prompt", op="ln_fwd", rows=16384, cols=4096, dtype="bf16", wdtype="f32", residual=True),
        # a small training step in 32 bits
        dict(name="ln_bwd_small", op="ln_bwd", rows=240, cols=384, dtype="f32", wdtype="f32", residual=False),
        # the same tokens and the same training batch, backward
        dict(name="ln_bwd_tokens", op="ln_bwd", rows=65536, cols=512, dtype="bf16", wdtype="bf16", residual=False),
        dict(name="ln_bwd_prompt", op="ln_bwd", rows=16384, cols=4096, dtype="bf16", wdtype="f32", residual=True),
        # the gradients of two blocks of width 384, in 32 bits
        dict(name="clip_small", op="clip", layers=2, width=384, vocab=0, dtype="f32"),
        # the gradients of 24 blocks of width 1024 and two tables of 32000 rows: 16-bit matrices, 32-bit norm weights
        dict(name="clip_large", op="clip", layers=24, width=1024, vocab=32000, dtype="bf16"),
        # a small activation split over two patches
        dict(name="gn_bwd_small", op="gn_bwd", N=1, C=64, D=1, H=15, W=32, patches=2, axis="h", groups=8,
             dtype="bf16", silu=True),
        # the library's 4D and 5D GroupNorm workloads, backward
        dict(name="gn_bwd_4d", op="gn_bwd", N=1, C=512, D=1, H=256, W=256, patches=4, axis="h", groups=32,
             dtype="bf16", silu=True),
        dict(name="gn_bwd_5d", op="gn_bwd", N=1, C=384, D=13, H=120, W=208, patches=4, axis="w", groups=32,
             dtype="bf16", silu=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "clip", "gn_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("ln_fwd", "ln_bwd"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.6:  # most widths are whole vectors
            cols = max(64, cols // 64 * 64)
        if cols == 3072:
            cols += 64
        rows = _log(rng, 1 if op == "ln_fwd" else 16, min(65536, 16384 * 4096 // cols))
        if dtype == "f32":
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, wdtype=rng.choice([dtype, "f32"]),
                    residual=rng.random() < 0.5)
    if op == "clip":
        width = _log(rng, 65, 1023)
        if rng.random() < 0.5:
            width = max(64, width // 64 * 64)
        if width in (768, 1536):
            width += 64
        return dict(op=op, layers=_log(rng, 1, 24 if dtype != "f32" else 12), width=width,
                    vocab=rng.choice([0, _log(rng, 100, 32000)]), dtype=dtype)
    groups = rng.choice([1, 4, 8, 16, 32])
    C = groups * rng.randint(1, max(1, 512 // groups))
    D = rng.choice([1, 1, rng.randint(2, 13)])
    N = rng.choice([1, 1, 2, 3])
    most = 384 * 13 * 120 * 208 // (N * C * D * (2 if dtype == "f32" else 1))
    H = _log(rng, 4, max(5, min(256, int(math.sqrt(most)))))
    W = _log(rng, 4, max(5, min(256, most // H)))
    if rng.random() < 0.6:
        W = max(8, W // 8 * 8)
    axis = rng.choice(["h", "w"])
    return dict(op=op, N=N, C=C, D=D, H=H, W=W, patches=rng.randint(1, min(4, H if axis == "h" else W)), axis=axis,
                groups=groups, dtype=dtype, silu=rng.random() < 0.7)


def _sizes(case):
    """(numel, dtype) of every gradient of a ``clip`` case: per block four
    projections, two matrices four times as wide, their biases and two norms'
    weights (32 bits), and two tables."""
    d, t = case["width"], case["dtype"]
    block = [(d * d, t)] * 4 + [(4 * d * d, t)] * 2 + [(4 * d, t), (d, t)] + [(d, "f32")] * 4
    return block * case["layers"] + [(case["vocab"] * d, t)] * (2 if case["vocab"] else 0)


def _numel(case):
    return case["N"] * case["C"] * case["D"] * case["H"] * case["W"]


def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        n, es = case["rows"] * case["cols"], TYPES[case["dtype"]].itemsize
        ws = TYPES[case["wdtype"]].itemsize
        moved = 2 + 2 * case["residual"] if op == "ln_fwd" else 3 + case["residual"]
        weights = (2 if op == "ln_fwd" else 3) * case["cols"] * ws
        return {"bytes": n * es * moved + weights + 8 * case["rows"], "flops": n * (8 if op == "ln_fwd" else 14)}
    if op == "clip":
        s = _sizes(case)
        return {"bytes": sum(2 * n * TYPES[t].itemsize for n, t in s) + 4, "flops": sum(3 * n for n, _ in s)}
    n, es = _numel(case), TYPES[case["dtype"]].itemsize
    return {"bytes": 3 * n * es + 4 * case["C"] * es, "flops": n * (28 if case["silu"] else 14)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype, scale=1.0, offset=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale + offset).to(dtype)


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _prepare_ln(case, seed):
    g = _gen(seed)
    dt, wt = TYPES[case["dtype"]], TYPES[case["wdtype"]]
    R, C = case["rows"], case["cols"]
    # activations: unit channels, one in 64 an outlier as residual streams have them
    chan = torch.where(torch.rand(C, generator=g, device="cuda") < 1 / 64, 12.0, 1.0)
    x = (torch.randn((R, C), generator=g, device="cuda") * chan + 0.1).to(dt)
    s = dict(case=case, gamma=_randn(g, C, wt, 0.1, 1.0), beta=_randn(g, C, wt, 0.1))
    if case["op"] == "ln_fwd":
        s.update(x=x, residual=_randn(g, (R, C), dt) if case["residual"] else None, y=torch.empty_like(x),
                 total=torch.empty_like(x) if case["residual"] else None, mean=_empty(R), rstd=_empty(R))
        return s
    # the forward pass left the rows' statistics; its workspace is kept from step to step
    xf = x.float()
    mean = xf.mean(1)
    rstd = 1.0 / torch.sqrt(((xf - mean[:, None]) ** 2).mean(1) + EPS)
    s.update(x=x, mean=mean, rstd=rstd, dy=_randn(g, (R, C), dt, 0.02),
             dtotal=_randn(g, (R, C), dt, 0.02) if case["residual"] else None, dx=torch.empty_like(x),
             dgamma=torch.empty_like(s["gamma"]), dbeta=torch.empty_like(s["beta"]))
    if own:
        s["workspace"] = _lib().ln_workspace(R, C)
    return s


def _prepare_clip(case, seed):
    g = _gen(seed)
    sizes = _sizes(case)
    # every tensor's gradients have a scale of their own, as layers do
    scales = (10.0 ** (torch.rand(len(sizes), generator=torch.Generator().manual_seed(seed)) * 3 - 5)).tolist()
    grads = [_randn(g, n, TYPES[t], sc) for (n, t), sc in zip(sizes, scales)]
    # the optimizer's flat buffers: one per type, each tensor's part starting on 16 bytes
    used = sorted({t for _, t in sizes})
    flat = {t: torch.zeros(sum(-(-n // 8) * 8 for n, u in sizes if u == t), dtype=TYPES[t], device="cuda")
            for t in used}
    at, outs = dict.fromkeys(used, 0), []
    for n, t in sizes:
        outs.append(flat[t][at[t]:at[t] + n])
        at[t] += -(-n // 8) * 8
    s = dict(case=case, grads=grads, outs=outs, flat=flat, norm=_empty(1), max_norm=1.0)
    if own:  # the table of the parameters' gradients that a training program makes once
        tb = _lib()
        s["table"] = tb.GradTable(grads, outs)
        s["records"] = tb.new_grad_records(len(grads))
    return s


def _patch_shapes(case):
    full = [case["N"], case["C"]] + ([case["D"]] if case["D"] > 1 else []) + [case["H"], case["W"]]
    dim = len(full) - (2 if case["axis"] == "h" else 1)
    P = case["patches"]
    each, extra = divmod(full[dim], P)
    return [tuple(full[:dim] + [each + (p < extra)] + full[dim + 1:]) for p in range(P)]


def _prepare_gn(case, seed):
    g = _gen(seed)
    dt, N, C, G = TYPES[case["dtype"]], case["N"], case["C"], case["groups"]
    shapes = _patch_shapes(case)
    means = [2.0 * p - len(shapes) + 1 for p in range(len(shapes))]
    xs = [_randn(g, sh, dt, 1.0, m) for sh, m in zip(shapes, means)]
    # the forward pass left its statistics records: (count, mean, M2) of every patch, sample and group
    rec = torch.zeros((len(xs), N, G, PARTS, 2), dtype=torch.int64, device="cuda")
    flat = [x.reshape(N, G, -1).float() for x in xs]
    rec[:, :, :, 0, 0] = torch.tensor([f.shape[2] for f in flat], device="cuda")[:, None, None]
    mean = torch.stack([f.mean(2) for f in flat])
    m2 = torch.stack([((f - m[..., None]) ** 2).sum(2) for f, m in zip(flat, mean)])
    rec[:, :, :, 0, 1] = torch.stack([mean, m2], -1).contiguous().view(torch.int64)[..., 0]
    s = dict(case=case, xs=xs, dys=[_randn(g, sh, dt, 0.02) for sh in shapes], records=rec,
             gamma=_randn(g, C, dt, 0.1, 1.0), beta=_randn(g, C, dt, 0.1), dxs=[torch.empty_like(x) for x in xs],
             dgamma=_empty(C, dtype=dt), dbeta=_empty(C, dtype=dt))
    if own:
        s["grad_records"] = _lib().new_grad_partials(len(xs), N, C)
    return s


def prepare(case, seed):
    return {"ln_fwd": _prepare_ln, "ln_bwd": _prepare_ln, "clip": _prepare_clip,
            "gn_bwd": _prepare_gn}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# the operators, plain and the library's
# ---------------------------------------------------------------------------

def _ln_fwd(s):
    x, r = s["x"], s["residual"]
    if own:
        _lib().tb_layer_norm(x, s["y"], s["gamma"], s["beta"], EPS, mean=s["mean"], rstd=s["rstd"], residual=r,
                             total=s["total"])
        out = dict(y=s["y"], mean=s["mean"], rstd=s["rstd"])
        return out if r is None else dict(out, total=s["total"])
    total = x if r is None else (x.float() + r.float()).to(x.dtype)
    h = total.float()
    mean = h.sum(1) / h.shape[1]
    d = h - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / h.shape[1] + EPS)
    y = (d * rstd[:, None] * s["gamma"].float() + s["beta"].float()).to(x.dtype)
    out = dict(y=y, mean=mean, rstd=rstd)
    return out if r is None else dict(out, total=total)


def _ln_bwd(s):
    x, dy, gamma = s["x"], s["dy"], s["gamma"]
    if own:
        _lib().tb_layer_norm_backward(dy, x, s["mean"], s["rstd"], gamma, s["dx"], s["dgamma"], s["dbeta"],
                                      s["workspace"], dtotal=s["dtotal"])
        return dict(dx=s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"])
    n, rstd = x.shape[1], s["rstd"][:, None]
    dyf = dy.float()
    xhat = (x.float() - s["mean"][:, None]) * rstd
    g = dyf * gamma.float()
    dx = rstd * (g - g.sum(1, keepdim=True) / n - xhat * ((g * xhat).sum(1, keepdim=True) / n))
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].float()
    return dict(dx=dx.to(x.dtype), dgamma=(dyf * xhat).sum(0).to(gamma.dtype), dbeta=dyf.sum(0).to(gamma.dtype))


def _clip(s):
    if own:
        _lib().clip_grad_norm(s["table"], s["max_norm"], records=s["records"], norm=s["norm"])
        return dict(flat=s["flat"], norm=s["norm"])
    norm = torch.sqrt(torch.stack([(g.float() * g.float()).sum() for g in s["grads"]]).sum()).reshape(1)
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["outs"])]
    return dict(flat=s["flat"], norm=norm)


def _gn_bwd(s):
    case, xs, dys, gamma, beta = s["case"], s["xs"], s["dys"], s["gamma"], s["beta"]
    N, C, G = case["N"], case["C"], case["groups"]
    if own:
        _lib().patch_group_norm_backward(dys, xs, G, s["records"], gamma, beta, EPS, silu=case["silu"], dxs=s["dxs"],
                                         dgamma=s["dgamma"], dbeta=s["dbeta"], grad_partials=s["grad_records"])
        return dict(dx=s["dxs"], dgamma=s["dgamma"], dbeta=s["dbeta"])
    # pool the records: counts, means about the pooled one, variances
    r = s["records"][:, :, :, 0]
    n = r[..., 0].float()
    m, m2 = r[..., 1:].contiguous().view(torch.float32).unbind(-1)
    count = n.sum(0)
    mean = (n * m).sum(0) / count
    rstd = 1.0 / torch.sqrt((m2 + n * (m - mean) ** 2).sum(0) / count + EPS)
    x = torch.cat([t.reshape(N, G, C // G, -1) for t in xs], 3).float()
    dz = torch.cat([t.reshape(N, G, C // G, -1) for t in dys], 3).float()
    xhat = (x - mean[..., None, None]) * rstd[..., None, None]
    gam, bet = gamma.float().reshape(G, -1, 1), beta.float().reshape(G, -1, 1)
    if case["silu"]:
        z = xhat * gam + bet
        sig = 1.0 / (1.0 + torch.exp(-z))
        dz = dz * (sig * (1.0 + z * (1.0 - sig)))
    B, A = dz.sum(3), (dz * xhat).sum(3)
    c1 = (B * gam[..., 0]).sum(2) / count
    c2 = (A * gam[..., 0]).sum(2) / count
    dx = (rstd[..., None, None] * (dz * gam - c1[..., None, None] - xhat * c2[..., None, None])).to(xs[0].dtype)
    dxs = [p.reshape(t.shape) for p, t in zip(dx.split([t[0, 0].numel() for t in xs], 3), xs)]
    return dict(dx=dxs, dgamma=A.sum(0).reshape(C).to(gamma.dtype), dbeta=B.sum(0).reshape(C).to(gamma.dtype))


def run(state):
    return {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "clip": _clip, "gn_bwd": _gn_bwd}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "ln_fwd":
        x = s["x"]
        total = None if s["residual"] is None else (x.to(f8) + s["residual"].to(f8)).to(x.dtype)
        h = (x if total is None else total).to(f8)
        var, mean = torch.var_mean(h, 1, correction=0, keepdim=True)
        rstd = (var + EPS).rsqrt()
        out = dict(y=(h - mean) * rstd * s["gamma"].to(f8) + s["beta"].to(f8), mean=mean[:, 0], rstd=rstd[:, 0])
        return out if total is None else dict(out, total=total.to(f8))
    if case["op"] == "ln_bwd":
        # dx = rstd (I - 1 1'/n - xhat xhat'/n) (dy gamma), with the statistics that the forward pass kept
        dy, rstd = s["dy"].to(f8), s["rstd"].to(f8)[:, None]
        xhat = (s["x"].to(f8) - s["mean"].to(f8)[:, None]) * rstd
        v = dy * s["gamma"].to(f8)
        along = torch.einsum("rc,rc->r", v, xhat)[:, None] / case["cols"]
        dx = (v - v.mean(1, keepdim=True) - along * xhat) * rstd
        if s["dtotal"] is not None:
            dx += s["dtotal"].to(f8)
        return dict(dx=dx, dgamma=torch.einsum("rc,rc->c", dy, xhat), dbeta=dy.sum(0))
    if case["op"] == "clip":
        norm = math.sqrt(math.fsum(float(torch.dot(g.to(f8), g.to(f8))) for g in s["grads"]))
        coef = min(1.0, s["max_norm"] / (norm + 1e-6))
        flat = {t: torch.zeros_like(v, dtype=f8) for t, v in s["flat"].items()}
        at = dict.fromkeys(flat, 0)
        for (n, t), g in zip(_sizes(case), s["grads"]):
            flat[t][at[t]:at[t] + n] = g.to(f8) * coef
            at[t] += -(-n // 8) * 8
        return dict(flat=flat, norm=torch.tensor([norm], dtype=f8))
    # gn_bwd: sample by sample and group by group, from the elements themselves
    N, C, G = case["N"], case["C"], case["groups"]
    if N * G > 256:
        return None
    K = C // G
    xs, dys = s["xs"], s["dys"]
    gam, bet = s["gamma"].to(f8).reshape(G, K, 1), s["beta"].to(f8).reshape(G, K, 1)
    dxs = [torch.empty_like(x, dtype=f8) for x in xs]
    dgamma, dbeta = torch.zeros(G, K, dtype=f8, device="cuda"), torch.zeros(G, K, dtype=f8, device="cuda")
    for n in range(N):
        for g in range(G):
            cut = [t[n, g * K:(g + 1) * K].reshape(K, -1).shape[1] for t in xs]
            x = torch.cat([t[n, g * K:(g + 1) * K].reshape(K, -1) for t in xs], 1).to(f8)
            dz = torch.cat([t[n, g * K:(g + 1) * K].reshape(K, -1) for t in dys], 1).to(f8)
            rstd = (x.var(correction=0) + EPS).rsqrt()
            xhat = (x - x.mean()) * rstd
            if case["silu"]:
                z = xhat * gam[g] + bet[g]
                sig = torch.sigmoid(z)
                dz = dz * (sig + z * sig * (1 - sig))
            dgamma[g] += (dz * xhat).sum(1)
            dbeta[g] += dz.sum(1)
            v = dz * gam[g]
            dx = (v - v.mean() - xhat * (v * xhat).mean()) * rstd
            for t, part in zip(dxs, dx.split(cut, 1)):
                t[n, g * K:(g + 1) * K] = part.reshape(t[n, g * K:(g + 1) * K].shape)
    return dict(dx=dxs, dgamma=dgamma.reshape(C), dbeta=dbeta.reshape(C))
