"""Measured cases of the channels-last training block's operators: PatchGroupNorm
(+ SiLU) over channels-last patches, forward and backward, and dropout whose mask
comes from a counter-based generator and is never stored, with an optional
residual.

``own`` false: plain torch, in 32 bits, rounded once at the end.  ``own``
true: the calls a user makes of ``patch_groupnorm_gb300.tileblend``.

A case's ``op`` is one of

* ``gn_fwd``   y = silu(GN(x)) over patches [N, *spatial_p, C]
* ``gn_bwd``   dx, dgamma, dbeta of the same, from the forward pass's records
* ``drop_fwd`` y = residual + dropout(x), or dropout(x)
* ``drop_bwd`` dx = the same mask and scale applied to dy
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
        # a small activation split over two patches: latency counts
        dict(name="gn_fwd_small", op="gn_fwd", N=1, C=64, D=1, H=15, W=32, patches=2, axis="h", groups=8,
             dtype="bf16", silu=True),
        # an odd channel count and an odd image, three samples: no row but a sample's first is aligned
        dict(name="gn_fwd_odd", op="gn_fwd", N=3, C=515, D=1, H=37, W=83, patches=1, axis="h", groups=5,
             dtype="f16", silu=True),
        # the library's 4D and 5D GroupNorm workloads, channels last
        dict(name="gn_fwd_4d", op="gn_fwd", N=1, C=512, D=1, H=256, W=256, patches=4, axis="h", groups=32,
             dtype="bf16", silu=True),
        dict(name="gn_fwd_5d", op="gn_fwd", N=1, C=384, D=13, H=120, W=208, patches=4, axis="w", groups=32,
             dtype="bf16", silu=True),
        # a small training step in 32 bits, backward; and the two workloads backward
        dict(name="gn_bwd_small", op="gn_bwd", N=1, C=64, D=1, H=15, W=32, patches=2, axis="h", groups=8,
             dtype="f32", silu=True),
        dict(name="gn_bwd_4d", op="gn_bwd", N=1, C=512, D=1, H=256, W=256, patches=4, axis="h", groups=32,
             dtype="bf16", silu=True),
        dict(name="gn_bwd_5d", op="gn_bwd", N=1, C=384, D=13, H=120, W=208, patches=4, axis="w", groups=32,
             dtype="bf16", silu=True),
        # a small training step in 32 bits
        dict(name="drop_fwd_small", op="drop_fwd", rows=240, cols=384, dtype="f32", residual=True, wide=False, p=0.1),
        # a ragged batch with an odd width, cut out of rows twice as wide
        dict(name="drop_fwd_odd", op="drop_fwd", rows=4099, cols=1111, dtype="f16", residual=True, wide=True, p=0.2),
        # the positions of a 512 x 256 x 256 decoder activation, as tokens, onto their residual stream
        dict(name="drop_fwd_tokens", op="drop_fwd", rows=65536, cols=512, dtype="bf16", residual=True, wide=False,
             p=0.1),
        # a training batch of a residual stream of 4096, forward without the residual, and backward
        dict(name="drop_fwd_prompt", op="drop_fwd", rows=16384, cols=4096, dtype="bf16", residual=False, wide=False,
             p=0.1),
        dict(name="drop_bwd_tokens", op="drop_bwd", rows=65536, cols=512, dtype="bf16", residual=False, wide=False,
             p=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_bwd", "drop_fwd", "drop_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("drop_fwd", "drop_bwd"):
        cols = _log(rng, 32, 16384)
        if rng.random() < 0.6:  # most widths are whole vectors
            cols = max(32, cols // 32 * 32)
        rows = _log(rng, 1, min(65536, 16384 * 4096 // cols))
        if dtype == "f32":
            rows = max(1, rows // 2)
        residual = op == "drop_fwd" and rng.random() < 0.5
        if residual:
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=residual, wide=rng.random() < 0.3,
                    p=rng.choice([0.05, 0.1, 0.2, 0.5]))
    groups = rng.choice([1, 4, 8, 16, 32])
    C = groups * rng.randint(1, max(1, 512 // groups))
    D = rng.choice([1, 1, rng.randint(2, 13)])
    N = rng.choice([1, 1, 2, 3])
    most = 384 * 13 * 120 * 208 // (N * C * D * (2 if dtype == "f32" else 1))
    H = _log(rng, 4, max(5, min(256, int(math.sqrt(most)))))
    W = _log(rng, 4, max(5, min(256, most // H)))
    axis = rng.choice(["h", "w"])
    return dict(op=op, N=N, C=C, D=D, H=H, W=W, patches=rng.randint(1, min(4, H if axis == "h" else W)), axis=axis,
                groups=groups, dtype=dtype, silu=rng.random() < 0.7)


def _numel(case):
    return case["N"] * case["C"] * case["D"] * case["H"] * case["W"]


def work(case):
    op, es = case["op"], TYPES[case["dtype"]].itemsize
    if op == "gn_fwd":
        n = _numel(case)
        return {"bytes": 2 * n * es + 2 * case["C"] * es, "flops": n * (12 if case["silu"] else 7)}
    if op == "gn_bwd":
        n = _numel(case)
        return {"bytes": 3 * n * es + 4 * case["C"] * es, "flops": n * (28 if case["silu"] else 14)}
    n = case["rows"] * case["cols"]
    # an eighth of a block of ten rounds: two products, two sums of three bits each; then compare, scale, add
    return {"bytes": (2 + case["residual"]) * n * es, "flops": n * 8}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype, scale=1.0, offset=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale + offset).to(dtype)


def _patch_shapes(case):
    full = [case["N"]] + ([case["D"]] if case["D"] > 1 else []) + [case["H"], case["W"], case["C"]]
    dim = len(full) - (3 if case["axis"] == "h" else 2)
    P = case["patches"]
    each, extra = divmod(full[dim], P)
    return [tuple(full[:dim] + [each + (p < extra)] + full[dim + 1:]) for p in range(P)]


def _prepare_gn(case, seed):
    g = _gen(seed)
    dt, N, C, G = TYPES[case["dtype"]], case["N"], case["C"], case["groups"]
    shapes = _patch_shapes(case)
    means = [2.0 * p - len(shapes) + 1 for p in range(len(shapes))]
    xs = [_randn(g, sh, dt, 1.0, m) for sh, m in zip(shapes, means)]
    s = dict(case=case, xs=xs, gamma=_randn(g, C, dt, 0.1, 1.0), beta=_randn(g, C, dt, 0.1),
             outs=[torch.empty_like(x) for x in xs])
    rec = torch.zeros((len(xs), N, G, PARTS, 2), dtype=torch.int64, device="cuda")
    s["records"] = rec
    if case["op"] == "gn_fwd":
        return s
    # the forward pass left its statistics records: (count, mean, M2) of every patch, sample and group
    flat = [x.reshape(N, -1, G, C // G).float() for x in xs]
    rec[:, :, :, 0, 0] = torch.tensor([f.shape[1] * f.shape[3] for f in flat], device="cuda")[:, None, None]
    mean = torch.stack([f.mean((1, 3)) for f in flat])
    m2 = torch.stack([((f - m[:, None, :, None]) ** 2).sum((1, 3)) for f, m in zip(flat, mean)])
    rec[:, :, :, 0, 1] = torch.stack([mean, m2], -1).contiguous().view(torch.int64)[..., 0]
    s.update(dys=[_randn(g, sh, dt, 0.02) for sh in shapes], dgamma=torch.empty(C, dtype=dt, device="cuda"),
             dbeta=torch.empty(C, dtype=dt, device="cuda"))
    if own:  # workspaces that a training program keeps from step to step
        s["grad_records"] = _lib().new_grad_partials(len(xs), N, C)
        s["workspace"] = _lib().gn_workspace_cl(N, G)
    return s


def _prepare_drop(case, seed):
    g = _gen(seed)
    dt, R, C = TYPES[case["dtype"]], case["rows"], case["cols"]
    x = _randn(g, (R, 2 * C if case["wide"] else C), dt, 0.02 if case["op"] == "drop_bwd" else 1.0)[:, :C]
    return dict(case=case, x=x, residual=_randn(g, (R, C), dt) if case["residual"] else None,
                y=torch.empty((R, C), dtype=dt, device="cuda"), p=case["p"],
                # the layer's key, and the step and layer that the mask is drawn for
                seed=(seed + 1) * 0x2545F4914F6CDD1D % 2 ** 64, offset=(seed % 1000) * 64 + 7)


def prepare(case, seed):
    return (_prepare_gn if case["op"] in ("gn_fwd", "gn_bwd") else _prepare_drop)(case, seed)


# ---------------------------------------------------------------------------
# the operators, plain and the library's
# ---------------------------------------------------------------------------

def _gn_fwd(s):
    case, xs, gamma, beta = s["case"], s["xs"], s["gamma"], s["beta"]
    N, C, G = case["N"], case["C"], case["groups"]
    if own:
        _lib().patch_group_norm_cl(xs, G, gamma, beta, EPS, silu=case["silu"], outs=s["outs"], partials=s["records"])
        return dict(y=s["outs"])
    x = torch.cat([t.reshape(N, -1, G, C // G) for t in xs], 1).float()
    count = x.shape[1] * x.shape[3]
    mean = x.sum((1, 3), keepdim=True) / count
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).sum((1, 3), keepdim=True) / count + EPS)
    z = d * rstd * gamma.float().reshape(G, -1) + beta.float().reshape(G, -1)
    if case["silu"]:
        z = z / (1.0 + torch.exp(-z))
    y = z.to(xs[0].dtype)
    return dict(y=[p.reshape(t.shape) for p, t in zip(y.split([t[0].numel() // C for t in xs], 1), xs)])


def _gn_bwd(s):
    case, xs, dys, gamma, beta = s["case"], s["xs"], s["dys"], s["gamma"], s["beta"]
    N, C, G = case["N"], case["C"], case["groups"]
    if own:
        _lib().patch_group_norm_backward_cl(dys, xs, G, s["records"], gamma, beta, EPS, silu=case["silu"],
                                            dxs=s["outs"], dgamma=s["dgamma"], dbeta=s["dbeta"],
                                            grad_partials=s["grad_records"], workspace=s["workspace"])
        return dict(dx=s["outs"], dgamma=s["dgamma"], dbeta=s["dbeta"])
    # pool the records: counts, means about the pooled one, variances
    r = s["records"][:, :, :, 0]
    n = r[..., 0].float()
    m, m2 = r[..., 1:].contiguous().view(torch.float32).unbind(-1)
    count = n.sum(0)
    mean = (n * m).sum(0) / count
    rstd = 1.0 / torch.sqrt((m2 + n * (m - mean) ** 2).sum(0) / count + EPS)
    x = torch.cat([t.reshape(N, -1, G, C // G) for t in xs], 1).float()
    dz = torch.cat([t.reshape(N, -1, G, C // G) for t in dys], 1).float()
    xhat = (x - mean[:, None, :, None]) * rstd[:, None, :, None]
    gam, bet = gamma.float().reshape(G, -1), beta.float().reshape(G, -1)
    if case["silu"]:
        z = xhat * gam + bet
        sig = 1.0 / (1.0 + torch.exp(-z))
        dz = dz * (sig * (1.0 + z * (1.0 - sig)))
    B, A = dz.sum(1), (dz * xhat).sum(1)
    c1 = ((B * gam).sum(2) / count)[:, None, :, None]
    c2 = ((A * gam).sum(2) / count)[:, None, :, None]
    dx = (rstd[:, None, :, None] * (dz * gam - c1 - xhat * c2)).to(xs[0].dtype)
    dxs = [p.reshape(t.shape) for p, t in zip(dx.split([t[0].numel() // C for t in xs], 1), xs)]
    return dict(dx=dxs, dgamma=A.sum(0).reshape(C).to(gamma.dtype), dbeta=B.sum(0).reshape(C).to(gamma.dtype))


M32 = 0xFFFFFFFF


def _bits(n, seed, offset):
    """n numbers of 16 bits: Philox 4x32 with ten rounds, key = seed, counter =
    (number of the block of eight, offset), each word's low half first."""
    b = torch.arange(-(-n // 8), device="cuda")
    c0, c1 = b & M32, b >> 32
    c2, c3 = torch.full_like(b, offset & M32), torch.full_like(b, offset >> 32 & M32)
    k0, k1 = seed & M32, seed >> 32 & M32
    for _ in range(10):
        # the products of 32-bit words wrap in int64; shifted and masked, their halves are right
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = p1 >> 32 & M32 ^ c1 ^ k0, p1 & M32, p0 >> 32 & M32 ^ c3 ^ k1, p0 & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    words = torch.stack([c0, c1, c2, c3], 1).reshape(-1)
    return torch.stack([words & 0xFFFF, words >> 16], 1).reshape(-1)[:n]


def _drop(s):
    x, r = s["x"], s["residual"]
    if own:
        _lib().tb_dropout(x, s["y"], s["p"], s["seed"], s["offset"], residual=r)
        return s["y"]
    t = math.floor(s["p"] * 65536 + 0.5)  # dropped: bits below t of 65536
    kept = (_bits(x.numel(), s["seed"], s["offset"]) >= t).reshape(x.shape)
    y = torch.where(kept, x.float() * (65536.0 / (65536 - t)), 0.0)
    return (y if r is None else y + r.float()).to(x.dtype)


def run(state):
    return {"gn_fwd": _gn_fwd, "gn_bwd": _gn_bwd, "drop_fwd": _drop, "drop_bwd": _drop}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _mul32(a, m):
    """(high, low) 32 bits of a * m for 32-bit values, from 16-bit digits of a."""
    lo, hi = (a % 65536) * m, torch.div(a, 65536, rounding_mode="floor") * m
    low = (lo + (hi % 65536) * 65536) % 2 ** 32
    high = torch.div(hi + torch.div(lo, 65536, rounding_mode="floor"), 65536, rounding_mode="floor")
    return high, low


def _exact_drop(case, s):
    x = s["x"].to(torch.float64)
    t = math.floor(case["p"] * 65536 + 0.5)
    flat = x.reshape(-1).clone()
    blocks = -(-flat.numel() // 8)
    ctr = [torch.arange(blocks, device="cuda"), 0, s["offset"], 0]  # no case has 2^32 blocks, no offset 2^32
    ctr = [torch.as_tensor(c, device="cuda").expand(blocks) for c in ctr]
    for k in range(10):
        key = [(s["seed"] % 2 ** 32 + k * 0x9E3779B9) % 2 ** 32, (s["seed"] // 2 ** 32 + k * 0xBB67AE85) % 2 ** 32]
        h0, l0 = _mul32(ctr[0], 0xD2511F53)
        h1, l1 = _mul32(ctr[2], 0xCD9E8D57)
        ctr = [h1.bitwise_xor(ctr[1]).bitwise_xor(key[0]), l1, h0.bitwise_xor(ctr[3]).bitwise_xor(key[1]), l0]
    for e in range(8):  # element 8 b + e has the half e % 2 of word e / 2 of block b
        half = ctr[e // 2] % 65536 if e % 2 == 0 else torch.div(ctr[e // 2], 65536, rounding_mode="floor")
        part = flat[e::8]
        part.mul_((half[:part.numel()] >= t).to(torch.float64))
    y = (flat * 65536 / (65536 - t)).reshape(x.shape)
    return y if s["residual"] is None else y + s["residual"].to(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("drop_fwd", "drop_bwd"):
        return _exact_drop(case, s)
    # sample by sample and group by group, from the elements themselves
    f8 = torch.float64
    N, C, G = case["N"], case["C"], case["groups"]
    if N * G > 256:
        return None
    K = C // G
    xs = s["xs"]
    gam, bet = s["gamma"].to(f8).reshape(G, 1, K), s["beta"].to(f8).reshape(G, 1, K)
    outs = [torch.empty_like(x, dtype=f8) for x in xs]
    dgamma, dbeta = torch.zeros(G, K, dtype=f8, device="cuda"), torch.zeros(G, K, dtype=f8, device="cuda")
    for n in range(N):
        for g in range(G):
            def cut(ts):
                return [t[n].reshape(-1, C)[:, g * K:(g + 1) * K] for t in ts]
            x = torch.cat(cut(xs)).to(f8)
            rstd = (x.var(correction=0) + EPS).rsqrt()
            xhat = (x - x.mean()) * rstd
            z = xhat * gam[g] + bet[g]
            sig = torch.sigmoid(z)
            if case["op"] == "gn_fwd":
                out = z * sig if case["silu"] else z
            else:
                dz = torch.cat(cut(s["dys"])).to(f8)
                if case["silu"]:
                    dz = dz * (sig + z * sig * (1 - sig))
                dgamma[g] += (dz * xhat).sum(0)
                dbeta[g] += dz.sum(0)
                v = dz * gam[g]
                out = (v - v.mean() - xhat * (v * xhat).mean()) * rstd
            for t, part in zip(outs, out.split([len(c) for c in cut(xs)])):
                t[n].reshape(-1, C)[:, g * K:(g + 1) * K] = part
    if case["op"] == "gn_fwd":
        return dict(y=outs)
    return dict(dx=outs, dgamma=dgamma.reshape(C), dbeta=dbeta.reshape(C))
