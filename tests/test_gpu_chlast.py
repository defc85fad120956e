"""GPU parity of channels-last PatchGroupNorm against the float64 oracle, which
sees the same tensors with the channels moved forward.

Forward tolerances as for the channels-first calls (``tests/tolerance.py``) where
inputs are of order one, else derived at the test; backward tolerances as derived
at the head of ``test_gpu_training.py`` (rounding of the output and K u times the
magnitudes that make it)."""
import numpy as np
import pytest
import torch

from oracle import groupnorm as GN
from tests.test_gpu_training import DT, HALF, TINY, U, check, check_gn, f64, rows_of, weights_of
from tests.tolerance import gn_violation

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tbl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import tileblend
    return tileblend


def cf(ts):
    return [t.movedim(-1, 1) for t in ts]


def check_forward(xs, G, gamma, beta, eps, silu, outs):
    name = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[xs[0].dtype]
    assert gn_violation(cf(outs), cf(xs), gamma, beta, G, eps, silu, name) <= 1.0


def check_backward(dys, xs, G, gamma, beta, eps, silu, dxs, dgamma, dbeta):
    check_gn(cf(dys), cf(xs), G, gamma, beta, eps, silu, cf(dxs), dgamma, dbeta, 2e-5)


def run(tbl, xs, dys, G, gamma, beta, eps, silu):
    part = tbl.new_partials(len(xs), xs[0].shape[0], G)
    part.fill_(-1)
    outs = tbl.patch_group_norm_cl(xs, G, gamma, beta, eps, silu, partials=part)
    check_forward(xs, G, gamma, beta, eps, silu, outs)
    dxs, dg, db = tbl.patch_group_norm_backward_cl(dys, xs, G, part, gamma, beta, eps, silu)
    check_backward(dys, xs, G, gamma, beta, eps, silu, dxs, dg, db)
    return part, outs, dxs, dg, db


# shape [N, *spatial, C], split axis, sizes, groups
CASES = [
    ((1, 24, 40, 32), 1, [6, 6, 6, 6], 4),
    ((2, 10, 33, 16), 2, [9, 8, 8, 8], 4),
    ((1, 5, 12, 16, 24), 3, [4, 4, 4, 4], 4),
    ((1, 3, 7, 9, 12), 2, [4, 3], 2),             # a position is not a whole number of chunks
    ((3, 64, 8), 1, [64], 4),
    ((2, 1, 6), 1, [1], 3),                        # one position
    ((1, 8, 16, 4), 1, [3, 0, 5], 1),              # an empty patch in the middle
    ((3, 17, 3, 5), 1, [10, 7], 5),                # samples at odd addresses; one channel a group
    ((1, 1, 1, 1), 1, [1], 1),                     # a single element
    ((2, 2, 3), 1, [1, 1], 1),                     # fewer elements than a chunk
    ((1, 900, 67), 1, [450, 450], 67),
    ((1, 50, 515), 1, [20, 30], 5),                # a period wider than a CTA
    ((2, 9, 1300), 1, [9], 26),                    # more columns than threads in 32 bits
    ((1, 3, 2051), 1, [3], 7),
    ((1, 7000, 40), 1, [3501, 3499], 5),           # many turns of a CTA
    ((1, 33000, 8), 1, [33000], 2),
    ((1, 4001, 64), 1, [1, 4000], 8),              # patches of very different size
    ((70, 5, 24), 1, [2, 3], 3),                   # many samples
]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[0])))
def test_forward_and_backward(tbl, case, dtype, silu):
    shape, dim, sizes, G = case
    dt = DT[dtype]
    x = rows_of(sum(shape), shape, torch.float64, 1.5)
    xs = [(p + m).to(dt).contiguous() for p, m in zip(x.split(sizes, dim), [-3.0, 3.0, -1.0, 1.0])]
    dys = [p.contiguous() for p in rows_of(7, shape, dt, 0.5).split(sizes, dim)]
    gamma, beta = weights_of(8, shape[-1], dt)
    run(tbl, xs, dys, G, gamma, beta, 1e-6, silu)
    run(tbl, xs, dys, G, None, None, 1e-6, silu)
    run(tbl, xs, dys, G, gamma, None, 1e-6, silu)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("C,G", [(48, 4), (50, 5), (515, 103)])
def test_in_place_misaligned_and_guard_bands(tbl, C, G, dtype):
    dt = DT[dtype]
    shape = (2, 30, C)
    x, dy = rows_of(1, shape, dt, 1.0, 0.5), rows_of(2, shape, dt)
    gamma, beta = weights_of(3, C, dt)
    part, (y,), (dx,), dg, db = run(tbl, [x], [dy], G, gamma, beta, 1e-6, True)
    t = x.clone()
    assert torch.equal(tbl.patch_group_norm_cl([t], G, gamma, beta, 1e-6, outs=[t])[0], y)
    for which in (0, 1):
        t = [dy.clone(), x.clone()]
        (o,), g2, b2 = tbl.patch_group_norm_backward_cl([t[0]], [t[1]], G, part, gamma, beta, 1e-6, dxs=[t[which]])
        assert torch.equal(o, dx) and torch.equal(g2, dg) and torch.equal(b2, db)
    # all tensors at one offset, then at several; what lies around them stays
    n = x.numel()
    for at in ((1, 1, 1), (3, 3, 3), (0, 1, 2), (1, 0, 0)):
        buf = torch.full((3, (n + 24) // 8 * 8), 7.0, dtype=dt, device="cuda")
        mx, md, mo = (b[a:a + n].view(shape) for a, b in zip(at, buf))
        mx.copy_(x)
        md.copy_(dy)
        tbl.patch_group_norm_cl([mx], G, gamma, beta, 1e-6, outs=[mo])
        check_forward([x], G, gamma, beta, 1e-6, True, [mo])
        _, g2, b2 = tbl.patch_group_norm_backward_cl([md], [mx], G, part, gamma, beta, 1e-6, dxs=[mo])
        check_backward([dy], [x], G, gamma, beta, 1e-6, True, [mo], g2, b2)
        assert torch.equal(mx, x) and torch.equal(md, dy)
        for a, b in zip(at, buf):
            assert (b[:a] == 7.0).all() and (b[a + n:] == 7.0).all()


def test_records_are_those_of_the_channels_first_calls(tbl):
    # either statistics serve either apply; the pooled sums agree
    dt, G = torch.float32, 4
    xs = [p.contiguous() for p in rows_of(1, (2, 12, 8, 16), dt, 1.0, 2.0).split([5, 7], 1)]
    fs = [x.movedim(-1, 1).contiguous() for x in xs]
    gamma, beta = weights_of(2, 16, dt)
    a = tbl.tb_patch_gn_stats_cl(xs, G, tbl.new_partials(2, 2, G))
    b = tbl.tb_patch_gn_stats(fs, G, tbl.new_partials(2, 2, G))
    assert torch.equal(a[..., 0].sum(-1), b[..., 0].sum(-1))
    ya = tbl.tb_patch_gn_apply_cl(xs, [torch.empty_like(x) for x in xs], G, b, 2, gamma, beta, 1e-6)
    check_forward(xs, G, gamma, beta, 1e-6, True, ya)
    yb = tbl.tb_patch_gn_apply(fs, [torch.empty_like(f) for f in fs], G, a, gamma, beta, 1e-6)
    check_forward(xs, G, gamma, beta, 1e-6, True, [y.movedim(1, -1) for y in yb])
    dys = [rows_of(5 + k, x.shape, dt) for k, x in enumerate(xs)]
    ga = tbl.tb_patch_gn_grad_stats_cl(dys, xs, G, b, 2, gamma, beta, 1e-6, tbl.new_grad_partials(2, 2, 16))
    dfs = [torch.empty_like(f) for f in fs]
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    tbl.tb_patch_gn_grad_apply([d.movedim(-1, 1).contiguous() for d in dys], fs, dfs, G, b, ga, 2, gamma, beta, 1e-6, dg,
                               db)
    check_gn(cf(dys), cf(xs), G, gamma, beta, 1e-6, True, dfs, dg, db, 2e-5)


@pytest.mark.parametrize("R", [2, 6])
def test_gathered_records(tbl, R):
    # ranks with one patch each: records of both passes gathered, each rank's results equal the unsharded ones
    dt, G = torch.bfloat16, 4
    x, dy = rows_of(1, (2, 4 * R, 8, 16), dt, 1.0, 0.5), rows_of(2, (2, 4 * R, 8, 16), dt)
    sizes = [3, 5] + [4] * (R - 2)
    xs, dys = ([p.contiguous() for p in t.split(sizes, 1)] for t in (x, dy))
    gamma, beta = weights_of(3, 16, dt)
    part = torch.cat([tbl.tb_patch_gn_stats_cl([p], G, tbl.new_partials(1, 2, G)) for p in xs])
    ys = [tbl.tb_patch_gn_apply_cl([p], [torch.empty_like(p)], G, part, R, gamma, beta, 1e-6)[0] for p in xs]
    check_forward(xs, G, gamma, beta, 1e-6, True, ys)
    grad = torch.cat([tbl.tb_patch_gn_grad_stats_cl([d], [p], G, part, R, gamma, beta, 1e-6,
                                                    tbl.new_grad_partials(1, 2, 16)) for d, p in zip(dys, xs)])
    ws = tbl.gn_workspace_cl(2, G)
    dxs, dgs, dbs = [], [], []
    for d, p in zip(dys, xs):
        o, dg, db = torch.empty_like(p), torch.empty_like(gamma), torch.empty_like(gamma)
        tbl.tb_patch_gn_grad_apply_cl([d], [p], [o], G, part, grad, R, gamma, beta, 1e-6, ws, dg, db)
        dxs.append(o)
        dgs.append(dg)
        dbs.append(db)
    check_backward(dys, xs, G, gamma, beta, 1e-6, True, dxs, dgs[0], dbs[0])
    assert all(torch.equal(dgs[0], t) for t in dgs) and all(torch.equal(dbs[0], t) for t in dbs)
    # a rank whose patch is empty still gets the weight gradients
    empty = torch.empty(2, 0, 8, 16, dtype=dt, device="cuda")
    dg, db = torch.full_like(gamma, 9.0), torch.full_like(gamma, 9.0)
    tbl.tb_patch_gn_grad_apply_cl([empty], [empty], [empty], G, part, grad, R, gamma, beta, 1e-6, ws, dg, db)
    assert torch.equal(dg, dgs[0]) and torch.equal(db, dbs[0])


def test_empty_sets_of_records_come_first(tbl):
    # five ranks without elements before the one that has them all
    x = rows_of(1, (1, 40, 16), torch.float32, 1.0, 100.0)
    none = x[:, :0].contiguous()
    part = torch.cat([tbl.tb_patch_gn_stats_cl([t], 2, tbl.new_partials(1, 1, 2)) for t in [none] * 5 + [x]])
    y, = tbl.tb_patch_gn_apply_cl([x], [torch.empty_like(x)], 2, part, 6, None, None, 1e-6)
    want, = tbl.tb_patch_gn_apply_cl([x], [torch.empty_like(x)], 2, part[5:], 1, None, None, 1e-6)
    assert torch.equal(y, want)
    check_forward([x], 2, None, None, 1e-6, True, [y])


def test_checks_and_empty_batches(tbl):
    x = rows_of(1, (1, 4, 8), torch.float32)
    part = tbl.tb_patch_gn_stats_cl([x], 2, tbl.new_partials(1, 1, 2))
    with pytest.raises(ValueError):
        tbl.tb_patch_gn_stats_cl([x], 4, part)                                       # records of another size
    with pytest.raises(ValueError):
        tbl.tb_patch_gn_stats_cl([x.transpose(1, 2)], 2, part)                       # not contiguous
    with pytest.raises(ValueError):
        tbl.patch_group_norm_cl([x, x.half()], 2, None, None, 1e-6)
    with pytest.raises(ValueError):
        tbl.patch_group_norm_cl([x], 2, torch.ones(4, device="cuda"), None, 1e-6)
    with pytest.raises(ValueError):
        tbl.patch_group_norm_cl([x], 2, None, None, 1e-6, outs=[x[:, :2]])
    with pytest.raises(ValueError):
        tbl.patch_group_norm_backward_cl([x.half()], [x], 2, part, None, None, 1e-6)
    with pytest.raises(ValueError):
        tbl.patch_group_norm_backward_cl([x], [x], 2, part, None, None, 1e-6, grad_partials=torch.empty(4, device="cuda"))
    with pytest.raises(tbl.TileBlendError):
        tbl.patch_group_norm_backward_cl([x], [x], 2, part, None, None, 1e-6, workspace=torch.empty(4, device="cuda"))
    with pytest.raises(tbl.TileBlendError):
        tbl.patch_group_norm_cl([x], 3, None, None, 1e-6)                            # 8 channels in 3 groups
    e = torch.empty(0, 4, 8, device="cuda")
    part = tbl.new_partials(1, 0, 2)
    assert tbl.patch_group_norm_cl([e], 2, None, None, 1e-6, partials=part)[0].shape == e.shape
    dxs, dg, db = tbl.patch_group_norm_backward_cl([e], [e], 2, part, None, None, 1e-6)
    assert dxs[0].shape == e.shape and (dg == 0).all() and (db == 0).all()
    e = torch.empty(2, 0, 8, device="cuda")                                          # no positions at all
    part = tbl.tb_patch_gn_stats_cl([e], 2, tbl.new_partials(1, 2, 2).fill_(-1))
    assert (part[..., 0] == 0).all()
    dxs, dg, db = tbl.patch_group_norm_backward_cl([e], [e], 2, part, None, None, 1e-6)
    assert dxs[0].shape == e.shape and (dg == 0).all() and (db == 0).all()


def test_far_means_and_an_outlier(tbl):
    # statistics about a shift: a mean a thousand deviations away, a first
    # element far from all others, a constant group.  The result's own bound: 4 u
    # of the mean move xhat by 4 u * |mean| * rstd, the sum of what is left of the
    # elements past their shift is off by 64 u of its magnitudes, the mean of
    # |x - mean|, and the variance's error is that of 64 sums, relative to itself
    x = rows_of(1, (1, 5000, 32), torch.float64)
    x[..., 8:16] += 1000.0
    x[0, 0, 16] = 1e4
    x[..., 24:] = 3.25
    x = x.float()
    part = tbl.new_partials(1, 1, 4)
    y, = tbl.patch_group_norm_cl([x], 4, None, None, 1e-6, silu=False, partials=part)
    h = f64(x).reshape(5000, 4, 8)
    mu = h.mean((0, 2), keepdims=True)
    r = 1 / np.sqrt(((h - mu) ** 2).mean((0, 2), keepdims=True) + 1e-6)
    want = ((h - mu) * r).reshape(1, 5000, 32)
    away = np.abs(h - mu).mean((0, 2), keepdims=True)
    scale = ((np.abs(mu) / 16 + away) * r + np.abs((h - mu) * r)).reshape(1, 5000, 32)
    scale[..., 24:] = 0
    check(y, want, scale)
    assert (y[..., 24:] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_values_stay_in_their_group(tbl, bad):
    x = rows_of(1, (2, 300, 16), torch.float32)
    clean, = tbl.patch_group_norm_cl([x], 4, None, None, 1e-6)
    t = x.clone()
    t[1, 123, 5] = bad
    y, = tbl.patch_group_norm_cl([t], 4, None, None, 1e-6)
    assert torch.isnan(y[1, :, 4:8]).all()
    y[1, :, 4:8] = clean[1, :, 4:8]
    assert torch.equal(y, clean)


def test_extreme_activations(tbl):
    # z far on either side of zero: silu' goes to 1 and to 0, and never to NaN
    x = rows_of(1, (1, 256, 4), torch.float32)
    gamma = torch.tensor([1.0, 500.0, -500.0, 1e-3], device="cuda")
    beta = torch.tensor([0.0, 200.0, -200.0, -90.0], device="cuda")
    part = tbl.tb_patch_gn_stats_cl([x], 1, tbl.new_partials(1, 1, 1))
    dy = rows_of(2, (1, 256, 4), torch.float32)
    dxs, dg, db = tbl.patch_group_norm_backward_cl([dy], [x], 1, part, gamma, beta, 1e-6)
    check_backward([dy], [x], 1, gamma, beta, 1e-6, True, dxs, dg, db)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape,G", [((1, 3000, 64), 8), ((2, 700, 515), 5), ((1, 40, 1300), 10)])
def test_every_element_is_counted_once(tbl, shape, G, dtype):
    # small integers: sums are exact, so one element left out or taken twice fails
    dt = DT[dtype]
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-2, 3, shape, generator=g).to(dt).cuda()
    dy = torch.randint(-2, 3, shape, generator=g).to(dt).cuda()
    N, S, C = shape
    # a forward pass whose records say mean 0 and variance 1: xhat = x
    part = torch.zeros(1, N, G, 8, 2, dtype=torch.int64, device="cuda")
    part[..., 0, 0] = S * C // G
    part.view(torch.float32)[..., 0, 3] = float(S * C // G)
    grec = tbl.new_grad_partials(1, N, C).fill_(float("nan"))
    tbl.tb_patch_gn_grad_stats_cl([dy], [x], G, part, 1, None, None, 0.0, grec, silu=False)
    assert torch.equal(grec[0, ..., 0].sum(-1), dy.float().sum(1))
    assert torch.equal(grec[0, ..., 1].sum(-1), (dy.float() * x.float()).sum(1))
    rec = tbl.tb_patch_gn_stats_cl([x], G, tbl.new_partials(1, N, G).fill_(-1))
    assert (rec[..., 0].sum(-1) == S * C // G).all()


def test_deterministic_and_in_any_order_of_calls(tbl):
    x, dy = rows_of(1, (1, 96 * 96, 64), torch.bfloat16), rows_of(2, (1, 96 * 96, 64), torch.bfloat16)
    gamma, beta = weights_of(3, 64, torch.bfloat16)
    first = None
    for _ in range(50):
        part = tbl.new_partials(1, 1, 32)
        y, = tbl.patch_group_norm_cl([x], 32, gamma, beta, 1e-6, partials=part)
        (dx,), dg, db = tbl.patch_group_norm_backward_cl([dy], [x], 32, part, gamma, beta, 1e-6)
        got = [part, y, dx, dg, db]
        if first is None:
            first = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_matches_differences(tbl, dtype):
    # the formula's gradient against differences of the oracle's forward pass
    x, v, dy = rows_of(1, (1, 60, 24), torch.float64), rows_of(2, (1, 60, 24), torch.float64), rows_of(3, (1, 60, 24),
                                                                                                       torch.float64)
    dt = DT[dtype]
    x, dy = x.to(dt), dy.to(dt)
    gamma, beta = weights_of(4, 24, dt)
    part = tbl.tb_patch_gn_stats_cl([x], 3, tbl.new_partials(1, 1, 3))
    (dx,), _, _ = tbl.patch_group_norm_backward_cl([dy], [x], 3, part, gamma, beta, 1e-6)
    h = 1e-5

    def f(s):
        return float((GN.patch_group_norm([(f64(x) + s * f64(v)).transpose(0, 2, 1)], 3, f64(gamma), f64(beta), 1e-6)[0]
                      .transpose(0, 2, 1) * f64(dy)).sum())
    want = (f(h) - f(-h)) / (2 * h)
    got = float((f64(dx) * f64(v)).sum())
    # each gradient is off by half a step of its type and 64 u; differences of h by h^2
    bound = (np.abs(f64(dx) * f64(v)) * (HALF[dt] + 64 * U)).sum() + 1e-5 + TINY[dt]
    assert abs(got - want) <= bound


def test_offsets_past_32_bits(tbl):
    # a patch of more than 2^31 elements: constant but for a few positions near its end
    S, C, G = (1 << 31) // 64 + 4096, 64, 2
    x = torch.zeros(1, S, C, dtype=torch.bfloat16, device="cuda")
    x[0, ::2] = 1.0
    x[0, 1::2] = -1.0
    x[0, -1, 5] = 40.0
    y, = tbl.patch_group_norm_cl([x], G, None, None, 0.0, silu=False)
    # mean and variance move by less than 1e-6: the step of bf16 is far wider
    assert torch.equal(y, x)
    del y
    part = tbl.tb_patch_gn_stats_cl([x], G, tbl.new_partials(1, 1, G))
    dy = torch.zeros_like(x)
    dy[0, -1, 7] = 1.0
    dy[0, 0, 40] = 2.0
    (dx,), dg, db = tbl.patch_group_norm_backward_cl([dy], [x], G, part, None, None, 0.0, silu=False)
    assert db.tolist() == [1.0 if c == 7 else 2.0 if c == 40 else 0.0 for c in range(C)]
    assert dx[0, -1, 7] == 1.0 and dx[0, 0, 40] == 2.0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 8192])
def test_the_most_channels(tbl, G, dtype):
    # one group of all of them, and a group each; the records of two patches
    dt = DT[dtype]
    xs = [rows_of(k, (1, 40 + k, 8192), dt, 1.0, 0.5) for k in (1, 2)]
    dys = [rows_of(5 + k, x.shape, dt) for k, x in enumerate(xs)]
    gamma, beta = weights_of(3, 8192, dt)
    x = torch.cat(xs, 1).double().reshape(1, -1, G, 8192 // G)
    mu = x.mean((1, 3), keepdim=True)
    rstd = 1 / (((x - mu) ** 2).mean((1, 3), keepdim=True) + 1e-6).sqrt()
    xhat = (x - mu) * rstd
    z = xhat * gamma.double().reshape(G, -1) + beta.double().reshape(G, -1)
    part = tbl.new_partials(2, 1, G)
    ys = tbl.patch_group_norm_cl(xs, G, gamma, beta, 1e-6, partials=part)
    got = torch.cat(ys, 1).double().reshape(x.shape)
    want = z * torch.sigmoid(z)
    # half a step of the output, and 64 u of z (at most 40 and of slope 1.1) and of the statistics
    assert ((got - want).abs() <= want.abs() * HALF[dt] + 64 * U * (z.abs() + 8) * 1.1).all()
    dxs, dg, db = tbl.patch_group_norm_backward_cl(dys, xs, G, part, gamma, beta, 1e-6)
    s = torch.sigmoid(z)
    dz = torch.cat(dys, 1).double().reshape(x.shape) * s * (1 + z * (1 - s))
    gam = gamma.double().reshape(G, -1)
    v = dz * gam
    dx = (v - v.mean((1, 3), keepdim=True) - xhat * (v * xhat).mean((1, 3), keepdim=True)) * rstd
    scale = rstd.max() * (v.abs() + 1 + xhat.abs()) * 8
    assert ((torch.cat(dxs, 1).double().reshape(x.shape) - dx).abs() <= dx.abs() * HALF[dt] + 64 * U * scale).all()
    for t, w, m in ((dg, (dz * xhat).sum(1), (dz * xhat).abs().sum(1)), (db, dz.sum(1), dz.abs().sum(1))):
        assert ((t.double() - w.reshape(-1)).abs() <= w.reshape(-1).abs() * HALF[dt] + 128 * U * (m.reshape(-1) + 1)).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_more_columns_than_a_cluster_takes(tbl, dtype):
    # tensors at different offsets (single elements), each CTA with all columns in turn
    dt = DT[dtype]
    shape, C, G = (1, 5, 2601), 2601, 9
    x, dy = rows_of(1, shape, dt, 1.0, 0.5), rows_of(2, shape, dt)
    gamma, beta = weights_of(3, C, dt)
    buf = torch.full((3, (x.numel() + 24) // 8 * 8), 7.0, dtype=dt, device="cuda")
    mx, md, mo = (b[a:a + x.numel()].view(shape) for a, b in zip((1, 2, 3), buf))
    mx.copy_(x)
    md.copy_(dy)
    part = tbl.new_partials(1, 1, G)
    tbl.patch_group_norm_cl([mx], G, gamma, beta, 1e-6, outs=[mo], partials=part)
    check_forward([x], G, gamma, beta, 1e-6, True, [mo])
    _, dg, db = tbl.patch_group_norm_backward_cl([md], [mx], G, part, gamma, beta, 1e-6, dxs=[mo])
    check_backward([dy], [x], G, gamma, beta, 1e-6, True, [mo], dg, db)


def test_the_two_ways_agree(tbl):
    # in one launch, and in the launches of the general path
    for shape, G in (((1, 1024, 512), 32), ((2, 500, 64), 8), ((1, 700, 37), 1)):
        for dt in (torch.float32, torch.bfloat16):
            x, dy = rows_of(1, shape, dt, 1.0, 3.0), rows_of(2, shape, dt)
            gamma, beta = weights_of(3, shape[-1], dt)
            part = tbl.new_partials(1, shape[0], G)
            y, = tbl.patch_group_norm_cl([x], G, gamma, beta, 1e-6, partials=part)
            rec = tbl.tb_patch_gn_stats_cl([x], G, tbl.new_partials(1, shape[0], G))
            w, = tbl.tb_patch_gn_apply_cl([x], [torch.empty_like(x)], G, rec, 1, gamma, beta, 1e-6)
            (dx,), dg, db = tbl.patch_group_norm_backward_cl([dy], [x], G, part, gamma, beta, 1e-6)
            grec = tbl.tb_patch_gn_grad_stats_cl([dy], [x], G, rec, 1, gamma, beta, 1e-6,
                                                 tbl.new_grad_partials(1, shape[0], shape[-1]))
            vg, vb, vx = torch.empty_like(dg), torch.empty_like(db), torch.empty_like(x)
            tbl.tb_patch_gn_grad_apply_cl([dy], [x], [vx], G, rec, grec, 1, gamma, beta, 1e-6,
                                          tbl.gn_workspace_cl(shape[0], G), vg, vb)
            # both round once what differs by fp32 arithmetic: a step apart at most, or 64 u of the values' size
            for a, b in ((y, w), (dx, vx), (dg, vg), (db, vb)):
                a, b = a.double(), b.double()
                assert ((a - b).abs() <= 2 * HALF[dt] * b.abs() + 64 * U * b.abs().max()).all()


def _pass(tbl, x, dy, gamma, beta, stream=None):
    part = tbl._on_stream(lambda: tbl.new_partials(1, 1, 4), stream)
    y = tbl.patch_group_norm_cl([x], 4, gamma, beta, 1e-6, partials=part, stream=stream)
    dxs, dg, db = tbl.patch_group_norm_backward_cl([dy], [x], 4, part, gamma, beta, 1e-6, stream=stream)
    return [*y, *dxs, dg, db]


# one that fits into shared memory, one that does not
LENGTHS = [500, 600000]


def _inputs(length, seed=0):
    bf = torch.bfloat16
    return [rows_of(seed + 1, (1, length, 16), bf), rows_of(seed + 2, (1, length, 16), bf), *weights_of(seed + 3, 16, bf)]


@pytest.mark.parametrize("length", LENGTHS)
@pytest.mark.parametrize("raw", [False, True])
def test_on_another_stream(tbl, raw, length):
    ins = _inputs(length)
    want = _pass(tbl, *ins)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(20):
        got = _pass(tbl, *ins, stream=s.cuda_stream if raw else s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("length", LENGTHS)
def test_replay_from_a_graph(tbl, length):
    ins = _inputs(length)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _pass(tbl, *ins)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = _pass(tbl, *ins)
    for seed in (100, 200):
        for t, u in zip(ins, _inputs(length, seed)):
            t.copy_(u)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, _pass(tbl, *ins)))


def test_calls_in_turn_share_a_workspace(tbl):
    # dx is launched before the constants are written: each call's are its own, not the last call's
    sets = [(rows_of(k, (1, 70000, 64), torch.bfloat16, 1.0 + k, 2.0 * k), rows_of(20 + k, (1, 70000, 64), torch.bfloat16),
             *weights_of(40 + k, 64, torch.bfloat16)) for k in range(6)]
    part, grec = [tbl.new_partials(1, 1, 8) for _ in sets], tbl.new_grad_partials(1, 1, 64)
    ws = tbl.gn_workspace_cl(1, 8)
    for p, (x, *_) in zip(part, sets):
        tbl.tb_patch_gn_stats_cl([x], 8, p)

    def backward(k):
        x, dy, gamma, beta = sets[k]
        return tbl.patch_group_norm_backward_cl([dy], [x], 8, part[k], gamma, beta, 1e-6, grad_partials=grec, workspace=ws)
    alone = []
    for k in range(len(sets)):
        ws.fill_(255)
        alone.append(backward(k))
        torch.cuda.synchronize()
    for _ in range(5):
        got = [backward(k) for k in range(len(sets))]
        for ((dx,), dg, db), ((wx,), wg, wb) in zip(got, alone):
            assert torch.equal(dx, wx) and torch.equal(dg, wg) and torch.equal(db, wb)


# [N, *spatial, C] of two patches, split axis 1: calls that fit into shared memory in every
# type.  Chunks of 8 halves (4 floats) that two groups share leave two sums where a group has
# a chunk's channels, so these have odd and small multiples of channels a group
ONE_LAUNCH = [
    (1, 515, 5, (24, 16)),      # a chunk over the end of a position; several slabs of columns
    (1, 67, 67, (40, 24)),      # a channel a group
    (2, 184, 8, (600, 18)),     # 23 channels a group, whole chunks a position
    (1, 400, 8, (300, 300)),    # 50 channels a group, the groups split among clusters
    (2, 400, 8, (200, 50)),
    (2, 1200, 8, (90, 31)),     # 150
    (1, 37, 1, (1312, 8)),      # both sums of a chunk over a position's end are one group's
    (2, 36, 4, (50, 30)),       # 9
    (4, 88, 8, (40, 41)),       # 11
    (2, 9, 1, (8, 72)),         # a position of a chunk and an element
    (3, 1029, 7, (8, 16)),      # 147 channels, a period of more than a thousand chunks in halves
    (1, 24, 2, (40, 41)),       # 12: a sum for every four
]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,C,G,sizes", ONE_LAUNCH, ids=lambda v: str(v))
def test_one_launch_of_every_kind_of_group(tbl, N, C, G, sizes, dtype, silu):
    dt = DT[dtype]
    x = rows_of(C, (N, sum(sizes), C), torch.float64, 1.5)
    xs = [(p + m).to(dt).contiguous() for p, m in zip(x.split(sizes, 1), (-2.0, 1.0))]
    dys = [p.contiguous() for p in rows_of(7, x.shape, dt, 0.5).split(sizes, 1)]
    gamma, beta = weights_of(8, C, dt)
    part = tbl.new_partials(2, N, G).fill_(-1)
    outs = tbl.patch_group_norm_cl(xs, G, gamma, beta, 1e-6, silu, partials=part)
    check_forward(xs, G, gamma, beta, 1e-6, silu, outs)
    # one launch leaves one record of the patches together
    assert (part[0, ..., 0, 0] == sum(sizes) * (C // G)).all() and (part[1] == 0).all() and (part[0, ..., 1:, :] == 0).all()
    grec = tbl.new_grad_partials(2, N, C).fill_(float("nan"))
    dxs, dg, db = tbl.patch_group_norm_backward_cl(dys, xs, G, part, gamma, beta, 1e-6, silu, grad_partials=grec)
    check_backward(dys, xs, G, gamma, beta, 1e-6, silu, dxs, dg, db)
    # and uses no records of the gradients, or one a sample
    assert grec.isnan().all() if N == 1 else (grec[1] == 0).all() and (grec[0, ..., 1:, :] == 0).all()


def _general(tbl, x, dy, G, gamma, beta):
    N, C = x.shape[0], x.shape[-1]
    rec = tbl.tb_patch_gn_stats_cl([x], G, tbl.new_partials(1, N, G))
    y, = tbl.tb_patch_gn_apply_cl([x], [torch.empty_like(x)], G, rec, 1, gamma, beta, 1e-6)
    grec = tbl.tb_patch_gn_grad_stats_cl([dy], [x], G, rec, 1, gamma, beta, 1e-6, tbl.new_grad_partials(1, N, C))
    dg, db, dx = torch.empty_like(gamma), torch.empty_like(gamma), torch.empty_like(x)
    tbl.tb_patch_gn_grad_apply_cl([dy], [x], [dx], G, rec, grec, 1, gamma, beta, 1e-6, tbl.gn_workspace_cl(N, G), dg, db)
    return rec, y, dx, dg, db


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape,G", [((1, 4000, 400), 8), ((2, 1500, 1200), 8), ((1, 900, 880), 16)])
def test_split_channels_with_chunks_of_two_groups(tbl, shape, G, dtype):
    # the launches of the general path, their statistics split by channels
    dt = DT[dtype]
    x, dy = rows_of(1, shape, dt, 1.5, 0.5), rows_of(2, shape, dt, 0.5)
    gamma, beta = weights_of(3, shape[-1], dt)
    rec, y, dx, dg, db = _general(tbl, x, dy, G, gamma, beta)
    assert (rec[..., 0].sum(-1) == shape[1] * (shape[2] // G)).all()
    check_forward([x], G, gamma, beta, 1e-6, True, [y])
    check_backward([dy], [x], G, gamma, beta, 1e-6, True, [dx], dg, db)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape,G", [((1, 704, 37), 1), ((1, 1312, 37), 1), ((2, 600, 184), 8), ((1, 600, 400), 8)])
def test_one_launch_and_several_agree(tbl, shape, G, dtype):
    dt = DT[dtype]
    x, dy = rows_of(1, shape, dt, 1.0, 3.0), rows_of(2, shape, dt)
    gamma, beta = weights_of(3, shape[-1], dt)
    part = tbl.new_partials(1, shape[0], G)
    y, = tbl.patch_group_norm_cl([x], G, gamma, beta, 1e-6, partials=part)
    grec = tbl.new_grad_partials(1, shape[0], shape[-1]).fill_(float("nan"))
    (dx,), dg, db = tbl.patch_group_norm_backward_cl([dy], [x], G, part, gamma, beta, 1e-6, grad_partials=grec)
    rec, *several = _general(tbl, x, dy, G, gamma, beta)
    # two ways: one record, and one from each of several clusters
    assert (part[..., 1:, 0] == 0).all() and (rec[..., 1, 0] > 0).all()
    assert grec.isnan().all() if shape[0] == 1 else (grec[..., 1:, :] == 0).all()
    # both round once what differs by fp32 arithmetic: a step apart at most, or 64 u of the values' size
    for a, b in zip((y, dx, dg, db), several):
        a, b = a.double(), b.double()
        assert ((a - b).abs() <= 2 * HALF[dt] * b.abs() + 64 * U * b.abs().max()).all()


def _ranks(tbl, xs, dys, gamma, beta, G=4):
    """The four separate calls of a rank with the first two patches and of one with the
    others, and the records of both gathered: R > P."""
    N, C = xs[0].shape[0], xs[0].shape[-1]
    ranks = [(xs[:2], dys[:2]), (xs[2:], dys[2:])]
    R = len(xs)
    rec = torch.cat([tbl.tb_patch_gn_stats_cl(x, G, tbl.new_partials(len(x), N, G)) for x, _ in ranks])
    ys = [y for x, _ in ranks
          for y in tbl.tb_patch_gn_apply_cl(x, [torch.empty_like(t) for t in x], G, rec, R, gamma, beta, 1e-6)]
    grec = torch.cat([tbl.tb_patch_gn_grad_stats_cl(d, x, G, rec, R, gamma, beta, 1e-6, tbl.new_grad_partials(len(x), N, C))
                      for x, d in ranks])
    ws, dxs, weights = tbl.gn_workspace_cl(N, G), [], []
    for x, d in ranks:
        dg, db = torch.empty_like(gamma), torch.empty_like(beta)
        dxs += tbl.tb_patch_gn_grad_apply_cl(d, x, [torch.empty_like(t) for t in x], G, rec, grec, R, gamma, beta, 1e-6,
                                             ws, dg, db)
        weights += [dg, db]
    return ys, dxs, weights


def _rank_inputs(seed, C=24):
    x, dy = rows_of(seed, (2, 400, C), torch.bfloat16, 1.5, 0.5), rows_of(seed + 1, (2, 400, C), torch.bfloat16)
    cut = [101, 99, 150, 50]
    return ([p.contiguous() for p in x.split(cut, 1)], [p.contiguous() for p in dy.split(cut, 1)],
            *weights_of(seed + 2, C, torch.bfloat16))


def test_separate_calls_replay_from_a_graph(tbl):
    ins = _rank_inputs(1)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _ranks(tbl, *ins)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ys, dxs, weights = _ranks(tbl, *ins)
    for seed in (100, 200, 300):
        xs, dys, gamma, beta = ins
        for t, u in zip([*xs, *dys, gamma, beta], (lambda a, b, c, d: [*a, *b, c, d])(*_rank_inputs(seed))):
            t.copy_(u)
        g.replay()
        torch.cuda.synchronize()
        check_forward(xs, 4, gamma, beta, 1e-6, True, ys)
        check_backward(dys, xs, 4, gamma, beta, 1e-6, True, dxs, *weights[:2])
        want = _ranks(tbl, *ins)
        assert all(torch.equal(a, b) for a, b in zip([*ys, *dxs, *weights], [t for ts in want for t in ts]))
