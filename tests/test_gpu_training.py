"""GPU parity of the training calls against the float64 oracle.

Tolerances, per element, from the arithmetic (u = 2^-24, one fp32 rounding):

* every output is rounded once into its type: half a unit in the last place,
  |v| * HALF[type], plus half the type's smallest subnormal;
* before that, fp32 arithmetic: K * u times the sum of the magnitudes that were
  added or cancelled to make the value (``scale`` below, each from the formula).
  A sum of m terms in any order is off by at most (m - 1) * u times the sum of
  their magnitudes; the row sums are split over at least 32 threads and then
  joined pairwise, so K = 64 covers rows of up to 2048 elements in full and is
  never reached by rounding errors of random sign in longer ones.  Column sums
  (dgamma, dbeta) get their full bound, K = rows + 8;
* SiLU's exponential and reciprocal are approximate to 2^-22 each: K = 64 covers
  them as well.
"""
import numpy as np
import pytest
import torch

from oracle import training as T

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
K = 64


@pytest.fixture(scope="module")
def tbl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import tileblend
    return tileblend


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def check(got, want, scale, k=K):
    """|got - want| within the rounding of got's type and k * u * scale."""
    g = f64(got)
    assert g.shape == want.shape
    tol = np.abs(want) * HALF[got.dtype] + TINY[got.dtype] + k * U * scale
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), "%d of %d off, worst %.3g of the bound" % (
        bad.sum(), bad.size, float(np.nanmax(np.abs(g - want) / tol)))


def check_ln(x, gamma, beta, eps, y, mean, rstd, total=None, residual=None):
    h = f64(x)
    if residual is not None:
        s = (x.float() + residual.float()).to(x.dtype)   # one fp32 add, one rounding
        assert torch.equal(total.cpu(), s.cpu())
        h = f64(s)
    h = h.reshape(-1, h.shape[-1])
    wy, wm, wr = T.layer_norm(h, f64(gamma), f64(beta), eps)
    mag = np.abs(h).mean(1)
    if mean is not None:
        check(mean.reshape(-1), wm, mag)
    # the mean's error enters the variance squared: it moves it by
    # (mean error / deviation)^2, relatively
    shift = (K * U * mag * wr) ** 2
    if rstd is not None:
        check(rstd.reshape(-1), wr, wr * (1 + shift / U))
    g = np.ones(h.shape[1]) if gamma is None else np.abs(f64(gamma))
    b = np.zeros(h.shape[1]) if beta is None else np.abs(f64(beta))
    scale = (np.abs(h) + mag[:, None]) * wr[:, None] * g * (1 + shift[:, None] / U) + b
    check(y.reshape(-1, h.shape[1]), wy, scale)


def check_ln_bwd(dy, x, mean, rstd, gamma, dtotal, dx, dgamma, dbeta):
    cols = x.shape[-1]
    d, h = f64(dy).reshape(-1, cols), f64(x).reshape(-1, cols)
    m, r = f64(mean).reshape(-1), f64(rstd).reshape(-1)
    t = None if dtotal is None else f64(dtotal).reshape(-1, cols)
    wdx, wdg, wdb = T.layer_norm_backward(d, h, m, r, f64(gamma), t)
    xh = (np.abs(h) + np.abs(m)[:, None]) * r[:, None]
    g = np.abs(d) * (1 if gamma is None else np.abs(f64(gamma)))
    if dx is not None:
        scale = r[:, None] * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True))
        check(dx.reshape(-1, cols), wdx, scale + (0 if t is None else np.abs(t)))
    rows = d.shape[0]
    if dgamma is not None:
        check(dgamma, wdg, (np.abs(d) * xh).sum(0), rows + 8)
    if dbeta is not None:
        check(dbeta, wdb, np.abs(d).sum(0), rows + 8)


def rows_of(seed, shape, dtype, scale=1.0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale + offset).to(dtype).cuda()


def weights_of(seed, cols, dtype):
    return rows_of(seed, (cols,), dtype, 0.3, 1.0), rows_of(seed + 1, (cols,), dtype, 0.3)


def run_ln(tbl, x, gamma, beta, eps, dy, residual=None, dtotal=None):
    """Forward and backward through the allocating entry points, checked."""
    out = tbl.layer_norm(x, gamma, beta, eps, residual)
    y, mean, rstd = out[:3]
    total = out[3] if residual is not None else None
    check_ln(x, gamma, beta, eps, y, mean, rstd, total, residual)
    h = x if total is None else total
    dx, dgamma, dbeta = tbl.layer_norm_backward(dy, h, mean, rstd, gamma, dtotal)
    check_ln_bwd(dy, h, mean, rstd, gamma, dtotal, dx, dgamma, dbeta)


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------

COLS = [1, 2, 3, 7, 8, 31, 64, 100, 129, 256, 257, 512, 520, 777, 1000, 1024, 1111, 2048, 2056, 4096, 4104, 4111, 8192,
        8200, 8197, 16384]


@pytest.mark.parametrize("wide", [False, True], ids=["w", "w32"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", COLS)
def test_layer_norm_widths(tbl, cols, dtype, wide):
    dt = DT[dtype]
    wt = torch.float32 if wide else dt
    rows = 37 if cols < 4096 else 5
    gamma, beta = weights_of(cols, cols, wt)
    x, dy = rows_of(1, (rows, cols), dt, 1.0, 0.3), rows_of(2, (rows, cols), dt, 0.5)
    run_ln(tbl, x, gamma, beta, 1e-5, dy)
    run_ln(tbl, x, gamma, beta, 1e-5, dy, residual=rows_of(3, (rows, cols), dt), dtotal=rows_of(4, (rows, cols), dt))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [16392, 33000, 32768, 40001, 70000])
def test_layer_norm_rows_longer_than_a_cta_holds(tbl, cols, dtype):
    dt = DT[dtype]
    gamma, beta = weights_of(cols, cols, torch.float32)
    for rows in (1, 3):
        x, dy = rows_of(1, (rows, cols), dt, 1.0, -0.2), rows_of(2, (rows, cols), dt)
        run_ln(tbl, x, gamma, beta, 1e-6, dy, residual=rows_of(3, (rows, cols), dt), dtotal=rows_of(4, (rows, cols), dt))
        run_ln(tbl, x, None, None, 1e-6, dy)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [1, 2, 3, 8, 31, 300, 2000, 5003])
@pytest.mark.parametrize("cols", [40, 129, 512, 1024])
def test_layer_norm_row_counts(tbl, rows, cols, dtype):
    dt = DT[dtype]
    gamma, beta = weights_of(rows, cols, dt)
    run_ln(tbl, rows_of(1, (rows, cols), dt), gamma, beta, 1e-6, rows_of(2, (rows, cols), dt, 0.1))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [1, 5, 33, 130, 30001])
@pytest.mark.parametrize("cols", [4, 16, 33, 63, 65, 72, 127, 128, 200])
def test_layer_norm_short_rows(tbl, cols, rows, dtype):
    # several rows to a warp: warps whose last rows are missing, lanes without a column
    dt = DT[dtype]
    gamma, beta = weights_of(7, cols, dt)
    x, dy = rows_of(1, (rows, cols), dt, 1.0, 0.2), rows_of(2, (rows, cols), dt, 0.3)
    run_ln(tbl, x, gamma, beta, 1e-5, dy, residual=rows_of(3, (rows, cols), dt), dtotal=rows_of(4, (rows, cols), dt))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [5001, 8192, 8191, 12008, 12001, 16384, 16383])
def test_layer_norm_wide_rows_many_to_a_cta(tbl, cols, dtype):
    # every row buffer of the backward kernel is filled and read several times
    dt = DT[dtype]
    if dtype == "f32":
        cols = (cols + 1) // 2
    rows = 1001
    gamma, beta = weights_of(6, cols, dt)
    x, dy = rows_of(1, (rows, cols), dt, 1.0, 0.1), rows_of(2, (rows, cols), dt, 0.1)
    run_ln(tbl, x, gamma, beta, 1e-6, dy)
    run_ln(tbl, x, gamma, beta, 1e-6, dy, dtotal=rows_of(3, (rows, cols), dt))


@pytest.mark.parametrize("dtype", list(DT))
def test_layer_norm_more_long_rows_than_ctas(tbl, dtype):
    # the long-row kernels loop over rows, the weight gradients add up in each
    # CTA's own slice; more rows than workspace parts
    dt = DT[dtype]
    rows, cols = 700, 16400 if dtype != "f32" else 8208
    gamma, beta = weights_of(5, cols, dt)
    run_ln(tbl, rows_of(1, (rows, cols), dt), gamma, beta, 1e-6, rows_of(2, (rows, cols), dt, 0.1))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [64, 100, 2048])
def test_layer_norm_strided_and_misaligned_rows(tbl, cols, dtype):
    dt = DT[dtype]
    gamma, beta = weights_of(3, cols, dt)
    n = 9
    wide = rows_of(1, (n, 3 * cols + 5), dt)
    for at in (0, 1, 3, 8, cols):   # slices of wider rows: any stride, any alignment
        x = wide[:, at:at + cols]
        dy = rows_of(2, (n, cols + 16), dt)[:, 8:8 + cols]
        y = torch.full((n, cols + 7), 3.0, dtype=dt, device="cuda")
        stats = torch.empty(2, n, device="cuda")
        tbl.tb_layer_norm(x, y[:, 2:2 + cols], gamma, beta, 1e-6, stats[0], stats[1])
        check_ln(x, gamma, beta, 1e-6, y[:, 2:2 + cols], stats[0], stats[1])
        assert (y[:, :2] == 3.0).all() and (y[:, 2 + cols:] == 3.0).all()
        dx = torch.full((n, cols + 8), 5.0, dtype=dt, device="cuda")
        dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
        tbl.tb_layer_norm_backward(dy, x, stats[0], stats[1], gamma, dx[:, 8:], dg, db, tbl.ln_workspace(n, cols))
        check_ln_bwd(dy, x, stats[0], stats[1], gamma, None, dx[:, 8:], dg, db)
        assert (dx[:, :8] == 5.0).all()
    # misaligned weights with aligned rows
    g2 = torch.zeros(cols + 1, dtype=dt, device="cuda")[1:]
    g2.copy_(gamma)
    run_ln(tbl, wide[:, :cols].contiguous(), g2, beta, 1e-6, rows_of(4, (n, cols), dt))


def test_layer_norm_batched_shapes_and_refused_layouts(tbl):
    x = rows_of(1, (2, 3, 4, 64), torch.bfloat16)
    gamma, beta = weights_of(2, 64, torch.bfloat16)
    y, mean, rstd = tbl.layer_norm(x, gamma, beta, 1e-6)
    assert y.shape == x.shape and mean.shape == x.shape[:-1]
    check_ln(x, gamma, beta, 1e-6, y, mean, rstd)
    z = rows_of(1, (2, 3, 4, 128), torch.bfloat16)[..., 64:]      # one row stride over all axes
    y, mean, rstd = tbl.layer_norm(z, gamma, beta, 1e-6)
    check_ln(z, gamma, beta, 1e-6, y, mean, rstd)
    out = torch.empty(2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (x.transpose(1, 2), x[:, :, :3], x[..., ::2], rows_of(1, (64, 2), torch.bfloat16).t(),
                rows_of(1, (1, 64), torch.bfloat16).expand(2, 64)):
        with pytest.raises(ValueError):
            tbl.tb_layer_norm(bad, torch.empty(bad.shape, dtype=bad.dtype, device="cuda"), None, None, 1e-6)
    with pytest.raises(ValueError):
        tbl.tb_layer_norm(out, out, gamma[:32], None, 1e-6)
    with pytest.raises(ValueError):
        tbl.tb_layer_norm(out, out.float(), None, None, 1e-6)
    with pytest.raises(ValueError):
        tbl.tb_layer_norm(out, out, gamma.half(), None, 1e-6)
    with pytest.raises(ValueError):
        tbl.tb_layer_norm(out, out, gamma, beta.float(), 1e-6)
    with pytest.raises(ValueError):
        tbl.tb_layer_norm(out, out, None, None, 1e-6, residual=out)
    with pytest.raises(ValueError):
        tbl.tb_layer_norm(out, out, None, None, 1e-6, mean=torch.empty(3, device="cuda"))
    with pytest.raises(tbl.TileBlendError) as e:
        tbl.tb_layer_norm(out, out, None, None, -1.0)
    assert e.value.status == tbl.TB_ERR_SHAPE
    with pytest.raises(tbl.TileBlendError) as e:
        tbl.tb_layer_norm_backward(out, out, torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), gamma, out,
                                   torch.empty_like(gamma), None, tbl.ln_workspace(1, 64))
    assert e.value.status == tbl.TB_ERR_SHAPE


@pytest.mark.parametrize("dtype", list(DT))
def test_layer_norm_in_place(tbl, dtype):
    dt = DT[dtype]
    for cols in (64, 1000, 40000):
        gamma, beta = weights_of(1, cols, dt)
        x, r = rows_of(2, (6, cols), dt), rows_of(3, (6, cols), dt)
        want = tbl.layer_norm(x, gamma, beta, 1e-6)[0]
        a = x.clone()
        tbl.tb_layer_norm(a, a, gamma, beta, 1e-6)
        assert torch.equal(a, want)
        y, mean, rstd, total = tbl.layer_norm(x, gamma, beta, 1e-6, r)
        for into in (0, 1):      # the sum over x, or over the residual
            ab = [x.clone(), r.clone()]
            y2 = torch.empty_like(x)
            tbl.tb_layer_norm(ab[0], y2, gamma, beta, 1e-6, residual=ab[1], total=ab[into])
            assert torch.equal(y2, y) and torch.equal(ab[into], total)
        dy, dt_ = rows_of(4, (6, cols), dt), rows_of(5, (6, cols), dt)
        dx, dg, db = tbl.layer_norm_backward(dy, total, mean, rstd, gamma, dt_)
        for which in range(3):   # dx over dy, over x, over dtotal
            t = [dy.clone(), total.clone(), dt_.clone()]
            g2, b2 = torch.empty_like(dg), torch.empty_like(db)
            tbl.tb_layer_norm_backward(t[0], t[1], mean, rstd, gamma, t[which], g2, b2, tbl.ln_workspace(6, cols),
                                       dtotal=t[2])
            assert torch.equal(t[which], dx) and torch.equal(g2, dg) and torch.equal(b2, db)


@pytest.mark.parametrize("cols", [96, 1000, 50000])
def test_layer_norm_backward_parts_on_their_own(tbl, cols):
    x, dy = rows_of(1, (20, cols), torch.bfloat16), rows_of(2, (20, cols), torch.bfloat16)
    gamma, beta = weights_of(3, cols, torch.float32)
    _, mean, rstd = tbl.layer_norm(x, gamma, beta, 1e-6)
    dx, dg, db = tbl.layer_norm_backward(dy, x, mean, rstd, gamma)
    a = torch.empty_like(dx)
    tbl.tb_layer_norm_backward(dy, x, mean, rstd, gamma, a, None, None, None)
    assert torch.equal(a, dx)
    g2, b2 = torch.full_like(dg, 9.0), torch.full_like(db, 9.0)
    ws = tbl.ln_workspace(20, cols)
    tbl.tb_layer_norm_backward(dy, x, mean, rstd, gamma, None, g2, None, ws)
    tbl.tb_layer_norm_backward(dy, x, mean, rstd, gamma, None, None, b2, ws)
    assert torch.equal(g2, dg) and torch.equal(b2, db)


def test_layer_norm_empty_batches(tbl):
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gamma, beta = weights_of(1, 64, torch.bfloat16)
    y, mean, rstd = tbl.layer_norm(e, gamma, beta, 1e-6)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dg, db = tbl.layer_norm_backward(e, e, mean, rstd, gamma)
    assert dx.shape == (0, 64) and (dg == 0).all() and (db == 0).all()


def test_layer_norm_hard_rows(tbl):
    cols = 1000
    gamma, beta = weights_of(1, cols, torch.float32)
    rows = rows_of(2, (8, cols), torch.float32)
    rows[0] = 7.25                      # no variance: y = beta
    rows[1] += 1.0e4                    # a large offset
    rows[2, 0] = 1.0e5                  # one outlier
    rows[3] *= 1e-12                    # variance far below eps
    rows[4] *= 1e15
    rows[5, 17] = float("nan")
    rows[6, 3] = float("inf")
    y, mean, rstd = tbl.layer_norm(rows, gamma, beta, 1e-5)
    keep = [0, 1, 2, 3, 4, 7]
    check_ln(rows[keep], gamma, beta, 1e-5, y[keep], mean[keep], rstd[keep])
    assert torch.equal(y[0], beta)
    assert torch.isnan(y[5]).all() and torch.isnan(y[6]).all()
    # the largest f16 values
    h = torch.full((2, 512), 65504.0, dtype=torch.float16, device="cuda")
    h[:, ::2] = -65504.0
    y, mean, rstd = tbl.layer_norm(h, None, None, 0.0)
    check_ln(h, None, None, 0.0, y, mean, rstd)


@pytest.mark.parametrize("cols", [512, 1023])
def test_layer_norm_guard_bands(tbl, cols):
    rows, guard, dt = 41, 512, torch.bfloat16
    gamma, beta = weights_of(1, cols, dt)
    x, dy = rows_of(2, (rows, cols), dt), rows_of(3, (rows, cols), dt)

    def banded(n, dtype, value=7.0):
        buf = torch.full((n + 2 * guard,), value, dtype=dtype, device="cuda")
        return buf, buf[guard:guard + n]
    bufs = [banded(rows * cols, dt), banded(rows, torch.float32), banded(rows, torch.float32), banded(rows * cols, dt),
            banded(cols, dt), banded(cols, dt), banded(tbl._lib.tb_layer_norm_workspace(rows, cols) // 4, torch.float32)]
    y, mean, rstd, dx, dg, db, ws = (b[1] for b in bufs)
    keep = x.clone(), dy.clone()
    tbl.tb_layer_norm(x, y.view(rows, cols), gamma, beta, 1e-6, mean, rstd)
    tbl.tb_layer_norm_backward(dy, x, mean, rstd, gamma, dx.view(rows, cols), dg, db, ws)
    torch.cuda.synchronize()
    for buf, v in bufs:
        assert (buf[:guard] == 7.0).all() and (buf[guard + v.numel():] == 7.0).all()
    assert torch.equal(x, keep[0]) and torch.equal(dy, keep[1])
    check_ln_bwd(dy, x, mean, rstd, gamma, None, dx.view(rows, cols), dg, db)


def test_layer_norm_is_deterministic(tbl):
    x, dy = rows_of(1, (4000, 512), torch.bfloat16), rows_of(2, (4000, 512), torch.bfloat16)
    gamma, beta = weights_of(3, 512, torch.float32)
    _, mean, rstd = tbl.layer_norm(x, gamma, beta, 1e-6)
    a = tbl.layer_norm_backward(dy, x, mean, rstd, gamma)
    for _ in range(3):
        b = tbl.layer_norm_backward(dy, x, mean, rstd, gamma)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_layer_norm_offsets_past_32_bits(tbl):
    ld, rows, cols = 1 << 20, 2100, 256     # row offsets past 2^31 elements
    big = torch.empty(rows, ld, dtype=torch.float16, device="cuda")
    x = big[:, 64:64 + cols]
    x.copy_(rows_of(1, (rows, cols), torch.float16))
    gamma, beta = weights_of(2, cols, torch.float16)
    y, mean, rstd = tbl.layer_norm(x, gamma, beta, 1e-6)
    check_ln(x, gamma, beta, 1e-6, y, mean, rstd)
    dy = rows_of(3, (rows, cols), torch.float16)
    dx = big[:, 1024:1024 + cols]
    tbl.tb_layer_norm_backward(dy, x, mean, rstd, gamma, dx, None, None, None)
    check_ln_bwd(dy, x, mean, rstd, gamma, None, dx, None, None)


def test_layer_norm_gradient_matches_differences(tbl):
    # d/dt of sum(w * LN(x + t v)) by central differences of the 64-bit oracle
    x, w, v = (rows_of(s, (6, 96), torch.float32) for s in (1, 2, 3))
    gamma, beta = weights_of(4, 96, torch.float32)
    _, mean, rstd = tbl.layer_norm(x, gamma, beta, 1e-5)
    dx, dg, db = tbl.layer_norm_backward(w, x, mean, rstd, gamma)
    h = 1e-6

    def loss(t=0.0, tg=0.0, tb=0.0):
        y, _, _ = T.layer_norm(f64(x) + t * f64(v), f64(gamma) + tg * f64(v)[0], f64(beta) + tb * f64(v)[0], 1e-5)
        return float((y * f64(w)).sum())
    for kw, grad, along in (("t", dx, f64(v)), ("tg", dg, f64(v)[0]), ("tb", db, f64(v)[0])):
        diff = (loss(**{kw: h}) - loss(**{kw: -h})) / (2 * h)
        terms = f64(grad) * along
        # fp32 gradients: 1e-5 of the terms' magnitudes, far above their rounding and the differences' error
        assert abs(diff - terms.sum()) <= 1e-5 * np.abs(terms).sum()


# --------------------------------------------------------------------------
# gradient norm and clip
# --------------------------------------------------------------------------

def run_clip(tbl, grads, max_norm, outs=None):
    keep = [f64(g) for g in grads]
    table = tbl.GradTable(grads, outs)
    norm = tbl.clip_grad_norm(table, max_norm)
    want = T.grad_norm(keep)
    # 36 fp32 roundings in a thread's sum of squares, halved by the root, and the last one
    assert abs(float(norm) - want) <= 20 * U * want
    c = T.clip_factor(want, max_norm)
    for o, k in zip(table.outs, keep):
        check(o.reshape(-1), k.reshape(-1) * c, np.abs(k.reshape(-1) * c), 24)
    return norm


CLIP_SETS = {
    "one": [1],
    "tiny": [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 31, 33],
    "empty_among": [0, 100, 0, 0, 4097, 0],
    "piece_edges": [8191, 8192, 8193, 16384, 4096, 4095, 24577],
    "ragged": [1000003, 17, 65536, 12345, 777],
}


@pytest.mark.parametrize("dtype", list(DT) + ["mixed"])
@pytest.mark.parametrize("name", list(CLIP_SETS))
def test_clip_sets(tbl, name, dtype):
    kinds = list(DT.values())
    grads = [rows_of(k, (n,), kinds[k % 3] if dtype == "mixed" else DT[dtype], 0.1 * (k + 1))
             for k, n in enumerate(CLIP_SETS[name])]
    for max_norm in (0.01, 1e6, 0.0, float("inf")):
        outs = [torch.full_like(g, 7.0) for g in grads]
        before = [g.clone() for g in grads]
        run_clip(tbl, grads, max_norm, outs)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
        if max_norm >= 1e6:
            assert all(torch.equal(a, b) for a, b in zip(grads, outs))
        run_clip(tbl, [g.clone() for g in grads], max_norm)       # in place


@pytest.mark.parametrize("dtype", list(DT))
def test_clip_views_of_flat_buffers(tbl, dtype):
    # views at every element offset; outputs that share the alignment, and ones that do not
    dt = DT[dtype]
    sizes = [1, 3, 5, 1000, 4099, 64, 20000, 7, 9]
    flat = rows_of(1, (sum(sizes),), dt)
    views = list(flat.split(sizes))
    for shift in (0, 1, 3):
        buf = torch.full((sum(sizes) + 16,), 7.0, dtype=dt, device="cuda")
        outs = list(buf[shift:shift + sum(sizes)].split(sizes))
        run_clip(tbl, views, 0.5, outs)
        assert (buf[:shift] == 7.0).all() and (buf[shift + sum(sizes):] == 7.0).all()
    # in place, with canaries around
    buf = torch.full((sum(sizes) + 10,), 7.0, dtype=dt, device="cuda")
    buf[5:5 + sum(sizes)] = flat
    run_clip(tbl, list(buf[5:5 + sum(sizes)].split(sizes)), 0.5)
    assert (buf[:5] == 7.0).all() and (buf[5 + sum(sizes):] == 7.0).all()


@pytest.mark.parametrize("count", [64, 65, 1024, 1025, 2500])
def test_clip_many_tensors(tbl, count):
    g = torch.Generator().manual_seed(count)
    sizes = torch.randint(0, 300, (count,), generator=g).tolist()
    kinds = list(DT.values())
    run_clip(tbl, [rows_of(k, (n,), kinds[k % 3]) for k, n in enumerate(sizes)], 1.0)


def test_clip_of_nothing(tbl):
    assert float(tbl.clip_grad_norm([], 1.0)) == 0.0
    assert float(tbl.clip_grad_norm([torch.empty(0, device="cuda")], 1.0)) == 0.0


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e10, 1e19, 1e30, 1e36])
def test_clip_values_whose_squares_leave_fp32(tbl, scale):
    grads = [rows_of(1, (5000,), torch.float32, scale), rows_of(2, (77,), torch.bfloat16, scale)]
    table = tbl.GradTable(grads)
    records = tbl.new_grad_records(2)
    norm = torch.empty(1, device="cuda")
    tbl.tb_grad_norm(tbl.tb_grad_stats(table, records), norm)
    want = T.grad_norm([f64(g) for g in grads])
    # a norm below fp32's normal range is rounded to a multiple of 2^-149
    assert abs(float(norm) - want) <= 20 * U * want + 2.0 ** -149
    if scale >= 1e10:
        run_clip(tbl, grads, 1.0)


def test_clip_of_infinite_and_nan_gradients(tbl):
    a, b = rows_of(1, (100,), torch.float32), rows_of(2, (100,), torch.bfloat16)
    a[3] = float("inf")
    norm = tbl.clip_grad_norm([a, b], 1.0)
    assert torch.isinf(norm).all()
    assert torch.isnan(a[3]) and (a[:3] == 0).all() and (b == 0).all()
    b[5] = float("nan")
    norm = tbl.clip_grad_norm([b, a[:3]], 1.0)
    assert torch.isnan(norm).all() and torch.isnan(b).all()


def test_clip_records_of_several_calls_join(tbl):
    # two ranks' gradients: each writes its records, all of them give both clips
    ranks = [[rows_of(1, (1000,), torch.float32), rows_of(2, (333,), torch.bfloat16)],
             [rows_of(3, (77777,), torch.float16, 3.0)]]
    tables = [tbl.GradTable(g, [torch.empty_like(t) for t in g]) for g in ranks]
    sets = [tbl.tb_grad_stats(t, tbl.new_grad_records(len(t))) for t in tables]
    every = torch.cat(sets)
    want = T.grad_norm([f64(g) for r in ranks for g in r])
    for t in tables:
        norm = torch.empty(1, device="cuda")
        tbl.tb_grad_clip(t, every, 2.0, norm)
        assert abs(float(norm) - want) <= 20 * U * want
        for g, o in zip(t.grads, t.outs):
            w = f64(g) * T.clip_factor(want, 2.0)
            check(o, w, np.abs(w), 24)


def test_clip_is_deterministic_and_checks_its_arguments(tbl):
    grads = [rows_of(k, (50000 + k,), torch.bfloat16) for k in range(20)]
    table = tbl.GradTable(grads, [torch.empty_like(g) for g in grads])
    norms = [tbl.clip_grad_norm(table, 1.0).item() for _ in range(4)]
    assert len(set(norms)) == 1
    with pytest.raises(ValueError):
        tbl.GradTable(grads, grads[:3])
    with pytest.raises(ValueError):
        tbl.GradTable([grads[0][::2]])
    with pytest.raises(ValueError):
        tbl.GradTable([grads[0]], [grads[0].float()])
    with pytest.raises(ValueError):
        tbl.tb_grad_stats(table, torch.empty(3, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        tbl.tb_grad_stats(table, torch.empty(tbl.TB_GRAD_PARTS, device="cuda"))
    with pytest.raises(tbl.TileBlendError):
        tbl.clip_grad_norm(table, -1.0)
    with pytest.raises(TypeError):
        tbl.GradTable([torch.zeros(4, dtype=torch.int32, device="cuda")])


def test_clip_tensor_past_32_bits(tbl):
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 5, n // 2, (1 << 31) - 1, 1 << 31, n - 1], device="cuda")
    g[at] = 3.0
    norm = tbl.clip_grad_norm([g], 1.0)
    assert abs(float(norm) - np.sqrt(54.0)) <= 20 * U * np.sqrt(54.0)
    assert int((g != 0).sum()) == at.numel()
    want = 3.0 / (np.sqrt(54.0) + 1e-6)
    assert (g[at].double() - want).abs().max().item() <= want * 2.0 ** -8


# --------------------------------------------------------------------------
# PatchGroupNorm backward
# --------------------------------------------------------------------------

def check_gn(dys, xs, G, gamma, beta, eps, silu, dxs, dgamma, dbeta, rel=0.0):
    """``rel``: the statistics' own relative error (2e-5 at most, tested with
    the forward pass)."""
    hx, hd = [f64(t) for t in xs], [f64(t) for t in dys]
    N, C = hx[0].shape[:2]
    cg = C // G
    want, wg, wb = T.group_norm_backward(hd, hx, G, f64(gamma), f64(beta), eps, silu)
    gam = np.ones(C) if gamma is None else np.abs(f64(gamma))
    bet = np.zeros(C) if beta is None else np.abs(f64(beta))
    sg, sb = np.zeros(C), np.zeros(C)
    scales = [np.zeros(x.shape) for x in hx]
    for n in range(N):
        for g in range(G):
            ch = slice(g * cg, (g + 1) * cg)
            flat = np.concatenate([x[n, ch].reshape(cg, -1) for x in hx], 1)
            mu = flat.mean()
            r = 1.0 / np.sqrt(((flat - mu) ** 2).mean() + eps)
            ga, be = gam[ch, None], bet[ch, None]
            d = np.abs(np.concatenate([t[n, ch].reshape(cg, -1) for t in hd], 1))
            xh = (np.abs(flat) + abs(mu)) * r
            # an error of z of u * (|xhat gamma| + |beta|) moves silu' by at most half of it
            dz = d * (1.1 + xh * ga + be) if silu else d
            sb[ch] += dz.sum(1)
            sg[ch] += (dz * xh).sum(1)
            cnt = flat.size
            c1, c2 = (dz * ga).sum() / cnt, (dz * xh * ga).sum() / cnt
            s = r * (ga * dz + c1 + xh * c2)
            at = 0
            for p, x in enumerate(hx):
                w = x[n, ch].reshape(cg, -1).shape[1]
                scales[p][n, ch] = s[:, at:at + w].reshape(x[n, ch].shape)
                at += w
    k = K + rel / U
    for o, w, s in zip(dxs, want, scales):
        check(o, w, s, k)
    if dgamma is not None:
        check(dgamma, wg, sg, k)
    if dbeta is not None:
        check(dbeta, wb, sb, k)


def run_gn(tbl, xs, dys, G, gamma, beta, eps, silu):
    part = tbl.new_partials(len(xs), xs[0].shape[0], G)
    tbl.tb_patch_gn_stats(xs, G, part)
    dxs, dg, db = tbl.patch_group_norm_backward(dys, xs, G, part, gamma, beta, eps, silu)
    check_gn(dys, xs, G, gamma, beta, eps, silu, dxs, dg, db, 2e-5)
    return part, dxs, dg, db


GN_CASES = [
    ((1, 32, 24, 40), 2, [6, 6, 6, 6], 4),
    ((2, 16, 10, 33), 3, [9, 8, 8, 8], 4),        # odd rows: the element path
    ((1, 24, 5, 12, 16), 4, [4, 4, 4, 4], 4),
    ((1, 12, 3, 7, 9), 3, [4, 3], 2),
    ((3, 8, 64), 2, [64], 4),
    ((2, 6, 1), 2, [1], 3),                        # one position
    ((1, 4, 8, 16), 2, [3, 0, 5], 1),              # an empty patch in the middle
    ((1, 4, 16384 + 64), 2, [8192, 8256], 2),      # several parts and segments of a row
    ((1, 2, 200, 1000), 2, [200], 1),
    ((1, 2, 199, 1001), 2, [99, 100], 2),
]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", GN_CASES, ids=lambda c: "x".join(map(str, c[0])))
def test_groupnorm_backward(tbl, case, dtype, silu):
    shape, dim, sizes, G = case
    dt = DT[dtype]
    x = rows_of(sum(shape), shape, torch.float64, 1.5)
    xs = [(p + m).to(dt).contiguous() for p, m in zip(x.split(sizes, dim), [-3.0, 3.0, -1.0, 1.0])]
    dys = [p.contiguous() for p in rows_of(7, shape, dt, 0.5).split(sizes, dim)]
    gamma, beta = weights_of(8, shape[1], dt)
    run_gn(tbl, xs, dys, G, gamma, beta, 1e-6, silu)
    run_gn(tbl, xs, dys, G, None, None, 1e-6, silu)


@pytest.mark.parametrize("dtype", list(DT))
def test_groupnorm_backward_in_place_and_misaligned(tbl, dtype):
    dt = DT[dtype]
    shape = (2, 8, 6, 32)
    x, dy = rows_of(1, shape, dt), rows_of(2, shape, dt)
    gamma, beta = weights_of(3, 8, dt)
    part, (dx,), dg, db = run_gn(tbl, [x], [dy], 4, gamma, beta, 1e-6, True)
    for which in (0, 1):
        t = [dy.clone(), x.clone()]
        (o,), g2, b2 = tbl.patch_group_norm_backward([t[0]], [t[1]], 4, part, gamma, beta, 1e-6, dxs=[t[which]])
        assert torch.equal(o, dx) and torch.equal(g2, dg) and torch.equal(b2, db)
    # views one element past a boundary: the element path, with canaries
    buf = torch.full((3, x.numel() + 8), 7.0, dtype=dt, device="cuda")
    mx, md, mo = (b[1:1 + x.numel()].view(shape) for b in buf)
    mx.copy_(x)
    md.copy_(dy)
    _, g2, b2 = tbl.patch_group_norm_backward([md], [mx], 4, part, gamma, beta, 1e-6, dxs=[mo])
    check_gn([dy], [x], 4, gamma, beta, 1e-6, True, [mo], g2, b2, 2e-5)
    assert (buf[:, 0] == 7.0).all() and (buf[:, 1 + x.numel():] == 7.0).all()


def test_groupnorm_backward_of_gathered_records(tbl):
    # two ranks with one patch each: records of both passes gathered, each rank's gradients equal the unsharded ones
    dt, G = torch.bfloat16, 4
    x, dy = rows_of(1, (2, 16, 12, 8), dt, 1.0, 0.5), rows_of(2, (2, 16, 12, 8), dt)
    xs, dys = ([p.contiguous() for p in t.split([5, 7], 2)] for t in (x, dy))
    gamma, beta = weights_of(3, 16, dt)
    part = torch.cat([tbl.tb_patch_gn_stats([p], G, tbl.new_partials(1, 2, G)) for p in xs])
    grad = torch.cat([tbl.tb_patch_gn_grad_stats([d], [p], G, part, 2, gamma, beta, 1e-6, tbl.new_grad_partials(1, 2, 16))
                      for d, p in zip(dys, xs)])
    dxs, dgs, dbs = [], [], []
    for d, p in zip(dys, xs):
        o, dg, db = torch.empty_like(p), torch.empty_like(gamma), torch.empty_like(gamma)
        tbl.tb_patch_gn_grad_apply([d], [p], [o], G, part, grad, 2, gamma, beta, 1e-6, dg, db)
        dxs.append(o)
        dgs.append(dg)
        dbs.append(db)
    check_gn(dys, xs, G, gamma, beta, 1e-6, True, dxs, dgs[0], dbs[0], 2e-5)
    assert torch.equal(dgs[0], dgs[1]) and torch.equal(dbs[0], dbs[1])
    # a rank whose patch is empty still gets the weight gradients
    empty = torch.empty(2, 16, 0, 8, dtype=dt, device="cuda")
    dg, db = torch.full_like(gamma, 9.0), torch.full_like(gamma, 9.0)
    tbl.tb_patch_gn_grad_apply([empty], [empty], [empty], G, part, grad, 2, gamma, beta, 1e-6, dg, db)
    assert torch.equal(dg, dgs[0]) and torch.equal(db, dbs[0])


def test_groupnorm_backward_checks_and_empty_batch(tbl):
    x = rows_of(1, (1, 8, 4, 8), torch.float32)
    part = tbl.tb_patch_gn_stats([x], 2, tbl.new_partials(1, 1, 2))
    with pytest.raises(ValueError):
        tbl.patch_group_norm_backward([x, x], [x], 2, part, None, None, 1e-6)
    with pytest.raises(ValueError):
        tbl.patch_group_norm_backward([x.half()], [x], 2, part, None, None, 1e-6)
    with pytest.raises(ValueError):
        tbl.patch_group_norm_backward([x], [x], 4, part, None, None, 1e-6)
    with pytest.raises(ValueError):
        tbl.patch_group_norm_backward([x], [x], 2, part, None, None, 1e-6, dgamma=torch.empty(4, device="cuda"))
    with pytest.raises(ValueError):
        tbl.patch_group_norm_backward([x], [x], 2, part, None, None, 1e-6, grad_partials=torch.empty(4, device="cuda"))
    e = torch.empty(0, 8, 4, 4, device="cuda")
    dxs, dg, db = tbl.patch_group_norm_backward([e], [e], 2, tbl.new_partials(1, 0, 2), None, None, 1e-6)
    assert dxs[0].shape == e.shape and (dg == 0).all() and (db == 0).all()
    e = torch.empty(2, 8, 0, 4, device="cuda")            # no positions at all
    part = tbl.tb_patch_gn_stats([e], 2, tbl.new_partials(1, 2, 2))
    dxs, dg, db = tbl.patch_group_norm_backward([e], [e], 2, part, None, None, 1e-6)
    assert dxs[0].shape == e.shape and (dg == 0).all() and (db == 0).all()


def test_groupnorm_backward_extreme_activations(tbl):
    # z far on either side of zero: silu' goes to 1 and to 0, and never to NaN
    x = rows_of(1, (1, 4, 16, 16), torch.float32)
    gamma = torch.tensor([1.0, 500.0, -500.0, 1e-3], device="cuda")
    beta = torch.tensor([0.0, 200.0, -200.0, -90.0], device="cuda")
    run_gn(tbl, [x], [rows_of(2, (1, 4, 16, 16), torch.float32)], 1, gamma, beta, 1e-6, True)


def test_groupnorm_backward_is_deterministic(tbl):
    x, dy = rows_of(1, (1, 64, 96, 96), torch.bfloat16), rows_of(2, (1, 64, 96, 96), torch.bfloat16)
    gamma, beta = weights_of(3, 64, torch.bfloat16)
    part = tbl.tb_patch_gn_stats([x], 32, tbl.new_partials(1, 1, 32))
    a = tbl.patch_group_norm_backward([dy], [x], 32, part, gamma, beta, 1e-6)
    b = tbl.patch_group_norm_backward([dy], [x], 32, part, gamma, beta, 1e-6)
    assert torch.equal(a[0][0], b[0][0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


def test_groupnorm_backward_over_many_passes(tbl):
    # warps of a CTA run apart by up to two stages of its ring: every pass must
    # give the same bits, and no wait may run out
    tbl.tb_device_status(clear=True)
    x, dy = rows_of(1, (1, 48, 40, 1000), torch.bfloat16), rows_of(2, (1, 48, 40, 1000), torch.bfloat16)
    gamma, beta = weights_of(3, 48, torch.bfloat16)
    part = tbl.tb_patch_gn_stats([x], 16, tbl.new_partials(1, 1, 16))
    first = None
    for _ in range(600):
        (dx,), dg, db = tbl.patch_group_norm_backward([dy], [x], 16, part, gamma, beta, 1e-6)
        if first is None:
            first = [t.clone() for t in (dx, dg, db)]
        assert all(torch.equal(a, b) for a, b in zip(first, (dx, dg, db)))
    assert tbl.tb_device_status() == tbl.TB_DEV_OK


# --------------------------------------------------------------------------
# streams and graphs
# --------------------------------------------------------------------------

def _step(tbl, x, dy, gamma, beta, gx, gdy, ggam, gbet, grads, stream=None):
    y, mean, rstd = tbl.layer_norm(x, gamma, beta, 1e-6, stream=stream)
    dx, dg, db = tbl.layer_norm_backward(dy, x, mean, rstd, gamma, stream=stream)
    part = tbl._on_stream(lambda: tbl.new_partials(1, 1, 4), stream)
    tbl.tb_patch_gn_stats([gx], 4, part, stream)
    gdx, gdg, gdb = tbl.patch_group_norm_backward([gdy], [gx], 4, part, ggam, gbet, 1e-6, stream=stream)
    norm = tbl.clip_grad_norm(grads, 0.5, stream=stream)
    return [y, dx, dg, db, gdx[0], gdg, gdb, norm]


def _step_inputs():
    bf = torch.bfloat16
    return [rows_of(1, (300, 256), bf), rows_of(2, (300, 256), bf), *weights_of(3, 256, bf), rows_of(5, (1, 16, 8, 8), bf),
            rows_of(6, (1, 16, 8, 8), bf), *weights_of(7, 16, bf)]


@pytest.mark.parametrize("raw", [False, True])
def test_training_calls_on_another_stream(tbl, raw):
    ins = _step_inputs()
    grads = [rows_of(9, (5000,), torch.float32)]
    want = _step(tbl, *ins, tbl.GradTable(grads, [torch.empty_like(grads[0])]))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    arg = s.cuda_stream if raw else s
    for _ in range(20):
        got = _step(tbl, *ins, tbl.GradTable(grads, [torch.empty_like(grads[0])]), stream=arg)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_training_calls_replay_from_a_graph(tbl):
    ins = _step_inputs()
    grads = [rows_of(9, (5000,), torch.float32), rows_of(10, (33,), torch.bfloat16)]
    table = tbl.GradTable(grads, [torch.empty_like(g) for g in grads])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _step(tbl, *ins, table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = _step(tbl, *ins, table)
    for seed in (100, 200):
        for k, t in enumerate(ins + grads):
            t.copy_(rows_of(seed + k, t.shape, t.dtype, 0.7, 0.2))
        g.replay()
        torch.cuda.synchronize()
        clipped = [o.clone() for o in table.outs]
        want = _step(tbl, *ins, table)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(a, b) for a, b in zip(clipped, table.outs))
