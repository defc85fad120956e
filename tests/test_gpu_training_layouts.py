"""GPU parity of the training calls on tensors whose offsets from 16-byte
boundaries differ from one another, on strided and misaligned wide rows, and
exact weight gradients.

The GroupNorm's backward pass takes its ring kernel when x, dy and dx of every
patch share their offset, aligned or not, whatever the row length; only tensors
whose offsets differ take its element kernels.  (The offsets are asserted here:
views at one offset into rows of one buffer may well share theirs, as those of
test_groupnorm_backward_in_place_and_misaligned do.)

The weight gradients' tests use integers: dy and x small integers, mean 0 and
rstd 1 given.  Every product and partial sum is then an integer below 2^24, so
fp32 sums in any order are exact, and one row left out or taken twice fails.
"""
import pytest
import torch

from tests.test_gpu_training import DT, check, check_gn, check_ln, check_ln_bwd, f64, rows_of, weights_of

pytestmark = pytest.mark.gpu

ES = {torch.float32: 4, torch.float16: 2, torch.bfloat16: 2}


@pytest.fixture(scope="module")
def tbl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import tileblend
    return tileblend


def at_offset(src, k, fill=7.0):
    """(buffer, view): a copy of ``src`` that starts k elements past a 16-byte
    boundary, with canaries on either side."""
    es = src.element_size()
    buf = torch.full((src.numel() + 64,), fill, dtype=src.dtype, device="cuda")
    v = buf[16 + k:16 + k + src.numel()].view(src.shape)
    v.copy_(src)
    assert v.numel() == 0 or v.data_ptr() % 16 == k * es % 16
    return buf, v


def untouched(buf, k, n, fill=7.0):
    return bool((buf[:16 + k] == fill).all() and (buf[16 + k + n:] == fill).all())


# --------------------------------------------------------------------------
# PatchGroupNorm backward
# --------------------------------------------------------------------------

GN_SHAPES = [
    ((1, 8, 6, 32), 2, [6], 4),
    ((2, 12, 10, 33), 2, [4, 0, 6], 3),             # an empty patch, odd rows
    ((1, 4, 9001), 2, [9001], 2),                   # rows of more than two segments
    ((1, 40, 3, 11), 3, [5, 6], 4),                 # many short rows to a group
    ((2, 2, 70001), 2, [35000, 35001], 1),          # several parts of a row
]
# elements past a boundary of x, dy and dx
GN_OFFSETS = {"all": (1, 2, 3), "dx": (0, 0, 1), "dy": (2, 1, 2), "x": (3, 0, 0)}


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("offsets", list(GN_OFFSETS))
@pytest.mark.parametrize("case", GN_SHAPES, ids=lambda c: "x".join(map(str, c[0])))
def test_groupnorm_backward_at_different_offsets(tbl, case, offsets, dtype, silu):
    shape, dim, sizes, G = case
    dt = DT[dtype]
    xs = [p.contiguous() for p in rows_of(sum(shape), shape, dt, 1.5, 0.5).split(sizes, dim)]
    dys = [p.contiguous() for p in rows_of(7, shape, dt, 0.5).split(sizes, dim)]
    gamma, beta = weights_of(8, shape[1], dt)
    part = tbl.tb_patch_gn_stats(xs, G, tbl.new_partials(len(xs), shape[0], G))
    kx, kd, ko = GN_OFFSETS[offsets]
    vx, vd = [at_offset(t, kx)[1] for t in xs], [at_offset(t, kd)[1] for t in dys]
    outs = [at_offset(t, ko) for t in xs]
    assert any(len({t[q].data_ptr() % 16 for t in (vx, vd, [o for _, o in outs])}) > 1 for q in range(len(xs)))
    _, dg, db = tbl.patch_group_norm_backward(vd, vx, G, part, gamma, beta, 1e-6, silu, dxs=[o for _, o in outs])
    check_gn(dys, xs, G, gamma, beta, 1e-6, silu, [o for _, o in outs], dg, db, 2e-5)
    assert all(untouched(b, ko, o.numel()) for b, o in outs)
    assert all(torch.equal(a, b) for a, b in zip(vx + vd, xs + dys))
    # without weights, and the same bits from a second call
    again = [torch.empty_like(t) for t in (dg, db)]
    outs2 = [at_offset(t, ko)[1] for t in xs]
    tbl.patch_group_norm_backward(vd, vx, G, part, gamma, beta, 1e-6, silu, dxs=outs2, dgamma=again[0], dbeta=again[1])
    assert all(torch.equal(a, b) for (_, a), b in zip(outs, outs2))
    assert torch.equal(again[0], dg) and torch.equal(again[1], db)
    _, dg, db = tbl.patch_group_norm_backward(vd, vx, G, part, None, None, 1e-6, silu, dxs=outs2)
    check_gn(dys, xs, G, None, None, 1e-6, silu, outs2, dg, db, 2e-5)


@pytest.mark.parametrize("dtype", list(DT))
def test_groupnorm_backward_in_place_at_different_offsets(tbl, dtype):
    dt, shape, G = DT[dtype], (2, 8, 5, 77), 4
    x, dy = rows_of(1, shape, dt), rows_of(2, shape, dt)
    gamma, beta = weights_of(3, 8, dt)
    part = tbl.tb_patch_gn_stats([x], G, tbl.new_partials(1, 2, G))
    vx, vd, vo = at_offset(x, 1)[1], at_offset(dy, 2)[1], at_offset(x, 3)[1]
    (dx,), dg, db = tbl.patch_group_norm_backward([vd], [vx], G, part, gamma, beta, 1e-6, dxs=[vo])
    for which in (0, 1):
        t = [at_offset(dy, 2), at_offset(x, 1)]
        (o,), g2, b2 = tbl.patch_group_norm_backward([t[0][1]], [t[1][1]], G, part, gamma, beta, 1e-6,
                                                     dxs=[t[which][1]])
        assert torch.equal(o, dx) and torch.equal(g2, dg) and torch.equal(b2, db)
        assert untouched(t[which][0], (2, 1)[which], x.numel())


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape,G", [((1, 8, 6, 32), 4), ((3, 12, 10, 33), 3), ((1, 4, 9001), 2), ((2, 40, 31), 4),
                                     ((1, 2, 140003), 1), ((5, 96, 7), 2)])
def test_groupnorm_weight_gradients_are_exact(tbl, shape, G, dtype, offset):
    # offset 1 (of dy): the element kernels
    dt = DT[dtype]
    g = torch.Generator().manual_seed(sum(shape))
    x, dy = (torch.randint(-m, m + 1, shape, generator=g).to(dt).cuda() for m in (3, 2))
    N, C = shape[:2]
    count = x.numel() // (N * G)
    # records of mean 0 and variance 1, whatever x is: rstd = 1 with eps = 0
    rec = torch.zeros((1, N, G, tbl.TB_GN_PARTS, 2), dtype=torch.int64, device="cuda")
    rec[..., 0, 0] = count
    rec[..., 0, 1] = torch.tensor([0.0, float(count)]).view(torch.int64).item()
    vd = at_offset(dy, offset)[1]
    for dxs in ([torch.empty_like(x)], [at_offset(x, offset)[1]]):
        _, dg, db = tbl.patch_group_norm_backward([vd], [x], G, rec, None, None, 0.0, False, dxs=dxs)
        d, h = dy.double().reshape(N, C, -1), x.double().reshape(N, C, -1)
        assert torch.equal(dg, (d * h).sum((0, 2)).to(dt)) and torch.equal(db, d.sum((0, 2)).to(dt))


# --------------------------------------------------------------------------
# layer norm backward: wide rows at any offset and stride
# --------------------------------------------------------------------------

WIDE = [(d, c) for d in ("bf16", "f16") for c in (4097, 5001, 8192, 12001, 16383)] + \
       [("f32", c) for c in (4097, 5001, 8191)]


@pytest.mark.parametrize("total", [False, True])
@pytest.mark.parametrize("dtype,cols", WIDE)
def test_layer_norm_backward_of_wide_rows_at_different_offsets(tbl, cols, dtype, total):
    # every tensor with a row stride and a first element of its own, so that each
    # row has another offset; more rows than CTAs times the ring's stages
    dt = DT[dtype]
    rows = 1300 if cols * ES[dt] <= 10400 else 700
    gamma, beta = weights_of(3, cols, torch.float32)

    def strided(seed, pad, first, scale):
        return rows_of(seed, (rows, cols + pad), dt, scale)[:, first:first + cols]
    x, dy = strided(1, 5, 3, 1.0), strided(2, 8, 1, 0.2)
    dtot = strided(4, 3, 2, 0.3) if total else None
    mean, rstd = tbl.layer_norm(x.contiguous(), gamma, beta, 1e-6)[1:]
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    got = []
    for first in (6, 0):
        out = torch.full((rows, cols + 7), 5.0, dtype=dt, device="cuda")
        dx = out[:, first:first + cols]
        tbl.tb_layer_norm_backward(dy, x, mean, rstd, gamma, dx, dg, db, tbl.ln_workspace(rows, cols), dtotal=dtot)
        assert (out[:, :first] == 5.0).all() and (out[:, first + cols:] == 5.0).all()
        got.append(dx)
    check_ln_bwd(dy, x, mean, rstd, gamma, dtot, got[0], dg, db)
    assert torch.equal(got[0], got[1])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [64, 1024, 4104, 8192, 16384])
def test_layer_norm_of_aligned_rows_with_misaligned_weights(tbl, cols, dtype):
    # whole 16-byte words, but the weights start past a boundary: rows go element by element
    dt = DT[dtype]
    if dtype == "f32":
        cols //= 2
    rows = 400
    gamma, beta = (at_offset(t, 1)[1] for t in weights_of(3, cols, dt))
    x, dy, dtot = (rows_of(k, (rows, cols), dt, 0.5) for k in (1, 2, 4))
    y, mean, rstd = tbl.layer_norm(x, gamma, beta, 1e-6)
    check_ln(x, gamma, beta, 1e-6, y, mean, rstd)
    dx, dg, db = tbl.layer_norm_backward(dy, x, mean, rstd, gamma, dtot)
    check_ln_bwd(dy, x, mean, rstd, gamma, dtot, dx, dg, db)


# --------------------------------------------------------------------------
# layer norm backward: weight gradients
# --------------------------------------------------------------------------

# (rows, columns): every kernel of the dispatch, last rows of warps, CTAs and rings
SUMS = [(30001, c) for c in (4, 16, 33, 63, 64, 65, 72, 127, 128, 129, 200, 256, 257)] + \
       [(5003, c) for c in (512, 515, 1000, 1024, 1025, 2040, 2047)] + \
       [(1001, c) for c in (2048, 4095, 4096, 4097, 5001, 8191, 8192)] + \
       [(313, c) for c in (8193, 12001, 16384, 16383, 16385, 16392, 33000)] + [(1, 40), (2, 515), (3, 8192), (153, 16400)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SUMS)
def test_layer_norm_weight_gradients_are_exact(tbl, rows, cols, dtype):
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x, dy = (torch.randint(-m, m + 1, (rows, cols), generator=g, device="cuda").to(dt) for m in (3, 2))
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    gamma = torch.ones(cols, device="cuda")
    want = (dy.double() * x.double()).sum(0).float(), dy.double().sum(0).float()
    for dtotal in (None, dy):
        _, dg, db = tbl.layer_norm_backward(dy, x, mean, rstd, gamma, dtotal)
        assert torch.equal(dg, want[0]) and torch.equal(db, want[1])


@pytest.mark.parametrize("rows,cols", [(30001, 63), (30001, 128), (5003, 1024), (1001, 5001), (313, 16400)])
def test_layer_norm_weight_gradients_within_their_sums_length(tbl, rows, cols):
    # A column's sum is a chain over the rows of a thread (rows / CTAs at most),
    # then over the row groups of a CTA (64 at most), the parts of a slice
    # (TB_LN_PARTS / 32) and five pairwise steps; a term itself is rounded three
    # times (x - mean, dy * rstd, their product within the sum's step).
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    k = -(-rows // min(sms, tbl.TB_LN_PARTS)) + 64 + tbl.TB_LN_PARTS // 32 + 5 + 3
    x, dy = rows_of(1, (rows, cols), torch.float32, 1.0, 0.2), rows_of(2, (rows, cols), torch.float32, 0.3)
    gamma, beta = weights_of(3, cols, torch.float32)
    _, mean, rstd = tbl.layer_norm(x, gamma, beta, 1e-6)
    _, dg, db = tbl.layer_norm_backward(dy, x, mean, rstd, gamma)
    d, h, m, r = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    terms = d * ((h - m) * r)
    scale = (d.abs() * (h.abs() + m.abs()) * r).sum(0)
    check(dg, f64(terms.sum(0)), f64(scale), k)
    check(db, f64(d.sum(0)), f64(d.abs().sum(0)), k)
