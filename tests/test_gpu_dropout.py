"""GPU parity of dropout against the oracle: the mask bit for bit, the values
within one rounding of the output (half a step) and two fp32 roundings (of the
scale and of the product and sum, 2 u of the magnitudes)."""
import numpy as np
import pytest
import torch

from oracle import dropout as D
from tests.test_gpu_training import DT, HALF, TINY, U, f64, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tbl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import tileblend
    return tileblend


def check(y, x, p, seed, offset, residual=None, first=0):
    want = D.dropout(f64(x), p, seed, offset, None if residual is None else f64(residual), first)
    scale = np.abs(D.dropout(np.abs(f64(x)), p, seed, offset, None if residual is None else np.abs(f64(residual)), first))
    got = f64(y)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= np.abs(want) * HALF[y.dtype] + TINY[y.dtype] + 3 * U * scale)
    assert not bad.any(), "%d of %d off" % (bad.sum(), bad.size)
    if residual is None:  # what is dropped is zero, and nothing else
        kept = D.bits(first, got.size, seed, offset).reshape(got.shape) >= D.threshold(p)
        assert (got[~kept] == 0).all() and ((got != 0) == (kept & (f64(x) != 0))).all()


SEED, OFFSET = 0x9123456789ABCDEF, (1 << 40) + 17


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (1, 8), (3, 5), (2, 9), (5, 64), (1, 4096), (33, 255), (33, 256),
                                   (33, 257), (7, 1111), (4099, 24), (301, 2048), (2, 3, 40), (8193,)],
                         ids=lambda s: "x".join(map(str, s)))
def test_shapes(tbl, shape, dtype, residual):
    x = rows_of(1, shape, DT[dtype], 1.5)
    r = rows_of(2, shape, DT[dtype]) if residual else None
    check(tbl.dropout(x, 0.3, SEED, OFFSET, r), x, 0.3, SEED, OFFSET, r)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -17, 1e-4, 0.1, 0.5, 0.999, 1 - 2.0 ** -16, 1 - 2.0 ** -18, 1.0])
def test_probabilities(tbl, p):
    x, r = rows_of(1, (100, 96), torch.float32), rows_of(2, (100, 96), torch.float32)
    check(tbl.dropout(x, p, 3, 4), x, p, 3, 4)
    check(tbl.dropout(x, p, 3, 4, r), x, p, 3, 4, r)
    odd = x[:, :95]
    check(tbl.dropout(odd, p, 3, 4, r[:, 1:]), odd, p, 3, 4, r[:, 1:])
    if p == 0:
        assert torch.equal(tbl.dropout(x, p, 3, 4), x)
    if p == 1:
        assert (tbl.dropout(x, p, 3, 4) == 0).all() and torch.equal(tbl.dropout(x, p, 3, 4, r), r)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("cols", [8, 24, 64, 100, 264, 1000])
def test_strides_offsets_and_guard_bands(tbl, cols, dtype):
    # every tensor cut out of wider rows, aligned and not; the mask goes by the
    # element's number in the rows, whatever their layout
    dt = DT[dtype]
    rows = 37
    x, r = rows_of(1, (rows, cols), dt), rows_of(2, (rows, cols), dt)
    want = tbl.dropout(x, 0.25, SEED, 5, r)
    check(want, x, 0.25, SEED, 5, r)
    for pad, at in ((8, 0), (8, 8), (16, 4), (9, 0), (7, 3), (0, 0)):
        buf = torch.full((3, rows, cols + pad), 7.0, dtype=dt, device="cuda")
        at = min(at, pad)
        vx, vr, vy = (b[:, at:at + cols] for b in buf)
        vx.copy_(x)
        vr.copy_(r)
        tbl.tb_dropout(vx, vy, 0.25, SEED, 5, residual=vr)
        assert torch.equal(vy, want) and torch.equal(vx, x) and torch.equal(vr, r)
        assert (buf[:, :, :at] == 7.0).all() and (buf[:, :, at + cols:] == 7.0).all()
        # mixed layouts
        assert torch.equal(tbl.dropout(vx, 0.25, SEED, 5, r), want)
        assert torch.equal(tbl.dropout(x, 0.25, SEED, 5, vr), want)
        # in place, over either input
        tbl.tb_dropout(vx, vx, 0.25, SEED, 5, residual=vr)
        assert torch.equal(vx, want)
        vx.copy_(x)
        tbl.tb_dropout(vx, vr, 0.25, SEED, 5, residual=vr)
        assert torch.equal(vr, want)
    flat = torch.full((rows * cols + 24,), 7.0, dtype=dt, device="cuda")   # dense, at odd addresses
    for at in (1, 3, 8):
        v = flat[at:at + rows * cols].view(rows, cols)
        v.copy_(x)
        tbl.tb_dropout(v, v, 0.25, SEED, 5, residual=r)
        assert torch.equal(v, want) and (flat[:at] == 7.0).all() and (flat[at + rows * cols:] == 7.0).all()
        flat.fill_(7.0)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows, cols", [(6, 319), (6, 320), (1, 761), (5, 767), (5, 769), (40, 1537), (3, 2311)])
def test_odd_rows_of_halves(tbl, rows, cols, dtype, residual):
    # every alignment of x, of the residual and of y against 16 bytes, rows of one and of
    # several warps, and in place
    dt = DT[dtype]
    x, r = rows_of(1, (rows, cols), dt), rows_of(2, (rows, cols), dt) if residual else None
    want = tbl.dropout(x, 0.3, SEED, 9, r)
    check(want, x, 0.3, SEED, 9, r)
    for at in range(8):
        buf = torch.full((3, rows * (cols + 11) + 8), 7.0, dtype=dt, device="cuda")
        vx, vr, vy = (b[k:k + rows * ld].view(rows, ld)[:, :cols]
                      for b, k, ld in zip(buf, (at, 3 * at % 8, 5 * at % 8), (cols + 3, cols + at, cols + 11)))
        vx.copy_(x)
        if residual:
            vr.copy_(r)
        tbl.tb_dropout(vx, vy, 0.3, SEED, 9, residual=vr if residual else None)
        assert torch.equal(vy, want) and torch.equal(vx, x)
        vy.fill_(7.0)
        assert (buf[2] == 7.0).all()
        into = vr if residual and at % 2 else vx
        tbl.tb_dropout(vx, into, 0.3, SEED, 9, residual=vr if residual else None)
        assert torch.equal(into, want)
        into.fill_(7.0)
        assert (buf[1 if into is vr else 0] == 7.0).all()


def test_odd_rows_of_halves_by_state_and_special_values(tbl):
    x, r = rows_of(1, (33, 1001), torch.bfloat16), rows_of(2, (33, 1001), torch.bfloat16)
    state = torch.tensor([5, 3], dtype=torch.int64, device="cuda")
    assert torch.equal(tbl.dropout(x[:, 1:], 0.3, 11, 2, r[:, 1:], state), tbl.dropout(x[:, 1:], 0.3, 16, 5, r[:, 1:]))
    odd = torch.full((33, 1003), float("nan"), dtype=torch.bfloat16, device="cuda")[:, 1:-1]
    assert torch.equal(tbl.dropout(odd, 1.0, 1, 2, r), r) and (tbl.dropout(odd, 1.0, 1, 2) == 0).all()
    assert torch.equal(tbl.dropout(x[:, 1:], 0.0, 1), x[:, 1:])
    keep = tbl.dropout(torch.ones_like(x), 0.5, 3, 4) != 0
    y = tbl.dropout(odd, 0.5, 3, 4, r)
    assert torch.equal(y.isnan(), keep) and torch.equal(y[~keep], r[~keep])


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
# the last ones: a row's last run is 32, 64 or 96 units at some alignments, or at all of them
@pytest.mark.parametrize("rows, cols", [(6, 319), (6, 320), (1, 761), (5, 767), (5, 769), (40, 1537), (3, 2311),
                                        (4, 505), (9, 511), (3, 512), (8, 1021), (4, 1111), (2, 1279), (5, 1535),
                                        (5, 2000)])
def test_odd_rows_of_halves_all_kept_or_all_dropped(tbl, rows, cols, dtype, residual):
    # at every alignment what is not random is exact: x (and the residual, one rounding), or
    # the residual alone (or zero)
    dt = DT[dtype]
    x, r = rows_of(1, (rows, cols), dt), rows_of(2, (rows, cols), dt) if residual else None
    kept = (x.float() + r.float()).to(dt) if residual else x
    gone = r if residual else torch.zeros_like(x)
    for at in range(8):
        buf = torch.full((3, rows * (cols + 11) + 8), 7.0, dtype=dt, device="cuda")
        vx, vr, vy = (b[k:k + rows * ld].view(rows, ld)[:, :cols]
                      for b, k, ld in zip(buf, (at, 3 * at % 8, 5 * at % 8), (cols + 3, cols + at, cols + 11)))
        for p, want in ((0.0, kept), (2.0 ** -18, kept), (1 - 2.0 ** -18, gone), (1.0, gone)):
            for into in (vy, vx, vr) if residual else (vy, vx):
                buf.fill_(7.0)
                vx.copy_(x)
                if residual:
                    vr.copy_(r)
                tbl.tb_dropout(vx, into, p, SEED, 9, residual=vr if residual else None)
                assert torch.equal(into, want)
                into.fill_(7.0)
                assert (buf[2 if into is vy else 0 if into is vx else 1] == 7.0).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows, cols", [(4099, 8), (2053, 16), (1031, 40), (130, 2040), (130, 2048), (130, 2056)])
def test_rows_that_a_thread_steps_over(tbl, rows, cols, residual):
    # whole blocks out of wider rows: a thread's blocks lie 256 apart, many rows or less
    # than one
    buf = rows_of(1, (2, rows, cols + 8), torch.bfloat16)
    x, r = buf[0, :, 8:], buf[1, :, :cols] if residual else None
    check(tbl.dropout(x, 0.3, SEED, 3, r), x, 0.3, SEED, 3, r)



def test_dropped_bad_values_are_gone(tbl):
    for bad in (float("nan"), float("inf")):
        x = torch.full((64, 40), bad, device="cuda")
        for t, r in ((x, None), (x, torch.ones_like(x)), (x[:, :39], None)):
            y = tbl.dropout(t, 0.5, 1, 2, r)
            kept = torch.from_numpy(D.bits(0, t.numel(), 1, 2).reshape(t.shape) >= 32768).cuda()
            assert (y[~kept] == (0 if r is None else 1)).all() and not torch.isfinite(y[kept]).any()


def test_the_backward_pass_is_the_same_call(tbl):
    # <dropout(x), dy> = <x, dropout(dy)> with equal masks, and differences of the
    # (linear) call are the call itself
    x, dy = rows_of(1, (50, 120), torch.float32), rows_of(2, (50, 120), torch.float32)
    y, dx = tbl.dropout(x, 0.4, 9, 1), tbl.dropout(dy, 0.4, 9, 1)
    a, b = float((f64(y) * f64(dy)).sum()), float((f64(x) * f64(dx)).sum())
    assert abs(a - b) <= 4 * U * float(np.abs(f64(y) * f64(dy)).sum())
    assert torch.equal(tbl.dropout(x + x, 0.4, 9, 1), y + y)


def test_seed_offset_and_device_state(tbl):
    x = rows_of(1, (40, 64), torch.float32)
    big = (1 << 64) - 1
    state = torch.tensor([5, -3], dtype=torch.int64, device="cuda")
    for t in (x, x[:, :63]):
        y = tbl.dropout(t, 0.5, 2, 7, state=state)
        assert torch.equal(y, tbl.dropout(t, 0.5, 7, 4))
        assert torch.equal(tbl.dropout(t, 0.5, big, 1, state=state), tbl.dropout(t, 0.5, 4, -2))   # modulo 2^64
        assert torch.equal(tbl.dropout(t, 0.0, 2, 7, state=state), t.contiguous())
        check(y, t, 0.5, 7, 4)
    assert not torch.equal(tbl.dropout(x, 0.5, 1, 0), tbl.dropout(x, 0.5, 0, 1))


def test_checks(tbl):
    x = rows_of(1, (4, 8), torch.float32)
    for call in (lambda: tbl.tb_dropout(x, x.half(), 0.1, 1), lambda: tbl.tb_dropout(x, x[:2], 0.1, 1),
                 lambda: tbl.dropout(x, 0.1, 1, residual=x[:, :4]), lambda: tbl.dropout(x.t(), 0.1, 1),
                 lambda: tbl.dropout(x[:, ::2], 0.1, 1), lambda: tbl.dropout(x.expand(3, 4, 8), 0.1, 1),
                 lambda: tbl.dropout(x, 0.1, 1, state=torch.zeros(2, device="cuda")),
                 lambda: tbl.dropout(x, 0.1, 1, state=torch.zeros(3, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(tbl.TileBlendError):
            tbl.dropout(x, p, 1)
    for shape in ((0, 8), (4, 0), (0,)):
        e = torch.empty(shape, device="cuda")
        assert tbl.dropout(e, 0.1, 1).shape == e.shape


def test_offsets_past_32_bits(tbl):
    # more than 2^32 elements: the last ones against the oracle
    n = (1 << 32) + 1003
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    tbl.tb_dropout(x, x, 0.5, SEED, OFFSET)
    check(x[-4000:], torch.ones(4000, dtype=torch.bfloat16), 0.5, SEED, OFFSET, first=n - 4000)
    check(x[:4000], torch.ones(4000, dtype=torch.bfloat16), 0.5, SEED, OFFSET)
    x.fill_(1.0)
    v = x[: (n // 9) * 9].view(-1, 9)[:, :7]      # 2^31.6 elements at strides of nine
    tbl.tb_dropout(v, v, 0.5, SEED, OFFSET)
    rows = v.shape[0]
    tail = v[-500:].contiguous()
    check(tail, torch.ones_like(tail), 0.5, SEED, OFFSET, first=(rows - 500) * 7)
    assert (x[: (n // 9) * 9].view(-1, 9)[:, 7:] == 1).all()


@pytest.mark.parametrize("rows, cols, pad", [(3870000, 1111, 1), (3, (1 << 31) + 5, 2), (4200000, 1024, 8), (1, (1 << 32) + 21, 0)])
def test_odd_rows_past_32_bits(tbl, rows, cols, pad):
    # more than 2^32 elements out of wider rows, and from an odd address: the first and the
    # last ones of some rows
    buf = torch.ones(rows * (cols + pad) + 8, dtype=torch.bfloat16, device="cuda")
    v = buf[8 if pad == 8 else 3:][:rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    assert v.numel() > 1 << 32
    tbl.tb_dropout(v, v, 0.5, SEED, OFFSET)
    for row in sorted({0, rows // 2, rows - 1}):
        for at in (0, cols - 600):
            got = v[row, at:at + 600]
            check(got, torch.ones(600, dtype=torch.bfloat16), 0.5, SEED, OFFSET, first=row * cols + at)
    if pad:
        gaps = buf[8 if pad == 8 else 3:][:rows * (cols + pad)].view(rows, cols + pad)[:, cols:]
        assert (gaps == 1).all()


@pytest.mark.parametrize("raw", [False, True])
def test_on_another_stream(tbl, raw):
    x, r = rows_of(1, (300, 256), torch.bfloat16), rows_of(2, (300, 256), torch.bfloat16)
    want = tbl.dropout(x, 0.1, 3, 4, r)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(20):
        got = tbl.dropout(x, 0.1, 3, 4, r, stream=s.cuda_stream if raw else s)
        s.synchronize()
        assert torch.equal(got, want)


def test_a_graph_draws_new_masks(tbl):
    x, r = rows_of(1, (30, 256), torch.bfloat16), rows_of(2, (30, 256), torch.bfloat16)
    state = torch.zeros(2, dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tbl.dropout(x, 0.3, 11, 1, r, state)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        y = tbl.dropout(x, 0.3, 11, 1, r, state)
        dx = tbl.dropout(r, 0.3, 11, 1, state=state)
        state[1] += 1
    for step in range(3):
        x.copy_(rows_of(10 + step, x.shape, x.dtype))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, tbl.dropout(x, 0.3, 11, 1 + step, r))
        assert torch.equal(dx, tbl.dropout(r, 0.3, 11, 1 + step))
        assert int(state[1]) == step + 1
