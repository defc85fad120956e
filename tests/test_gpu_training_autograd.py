"""The training module's autograd functions on the kernels themselves: second
derivatives are refused, and gradients that are not wanted leave the others as
they are, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def training():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import training
    return training


def _randn(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=torch.float64).to(dtype).cuda()


def test_second_derivatives_are_refused(training):
    x, w, b = (t.requires_grad_() for t in (_randn(1, 5, 96), _randn(2, 96), _randn(3, 96)))
    y = training.layer_norm(x, w, b)
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        (y.mean() + g.square().sum()).backward()
    xs = [_randn(4, 1, 8, 3, 8).requires_grad_(), _randn(5, 1, 8, 5, 8).requires_grad_()]
    w, b = _randn(6, 8).requires_grad_(), _randn(7, 8).requires_grad_()
    ys = training.patch_group_norm(xs, 4, w, b)
    gs = torch.autograd.grad(sum(t.sum() for t in ys), xs, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        (ys[0].mean() + gs[1].square().sum()).backward()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [96, 515, 5001, 40001])
def test_gradients_on_their_own(training, cols, dtype):
    tb = training.tb
    x, dy, r, t = (_randn(k, 30, cols, dtype=dtype) for k in range(4))
    w, b = _randn(5, cols), _randn(6, cols)
    _, mean, rstd, total = tb.layer_norm(x, w, b, 1e-6, r)
    want = tb.layer_norm_backward(dy, total, mean, rstd, w, t)
    for k in range(1, 8):
        needs = tuple(bool(k >> q & 1) for q in range(3))
        got = tb.layer_norm_backward(dy, total, mean, rstd, w, t, needs=needs)
        assert all(g is None if not n else torch.equal(g, a) for g, n, a in zip(got, needs, want))
    assert tb.layer_norm_backward(dy, total, mean, rstd, w, t, needs=(False,) * 3) == (None,) * 3


def test_unused_outputs_and_frozen_inputs(training):
    def grads(frozen, use_y, use_total):
        ts = [_randn(k, *s).requires_grad_(k not in frozen) for k, s in enumerate([(7, 96), (96,), (96,), (7, 96)])]
        y, total = training.layer_norm(*ts[:3], 1e-5, ts[3])
        loss = (y * _randn(8, 7, 96)).sum() if use_y else 0
        (loss + (total * _randn(9, 7, 96)).sum() if use_total else loss).backward()
        return [t.grad for t in ts]
    every = grads((), True, True)
    for frozen in ((0,), (1, 2), (3,), (0, 3), (1,), (0, 2, 3)):
        for k, (a, c) in enumerate(zip(grads(frozen, True, True), every)):
            assert a is None if k in frozen else torch.equal(a, c)
    only = grads((), False, True)
    assert only[1] is None and only[2] is None
    assert torch.equal(only[0], _randn(9, 7, 96)) and torch.equal(only[3], only[0])
    # a sum that is not used adds nothing: dx is the norm's own
    x, w, b, r = _randn(0, 7, 96), _randn(1, 96), _randn(2, 96), _randn(3, 7, 96)
    _, mean, rstd, total = training.tb.layer_norm(x, w, b, 1e-5, r)
    dx, dw, db = training.tb.layer_norm_backward(_randn(8, 7, 96), total, mean, rstd, w)
    got = grads((), True, False)
    assert all(torch.equal(a, c) for a, c in zip(got, (dx, dw, db, dx)))
