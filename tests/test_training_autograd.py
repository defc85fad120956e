"""CPU checks of the training module's autograd functions and step.  The
library's kernels are replaced by the same formulas in torch, run without a
graph as the kernels run: what is tested is what the module makes of them."""
import pytest
import torch
import torch.nn.functional as F


def _layer_norm(x, gamma, beta, eps, residual=None, stream=None):
    with torch.no_grad():
        h = x if residual is None else x + residual
        mean = h.mean(-1)
        rstd = 1.0 / torch.sqrt(h.var(-1, unbiased=False) + eps)
        y = (h - mean[..., None]) * rstd[..., None]
        y = y if gamma is None else y * gamma.reshape(-1)
        y = y if beta is None else y + beta.reshape(-1)
    return (y, mean, rstd) if residual is None else (y, mean, rstd, h)


def _layer_norm_backward(dy, x, mean, rstd, gamma, dtotal=None, wdtype=None, stream=None, needs=(True, True, True)):
    with torch.no_grad():
        n, r = x.shape[-1], rstd[..., None]
        xhat = (x - mean[..., None]) * r
        g = dy if gamma is None else dy * gamma.reshape(-1)
        dx = r * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
        dx = dx if dtotal is None else dx + dtotal
        out = dx, (dy * xhat).reshape(-1, n).sum(0), dy.reshape(-1, n).sum(0)
        return tuple(t if want else None for t, want in zip(out, needs))


def _patch_group_norm(patches, G, gamma, beta, eps, silu=True, outs=None, partials=None, stream=None):
    with torch.no_grad():
        y = F.group_norm(torch.cat(list(patches), 2), G, gamma.reshape(-1), beta.reshape(-1), eps)
        return list((F.silu(y) if silu else y).split([p.shape[2] for p in patches], 2))


def _patch_group_norm_backward(grads, patches, G, partials, gamma, beta, eps, silu=True):
    with torch.enable_grad():
        xs = [p.detach().requires_grad_() for p in patches]
        w, b = (t.detach().reshape(-1).requires_grad_() for t in (gamma, beta))
        y = F.group_norm(torch.cat(xs, 2), G, w, b, eps)
        out = torch.autograd.grad(F.silu(y) if silu else y, [*xs, w, b], torch.cat(list(grads), 2))
    return list(out[:-2]), out[-2], out[-1]


@pytest.fixture
def training(monkeypatch):
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import training
    for name, f in (("layer_norm", _layer_norm), ("layer_norm_backward", _layer_norm_backward),
                    ("patch_group_norm", _patch_group_norm), ("patch_group_norm_backward", _patch_group_norm_backward),
                    ("new_partials", lambda *a: torch.zeros(1)), ("_row_ld", lambda t, *a: t.stride(0))):
        monkeypatch.setattr(training.tb, name, f)
    return training


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


# --------------------------------------------------------------------------
# second derivatives: the kernels compute none, so asking for one is an error
# --------------------------------------------------------------------------

@pytest.mark.parametrize("residual", [False, True])
def test_layer_norm_second_derivative_is_refused(training, residual):
    x, w, b = _randn(1, 3, 8).requires_grad_(), _randn(2, 8).requires_grad_(), _randn(3, 8).requires_grad_()
    r = _randn(4, 3, 8).requires_grad_() if residual else None

    def penalised(dy):
        y = training.layer_norm(x, w, b, 1e-5, r)
        y = y[0] if residual else y
        g, = torch.autograd.grad(y, x, dy, create_graph=True)
        return y.square().mean() + g.square().sum()   # the first term has a graph of its own
    # the gradient of y may itself be a constant, or not
    for dy in (_randn(5, 3, 8), _randn(5, 3, 8).requires_grad_()):
        with pytest.raises(RuntimeError, match="second derivative"):
            penalised(dy).backward()
    # first derivatives with create_graph are what they are without it
    y = training.layer_norm(x, w, b, 1e-5)
    a = torch.autograd.grad(y, [x, w, b], _randn(6, 3, 8), create_graph=True)
    y = training.layer_norm(x, w, b, 1e-5)
    c = torch.autograd.grad(y, [x, w, b], _randn(6, 3, 8))
    assert all(torch.equal(p, q) for p, q in zip(a, c))


def test_group_norm_second_derivative_is_refused(training):
    xs = [_randn(1, 2, 4, 3, 5).requires_grad_(), _randn(2, 2, 4, 2, 5).requires_grad_()]
    w, b = _randn(3, 4).requires_grad_(), _randn(4, 4).requires_grad_()
    for last in (False, True):
        dys = [_randn(5 + k, *x.shape) for k, x in enumerate(xs)]
        dys[1].requires_grad_(last)
        outs = training.patch_group_norm(xs, 2, w, b)
        gs = torch.autograd.grad(outs, xs, dys, create_graph=True)
        loss = sum(o.square().mean() for o in outs) + sum(g.square().sum() for g in gs)
        with pytest.raises(RuntimeError, match="second derivative"):
            loss.backward()


# --------------------------------------------------------------------------
# only what is asked for is computed
# --------------------------------------------------------------------------

@pytest.fixture
def calls(training, monkeypatch):
    """The arguments (dtotal, needs) of every backward call."""
    seen = []

    def backward(dy, x, mean, rstd, gamma, dtotal=None, wdtype=None, stream=None, needs=(True, True, True)):
        seen.append((dtotal, tuple(needs)))
        return _layer_norm_backward(dy, x, mean, rstd, gamma, dtotal, needs=needs)
    monkeypatch.setattr(training.tb, "layer_norm_backward", backward)
    return seen


def _leaves():
    return (_randn(1, 3, 8).requires_grad_(), _randn(2, 8).requires_grad_(), _randn(3, 8).requires_grad_(),
            _randn(4, 3, 8).requires_grad_())


def _plain(x, w, b, r):
    total = x + r
    return F.layer_norm(total, (8,), w, b, 1e-5), total


@pytest.mark.parametrize("used", ["y", "total", "both"])
def test_layer_norm_outputs_that_are_not_used_cost_nothing(training, calls, used):
    def grads(f):
        ts = _leaves()
        y, total = f(*ts)
        v, u = _randn(5, 3, 8), _randn(6, 3, 8)
        sum(t for name, t in (("y", (y * v).sum()), ("total", (total * u).sum())) if used in (name, "both")).backward()
        return [t.grad for t in ts]
    got = grads(lambda x, w, b, r: training.layer_norm(x, w, b, 1e-5, r))
    for a, c in zip(got, grads(_plain)):
        assert a is None and c is None or torch.allclose(a, c, rtol=1e-10, atol=1e-12)
    if used == "total":
        assert calls == []
    else:
        (dtotal, needs), = calls
        assert (dtotal is None) == (used == "y") and needs == (True, True, True)


@pytest.mark.parametrize("frozen", [(1, 2), (0,), (0, 3), (1,), (2, 0, 3)])
def test_layer_norm_gradients_that_are_not_wanted_are_not_computed(training, calls, frozen):
    ts, plain = _leaves(), _leaves()
    for k in frozen:
        ts[k].requires_grad_(False)
    v = _randn(5, 3, 8)
    (training.layer_norm(*ts[:3], 1e-5, ts[3])[0] * v).sum().backward()
    (_plain(*plain)[0] * v).sum().backward()
    for k, (t, p) in enumerate(zip(ts, plain)):
        assert t.grad is None if k in frozen else torch.allclose(t.grad, p.grad, rtol=1e-10, atol=1e-12)
    (_, needs), = calls
    assert needs == (not {0, 3} <= set(frozen), 1 not in frozen, 2 not in frozen)


# --------------------------------------------------------------------------
# the step
# --------------------------------------------------------------------------

class _Table:
    def __init__(self, grads, outs=None):
        self.grads = list(grads)


def _clip_grad_norm(table, max_norm, records=None, norm=None, stream=None):
    n = torch.sqrt(sum(g.square().sum() for g in table.grads))
    for g in table.grads:
        g.mul_(torch.clamp(max_norm / (n + 1e-6), max=1.0))
    return n.reshape(1)


@pytest.mark.parametrize("between", ["nothing", "dropped", "replaced", "scaled"])
def test_step_clips_the_gradients_it_applies(training, monkeypatch, between):
    # whatever a program did to the parameters' .grad since the last step
    for name, f in (("GradTable", _Table), ("new_grad_records", lambda *a: None), ("clip_grad_norm", _clip_grad_norm)):
        monkeypatch.setattr(training.tb, name, f)
    w, b = _randn(1, 4, 4).requires_grad_(), _randn(2, 4).requires_grad_()
    trainer = training.Trainer([w, b], lr=0.5, max_norm=0.25)
    x = _randn(3, 5, 4)
    for _ in range(2):
        for p in (w, b):
            if between == "dropped":
                p.grad = None
            elif between == "replaced":
                p.grad = torch.full_like(p, 3.0)
            elif between == "scaled":
                p.grad *= 7.0
        ps = [p.detach().clone().requires_grad_() for p in (w, b)]
        (x @ ps[0] + ps[1]).square().mean().backward()
        want = torch.nn.utils.clip_grad_norm_(ps, 0.25)
        norm = trainer.step((x @ w + b).square().mean())
        assert want > 0.25 and torch.allclose(norm, want)
        for p, q in zip((w, b), ps):
            assert torch.allclose(p.grad, q.grad) and torch.allclose(p.detach(), q.detach() - 0.5 * q.grad)


# --------------------------------------------------------------------------
# weights of any shape of the right size
# --------------------------------------------------------------------------

def test_weight_gradients_have_their_weights_shapes(training):
    x, w, b = _randn(1, 3, 8).requires_grad_(), _randn(2, 1, 1, 8).requires_grad_(), _randn(3, 8, 1).requires_grad_()
    v = _randn(4, 3, 8)
    (training.layer_norm(x, w, b, 1e-5) * v).sum().backward()
    ps = [t.detach().reshape(-1).requires_grad_() for t in (w, b)]
    (F.layer_norm(x.detach(), (8,), *ps, 1e-5) * v).sum().backward()
    for t, p in zip((w, b), ps):
        assert t.grad.shape == t.shape and torch.allclose(t.grad.reshape(-1), p.grad)
    xs = [_randn(5, 2, 4, 3, 5), _randn(6, 2, 4, 2, 5)]
    w, b = _randn(7, 1, 4, 1, 1).requires_grad_(), _randn(8, 4, 1).requires_grad_()
    v = _randn(9, 2, 4, 5, 5)
    (torch.cat(training.patch_group_norm(xs, 2, w, b), 2) * v).sum().backward()
    ps = [t.detach().reshape(-1).requires_grad_() for t in (w, b)]
    (F.silu(F.group_norm(torch.cat(xs, 2), 2, *ps, 1e-6)) * v).sum().backward()
    for t, p in zip((w, b), ps):
        assert t.grad.shape == t.shape and torch.allclose(t.grad.reshape(-1), p.grad)
