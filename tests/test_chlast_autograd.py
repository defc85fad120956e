"""CPU checks of the channels-last functions of the training module, with torch
in the kernels' place: what autograd makes of them, and where they are refused."""
import pytest
import torch

from oracle import dropout as D
from tests.test_training_autograd import _patch_group_norm, _patch_group_norm_backward, _randn
from tests.test_training_devices import Library, t


def _dropout(x, p, seed, offset=0, residual=None, state=None, stream=None):
    with torch.no_grad():
        s, o = (0, 0) if state is None else state.tolist()
        keep = D.bits(0, x.numel(), (seed + s) % 2 ** 64, (offset + o) % 2 ** 64) >= D.threshold(p)
        y = torch.where(torch.from_numpy(keep).view(x.shape), x, 0.0) * (65536 / max(1, 65536 - D.threshold(p)))
        return y if residual is None else y + residual


def _forward(patches, G, gamma, beta, eps, silu=True, outs=None, partials=None, stream=None):
    ys = _patch_group_norm([p.movedim(-1, 1).flatten(2) for p in patches], G, gamma, beta, eps, silu)
    return [y.movedim(1, -1).reshape(p.shape) for y, p in zip(ys, patches)]


def _backward(grads, patches, G, partials, gamma, beta, eps, silu=True):
    def cf(ts):
        return [x.movedim(-1, 1).flatten(2) for x in ts]
    dxs, dg, db = _patch_group_norm_backward(cf(grads), cf(patches), G, partials, gamma, beta, eps, silu)
    return [d.movedim(1, -1).reshape(p.shape) for d, p in zip(dxs, patches)], dg, db


@pytest.fixture
def training(monkeypatch):
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import training
    for name, f in (("dropout", _dropout), ("patch_group_norm_cl", _forward),
                    ("patch_group_norm_backward_cl", _backward), ("new_partials", lambda *a: torch.zeros(1)),
                    ("_row_ld", lambda x, *a: x.stride(0))):
        monkeypatch.setattr(training.tb, name, f)
    return training


def test_dropout_gradients_of_every_order(training):
    x, r = _randn(1, 6, 8).requires_grad_(), _randn(2, 6, 8).requires_grad_()
    assert torch.autograd.gradcheck(lambda a, b: training.dropout(a, 0.4, 3, 5, b), (x, r))
    assert torch.autograd.gradgradcheck(lambda a, b: training.dropout(a, 0.4, 3, 5, b) ** 2, (x, r))
    y = training.dropout(x, 0.4, 3, 5, r)
    dy = _randn(3, 6, 8)
    gx, gr = torch.autograd.grad(y, (x, r), dy)
    assert torch.equal(gx, _dropout(dy, 0.4, 3, 5)) and torch.equal(gr, dy)
    y = training.dropout(x, 0.4, 3, 5, r.detach())
    assert torch.equal(torch.autograd.grad(y, x, dy)[0], gx)
    y = training.dropout(x.detach(), 0.4, 3, 5, r)
    assert torch.equal(torch.autograd.grad(y, r, dy)[0], dy)


def test_a_state_that_changed_before_the_backward_pass_is_refused(training):
    state = torch.tensor([1, 2])
    x = _randn(1, 6, 8).requires_grad_()
    y = training.dropout(x, 0.4, 3, 5, state=state)
    assert torch.equal(torch.autograd.grad(y.sum(), x)[0], _dropout(torch.ones(6, 8, dtype=torch.float64), 0.4, 4, 7))
    y = training.dropout(x, 0.4, 3, 5, state=state)
    state[1] += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_group_norm_gradients_and_refused_second_derivative(training):
    xs = [_randn(1, 2, 3, 5, 4).requires_grad_(), _randn(2, 2, 2, 5, 4).requires_grad_()]
    w, b = _randn(3, 1, 4).requires_grad_(), _randn(4, 4).requires_grad_()
    assert torch.autograd.gradcheck(lambda *a: training.patch_group_norm_cl(a[2:], 2, a[0], a[1]), (w, b, *xs))
    outs = training.patch_group_norm_cl(xs, 2, w, b)
    gs = torch.autograd.grad(outs, xs, [_randn(5 + k, *x.shape) for k, x in enumerate(xs)], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        (outs[0].square().mean() + gs[1].square().sum()).backward()


@pytest.fixture
def devices(monkeypatch):
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import tileblend

    class Lib(Library):
        def __getattr__(self, name):
            return getattr(self._real, name) if name == "tb_patch_gn_workspace_cl" else super().__getattr__(name)
    monkeypatch.setattr(tileblend, "_lib", Lib(tileblend._lib))
    monkeypatch.setattr(tileblend, "_current_device", lambda: 0)
    monkeypatch.setattr(tileblend, "_raw_stream", lambda device: 0)
    return tileblend


def _calls(tbl, d, **at):
    def on(name, *shape, dtype=torch.float32):
        return t(at.get(name, d), *shape, dtype=dtype)
    x, y, r, s = on("x", 4, 8), on("y", 4, 8), on("r", 4, 8), on("s", 2, dtype=torch.int64)
    p, o, g = on("p", 1, 4, 4), on("o", 1, 4, 4), on("g", 1, 4, 4)
    rec, w = on("rec", 1, 1, 2, tbl.TB_GN_PARTS, 16, dtype=torch.uint8), on("w", 4)
    grec, ws, dw = on("grec", 1, 1, 4, tbl.TB_GN_PARTS, 2), on("ws", 32, dtype=torch.uint8), on("dw", 4)
    return {
        "dropout": lambda: tbl.tb_dropout(x, y, 0.1, 1, 2, r, s),
        "stats": lambda: tbl.tb_patch_gn_stats_cl([p], 2, rec),
        "apply": lambda: tbl.tb_patch_gn_apply_cl([p], [o], 2, rec, 1, w, w, 1e-6),
        "both": lambda: tbl.patch_group_norm_cl([p], 2, w, w, 1e-6, outs=[o], partials=rec),
        "grad_stats": lambda: tbl.tb_patch_gn_grad_stats_cl([g], [p], 2, rec, 1, w, w, 1e-6, grec),
        "grad_apply": lambda: tbl.tb_patch_gn_grad_apply_cl([g], [p], [o], 2, rec, grec, 1, w, w, 1e-6, ws, dw, dw),
        "grad_both": lambda: tbl.patch_group_norm_backward_cl([g], [p], 2, rec, w, w, 1e-6, dxs=[o], dgamma=dw, dbeta=dw,
                                                              grad_partials=grec, workspace=ws),
    }


USES = {"dropout": "xyrs", "stats": ["p", "rec"], "apply": ["p", "o", "rec", "w"], "both": ["p", "o", "rec", "w"],
        "grad_stats": ["g", "p", "rec", "w", "grec"], "grad_apply": ["g", "p", "o", "rec", "grec", "w", "ws", "dw"],
        "grad_both": ["g", "p", "o", "rec", "grec", "w", "ws", "dw"]}


@pytest.mark.parametrize("call", list(USES))
def test_tensors_of_another_device_are_refused(devices, call):
    _calls(devices, 0)[call]()
    assert devices._lib.calls
    devices._lib.calls.clear()
    with pytest.raises(ValueError):
        _calls(devices, 1)[call]()                     # all of them on a device that is not the current one
    for name in USES[call]:
        with pytest.raises(ValueError):
            _calls(devices, 0, **{name: 1})[call]()
    assert not devices._lib.calls
