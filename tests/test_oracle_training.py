"""The training oracle against independent statements: torch's float64 layer
norm and group norm and their autograd, and central differences."""
import numpy as np
import torch
import torch.nn.functional as F

from oracle import training as T


def test_layer_norm_and_its_gradients_match_torch_in_64_bits():
    g = torch.Generator().manual_seed(1)
    for rows, cols in ((1, 1), (3, 2), (5, 17), (2, 64)):
        x = torch.randn(rows, cols, generator=g, dtype=torch.float64).requires_grad_()
        w = torch.randn(cols, generator=g, dtype=torch.float64).requires_grad_()
        b = torch.randn(cols, generator=g, dtype=torch.float64).requires_grad_()
        dy = torch.randn(rows, cols, generator=g, dtype=torch.float64)
        y = F.layer_norm(x, (cols,), w, b, 1e-5)
        y.backward(dy)
        oy, mean, rstd = T.layer_norm(x.detach().numpy(), w.detach().numpy(), b.detach().numpy(), 1e-5)
        dx, dw, db = T.layer_norm_backward(dy.numpy(), x.detach().numpy(), mean, rstd, w.detach().numpy())
        for a, r in ((oy, y), (dx, x.grad), (dw, w.grad), (db, b.grad)):
            assert np.allclose(a, r.detach().numpy(), rtol=1e-10, atol=1e-10)


def test_group_norm_gradients_match_torch_in_64_bits():
    g = torch.Generator().manual_seed(2)
    for silu in (False, True):
        x = torch.randn(2, 8, 6, 5, generator=g, dtype=torch.float64).requires_grad_()
        w = torch.randn(8, generator=g, dtype=torch.float64).requires_grad_()
        b = torch.randn(8, generator=g, dtype=torch.float64).requires_grad_()
        dy = torch.randn(2, 8, 6, 5, generator=g, dtype=torch.float64)
        y = F.group_norm(x, 4, w, b, 1e-6)
        (F.silu(y) if silu else y).backward(dy)
        cut = [4, 2]
        dxs, dw, db = T.group_norm_backward([p.numpy() for p in dy.split(cut, 2)],
                                            [p.numpy() for p in x.detach().split(cut, 2)], 4, w.detach().numpy(),
                                            b.detach().numpy(), 1e-6, silu)
        assert np.allclose(np.concatenate(dxs, 2), x.grad.numpy(), rtol=1e-9, atol=1e-9)
        assert np.allclose(dw, w.grad.numpy(), rtol=1e-9, atol=1e-9)
        assert np.allclose(db, b.grad.numpy(), rtol=1e-9, atol=1e-9)


def test_layer_norm_gradient_matches_differences():
    rnd = np.random.RandomState(3)
    x, w, b = rnd.randn(3, 9), rnd.randn(9), rnd.randn(9)
    dy, v = rnd.randn(3, 9), rnd.randn(3, 9)
    _, mean, rstd = T.layer_norm(x, w, b, 1e-5)
    dx, _, _ = T.layer_norm_backward(dy, x, mean, rstd, w)
    h = 1e-6
    up, down = (float((T.layer_norm(x + s * v, w, b, 1e-5)[0] * dy).sum()) for s in (h, -h))
    assert abs((up - down) / (2 * h) - float((dx * v).sum())) < 1e-7


def test_clip_matches_torch():
    g = torch.Generator().manual_seed(4)
    ps = [torch.nn.Parameter(torch.zeros(n, dtype=torch.float64)) for n in (3, 1, 20)]
    for p in ps:
        p.grad = torch.randn(p.shape, generator=g, dtype=torch.float64)
    grads = [p.grad.numpy().copy() for p in ps]
    want = torch.nn.utils.clip_grad_norm_(ps, 0.5)
    norm = T.grad_norm(grads)
    assert abs(norm - float(want)) < 1e-12
    c = T.clip_factor(norm, 0.5)
    assert all(np.allclose(p.grad.numpy(), a * c, rtol=1e-12) for p, a in zip(ps, grads))
    assert T.clip_factor(0.1, 0.5) == 1.0
