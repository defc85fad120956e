"""The training module: gradients of a whole block against torch's float64
autograd of the plain formulas, the clipped step, and the command."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def training():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import training
    return training


def _block(training):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(2, 16, 9, 10, generator=g, device="cuda") + 0.5
    patches = [p.contiguous().requires_grad_() for p in x.split([4, 5], 2)]
    stream = torch.randn(2, 90, 40, generator=g, device="cuda").requires_grad_()
    target = torch.randn(2, 90, 16, generator=g, device="cuda")
    return training.DecoderBlock(16, 40, 4, seed=5), patches, stream, target


def _plain(block, patches, stream, target):
    """The same loss in 64 bits; (loss, gradients of params, patches, stream)."""
    ps = [p.detach().double().requires_grad_() for p in block.params()]
    xs = [p.detach().double().requires_grad_() for p in patches]
    st = stream.detach().double().requires_grad_()
    h = F.silu(F.group_norm(torch.cat(xs, 2), block.groups, ps[0], ps[1], 1e-6))
    t = h.flatten(2).transpose(1, 2) @ ps[2] + st
    y = F.layer_norm(t, (t.shape[-1],), ps[3], ps[4], 1e-6) @ ps[5]
    loss = (y - target.double()).square().mean()
    loss.backward()
    return loss, [t.grad for t in ps + xs + [st]]


def test_gradients_of_the_block(training):
    block, patches, stream, target = _block(training)
    params = block.params()
    trainer = training.Trainer(params, lr=0.5, max_norm=0.25)
    want_loss, want = _plain(block, patches, stream, target)
    before = [p.detach().clone() for p in params]
    loss = (block(patches, stream) - target).square().mean()
    norm = trainer.step(loss)
    # fp32 (torch's fp32 products among it): 1e-4 of each gradient's norm
    assert abs(loss.item() - want_loss.item()) <= 1e-5 * want_loss.item()
    wn = torch.sqrt(sum((w ** 2).sum() for w in want[:len(params)])).item()
    assert abs(norm.item() - wn) <= 1e-4 * wn and wn > 0.25
    coef = 0.25 / (wn + 1e-6)
    for p, b, w in zip(params, before, want):
        assert (p.grad.double() - w * coef).norm() <= 1e-4 * w.norm() * coef
        assert torch.equal(p.detach(), b - 0.5 * p.grad)
    for t, w in zip(patches + [stream], want[len(params):]):
        assert (t.grad.double() - w).norm() <= 1e-4 * w.norm()


def test_steps_lower_the_loss(training):
    block, patches, stream, target = _block(training)
    trainer = training.Trainer(block.params(), lr=0.2, max_norm=1.0)
    losses = []
    for _ in range(30):
        loss = (block([p.detach() for p in patches], stream.detach()) - target).square().mean()
        trainer.step(loss)
        losses.append(loss.item())
    assert np.isfinite(losses).all() and losses[-1] < 0.9 * losses[0]


def test_layer_norm_of_transposed_gradients_and_absent_weights(training):
    x = torch.randn(6, 40, device="cuda").requires_grad_()
    y = training.layer_norm(x, None, None)
    w = torch.randn(40, 6, device="cuda")
    (y.t() * w).sum().backward()           # dy arrives with strided elements
    xd = x.detach().double().requires_grad_()
    (F.layer_norm(xd, (40,), None, None, 1e-6).t() * w.double()).sum().backward()
    assert (x.grad.double() - xd.grad).norm() <= 1e-5 * xd.grad.norm()


def test_the_command_runs(training, capsys):
    training.main(["--steps", "3"])
    out = capsys.readouterr().out.strip().splitlines()
    assert len(out) == 3 and all("gradient norm" in line for line in out)
