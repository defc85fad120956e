"""The channels-last calls together, as a training step runs them: GroupNorm,
projection, dropout onto the residual stream, layer norm, projection; gradients
against the same block in torch's float64, graphs, and the command."""
import subprocess
import sys

import pytest
import torch
import torch.nn.functional as F

from oracle import dropout as D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def training():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import training
    return training


def _inputs(seed=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, 9, 8, 32, generator=g, dtype=torch.float64)
    stream = torch.randn(2, 72, 48, generator=g, dtype=torch.float64)
    return x.float().cuda(), stream.float().cuda()


def _patches(x):
    return [p.contiguous().requires_grad_() for p in x.split([4, 5], 1)]


def _reference(block, xs, stream, step, grads):
    """The block and its gradients in float64."""
    params = [p.detach().double().cpu().requires_grad_() for p in block.params()]
    gw, gb, up, lw, lb, down = params
    xs = [x.detach().double().cpu().requires_grad_() for x in xs]
    s = stream.detach().double().cpu().requires_grad_()
    h = F.silu(F.group_norm(torch.cat([x.flatten(1, -2) for x in xs], 1).transpose(1, 2), block.groups, gw, gb, 1e-6))
    tokens = h.transpose(1, 2) @ up
    keep = torch.from_numpy(D.bits(0, tokens.numel(), block.seed, step) >= D.threshold(block.dropout)).view(tokens.shape)
    tokens = torch.where(keep, tokens, 0.0) * (65536 / (65536 - D.threshold(block.dropout)))
    y = F.layer_norm(tokens + s, (up.shape[1],), lw, lb, 1e-6) @ down
    return y, torch.autograd.grad(y, [*xs, s, *params], grads.double().cpu())


def _close(a, b, rel):
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    assert (a - b).norm() <= rel * b.norm()


def test_block_and_its_gradients(training):
    x, stream = _inputs()
    xs, stream = _patches(x), stream.requires_grad_()
    block = training.DecoderBlock(32, 48, 4, seed=3, channels_last=True, dropout=0.2)
    y = block(xs, stream, 7)
    dy = torch.randn(y.shape, generator=torch.Generator().manual_seed(2)).cuda()
    got = torch.autograd.grad(y, [*xs, stream, *block.params()], dy)
    want_y, want = _reference(block, xs, stream, 7, dy)
    # products of 48 and 32 terms in tf32 at worst (2^-11 each), everything else in fp32
    _close(y, want_y, 2e-3)
    for a, b in zip(got, want):
        _close(a, b, 4e-3)


def test_channels_last_and_first_agree(training):
    x, stream = _inputs()
    a = training.DecoderBlock(32, 48, 4, seed=3, channels_last=True)
    b = training.DecoderBlock(32, 48, 4, seed=3)
    xs = _patches(x)
    fs = [p.detach().movedim(-1, 1).contiguous().requires_grad_() for p in xs]
    ya, yb = a(xs, stream), b(fs, stream)
    _close(ya, yb, 1e-5 if not torch.backends.cuda.matmul.allow_tf32 else 2e-3)
    ga = torch.autograd.grad(ya.sum(), xs)
    gb = torch.autograd.grad(yb.sum(), fs)
    for p, q in zip(ga, gb):
        _close(p, q.movedim(1, -1), 1e-4 if not torch.backends.cuda.matmul.allow_tf32 else 4e-3)


def test_a_captured_step_draws_new_masks(training):
    x, stream = _inputs()
    block = training.DecoderBlock(32, 48, 4, seed=3, channels_last=True, dropout=0.2)
    xs = [p.contiguous() for p in x.split([4, 5], 1)]
    state = torch.zeros(2, dtype=torch.int64, device="cuda")

    def step():
        y = block(xs, stream, 0, state)
        return [y, *torch.autograd.grad(y.square().mean(), block.params())]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
        state[1] += 1
    for k in range(3):
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        y = block(xs, stream, k)
        want = [y, *torch.autograd.grad(y.square().mean(), block.params())]
        for a, b in zip(got, want):
            _close(a, b, 1e-5)
    assert int(state[1]) == 3


def test_gradients_of_any_layout_and_frozen_inputs(training):
    # gradients that are expanded, or not contiguous; inputs that want none
    g = torch.Generator().manual_seed(4)
    x = torch.randn(5, 7, 24, generator=g).cuda().requires_grad_()
    r = torch.randn(5, 7, 24, generator=g).cuda().requires_grad_()
    keep = torch.from_numpy(D.bits(0, x.numel(), 3, 5) >= D.threshold(0.25)).view(x.shape).cuda()
    gx, gr = torch.autograd.grad(training.dropout(x, 0.25, 3, 5, r).sum(), (x, r))
    scale = torch.tensor(65536 / (65536 - D.threshold(0.25)), device="cuda")
    assert torch.equal(gx, torch.where(keep, scale, torch.zeros_like(scale))) and (gr == 1).all()
    dy = torch.randn(24, 7, 5, generator=g).cuda().permute(2, 1, 0)
    gx, gr = torch.autograd.grad(training.dropout(x, 0.25, 3, 5, r), (x, r), dy)
    assert torch.equal(gx, torch.where(keep, dy * scale, torch.zeros_like(scale))) and torch.equal(gr, dy)
    w, b = torch.ones(24, device="cuda", requires_grad=True), torch.zeros(24, device="cuda")
    y, = training.patch_group_norm_cl([x], 4, w, b)
    want = torch.autograd.grad(y, (x, w), dy.contiguous())
    y, = training.patch_group_norm_cl([x], 4, w, b)
    got = torch.autograd.grad(y, (x, w), dy)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    y, = training.patch_group_norm_cl([x.detach()], 4, w, b)
    assert torch.equal(torch.autograd.grad(y, w, dy)[0], want[1])
    y, = training.patch_group_norm_cl([x], 4, None, None)
    assert torch.isfinite(torch.autograd.grad(y.sum(), x)[0]).all()


def test_the_command_runs(training):
    r = subprocess.run([sys.executable, "-m", "patch_groupnorm_gb300.training", "--steps", "3", "--channels-last",
                        "--dropout", "0.1"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.count("step") == 3 and "nan" not in r.stdout
