"""The training calls as autograd functions, and a small training step that
runs them together.

``layer_norm`` and ``patch_group_norm`` take tensors that require gradients;
their backward passes run in the library's kernels, and a second derivative
through them raises an error.  ``Trainer`` keeps a
parameter set's gradient table and clips it by its global norm before a plain
gradient step.

    python -m patch_groupnorm_gb300.training --steps 20

trains a block of a patch-parallel decoder -- GroupNorm and SiLU over patches,
a projection of every position, a layer norm with the residual stream, a
second projection -- on one synthetic target, and prints the loss and the
gradients' norm before the clip.
"""
import argparse
import math
from typing import List, Optional, Sequence, Tuple

import torch

from . import tileblend as tb


def _rows(t: torch.Tensor) -> torch.Tensor:
    """``t``, or a copy if its rows do not have one stride."""
    try:
        tb._row_ld(t, t.shape, t.dtype, t.get_device(), "gradient")
        return t
    except ValueError:
        return t.contiguous()


def _like(grad: Optional[torch.Tensor], weight: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """A weight's gradient in the weight's shape (the kernels see vectors)."""
    return None if grad is None or weight is None else grad.view(weight.shape)


# The gradients are nodes of their own.  A graph made of them (create_graph)
# then reaches back to the norm's inputs and ends in an error: the kernels have
# no second derivatives, and gradients without a node would be taken for
# constants whenever dy is one.

class _LayerNormGrad(torch.autograd.Function):
    @staticmethod
    def forward(ctx, dy, h, mean, rstd, gamma, wdtype, dtotal, needs):
        return tb.layer_norm_backward(dy, h, mean, rstd, gamma, dtotal, wdtype=wdtype, needs=needs)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the layer norm has no second derivative")


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, eps, residual):
        out = tb.layer_norm(x, gamma, beta, eps, residual)
        h = x if residual is None else out[3]
        ctx.save_for_backward(h, out[1], out[2], gamma, beta)
        ctx.set_materialize_grads(False)
        return out[0] if residual is None else (out[0], out[3])

    @staticmethod
    def backward(ctx, dy, dtotal=None):
        x_, gamma_, beta_, _, residual_ = ctx.needs_input_grad
        if dy is None:  # only the sum was used
            return dtotal if x_ else None, None, None, None, dtotal if residual_ else None
        h, mean, rstd, gamma, beta = ctx.saved_tensors
        dx, dgamma, dbeta = _LayerNormGrad.apply(_rows(dy), h, mean, rstd, gamma, None if beta is None else beta.dtype,
                                                 None if dtotal is None else _rows(dtotal),
                                                 (x_ or residual_, gamma_, beta_))
        return dx if x_ else None, _like(dgamma, gamma), _like(dbeta, beta), None, dx if residual_ else None


def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor], eps: float = 1e-6,
               residual: Optional[torch.Tensor] = None):
    """Layer norm over the last axis, differentiable once (a second derivative
    raises).  With a residual: ``(LN(x + residual), x + residual)``."""
    return _LayerNorm.apply(x, gamma, beta, eps, residual)


class _PatchGroupNormGrad(torch.autograd.Function):
    @staticmethod
    def forward(ctx, args, partials, gamma, beta, *dys_and_patches):
        P = len(dys_and_patches) // 2
        G, eps, silu = args
        dxs, dgamma, dbeta = tb.patch_group_norm_backward(dys_and_patches[:P], dys_and_patches[P:], G, partials, gamma,
                                                          beta, eps, silu)
        return dgamma, dbeta, *dxs

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the patch group norm has no second derivative")


class _PatchGroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, G, eps, silu, gamma, beta, *patches):
        partials = tb.new_partials(len(patches), patches[0].shape[0], G, patches[0].device)
        outs = tb.patch_group_norm(patches, G, gamma, beta, eps, silu, partials=partials)
        ctx.save_for_backward(partials, gamma, beta, *patches)
        ctx.args = G, eps, silu
        return tuple(outs)

    @staticmethod
    def backward(ctx, *dys):
        partials, gamma, beta, *patches = ctx.saved_tensors
        dgamma, dbeta, *dxs = _PatchGroupNormGrad.apply(ctx.args, partials, gamma, beta,
                                                        *[d.contiguous() for d in dys], *patches)
        return (None, None, None, _like(dgamma, gamma), _like(dbeta, beta), *dxs)


def patch_group_norm(patches: Sequence[torch.Tensor], G: int, gamma: Optional[torch.Tensor],
                     beta: Optional[torch.Tensor], eps: float = 1e-6, silu: bool = True) -> Tuple[torch.Tensor, ...]:
    """GroupNorm (+ SiLU) of the whole tensor over its patches, differentiable
    once (a second derivative raises)."""
    return _PatchGroupNorm.apply(G, eps, silu, gamma, beta, *patches)


class Trainer:
    """Gradient descent on ``params`` with the gradients clipped to
    ``max_norm`` by their global norm.  The gradients live in buffers made
    once, so their table and its records are made once too."""

    def __init__(self, params: Sequence[torch.Tensor], lr: float, max_norm: float):
        self.params = list(params)
        self.lr, self.max_norm = lr, max_norm
        for p in self.params:
            p.grad = torch.zeros_like(p)
        self.table = tb.GradTable([p.grad for p in self.params])
        self.records = tb.new_grad_records(len(self.params), self.params[0].device)

    def step(self, loss: torch.Tensor) -> torch.Tensor:
        """Backward pass, clip and update; returns the norm before the clip."""
        for p, g in zip(self.params, self.table.grads):
            p.grad = g.zero_()  # a program may have dropped or replaced it since
        loss.backward()
        norm = tb.clip_grad_norm(self.table, self.max_norm, records=self.records)
        with torch.no_grad():
            for p, g in zip(self.params, self.table.grads):
                p -= self.lr * g
        return norm


class DecoderBlock:
    """GroupNorm + SiLU over patches, a projection of every position to
    ``width``, a layer norm with the residual stream, and a projection back."""

    def __init__(self, channels: int, width: int, groups: int, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, scale=1.0, offset=0.0):
            t = torch.randn(shape, generator=g, dtype=torch.float64) * scale + offset
            return t.float().to(device).requires_grad_()
        self.groups = groups
        self.gn = normal(channels, scale=0.1, offset=1.0), normal(channels, scale=0.1)
        self.up = normal(channels, width, scale=1.0 / math.sqrt(channels))
        self.ln = normal(width, scale=0.1, offset=1.0), normal(width, scale=0.1)
        self.down = normal(width, channels, scale=1.0 / math.sqrt(width))

    def params(self) -> List[torch.Tensor]:
        return [*self.gn, self.up, *self.ln, self.down]

    def __call__(self, patches: Sequence[torch.Tensor], stream: torch.Tensor) -> torch.Tensor:
        """patches [N, C, *spatial_p]; ``stream`` [N, positions, width] -> [N, positions, C]."""
        outs = patch_group_norm(patches, self.groups, *self.gn)
        tokens = torch.cat([o.flatten(2) for o in outs], 2).transpose(1, 2) @ self.up
        y, _ = layer_norm(tokens, *self.ln, residual=stream)
        return y @ self.down


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.05)
    ap.add_argument("--max-norm", type=float, default=1.0)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, 64, 32, 32, generator=g, device="cuda")
    patches = [p.contiguous() for p in x.split([20, 12], 2)]
    stream = torch.randn(1, 1024, 128, generator=g, device="cuda")
    target = torch.randn(1, 1024, 64, generator=g, device="cuda") * 0.1
    block = DecoderBlock(64, 128, 8)
    trainer = Trainer(block.params(), a.lr, a.max_norm)
    for k in range(a.steps):
        loss = (block(patches, stream) - target).square().mean()
        norm = trainer.step(loss)
        print("step %3d  loss %.5f  gradient norm %.4f" % (k, loss.item(), norm.item()))


if __name__ == "__main__":
    main()
