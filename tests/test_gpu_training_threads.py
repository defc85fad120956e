"""Several host threads in the training calls at once, each on its own stream:
every launch succeeds and gives the bits that it gives alone."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tbl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import tileblend
    return tileblend


# pairs of widths that one kernel takes with different amounts of shared memory
@pytest.mark.parametrize("widths", [(8192, 4104), (8191, 4097), (2048, 1032), (512, 264)])
def test_backward_passes_of_different_widths(tbl, widths):
    def inputs(cols, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x, dy = (torch.randn(6, cols, generator=g, device="cuda").bfloat16() for _ in range(2))
        gamma = torch.randn(cols, generator=g, device="cuda").bfloat16()
        _, mean, rstd = tbl.layer_norm(x, gamma, gamma, 1e-6)
        outs = [torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)]
        return dy, x, mean, rstd, gamma, *outs, tbl.ln_workspace(6, cols)
    work = [inputs(c, k) for k, c in enumerate(widths)]
    want = []
    for w in work:
        tbl.tb_layer_norm_backward(*w)
        want.append([t.clone() for t in w[5:8]])
    torch.cuda.synchronize()
    streams, errors = [torch.cuda.Stream() for _ in work], []
    start = threading.Barrier(len(work))

    def loop(k):
        start.wait()
        try:
            for _ in range(3000):
                tbl.tb_layer_norm_backward(*work[k], stream=streams[k])
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)
    threads = [threading.Thread(target=loop, args=(k,)) for k in range(len(work))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors, errors
    for w, o in zip(work, want):
        assert all(torch.equal(a, b) for a, b in zip(w[5:8], o))
