"""CPU-only checks of the channels-last calls: sizes, and refusals on the host
before a GPU is touched."""
import ctypes
import os
import re

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "patch_groupnorm_gb300", "csrc")


@pytest.fixture(scope="module")
def tbl():
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import tileblend
    return tileblend


def _ptrs(*at):
    return (ctypes.c_void_p * max(1, len(at)))(*at)


def _sizes(*n):
    return (ctypes.c_int64 * max(1, len(n)))(*n)


class Call:
    """One call of each kind with the same arguments; results are statuses."""

    def __init__(self, tbl, patches=(16,), grads=(16,), outs=(16,), P=1, dt=2, N=1, C=8, sp=(4,), G=2, part=16, R=1,
                 gamma=None, beta=None, eps=1e-6, grec=16, dg=None, db=None, ws=16, wb=1 << 20):
        lib = tbl._lib
        x, d, o = (None if t is None else _ptrs(*t) for t in (patches, grads, outs))
        s = None if sp is None else _sizes(*sp)
        self.calls = {
            "stats": lambda: lib.tb_patch_gn_stats_cl(x, P, dt, N, C, s, G, part, None),
            "apply": lambda: lib.tb_patch_gn_apply_cl(x, o, P, dt, N, C, s, G, part, R, gamma, beta, eps, 1, None),
            "both": lambda: lib.tb_patch_group_norm_cl(x, o, P, dt, N, C, s, G, part, gamma, beta, eps, 1, None),
            "grad_stats": lambda: lib.tb_patch_gn_grad_stats_cl(x, d, P, dt, N, C, s, G, part, R, gamma, beta, eps, 1,
                                                                grec, None),
            "grad_apply": lambda: lib.tb_patch_gn_grad_apply_cl(x, d, o, P, dt, N, C, s, G, part, grec, R, gamma, beta,
                                                                eps, 1, dg, db, ws, wb, None),
            "grad_both": lambda: lib.tb_patch_group_norm_backward_cl(x, d, o, P, dt, N, C, s, G, part, grec, gamma,
                                                                     beta, eps, 1, dg, db, ws, wb, None),
        }

    def all(self, status, *names):
        for n in names or self.calls:
            assert self.calls[n]() == status, n


FORWARD, BACKWARD = ("stats", "apply", "both"), ("grad_stats", "grad_apply", "grad_both")
APPLY = ("apply", "both", "grad_stats", "grad_apply", "grad_both")


def test_group_norm_refuses_before_launch(tbl):
    def refused(status, *names, **at):
        Call(tbl, **at).all(status, *names)
    refused(tbl.TB_ERR_DTYPE, dt=3)
    refused(tbl.TB_ERR_SHAPE, P=0)
    refused(tbl.TB_ERR_SHAPE, N=-1)
    refused(tbl.TB_ERR_SHAPE, C=-2)
    refused(tbl.TB_ERR_SHAPE, G=0)
    refused(tbl.TB_ERR_SHAPE, G=3)                                        # 8 channels in 3 groups
    refused(tbl.TB_ERR_SHAPE, "apply", "grad_stats", "grad_apply", R=0)
    refused(tbl.TB_ERR_SHAPE, sp=(-1,))
    for eps in (-1.0, float("nan"), float("inf")):
        refused(tbl.TB_ERR_SHAPE, *APPLY, eps=eps)
    refused(tbl.TB_ERR_UNSUPPORTED, P=65, patches=(16,) * 65, grads=(16,) * 65, outs=(16,) * 65, sp=(1,) * 65)
    refused(tbl.TB_ERR_UNSUPPORTED, C=tbl.TB_GN_CL_MAX_CHANNELS + 2)
    refused(tbl.TB_ERR_UNSUPPORTED, "apply", "grad_stats", "grad_apply", R=65537)
    refused(tbl.TB_ERR_UNSUPPORTED, N=1 << 40)                            # records past their limit
    refused(tbl.TB_ERR_UNSUPPORTED, sp=(1 << 42,))
    refused(tbl.TB_ERR_NULL, patches=None)
    refused(tbl.TB_ERR_NULL, patches=(None,))
    refused(tbl.TB_ERR_NULL, sp=None)
    refused(tbl.TB_ERR_NULL, part=None)
    refused(tbl.TB_ERR_NULL, "apply", "both", "grad_apply", "grad_both", outs=None)
    refused(tbl.TB_ERR_NULL, "apply", "both", "grad_apply", "grad_both", outs=(None,))
    refused(tbl.TB_ERR_NULL, *BACKWARD, grads=None)
    refused(tbl.TB_ERR_NULL, *BACKWARD, grads=(None,))
    refused(tbl.TB_ERR_NULL, *BACKWARD, grec=None)
    refused(tbl.TB_ERR_NULL, "grad_apply", "grad_both", ws=None)
    refused(tbl.TB_ERR_SHAPE, "grad_apply", "grad_both", wb=31)
    refused(tbl.TB_ERR_UNSUPPORTED, patches=(17,))
    refused(tbl.TB_ERR_UNSUPPORTED, part=24)
    refused(tbl.TB_ERR_UNSUPPORTED, *APPLY, gamma=17)
    refused(tbl.TB_ERR_UNSUPPORTED, *APPLY, beta=17)
    refused(tbl.TB_ERR_UNSUPPORTED, "apply", "both", outs=(17,))
    refused(tbl.TB_ERR_UNSUPPORTED, *BACKWARD, grads=(17,))
    refused(tbl.TB_ERR_UNSUPPORTED, *BACKWARD, grec=8)
    refused(tbl.TB_ERR_UNSUPPORTED, "grad_apply", "grad_both", dg=17)
    refused(tbl.TB_ERR_UNSUPPORTED, "grad_apply", "grad_both", ws=8)
    # nothing to do
    refused(tbl.TB_OK, N=0, part=None, grec=None, ws=None, patches=(None,), grads=(None,), outs=(None,))
    refused(tbl.TB_OK, C=0, part=None, grec=None, ws=None, patches=(None,), grads=(None,), outs=(None,))


def test_workspace_sizes(tbl):
    w = tbl._lib.tb_patch_gn_workspace_cl
    assert w(0, 4) == 0 and w(1, 1) == 16 and w(3, 32) == 3 * 32 * 16
    assert w(-1, 4) == -1 and w(1, 0) == -1 and w(1, tbl.TB_GN_CL_MAX_CHANNELS + 1) == -1


def _drop(tbl, x=16, x_ld=8, r=None, r_ld=0, dt=2, rows=4, cols=8, p=0.1, seed=1, offset=2, state=None, y=16, y_ld=8):
    return tbl._lib.tb_dropout(x, x_ld, r, r_ld, dt, rows, cols, p, seed, offset, state, y, y_ld, None)


def test_dropout_refuses_before_launch(tbl):
    assert _drop(tbl, dt=5) == tbl.TB_ERR_DTYPE
    assert _drop(tbl, rows=-1) == tbl.TB_ERR_SHAPE
    assert _drop(tbl, cols=-1) == tbl.TB_ERR_SHAPE
    for p in (-0.1, 1.1, float("nan"), float("inf")):
        assert _drop(tbl, p=p) == tbl.TB_ERR_SHAPE
    assert _drop(tbl, x_ld=7) == tbl.TB_ERR_SHAPE
    assert _drop(tbl, y_ld=7) == tbl.TB_ERR_SHAPE
    assert _drop(tbl, r=16, r_ld=7) == tbl.TB_ERR_SHAPE
    assert _drop(tbl, x=None) == tbl.TB_ERR_NULL
    assert _drop(tbl, y=None) == tbl.TB_ERR_NULL
    assert _drop(tbl, rows=1 << 30, cols=1 << 11, x_ld=1 << 11, y_ld=1 << 11) == tbl.TB_ERR_UNSUPPORTED
    assert _drop(tbl, x=17) == tbl.TB_ERR_UNSUPPORTED
    assert _drop(tbl, y=17) == tbl.TB_ERR_UNSUPPORTED
    assert _drop(tbl, r=17, r_ld=8) == tbl.TB_ERR_UNSUPPORTED
    assert _drop(tbl, state=12) == tbl.TB_ERR_UNSUPPORTED
    assert _drop(tbl, rows=0, x=None, y=None) == tbl.TB_OK
    assert _drop(tbl, cols=0, x=None, y=None) == tbl.TB_OK


def test_bindings_refuse_cpu_tensors(tbl):
    x = torch.zeros(1, 4, 8)
    part = torch.zeros(1, 1, 2, 8, 2, dtype=torch.int64)
    for call in (lambda: tbl.tb_dropout(x, x, 0.1, 1), lambda: tbl.dropout(x, 0.1, 1),
                 lambda: tbl.patch_group_norm_cl([x], 2, None, None, 1e-6, partials=part),
                 lambda: tbl.tb_patch_gn_stats_cl([x], 2, part)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("name", ["tb_gncl.cuh", "tb_gncl.cu", "tb_gncl_bwd.cu", "tb_gncl_fused.cu", "tb_dropout.cu"])
def test_kernels_launched_early_read_coherently(name):
    # records, constants, states and tensors may be written while these kernels are resident
    # already, so none is read through the read-only path
    source = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert not re.findall(r"__ldg\s*\(|\.nc\b|__restrict__", source)


@pytest.mark.parametrize("name", ["tb_gncl.cuh", "tb_gncl.cu", "tb_gncl_bwd.cu", "tb_gncl_fused.cu", "tb_dropout.cu"])
def test_accesses_of_global_memory_are_behind_checks(name):
    # in the bounds-checked build: whatever function reads or writes a tensor, a weight or a
    # record by address checks it, or calls one that does
    source = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    access = (r"__ldcs\(|__stcs\(|cp\.async\.cg|from\[\d\]|\*at = |\*reinterpret_cast<(?:const )?(?:W|longlong2|uint4)\*>"
              r"|at->n|weight_at\(w")
    for f in re.split(r"\n(?=(?:template|__device__|__global__|static|inline|struct)\b)", source):
        if re.search(access, f):
            assert re.search(r"in_bounds\(|index_ok\(", f), f[:200]
    # single elements and weights go through the checked helpers
    assert not re.search(r"(?<!cl_)(?:\bweight_at|\bstore_weight)\((?!w, DT)", source)
    for call in re.findall(r"(?:cl_elem<DT>|cl_store_elem<DT>|load_unit<(?:true|false)>)\(.*?[;?]", source, re.S):
        assert "status" in call, call
    # what is left of the last block: all three tensors
    if name == "tb_dropout.cu":
        rest = source[source.index("if (e < rest)"):source.index("pack<DT, 1>(f);")]
        assert [t for t in ("x", "res", "y") if "in_bounds(%s + i * ES" % t in rest] == ["x", "res", "y"]


def test_bindings_refuse_patches_without_channels(tbl):
    for x in (torch.zeros(()), torch.zeros(8)):
        for call in (lambda: tbl.patch_group_norm_cl([x], 2, None, None, 1e-6), lambda: tbl.patch_group_norm_cl([], 2, None, None, 1e-6),
                     lambda: tbl.patch_group_norm_backward_cl([x], [x], 2, None, None, None, 1e-6)):
            with pytest.raises(ValueError):
                call()
