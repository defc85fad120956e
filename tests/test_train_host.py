"""CPU-only checks of the training calls: sizes of workspaces and records, and
refusals on the host before a GPU is touched."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def tbl():
    from patch_groupnorm_gb300 import build
    build.build()
    from patch_groupnorm_gb300 import tileblend
    return tileblend


def _ln(tbl, x=16, x_ld=8, res=None, r_ld=0, dt=2, rows=4, cols=8, gamma=16, beta=16, wdt=2, eps=1e-6, total=None,
        t_ld=0, y=16, y_ld=8, mean=None, rstd=None):
    return tbl._lib.tb_layer_norm(x, x_ld, res, r_ld, dt, rows, cols, gamma, beta, wdt, eps, total, t_ld, y, y_ld,
                                  mean, rstd, None)


def test_layer_norm_refuses_before_launch(tbl):
    assert _ln(tbl, dt=3) == tbl.TB_ERR_DTYPE
    assert _ln(tbl, wdt=9) == tbl.TB_ERR_DTYPE
    assert _ln(tbl, dt=2, wdt=1) == tbl.TB_ERR_DTYPE       # bf16 rows with f16 weights
    assert _ln(tbl, dt=0, wdt=2) == tbl.TB_ERR_DTYPE       # f32 rows with bf16 weights
    assert _ln(tbl, rows=-1) == tbl.TB_ERR_SHAPE
    assert _ln(tbl, cols=0) == tbl.TB_ERR_SHAPE
    assert _ln(tbl, x_ld=7) == tbl.TB_ERR_SHAPE
    assert _ln(tbl, y_ld=-8) == tbl.TB_ERR_SHAPE
    assert _ln(tbl, rows=2 ** 40, x_ld=2 ** 40) == tbl.TB_ERR_SHAPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _ln(tbl, eps=eps) == tbl.TB_ERR_SHAPE
    assert _ln(tbl, cols=2 ** 30 + 1, x_ld=2 ** 31, y_ld=2 ** 31) == tbl.TB_ERR_UNSUPPORTED
    assert _ln(tbl, x=None) == tbl.TB_ERR_NULL
    assert _ln(tbl, y=None) == tbl.TB_ERR_NULL
    assert _ln(tbl, res=16, r_ld=8) == tbl.TB_ERR_NULL     # a residual without a total
    assert _ln(tbl, res=16, r_ld=4, total=16, t_ld=8) == tbl.TB_ERR_SHAPE
    assert _ln(tbl, x=17) == tbl.TB_ERR_UNSUPPORTED
    assert _ln(tbl, gamma=17) == tbl.TB_ERR_UNSUPPORTED
    assert _ln(tbl, mean=18) == tbl.TB_ERR_UNSUPPORTED
    assert _ln(tbl, rows=0, x=None, y=None) == tbl.TB_OK   # nothing to do


def _lnb(tbl, dy=16, dy_ld=8, x=16, x_ld=8, dt=2, rows=4, cols=8, mean=16, rstd=16, gamma=16, wdt=2, dtot=None, dt_ld=0,
         dx=16, dx_ld=8, dg=16, db=16, ws=16, wb=1 << 20):
    return tbl._lib.tb_layer_norm_backward(dy, dy_ld, x, x_ld, dt, rows, cols, mean, rstd, gamma, wdt, dtot, dt_ld, dx,
                                           dx_ld, dg, db, ws, wb, None)


def test_layer_norm_backward_refuses_before_launch(tbl):
    assert _lnb(tbl, dt=-1) == tbl.TB_ERR_DTYPE
    assert _lnb(tbl, wdt=1) == tbl.TB_ERR_DTYPE
    assert _lnb(tbl, rows=-2) == tbl.TB_ERR_SHAPE
    assert _lnb(tbl, dy_ld=3) == tbl.TB_ERR_SHAPE
    assert _lnb(tbl, dx_ld=3) == tbl.TB_ERR_SHAPE
    assert _lnb(tbl, dtot=16, dt_ld=3) == tbl.TB_ERR_SHAPE
    assert _lnb(tbl, wb=4 * 8 * 8 - 1) == tbl.TB_ERR_SHAPE          # workspace too small
    assert _lnb(tbl, ws=None) == tbl.TB_ERR_NULL
    assert _lnb(tbl, ws=24) == tbl.TB_ERR_UNSUPPORTED
    assert _lnb(tbl, mean=None) == tbl.TB_ERR_NULL
    assert _lnb(tbl, rstd=None) == tbl.TB_ERR_NULL
    assert _lnb(tbl, dy=None) == tbl.TB_ERR_NULL
    assert _lnb(tbl, db=17) == tbl.TB_ERR_UNSUPPORTED
    # nothing asked for
    assert _lnb(tbl, dx=None, dg=None, db=None, ws=None, wb=0) == tbl.TB_OK
    assert _lnb(tbl, rows=0, dy=None, x=None, mean=None, rstd=None, dg=None, db=None) == tbl.TB_OK


def test_workspace_and_record_sizes(tbl):
    w = tbl._lib.tb_layer_norm_workspace
    assert w(0, 8) == 0
    assert w(3, 100) == 3 * 100 * 8
    assert w(10 ** 6, 4096) == tbl.TB_LN_PARTS * 4096 * 8
    assert w(-1, 8) == -1 and w(4, 0) == -1 and w(1, 2 ** 30 + 1) == -1
    r = tbl._lib.tb_grad_records
    assert r(0) == r(1) == r(tbl.TB_GRAD_TABLE) == tbl.TB_GRAD_PARTS
    assert r(tbl.TB_GRAD_TABLE + 1) == 2 * tbl.TB_GRAD_PARTS
    assert r(-1) == -1 and r(tbl.TB_MAX_GRADS + 1) == -1
    with pytest.raises(ValueError):
        tbl.ln_workspace(4, 0)
    with pytest.raises(ValueError):
        tbl.new_grad_records(tbl.TB_MAX_GRADS + 1)


def test_gradient_calls_refuse_before_launch(tbl):
    ptrs = (ctypes.c_void_p * 2)(16, 32)
    odd = (ctypes.c_void_p * 2)(16, 33)
    null = (ctypes.c_void_p * 2)(16, None)
    n = (ctypes.c_int64 * 2)(5, 7)
    d = (ctypes.c_int32 * 2)(0, 2)
    f = tbl._lib.tb_grad_stats
    assert f(ptrs, n, (ctypes.c_int32 * 2)(0, 3), 2, 16, None) == tbl.TB_ERR_DTYPE
    assert f(ptrs, (ctypes.c_int64 * 2)(5, -1), d, 2, 16, None) == tbl.TB_ERR_SHAPE
    assert f(ptrs, n, d, -1, 16, None) == tbl.TB_ERR_SHAPE
    assert f(ptrs, n, d, tbl.TB_MAX_GRADS + 1, 16, None) == tbl.TB_ERR_UNSUPPORTED
    assert f(ptrs, (ctypes.c_int64 * 2)(5, 2 ** 42 + 1), d, 2, 16, None) == tbl.TB_ERR_UNSUPPORTED
    assert f(odd, n, d, 2, 16, None) == tbl.TB_ERR_UNSUPPORTED
    assert f(null, n, d, 2, 16, None) == tbl.TB_ERR_NULL
    assert f(None, n, d, 2, 16, None) == tbl.TB_ERR_NULL
    assert f(ptrs, n, d, 2, None, None) == tbl.TB_ERR_NULL
    assert f(ptrs, n, d, 2, 20, None) == tbl.TB_ERR_UNSUPPORTED
    c = tbl._lib.tb_grad_clip
    assert c(ptrs, ptrs, n, d, 2, 16, 1024, -1.0, None, None) == tbl.TB_ERR_SHAPE
    assert c(ptrs, ptrs, n, d, 2, 16, 1024, float("nan"), None, None) == tbl.TB_ERR_SHAPE
    assert c(ptrs, ptrs, n, d, 2, 16, -1, 1.0, None, None) == tbl.TB_ERR_SHAPE
    assert c(ptrs, ptrs, n, d, 2, None, 1024, 1.0, None, None) == tbl.TB_ERR_NULL
    assert c(ptrs, null, n, d, 2, 16, 1024, 1.0, None, None) == tbl.TB_ERR_NULL
    assert c(ptrs, None, n, d, 2, 16, 1024, 1.0, None, None) == tbl.TB_ERR_NULL
    assert c(ptrs, odd, n, d, 2, 16, 1024, 1.0, None, None) == tbl.TB_ERR_UNSUPPORTED
    m = tbl._lib.tb_grad_norm
    assert m(16, 1024, None, None) == tbl.TB_ERR_NULL
    assert m(None, 1024, 16, None) == tbl.TB_ERR_NULL
    assert m(16, -1, 16, None) == tbl.TB_ERR_SHAPE
    assert m(16, 1024, 18, None) == tbl.TB_ERR_UNSUPPORTED


def test_groupnorm_backward_refuses_before_launch(tbl):
    ptrs = (ctypes.c_void_p * 4)(16, 32, 48, 64)
    null = (ctypes.c_void_p * 4)(16, 32, None, 64)
    sp = (ctypes.c_int64 * 4)(100, 100, 100, 100)
    f, g = tbl._lib.tb_patch_gn_grad_stats, tbl._lib.tb_patch_gn_grad_apply

    def stats(xs=ptrs, ds=ptrs, P=4, dt=2, N=1, C=64, s=sp, G=32, part=16, R=4, gam=None, bet=None, eps=1e-6, out=16):
        return f(xs, ds, P, dt, N, C, s, G, part, R, gam, bet, eps, 1, out, None)
    assert stats(dt=4) == tbl.TB_ERR_DTYPE
    assert stats(C=60) == tbl.TB_ERR_SHAPE
    assert stats(P=0) == tbl.TB_ERR_SHAPE
    assert stats(R=0) == tbl.TB_ERR_SHAPE
    assert stats(eps=-1.0) == tbl.TB_ERR_SHAPE
    assert stats(s=(ctypes.c_int64 * 4)(100, -1, 100, 100)) == tbl.TB_ERR_SHAPE
    assert stats(P=65) == tbl.TB_ERR_UNSUPPORTED
    assert stats(R=65537) == tbl.TB_ERR_UNSUPPORTED
    assert stats(N=2 ** 20, C=2 ** 10) == tbl.TB_ERR_UNSUPPORTED
    assert stats(xs=null) == tbl.TB_ERR_NULL
    assert stats(ds=null) == tbl.TB_ERR_NULL
    assert stats(s=None) == tbl.TB_ERR_NULL
    assert stats(part=None) == tbl.TB_ERR_NULL
    assert stats(out=None) == tbl.TB_ERR_NULL
    assert stats(gam=17) == tbl.TB_ERR_UNSUPPORTED
    assert stats(ds=(ctypes.c_void_p * 4)(16, 33, 48, 64)) == tbl.TB_ERR_UNSUPPORTED
    assert stats(N=0, part=None, out=None) == tbl.TB_OK

    def apply(outs=ptrs, dg=None, db=None, N=1):
        return g(ptrs, ptrs, outs, 4, 2, N, 64, sp, 32, 16, 16, 4, None, None, 1e-6, 1, dg, db, None)
    assert apply(outs=None) == tbl.TB_ERR_NULL
    assert apply(outs=null) == tbl.TB_ERR_NULL
    assert apply(dg=17) == tbl.TB_ERR_UNSUPPORTED
    assert apply(N=0) == tbl.TB_OK


def test_binding_refuses_cpu_tensors(tbl):
    x, w, r = torch.zeros(2, 8), torch.zeros(8), torch.zeros(2)
    with pytest.raises(ValueError):
        tbl.tb_layer_norm(x, x, w, w, 1e-6)
    with pytest.raises(ValueError):
        tbl.tb_layer_norm_backward(x, x, r, r, w, x, w, w, None)
    with pytest.raises(ValueError):
        tbl.GradTable([x])
    with pytest.raises(ValueError):
        tbl.patch_group_norm_backward([x], [x], 2, torch.zeros(4), None, None, 1e-6, dxs=[x], dgamma=w, dbeta=w,
                                      grad_partials=r)
