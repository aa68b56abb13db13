"""Refusals of the norm, expert-row and dense int8 calls, without a GPU: every
bad argument is turned down before anything is enqueued."""
from __future__ import annotations

import ctypes

import pytest
import torch

from ternary_weight_amd import tq

A, B, C, D, E, F = (0x100000000 * i for i in range(1, 7))        # addresses far apart, never read


def norm(M=4, K=64, xt=tq.F32, x=A, rt=tq.F32, res=None, ro=None, w=B, eps=1e-5, yt=tq.F32, y=C, ys=None):
    return tq.lib().tq_rmsnorm(M, K, xt, x, rt, res, ro, w, eps, yt, y, ys, None)


def test_norm_refusals():
    assert norm(M=-1) == tq.ERR_ARG and norm(K=-16) == tq.ERR_ARG
    for k in (0, 8, 40, 65552):
        assert norm(K=k) == tq.ERR_SHAPE
    assert norm(M=1 << 31) == tq.ERR_SHAPE
    for t in (tq.I8, tq.F32_Q8, -1):
        assert norm(xt=t) == tq.ERR_ARG
        assert norm(rt=t, res=D) == tq.ERR_ARG
    assert norm(yt=tq.F32_Q8) == tq.ERR_ARG
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(eps=eps) == tq.ERR_VALUE
    assert norm(x=None) == tq.ERR_ARG and norm(w=None) == tq.ERR_ARG and norm(y=None) == tq.ERR_ARG
    assert norm(yt=tq.I8) == tq.ERR_ARG                          # no scales
    assert norm(ro=D) == tq.ERR_ARG                              # a sum to store, nothing added
    assert norm(x=A + 4) == tq.ERR_ALIGN and norm(res=D + 8) == tq.ERR_ALIGN and norm(w=B + 4) == tq.ERR_ALIGN
    assert norm(y=C + 4) == tq.ERR_ALIGN and norm(yt=tq.I8, ys=D + 2) == tq.ERR_ALIGN
    # overlaps: a shifted output, another type in place, the sum over x, scales over y
    assert norm(y=A + 256) == tq.ERR_ARG and norm(yt=tq.BF16, y=A) == tq.ERR_ARG
    assert norm(res=D, ro=D + 256) == tq.ERR_ARG and norm(res=D, ro=A) == tq.ERR_ARG
    assert norm(res=D, y=D) == tq.ERR_ARG and norm(yt=tq.I8, ys=C + 64) == tq.ERR_ARG
    assert norm(y=B) == tq.ERR_ARG
    assert norm(M=0, x=None, w=None, y=None) == tq.OK and tq.last_error() == ""


def dispatch(T=6, k=2, n=4, ids=A, rows=B, pairs=C, offs=D, width=0, xt=tq.F32, x=None, xsc=None, xs=None, xss=None,
             ws=None, nws=0):
    return tq.lib().tq_moe_dispatch(T, k, n, ids, rows, pairs, offs, width, xt, x, xsc, xs, xss, ws, nws, None)


def test_dispatch_refusals():
    assert dispatch(T=-1) == tq.ERR_ARG and dispatch(width=-16) == tq.ERR_ARG
    for k in (0, -1, 65):
        assert dispatch(k=k) == tq.ERR_ARG
    for n in (0, 1025):
        assert dispatch(n=n) == tq.ERR_ARG
    assert dispatch(T=(1 << 29) + 1) == tq.ERR_SHAPE
    assert dispatch(width=24, x=E, xs=F) == tq.ERR_SHAPE and dispatch(width=65552, x=E, xs=F) == tq.ERR_SHAPE
    assert dispatch(width=16, x=E, xs=F, xt=tq.F32_Q8) == tq.ERR_ARG
    for name in ("ids", "rows", "pairs", "offs"):
        assert dispatch(**{name: None}) == tq.ERR_ARG
        assert dispatch(**{name: E + 2}) == tq.ERR_ALIGN
    assert dispatch(width=16, x=E) == tq.ERR_ARG                                  # nowhere to copy to
    assert dispatch(width=16, x=E, xs=F + 8) == tq.ERR_ALIGN
    assert dispatch(width=16, x=E, xs=F, xt=tq.I8) == tq.ERR_ARG                  # no scales
    assert dispatch(width=16, x=E, xs=F, xt=tq.I8, xsc=7 * A) == tq.ERR_ARG
    assert dispatch(rows=A) == tq.ERR_ARG and dispatch(pairs=B + 4) == tq.ERR_ARG  # overlaps
    assert dispatch(width=16, x=E, xs=E) == tq.ERR_ARG and dispatch(offs=C + 8) == tq.ERR_ARG
    need = tq.moe_dispatch_workspace_size(10000, 2, 4)
    assert need > 0 and tq.moe_dispatch_workspace_size(64, 8, 128) == 0
    assert tq.moe_dispatch_workspace_size(1, 1, 1024) == 0 and tq.moe_dispatch_workspace_size(1025, 1, 1024) > 0
    assert dispatch(T=10000) == tq.ERR_ARG and dispatch(T=10000, ws=E, nws=need - 1) == tq.ERR_ARG
    assert dispatch(T=10000, ws=E + 4, nws=need) == tq.ERR_ALIGN and dispatch(T=10000, ws=A, nws=need) == tq.ERR_ARG
    with pytest.raises(tq.TQError) as e:
        tq.moe_dispatch_workspace_size(1, 1, 0)
    assert e.value.status == tq.ERR_ARG
    assert tq.lib().tq_moe_dispatch_workspace_size(1, 1, 1, None) == tq.ERR_ARG


def combine(T=6, k=2, H=64, R=12, rows=A, w=B, st=tq.F32, ys=C, yt=tq.F32, y=D):
    return tq.lib().tq_moe_combine(T, k, H, R, rows, w, st, ys, yt, y, None)


def grad(T=6, k=2, H=64, R=12, rows=A, w=B, dt=tq.F32, dy=C, st=tq.F32, ys=D, dys=E, dw=F):
    return tq.lib().tq_moe_combine_grad(T, k, H, R, rows, w, dt, dy, st, ys, dys, dw, None)


def test_combine_refusals():
    for call in (combine, grad):
        assert call(T=-1) == tq.ERR_ARG and call(k=0) == tq.ERR_ARG and call(k=65) == tq.ERR_ARG
        assert call(H=-16) == tq.ERR_ARG and call(H=40) == tq.ERR_SHAPE and call(H=65552) == tq.ERR_SHAPE
        assert call(R=-1) == tq.ERR_ARG and call(R=1 << 31) == tq.ERR_ARG and call(st=tq.I8) == tq.ERR_ARG
        assert call(rows=None) == tq.ERR_ARG and call(rows=7 * A + 2) == tq.ERR_ALIGN
        assert call(w=7 * A + 1) == tq.ERR_ALIGN and call(ys=None) == tq.ERR_ARG and call(ys=7 * A + 8) == tq.ERR_ALIGN
        assert call(T=0) == tq.OK
    assert combine(yt=tq.I8) == tq.ERR_ARG and combine(y=None) == tq.ERR_ARG and combine(y=D + 4) == tq.ERR_ALIGN
    assert combine(y=C + 16) == tq.ERR_ARG and combine(y=A) == tq.ERR_ARG
    assert combine(H=0, rows=None, ys=None, y=None) == tq.OK
    assert grad(dt=tq.I8) == tq.ERR_ARG and grad(dy=None) == tq.ERR_ARG and grad(dys=E + 4) == tq.ERR_ALIGN
    assert grad(dw=F + 2) == tq.ERR_ALIGN and grad(dys=D) == tq.ERR_ARG and grad(dw=B) == tq.ERR_ARG
    assert grad(dys=C, ys=None, dw=None) == tq.ERR_ARG
    assert grad(dys=None, dw=None, rows=None) == tq.OK


def dense(M=4, N=8, K=64, x=A, xs=B, w=C, ws=D, yt=tq.F32, y=E):
    return tq.lib().tq_gemm_dense_i8(M, N, K, x, xs, w, ws, yt, y, None)


def test_dense_refusals():
    assert dense(M=-1) == tq.ERR_ARG and dense(N=-1) == tq.ERR_ARG and dense(K=-16) == tq.ERR_ARG
    assert dense(yt=tq.I8) == tq.ERR_ARG and dense(K=40) == tq.ERR_SHAPE and dense(K=65552) == tq.ERR_SHAPE
    assert dense(M=(1 << 24) + 1) == tq.ERR_SHAPE and dense(N=(1 << 24) + 1) == tq.ERR_SHAPE
    for name in ("x", "xs", "w", "ws", "y"):
        assert dense(**{name: None}) == tq.ERR_ARG
    assert dense(x=A + 8) == tq.ERR_ALIGN and dense(w=C + 8) == tq.ERR_ALIGN
    for name in ("xs", "ws", "y"):
        assert dense(**{name: F + 2}) == tq.ERR_ALIGN
    for at in (A, B, C + 64, D):
        assert dense(y=at) == tq.ERR_ARG
    assert dense(M=0, x=None, xs=None, w=None, ws=None, y=None) == tq.OK and dense(N=0, y=None) == tq.OK


def test_binding_checks_tensors():
    """What the C call cannot see of a tensor: layout, type, length, device."""
    x, w, y = torch.zeros(4, 64), torch.ones(64), torch.zeros(4, 64)
    for bad, text in ((dict(x=torch.zeros(64, 4).t()), "not contiguous"), (dict(x=x.half()), "torch.float16"),
                      (dict(x=x[:3]), "192 elements"), (dict(), "not a GPU tensor")):
        a = dict(x=x, w=w, y=y)
        a.update(bad)
        with pytest.raises(ValueError, match=text):
            tq.rmsnorm(4, 64, tq.F32, a["x"], a["w"], 1e-5, tq.F32, a["y"], stream=0)
    with pytest.raises(ValueError, match="torch.int64"):
        tq.moe_dispatch(4, 2, 8, torch.zeros(4, 2, dtype=torch.int64), A, B, C, stream=0)
    with pytest.raises(ValueError, match="torch.uint8"):
        tq.gemm_dense_i8(1, 1, 16, torch.zeros(16, dtype=torch.uint8), A, B, C, tq.F32, D, stream=0)
    with pytest.raises(ValueError, match="d_weights: 7 elements"):
        tq.moe_combine_grad(4, 2, 64, 8, A, B, tq.F32, C, tq.F32, D, E, torch.zeros(7), stream=0)
    with pytest.raises(tq.TQError):
        tq.gemm_dense_i8(1, 1, 8, A, B, C, D, tq.F32, E, stream=0)
    for bad, error in (([1.0], TypeError), ("x", TypeError)):
        with pytest.raises(error):
            tq.rmsnorm(1, 16, tq.F32, bad, B, 1e-5, tq.F32, C, stream=0)
    with pytest.raises(OverflowError):
        tq.rmsnorm(1, 16, 1 << 40, A, B, 1e-5, tq.F32, C, stream=0)
    with pytest.raises(ValueError, match="xq: 16 elements, needs"):          # a count past 64 bits
        tq.gemm_dense_i8(1 << 60, 1, 1 << 20, torch.zeros(16, dtype=torch.int8), A, B, C, tq.F32, D, stream=0)
    for call in (lambda: tq.rmsnorm(None, 16, tq.F32, A, B, 1e-5, tq.F32, C, stream=0),
                 lambda: tq.moe_combine(1, 1, 16, 1, A, B, tq.F32, C, tq.F32, D, stream=object())):
        with pytest.raises((TypeError, AttributeError)):
            call()
    assert ctypes.sizeof(ctypes.c_void_p) == 8
    with pytest.raises(ValueError, match="workspace_bytes = -1"):       # not the largest size_t
        tq.moe_dispatch(10000, 2, 8, A, B, C, D, workspace=E, workspace_bytes=-1, stream=0)
