"""Host-side refusals of the layer-norm and adapter entry points (CPU only:
every call here is rejected before anything touches a device)."""
import ctypes

import pytest
import torch

from tests.test_abi import q  # noqa: F401  (the built library)

P = ctypes.c_void_p(4096)     # a fake aligned device address: validation fails before any use
ODD = ctypes.c_void_p(4104)   # 8-byte aligned only


def _norm_fwd(q, X=P, dt=1, M=4, K=64, gamma=None, beta=None, eps=1e-6, Y=P):
    return q.lib.qlin_layer_norm_forward(X, dt, M, K, gamma, beta, eps, Y, None, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(K=24), 3), (dict(K=0), 3), (dict(K=32784), 2), (dict(dt=5), 1), (dict(M=-1), 1), (dict(X=None), 1), (dict(X=ODD), 3),
    (dict(gamma=ODD), 3), (dict(beta=ODD), 3), (dict(Y=None), 1), (dict(Y=ODD), 3), (dict(eps=-1.0), 1), (dict(eps=float("inf")), 1),
    (dict(eps=float("nan")), 1), (dict(M=0), 0)])
def test_layer_norm_forward_refusals(q, kw, want):
    assert _norm_fwd(q, **kw) == want


def test_layer_norm_prep_refusals(q):
    f = q.lib.qlin_layer_norm_fp8_prep
    assert f(P, 1, 4, 64, None, None, 1e-6, None, P, None, None) == q.QLIN_ERR_INVALID_ARG   # dynamic scales need s_x
    assert f(P, 1, 4, 64, None, None, 1e-6, None, None, P, None) == q.QLIN_ERR_INVALID_ARG
    assert f(P, 1, 4, 40, None, None, 1e-6, None, P, P, None) == q.QLIN_ERR_ALIGNMENT
    f = q.lib.qlin_layer_norm_w4a8_prep
    assert f(P, 1, 4, 64, None, None, 1e-6, P, None, None) == q.QLIN_ERR_INVALID_ARG
    assert f(P, 1, 4, 64, None, None, 1e-6, ODD, P, None) == q.QLIN_ERR_ALIGNMENT


def _norm_bwd(q, dY=P, X=P, dt=1, M=4, K=64, mean=P, rstd=P, dX=P, dgamma=P, dbeta=P, ws=P, n=None):
    n = q.qlin_workspace_bytes(q.QLIN_OP_LAYER_NORM_BACKWARD, max(M, 0), 0, K) if n is None else n
    return q.lib.qlin_layer_norm_backward(dY, X, dt, M, K, None, mean, rstd, dX, dgamma, dbeta, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(K=24), 3), (dict(K=16400), 2), (dict(dY=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1), (dict(dX=None), 1), (dict(dX=ODD), 3),
    (dict(dgamma=ODD), 3), (dict(ws=None), 4), (dict(n=16), 4), (dict(M=0, dgamma=None, dbeta=None), 0)])
def test_layer_norm_backward_refusals(q, kw, want):
    assert _norm_bwd(q, **kw) == want


def test_layer_norm_workspace(q):
    # two K-column fp32 sums for each CTA, at most one CTA per row
    assert q.qlin_workspace_bytes(q.QLIN_OP_LAYER_NORM_BACKWARD, 1, 0, 4096) == 8 * 4096
    assert q.qlin_workspace_bytes(q.QLIN_OP_LAYER_NORM_BACKWARD, 1 << 20, 0, 4096) <= 8 * 4096 * 4736


def _plan_bytes(q, M, L):
    return q.lib.qlin_lora_plan_bytes(M, L)


def test_plan_sizes(q):
    assert _plan_bytes(q, 0, 1) > 0
    assert _plan_bytes(q, 4, 0) == 0 and _plan_bytes(q, 4, 1025) == 0 and _plan_bytes(q, -1, 2) == 0 and _plan_bytes(q, (1 << 28) + 1, 2) == 0
    for M, L in ((1, 1), (127, 3), (128, 1), (129, 1024), (5000, 7)):
        tiles = M // 128 + min(L, M)
        # header, first tiles, tile records and 128 row numbers a tile
        assert _plan_bytes(q, M, L) >= 4 * (16 + L + 1 + 2 * tiles + 128 * tiles)
        # ceil(rows / 128) summed over adapters stays within `tiles` for the split that needs most
        n = min(L, M)
        rows = [1] * (n - 1) + [M - (n - 1)]
        assert sum((r + 127) // 128 for r in rows) <= tiles


@pytest.mark.parametrize("idx,M,L,plan,short,want", [(None, 4, 2, P, 0, 1), (P, 4, 0, P, 0, 2), (P, 4, 1025, P, 0, 2), (P, -1, 2, P, 0, 1),
                                                     (P, 4, 2, None, 0, 1), (P, 4, 2, ODD, 0, 3), (ODD, 4, 2, P, 0, 3), (P, 4, 2, P, 1, 4)])
def test_plan_refusals(q, idx, M, L, plan, short, want):
    assert q.lib.qlin_lora_plan(idx, M, L, plan, max(_plan_bytes(q, M, L), 64) - short * 32, None) == want


def _fwd(q, X=P, dt=1, M=4, K=64, A=P, B=P, scale=P, L=2, R=16, N=32, plan=P, H=P, Y=P, short=0):
    return q.lib.qlin_lora_forward(X, dt, M, K, A, B, scale, L, R, N, plan, _plan_bytes(q, M, L) - short, H, Y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(K=20), 3), (dict(K=32784), 2), (dict(dt=3), 1), (dict(M=-2), 1), (dict(X=ODD), 3), (dict(A=None), 1), (dict(B=ODD), 3), (dict(scale=None), 1),
    (dict(L=0), 2), (dict(L=1025), 2), (dict(R=12), 3), (dict(R=0), 3), (dict(R=136), 2), (dict(plan=None), 1), (dict(short=4), 4), (dict(H=None, M=500), 1),
    (dict(H=ODD), 3), (dict(Y=None), 1), (dict(N=-1), 1), (dict(N=0), 0), (dict(M=0), 0)])
def test_lora_forward_refusals(q, kw, want):
    assert _fwd(q, **kw) == want


def test_h_is_scratch_for_more_than_a_few_rows(q):
    assert q.lib.qlin_lora_forward_h_bytes(4, 16) == 0 and q.lib.qlin_lora_forward_h_bytes(256, 16) == 0
    assert q.lib.qlin_lora_forward_h_bytes(257, 16) == 4 * 257 * 16 and q.lib.qlin_lora_forward_h_bytes(8, 64) == 4 * 8 * 64
    assert q.lib.qlin_lora_forward_h_bytes(-1, 16) == 0 and q.lib.qlin_lora_forward_h_bytes(8, 0) == 0


def _bwd(q, dY=P, X=P, dt=1, M=4, K=64, L=2, R=16, N=32, H=P, dX=P, dA=P, dB=P, ws=P, n=None):
    n = q.lib.qlin_lora_backward_workspace_bytes(M, R) if n is None else n
    return q.lib.qlin_lora_backward(dY, X, dt, M, K, P, P, P, L, R, N, P, _plan_bytes(q, M, L), H, dX, dA, dB, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=0), 2), (dict(N=36), 3), (dict(N=0), 3), (dict(R=20), 3), (dict(R=144), 2), (dict(L=0), 2), (dict(dY=None), 1), (dict(H=None), 1),
    (dict(dX=ODD), 3), (dict(dA=None), 1), (dict(dB=ODD), 3), (dict(ws=None), 4), (dict(n=256), 4)])
def test_lora_backward_refusals(q, kw, want):
    assert _bwd(q, **kw) == want


def test_binding_refuses_cpu_and_wrong_arguments(q):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: q.qlin_layer_norm_forward(x), lambda: q.qlin_layer_norm_fp8_prep(x), lambda: q.qlin_layer_norm_w4a8_prep(x),
                 lambda: q.qlin_layer_norm_backward(x, x, torch.zeros(4), torch.zeros(4)),
                 lambda: q.qlin_lora_plan(torch.zeros(4, dtype=torch.int32), 2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        q.qlin_lora_plan(torch.zeros(4, dtype=torch.int64), 2)
