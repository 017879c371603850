"""Layer norm, quantized projection and adapters run together, as a block
uses them, forward and backward, against the same chain in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import norm_lora as o

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_w8a8_linear_b200 as q
    torch.cuda.init()
    assert q.qlin_get_device_status(reset=True) == 0
    yield q
    assert q.qlin_get_device_status() == 0


def _inputs(M, K, N, L, R, seed):
    g = torch.Generator().manual_seed(seed)
    bf = lambda t: t.to(torch.bfloat16)   # noqa: E731
    idx = torch.randint(-1, L, (M,), generator=g).to(torch.int32)
    return dict(X=bf(torch.randn((M, K), generator=g) + 0.3), gamma=bf(1 + 0.2 * torch.randn(K, generator=g)), beta=bf(0.1 * torch.randn(K, generator=g)),
                W=bf(torch.randn((N, K), generator=g) / K ** 0.5), bias=bf(0.1 * torch.randn(N, generator=g)),
                A=bf(torch.randn((L, R, K), generator=g) / K ** 0.5), B=bf(0.2 * torch.randn((L, N, R), generator=g)),
                scale=0.5 + torch.rand(L, generator=g), idx=idx, dY=bf(torch.randn((M, N), generator=g)))


def _rel(got, want):
    return np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)


@pytest.mark.parametrize("M,K,N,L,R", [(200, 512, 384, 3, 16), (37, 1024, 256, 5, 8)])
def test_fp8_and_w4a8_block_forward(q, M, K, N, L, R):
    """Norm to codes -> quantized GEMM -> adapters on the 16-bit norm. The codes are
    within half a step of the norm (e4m3 2^-4, int8 1/2 of absmax/127), so the
    chain is compared with the GEMM of the kernel's own codes in 64 bits."""
    c = _inputs(M, K, N, L, R, 1)
    d = {k: v.cuda() for k, v in c.items()}
    plan = q.qlin_lora_plan(d["idx"], L)
    xn = q.qlin_layer_norm_forward(d["X"], d["gamma"], d["beta"])
    W8, s8 = q.qlin_quantize_weight(d["W"], q.QLIN_W_FP8_CHANNEL)
    Xq, sx = q.qlin_layer_norm_fp8_prep(d["X"], d["gamma"], d["beta"])
    Y = q.qlin_fp8_gemm(Xq, sx, W8, s8, q.QLIN_W_FP8_CHANNEL, torch.bfloat16, bias=d["bias"])
    base = (Xq.cpu().view(torch.float8_e4m3fn).double() * sx.cpu().double()[:, None]) @ \
        (W8.cpu().view(torch.float8_e4m3fn).double() * s8.cpu().double()).T + c["bias"].double()
    q.qlin_lora_forward(xn, d["A"], d["B"], d["scale"], plan, Y)
    want, _ = o.lora_forward(xn.cpu(), c["A"], c["B"], c["scale"], c["idx"].numpy(), base)
    assert _rel(Y, want) <= 2 * 2.0 ** -8      # two roundings to bf16 (base, sum), half a step each
    # the codes really stand for the norm
    y64, _, _ = o.layer_norm_forward(c["X"], c["gamma"], c["beta"])
    assert _rel(Xq.cpu().view(torch.float8_e4m3fn).double() * sx.cpu().double()[:, None], y64) <= 2.0 ** -4
    W4, s4 = q.qlin_quantize_weight(d["W"], q.QLIN_W_INT4_G128)
    Xi, si = q.qlin_layer_norm_w4a8_prep(d["X"], d["gamma"], d["beta"])
    Y = q.qlin_w4a8_gemm(Xi, si, W4, s4, torch.bfloat16)
    Y2 = Y.clone()
    q.qlin_lora_forward(xn, d["A"], d["B"], d["scale"], plan, Y2)
    want, _ = o.lora_forward(xn.cpu(), c["A"], c["B"], c["scale"], c["idx"].numpy(), Y.cpu())
    assert _rel(Y2, want) <= 2.0 ** -8


@pytest.mark.parametrize("M,K,N,L,R", [(200, 512, 384, 3, 16), (130, 256, 528, 2, 64)])
def test_training_step_gradients(q, M, K, N, L, R):
    """Norm -> frozen 16-bit projection + adapters, and back: every gradient against
    float64 autograd of the same chain. Each kernel's inputs carry the roundings of
    the ones before it (norm, H in fp32, dX base, dX sum): at most four halves of a
    bf16 step normwise."""
    c = _inputs(M, K, N, L, R, 2)
    d = {k: v.cuda() for k, v in c.items()}
    plan = q.qlin_lora_plan(d["idx"], L)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    xn = q.qlin_layer_norm_forward(d["X"], d["gamma"], d["beta"], mean=mean, rstd=rstd)
    Y = q.qlin_fp_linear_forward(xn, d["W"], bias=d["bias"])
    H = torch.empty((M, R), device="cuda")
    q.qlin_lora_forward(xn, d["A"], d["B"], d["scale"], plan, Y, H=H)
    Wt = d["W"].t().contiguous()                      # the frozen weight's transpose, laid out once
    dxn = q.qlin_fp_linear_forward(d["dY"], Wt)
    dxn, dA, dB = q.qlin_lora_backward(d["dY"], xn, d["A"], d["B"], d["scale"], plan, H, dX=dxn)
    dX, dgamma, dbeta = q.qlin_layer_norm_backward(dxn, d["X"], mean, rstd, gamma=d["gamma"])

    p = {k: v.double().requires_grad_(k in ("X", "gamma", "beta", "A", "B")) for k, v in c.items() if k != "idx"}
    x64 = torch.nn.functional.layer_norm(p["X"], (K,), p["gamma"], p["beta"], 1e-6)
    on = (c["idx"] >= 0).double()[:, None]
    at = c["idx"].clamp(min=0).long()
    h = torch.einsum("mk,mrk->mr", x64, p["A"][at])
    y64 = x64 @ p["W"].T + p["bias"] + on * p["scale"][at][:, None] * torch.einsum("mr,mnr->mn", h, p["B"][at])
    y64.backward(p["dY"])
    tol = 4 * 2.0 ** -8
    for name, got, want in (("Y", Y, y64.detach()), ("dX", dX, p["X"].grad), ("dgamma", dgamma, p["gamma"].grad), ("dbeta", dbeta, p["beta"].grad),
                            ("dA", dA, p["A"].grad), ("dB", dB, p["B"].grad)):
        assert _rel(got, want.numpy()) <= tol, name
