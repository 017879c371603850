"""Layer norm of rows whose mean is large beside their spread. With u = 2^-24
and at most D = 80 roundings on a value's way through a sum (as in
test_gpu_layer_norm.py): the row's values are multiples of the type's step in
one binade, so their sums are exact while they need no more than 24 bits: over
65536 bf16 or 8192 fp16 values, beyond that with a rounding for each doubling
(G of them). The mean's own rounding is taken out again, so the differences
d = x - mean are off by u |d| and G u |mean|, and xh by
  E = (G u |mean| + (D + 2) u mean|d|) rstd (1 + |xh|) + (D + 8) u |xh|,
and the mean that is kept by half a step of it, G u |mean| and 2 u mean|d|."""
import numpy as np
import pytest
import torch

from oracle import norm_lora as o

pytestmark = pytest.mark.gpu
U, D = 2.0 ** -24, 80


@pytest.fixture(scope="module")
def q():
    import quantized_w8a8_linear_b200 as q
    torch.cuda.init()
    assert q.qlin_get_device_status(reset=True) == 0
    yield q
    assert q.qlin_get_device_status() == 0


@pytest.mark.parametrize("M,K", [(200, 96), (200, 1040), (300, 4096), (50, 12288), (20, 20480)])
@pytest.mark.parametrize("dtype,mean", [(torch.float16, 2000.0), (torch.float16, -40000.0), (torch.bfloat16, 300.0)])
def test_a_large_mean_costs_no_bits(q, M, K, dtype, mean):
    g = torch.Generator().manual_seed(M + K)
    spread = mean * torch.finfo(dtype).eps * (0.5 + 2 * torch.rand((M, 1), generator=g))     # a few steps of the type
    x = (mean + spread * torch.randn((M, K), generator=g)).to(dtype)
    gamma = (1 + 0.1 * torch.randn(K, generator=g)).to(dtype)
    kept, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    y = q.qlin_layer_norm_forward(x.cuda(), gamma.cuda(), mean=kept, rstd=rstd).double().cpu().numpy()
    want, m64, r64 = o.layer_norm_forward(x, gamma)
    xa, ga = x.double().numpy(), np.abs(gamma.double().numpy())
    d = np.abs(xa - m64[:, None]).mean(axis=1)
    xh = np.abs(xa - m64[:, None]) * r64[:, None]
    G = max(0, int(np.ceil(np.log2(K / (8192 if dtype == torch.float16 else 65536)))))
    e = ((G * U * np.abs(m64) + (D + 2) * U * d) * r64)[:, None] * (1 + xh) + (D + 10) * U * xh
    e = e * ga
    assert (np.abs(y - want) <= e + torch.finfo(dtype).eps / 2 * (np.abs(want) + e) + (2.0 ** -25 if dtype == torch.float16 else 0)).all()
    assert (np.abs(kept.double().cpu().numpy() - m64) <= (1 + G) * U * np.abs(m64) + 2 * U * d).all()


@pytest.mark.parametrize("K", [48, 96, 528, 1040, 3088, 12304, 20480])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rows_of_one_value(q, K, dtype):
    # xh is 0. The rounded mean is off by D u c at most, what is left of that by D u of it.
    c = torch.tensor([0.0, 1.0, -3.0, 10.0, 100.0, 1000.0, -1600.0, 30000.0])
    x = c[:, None].expand(-1, K).to(dtype).contiguous()
    beta = torch.linspace(-1, 1, K).to(dtype)
    y = q.qlin_layer_norm_forward(x.cuda(), None, beta.cuda()).double().cpu()
    off = (D * U) ** 2 * x.double().abs() * 1000.0     # rstd = 1 / sqrt(eps) at most
    assert ((y - beta.double()).abs() <= off + torch.finfo(dtype).eps / 2 * (beta.double().abs() + off) + 2.0 ** -25).all()
    codes, s = q.qlin_layer_norm_w4a8_prep(x.cuda())
    assert ((codes.cpu().double() * s.cpu().double()[:, None]).abs() <= 1.01 * off).all()
