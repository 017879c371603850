"""Rows of the layer norm that are not finite, as codes: a NaN stays visible in
the row's scale, or in its codes, and in what the GEMM makes of the row."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import quantized_w8a8_linear_b200 as q
    torch.cuda.init()
    assert q.qlin_get_device_status(reset=True) == 0
    yield q
    assert q.qlin_get_device_status() == 0


def _case(M, K, dtype):
    g = torch.Generator().manual_seed(M + K)
    X = torch.randn((M, K), generator=g).to(dtype).cuda()
    gamma = (1 + 0.1 * torch.randn(K, generator=g)).to(dtype).cuda()
    bad = X.clone()
    bad[1, K // 2] = float("nan")
    bad[3, 0] = float("inf")
    bad[4, K - 1] = -float("inf")
    rows = torch.tensor([1, 3, 4], device="cuda")
    good = torch.ones(M, dtype=torch.bool, device="cuda")
    good[rows] = False
    return X, bad, gamma, rows, good


# a warp a row, several warps, rows whose threads do not all have columns, two-row CTAs' widths
@pytest.mark.parametrize("K", [128, 512, 1040, 4096, 9216, 16384])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_codes_of_rows_that_are_not_finite(q, K, dtype):
    X, bad, gamma, rows, good = _case(9, K, dtype)
    for prep, values in ((q.qlin_layer_norm_w4a8_prep, lambda c: c.float()), (q.qlin_layer_norm_fp8_prep, lambda c: c.view(torch.float8_e4m3fn).float())):
        codes, s = prep(X, gamma)
        got, t = prep(bad, gamma)
        assert torch.equal(got[good], codes[good]) and torch.equal(t[good], s[good])
        assert torch.isnan(values(got[rows]) * t[rows][:, None]).all()
    static, _ = q.qlin_layer_norm_fp8_prep(bad, gamma, x_scale=torch.full((1,), 0.01, device="cuda"))
    assert torch.isnan(static.view(torch.float8_e4m3fn).float()[rows]).all()


@pytest.mark.parametrize("prep", ["w4a8", "fp8"])
def test_nan_in_gamma_reaches_every_row(q, prep):
    X, _, gamma, _, _ = _case(9, 1040, torch.bfloat16)
    gamma[1039] = float("nan")
    codes, s = q.qlin_layer_norm_w4a8_prep(X, gamma) if prep == "w4a8" else q.qlin_layer_norm_fp8_prep(X, gamma)
    assert torch.isnan(s).all()


def test_projections_of_rows_that_are_not_finite(q):
    M, K, N = 9, 1024, 256
    X, bad, gamma, rows, good = _case(M, K, torch.bfloat16)
    W = (0.02 * torch.randn((N, K), generator=torch.Generator().manual_seed(0))).to(torch.bfloat16).cuda()
    W4, s4 = q.qlin_quantize_weight(W, q.QLIN_W_INT4_G128)
    W8, s8 = q.qlin_quantize_weight(W, q.QLIN_W_FP8_CHANNEL)
    for f in (lambda x: q.qlin_w4a8_gemm(*q.qlin_layer_norm_w4a8_prep(x, gamma), W4, s4, torch.bfloat16),
              lambda x: q.qlin_fp8_gemm(*q.qlin_layer_norm_fp8_prep(x, gamma), W8, s8, q.QLIN_W_FP8_CHANNEL, torch.bfloat16)):
        clean, Y = f(X), f(bad)
        assert torch.equal(Y[good], clean[good]) and torch.isnan(Y[rows]).all()
