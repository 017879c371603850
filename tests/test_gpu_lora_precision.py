"""How many bits the adapters' sums keep, at inputs that show it.

An MMA adds 16 products to its fp32 accumulator and cuts off instead of
rounding. A step is 2^-23 of the sum so far: the sum loses less than one, and
each product, aligned with the sum before they are added, what lies below the
bits kept for that (two or three past the step, going by the sums measured:
16 products lose less than three steps). So an MMA loses less than four
steps, as the elementwise tolerances of the adapters' other tests have it,
and where all products are positive, so that the sum grows evenly, a chain of
n MMAs less than 4 (n + 1) / 2 steps of its result.
"""
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


def _positive(g, shape, dtype, scale=1.0):
    return (scale * (0.5 + torch.rand(shape, generator=g, device="cuda"))).to(dtype)


# 4096 products are 256 MMAs: in eight chains (R <= 64, tiles enough for a CTA an
# SM), in four (R > 64), or cut between the CTAs of a cluster as well
@pytest.mark.parametrize("M,R,chain", [(9700, 16, 32), (9700, 72, 64), (300, 16, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_h_is_summed_in_short_chains(q, M, R, chain, dtype):
    K, N, L = 4096, 64, 2
    g = torch.Generator(device="cuda").manual_seed(M + R)
    X, A, B = _positive(g, (M, K), dtype), _positive(g, (L, R, K), dtype, 1 / 64), _positive(g, (L, N, R), dtype)
    idx = (torch.arange(M, device="cuda") * L // M).to(torch.int32)
    H = torch.zeros((M, R), device="cuda")
    Y = torch.zeros((M, N), dtype=dtype, device="cuda")
    q.qlin_lora_forward(X, A, B, torch.full((L,), 1e-4, device="cuda"), q.qlin_lora_plan(idx, L), Y, H=H)
    h = torch.cat([X[idx == a].double() @ A[a].double().T for a in range(L)])
    # the chains' sums, then at most eight of them (four, and the parts of eight CTAs) added with a rounding each
    tol = 4 * (chain + 1) / 2 * 2.0 ** -23 + 11 * 2.0 ** -24
    assert ((H.double() - h).abs() / h).max().item() <= tol
