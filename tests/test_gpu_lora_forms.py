"""Adapters of so many rows that every form of the first product is reached:
clusters of eight, four and two CTAs, one CTA a tile with two or four stages,
several rounds of tiles. Against 64 bits, with the tolerances derived in
test_gpu_lora.py (H in fp32's 24 bits)."""
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


def G(C, parts=8):
    return (4 * (C / 16 + 1) + 2 * parts) * 2.0 ** -23


# rows in tiles of 128: up to 33 and 71 tiles go to clusters of eight and four, 112 to 148 and 371 to 444 to one CTA an SM
@pytest.mark.parametrize("tiles", [16, 33, 34, 71, 72, 111, 112, 148, 149, 300, 375])
@pytest.mark.parametrize("R,dtype", [(8, torch.bfloat16), (64, torch.float16), (64, torch.bfloat16), (72, torch.bfloat16)])
def test_forward_and_gradients_over_many_tiles(q, tiles, R, dtype):
    M, K, N, L = tiles * 128 - 5, 1040, 72, 1
    g = torch.Generator(device="cuda").manual_seed(tiles + R)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    X, A, B = n(M, K).to(dtype), (n(L, R, K) / K ** 0.5).to(dtype), (0.3 * n(L, N, R)).to(dtype)
    Y, scale = n(M, N).to(dtype), torch.full((L,), 0.75, device="cuda")
    idx = torch.zeros(M, dtype=torch.int32, device="cuda")
    idx[::1001] = -1
    on = idx == 0
    plan = q.qlin_lora_plan(idx, L)
    H = torch.zeros((M, R), device="cuda")
    got = q.qlin_lora_forward(X, A, B, scale, plan, Y.clone(), H=H)
    assert torch.equal(got[~on], Y[~on]) and not H[~on].any()
    half, tiny = torch.finfo(dtype).eps / 2, 2.0 ** -25 if dtype == torch.float16 else 0.0
    x, a, b, y = X.double()[on], A[0].double(), B[0].double(), Y.double()[on]
    h, ha = x @ a.T, x.abs() @ a.abs().T
    eh = G(K) * ha
    assert ((H.double()[on] - h).abs() <= eh).all()
    want = y + 0.75 * h @ b.T
    e = 0.75 * (eh + G(3 * R) * (h.abs() + eh)) @ b.abs().T + 2.0 ** -23 * (y.abs() + want.abs())
    assert ((got.double()[on] - want).abs() <= e + half * (want.abs() + e) + tiny).all()
    if dtype != torch.bfloat16:
        return
    dY, dX = n(M, N).to(dtype), n(M, K).to(dtype)
    gX, dA, dB = q.qlin_lora_backward(dY, X, A, B, scale, plan, H, dX=dX.clone())
    assert torch.equal(gX[~on], dX[~on])
    dy, dx, hk = dY.double()[on], dX.double()[on], H.double()[on]
    dh = 0.75 * dy @ b
    ed = 0.75 * G(N) * (dy.abs() @ b.abs())
    dm = dh.abs() + ed
    want = dx + dh @ a
    e = (ed + G(3 * R) * dm) @ a.abs() + 2.0 ** -23 * (dx.abs() + want.abs())
    assert ((gX.double()[on] - want).abs() <= e + half * (want.abs() + e)).all()
    rows = int(on.sum())
    wA, eA = dh.T @ x, (ed + G(3 * rows, 160) * dm).T @ x.abs()
    wB, eB = 0.75 * dy.T @ hk, 0.75 * (G(3 * rows, 160) + 2.0 ** -23) * (dy.abs().T @ hk.abs())
    for got, w, e in ((dA[0], wA, eA), (dB[0], wB, eB)):
        assert ((got.double() - w).abs() <= e + half * (w.abs() + e)).all()
