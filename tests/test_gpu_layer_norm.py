"""GPU layer norm (forward, fused codes, backward) against the 64-bit oracle.

Tolerances, elementwise. u = 2^-24 is half a step of fp32; h = eps / 2 half a
step of the output type (eps of torch.finfo). A sum of K values by a thread
(8 V <= 64 of them), a warp (5 levels) and a CTA (4 levels) has at most
D = 80 roundings on any value's way, so it is off by at most D u sum|v|.
  mean: D u mean|x|;  x - mean adds u |x - mean|;
  var (from differences, relative): 2 (D u mean|x| rstd + u) + D u, rstd half of that plus 4 u
  xh:  E = D u rstd mean|x| * (1 + |xh|) + (D + 8) u |xh|
  y = xh gamma + beta: E |gamma| + 2 u (|xh gamma| + |y|), then h |y| for the output's rounding
      (and half the smallest subnormal of fp16, 2^-25).
Codes: y / s_x rounded to a code is half a code's step off (e4m3: 2^-4 of the
value, at least 2^-10; int8: 1/2), with s_x off by the error of the row's
largest |y|. Backward, with the given mean and rstd: xh is off by 2 u |xh| +
u rstd |x - mean|; the row sums by D u sum|.|; dX by rstd times
(4 u |d| + D u (mean|d| + |xh| mean|d xh|) + 4 u |xh| mean|d xh|); column sums
over M rows of products of two roundings each by (M + 4) u sum|.| (each CTA
adds its rows one after another, then the CTAs' sums are added).
"""
import numpy as np
import pytest
import torch

from oracle import norm_lora as o

pytestmark = pytest.mark.gpu

U, D = 2.0 ** -24, 80
SHAPES = [(1, 16), (1, 4096), (3, 48), (13, 1040), (37, 4096), (5, 8192), (600, 528), (700, 2064), (2, 32768), (9, 12288),
          (640, 4096), (650, 12304), (620, 32768), (1500, 16), (300, 8208), (5, 16384), (7, 16400), (4, 24576), (3, 24592)]


@pytest.fixture(scope="module")
def q():
    import quantized_w8a8_linear_b200 as q
    torch.cuda.init()
    assert q.qlin_get_device_status(reset=True) == 0
    yield q
    assert q.qlin_get_device_status() == 0


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def _case(M, K, dtype, affine, seed=0):
    g = torch.Generator().manual_seed(seed + M * 7 + K)
    x = torch.randn((M, K), generator=g) + 0.5
    x[:, 3 % K] += 40.0                      # a channel of large values
    x[M // 2] *= 100.0
    gamma = (1 + 0.3 * torch.randn(K, generator=g)).to(dtype) if affine else None
    beta = (0.2 * torch.randn(K, generator=g)).to(dtype) if affine else None
    return x.to(dtype), gamma, beta, torch.randn((M, K), generator=g).to(dtype)


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _forward_error(x, gamma, beta, eps):
    """(y64, mean, rstd, elementwise error of y before its rounding)"""
    y, mean, rstd = o.layer_norm_forward(x, gamma, beta, eps)
    xa = x.double().numpy()
    ga = np.ones(xa.shape[1]) if gamma is None else gamma.double().numpy()
    xh = (xa - mean[:, None]) * rstd[:, None]
    r = rstd[:, None] * np.abs(xa).mean(axis=1, keepdims=True)
    E = D * U * r * (1 + np.abs(xh)) + (D + 8) * U * np.abs(xh)
    return y, mean, rstd, E * np.abs(ga) + 2 * U * (np.abs(xh * ga) + np.abs(y))


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("affine", [True, False])
def test_forward(q, M, K, dtype, affine):
    x, gamma, beta, _ = _case(M, K, dtype, affine)
    eps = 1e-5
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    got = q.qlin_layer_norm_forward(*_cuda(x, gamma, beta), eps=eps, mean=mean, rstd=rstd).double().cpu().numpy()
    y, m64, r64, err = _forward_error(x, gamma, beta, eps)
    assert (np.abs(got - y) <= err * 1.01 + _half(dtype) * np.abs(y) * 1.01 + _tiny(dtype)).all()
    xa = np.abs(x.double().numpy()).mean(axis=1)
    assert (np.abs(mean.cpu().numpy() - m64) <= D * U * xa).all()
    assert (np.abs(rstd.cpu().numpy() / r64 - 1) <= D * U * xa * r64 + (D / 2 + 8) * U).all()


@pytest.mark.parametrize("M,K", [(1, 16), (13, 1040), (640, 528), (37, 4096), (2, 32768)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("affine", [True, False])
def test_fp8_codes(q, M, K, dtype, affine):
    x, gamma, beta, _ = _case(M, K, dtype, affine, 1)
    y, _, _, err = _forward_error(x, gamma, beta, 1e-6)
    codes, s = q.qlin_layer_norm_fp8_prep(*_cuda(x, gamma, beta))
    dec = codes.cpu().view(torch.float8_e4m3fn).double().numpy()
    s = s.double().cpu().numpy()
    s64 = np.abs(y).max(axis=1) / 448
    assert (np.abs(s - s64) <= err.max(axis=1) / 448 + 4 * U * s64).all()
    t = y / s[:, None]                        # the value the code stands for, at the kernel's own scale
    terr = err / s[:, None] + 4 * U * np.abs(t)
    assert (np.abs(dec - t) <= np.maximum(2.0 ** -4 * (np.abs(t) + terr), 2.0 ** -10) + terr).all()
    # static scale: absmax of another batch, so some values saturate
    xs = torch.tensor([float(np.abs(y).max()) / 448 / 1.5], dtype=torch.float32)
    codes, none = q.qlin_layer_norm_fp8_prep(*_cuda(x, gamma, beta), x_scale=xs.cuda())
    assert none is None
    t = np.clip(y / float(xs), -448, 448)
    terr = err / float(xs) + 4 * U * np.abs(t)
    dec = codes.cpu().view(torch.float8_e4m3fn).double().numpy()
    assert (np.abs(dec - t) <= np.maximum(2.0 ** -4 * (np.abs(t) + terr), 2.0 ** -10) + terr).all()


@pytest.mark.parametrize("M,K", [(1, 128), (13, 1152), (640, 512), (37, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_int8_codes(q, M, K, dtype):
    x, gamma, beta, _ = _case(M, K, dtype, True, 2)
    y, _, _, err = _forward_error(x, gamma, beta, 1e-6)
    codes, s = q.qlin_layer_norm_w4a8_prep(*_cuda(x, gamma, beta))
    s = s.double().cpu().numpy()
    s64 = np.abs(y).max(axis=1) / 127
    assert (np.abs(s - s64) <= err.max(axis=1) / 127 + 4 * U * s64).all()
    t = y / s[:, None]
    assert (np.abs(codes.cpu().double().numpy() - t) <= 0.5 + err / s[:, None] + 4 * U * np.abs(t)).all()
    assert codes.abs().max().item() <= 127


def test_constant_and_zero_rows(q):
    # var = 0: rstd = 1 / sqrt(eps), y = beta exactly; without beta the codes and their scale are 0
    x = torch.full((3, 256), 2.5, dtype=torch.bfloat16, device="cuda")
    x[1] = 0.0
    beta = torch.randn(256, device="cuda").to(torch.bfloat16)
    assert torch.equal(q.qlin_layer_norm_forward(x, None, beta), beta.expand(3, 256))
    for prep in (q.qlin_layer_norm_fp8_prep, q.qlin_layer_norm_w4a8_prep):
        codes, s = prep(x)
        assert not codes.any() and not s.any()


def test_rows_with_nan_and_inf_stay_alone(q):
    x, gamma, beta, dy = _cuda(*_case(40, 1040, torch.bfloat16, True, 3))
    clean = q.qlin_layer_norm_forward(x, gamma, beta)
    bad = x.clone()
    bad[5, 7], bad[20, 0] = float("nan"), float("inf")
    got = q.qlin_layer_norm_forward(bad, gamma, beta)
    keep = [i for i in range(40) if i not in (5, 20)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[5]).all() and torch.isnan(got[20, 0])


BWD = [(1, 16), (1, 4096), (13, 1040), (37, 4096), (5, 8192), (700, 528), (1500, 2064), (9, 12288), (3, 16384),
       (2, 512), (9, 1024), (3000, 1008), (5000, 160), (2500, 496), (700, 4096), (350, 16384)]


@pytest.mark.parametrize("M,K", BWD)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("affine", [True, False])
def test_backward(q, M, K, dtype, affine):
    x, gamma, _, dy = _case(M, K, dtype, affine, 4)
    _, m64, r64 = o.layer_norm_forward(x, eps=1e-5)
    mean, rstd = torch.from_numpy(m64).float(), torch.from_numpy(r64).float()
    dx, dg, db = q.qlin_layer_norm_backward(*_cuda(dy, x, mean, rstd), gamma=None if gamma is None else gamma.cuda())
    want, wg, wb = o.layer_norm_backward(dy, x, mean, rstd, gamma)
    xa, dya, r = x.double().numpy(), dy.double().numpy(), rstd.double().numpy()[:, None]
    diff = np.abs(xa - mean.double().numpy()[:, None])
    xh = diff * r
    xh_err = 2 * U * xh + U * r * diff
    d = np.abs(dya) * (1.0 if gamma is None else np.abs(gamma.double().numpy()))
    md, mdx = d.mean(axis=1, keepdims=True), (d * xh).mean(axis=1, keepdims=True)
    err = r * (4 * U * d + (D + 4) * U * (md + xh * mdx) + 4 * U * xh * mdx) + 4 * U * np.abs(want)
    h = _half(dtype)
    assert (np.abs(dx.double().cpu().numpy() - want) <= 1.01 * (err + h * np.abs(want)) + _tiny(dtype)).all()
    if gamma is None:
        assert dg is None and db is None
        return
    eg = (M + 4) * U * (np.abs(dya) * xh).sum(axis=0) + (np.abs(dya) * xh_err).sum(axis=0)
    eb = (M + 4) * U * np.abs(dya).sum(axis=0)
    assert (np.abs(dg.double().cpu().numpy() - wg) <= 1.01 * (eg + h * np.abs(wg)) + _tiny(dtype)).all()
    assert (np.abs(db.double().cpu().numpy() - wb) <= 1.01 * (eb + h * np.abs(wb)) + _tiny(dtype)).all()


def test_backward_outputs_asked_for(q):
    x, gamma, _, dy = _cuda(*_case(300, 528, torch.bfloat16, True, 5))
    mean, rstd = torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    q.qlin_layer_norm_forward(x, gamma, mean=mean, rstd=rstd)
    dx, dg, db = q.qlin_layer_norm_backward(dy, x, mean, rstd, gamma=gamma)
    a = q.qlin_layer_norm_backward(dy, x, mean, rstd, gamma=gamma, beta_grad=False)
    assert torch.equal(a[0], dx) and torch.equal(a[1], dg) and a[2] is None
    b = q.qlin_layer_norm_backward(dy, x, mean, rstd, beta_grad=True)   # beta without gamma
    assert b[1] is None and torch.equal(b[2], db)
    # in place: dX over dY, over X
    for into in ("dY", "X"):
        t = {"dY": dy.clone(), "X": x.clone()}
        got = q.qlin_layer_norm_backward(t["dY"], t["X"], mean, rstd, gamma=gamma, dX=t[into])
        assert got[0] is t[into] and torch.equal(got[0], dx) and torch.equal(got[1], dg)
    e = torch.empty((0, 528), dtype=torch.bfloat16, device="cuda")
    z = torch.empty(0, device="cuda")
    _, dg0, db0 = q.qlin_layer_norm_backward(e, e, z, z, gamma=gamma)
    assert not dg0.any() and not db0.any()
    assert q.qlin_layer_norm_forward(e).shape == (0, 528)


def test_forward_in_place_and_same_bits_again(q):
    x, gamma, beta, dy = _cuda(*_case(1000, 4096, torch.bfloat16, True, 6))
    want = q.qlin_layer_norm_forward(x, gamma, beta)
    y = x.clone()
    assert torch.equal(q.qlin_layer_norm_forward(y, gamma, beta, Y=y), want)
    mean, rstd = torch.empty(1000, device="cuda"), torch.empty(1000, device="cuda")
    q.qlin_layer_norm_forward(x, gamma, mean=mean, rstd=rstd)
    first = q.qlin_layer_norm_backward(dy, x, mean, rstd, gamma=gamma)
    for _ in range(3):
        again = q.qlin_layer_norm_backward(dy, x, mean, rstd, gamma=gamma)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_streams_and_graph(q):
    x, gamma, beta, dy = _cuda(*_case(257, 1040, torch.bfloat16, True, 7))
    mean, rstd = torch.empty(257, device="cuda"), torch.empty(257, device="cuda")
    want = q.qlin_layer_norm_forward(x, gamma, beta, mean=mean, rstd=rstd)
    grads = q.qlin_layer_norm_backward(dy, x, mean, rstd, gamma=gamma)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = [q.qlin_layer_norm_backward(dy, x, mean, rstd, gamma=gamma) for _ in range(3)]
    b = [q.qlin_layer_norm_backward(dy, x, mean, rstd, gamma=gamma) for _ in range(3)]   # beside the side stream's
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for t in a + b for u, v in zip(t, grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = q.qlin_layer_norm_forward(x, gamma, beta, mean=mean, rstd=rstd)
        out = q.qlin_layer_norm_backward(dy, x, mean, rstd, gamma=gamma)
    dy2 = dy.flip(0).contiguous()
    want2 = q.qlin_layer_norm_backward(dy2, x, mean, rstd, gamma=gamma)
    dy.copy_(dy2)
    for t in (y, *out):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all(torch.equal(u, v) for u, v in zip(out, want2))


def test_binding_refusals(q):
    x, gamma, beta, dy = _cuda(*_case(4, 64, torch.bfloat16, True, 8))
    m = torch.zeros(4, device="cuda")
    for bad in (dict(gamma=gamma[:32]), dict(Y=torch.empty((4, 32), device="cuda", dtype=x.dtype)), dict(mean=m[:3])):
        with pytest.raises(ValueError):
            q.qlin_layer_norm_forward(x, **bad)
    with pytest.raises(TypeError):
        q.qlin_layer_norm_forward(x, gamma.half())
    with pytest.raises(TypeError):
        q.qlin_layer_norm_backward(dy, x, m.double(), m)
    with pytest.raises(ValueError):
        q.qlin_layer_norm_forward(x.t())
    with pytest.raises(q.QlinError):
        q.qlin_layer_norm_forward(x[:, :40].contiguous())
