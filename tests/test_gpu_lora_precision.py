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


def _ladder(g, L, R, C, dtype):
    """[L,R,C] positive, row r 4^-r the size of row 0: the largest and the smallest of a row of H are 2^14 apart."""
    return (16.0 * 4.0 ** -torch.arange(R, device="cuda")[:, None] * (0.5 + torch.rand((L, R, C), generator=g, device="cuda"))).to(dtype)


def _pick(g, L, R, C, dtype):
    """[L,C,R] with one positive weight a column: column c reads element c % R of H alone."""
    b = torch.zeros((L, C, R), device="cuda")
    c = torch.arange(C, device="cuda")
    b[:, c, c % R] = 0.5 + torch.rand((L, C), generator=g, device="cuda")
    return b.to(dtype)


def _check_difference(got, base, update, dtype):
    """got = T(base + update), where base = -T(update): what is left is as small as the roundings of `update`. Two
    MMAs in line lose four steps each of their sums (16 products, then H's largest part's one; the smaller parts'
    sums are 2^-8 of that at most, and their losses less than another step), and the last addition rounds once."""
    want = base.double() + update
    e = (4 + 4 + 1) * 2.0 ** -23 * update.abs()
    tol = e + torch.finfo(dtype).eps / 2 * (want.abs() + e) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("M,R", [(200, 8), (300, 8), (300, 72)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_y_sees_all_bits_of_h(q, M, R, dtype):
    # 16 products, one MMA, for each element of H: what is left of Y + update - T(update) shows how exactly H entered.
    # 200 rows of rank 8 go through the kernel of few rows, in the batch of 300 through the tiles'
    K, N, L = 16, 520, 3
    g = torch.Generator(device="cuda").manual_seed(M + R)
    X, A, B = _positive(g, (M, K), dtype), torch.zeros((L, R, K), dtype=dtype, device="cuda"), torch.zeros((L, N, R), dtype=dtype, device="cuda")
    A[:, -8:], B[:, :, -8:] = _ladder(g, L, 8, K, dtype), _pick(g, L, 8, N, dtype)
    idx = (torch.arange(M, device="cuda") % L).to(torch.int32)
    scale = 0.5 + torch.rand(L, generator=g, device="cuda")
    update = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    for a in range(L):
        update[idx == a] = scale[a].double() * (X[idx == a].double() @ A[a].double().T @ B[a].double().T)
    base = -update.to(dtype)
    Y = q.qlin_lora_forward(X, A, B, scale, q.qlin_lora_plan(idx, L), base.clone())
    _check_difference(Y, base, update, dtype)


@pytest.mark.parametrize("R", [8, 72])
def test_dx_sees_all_bits_of_dh(q, R):
    dtype, M, K, N, L = torch.bfloat16, 300, 528, 16, 3
    g = torch.Generator(device="cuda").manual_seed(R)
    X, dY = _positive(g, (M, K), dtype), _positive(g, (M, N), dtype)
    A, B = torch.zeros((L, R, K), dtype=dtype, device="cuda"), torch.zeros((L, N, R), dtype=dtype, device="cuda")
    A[:, -8:], B[:, :, -8:] = _pick(g, L, 8, K, dtype).transpose(1, 2), _ladder(g, L, 8, N, dtype).transpose(1, 2)
    idx = (torch.arange(M, device="cuda") % L).to(torch.int32)
    scale = 0.5 + torch.rand(L, generator=g, device="cuda")
    update = torch.zeros((M, K), dtype=torch.float64, device="cuda")
    for a in range(L):
        update[idx == a] = scale[a].double() * (dY[idx == a].double() @ B[a].double() @ A[a].double())
    base = -update.to(dtype)
    dX, _, _ = q.qlin_lora_backward(dY, X, A, B, scale, q.qlin_lora_plan(idx, L), torch.zeros((M, R), device="cuda"), dX=base.clone())
    _check_difference(dX, base, update, dtype)


def test_gradient_is_summed_in_short_chains(q):
    # 8192 rows of one adapter under columns enough that a CTA takes all of a column's tiles: 512 MMAs in line, in chains
    # of 64, for each element of dB. bf16's steps are 2^-8 to 2^-7 of a value, and the elements lie anywhere between them
    # (a factor for each column), so of sums that are too small by e on average at most 2^8 e are rounded the other way.
    # What is cut off is half of the most on average: two steps an MMA. H in 8 bits, so that it is its own first part.
    M, K, N, R, dtype = 8192, 26112, 12288, 8, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(5)
    dY = ((0.5 + torch.rand((M, N), generator=g, device="cuda")) * 2.0 ** torch.rand(N, generator=g, device="cuda")).to(dtype)
    X = torch.ones((M, K), dtype=dtype, device="cuda")
    A, B = torch.ones((1, R, K), dtype=dtype, device="cuda"), torch.ones((1, N, R), dtype=dtype, device="cuda")
    H = _positive(g, (M, R), dtype).float()
    plan = q.qlin_lora_plan(torch.zeros(M, dtype=torch.int32, device="cuda"), 1)
    _, _, dB = q.qlin_lora_backward(dY, X, A, B, torch.ones(1, device="cuda"), plan, H)
    want = torch.cat([dY[:, n:n + 1024].double().T @ H.double() for n in range(0, N, 1024)]).to(dtype)
    e = 2 * (64 + 1) / 2 * 2.0 ** -23 + 8 * 2.0 ** -25
    assert (dB[0] != want).float().mean().item() <= 2.0 ** 8 * e


def _two_rows(M, L):
    """For each adapter of idx = m % L: a row among the first and one among the last, of other tiles or MMAs."""
    return [(a, a + (M - L) // L * L) for a in range(L)]


@pytest.mark.parametrize("R", [8, 72])
def test_db_sees_all_bits_of_h(q, R):
    # rows +c and -c of dY against rows of H that differ by 2^-12: what is left of the sum shows how exactly H entered.
    # Two MMAs with anything in them lose four steps each, the parts are added in two roundings.
    dtype, M, K, N, L = torch.bfloat16, 300, 32, 520, 3
    g = torch.Generator(device="cuda").manual_seed(R)
    idx = (torch.arange(M, device="cuda") % L).to(torch.int32)
    H = 0.5 + torch.rand((M, R), generator=g, device="cuda")
    dY, c = torch.zeros((M, N), dtype=dtype, device="cuda"), _positive(g, (N,), dtype)
    scale = 0.5 + torch.rand(L, generator=g, device="cuda")
    want, size = torch.zeros((L, N, R), dtype=torch.float64, device="cuda"), torch.zeros((L, N, R), dtype=torch.float64, device="cuda")
    for a, (i, j) in enumerate(_two_rows(M, L)):
        H[j] = H[i] * (1 + 2.0 ** -12 * torch.rand(R, generator=g, device="cuda"))
        dY[i], dY[j] = c, -c
        want[a] = scale[a].double() * torch.outer(c.double(), H[i].double() - H[j].double())
        size[a] = scale[a].double() * torch.outer(c.double(), H[j].double())
    X, A, B = _positive(g, (M, K), dtype), _positive(g, (L, R, K), dtype), _positive(g, (L, N, R), dtype)
    _, _, dB = q.qlin_lora_backward(dY, X, A, B, scale, q.qlin_lora_plan(idx, L), H)
    e = (4 + 4 + 1) * 2.0 ** -23 * size
    assert ((dB.double() - want).abs() <= e + 2.0 ** -8 * (want.abs() + e)).all()


@pytest.mark.parametrize("R", [8, 72])
def test_da_sees_all_bits_of_dh(q, R):
    # the same for dA: rows +x and -x of X against dH = s (d1 B[n1] + d2 B[n2]) whose d2, 2^-12 of d1, differ. The MMA
    # and the scale of each dH lose four steps and half a one.
    dtype, M, K, N, L = torch.bfloat16, 300, 528, 16, 3
    g = torch.Generator(device="cuda").manual_seed(R)
    idx = (torch.arange(M, device="cuda") % L).to(torch.int32)
    A, B = _positive(g, (L, R, K), dtype), _positive(g, (L, N, R), dtype)
    dY, X, x = torch.zeros((M, N), dtype=dtype, device="cuda"), torch.zeros((M, K), dtype=dtype, device="cuda"), _positive(g, (K,), dtype)
    scale = 0.5 + torch.rand(L, generator=g, device="cuda")
    want, size = torch.zeros((L, R, K), dtype=torch.float64, device="cuda"), torch.zeros((L, R, K), dtype=torch.float64, device="cuda")
    for a, (i, j) in enumerate(_two_rows(M, L)):
        dY[i, 3] = dY[j, 3] = 1.5
        dY[i, 11], dY[j, 11] = 2.0 ** -12, 2.0 ** -13
        X[i], X[j] = x, -x
        dh = scale[a].double() * (dY[[i, j]].double() @ B[a].double())
        want[a], size[a] = torch.outer(dh[0] - dh[1], x.double()), torch.outer(dh[0], x.double())
    _, dA, _ = q.qlin_lora_backward(dY, X, A, B, scale, q.qlin_lora_plan(idx, L), torch.zeros((M, R), device="cuda"))
    e = (2 * (4 + 0.5) + 4 + 4 + 1) * 2.0 ** -23 * size
    assert ((dA.double() - want).abs() <= e + 2.0 ** -8 * (want.abs() + e)).all()
