"""GPU low-rank adapters (plan, forward, backward) against the 64-bit oracle.

Tolerances, elementwise. h = eps / 2 is half a step of the 16-bit type. An
MMA adds 16 exact products to an fp32 accumulator; its rounding is not
documented, so four steps of 2^-23 of the sum of absolute values are allowed
for each, and two for each of the at most 8 partial sums of a cluster (or at
most 160 of the gradients' CTAs): over C products the sum is off by at most
  G(C) = (4 (C / 16 + 1) + 2 P) 2^-23, times the sum of absolute values.
H: G(K) sum|x a|. Its 16-bit parts: 2^-16 of |h| in bf16 (two halves of 8
bits, each off by half a step), 2^-22 of the row's largest |h| (and 2^-25 of
it where lo is subnormal) in fp16; 2^-16 of the row's largest covers both.
Y: |s| (sum_r (G(K) sum|x a| + 2^-16 max|h|) |b| + G(2 R) sum|h b|) +
2 2^-24 (|y0| + |y|), then h |y|. The gradients likewise, with dH in H's place.
"""
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


def G(C, parts=8):
    return (4 * (C / 16 + 1) + 2 * parts) * 2.0 ** -23


def _case(M, K, N, L, R, dtype, idx, seed=0):
    g = torch.Generator().manual_seed(seed + M + 3 * K + 5 * N + 7 * L + 11 * R)
    n = lambda *s: torch.randn(s, generator=g)   # noqa: E731
    c = dict(X=n(M, K).to(dtype), A=(n(L, R, K) / K ** 0.5).to(dtype), B=(0.3 * n(L, N, R)).to(dtype), scale=0.5 + torch.rand(L, generator=g),
             Y=n(M, N).to(dtype), dY=n(M, N).to(dtype), dX=n(M, K).to(dtype))
    if idx == "tokens":
        c["idx"] = torch.randint(-1, L + 1, (M,), generator=g).to(torch.int32)     # -1 and L: none
    elif idx == "spans":
        c["idx"] = (torch.arange(M) * L // max(M, 1)).flip(0).to(torch.int32)
    else:
        c["idx"] = torch.full((M,), idx, dtype=torch.int32)
    return c


def _forward(q, c, H=None):
    d = {k: v.cuda() for k, v in c.items()}
    plan = q.qlin_lora_plan(d["idx"], d["A"].shape[0])
    Y = d["Y"].clone()
    assert q.qlin_lora_forward(d["X"], d["A"], d["B"], d["scale"], plan, Y, H=H) is Y
    return Y, plan, d


def _abs(c):
    return {k: (v.double().abs().numpy() if k != "idx" else v.numpy()) for k, v in c.items()}


def _check_forward(c, Y, H, dtype):
    idx = c["idx"].numpy()
    y64, h64 = o.lora_forward(c["X"], c["A"], c["B"], c["scale"], idx, c["Y"])
    a = _abs(c)
    L, R, K = c["A"].shape
    got, h = Y.double().cpu().numpy(), H.double().cpu().numpy()
    half = torch.finfo(dtype).eps / 2
    for m, l in enumerate(idx):
        if not 0 <= l < L:
            assert np.array_equal(got[m], c["Y"][m].double().numpy())          # bit for bit
            assert (h[m] == 77.0).all()                                        # left as it was
            continue
        eh = G(K) * (a["A"][l] @ a["X"][m])
        assert (np.abs(h[m] - h64[m]) <= eh).all()
        hm = np.abs(h64[m]) + eh
        e = a["scale"][l] * (a["B"][l] @ (eh + 2.0 ** -16 * hm.max()) + G(2 * R) * (a["B"][l] @ hm)) + 2.0 ** -23 * (a["Y"][m] + np.abs(y64[m]))
        assert (np.abs(got[m] - y64[m]) <= e + half * (np.abs(y64[m]) + e) + (2.0 ** -25 if dtype == torch.float16 else 0)).all()


FWD = [(1, 16, 8, 1, 8, 0), (1, 64, 64, 1, 16, 0), (1, 4096, 1000, 2, 16, 1), (5, 80, 1, 3, 8, "tokens"), (7, 256, 65, 1, 128, "tokens"),
       (64, 1024, 264, 32, 16, "tokens"), (127, 208, 72, 2, 24, "spans"), (128, 512, 256, 1, 64, "spans"), (129, 512, 136, 2, 72, "tokens"),
       (130, 64, 515, 1, 40, "spans"), (300, 528, 63, 4, 120, "tokens"), (257, 1040, 200, 100, 8, "tokens"), (40, 128, 129, 1024, 8, "tokens"),
       (33, 128, 64, 3, 16, -1), (1100, 144, 96, 2, 32, "spans"),
       # both sides of the choice between the kernel of few rows and the tiles' (M <= 256, R <= 32, M R <= 4096)
       (256, 128, 72, 3, 16, "tokens"), (257, 128, 72, 3, 16, "tokens"), (128, 96, 41, 2, 32, "tokens"), (129, 96, 41, 2, 32, "tokens"),
       (60, 96, 41, 2, 40, "tokens"), (1, 32768, 16, 1, 32, 0), (9, 16, 3, 2, 8, "tokens"),
       # tiles enough for one CTA an SM and no clusters
       (9700, 144, 64, 3, 16, "spans")]


@pytest.mark.parametrize("M,K,N,L,R,idx", FWD)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_forward(q, M, K, N, L, R, idx, dtype):
    c = _case(M, K, N, L, R, dtype, idx)
    H = torch.full((M, R), 77.0, device="cuda")
    Y, _, _ = _forward(q, c, H)
    _check_forward(c, Y, H, dtype)


BWD = [(1, 16, 8, 1, 8, 0), (1, 64, 64, 2, 16, 1), (5, 80, 8, 3, 8, "tokens"), (7, 256, 72, 1, 128, "tokens"), (64, 1024, 264, 32, 16, "tokens"),
       (127, 208, 72, 2, 24, "spans"), (128, 512, 256, 1, 64, "spans"), (129, 512, 136, 2, 72, "tokens"), (300, 528, 72, 4, 120, "tokens"),
       (257, 1040, 200, 100, 8, "tokens"), (40, 128, 136, 1024, 8, "tokens"), (33, 128, 64, 3, 16, -1), (1100, 144, 96, 2, 32, "spans"),
       (1500, 272, 528, 1, 16, "spans"), (1300, 528, 272, 3, 128, "spans"),
       # gradients cut between CTAs: fewer units than CTAs, and more
       (3000, 416, 680, 3, 32, "tokens"), (1200, 2064, 1304, 1, 72, "spans"), (2300, 1040, 2600, 5, 8, "tokens"), (9700, 80, 72, 2, 16, "spans")]


@pytest.mark.parametrize("M,K,N,L,R,idx", BWD)
def test_backward(q, M, K, N, L, R, idx):
    c = _case(M, K, N, L, R, torch.bfloat16, idx, 1)
    H = torch.full((M, R), 77.0, device="cuda")
    _, plan, d = _forward(q, c, H)
    dX = d["dX"].clone()
    got, dA, dB = q.qlin_lora_backward(d["dY"], d["X"], d["A"], d["B"], d["scale"], plan, H, dX=dX)
    assert got is dX
    ix = c["idx"].numpy()
    h = H.double().cpu().numpy()
    wX, wA, wB, dh = o.lora_backward(c["dY"], c["X"], c["A"], c["B"], c["scale"], ix, h, c["dX"])
    a = _abs(c)
    on = (ix >= 0) & (ix < L)
    half = 2.0 ** -8
    eA, eB = np.zeros(wA.shape), np.zeros(wB.shape)
    gX = dX.double().cpu().numpy()
    for m, l in enumerate(ix):
        if not on[m]:
            assert np.array_equal(gX[m], c["dX"][m].double().numpy())
            continue
        ed = a["scale"][l] * G(N) * (a["dY"][m] @ a["B"][l])
        dm = np.abs(dh[m]) + ed
        part = ed + 2.0 ** -16 * dm
        e = part @ a["A"][l] + G(2 * R) * (dm @ a["A"][l]) + 2.0 ** -23 * (a["dX"][m] + np.abs(wX[m]))
        assert (np.abs(gX[m] - wX[m]) <= e + half * (np.abs(wX[m]) + e)).all()
        n = int((ix == l).sum())
        eA[l] += np.outer(part + G(2 * n, 160) * dm, a["X"][m])
        eB[l] += a["scale"][l] * np.outer(a["dY"][m], (2.0 ** -16 + G(2 * n, 160) + 2.0 ** -23) * np.abs(h[m]))
    for g, w, e in ((dA, wA, eA), (dB, wB, eB)):
        g = g.double().cpu().numpy()
        assert (np.abs(g - w) <= e + half * (np.abs(w) + e)).all()
        empty = [l for l in range(L) if not (ix == l).any()]
        assert not g[empty].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_alignment_of_a_row(q, dtype):
    # rows whose start is any even number of bytes past 16, whole and partial last columns
    for N in list(range(120, 137)) + [1, 7, 63, 191, 193, 261]:
        c = _case(300, 64, N, 3, 16, dtype, "tokens", 20)
        H = torch.full((300, 16), 77.0, device="cuda")
        Y, _, _ = _forward(q, c, H)
        _check_forward(c, Y, H, dtype)


def test_order_of_rows_does_not_matter(q):
    c = _case(500, 256, 136, 5, 16, torch.bfloat16, "tokens", 2)
    Y, _, _ = _forward(q, c)
    g = torch.Generator().manual_seed(0)
    p = torch.randperm(500, generator=g)
    c2 = dict(c, X=c["X"][p], Y=c["Y"][p], idx=c["idx"][p])
    Y2, _, _ = _forward(q, c2)
    assert torch.equal(Y2.cpu(), Y.cpu()[p])


@pytest.mark.parametrize("M,R", [(3, 16), (200, 16), (40, 64), (300, 8)])
def test_h_not_kept(q, M, R):
    c = _case(M, 256, 136, 3, R, torch.bfloat16, "tokens", 13)
    H = torch.zeros((M, R), device="cuda")
    kept, _, _ = _forward(q, c, H)
    Y, _, _ = _forward(q, c)
    assert torch.equal(Y, kept)


def test_update_alone_and_zero_weights(q):
    # B = 0 keeps Y's bits; Y = 0 leaves the update alone
    c = _case(200, 128, 72, 2, 16, torch.bfloat16, "spans", 3)
    Y, _, _ = _forward(q, dict(c, B=torch.zeros_like(c["B"])))
    assert torch.equal(Y.cpu(), c["Y"])
    c0 = dict(c, Y=torch.zeros_like(c["Y"]))
    H = torch.full((200, 16), 77.0, device="cuda")
    Y, _, _ = _forward(q, c0, H)
    _check_forward(c0, Y, H, torch.bfloat16)


@pytest.mark.parametrize("big", [3e4, 1e-6])
def test_fp16_range_of_h(q, big):
    # h past fp16's largest value, and down among its subnormals: the parts are taken of a scaled row
    c = _case(150, 512, 72, 2, 24, torch.float16, "tokens", 4)
    if big > 1:
        c["X"] = (c["X"].float() * 300).half()
        c["A"] = (c["A"].float() * 400).half()
        c["B"] = (c["B"].float() * 1e-4).half()
    else:
        c["X"] = (c["X"].float() * 1e-3).half()
        c["A"] = (c["A"].float() * 1e-2).half()
        c["B"] = (c["B"].float() * 100).half()
    H = torch.full((150, 24), 77.0, device="cuda")
    Y, _, _ = _forward(q, c, H)
    on = (c["idx"] >= 0) & (c["idx"] < 2)
    assert (H[on.cuda()].abs().max().item() > 65504) == (big > 1)
    _check_forward(c, Y, H, torch.float16)


def test_nan_and_inf_stay_in_their_rows_and_adapters(q):
    c = _case(300, 256, 136, 4, 16, torch.bfloat16, "tokens", 5)
    c["idx"][10], c["idx"][11] = 1, 1
    H = torch.full((300, 16), 0.0, device="cuda")
    clean, plan, d = _forward(q, c, H)
    gX, gA, gB = q.qlin_lora_backward(d["dY"], d["X"], d["A"], d["B"], d["scale"], plan, H, dX=d["dX"].clone())
    c2 = {k: v.clone() for k, v in c.items()}
    c2["X"][10, 3] = float("nan")
    c2["X"][c2["idx"] < 0] = float("inf")            # rows without an adapter are not read into anything
    c2["dY"][c2["idx"] < 0] = float("nan")
    H2 = torch.full((300, 16), float("nan"), device="cuda")   # nor are their rows of H
    Y, plan2, d2 = _forward(q, c2, H2)
    keep = torch.arange(300) != 10
    assert torch.equal(Y.cpu()[keep], clean.cpu()[keep]) and torch.isnan(Y[10]).all()
    hX, hA, hB = q.qlin_lora_backward(d2["dY"], d2["X"], d2["A"], d2["B"], d2["scale"], plan2, H2, dX=d2["dX"].clone())
    others = [0, 2, 3]
    assert torch.equal(hA[others], gA[others]) and torch.equal(hB[others], gB[others])
    assert torch.isnan(hA[1]).any() and torch.isnan(hB[1]).any() and torch.equal(hX, gX)
    # an adapter of NaN and infinities touches its own rows only
    c3 = {k: v.clone() for k, v in c.items()}
    c3["A"][1], c3["B"][1, 5] = float("nan"), float("inf")
    Y, _, _ = _forward(q, c3)
    other = (c["idx"] != 1)
    assert torch.equal(Y.cpu()[other], clean.cpu()[other]) and torch.isnan(Y[10]).all()


def test_same_bits_again_streams_and_graph(q):
    c = _case(700, 528, 264, 3, 32, torch.bfloat16, "spans", 6)
    H = torch.zeros((700, 32), device="cuda")
    want, plan, d = _forward(q, c, H)
    run = lambda: q.qlin_lora_backward(d["dY"], d["X"], d["A"], d["B"], d["scale"], plan, H, dX=d["dX"].clone())   # noqa: E731
    grads = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = [run() for _ in range(3)]
    b = [run() for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for t in a + b for u, v in zip(t, grads))
    # one captured step, replayed on another batch: the plan is made inside the graph
    Y, dX, H2 = d["Y"].clone(), d["dX"].clone(), torch.zeros_like(H)
    X, idx = d["X"].clone(), d["idx"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = q.qlin_lora_plan(idx, 3)
        q.qlin_lora_forward(X, d["A"], d["B"], d["scale"], p, Y, H=H2)
        out = q.qlin_lora_backward(d["dY"], X, d["A"], d["B"], d["scale"], p, H2, dX=dX)
    perm = torch.randperm(700, generator=torch.Generator().manual_seed(1)).cuda()
    X.copy_(d["X"][perm])
    idx.copy_(d["idx"][perm])
    Y.copy_(d["Y"][perm])
    dX.copy_(d["dX"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want[perm])
    c2 = dict(c, X=X.cpu(), idx=idx.cpu(), Y=c["Y"][perm.cpu()])
    Hr = torch.zeros_like(H)
    _, plan2, d2 = _forward(q, c2, Hr)
    ref = q.qlin_lora_backward(d["dY"], X, d["A"], d["B"], d["scale"], plan2, Hr, dX=d["dX"].clone())
    assert all(torch.equal(u, v) for u, v in zip(out, ref))


def test_without_dx_and_without_rows(q):
    c = _case(150, 128, 72, 2, 16, torch.bfloat16, "spans", 7)
    H = torch.zeros((150, 16), device="cuda")
    _, plan, d = _forward(q, c, H)
    full = q.qlin_lora_backward(d["dY"], d["X"], d["A"], d["B"], d["scale"], plan, H, dX=d["dX"].clone())
    none, dA, dB = q.qlin_lora_backward(d["dY"], d["X"], d["A"], d["B"], d["scale"], plan, H)
    assert none is None and torch.equal(dA, full[1]) and torch.equal(dB, full[2])
    e = {k: d[k][:0] for k in ("X", "Y", "dY", "dX", "idx")}
    plan0 = q.qlin_lora_plan(e["idx"], 2)
    assert q.qlin_lora_forward(e["X"], d["A"], d["B"], d["scale"], plan0, e["Y"]).shape == (0, 72)
    _, dA, dB = q.qlin_lora_backward(e["dY"], e["X"], d["A"], d["B"], d["scale"], plan0, H[:0], dX=e["dX"])
    assert not dA.any() and not dB.any()


@pytest.mark.parametrize("M,L", [(1, 1), (31, 1024), (256, 3), (257, 3), (1000, 1000), (4352, 48), (20000, 2), (33000, 1024)])
def test_plan_is_a_stable_sort(q, M, L):
    g = torch.Generator().manual_seed(M + L)
    idx = torch.randint(-2, L + 2, (M,), generator=g, dtype=torch.int32)
    plan = q.qlin_lora_plan(idx.cuda(), L).view(torch.int32).cpu()
    most = M // 128 + min(L, M)
    info_at = 16 + (L + 4) // 4 * 4
    rows_at = info_at + (2 * most + 3) // 4 * 4
    info, rows = plan[info_at:info_at + 2 * most].view(-1, 2), plan[rows_at:rows_at + 128 * most].view(-1, 128)
    tiles = int(plan[2])
    assert plan[0] == M and plan[1] == L and tiles <= most and plan[16 + L] == tiles
    on = ((idx >= 0) & (idx < L)).nonzero()[:, 0]
    want = on[torch.sort(idx[on], stable=True).indices].int()
    got = [rows[t][:int(info[t, 1])] for t in range(tiles)]
    assert torch.equal(torch.cat(got) if got else want[:0], want)
    assert all((rows[t][int(info[t, 1]):] == M).all() and (idx[got[t].long()] == info[t, 0]).all() for t in range(tiles))
    octets = int(plan[3])
    assert (octets > 0) == (M <= 256 and want.numel() > 0)
    at = rows_at + 128 * most
    o = plan[at:at + 12 * octets].view(-1, 12)
    eights = [o[t, 4:4 + int(o[t, 1])] for t in range(octets)]
    if octets:
        assert torch.equal(torch.cat(eights), want)
        assert all((o[t, 4 + int(o[t, 1]):] == M).all() and (idx[eights[t].long()] == o[t, 0]).all() for t in range(octets))


def test_plan_of_another_batch_is_refused(q):
    c = _case(150, 128, 72, 2, 16, torch.bfloat16, "spans", 8)
    _, plan, d = _forward(q, c)
    with pytest.raises(ValueError):
        q.qlin_lora_forward(d["X"][:20], d["A"], d["B"], d["scale"], plan, d["Y"][:20])
    # the same size, another M: caught on the device, nothing is written
    other = plan.clone()
    other.view(torch.int32)[0] = 149
    Y = d["Y"].clone()
    q.qlin_lora_forward(d["X"], d["A"], d["B"], d["scale"], other, Y)
    H = torch.zeros((150, 16), device="cuda")
    dX, dA, dB = q.qlin_lora_backward(d["dY"], d["X"], d["A"], d["B"], d["scale"], other, H, dX=d["dX"].clone())
    assert q.qlin_get_device_status(reset=True) == q.QLIN_ERR_INVALID_ARG
    assert torch.equal(Y, d["Y"]) and torch.equal(dX, d["dX"]) and not dA.any() and not dB.any()


def test_rows_behind_the_last_and_far_offsets(q):
    # rows past M are another tensor's; element offsets pass 2^31
    M, N, K, R = 180000, 12288, 64, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    Y = torch.zeros((M + 2, N), dtype=torch.bfloat16, device="cuda")
    X = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    A = torch.randn((1, R, K), generator=g, device="cuda").to(torch.bfloat16)
    B = torch.randn((1, N, R), generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 131071, 174762, 174763, M - 1], device="cuda")
    idx[rows] = 0
    Y[M:] = 5.0
    plan = q.qlin_lora_plan(idx, 1)
    q.qlin_lora_forward(X, A, B, torch.ones(1, device="cuda"), plan, Y[:M])
    want = (X[rows].double() @ A[0].double().T @ B[0].double().T)
    err = (Y[rows].double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 1e-2).all()      # the update is about 23 in size
    assert (Y[M:] == 5.0).all()
    others = torch.ones(M, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert not any(Y[:M][i:i + 20000][others[i:i + 20000]].any().item() for i in range(0, M, 20000))


def test_binding_refusals(q):
    c = _case(20, 64, 24, 2, 16, torch.bfloat16, "spans", 9)
    Y, plan, d = _forward(q, c)
    f = lambda **k: q.qlin_lora_forward(*[{**d, **k}[n] for n in ("X", "A", "B", "scale")], plan, k.get("Y", Y))   # noqa: E731
    with pytest.raises(ValueError):
        f(A=d["A"][:, :, :48].contiguous())
    with pytest.raises(ValueError):
        f(B=d["B"].transpose(1, 2))
    with pytest.raises(ValueError):
        f(Y=Y[:, :16])
    with pytest.raises(ValueError):
        f(scale=d["scale"].cpu())
    with pytest.raises(TypeError):
        f(A=d["A"].half())
    with pytest.raises(TypeError):
        f(scale=d["scale"].double())
    with pytest.raises(q.QlinError):
        f(A=d["A"][:, :12].contiguous(), B=d["B"][:, :, :12].contiguous())
    with pytest.raises(q.QlinError):
        h = {k: v.half() if v.dtype == torch.bfloat16 else v for k, v in d.items()}
        q.qlin_lora_backward(h["dY"], h["X"], h["A"], h["B"], h["scale"], plan, torch.zeros((20, 16), device="cuda"))
