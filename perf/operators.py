"""Cases of the layer-norm and low-rank-adapter operators, their plain forms and their values in 64 bits.

Four operators around one quantized projection, as a model's block uses them:

- lora_forward: adapters of many requests beside a shared projection,
  Y[m] += scale[a] * (X[m] A[a]^T) B[a]^T with a = idx[m] (rows with idx < 0 keep their Y);
- lora_backward: its gradients dX (added to the projection's own), dA, dB;
- norm_forward: layer norm in front of the projection, with a 16-bit output or with the
  FP8 codes and per-token scales that the projection's GEMM takes;
- norm_backward: dX and the weight's and bias's gradients.

`own` selects the framework's kernels instead of the plain forms.
"""
import math

import torch

own = False

_EPS = 1e-6
_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one token of one request through an attention output projection: latency alone
        dict(name="lora_one_token", op="lora_forward", M=1, K=4096, N=4096, L=1, R=16, mix="tokens", bare=0.0, dt="bf16"),
        # a decode step: 64 requests, 32 adapters in use, some requests without one, through an MLP projection
        dict(name="lora_decode_64", op="lora_forward", M=64, K=4096, N=12288, L=32, R=16, mix="tokens", bare=0.1, dt="bf16"),
        # prompts of eight requests, of ragged lengths, in one batch, fp16
        dict(name="lora_prompts", op="lora_forward", M=1777, K=4096, N=12288, L=8, R=32, mix="spans", bare=0.1, dt="fp16"),
        # tokens of 48 adapters in no order, an odd output width
        dict(name="lora_mixed_tokens", op="lora_forward", M=4352, K=4096, N=4099, L=48, R=8, mix="tokens", bare=0.0, dt="bf16"),
        # the largest: a 2048 x 2048 image's tokens, four adapters of rank 64
        dict(name="lora_image_tokens", op="lora_forward", M=16640, K=4096, N=12288, L=4, R=64, mix="spans", bare=0.0, dt="bf16"),
        # training one small adapter on a short batch
        dict(name="lora_grad_small", op="lora_backward", M=512, K=4096, N=4096, L=1, R=16, mix="spans", bare=0.0, dt="bf16"),
        # training several adapters over ragged spans, rank 64
        dict(name="lora_grad_large", op="lora_backward", M=8191, K=4096, N=12288, L=6, R=64, mix="spans", bare=0.0, dt="bf16"),
        # the norm of a decode step
        dict(name="norm_decode", op="norm_forward", M=64, K=4096, out="same", affine=True, dt="bf16"),
        # the norm over a 2048 x 2048 image's tokens
        dict(name="norm_image_tokens", op="norm_forward", M=16640, K=4096, out="same", affine=True, dt="bf16"),
        # the norm in front of an FP8 projection: codes and scales instead of 16 bits, no weight of its own
        dict(name="norm_to_fp8", op="norm_forward", M=4352, K=4096, out="fp8", affine=False, dt="bf16"),
        # gradients on a short batch of wide rows, fp16
        dict(name="norm_grad_small", op="norm_backward", M=515, K=12288, out="same", affine=True, dt="fp16"),
        # gradients over a 2048 x 2048 image's tokens
        dict(name="norm_grad_large", op="norm_backward", M=16640, K=4096, out="same", affine=True, dt="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora_forward", "lora_forward", "lora_backward", "norm_forward", "norm_backward"])
    dt = rng.choice(["bf16", "fp16"])
    K = 16 * _log(rng, 8, 768)
    if op.startswith("norm"):
        M = _log(rng, 1, 16640)
        while M * K > 16640 * 4096:
            M = max(1, M // 2)
        out = rng.choice(["same", "fp8"]) if op == "norm_forward" else "same"
        return dict(op=op, M=M, K=K, out=out, affine=rng.random() < 0.7, dt=dt)
    if op == "lora_backward":
        M, N, dt, most = _log(rng, 1, 8191), 8 * _log(rng, 8, 1536), "bf16", 8191 * (4096 + 12288) * 6 * 64
    else:
        M, N, most = _log(rng, 1, 16640), _log(rng, 64, 12288), 16640 * (4096 + 12288) * 4 * 64
    L, R = _log(rng, 1, 64), 8 * _log(rng, 1, 16)
    while M * (K + N) * L * R > most:
        M, L = (M, max(1, L // 2)) if L > 8 else (max(1, M // 2), L)
    return dict(op=op, M=M, K=K, N=N, L=L, R=R, mix=rng.choice(["spans", "tokens"]), bare=rng.choice([0.0, 0.0, 0.1, 0.5]), dt=dt)


def _adapted(case):
    """Rows that have an adapter."""
    return case["M"] - int(case["bare"] * case["M"])


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "norm_forward":
        out = M * K * 2 if case["out"] == "same" else M * K + 4 * M
        return {"bytes": M * K * 2 + out + (4 * K if case["affine"] else 0), "flops": 8 * M * K}
    if case["op"] == "norm_backward":
        return {"bytes": 3 * M * K * 2 + 8 * M + (6 * K if case["affine"] else 0), "flops": 12 * M * K}
    N, L, R = case["N"], case["L"], case["R"]
    rows = _adapted(case)
    used = min(L, rows)
    if case["op"] == "lora_forward":
        return {"bytes": 2 * (rows * K + 2 * rows * N + used * R * (K + N)) + 4 * (M + L), "flops": 2 * rows * R * (K + N)}
    return {"bytes": 2 * (rows * N + 3 * rows * K + used * R * (K + N) + L * R * (K + N)) + 4 * (rows * R + M + L),
            "flops": 4 * rows * R * (K + N)}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, std, dt):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)


def _activations(g, M, K, dt):
    """N(0, 1) with a few channels of large values, as the projections' inputs have."""
    x = torch.randn((M, K), generator=g, device="cuda")
    x[:, 17 % K] *= 12.0
    x[: min(M, 4), 100 % K] = 900.0
    return x.to(dt)


def _idx(case, g):
    """The adapter of each row: requests are spans of rows, or each row is a request; `bare` of the rows have none."""
    M, L = case["M"], case["L"]
    if case["mix"] == "spans":
        cuts = torch.randint(0, M + 1, (L - 1,), generator=g, device="cuda").sort().values
        order = torch.randperm(L, generator=g, device="cuda")
        idx = order[torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)]
    else:
        idx = torch.randint(0, L, (M,), generator=g, device="cuda")
    idx = idx.to(torch.int32)
    bare = M - _adapted(case)
    at = (M - bare) // 2
    if case["mix"] == "spans":
        idx[at:at + bare] = -1
    else:
        idx[torch.randperm(M, generator=g, device="cuda")[:bare]] = -1
    return idx


def prepare(case, seed):
    g, dt, M, K = _gen(seed), _DT[case["dt"]], case["M"], case["K"]
    s = {"op": case["op"], "x": _activations(g, M, K, dt)}
    if case["op"].startswith("norm"):
        s["out"] = case["out"]
        s["x"] += 0.25
        s["gamma"] = (1.0 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(dt) if case["affine"] else None
        s["beta"] = _normal(g, (K,), 0.1, dt) if case["affine"] else None
        if case["op"] == "norm_backward":
            s["dy"] = _normal(g, (M, K), 0.5, dt)
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + _EPS).rsqrt().float()
        return s
    N, L, R = case["N"], case["L"], case["R"]
    s["A"] = _normal(g, (L, R, K), 1.0 / math.sqrt(K), dt)
    s["B"] = _normal(g, (L, N, R), 0.05, dt)
    s["scale"] = 0.5 + torch.rand(L, generator=g, device="cuda")
    s["idx"] = _idx(case, g)
    if case["op"] == "lora_forward":
        s["y"] = _normal(g, (M, N), 0.5, dt)          # what the shared projection gave
    else:
        s["dy"] = _normal(g, (M, N), 0.1, dt)
        s["dx"] = _normal(g, (M, K), 0.1, dt)         # what the shared projection gave
        s["h"] = torch.zeros((M, R), device="cuda")   # X A^T, kept by the forward pass
        for a in range(L):
            at = (s["idx"] == a).nonzero()[:, 0]
            s["h"][at] = s["x"][at].float() @ s["A"][a].float().T
    if own:   # the batch's plan, made once for all projections of a model
        import quantized_w8a8_linear_b200 as q
        s["plan"] = q.qlin_lora_plan(s["idx"], L)
    return s


def _run_own(s):
    import quantized_w8a8_linear_b200 as q
    if s["op"] == "lora_forward":
        return q.qlin_lora_forward(s["x"], s["A"], s["B"], s["scale"], s["plan"], s["y"])
    if s["op"] == "lora_backward":
        return q.qlin_lora_backward(s["dy"], s["x"], s["A"], s["B"], s["scale"], s["plan"], s["h"], dX=s["dx"])
    if s["op"] == "norm_backward":
        out = q.qlin_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], gamma=s["gamma"])
        return out if s["gamma"] is not None else out[0]
    if s["out"] == "fp8":
        codes, s_x = q.qlin_layer_norm_fp8_prep(s["x"], s["gamma"], s["beta"], eps=_EPS)
        return codes.view(torch.float8_e4m3fn), s_x
    return q.qlin_layer_norm_forward(s["x"], s["gamma"], s["beta"], eps=_EPS)


def _one_hot(idx, L):
    return (idx[:, None] == torch.arange(L, device=idx.device)).float()


def _plain_lora_forward(s):
    x, A, B, y = s["x"].float(), s["A"].float(), s["B"].float(), s["y"]
    L, R, K = A.shape
    pick = (_one_hot(s["idx"], L) * s["scale"])[:, :, None]
    h = (x @ A.reshape(L * R, K).T).reshape(-1, L, R) * pick
    add = h.reshape(-1, L * R) @ B.transpose(1, 2).reshape(L * R, -1)
    s["y"] = (y.float() + add).to(y.dtype)
    return s["y"]


def _plain_lora_backward(s):
    x, dy, A, B, dt = s["x"].float(), s["dy"].float(), s["A"].float(), s["B"].float(), s["x"].dtype
    L, R, K = A.shape
    N = B.shape[1]
    pick = (_one_hot(s["idx"], L) * s["scale"])[:, :, None]
    h = (s["h"][:, None, :] * pick).reshape(-1, L * R)
    dh = ((dy @ B.transpose(0, 1).reshape(N, L * R)).reshape(-1, L, R) * pick).reshape(-1, L * R)
    dB = (h.T @ dy).reshape(L, R, N).transpose(1, 2).contiguous().to(dt)
    dA = (dh.T @ x).reshape(L, R, K).to(dt)
    s["dx"] = (s["dx"].float() + dh @ A.reshape(L * R, K)).to(dt)
    return s["dx"], dA, dB


def _plain_norm_forward(s):
    x = s["x"].float()
    c = x - x.mean(1, keepdim=True)
    y = c * torch.rsqrt((c * c).mean(1, keepdim=True) + _EPS)
    if s["gamma"] is not None:
        y = y * s["gamma"].float() + s["beta"].float()
    if s["out"] == "same":
        return y.to(s["x"].dtype)
    s_x = y.abs().amax(1) / 448.0
    return (y * (1.0 / s_x)[:, None]).to(torch.float8_e4m3fn), s_x


def _plain_norm_backward(s):
    x, dy, dt = s["x"].float(), s["dy"].float(), s["x"].dtype
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    d = dy if s["gamma"] is None else dy * s["gamma"].float()
    dx = (s["rstd"][:, None] * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))).to(dt)
    if s["gamma"] is None:
        return dx
    return dx, (dy * xh).sum(0).to(dt), dy.sum(0).to(dt)


def run(state):
    if own:
        return _run_own(state)
    return {"lora_forward": _plain_lora_forward, "lora_backward": _plain_lora_backward,
            "norm_forward": _plain_norm_forward, "norm_backward": _plain_norm_backward}[state["op"]](state)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"].startswith("norm"):
        n = x.shape[1]
        mean = x.sum(1, keepdim=True) / n
        var = ((x - mean) ** 2).sum(1, keepdim=True) / n
        gamma = torch.ones(n, dtype=torch.float64, device="cuda") if s["gamma"] is None else s["gamma"].double()
        if case["op"] == "norm_forward":
            y = (x - mean) / torch.sqrt(var + _EPS) * gamma + (0.0 if s["beta"] is None else s["beta"].double())
            if case["out"] == "same":
                return y
            s_x = y.abs().max(1).values / 448.0
            return y / s_x[:, None], s_x
        dy, r = s["dy"].double(), s["rstd"].double()[:, None]
        xh = (x - s["mean"].double()[:, None]) * r
        g = dy * gamma
        dx = r * g - r / n * (g.sum(1, keepdim=True) + xh * (g * xh).sum(1, keepdim=True))
        return dx if s["gamma"] is None else (dx, torch.einsum("mk,mk->k", dy, xh), dy.sum(0))
    # one adapter at a time, over its own rows
    L = case["L"]
    if case["op"] == "lora_forward":
        y = s["y"].double()
        for a in range(L):
            at = (s["idx"] == a).nonzero()[:, 0]
            y[at] += s["scale"][a].double() * (x[at] @ s["A"][a].double().T @ s["B"][a].double().T)
        return y
    dx, dA, dB = s["dx"].double(), torch.zeros_like(s["A"], dtype=torch.float64), torch.zeros_like(s["B"], dtype=torch.float64)
    for a in range(L):
        at = (s["idx"] == a).nonzero()[:, 0]
        dy, c = s["dy"][at].double(), s["scale"][a].double()
        dh = c * (dy @ s["B"][a].double())
        dB[a] = c * (dy.T @ s["h"][at].double())
        dA[a] = dh.T @ x[at]
        dx[at] += dh @ s["A"][a].double()
    return dx, dA, dB
