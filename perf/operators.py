"""Cases for the operators around a frozen, pruned linear layer: low-rank adapters and layer norm.

Kinds of case:

* ``lora``        the adapters of many requests added to a shared projection's output (serving);
* ``lora_train``  the same forward, then its gradients (fine-tuning beside a frozen weight);
* ``ln``          layer norm, with or without the residual sum in front of it, keeping the statistics;
* ``ln_s8``       layer norm quantised to the int8 activations of a fixed-point layer;
* ``ln_bwd``      layer norm's gradients, with the reduction of the weight's gradient.

``own = False`` computes the formulas with elementary torch operations in 32 bits; ``own = True`` makes
the calls of this repository's library.  Matrices are row-major with rows padded to 16 bytes.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    lora = {"kind": "lora", "none": 0.1, "order": "requests"}
    return [
        # one new token of one request beside a large projection: latency alone
        {**lora, "name": "lora decode 1", "M": 1, "N": 16384, "K": 4096, "R": 16, "L": 8, "dtype": "bf16", "order": "mixed", "none": 0.0},
        # a decode step of 64 requests, nearly each with an adapter of its own: the adapters' weights are the traffic
        {**lora, "name": "lora decode 64", "M": 64, "N": 16384, "K": 4096, "R": 16, "L": 64, "dtype": "bf16", "order": "mixed"},
        # 32 images of 197 tokens through a vision transformer's second MLP layer, six fine-tuned variants of it
        {**lora, "name": "lora vit", "M": 6304, "N": 1024, "K": 4096, "R": 32, "L": 6, "dtype": "f16"},
        # a prefill batch of several requests beside the large projection
        {**lora, "name": "lora prefill", "M": 8192, "N": 16384, "K": 4096, "R": 16, "L": 8, "dtype": "bf16"},
        # fine-tuning steps: rows of five adapters in no order with odd sizes, and one large batch of a few tasks
        {**lora, "kind": "lora_train", "name": "lora train ragged", "M": 1970, "N": 1001, "K": 776, "R": 8, "L": 5, "dtype": "f16", "order": "mixed"},
        {**lora, "kind": "lora_train", "name": "lora train", "M": 8192, "N": 16384, "K": 4096, "R": 64, "L": 4, "dtype": "bf16", "none": 0.0},
        # the norm in front of a decode step, after the residual sum
        {"kind": "ln", "name": "ln decode", "M": 16, "C": 4096, "dtype": "bf16", "weight": "bf16", "residual": True},
        # 64 images of 197 tokens, the norm in front of a vision transformer's MLP block
        {"kind": "ln", "name": "ln vit", "M": 12608, "C": 768, "dtype": "f16", "weight": "f16", "residual": False},
        # the norm in front of the fixed-point layer: one image, and 32 images
        {"kind": "ln_s8", "name": "ln int8 small", "M": 197, "C": 1024, "dtype": "f16", "weight": "f16", "residual": False},
        {"kind": "ln_s8", "name": "ln int8", "M": 6304, "C": 1024, "dtype": "f16", "weight": "f16", "residual": True},
        # gradients: odd sizes in 32 bits, and a large batch with the residual path's gradient added
        {"kind": "ln_bwd", "name": "ln bwd ragged", "M": 1970, "C": 1001, "dtype": "f32", "weight": "f32", "residual": False},
        {"kind": "ln_bwd", "name": "ln bwd", "M": 8192, "C": 4096, "dtype": "bf16", "weight": "f32", "residual": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    kind = rng.choice(["lora", "lora", "lora_train", "ln", "ln_s8", "ln_bwd"])
    if kind.startswith("lora"):
        M, N, K = _log(rng, 1, 8192), _log(rng, 64, 16384), 8 * _log(rng, 8, 1024)
        L, R = _log(rng, 1, 64), 8 * rng.choice([1, 2, 3, 4, 8, 12, 16])
        if kind == "lora_train":  # the products of the plain form grow with L * R
            L = min(L, max(1, 256 // R))
        while M * (N + K) > 8192 * 20480 or M * (N + K) * L * R > 8192 * 20480 * 256:
            M = max(1, M // 2)
        return {"kind": kind, "M": M, "N": N, "K": K, "R": R, "L": L, "dtype": rng.choice(["f16", "bf16"]),
                "order": rng.choice(["requests", "mixed"]), "none": rng.choice([0.0, 0.1, 0.5])}
    C = _log(rng, 8, 16384)
    M = _log(rng, 1, min(65536, (8192 * 4096) // C))
    dtype = rng.choice(["f16", "bf16"] if kind == "ln_s8" else ["f16", "bf16", "f32"])
    return {"kind": kind, "M": M, "C": C, "dtype": dtype, "weight": rng.choice([dtype, "f32"]),
            "residual": rng.choice([True, False])}


def _matrix(gen, rows, cols, dtype, std):
    """A [rows, cols] matrix of normal values whose rows are padded to a multiple of 16 bytes."""
    step = 16 // torch.empty((), dtype=dtype).element_size()
    buf = torch.randn(rows, -(-cols // step) * step, generator=gen, device="cuda", dtype=torch.float32)
    return buf.mul_(std).to(dtype)[:, :cols]


def _index(rng, case):
    """The adapter of each row, -1 for none: runs of rows as requests come, or rows in no order."""
    M, L = case["M"], case["L"]
    out = []
    while len(out) < M:
        n = 1 if case["order"] == "mixed" else _log(rng, 8, 2048)
        out += [-1 if rng.random() < case["none"] else rng.randrange(L)] * n
    return torch.tensor(out[:M], dtype=torch.int32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = random.Random(int(seed))
    M, dt = case["M"], DTYPES[case["dtype"]]
    s = {"case": case}
    if case["kind"].startswith("lora"):
        N, K, R, L = case["N"], case["K"], case["R"], case["L"]
        s["index"] = _index(rng, case)
        s["X"] = _matrix(gen, M, K, dt, 1.0)
        s["A"] = _matrix(gen, L * R, K, dt, 0.02).view(L, R, K)
        s["B"] = _matrix(gen, L * N, R, dt, 0.02).view(L, N, R)
        s["scale"] = torch.rand(L, generator=gen, device="cuda") * 1.5 + 0.5
        s["base"] = _matrix(gen, M, N, dt, 1.0)  # the shared projection's output
        if case["kind"] == "lora_train":
            s["dY"] = _matrix(gen, M, N, dt, 0.05)
            s["dbase"] = _matrix(gen, M, K, dt, 0.05)  # the shared projection's gradient of X
        return s
    C, wdt = case["C"], DTYPES[case["weight"]]
    s["eps"] = 1e-5
    s["X"] = _matrix(gen, M, C, dt, 1.5)
    s["gamma"] = (1.0 + 0.2 * torch.randn(C, generator=gen, device="cuda")).to(wdt)
    s["beta"] = (0.1 * torch.randn(C, generator=gen, device="cuda")).to(wdt)
    s["qscale"] = 127.0 / 4.0  # four standard deviations of a normalised row
    s["residual"] = _matrix(gen, M, C, dt, 0.5) if case["residual"] else None
    if case["kind"] == "ln_bwd":
        s["dY"] = _matrix(gen, M, C, dt, 0.1)
        x = s["X"].float()
        s["mean"] = x.mean(1)
        s["rstd"] = (x - s["mean"][:, None]).square().mean(1).add_(s["eps"]).rsqrt_()
    return s


def _plain_lora(s, train):
    """All adapters' products at once; a mask keeps each row's own."""
    dt = s["X"].dtype
    L, R, K = s["A"].shape
    N = s["B"].shape[1]
    X = s["X"].float()
    A = s["A"].float().reshape(L * R, K)
    B = s["B"].float().transpose(1, 2).reshape(L * R, N)
    own_row = s["index"][:, None] == torch.arange(L, device=X.device, dtype=torch.int32)[None, :]
    mask = own_row.float().repeat_interleave(R, 1)
    scaled = (own_row.float() * s["scale"][None, :]).repeat_interleave(R, 1)
    P = X @ A.T
    Y = s["base"].float() + (P * scaled) @ B
    V = (P * mask).view(-1, L, R).sum(1)
    if not train:
        return {"Y": Y.to(dt), "V": V.to(dt)}
    dY = s["dY"].float()
    U = (dY @ B.T) * scaled
    dX = s["dbase"].float() + U @ A
    dA = (U.T @ X).view(L, R, K)
    dB = (dY.T @ (P * scaled)).view(N, L, R).transpose(0, 1).contiguous()
    return {"Y": Y.to(dt), "V": V.to(dt), "dX": dX.to(dt), "dA": dA.to(dt), "dB": dB.to(dt)}


def _plain_ln(s):
    h = s["X"].float()
    H = None
    if s["residual"] is not None:
        H = (h + s["residual"].float()).to(s["X"].dtype)  # the sum is kept for the backward pass: rounded here
        h = H.float()
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = (d.square().mean(1) + s["eps"]).rsqrt()
    return d * rstd[:, None] * s["gamma"].float() + s["beta"].float(), H, mean, rstd


def _plain_ln_bwd(s):
    xhat = (s["X"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dY = s["dY"].float()
    g = dY * s["gamma"].float()
    dX = s["rstd"][:, None] * (g - g.mean(1)[:, None] - xhat * (g * xhat).mean(1)[:, None])
    if s["residual"] is not None:  # in this case the gradient that reaches the sum by the other path
        dX = dX + s["residual"].float()
    return {"dX": dX.to(s["X"].dtype), "dgamma": (dY * xhat).sum(0).to(s["gamma"].dtype), "dbeta": dY.sum(0).to(s["gamma"].dtype)}


def _own(s):
    import structured_sparse_gemm_02_b200 as spg

    kind = s["case"]["kind"]
    if kind.startswith("lora"):
        plan = spg.lora_plan(s["index"], s["A"].shape[0])
        Y, V = spg.lora_f16(s["X"], s["A"], s["B"], plan, scale=s["scale"], base=s["base"])
        if kind == "lora":
            return {"Y": Y, "V": V}
        dX, dA, dB = spg.lora_f16_bwd(s["dY"], s["X"], V, s["A"], s["B"], plan, scale=s["scale"], dbase=s["dbase"])
        return {"Y": Y, "V": V, "dX": dX, "dA": dA, "dB": dB}
    if kind == "ln":
        Y, H, mean, rstd = spg.layernorm(s["X"], s["gamma"], s["beta"], s["eps"], residual=s["residual"], stats=True)
        return {"Y": Y, "H": H, "mean": mean, "rstd": rstd}
    if kind == "ln_s8":
        Yq, H = spg.layernorm_s8(s["X"], s["gamma"], s["beta"], s["qscale"], s["eps"], residual=s["residual"])
        return {"Y": Yq.to(torch.float16), "H": H}
    dX, dgamma, dbeta = spg.layernorm_bwd(s["dY"], s["X"], s["mean"], s["rstd"], s["gamma"], dH=s["residual"])
    return {"dX": dX, "dgamma": dgamma, "dbeta": dbeta}


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind.startswith("lora"):
        return _plain_lora(state, kind == "lora_train")
    if kind == "ln_bwd":
        return _plain_ln_bwd(state)
    y, H, mean, rstd = _plain_ln(state)
    if kind == "ln_s8":
        return {"Y": (y * state["qscale"]).round().clamp(-127, 127).to(torch.float16), "H": H}
    return {"Y": y.to(state["X"].dtype), "H": H, "mean": mean, "rstd": rstd}


def work(case):
    M = case["M"]
    if case["kind"].startswith("lora"):
        N, K, R, L = case["N"], case["K"], case["R"], case["L"]
        rows = M * (1.0 - case["none"])
        runs = rows if case["order"] == "mixed" else rows / 368 + 1  # 368: the mean length of a request's run
        weights = L * (1.0 - (1.0 - 1.0 / L) ** runs) * R * (N + K)  # of the adapters that are drawn at all
        elems = rows * K + M * (2 * N + R) + weights
        flops = 2.0 * rows * R * (N + K)
        if case["kind"] == "lora_train":  # dY, dbase and dX once more each, and the weights' gradients
            elems += M * (N + 2 * K) + L * R * (N + K)
            flops *= 3.0
        return {"bytes": 2 * elems + 4 * M + 4 * L, "flops": flops}
    C = case["C"]
    es, ws = (4 if case[k] == "f32" else 2 for k in ("dtype", "weight"))
    if case["kind"] == "ln_bwd":
        return {"bytes": es * M * C * (4 if case["residual"] else 3) + 8 * M + 3 * ws * C, "flops": 12.0 * M * C}
    out = 1 if case["kind"] == "ln_s8" else es
    stats = 8 * M if case["kind"] == "ln" else 0
    return {"bytes": M * C * (es + out + (2 * es if case["residual"] else 0)) + stats + 2 * ws * C, "flops": 8.0 * M * C}


def exact(case, seed):
    """The same outputs from the definitions, adapter by adapter and in 64 bits."""
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["kind"].startswith("lora"):
        Y, V = d["base"].clone(), torch.zeros(case["M"], case["R"], dtype=torch.float64, device="cuda")
        train = case["kind"] == "lora_train"
        out = {"Y": Y, "V": V}
        if train:
            out.update(dX=d["dbase"].clone(), dA=torch.zeros_like(d["A"]), dB=torch.zeros_like(d["B"]))
        for a in range(case["L"]):
            rows = torch.nonzero(s["index"] == a).flatten()
            x, f = d["X"][rows], float(s["scale"][a])
            V[rows] = v = torch.einsum("mk,rk->mr", x, d["A"][a])
            Y[rows] += f * torch.einsum("mr,nr->mn", v, d["B"][a])
            if train:
                g = d["dY"][rows]
                u = f * torch.einsum("mn,nr->mr", g, d["B"][a])
                out["dX"][rows] += torch.einsum("mr,rk->mk", u, d["A"][a])
                out["dA"][a] = torch.einsum("mr,mk->rk", u, x)
                out["dB"][a] = f * torch.einsum("mn,mr->nr", g, v)
        return out
    gamma, beta = d["gamma"], d["beta"]
    if case["kind"] == "ln_bwd":
        mu, r = d["mean"].unsqueeze(1), d["rstd"].unsqueeze(1)
        z = (d["X"] - mu) * r
        a = d["dY"] * gamma
        C = case["C"]
        dX = r / C * (C * a - a.sum(1, keepdim=True) - z * (a * z).sum(1, keepdim=True))
        return {"dX": dX if s["residual"] is None else dX + d["residual"], "dgamma": torch.einsum("mc,mc->c", d["dY"], z), "dbeta": d["dY"].sum(0)}
    H = None
    h = d["X"]
    if s["residual"] is not None:
        H = (h + d["residual"]).to(s["X"].dtype).double()
        h = H
    var, mu = torch.var_mean(h, dim=1, correction=0)
    r = 1.0 / torch.sqrt(var + s["eps"])
    y = (h - mu.unsqueeze(1)) * r.unsqueeze(1) * gamma + beta
    if case["kind"] == "ln_s8":
        return {"Y": torch.clamp(torch.round(y * s["qscale"]), -127, 127), "H": H}
    return {"Y": y, "H": H, "mean": mu, "rstd": r}
