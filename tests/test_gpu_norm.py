"""Layer norm (forward, int8 output, backward) against its formulas in 64 bits.

Tolerances, from the arithmetic: each output is rounded once to its type (half
a step, ``finfo.eps / 2`` relative to the value, or half the smallest subnormal); before that all is
fp32.  A row's sums take at most 64 roundings one after another (32 columns a
thread, then a tree and at most 32 partial sums), so a mean is off by at most
64 * 2^-24 = 2^-18 of the mean of the magnitudes; the statistics' own error and the few
roundings of an element stay below 2^-18 of the terms that are added.  A
column's sum takes at most 256 roundings (rows of a block, then the blocks'
partial sums): 2^-16 of the sum of the magnitudes."""
import numpy as np
import pytest

from tests.gpu_util import Guarded, need_gpu

pytestmark = pytest.mark.gpu

E = 2.0 ** -18


def _dt(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[name]


def _half(y, dtype):
    import torch
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]
    return torch.clamp(y.abs() * torch.finfo(dtype).eps / 2, min=tiny)


def _mat(g, M, C, dt, std=1.0, mean=0.0, ld=None):
    import torch
    buf = torch.full((max(M, 1), ld or C), float("nan"), dtype=dt, device="cuda")
    buf[:M, :C] = (torch.randn(M, C, generator=g, device="cuda") * std + mean).to(dt)
    return buf[:M, :C]


def _gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ref_fwd(h, gamma, beta, eps):
    h = h.double()
    mu = h.mean(1, keepdim=True)
    r = 1.0 / ((h - mu).square().mean(1, keepdim=True) + eps).sqrt()
    z = (h - mu) * r
    zg = z * gamma.double()
    y = zg + (0 if beta is None else beta.double())
    # the mean's error moves every element of the row, through r and gamma
    tol = E * (zg.abs() + y.abs() + r * gamma.double().abs() * h.abs().mean(1, keepdim=True))
    return y, mu[:, 0], r[:, 0], tol


FWD = [  # M, C, dtype, weight's dtype, residual, beta
    (1, 1, "f16", "f16", False, True), (3, 2, "f32", "f32", True, True), (257, 8, "bf16", "f32", True, False),
    (130, 33, "f16", "f16", False, True), (64, 255, "bf16", "bf16", True, True), (65, 256, "f32", "f32", False, True),
    (37, 257, "f16", "f32", True, True), (1, 768, "f16", "f16", False, True), (515, 768, "f16", "f16", True, True),
    (19, 1001, "bf16", "bf16", False, True), (100, 1024, "bf16", "f32", True, True), (9, 1025, "f16", "f16", True, True),
    (16, 4096, "bf16", "bf16", True, True), (5, 4104, "f32", "f32", False, False), (7, 8191, "f16", "f32", False, True),
    (3, 16384, "bf16", "bf16", True, True), (2, 16384, "f32", "f32", True, True), (3, 12345, "f32", "f32", False, True),
]


@pytest.mark.parametrize("M,C,dt,wdt,residual,beta", FWD)
def test_forward(M, C, dt, wdt, residual, beta):
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    dt, wdt = _dt(dt), _dt(wdt)
    g = _gen(M * 31 + C)
    X = _mat(g, M, C, dt, 1.5, 0.25, ld=C + (8 if C % 2 else 0))
    R = _mat(g, M, C, dt, 0.5) if residual else None
    gamma = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(wdt)
    b = (0.1 * torch.randn(C, generator=g, device="cuda")).to(wdt) if beta else None
    Y, H, mean, rstd = spg.layernorm(X, gamma, b, 1e-5, residual=R, stats=True)
    h = X
    if residual:
        h = (X.float() + R.float()).to(dt)
        assert torch.equal(H, h)
    y, mu, r, tol = _ref_fwd(h, gamma, b, 1e-5)
    assert Y.dtype == dt and torch.all((Y.double() - y).abs() <= tol + _half(y, dt))
    assert torch.all((mean.double() - mu).abs() <= E * h.double().abs().mean(1) + 2.0 ** -24 * mu.abs())
    # d(rstd) / rstd is half the variance's relative error, which the mean's error enters squared
    var = (1 / r ** 2)
    dmu = E * h.double().abs().mean(1)
    assert torch.all((rstd.double() - r).abs() <= r * (E + dmu ** 2 / var))


@pytest.mark.parametrize("M,C,dt,wdt,residual", [(1, 16, "f16", "f16", False), (197, 1024, "f16", "f16", True),
                                                  (33, 1001, "bf16", "f32", True), (6, 16384, "bf16", "bf16", False),
                                                  (40, 7, "f32", "f32", False), (70, 300, "f32", "f32", True)])
def test_int8_output(M, C, dt, wdt, residual):
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    dt, wdt = _dt(dt), _dt(wdt)
    g = _gen(M + C)
    X = _mat(g, M, C, dt, 2.0)
    R = _mat(g, M, C, dt, 1.0) if residual else None
    gamma = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(wdt)
    b = (0.1 * torch.randn(C, generator=g, device="cuda")).to(wdt)
    qs = 127.0 / 2.5  # some values clip
    Yq, H = spg.layernorm_s8(X, gamma, b, qs, residual=R)
    h = (X.float() + R.float()).to(dt) if residual else X
    y, _, _, tol = _ref_fwd(h, gamma, b, 1e-5)
    q32 = float(np.float32(qs))
    v = y * q32
    assert Yq.dtype == torch.int8 and int(Yq.min()) >= -127
    assert torch.all((Yq.double() - v.clamp(-127, 127)).abs() <= 0.5 + tol * q32 + E * v.abs())


def test_int8_output_feeds_the_int8_layer():
    """layernorm_s8 -> spgemm_24_s8: the layer's product of the codes, bit for bit, on padded rows too."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    g = _gen(5)
    M, C, N = 197, 1024, 640
    X = _mat(g, M, C, torch.float16, 1.5)
    gamma = torch.ones(C, dtype=torch.float16, device="cuda")
    W = torch.randint(-127, 128, (N, C), generator=g, device="cuda", dtype=torch.int8)
    Wv, meta = spg.sparse_compress_24(W)
    Wm = spg.sparse_prune_24(W)
    buf = torch.zeros(M, C + 64, dtype=torch.int8, device="cuda")
    Yq, _ = spg.layernorm_s8(X, gamma, None, 32.0, Yq=buf[:, :C])
    acc = spg.spgemm_24_s8(Yq, Wv, meta, out_mode=spg.SPG_OUT_S32)
    assert torch.equal(acc.double(), Yq.double() @ Wm.double().T)
    assert not buf[:, C:].any()


BWD = [(1, 1, "f16", "f16", False), (300, 8, "bf16", "f32", True), (5000, 24, "f32", "f32", False),
       (1000, 255, "bf16", "bf16", True), (777, 257, "f16", "f32", False), (640, 768, "f16", "f16", True),
       (1970, 1001, "f32", "f32", True), (2, 2048, "bf16", "bf16", False), (900, 4096, "bf16", "f32", True),
       (301, 4104, "f16", "f16", False), (120, 8000, "bf16", "bf16", True), (40, 16384, "bf16", "f32", True),
       (40, 16384, "f32", "f32", True), (33, 12345, "f32", "f32", False), (20000, 64, "f16", "f32", False)]


def _ref_bwd(dY, X, mean, rstd, gamma, dH):
    dy, x, ga = dY.double(), X.double(), gamma.double()
    mu, r = mean.double()[:, None], rstd.double()[:, None]
    z = (x - mu) * r
    gr = dy * ga
    m1, m2 = gr.mean(1, keepdim=True), (gr * z).mean(1, keepdim=True)
    dx = r * (gr - m1 - z * m2)
    tol = E * r * (gr.abs() + gr.abs().mean(1, keepdim=True) + z.abs() * (gr * z).abs().mean(1, keepdim=True))
    if dH is not None:
        dx = dx + dH.double()
        tol = tol + E * dH.double().abs()
    return dx, tol, (dy * z).sum(0), (dy * z).abs().sum(0), dy.sum(0), dy.abs().sum(0)


@pytest.mark.parametrize("M,C,dt,wdt,residual", BWD)
def test_backward(M, C, dt, wdt, residual):
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    dt, wdt = _dt(dt), _dt(wdt)
    g = _gen(M * 7 + C)
    X = _mat(g, M, C, dt, 1.5, 0.25, ld=C + (8 if C % 2 else 0))
    dY = _mat(g, M, C, dt, 0.3)
    dH = _mat(g, M, C, dt, 0.3, ld=C + 16) if residual else None
    gamma = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(wdt)
    _, _, mean, rstd = spg.layernorm(X, gamma, None, 1e-5, stats=True)
    dX, dga, dbe = spg.layernorm_bwd(dY, X, mean, rstd, gamma, dH=dH)
    dx, tol, rg, sg, rb, sb = _ref_bwd(dY, X, mean, rstd, gamma, dH)
    assert torch.all((dX.double() - dx).abs() <= tol + _half(dx, dt))
    assert dga.dtype == wdt and dbe.dtype == wdt
    assert torch.all((dga.double() - rg).abs() <= 2.0 ** -16 * sg + _half(rg, wdt))
    assert torch.all((dbe.double() - rb).abs() <= 2.0 ** -16 * sb + _half(rb, wdt))
    again = spg.layernorm_bwd(dY, X, mean, rstd, gamma, dH=dH)  # the sums' order is fixed
    assert all(torch.equal(a, b) for a, b in zip((dX, dga, dbe), again))


def test_gradient_against_differences():
    """fp32 gradients against central differences of the forward formula in 64 bits."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    g = _gen(11)
    M, C, eps = 3, 20, 1e-5
    X = _mat(g, M, C, torch.float32)
    dY = _mat(g, M, C, torch.float32)
    gamma = 1 + 0.2 * torch.randn(C, generator=g, device="cuda")
    _, _, mean, rstd = spg.layernorm(X, gamma, None, eps, stats=True)
    dX, dga, dbe = spg.layernorm_bwd(dY, X, mean, rstd, gamma)

    def loss(x, ga, be):
        mu = x.mean(1, keepdim=True)
        z = (x - mu) / ((x - mu).square().mean(1, keepdim=True) + eps).sqrt()
        return ((z * ga + be) * dY.double()).sum()

    args = [X.double(), gamma.double(), torch.zeros(C, device="cuda", dtype=torch.float64)]
    h = 1e-4  # the differences' own error is h^2 / 6 of a third derivative of order 10: about 2e-8
    for k, grad in enumerate((dX, dga, dbe)):
        flat = args[k].flatten()
        for j in range(0, flat.numel(), 7):
            d = torch.zeros_like(flat)
            d[j] = h
            hi, lo = ([a + (s * d).view_as(a) if i == k else a for i, a in enumerate(args)] for s in (1, -1))
            want = float((loss(*hi) - loss(*lo)) / (2 * h))
            assert abs(float(grad.flatten()[j]) - want) <= 1e-5 * max(1.0, abs(want))


def test_layouts_aliasing_and_guards():
    """Unaligned rows give the bits of aligned ones; outputs in place of inputs; nothing outside is written."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    g = _gen(3)
    M, C, dt = 77, 768, torch.float16
    X, R = _mat(g, M, C, dt), _mat(g, M, C, dt)
    gamma = (1 + 0.1 * torch.randn(C, generator=g, device="cuda")).to(dt)
    beta = (0.1 * torch.randn(C, generator=g, device="cuda")).to(dt)
    Y, H, mean, rstd = spg.layernorm(X, gamma, beta, residual=R, stats=True)
    odd = torch.empty(M * (C + 1) + 1, dtype=dt, device="cuda")[1:].view(M, C + 1)[:, :C]
    odd.copy_(X)
    Yg, Hg = Guarded((M, C + 3), dt), Guarded((M, C), dt)
    Yg.t.fill_(7.0)
    spg.layernorm(odd, gamma, beta, residual=R, H=Hg.t, Y=Yg.t[:, :C])
    assert torch.equal(Yg.t[:, :C], Y) and torch.equal(Hg.t, H) and Yg.intact() and Hg.intact()
    assert bool((Yg.t[:, C:] == 7.0).all())
    x2, r2 = X.clone(), R.clone()
    spg.layernorm(x2, gamma, beta, residual=r2, H=r2, Y=x2)
    assert torch.equal(x2, Y) and torch.equal(r2, H)
    dY = _mat(g, M, C, dt)
    want = spg.layernorm_bwd(dY, H, mean, rstd, gamma, dH=R)
    d2, h2 = dY.clone(), R.clone()
    got = spg.layernorm_bwd(d2, H, mean, rstd, gamma, dH=h2, dX=d2)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    got = spg.layernorm_bwd(dY, H, mean, rstd, gamma, dH=h2, dX=h2)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_bad_rows_stay_alone_and_empty_batches():
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    g = _gen(4)
    M, C, dt = 40, 512, torch.bfloat16
    X = _mat(g, M, C, dt)
    gamma, beta = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    clean = spg.layernorm(X, gamma, beta)[0]
    X2 = X.clone()
    X2[3, 5], X2[9, 0], X2[20] = float("nan"), float("inf"), 2.5  # the last: a constant row, variance 0
    got = spg.layernorm(X2, gamma, beta)[0]
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[[3, 9, 20]] = False
    assert torch.equal(got[keep], clean[keep])
    assert got[3].isnan().all() and got[9].isnan().all() and bool((got[20] == 0).all())
    codes, _ = spg.layernorm_s8(X2, gamma, beta, 30.0)
    assert not codes[3].any()
    E0 = torch.empty(0, C, dtype=dt, device="cuda")
    Y, H, mean, rstd = spg.layernorm(E0, gamma, beta, residual=E0, stats=True)
    assert Y.shape == (0, C) and H.shape == (0, C) and mean.shape == (0,)
    dX, dga, dbe = spg.layernorm_bwd(E0, E0, mean, rstd, gamma)
    assert dX.shape == (0, C) and not dga.any() and not dbe.any()


def test_streams_and_graph():
    """On a stream of its own, and captured: the replay reads the inputs' new values."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    g = _gen(6)
    M, C, dt = 500, 1024, torch.bfloat16
    X, dY = _mat(g, M, C, dt), _mat(g, M, C, dt)
    gamma, beta = torch.ones(C, dtype=dt, device="cuda"), torch.zeros(C, dtype=dt, device="cuda")

    def step(stream=None):
        Y, _, mean, rstd = spg.layernorm(X, gamma, beta, stats=True, stream=stream)
        return (Y,) + spg.layernorm_bwd(dY, X, mean, rstd, gamma, stream=stream)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    X.copy_(_mat(g, M, C, dt))
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
