"""Low-rank adapters (plan, forward, backward) against their formulas in 64 bits.

Tolerances, from the arithmetic: an output is rounded once to its type
(``finfo.eps / 2`` relative, or half the smallest subnormal).  A sum of n products of 16-bit
values in fp32 is off by at most n * 2^-23 of the sum of the magnitudes (the
products are exact; twice the unit roundoff per addition covers the tensor
cores' truncation), plus 16 * 2^-23 for the scale and the last additions.  V is
an output: what follows from it is tested from the V the call returned.  U is
internal: its rounding and sum errors enter dX and dA through the magnitudes
of A and X."""
import pytest

from tests.gpu_util import Guarded, need_gpu

pytestmark = pytest.mark.gpu

E = 2.0 ** -23


def _dt(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def _half(y, dtype):
    import torch
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}[dtype]
    return torch.clamp(y.abs() * torch.finfo(dtype).eps / 2, min=tiny)


def _mat(g, shape, dt, std=1.0, pad=0):
    """Random [rows, cols] (or more dims, contiguous); rows padded to 8 elements and `pad` more, the padding NaN."""
    import torch
    if len(shape) != 2:
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)
    M, C = shape
    buf = torch.full((max(1, M), (C + 7) // 8 * 8 + pad), float("nan"), dtype=dt, device="cuda")
    buf[:M, :C] = (torch.randn(M, C, generator=g, device="cuda") * std).to(dt)
    return buf[:M, :C]


def _problem(M, N, K, R, L, dt, none=0.2, order="mixed", seed=0, pad=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + M + N + K)
    index = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    if order == "runs":
        index = index.sort().values.to(torch.int32)
    gone = torch.rand(M, generator=g, device="cuda") < none
    index[gone] = torch.where(torch.rand(int(gone.sum()), generator=g, device="cuda") < 0.5, -1, L + 3).int()
    return dict(index=index, X=_mat(g, (M, K), dt, pad=pad), A=_mat(g, (L, R, K), dt, 0.05), B=_mat(g, (L, N, R), dt, 0.05),
                scale=torch.rand(L, generator=g, device="cuda") * 1.5 + 0.5, base=_mat(g, (M, N), dt, pad=pad),
                dY=_mat(g, (M, N), dt, 0.1, pad=pad), dbase=_mat(g, (M, K), dt, 0.1, pad=pad), L=L)


def _check_forward(p, Y, V):
    import torch
    dt, L = p["X"].dtype, p["L"]
    M, K = p["X"].shape
    R = p["A"].shape[1]
    none = (p["index"] < 0) | (p["index"] >= L)
    assert not V[none].any() and torch.equal(Y[none], (torch.zeros_like(Y) if p["base"] is None else p["base"])[none])
    for a in range(L):
        rows = torch.nonzero(p["index"] == a).flatten()
        if not len(rows):
            continue
        x, A, B = p["X"][rows].double(), p["A"][a].double(), p["B"][a].double()
        v = x @ A.T
        tol = (K + 16) * E * (x.abs() @ A.abs().T)
        assert torch.all((V[rows].double() - v).abs() <= tol + _half(v, dt)), a
        s = 1.0 if p["scale"] is None else float(p["scale"][a])
        v = V[rows].double()
        y = s * (v @ B.T) + (0 if p["base"] is None else p["base"][rows].double())
        tol = (R + 16) * E * (s * (v.abs() @ B.abs().T) + y.abs())
        assert torch.all((Y[rows].double() - y).abs() <= tol + _half(y, dt)), a


def _check_backward(p, V, dX, dA, dB):
    import torch
    dt, L = p["X"].dtype, p["L"]
    N = p["B"].shape[1]
    R = p["A"].shape[1]
    none = (p["index"] < 0) | (p["index"] >= L)
    if dX is not None:
        assert torch.equal(dX[none], (torch.zeros_like(dX) if p["dbase"] is None else p["dbase"])[none])
    for a in range(L):
        rows = torch.nonzero(p["index"] == a).flatten()
        if not len(rows):
            assert not dA[a].any() and not dB[a].any()
            continue
        x, A, B = p["X"][rows].double(), p["A"][a].double(), p["B"][a].double()
        s = 1.0 if p["scale"] is None else float(p["scale"][a])
        dy, v = p["dY"][rows].double(), V[rows].double()
        u = s * (dy @ B)
        du = _half(u, dt) + (N + 16) * E * s * (dy.abs() @ B.abs())
        if dX is not None:
            want = u @ A + (0 if p["dbase"] is None else p["dbase"][rows].double())
            tol = (du @ A.abs()) + (R + 16) * E * ((u.abs() + du) @ A.abs() + want.abs())
            assert torch.all((dX[rows].double() - want).abs() <= tol + _half(want.abs() + tol, dt)), a
        want = u.T @ x
        tol = du.T @ x.abs() + (len(rows) + 16) * E * ((u.abs() + du).T @ x.abs())
        assert torch.all((dA[a].double() - want).abs() <= tol + _half(want.abs() + tol, dt)), a
        want = s * (dy.T @ v)
        tol = (len(rows) + 16) * E * s * (dy.abs().T @ v.abs())
        assert torch.all((dB[a].double() - want).abs() <= tol + _half(want.abs() + tol, dt)), a


@pytest.mark.parametrize("M,L", [(1, 1), (5, 3), (31, 8), (64, 64), (1000, 7), (4097, 300), (300, 8192), (9000, 1)])
def test_plan(M, L):
    """The plan's words: groups in order, rows of a group ascending, tiles of at most 128 rows of one group."""
    need_gpu()
    import numpy as np
    import torch
    import structured_sparse_gemm_02_b200 as spg
    idx = np.random.default_rng(M + L).integers(-2, L + 2, M).astype(np.int32)
    plan = spg.lora_plan(torch.from_numpy(idx).cuda(), L)
    w = plan.buf.cpu().numpy()
    g = np.where((idx >= 0) & (idx < L), idx, L)
    start = np.searchsorted(np.sort(g), np.arange(L + 2))
    r4 = lambda v: (v + 3) // 4 * 4
    assert np.array_equal(w[4:4 + L + 2], start)
    o = 4 + r4(L + 2)
    assert np.array_equal(w[o:o + M], np.argsort(g, kind="stable"))
    o += r4(M)
    want = [(a if a < L else -1, b, min(128, start[a + 1] - b), 0) for a in range(L + 1)
            for b in range(start[a], start[a + 1], 128)]
    assert w[0] == len(want) and np.array_equal(w[o:o + 4 * len(want)].reshape(-1, 4), np.array(want).reshape(-1, 4))


SIZES = [  # M, N, K, R, L, dtype, rows' order, rows without an adapter, further padding
    (1, 1, 8, 8, 1, "f16", "mixed", 0.0, 0), (3, 7, 16, 8, 2, "bf16", "mixed", 0.3, 8), (16, 64, 64, 16, 4, "f16", "mixed", 0.0, 0),
    (129, 130, 136, 24, 3, "bf16", "runs", 0.2, 0), (64, 1000, 776, 16, 64, "f16", "mixed", 0.1, 16), (300, 257, 520, 40, 5, "f16", "runs", 0.5, 0),
    (777, 768, 768, 32, 6, "bf16", "mixed", 0.1, 0), (500, 500, 200, 64, 2, "f16", "runs", 0.0, 8), (257, 384, 1024, 72, 3, "bf16", "mixed", 0.2, 0),
    (400, 333, 640, 128, 4, "f16", "mixed", 0.2, 0), (2000, 1001, 264, 8, 1, "bf16", "mixed", 0.0, 0), (1200, 640, 4096, 16, 2, "bf16", "runs", 0.1, 0),
    (130, 4096, 64, 96, 200, "bf16", "mixed", 0.1, 0), (40, 100, 8192, 16, 3, "f16", "mixed", 1.0, 0),
]


@pytest.mark.parametrize("M,N,K,R,L,dt,order,none,pad", SIZES)
def test_forward_and_backward(M, N, K, R, L, dt, order, none, pad):
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    p = _problem(M, N, K, R, L, _dt(dt), none, order, pad=pad)
    plan = spg.lora_plan(p["index"], L)
    Y, V = spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"], base=p["base"])
    torch.cuda.synchronize()
    assert spg.check_device_error() == 0
    _check_forward(p, Y, V)
    dX, dA, dB = spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], plan, scale=p["scale"], dbase=p["dbase"])
    torch.cuda.synchronize()
    assert spg.check_device_error() == 0
    _check_backward(p, V, dX, dA, dB)
    again = spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"], base=p["base"]) + spg.lora_f16_bwd(
        p["dY"], p["X"], V, p["A"], p["B"], plan, scale=p["scale"], dbase=p["dbase"])
    assert all(torch.equal(a, b) for a, b in zip((Y, V, dX, dA, dB), again))


def test_without_base_scale_or_dx_and_in_place():
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    p = _problem(300, 200, 256, 16, 3, torch.bfloat16)
    plan = spg.lora_plan(p["index"], 3)
    Y, V = spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"], base=p["base"])
    acc = p["base"].clone()
    got, _ = spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"], base=acc, Y=acc)
    assert got is acc and torch.equal(acc, Y)
    dX, dA, dB = spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], plan, scale=p["scale"], dbase=p["dbase"])
    acc = p["dbase"].clone()
    got = spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], plan, scale=p["scale"], dbase=acc, dX=acc)
    assert got[0] is acc and torch.equal(acc, dX) and torch.equal(got[1], dA) and torch.equal(got[2], dB)
    none, dA2, dB2 = spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], plan, scale=p["scale"], need_dx=False)
    assert none is None and torch.equal(dA2, dA) and torch.equal(dB2, dB)
    q = dict(p, base=None, dbase=None, scale=None)
    Y, V = spg.lora_f16(p["X"], p["A"], p["B"], plan)
    _check_forward(q, Y, V)
    _check_backward(q, V, *spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], plan))


def test_bad_values_stay_with_their_rows_and_adapters():
    """NaN and infinities in one row, one adapter or the padding leave every other result's bits alone."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    M, N, K, R, L = 260, 203, 72, 8, 4
    p = _problem(M, N, K, R, L, torch.float16, none=0.1)
    plan = spg.lora_plan(p["index"], L)

    def run(q):
        Y, V = spg.lora_f16(q["X"], q["A"], q["B"], plan, scale=q["scale"], base=q["base"])
        return (Y, V) + spg.lora_f16_bwd(q["dY"], q["X"], V, q["A"], q["B"], plan, scale=q["scale"], dbase=q["dbase"])

    clean = run(p)
    gen = torch.Generator(device="cuda")
    q = dict(p, X=p["X"].clone(), dY=_mat(gen, (M, N), torch.float16).copy_(p["dY"]),  # a clone has no padded rows
             A=p["A"].clone(), B=p["B"].clone())
    q["A"][1], q["B"][1] = float("nan"), float("inf")
    row = int(torch.nonzero(p["index"] == 2)[0])
    q["X"][row, 3], q["dY"][row, 5] = float("inf"), float("nan")
    none = torch.nonzero((p["index"] < 0) | (p["index"] >= L)).flatten()
    q["X"][none], q["dY"][none] = float("nan"), float("nan")
    got = run(q)
    keep = p["index"] != 1
    keep[row] = False
    for a, b in zip(clean[:3], got[:3]):
        assert torch.equal(a[keep], b[keep])
    for a, b in zip(clean[3:], got[3:]):
        assert torch.equal(a[[0, 3]], b[[0, 3]])
    assert got[0][row].isnan().any() and got[3][1].isnan().all()


def test_guards_and_rows_behind_the_batch():
    """Nothing outside the outputs is written: not their padding, not the rows behind M."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    M, N, K, R, L = 141, 93, 72, 16, 3
    dt = torch.bfloat16
    p = _problem(M, N, K, R, L, dt)
    plan = spg.lora_plan(p["index"], L)
    Yg, Vg, Xg = Guarded((M + 5, 104), dt), Guarded((M + 5, 24), dt), Guarded((M + 5, 80), dt)
    for t in (Yg, Vg, Xg):
        t.t.fill_(3.0)
    Ag, Bg = Guarded((L, R, K), dt), Guarded((L, N, R), dt)
    Y, V = Yg.t[:M, :N], Vg.t[:M, :R]
    spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"], base=p["base"], Y=Y, V=V)
    spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], plan, scale=p["scale"], dbase=p["dbase"], dX=Xg.t[:M, :K],
                     dA=Ag.t, dB=Bg.t)
    torch.cuda.synchronize()
    _check_forward(p, Y, V)
    _check_backward(p, V, Xg.t[:M, :K], Ag.t, Bg.t)
    for g, c in ((Yg, N), (Vg, R), (Xg, K)):
        assert g.intact() and bool((g.t[M:] == 3.0).all()) and bool((g.t[:, c:] == 3.0).all())
    assert Ag.intact() and Bg.intact()


def test_empty_batch():
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    p = _problem(4, 40, 48, 8, 2, torch.float16)
    plan = spg.lora_plan(p["index"][:0], 2)
    Y, V = spg.lora_f16(p["X"][:0], p["A"], p["B"], plan, base=p["base"][:0])
    assert Y.shape == (0, 40) and V.shape == (0, 8)
    dX, dA, dB = spg.lora_f16_bwd(p["dY"][:0], p["X"][:0], V, p["A"], p["B"], plan)
    assert dX.shape == (0, 48) and not dA.any() and not dB.any()


def test_graph_follows_a_refilled_plan_and_streams():
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    M, N, K, R, L = 200, 320, 256, 16, 5
    p = _problem(M, N, K, R, L, torch.bfloat16, none=0.1)
    plan = spg.lora_plan(p["index"], L)

    def step(pl, stream=None):
        Y, V = spg.lora_f16(p["X"], p["A"], p["B"], pl, scale=p["scale"], base=p["base"], stream=stream)
        return (Y, V) + spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], pl, scale=p["scale"], dbase=p["dbase"],
                                         stream=stream)

    want = step(plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(plan, s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spg.lora_plan(p["index"], L, plan=plan)
        outs = step(plan)
    p["index"].copy_(p["index"].flip(0))
    p["X"].copy_(p["X"].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    want = step(spg.lora_plan(p["index"], L))
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    assert spg.check_device_error() == 0


def test_gradients_against_differences():
    """dX, dA and dB of the sum of Y * dY against central differences of the formula in 64 bits.
    The loss is a polynomial (at most bilinear in each input alone), so the differences are exact to
    64-bit rounding; the tolerance is the backward pass's own roundings: three of them (V, U,
    the result) of half a step each, in the root of the sum of squares of a gradient."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    M, N, K, R, L = 6, 9, 16, 8, 2
    p = _problem(M, N, K, R, L, torch.float16, none=0.0)
    plan = spg.lora_plan(p["index"], L)
    _, V = spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"])
    grads = spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], plan, scale=p["scale"])
    args = [p["X"].double(), p["A"].double(), p["B"].double()]
    idx = p["index"].long()

    def loss(X, A, B):
        v = torch.einsum("mk,mrk->mr", X, A[idx])
        return (p["scale"].double()[idx][:, None] * torch.einsum("mr,mnr->mn", v, B[idx]) * p["dY"].double()).sum()

    for k, g in enumerate(grads):
        want = torch.zeros_like(args[k]).flatten()
        for j in range(want.numel()):
            d = torch.zeros_like(want)
            d[j] = 0.5
            hi, lo = ([a + (s * d).view_as(a) if i == k else a for i, a in enumerate(args)] for s in (1, -1))
            want[j] = loss(*hi) - loss(*lo)
        off = (g.double().flatten() - want).norm()
        assert off <= 3 * 2.0 ** -11 * want.norm()


@pytest.mark.parametrize("M,N,K,R,L,dt", [(200, 5001, 264, 16, 64, "bf16"), (130, 9000, 72, 24, 40, "f16"),
                                          (64, 16384, 128, 32, 64, "bf16"), (33, 20000, 520, 8, 300, "f16"),
                                          (97, 2000, 1032, 128, 64, "bf16"), (127, 700, 2056, 56, 3, "f16"),
                                          (500, 4099, 1024, 16, 33, "bf16"), (5, 30001, 8, 16, 500, "bf16")])
def test_few_rows_in_skewed_groups(M, N, K, R, L, dt):
    """Fewer than 64 rows an adapter, but most of them on one: groups of one row, of several tiles, and none."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    p = _problem(M, N, K, R, L, _dt(dt), none=0.1, seed=21)
    p["index"][: 2 * M // 3] = L // 2
    p["index"][M // 4: M // 3] = -1
    plan = spg.lora_plan(p["index"], L)
    Y, V = spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"], base=p["base"])
    _check_forward(p, Y, V)
    rows = torch.empty_strided(p["base"].shape, p["base"].stride(), dtype=_dt(dt), device="cuda")
    rows.copy_(p["base"])
    spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"], base=rows, Y=rows)
    assert torch.equal(rows, Y)
    Y0, V0 = spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"])
    assert torch.equal(V0, V)
    _check_forward(dict(p, base=None), Y0, V0)
    dX, dA, dB = spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], plan, scale=p["scale"], dbase=p["dbase"])
    _check_backward(p, V, dX, dA, dB)
    assert spg.check_device_error() == 0


@pytest.mark.parametrize("M,K,R,L,dt", [(64, 4096, 72, 64, "bf16"), (30, 8192, 80, 60, "f16"), (96, 4096, 104, 96, "bf16"),
                                        (64, 4096, 40, 64, "f16")])
def test_few_rows_wide_ranks(M, K, R, L, dt):
    """A tile an adapter with blocks that take much of an SM's tensor memory, on two streams at once."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    p = _problem(M, 1000, K, R, L, _dt(dt), none=0.0, seed=31)
    p["index"].copy_(torch.arange(M, dtype=torch.int32) % L)
    plan = spg.lora_plan(p["index"], L)

    def step():
        Y, V = spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"], base=p["base"])
        return Y, V, *spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], plan, scale=p["scale"], dbase=p["dbase"])
    want = step()
    _check_forward(p, *want[:2])
    _check_backward(p, *want[1:])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(step())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for got in outs for a, b in zip(got, want))
    assert spg.check_device_error() == 0
