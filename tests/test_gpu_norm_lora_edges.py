"""Layer norm and low-rank adapters at sizes and in orders of calls where the launch itself, or the
hand-over of a buffer inside a kernel, can go wrong.  The results are compared as in the operators'
own tests, whose tolerances are derived there."""
import os
import subprocess
import sys

import pytest

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("M,L", [(1000, 383), (993, 381), (512, 767), (481, 762), (256, 1535), (225, 1524)])
def test_first_plan_of_a_process(M, L):
    """Counters of just under 48 KB beside the kernel's static arrays, with no larger plan before them in the process."""
    need_gpu()
    p = subprocess.run([sys.executable, "-c", f"from tests.test_gpu_lora import test_plan; test_plan({M}, {L})"],
                       cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


@pytest.mark.parametrize("C,dt", [(512, "f16"), (768, "f16"), (1024, "bf16"), (1001, "f16"), (260, "f32"), (512, "f32")])
def test_backward_through_many_turns_of_the_ring(C, dt):
    """Rows of 33 to 128 vectors, tens of turns of every warp's ring with the residual path's gradient in it: a
    stage that is filled before all of it has been read would change dX.  The same bits from run to run, in place too."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    from tests.test_gpu_norm import _dt, _gen, _half, _mat, _ref_bwd
    dt, g, M = _dt(dt), _gen(C), 60000
    ld = (C + 7) // 8 * 8
    X, dY, dH = _mat(g, M, C, dt, 1.5, 0.25, ld), _mat(g, M, C, dt, 0.3, ld=ld), _mat(g, M, C, dt, 0.3, ld=ld)
    gamma = 1 + 0.2 * torch.randn(C, generator=g, device="cuda")
    _, _, mean, rstd = spg.layernorm(X, gamma, None, 1e-5, stats=True)
    dX, dga, dbe = spg.layernorm_bwd(dY, X, mean, rstd, gamma, dH=dH)
    for i in range(0, M, 20000):  # in parts: the reference holds 64 bits
        r = slice(i, i + 20000)
        want, tol, *_ = _ref_bwd(dY[r], X[r], mean[r], rstd[r], gamma, dH[r])
        assert torch.all((dX[r].double() - want).abs() <= tol + _half(want, dt))
    for turn in range(8):
        out = torch.empty_strided(dH.shape, dH.stride(), dtype=dt, device="cuda").copy_(dH) if turn % 2 else None
        got = spg.layernorm_bwd(dY, X, mean, rstd, gamma, dH=dH if out is None else out, dX=out)
        assert all(torch.equal(a, b) for a, b in zip(got, (dX, dga, dbe)))
    assert spg.check_device_error() == 0


def test_plan_follows_the_kernel_that_writes_its_index():
    """The index comes from a kernel of this library, which lets the plan's start before its own end: each plan
    groups the values of its turn."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    M, N, K, L = 64, 256, 128, 40
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    W = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    W[:, 0] = torch.randint(0, L, (N,), generator=g, device="cuda")
    W[:, 4] = torch.randint(0, L, (N,), generator=g, device="cuda")
    Wv, meta = spg.sparse_compress_24(W)
    picks = []  # the product of such rows is column 0 or column 4 of W
    for c in (0, 4):
        X = torch.zeros(M, K, dtype=torch.int8, device="cuda")
        X[:, c] = 1
        X[1::3] = 0
        picks.append(X)
    rows = torch.empty(M, N, dtype=torch.int32, device="cuda")
    want = []
    for X in picks:
        spg.spgemm_24_s8(X, Wv, meta, Y=rows, out_mode=spg.SPG_OUT_S32)
        assert torch.equal(rows, X.int().sum(1)[:, None] * W[:, 0 if X is picks[0] else 4].int()[None])
        want.append(torch.sort(rows.flatten(), stable=True)[1].int())
    plans = [spg.lora_plan(rows.flatten(), L) for _ in range(50)]
    torch.cuda.synchronize()
    for i, plan in enumerate(plans):  # nothing else between the two calls
        spg.spgemm_24_s8(picks[i % 2], Wv, meta, Y=rows, out_mode=spg.SPG_OUT_S32)
        spg.lora_plan(rows.view(-1), L, plan=plan)
    at = 4 + (L + 2 + 3) // 4 * 4
    for i, plan in enumerate(plans):
        assert torch.equal(plan.buf[at:at + M * N], want[i % 2]), i


@pytest.mark.parametrize("M,C,dt", [(300, 64, "bf16"), (500, 768, "f16"), (500, 769, "f16"), (120, 4104, "bf16"), (40, 16384, "bf16"),
                                    (30, 12345, "f32"), (77, 1001, "f32")])
def test_norm_backward_in_place_of_its_input(M, C, dt):
    """dX over X, as over dY and dH: the bits of a call with memory of its own, with rows of every kind of kernel."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    from tests.test_gpu_norm import _dt, _gen, _mat
    dt, g = _dt(dt), _gen(M + C)
    for ld in (C, (C + 7) // 8 * 8):
        X, dY, dH = (_mat(g, M, C, dt, 0.5, ld=ld) for _ in range(3))
        gamma = 1 + 0.2 * torch.randn(C, generator=g, device="cuda")
        _, _, mean, rstd = spg.layernorm(X, gamma, None, 1e-5, stats=True)
        want = spg.layernorm_bwd(dY, X, mean, rstd, gamma, dH=dH)
        for place in (X, dY, dH):
            kept = place.clone()
            got = spg.layernorm_bwd(dY, X, mean, rstd, gamma, dH=dH, dX=place)
            assert got[0] is place and all(torch.equal(a, b) for a, b in zip(got, want))
            place.copy_(kept)


@pytest.mark.parametrize("M,K,R,L,dt", [(300, 264, 16, 3, "bf16"), (700, 512, 72, 4, "f16"), (40, 4096, 16, 40, "bf16")])
def test_adapters_outputs_over_what_has_been_read(M, K, R, L, dt):
    """Y over X, and dX over X or dY: square layers whose input is not needed any more."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    from tests.test_gpu_lora import _dt, _problem
    p = _problem(M, K, K, R, L, _dt(dt))
    plan = spg.lora_plan(p["index"], L)
    A, B, scale = p["A"], p["B"], p["scale"]
    Y, V = spg.lora_f16(p["X"], A, B, plan, scale=scale, base=p["base"])
    want = spg.lora_f16_bwd(p["dY"], p["X"], V, A, B, plan, scale=scale, dbase=p["dbase"])
    for name in ("X", "dY"):
        q = dict(p)
        q[name] = torch.empty_strided(p[name].shape, p[name].stride(), dtype=_dt(dt), device="cuda").copy_(p[name])
        if name == "X":
            got, _ = spg.lora_f16(q["X"], A, B, plan, scale=scale, base=p["base"], Y=q["X"])
            assert torch.equal(got, Y)
            q["X"].copy_(p["X"])
        got = spg.lora_f16_bwd(q["dY"], q["X"], V, A, B, plan, scale=scale, dbase=p["dbase"], dX=q[name])
        assert got[0] is q[name] and all(torch.equal(a, b) for a, b in zip(got, want))


def _torch():
    import torch
    return torch


@pytest.mark.parametrize("C", [64, 100, 768, 1001, 4096, 4099])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_norm_of_views(C, dt):
    """Weights, statistics and outputs that start anywhere inside their buffers, columns of wider buffers, the
    residual that is X itself: the bits of the same call on memory of its own, and nothing beside the views written."""
    need_gpu()
    torch = _torch()
    import structured_sparse_gemm_02_b200 as spg
    from tests.test_gpu_norm import _dt, _gen, _mat
    dt, g, M = _dt(dt), _gen(C), 37
    X, R, dY = (_mat(g, M, C, dt, 1.0) for _ in range(3))
    gamma, beta = (torch.randn(C, generator=g, device="cuda").to(dt) for _ in range(2))
    want = spg.layernorm(X, gamma, beta, residual=R, stats=True)
    grads = spg.layernorm_bwd(dY, want[1], want[2], want[3], gamma)
    codes = spg.layernorm_s8(X, gamma, beta, 20.0, residual=R)[0]

    def inside(t, at):  # a copy of t whose first element is `at` into its buffer; behind it stays 7
        buf = torch.full((t.numel() + at + 3,), 7, dtype=t.dtype, device="cuda")
        buf[at:at + t.numel()].copy_(t.flatten())
        return buf, buf[at:at + t.numel()].view(t.shape)

    def columns(t, at):  # columns `at` .. of a wider buffer
        buf = torch.full((M, C + at + 5), 7, dtype=t.dtype, device="cuda")
        buf[:, at:at + C].copy_(t)
        return buf, buf[:, at:at + C]

    for at in (1, 3):
        ga, be = inside(gamma, at)[1], inside(beta, at + 1)[1]
        bufs = [columns(X, at) for _ in range(2)]
        got = spg.layernorm(columns(X, at)[1], ga, be, residual=columns(R, at)[1], H=bufs[0][1], Y=bufs[1][1], stats=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        q = columns(torch.zeros_like(codes), at)
        assert torch.equal(spg.layernorm_s8(X, ga, be, 20.0, residual=R, Yq=q[1])[0], codes)
        mean, rstd = inside(want[2], at)[1], inside(want[3], at)[1]
        dx, outs = columns(X, at), [inside(gamma, at), inside(gamma, at + 2)]
        got = spg.layernorm_bwd(columns(dY, at)[1], want[1], mean, rstd, ga, dX=dx[1], dgamma=outs[0][1], dbeta=outs[1][1])
        # rows that are not aligned may be summed in another order
        for a, b, c in zip(got, grads, (1, M, M)):
            assert (a.double() - b.double()).abs().max() <= 2.0 ** -9 * b.double().abs().max(), c
        for buf, view in bufs + [q, dx]:
            assert bool((buf[:, :at] == 7).all()) and bool((buf[:, at + C:] == 7).all())
        for buf, view in outs:
            assert bool((buf[C + 8:] == 7).all()) and bool((buf[:at] == 7).all())
    same = spg.layernorm(X, gamma, beta, residual=X)
    place = X.clone()
    got = spg.layernorm(place, gamma, beta, residual=place, H=place)
    assert torch.equal(got[0], same[0]) and torch.equal(place, same[1])


@pytest.mark.parametrize("how", ["stream", "handle", "current", "default handle"])
def test_calls_on_streams_given_in_every_way(how):
    """A stream object, its raw handle, the current stream and the default stream's handle: one result."""
    need_gpu()
    torch = _torch()
    import structured_sparse_gemm_02_b200 as spg
    from tests.test_gpu_lora import _problem
    p = _problem(200, 136, 264, 16, 3, torch.bfloat16)
    gamma = torch.ones(264, device="cuda")

    def step(stream):
        plan = spg.lora_plan(p["index"], 3, stream=stream)
        Y, _, mean, rstd = spg.layernorm(p["X"], gamma, None, stats=True, stream=stream)
        out, V = spg.lora_f16(Y, p["A"], p["B"], plan, base=p["base"], stream=stream)
        dY, dA, dB = spg.lora_f16_bwd(p["dY"], Y, V, p["A"], p["B"], plan, dbase=p["dbase"], stream=stream)
        return (out, dA, dB) + spg.layernorm_bwd(dY, p["X"], mean, rstd, gamma, stream=stream)
    want = step(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    if how == "current":
        with torch.cuda.stream(s):
            got = step(None)
    else:
        got = step({"stream": s, "handle": s.cuda_stream, "default handle": torch.cuda.default_stream().cuda_stream}[how])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_single_rows_and_parameters():
    """One row cut out of other memory (whatever its strides say), parameters, inference mode."""
    need_gpu()
    torch = _torch()
    import structured_sparse_gemm_02_b200 as spg
    from tests.test_gpu_lora import _problem
    p = _problem(40, 72, 64, 8, 3, torch.float16, none=0.0)
    gamma = torch.nn.Parameter(torch.ones(64, device="cuda"))
    Y = spg.layernorm(p["X"], gamma)[0]
    plan = spg.lora_plan(p["index"], 3)
    out, V = spg.lora_f16(Y, p["A"], p["B"], plan, base=p["base"])
    with torch.inference_mode():
        for r in (0, 7, 39):
            for row in (p["X"][r:r + 1], p["X"][r].clone().view(64, 1).t(), p["X"][r::40][:1]):
                y = spg.layernorm(row, gamma)[0]
                assert torch.equal(y[0], Y[r])
                one = spg.lora_plan(p["index"][r:r + 1], 3)
                a, b = torch.nn.Parameter(p["A"]), torch.nn.Parameter(p["B"])
                got, v = spg.lora_f16(y, a, b, one, base=p["base"][r:r + 1])
                # the sums of few rows may be split in another way
                assert (got[0].double() - out[r].double()).abs().max() <= 2.0 ** -9 * out[r].abs().max()
                assert (v[0].double() - V[r].double()).abs().max() <= 2.0 ** -9 * V[r].abs().max()


@pytest.mark.parametrize("C,dt", [(64, "f16"), (768, "bf16"), (1001, "f16"), (4096, "bf16"), (4100, "f32"), (16384, "f16")])
def test_a_row_of_the_norm_does_not_depend_on_its_batch(C, dt):
    """Rows alone, in a small batch and in a large one: the same bits of Y, the statistics and dX."""
    need_gpu()
    torch = _torch()
    import structured_sparse_gemm_02_b200 as spg
    from tests.test_gpu_norm import _dt, _gen, _mat
    dt, g, M = _dt(dt), _gen(C), 3000
    ld = (C + 7) // 8 * 8
    X, dY, dH = (_mat(g, M, C, dt, 1.0, ld=ld) for _ in range(3))
    gamma = torch.randn(C, generator=g, device="cuda")

    def both(rows):
        Y, _, mean, rstd = spg.layernorm(X[rows], gamma, None, stats=True)
        return Y, mean, rstd, spg.layernorm_bwd(dY[rows], X[rows], mean, rstd, gamma, dH=dH[rows])[0]
    want = both(slice(0, M))
    for rows in (slice(0, 1), slice(7, 8), slice(M - 1, M), slice(100, 117), slice(512, 1536)):
        assert all(torch.equal(a, b[rows]) for a, b in zip(both(rows), want)), rows
