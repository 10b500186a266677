"""Layer norm, pruned layer and low-rank adapters together, as a block uses them: fine-tuning
(forward and backward), int8 serving, single tokens, captured graphs, streams and threads.

Each stage is checked against its formula in 64 bits from the inputs it really had, with the
tolerances of the operators' own tests; the pruned layer's product of n kept terms is off by
at most n * 2^-23 of the sum of their magnitudes and one rounding (half a step).  Runs that
do the same work in another way have to give the same bits."""
import threading

import pytest

from tests.gpu_util import need_gpu
from tests.test_gpu_lora import _check_backward, _check_forward, _problem
from tests.test_gpu_lora import _half as _half16
from tests.test_gpu_norm import E as E_LN
from tests.test_gpu_norm import _half, _ref_bwd, _ref_fwd

pytestmark = pytest.mark.gpu


def _block(M, C, N, R, L, dt, seed, order="mixed"):
    """A block's parameters and a batch; W is 2:4 pruned, `Wm` its masked dense form."""
    import torch
    import structured_sparse_gemm_02_b200 as spg
    p = _problem(M, N, C, R, L, dt, none=0.2, order=order, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)
    W = rand(N, C, std=0.05)
    p.update(x=rand(M, C), res=rand(M, C), gamma=(1 + rand(C, std=0.2)), beta=rand(C, std=0.2), bias=rand(N, std=0.2),
             dH=rand(M, C, std=0.1), dOut=rand(M, N, std=0.1), Wm=spg.sparse_prune_24(W))
    p["Wv"], p["meta"] = spg.sparse_compress_24(W)
    return p


def _forward(p, plan, stats=True, stream=None):
    import structured_sparse_gemm_02_b200 as spg
    Y, H, mean, rstd = spg.layernorm(p["x"], p["gamma"], p["beta"], 1e-5, residual=p["res"], stats=stats, stream=stream)
    P = spg.spgemm_24_f16(Y, p["Wv"], p["meta"], p["bias"], stream=stream)
    base = P.clone() if p.get("keep") else None
    out, V = spg.lora_f16(Y, p["A"], p["B"], plan, scale=p["scale"], base=P, Y=P, stream=stream)
    return dict(Y=Y, H=H, mean=mean, rstd=rstd, base=base, out=out, V=V)


def _backward(p, f, plan, stream=None):
    import torch
    import structured_sparse_gemm_02_b200 as spg
    dbase = torch.matmul(p["dOut"], p["Wm"])  # the frozen layer's gradient of its input
    kept = dbase.clone() if p.get("keep") else None
    dY, dA, dB = spg.lora_f16_bwd(p["dOut"], f["Y"], f["V"], p["A"], p["B"], plan, scale=p["scale"], dbase=dbase,
                                  dX=dbase, stream=stream)
    before = dY.clone() if p.get("keep") else None
    dx, dga, dbe = spg.layernorm_bwd(dY, f["H"], f["mean"], f["rstd"], p["gamma"], dH=p["dH"], dX=dY, stream=stream)
    return dict(dbase=kept, dY=before, dA=dA, dB=dB, dx=dx, dgamma=dga, dbeta=dbe)


def _check(p, f, b=None):
    """Every stage from the inputs that it had (p["keep"] saved what the next one overwrites)."""
    import torch
    dt, C = p["x"].dtype, p["x"].shape[1]
    h = (p["x"].float() + p["res"].float()).to(dt)
    assert torch.equal(f["H"], h)
    y, _, _, tol = _ref_fwd(h, p["gamma"], p["beta"], 1e-5)
    assert torch.all((f["Y"].double() - y).abs() <= tol + _half(y, dt))
    w = p["Wm"].double()
    y = f["Y"].double() @ w.T + p["bias"].double()
    tol = (C // 2 + 16) * 2.0 ** -23 * (f["Y"].double().abs() @ w.abs().T + p["bias"].double().abs())
    assert torch.all((f["base"].double() - y).abs() <= tol + _half16(y.abs() + tol, dt))
    q = dict(p, X=f["Y"], base=f["base"], dY=p["dOut"])
    _check_forward(q, f["out"], f["V"])
    if b is None:
        return
    q["dbase"] = b["dbase"]
    _check_backward(q, f["V"], b["dY"], b["dA"], b["dB"])
    dx, tol, rg, sg, rb, sb = _ref_bwd(b["dY"], f["H"], f["mean"], f["rstd"], p["gamma"], p["dH"])
    assert torch.all((b["dx"].double() - dx).abs() <= tol + _half(dx, dt))
    assert torch.all((b["dgamma"].double() - rg).abs() <= 2.0 ** -16 * sg + _half(rg, dt))
    assert torch.all((b["dbeta"].double() - rb).abs() <= 2.0 ** -16 * sb + _half(rb, dt))


def _outputs(f, b):
    return [f[k] for k in ("Y", "H", "mean", "rstd", "out", "V")] + [b[k] for k in ("dA", "dB", "dx", "dgamma", "dbeta")]


BLOCKS = [(1, 768, 2304, 16, 1, "f16"), (70, 512, 384, 40, 7, "bf16"), (591, 1024, 640, 8, 4, "f16"),
          (1030, 768, 1160, 72, 3, "bf16")]


@pytest.mark.parametrize("M,C,N,R,L,dt", BLOCKS)
def test_training_step(M, C, N, R, L, dt):
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    p = _block(M, C, N, R, L, {"f16": torch.float16, "bf16": torch.bfloat16}[dt], M)
    p["keep"] = True
    plan = spg.lora_plan(p["index"], L)
    f = _forward(p, plan)
    b = _backward(p, f, plan)
    _check(p, f, b)
    assert spg.check_device_error() == 0


def test_captured_step_follows_its_inputs():
    """Plan, forward and backward in one graph, captured beside an eager step: each replay gives the
    bits of an eager step on the inputs and the index that it finds."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    M, C, N, R, L = 300, 768, 640, 16, 5
    p = _block(M, C, N, R, L, torch.bfloat16, 3)
    other = _block(M, C, N, R, L, torch.bfloat16, 4, order="runs")

    def step():
        plan = spg.lora_plan(p["index"], L)
        f = _forward(p, plan)
        return _outputs(f, _backward(p, f, plan))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    held = step()  # an eager step's tensors live through the capture
    bits = [t.clone() for t in held]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for turn in range(3):
        if turn == 1:
            for k in ("x", "res", "dOut", "dH", "index", "scale"):
                p[k].copy_(other[k])
        graph.replay()
        got = [t.clone() for t in outs]
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn
    assert all(torch.equal(a, b) for a, b in zip(held, bits))
    assert spg.check_device_error() == 0


def test_two_threads_and_two_graphs_at_once():
    """Two host threads with a stream each, then two graphs on two streams, one plan read by both:
    the bits of the same steps one after the other."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    M, C, N, R, L = 600, 1024, 1160, 72, 4
    ps = [_block(M, C, N, R, L, torch.float16, s) for s in (5, 6)]
    ps[1]["index"] = ps[0]["index"]
    plan = spg.lora_plan(ps[0]["index"], L)

    def step(p):
        f = _forward(p, plan)
        return _outputs(f, _backward(p, f, plan))
    want = [step(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[], []]
    errors = []

    def run(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(8):
                    got[i].append(step(ps[i]))
            streams[i].synchronize()
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for i in range(2):
        assert all(torch.equal(a, b) for outs in got[i] for a, b in zip(outs, want[i]))
    graphs, outs = [], []
    for i, p in enumerate(ps):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[i]):
            outs.append(step(p))
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(8):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
    assert spg.check_device_error() == 0


def test_calls_on_a_named_stream():
    """stream= moves a whole step to that stream while another one is current."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    p = _block(130, 512, 384, 16, 3, torch.float16, 7)
    plan = spg.lora_plan(p["index"], 3)
    want = _forward(p, plan)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    plan2 = spg.lora_plan(p["index"], 3, stream=s)
    Y, H, mean, rstd = spg.layernorm(p["x"], p["gamma"], p["beta"], 1e-5, residual=p["res"], stats=True, stream=s)
    base = torch.zeros(130, 384, dtype=torch.float16, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    spg.spgemm_24_f16(Y, p["Wv"], p["meta"], p["bias"], Y=base, stream=s)
    out, V = spg.lora_f16(Y, p["A"], p["B"], plan2, scale=p["scale"], base=base, stream=s)
    s.synchronize()
    for a, b in ((Y, "Y"), (H, "H"), (mean, "mean"), (rstd, "rstd"), (out, "out"), (V, "V")):
        assert torch.equal(a, want[b])


def test_single_tokens():
    """Decode: one captured step of a few requests with an adapter each, its index refilled between replays."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    M, C, N, R, L = 6, 768, 2304, 16, 32
    p = _block(M, C, N, R, L, torch.float16, 9)
    p["keep"] = True
    plan = spg.lora_plan(p["index"], L)
    _forward(p, plan, stats=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spg.lora_plan(p["index"], L, plan=plan)
        f = _forward(p, plan, stats=False)
    for index in ([0, 1, 2, 3, 4, 5], [31, 31, -1, 31, 32, 0], [-1] * 6):
        p["index"].copy_(torch.tensor(index, dtype=torch.int32))
        graph.replay()
        _check(p, f)


def test_int8_layer_with_adapters():
    """The norm's int8 codes feed the int8 layer, its fp16 copy the adapters of the same rows."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    M, C, N, R, L = 197, 1024, 640, 16, 4
    p = _block(M, C, N, R, L, torch.float16, 11)
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    Wq = torch.randint(-127, 128, (N, C), generator=g, device="cuda", dtype=torch.int8)
    Wv, meta = spg.sparse_compress_24(Wq)
    scale = torch.full((N,), 2.0 ** -18, device="cuda")
    Yq, Hq = spg.layernorm_s8(p["x"], p["gamma"], p["beta"], 32.0, residual=p["res"])
    Y, H, _, _ = spg.layernorm(p["x"], p["gamma"], p["beta"], residual=p["res"])
    assert torch.equal(H, Hq)
    y, _, _, tol = _ref_fwd(H, p["gamma"], p["beta"], 1e-5)
    want = (y * 32).clamp(-127, 127)
    assert torch.all((Yq.double() - want).abs() <= 0.5 + 32 * tol + E_LN * want.abs())
    base = spg.spgemm_24_s8(Yq, Wv, meta, scale=scale)
    acc = spg.spgemm_24_s8(Yq, Wv, meta, out_mode=spg.SPG_OUT_S32)
    assert torch.equal(base, (acc.float() * scale).half())
    plan = spg.lora_plan(p["index"], L)
    out, V = spg.lora_f16(Y, p["A"], p["B"], plan, scale=p["scale"], base=base)
    _check_forward(dict(p, X=Y, base=base), out, V)


def test_wide_layers():
    """Layers and batches whose blocks take several tiles of columns, with a ragged last one, in place."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    for M, N, K, R, L, order in ((8200, 14001, 264, 72, 3, "mixed"), (8200, 264, 14008, 48, 3, "runs")):
        p = _problem(M, N, K, R, L, torch.bfloat16, none=0.1, order=order, seed=13)
        plan = spg.lora_plan(p["index"], L)
        Y, V = spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"], base=p["base"])
        _check_forward(p, Y, V)
        buf = torch.empty_strided(p["base"].shape, p["base"].stride(), dtype=torch.bfloat16, device="cuda")
        buf.copy_(p["base"])
        spg.lora_f16(p["X"], p["A"], p["B"], plan, scale=p["scale"], base=buf, Y=buf)
        assert torch.equal(buf, Y)
        del Y, buf
        dX, dA, dB = spg.lora_f16_bwd(p["dY"], p["X"], V, p["A"], p["B"], plan, scale=p["scale"], dbase=p["dbase"])
        _check_backward(p, V, dX, dA, dB)
    assert spg.check_device_error() == 0


@pytest.mark.parametrize("C,dt", [(1001, "f16"), (2049, "bf16"), (4097, "bf16"), (8191, "f16"), (3001, "f32"),
                                  (16383, "bf16"), (12345, "f32"), (770, "f32"), (15, "f16")])
@pytest.mark.parametrize("residual", [False, True])
def test_padded_odd_rows(C, dt, residual):
    """Rows of any length padded to 16 bytes, the padding NaN: read in vectors, its content without effect, and
    the padding of the outputs as it was."""
    need_gpu()
    import torch
    import structured_sparse_gemm_02_b200 as spg
    dt = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dt]
    M, step = 203, 16 // dt.itemsize
    ld = (C + step - 1) // step * step
    g = torch.Generator(device="cuda")
    g.manual_seed(C)

    def mat(std, data=True):
        buf = torch.full((M, ld), float("nan"), dtype=dt, device="cuda")
        if data:
            buf[:, :C] = (torch.randn(M, C, generator=g, device="cuda") * std).to(dt)
        return buf
    x, dy, dh, out, hh = mat(1.5), mat(0.3), mat(0.3), mat(0, False), mat(0, False)
    gamma = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(dt)
    beta = (0.2 * torch.randn(C, generator=g, device="cuda")).to(dt)
    res = dh[:, :C] if residual else None
    Y, H, mean, rstd = spg.layernorm(x[:, :C], gamma, beta, 1e-5, residual=res, H=hh[:, :C] if residual else None,
                                     Y=out[:, :C], stats=True)
    h = (x[:, :C].float() + dh[:, :C].float()).to(dt) if residual else x[:, :C]
    y, _, _, tol = _ref_fwd(h, gamma, beta, 1e-5)
    assert torch.all((Y.double() - y).abs() <= tol + _half(y, dt)) and out[:, C:].isnan().all()
    if residual:
        assert torch.equal(H, h) and hh[:, C:].isnan().all()
    hx = hh[:, :C] if residual else x[:, :C]
    dx, dga, dbe = spg.layernorm_bwd(dy[:, :C], hx, mean, rstd, gamma, dH=res, dX=out[:, :C])
    want, tol, rg, sg, rb, sb = _ref_bwd(dy[:, :C], hx, mean, rstd, gamma, res)
    assert torch.all((dx.double() - want).abs() <= tol + _half(want, dt)) and out[:, C:].isnan().all()
    assert torch.all((dga.double() - rg).abs() <= 2.0 ** -16 * sg + _half(rg, dt))
    assert torch.all((dbe.double() - rb).abs() <= 2.0 ** -16 * sb + _half(rb, dt))
