"""Layer norm and low-rank adapters: what is refused, before anything is launched (CPU only).

The C entry points check sizes, pitches, pointers and alignment on the host;
the binding checks dtypes, shapes, layouts, devices and overlapping outputs.
The launching entry points are replaced by a recorder for the latter, as in
the other binding tests."""
import inspect

import pytest
import torch

import structured_sparse_gemm_02_b200 as spg

HOST_ONLY = {"lora_plan_size", "lora_bwd_workspace_size", "layernorm_bwd_workspace_size"}
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3


class Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name in HOST_ONLY:
            return getattr(self.real, name)

        def f(*args):
            self.calls.append((name, args))
            return 0
        return f


@pytest.fixture
def rec(monkeypatch):
    r = Recorder(spg.lib())
    monkeypatch.setattr(spg, "_lib", r)
    monkeypatch.setattr(spg, "_on_device", lambda t, name: None)
    monkeypatch.setattr(spg, "_stream", lambda s: 0)
    return r


def _f(*shape, dt=torch.float16):
    return torch.zeros(shape, dtype=dt)


# ---- the C entry points -----------------------------------------------------------------

def _ln(**k):
    a = dict(X=16, ldx=64, res=None, ldres=0, H=None, ldh=0, gamma=16, beta=16, eps=1e-5, Y=16, ldy=64, mean=None,
             rstd=None, M=4, C=64, dtype=0, wdtype=0, stream=None)
    assert set(k) <= set(a)
    return spg.lib().layernorm(*{**a, **k}.values())


def _ln8(**k):
    a = dict(X=16, ldx=64, res=None, ldres=0, H=None, ldh=0, gamma=16, beta=16, eps=1e-5, qscale=30.0, Y=16, ldy=64,
             M=4, C=64, dtype=0, wdtype=0, stream=None)
    assert set(k) <= set(a)
    return spg.lib().layernorm_s8(*{**a, **k}.values())


def _lnb(**k):
    a = dict(dY=16, lddy=64, X=16, ldx=64, mean=16, rstd=16, gamma=16, dH=None, lddh=0, dX=16, lddx=64, dgamma=16,
             dbeta=16, ws=16, ws_bytes=1 << 30, M=4, C=64, dtype=0, wdtype=0, stream=None)
    assert set(k) <= set(a)
    return spg.lib().layernorm_bwd(*{**a, **k}.values())


@pytest.mark.parametrize("f", [_ln, _ln8, _lnb])
def test_norm_argument_errors(f):
    nan, inf = float("nan"), float("inf")
    for k, want in [(dict(C=0), INVALID), (dict(M=-1), INVALID), (dict(ldx=63), INVALID), (dict(X=None), INVALID),
                    (dict(gamma=None), INVALID), (dict(dtype=2), INVALID), (dict(dtype=9), INVALID),
                    (dict(wdtype=1), INVALID), (dict(C=16385, ldx=20000), None), (dict(M=1 << 31), SHAPE),
                    (dict(X=17), MISALIGNED), (dict(gamma=17), MISALIGNED), (dict(gamma=18, wdtype=3), MISALIGNED),
                    (dict(X=18, dtype=3, wdtype=3), MISALIGNED)]:
        if want is None:  # every pitch has to hold the row before the size is looked at
            k, want = {**k, **({"ldy": 20000} if f is not _lnb else {"lddy": 20000, "lddx": 20000})}, SHAPE
        assert f(**k) == want, k
    if f is not _lnb:
        assert f(ldy=63) == INVALID and f(Y=None) == INVALID
        assert f(eps=-1.0) == INVALID and f(eps=nan) == INVALID and f(eps=inf) == INVALID
        assert f(res=16, ldres=64) == INVALID          # a residual without a place for the sum
        assert f(H=16, ldh=64) == INVALID              # and the other way round
        assert f(res=16, ldres=63, H=16, ldh=64) == INVALID and f(res=16, ldres=64, H=16, ldh=63) == INVALID
        assert f(beta=17) == MISALIGNED and f(res=17, ldres=64, H=16, ldh=64) == MISALIGNED
        assert f(M=0, X=None, Y=None) == OK
    else:
        assert f(mean=None) == INVALID and f(dgamma=None) == INVALID and f(lddy=63) == INVALID
        assert f(lddx=63) == INVALID and f(dH=16, lddh=63) == INVALID and f(ws_bytes=63) == INVALID
        assert f(ws=None) == INVALID and f(ws=24) == MISALIGNED and f(mean=18) == MISALIGNED
    if f is _ln:
        assert f(mean=18) == MISALIGNED
    if f is _ln8:
        for q in (0.0, -1.0, nan, inf):
            assert f(qscale=q) == INVALID


def test_norm_in_place_errors():
    """In place means the same rows: another pitch, two outputs in one place or codes over their input are refused."""
    two = dict(res=4096, ldres=64, H=8192, ldh=64)
    assert _ln(ldy=72) == INVALID                                        # Y is X
    assert _ln(Y=4096, **{**two, "ldres": 72}) == INVALID                # Y is res
    assert _ln(Y=12288, **{**two, "H": 16, "ldh": 72}) == INVALID        # H is X
    assert _ln(Y=12288, **{**two, "H": 4096, "ldh": 72}) == INVALID      # H is res
    assert _ln(Y=8192, **two) == INVALID and _ln8(Y=8192, **two) == INVALID  # Y is H
    assert _ln8() == INVALID and _ln8(Y=4096, **two) == INVALID          # codes over X, over res
    assert _lnb(lddx=72) == INVALID                                      # dX is dY
    assert _lnb(dY=4096, dH=16, lddh=72) == INVALID                      # dX is dH
    assert _ln(M=0, ldy=72) == OK                                        # nothing is written


def test_norm_workspace_size():
    size = spg.lib().layernorm_bwd_workspace_size
    assert size(0, 64, 0) == 0 and size(5, 0, 0) == 0 and size(5, 16385, 0) == 0 and size(5, 64, 2) == 0
    assert size(1, 4096, 1) == 2 * 4096 * 4                       # one block, one row of partial sums
    assert size(1 << 20, 16384, 3) <= 148 * 8 * 2 * 16384 * 4


def _lora(**k):
    a = dict(X=16, ldx=64, A=16, B=16, scale=None, plan=16, V=16, ldv=8, base=None, ldbase=0, Y=16, ldy=104, M=4, N=100,
             K=64, R=8, L=2, dtype=0, stream=None)
    assert set(k) <= set(a)
    return spg.lib().lora_f16(*{**a, **k}.values())


def _lorab(**k):
    a = dict(dY=16, lddy=104, X=16, ldx=64, V=16, ldv=8, A=16, B=16, scale=None, plan=16, dbase=None, lddbase=0, dX=16,
             lddx=64, dA=16, dB=16, ws=16, ws_bytes=1 << 20, M=4, N=100, K=64, R=8, L=2, dtype=0, stream=None)
    assert set(k) <= set(a)
    return spg.lib().lora_f16_bwd(*{**a, **k}.values())


@pytest.mark.parametrize("f", [_lora, _lorab])
def test_lora_argument_errors(f):
    big = 1 << 31
    for k, want in [(dict(dtype=2), INVALID), (dict(dtype=3), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID),
                    (dict(K=0), INVALID), (dict(R=0), INVALID), (dict(L=0), INVALID), (dict(ldx=63), INVALID),
                    (dict(ldv=7), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(X=None), INVALID),
                    (dict(V=None), INVALID), (dict(plan=None), INVALID), (dict(K=60), SHAPE), (dict(R=4, ldv=8), SHAPE),
                    (dict(R=136, ldv=136), SHAPE), (dict(L=8193), SHAPE), (dict(M=1 << 22), SHAPE),
                    (dict(K=big, ldx=big), SHAPE), (dict(X=24), MISALIGNED), (dict(ldx=68), MISALIGNED),
                    (dict(V=24), MISALIGNED), (dict(ldv=12), MISALIGNED), (dict(A=24), MISALIGNED),
                    (dict(B=24), MISALIGNED), (dict(scale=18), MISALIGNED), (dict(plan=24), MISALIGNED)]:
        assert f(**k) == want, k
    if f is _lora:
        assert f(ldy=99) == INVALID and f(Y=None) == INVALID and f(base=32, ldbase=99) == INVALID
        assert f(base=16, ldbase=112) == INVALID       # in place with another pitch
        assert f(Y=24) == MISALIGNED and f(ldy=100) == MISALIGNED and f(base=24, ldbase=104) == MISALIGNED
        assert f(M=0, X=None, V=None, Y=None, plan=None) == OK
    else:
        assert f(lddy=99) == INVALID and f(dA=None) == INVALID and f(dB=None) == INVALID and f(lddx=63) == INVALID
        assert f(dbase=16, lddbase=72) == INVALID and f(dbase=32, lddbase=63) == INVALID
        assert f(dY=None) == INVALID and f(ws=None) == INVALID and f(ws_bytes=1) == INVALID
        assert f(dA=24) == MISALIGNED and f(dB=24) == MISALIGNED and f(dY=24) == MISALIGNED
        assert f(lddx=68) == MISALIGNED and f(dbase=24, lddbase=64) == MISALIGNED and f(ws=24) == MISALIGNED


def test_lora_pitch_limits():
    big = 1 << 31
    for k in (dict(ldx=big), dict(ldv=big), dict(ldy=big), dict(base=32, ldbase=big), dict(N=big - 256, ldy=big - 8)):
        assert _lora(**k) == SHAPE, k
    for k in (dict(ldx=big), dict(ldv=big), dict(lddy=big), dict(lddx=big), dict(dbase=32, lddbase=big)):
        assert _lorab(**k) == SHAPE, k
    assert _lorab(dX=None, lddx=big, dY=None) == INVALID  # a pitch that is not used; the call fails for its dY


def test_lora_plan_errors_and_sizes():
    L = spg.lib()
    assert L.lora_plan_size(-1, 2) == 0 and L.lora_plan_size(4, 0) == 0 and L.lora_plan_size(4, 8193) == 0
    assert L.lora_plan_size(1 << 22, 2) == 0
    # header, group starts, rows and at most M / 128 + (L + 1) tiles of four words
    assert L.lora_plan_size(300, 5) == 4 * (4 + 8 + 300 + 4 * (2 + 6))
    need = L.lora_plan_size(300, 5)
    assert L.lora_plan(16, -1, 5, 16, need, None) == INVALID and L.lora_plan(16, 300, 0, 16, need, None) == INVALID
    assert L.lora_plan(None, 300, 5, 16, need, None) == INVALID and L.lora_plan(16, 300, 5, None, need, None) == INVALID
    assert L.lora_plan(16, 300, 5, 16, need - 1, None) == INVALID
    assert L.lora_plan(16, 300, 8193, 16, 1 << 30, None) == SHAPE
    assert L.lora_plan(16, 1 << 22, 5, None, 0, None) == SHAPE  # as the binding calls it: no size, no plan
    assert L.lora_plan(18, 300, 5, 16, need, None) == MISALIGNED and L.lora_plan(16, 300, 5, 24, need, None) == MISALIGNED
    assert L.lora_bwd_workspace_size(300, 64, 64, 8, 5) >= 300 * 8 * 2 and L.lora_bwd_workspace_size(0, 64, 64, 8, 5) == 0


# ---- the binding --------------------------------------------------------------------------

def _names(fn, args):
    """The recorded arguments under the C declaration's order, as the tests above name them."""
    helper = {"layernorm": _ln, "layernorm_s8": _ln8, "layernorm_bwd": _lnb, "lora_f16": _lora, "lora_f16_bwd": _lorab}
    src = inspect.getsource(helper[fn])
    keys = [p.split("=")[0].strip() for p in src[src.index("dict(") + 5:src.index("stream=None)")].replace("\n", " ").split(",")]
    return dict(zip([k for k in keys if k] + ["stream"], args))


def test_norm_calls_reach_the_library(rec):
    M, C = 6, 40
    X, g = _f(M, C + 8)[:, :C], torch.ones(C)
    Y, H, mean, rstd = spg.layernorm(X, g)
    assert H is None and mean is None and rstd is None and Y.shape == (M, C)
    a = _names(*rec.calls[-1])
    assert a["ldx"] == C + 8 and a["wdtype"] == spg.SPG_F32 and a["dtype"] == spg.SPG_F16 and a["beta"] is None
    Y, H, mean, rstd = spg.layernorm(X, g.half(), g.half(), residual=_f(M, C), stats=True)
    assert H.shape == (M, C) and mean.shape == (M,) and mean.dtype == torch.float32
    Y, H = spg.layernorm_s8(X, g, None, 31.5)
    assert Y.dtype == torch.int8 and H is None and _names(*rec.calls[-1])["qscale"] == 31.5
    odd = spg.layernorm(_f(M, 13), g[:13])[0]
    assert odd.stride(0) == 16                                     # rows padded to 16 bytes
    assert _names("layernorm", rec.calls[-1][1])["ldy"] == 16
    dX, dga, dbe = spg.layernorm_bwd(_f(M, C), X, mean, rstd, g, dH=_f(M, C))
    assert dX.dtype == torch.float16 and dga.dtype == torch.float32 and dbe.shape == (C,)
    # one row, whatever its stride: the pitch only has to hold it
    spg.layernorm(_f(C, 1).t(), g)
    assert _names("layernorm", rec.calls[-1][1])["ldx"] >= C
    assert spg.layernorm(_f(0, C), g, residual=_f(0, C), stats=True)[0].shape == (0, C)


@pytest.mark.parametrize("call", [
    lambda X, g: spg.layernorm(X.t(), g[:4]),                               # columns are not contiguous
    lambda X, g: spg.layernorm(X[0], g),                                    # 1-D
    lambda X, g: spg.layernorm(X.double(), g),
    lambda X, g: spg.layernorm(X, g[:-1]),
    lambda X, g: spg.layernorm(X, g.bfloat16()),                            # neither X's dtype nor fp32
    lambda X, g: spg.layernorm(X, torch.ones(80)[::2]),                     # a weight with a stride
    lambda X, g: spg.layernorm(X, None),
    lambda X, g: spg.layernorm(X, g, g.half()),                             # beta in another dtype than gamma
    lambda X, g: spg.layernorm(X, g, residual=X.bfloat16()),
    lambda X, g: spg.layernorm(X, g, residual=X[:2]),
    lambda X, g: spg.layernorm(X, g, H=X),                                  # a sum without a residual
    lambda X, g: spg.layernorm(X, g, Y=X.float()),
    lambda X, g: spg.layernorm(X, g, residual=X, H=X, Y=X),                 # two outputs in one place
    lambda X, g: spg.layernorm_s8(X, g, None, 1.0, Yq=X),
    lambda X, g: spg.layernorm_bwd(X, X, torch.zeros(3), torch.zeros(4), g),
    lambda X, g: spg.layernorm_bwd(X, X, torch.zeros(4), torch.zeros(4).double(), g),
    lambda X, g: spg.layernorm_bwd(X, X, torch.zeros(4), torch.zeros(4), g, dgamma=torch.zeros(40).half()),
    lambda X, g: spg.layernorm_bwd(X, X, torch.zeros(4), torch.zeros(4), g, dgamma=(z := torch.zeros(40)), dbeta=z),
    lambda X, g: spg.layernorm_bwd(X, X, torch.zeros(4), torch.zeros(4), g, workspace=torch.zeros(8, dtype=torch.uint8)),
])
def test_norm_refusals(rec, call):
    with pytest.raises((ValueError, TypeError)):
        call(_f(4, 40), torch.ones(40))
    assert not rec.calls


def _lora_args(M=6, N=20, K=16, R=8, L=3, dt=torch.bfloat16):
    return _f(M, K, dt=dt), _f(L, R, K, dt=dt), _f(L, N, R, dt=dt), spg.LoraPlan(torch.zeros(400, dtype=torch.int32), M, L)


def test_lora_calls_reach_the_library(rec):
    plan = spg.lora_plan(torch.zeros(6, dtype=torch.int32), 3)
    assert (plan.M, plan.L) == (6, 3) and plan.buf.numel() * 4 == spg.lib().lora_plan_size(6, 3)
    assert spg.lora_plan(torch.ones(6, dtype=torch.int32), 3, plan=plan) is plan
    X, A, B, plan = _lora_args()
    Y, V = spg.lora_f16(X, A, B, plan)
    assert Y.shape == (6, 20) and Y.stride(0) == 24 and V.shape == (6, 8)
    a = _names(*rec.calls[-1])
    assert a["base"] is None and a["scale"] is None and a["dtype"] == spg.SPG_BF16 and (a["N"], a["K"], a["R"]) == (20, 16, 8)
    base = _f(6, 24, dt=torch.bfloat16)[:, :20]
    assert spg.lora_f16(X, A, B, plan, scale=torch.ones(3), base=base, Y=base)[0] is base
    dX, dA, dB = spg.lora_f16_bwd(base, X, V, A, B, plan, dbase=X)
    assert dX.shape == X.shape and dA.shape == A.shape and dB.shape == B.shape
    assert spg.lora_f16_bwd(base, X, V, A, B, plan, need_dx=False)[0] is None
    assert _names(*rec.calls[-1])["dX"] is None


@pytest.mark.parametrize("call", [
    lambda X, A, B, p: spg.lora_plan(torch.zeros(6, dtype=torch.int64), 3),
    lambda X, A, B, p: spg.lora_plan(torch.zeros(6, 1, dtype=torch.int32), 3),
    lambda X, A, B, p: spg.lora_plan(torch.zeros(12, dtype=torch.int32)[::2], 3),
    lambda X, A, B, p: spg.lora_plan(torch.zeros(5, dtype=torch.int32), 3, plan=p),     # a plan for other rows
    lambda X, A, B, p: spg.lora_plan(torch.zeros(6, dtype=torch.int32), 2, plan=p),     # and for other adapters
    lambda X, A, B, p: spg.lora_f16(X, A, B, p.buf),
    lambda X, A, B, p: spg.lora_f16(X[:5], A, B, p),
    lambda X, A, B, p: spg.lora_f16(X.float(), A, B, p),
    lambda X, A, B, p: spg.lora_f16(X, A.half(), B, p),
    lambda X, A, B, p: spg.lora_f16(X, A[:2], B, p),
    lambda X, A, B, p: spg.lora_f16(X, A[:, :, :8], B, p),
    lambda X, A, B, p: spg.lora_f16(X, A.transpose(1, 2).contiguous().transpose(1, 2), B, p),
    lambda X, A, B, p: spg.lora_f16(X, A, B[:, ::2], p),
    lambda X, A, B, p: spg.lora_f16(X, A, B[:, :, :4], p),
    lambda X, A, B, p: spg.lora_f16(X, A[0], B[0], p),
    lambda X, A, B, p: spg.lora_f16(X, A, B, p, scale=torch.ones(2)),
    lambda X, A, B, p: spg.lora_f16(X, A, B, p, scale=torch.ones(3).double()),
    lambda X, A, B, p: spg.lora_f16(X, A, B, p, base=X),
    lambda X, A, B, p: spg.lora_f16(X, A, B, p, V=(b := torch.zeros(6, 32, dtype=X.dtype))[:, :8], Y=b[:, 8:28]),
    lambda X, A, B, p: spg.lora_f16_bwd(X, X, X[:, :8], A, B, p),
    lambda X, A, B, p: spg.lora_f16_bwd(_f(6, 20, dt=X.dtype), X, X, A, B, p),
    lambda X, A, B, p: spg.lora_f16_bwd(_f(6, 20, dt=X.dtype), X, _f(6, 8, dt=X.dtype), A, B, p, dA=A.float()),
    lambda X, A, B, p: spg.lora_f16_bwd(_f(6, 20, dt=X.dtype), X, _f(6, 8, dt=X.dtype), A, B, p, need_dx=False, dbase=X),
    lambda X, A, B, p: spg.lora_f16_bwd(_f(6, 20, dt=X.dtype), X, _f(6, 8, dt=X.dtype), A, B, p,
                                        workspace=torch.zeros(8, dtype=torch.uint8)),
])
def test_lora_refusals(rec, call):
    X, A, B, plan = _lora_args()
    with pytest.raises((ValueError, TypeError)):
        call(X, A, B, plan)
    assert not rec.calls


def test_host_tensors_are_refused():
    X, g = _f(4, 40), torch.ones(40)
    with pytest.raises(ValueError, match="CUDA"):
        spg.layernorm(X, g)
    with pytest.raises(ValueError, match="CUDA"):
        spg.lora_plan(torch.zeros(6, dtype=torch.int32), 3)
