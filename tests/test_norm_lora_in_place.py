"""Outputs over memory that the same call still reads are refused, before anything is launched (CPU only).

Every call below has an output in a place where it is not allowed, and otherwise valid arguments."""
import pytest

import structured_sparse_gemm_02_b200 as spg

INVALID = 1
M, N, K, R, L = 4, 64, 64, 64, 2  # square, so that every matrix of the adapters fits every other one's place


def _forward(**k):
    a = dict(X=1 << 20, ldx=64, A=2 << 20, B=3 << 20, scale=None, plan=4 << 20, V=5 << 20, ldv=64, base=6 << 20, ldbase=64,
             Y=7 << 20, ldy=64)
    for out, other in k.items():
        a[out] = a[other]
    return spg.lib().lora_f16(*a.values(), M, N, K, R, L, 0, None)


def _backward(**k):
    a = dict(dY=1 << 20, lddy=64, X=2 << 20, ldx=64, V=3 << 20, ldv=64, A=4 << 20, B=5 << 20, scale=None, plan=6 << 20,
             dbase=7 << 20, lddbase=64, dX=8 << 20, lddx=64, dA=9 << 20, dB=10 << 20, ws=11 << 20)
    for out, other in k.items():
        a[out] = a[other]
    return spg.lib().lora_f16_bwd(*a.values(), 1 << 20, M, N, K, R, L, 0, None)


@pytest.mark.parametrize("out,other", [("V", o) for o in ("X", "A", "B", "base", "Y")] + [("Y", "A"), ("Y", "B")])
def test_adapters_forward(out, other):
    assert _forward(**{out: other}) == INVALID


@pytest.mark.parametrize("out,other", [(o, i) for o in ("dA", "dB", "ws") for i in ("dY", "X", "V", "A", "B", "dbase", "dX")]
                         + [("dX", "A"), ("dX", "B"), ("dB", "dA"), ("ws", "dA"), ("ws", "dB")])
def test_adapters_backward(out, other):
    assert _backward(**{out: other}) == INVALID


@pytest.mark.parametrize("dX,pitch", [(1 << 20, 72), (2 << 20, 72), (3 << 20, 72)])
def test_norm_backward_in_place_with_another_pitch(dX, pitch):
    assert spg.lib().layernorm_bwd(1 << 20, 64, 2 << 20, 64, 4 << 20, 5 << 20, 6 << 20, 3 << 20, 64, dX, pitch, 7 << 20,
                                   8 << 20, 9 << 20, 1 << 20, 4, 64, 0, 0, None) == INVALID
