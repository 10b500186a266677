"""What the binding passes on for views whose strides say little: single rows and empty batches (CPU only)."""
import pytest
import torch

import structured_sparse_gemm_02_b200 as spg
from tests.test_norm_lora_checks import _f, _names, rec  # noqa: F401 (rec is a fixture)

C, R, L = 64, 16, 3


def _row(rows, dt=torch.float16):
    """A [rows, C] view, at most one row, whose first stride does not hold a row."""
    return torch.zeros(C, rows, dtype=dt).t()


@pytest.mark.parametrize("rows", [0, 1])
def test_pitches_of_new_outputs_hold_their_row(rec, rows):  # noqa: F811
    X, gamma = _row(rows), torch.ones(C)
    assert X.is_contiguous() and X.stride(0) < C
    Y, H, mean, rstd = spg.layernorm(X, gamma, residual=X, stats=True)
    a = _names(*rec.calls[-1])
    assert min(a["ldx"], a["ldres"], a["ldh"], a["ldy"]) >= C and Y.shape == H.shape == (rows, C)
    spg.layernorm_s8(X, gamma, None, 1.0, residual=X)
    a = _names(*rec.calls[-1])
    assert min(a["ldx"], a["ldres"], a["ldh"], a["ldy"]) >= C
    spg.layernorm_bwd(X, X, mean, rstd, gamma, dH=X)
    a = _names(*rec.calls[-1])
    assert min(a["lddy"], a["ldx"], a["lddh"], a["lddx"]) >= C
    A, B, plan = _f(L, R, C), _f(L, C, R), spg.LoraPlan(torch.zeros(400, dtype=torch.int32), rows, L)
    Y, V = spg.lora_f16(X, A, B, plan, base=X)
    a = _names(*rec.calls[-1])
    assert min(a["ldx"], a["ldbase"], a["ldy"]) >= C and a["ldv"] >= R
    spg.lora_f16_bwd(X, X, V, A, B, plan, dbase=X)
    a = _names(*rec.calls[-1])
    assert min(a["lddy"], a["ldx"], a["lddbase"], a["lddx"]) >= C and a["ldv"] >= R
