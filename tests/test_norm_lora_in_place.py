"""Outputs over memory that the same call still reads are refused, before anything is launched (CPU only).

Every call below has an output in a place where it is not allowed, and otherwise valid arguments."""
import pytest

import structured_sparse_gemm_02_b200 as spg

INVALID = 1


@pytest.mark.parametrize("dX,pitch", [(1 << 20, 72), (2 << 20, 72), (3 << 20, 72)])
def test_norm_backward_in_place_with_another_pitch(dX, pitch):
    assert spg.lib().layernorm_bwd(1 << 20, 64, 2 << 20, 64, 4 << 20, 5 << 20, 6 << 20, 3 << 20, 64, dX, pitch, 7 << 20,
                                   8 << 20, 9 << 20, 1 << 20, 4, 64, 0, 0, None) == INVALID
