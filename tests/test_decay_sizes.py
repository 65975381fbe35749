"""Sizes at the limits of the decayed calls, without a GPU: what a call refuses, its workspace
query and its path query refuse too."""
import pytest

from kernelized_linear_attention_unit_b200 import binding as bd
from test_decay_abi import NO, _bwd, _copy, _decode, _fwd

MAX_BH, MAX_L = 65535 // 3, 64 * 65535


@pytest.mark.parametrize("dt", [bd.SLAY_F32, bd.SLAY_BF16])
@pytest.mark.parametrize("B,H,L", [(MAX_BH + 1, 1, 4), (2, 20000, 4), (1 << 20, 1 << 10, 1), (1, 1, MAX_L + 1), (MAX_BH + 1, 1, 0)])
def test_refused_sizes_have_no_workspace_and_no_path(dt, B, H, L):
    for op, call in ((bd.OP_DECAY_FWD, _fwd), (bd.OP_DECAY_BWD, _bwd)):
        assert call(B=B, H=H, L=L, dt=dt) == NO
        with pytest.raises(bd.SlayError):
            bd.slay_workspace_bytes(op, dt, B, H, L, 64, 64, 1, 64)
        with pytest.raises(bd.SlayError):
            bd.slay_path(op, dt, B, H, L, 64, 64, 1, 64)


@pytest.mark.parametrize("B,H,L", [(MAX_BH, 1, 4), (1, 1, MAX_L)])
def test_largest_sizes_are_taken(B, H, L):
    for op in (bd.OP_DECAY_FWD, bd.OP_DECAY_BWD):
        assert bd.slay_workspace_bytes(op, bd.SLAY_BF16, B, H, L, 64, 64, 1, 64) > 0
        assert bd.slay_path(op, bd.SLAY_BF16, B, H, L, 64, 64, 1, 64) == bd.PATH_TC_CONTRACTION


def test_pool_calls_refuse_beyond_their_limits():
    assert _decode(Bt=(1 << 27) + 1, H=1) == NO
    assert _decode(Bt=1 << 14, H=(1 << 13) + 1) == NO
    assert _copy(H=(1 << 18) + 1, F=64) == NO
    assert _copy(H=(1 << 14) + 1, F=1024) == NO
