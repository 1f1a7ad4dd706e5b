"""The scratch sizes of the gated delta rule are the documented ones: whole
chunks of 64 steps, however few of them a call has."""
import pytest

import rwkv_wkv_mixing_b200 as wkv


def up(x, a):
    return -(-x // a) * a


@pytest.mark.parametrize("B,HV", [(1, 4), (2, 74), (3, 50)])
@pytest.mark.parametrize("DK,DV", [(64, 64), (128, 64), (8, 16), (72, 104), (96, 128), (33, 64), (64, 60)])
@pytest.mark.parametrize("T", [1, 2, 32, 33, 56, 57, 64, 65, 333, 4096])
def test_forward(B, HV, DK, DV, T):
    chunks = B * HV * up(T, 64) // 64
    first = 33 if B * HV <= 148 or DV > 64 else 57
    for state, per in ((0, 33792), (1, 41984)):
        want = chunks * per if T >= first and DK % 8 == 0 and DV % 8 == 0 else 0
        assert wkv.lib.gated_delta_scratch(B, T, HV, DK, DV, 2, state) == want
        assert wkv.lib.gated_delta_scratch(B, T, HV, DK, DV, 4, state) == 0


@pytest.mark.parametrize("DK,DV", [(64, 64), (128, 64), (8, 16), (72, 104), (96, 128), (33, 64), (64, 60), (1, 1)])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 333])
def test_backward(DK, DV, T):
    for B, HV in ((1, 1), (2, 6)):
        chunks = B * HV * up(T, 64) // 64
        for es in (2, 4):
            want = chunks * 8 * up(DV, 16) * (DK + 64)
            if es == 2 and DK % 8 == 0 and DV % 8 == 0:
                want += chunks * (100352 if DK <= 64 else 124928)
            else:
                want += B * HV * T * 8 * DK
            assert 0 <= wkv.lib.gated_delta_backward_scratch(B, T, HV, DK, DV, es) - want <= 1024
