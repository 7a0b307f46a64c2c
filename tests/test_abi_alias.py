"""Outputs of the layer's entry points that would be written over inputs still being read are refused on the
host, before CUDA is touched.  No GPU needed."""
import ctypes

import pytest

import gated_delta_rule_95_b200 as g

P = ctypes.c_void_p
SHAPE = 2
C = 64
W, FAR = 0x100000, 0x200000  # aligned, never dereferenced


@pytest.mark.parametrize("dweight,dbias", [
    (W, FAR), (W + 16, FAR), (W + 16 * C - 16, FAR), (W - 16 * C + 16, FAR), (W, None),
    (FAR, W), (FAR, W + 16), (FAR, W + 16 * C - 16), (FAR, W - 4 * C + 16)])
def test_the_taps_gradients_over_the_taps_beside_dhist(dweight, dbias):
    # (the history's gradient reads the taps while their gradient is written)
    assert g.lib().gdn2_short_conv_bwd(P(0x10000), P(0x20000), P(W), None, None, None, P(0x30000), P(dweight), P(dbias), P(0x50000), 2, 10, C, 1,
                                       P(0x40000), 1 << 30, None) == SHAPE


STATE = 4 * 64 * 128  # bytes of one


@pytest.mark.parametrize("shift", [16, STATE, 5 * STATE, 6 * STATE - 16, -16, -STATE, -6 * STATE + 16])
def test_states_shifted_over_the_entering_ones(shift):
    # 3 sequences of 2 value heads: some block's state would be written before another one has read it
    args = P(0x10000), P(0x20000), P(0x30000), P(0x40000), P(0x50000)
    assert g.lib().gdn2_gdr_chunk_fwd(*args, None, P(W), P(0x60000), P(W + shift), 3, 10, 1, 2, 64, 128, 1.0, 1, P(0x800000), 1 << 30, None) == SHAPE
    assert g.lib().gdn2_gdr_decode_step(*args, P(W), P(W + shift), P(0x60000), 3, 1, 2, 64, 128, 1.0, 1, None) == SHAPE
