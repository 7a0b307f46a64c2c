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


X = 0x4000000  # a tensor of N bytes
N = 2 * 300 * 64 * 2  # [2, 300, 64] bf16
SHIFTS = [0, 16, 128, N - 16, -16, -N + 16]
A, B, D, E, F = (P(i << 28) for i in range(1, 6))  # apart from it and each other


@pytest.mark.parametrize("shift", SHIFTS)
def test_outputs_over_inputs(shift):
    L, x, y = g.lib(), P(X), P(X + shift)
    conv = lambda dy, xx, dx, **k: L.gdn2_short_conv_bwd(dy, xx, A, None, None, k.get("dho"), dx, B, None, k.get("dh"), 2, 300, 64, 1, D, 1 << 30, None)  # noqa: E731
    fwd = lambda xx, r, yy, s=None: L.gdn2_layer_norm_fwd(xx, r, A, B, yy, s, D, E, 600, 64, 1e-5, 1, None)  # noqa: E731
    bwd = lambda dy, s, ds, dx: L.gdn2_layer_norm_bwd(dy, s, A, B, D, ds, dx, E, None, 600, 64, 1, F, 1 << 27, None)  # noqa: E731
    chunk = lambda q, k, v, o: L.gdn2_gdr_chunk_fwd(q, k, v, A, B, None, None, o, None, 2, 300, 1, 1, 64, 64, 1.0, 1, D, 1 << 28, None)  # noqa: E731
    step = lambda q, k, v, o: L.gdn2_gdr_decode_step(q, k, v, A, B, D, E, o, 600, 1, 1, 64, 64, 1.0, 1, None)  # noqa: E731
    far = P(0x8000000)
    calls = [conv(x, far, y), conv(far, x, y), fwd(x, None, y), fwd(far, x, y), fwd(far, P(0xA000000), x, y), bwd(x, far, None, y),
             bwd(far, x, None, y), bwd(far, P(0xA000000), x, y)]
    calls += [f(*(x if i == j else P(0x8000000 + 0x100000 * j) for j in range(3)), y) for f in (chunk, step) for i in range(3)]
    if shift:  # in place is allowed
        calls += [fwd(x, None, far, y), fwd(far, x, P(0xA000000), y)]
    assert calls == [SHAPE] * len(calls)


@pytest.mark.parametrize("shift", [16, 3 * 64 * 2, -16, -3 * 64 * 2])
def test_the_history_gradient_shifted_over_the_one_handed_in(shift):
    assert g.lib().gdn2_short_conv_bwd(P(X), P(0x8000000), A, None, None, E, P(0xA000000), B, None, P(E.value + shift), 2, 300, 64, 1, D, 1 << 28,
                                       None) == SHAPE


@pytest.mark.parametrize("over", ["weight", "bias", "mean", "rstd"])
def test_a_norms_rows_over_its_vectors(over):
    at = {"weight": A, "bias": B, "mean": D, "rstd": E}
    L, y = g.lib(), P(at[over].value - 64)
    assert L.gdn2_layer_norm_fwd(P(X), None, A, B, y, None, D, E, 600, 64, 1e-5, 1, None) == SHAPE
    if over != "bias":
        assert L.gdn2_layer_norm_bwd(P(X), P(0x8000000), A, D, E, None, y, P(0xA000000), None, 600, 64, 1, F, 1 << 27, None) == SHAPE
