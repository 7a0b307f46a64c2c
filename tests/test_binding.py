"""The ctypes binding on the host: sizes that the library's ints do not hold.  No GPU needed."""
import ctypes

import pytest
import torch

import gated_delta_rule_95_b200 as g

I, P = ctypes.c_int, ctypes.c_void_p


def _entry_points():
    """Every function of the library that takes tensors and sizes."""
    L = g.lib()
    return [n for n, f in vars(L).items() if n.startswith("gdn2_") and P in (f.argtypes or ()) and I in f.argtypes]


def test_every_entry_point_has_its_sizes():
    names = _entry_points()
    assert {"gdn2_chunk_fwd", "gdn2_chunk_fwd_csize", "gdn2_chunk_bwd", "gdn2_short_conv", "gdn2_short_conv_bwd", "gdn2_decode_step",
            "gdn2_layer_norm_fwd", "gdn2_layer_norm_bwd", "gdn2_gdr_chunk_fwd", "gdn2_gdr_decode_step"} <= set(names)
    for n in names:
        types = getattr(g.lib(), n).argtypes
        at = types.index(I)
        # the run after the pointers: at least two sizes (rows and columns) and none of another type
        assert all(t is P for t in types[:at]) and all(t is I for t in types[at:at + 2])


@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32 + 5, 2 ** 40])
@pytest.mark.parametrize("name", ["gdn2_chunk_fwd", "gdn2_chunk_bwd", "gdn2_short_conv", "gdn2_short_conv_bwd", "gdn2_decode_step",
                                  "gdn2_layer_norm_fwd", "gdn2_layer_norm_bwd", "gdn2_gdr_chunk_fwd", "gdn2_gdr_decode_step"])
def test_sizes_past_32_bits_are_refused(name, size):
    f = getattr(g.lib(), name)
    at, n = f.argtypes.index(I), 0
    while f.argtypes[at + n] is I:
        n += 1
    for i in range(n):
        args = [None] * at + [1] * n + [0] * (len(f.argtypes) - at - n - 1)
        args[at + i] = size
        for call in (lambda: g._call(name, torch.device("cuda", 0), *args), lambda: g._on(torch.device("cuda", 0), f, *args, None)):
            with pytest.raises(ValueError, match=name):
                call()
