"""The entry points around the channel-wise mixer (scalar-gate rule, layer norm, gradients of the norm and
of the short convolution) on the host: bad arguments are refused before CUDA is touched, sizes of
workspaces, the binding's own checks.  No GPU needed."""
import ctypes

import pytest
import torch

import gated_delta_rule_95_b200 as g

P = ctypes.c_void_p
A = P(0x10000)   # aligned, never dereferenced
M = P(0x10008)   # not on 16 bytes
Q = P(0x10002)   # not on 4 bytes
OUT, OUT2, WS = P(0x20000), P(0x30000), P(0x40000)
OK, NULL, SHAPE, DTYPE, ALIGN = 0, 1, 2, 3, 4


def gdr(q=A, k=A, v=A, ga=A, be=A, cu=None, S0=None, o=OUT, ST=None, B=2, T=100, Hk=2, Hv=4, dk=128, dv=64, scale=1.0, dt=1,
        ws=WS, wsb=1 << 30):
    return g.lib().gdn2_gdr_chunk_fwd(q, k, v, ga, be, cu, S0, o, ST, B, T, Hk, Hv, dk, dv, scale, dt, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dk=96), SHAPE), (dict(dv=32), SHAPE), (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(Hk=-1), SHAPE),
    (dict(Hk=3), SHAPE), (dict(Hk=8), SHAPE), (dict(Hk=0), SHAPE), (dict(Hv=0), SHAPE), (dict(Hv=-4), SHAPE),
    (dict(B=1 << 30, Hv=4), SHAPE), (dict(B=1 << 30, cu=A), SHAPE), (dict(T=2 ** 31 - 1), SHAPE),
    (dict(dt=2), DTYPE), (dict(dt=-1), DTYPE),
    *[({n: None}, NULL) for n in ("q", "k", "v", "ga", "be", "o", "ws")],
    *[({n: M}, ALIGN) for n in ("q", "k", "v", "S0", "o", "ST", "ws")],
    *[({n: Q}, ALIGN) for n in ("ga", "be", "cu")],
    (dict(o=A), SHAPE), (dict(wsb=0), SHAPE), (dict(wsb=2 * 2 * 4 * 16 * 1024 - 1), SHAPE),
    (dict(B=0), OK), (dict(Hk=0, Hv=0), OK), (dict(B=0, q=None, ws=None, wsb=0), OK),
])
def test_gdr_chunk_validation(kw, status):
    assert gdr(**kw) == status


def step(q=A, k=A, v=A, ga=A, be=A, S=A, So=A, o=OUT, B=3, Hk=2, Hv=4, dk=64, dv=128, scale=1.0, dt=0):
    return g.lib().gdn2_gdr_decode_step(q, k, v, ga, be, S, So, o, B, Hk, Hv, dk, dv, scale, dt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dk=32), SHAPE), (dict(dv=256), SHAPE), (dict(B=-1), SHAPE), (dict(Hk=3), SHAPE), (dict(Hk=0), SHAPE),
    (dict(B=1 << 30), SHAPE), (dict(dt=3), DTYPE),
    *[({n: None}, NULL) for n in ("q", "k", "v", "ga", "be", "S", "So", "o")],
    *[({n: M}, ALIGN) for n in ("q", "k", "v", "S", "So", "o")],
    *[({n: Q}, ALIGN) for n in ("ga", "be")],
    (dict(o=A), SHAPE), (dict(B=0), OK), (dict(Hk=0, Hv=0), OK),
])
def test_gdr_decode_validation(kw, status):
    assert step(**kw) == status


def norm(x=A, r=None, w=A, b=None, y=OUT, s=None, mean=None, rstd=None, rows=5, cols=64, eps=1e-5, dt=1):
    return g.lib().gdn2_layer_norm_fwd(x, r, w, b, y, s, mean, rstd, rows, cols, eps, dt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(cols=(1 << 24) + 1), SHAPE), (dict(rows=2 ** 31 - 1), SHAPE),
    (dict(rows=1 << 30, cols=1 << 17), SHAPE), (dict(eps=-1e-5), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(dt=2), DTYPE),
    *[({n: None}, NULL) for n in ("x", "w", "y")],
    *[({n: M}, ALIGN) for n in ("x", "r", "w", "b", "y", "s")],
    *[({n: Q}, ALIGN) for n in ("mean", "rstd")],
    (dict(y=A), SHAPE), (dict(r=OUT), SHAPE), (dict(s=OUT), SHAPE),
    (dict(rows=0), OK), (dict(cols=0), OK),
])
def test_layer_norm_validation(kw, status):
    assert norm(**kw) == status


def norm_bwd(dy=A, s=A, w=A, mean=A, rstd=A, ds=None, dx=OUT, dw=OUT2, db=None, rows=5, cols=64, dt=1, ws=WS, wsb=1 << 30):
    return g.lib().gdn2_layer_norm_bwd(dy, s, w, mean, rstd, ds, dx, dw, db, rows, cols, dt, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(cols=(1 << 24) + 1), SHAPE), (dict(dt=2), DTYPE),
    *[({n: None}, NULL) for n in ("dy", "s", "w", "mean", "rstd", "dx", "dw", "ws")],
    *[({n: M}, ALIGN) for n in ("dy", "s", "w", "ds", "dx", "dw", "db", "ws")],
    *[({n: Q}, ALIGN) for n in ("mean", "rstd")],
    (dict(dx=A), SHAPE), (dict(ds=OUT), SHAPE), (dict(wsb=16), SHAPE), (dict(cols=0), OK),
])
def test_layer_norm_bwd_validation(kw, status):
    assert norm_bwd(**kw) == status


def conv_bwd(dy=A, x=A, w=A, cu=None, hist=None, dho=None, dx=OUT, dw=OUT2, db=None, dh=None, B=2, T=10, C=64, dt=1, ws=WS,
             wsb=1 << 30):
    return g.lib().gdn2_short_conv_bwd(dy, x, w, cu, hist, dho, dx, dw, db, dh, B, T, C, dt, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(C=60), SHAPE), (dict(C=-8), SHAPE), (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(C=(1 << 24) + 8), SHAPE),
    (dict(B=1 << 16, T=1 << 16), SHAPE), (dict(dt=4), DTYPE),
    *[({n: None}, NULL) for n in ("dy", "x", "w", "dx", "dw", "ws")],
    *[({n: M}, ALIGN) for n in ("dy", "x", "w", "hist", "dho", "dx", "dw", "db", "dh", "ws")],
    (dict(cu=Q), ALIGN), (dict(dx=A), SHAPE), (dict(wsb=16), SHAPE), (dict(C=0), OK),
])
def test_short_conv_bwd_validation(kw, status):
    assert conv_bwd(**kw) == status


def test_workspace_sizes():
    L = g.lib()
    f = L.gdn2_gdr_chunk_fwd_workspace_bytes
    rec = 16 * 1024
    assert f(2, 100, 4, 128, 64, 0, 1) == 2 * 2 * 4 * rec       # two chunks a sequence
    assert f(3, 100, 4, 128, 64, 1, 1) == (100 // 64 + 3) * 4 * rec
    assert f(8, 4096, 16, 128, 128, 0, 1) == 8 * 64 * 16 * rec  # 128 units: whole sequences
    segs = (f(1, 65536, 16, 128, 128, 0, 1) - 1024 * 16 * rec) / (16 * 128 * 128 * 4)
    assert segs > 0 and (segs + 3) % 3 == 0                     # 2 P - 3 and P states a unit
    assert f(1, 65536, 16, 128, 64, 0, 1) == 1024 * 16 * rec    # (a transition is d_k x d_k: only square states are split)
    for bad in ((2, 100, 4, 96, 64, 0, 1), (-1, 100, 4, 64, 64, 0, 1), (2, -1, 4, 64, 64, 0, 1), (2, 100, 4, 64, 64, 0, 0),
                (2, 100, 4, 64, 64, 0, 7), (0, 100, 4, 64, 64, 0, 1), (1, 0, 4, 64, 64, 0, 1), (1, 1, 0, 64, 64, 0, 1)):
        assert f(*bad) == 0
    assert L.gdn2_layer_norm_bwd_workspace_bytes(-1, 8) == 0 and L.gdn2_layer_norm_bwd_workspace_bytes(1, 1 << 25) == 0
    assert L.gdn2_short_conv_bwd_workspace_bytes(-1, 8) == 0 and L.gdn2_short_conv_bwd_workspace_bytes(1, 12) == 0
    # partial sums of as many blocks as there is work for: at least a row of them, and they stop growing
    assert L.gdn2_layer_norm_bwd_workspace_bytes(1, 64) >= 64 * 4 * 2
    assert L.gdn2_layer_norm_bwd_workspace_bytes(1 << 20, 64) == L.gdn2_layer_norm_bwd_workspace_bytes(1 << 21, 64)
    assert L.gdn2_short_conv_bwd_workspace_bytes(1, 64) >= 64 * 4 * 5


def test_entry_points_are_public():
    for n in ("gdn2_gdr_chunk_fwd", "gdn2_gdr_decode_step", "gdn2_layer_norm_fwd", "gdn2_layer_norm_bwd", "gdn2_short_conv_bwd"):
        assert n in g.__all__ and getattr(g, n).__doc__


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(2, 10, 64)
    w, c, s = torch.zeros(64), torch.zeros(64, 4), torch.zeros(2, 10)
    q, v, b = torch.zeros(2, 10, 2, 64), torch.zeros(2, 10, 4, 64), torch.zeros(2, 10, 4)
    S = torch.zeros(2, 4, 64, 64)
    calls = [lambda: g.gdn2_layer_norm_fwd(x, w), lambda: g.gdn2_layer_norm_bwd(x, x, w, s, s), lambda: g.gdn2_short_conv_bwd(x, x, c),
             lambda: g.gdn2_gdr_chunk_fwd(q, q, v, b, b), lambda: g.gdn2_gdr_decode_step(q[:, 0], q[:, 0], v[:, 0], b[:, 0], b[:, 0], S),
             # numbers of axes and types are looked at first
             lambda: g.gdn2_gdr_chunk_fwd(q, q, v[0], b, b), lambda: g.gdn2_gdr_chunk_fwd(q[0], q, v, b, b),
             lambda: g.gdn2_gdr_decode_step(q, q, v, b, b, S), lambda: g.gdn2_short_conv_bwd(x[0], x[0], c),
             lambda: g.gdn2_layer_norm_fwd(x.double(), w), lambda: g.gdn2_layer_norm_fwd(torch.zeros(()), w),
             lambda: g.gdn2_layer_norm_fwd(torch.zeros(3, 0), w)]
    for call in calls:
        with pytest.raises(ValueError, match="gdn2_"):
            call()
