"""The backward of the short convolution on the GPU against fp64: fixed and packed batches
with empty and short sequences, carried history and its gradients, strips that end in and at
sequences, streams, captured graphs, bad offsets.

Tolerances, from the arithmetic (u = 2^-24): dx and dhist are at most five products and sums in
fp32 and one rounding to the type; dweight and dbias are sums over the tokens, at most 256 in
one chain, then the strips in chains of an eighth of them."""
import numpy as np
import pytest
import torch

import gated_delta_rule_95_b200 as g
from oracle import layer

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
GDN2_ERR_SHAPE = 2


def _f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def _draw(shape, seed, dtype=torch.float32, std=1.0):
    return torch.from_numpy((np.random.default_rng(seed).standard_normal(shape) * std).astype(np.float32)).to(dtype)


def _cuda(t):
    return None if t is None else t.cuda()


def _check(r, dy, x, w, hist, dho, spans, dtype):
    """Every sequence's [lo, hi) of the flat token axis."""
    C = x.shape[-1]
    dyf, xf, wf = _f64(dy).reshape(-1, C), _f64(x).reshape(-1, C), _f64(w)
    dx = _f64(r["dx"]).reshape(-1, C)
    dw, db, dwm, dbm = np.zeros((C, 4)), np.zeros(C), np.zeros((C, 4)), np.zeros(C)
    for n, (lo, hi) in enumerate(spans):
        h = None if hist is None else _f64(hist[n])
        d = None if dho is None else _f64(dho[n])
        a = layer.short_conv_backward(dyf[lo:hi], xf[lo:hi], wf, h, d)
        m = layer.short_conv_backward(*(None if t is None else np.abs(t) for t in (dyf[lo:hi], xf[lo:hi], wf, h, d)))
        for got, ref, mag in [(dx[lo:hi], a[0], m[0])] + ([(_f64(r["dhist"][n]), a[3], m[3])] if r["dhist"] is not None else []):
            bound = 6 * U * mag
            bound = bound + HALF[dtype] * (np.abs(ref) + bound) + 1e-38
            assert np.all(np.abs(got - ref) <= bound), n
        dw, db, dwm, dbm = dw + a[1], db + a[2], dwm + m[1], dbm + m[2]
    chain = 256 + len(dyf) / 16 / 8 + 16
    assert np.all(np.abs(_f64(r["dweight"]).reshape(C, 4) - dw) <= chain * U * dwm + 1e-38)
    if r["dbias"] is not None:
        assert np.all(np.abs(_f64(r["dbias"]) - db) <= chain * U * dbm + 1e-38)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,C,carried", [(1, 1, 8, False), (2, 2, 8, True), (3, 3, 16, True), (3, 37, 72, True),
                                           (2, 300, 520, False), (5, 64, 1032, True), (1, 1500, 40, True)])
def test_fixed_length(B, T, C, carried, dtype):
    dy, x, w = _draw((B, T, C), 1, dtype), _draw((B, T, C), 2, dtype), _draw((C, 4), 3, std=0.5)
    hist, dho = (_draw((B, 3, C), 4, dtype), _draw((B, 3, C), 5, dtype)) if carried else (None, None)
    r = g.gdn2_short_conv_bwd(dy.cuda(), x.cuda(), w.cuda(), hist=_cuda(hist), dhist_out=_cuda(dho))
    torch.cuda.synchronize()
    assert (r["dhist"] is not None) == carried
    _check(r, dy, x, w, hist, dho, [(n * T, (n + 1) * T) for n in range(B)], dtype)
    assert g.gdn2_device_status() == 0


LENGTHS = [[0, 1, 2, 5, 40, 0, 17, 3], [300, 0, 0, 1, 1, 700, 64, 8], [16] * 9, [5], [0, 0, 9, 0]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("hist_given,dho_given", [(True, True), (False, True), (True, False)])
def test_packed(lengths, hist_given, dho_given, dtype):
    T, C, N = sum(lengths), 24, len(lengths)
    dy, x, w = _draw((T, C), 6, dtype), _draw((T, C), 7, dtype), _draw((C, 1, 4), 8, std=0.5)
    hist = _draw((N, 3, C), 9, dtype) if hist_given else None
    dho = _draw((N, 3, C), 10, dtype) if dho_given else None
    at = np.concatenate([[0], np.cumsum(lengths)])
    cu = torch.tensor(at, dtype=torch.int32).cuda()
    r = g.gdn2_short_conv_bwd(dy.cuda(), x.cuda(), w.cuda(), cu_seqlens=cu, hist=_cuda(hist), dhist_out=_cuda(dho),
                              want_dbias=False, want_dhist=True)
    torch.cuda.synchronize()
    assert r["dbias"] is None and r["dweight"].shape == (C, 1, 4)
    _check(r, dy, x, w.reshape(C, 4), hist, dho, list(zip(at[:-1], at[1:])), dtype)
    assert g.gdn2_device_status() == 0


def test_no_tokens():
    w = _draw((16, 4), 11).cuda()
    x = torch.empty(2, 0, 16, device="cuda")
    dho = _draw((2, 3, 16), 12)
    r = g.gdn2_short_conv_bwd(x, x, w, dhist_out=dho.cuda(), want_dhist=True)
    assert torch.equal(r["dweight"].cpu(), torch.zeros(16, 4)) and torch.equal(r["dbias"].cpu(), torch.zeros(16))
    assert torch.equal(r["dhist"].cpu(), dho)


def test_against_differences():
    # the loss reads y and the history handed on; the gradient of every input by differences of
    # the forward's own fp64 oracle
    import oracle
    rng = np.random.default_rng(13)
    x, w, h, dy, dho = (rng.standard_normal(n) for n in ((5, 8), (8, 4), (3, 8), (5, 8), (3, 8)))

    def loss(x, w, h):
        y, hist = oracle.short_conv(x, w, None, h)
        return float((y * dy).sum() + (hist * dho).sum())

    dev = {n: torch.from_numpy(np.float32(t)).cuda() for n, t in dict(x=x, w=w, h=h, dy=dy, dho=dho).items()}
    r = g.gdn2_short_conv_bwd(dev["dy"][None], dev["x"][None], dev["w"], hist=dev["h"][None],
                              dhist_out=dev["dho"][None])
    got = dict(x=_f64(r["dx"][0]), w=_f64(r["dweight"]), h=_f64(r["dhist"][0]))
    step = 1e-5
    for i, name in enumerate(("x", "w", "h")):
        for at in [(0, 0), (1, 1), (2, 3)] + ([(4, 7)] if name == "x" else []):
            args = [x.copy(), w.copy(), h.copy()]
            args[i][at] += step
            up = loss(*args)
            args[i][at] -= 2 * step
            assert abs((up - loss(*args)) / (2 * step) - got[name][at]) < 1e-4, (name, at)


def test_offsets_out_of_order_are_reported():
    x = _draw((30, 16), 14, torch.bfloat16).cuda()
    w = _draw((16, 4), 15).cuda()
    for offsets in ([0, 20, 10, 30], [0, 10, 40], [-5, 10, 30], [0, 10, 29]):
        cu = torch.tensor(offsets, dtype=torch.int32).cuda()
        g.gdn2_short_conv_bwd(x, x, w, cu_seqlens=cu, want_dhist=True)
        assert g.gdn2_device_status() == GDN2_ERR_SHAPE, offsets
        assert g.gdn2_device_status() == 0


def test_other_stream_and_captured():
    dy, x, w = _draw((3, 200, 64), 16).cuda(), _draw((3, 200, 64), 17).cuda(), _draw((64, 4), 18).cuda()
    ref = g.gdn2_short_conv_bwd(dy, x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = g.gdn2_short_conv_bwd(dy, x, w, stream=side)
    side.synchronize()
    out = dict(dx=torch.zeros_like(x), dweight=torch.zeros_like(w), dbias=torch.zeros(64, device="cuda"), dhist=None)
    ws = torch.empty(g.lib().gdn2_short_conv_bwd_workspace_bytes(600, 64), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        g.gdn2_short_conv_bwd(dy, x, w, workspace=ws, out=out)
    graph.replay()
    torch.cuda.synchronize()
    for n in ("dx", "dweight", "dbias"):
        assert torch.equal(ref[n], other[n]) and torch.equal(ref[n], out[n]), n
