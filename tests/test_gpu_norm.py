"""Layer norm and its backward on the GPU against fp64: row widths held by part of a warp, a
warp, a block and none of these, odd and unaligned widths, one row and many, in-place residual
sums, constant and far-off rows, other streams, captured graphs.

Tolerances, from the arithmetic.  u = 2^-24.  A row's mean is a fp32 sum of n terms added in a
tree of depth at most 64 + 10 (64 values a thread at most, then 10 halvings), so it is off by at most
74 u mean|s| <= 74 u A with A = max |s| of the row; the deviations d = s - mu inherit that, so
xh = d rho is off by at most 75 u A rho + (74 + 4) u |xh| (the variance's own sum, rsqrt and the
products).  y adds the weight's product and the bias and one rounding to the output type (half
a step: 2^-8 relative for bf16, 2^-24 for fp32)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_95_b200 as g
from oracle import layer

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DEPTH = 74


def _f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def _draw(shape, seed, dtype=torch.float32, std=1.0, mean=0.0):
    x = np.random.default_rng(seed).standard_normal(shape) * std + mean
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def _within(got, ref, bound):
    err = np.abs(_f64(got) - ref)
    assert np.all(err <= bound), float(np.max(err / bound))


def _depth(cols):
    """Longest chain of a row's sum: the values of one thread, then the halvings."""
    return max(DEPTH, cols / 512 + 16)


def _check_fwd(x, r, w, b, out, eps, dtype):
    y, s, mean, rstd = out
    sf = _f64(x) if r is None else _f64((x.float() + r.float()).to(dtype))
    if r is not None:
        assert torch.equal(s.cpu(), (x.float() + r.float()).to(dtype))
    else:
        assert s is None
    y_ref, m_ref, r_ref = layer.layer_norm(sf, _f64(w), _f64(b), eps)
    n = _depth(x.shape[-1])
    A = np.abs(sf).max(-1)
    dm = n * U * A + 1e-38
    _within(mean, m_ref, dm)
    # the variance is off by its own sum and by the mean's square; rho by half of that
    dr = r_ref * ((n + 6) * U + 2 * (dm * r_ref) ** 2 + 2 * U * A * r_ref)
    _within(rstd, r_ref, dr)
    xh = np.abs(sf - m_ref[:, None]) * r_ref[:, None]
    wa = np.abs(_f64(w))
    bound = wa * (xh * (dr / r_ref + 4 * U)[:, None] + ((dm + U * A) * r_ref)[:, None]) * 1.01
    bound = bound + 2 * U * (xh * wa + (0 if b is None else np.abs(_f64(b))))
    _within(y, y_ref, bound + HALF[dtype] * (np.abs(y_ref) + bound) + 1e-38)


WIDTHS = [1, 2, 7, 8, 24, 33, 64, 100, 128, 250, 256, 257, 1000, 1001, 2048, 2056, 4099, 8192, 8200, 20000, 33000]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", WIDTHS)
def test_forward_widths(cols, dtype):
    rows = 37 if cols < 3000 else 5
    x, w, b = _draw((rows, cols), 1, dtype), _draw((cols,), 2, std=0.3, mean=1.0), _draw((cols,), 3)
    r = _draw((rows, cols), 4, dtype) if cols % 3 else None
    out = g.gdn2_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), None if r is None else r.cuda(), eps=1e-5)
    torch.cuda.synchronize()
    _check_fwd(x, r, w, b, out, 1e-5, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (3, 513), (129, 8), (4097, 40), (1000, 2048)])
def test_forward_rows_without_bias(rows, cols, dtype):
    x, w = _draw((rows, cols), 5, dtype), _draw((cols,), 6)
    out = g.gdn2_layer_norm_fwd(x.cuda(), w.cuda(), eps=1e-3)
    torch.cuda.synchronize()
    _check_fwd(x, None, w, None, out, 1e-3, dtype)


def test_forward_far_off_and_constant_rows():
    # a mean a thousand deviations away (two passes lose nothing), and rows without variance
    x = torch.cat([_draw((4, 640), 7, std=1.0, mean=1000.0), torch.full((3, 640), 2.5), torch.zeros(2, 640)])
    w, b = _draw((640,), 8), _draw((640,), 9)
    out = g.gdn2_layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=1e-5)
    torch.cuda.synchronize()
    _check_fwd(x, None, w, b, out, 1e-5, torch.float32)
    assert torch.equal(out[0].cpu()[4:], b.expand(5, -1))


@pytest.mark.parametrize("where", ["x", "residual"])
def test_sum_in_place_and_leading_axes(where):
    x, r = _draw((2, 3, 5, 264), 10, torch.bfloat16), _draw((2, 3, 5, 264), 11, torch.bfloat16)
    w = _draw((264,), 12)
    xd, rd = x.cuda(), r.cuda()
    into = xd if where == "x" else rd
    y, s, mean, rstd = g.gdn2_layer_norm_fwd(xd, w.cuda(), None, rd, sum_out=into)
    torch.cuda.synchronize()
    assert s.data_ptr() == into.data_ptr() and mean.shape == (2, 3, 5) and y.shape == x.shape
    flat = (y.reshape(-1, 264), s.reshape(-1, 264), mean.reshape(-1), rstd.reshape(-1))
    _check_fwd(x.reshape(-1, 264), r.reshape(-1, 264), w, None, flat, 1e-5, torch.bfloat16)


def test_empty():
    w = torch.ones(16, device="cuda")
    y, _, mean, _ = g.gdn2_layer_norm_fwd(torch.empty(0, 16, device="cuda"), w)
    assert y.shape == (0, 16) and mean.shape == (0,)
    e = torch.empty(0, device="cuda")
    r = g.gdn2_layer_norm_bwd(y, y, w, e, e)
    assert torch.equal(r["dweight"].cpu(), torch.zeros(16)) and torch.equal(r["dbias"].cpu(), torch.zeros(16))


def _check_bwd(dy, s, w, mean, rstd, ds, r, dtype):
    f = [_f64(t) for t in (dy, s, w, mean, rstd)]
    dx_ref, dw_ref, db_ref = layer.layer_norm_backward(*f, ds=_f64(ds))
    dyf, sf, wf, mf, rf = f
    rows, cols = sf.shape
    n = _depth(cols)
    xh = np.abs(sf - mf[:, None]) * rf[:, None]
    h = np.abs(dyf * wf)
    # m0 and m1 are sums of cols terms in a tree, their terms off by a few u each
    m0, m1 = h.mean(-1, keepdims=True), (h * xh).mean(-1, keepdims=True)
    bound = rf[:, None] * (n + 8) * U * (h + m0 + xh * m1) + 2 * U * (0 if ds is None else np.abs(_f64(ds)))
    _within(r["dx"], dx_ref, bound + HALF[dtype] * (np.abs(dx_ref) + bound) + 1e-38)
    # column sums: at most a block's rows in one chain, then the partial rows in chains of
    # an eighth of them; every term xh is off by 3 u
    chain = rows / min(rows, 592) + 592 / 8 + 16 + 128 + 4
    _within(r["dweight"], dw_ref, chain * U * (np.abs(dyf) * xh).sum(0) + 1e-38)
    if r["dbias"] is not None:
        _within(r["dbias"], db_ref, chain * U * np.abs(dyf).sum(0) + 1e-38)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", WIDTHS)
def test_backward_widths(cols, dtype):
    rows = 41 if cols < 3000 else 6
    s, dy, w = _draw((rows, cols), 20, dtype), _draw((rows, cols), 21, dtype), _draw((cols,), 22)
    ds = _draw((rows, cols), 23, dtype) if cols % 3 else None
    _, _, mean, rstd = g.gdn2_layer_norm_fwd(s.cuda(), w.cuda())
    r = g.gdn2_layer_norm_bwd(dy.cuda(), s.cuda(), w.cuda(), mean, rstd, None if ds is None else ds.cuda())
    torch.cuda.synchronize()
    _check_bwd(dy, s, w, mean, rstd, ds, r, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (2, 513), (130, 8), (5000, 40), (2500, 2048), (700, 8193)])
def test_backward_rows(rows, cols, dtype):
    s, dy, w = _draw((rows, cols), 24, dtype), _draw((rows, cols), 25, dtype), _draw((cols,), 26)
    _, _, mean, rstd = g.gdn2_layer_norm_fwd(s.cuda(), w.cuda())
    r = g.gdn2_layer_norm_bwd(dy.cuda(), s.cuda(), w.cuda(), mean, rstd, want_dbias=False)
    torch.cuda.synchronize()
    assert r["dbias"] is None
    _check_bwd(dy, s, w, mean, rstd, None, r, dtype)


def test_backward_against_differences():
    rng = np.random.default_rng(30)
    s, dy, w, b = (rng.standard_normal(n) for n in ((3, 20), (3, 20), 20, 20))
    _, mean, rstd = layer.layer_norm(s, w, b)

    def loss(s, w, b):
        return float((layer.layer_norm(s, w, b)[0] * dy).sum())

    dev = [torch.from_numpy(np.float32(t)).cuda() for t in (dy, s, w, mean, rstd)]
    r = {n: _f64(t) for n, t in g.gdn2_layer_norm_bwd(*dev).items()}
    step = 1e-5
    for name, at, i in [("dx", 0, (1, 7)), ("dx", 0, (2, 0)), ("dweight", 1, (5,)), ("dbias", 2, (11,))]:
        args = [s.copy(), w.copy(), b.copy()]
        args[at][i] += step
        up = loss(*args)
        args[at][i] -= 2 * step
        # central differences are off by about step^2 and 2^-52 |loss| / step; the kernel by fp32
        assert abs((up - loss(*args)) / (2 * step) - r[name][i]) < 1e-4, (name, i)


def test_same_result_twice_and_on_another_stream():
    s, dy, w = (_draw(n, 31 + i, t).cuda() for i, (n, t) in enumerate(
        [((3001, 520), torch.bfloat16), ((3001, 520), torch.bfloat16), ((520,), torch.float32)]))
    _, _, mean, rstd = g.gdn2_layer_norm_fwd(s, w)
    a = g.gdn2_layer_norm_bwd(dy, s, w, mean, rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = g.gdn2_layer_norm_bwd(dy, s, w, mean, rstd, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_captured_forward_and_backward():
    x, r, dy, w = (_draw(n, 40 + i).cuda() for i, n in enumerate([(65, 300), (65, 300), (65, 300), (300,)]))
    ws = torch.empty(g.lib().gdn2_layer_norm_bwd_workspace_bytes(65, 300), dtype=torch.uint8, device="cuda")
    y, s, mean, rstd = g.gdn2_layer_norm_fwd(x, w, None, r)
    ref = g.gdn2_layer_norm_bwd(dy, s, w, mean, rstd)
    out = {n: torch.zeros_like(t) for n, t in ref.items()}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _, s2, m2, r2 = g.gdn2_layer_norm_fwd(x, w, None, r)
        g.gdn2_layer_norm_bwd(dy, s2, w, m2, r2, workspace=ws, out=out)
    for scale in (1.0, 2.0):
        dy.copy_(dy * scale)
        graph.replay()
        torch.cuda.synchronize()
        want = g.gdn2_layer_norm_bwd(dy, s, w, mean, rstd)
        for n in out:
            assert torch.equal(out[n], want[n]), n
