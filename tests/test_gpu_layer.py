"""The layer's operators one after the other on the GPU, as they are used: a prompt of packed sequences
and steps after it (convolution, scalar-gate rule, layer norm), and a training step
(convolution, channel-wise mixer with one gate, layer norm, and the three backward passes).

Each stage is held against fp64 from the inputs that it got, within that operator's own tolerance
(what the tests of the single operators derive); the training step's gradients are also held
against differences of the whole in fp64, the tolerance being each stage's error carried to
the loss."""
import numpy as np
import pytest
import torch

import gated_delta_rule_95_b200 as g
import oracle
from oracle import backward as ob, layer
from tests.parity import TOL, rel_err
from tests.test_gpu_gdr import check_sequence
from tests.test_gpu_norm import _check_fwd

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HK, HV, D = 2, 4, 64
C = (2 * HK + HV) * D


def _f64(t):
    return t.detach().cpu().double().numpy()


def _draw(rng, *shape, std=1.0, dtype=F32):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(dtype).cuda()


def _check_conv(x, w, b, y, spans):
    """4 products and sums in fp32 and one rounding to bf16."""
    for lo, hi, hist in spans:
        ref, _ = oracle.short_conv(_f64(x[lo:hi]), _f64(w), _f64(b), hist)
        mag, _ = oracle.short_conv(np.abs(_f64(x[lo:hi])), np.abs(_f64(w)), np.abs(_f64(b)), None if hist is None else np.abs(hist))
        bound = 5 * U * mag
        assert np.all(np.abs(_f64(y[lo:hi]) - ref) <= bound + 2.0 ** -8 * (np.abs(ref) + bound))


def _heads(y, rng, lead):
    """q, k (normed, the lengths 1 at most), v, g, beta of the rows y [..., C]."""
    def unit(t):
        t = t.float()
        return (t / t.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6) * (1 - 2 ** -7)).to(BF).contiguous()
    q, k, v = y.split([HK * D, HK * D, HV * D], -1)
    q, k, v = unit(q.reshape(*lead, HK, D)), unit(k.reshape(*lead, HK, D)), v.reshape(*lead, HV, D).contiguous()
    gg = -torch.nn.functional.softplus(_draw(rng, *lead, HV)) / 8
    return q, k, v, gg, torch.sigmoid(_draw(rng, *lead, HV))


def test_prompt_and_steps():
    rng = np.random.default_rng(1)
    lengths = [70, 1, 200, 0, 64]
    N, T = len(lengths), sum(lengths)
    at = np.concatenate([[0], np.cumsum(lengths)])
    cu = torch.tensor(at, dtype=torch.int32).cuda()
    w, b = _draw(rng, C, 4, std=0.5), _draw(rng, C, std=0.1)
    nw, nb = _draw(rng, HV * D, std=0.2) + 1, _draw(rng, HV * D, std=0.2)
    x, hist0 = _draw(rng, T, C, dtype=BF), _draw(rng, N, 3, C, dtype=BF)
    hist = hist0.clone()

    y, _ = g.gdn2_short_conv(x, w, b, cu_seqlens=cu, hist=hist, hist_out=hist)
    q, k, v, gg, beta = _heads(y, rng, (T,))
    o, S = g.gdn2_gdr_chunk_fwd(q, k, v, gg, beta, cu_seqlens=cu, scale=D ** -0.5)
    out = g.gdn2_layer_norm_fwd(o.reshape(T, -1), nw, nb, v.reshape(T, -1), eps=1e-5)
    torch.cuda.synchronize()
    _check_conv(x, w, b, y, [(at[n], at[n + 1], _f64(hist0[n])) for n in range(N) if lengths[n]])
    d = dict(q=q, k=k, v=v, g=gg, beta=beta)
    for n in range(N):
        if lengths[n]:
            check_sequence(d, slice(at[n], at[n + 1]), o[at[n]:at[n + 1]], S[n], None, D ** -0.5, BF, True)
    _check_fwd(o.reshape(T, -1).cpu(), v.reshape(T, -1).cpu(), nw, nb, out, 1e-5, BF)

    for _ in range(3):  # steps: the state and the history go from call to call in place
        x1 = _draw(rng, N, 1, C, dtype=BF)
        before, S0 = _f64(hist), S.clone()
        y1, _ = g.gdn2_short_conv(x1, w, b, hist=hist, hist_out=hist)
        q, k, v, gg, beta = _heads(y1[:, 0], rng, (N,))
        o = g.gdn2_gdr_decode_step(q, k, v, gg, beta, S, scale=D ** -0.5)
        out = g.gdn2_layer_norm_fwd(o.reshape(N, -1), nw, nb, v.reshape(N, -1), eps=1e-5)
        torch.cuda.synchronize()
        for n in range(N):
            _check_conv(x1[n], w, b, y1[n], [(0, 1, before[n])])
            d = {m: t[n:n + 1] for m, t in dict(q=q, k=k, v=v, g=gg, beta=beta).items()}
            check_sequence(d, slice(0, 1), o[n:n + 1], S[n], S0[n], D ** -0.5, BF, False)
        _check_fwd(o.reshape(N, -1).cpu(), v.reshape(N, -1).cpu(), nw, nb, out, 1e-5, BF)
    assert g.gdn2_device_status() == 0


def _model(x, r, w4, b4, la, gate, nw, nb, H, cy, cs):
    """fp64: the loss, o, s and y of the training step."""
    conv = np.stack([oracle.short_conv(t, w4, b4)[0] for t in x])
    q, k, v = (t.reshape(*t.shape[:2], H, D) for t in np.split(conv, 3, -1))
    o, _ = oracle.forward(q, k, v, la, gate, gate)
    s = o.reshape(r.shape) + r
    y, mean, rstd = layer.layer_norm(s.reshape(-1, s.shape[-1]), nw, nb)
    return (y.reshape(s.shape) * cy).sum() + (s * cs).sum(), conv, o, rstd


def test_training_step():
    rng = np.random.default_rng(2)
    B, T, H = 2, 130, 2
    x, r = _draw(rng, B, T, 3 * H * D, std=0.3), _draw(rng, B, T, H * D)
    w4, b4 = _draw(rng, 3 * H * D, 4, std=0.3), _draw(rng, 3 * H * D, std=0.05)
    la = (-torch.nn.functional.softplus(_draw(rng, B, T, H, 1)) / 16).expand(B, T, H, D).contiguous()
    gate = torch.sigmoid(_draw(rng, B, T, H, 1)).expand(B, T, H, D).contiguous()
    nw, nb = _draw(rng, H * D, std=0.2) + 1, _draw(rng, H * D, std=0.2)
    cy, cs = _draw(rng, B, T, H * D), _draw(rng, B, T, H * D)

    conv, _ = g.gdn2_short_conv(x, w4, b4)
    q, k, v = (t.reshape(B, T, H, D).contiguous() for t in conv.split(H * D, -1))
    o, _ = g.gdn2_chunk_fwd(q, k, v, la, gate, gate)
    y, s, mean, rstd = g.gdn2_layer_norm_fwd(o.reshape(B, T, H * D), nw, nb, r)
    n = g.gdn2_layer_norm_bwd(cy, s, nw, mean, rstd, cs)
    m = g.gdn2_chunk_bwd(q, k, v, la, gate, gate, None, n["dx"].reshape(B, T, H, D), want_dS0=False)
    dconv = torch.cat([m[t].reshape(B, T, H * D) for t in ("dq", "dk", "dv")], -1)
    c = g.gdn2_short_conv_bwd(dconv, x, w4)
    torch.cuda.synchronize()
    assert g.gdn2_device_status() == 0

    # stage by stage
    f = {t: _f64(a) for t, a in dict(x=x, r=r, w4=w4, b4=b4, la=la, gate=gate, nw=nw, nb=nb, cy=cy, cs=cs).items()}
    rows = (B * T, H * D)
    flat = [_f64(t).reshape(rows) for t in (cy, s, cs)]
    dx, dw, db = layer.layer_norm_backward(flat[0], flat[1], f["nw"], _f64(mean).reshape(-1), _f64(rstd).reshape(-1), flat[2])
    h = np.abs(flat[0] * f["nw"])
    xh = np.abs(flat[1] - _f64(mean).reshape(-1, 1)) * _f64(rstd).reshape(-1, 1)
    # two means of 128 products (a tree of 4 + 10), three products and sums
    bound = 20 * U * (_f64(rstd).reshape(-1, 1) * (h + h.mean(-1, keepdims=True) + xh * (h * xh).mean(-1, keepdims=True)) + np.abs(flat[2]))
    assert np.all(np.abs(_f64(n["dx"]).reshape(rows) - dx) <= bound)
    assert np.all(np.abs(_f64(n["dweight"]) - dw) <= (B * T + 8) * U * (np.abs(flat[0]) * xh).sum(0))
    assert np.all(np.abs(_f64(n["dbias"]) - db) <= (B * T + 8) * U * np.abs(flat[0]).sum(0))
    ref = ob.backward(*(_f64(t) for t in (q, k, v, la, gate, gate)), S0=None, do=_f64(n["dx"]).reshape(B, T, H, D), dS_T=None)
    for t in ("dq", "dk", "dv", "dlog_alpha", "db", "dw"):
        assert rel_err(_f64(m[t]), ref[t]) <= TOL["f32"], t
    dw4, db4 = np.zeros((3 * H * D, 4)), np.zeros(3 * H * D)
    mw4, mb4 = np.zeros_like(dw4), np.zeros_like(db4)
    for i in range(B):
        a = layer.short_conv_backward(_f64(dconv[i]), f["x"][i], f["w4"])
        mag = layer.short_conv_backward(np.abs(_f64(dconv[i])), np.abs(f["x"][i]), np.abs(f["w4"]))
        assert np.all(np.abs(_f64(c["dx"][i]) - a[0]) <= 7 * U * mag[0])
        dw4, db4, mw4, mb4 = dw4 + a[1], db4 + a[2], mw4 + mag[1], mb4 + mag[2]
    assert np.all(np.abs(_f64(c["dweight"]) - dw4) <= (B * T + 8) * U * mw4)
    assert np.all(np.abs(_f64(c["dbias"]) - db4) <= (B * T + 8) * U * mb4)

    # the whole against central differences along one direction of each leaf
    names = ("x", "r", "w4", "b4", "nw", "nb")
    grads = dict(x=c["dx"], r=n["dx"], w4=c["dweight"], b4=c["dbias"], nw=n["dweight"], nb=n["dbias"])
    order = ("x", "r", "w4", "b4", "la", "gate", "nw", "nb")
    for leaf in names:
        e = rng.standard_normal(f[leaf].shape)
        step = 1e-4
        ends = [_model(*(f[t] + sgn * step * e if t == leaf else f[t] for t in order), H, f["cy"], f["cs"]) for sgn in (1, -1)]
        want = (ends[0][0] - ends[1][0]) / (2 * step)
        got = (_f64(grads[leaf]) * e).sum()
        J_conv, J_o = ((ends[0][i] - ends[1][i]) / (2 * step) for i in (1, 2))
        # The mixer's o is off by d = 1e-4 rms(o) at most (its bar); a row's xh and rstd then by
        # e = d rstd in 6 e |xh|-sized terms (mean, deviation, scale), the norm's gradient in 13 such of
        # its h rstd; that error meets J_o along the direction.  The mixer's own gradient is off by 1e-4
        # of its rms, and meets J_conv.  nw's gradient sees xh itself.  The rest is fp32 (2e-6) and
        # the difference's own error (step^2 of the third derivative, and 1e-16 / step of the loss).
        o_rms = np.sqrt((ends[0][2] ** 2).mean())
        off = TOL["f32"] * o_rms * ends[0][3].max()
        hr = np.sqrt((h ** 2).sum()) * ends[0][3].max()
        tol = 13 * off * hr * np.sqrt((J_o ** 2).sum())
        tol += TOL["f32"] * np.sqrt((_f64(dconv) ** 2).mean() * dconv.numel()) * np.sqrt((J_conv ** 2).sum())
        if leaf in ("nw", "nb"):
            tol += 6 * off * np.sqrt((flat[0] ** 2).sum()) * np.sqrt(rows[0]) * np.sqrt((e ** 2).sum()) / np.sqrt(e.size)
        tol += 2e-6 * np.sqrt((_f64(grads[leaf]) ** 2).sum() * (e ** 2).sum()) + 1e-6 * abs(want) + 1e-9
        assert abs(got - want) <= tol, (leaf, got, want, tol)


def test_binding_refuses_on_the_device():
    z = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    x, w, c, st = z(2, 10, 64), z(64), z(64, 4), z(2, 10)
    q, v, b, S, cu = z(2, 10, 2, 64), z(2, 10, 4, 64), z(2, 10, 4), z(2, 4, 64, 64), z(3, dt=torch.int32)
    one = dict(q=q[:, 0].contiguous(), k=q[:, 0].contiguous(), v=v[:, 0].contiguous(), g=b[:, 0].contiguous(), beta=b[:, 0].contiguous(), S=S)
    far = q.transpose(1, 2).contiguous().transpose(1, 2)  # the right shape, other strides
    calls = [
        lambda: g.gdn2_layer_norm_fwd(x.transpose(0, 1), w), lambda: g.gdn2_layer_norm_fwd(x, w[:63]), lambda: g.gdn2_layer_norm_fwd(x, w.cpu()),
        lambda: g.gdn2_layer_norm_fwd(x, w.to(BF)), lambda: g.gdn2_layer_norm_fwd(x, w, w[:1]), lambda: g.gdn2_layer_norm_fwd(x, w, None, x.to(BF)),
        lambda: g.gdn2_layer_norm_fwd(x, w, sum_out=x), lambda: g.gdn2_layer_norm_fwd(x, w, y=z(2, 10, 63)),
        lambda: g.gdn2_layer_norm_bwd(x[:1], x, w, st, st), lambda: g.gdn2_layer_norm_bwd(x, x, w, st[:1], st),
        lambda: g.gdn2_layer_norm_bwd(x, x, w, st, st.to(BF)), lambda: g.gdn2_layer_norm_bwd(x, x, w, st, st, st),
        lambda: g.gdn2_layer_norm_bwd(x, x, w, st, st, workspace=torch.zeros(9, dtype=torch.uint8)),
        lambda: g.gdn2_short_conv_bwd(x, x, c[:63]), lambda: g.gdn2_short_conv_bwd(x.to(BF), x, c), lambda: g.gdn2_short_conv_bwd(x, x, c, hist=z(2, 2, 64)),
        lambda: g.gdn2_short_conv_bwd(x[0], x[0], c, cu_seqlens=cu.long()), lambda: g.gdn2_short_conv_bwd(x[0], x[0], c, cu_seqlens=cu.cpu()),
        lambda: g.gdn2_gdr_chunk_fwd(far, q, v, b, b), lambda: g.gdn2_gdr_chunk_fwd(q, q[:, :, :1], v, b, b), lambda: g.gdn2_gdr_chunk_fwd(q, q, v, b[..., :3], b),
        lambda: g.gdn2_gdr_chunk_fwd(q, q, v.to(BF), b, b), lambda: g.gdn2_gdr_chunk_fwd(q, q, v, b.to(BF), b), lambda: g.gdn2_gdr_chunk_fwd(q, q, v, b, b, S[:1]),
        lambda: g.gdn2_gdr_chunk_fwd(q, q, v, b, b, S_T=S.transpose(2, 3)), lambda: g.gdn2_gdr_chunk_fwd(q, q, v, b, b, o=q),
        lambda: g.gdn2_gdr_chunk_fwd(q[0], q[0], v[0], b[0], b[0], cu_seqlens=cu.cpu()),
        lambda: g.gdn2_gdr_decode_step(**{**one, "S": S[:1]}), lambda: g.gdn2_gdr_decode_step(**{**one, "g": one["g"].to(BF)}),
        lambda: g.gdn2_gdr_decode_step(**one, S_out=S.transpose(2, 3)), lambda: g.gdn2_gdr_decode_step(**one, o=one["q"]),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="gdn2_"):
            call()
    small = torch.zeros(16, dtype=torch.uint8, device="cuda")
    late = [lambda: g.gdn2_gdr_chunk_fwd(z(2, 10, 3, 64), z(2, 10, 3, 64), v, b, b), lambda: g.gdn2_gdr_chunk_fwd(*(z(2, 10, 2, 32),) * 2, v, b, b),
            lambda: g.gdn2_gdr_chunk_fwd(q.to(BF), q.to(BF), v.to(BF), b, b, workspace=small), lambda: g.gdn2_layer_norm_bwd(x, x, w, st, st, workspace=small),
            lambda: g.gdn2_layer_norm_fwd(x, w, y=x), lambda: g.gdn2_gdr_chunk_fwd(v, v, v, b, b, o=v),
            lambda: g.gdn2_layer_norm_fwd(x.flatten()[1:].view(1, -1), z(1279)), lambda: g.gdn2_short_conv_bwd(z(2, 10, 60), z(2, 10, 60), z(60, 4))]
    for call in late:
        with pytest.raises(g.GDN2Error):
            call()
    torch.cuda.synchronize()
    assert g.gdn2_device_status() == 0


def test_two_streams_and_two_graphs_at_once():
    # prefill (split and whole), norm and convolution gradients on two streams, each call with its own
    # workspace, then as two captured graphs replayed side by side: what one alone gives, bit by bit
    rng = np.random.default_rng(3)

    def job(T):
        q, v = _draw(rng, 1, T, 2, 128, std=0.08, dtype=BF), _draw(rng, 1, T, 2, 128, dtype=BF)
        gg, beta = -torch.nn.functional.softplus(_draw(rng, 1, T, 2)), torch.sigmoid(_draw(rng, 1, T, 2))
        dy, w, c = _draw(rng, 1, T, 256, dtype=BF), _draw(rng, 256), _draw(rng, 256, 4)

        def run():
            o, S = g.gdn2_gdr_chunk_fwd(q, q, v, gg, beta)
            y, s, mean, rstd = g.gdn2_layer_norm_fwd(o.view(1, T, 256), w, None, dy)
            n = g.gdn2_layer_norm_bwd(dy, s, w, mean, rstd, want_dbias=False)
            r = g.gdn2_short_conv_bwd(n["dx"], s, c)
            return [o, S, y, n["dx"], n["dweight"], r["dx"], r["dweight"], r["dbias"]]
        return run
    jobs = [job(2600), job(300)]
    want = [run() for run in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        got = []
        for run, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(run())
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    graphs, outs = [], []
    for run in jobs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(run())
        graphs.append(gr)
    for _ in range(3):
        for t in [t for out in outs for t in out]:
            t.zero_()
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("as_handle", [False, True])
def test_a_given_stream_keeps_its_memory(as_handle):
    # the call waits on its stream while other work takes memory of the same sizes on the current one
    rng = np.random.default_rng(4)
    T = 2600
    q, v = _draw(rng, 1, T, 1, 128, std=0.08, dtype=BF), _draw(rng, 1, T, 1, 128, dtype=BF)
    gg, beta = -torch.nn.functional.softplus(_draw(rng, 1, T, 1)), torch.sigmoid(_draw(rng, 1, T, 1))
    x, dy, w, c = _draw(rng, 1, 4096, 2048, dtype=BF), _draw(rng, 1, 4096, 2048, dtype=BF), _draw(rng, 2048), _draw(rng, 2048, 4)
    _, _, mean, rstd = g.gdn2_layer_norm_fwd(x, w)
    L = g.lib()
    calls = [(lambda **k: g.gdn2_gdr_chunk_fwd(q, q, v, gg, beta, **k), L.gdn2_gdr_chunk_fwd_workspace_bytes(1, T, 1, 128, 128, 0, 1)),
             (lambda **k: tuple(g.gdn2_layer_norm_bwd(dy, x, w, mean, rstd, **k).values()), L.gdn2_layer_norm_bwd_workspace_bytes(4096, 2048)),
             (lambda **k: tuple(t for t in g.gdn2_short_conv_bwd(dy, x, c, **k).values() if t is not None), L.gdn2_short_conv_bwd_workspace_bytes(4096, 2048))]
    side = torch.cuda.Stream()
    for call, size in calls:
        want = call()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # about 0.1 s
        got = call(stream=side.cuda_stream if as_handle else side)
        taken = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        del taken
    assert g.gdn2_device_status() == 0


def test_offsets_past_32_bits():
    # tensors of more than 2^31 elements: what lies at their end is what it is alone
    def tail(t, n):
        return t[-n:].contiguous()
    gen = torch.Generator(device="cuda").manual_seed(5)

    def rand(*s, dt=BF):
        return torch.randn(s, generator=gen, device="cuda", dtype=dt)
    rows, n = (1 << 20) + 5000, 64
    x, w = rand(rows, 2048), rand(2048, dt=F32)
    y, _, mean, rstd = g.gdn2_layer_norm_fwd(x, w)
    y1, _, m1, r1 = g.gdn2_layer_norm_fwd(tail(x, n), w)
    assert torch.equal(tail(y, n), y1) and torch.equal(tail(mean, n), m1) and torch.equal(tail(rstd, n), r1)
    dx = g.gdn2_layer_norm_bwd(y, x, w, mean, rstd, want_dbias=False)["dx"]
    assert torch.equal(tail(dx, n), g.gdn2_layer_norm_bwd(y1, tail(x, n), w, m1, r1, want_dbias=False)["dx"])
    del dx
    c = rand(2048, 4, dt=F32)
    dx = g.gdn2_short_conv_bwd(y[None], x[None], c, want_dbias=False)["dx"][0]
    alone = g.gdn2_short_conv_bwd(tail(y, n)[None], tail(x, n)[None], c, want_dbias=False)["dx"][0]
    # four products and sums in another order, then one rounding: one step of bf16 at most, and fp32's
    assert torch.all((tail(dx, n).float() - alone.float()).abs() <= 2.0 ** -7 * alone.float().abs() + 1e-5)
    del x, y, dx, mean, rstd
    B, H = 2200, 64
    S, S2 = rand(B, H, 128, 128, dt=F32), torch.empty(B, H, 128, 128, device="cuda")
    q, v, gg = torch.nn.functional.normalize(rand(B, 1, 128, dt=F32), dim=-1), rand(B, H, 128, dt=F32), -rand(B, H, dt=F32).abs()
    o = g.gdn2_gdr_decode_step(q, q, v, gg, torch.sigmoid(gg), S, S_out=S2)
    t = [tail(a, 2) for a in (q, q, v, gg, torch.sigmoid(gg), S)]
    o1 = g.gdn2_gdr_decode_step(*t)
    assert torch.equal(tail(o, 2), o1) and torch.equal(tail(S2, 2), t[-1])
    del S, S2, o
    # a prompt of one key head and 128 value heads; the decay leaves nothing of what is 512 tokens back
    T, H = (1 << 17) + 1000, 128
    q, k = (torch.nn.functional.normalize(rand(1, T, 1, 128, dt=F32), dim=-1).to(BF) for _ in range(2))
    v, gg, beta = rand(1, T, H, 128), -1 - rand(1, T, H, dt=F32).abs(), torch.sigmoid(rand(1, T, H, dt=F32))
    o, S = g.gdn2_gdr_chunk_fwd(q, k, v, gg, beta)
    torch.cuda.synchronize()
    for h in (0, 127):
        a = [t[0, -576:].cpu().double().numpy() for t in (q, k, v[..., h:h + 1, :], gg[..., h:h + 1], beta[..., h:h + 1])]
        o_ref, S_ref = layer.gdr_forward(*a)
        # the rounding of o, and of the products 1e-5 of the values' size (test_gpu_gdr derives the bound for each)
        got, ref = _f64(o[0, -64:, h]), o_ref[-64:, 0]
        assert np.all(np.abs(got - ref) <= 2.0 ** -6 * np.abs(ref) + 2.0 ** -6 * np.sqrt((ref ** 2).mean()))
        assert np.linalg.norm(_f64(S[0, h]) - S_ref[0]) <= 2e-5 * np.linalg.norm(S_ref[0])
    assert g.gdn2_device_status() == 0


def test_the_most_tokens_of_the_convolution_backward():
    # as many tokens as the entry point takes, zero but for the last: the strips' bounds and count fill 31 bits
    T, C, n = 2 ** 31 - 65, 8, 4096
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80e9:
        pytest.skip("needs 70 GB of device memory")
    x = torch.zeros(1, T, C, dtype=BF, device="cuda")
    x[0, -n:].normal_(generator=torch.Generator(device="cuda").manual_seed(6))
    c = torch.randn(C, 4, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    out = dict(dx=torch.full_like(x, 7.0), dweight=torch.empty_like(c), dbias=torch.empty(C, device="cuda"))
    g.gdn2_short_conv_bwd(x, x, c, out=out)
    alone = g.gdn2_short_conv_bwd(*(x[:, -n:].contiguous(),) * 2, c)
    assert torch.equal(out["dx"][:, -n:], alone["dx"])
    for part in (out["dx"][0, :1 << 20], out["dx"][0, T // 2:T // 2 + (1 << 20)], out["dx"][0, -n - 1000:-n - 3]):
        assert not part.any()
    # sums of the same n products, in chains of n at most
    a = x[0, -n:].float()
    for got, want, mag in ((out["dbias"], alone["dbias"], a.abs().sum(0)), (out["dweight"], alone["dweight"], a.square().sum(0)[:, None])):
        assert torch.all((got - want).abs() <= 2 * n * U * mag)
    assert g.gdn2_device_status() == 0
