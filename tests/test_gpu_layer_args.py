"""The layer's entry points on the GPU: stream handles, sizes past 32 bits, a workspace used call after call,
what outputs held before."""
import pytest
import torch

import gated_delta_rule_95_b200 as g

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def test_the_default_stream_by_its_handle():
    # handle 0 is the default stream: a call on it waits for what is queued there, whatever stream is current
    assert torch.cuda.default_stream().cuda_stream == 0
    x, w, side = torch.zeros(64, 256, device="cuda"), torch.ones(256, device="cuda"), torch.cuda.Stream()
    new = torch.randn(64, 256, device="cuda")
    want = g.gdn2_layer_norm_fwd(new, w)[0]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s, on the default stream
    x.copy_(new)
    with torch.cuda.stream(side):
        y = g.gdn2_layer_norm_fwd(x, w, stream=0)[0]
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.large
def test_more_rows_than_the_library_counts():
    # 2^32 + 5 rows are not 5
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 26 GB of device memory")
    x, w = torch.empty(2 ** 32 + 5, 1, dtype=BF, device="cuda"), torch.ones(1, device="cuda")
    for call in (lambda: g.gdn2_layer_norm_fwd(x, w, want_stats=False), lambda: g.gdn2_short_conv(x.view(1, -1, 1), torch.ones(1, 4, device="cuda")),
                 lambda: g.gdn2_short_conv_bwd(x.view(1, -1, 1), x.view(1, -1, 1), torch.ones(1, 4, device="cuda"))):
        with pytest.raises(ValueError, match="gdn2_"):
            call()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_workspace_call_after_call(dtype):
    # the sums over partial results start before the kernel in front is done: each call's are its own, not what the
    # workspace held; and the history's gradient may replace dhist_out
    gen = torch.Generator(device="cuda").manual_seed(1)

    def rand(*s, dt=dtype):
        return torch.randn(s, generator=gen, device="cuda", dtype=dt)
    lengths = [0, 1, 2, 500, 3, 0, 700, 40]
    T, N, C = sum(lengths), len(lengths), 264
    cu = torch.tensor([sum(lengths[:i]) for i in range(N + 1)], dtype=torch.int32, device="cuda")
    w, c = rand(C, dt=F32), rand(C, 4, dt=F32)
    ins = [(rand(T, C), rand(T, C), rand(N, 3, C), rand(N, 3, C), rand(T, dt=F32), rand(T, dt=F32)) for _ in range(4)]
    L = g.lib()
    ws = torch.empty(max(L.gdn2_short_conv_bwd_workspace_bytes(T, C), L.gdn2_layer_norm_bwd_workspace_bytes(T, C)), dtype=torch.uint8, device="cuda")

    def run(i, workspace, in_place):
        x, dy, hist, dho, mean, rstd = ins[i]
        dho = dho.clone()
        out = dict(dx=torch.empty_like(x), dweight=torch.empty_like(c), dbias=torch.empty_like(w), dhist=dho if in_place else torch.empty_like(dho))
        a = g.gdn2_short_conv_bwd(dy, x, c, cu_seqlens=cu, hist=hist, dhist_out=dho, out=out, workspace=workspace)
        b = g.gdn2_layer_norm_bwd(dy, x, w, mean, rstd, workspace=workspace)
        return [t.clone() for r in (a, b) for t in r.values()]
    want = []
    for i in range(4):
        want.append(run(i, None, False))
        torch.cuda.synchronize()
    got = [run(i % 4, ws, True) for i in range(12)]
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(want[i % 4], r)), i
    assert g.gdn2_device_status() == 0


def test_the_taps_gradient_in_their_place():
    # without the history's gradient the taps are read before their gradient is written
    x, dy, c = torch.randn(2, 300, 64, device="cuda"), torch.randn(2, 300, 64, device="cuda"), torch.randn(64, 4, device="cuda")
    want = g.gdn2_short_conv_bwd(dy, x, c)
    out = dict(dx=torch.empty_like(x), dweight=c, dbias=torch.empty(64, device="cuda"), dhist=None)
    g.gdn2_short_conv_bwd(dy, x, c, out=out)
    assert torch.equal(out["dx"], want["dx"]) and torch.equal(out["dweight"], want["dweight"]) and torch.equal(out["dbias"], want["dbias"])
    c = want["dweight"].clone()
    with pytest.raises(g.GDN2Error):
        g.gdn2_short_conv_bwd(dy, x, c, out=dict(out, dweight=c, dhist=torch.empty(2, 3, 64, device="cuda")))


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("lengths", [[70, 0, 64, 1, 130], [3000, 5, 63, 2000], None])
def test_what_the_outputs_held_before_is_nothing(lengths, dk, dv):
    # o holds intermediate values while the call runs; what it held before the call, and what the rows past a sequence's
    # end hold, reaches no result, and rows of no sequence are left as they were
    gen = torch.Generator(device="cuda").manual_seed(2)

    def rand(*s, dt=BF):
        return torch.randn(s, generator=gen, device="cuda").to(dt)
    lead = (2, 333) if lengths is None else (sum(lengths) + 90,)
    kw, mine = {}, slice(None)
    if lengths is not None:
        at = [20 + sum(lengths[:i]) for i in range(len(lengths) + 1)]
        kw, mine = dict(cu_seqlens=torch.tensor(at, dtype=torch.int32, device="cuda")), slice(20, at[-1])
    q, k = (torch.nn.functional.normalize(rand(*lead, 2, dk, dt=F32), dim=-1).to(BF) for _ in range(2))
    v, gg, beta = rand(*lead, 4, dv), -rand(*lead, 4, dt=F32).abs(), torch.sigmoid(rand(*lead, 4, dt=F32))
    want = g.gdn2_gdr_chunk_fwd(q, k, v, gg, beta, o=torch.zeros_like(v), **kw)
    for fill in (float("nan"), float("inf"), -3e38):
        o = torch.full_like(v, fill)
        before = o.clone()
        _, S = g.gdn2_gdr_chunk_fwd(q, k, v, gg, beta, o=o, **kw)
        assert torch.equal(o[mine], want[0][mine]) and torch.equal(S, want[1])
        if lengths is not None:
            for rows in (slice(0, 20), slice(at[-1], None)):
                assert torch.equal(o[rows].view(torch.int16), before[rows].view(torch.int16))
    assert torch.isfinite(want[0][mine]).all() and g.gdn2_device_status() == 0
