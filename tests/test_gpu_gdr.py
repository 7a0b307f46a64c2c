"""The gated delta rule with scalar gates on the GPU against the fp64 recurrence: both types,
all head sizes, shared key heads, lengths around the chunk of 64, packed batches with empty
sequences and rows of nobody, cleared states (g = -inf), write strengths up to 2, decode steps
that equal the prompt, streams, captured graphs, bad offsets.

Tolerances, from the arithmetic.  The rule contracts (|1 - beta k k^T| <= 1 for |k| <= 1 and
beta <= 2, alpha <= 1), so an error of the state in the Frobenius norm never grows, and the
state's error is at most the sum of what each step adds.
  token by token (u = 2^-24): the key sum of at most 128 terms in a tree of 16 + 3 (the scan)
    or 16 + 8 (the step), the decay's exponential and the update add at most
    40 u (|S before| + |S after| + beta |v|);
  chunks on the tensor cores: T = (I + A)^-1 diag(beta), R = -e^G K S, U = T V + T R.  S, R, U
    and T enter their products in two bf16 parts (2^-16 of the value each), T R drops the
    product of both second parts and T itself is off by its solve (2^-16 each); fp32 sums add
    less than 2^-17 of their terms' magnitudes.  So with the fp64 chunk quantities
      dR = 2^-15 e^G |K| |S|,  dU = |T| dR + 2^-14 |T| (|V| + |R|),
      dS = 2^-16 |S| + |K|^T e^(G_C - G) (dU + 2^-15 |U|),
    and o adds |P| dU + 2 2^-8 |P| |U| (P and U as single bf16) and 2^-8 |o|;
  segments: the state after one is M S + N with M and N run through its chunks from S = I without V
    and from S = 0, each off by what its own chunks add, the sum M S + N in fp32 by 130 u |M| |S|."""
import numpy as np
import pytest
import torch

import gated_delta_rule_95_b200 as g
from oracle import layer

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
GDN2_ERR_SHAPE = 2
BF, F32 = torch.bfloat16, torch.float32


def _f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def _cuda(t):
    return None if t is None else t.cuda()


def draw(lead, Hk, Hv, dk, dv, dtype, seed, decay=1 / 16, beta_max=1.0, n=None, state=False):
    """Inputs over the leading axes; keys and queries of norm 1 at most."""
    rng = np.random.default_rng(seed)

    def unit(*s):
        x = rng.standard_normal(s)
        return torch.from_numpy((x / np.linalg.norm(x, axis=-1, keepdims=True) * (1 - 2 ** -7)).astype(np.float32)).to(dtype)

    d = dict(q=unit(*lead, Hk, dk), k=unit(*lead, Hk, dk),
             v=torch.from_numpy(rng.standard_normal((*lead, Hv, dv)).astype(np.float32)).to(dtype),
             g=torch.from_numpy((-np.logaddexp(0, rng.standard_normal((*lead, Hv))) * decay).astype(np.float32)),
             beta=torch.from_numpy((beta_max / (1 + np.exp(-rng.standard_normal((*lead, Hv))))).astype(np.float32)))
    d["S0"] = torch.from_numpy((0.1 * rng.standard_normal((n, Hv, dk, dv))).astype(np.float32)) if state else None
    return d


def run(d, **kw):
    a = {n: _cuda(t) for n, t in d.items()}
    out = g.gdn2_gdr_chunk_fwd(a["q"], a["k"], a["v"], a["g"], a["beta"], a["S0"], **kw)
    torch.cuda.synchronize()
    return out


def _norm(x):
    return np.sqrt((x * x).sum((-2, -1)))


def chunk_parts(q, k, v, gg, beta, S):
    """For one chunk from the state S [Hv, dk, dv]: what its arithmetic adds to the state's error (norm) and
    to the outputs' errors [Hv, t, dv], scale 1."""
    n, head = len(q), np.arange(v.shape[1]) // (v.shape[1] // q.shape[1])
    with np.errstate(invalid="ignore"):
        G = np.cumsum(np.maximum(gg, -1e4), 0).T  # [H, t]
        D = np.exp(np.minimum(G[:, :, None] - G[:, None, :], 0.0)) * np.tril(np.ones((n, n)))
    K, Q = (x[:, head].transpose(1, 0, 2) for x in (k, q))
    V, b = v.transpose(1, 0, 2), beta.T[:, :, None]
    A = np.tril(b * D * (K @ K.transpose(0, 2, 1)), -1)
    Tm = np.linalg.inv(np.eye(n) + A) * b.transpose(0, 2, 1)
    eG, eE = np.exp(G)[:, :, None], np.exp(G[:, -1:] - G)[:, :, None]
    R = -eG * (K @ S)
    Uu, P = Tm @ (V + R), D * (Q @ K.transpose(0, 2, 1))
    dU = np.abs(Tm) @ (2.0 ** -15 * eG * (np.abs(K) @ np.abs(S)) + 2.0 ** -14 * (np.abs(V) + np.abs(R)))
    add = _norm(2.0 ** -16 * np.abs(S) + np.abs(K).transpose(0, 2, 1) @ (eE * (dU + 2.0 ** -15 * np.abs(Uu))))
    return add, 2.0 ** -15 * eG * (np.abs(Q) @ np.abs(S)) + np.abs(P) @ (dU + 2.0 ** -7 * np.abs(Uu))


def segment_errors(q, k, v, gg, beta, S0, starts):
    """What the states at the tokens `starts` (ascending, of chunks) are off by when the segments before
    them are joined, {token: [Hv]}."""
    Hv, dk = v.shape[1], q.shape[2]
    none = np.zeros((64, Hv, dk))
    S, err, out = S0, np.zeros(Hv), {}
    for begin, end in zip([0, *starts], starts):
        N, M = (np.zeros_like(S0) if begin else S0), np.broadcast_to(np.eye(dk), (Hv, dk, dk))
        eN, eM = np.zeros(Hv), np.zeros(Hv)
        for lo in range(begin, end, 64):
            c = slice(lo, lo + 64)
            eN = eN + chunk_parts(q[c], k[c], v[c], gg[c], beta[c], N)[0]
            N = layer.gdr_forward(q[c], k[c], v[c], gg[c], beta[c], N, 1.0)[1]
            if begin:
                eM = eM + chunk_parts(q[c], k[c], none, gg[c], beta[c], M)[0]
                M = layer.gdr_forward(q[c], k[c], none, gg[c], beta[c], M, 1.0)[1]
        if begin:
            err = err + eN + (eM + 130 * U * _norm(M)) * (_norm(S) + err)
            S = M @ S + N
        else:
            err, S = eN, N
        out[end] = err
    return out


def check_sequence(d, sl, o, S, S0, scale, dtype, chunked, segments=1):
    """One sequence's outputs o [T, Hv, dv] and S [Hv, dk, dv] (None: not asked)."""
    q, k, v, gg, beta = (_f64(d[n][sl]) for n in ("q", "k", "v", "g", "beta"))
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1:]
    S_ref = np.zeros((Hv, dk, dv)) if S0 is None else _f64(S0)
    err = np.zeros(Hv)  # of the state, in the norm
    per = -(-(-(-T // 64)) // segments) * 64
    starts = [s * per for s in range(1, segments) if s * per < T]
    joined = segment_errors(q, k, v, gg, beta, S_ref, starts) if starts else {}
    o_ref, o_tol = np.zeros((T, Hv, dv)), np.zeros((T, Hv, dv))
    for lo in range(0, T, 64):
        hi = min(T, lo + 64)
        c = slice(lo, hi)
        if chunked:
            err = joined.get(lo, err)
            add, tol = chunk_parts(q[c], k[c], v[c], gg[c], beta[c], S_ref)
            o_ref[c], S_new = layer.gdr_forward(q[c], k[c], v[c], gg[c], beta[c], S_ref, scale)
            # what the state was off, through Q and (|T K dS| <= the contraction's bound) through U
            tol = tol + err[:, None, None] * (1 + np.sqrt(hi - lo))
            o_tol[c] = abs(scale) * tol.transpose(1, 0, 2)
            err, S_ref = err + add, S_new
        else:
            for t in range(lo, hi):
                o_ref[t:t + 1], S_new = layer.gdr_forward(*(x[t:t + 1] for x in (q, k, v, gg, beta)), S_ref, scale)
                err = np.exp(gg[t]) * err + 40 * U * (_norm(S_ref) + _norm(S_new) + beta[t] * np.linalg.norm(v[t], axis=-1))
                S_ref = S_new
                o_tol[t] = (abs(scale) * (err + 24 * U * _norm(S_ref)))[:, None]
    o_tol = o_tol + HALF[dtype] * (np.abs(o_ref) + o_tol) + 1e-38
    bad = np.abs(_f64(o) - o_ref) / o_tol
    assert np.all(bad <= 1), ("o", float(np.nanmax(bad)), bool(np.isnan(bad).any()))
    if S is not None:
        off = _norm(_f64(S) - S_ref)
        assert np.all(off <= err + 1e-30), ("S", float(np.max(off / (err + 1e-30))))


def is_chunked(dtype):
    return dtype == BF


SIZES = [(128, 128), (64, 64), (128, 64), (64, 128)]
LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 330]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(T, dtype):
    d = draw((2, T), 1, 2, 128, 128, dtype, seed=T, n=2, state=T % 2 == 0)
    o, S = run(d, scale=0.5)
    for n in range(2):
        check_sequence(d, n, o[n], S[n], None if d["S0"] is None else d["S0"][n], 0.5, dtype, is_chunked(dtype))
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("Hk,Hv", [(1, 1), (3, 3), (2, 8)])
def test_head_sizes_and_groups(dk, dv, Hk, Hv, dtype):
    d = draw((2, 150), Hk, Hv, dk, dv, dtype, seed=dk + dv + Hv, n=2, state=True)
    o, S = run(d, scale=dk ** -0.5)
    assert o.dtype == dtype and S.dtype == F32
    for n in range(2):
        check_sequence(d, n, o[n], S[n], d["S0"][n], dk ** -0.5, dtype, is_chunked(dtype))
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("decay,beta_max", [(0.0, 1.0), (3.0, 1.0), (40.0, 1.0), (1 / 16, 2.0), (1 / 16, 0.0)])
def test_decays_and_strengths(decay, beta_max, dtype):
    # no decay at all, decays far past what one chunk's exponentials could hold (e^-2500),
    # overshooting writes, no writes
    d = draw((1, 300), 2, 2, 64, 128, dtype, seed=7, decay=decay, beta_max=beta_max, n=1, state=True)
    o, S = run(d)
    check_sequence(d, 0, o[0], S[0], d["S0"][0], 1.0, dtype, is_chunked(dtype))
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_same_key_again_and_again(dtype):
    # T = (I + A)^-1 at its least benign: one key, full strength, no decay
    d = draw((1, 200), 1, 2, 128, 128, dtype, seed=8, decay=0.0)
    d["k"] = d["k"][:, :1].expand_as(d["k"]).contiguous()
    d["beta"] = torch.ones_like(d["beta"])
    o, S = run(d)
    check_sequence(d, 0, o[0], S[0], None, 1.0, dtype, is_chunked(dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_cleared_states(dtype):
    # g = -inf: nothing before the token is left; everything from there on is as from a zero state
    d = draw((1, 190), 1, 2, 64, 64, dtype, seed=9, n=1, state=True)
    for t in (0, 5, 64, 100, 101, 189):
        d["g"][0, t] = -float("inf")
    o, S = run(d)
    check_sequence(d, 0, o[0], S[0], d["S0"][0], 1.0, dtype, is_chunked(dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lengths", [[5, 0, 64, 1, 130, 63, 0], [0, 0], [300], [1] * 9, [64, 64, 65]])
def test_packed(lengths, dtype):
    T, N = sum(lengths), len(lengths)
    d = draw((T,), 2, 4, 64, 128, dtype, seed=10 + T, n=N, state=True)
    at = np.concatenate([[0], np.cumsum(lengths)])
    cu = torch.tensor(at, dtype=torch.int32).cuda()
    S = _cuda(d["S0"])  # states in place
    a = {n: _cuda(t) for n, t in d.items()}
    o, S2 = g.gdn2_gdr_chunk_fwd(a["q"], a["k"], a["v"], a["g"], a["beta"], S, cu_seqlens=cu, S_T=S, scale=0.25)
    torch.cuda.synchronize()
    assert S2.data_ptr() == S.data_ptr()
    for n in range(N):
        if lengths[n]:
            check_sequence(d, slice(at[n], at[n + 1]), o[at[n]:at[n + 1]], S[n], d["S0"][n], 0.25, dtype, is_chunked(dtype))
        else:
            assert torch.equal(S[n].cpu(), d["S0"][n])
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_nobody(dtype):
    # rows before the first sequence and after the last hold NaN: they are neither read into a
    # sequence's results nor written
    T, lo, hi = 260, 30, 201
    d = draw((T,), 1, 2, 128, 64, dtype, seed=11)
    for n in ("q", "k", "v", "g", "beta"):
        d[n][:lo] = float("nan")
        d[n][hi:] = float("nan")
    o = torch.full((T, 2, 64), 7.0, dtype=dtype, device="cuda")
    cu = torch.tensor([lo, 100, hi], dtype=torch.int32).cuda()
    o, S = run(d, cu_seqlens=cu, o=o)
    for n, (a, b) in enumerate([(lo, 100), (100, hi)]):
        check_sequence(d, slice(a, b), o[a:b], S[n], None, 1.0, dtype, is_chunked(dtype))
    assert torch.all(o[:lo] == 7) and torch.all(o[hi:] == 7)
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("offsets", [[0, 20, 10, 30], [0, 10, 40], [-5, 10, 30]])
def test_bad_offsets_are_reported(offsets, dtype):
    d = draw((30,), 1, 1, 64, 64, dtype, seed=12)
    run(d, cu_seqlens=torch.tensor(offsets, dtype=torch.int32).cuda())
    assert g.gdn2_device_status() == GDN2_ERR_SHAPE
    assert g.gdn2_device_status() == 0


def test_empty_batches():
    for dtype in (BF, F32):
        d = draw((2, 0), 1, 2, 64, 64, dtype, seed=13, n=2, state=True)
        o, S = run(d)
        assert o.shape == (2, 0, 2, 64) and torch.equal(S.cpu(), d["S0"])
        d = draw((0,), 1, 2, 64, 64, dtype, seed=14, n=3, state=True)
        o, S = run(d, cu_seqlens=torch.zeros(4, dtype=torch.int32, device="cuda"))
        assert torch.equal(S.cpu(), d["S0"])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("B,Hk,Hv", [(1, 1, 1), (5, 2, 4), (33, 3, 3)])
@pytest.mark.parametrize("in_place", [True, False])
def test_decode_step(B, Hk, Hv, dk, dv, dtype, in_place):
    d = draw((B, 1), Hk, Hv, dk, dv, dtype, seed=B + dk, n=B, state=True)
    d["g"][0, 0, 0] = -float("inf")
    a = {n: t.cuda() for n, t in d.items()}
    q, k, v, gg, beta = (a[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta"))
    S = a["S0"]
    out = None if in_place else torch.empty_like(S)
    o = g.gdn2_gdr_decode_step(q, k, v, gg, beta, S, S_out=out, scale=0.3)
    torch.cuda.synchronize()
    if not in_place:
        assert torch.equal(S.cpu(), d["S0"])
    for n in range(B):
        check_sequence(d, n, o[n:n + 1], (S if in_place else out)[n], d["S0"][n], 0.3, dtype, False)


def test_prompt_then_steps_equal_the_prompt():
    # serving: a prompt, then token by token, against the whole prompt at once (each within its
    # own tolerance of the fp64 recurrence)
    T, P = 150, 101
    d = draw((3, T), 2, 4, 128, 128, BF, seed=15, n=3, state=True)
    head = {n: (t if n == "S0" else t[:, :P].contiguous()) for n, t in d.items()}
    o, S = run(head)
    outs = [o]
    a = {n: t.cuda() for n, t in d.items()}
    for t in range(P, T):
        x = [a[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")]
        outs.append(g.gdn2_gdr_decode_step(*x, S)[:, None])
    torch.cuda.synchronize()
    o = torch.cat(outs, 1)
    for n in range(3):
        check_sequence(d, n, o[n], S[n], d["S0"][n], 1.0, BF, True)


def test_streams_and_captured_graphs():
    d = {n: _cuda(t) for n, t in draw((2, 140), 2, 2, 128, 128, BF, seed=16, n=2, state=True).items()}
    args = [d[n] for n in ("q", "k", "v", "g", "beta", "S0")]
    ref = g.gdn2_gdr_chunk_fwd(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = g.gdn2_gdr_chunk_fwd(*args, stream=side)
    side.synchronize()
    assert torch.equal(ref[0], other[0]) and torch.equal(ref[1], other[1])
    o, S = torch.zeros_like(ref[0]), torch.zeros_like(ref[1])
    step = [d[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        g.gdn2_gdr_chunk_fwd(*args, o=o, S_T=S)
        o1 = g.gdn2_gdr_decode_step(*step, S)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref[0])
        S_ref = ref[1].clone()
        assert torch.equal(o1, g.gdn2_gdr_decode_step(*step, S_ref)) and torch.equal(S, S_ref)


def test_channelwise_rule_with_collapsed_gates_agrees():
    # the channel-wise mixer with b = w = beta and a scalar decay is the same rule; its own
    # tolerance (2e-2 of the RMS) holds between the two
    d = draw((1, 200), 2, 2, 128, 128, BF, seed=17)
    d["beta"] = d["beta"].to(BF).float()
    o, S = run(d)
    a = {n: _cuda(t) for n, t in d.items()}
    wide = a["beta"][..., None].expand(1, 200, 2, 128).to(BF).contiguous()
    la = a["g"][..., None].expand(1, 200, 2, 128).contiguous()
    o2, S2 = g.gdn2_chunk_fwd(a["q"], a["k"], a["v"], la, wide, wide)
    torch.cuda.synchronize()
    for x, y in ((o.float(), o2), (S, S2)):
        # 2e-2 of the RMS for the channel-wise rule, half a bf16 step of the value for o
        assert torch.all((x - y).abs() <= 2e-2 * y.square().mean().sqrt() + 2.0 ** -7 * y.abs())


def segments_of(B, T, Hv, d, packed):
    """Segments of a sequence, from the workspace: 16 KB a chunk and value head, then states: 2 P - 3 and P a unit."""
    slots = T // 64 + B if packed else B * -(-T // 64)
    states = (g.lib().gdn2_gdr_chunk_fwd_workspace_bytes(B, T, Hv, d, d, int(packed), 1) - slots * Hv * 16 * 1024) // (B * Hv * d * d * 4)
    return (states + 3) // 3 if states else 1


@pytest.mark.parametrize("T,B,Hk,Hv,d,decay,beta_max,state,want", [
    (2560, 1, 1, 1, 128, 1 / 16, 1.0, True, True), (2561, 1, 1, 2, 64, 1 / 16, 2.0, False, True),
    (2500, 2, 1, 1, 128, 3.0, 1.0, True, False), (3000, 1, 1, 1, 64, 0.0, 1.0, True, True)])
def test_long_sequences_in_segments(T, B, Hk, Hv, d, decay, beta_max, state, want):
    x = draw((B, T), Hk, Hv, d, d, BF, seed=19 + T, decay=decay, beta_max=beta_max, n=B, state=state)
    P = segments_of(B, T, Hv, d, False)
    assert P > 1
    o, S = run(x, scale=0.5, want_state=want)
    assert (S is not None) == want
    for n in range(B):
        check_sequence(x, n, o[n], S[n] if want else None, x["S0"][n] if state else None, 0.5, BF, True, P)
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("lengths", [[2700, 0, 3, 1301, 4500], [1, 0, 6200]])
def test_packed_sequences_in_segments(lengths):
    # segments are the same part of every sequence, none of them where it is too short
    T, N = sum(lengths), len(lengths)
    d = draw((T + 70,), 1, 2, 64, 64, BF, seed=23 + N, n=N, state=True)
    at = np.concatenate([[0], np.cumsum(lengths)])
    P = segments_of(N, T + 70, 2, 64, True)
    assert P > 1
    for n in ("q", "k", "v", "g", "beta"):
        d[n][T:] = float("nan")
    S0 = _cuda(d["S0"])
    a = {n: _cuda(t) for n, t in d.items()}
    o = torch.full((T + 70, 2, 64), 7.0, dtype=BF, device="cuda")
    g.gdn2_gdr_chunk_fwd(a["q"], a["k"], a["v"], a["g"], a["beta"], S0, cu_seqlens=torch.tensor(at, dtype=torch.int32).cuda(), S_T=S0, o=o)
    torch.cuda.synchronize()
    for n in range(N):
        if lengths[n]:
            check_sequence(d, slice(at[n], at[n + 1]), o[at[n]:at[n + 1]], S0[n], d["S0"][n], 1.0, BF, True, P)
        else:
            assert torch.equal(S0[n].cpu(), d["S0"][n])
    assert torch.all(o[T:] == 7)
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("dim", [64, 128])
def test_packed_sequences_that_end_before_their_last_segment(dim):
    # 1 to 9 chunks, the last one ragged, among long ones: the segment that ends such a sequence may be
    # any of them, and those after it are empty
    lengths = [5000] + [64 * n - 7 for n in range(1, 10)] + [5000, 4990]
    T, N = sum(lengths), len(lengths)
    d = draw((T,), 1, 1, dim, dim, BF, seed=37, n=N, state=True)
    at = np.concatenate([[0], np.cumsum(lengths)])
    P = segments_of(N, T, 1, dim, True)
    ends = {(-(-n // 64) - 1) // -(-(-(-n // 64)) // P) for n in lengths}  # segments that sequences end in
    assert P >= 4 and ends & set(range(1, P - 1))
    o, S = run(d, cu_seqlens=torch.tensor(at, dtype=torch.int32).cuda())
    for n in range(N):
        check_sequence(d, slice(at[n], at[n + 1]), o[at[n]:at[n + 1]], S[n], d["S0"][n], 1.0, BF, True, P)
    assert g.gdn2_device_status() == 0


@pytest.mark.parametrize("lengths", [None, [2700, 0, 3, 1301, 4500]])
def test_segments_with_the_states_in_place(lengths):
    # a sequence's last segment writes the state over the one its first segment starts from
    N, T = (3, 2600) if lengths is None else (len(lengths), sum(lengths))
    d = draw((N, T) if lengths is None else (T,), 1, 2, 128, 128, BF, seed=29, n=N, state=True)
    assert segments_of(N, T, 2, 128, lengths is not None) > 1
    a = {n: _cuda(t) for n, t in d.items()}
    kw = {} if lengths is None else dict(cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda())
    x = [a[n] for n in ("q", "k", "v", "g", "beta")]
    o, S = g.gdn2_gdr_chunk_fwd(*x, a["S0"], **kw)
    for _ in range(5):
        S1 = a["S0"].clone()
        o1, _ = g.gdn2_gdr_chunk_fwd(*x, S1, S_T=S1, **kw)
        assert torch.equal(o, o1) and torch.equal(S, S1)


def test_many_units_and_a_long_sequence_sampled():
    d = draw((2, 2100), 8, 16, 128, 128, BF, seed=18, decay=1 / 8)
    o, S = run(d)
    for n, h in ((0, 0), (1, 15), (0, 9)):
        one = {m: (None if t is None else t[:, :, h // 2:h // 2 + 1] if m in ("q", "k") else t[:, :, h:h + 1]) for m, t in d.items()}
        check_sequence(one, n, o[n][:, h:h + 1], S[n][h:h + 1], None, 1.0, BF, True)
