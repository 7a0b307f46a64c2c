"""How far the scalar-gate prompt's outputs and states may be off for bf16 inputs, in the 2-norm: random,
correlated and repeated keys, write strengths up to 2, one chunk and many, segments.

The tolerance is the error that the arithmetic makes by itself.  S, R, U, T and P are fp32 values that
enter the tensor cores in two bf16 parts: off by w = 2^-16 of the value at most, and a product of two such
operands drops that of both second parts, another w.  (The blocked solve's tf32 products are off by
2^-21 of A, the state's fp32 sum by 2^-24.)  Roundings of different values are independent, so their squares add.  Over
a chunk with T = (I + A)^-1 diag(beta), R = -e^G K S, U = T (V + R) and ^2 element by element, the mean squares are

    R: w^2 ((e^G)^2 K^2 S^2 + R^2)
    U: T^2 R: + w^2 T^2 (V^2 + 2 R^2) + (T1^2 (2^-21 A)^2 T^2) (V^2 + R^2),      T1 = (I + A)^-1
    S: K^T diag over the tokens of (e^(G_C - G))^2 (U: + w^2 U^2) K + 2^-48 S^2      (a covariance over the key axis)
    O: (e^G)^2 Q^2 w^2 S^2 + P^2 (U: + 3 w^2 U^2),

and what the state was off before the chunk goes through it by the chunk's own matrices: S by
e^(G_C) I - K^T e^(G_C - G) T e^G K, O by e^G Q - P T e^G K.  A segment's first state is M S + N, whose errors are
those of M, each column as large as the row of S that it meets, of N, and of S through M.  The largest
error of a rounding stands for its root mean square, which is a sixth of it for two bf16 parts: what is
left over is the room between the expected error and the tolerance.  (One key without decay and with
one strength has the same T in every chunk: its errors add up themselves over the chunks, not their squares.)

o is rounded to bf16 at the end: what counts is by how much it is further from the definition
than half a step."""
import numpy as np
import pytest
import torch

import gated_delta_rule_95_b200 as g
from oracle import layer
from tests.test_gpu_gdr import segments_of

pytestmark = pytest.mark.gpu
W = 2.0 ** -16
BF, F32 = torch.bfloat16, torch.float32


def chunk(q, k, v, gg, beta, S, cov, weight):
    """One chunk of one head from the state S [dk, n], whose error has the covariance cov [dk, dk] (summed over the
    columns, column j counted weight[j] times): the matrices through S and O, the covariance after it and
    the outputs' mean squares (scale 1)."""
    n, sq = len(q), np.square
    G = np.cumsum(np.maximum(gg, -1e4))
    D = np.exp(np.minimum(G[:, None] - G[None], 0.0)) * np.tril(np.ones((n, n)))
    A = np.tril(beta[:, None] * D * (k @ k.T), -1)
    T1 = np.linalg.inv(np.eye(n) + A)
    T, P = T1 * beta, D * (q @ k.T)
    eG, eE = np.exp(G)[:, None], np.exp(G[-1] - G)[:, None]
    R = -eG * (k @ S)
    U = T @ (v + R)
    R2 = W ** 2 * (sq(eG) * (sq(k) @ sq(S)) + sq(R))
    U2 = sq(T) @ (R2 + W ** 2 * (sq(v) + 2 * sq(R))) + sq(T1) @ sq(2.0 ** -21 * A) @ sq(T) @ (sq(v) + sq(R))
    through_S = eG[-1] * np.eye(k.shape[1]) - (k * eE).T @ T @ (eG * k)
    through_O = eG * q - P @ T @ (eG * k)
    after = through_S @ cov @ through_S.T + (k * sq(eE) * ((U2 + W ** 2 * sq(U)) @ weight)[:, None]).T @ k
    after = after + np.diag(2.0 ** -48 * (sq(S) @ weight))
    O2 = (sq(eG) * (sq(q) @ sq(S)) * W ** 2 + sq(P) @ (U2 + 3 * W ** 2 * sq(U))) @ weight
    return after, O2 + np.einsum("td,de,te->t", through_O, cov, through_O)


def predicted(q, k, v, gg, beta, S0, scale, segments=1):
    """One head's o, S in fp64 and the mean squares of their errors, over o and over S: q, k [T, dk], v [T, dv]."""
    T, dk = k.shape

    def run(lo, hi, S, cov, v, weight, o=None):
        off = 0.0
        for a in range(lo, hi, 64):
            c = slice(a, min(hi, a + 64))
            cov, O2 = chunk(q[c], k[c], v[c], gg[c], beta[c], S, cov, weight)
            out, S = layer.gdr_forward(q[c, None], k[c, None], v[c, None], gg[c, None], beta[c, None], S[None], scale)
            S = S[0]
            if o is not None:
                o[c] = out[:, 0]
            off += scale ** 2 * O2.sum()
        return S, cov, off
    S, cov = (np.zeros((dk, v.shape[1])) if S0 is None else S0), np.zeros((dk, dk))
    per = -(-(-(-T // 64)) // segments) * 64
    o, off, one = np.zeros(v.shape), 0.0, np.ones(v.shape[1])
    for s in range(segments):
        lo, hi = min(T, s * per), min(T, (s + 1) * per)
        if lo == hi:
            break
        S1, cov1, add = run(lo, hi, S, cov, v, one, o)
        off += add
        if s and hi < T:  # the next segment starts from M S + N
            M, cov_M, _ = run(lo, hi, np.eye(dk), np.zeros((dk, dk)), np.zeros((T, dk)), np.square(S).sum(1))
            _, cov_N, _ = run(lo, hi, np.zeros_like(S), np.zeros((dk, dk)), v, one)
            cov1 = cov_M + cov_N + M @ cov @ M.T
        S, cov = S1, cov1
    return o, S, off, np.trace(cov)


def excess(o, ref):
    """By how much o is further from ref than half a step of bf16 at ref."""
    half = np.exp2(np.floor(np.log2(np.maximum(np.abs(ref), 1e-30))) - 8)
    return np.maximum(np.abs(o - ref) - half, 0.0)


def draw(T, kind, decay, strength, seed, dk=128, dv=128, heads=2, state=True, even=False):
    """One key head; queries and keys of norm 1 at most.  kind: random; correlated (a common direction and 0.3 of
    noise in each channel, queries like the keys); the same key all over."""
    rng = np.random.default_rng(seed)

    def unit(common):
        x = rng.standard_normal((T, dk))
        x = 0.3 * x + rng.standard_normal(dk) if common else x
        return x / np.linalg.norm(x, axis=-1, keepdims=True) * (1 - 2 ** -7)
    k = unit(kind == "correlated")
    k = np.broadcast_to(k[:1], k.shape) if kind == "same" else k
    q = unit(False) if kind == "random" else k
    d = {n: torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(BF).reshape(1, T, 1, dk) for n, x in (("q", q), ("k", k))}
    d["v"] = torch.from_numpy(rng.standard_normal((1, T, heads, dv)).astype(np.float32)).to(BF)
    d["g"] = torch.from_numpy((-np.logaddexp(0, rng.standard_normal((1, T, heads))) * decay).astype(np.float32))
    beta = np.full((1, T, heads), strength) if even else strength / (1 + np.exp(-rng.standard_normal((1, T, heads))))
    d["beta"] = torch.from_numpy(beta.astype(np.float32))
    d["S0"] = torch.from_numpy((0.1 * rng.standard_normal((1, heads, dk, dv))).astype(np.float32)) if state else None
    return d


def errors(d, o, S, scale, segments=1):
    """Over all heads: (o's excess, its tolerance, |o|), (S's error, its tolerance, |S|) in the 2-norm."""
    f = {n: None if t is None else t.double().numpy()[0] for n, t in d.items()}
    sums = np.zeros(6)
    for h in range(f["v"].shape[1]):
        S0 = None if f["S0"] is None else f["S0"][h]
        o_ref, S_ref, o2, S2 = predicted(f["q"][:, 0], f["k"][:, 0], f["v"][:, h], f["g"][:, h], f["beta"][:, h], S0, scale, segments)
        sums += [np.square(excess(o[0, :, h], o_ref)).sum(), o2, np.square(o_ref).sum(), np.square(S[0, h] - S_ref).sum(), S2, np.square(S_ref).sum()]
    return np.sqrt(sums)


def check(d, scale=1.0, segments=1, times=1.0):
    """times: of the tolerances."""
    x = {n: None if t is None else t.cuda() for n, t in d.items()}
    o, S = g.gdn2_gdr_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["S0"], scale=scale)
    torch.cuda.synchronize()
    e = errors(d, o.cpu().double().numpy(), S.cpu().double().numpy(), scale, segments)
    e[[1, 4]] *= times
    assert e[0] <= e[1] and e[3] <= e[4], dict(zip(("o past rounding", "its tolerance", "|o|", "S", "its tolerance", "|S|"), e))
    assert g.gdn2_device_status() == 0


KEYS = [("random", 1 / 16, 1.0, False), ("random", 0.0, 1.0, False), ("random", 3.0, 1.0, False), ("random", 1 / 16, 2.0, False),
        ("random", 0.0, 1.99, True), ("correlated", 1 / 16, 1.0, False), ("correlated", 0.0, 1.0, False),
        ("correlated", 1 / 16, 1.5, False), ("correlated", 0.0, 1.99, True), ("same", 0.0, 1.0, True),
        ("same", 1 / 16, 1.99, True), ("same", 0.0, 1.99, True)]


@pytest.mark.parametrize("T,state", [(64, False), (64, True), (330, True), (1500, True)])
@pytest.mark.parametrize("kind,decay,strength,even", KEYS)
def test_outputs_and_states(kind, decay, strength, even, T, state):
    times = (-(-T // 64)) ** 0.5 if kind == "same" and decay == 0 else 1.0
    check(draw(T, kind, decay, strength, 50 + T, state=state, even=even), scale=0.5, times=times)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("kind", ["random", "correlated"])
def test_head_sizes(kind, dk, dv):
    check(draw(330, kind, 1 / 16, 1.0, 60, dk, dv), scale=0.5)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kind,decay,strength", [("random", 1 / 16, 1.0), ("random", 0.0, 2.0), ("correlated", 1 / 16, 1.5)])
def test_segments(kind, decay, strength, dim):
    T = 2600
    P = segments_of(1, T, 1, dim, False)
    assert P > 1
    check(draw(T, kind, decay, strength, 70, dim, dim, heads=1), segments=P)
