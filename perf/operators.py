"""Performance cases of the Gated DeltaNet layer's operators.

Five operators that a layer built on this library runs next to the channel-wise mixer:

* ``gdr_chunk``: the gated delta rule with one decay and one write strength per token and
  head (the scalar-gate form of the mixer), chunked over a prompt or a packed batch;
* ``gdr_decode``: the same rule for one new token per sequence, state updated;
* ``norm_fwd``, ``norm_bwd``: layer norm over the residual sum, and its gradients with the
  reduction of the weight's and the bias's;
* ``conv_bwd``: the gradients of the 4-tap short convolution.

A case is a dict of plain values; ``run`` computes it in elementary torch operations, or
with this library's kernels when ``own`` is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64
TAPS = 4
EPS = 1e-5

# ------------------------------------------------------------------------------- cases


def _gdr(B, T, Hk, Hv, dk, dv, dtype, packed=False, state=False, heavy=False):
    return dict(op="gdr_chunk", B=B, T=T, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype, packed=packed, state=state,
                heavy=heavy)


def _step(B, Hk, Hv, dk, dv, dtype):
    return dict(op="gdr_decode", B=B, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype=dtype)


def _norm(op, rows, cols, dtype, residual, bias):
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=residual, bias=bias)


def _conv(B, T, C, dtype, packed, bias):
    return dict(op="conv_bwd", B=B, T=T, C=C, dtype=dtype, packed=packed, bias=bias)


def listed():
    return [
        # a prefill batch at the 1.3B layer's shape: the ordinary case of the chunked form
        dict(_gdr(8, 4096, 16, 16, 128, 128, "bf16"), name="prefill_b8_h16_t4096"),
        # one long document, few heads: the longest chain of chunks, with the heavy-tailed decay
        dict(_gdr(1, 65536, 16, 16, 128, 128, "bf16", heavy=True), name="long_b1_h16_t65536"),
        # a serving batch of ragged prompts, each continuing from its state, four value heads
        # to a key head
        dict(_gdr(24, 2048, 4, 16, 128, 128, "bf16", packed=True, state=True), name="packed_n24_h16"),
        # one short prompt of one fp32 head: latency
        dict(_gdr(1, 256, 1, 1, 64, 64, "f32"), name="tiny_f32"),
        # decode at full batch: the state streams once
        dict(_step(256, 16, 16, 128, 128, "bf16"), name="decode_b256_h16"),
        # decode of a few sequences, uneven head sizes, fp32: latency
        dict(_step(3, 2, 4, 64, 128, "f32"), name="decode_b3_h4_f32"),
        # the norm after the mixer over the prefill batch, with the residual sum
        dict(_norm("norm_fwd", 32768, 2048, "bf16", True, True), name="norm_fwd_32768x2048"),
        # the same norm over one decode step's tokens: latency
        dict(_norm("norm_fwd", 256, 2048, "bf16", True, True), name="norm_fwd_256x2048"),
        # its gradients over the training batch, with the gradient of the residual stream
        dict(_norm("norm_bwd", 32768, 2048, "bf16", True, True), name="norm_bwd_32768x2048"),
        # an odd, unaligned width in fp32
        dict(_norm("norm_bwd", 1031, 1001, "f32", False, False), name="norm_bwd_1031x1001_f32"),
        # gradients of the convolution over the value projection of the training batch
        dict(_conv(8, 4096, 2048, "bf16", False, True), name="conv_bwd_b8_t4096_c2048"),
        # a packed ragged batch with carried history, fp32
        dict(_conv(24, 1000, 1000, "f32", True, False), name="conv_bwd_n24_c1000_f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["gdr_chunk", "gdr_chunk", "gdr_decode", "norm_fwd", "norm_bwd", "conv_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "gdr_chunk":
        Hk, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 4])
        B, T = _log(rng, 1, 24), _log(rng, 1, 8192)
        while B * T * Hk * group > (1 << 19 if dtype == "bf16" else 1 << 17):  # half the ordinary case at most
            T = max(1, T // 2)
        return _gdr(B, T, Hk, Hk * group, rng.choice([64, 128]), rng.choice([64, 128]), dtype, rng.random() < 0.4,
                    rng.random() < 0.5, rng.random() < 0.3)
    if op == "gdr_decode":
        Hk, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2])
        return _step(_log(rng, 1, 128), Hk, Hk * group, rng.choice([64, 128]), rng.choice([64, 128]), dtype)
    if op == "conv_bwd":
        B, T, C = _log(rng, 1, 24), _log(rng, 1, 4096), 8 * _log(rng, 1, 512)
        while B * T * C > 1 << 25:
            T = max(1, T // 2)
        return _conv(B, T, C, dtype, rng.random() < 0.5, rng.random() < 0.5)
    rows, cols = _log(rng, 1, 32768), _log(rng, 1, 8192)
    if rng.random() < 0.5:
        cols = 8 * ((cols + 7) // 8)
    while rows * cols > 1 << 25:
        rows = max(1, rows // 2)
    return _norm(op, rows, cols, dtype, rng.random() < 0.6, rng.random() < 0.6)


def _lengths(case):
    """Sequence lengths of a packed batch: log-uniform in [1, T], the first one T."""
    r = random.Random(1000003 * case["B"] + case["T"])
    return [case["T"]] + [_log(r, 1, case["T"]) for _ in range(case["B"] - 1)]


# ------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    def unit(*shape):
        return torch.nn.functional.normalize(torch.randn(*shape, generator=gen, device="cuda"), dim=-1).to(dt)

    s = dict(case=dict(case))
    op = case["op"]
    if op in ("gdr_chunk", "gdr_decode"):
        B, Hk, Hv, dk, dv = (case[n] for n in ("B", "Hk", "Hv", "dk", "dv"))
        if op == "gdr_decode":
            lead = (B,)
        elif case["packed"]:
            lens = _lengths(case)
            lead = (sum(lens),)
            s["cu"] = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
            s["lens"] = lens
        else:
            lead = (B, case["T"])
        s["q"], s["k"], s["v"] = unit(*lead, Hk, dk), unit(*lead, Hk, dk), normal(*lead, Hv, dv, dtype=dt)
        x = normal(*lead, Hv)
        s["g"] = -torch.nn.functional.softplus(2 * x) / 8 if case.get("heavy") else -torch.nn.functional.softplus(x) / 16
        s["beta"] = torch.sigmoid(normal(*lead, Hv))
        s["scale"] = dk ** -0.5
        std = 0.02 if op == "gdr_decode" else 0.05
        s["S"] = normal(B, Hv, dk, dv, std=std) if op == "gdr_decode" or case["state"] else None
    elif op == "conv_bwd":
        B, T, C = case["B"], case["T"], case["C"]
        if case["packed"]:
            lens = _lengths(case)
            lead = (sum(lens),)
            s["cu"] = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
            s["lens"] = lens
            s["hist"], s["dhist_out"] = normal(B, 3, C, dtype=dt), normal(B, 3, C, dtype=dt)
        else:
            lead = (B, T)
        s["x"], s["dy"] = normal(*lead, C, dtype=dt), normal(*lead, C, dtype=dt)
        s["weight"] = normal(C, TAPS, std=0.5)
    else:
        rows, cols = case["rows"], case["cols"]
        s["x"] = normal(rows, cols, dtype=dt)
        s["weight"] = 1.0 + normal(cols, std=0.1)
        if op == "norm_fwd":
            s["residual"] = normal(rows, cols, dtype=dt) if case["residual"] else None
            s["bias"] = normal(cols, std=0.1) if case["bias"] else None
        else:
            xd = s["x"].double()
            mean = xd.mean(-1)
            s["mean"] = mean.float()
            s["rstd"] = ((xd - mean[:, None]).square().mean(-1) + EPS).rsqrt().float()
            s["dy"] = normal(rows, cols, dtype=dt)
            s["ds"] = normal(rows, cols, dtype=dt) if case["residual"] else None
    return s


# ---------------------------------------------------------------------- the plain forms


def _pad(x, s):
    """Packed [tokens, ...] to [sequences, longest, ...] (zeros after each sequence's end)."""
    at = torch.arange(max(s["lens"]), device=x.device)
    idx = (s["cu"][:-1, None].long() + at).clamp(max=x.shape[0] - 1)
    keep = at < s["cu"].diff()[:, None]
    return torch.where(keep.reshape(*keep.shape, *[1] * (x.dim() - 1)), x[idx], torch.zeros((), dtype=x.dtype, device=x.device))


def _unpad(x, s):
    """The reverse of _pad."""
    total = sum(s["lens"])
    seq = torch.repeat_interleave(s["cu"].diff().long(), output_size=total)
    return x[seq, torch.arange(total, device=x.device) - s["cu"].long()[seq]]


def _gdr_chunk(s):
    c = s["case"]
    q, k, v, g, beta = (s[n] for n in ("q", "k", "v", "g", "beta"))
    if c["packed"]:
        q, k, v, g, beta = (_pad(x, s) for x in (q, k, v, g, beta))
    N, T, Hv, dv = v.shape
    dk, group, dt = q.shape[-1], c["Hv"] // c["Hk"], q.dtype
    nc = -(-T // CHUNK)

    def chunks(x):  # [N, T, H, D] -> [N, H, chunks, CHUNK, D] in fp32, zeros after the end
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, nc * CHUNK - T))
        return x.reshape(N, nc, CHUNK, x.shape[2], -1).permute(0, 3, 1, 2, 4)

    q, k = (chunks(x).repeat_interleave(group, 1) for x in (q, k))
    v, beta = chunks(v), chunks(beta[..., None])
    G = chunks(g[..., None])[..., 0].double().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    D = torch.where(low, (G[..., :, None] - G[..., None, :]).clamp(max=0).exp(), 0.0).float()
    eG, eE = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None]
    P = (q @ k.transpose(-1, -2)) * D
    X = torch.eye(CHUNK, device=q.device) - ((k @ k.transpose(-1, -2)) * D * beta).tril(-1)
    for i in range(2, CHUNK):  # forward substitution of (I + A)^-1, a row at a time
        row = X[..., i, :i].clone()
        X[..., i, :i] = row + (row[..., None, :] @ (X[..., :i, :i] - torch.eye(i, device=q.device)))[..., 0, :]
    U, W = X @ (beta * v), X @ (beta * eG * k)
    qe, ke, end = q * eG, (k * eE).transpose(-1, -2), G[..., -1].exp().float()
    S = torch.zeros(N, Hv, dk, dv, device=q.device) if s["S"] is None else s["S"]
    o = torch.empty_like(v)
    for i in range(nc):  # the state's way through the chunks
        u = U[:, :, i] - W[:, :, i] @ S
        o[:, :, i] = qe[:, :, i] @ S + P[:, :, i] @ u
        S = end[:, :, i, None, None] * S + ke[:, :, i] @ u
    o = (o * s["scale"]).permute(0, 2, 3, 1, 4).reshape(N, nc * CHUNK, Hv, dv)[:, :T]
    return (_unpad(o, s) if c["packed"] else o).to(dt), S


def _gdr_decode(s):
    c, dt = s["case"], s["q"].dtype
    group = c["Hv"] // c["Hk"]
    q, k = (s[n].float().repeat_interleave(group, 1) for n in ("q", "k"))
    S = s["S"] * s["g"].exp()[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (k[..., None, :] @ S)[..., 0, :])
    S = S + k[..., None] * u[..., None, :]
    return ((q[..., None, :] @ S)[..., 0, :] * s["scale"]).to(dt), S


def _norm_fwd(s):
    dt = s["x"].dtype
    x = s["x"].float()
    if s["residual"] is not None:
        x = (x + s["residual"].float()).to(dt).float()
    mean = x.mean(-1)
    d = x - mean[:, None]
    rstd = (d.square().mean(-1) + EPS).rsqrt()
    y = d * rstd[:, None] * s["weight"]
    y = y if s["bias"] is None else y + s["bias"]
    return y.to(dt), x.to(dt) if s["residual"] is not None else None, mean, rstd


def _norm_bwd(s):
    dt = s["x"].dtype
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    h = dy * s["weight"]
    dx = (h - h.mean(-1, keepdim=True) - xhat * (h * xhat).mean(-1, keepdim=True)) * s["rstd"][:, None]
    dx = dx if s["ds"] is None else dx + s["ds"].float()
    return dx.to(dt), (dy * xhat).sum(0), dy.sum(0) if s["case"]["bias"] else None


def _conv_bwd(s):
    dt, C = s["x"].dtype, s["case"]["C"]
    x, dy = s["x"].float(), s["dy"].float()
    if s["case"]["packed"]:
        x, dy = _pad(x, s), _pad(dy, s)
    N, T, _ = x.shape
    hist = torch.zeros(N, 3, C, device=x.device) if s.get("hist") is None else s["hist"].float()
    xp = torch.cat([hist, x], 1)  # [history | tokens]
    dxp = torch.zeros_like(xp)
    dw = []
    for j in range(TAPS):
        dw.append((dy * xp[:, j:j + T]).sum((0, 1)))
        dxp[:, j:j + T] += dy * s["weight"][:, j]
    if s.get("dhist_out") is not None:  # the last three inputs were handed on
        lens = torch.full((N,), T, device=x.device) if not s["case"]["packed"] else s["cu"].diff().long()
        at = (lens[:, None] + torch.arange(3, device=x.device))[..., None].expand(N, 3, C)
        dxp = dxp.scatter_add(1, at, s["dhist_out"].float())
    dx = dxp[:, 3:]
    dx = _unpad(dx, s) if s["case"]["packed"] else dx
    return (dx.to(dt), torch.stack(dw, -1), dy.sum((0, 1)) if s["case"]["bias"] else None,
            None if s.get("hist") is None else dxp[:, :3].to(dt))


def run(state):
    op = state["case"]["op"]
    if own:
        import gated_delta_rule_95_b200 as g
        if op == "gdr_chunk":
            return g.gdn2_gdr_chunk_fwd(state["q"], state["k"], state["v"], state["g"], state["beta"], state["S"],
                                        scale=state["scale"], cu_seqlens=state.get("cu"))
        if op == "gdr_decode":
            S = torch.empty_like(state["S"])  # the new state beside the old one, as a server that may roll back keeps it
            o = g.gdn2_gdr_decode_step(state["q"], state["k"], state["v"], state["g"], state["beta"], state["S"],
                                       S_out=S, scale=state["scale"])
            return o, S
        if op == "norm_fwd":
            return g.gdn2_layer_norm_fwd(state["x"], state["weight"], state["bias"], state["residual"], eps=EPS)
        if op == "norm_bwd":
            r = g.gdn2_layer_norm_bwd(state["dy"], state["x"], state["weight"], state["mean"], state["rstd"],
                                      state["ds"], want_dbias=state["case"]["bias"])
            return r["dx"], r["dweight"], r["dbias"]
        r = g.gdn2_short_conv_bwd(state["dy"], state["x"], state["weight"], cu_seqlens=state.get("cu"),
                                  hist=state.get("hist"), dhist_out=state.get("dhist_out"),
                                  want_dbias=state["case"]["bias"])
        return r["dx"], r["dweight"], r["dbias"], r["dhist"]
    return {"gdr_chunk": _gdr_chunk, "gdr_decode": _gdr_decode, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd,
            "conv_bwd": _conv_bwd}[op](state)


# --------------------------------------------------------- what a pass cannot do without


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("gdr_chunk", "gdr_decode"):
        B, Hk, Hv, dk, dv = (case[n] for n in ("B", "Hk", "Hv", "dk", "dv"))
        n = B if op == "gdr_decode" else sum(_lengths(case)) if case["packed"] else B * case["T"]
        states = 2 if op == "gdr_decode" or case["state"] else 1
        return {"bytes": n * (2 * Hk * dk * e + 2 * Hv * dv * e + 8 * Hv) + 4 * states * B * Hv * dk * dv,
                "flops": 7 * n * Hv * dk * dv}
    if op == "conv_bwd":
        C = case["C"]
        n = sum(_lengths(case)) if case["packed"] else case["B"] * case["T"]
        extra = case["B"] * 3 * C * 3 * e if case["packed"] else 0
        return {"bytes": 3 * n * C * e + extra + 2 * 4 * TAPS * C + (4 * C if case["bias"] else 0), "flops": 17 * n * C}
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if op == "norm_fwd":
        return {"bytes": (4 if case["residual"] else 2) * n * e + 8 * rows + 4 * cols * (2 if case["bias"] else 1),
                "flops": 8 * n}
    return {"bytes": (4 if case["residual"] else 3) * n * e + 8 * rows + 4 * cols * (3 if case["bias"] else 2),
            "flops": 14 * n}


# --------------------------------------------------------------- the definitions, 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = {n: x.double() for n, x in s.items() if isinstance(x, torch.Tensor) and x.is_floating_point()}
    if op in ("gdr_chunk", "gdr_decode"):
        # the recurrence itself, a token at a time: S <- exp(g) S, S <- S + k (beta (v - S^T k))^T
        group = case["Hv"] // case["Hk"]
        q, k = (f[n].repeat_interleave(group, -2) for n in ("q", "k"))
        v, g, beta = f["v"], f["g"], f["beta"]
        S = f["S"].clone() if "S" in f else torch.zeros(case["B"], case["Hv"], case["dk"], case["dv"],
                                                        dtype=torch.float64, device="cuda")
        if op == "gdr_decode":
            q, k, v, g, beta = (x[:, None] for x in (q, k, v, g, beta))
        lens = s["lens"] if case.get("packed") else [1 if op == "gdr_decode" else case["T"]] * case["B"]
        order = sorted(range(case["B"]), key=lambda n: -lens[n])  # the longest first: the ones alive are a prefix
        at = torch.tensor(order, device="cuda")
        first = s["cu"][at].long() if case.get("packed") else None
        S = S[at]
        o = torch.empty_like(v)
        for t in range(max(lens)):
            alive = sum(1 for n in lens if n > t) if case.get("packed") else case["B"]
            rows = (first[:alive] + t) if first is not None else (at[:alive], t)
            St = S[:alive] * g[rows].exp()[..., None, None]
            kt = k[rows]
            u = beta[rows][..., None] * (v[rows] - torch.einsum("nhk,nhkv->nhv", kt, St))
            St = St + kt[..., None] * u[..., None, :]
            o[rows] = s["scale"] * torch.einsum("nhk,nhkv->nhv", q[rows], St)
            S = St if alive == case["B"] else torch.cat([St, S[alive:]])
        back = torch.empty_like(S)
        back[at] = S
        return (o[:, 0] if op == "gdr_decode" else o), back
    if op == "norm_fwd":
        x = f["x"]
        if s["residual"] is not None:
            x = (x + f["residual"]).to(s["x"].dtype).double()  # the sum as it is stored
        var, mean = torch.var_mean(x, -1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        y = torch.nn.functional.layer_norm(x, x.shape[-1:], f["weight"], f.get("bias"), EPS)
        return y, x if s["residual"] is not None else None, mean, rstd
    if op == "norm_bwd":  # reverse mode over the definition
        x, w = f["x"].requires_grad_(), f["weight"].requires_grad_()
        b = torch.zeros_like(w).requires_grad_()
        torch.nn.functional.layer_norm(x, x.shape[-1:], w, b, EPS).backward(f["dy"])
        dx = x.grad if s["ds"] is None else x.grad + f["ds"]
        return dx, w.grad, b.grad if case["bias"] else None
    B, C = case["B"], case["C"]
    lens = s["lens"] if case["packed"] else [case["T"]] * B
    x, w = f["x"].reshape(-1, C).requires_grad_(), f["weight"].requires_grad_()
    hist = (f["hist"] if "hist" in f else torch.zeros(B, 3, C, dtype=torch.float64, device="cuda")).requires_grad_()
    dy, first, loss, dbias = f["dy"].reshape(-1, C), 0, 0.0, 0.0
    for n, length in enumerate(lens):
        xs = torch.cat([hist[n], x[first:first + length]])
        y = sum(w[:, j] * xs[j:j + length] for j in range(TAPS))
        loss = loss + (y * dy[first:first + length]).sum()
        if "dhist_out" in f:
            loss = loss + (xs[length:] * f["dhist_out"][n]).sum()
        first += length
    loss.backward()
    return (x.grad.reshape(f["x"].shape), w.grad, dy.sum(0) if case["bias"] else None,
            hist.grad if s.get("hist") is not None else None)
