"""The measured cases of the gated delta rule (a prompt, a gradient, a
single-token step) and of the group norm with an activation (channels last,
over a sample's pixels or over each token by itself, and its gradient).

`run` computes them in plain torch operations (own = False) or through the
package (own = True); `exact` evaluates the definitions in 64 bits, the delta
rule token by token.
"""
import math

import torch

own = False

CHUNK = 64     # tokens whose scores the plain delta rule forms at once


def listed():
    return [
        # one prompt of ordinary length through a mixer with 32 value heads of 128 on 16 heads of keys
        {"name": "delta prompt bf16", "op": "delta", "dtype": "bf16", "N": 1, "L": 4096, "H": 32, "P": 128, "G": 16,
         "S": 128, "ragged": False, "state": False},
        # the largest: a long document through the same layer
        {"name": "delta long bf16", "op": "delta", "dtype": "bf16", "N": 1, "L": 16384, "H": 32, "P": 128, "G": 16,
         "S": 128, "ragged": False, "state": False},
        # a padded batch of prompts that continue cached states, smaller heads
        {"name": "delta ragged bf16", "op": "delta", "dtype": "bf16", "N": 6, "L": 1000, "H": 8, "P": 64, "G": 8,
         "S": 64, "ragged": True, "state": True},
        # full precision, heads and keys that fill no tile
        {"name": "delta odd f32", "op": "delta", "dtype": "f32", "N": 2, "L": 777, "H": 6, "P": 40, "G": 2, "S": 24,
         "ragged": False, "state": True},
        # one layer's mixer in a training step
        {"name": "delta gradient bf16", "op": "delta_grad", "dtype": "bf16", "N": 2, "L": 2048, "H": 16, "P": 128,
         "G": 16, "S": 128, "ragged": False, "state": False},
        # the gradient through a ragged batch and its states in full precision
        {"name": "delta gradient odd f32", "op": "delta_grad", "dtype": "f32", "N": 2, "L": 413, "H": 6, "P": 40,
         "G": 3, "S": 24, "ragged": True, "state": True},
        # the smallest: one token of one sequence
        {"name": "delta step one bf16", "op": "delta_step", "dtype": "bf16", "N": 1, "L": 1, "H": 32, "P": 128, "G": 16,
         "S": 128, "ragged": False, "state": True},
        # one token for each sequence of a full serving batch: the states' bytes
        {"name": "delta step batch bf16", "op": "delta_step", "dtype": "bf16", "N": 64, "L": 1, "H": 32, "P": 128,
         "G": 16, "S": 128, "ragged": False, "state": True},
        # behind a 2-D convolution of 4 x 64 channels on 56 x 56 pixels, groups of 8 channels
        {"name": "norm image bf16", "op": "norm", "dtype": "bf16", "N": 8, "L": 3136, "G": 32, "C": 8,
         "per_token": False, "act": "silu", "bias": True, "gated": False, "center": True, "ragged": False},
        # behind the audio frontend's first convolution in full precision, batch 1
        {"name": "norm audio f32", "op": "norm", "dtype": "f32", "N": 1, "L": 3000, "G": 8, "C": 48,
         "per_token": False, "act": "gelu", "bias": True, "gated": False, "center": True, "ragged": False},
        # behind the mixer: every head of every token by itself, without its mean, times a gate
        {"name": "norm gated heads bf16", "op": "norm", "dtype": "bf16", "N": 1, "L": 4096, "G": 32, "C": 128,
         "per_token": True, "act": "silu", "bias": False, "gated": True, "center": False, "ragged": False},
        # the image's norm in a training step
        {"name": "norm gradient bf16", "op": "norm_grad", "dtype": "bf16", "N": 8, "L": 3136, "G": 32, "C": 8,
         "per_token": False, "act": "silu", "bias": True, "gated": False, "center": True, "ragged": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "delta_grad", "delta_grad", "delta_step", "norm", "norm", "norm_grad",
                     "norm_grad"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "ragged": rng.random() < 0.4}
    if op.startswith("norm"):
        c.update(per_token=rng.random() < 0.4, act=rng.choice(["none", "silu", "silu", "gelu"]),
                 bias=rng.random() < 0.6, gated=rng.random() < 0.3, center=rng.random() < 0.7, N=_log(rng, 1, 16))
        c["G"] = rng.choice([1, 2, 4, 8, 16, 32, 32])
        c["C"] = rng.choice([3, 8, 12, 16, 24, 48, 64, 128])
        c["L"] = _log(rng, 1, max(1, min(8192, (1 << 24) // (c["N"] * c["G"] * c["C"]))))
        return c
    c["state"] = rng.random() < 0.5
    c["G"] = rng.choice([1, 1, 2, 4, 8])
    c.update(N=_log(rng, 1, 12), H=c["G"] * _log(rng, 1, 32 // c["G"]), P=rng.choice([16, 32, 40, 64, 64, 128, 128, 256]),
             S=rng.choice([16, 24, 64, 64, 96, 128, 128, 256]))
    most = (1 << 22) if op == "delta_grad" else (1 << 24)
    c["L"] = _log(rng, 1, max(1, min(8192, most // (c["N"] * c["H"] * max(c["P"], c["S"])))))
    if c["dtype"] == "f32":
        c["L"] = max(1, c["L"] // 4)
    if op == "delta_step":
        c.update(N=_log(rng, 1, 64), L=1, ragged=False, state=True)
    return c


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    t = _type(case)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=dev)
    uniform = lambda lo, hi, *shape: torch.rand(shape, generator=gen, device=dev) * (hi - lo) + lo
    N, L, G, op = case["N"], case["L"], case["G"], case["op"]
    s = {"case": case, "lengths": None, "state": None}
    if case["ragged"]:
        # some sequences full, some short, one cut off near the front
        n = torch.randint(0, L + 1, (N,), generator=gen, device=dev, dtype=torch.int32)
        n[0] = L
        s["lengths"] = n
    if op.startswith("norm"):
        C = case["C"]
        # what a layer hands on: channels of unequal size around means of their own
        s["x"] = (normal(N, L, G, C) * uniform(0.5, 2, G, C) + normal(G, C)).to(t)
        s["w"] = (1 + 0.1 * normal(G, C)).to(t)
        s["bias"] = (0.1 * normal(G, C)).to(t) if case["bias"] else None
        s["gate"] = normal(N, L, G, C).to(t) if case["gated"] else None
        if op == "norm_grad":
            s["dy"] = normal(N, L, G, C).to(t)
        if own:
            from convolution_forward_implicit_amd import GroupNorm
            s["plan"] = GroupNorm({"N": N, "L": L, "G": G, "C": C}, case["dtype"], act=case["act"],
                                  has_bias=case["bias"], gated=case["gated"], center=case["center"],
                                  per_token=case["per_token"])
        return s
    H, P, S = case["H"], case["P"], case["S"]
    lead = (N,) if op == "delta_step" else (N, L)
    unit = lambda v: v / (v.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    # queries and keys of unit length, values as the column range of a convolution's output, rates and decays as
    # a gate's projections leave them
    s["q"] = unit(normal(*lead, G, S)).to(t)
    s["k"] = unit(normal(*lead, G, S)).to(t)
    u = normal(*lead, 2 * G * S + H * P)
    s["v"] = (u * torch.sigmoid(u)).to(t)[..., 2 * G * S:].unflatten(-1, (H, P))
    s["beta"] = torch.sigmoid(normal(*lead, H)).to(t)
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))
    raw = 0.5 * normal(*lead, H) + step + torch.log(-torch.expm1(-step))
    s["g"] = -uniform(1, 16, H) * torch.nn.functional.softplus(raw)
    if case["state"]:
        s["state"] = 0.3 * normal(N, H, P, S)
    if op == "delta_grad":
        s["dy"] = normal(N, L, H, P).to(t)
        s["dstate_out"] = 0.1 * normal(N, H, P, S) if case["state"] else None
    if own:
        from convolution_forward_implicit_amd import DeltaRule
        s["plan"] = DeltaRule({"N": N, "L": L, "H": H, "P": P, "G": G, "S": S}, case["dtype"])
    return s


# ---- the calls of the package -----------------------------------------------

GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dstate")
NORM_GRADS = ("dx", "dw", "dbias", "dgate")


def _own(s):
    c, op, p = s["case"], s["case"]["op"], s["plan"]
    if op == "norm":
        return p(s["x"], s["w"], s["bias"], gate=s["gate"], lengths=s["lengths"])
    if op == "norm_grad":
        g = p.backward(s["dy"], s["x"], s["w"], s["bias"], gate=s["gate"], lengths=s["lengths"])
        return [g[k] for k in NORM_GRADS if g[k] is not None]
    a = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if op == "delta":
        out = torch.empty((c["N"], c["H"], c["P"], c["S"]), dtype=torch.float32, device=s["q"].device)
        return p(*a, state=s["state"], lengths=s["lengths"], state_out=out), out
    if op == "delta_step":
        return p.step(*a, s["state"]), s["state"]
    g = p.backward(s["dy"], *a, state=s["state"], lengths=s["lengths"], dstate_out=s["dstate_out"])
    return [g[k] for k in GRADS if g[k] is not None]


# ---- the plain forms --------------------------------------------------------

def _inside(s):
    """[N, L]: the tokens that belong to their sequence."""
    if s["lengths"] is None:
        return None
    t = torch.arange(s["case"]["L"], device=s["lengths"].device)
    return t[None, :] < s["lengths"][:, None]


def _act(name, v):
    """An activation and its derivative."""
    if name == "silu":
        sg = 1 / (1 + torch.exp(-v))
        return v * sg, sg * (1 + v * (1 - sg))
    if name == "gelu":
        phi = 0.5 * (1 + torch.erf(v / math.sqrt(2)))
        return v * phi, phi + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    return v, torch.ones_like(v)


EPS = 1e-5


def _norm_parts(s):
    c = s["case"]
    x = s["x"].float()
    keep = _inside(s)
    dims = (3,) if c["per_token"] else (1, 3)
    count = torch.full((1, 1, 1, 1), float(c["C"] if c["per_token"] else c["L"] * c["C"]), device=x.device)
    if keep is not None:
        keep = keep[..., None, None]
        x = torch.where(keep, x, 0.0)
        if not c["per_token"]:
            count = (s["lengths"].float() * c["C"]).clamp(min=1)[:, None, None, None]
    d = x
    if c["center"]:
        d = x - x.sum(dims, keepdim=True) / count
        if keep is not None:
            d = torch.where(keep, d, 0.0)
    r = 1 / (d.square().sum(dims, keepdim=True) / count + EPS).sqrt()
    xhat = d * r
    v = xhat * s["w"].float()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    return keep, dims, count, r, xhat, v


def _plain_norm(s):
    c, t = s["case"], s["x"].dtype
    keep, _, _, _, _, v = _norm_parts(s)
    y = v * _act(c["act"], s["gate"].float())[0] if c["gated"] else _act(c["act"], v)[0]
    if keep is not None:
        y = torch.where(keep, y, 0.0)
    return y.to(t)


def _plain_norm_grad(s):
    c, t = s["case"], s["x"].dtype
    keep, dims, count, r, xhat, v = _norm_parts(s)
    dy = s["dy"].float()
    clear = (lambda z: z) if keep is None else (lambda z: torch.where(keep, z, 0.0))
    if c["gated"]:
        a, da = _act(c["act"], s["gate"].float())
        d, dgate = clear(dy * a), clear(dy * v * da)
    else:
        d, dgate = clear(dy * _act(c["act"], v)[1]), None
    dw, db = (d * xhat).sum((0, 1)), d.sum((0, 1))
    d = d * s["w"].float()
    dx = d - xhat * ((d * xhat).sum(dims, keepdim=True) / count)
    if c["center"]:
        dx = dx - d.sum(dims, keepdim=True) / count
    got = [clear(dx * r).to(t), dw.to(t)]
    return got + ([db.to(t)] if s["bias"] is not None else []) + ([dgate.to(t)] if dgate is not None else [])


def _chunks(v, K, Q):
    """[N, L, heads, ...] as [N, chunk, heads, Q, ...] with zeros behind the end."""
    v = torch.cat([v, v.new_zeros(v.shape[0], K * Q - v.shape[1], *v.shape[2:])], 1)
    return v.unflatten(1, (K, Q)).transpose(2, 3)


def _joined(v, L):
    """The inverse of _chunks."""
    return v.transpose(2, 3).flatten(1, 2)[:, :L]


def _tr(v):
    return v.transpose(-1, -2).contiguous()


def _delta_parts(s):
    """What the delta rule and its gradient share: the chunked inputs, the decays inside a chunk (their exponents
    are summed in 64 bits: long sums) and the matrix that a chunk's own keys act by on what the state lacks."""
    c = s["case"]
    N, L, H, G = (c[k] for k in "NLHG")
    Q = CHUNK
    K = max(1, -(-L // Q))
    keep = _inside(s)
    clear = (lambda v: v.float()) if keep is None else (
        lambda v: torch.where(keep.view(*keep.shape, *[1] * (v.dim() - 2)), v.float(), 0.0))
    heads = lambda v: _chunks(clear(v), K, Q).repeat_interleave(H // G, 2)     # a head's own copy of its group's
    p = {"K": K, "keep": keep, "q": heads(s["q"]), "k": heads(s["k"]), "v": _chunks(clear(s["v"]), K, Q),
         "beta": _chunks(clear(s["beta"]), K, Q)}
    cum = _chunks(clear(s["g"]), K, Q).double().cumsum(-1)                      # [N, K, H, Q]
    low = torch.ones(Q, Q, dtype=torch.bool, device=cum.device).tril()
    p["decay"] = torch.exp(torch.where(low, cum[..., :, None] - cum[..., None, :], -math.inf)).float()
    p["from_start"] = torch.exp(cum).float()[..., None]
    p["to_end"] = torch.exp(cum[..., -1:] - cum).float()[..., None]
    p["total"] = p["from_start"][..., -1:, :]
    p["T"] = (torch.matmul(p["k"], _tr(p["k"])) * p["decay"]).tril(-1)
    power = -(p["T"] * p["beta"][..., None, :]).double()
    inverse = power + torch.eye(Q, dtype=torch.float64, device=cum.device)
    for _ in range(int(math.log2(Q)) - 1):                                     # (1 + X)(1 + X^2)(1 + X^4) ..., X^Q = 0
        power = torch.matmul(power, power)
        inverse = inverse + torch.matmul(inverse, power)
    p["act"] = torch.matmul(inverse, p["T"].double()).float()
    p["scale"] = c["S"] ** -0.5
    p["M"] = torch.matmul(p["q"], _tr(p["k"])) * p["decay"] * p["scale"]
    return p


def _delta_chunk(p, j, S):
    """What chunk j adds under its keys, without and with its rates, and the state behind it."""
    k, beta = p["k"][:, j], p["beta"][:, j, ..., None]
    z = p["v"][:, j] - p["from_start"][:, j] * torch.matmul(k, _tr(S))
    y = z - torch.matmul(p["act"][:, j], beta * z)
    u = beta * y
    return y, u, p["total"][:, j] * S + torch.matmul(_tr(u * p["to_end"][:, j]), k)


def _first(s):
    c = s["case"]
    return s["state"] if s["state"] is not None else torch.zeros(c["N"], c["H"], c["P"], c["S"], device=s["q"].device)


def _plain_delta(s):
    c, t = s["case"], s["q"].dtype
    p = _delta_parts(s)
    S, out = _first(s), []
    for j in range(p["K"]):
        _, u, after = _delta_chunk(p, j, S)
        out.append(torch.matmul(p["q"][:, j], _tr(S)) * (p["from_start"][:, j] * p["scale"]) + torch.matmul(p["M"][:, j], u))
        S = after
    return _joined(torch.stack(out, 1), c["L"]).to(t), S


def _plain_delta_step(s):
    c, t = s["case"], s["q"].dtype
    r = c["H"] // c["G"]
    q, k = s["q"].float().repeat_interleave(r, 1), s["k"].float().repeat_interleave(r, 1)
    h = s["state"]
    h.mul_(torch.exp(s["g"])[..., None, None])
    e = s["v"].float() - (h * k[:, :, None]).sum(-1)
    h.add_((s["beta"].float()[..., None] * e)[..., None] * k[:, :, None])
    return ((h * q[:, :, None]).sum(-1) * c["S"] ** -0.5).to(t), h


def _plain_delta_grad(s):
    c, t = s["case"], s["q"].dtype
    L, G, H = c["L"], c["G"], c["H"]
    p = _delta_parts(s)
    dy = s["dy"].float()
    if p["keep"] is not None:
        dy = torch.where(p["keep"][..., None, None], dy, 0.0)
    dy = _chunks(dy, p["K"], CHUNK)
    S, start, ys, us = _first(s), [], [], []
    for j in range(p["K"]):
        start.append(S)
        y, u, S = _delta_chunk(p, j, S)
        ys.append(y)
        us.append(u)
    start, y, u = torch.stack(start, 1), torch.stack(ys, 1), torch.stack(us, 1)
    dS = s["dstate_out"] if s["dstate_out"] is not None else torch.zeros_like(S)
    ends, es = [None] * p["K"], [None] * p["K"]
    for j in reversed(range(p["K"])):
        ends[j] = dS
        beta = p["beta"][:, j, ..., None]
        du = torch.matmul(_tr(p["M"][:, j]), dy[:, j]) + p["to_end"][:, j] * torch.matmul(p["k"][:, j], _tr(dS))
        es[j] = du - torch.matmul(_tr(p["act"][:, j]), beta * du)
        dS = (p["total"][:, j] * dS + torch.matmul(_tr(dy[:, j] * (p["from_start"][:, j] * p["scale"])), p["q"][:, j])
              - torch.matmul(_tr(beta * es[j] * p["from_start"][:, j]), p["k"][:, j]))
    end, e = torch.stack(ends, 1), torch.stack(es, 1)
    beta = p["beta"][..., None]
    dv = beta * e
    dM = torch.matmul(dy, _tr(u))
    W = torch.matmul(dv, _tr(u))
    low, below = (dM * p["decay"]).tril() * p["scale"], (W * p["decay"]).tril(-1)
    by_start = torch.matmul(dy, start) * (p["from_start"] * p["scale"])         # of q by the state in front
    old = torch.matmul(dv, start) * p["from_start"]
    new = torch.matmul(u, end) * p["to_end"]
    dq = by_start + torch.matmul(low, p["k"])
    dk = torch.matmul(_tr(low), p["q"]) - old + new - torch.matmul(below + _tr(below), p["k"])
    # the logarithms of the decays: sums of like size that cancel, so in 64 bits
    pairs = dM.double() * p["M"] - W.double() * p["T"]
    front = pairs.sum(-1) - pairs.sum(-2) + (by_start.double() * p["q"]).sum(-1) - (old.double() * p["k"]).sum(-1)
    behind = (new.double() * p["k"]).sum(-1)
    across = (p["total"].double() * start * end).sum((-1, -2))[..., None]
    dg = front.flip(-1).cumsum(-1).flip(-1) + across + behind.cumsum(-1) - behind
    groups = lambda w: _joined(w, L).unflatten(2, (G, H // G)).sum(3)
    keep = p["keep"]
    clear = (lambda w: w) if keep is None else (lambda w: torch.where(keep.view(*keep.shape, *[1] * (w.dim() - 2)), w, 0.0))
    got = [clear(groups(dq)).to(t), clear(groups(dk)).to(t), clear(_joined(dv, L)).to(t),
           clear(_joined(dg, L)).float(), clear(_joined((e * y).sum(-1), L)).to(t)]
    return got + ([dS] if s["state"] is not None else [])


PLAIN = {"delta": _plain_delta, "delta_step": _plain_delta_step, "delta_grad": _plain_delta_grad, "norm": _plain_norm,
         "norm_grad": _plain_norm_grad}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    N, L, G, op = case["N"], case["L"], case["G"], case["op"]
    if op.startswith("norm"):
        n = N * L * G * case["C"]
        w = G * case["C"] * e * (2 if case["bias"] else 1)
        if op == "norm":
            return {"bytes": n * e * (3 if case["gated"] else 2) + w, "flops": 12 * n}
        return {"bytes": n * e * (5 if case["gated"] else 3) + 2 * w, "flops": 30 * n}
    H, P, S = case["H"], case["P"], case["S"]
    rows, state = N * L, N * H * P * S * 4
    inputs = rows * ((2 * G * S + H * P + H) * e + H * 4)
    out = rows * H * P * e
    if op == "delta":
        return {"bytes": inputs + out + state * (2 if case["state"] else 1), "flops": 6 * rows * H * P * S}
    if op == "delta_step":
        return {"bytes": inputs + out + 2 * state, "flops": 7 * rows * H * P * S}
    return {"bytes": 2 * inputs + out + (3 * state if case["state"] else 0), "flops": 18 * rows * H * P * S}


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    def norm(s, grad):
        c = case
        wide = lambda v: None if v is None else v.double().requires_grad_(grad)
        x, w, b, z = wide(s["x"]), wide(s["w"]), wide(s["bias"]), wide(s["gate"])
        act = {"none": lambda v: v, "silu": lambda v: v * torch.sigmoid(v),
               "gelu": lambda v: v * torch.special.ndtr(v)}[c["act"]]
        n = s["lengths"].tolist() if s["lengths"] is not None else [c["L"]] * c["N"]
        rows = []
        for i in range(c["N"]):
            xi = x[i, :n[i]]
            over = (-1,) if c["per_token"] else (0, 2)
            if n[i]:
                if c["center"]:
                    xi = xi - xi.mean(over, keepdim=True)
                xi = xi / ((xi * xi).mean(over, keepdim=True) + EPS).sqrt()
            v = xi * w
            if b is not None:
                v = v + b
            y = v * act(z[i, :n[i]]) if z is not None else act(v)
            rows.append(torch.cat([y, torch.zeros_like(x[i, n[i]:])]))
        y = torch.stack(rows)
        if not grad:
            return y
        y.backward(s["dy"].double())
        return [v.grad for v in (x, w, b, z) if v is not None]

    def delta(s, grad):
        N, L, H, P, G, S = (case[k] for k in "NLHPGS")
        r, dev, scale = H // G, s["q"].device, case["S"] ** -0.5
        step = case["op"] == "delta_step"
        wide = lambda v: v.double()[:, None] if step else v.double()
        q, k = wide(s["q"]).repeat_interleave(r, 2), wide(s["k"]).repeat_interleave(r, 2)
        v, a, beta = wide(s["v"]), torch.exp(wide(s["g"])), wide(s["beta"])
        n = s["lengths"] if s["lengths"] is not None else torch.full((N,), L, device=dev)
        live = torch.arange(L, device=dev)[None, :] < n[:, None]
        on = live.double()[..., None]
        a, beta = torch.where(live[..., None], a, 1.0), beta * on               # a row behind leaves the state
        h = s["state"].double().clone() if s["state"] is not None else torch.zeros(N, H, P, S, dtype=torch.float64, device=dev)

        def after(h, t):
            h = a[:, t, :, None, None] * h
            e = v[:, t] - torch.matmul(h, k[:, t, :, :, None])[..., 0]
            return h, e, h + (beta[:, t, :, None] * e)[..., None] * k[:, t, :, None, :]

        if not grad:
            y = torch.zeros(N, L, H, P, dtype=torch.float64, device=dev)
            for t in range(L):
                h = after(h, t)[2]
                y[:, t] = torch.matmul(h, q[:, t, :, :, None])[..., 0]
            y = y * scale * on[..., None]
            return (y[:, 0] if step else y), h
        dy = s["dy"].double() * on[..., None] * scale
        near, marks = 32, []
        for t in range(L):
            if t % near == 0:
                marks.append(h)
            h = after(h, t)[2]
        u = s["dstate_out"].double().clone() if s["dstate_out"] is not None else torch.zeros_like(h)
        dq, dk, dv, dg, db = (torch.zeros_like(w) for w in (q, k, v, a, beta))
        for m in reversed(range(len(marks))):
            steps, h = [], marks[m]
            for t in range(m * near, min(L, (m + 1) * near)):
                steps.append((h,) + after(h, t))
                h = steps[-1][3]
            for t in reversed(range(m * near, min(L, (m + 1) * near))):
                before, faded, e, now = steps[t - m * near]
                dq[:, t] = torch.matmul(dy[:, t, :, None, :], now)[..., 0, :]
                u = u + dy[:, t, :, :, None] * q[:, t, :, None, :]
                uk = torch.matmul(u, k[:, t, :, :, None])[..., 0]
                db[:, t] = (uk * e).sum(-1)
                de = beta[:, t, :, None] * uk
                dv[:, t] = de
                dk[:, t] = (torch.matmul((beta[:, t, :, None] * e)[..., None, :], u) - torch.matmul(de[..., None, :], faded))[..., 0, :]
                u = u - de[..., None] * k[:, t, :, None, :]
                dg[:, t] = (u * faded).sum((-1, -2))
                u = a[:, t, :, None, None] * u
        group = lambda w: (w * on[..., None]).unflatten(2, (G, r)).sum(3)
        got = [group(dq), group(dk), dv, dg * on, db * on]
        return got + ([u] if s["state"] is not None else [])

    s = prepare(case, seed)
    f = norm if case["op"].startswith("norm") else delta
    return f(s, case["op"].endswith("grad"))
