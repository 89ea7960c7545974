"""Workloads of the gated delta rule (prompt scan and decode step) and of the per-token
group norm that follows it, for timing and for comparing outputs.

With ``own`` false, run() evaluates the formulas with elementary torch operations in 32
bits; with ``own`` true it calls the package's entry points.  exact() evaluates the
definitions in 64 bits, token by token.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}
CHUNK = 64  # tokens per chunk of the plain chunked form
NORM_EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------

def _scan(name, batch, seq, heads_k, heads_v, dk, dv, dtype, doc=0, h0=False):
    return {"name": name, "op": "delta_scan", "batch": batch, "seq": seq, "heads_k": heads_k, "heads_v": heads_v,
            "dk": dk, "dv": dv, "dtype": dtype, "doc": doc, "h0": h0}


def _update(name, batch, heads_k, heads_v, dk, dv, dtype):
    return {"name": name, "op": "delta_update", "batch": batch, "heads_k": heads_k, "heads_v": heads_v, "dk": dk,
            "dv": dv, "dtype": dtype}


def _norm(name, rows, groups, size, dtype, center, gate, act, shared):
    return {"name": name, "op": "group_norm", "rows": rows, "groups": groups, "size": size, "dtype": dtype,
            "center": center, "gate": gate, "act": act, "shared": shared}


def listed():
    return [
        # a short question to one model layer: one chunk of tokens, latency counts
        _scan("prompt_short", 1, 64, 16, 32, 128, 128, BF16),
        # one long document, a single request: few heads, a long chain of chunks
        _scan("prompt_long", 1, 16384, 16, 32, 128, 128, BF16),
        # several requests prefilled together, continued from a cached state
        _scan("prompt_batch", 8, 2048, 16, 32, 128, 128, BF16, h0=True),
        # packed documents of odd lengths, narrower heads, a ragged last chunk
        _scan("prompt_packed", 3, 1531, 4, 12, 96, 64, BF16, doc=200, h0=True),
        # a small model checked in full precision
        _scan("prompt_f32", 2, 300, 4, 4, 64, 64, F32),
        # one token for one user: latency counts
        _update("decode_one", 1, 16, 32, 128, 128, BF16),
        # one token for a full serving batch: the state is read and written once
        _update("decode_batch", 256, 16, 32, 128, 128, BF16),
        # an odd batch with sizes that are no power of two, full precision
        _update("decode_f32_odd", 37, 3, 6, 96, 80, F32),
        # the gated norm of one decode step's heads
        _norm("norm_decode", 256, 32, 128, BF16, False, "after", False, True),
        # the gated norm of a long prompt's heads, one weight for all heads
        _norm("norm_prompt", 16384, 32, 128, BF16, False, "after", False, True),
        # centred group norm with SiLU over a few wide groups (5120 channels)
        _norm("norm_wide_f32", 4096, 8, 640, F32, True, "none", True, False),
        # an odd number of rows and a group size that no vector load divides
        _norm("norm_odd", 4099, 5, 83, BF16, True, "before", False, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(("delta_scan", "delta_scan", "delta_update", "group_norm"))
    dtype = BF16 if rng.random() < 0.7 else F32
    size = (lambda: rng.choice((32, 64, 96, 128)) if rng.random() < 0.6 else rng.randint(9, 128))
    if op == "group_norm":
        groups, width = _log_int(rng, 1, 64), _log_int(rng, 16, 1024)
        rows = min(_log_int(rng, 1, 16384), max(1, 16384 * 4096 // (groups * width)))
        c = _norm("", rows, groups, width, dtype, rng.random() < 0.5, rng.choice(("none", "before", "after")),
                  rng.random() < 0.5, rng.random() < 0.5)
    elif op == "delta_update":
        hk, ratio = rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((1, 2, 4))
        batch = min(_log_int(rng, 1, 256), 256 * 32 // (hk * ratio))
        c = _update("", batch, hk, hk * ratio, size(), size(), dtype)
    else:
        hk, ratio, batch = rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((1, 2, 4)), _log_int(rng, 1, 8)
        top = min(16384, max(1, 16384 * 32 // (batch * hk * ratio)))
        c = _scan("", batch, _log_int(rng, 1, top), hk, hk * ratio, size(), size(), dtype,
                  rng.choice((0, 0, 50, 500)), rng.random() < 0.5)
    del c["name"]
    return c


# ---- inputs --------------------------------------------------------------------------

def _gates(gen, lead, heads):
    """Log decays g = -A softplus(a + dt_bias) and write strengths beta = sigmoid(b), with
    A in [1, 16] and steps log-uniform in [1e-3, 1e-1] as state-space layers start."""
    dev = gen.device
    A = 1 + 15 * torch.rand(heads, generator=gen, device=dev)
    u = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(heads, generator=gen, device=dev))
    a = torch.randn(*lead, heads, generator=gen, device=dev)
    g = -A * torch.nn.functional.softplus(a + torch.log(torch.expm1(u)))
    return g, torch.sigmoid(torch.randn(*lead, heads, generator=gen, device=dev))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    t = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def conv_out(*shape):  # q, k and v come out of a convolution and a SiLU
        return torch.nn.functional.silu(normal(*shape)).to(t)

    s = {"case": case}
    if case["op"] == "group_norm":
        rows, ch = case["rows"], case["groups"] * case["size"]
        s["x"] = (normal(rows, ch) * 0.5 + 0.1).to(t)
        s["gate"] = normal(rows, ch).to(t) if case["gate"] != "none" else None
        n = case["size"] if case["shared"] else ch
        s["weight"] = 1 + 0.1 * normal(n)
        s["bias"] = 0.1 * normal(n) if case["center"] else None
        return s
    b, hk, hv, dk, dv = (case[n] for n in ("batch", "heads_k", "heads_v", "dk", "dv"))
    lead = (b,) if case["op"] == "delta_update" else (b, case["seq"])
    # one projection holds q, k and v side by side, as the layer's convolution leaves them
    qkv = conv_out(*lead, 2 * hk * dk + hv * dv)
    s["q"] = qkv[..., : hk * dk].unflatten(-1, (hk, dk))
    s["k"] = qkv[..., hk * dk: 2 * hk * dk].unflatten(-1, (hk, dk))
    s["v"] = qkv[..., 2 * hk * dk:].unflatten(-1, (hv, dv))
    s["g"], s["beta"] = _gates(gen, lead, hv)
    if case["op"] == "delta_update":
        s["state"] = 0.3 * normal(b, hv, dk, dv)
        return s
    s["h0"] = 0.3 * normal(b, hv, dk, dv) if case["h0"] else None
    s["reset"] = None
    if case["doc"]:
        s["reset"] = torch.rand(*lead, generator=gen, device=dev) < 1.0 / case["doc"]
    return s


# ---- plain forms ---------------------------------------------------------------------

def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + NORM_EPS)


def _heads(x, heads_v):
    """[..., heads_k, d] -> [..., heads_v, d]: value head h reads key head h // ratio."""
    return x.repeat_interleave(heads_v // x.shape[-2], dim=-2)


def _plain_scan(s):
    c = s["case"]
    hv, dk, L = c["heads_v"], c["dk"], c["seq"]
    n = -(-L // CHUNK)
    pad = n * CHUNK - L

    def chunks(x):  # [b, L, h, d] -> [b, h, n, C, d]; padding tokens are zero
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad))
        return x.transpose(1, 2).unflatten(2, (n, CHUNK))

    q = chunks(_heads(_unit(s["q"].float()), hv) * dk ** -0.5)
    k = chunks(_heads(_unit(s["k"].float()), hv))
    v = chunks(s["v"].float())
    beta = chunks(s["beta"][..., None])
    # decays between two tokens of a chunk, from sums of logs in 64 bits; a reset cuts them
    G = chunks(s["g"][..., None].double())[..., 0]
    cut = torch.zeros_like(G, dtype=torch.long)
    if s["reset"] is not None:
        cut = chunks(s["reset"][:, :, None, None].long().expand(-1, -1, hv, 1))[..., 0]
        G = G * (cut == 0)
    G, N = G.cumsum(-1), cut.cumsum(-1)
    i = torch.arange(CHUNK, device=G.device)
    keep = (N[..., :, None] == N[..., None, :]) & (i[:, None] >= i[None, :])
    between = torch.where(keep, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    enter = torch.where(N == 0, G, -math.inf).exp().float()[..., None]
    leave = torch.where(N == N[..., -1:], G[..., -1:] - G, -math.inf).exp().float()[..., None]
    last = enter[..., -1:, :]
    eye = torch.eye(CHUNK, device=G.device)
    low = beta * (k @ k.mT) * between * (1 - eye) + eye
    both = torch.linalg.solve_triangular(low, beta * torch.cat((v, enter * k), -1), upper=False, unitriangular=True)
    uv, uk = both.split((c["dv"], dk), -1)
    H = s["h0"].float() if s["h0"] is not None else torch.zeros(c["batch"], hv, dk, c["dv"], device=G.device)
    kl = (leave * k).mT
    states, us = [], []
    for j in range(n):
        states.append(H)
        us.append(uv[:, :, j] - uk[:, :, j] @ H)
        H = last[:, :, j] * H + kl[:, :, j] @ us[-1]
    states, us = torch.stack(states, 2), torch.stack(us, 2)
    y = (enter * q) @ states + ((q @ k.mT) * between) @ us
    y = y.flatten(2, 3)[:, :, :L].transpose(1, 2)
    return {"outputs": y.to(s["q"].dtype), "final_state": H}


def _plain_update(s):
    c = s["case"]
    q = _heads(_unit(s["q"].float()), c["heads_v"]) * c["dk"] ** -0.5
    k = _heads(_unit(s["k"].float()), c["heads_v"])
    S = s["state"]
    S *= s["g"].exp()[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (k[..., None, :] @ S)[..., 0, :])
    S += k[..., :, None] * u[..., None, :]
    return {"outputs": (q[..., None, :] @ S)[..., 0, :].to(s["q"].dtype), "state": S}


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    gate = s["gate"].float() if s["gate"] is not None else None
    if c["gate"] == "before":
        x = x * (gate * torch.sigmoid(gate))
    x = x.unflatten(-1, (c["groups"], c["size"]))
    if c["center"]:
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS)
    shape = (1, c["size"]) if c["shared"] else (c["groups"], c["size"])
    x = x * s["weight"].view(shape)
    if s["bias"] is not None:
        x = x + s["bias"].view(shape)
    x = x.flatten(-2)
    if c["act"]:
        x = x * torch.sigmoid(x)
    if c["gate"] == "after":
        x = x * (gate * torch.sigmoid(gate))
    return x.to(s["x"].dtype)


# ---- one pass ------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        from selective_state_space_18_b200 import ssscan
        if op == "delta_scan":
            return ssscan.ss_delta_scan(state["q"], state["k"], state["v"], state["g"], state["beta"],
                                        reset=state["reset"], h0=state["h0"], qk_l2norm=True)
        if op == "delta_update":
            y = ssscan.ss_delta_update(state["state"], state["q"], state["k"], state["v"], state["g"], state["beta"],
                                       qk_l2norm=True)
            return {"outputs": y, "state": state["state"]}
        c = state["case"]
        return ssscan.ss_group_norm(state["x"], c["groups"], state["weight"], state["bias"], gate=state["gate"],
                                    gate_first=c["gate"] == "before", center=c["center"],
                                    activation="silu" if c["act"] else None, eps=NORM_EPS)
    if op == "delta_scan":
        return _plain_scan(state)
    return _plain_update(state) if op == "delta_update" else _plain_norm(state)


def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    if case["op"] == "group_norm":
        n = case["rows"] * case["groups"] * case["size"]
        return {"bytes": n * e * (2 if case["gate"] == "none" else 3), "flops": 6 * n}
    b, hk, hv, dk, dv = (case[n] for n in ("batch", "heads_k", "heads_v", "dk", "dv"))
    tokens = b * case.get("seq", 1)
    state = b * hv * dk * dv * 4
    # q, k, v and the output, g and beta; the state written, and read where there is one
    n = tokens * (e * (2 * hk * dk + 2 * hv * dv) + 8 * hv) + state
    if case["op"] == "delta_update" or case["h0"]:
        n += state
    if case.get("doc"):
        n += tokens
    # per token and value head: k^T S, the outer product's update of S, q^T S
    return {"bytes": n, "flops": 6 * tokens * hv * dk * dv}


# ---- the definitions in 64 bits --------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "group_norm":
        x = s["x"].double().view(case["rows"], case["groups"], case["size"])
        gate = None
        if s["gate"] is not None:
            z = s["gate"].double()
            gate = (z / (1 + torch.exp(-z))).view(x.shape)
        if case["gate"] == "before":
            x = x * gate
        mean = x.sum(-1, keepdim=True) / case["size"] if case["center"] else torch.zeros_like(x[..., :1])
        var = ((x - mean) ** 2).sum(-1, keepdim=True) / case["size"]
        y = (x - mean) / torch.sqrt(var + NORM_EPS)
        one = (1, 1, case["size"]) if case["shared"] else (1, case["groups"], case["size"])
        y = y * s["weight"].double().view(one)
        if s["bias"] is not None:
            y = y + s["bias"].double().view(one)
        if case["act"]:
            y = y / (1 + torch.exp(-y))
        if case["gate"] == "after":
            y = y * gate
        return y.view(case["rows"], -1)
    hv, dk = case["heads_v"], case["dk"]

    def unit(x):
        x = x.double()
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) + NORM_EPS)
        return x.repeat_interleave(hv // x.shape[-2], dim=-2)

    q, k, v = unit(s["q"]) / math.sqrt(dk), unit(s["k"]), s["v"].double()
    decay, beta = torch.exp(s["g"].double()), s["beta"].double()
    if case["op"] == "delta_update":
        q, k, v, decay, beta = (x[:, None] for x in (q, k, v, decay, beta))
        S, steps = s["state"].double(), 1
    else:
        steps = case["seq"]
        S = s["h0"].double() if s["h0"] is not None else torch.zeros(case["batch"], hv, dk, case["dv"], device=q.device,
                                                                    dtype=torch.float64)
        if s["reset"] is not None:
            decay = decay * (~s["reset"])[..., None]
    y = torch.empty_like(v)
    for t in range(steps):
        S = S * decay[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(-2))
        S = S + k[:, t, :, :, None] * u[:, :, None, :]
        y[:, t] = (S * q[:, t, :, :, None]).sum(-2)
    if case["op"] == "delta_update":
        return {"outputs": y[:, 0], "state": S}
    return {"outputs": y, "final_state": S}
