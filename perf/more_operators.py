"""Cases for a gated linear recurrence (prompts, single tokens, gradient) and the RMS norm with the
residual's addition (the same type out, 8 bits out, gradient).

A case names an operator (`op`) and its sizes.  `run` computes it in plain torch, in 32 bits,
or, where `own` is set, through this package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FWD, BWD, NORM = 32768 * 4096, 16384 * 4096, 32768 * 4096  # the largest T * C of each
DECAY, EPS = 8.0, 1e-6


def listed():
    return [
        # a short prompt in one layer of a small model: latency counts
        dict(name="rec fwd short prompt", op="rec_fwd", N=1, T=64, C=1024, type="bf16", param=True, xgate=True, act="", scale="sqrt", init=False),
        # a batch of ragged prompts, some of them continued from a cached state, with the block's gated branch
        dict(name="rec fwd prompts", op="rec_fwd", N=16, T=32768, C=4096, type="bf16", param=True, xgate=True, act="gelu", scale="sqrt", init=True),
        # one very long document: the whole parallelism is in the channels
        dict(name="rec fwd long", op="rec_fwd", N=1, T=65536, C=2048, type="bf16", param=True, xgate=True, act="", scale="sqrt", init=False),
        # a few requests decoding in a small fp32 model whose decay is the forget gate itself
        dict(name="rec update few", op="rec_update", N=5, C=1032, type="f32", param=False, xgate=False, act="silu", scale="linear"),
        # one decode step at the benchmark's batch
        dict(name="rec update batch", op="rec_update", N=256, C=4096, type="bf16", param=True, xgate=True, act="gelu", scale="sqrt"),
        # gradients of a small, odd fp32 batch with state gradients
        dict(name="rec bwd odd", op="rec_bwd", N=3, T=301, C=520, type="f32", param=False, xgate=True, act="silu", scale="linear", init=True),
        # a training step's micro-batch of packed documents
        dict(name="rec bwd training", op="rec_bwd", N=8, T=16384, C=4096, type="bf16", param=True, xgate=True, act="gelu", scale="sqrt", init=False),
        # a handful of decoding tokens through the benchmark's channel count, back to bf16
        dict(name="norm decode", op="norm", T=7, d=8192, type="bf16", residual=True, group=None),
        # a prompt's rows in front of 8-bit projections, a scale for each 128 values
        dict(name="norm 8 bits prompt", op="norm", T=32768, d=4096, type="bf16", residual=True, group=128),
        # an odd fp32 batch without a residual, a scale for each row
        dict(name="norm 8 bits odd", op="norm", T=1001, d=1160, type="f32", residual=False, group=0),
        # gradients of a small, odd fp32 batch
        dict(name="norm bwd odd", op="norm_bwd", T=333, d=1032, type="f32", residual=False),
        # the benchmark's backward workload, 8 x 4096 tokens packed
        dict(name="norm bwd training", op="norm_bwd", T=32768, d=4096, type="bf16", residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rec_fwd", "rec_fwd", "rec_update", "rec_bwd", "rec_bwd", "norm", "norm", "norm_bwd"])
    t = rng.choice(["bf16", "f32"])
    half = 2 if t == "f32" else 1
    if op in ("norm", "norm_bwd"):
        d = 8 * _log(rng, 8, 2048)
        T = min(_log(rng, 1, 32768), max(1, NORM // (d * half)))
        c = dict(op=op, T=T, d=d, type=t, residual=rng.random() < 0.7)
        return c if op == "norm_bwd" else dict(c, group=rng.choice([None, None, 0, 32, 64, 128]))
    C = 8 * _log(rng, 8, 1024)
    param = rng.random() < 0.6
    kind = dict(type=t, param=param, xgate=rng.random() < (0.8 if param else 0.4), act=rng.choice(["", "silu", "gelu"]),
                scale=rng.choice(["sqrt", "sqrt", "linear", "one"] if param else ["linear", "linear", "sqrt", "one"]))
    if op == "rec_update":
        return dict(op=op, N=_log(rng, 1, 512), C=C, **kind)
    most = (FWD if op == "rec_fwd" else BWD) // (C * half)
    T = min(_log(rng, 1, 65536 if op == "rec_fwd" else 16384), max(1, most))
    return dict(op=op, N=rng.randint(1, min(T, 16)), T=T, C=C, **kind, init=rng.random() < 0.5)


def lengths(c):
    """Ragged lengths (an empty one among four or more) that sum to T."""
    r = random.Random(c["N"] * 1000003 + c["T"])
    w = [r.lognormvariate(0.0, 0.5) for _ in range(c["N"])]
    if c["N"] >= 4:
        w[1] = 0.0
    at = np.floor(np.cumsum(w) / sum(w) * c["T"] + 0.5).astype(int)
    at[-1] = c["T"]
    return np.diff(np.concatenate([[0], at])).tolist()


def _inputs(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    ty = TYPES[c["type"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = dict(c)
    if c["op"] in ("norm", "norm_bwd"):
        T, d = c["T"], c["d"]
        s["x"] = (randn(T, d) * torch.exp(0.5 * randn(T, 1))).to(ty)  # a token's rows grow and shrink along a model
        s["w"] = 1 + 0.1 * randn(d)
        if c["op"] == "norm":
            s["r"] = (2 * randn(T, d)).to(ty) if c["residual"] else None
        else:
            s["dy"] = randn(T, d).to(ty)
            s["dr"] = randn(T, d).to(ty) if c["residual"] else None
        return s
    C, T = c["C"], c.get("T", c["N"])
    if c["op"] != "rec_update":
        lens = lengths(c)
        s["longest"] = max(lens)
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    s["x"] = randn(T, C).to(ty)
    gates = randn(T, 2 * C)                                # both gates side by side, as one projection gives them
    if not c["param"]:
        gates[:, :C].mul_(1.5).add_(2.0)                   # forget gates that mostly keep
    gates = gates.to(ty)
    s["ag"], s["xg"] = gates[:, :C], gates[:, C:] if c["xgate"] else None
    s["z"] = randn(T, C).to(ty) if c["act"] else None
    keep = 0.9 + 0.099 * torch.rand(C, generator=gen, device=DEV)
    s["par"] = torch.log(torch.expm1(-torch.log(keep) / DECAY)) if c["param"] else None  # decays of 0.9 .. 0.999 at an open gate
    if c["op"] == "rec_bwd":
        s["dy"] = randn(T, C).to(ty)
        s["h0"] = randn(c["N"], C) if c["init"] else None
        s["dhT"] = randn(c["N"], C) if c["init"] else None
        return s
    slots = c["N"] + 3
    s["pool"] = randn(slots, C)
    s["idx"] = torch.randperm(slots, generator=gen, device=DEV)[:c["N"]].to(torch.int32)
    if c["op"] == "rec_fwd":
        has = torch.arange(c["N"], device=DEV) % 3 != 0 if c["init"] else torch.zeros(c["N"], device=DEV)
        s["has"] = has.to(torch.int32)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---------------------------------------------------------------- the plain forms


def _sig(x):
    return 1 / (1 + torch.exp(-x))


def _softplus(v):
    return torch.maximum(v, torch.zeros_like(v)) + torch.log1p(torch.exp(-v.abs()))


def _inner(act, z):
    """The sigmoid's argument of the branch's activation z * sigmoid(.), and its slope."""
    if act == "silu":
        return z, 1.0
    k = 2 * math.sqrt(2 / math.pi)
    return k * (z + 0.044715 * z * z * z), k * (1 + 3 * 0.044715 * z * z)


def _act(act, z):
    return z * _sig(_inner(act, z)[0])


def _dact(act, z):
    u, du = _inner(act, z)
    p = _sig(u)
    return p + z * p * (1 - p) * du


def _gates(s):
    """The log decay, the decay, the input's scale and the gated input of every token."""
    g, x = s["ag"].float(), s["x"].float()
    u = -DECAY * _softplus(s["par"]) * _sig(g) if s["param"] else -_softplus(-g)
    a, m = torch.exp(u), -torch.expm1(u)
    sc = torch.sqrt(m * (2 - m)) if s["scale"] == "sqrt" else m if s["scale"] == "linear" else torch.ones_like(m)
    return u, a, sc, x * _sig(s["xg"].float()) if s["xgate"] else x


def _recur(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; a_t is 0 where a sequence starts."""
    reach = 1
    while reach < longest:
        more = a[reach:] * b[:-reach]
        far = a[reach:] * a[:-reach]
        b[reach:] += more
        a[reach:] = far
        reach *= 2
    return b


def _edges(s, T):
    """Whether each token is its sequence's first, its last; each sequence's first and last token; which sequences have any."""
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    cu = s["cu"]
    seq = torch.searchsorted(cu[1:], t, right=True)
    start, end = cu[:-1].long().clamp(max=T - 1), (cu[1:].long() - 1).clamp(min=0)
    return (t == cu[seq])[:, None], (t == cu[seq + 1] - 1)[:, None], start, end, (cu[1:] > cu[:-1])[:, None]


def _rec_fwd(s):
    first, _, start, end, ran = _edges(s, s["x"].shape[0])
    _, a, sc, v = _gates(s)
    b = sc * v
    slot = s["idx"].long()
    h0 = s["pool"][slot] * (s["has"] != 0)[:, None]
    b.index_add_(0, start, torch.where(ran, a[start] * h0, 0))
    h = _recur(a * ~first, b, s["longest"])
    s["pool"][slot] = torch.where(ran, h[end], h0)
    return {"y": (h * _act(s["act"], s["z"].float()) if s["act"] else h).to(s["x"].dtype), "state": s["pool"]}


def _rec_update(s):
    _, a, sc, v = _gates(s)
    slot = s["idx"].long()
    h = a * s["pool"][slot] + sc * v
    s["pool"][slot] = h
    return {"y": (h * _act(s["act"], s["z"].float()) if s["act"] else h).to(s["x"].dtype), "state": s["pool"]}


def _rec_bwd(s):
    ty, x, dy = s["x"].dtype, s["x"].float(), s["dy"].float()
    first, last, start, end, ran = _edges(s, x.shape[0])
    u, a, sc, v = _gates(s)
    b = sc * v
    if s["h0"] is not None:
        b.index_add_(0, start, torch.where(ran, a[start] * s["h0"], 0))
    h = _recur(a * ~first, b, s["longest"])
    old = torch.cat([torch.zeros_like(h[:1]), h[:-1]]) * ~first
    if s["h0"] is not None:
        old.index_add_(0, start, torch.where(ran, s["h0"], 0))
    out, e = {}, dy
    if s["act"]:
        z = s["z"].float()
        out["dz"] = (dy * h * _dact(s["act"], z)).to(ty)
        e = dy * _act(s["act"], z)
    if s["dhT"] is not None:
        e = e.index_add(0, end, torch.where(ran, s["dhT"], 0))
    after = torch.cat([a[1:], torch.zeros_like(a[:1])]) * ~last
    g = _recur(after.flip(0), e.flip(0), s["longest"]).flip(0)
    dv = g * sc
    if s["xgate"]:
        p = _sig(s["xg"].float())
        out["dx"], out["dx_gate"] = (dv * p).to(ty), (dv * v * (1 - p)).to(ty)
    else:
        out["dx"] = dv.to(ty)
    q = a * old
    if s["scale"] == "sqrt":
        q = q - v * a * a / sc
    elif s["scale"] == "linear":
        q = q - v * a
    q = q * g
    if s["param"]:
        r = _sig(s["ag"].float())
        out["da_gate"] = (q * u * _sig(-s["ag"].float())).to(ty)
        out["da_param"] = -DECAY * (q * r).sum(0) * _sig(s["par"])
    else:
        out["da_gate"] = (q * -torch.expm1(u)).to(ty)
    if s["init"]:
        out["d_init_state"] = torch.where(ran, (a * g)[start], s["dhT"])
    return out


def _norm(s):
    x, ty = s["x"].float(), s["x"].dtype
    out = {}
    if s["r"] is not None:
        out["residual"] = (x + s["r"].float()).to(ty)
        x = out["residual"].float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"]
    if s["group"] is None:
        out["y"] = n.to(ty)
        return out
    T, d = n.shape
    per = s["group"] or d
    cols = -(-d // per)
    most = torch.cat([n.abs(), n.new_zeros(T, cols * per - d)], 1).unflatten(1, (cols, per)).amax(-1)
    out["scales"] = (most / 448).clamp(min=2.0 ** -126)
    out["y"] = (n / out["scales"].repeat_interleave(per, 1)[:, :d]).to(torch.float8_e4m3fn)
    return out


def _norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    g = dy * s["w"]
    dx = r * g - x * r ** 3 * (g * x).mean(-1, keepdim=True)
    if s["dr"] is not None:
        dx = dx + s["dr"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * x * r).sum(0)}


def run(state):
    s = state
    if own:
        return _own(s)
    return {"rec_fwd": _rec_fwd, "rec_update": _rec_update, "rec_bwd": _rec_bwd, "norm": _norm, "norm_bwd": _norm_bwd}[s["op"]](s)


# ---------------------------------------------------------------- this package's entry points


def _own(s):
    import invariant_linear_attention_gb300 as gdn
    op = s["op"]
    if op == "norm":
        if s["group"] is None:
            y, res = gdn.gdn_add_rmsnorm(s["x"], s["w"], residual=s["r"], eps=EPS)
            return {"y": y, **({} if res is None else {"residual": res})}
        y, scales, res = gdn.gdn_add_rmsnorm_fp8(s["x"], s["w"], residual=s["r"], eps=EPS, group=s["group"])
        return {"y": y, "scales": scales, **({} if res is None else {"residual": res})}
    if op == "norm_bwd":
        return gdn.gdn_add_rmsnorm_bwd(s["x"], s["w"], s["dy"], d_residual_out=s["dr"], eps=EPS)
    kind = dict(a_param=s["par"], x_gate=s["xg"], z=s["z"], input_scale=s["scale"], decay=DECAY, activation=s["act"] or "silu")
    if op == "rec_fwd":
        y = gdn.gdn_linear_recurrence_fwd(s["x"], s["ag"], s["cu"], state=s["pool"], state_indices=s["idx"], has_initial_state=s["has"], **kind)
        return {"y": y, "state": s["pool"]}
    if op == "rec_update":
        y = gdn.gdn_linear_recurrence_update(s["x"], s["ag"], s["pool"], state_indices=s["idx"], **kind)
        return {"y": y, "state": s["pool"]}
    return gdn.gdn_linear_recurrence_bwd(s["x"], s["ag"], s["cu"], s["dy"], init_state=s["h0"], d_final_state=s["dhT"],
                                         need_d_init_state=s["init"], **kind)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    e = 2 if c["type"] == "bf16" else 4
    if c["op"] in ("norm", "norm_bwd"):
        n, d = c["T"] * c["d"], c["d"]
        if c["op"] == "norm_bwd":
            return {"bytes": n * e * (4 if c["residual"] else 3) + 8 * d, "flops": n * 12}
        moved = n * e * (3 if c["residual"] else 1) + 4 * d
        if c["group"] is None:
            return {"bytes": moved + n * e, "flops": n * 6}
        return {"bytes": moved + n + 4 * c["T"] * (-(-d // c["group"]) if c["group"] else 1), "flops": n * 8}
    T, C = c.get("T", c["N"]), c["C"]
    n, par, states = T * C, 4 * C if c["param"] else 0, 4 * c["N"] * C
    read = 2 + c["xgate"] + bool(c["act"])
    if c["op"] == "rec_bwd":
        return {"bytes": n * e * (2 * read + 1) + 2 * par + (3 * states if c["init"] else 0), "flops": n * 60}
    used = sum(i % 3 != 0 for i in range(c["N"])) / c["N"] if c.get("init") else 0 if c["op"] == "rec_fwd" else 1
    return {"bytes": n * e * (read + 1) + par + states * (1 + used), "flops": n * 30}


# ---------------------------------------------------------------- the definitions, in 64 bits


def _pad(v, lens, longest):
    """Packed rows as [sequence, row, ...], the rows behind a sequence's end filled with its neighbours'."""
    at = np.concatenate([[0], np.cumsum(lens)[:-1]])[:, None] + np.arange(longest)
    return v[torch.from_numpy(np.minimum(at, v.shape[0] - 1)).to(v.device)]


def _pack(v, lens):
    return torch.cat([v[n, :m] for n, m in enumerate(lens)])


def _walk(a, b, h, lens):
    """The recurrence token by token, all sequences side by side: the states after each token (past a sequence's end, anything)."""
    longest = max(lens)
    hs = []
    for at, bt in zip(_pad(a, lens, longest).unbind(1), _pad(b, lens, longest).unbind(1)):
        h = torch.addcmul(bt, at, h)
        hs.append(h)
    return hs


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    F = torch.nn.functional
    if c["op"] in ("norm", "norm_bwd"):
        T, d = c["T"], c["d"]
        x, w = s["x"].double(), s["w"].double()
        if c["op"] == "norm_bwd":
            x.requires_grad_()
            w.requires_grad_()
            y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w
            loss = (y * s["dy"].double()).sum()
            if s["dr"] is not None:
                loss = loss + (x * s["dr"].double()).sum()
            dx, dw = torch.autograd.grad(loss, (x, w))
            return {"dx": dx, "dweight": dw}
        got = {}
        if s["r"] is not None:
            got["residual"] = x + s["r"].double()
            x = got["residual"].to(s["x"].dtype).double()  # the norm is defined on the sum as it is stored
        n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        if c["group"] is None:
            return {**got, "y": n}
        parts = n.split(c["group"] or d, dim=1)
        sc = [(p.abs().amax(1, keepdim=True) / 448).clamp(min=2.0 ** -126) for p in parts]
        q = torch.cat([(p / k).clamp(-448, 448).to(torch.float8_e4m3fn).double() for p, k in zip(parts, sc)], 1)
        return {**got, "scales": torch.cat(sc, 1), "y": q}
    T, C, N = c.get("T", c["N"]), c["C"], c["N"]
    lens = lengths(c) if c["op"] != "rec_update" else [1] * N
    if N * max(lens) * C * 8 * (12 if c["op"] == "rec_bwd" else 6) > 150e9:
        return None
    leaf = {k: s[k].double() for k in ("x", "ag", "xg", "z", "par") if s[k] is not None}
    if c["op"] == "rec_bwd":
        leaf["h0"] = torch.zeros(N, C, dtype=torch.float64, device=DEV) if s["h0"] is None else s["h0"].double()
        for v in leaf.values():
            v.requires_grad_()
        h0 = leaf["h0"]
    else:
        h0 = s["pool"].double()[s["idx"].long()]
        if c["op"] == "rec_fwd":
            h0 = h0 * (s["has"] != 0)[:, None]
    v = leaf["x"] * torch.sigmoid(leaf["xg"]) if c["xgate"] else leaf["x"]
    u = -DECAY * F.softplus(leaf["par"], threshold=40.0) * torch.sigmoid(leaf["ag"]) if c["param"] else F.logsigmoid(leaf["ag"])
    b = v * {"sqrt": lambda: torch.sqrt(-torch.expm1(2 * u)), "linear": lambda: -torch.expm1(u), "one": lambda: 1.0}[c["scale"]]()
    hs = _walk(torch.exp(u), b, h0, lens)
    last = torch.stack([hs[m - 1][n] if m else h0[n] for n, m in enumerate(lens)])
    y = _pack(torch.stack(hs, 1), lens)
    if c["act"]:
        y = y * (F.silu(leaf["z"]) if c["act"] == "silu" else F.gelu(leaf["z"], approximate="tanh"))
    if c["op"] != "rec_bwd":
        pool = s["pool"].double()
        pool[s["idx"].long()] = last
        return {"y": y, "state": pool}
    loss = (y * s["dy"].double()).sum()
    if s["dhT"] is not None:
        loss = loss + (last * s["dhT"].double()).sum()
    names = {"x": "dx", "ag": "da_gate", "xg": "dx_gate", "z": "dz", "par": "da_param", "h0": "d_init_state"}
    got = dict(zip((names[k] for k in leaf), torch.autograd.grad(loss, list(leaf.values()))))
    if not c["init"]:
        del got["d_init_state"]
    return got
