"""Cases for the selective scan, the causal conv's gradient and the q/k norm with rotation.

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
SCAN_FWD, SCAN_BWD = 16384 * 8192 * 16, 8192 * 4096 * 16  # the largest scans' T * C * S
CONV, QK = 32768 * 8192, 32768 * 32 * 128                 # the largest convs' T * C, q/k passes' T * heads * d


def listed():
    return [
        # a short prompt in one layer of a small model: latency counts
        dict(name="scan fwd short prompt", op="scan_fwd", N=1, T=64, C=1024, S=16, G=1, type="bf16", gate=True, init=False),
        # a batch of ragged prompts, some of them continued from a cached state, at the benchmark's channel count
        dict(name="scan fwd prompts", op="scan_fwd", N=16, T=16384, C=8192, S=16, G=1, type="bf16", gate=True, init=True),
        # a few requests decoding in a small fp32 model with wide states in groups
        dict(name="scan update few", op="scan_update", N=5, C=1032, S=64, G=3, type="f32", gate=False),
        # one decode step at the benchmark's batch and channel count
        dict(name="scan update batch", op="scan_update", N=256, C=8192, S=16, G=1, type="bf16", gate=True),
        # gradients of a small, odd fp32 batch with state gradients
        dict(name="scan bwd odd", op="scan_bwd", N=3, T=301, C=520, S=32, G=1, type="f32", gate=False, init=True),
        # a training step's micro-batch of packed documents
        dict(name="scan bwd training", op="scan_bwd", N=8, T=8192, C=4096, S=16, G=1, type="bf16", gate=True, init=False),
        # a small odd batch with conv states on both ends
        dict(name="conv bwd odd", op="conv_bwd", N=5, T=333, C=1032, W=3, type="f32", act=True, init=True),
        # the benchmark's backward workload, 8 x 4096 tokens packed, over its 8192 channels
        dict(name="conv bwd training", op="conv_bwd", N=8, T=32768, C=8192, W=4, type="bf16", act=True, init=False),
        # a decode batch of the benchmark's size, partly rotated wide heads
        dict(name="qk decode", op="qk", T=256, HQ=16, HK=2, d=256, rd=64, type="bf16", norm="rms", weight=True, inter=False),
        # a prompt through the benchmark's heads, L2 norm, all of a head rotated
        dict(name="qk prompt", op="qk", T=32768, HQ=16, HK=16, d=128, rd=128, type="bf16", norm="l2", weight=False, inter=False),
        # an odd fp32 batch, neighbouring pairs rotated
        dict(name="qk bwd odd", op="qk_bwd", T=1001, HQ=6, HK=3, d=80, rd=80, type="f32", norm="rms", weight=True, inter=True),
        # the benchmark's backward workload with learned norm weights
        dict(name="qk bwd training", op="qk_bwd", T=32768, HQ=16, HK=16, d=128, rd=128, type="bf16", norm="rms", weight=True, inter=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_update", "scan_bwd", "conv_bwd", "qk", "qk_bwd"])
    t = rng.choice(["bf16", "f32"])
    if op in ("qk", "qk_bwd"):
        d = rng.choice([64, 80, 96, 112, 128, 192, 256])
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        hq = hk * rng.choice([1, 1, 2, 3, 8])
        rd = d if rng.random() < 0.6 else 16 * rng.randint(0, d // 16)
        T = min(_log(rng, 1, 32768), max(1, QK // ((hq + hk) * d * (2 if t == "f32" else 1))))
        norm = rng.choice(["rms", "l2"])
        return dict(op=op, T=T, HQ=hq, HK=hk, d=d, rd=rd, type=t, norm=norm, weight=norm == "rms", inter=rng.random() < 0.3)
    if op == "conv_bwd":
        C = 8 * _log(rng, 4, 1024)
        T = min(_log(rng, 1, 32768), max(1, CONV // (C * (2 if t == "f32" else 1))))
        return dict(op=op, N=rng.randint(1, min(T, 16)), T=T, C=C, W=rng.choice([2, 3, 4, 4, 5, 8]), type=t, act=rng.random() < 0.8,
                    init=rng.random() < 0.5)
    S = rng.choice([8, 16, 16, 32, 64])
    G = rng.choice([1, 1, 2, 3])
    C = 8 * G * _log(rng, 8, 1024 // G)
    if op == "scan_update":
        return dict(op=op, N=min(_log(rng, 1, 512), max(1, 256 * 8192 * 16 // (C * S * (2 if t == "f32" else 1)))), C=C, S=S, G=G,
                    type=t, gate=rng.random() < 0.5)
    most = (SCAN_FWD if op == "scan_fwd" else SCAN_BWD) // (C * S * (2 if t == "f32" else 1))
    T = min(_log(rng, 1, 16384), max(1, most))
    return dict(op=op, N=rng.randint(1, min(T, 16)), T=T, C=C, S=S, G=G, type=t, gate=rng.random() < 0.6, init=rng.random() < 0.5)


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
    if c["op"] in ("qk", "qk_bwd"):
        T, HQ, HK, d, rd = c["T"], c["HQ"], c["HK"], c["d"], c["rd"]
        qkv = randn(T, (HQ + 2 * HK) * d).to(ty)  # q, k and v side by side, as the projection or the conv leaves them
        s["q"] = qkv[:, :HQ * d].unflatten(1, (HQ, d))
        s["k"] = qkv[:, HQ * d:(HQ + HK) * d].unflatten(1, (HK, d))
        P = max(4096, T)
        angle = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rd, 2, device=DEV, dtype=torch.float64) / max(rd, 1))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["positions"] = torch.randint(0, P, (T,), generator=gen, device=DEV, dtype=torch.int32)
        s["qw"] = 1 + 0.1 * randn(d) if c["weight"] else None
        s["kw"] = 1 + 0.1 * randn(d) if c["weight"] else None
        if c["op"] == "qk_bwd":
            s["dqo"], s["dko"] = randn(T, HQ, d).to(ty), randn(T, HK, d).to(ty)
        return s
    C = c["C"]
    if c["op"] != "scan_update":
        lens = lengths(c)
        s["longest"] = max(lens)
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    if c["op"] == "conv_bwd":
        W = c["W"]
        s["x"], s["dy"] = randn(c["T"], C).to(ty), randn(c["T"], C).to(ty)
        s["w"], s["b"] = randn(C, W) / math.sqrt(W), 0.1 * randn(C)
        s["h0"] = randn(c["N"], W - 1, C).to(ty) if c["init"] else None
        s["dhT"] = randn(c["N"], W - 1, C).to(ty) if c["init"] else None
        return s
    T, S, G = c.get("T", c["N"]), c["S"], c["G"]
    s["x"] = randn(T, C).to(ty)
    s["dt"] = (0.5 * randn(T, C)).to(ty)
    s["z"] = randn(T, 2 * C).to(ty)[:, C:] if c["gate"] else None  # the second half of the input projection
    low = randn(T, 64 + 2 * G * S).to(ty)                          # a low-rank dt, then B and C, as one projection gives them
    s["B"] = low[:, 64:64 + G * S].unflatten(1, (G, S))
    s["C_"] = low[:, 64 + G * S:].unflatten(1, (G, S))
    s["A_log"] = torch.log(torch.arange(1, S + 1, device=DEV, dtype=torch.float32)).repeat(C, 1) + 0.05 * randn(C, S)
    step = torch.exp(math.log(1e-3) + torch.rand(C, generator=gen, device=DEV) * math.log(100.0))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))           # softplus(dt_bias) = step, in 0.001 .. 0.1
    s["D"] = 1 + 0.1 * randn(C)
    if c["op"] == "scan_bwd":
        s["dy"] = randn(T, C).to(ty)
        s["h0"] = randn(c["N"], C, S) if c["init"] else None
        s["dhT"] = randn(c["N"], C, S) if c["init"] else None
        return s
    slots = c["N"] + 3
    s["pool"] = randn(slots, C, S)
    s["idx"] = torch.randperm(slots, generator=gen, device=DEV)[:c["N"]].to(torch.int32)
    if c["op"] == "scan_fwd":
        has = torch.arange(c["N"], device=DEV) % 3 != 0 if c["init"] else torch.zeros(c["N"], device=DEV)
        s["has"] = has.to(torch.int32)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---------------------------------------------------------------- the plain forms


def _silu(x):
    return x / (1 + torch.exp(-x))


def _dsilu(x):
    p = 1 / (1 + torch.exp(-x))
    return p * (1 + x * (1 - p))


def _softplus(v):
    return torch.maximum(v, torch.zeros_like(v)) + torch.log1p(torch.exp(-v.abs()))


def _channels(v, C):
    """[T, G, S] of the groups as [T, C, S] of their channels."""
    return v.float().repeat_interleave(C // v.shape[1], dim=1)


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


def _where(s, T):
    """Each token's sequence, whether it is its first, whether it is its last."""
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:], t, right=True)
    return seq, t == s["cu"][seq], t == s["cu"][seq + 1] - 1


def _scan_fwd(s):
    T = s["x"].shape[0]
    seq, first, last = _where(s, T)
    x = s["x"].float()
    d = _softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(d[:, :, None] * -torch.exp(s["A_log"]))
    b = (d * x)[:, :, None] * _channels(s["B"], s["C"])
    slot = s["idx"].long()
    h0 = s["pool"][slot] * (s["has"] != 0)[:, None, None]
    start, keep = s["cu"][:-1].long(), s["cu"][1:] > s["cu"][:-1]
    at = start.clamp(max=T - 1)
    b.index_add_(0, at, torch.where(keep[:, None, None], a[at] * h0, 0))
    a.mul_(~first[:, None, None])
    h = _recur(a, b, s["longest"])
    y = (h * _channels(s["C_"], s["C"])).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    end = (s["cu"][1:].long() - 1).clamp(min=0)
    s["pool"][slot] = torch.where(keep[:, None, None], h[end], h0)
    return {"y": y.to(s["x"].dtype), "state": s["pool"]}


def _scan_update(s):
    x = s["x"].float()
    d = _softplus(s["dt"].float() + s["dt_bias"])
    slot = s["idx"].long()
    h = torch.exp(d[:, :, None] * -torch.exp(s["A_log"])) * s["pool"][slot] + (d * x)[:, :, None] * _channels(s["B"], s["C"])
    s["pool"][slot] = h
    y = (h * _channels(s["C_"], s["C"])).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"y": y.to(s["x"].dtype), "state": s["pool"]}


def _scan_bwd(s):
    T, C, G, ty = s["x"].shape[0], s["C"], s["G"], s["x"].dtype
    seq, first, last = _where(s, T)
    x, dy = s["x"].float(), s["dy"].float()
    raw = s["dt"].float() + s["dt_bias"]
    d = _softplus(raw)
    A = -torch.exp(s["A_log"])
    a = torch.exp(d[:, :, None] * A)
    Bc, Cc = _channels(s["B"], C), _channels(s["C_"], C)
    b = (d * x)[:, :, None] * Bc
    ran = s["cu"][1:] > s["cu"][:-1]
    start, end = s["cu"][:-1].long().clamp(max=T - 1), (s["cu"][1:].long() - 1).clamp(min=0)
    if s["h0"] is not None:
        b.index_add_(0, start, torch.where(ran[:, None, None], a[start] * s["h0"], 0))
    h = _recur(a * ~first[:, None, None], b, s["longest"])
    old = torch.cat([torch.zeros_like(h[:1]), h[:-1]]) * ~first[:, None, None]
    if s["h0"] is not None:
        old.index_add_(0, start, torch.where(ran[:, None, None], s["h0"], 0))
    out = {}
    e = dy
    if s["z"] is not None:
        z = s["z"].float()
        out["dz"] = (dy * ((h * Cc).sum(-1) + s["D"] * x) * _dsilu(z)).to(ty)
        e = dy * _silu(z)
    g = e[:, :, None] * Cc
    if s["dhT"] is not None:
        g.index_add_(0, end, torch.where(ran[:, None, None], s["dhT"], 0))
    after = torch.cat([a[1:], torch.zeros_like(a[:1])]) * ~last[:, None, None]
    g = _recur(after.flip(0), g.flip(0), s["longest"]).flip(0)
    s1 = (g * Bc).sum(-1)
    w = g * a * old
    out["dx"] = (d * s1 + s["D"] * e).to(ty)
    ddt = (x * s1 + (w * A).sum(-1)) / (1 + torch.exp(-raw))
    out["ddt"] = ddt.to(ty)
    out["dA_log"] = (w * d[:, :, None]).sum(0) * A
    out["dB"] = (g * (d * x)[:, :, None]).unflatten(1, (G, C // G)).sum(2).to(ty)
    out["dC"] = (h * e[:, :, None]).unflatten(1, (G, C // G)).sum(2).to(ty)
    out["dD"] = (e * x).sum(0)
    out["ddt_bias"] = ddt.sum(0)
    if s["h0"] is not None:
        out["d_init_state"] = torch.where(ran[:, None, None], (a * g)[start], s["dhT"])
    return out


def _conv_bwd(s):
    T, W, N, ty = s["x"].shape[0], s["W"], s["N"], s["x"].dtype
    seq, _, _ = _where(s, T)
    cu = s["cu"].long()
    bos, eos = cu[:-1], cu[1:]
    x, w = s["x"].float(), s["w"].t()
    tap = torch.arange(W, device=DEV)
    before = torch.arange(W - 1, device=DEV)
    zero = torch.zeros_like(x[:1])
    past = s["h0"].float().reshape(N * (W - 1), -1) if s["h0"] is not None else zero.expand(N * (W - 1), -1)
    t = torch.arange(T, device=DEV)
    src = t[:, None] - (W - 1) + tap
    src = torch.where(src >= bos[seq][:, None], src, T + seq[:, None] * (W - 1) + src - bos[seq][:, None] + W - 1)
    xw = torch.cat([x, past])[src]
    p = s["dy"].float()
    if s["act"]:
        p = p * _dsilu((xw * w).sum(1) + s["b"])
    out = {"dweight": (p[:, None] * xw).sum(0).t().contiguous(), "dbias": p.sum(0)}
    p = torch.cat([p, zero])
    to = t[:, None] + W - 1 - tap
    dx = (p[torch.where(to < eos[seq][:, None], to, T)] * w).sum(1)
    if s["dhT"] is not None:
        tail = torch.cat([s["dhT"].float().reshape(N * (W - 1), -1), zero])
        j = t - eos[seq] + W - 1
        dx = dx + tail[torch.where(j >= 0, seq * (W - 1) + j, N * (W - 1))]
        to = bos[:, None, None] + before[:, None] - tap
        dh = (p[torch.where((tap <= before[:, None]) & (to < eos[:, None, None]), to, T)] * w).sum(2)
        j = before - (eos - bos)[:, None]
        dh = dh + tail[torch.where(j >= 0, torch.arange(N, device=DEV)[:, None] * (W - 1) + j, N * (W - 1))]
        out["d_init_state"] = dh.to(ty)
    out["dx"] = dx.to(ty)
    return out


def _turn(s, n, back):
    """The rotation by each token's angles of the first rd values of a head; back: by their negatives."""
    rd, at = s["rd"], s["positions"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None] * (-1 if back else 1)
    u, v = (n[..., 0:rd:2], n[..., 1:rd:2]) if s["inter"] else (n[..., :rd // 2], n[..., rd // 2:rd])
    u, v = u * cos - v * sin, v * cos + u * sin
    front = torch.stack([u, v], -1).flatten(-2) if s["inter"] else torch.cat([u, v], -1)
    return torch.cat([front, n[..., rd:]], -1)


def _scale(s, x):
    ss = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((ss / s["d"] if s["norm"] == "rms" else ss) + 1e-6)


def _qk(s, x, w):
    x = x.float()
    n = x * _scale(s, x)
    return _turn(s, n if w is None else n * w, False).to(TYPES[s["type"]])


def _qk_bwd(s, x, w, do):
    x = x.float()
    r = _scale(s, x)
    dn = _turn(s, do.float(), True)
    g = dn if w is None else dn * w
    share = 1 / s["d"] if s["norm"] == "rms" else 1.0
    dx = r * g - x * r ** 3 * share * (g * x).sum(-1, keepdim=True)
    return dx.to(TYPES[s["type"]]), (dn * x * r).sum((0, 1)) if w is not None else None


def run(state):
    s = state
    op = s["op"]
    if own:
        return _own(s)
    if op == "scan_fwd":
        return _scan_fwd(s)
    if op == "scan_update":
        return _scan_update(s)
    if op == "scan_bwd":
        return _scan_bwd(s)
    if op == "conv_bwd":
        return _conv_bwd(s)
    if op == "qk":
        return {"q": _qk(s, s["q"], s["qw"]), "k": _qk(s, s["k"], s["kw"])}
    dq, dqw = _qk_bwd(s, s["q"], s["qw"], s["dqo"])
    dk, dkw = _qk_bwd(s, s["k"], s["kw"], s["dko"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


# ---------------------------------------------------------------- this package's entry points


def _own(s):
    import invariant_linear_attention_gb300 as gdn
    op = s["op"]
    if op == "scan_fwd":
        y = gdn.gdn_selective_scan_fwd(s["x"], s["dt"], s["A_log"], s["B"], s["C_"], s["cu"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                                       state=s["pool"], state_indices=s["idx"], has_initial_state=s["has"])
        return {"y": y, "state": s["pool"]}
    if op == "scan_update":
        y = gdn.gdn_selective_scan_update(s["x"], s["dt"], s["A_log"], s["B"], s["C_"], s["pool"], state_indices=s["idx"], D=s["D"],
                                          z=s["z"], dt_bias=s["dt_bias"])
        return {"y": y, "state": s["pool"]}
    if op == "scan_bwd":
        return gdn.gdn_selective_scan_bwd(s["x"], s["dt"], s["A_log"], s["B"], s["C_"], s["cu"], s["dy"], D=s["D"], z=s["z"],
                                          dt_bias=s["dt_bias"], init_state=s["h0"], d_final_state=s["dhT"], need_d_init_state=s["init"])
    if op == "conv_bwd":
        return gdn.gdn_causal_conv1d_bwd(s["x"], s["w"], s["cu"], s["dy"], bias=s["b"], init_state=s["h0"], d_final_state=s["dhT"],
                                         activation=s["act"], need_d_init_state=s["init"])
    if op == "qk":
        q, k = gdn.gdn_qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], positions=s["positions"], q_weight=s["qw"], k_weight=s["kw"],
                                    norm=s["norm"], eps=1e-6, interleaved=s["inter"])
        return {"q": q, "k": k}
    return gdn.gdn_qk_norm_rope_bwd(s["q"], s["k"], s["cos"], s["sin"], s["dqo"], s["dko"], positions=s["positions"], q_weight=s["qw"],
                                    k_weight=s["kw"], norm=s["norm"], eps=1e-6, interleaved=s["inter"])


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    e = 2 if c["type"] == "bf16" else 4
    if c["op"] in ("qk", "qk_bwd"):
        n = c["T"] * (c["HQ"] + c["HK"]) * c["d"]
        angles = 4 * c["T"] * (c["rd"] + 1)
        return {"bytes": n * e * (2 if c["op"] == "qk" else 3) + angles, "flops": n * (8 if c["op"] == "qk" else 16)}
    if c["op"] == "conv_bwd":
        n = c["T"] * c["C"]
        states = (3 if c["init"] else 0) * c["N"] * (c["W"] - 1) * c["C"] * e
        return {"bytes": 3 * n * e + states + 8 * c["C"] * (c["W"] + 1), "flops": n * (6 * c["W"] + 8)}
    T, C, S = c.get("T", c["N"]), c["C"], c["S"]
    n, bc, par, states = T * C, 2 * T * c["G"] * S, 4 * C * (S + 2), 4 * c["N"] * C * S
    if c["op"] == "scan_bwd":
        moved = n * e * (7 if c["gate"] else 5) + 2 * bc * e + 2 * par + (3 * states if c["init"] else 0)
        return {"bytes": moved, "flops": n * (26 * S + 30)}
    moved = n * e * (4 if c["gate"] else 3) + bc * e + par
    read = sum(i % 3 != 0 for i in range(c["N"])) / c["N"] if c.get("init") else 0 if c["op"] == "scan_fwd" else 1
    return {"bytes": moved + states * (1 + read), "flops": n * (7 * S + 20)}


# ---------------------------------------------------------------- the definitions, in 64 bits


def _f64(v):
    return None if v is None else v.double()


def _pad(v, lens, longest):
    """Packed rows as [sequence, row, ...], the rows behind a sequence's end filled with its neighbours'."""
    at = np.concatenate([[0], np.cumsum(lens)[:-1]])[:, None] + np.arange(longest)
    return v[torch.from_numpy(np.minimum(at, v.shape[0] - 1)).to(v.device)]


def _pack(v, lens):
    return torch.cat([v[n, :m] for n, m in enumerate(lens)])


def _walk(x, dt, z, B, C, A_log, D, bias, h, lens):
    """The recurrence token by token, all sequences side by side; (y [N, longest, C], the last states)."""
    m = torch.tensor(lens, device=x.device)[:, None, None]
    A = -torch.exp(A_log)
    per = A.shape[0] // B.shape[2]
    ys = []
    for t, (xt, dtt, zt, Bt, Ct) in enumerate(zip(*(v.unbind(1) for v in (x, dt, z, B, C)))):
        step = torch.nn.functional.softplus(dtt + bias, threshold=40.0)[..., None]
        new = torch.exp(step * A) * h + step * xt[..., None] * Bt.repeat_interleave(per, 1)
        ys.append((torch.einsum("ncs,ncs->nc", new, Ct.repeat_interleave(per, 1)) + D * xt) * zt)
        h = torch.where(t < m, new, h)
    return torch.stack(ys, 1), h


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    op = c["op"]
    if op in ("qk", "qk_bwd"):
        got = {}
        for name, w, do in (("q", "qw", "dqo"), ("k", "kw", "dko")):
            x = s[name].double().contiguous().requires_grad_()
            wt = torch.ones(c["d"], dtype=torch.float64, device=DEV) if s[w] is None else s[w].double()
            wt.requires_grad_()
            length = x.square().mean(-1, keepdim=True) if c["norm"] == "rms" else x.square().sum(-1, keepdim=True)
            n = x / torch.sqrt(length + 1e-6) * wt
            half = c["rd"] // 2
            pairs = n[..., :c["rd"]].unflatten(-1, (half, 2) if c["inter"] else (2, half))
            pairs = pairs if c["inter"] else pairs.transpose(-1, -2)
            spin = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"].long()][:, None]
            pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * spin)
            pairs = pairs if c["inter"] else pairs.transpose(-1, -2)
            o = torch.cat([pairs.reshape(*n.shape[:-1], c["rd"]), n[..., c["rd"]:]], -1)
            if op == "qk":
                got[name] = o.detach()
            else:
                got["d" + name], g = torch.autograd.grad(o, (x, wt), s[do].double())
                got["d" + name + "_weight"] = g if s[w] is not None else None
        return got
    T, C = c.get("T", c["N"]), c["C"]
    lens = lengths(c) if op != "scan_update" else [1] * c["N"]
    longest = max(lens)
    if op == "conv_bwd":
        W = c["W"]
        x, w, b = (_f64(s[k]).requires_grad_() for k in ("x", "w", "b"))
        h0 = (torch.zeros(c["N"], W - 1, C, dtype=torch.float64, device=DEV) if s["h0"] is None else _f64(s["h0"])).requires_grad_()
        at, loss = 0, 0.0
        for n, m in enumerate(lens):
            rows = torch.cat([h0[n], x[at:at + m]])
            if m:
                pre = b + sum(w[:, i] * rows[i:i + m] for i in range(W))
                y = torch.nn.functional.silu(pre) if c["act"] else pre
                loss = loss + (y * s["dy"][at:at + m].double()).sum()
            if s["dhT"] is not None:
                loss = loss + (rows[m:] * s["dhT"][n].double()).sum()
            at += m
        dx, dw, db, dh = torch.autograd.grad(loss, (x, w, b, h0))
        return {"dx": dx, "dweight": dw, "dbias": db, **({"d_init_state": dh} if c["init"] else {})}
    if c["N"] * longest * C * 8 * (10 * c["S"] if op == "scan_bwd" else 8) > 150e9:  # what autograd keeps, or the padded rows
        return None
    leaf = {k: _f64(s[k]) for k in ("x", "dt", "z", "B", "C_", "A_log", "D", "dt_bias") if s[k] is not None}
    if op == "scan_bwd":
        for v in leaf.values():
            v.requires_grad_()
    gate = torch.nn.functional.silu(leaf["z"]) if "z" in leaf else torch.ones(T, C, dtype=torch.float64, device=DEV)
    rows = [_pad(v, lens, longest) for v in (leaf["x"], leaf["dt"], gate, leaf["B"], leaf["C_"])]
    if op != "scan_bwd":
        slot = s["idx"].long()
        h0 = s["pool"].double()[slot]
        if op == "scan_fwd":
            h0 = h0 * (s["has"] != 0)[:, None, None]
        y, h = _walk(*rows, leaf["A_log"], leaf["D"], leaf["dt_bias"], h0, lens)
        pool = s["pool"].double()
        pool[slot] = h
        return {"y": _pack(y, lens), "state": pool}
    h0 = (torch.zeros(c["N"], C, c["S"], dtype=torch.float64, device=DEV) if s["h0"] is None else _f64(s["h0"])).requires_grad_()
    y, h = _walk(*rows, leaf["A_log"], leaf["D"], leaf["dt_bias"], h0, lens)
    loss = (_pack(y, lens) * s["dy"].double()).sum()
    if s["dhT"] is not None:
        loss = loss + (h * s["dhT"].double()).sum()
    names = {"x": "dx", "dt": "ddt", "z": "dz", "B": "dB", "C_": "dC", "A_log": "dA_log", "D": "dD", "dt_bias": "ddt_bias"}
    grads = torch.autograd.grad(loss, list(leaf.values()) + [h0])
    got = {names[k]: g for k, g in zip(leaf, grads)}
    if c["init"]:
        got["d_init_state"] = grads[-1]
    return got
