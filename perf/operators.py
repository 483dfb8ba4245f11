"""What is measured of the operators around the expert block: the residual
norm (the norms before and after a block with its gate, dropout, residual
scale and residual add), the dense gated feed-forward block beside the routed
experts, and dropout from a counter-based generator.

With ``own`` false, ``run`` computes an operator in elementary torch
operations in 32 bits; with ``own`` true it makes the library's calls.

Definitions (x^ = x * rstd(x), rstd(x) = 1 / sqrt(mean(x^2) + eps)):

  residual norm   b = y^ (w_offset + w_post)      (b = y without w_post)
                  b = keep * b / (1 - p)          (with p > 0)
                  r = res + scale * gate * b      -> r, in y's type
                  n = r^ (w_offset + w_pre)       -> n, in y's type
                  the backward takes the r that the forward returned
  gated FFN       [g | u] = X W1^T, h = act(g) * u, Y = add + h W2^T
                  W1 [2I, H], gate rows first; W2 [H, I]
  dropout         out = keep * x / (1 - p), keep = (bits >= round(p 2^32))
                  bits of element (t, c): word c % 4 of Philox4x32-10
                  (Salmon et al., SC11) at counter
                  (c / 4, t, offset low, offset high) and key (seed low,
                  seed high); rng = [seed, offset], 64 bits each
"""

from __future__ import annotations

import functools
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ cases
def _norm(name, T, H, dtype, gate="none", post=True, p=0.0, scale=1.0, w_offset=0.0,
          train=False):
    return {"name": name, "op": "residual_norm", "T": T, "H": H, "dtype": dtype, "gate": gate,
            "post": post, "p": p, "scale": scale, "w_offset": w_offset, "train": train}


def _ffn(name, T, H, I, dtype, act="silu", add=False, mode="infer"):
    return {"name": name, "op": "ffn", "T": T, "H": H, "I": I, "dtype": dtype, "act": act,
            "add": add, "mode": mode}


def _drop(name, T, H, dtype, p, train=False):
    return {"name": name, "op": "dropout", "T": T, "H": H, "dtype": dtype, "p": p,
            "train": train}


def listed():
    return [
        # one token of a decoding stream between two blocks: latency
        _norm("norm decode", 1, 7168, "bf16", scale=0.22),
        # a prompt's tokens, each block output weighted by a gate per token
        _norm("norm prompt token gate", 1021, 2048, "fp16", gate="token"),
        # fine-tuning with residual dropout and a trained scale per channel
        _norm("norm train", 8192, 7168, "bf16", gate="channel", p=0.1, scale=0.5, train=True),
        # full precision, a gate per element, weights stored as w - 1, odd width
        _norm("norm train odd fp32", 3001, 2051, "fp32", gate="element", w_offset=1.0,
              train=True),
        # shared expert of the 256-expert layer, one token: the weights' bytes
        _ffn("ffn decode", 1, 7168, 2048, "bf16", add=True),
        # a ragged decoding batch
        _ffn("ffn batch", 23, 2880, 2880, "bf16", add=True),
        # the tiny test layer as a training step: launches and latency
        _ffn("ffn train tiny", 512, 256, 512, "fp16", act="gelu_tanh", mode="train"),
        # a prompt through the 2048-wide layer's block
        _ffn("ffn prompt", 1021, 2048, 768, "bf16", add=True),
        # full fine-tuning of the large shared expert: forward and all gradients
        _ffn("ffn train", 8192, 7168, 2048, "bf16", mode="train"),
        # adapter fine-tuning: frozen weights, only the input's gradient
        _ffn("ffn train frozen", 16384, 2048, 768, "bf16", mode="frozen"),
        # a small activation, forward and backward
        _drop("dropout small", 512, 256, "fp16", 0.05, train=True),
        # the routed rows that feed the adapters of one step
        _drop("dropout rows", 32768, 2880, "bf16", 0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("residual_norm", "ffn", "dropout"))
    if kind == "ffn":
        H = 16 * _log(rng, 8, 448)
        I = 16 * _log(rng, 8, 180)
        T = min(_log(rng, 1, 16384), int(8192 * 7168 * 2048 / (H * I)))
        c = _ffn("", T, H, I, rng.choice(("bf16", "bf16", "fp16")),
                 rng.choice(("silu", "silu", "gelu_tanh")), rng.random() < 0.5,
                 rng.choice(("infer", "train", "frozen")))
    else:
        H = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            H = max(64, H // 16 * 16)
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        T = min(_log(rng, 1, 32768), 8192 * 7168 * 2 // (H * SIZE[dtype]))
        train = rng.random() < 0.6
        p = rng.choice((0.05, 0.1, 0.25, 0.5))
        if kind == "dropout":
            c = _drop("", T, H, dtype, p, train)
        else:
            c = _norm("", T, H, dtype, rng.choice(("none", "token", "channel", "element")),
                      rng.random() < 0.8, p if rng.random() < 0.5 else 0.0,
                      rng.choice((1.0, 0.5, 0.22)), rng.choice((0.0, 1.0)), train)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]
    T, H = case["T"], case["H"]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dt)

    s = {"case": case}
    if case["op"] == "ffn":
        I = case["I"]
        s["X"] = normal(T, H)
        s["W1"] = normal(2 * I, H, std=0.02)
        s["W2"] = normal(H, I, std=0.02)
        s["add"] = normal(T, H) if case["add"] else None
        s["dY"] = normal(T, H) if case["mode"] != "infer" else None
        s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
        return s
    # seeds and offsets of more than 32 bits, as a run of many steps has them
    s["rng"] = torch.tensor([0x5DEECE66D00000000 % (1 << 62) + seed, (1 << 33) + 7 * seed],
                            dtype=torch.int64, device="cuda")
    if case["op"] == "dropout":
        s["x"] = normal(T, H)
        s["dy"] = normal(T, H) if case["train"] else None
        return s
    s["y"] = normal(T, H)
    s["res"] = normal(T, H)
    shape = {"none": None, "token": (T, 1), "channel": (H,), "element": (T, H)}[case["gate"]]
    s["gate"] = None if shape is None else normal(*shape, std=0.3, mean=0.5)
    centre = 1.0 - case["w_offset"]
    s["w_post"] = normal(H, std=0.1, mean=centre) if case["post"] else None
    s["w_pre"] = normal(H, std=0.1, mean=centre)
    if case["train"]:
        s["dr"] = normal(T, H)
        s["dn"] = normal(T, H)
    s["out"] = (torch.empty_like(s["y"]), torch.empty_like(s["y"]),
                torch.empty(2, T, dtype=torch.float32, device="cuda"))
    return s


# ------------------------------------------------------- the plain forms
def _round(state, _):
    """One Philox round on (c0, c1, c2, c3, k0, k1), 32-bit words in int64;
    the products wrap in 64 bits, which leaves their bits as they are."""
    c0, c1, c2, c3, k0, k1 = state
    a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
    return (((b >> 32) & M32) ^ c1 ^ k0, b & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32,
            (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32)


def _keep(T, H, p, rng):
    dev = rng.device
    groups = torch.arange((H + 3) // 4, device=dev)[None, :].expand(T, -1)
    tokens = torch.arange(T, device=dev)[:, None].expand_as(groups)
    seed, offset = rng[0], rng[1]
    start = (groups, tokens, offset & M32, (offset >> 32) & M32, seed & M32, (seed >> 32) & M32)
    words = functools.reduce(_round, range(10), start)[:4]
    return torch.stack(words, -1).reshape(T, -1)[:, :H] >= round(p * 2 ** 32)


def _drop_plain(x, p, keep):
    return torch.where(keep, x.float() / (1 - p), 0.0)


def _norm_forward_plain(s):
    c = s["case"]
    y = s["y"].float()
    rs_post = None
    b = y
    if s["w_post"] is not None:
        rs_post = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        b = y * rs_post * (c["w_offset"] + s["w_post"].float())
    keep = _keep(*y.shape, c["p"], s["rng"]) if c["p"] else None
    if keep is not None:
        b = _drop_plain(b, c["p"], keep)
    add = c["scale"] * b if s["gate"] is None else c["scale"] * s["gate"].float() * b
    r = s["res"].float() + add
    rs_pre = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    n = r * rs_pre * (c["w_offset"] + s["w_pre"].float())
    return r, n, b, keep, rs_post, rs_pre


def _norm_plain(s):
    c = s["case"]
    dt = s["y"].dtype
    r, n, b, keep, rs_post, rs_pre = _norm_forward_plain(s)
    out = {"r": r.to(dt), "n": n.to(dt)}
    if not c["train"]:
        return out
    rhat = out["r"].float() * rs_pre
    dn = s["dn"].float()
    a = dn * (c["w_offset"] + s["w_pre"].float())
    dr = s["dr"].float() + rs_pre * (a - rhat * (a * rhat).mean(1, keepdim=True))
    out["dw_pre"] = (dn * rhat).sum(0).to(dt)
    out["dres"] = dr.to(dt)
    db = c["scale"] * dr
    if s["gate"] is not None:
        dgate = db * b
        shape = s["gate"].shape
        over = () if shape == dgate.shape else (1,) if len(shape) == 2 else (0,)
        if over:
            dgate = dgate.sum(over, keepdim=len(shape) == 2)
        out["dgate"] = dgate.reshape(shape).to(dt)
        db = db * s["gate"].float()
    if keep is not None:
        db = torch.where(keep, db / (1 - c["p"]), 0.0)
    if s["w_post"] is not None:
        yhat = s["y"].float() * rs_post
        out["dw_post"] = (db * yhat).sum(0).to(dt)
        a = db * (c["w_offset"] + s["w_post"].float())
        db = rs_post * (a - yhat * (a * yhat).mean(1, keepdim=True))
    out["dy"] = db.to(dt)
    return out


def _act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 0.134145 * g * g)


def _ffn_plain(s):
    c = s["case"]
    dt = s["X"].dtype
    X, W1, W2 = s["X"].float(), s["W1"].float(), s["W2"].float()
    g, u = (X @ W1.T).chunk(2, dim=1)
    a, da = _act(c["act"], g)
    h = a * u
    Y = h @ W2.T
    if s["add"] is not None:
        Y = Y + s["add"].float()
    out = {"Y": Y.to(dt)}
    if c["mode"] == "infer":
        return out
    dY = s["dY"].float()
    dh = dY @ W2
    dZ = torch.cat((dh * u * da, dh * a), dim=1)
    out["dX"] = (dZ @ W1).to(dt)
    if c["mode"] == "train":
        out["dW1"] = (dZ.T @ X).to(dt)
        out["dW2"] = (dY.T @ h).to(dt)
    return out


def _dropout_plain(s):
    c = s["case"]
    dt = s["x"].dtype
    keep = _keep(*s["x"].shape, c["p"], s["rng"])
    out = {"out": _drop_plain(s["x"], c["p"], keep).to(dt)}
    if c["train"]:
        out["dx"] = _drop_plain(s["dy"], c["p"], keep).to(dt)
    return out


# ------------------------------------------------------- the library's calls
def _norm_own(s):
    from moe_expert_grouped_softmax_b200 import ops
    c = s["case"]
    args = dict(w_post=s["w_post"], gate=s["gate"], scale=c["scale"], w_pre=s["w_pre"],
                w_offset=c["w_offset"], p=c["p"], rng=s["rng"] if c["p"] else None)
    r, n, stats = ops.residual_norm_fwd(s["y"], s["res"], eps=EPS, out=s["out"], **args)
    out = {"r": r, "n": n}
    if c["train"]:
        dres, dy, dgate, dw_post, dw_pre = ops.residual_norm_bwd(s["dr"], s["dn"], s["y"], r,
                                                                 stats, **args)
        out["dres"], out["dy"], out["dw_pre"] = dres, dy, dw_pre
        if dgate is not None:
            out["dgate"] = dgate
        if dw_post is not None:
            out["dw_post"] = dw_post
    return out


def _ffn_own(s):
    from moe_expert_grouped_softmax_b200 import ops
    c = s["case"]
    if c["mode"] == "infer":
        Y, _ = ops.ffn_fwd(s["X"], s["W1"], s["W2"], act=c["act"], add=s["add"], out=s["out"],
                           save=False)
        return {"Y": Y}
    Y, saved = ops.ffn_fwd(s["X"], s["W1"], s["W2"], act=c["act"], add=s["add"], out=s["out"])
    dX, dW1, dW2 = ops.ffn_bwd(s["dY"], s["X"], s["W1"], s["W2"], saved, act=c["act"],
                               need_dw=c["mode"] == "train")
    out = {"Y": Y, "dX": dX}
    if c["mode"] == "train":
        out["dW1"], out["dW2"] = dW1, dW2
    return out


def _dropout_own(s):
    from moe_expert_grouped_softmax_b200 import ops
    c = s["case"]
    out = {"out": ops.dropout_fwd(s["x"], c["p"], s["rng"])}
    if c["train"]:
        out["dx"] = ops.dropout_bwd(s["dy"], c["p"], s["rng"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        if op == "ffn":
            return _ffn_own(state)
        return _norm_own(state) if op == "residual_norm" else _dropout_own(state)
    if op == "ffn":
        return _ffn_plain(state)
    return _norm_plain(state) if op == "residual_norm" else _dropout_plain(state)


# ------------------------------------------------------- bytes and operations
def work(case):
    T, H, b = case["T"], case["H"], SIZE[case["dtype"]]
    if case["op"] == "ffn":
        I = case["I"]
        weights = 3 * H * I
        passes = {"infer": 1, "frozen": 2, "train": 3}[case["mode"]]
        values = weights + (2 + case["add"]) * T * H
        if case["mode"] != "infer":
            values += 2 * T * H
        if case["mode"] == "train":
            values += weights
        return {"bytes": values * b, "flops": passes * 2 * T * weights}
    if case["op"] == "dropout":
        return {"bytes": (4 if case["train"] else 2) * T * H * b,
                "flops": (2 if case["train"] else 1) * T * H}
    gate = {"none": 0, "token": T, "channel": H, "element": T * H}[case["gate"]]
    weights = (2 if case["post"] else 1) * H
    values = 4 * T * H + gate + weights
    flops = 10 * T * H
    if case["train"]:
        values += 4 * T * H + gate + weights
        flops += 25 * T * H
    return {"bytes": values * b, "flops": flops}


# ------------------------------------------------------- the definitions in 64 bits
def _mul_high_low(c, m):
    """High and low words of the product of 32-bit words c and a constant m,
    from 16-bit halves (nothing wraps)."""
    cl, ch, ml, mh = c & 0xFFFF, c >> 16, m & 0xFFFF, m >> 16
    low = cl * ml
    mid1 = ch * ml + (low >> 16)
    mid2 = cl * mh + (mid1 & 0xFFFF)
    return ch * mh + (mid1 >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (low & 0xFFFF)


def _exact_keep(T, H, p, rng):
    seed, offset = (int(v) for v in rng.tolist())
    key = [seed & M32, seed >> 32 & M32]
    G = -(-H // 4)
    dev = rng.device
    x = [torch.arange(G, device=dev).repeat(T), torch.arange(T, device=dev).repeat_interleave(G),
         torch.full((T * G,), offset & M32, device=dev),
         torch.full((T * G,), offset >> 32 & M32, device=dev)]
    for _ in range(10):
        ah, al = _mul_high_low(x[0], 0xD2511F53)
        bh, bl = _mul_high_low(x[2], 0xCD9E8D57)
        x = [bh ^ x[1] ^ key[0], bl, ah ^ x[3] ^ key[1], al]
        key = [(key[0] + 0x9E3779B9) & M32, (key[1] + 0xBB67AE85) & M32]
    bits = torch.empty(T, G * 4, dtype=torch.int64, device=dev)
    for i in range(4):
        bits[:, i::4] = x[i].view(T, G)
    return bits[:, :H] >= round(p * 4294967296)


def _exact_norm(case, s):
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and k != "rng"}
    T, H = case["T"], case["H"]
    factor = torch.full((T, H), case["scale"], dtype=torch.float64, device=d["y"].device)
    if case["p"]:
        factor = factor * _exact_keep(T, H, case["p"], s["rng"]) / (1 - case["p"])
    gate = d["gate"].expand(T, H) if "gate" in d else torch.ones_like(factor)
    if case["post"]:
        v_post = (d["y"].pow(2).sum(1, keepdim=True) / H + EPS).sqrt()
        yhat = d["y"] / v_post
        wp = d["w_post"] + case["w_offset"]
        b = yhat * wp
    else:
        b = d["y"]
    r = d["res"] + factor * gate * b
    v = (r.pow(2).sum(1, keepdim=True) / H + EPS).sqrt()
    rhat = r / v
    wn = d["w_pre"] + case["w_offset"]
    out = {"r": r, "n": rhat * wn}
    if not case["train"]:
        return out
    gn = d["dn"] * wn
    dr = d["dr"] + (gn - rhat * ((gn * rhat).sum(1, keepdim=True) / H)) / v
    out["dres"] = dr
    out["dw_pre"] = torch.einsum("th,th->h", d["dn"], rhat)
    if "gate" in d:
        full = dr * factor * b
        out["dgate"] = {"element": lambda: full, "token": lambda: full.sum(1, keepdim=True),
                        "channel": lambda: full.sum(0)}[case["gate"]]()
    db = dr * factor * gate
    if case["post"]:
        out["dw_post"] = torch.einsum("th,th->h", db, yhat)
        gb = db * wp
        db = (gb - yhat * ((gb * yhat).sum(1, keepdim=True) / H)) / v_post
    out["dy"] = db
    return out


def _exact_ffn(case, s):
    X, W1, W2 = (s[k].double() for k in ("X", "W1", "W2"))
    I = case["I"]
    g = X.matmul(W1[:I].t()).requires_grad_(case["mode"] != "infer")
    u = X.matmul(W1[I:].t())
    with torch.enable_grad():
        if case["act"] == "silu":
            a = g * torch.sigmoid(g)
        else:
            a = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
    h = a.detach() * u
    Y = h.matmul(W2.t())
    if case["add"]:
        Y += s["add"].double()
    out = {"Y": Y}
    if case["mode"] == "infer":
        return out
    dY = s["dY"].double()
    dh = dY.matmul(W2)
    dg, = torch.autograd.grad(a, g, dh * u)
    du = dh * a.detach()
    out["dX"] = dg.matmul(W1[:I]) + du.matmul(W1[I:])
    if case["mode"] == "train":
        out["dW1"] = torch.cat((dg.t().matmul(X), du.t().matmul(X)))
        out["dW2"] = dY.t().matmul(h)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ffn":
        return _exact_ffn(case, s)
    if case["op"] == "residual_norm":
        return _exact_norm(case, s)
    keep = _exact_keep(case["T"], case["H"], case["p"], s["rng"])
    out = {"out": s["x"].double() * keep / (1 - case["p"])}
    if case["train"]:
        out["dx"] = s["dy"].double() * keep / (1 - case["p"])
    return out
