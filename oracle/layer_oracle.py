"""Plain fp64 numpy implementations of the operators around the expert block:
the residual norm, the dense gated feed-forward block and counter-based
dropout, forward and backward, one formula per line.  Test infrastructure: no
code is shared with the CUDA path."""

from __future__ import annotations

import numpy as np

M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ dropout
def philox4x32(counter, key, rounds=10):
    """Philox4x32 (Salmon et al., SC11) on arrays of 32-bit words."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        lo, s = np.uint64(M32), np.uint64(32)
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & lo, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & lo]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def keep_mask(T, H, p, seed, offset):
    """True where element (t, c) is kept: word c % 4 at counter
    (c // 4, t, offset) and key seed is at least round(p 2^32)."""
    c = np.broadcast_to(np.arange(H), (T, H))
    t = np.broadcast_to(np.arange(T)[:, None], (T, H))
    full = np.zeros((T, H), dtype=np.uint64)
    words = philox4x32((c // 4, t, full + np.uint64(offset & M32),
                        full + np.uint64((offset >> 32) & M32)),
                       (seed & M32, (seed >> 32) & M32))
    bits = np.choose(c % 4, words)
    return (bits >= np.uint64(round(p * 2 ** 32))) if p < 1 else np.zeros((T, H), dtype=bool)


def dropout(x, p, keep):
    return np.where(keep, x / (1 - p) if p < 1 else 0.0, 0.0)


# ------------------------------------------------------------ residual norm
def rstd(x, eps):
    return 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)


def residual_norm_forward(y, res=None, w_post=None, gate=None, scale=1.0, w_pre=None,
                          w_offset=0.0, eps=1e-6, p=0.0, keep=None):
    """Returns a dict with r, n (with w_pre), b and the statistics."""
    o = {"rs_post": rstd(y, eps)}
    b = y if w_post is None else y * o["rs_post"] * (w_offset + w_post)
    if p > 0:
        b = dropout(b, p, keep)
    o["b"] = b
    add = scale * b * (1.0 if gate is None else gate)
    o["r"] = add if res is None else res + add
    o["rs_pre"] = rstd(o["r"], eps)
    if w_pre is not None:
        o["n"] = o["r"] * o["rs_pre"] * (w_offset + w_pre)
    return o


def _norm_backward(d, xhat, rs):
    return rs * (d - xhat * (d * xhat).mean(1, keepdims=True))


def residual_norm_backward(dr, dn, y, r, fwd, w_post=None, gate=None, scale=1.0, w_pre=None,
                           w_offset=0.0, p=0.0, keep=None):
    """``r`` may be the rounded stream the forward returned; the statistics
    are the forward's."""
    o = {}
    d = np.zeros_like(y) if dr is None else dr
    if w_pre is not None:
        rhat = r * fwd["rs_pre"]
        o["dw_pre"] = (dn * rhat).sum(0)
        d = d + _norm_backward(dn * (w_offset + w_pre), rhat, fwd["rs_pre"])
    o["dres"] = d
    d = scale * d
    if gate is not None:
        dg = d * fwd["b"]
        o["dgate"] = dg if gate.shape == dg.shape else (
            dg.sum(0) if gate.ndim == 1 else dg.sum(1, keepdims=True))
        d = d * gate
    if p > 0:
        d = dropout(d, p, keep)
    if w_post is not None:
        yhat = y * fwd["rs_post"]
        o["dw_post"] = (d * yhat).sum(0)
        d = _norm_backward(d * (w_offset + w_post), yhat, fwd["rs_post"])
    o["dy"] = d
    return o


# --------------------------------------------------------------- gated FFN
def act(name, x):
    """act(x) and act'(x)."""
    if name == "silu":
        s = 1 / (1 + np.exp(-x))
        return x * s, s + x * s * (1 - s)
    k, c = np.sqrt(2 / np.pi), 0.044715
    t = np.tanh(k * (x + c * x ** 3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * k * (1 + 3 * c * x * x)


def ffn_forward(X, W1, W2, name="silu", add=None):
    I = W2.shape[1]
    g, u = X @ W1[:I].T, X @ W1[I:].T
    h = act(name, g)[0] * u
    Y = h @ W2.T
    return {"g": g, "u": u, "h": h, "Y": Y if add is None else Y + add}


def ffn_backward(dY, X, W1, W2, fwd, name="silu", add=None):
    a, da = act(name, fwd["g"])
    dh = dY @ W2
    dZ = np.concatenate((dh * fwd["u"] * da, dh * a), 1)
    dX = dZ @ W1
    return {"dZ": dZ, "dh": dh, "dX": dX if add is None else dX + add, "dW1": dZ.T @ X,
            "dW2": dY.T @ fwd["h"]}
