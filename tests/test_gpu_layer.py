"""The residual norm, the dense gated feed-forward block and dropout on the
GPU against the fp64 oracle.

Tolerances.  u = finfo(type).eps / 2 is the half step that rounding to the
output's type may cost.  An fp32 sum of n terms, in any order, is off by at
most n 2^-24 times the sum of the terms' magnitudes; the tests bound every
other fp32 operation of a value by 64 more such steps (rsqrt, exp, division
and the few products of each formula), so G(n) = (n + 64) 2^-24.  The tensor
cores may cut rather than round: their sums count 2 G.  Each bound below adds
those terms along the formula; ``tiny`` is half of fp16's smallest step."""

import functools

import numpy as np
import pytest
import torch

from moe_expert_grouped_softmax_b200 import ops
from oracle import layer_oracle as LO

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = 2.0 ** -25


def half_step(name):
    return torch.finfo(TYPES[name]).eps / 2


def G(n):
    return (n + 64) * 2.0 ** -24


def n64(t):
    return None if t is None else t.double().cpu().numpy()


def randn(gen, *shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen) * std + mean).to(dtype).cuda()


def close(got, ref, bound, name):
    got = n64(got)
    assert got.shape == ref.shape, name
    off = np.abs(got - ref) - bound
    at = np.unravel_index(np.argmax(off), off.shape) if off.size else ()
    assert not off.size or off[at] <= 0, (
        f"{name}{list(map(int, at))}: {got[at]} for {ref[at]}, allowed {np.broadcast_to(bound, ref.shape)[at]}")


def status_ok():
    torch.cuda.synchronize()
    assert ops.device_status() == 0


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,shift", [(1, 1, 0), (1, 4, 0), (3, 7, 0), (5, 8, 0), (64, 208, 0),
                                       (33, 2880, 0), (7, 1111, 0), (9, 64, 1)])
def test_dropout(cuda_ok, dtype, T, H, shift):
    """Kept elements are x / (1 - p) with one rounding (two fp32 ones before
    it), dropped ones are zero; the mask is the oracle's bit for bit, on rows
    of any length and alignment (``shift``: elements past a 16-byte edge)."""
    p, seed, offset = 0.3, (5 << 40) + 17, (3 << 33) + 9
    gen = torch.Generator().manual_seed(T * H)
    x = torch.empty(T * H + shift, dtype=TYPES[dtype], device="cuda")[shift:].view(T, H)
    x.copy_(torch.randn(T, H, generator=gen))
    rng = torch.tensor([seed, offset], device="cuda")
    out = ops.dropout_fwd(x, p, rng)
    keep = LO.keep_mask(T, H, p, seed, offset)
    ref = LO.dropout(n64(x), p, keep)
    close(out, ref, (half_step(dtype) + 2.0 ** -22) * np.abs(ref) + TINY, "out")
    assert np.array_equal(n64(out) != 0, keep & (n64(x) != 0))
    # the backward draws the same mask; in place gives the same bytes
    dx = ops.dropout_bwd(x, p, rng)
    assert torch.equal(dx, out)
    assert torch.equal(ops.dropout_fwd(x, p, rng, out=x), out)
    status_ok()


def test_dropout_extremes(cuda_ok):
    """p = 0 keeps everything, p = 1 nothing; dropped infinities and NaN are
    zeros; negative seeds and offsets are 64-bit words; no rows."""
    x = torch.randn(40, 50, device="cuda", dtype=torch.bfloat16)
    rng = torch.tensor([-3, -(1 << 40)], device="cuda")
    assert torch.equal(ops.dropout_fwd(x, 0.0, rng), x)
    x[::2, ::3] = float("nan")
    x[1::2, ::3] = float("inf")
    assert not ops.dropout_fwd(x, 1.0, rng).any()
    keep = LO.keep_mask(40, 50, 0.5, -3 & (2 ** 64 - 1), -(1 << 40) & (2 ** 64 - 1))
    out = ops.dropout_fwd(x, 0.5, rng)
    assert not out[torch.tensor(~keep).cuda()].any()
    assert torch.equal(out.isnan().cpu(), x.isnan().cpu() & torch.tensor(keep))
    assert ops.dropout_fwd(x[:0], 0.5, rng).shape == (0, 50)
    status_ok()


# ------------------------------------------------------------ residual norm
NORM_CASES = [
    # T, H, dtype, gate, post, pre, res, p, scale, w_offset, shift
    (1, 64, "bf16", "none", True, True, True, 0.0, 1.0, 0.0, 0),
    (5, 7168, "bf16", "channel", True, True, True, 0.1, 0.5, 0.0, 0),
    (300, 256, "bf16", "channel", True, True, True, 0.25, 0.5, 1.0, 0),
    (37, 2880, "fp16", "token", True, True, True, 0.0, 0.22, 0.0, 0),
    (9, 2051, "fp32", "element", True, True, True, 0.0, 1.0, 1.0, 0),
    (13, 2051, "bf16", "element", True, True, True, 0.5, 1.0, 0.0, 0),
    (6, 1, "fp32", "channel", True, True, True, 0.0, 1.0, 0.0, 0),
    (11, 3, "fp16", "token", True, True, True, 0.1, 1.0, 0.0, 0),
    (3, 16384, "fp32", "channel", True, True, True, 0.1, 0.5, 0.0, 0),
    (3, 16384, "bf16", "element", True, True, True, 0.1, 0.5, 0.0, 0),
    (4, 16383, "fp16", "channel", True, True, True, 0.0, 0.5, 0.0, 0),
    (700, 520, "fp32", "none", True, True, True, 0.0, 1.0, 0.0, 1),
    (20, 512, "bf16", "none", False, True, False, 0.0, 1.0, 0.0, 0),   # norm before a block
    (20, 4096, "fp16", "none", False, True, True, 0.0, 1.0, 0.0, 0),   # residual add + norm
    (20, 512, "bf16", "token", True, False, True, 0.3, 0.7, 0.0, 0),   # norm after, no next
    (20, 130, "fp32", "channel", False, False, True, 0.3, 0.7, 0.0, 0),  # no norm at all
    (20, 512, "bf16", "none", True, False, False, 0.0, 1.0, 0.0, 0),
    (1500, 96, "bf16", "none", True, True, True, 0.1, 1.0, 0.0, 0),    # several rows a block
    (700, 8192, "bf16", "channel", True, True, True, 0.1, 0.5, 0.0, 0),
    (500, 7168, "fp32", "element", True, True, True, 0.1, 0.5, 0.0, 0),
    (600, 3584, "fp16", "token", True, True, True, 0.0, 0.5, 0.0, 0),
    (400, 4097, "bf16", "token", True, True, True, 0.2, 0.5, 1.0, 0),
    (350, 12288, "fp32", "none", True, True, True, 0.0, 0.5, 0.0, 0),
]


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: "-".join(map(str, c)))
def test_residual_norm(cuda_ok, case):
    T, H, dtype, gate, post, pre, with_res, p, scale, w_offset, shift = case
    dt, u, eps = TYPES[dtype], half_step(dtype), 1e-6
    gen = torch.Generator().manual_seed(T + H)

    def tensor(*shape, std=1.0, mean=0.0):
        n = int(np.prod(shape))
        t = torch.empty(n + shift, dtype=dt, device="cuda")[shift:].view(*shape)
        return t.copy_(torch.randn(*shape, generator=gen) * std + mean)

    y = tensor(T, H)
    res = tensor(T, H) if with_res else None
    shape = {"none": None, "token": (T, 1), "channel": (H,), "element": (T, H)}[gate]
    gt = None if shape is None else tensor(*shape, std=0.3, mean=0.5)
    w_post = tensor(H, std=0.1, mean=1 - w_offset) if post else None
    w_pre = tensor(H, std=0.1, mean=1 - w_offset) if pre else None
    dr, dn = tensor(T, H), tensor(T, H) if pre else None
    seed, offset = 1234567, 89
    rng = torch.tensor([seed, offset], device="cuda") if p else None
    keep = LO.keep_mask(T, H, p, seed, offset) if p else None
    args = dict(w_post=w_post, gate=gt, scale=scale, w_pre=w_pre, w_offset=w_offset, p=p, rng=rng)
    nargs = dict(w_post=n64(w_post), gate=n64(gt), scale=scale, w_pre=n64(w_pre),
                 w_offset=w_offset, p=p, keep=keep)

    r, n, stats = ops.residual_norm_fwd(y, res, eps=eps, **args)
    f = LO.residual_norm_forward(n64(y), n64(res), eps=eps, **nargs)
    # fp32 error of r: of b (a sum over H and a few products), then one sum
    ref_add = f["r"] - (0 if res is None else n64(res))
    r32 = G(H) * (np.abs(ref_add) + (0 if res is None else np.abs(n64(res))))
    close(r, f["r"], u * np.abs(f["r"]) + (1 + u) * r32 + TINY, "r")
    if pre:
        w = np.abs(w_offset + n64(w_pre))
        # r^ w: r's error, and the statistic's (relative: half of mean(r^2)'s,
        # which is at most G(H) + 2 sum|r| r32 / sum r^2)
        rel = G(H) + (np.abs(f["r"]) * r32).sum(1, keepdims=True) / (f["r"] ** 2).sum(1, keepdims=True)
        n32 = f["rs_pre"] * w * (r32 + rel * np.abs(f["r"]))
        close(n, f["n"], u * np.abs(f["n"]) + (1 + u) * n32 + TINY, "n")
    else:
        assert n is None

    got = ops.residual_norm_bwd(dr, dn, y, r, stats, **args)
    rr = n64(r)
    b = LO.residual_norm_backward(n64(dr), n64(dn), n64(y), rr, f, **nargs)
    # dres = dr + rs (a - r^ mean(a r^)): every term's magnitude, summed
    mag = np.abs(n64(dr))
    srel = G(H)
    if pre:
        a = np.abs(n64(dn)) * np.abs(w_offset + n64(w_pre))
        rhat = np.abs(rr) * f["rs_pre"]
        srel = 4 * (G(H) + rel)  # the saved statistic enters up to three times
        mag = mag + f["rs_pre"] * (a + rhat * (a * rhat).mean(1, keepdims=True))
        e = np.abs(n64(dn)) * rhat
        ref = b["dw_pre"]
        close(got[4], ref, u * np.abs(ref) + ((G(T) + srel) * e).sum(0) + TINY, "dw_pre")
    d32 = srel * mag
    close(got[0], b["dres"], u * np.abs(b["dres"]) + (1 + u) * d32 + TINY, "dres")
    ks = scale * (np.where(keep, 1 / (1 - p), 0) if p else 1.0)
    if gate != "none":
        bb = np.abs(scale * f["b"])
        e = bb * (d32 + G(H) * (np.abs(b["dres"]) + d32))
        if gate == "token":
            e = e.sum(1, keepdims=True) + G(H) * (bb * np.abs(b["dres"])).sum(1, keepdims=True)
        elif gate == "channel":
            e = e.sum(0) + G(T) * (bb * np.abs(b["dres"])).sum(0)
        close(got[2], b["dgate"], u * np.abs(b["dgate"]) + e + TINY, "dgate")
    else:
        assert got[2] is None
    gabs = 1.0 if gt is None else np.abs(n64(gt))
    db, db32 = ks * gabs * np.abs(b["dres"]), ks * gabs * (d32 + G(8) * np.abs(b["dres"]))
    if post:
        yhat = np.abs(n64(y)) * f["rs_post"]
        wp = np.abs(w_offset + n64(w_post))
        e = (yhat * (db32 + (G(H) + G(T)) * db)).sum(0)
        close(got[3], b["dw_post"], u * np.abs(b["dw_post"]) + e + TINY, "dw_post")
        x, x32 = db * wp, db32 * wp

        def through(v):
            return f["rs_post"] * (v + yhat * (v * yhat).mean(1, keepdims=True))

        db, db32 = through(x), through(x32) + 4 * G(H) * through(x)
    close(got[1], b["dy"], u * np.abs(b["dy"]) + (1 + u) * (db32 + G(8) * db) + TINY, "dy")
    # the same call again gives the same bytes
    again = ops.residual_norm_bwd(dr, dn, y, r, stats, **args)
    for x, z in zip(got, again):
        assert x is None or torch.equal(x, z)
    status_ok()


@pytest.mark.parametrize("T", [23, 900])
def test_residual_norm_in_place_and_empty(cuda_ok, T):
    """r over res and n over y, dres over dr and dy over dn, give the bytes of
    separate outputs (also where a block's later rows are on their way); rows
    behind T stay as they were; T = 0."""
    H = 2880
    gen = torch.Generator().manual_seed(1)
    y, res, dr, dn = (randn(gen, T + 2, H, dtype=torch.bfloat16) for _ in range(4))
    w = randn(gen, H, dtype=torch.bfloat16, std=0.1, mean=1.0)
    r, n, stats = ops.residual_norm_fwd(y[:T], res[:T], w_post=w, w_pre=w)
    want = ops.residual_norm_bwd(dr[:T], dn[:T], y[:T], r, stats, w_post=w, w_pre=w)
    tail = [t[T:].clone() for t in (y, res, dr, dn)]
    dw = [torch.empty_like(w) for _ in range(2)]
    keep_y = y[:T].clone()
    ops.residual_norm_bwd(dr[:T], dn[:T], keep_y, r, stats, w_post=w, w_pre=w,
                          out=(dr[:T], dn[:T], None, *dw))
    for a, b in zip((dr[:T], dn[:T], *dw), (want[0], want[1], want[3], want[4])):
        assert torch.equal(a, b)
    ops.residual_norm_fwd(y[:T], res[:T], w_post=w, w_pre=w, out=(res[:T], y[:T], stats))
    assert torch.equal(res[:T], r) and torch.equal(y[:T], n)
    for t, keep in zip((y, res, dr, dn), tail):
        assert torch.equal(t[T:], keep)
    r0, n0, s0 = ops.residual_norm_fwd(y[:0], res[:0], w_pre=w)
    assert n0.shape == (0, H)
    g0 = ops.residual_norm_bwd(None, n0, y[:0], r0, s0, w_pre=w)
    assert g0[0].shape == (0, H) and not g0[4].any()
    status_ok()


# --------------------------------------------------------------- gated FFN
def ffn_check(T, H, I, dtype, act, add, train, seed=0):
    dt, u = TYPES[dtype], half_step(dtype)
    gen = torch.Generator().manual_seed(seed + T + H + I)
    X = randn(gen, T, H, dtype=dt)
    W1 = randn(gen, 2 * I, H, dtype=dt, std=0.05)
    W2 = randn(gen, H, I, dtype=dt, std=0.05)
    ad = randn(gen, T, H, dtype=dt) if add else None
    x, w1, w2, nad = n64(X), n64(W1), n64(W2), n64(ad)
    f = LO.ffn_forward(x, w1, w2, act, nad)
    A = np.abs
    # g, u: sums over H.  h: |act'| <= 1.13 for both, exp and division within
    # G; one rounding.  Y: sum over I, of the rounded h; one rounding.
    gb, ub = (2 * G(H) * (A(x) @ A(w1[s]).T) for s in (slice(0, I), slice(I, 2 * I)))
    a, da = LO.act(act, f["g"])
    ab = 1.13 * gb + G(0) * (A(a) + A(f["g"]) * A(a))  # exp's error grows with |g|
    h32 = A(f["u"]) * ab + (A(a) + ab) * ub
    hb = u * A(f["h"]) + (1 + u) * h32 + TINY
    Yb = hb @ A(w2).T + 2 * G(I) * (A(f["h"]) + hb) @ A(w2).T + G(2) * A(f["Y"] if nad is None else nad)
    Y, saved = ops.ffn_fwd(X, W1, W2, act=act, add=ad, save=train)
    close(Y, f["Y"], u * A(f["Y"]) + (1 + u) * Yb + TINY, "Y")
    # the roundings of h and Y are independent of the signs they are summed
    # with: in the 2-norm each costs at most u
    def l2(got, ref, steps, name):
        err = np.linalg.norm(n64(got) - ref) / np.linalg.norm(ref)
        assert err <= steps * u + 2 * G(H + 2 * I + T), f"{name}: {err}"
    l2(Y, f["Y"], 2, "Y")
    if not train:
        assert saved is None
        status_ok()
        return
    dY = randn(gen, T, H, dtype=dt)
    ad2 = randn(gen, T, H, dtype=dt) if add else None
    dy = n64(dY)
    b = LO.ffn_backward(dy, x, w1, w2, f, act, n64(ad2))
    dX, dW1, dW2 = ops.ffn_bwd(dY, X, W1, W2, saved, act=act, add=ad2)
    # dh: a sum over H; |act''| <= 1.13 for both; dZ: one rounding
    dhb = 2 * G(H) * (A(dy) @ A(w2))
    dab = 1.13 * gb + G(0) * (1 + A(f["g"])) ** 2
    uu, dh = A(f["u"]), A(b["dh"])
    dgb = (dhb * uu * A(da) + dh * ub * A(da) + dh * uu * dab) * (1 + 2.0 ** -10) + G(0) * dh * uu * A(da)
    dub = (dhb * A(a) + dh * ab) * (1 + 2.0 ** -10) + G(0) * dh * A(a)
    dZb = np.concatenate((dgb, dub), 1) * (1 + u) + u * A(b["dZ"]) + TINY
    dZm = A(b["dZ"]) + dZb
    bound = dZb @ A(w1) + 2 * G(2 * I) * dZm @ A(w1) + (0 if ad2 is None else G(2) * A(n64(ad2)))
    close(dX, b["dX"], u * A(b["dX"]) + (1 + u) * bound + TINY, "dX")
    close(dW1, b["dW1"], u * A(b["dW1"]) + (1 + u) * (dZb.T @ A(x) + 2 * G(T) * dZm.T @ A(x)) + TINY,
          "dW1")
    close(dW2, b["dW2"], u * A(b["dW2"]) + (1 + u) * (A(dy).T @ hb + 2 * G(T) * A(dy).T @ (A(f["h"]) + hb))
          + TINY, "dW2")
    for got, name in ((dX, "dX"), (dW1, "dW1"), (dW2, "dW2")):
        l2(got, b[name], 2, name)
    # frozen weights: dX (perhaps by another split of the sums), nothing else
    fX, f1, f2 = ops.ffn_bwd(dY, X, W1, W2, saved, act=act, add=ad2, need_dw=False)
    assert f1 is None and f2 is None
    close(fX, b["dX"], u * A(b["dX"]) + (1 + u) * bound + TINY, "dX (frozen weights)")
    # inference gives the training forward's bytes
    assert torch.equal(ops.ffn_fwd(X, W1, W2, act=act, add=ad, save=False)[0], Y)
    status_ok()


@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 17, 23, 32, 33, 64, 100, 127, 128, 129, 255, 257])
def test_ffn_lengths(cuda_ok, T):
    ffn_check(T, 208, 80, "bf16", "silu", True, True)


@pytest.mark.parametrize("case", [
    (1, 64, 64, "bf16", "silu", False), (3, 64, 64, "fp16", "gelu_tanh", True),
    (1, 2880, 2880, "bf16", "silu", True), (16, 1024, 528, "fp16", "silu", False),
    (40, 2064, 272, "bf16", "gelu_tanh", True), (300, 256, 512, "fp16", "gelu_tanh", True),
    (513, 576, 304, "bf16", "silu", False), (1000, 128, 1040, "bf16", "silu", True),
    (600, 1040, 144, "fp16", "silu", False), (77, 528, 2064, "fp16", "silu", True),
], ids=lambda c: "-".join(map(str, c)))
def test_ffn_shapes(cuda_ok, case):
    ffn_check(*case, train=True)


@pytest.mark.parametrize("T", [1, 7, 50])
def test_ffn_inference_only(cuda_ok, T):
    ffn_check(T, 320, 192, "bf16", "silu", True, False)


@pytest.mark.parametrize("T,H,I,dtype,act", [
    (4153, 2064, 1040, "bf16", "silu"), (5000, 1536, 4112, "fp16", "gelu_tanh"),
    (1300, 4096, 2064, "bf16", "silu"), (9000, 768, 2320, "bf16", "silu"),
    (20000, 64, 80, "bf16", "silu"), (70000, 80, 64, "fp16", "gelu_tanh"),
])
def test_ffn_many_tiles(cuda_ok, T, H, I, dtype, act):
    """Several rounds of tiles per pair of CTAs, the gradients' GEMMs of
    unequal length in one launch, ragged in every dimension.  In the 2-norm a
    result's own rounding and that of the values it is summed from (h or dZ)
    cost at most u each, and the fp32 sums 2 G of their length; every 256th
    row is also held to twice that of its own norm (a row's roundings need
    not be as even as the whole's)."""
    u = half_step(dtype)
    gen = torch.Generator(device="cuda").manual_seed(T)

    def draw(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(TYPES[dtype])

    X, dY, W1, W2 = draw(T, H), draw(T, H), draw(2 * I, H, std=0.03), draw(H, I, std=0.03)
    Y, saved = ops.ffn_fwd(X, W1, W2, act=act)
    dX, dW1, dW2 = ops.ffn_bwd(dY, X, W1, W2, saved, act=act)
    x, dy, w1, w2 = X.double(), dY.double(), W1.double(), W2.double()
    g, up = (x @ w1.T).chunk(2, 1)
    g = g.clone().requires_grad_()
    a = torch.nn.functional.silu(g) if act == "silu" else \
        torch.nn.functional.gelu(g, approximate="tanh")
    dh = dy @ w2
    dg, = torch.autograd.grad(a, g, dh * up)
    a = a.detach()
    dZ = torch.cat((dg, dh * a), 1)
    for got, ref, n, name in ((Y, (a * up) @ w2.T, H + I, "Y"), (dX, dZ @ w1, H + 2 * I, "dX"),
                              (dW1, dZ.T @ x, H + T, "dW1"), (dW2, dy.T @ (a * up), H + T, "dW2")):
        err, norm = got.double() - ref, ref.norm()
        assert err.norm() <= (2 * u + 2 * G(n)) * norm, (name, float(err.norm() / norm))
        rows = err[::256].norm(dim=1) / ref[::256].norm(dim=1)
        assert rows.max() <= 2 * (2 * u + 2 * G(n)), (name, float(rows.max()))
    for _ in range(8):  # the same bytes every time
        Y2, saved = ops.ffn_fwd(X, W1, W2, act=act)
        again = ops.ffn_bwd(dY, X, W1, W2, saved, act=act)
        assert torch.equal(Y2, Y) and all(map(torch.equal, again, (dX, dW1, dW2)))
    status_ok()


@pytest.mark.parametrize("T", [1, 8, 16, 24, 32, 40, 128, 500])
def test_ffn_repeats(cuda_ok, T):
    """Wide weights at few rows: the same bytes every time, calls back to back
    on alternating inputs, and within the roundings' 2-norm of fp64."""
    H, I, u = 2880, 1440, half_step("bf16")
    gen = torch.Generator(device="cuda").manual_seed(T)

    def draw(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    W1, W2 = draw(2 * I, H, std=0.03), draw(H, I, std=0.03)
    X = [draw(T, H) for _ in range(2)]
    want = [ops.ffn_fwd(x, W1, W2, save=False)[0] for x in X]
    for x, y in zip(X, want):
        g, up = (x.double() @ W1.double().T).chunk(2, 1)
        ref = (torch.nn.functional.silu(g) * up) @ W2.double().T
        err = (y.double() - ref).norm() / ref.norm()
        assert err <= 2 * u + 2 * G(H + I), float(err)
    got = [ops.ffn_fwd(X[i % 2], W1, W2, save=False)[0] for i in range(40)]
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))
    status_ok()


def test_ffn_in_place_tail_and_empty(cuda_ok):
    """Y over add and dX over its add give the bytes of separate outputs; rows
    behind T stay as they were; no rows leave zero weight gradients."""
    H, I = 256, 144
    gen = torch.Generator().manual_seed(2)
    W1 = randn(gen, 2 * I, H, dtype=torch.bfloat16, std=0.05)
    W2 = randn(gen, H, I, dtype=torch.bfloat16, std=0.05)
    for T in (1, 13, 70, 300):
        X, ad, dY = (randn(gen, T + 3, H, dtype=torch.bfloat16) for _ in range(3))
        Y, saved = ops.ffn_fwd(X[:T], W1, W2, add=ad[:T])
        dX, _, _ = ops.ffn_bwd(dY[:T], X[:T], W1, W2, saved, add=ad[:T], need_dw=False)
        a1, a2 = ad.clone(), ad.clone()
        ops.ffn_fwd(X[:T], W1, W2, add=a1[:T], out=a1[:T])
        ops.ffn_bwd(dY[:T], X[:T], W1, W2, saved, add=a2[:T], need_dw=False,
                    out=(a2[:T], None, None))
        assert torch.equal(a1[:T], Y) and torch.equal(a2[:T], dX)
        assert torch.equal(a1[T:], ad[T:]) and torch.equal(a2[T:], ad[T:])
    Y, saved = ops.ffn_fwd(X[:0], W1, W2)
    dX, dW1, dW2 = ops.ffn_bwd(dY[:0], X[:0], W1, W2, saved)
    assert Y.shape == dX.shape == (0, H) and not dW1.any() and not dW2.any()
    status_ok()


# ------------------------------------------------- streams, graphs, failures
@pytest.mark.parametrize("gate", ["none", "token", "channel", "element"])
def test_residual_norm_against_differences(cuda_ok, gate):
    """<gradient, v> of the fp32 kernels against the central difference of
    their own forward along v.  Rows have norm sqrt(96) and move by 1e-2 of
    it, so the difference's truncation is of order 1e-4 of the derivative and
    fp32 rounding 1e-5; 5e-3 leaves room for the third derivative's factor."""
    T, H, p, h = 8, 96, 0.25, 1e-2
    gen = torch.Generator().manual_seed(5)
    x = {n: randn(gen, T, H, dtype=torch.float32) for n in ("y", "res", "dr", "dn")}
    x["w_post"], x["w_pre"] = (randn(gen, H, dtype=torch.float32, std=0.1, mean=1.0)
                               for _ in range(2))
    shape = {"none": None, "token": (T, 1), "channel": (H,), "element": (T, H)}[gate]
    x["gate"] = None if shape is None else randn(gen, *shape, dtype=torch.float32, mean=1.0)
    rng = torch.tensor([3, 4], device="cuda")

    def forward(a):
        return ops.residual_norm_fwd(a["y"], a["res"], a["w_post"], a["gate"], 0.7, a["w_pre"],
                                     p=p, rng=rng)

    def loss(a):
        r, n, _ = forward(a)
        return float((r.double() * x["dr"]).sum() + (n.double() * x["dn"]).sum())

    r, n, stats = forward(x)
    grads = ops.residual_norm_bwd(x["dr"], x["dn"], x["y"], r, stats, x["w_post"], x["gate"], 0.7,
                                  x["w_pre"], p=p, rng=rng)
    for name, g in zip(("res", "y", "gate", "w_post", "w_pre"), grads):
        if g is None:
            continue
        # along the gradient itself, scaled to a unit step per element
        v = g / g.square().mean().sqrt()
        up, down = dict(x), dict(x)
        up[name], down[name] = x[name] + h * v, x[name] - h * v
        want = float((g.double() * v).sum())
        got = (loss(up) - loss(down)) / (2 * h)
        assert abs(got - want) <= 5e-3 * abs(want), (name, got, want)


@pytest.mark.parametrize("T", [3, 70, 700])
def test_graphs_and_streams(cuda_ok, T):
    """Forward and backward of all three operators on a stream of its own, and
    captured into two graphs (each with buffers from its own pool), replayed
    in turn on new inputs, give the eager call's bytes."""
    H, I = 320, 192
    gen = torch.Generator().manual_seed(T)
    W1 = randn(gen, 2 * I, H, dtype=torch.bfloat16, std=0.05)
    W2 = randn(gen, H, I, dtype=torch.bfloat16, std=0.05)
    w = randn(gen, H, dtype=torch.bfloat16, std=0.1, mean=1.0)
    rng = torch.tensor([9, 9], device="cuda")
    inputs = [[randn(gen, T, H, dtype=torch.bfloat16) for _ in range(2)] for _ in range(3)]

    def run(x, g):
        r, n, st = ops.residual_norm_fwd(x, w_pre=w)
        y, saved = ops.ffn_fwd(n, W1, W2)
        d = ops.dropout_fwd(y, 0.25, rng)
        dy = ops.dropout_bwd(g, 0.25, rng)
        dn, d1, d2 = ops.ffn_bwd(dy, n, W1, W2, saved)
        dx, _, _, _, dw = ops.residual_norm_bwd(g, dn, x, r, st, w_pre=w)
        return d, dx, dw, d1, d2

    want = [run(*i) for i in inputs]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = run(*inputs[0])
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    bufs, graphs, outs = [], [], []
    for _ in range(2):
        x, g = inputs[0][0].clone(), inputs[0][1].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(x, g))
        bufs.append((x, g))
        graphs.append(graph)
    for i, j in ((0, 1), (1, 2), (2, 0)):
        for (x, g), graph, k in zip(bufs, graphs, (i, j)):
            x.copy_(inputs[k][0])
            g.copy_(inputs[k][1])
            graph.replay()
        torch.cuda.synchronize()
        for out, k in zip(outs, (i, j)):
            assert all(torch.equal(a, b) for a, b in zip(out, want[k]))
    status_ok()


@pytest.mark.parametrize("T", [64, 1500])
def test_wait_timeout_is_reported_and_context_survives(cuda_ok, T):
    """The dense kernels' waits are bounded too: on few rows (K split over a
    cluster) and on many (CTA pairs)."""
    H, I = 1024, 576
    gen = torch.Generator().manual_seed(T)
    W1 = randn(gen, 2 * I, H, dtype=torch.bfloat16, std=0.05)
    W2 = randn(gen, H, I, dtype=torch.bfloat16, std=0.05)
    X, dY = (randn(gen, T, H, dtype=torch.bfloat16) for _ in range(2))
    Y, saved = ops.ffn_fwd(X, W1, W2)
    want = ops.ffn_bwd(dY, X, W1, W2, saved)
    status_ok()
    ops.set_wait_limit_ns(2_000_000)  # 2 ms
    ops.test_inject_stall(True)
    try:
        s2 = ops.ffn_fwd(X, W1, W2)[1]
        ops.ffn_bwd(dY, X, W1, W2, s2)
        torch.cuda.synchronize()
        st = ops.device_status()
    finally:
        ops.test_inject_stall(False)
        ops.set_wait_limit_ns(0)
    assert st == 4, ops.STATUS_NAMES.get(st, st)
    Y2, saved = ops.ffn_fwd(X, W1, W2)
    assert torch.equal(Y2, Y)
    assert all(torch.equal(a, b) for a, b in zip(ops.ffn_bwd(dY, X, W1, W2, saved), want))
    status_ok()


def test_binding_refusals(cuda_ok):
    """Types, shapes, layouts and devices that the binding turns down."""
    bf = torch.bfloat16
    x = torch.zeros(6, 64, dtype=bf, device="cuda")
    w = torch.zeros(64, dtype=bf, device="cuda")
    w1, w2 = torch.zeros(256, 64, dtype=bf, device="cuda"), torch.zeros(64, 128, dtype=bf, device="cuda")
    rng = torch.zeros(2, dtype=torch.int64, device="cuda")
    saved = ops.ffn_fwd(x, w1, w2)[1]
    bad = [
        lambda: ops.dropout_fwd(x.double(), 0.5, rng),
        lambda: ops.dropout_fwd(x[0], 0.5, rng),
        lambda: ops.dropout_fwd(x.t(), 0.5, rng),
        lambda: ops.dropout_fwd(x[:, :32], 0.5, rng),
        lambda: ops.dropout_fwd(x, 1.5, rng),
        lambda: ops.dropout_fwd(x, 0.5, rng.int()),
        lambda: ops.dropout_fwd(x, 0.5, rng.cpu()),
        lambda: ops.dropout_fwd(x, 0.5, None),
        lambda: ops.residual_norm_fwd(x),
        lambda: ops.residual_norm_fwd(x, x.float(), w_pre=w),
        lambda: ops.residual_norm_fwd(x, x[:5], w_pre=w),
        lambda: ops.residual_norm_fwd(x, w_pre=w[:63]),
        lambda: ops.residual_norm_fwd(x, x, gate=w[:6]),
        lambda: ops.residual_norm_fwd(x, x, p=0.5),
        lambda: ops.residual_norm_bwd(x, x, x, x, torch.zeros(2, 6, device="cuda")),
        lambda: ops.residual_norm_bwd(None, None, x, x, torch.zeros(2, 6, device="cuda")),
        lambda: ops.residual_norm_bwd(x, x, x, x, torch.zeros(6, device="cuda"), w_pre=w),
        lambda: ops.ffn_fwd(x.float(), w1.float(), w2.float()),
        lambda: ops.ffn_fwd(x, w1[:128], w2),
        lambda: ops.ffn_fwd(x, w1, w2, act="relu"),
        lambda: ops.ffn_fwd(x, w1, w2, add=x.half()),
        lambda: ops.ffn_fwd(x, w1, w2, save=False, ws=torch.zeros(8, dtype=torch.uint8, device="cuda")),
        lambda: ops.ffn_bwd(x, x, w1, w2, saved[:-1]),
        lambda: ops.ffn_bwd(None, x, w1, w2, saved),
        lambda: ops.ffn_fwd(torch.zeros(6 * 64 + 1, dtype=bf, device="cuda")[1:].view(6, 64), w1, w2),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, ops.MoeError)):
            call()
            pytest.fail(f"call {i} was accepted")
    status_ok()


@pytest.mark.parametrize("T,H,dtype,status", [
    (2000, 2880, "bf16", [4, 4]), (20000, 64, "fp16", [4, 4]), (1500, 8192, "bf16", [4, 4]),
    (1000, 7168, "fp32", [0, 4]),  # this forward's threads load for themselves: no wait
])
def test_norm_wait_timeout_is_reported_and_context_survives(cuda_ok, T, H, dtype, status):
    """The norm's waits for its rows are bounded too, and after one that ran
    out no barrier is armed again: several rows a block and more than the ring
    holds, one to four of them in flight, rows of one warp."""
    gen = torch.Generator().manual_seed(T)
    y, res, dr, dn = (randn(gen, T, H, dtype=TYPES[dtype]) for _ in range(4))
    w = randn(gen, H, dtype=TYPES[dtype], std=0.1, mean=1.0)
    fwd = lambda: ops.residual_norm_fwd(y, res, w_post=w, w_pre=w)  # noqa: E731
    r, n, stats = fwd()
    bwd = lambda: ops.residual_norm_bwd(dr, dn, y, r, stats, w_post=w, w_pre=w)  # noqa: E731
    want = bwd()
    status_ok()
    seen = []
    ops.set_wait_limit_ns(2_000_000)  # 2 ms
    ops.test_inject_stall(True)
    try:
        for call in (fwd, bwd):
            call()
            torch.cuda.synchronize()
            seen.append(ops.device_status())
    finally:
        ops.test_inject_stall(False)
        ops.set_wait_limit_ns(0)
    assert seen == status, [ops.STATUS_NAMES.get(s, s) for s in seen]
    r2, n2, _ = fwd()
    assert torch.equal(r2, r) and torch.equal(n2, n)
    for a, b in zip(bwd(), want):
        assert b is None or torch.equal(a, b)
    status_ok()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("offset,word", [(1870304274, 0), (4265977243, 1), (491251087, 2)])
def test_dropout_at_the_largest_words(cuda_ok, dtype, offset, word):
    """Words 2^32 - 1 (the first two offsets) and 2^32 - 2 (the third) against
    the thresholds round(p 2^32) of 2^32 - 1 and, from p = 1 - 2^-33 on, 2^32,
    which no word reaches; scaled by 2^32 exactly, or zero.  Dropout alone and
    inside the norm."""
    seed, H = 77, 4
    x = torch.full((1, H), 2.0 ** -20, dtype=TYPES[dtype], device="cuda")
    rng = torch.tensor([seed, offset], device="cuda")
    for e in (32, 33, 34, 50):
        p = 1 - 2.0 ** -e
        keep = LO.keep_mask(1, H, p, seed, offset)
        assert keep.sum() == (e == 32 and word < 2) and (not keep.any() or keep[0, word])
        want = LO.dropout(n64(x), p, keep)
        assert np.array_equal(n64(ops.dropout_fwd(x, p, rng)), want), e
        assert np.array_equal(n64(ops.residual_norm_fwd(x, p=p, rng=rng)[0]), want), e
    status_ok()


@pytest.mark.parametrize("T", [9, 200, 5000])
def test_ffn_fp16_range(cuda_ok, T):
    """The documented range of fp16: h or dZ past 65504 becomes infinite where
    an fp32 pass would stay finite.  What is summed from it is infinite or NaN
    (that row of Y or dX, its column of dW2 or row of dW1); other rows have
    the bytes of a pass without it.  Token kernel, clusters and CTA pairs."""
    H, I, bad = 256, 320, T // 2
    gen = torch.Generator().manual_seed(T)
    X, dY = (randn(gen, T, H, dtype=torch.float16) for _ in range(2))
    W1 = randn(gen, 2 * I, H, dtype=torch.float16, std=0.05)
    W2 = randn(gen, H, I, dtype=torch.float16, std=0.001)
    others = torch.arange(T, device="cuda") != bad

    def row(x, w1, dy):
        f = LO.ffn_forward(n64(x[bad:bad + 1]), n64(w1), n64(W2), "silu")
        return f, LO.ffn_backward(n64(dy[bad:bad + 1]), n64(x[bad:bad + 1]), n64(w1), n64(W2), f, "silu")

    def past(v):
        over, under = (torch.tensor(m, device="cuda") for m in (np.abs(v) > 66000, np.abs(v) < 65000))
        assert over.any() and under.any()
        return over, under

    # h: g and u of standard deviation 240
    dY[bad] *= 0.01
    want = ops.ffn_fwd(X, W1, W2)[0]
    X2 = X.clone()
    X2[bad] *= 300
    f, _ = row(X2, W1, dY)
    over, under = past(f["h"][0])
    assert np.abs(f["Y"]).max() < 65000
    Y, saved = ops.ffn_fwd(X2, W1, W2)
    assert not Y[bad].isfinite().any()
    assert torch.equal(Y[others], want[others])
    dW2 = ops.ffn_bwd(dY, X2, W1, W2, saved)[2]
    assert not dW2[:, over].isfinite().any() and dW2[:, under].isfinite().all()

    # dZ: a row with one element, whose up weights give u = 80 beside a dh of
    # standard deviation 960
    X2, W3 = X.clone(), W1.clone()
    X2[:, 0] = X2[bad] = 0
    X2[bad, 0] = 0.5
    W3[:I, 0], W3[I:, 0] = 4, 160
    saved = ops.ffn_fwd(X2, W3, W2)[1]
    want = ops.ffn_bwd(dY, X2, W3, W2, saved)[0]
    dY2 = dY.clone()
    dY2[bad] = 60000 * dY[bad].sign()
    over, under = past(row(X2, W3, dY2)[1]["dZ"][0])
    dX, dW1, _ = ops.ffn_bwd(dY2, X2, W3, W2, saved)
    assert not dX[bad].isfinite().any()
    assert torch.equal(dX[others], want[others])
    assert not dW1[over, 0].isfinite().any() and dW1[under].isfinite().all()
    status_ok()


# ------------------------------------------------ many rows a block or thread
@pytest.mark.parametrize("case", [
    # more rows a block than its ring holds, so that stages are filled again
    (2000, 2880, "bf16", "element", True, True, True, 0.1, 0.5, 0.0, 0),
    (1000, 8192, "bf16", "channel", True, True, True, 0.0, 0.5, 0.0, 0),   # 16 elements a thread
    (1300, 2048, "fp32", "token", True, True, True, 0.0, 1.0, 1.0, 0),
    (12000, 64, "fp16", "none", True, True, True, 0.1, 1.0, 0.0, 0),       # rows of one warp
    (6000, 1024, "bf16", "channel", True, False, True, 0.1, 0.5, 0.0, 0),  # no norm after it
    (12000, 64, "bf16", "none", False, False, True, 0.0, 0.5, 0.0, 0),     # no sum at all
    (1500, 2051, "bf16", "element", True, True, True, 0.1, 0.5, 0.0, 0),   # without the ring
], ids=lambda c: "-".join(map(str, c)))
def test_residual_norm_many_rows_a_block(cuda_ok, case):
    test_residual_norm(cuda_ok, case)


def test_residual_norm_in_place_many_rows_a_block(cuda_ok):
    """Rows overwritten while later ones of the same block are on their way."""
    test_residual_norm_in_place_and_empty(cuda_ok, 2500)


@functools.lru_cache(maxsize=None)
def keep_mask(T, H, p, seed, offset):
    """The oracle's mask, drawn once per group of four columns."""
    groups, rows = np.arange((H + 3) // 4)[None, :], np.arange(T)[:, None]
    full = np.zeros((T, groups.size), dtype=np.uint64)
    words = LO.philox4x32((full + groups.astype(np.uint64), full + rows.astype(np.uint64),
                           full + np.uint64(offset & LO.M32), full + np.uint64(offset >> 32)),
                          (seed & LO.M32, seed >> 32))
    return np.stack(words, -1).reshape(T, -1)[:, :H] >= np.uint64(round(p * 2 ** 32))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,shift", [
    (3000, 2880, 0),      # 32-byte pieces, several strides of the grid
    (3000, 2888, 0),      # rows that are 16-byte aligned only, in the 16-bit types
    (3000, 2880, 16),     # bytes past a 32-byte edge
    (3000, 2880, 8),
    (4000, 2051, 0),      # unaligned
    (3, 1300016, 0),      # rows longer than the grid's stride
    (5, 700001, 0),
])
def test_dropout_many_pieces_a_thread(cuda_ok, dtype, T, H, shift):
    """Threads that take several pairs of pieces: the mask bit for bit, and
    kept elements scaled with one rounding."""
    p, seed, offset = 0.3, (5 << 40) + 17, (3 << 33) + 9
    shift //= TYPES[dtype].itemsize
    gen = torch.Generator(device="cuda").manual_seed(T)
    buf = torch.full((T * H + shift + 8,), 3.0, dtype=TYPES[dtype], device="cuda")
    out = buf[shift:shift + T * H].view(T, H)
    x = torch.empty(T * H + shift, dtype=TYPES[dtype], device="cuda")[shift:].view(T, H)
    x.copy_(torch.randn(T, H, generator=gen, device="cuda"))
    x[x == 0] = 1
    rng = torch.tensor([seed, offset], device="cuda")
    keep = torch.tensor(keep_mask(T, H, p, seed, offset), device="cuda")
    ops.dropout_fwd(x, p, rng, out=out)
    assert torch.equal(out != 0, keep)
    ref = torch.where(keep, x.double() / (1 - p), 0.0)
    bound = (half_step(dtype) + 2.0 ** -22) * ref.abs() + TINY
    assert ((out.double() - ref).abs() <= bound).all()
    assert (buf[:shift] == 3).all() and (buf[shift + T * H:] == 3).all()
    assert torch.equal(ops.dropout_fwd(x, p, rng, out=x), out)
    status_ok()


def test_past_32_bit_offsets(cuda_ok):
    """More than 2^31 elements a tensor: rows around each place where an
    element's or a byte's offset passes 32 bits, and the last ones."""
    T, H, p = 300007, 7168, 0.25
    rows = sorted({0, T // 2, T - 1} | {min(T - 1, 2 ** e // (H * b) + d) for e in (31, 32)
                                        for b in (1, 2) for d in (-1, 0, 1)})
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    rng = torch.tensor([3, 4], device="cuda")
    out = ops.dropout_fwd(x, p, rng)
    for t in rows:
        words = LO.philox4x32(tuple(np.broadcast_to(np.uint64(v), (H // 4,)) for v in
                                    (np.arange(H // 4), t, 4, 0)), (3, 0))
        keep = torch.tensor(np.stack(words, -1).reshape(-1) >= np.uint64(2 ** 30), device="cuda")
        ref = torch.where(keep, x[t].double() / (1 - p), 0.0)
        assert torch.equal(out[t], ref.to(torch.bfloat16)), t
    # r is one fp32 sum, rounded; n and dres: the statistic's sum over H, one
    # rounding; dw: one rounding, the additions' of random sign far below it
    w = torch.empty(H, dtype=torch.bfloat16, device="cuda").normal_(1, 0.1, generator=gen)
    r, n, stats = ops.residual_norm_fwd(x, out, w_pre=w)
    dres, dy, _, _, dw = ops.residual_norm_bwd(None, out, x, r, stats, w_pre=w)
    u = half_step("bf16")
    want_dw = torch.zeros(H, dtype=torch.float64, device="cuda")
    for t0 in range(0, T, 16384):
        rr = r[t0:t0 + 16384].double()
        rh = rr * (rr.square().mean(1, keepdim=True) + 1e-6).rsqrt()
        want_dw += (out[t0:t0 + 16384].double() * rh).sum(0)
    assert (dw.double() - want_dw).norm() <= 2 * u * want_dw.norm()
    for t in rows:
        v = x[t].float() + out[t].float()
        assert torch.equal(r[t], v.to(torch.bfloat16)), t
        v = v.double()
        rs = (v.square().mean() + 1e-6).rsqrt()
        ref = v * rs * w.double()
        assert ((n[t].double() - ref).abs() <= (u + 2 * G(H)) * ref.abs() + TINY).all(), t
        a, rh = out[t].double() * w.double(), r[t].double() * rs
        ref = rs * (a - rh * (a * rh).mean())
        mag = rs * (a.abs() + rh.abs() * (a * rh).abs().mean())
        assert ((dres[t].double() - ref).abs() <= u * ref.abs() + 4 * G(H) * mag + TINY).all(), t
    assert dy is dres
    status_ok()


def test_ffn_past_32_bit_offsets(cuda_ok):
    """More than 2^32 saved values, and a reduction over 300007 rows."""
    T, H, I, u = 300007, 128, 7168, half_step("bf16")
    gen = torch.Generator(device="cuda").manual_seed(2)

    def draw(*shape, std=1.0):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=gen)

    X, dY, W1, W2 = draw(T, H), draw(T, H), draw(2 * I, H, std=H ** -0.5), draw(H, I, std=I ** -0.5)
    Y, saved = ops.ffn_fwd(X, W1, W2)
    dX, dW1, dW2 = ops.ffn_bwd(dY, X, W1, W2, saved)
    w1, w2 = W1.double(), W2.double()
    want1, want2 = torch.zeros_like(w1), torch.zeros_like(w2)
    for t0 in range(0, T, 8192):
        x, dy = X[t0:t0 + 8192].double(), dY[t0:t0 + 8192].double()
        g, up = (x @ w1.T).chunk(2, 1)
        s = torch.sigmoid(g)
        a, dh = g * s, dy @ w2
        dZ = torch.cat((dh * up * s * (1 + g * (1 - s)), dh * a), 1)
        for got, ref in ((Y, (a * up) @ w2.T), (dX, dZ @ w1)):
            err = (got[t0:t0 + 8192].double() - ref).norm(dim=1) / ref.norm(dim=1)
            assert err.max() <= 2 * (2 * u + 2 * G(H + 2 * I)), t0
        want1 += dZ.T @ x
        want2 += dy.T @ (a * up)
    for got, ref in ((dW1, want1), (dW2, want2)):
        # its own rounding and dZ's or h's; each MMA of 16 rows may cut a step
        # of its partial sum
        assert (got.double() - ref).norm() <= (2 * u + T / 16 * 2.0 ** -23) * ref.norm()
    status_ok()
