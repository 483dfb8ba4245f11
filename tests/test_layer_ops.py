"""The operators around the expert block on the CPU: the fp64 oracle pinned
against published vectors, autograd and finite differences; the library's
argument checks, each of which returns before anything is launched; and the
binding's."""

import ctypes

import numpy as np
import pytest
import torch

from moe_expert_grouped_softmax_b200 import build, ops
from oracle import layer_oracle as LO


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.lib()


# ------------------------------------------------------------------ oracle
@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((LO.M32,) * 4, (LO.M32,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    """The known-answer vectors published with the generator."""
    assert tuple(int(w) for w in LO.philox4x32(counter, key)) == want


def test_keep_mask_share_and_independence():
    T, H, p = 200, 301, 0.3
    a = LO.keep_mask(T, H, p, 7, 1)
    # binomial: 60200 draws, sd of the share 0.0019; 5 sd
    assert abs(a.mean() - (1 - p)) < 5 * np.sqrt(p * (1 - p) / (T * H))
    b = LO.keep_mask(T, H, p, 7, 2)
    agree = (a == b).mean()
    want = (1 - p) ** 2 + p ** 2
    assert abs(agree - want) < 5 * np.sqrt(want * (1 - want) / (T * H))
    assert not LO.keep_mask(3, 5, 1.0, 7, 1).any()
    # the mask of a narrower tensor is the same rows' first columns
    assert np.array_equal(LO.keep_mask(T, 17, p, 7, 1), a[:, :17])


def _norm_inputs(T, H, gate, seed=0):
    rng = np.random.default_rng(seed)
    d = {n: rng.standard_normal((T, H)) for n in ("y", "res", "dr", "dn")}
    d["w_post"], d["w_pre"] = rng.normal(1, 0.1, H), rng.normal(1, 0.1, H)
    shape = {"none": None, "token": (T, 1), "channel": (H,), "element": (T, H)}[gate]
    d["gate"] = None if shape is None else rng.normal(0.5, 0.3, shape)
    return d


def _norm_torch(t, scale, w_offset, p, keep, eps):
    def norm(x, w):
        return x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * (w_offset + w)
    b = norm(t["y"], t["w_post"])
    if p:
        b = torch.where(keep, b / (1 - p), torch.zeros_like(b))
    r = t["res"] + scale * b * (1.0 if t["gate"] is None else t["gate"])
    return r, norm(r, t["w_pre"])


@pytest.mark.parametrize("gate", ["none", "token", "channel", "element"])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_residual_norm_oracle_against_autograd_and_differences(gate, p):
    T, H, scale, w_offset, eps = 3, 7, 0.6, 0.5, 1e-3
    d = _norm_inputs(T, H, gate)
    keep = LO.keep_mask(T, H, p, 11, 5)
    args = dict(w_post=d["w_post"], gate=d["gate"], scale=scale, w_pre=d["w_pre"],
                w_offset=w_offset, p=p, keep=keep)
    f = LO.residual_norm_forward(d["y"], d["res"], eps=eps, **args)
    b = LO.residual_norm_backward(d["dr"], d["dn"], d["y"], f["r"], f, **args)
    t = {k: None if v is None else torch.tensor(v, requires_grad=True) for k, v in d.items()}
    r, n = _norm_torch(t, scale, w_offset, p, torch.tensor(keep), eps)
    np.testing.assert_allclose(f["r"], r.detach(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(f["n"], n.detach(), rtol=1e-12, atol=1e-12)
    ((r * t["dr"]).sum() + (n * t["dn"]).sum()).backward()
    grads = {"dres": "res", "dy": "y", "dw_post": "w_post", "dw_pre": "w_pre"}
    if gate != "none":
        grads["dgate"] = "gate"
    for g, name in grads.items():
        np.testing.assert_allclose(b[g], t[name].grad, rtol=1e-10, atol=1e-11, err_msg=g)

    def loss(**new):
        a = dict(d, **new)
        o = LO.residual_norm_forward(a["y"], a["res"], a["w_post"], a["gate"], scale,
                                     a["w_pre"], w_offset, eps, p, keep)
        return (o["r"] * d["dr"]).sum() + (o["n"] * d["dn"]).sum()

    h = 1e-5
    for g, name in grads.items():
        for i in np.ndindex(d[name].shape):
            up, down = d[name].copy(), d[name].copy()
            up[i] += h
            down[i] -= h
            fd = (loss(**{name: up}) - loss(**{name: down})) / (2 * h)
            assert abs(fd - b[g][i]) < 1e-7 * max(1, abs(fd)), (g, i)


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_ffn_oracle_against_autograd_and_differences(name):
    T, H, I = 3, 5, 4
    rng = np.random.default_rng(3)
    d = {"X": rng.standard_normal((T, H)), "W1": rng.standard_normal((2 * I, H)),
         "W2": rng.standard_normal((H, I)), "add": rng.standard_normal((T, H))}
    dY = rng.standard_normal((T, H))
    f = LO.ffn_forward(d["X"], d["W1"], d["W2"], name, d["add"])
    b = LO.ffn_backward(dY, d["X"], d["W1"], d["W2"], f, name)
    t = {k: torch.tensor(v, requires_grad=True) for k, v in d.items()}
    g, u = (t["X"] @ t["W1"].T).chunk(2, 1)
    a = torch.nn.functional.silu(g) if name == "silu" else \
        torch.nn.functional.gelu(g, approximate="tanh")
    Y = t["add"] + (a * u) @ t["W2"].T
    np.testing.assert_allclose(f["Y"], Y.detach(), rtol=1e-12, atol=1e-12)
    Y.backward(torch.tensor(dY))
    for gname, n in (("dX", "X"), ("dW1", "W1"), ("dW2", "W2")):
        np.testing.assert_allclose(b[gname], t[n].grad, rtol=1e-10, atol=1e-11, err_msg=gname)

    def loss(**new):
        a = dict(d, **new)
        return (LO.ffn_forward(a["X"], a["W1"], a["W2"], name, a["add"])["Y"] * dY).sum()

    h = 1e-5
    for gname, n in (("dX", "X"), ("dW1", "W1"), ("dW2", "W2")):
        for i in np.ndindex(d[n].shape):
            up, down = d[n].copy(), d[n].copy()
            up[i] += h
            down[i] -= h
            fd = (loss(**{n: up}) - loss(**{n: down})) / (2 * h)
            assert abs(fd - b[gname][i]) < 1e-6 * max(1, abs(fd)), (gname, i)
    # the gradient of ``add`` is dY itself
    np.testing.assert_allclose(t["add"].grad, dY)


# ------------------------------------------------------- argument checks
class _Buffers:
    """Real memory for every pointer (see test_abi.py): a lost check would
    launch on valid buffers, not on made-up addresses."""

    def __init__(self):
        self.cuda, self.keep = torch.cuda.is_available(), []

    def __call__(self, nbytes):
        n = max(16, int(nbytes)) + 16
        if self.cuda:
            t = torch.zeros(n, dtype=torch.uint8, device="cuda")
            self.keep.append(t)
            return t.data_ptr()
        b = ctypes.create_string_buffer(n)
        self.keep.append(b)
        return (ctypes.addressof(b) + 15) & ~15


INVALID, UNSUPPORTED = 1, 2


def test_residual_norm_fwd_refusals(L):
    B = _Buffers()
    T, H = 4, 32
    ok = dict(y=B(T * H * 4), res=B(T * H * 4), w_post=B(H * 4), gate=None, kind=0, scale=1.0,
              w_pre=B(H * 4), w_offset=0.0, eps=1e-6, p=0.0, rng=None, T=T, H=H, dtype=2,
              r=B(T * H * 4), n=B(T * H * 4), stats=B(T * 8), stream=None)

    def call(**kw):
        return L.moe_residual_norm_fwd(*dict(ok, **kw).values())

    assert call(dtype=3) == UNSUPPORTED and call(dtype=-1) == UNSUPPORTED
    assert call(T=-1) == UNSUPPORTED and call(T=(1 << 30) + 1) == UNSUPPORTED
    assert call(H=0) == UNSUPPORTED and call(H=16385) == UNSUPPORTED
    assert call(kind=4) == UNSUPPORTED and call(kind=-1) == UNSUPPORTED
    assert call(kind=1) == INVALID and call(gate=ok["y"]) == INVALID
    assert call(p=0.5) == INVALID                       # no rng
    rng = B(16)
    assert call(p=-0.1, rng=rng) == INVALID and call(p=1.5, rng=rng) == INVALID
    assert call(p=float("nan"), rng=rng) == INVALID
    assert call(y=None) == INVALID and call(stats=None) == INVALID
    assert call(n=None) == INVALID and call(w_pre=None) == INVALID
    assert call(r=None, n=None, w_pre=None) == INVALID
    assert call(T=0) == 0


def test_residual_norm_bwd_refusals(L):
    B = _Buffers()
    T, H = 4, 32
    nb = L.moe_residual_norm_bwd_workspace_bytes(T, H, 2)
    assert nb >= 3 * H * 4
    t = B(T * H * 4)
    ok = dict(dr=t, dn=B(T * H * 4), y=B(T * H * 4), r=B(T * H * 4), stats=B(T * 8),
              w_post=B(H * 4), gate=None, kind=0, scale=1.0, w_pre=B(H * 4), w_offset=0.0, p=0.0,
              rng=None, T=T, H=H, dtype=2, dres=B(T * H * 4), dy=B(T * H * 4), dgate=None,
              dw_post=B(H * 4), dw_pre=B(H * 4), ws=B(nb), nb=nb, stream=None)

    def call(**kw):
        return L.moe_residual_norm_bwd(*dict(ok, **kw).values())

    assert call(dtype=3) == UNSUPPORTED and call(H=16385) == UNSUPPORTED
    assert call(T=-1) == UNSUPPORTED and call(kind=4) == UNSUPPORTED
    assert call(dw_post=None) == INVALID and call(dw_pre=None) == INVALID
    assert call(w_post=None) == INVALID and call(dn=None) == INVALID
    assert call(gate=t, kind=3) == INVALID              # no dgate
    assert call(dgate=t) == INVALID                     # no gate
    assert call(dy=None) == INVALID and call(r=None) == INVALID and call(y=None) == INVALID
    assert call(stats=None) == INVALID and call(p=0.5) == INVALID
    assert call(ws=None) == INVALID and call(nb=nb - 1) == INVALID
    assert call(dr=None, dn=None, w_pre=None, dw_pre=None) == INVALID


def test_dropout_refusals(L):
    B = _Buffers()
    x, o, rng = B(4 * 32 * 2), B(4 * 32 * 2), B(16)
    f = L.moe_dropout
    assert f(x, 4, 32, 3, 0.5, rng, o, None) == UNSUPPORTED
    assert f(x, -1, 32, 0, 0.5, rng, o, None) == UNSUPPORTED
    assert f(x, 4, 0, 0, 0.5, rng, o, None) == UNSUPPORTED
    assert f(x, 4, 32, 0, 1.01, rng, o, None) == INVALID
    assert f(x, 4, 32, 0, float("nan"), rng, o, None) == INVALID
    assert f(x, 4, 32, 0, 0.5, None, o, None) == INVALID
    assert f(None, 4, 32, 0, 0.5, rng, o, None) == INVALID
    assert f(x, 4, 32, 0, 0.5, rng, None, None) == INVALID
    assert f(None, 0, 32, 0, 0.5, rng, None, None) == 0


def test_ffn_refusals(L):
    B = _Buffers()
    T, H, I = 8, 64, 64
    sb, wb = L.moe_ffn_saved_bytes(T, H, I), L.moe_ffn_workspace_bytes(T, H, I)
    assert sb >= T * 2 * I * 4 + T * I * 2 and wb >= T * 2 * I * 2
    ok = dict(X=B(T * H * 2), W1=B(2 * I * H * 2), W2=B(H * I * 2), T=T, H=H, I=I, dtype=0,
              act=0, add=None, Y=B(T * H * 2), saved=B(sb), sb=sb, ws=None, wb=0, stream=None)

    def fwd(**kw):
        return L.moe_ffn_fwd(*dict(ok, **kw).values())

    for bad in (dict(H=48), dict(H=72), dict(I=48), dict(I=72), dict(dtype=2), dict(act=2),
                dict(T=-1), dict(T=(1 << 30) + 1)):
        assert fwd(**bad) == UNSUPPORTED, bad
    for bad in (dict(X=None), dict(W1=None), dict(W2=None), dict(Y=None), dict(sb=sb - 1),
                dict(saved=None, sb=0), dict(saved=None, sb=0, ws=ok["saved"], wb=wb - 1),
                dict(X=ok["X"] + 2), dict(add=ok["X"] + 8)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(T=0, X=None) == 0
    ok = dict(dY=B(T * H * 2), X=B(T * H * 2), W1=B(2 * I * H * 2), W2=B(H * I * 2), T=T, H=H,
              I=I, dtype=0, act=0, saved=B(sb), sb=sb, add=None, dX=B(T * H * 2),
              dW1=B(2 * I * H * 2), dW2=B(H * I * 2), ws=B(wb), wb=wb, stream=None)

    def bwd(**kw):
        return L.moe_ffn_bwd(*dict(ok, **kw).values())

    for bad in (dict(H=72), dict(dtype=2), dict(act=-1)):
        assert bwd(**bad) == UNSUPPORTED, bad
    for bad in (dict(dW1=None), dict(dW2=None), dict(dX=None), dict(saved=None), dict(sb=sb - 1),
                dict(ws=None), dict(wb=wb - 1), dict(dY=None), dict(dY=ok["dY"] + 4)):
        assert bwd(**bad) == INVALID, bad


def test_binding_refuses_host_tensors():
    """No tensor of the host reaches the library."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    rng = torch.zeros(2, dtype=torch.int64)
    w1, w2 = torch.zeros(128, 64, dtype=torch.bfloat16), torch.zeros(64, 64, dtype=torch.bfloat16)
    for call in (lambda: ops.dropout_fwd(x, 0.5, rng),
                 lambda: ops.residual_norm_fwd(x, w_pre=x[0]),
                 lambda: ops.residual_norm_bwd(x, None, x, x, torch.zeros(2, 4)),
                 lambda: ops.ffn_fwd(x, w1, w2),
                 lambda: ops.ffn_bwd(x, x, w1, w2, None)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ------------------------------------------------------------- the layer
def _layer(**kw):
    """A layer without memory behind its buffers: for checks that come before
    any call of the library."""
    T, H = 8, 64
    layer = ops.MoeLayer(T, H, 64, 4, 2, 16, 1.0, device="meta", **kw)
    t = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="meta")  # noqa: E731
    return layer, t(T, H), (t(H), t(H))


@pytest.mark.parametrize("I_shared", [0, 64])
def test_layer_refuses_a_missing_or_unknown_shared_expert(L, I_shared):
    """In both directions: a backward without the shared expert's weights
    would leave its part out of dX and the last step's dW1s, dW2s in place."""
    layer, X, norms = _layer(I_shared=I_shared)
    shared = None if I_shared else (X, X)
    with pytest.raises(ValueError, match="shared"):
        layer.forward(X, None, None, norms, shared)
    with pytest.raises(ValueError, match="shared"):
        layer.backward(X, X, None, norms, shared)
    with pytest.raises(ValueError, match="shared"):
        layer.step(X, None, X, None, norms, shared)


def test_layer_refuses_dropout_without_its_state(L):
    """Before anything of the step runs, for either dropout."""
    for kw in (dict(p=0.1), dict(p_in=0.1)):
        layer, X, norms = _layer(**kw)
        with pytest.raises(ValueError, match="rng"):
            layer.forward(X, None, None, norms)
        with pytest.raises(ValueError, match="rng"):
            layer.backward(X, X, None, norms)
    for kw in (dict(p=1.5), dict(p_in=-0.1), dict(p=float("nan")), dict(act="relu")):
        with pytest.raises(ValueError, match="p_in and p|act"):
            _layer(**kw)


def test_layer_and_block_run_on_their_own_device(L, monkeypatch):
    """Made on device 1 with device 0 the current one, every call of a step is
    made with device 1 current, the routed block's too (they take the current
    device's stream), and device 0 is back afterwards."""
    current, seen = [0], []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, current[0] = current[0], self.dev

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(ops, "_current_device", lambda: current[0])
    calls = ("residual_norm_fwd", "residual_norm_bwd", "dropout_fwd", "dropout_bwd", "ffn_fwd",
             "ffn_bwd", "route_topk", "permute", "unpermute", "lora_mlp_fwd", "lora_mlp_bwd")
    for name in calls:
        monkeypatch.setattr(ops, name, lambda *a, name=name, **k: seen.append((name, current[0])))
    layer, X, norms = _layer(I_shared=64, p=0.1, p_in=0.1)
    layer.dev = layer.block.dev = 1
    W = [None] * 6
    rng = torch.zeros(2, 2, dtype=torch.int64)
    layer.step(X, None, X, W, norms, (X, X), rng=rng)
    assert {n for n, _ in seen} == set(calls) and {d for _, d in seen} == {1}
    layer.forward(X, None, W, norms, (X, X), rng=rng)
    layer.backward(X, X, W, norms, (X, X), rng=rng)
    layer.block.step(X, None, X, W)
    layer.block.forward(X, None, W)
    layer.block.backward(X, W)
    assert {d for _, d in seen} == {1} and current == [0]


@pytest.mark.parametrize("T,H", [((1 << 32) + 8, 1), (8, (1 << 32) + 8), ((1 << 30) + 1, 1),
                                 (1, (1 << 30) + 1)])
def test_sizes_past_32_bits_are_refused(L, monkeypatch, T, H):
    """Rows and columns past 2^30 never reach the library, whose C ints would
    take them modulo 2^32 (2^32 + 8 rows as 8, the others left unwritten)."""
    class Rows:
        dtype, device = torch.bfloat16, torch.device("cuda", 0)

        def __init__(self, *shape):
            self.shape = torch.Size(shape)

        dim = lambda self: len(self.shape)              # noqa: E731
        get_device = lambda self: 0                     # noqa: E731
        is_contiguous = lambda self: True               # noqa: E731
        data_ptr = lambda self: 256                     # noqa: E731

    calls = []
    monkeypatch.setattr(ops, "_run", lambda *a: calls.append(a))
    x, rng = Rows(T, H), Rows(2)
    rng.dtype = torch.int64
    w1, w2 = Rows(2 * 64, H), Rows(H, 64)
    for call in (lambda: ops.dropout_fwd(x, 0.5, rng, out=x),
                 lambda: ops.residual_norm_fwd(x, w_pre=Rows(H), out=(x, x, None)),
                 lambda: ops.residual_norm_bwd(x, x, x, x, None, w_pre=Rows(H),
                                               out=(x, x, None, None, Rows(H))),
                 lambda: ops.ffn_fwd(x, w1, w2, out=x),
                 lambda: ops.ffn_bwd(x, x, w1, w2, x, out=(x, None, None)),
                 lambda: ops.ffn_fwd(Rows(4, 64), Rows(2 * T, 64), Rows(64, T), out=x)
                 if T > H else ops.dropout_bwd(x, 0.5, rng, out=x)):
        with pytest.raises(ValueError, match="2\\^30"):
            call()
    assert not calls


def test_addresses_inside_an_element_are_refused(L):
    """Addresses that are no multiple of the element's size (statistics and
    workspace: of 4, the dropout's state: of 8) are errors of the call, not of
    the device."""
    B = _Buffers()
    T, H = 4, 32
    t = B(T * H * 4)
    for dtype in (0, 1, 2):
        ok = dict(y=t, res=t, w_post=t, gate=t, kind=3, scale=1.0, w_pre=t, w_offset=0.0,
                  eps=1e-6, p=0.5, rng=B(16), T=T, H=H, dtype=dtype, r=t, n=t, stats=B(T * 8),
                  stream=None)
        for name in ("y", "res", "w_post", "gate", "w_pre", "r", "n", "stats", "rng"):
            bad = dict(ok, **{name: ok[name] + 1})
            assert L.moe_residual_norm_fwd(*bad.values()) == INVALID, name
        nb = L.moe_residual_norm_bwd_workspace_bytes(T, H, dtype)
        ok = dict(dr=t, dn=t, y=t, r=t, stats=B(T * 8), w_post=t, gate=t, kind=3, scale=1.0,
                  w_pre=t, w_offset=0.0, p=0.5, rng=B(16), T=T, H=H, dtype=dtype, dres=t, dy=t,
                  dgate=t, dw_post=t, dw_pre=t, ws=B(nb + 8), nb=nb, stream=None)
        for name in ("dr", "dn", "y", "r", "stats", "w_post", "gate", "w_pre", "rng", "dres",
                     "dy", "dgate", "dw_post", "dw_pre", "ws"):
            bad = dict(ok, **{name: ok[name] + 1})
            assert L.moe_residual_norm_bwd(*bad.values()) == INVALID, name
        assert L.moe_residual_norm_bwd(*dict(ok, ws=ok["ws"] + 2).values()) == INVALID
        rng = B(16)
        for p in (0.0, 0.5):
            assert L.moe_dropout(t + 1, T, H, dtype, p, rng, t, None) == INVALID
            assert L.moe_dropout(t, T, H, dtype, p, rng, t + 1, None) == INVALID
            assert L.moe_dropout(t, T, H, dtype, p, rng + 4, t, None) == INVALID


def test_inputs_larger_than_the_layer_are_refused(L, monkeypatch):
    """Logits of more tokens or experts, and adapters of a larger rank, than
    the layer's buffers hold: errors, not writes past their ends."""
    monkeypatch.setattr(ops, "_need", lambda *a: None)     # buffers without memory
    layer, X, norms = _layer(I_shared=64)                  # 8 tokens, 4 experts, 2 each, rank 16
    blk, R, H, I = layer.block, 16, 64, 64

    def t(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="meta")

    def weights(E, r):
        return (t(E, 2 * I, H), t(E, r, H), t(E, 2 * I, r), t(E, H, I), t(E, r, I), t(E, H, r))

    def refused(call, match):
        with pytest.raises(ValueError, match=match):
            call()

    W = weights(4, 16)
    for logits in (t(9, 4, dtype=torch.float32), t(8, 5, dtype=torch.float32)):
        refused(lambda: blk.forward(X, logits, W), "topk_idx|expert_counts")
    refused(lambda: ops.permute(t(9, H), t(9, 2), out=blk.Xp), "Xp")
    refused(lambda: ops.permute(X, blk.dest, Zp=t(R, H), dw=t(7, 2)), "dw")
    refused(lambda: ops.unpermute(blk.Z2, blk.dest, out=t(7, H)), "Y")
    refused(lambda: ops.lora_mlp_fwd(t(R + 1, H), blk.offsets, *W, 1.0, out=blk.Z2), "Z2")
    refused(lambda: ops.lora_mlp_bwd(blk.dZ2, blk.Xp, blk.offsets, *weights(4, 32), 1.0, blk.saved,
                                     out=(blk.dXp, blk.dA1, blk.dB1, blk.dA2, blk.dB2)), "dA1")
    refused(lambda: ops.router_bwd(blk.w, blk.w, blk.idx, blk.dest, blk.offsets, blk.Xp, t(4, H),
                                   blk.dXp, out=(blk.dX, t(3, H))), "dWr")
    refused(lambda: ops.ep_regroup(t(R, H), t(2, 4), 0, out=t(R - 1, H)), "out")
