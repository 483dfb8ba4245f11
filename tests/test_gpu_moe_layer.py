"""The whole expert half of a decoder layer (norm, dropout, routed experts,
shared expert, post norm, gate, residual) as one step: each part of the run
against the fp64 oracle on that part's own inputs, forward and backward, the
step eager and as a replayed graph, and a change of the dropout's state
between replays."""

import numpy as np
import pytest
import torch

import oracle as O
from moe_expert_grouped_softmax_b200 import ops
from moe_expert_grouped_softmax_b200 import synthetic as S
from oracle import layer_oracle as LO

from _common import assert_bf16_close, f32

pytestmark = pytest.mark.gpu

U = 2.0 ** -8  # half a step of bf16
NAMES = ("W1", "A1", "B1", "W2", "A2", "B2")


def l2(got, ref, steps, name):
    """2-norm error of at most `steps` roundings to bf16 (sums in fp32 add
    less than 1e-4 at these lengths)."""
    g = got.double().cpu().numpy()
    err = np.linalg.norm(g - ref) / np.linalg.norm(ref)
    assert err <= steps * U + 1e-4, f"{name}: {err}"


def make(T=None, p_in=0.1, p=0.2, gate="channel", seed=3, **block):
    cfg = S.make_config("tiny")
    if T:
        cfg["T"] = T
    inp = S.make_inputs(cfg)
    H, Is = cfg["H"], 144
    gen = torch.Generator().manual_seed(seed)

    def t(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen) * std + mean).to(torch.bfloat16).cuda()

    shape = {None: None, "channel": (H,), "token": (cfg["T"], 1)}[gate]
    a = dict(X=inp["X"].cuda(), logits=inp["logits"].cuda(), dOut=inp["dY"].cuda(),
             W=[inp[n].cuda() for n in NAMES], norms=(t(H, std=0.1, mean=1.0), t(H, std=0.1, mean=1.0)),
             shared=(t(2 * Is, H, std=0.05), t(H, Is, std=0.05)),
             gate=None if shape is None else t(*shape, std=0.3, mean=0.5),
             rng=torch.tensor([[11, 5], [12, 6]], device="cuda"))
    layer = ops.MoeLayer(*(cfg[x] for x in ("T", "H", "I", "E", "k", "r", "s")), I_shared=Is,
                         scale=0.5, p_in=p_in, p=p, gate_shape=shape, **block)
    return cfg, layer, a


def check(cfg, layer, a):
    n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    T, H = cfg["T"], cfg["H"]
    masks = [LO.keep_mask(T, H, p, *map(int, r)) for p, r in
             zip((layer.p_in, layer.p), a["rng"].tolist())]
    X, w_pre, w_post = n64(a["X"]), n64(a["norms"][0]), n64(a["norms"][1])
    gate = None if a["gate"] is None else n64(a["gate"])
    pre = LO.residual_norm_forward(X, w_pre=w_pre)
    # n's gradient form takes r itself: x / rms, not its rounding
    f = LO.residual_norm_forward(X, None, None, None, 1.0, w_pre)
    l2(layer.n, f["n"], 1, "n")
    nd = n64(layer.nd)
    if layer.p_in:
        l2(layer.nd, LO.dropout(n64(layer.n), layer.p_in, masks[0]), 1, "dropout(n)")
    W = [f32(w) for w in a["W"]]
    Y, ctx = O.block_forward(nd, a["logits"].cpu().numpy(), cfg["k"], *W, cfg["s"])
    assert_bf16_close(layer.block.Y, Y, "block.Y")
    w1, w2 = (n64(w) for w in a["shared"])
    ffn = LO.ffn_forward(nd, w1, w2, "silu", n64(layer.block.Y))
    l2(layer.y, ffn["Y"], 2, "y")
    args = dict(w_post=w_post, gate=gate, scale=layer.scale, p=layer.p, keep=masks[1])
    post = LO.residual_norm_forward(n64(layer.y), X, **args)
    l2(layer.out, post["r"], 1, "out")
    # backward
    b = LO.residual_norm_backward(n64(a["dOut"]), None, n64(layer.y), None, post, **args)
    l2(layer.dy, b["dy"], 1, "dy")
    l2(layer.dw_post, b["dw_post"], 1, "dw_post")
    if gate is not None:
        l2(layer.dgate, b["dgate"].reshape(gate.shape), 1, "dgate")
    dy = n64(layer.dy)
    g = O.block_backward(dy, ctx, base=layer.block.full_ft)
    assert_bf16_close(layer.block.dX, g["dX"], "block.dX")
    assert_bf16_close(layer.block.dA1, g["dA1"], "dA1")
    fb = LO.ffn_backward(dy, nd, w1, w2, ffn, "silu", n64(layer.block.dX))
    dn = fb["dX"]
    if layer.p_in:
        dn = LO.dropout(dn, layer.p_in, masks[0])
    l2(layer.dn, dn, 3, "dn")
    if layer.dW1s is not None:
        l2(layer.dW1s, fb["dW1"], 2, "dW1s")
        l2(layer.dW2s, fb["dW2"], 2, "dW2s")
    pb = LO.residual_norm_backward(n64(a["dOut"]), n64(layer.dn), X, X, pre, w_pre=w_pre)
    l2(layer.dX, pb["dres"], 1, "dX")
    l2(layer.dw_pre, pb["dw_pre"], 1, "dw_pre")
    torch.cuda.synchronize()
    assert ops.device_status() == 0


@pytest.mark.parametrize("case", [
    dict(), dict(gate="token", p_in=0.0, full_ft=True), dict(T=1, gate=None, p=0.0),
    dict(T=77, gate="token"),
], ids=["all", "full-ft", "one-token", "ragged"])
def test_layer_step_against_oracle(cuda_ok, case):
    cfg, layer, a = make(**case)
    layer.step(**a)
    check(cfg, layer, a)


def test_layer_graph_replay(cuda_ok):
    """A captured step gives the eager bytes; with another offset written in
    place a replay drops other elements and is right for those."""
    cfg, eager, a = make()
    eager.step(**a)
    _, graphed, _ = make()
    graphed.capture(**a)
    outs = ("out", "dX", "dw_pre", "dw_post", "dgate", "y", "n")
    for n in outs:
        getattr(graphed, n).zero_()
    graphed.replay()
    for n in outs:
        assert torch.equal(getattr(graphed, n), getattr(eager, n)), n
    a["rng"][:, 1] += 1
    graphed.replay()
    assert not torch.equal(graphed.nd, eager.nd)
    check(cfg, graphed, a)


def test_two_layers_on_two_streams(cuda_ok):
    """Two layers with buffers of their own, stepped at once on two streams,
    give what each gives alone."""
    made = [make(seed=s) for s in (3, 4)]
    want = []
    for _, layer, a in made:
        layer.step(**a)
        want.append([getattr(layer, n).clone() for n in ("out", "dX", "dw_post")])
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(5):
        for (_, layer, a), st in zip(made, streams):
            with torch.cuda.stream(st):
                layer.step(**a)
    torch.cuda.synchronize()
    for (_, layer, _), w in zip(made, want):
        for n, x in zip(("out", "dX", "dw_post"), w):
            assert torch.equal(getattr(layer, n), x), n
    assert ops.device_status() == 0


def test_layer_refusals(cuda_ok):
    cfg, layer, a = make()
    with pytest.raises(ValueError, match="shared"):
        layer.forward(a["X"], a["logits"], a["W"], a["norms"], None, a["gate"], a["rng"])
    with pytest.raises(ValueError, match="gate"):
        layer.forward(a["X"], a["logits"], a["W"], a["norms"], a["shared"], None, a["rng"])
    with pytest.raises(ValueError, match="w_post"):
        layer.forward(a["X"], a["logits"], a["W"], (a["norms"][0], None), a["shared"], a["gate"],
                      a["rng"])
