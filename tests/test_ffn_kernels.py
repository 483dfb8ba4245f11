"""Every kernel that a product of the dense gated feed-forward block can run
on: cases that take each of them (the choice is host logic, asserted here on
the CPU), and their results on the GPU, with and without ``add``."""

import pytest
import torch

from moe_expert_grouped_softmax_b200 import build, ops

# T, H, I, type, activation, weight gradients, then the kernels of gate_up,
# down, dh, dX (, dW1, dW2): T = token kernel, P = CTA pairs, M = the three in
# one launch, n/s = 128 x n tiles over clusters of s
CASES = [
    (23, 320, 144, "bf16", "silu", True, "T T 64/1 M M M"),
    (39, 64, 64, "fp16", "silu", True, "64/1 64/1 64/1 M M M"),
    (35, 1360, 64, "bf16", "gelu_tanh", False, "64/4 64/1 64/4 64/1"),
    (41, 880, 2464, "bf16", "silu", True, "64/1 64/4 64/2 64/4 128/1 128/1"),
    (404, 64, 3616, "fp16", "silu", True, "128/1 64/4 128/1 64/4 64/1 64/1"),
    (37, 2384, 1344, "fp16", "gelu_tanh", False, "128/4 128/4 64/4 128/4"),
    (34, 816, 4608, "bf16", "silu", True, "64/1 64/4 64/1 64/4 P P"),
    (2366, 1552, 80, "bf16", "silu", False, "64/2 P 128/4 P"),
    (8736, 160, 304, "fp16", "silu", True, "P 128/1 P 128/1 64/4 64/4"),
    (38, 2304, 4944, "bf16", "gelu_tanh", True, "64/1 64/4 128/2 M M M"),
    (37, 5456, 2512, "bf16", "silu", False, "128/2 128/2 128/4 128/2"),
    (2302, 96, 3488, "fp16", "silu", True, "P 64/4 P 64/4 128/2 128/4"),
    (2454, 64, 5104, "bf16", "silu", True, "P 64/4 P 64/4 64/1 128/2"),
    (8082, 144, 848, "bf16", "gelu_tanh", True, "P 128/1 P 128/1 128/4 64/4"),
    (8994, 64, 4720, "fp16", "silu", True, "P 64/2 P 64/2 64/2 128/4"),
    (6001, 2064, 1040, "bf16", "silu", False, "P P P P"),
    # the widths of a layer without routing
    (1, 4096, 14336, "bf16", "silu", False, "T T 128/1 128/4"),
    (65, 4096, 14336, "bf16", "silu", True, "128/1 128/4 128/1 M M M"),
    (2100, 2048, 28672, "bf16", "silu", True, "P P P P P P"),
]
IDS = ["-".join(map(str, c[:4])) for c in CASES]


def names(kernels):
    short = {"tokens": "T", "pairs": "P", "pairs merged": "M"}
    return [short[k] if k in short else f"{k[0]}/{k[1]}" for k in kernels.values()]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_cases_take_the_kernels_they_are_for(case):
    build.build()
    T, H, I, _, _, need_dw, want = case
    assert names(ops.ffn_kernels(T, H, I, need_dw)) == want.split()


def test_cases_take_every_kernel():
    """Both directions of every product: all that the choice can return (dW1
    and dW2 are one kernel, on either operand's shape)."""
    split = {f"{n}/{s}" for n in (64, 128) for s in (1, 2, 4)}
    seen = [set() for _ in range(6)]
    for case in CASES:
        for i, k in enumerate(case[6].split()):
            seen[i].add(k)
    gate_up, down, dh, dX, dW1, dW2 = seen
    assert gate_up == split | {"T", "P"} and dh == split | {"P"}
    assert down == split | {"T", "P"} and dX == split | {"P", "M"}
    assert dW1 == split | {"P", "M"} and dW2 <= dW1


def test_kernel_query_refusals():
    L = ops.lib()
    f = L.moe_ffn_kernel
    assert f(0, 64, 64, 0, 1) == f(-1, 64, 64, 0, 1) == f(40, 72, 64, 0, 1) == -1
    assert f(40, 64, 64, 6, 1) == f(40, 64, 64, -1, 1) == f(40, 64, 64, 4, 0) == -1
    with pytest.raises(ValueError):
        ops.ffn_kernels(40, 64, 72)


def G(n):
    """Steps of an fp32 sum of n terms and 64 more operations, twice (the
    tensor cores may cut rather than round)."""
    return 2 * (n + 64) * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_every_kernel_against_fp64(cuda_ok, case):
    """In the 2-norm a result's own rounding costs at most u of itself; that of
    the values it is summed from (h or dZ) at most u, and the fp32 sums G of
    their length, of the product.  Every 64th row is held to twice that."""
    T, H, I, dtype, act, need_dw, _ = case
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    u = torch.finfo(dt).eps / 2
    gen = torch.Generator(device="cuda").manual_seed(T + H + I)

    def draw(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dt)

    X, dY, W1, W2 = draw(T, H), draw(T, H), draw(2 * I, H, std=H ** -0.5), draw(H, I, std=I ** -0.5)
    adds = (None, None), (draw(T, H), draw(T, H))
    x, dy, w1, w2 = X.double(), dY.double(), W1.double(), W2.double()
    g, up = (x @ w1.T).chunk(2, 1)
    g = g.clone().requires_grad_()
    a = torch.nn.functional.silu(g) if act == "silu" else \
        torch.nn.functional.gelu(g, approximate="tanh")
    dg, = torch.autograd.grad(a, g, (dy @ w2) * up)
    a = a.detach()
    dZ = torch.cat((dg, (dy @ w2) * a), 1)
    prod = {"Y": ((a * up) @ w2.T, H + I), "dX": (dZ @ w1, H + 2 * I),
            "dW1": (dZ.T @ x, H + T), "dW2": (dy.T @ (a * up), H + T)}

    def close(got, name, add=None):
        p, n = prod[name]
        ref = p if add is None else p + add.double()
        err = got.double() - ref
        for e, r, q, factor in ((err.norm(), ref.norm(), p.norm(), 1),
                                (err[::64].norm(dim=1), ref[::64].norm(dim=1), p[::64].norm(dim=1), 2)):
            bound = factor * (u * r + (u + G(n)) * (1 + u) * q)
            assert (e <= bound).all(), (name, float((e / bound).max()))

    for add_f, add_b in adds:
        Y, saved = ops.ffn_fwd(X, W1, W2, act=act, add=add_f)
        close(Y, "Y", add_f)
        assert torch.equal(ops.ffn_fwd(X, W1, W2, act=act, add=add_f, save=False)[0], Y)
        grads = ops.ffn_bwd(dY, X, W1, W2, saved, act=act, add=add_b, need_dw=need_dw)
        close(grads[0], "dX", add_b)
        if need_dw:
            close(grads[1], "dW1")
            close(grads[2], "dW2")
        for _ in range(3):  # the same bytes every time
            again = ops.ffn_bwd(dY, X, W1, W2, saved, act=act, add=add_b, need_dw=need_dw)
            assert all(p is q or torch.equal(p, q) for p, q in zip(again, grads))
    torch.cuda.synchronize()
    assert ops.device_status() == 0
