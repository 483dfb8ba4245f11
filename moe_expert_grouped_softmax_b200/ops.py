"""Python binding of libmoe_lora.so (ctypes).

Argument marshalling only: every step of the block runs in the library's
CUDA kernels.  Tensors are passed by ``data_ptr()`` with the current CUDA
stream.  If the library is missing, every call raises; there is no fallback.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_lora.so")
_lib = None

MOE_OK = 0
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported shape",
                3: "CUDA error", 4: "device wait timed out",
                5: "device index out of range"}

EXPORTS = [
    "moe_route_workspace_bytes", "moe_route_topk", "moe_permute", "moe_unpermute",
    "moe_saved_bytes", "moe_saved_part_offset", "moe_workspace_bytes",
    "moe_lora_mlp_fwd", "moe_lora_mlp_bwd", "moe_lora_mlp_bwd_full", "moe_get_device_status",
    "moe_status_string", "moe_set_wait_limit_ns", "moe_test_inject_stall",
    "moe_set_cta_pairs", "moe_uses_cta_pairs", "moe_kernel_launches", "moe_profile_enable",
    "moe_router_fwd", "moe_router_bwd_workspace_bytes", "moe_router_bwd",
    "moe_profile_collect", "moe_ep_regroup",
    "moe_residual_norm_fwd", "moe_residual_norm_bwd_workspace_bytes", "moe_residual_norm_bwd",
    "moe_dropout", "moe_ffn_kernel", "moe_ffn_saved_bytes", "moe_ffn_workspace_bytes", "moe_ffn_fwd",
    "moe_ffn_bwd",
]

PROF_KINDS = {"route": 0, "permute": 1, "gate_up_fwd": 2, "down_fwd": 3,
              "unpermute": 4, "down_bwd": 5, "gate_up_bwd": 6, "lora_grad": 7,
              "transpose": 8, "base_grad": 9, "router_fwd": 10, "router_bwd": 11,
              "rank_down": 12, "ffn_gate_up": 13, "ffn_down": 14, "ffn_dh": 15, "ffn_dx": 16,
              "ffn_dw": 17, "norm_fwd": 18, "norm_bwd": 19, "dropout": 20}


class MoeError(RuntimeError):
    def __init__(self, code, where):
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} ({code})")
        self.code = code


def lib():
    """The loaded library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build it with "
                "`python -m moe_expert_grouped_softmax_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        P, I, S, F, U64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t,
                           ctypes.c_float, ctypes.c_uint64)
        L.moe_route_workspace_bytes.argtypes = [I, I, I]
        L.moe_route_workspace_bytes.restype = S
        L.moe_route_topk.argtypes = [P, I, I, I, P, P, P, P, P, P, S, P]
        L.moe_route_topk.restype = I
        L.moe_permute.argtypes = [P, P, P, I, I, I, P, P, P, P]
        L.moe_permute.restype = I
        L.moe_unpermute.argtypes = [P, P, P, I, I, I, P, P]
        L.moe_unpermute.restype = I
        L.moe_router_fwd.argtypes = [P, P, I, I, I, P, P]
        L.moe_router_fwd.restype = I
        L.moe_router_bwd_workspace_bytes.argtypes = [I, I]
        L.moe_router_bwd_workspace_bytes.restype = S
        L.moe_router_bwd.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, P, P, P, S, P]
        L.moe_router_bwd.restype = I
        L.moe_saved_bytes.argtypes = [I, I, I, I]
        L.moe_saved_bytes.restype = S
        L.moe_saved_part_offset.argtypes = [I, I, I, I, I]
        L.moe_saved_part_offset.restype = S
        L.moe_workspace_bytes.argtypes = [I, I, I, I, I]
        L.moe_workspace_bytes.restype = S
        L.moe_lora_mlp_fwd.argtypes = [P, P, I, I, I, I, F, P, P, P, P, P, P, I, P,
                                       P, S, P, S, P]
        L.moe_lora_mlp_fwd.restype = I
        L.moe_lora_mlp_bwd.argtypes = [P, P, P, I, I, I, I, F, P, P, P, P, P, P, P,
                                       S, I, P, P, P, P, P, P, S, P]
        L.moe_lora_mlp_bwd.restype = I
        L.moe_lora_mlp_bwd_full.argtypes = [P, P, P, I, I, I, I, F, P, P, P, P, P, P, P,
                                            S, I, P, P, P, P, P, P, P, P, S, P]
        L.moe_lora_mlp_bwd_full.restype = I
        L.moe_get_device_status.argtypes = [P]
        L.moe_get_device_status.restype = I
        L.moe_status_string.argtypes = [I]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_set_wait_limit_ns.argtypes = [U64]
        L.moe_set_wait_limit_ns.restype = None
        L.moe_set_cta_pairs.argtypes = [I]
        L.moe_set_cta_pairs.restype = None
        L.moe_uses_cta_pairs.argtypes = [I, I, I]
        L.moe_uses_cta_pairs.restype = I
        L.moe_kernel_launches.argtypes = []
        L.moe_kernel_launches.restype = ctypes.c_ulonglong
        L.moe_test_inject_stall.argtypes = [I]
        L.moe_test_inject_stall.restype = None
        L.moe_profile_enable.argtypes = [I]
        L.moe_profile_enable.restype = I
        L.moe_profile_collect.argtypes = [I, ctypes.POINTER(ctypes.c_float), I]
        L.moe_profile_collect.restype = I
        L.moe_ep_regroup.argtypes = [P, P, I, I, I, I, I, P, P, P]
        L.moe_ep_regroup.restype = I
        D = ctypes.c_double
        L.moe_residual_norm_fwd.argtypes = [P, P, P, P, I, F, P, F, F, D, P, I, I, I, P, P, P, P]
        L.moe_residual_norm_fwd.restype = I
        L.moe_residual_norm_bwd_workspace_bytes.argtypes = [I, I, I]
        L.moe_residual_norm_bwd_workspace_bytes.restype = S
        L.moe_residual_norm_bwd.argtypes = [P, P, P, P, P, P, P, I, F, P, F, D, P, I, I, I, P, P,
                                            P, P, P, P, S, P]
        L.moe_residual_norm_bwd.restype = I
        L.moe_dropout.argtypes = [P, I, I, I, D, P, P, P]
        L.moe_dropout.restype = I
        L.moe_ffn_saved_bytes.argtypes = [I, I, I]
        L.moe_ffn_saved_bytes.restype = S
        L.moe_ffn_workspace_bytes.argtypes = [I, I, I]
        L.moe_ffn_workspace_bytes.restype = S
        L.moe_ffn_kernel.argtypes = [I, I, I, I, I]
        L.moe_ffn_kernel.restype = I
        L.moe_ffn_fwd.argtypes = [P, P, P, I, I, I, I, I, P, P, P, S, P, S, P]
        L.moe_ffn_fwd.restype = I
        L.moe_ffn_bwd.argtypes = [P, P, P, P, I, I, I, I, I, P, S, P, P, P, P, P, S, P]
        L.moe_ffn_bwd.restype = I
        _lib = L
    return _lib


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(code, where):
    if code != MOE_OK:
        raise MoeError(code, where)


def _need(t, dtype, shape, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _room(*outs):
    """Each (output, elements that the call writes, name) is large enough."""
    for t, n, name in outs:
        if t.numel() < n:
            raise ValueError(f"{name}: expected at least {n} elements, got {t.numel()}")


def device_status():
    """Synchronise, return and clear the device-side status word."""
    return lib().moe_get_device_status(_stream())


def set_wait_limit_ns(ns):
    lib().moe_set_wait_limit_ns(int(ns))


def kernel_launches():
    """Kernels this library has launched in this process (host-side count)."""
    return int(lib().moe_kernel_launches())


def set_cta_pairs(on=True):
    """Grouped GEMMs on CTA pairs (True, 256-row tiles), single CTAs (False)
    or chosen per GEMM from the rows per expert and K (None, the default)."""
    lib().moe_set_cta_pairs(-1 if on is None else (1 if on else 0))


def uses_cta_pairs(R, E, K):
    """Whether a grouped GEMM over R routed rows, E experts and reduction
    length K runs on CTA pairs under the current setting (the library's own
    choice; host-side, no GPU needed)."""
    return bool(lib().moe_uses_cta_pairs(R, E, K))


def test_inject_stall(on=True):
    lib().moe_test_inject_stall(1 if on else 0)


def profile_enable(on=True):
    _check(lib().moe_profile_enable(1 if on else 0), "moe_profile_enable")


def profile_collect(kind):
    """Durations (ms) of the recorded launches of one kernel kind."""
    buf = (ctypes.c_float * 512)()
    n = lib().moe_profile_collect(PROF_KINDS[kind], buf, 512)
    if n < 0:
        raise MoeError(3, "moe_profile_collect")
    return [buf[i] for i in range(n)]


# ------------------------------------------------------------------ sizes
def route_workspace_bytes(T, E, k):
    return lib().moe_route_workspace_bytes(T, E, k)


def saved_bytes(R, H, I, r):
    return lib().moe_saved_bytes(R, H, I, r)


def saved_part_offset(R, H, I, r, part):
    return lib().moe_saved_part_offset(R, H, I, r, part)


def workspace_bytes(R, E, H, I, r):
    return lib().moe_workspace_bytes(R, E, H, I, r)


def ld_rank(R):
    """Row pitch (elements) of the transposed rank-r saved parts."""
    return (R + 63) // 64 * 64


def saved_views(saved, R, H, I, r):
    """Views of the saved-activation buffer: Z1, h, XA1t, HA2t."""
    b = saved
    o = [saved_part_offset(R, H, I, r, i) for i in range(5)]
    ld = ld_rank(R)

    def view(i, shape):
        n = 1
        for d in shape:
            n *= d
        return b[o[i]:o[i] + 2 * n].view(torch.bfloat16).view(*shape)

    return (view(0, (R, 2 * I)), view(1, (R, I)), view(2, (r, ld)), view(3, (r, ld)))


# ------------------------------------------------------------------ ops
def route_topk(logits, k, out=None, ws=None):
    """a1: returns (topk_idx, topk_w, expert_counts, expert_offsets, dest)."""
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    dev = logits.device
    if out is None:
        out = (torch.empty((T, k), dtype=torch.int32, device=dev),
               torch.empty((T, k), dtype=torch.float32, device=dev),
               torch.empty((E,), dtype=torch.int32, device=dev),
               torch.empty((E + 1,), dtype=torch.int32, device=dev),
               torch.empty((T, k), dtype=torch.int32, device=dev))
    idx, w, counts, offsets, dest = out
    _room((idx, T * k, "topk_idx"), (w, T * k, "topk_w"), (counts, E, "expert_counts"),
          (offsets, E + 1, "expert_offsets"), (dest, T * k, "dest"))
    nbytes = route_workspace_bytes(T, E, k)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(lib().moe_route_topk(_p(logits), T, E, k, _p(idx), _p(w), _p(counts),
                                _p(offsets), _p(dest), _p(ws), ws.numel(), _stream()),
           "moe_route_topk")
    return idx, w, counts, offsets, dest


def permute(X, dest, scale=None, Zp=None, out=None, dw=None):
    """a2 / a6: Xp[dest[t, j]] = scale[t, j] * X[t]; optional dw = <X[t], Zp[dest]>."""
    T, H = X.shape
    k = dest.shape[1]
    _need(X, torch.bfloat16, (T, H), "X")
    _need(dest, torch.int32, (T, k), "dest")
    if scale is not None:
        _need(scale, torch.float32, (T, k), "scale")
    if out is None:
        out = torch.empty((T * k, H), dtype=torch.bfloat16, device=X.device)
    if Zp is not None:
        _need(Zp, torch.bfloat16, (T * k, H), "Zp")
        if dw is None:
            dw = torch.empty((T, k), dtype=torch.float32, device=X.device)
        _room((dw, T * k, "dw"))
    _room((out, T * k * H, "Xp"))
    _check(lib().moe_permute(_p(X), _p(dest), _p(scale), T, H, k, _p(out), _p(Zp),
                             _p(dw), _stream()), "moe_permute")
    return (out, dw) if Zp is not None else out


def router_fwd(X, Wr, out=None):
    """Trained router: logits [T, E] fp32 = X Wr^T."""
    T, H = X.shape
    E = Wr.shape[0]
    _need(X, torch.bfloat16, (T, H), "X")
    _need(Wr, torch.bfloat16, (E, H), "Wr")
    if out is None:
        out = torch.empty((T, E), dtype=torch.float32, device=X.device)
    _need(out, torch.float32, (T, E), "logits")
    _check(lib().moe_router_fwd(_p(X), _p(Wr), T, H, E, _p(out), _stream()), "moe_router_fwd")
    return out


def router_bwd(w, dw, idx, dest, offsets, Xp, Wr, dXp, out=None, ws=None):
    """Trained router backward: returns (dX with the router's part, dWr fp32)."""
    T, k = w.shape
    E, H = Wr.shape
    for t, dt, sh, n in ((w, torch.float32, (T, k), "w"), (dw, torch.float32, (T, k), "dw"),
                         (idx, torch.int32, (T, k), "idx"), (dest, torch.int32, (T, k), "dest"),
                         (offsets, torch.int32, (E + 1,), "offsets"),
                         (Xp, torch.bfloat16, (T * k, H), "Xp"), (Wr, torch.bfloat16, (E, H), "Wr"),
                         (dXp, torch.bfloat16, (T * k, H), "dXp")):
        _need(t, dt, sh, n)
    dev = Xp.device
    if out is None:
        out = (torch.empty((T, H), dtype=torch.bfloat16, device=dev),
               torch.empty((E, H), dtype=torch.float32, device=dev))
    dX, dWr = out
    _room((dX, T * H, "dX"), (dWr, E * H, "dWr"))
    nb = int(lib().moe_router_bwd_workspace_bytes(T, k))
    if ws is None or ws.numel() < nb:
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
    _check(lib().moe_router_bwd(_p(w), _p(dw), _p(idx), _p(dest), _p(offsets), _p(Xp), _p(Wr),
                                _p(dXp), T, H, E, k, _p(dX), _p(dWr), _p(ws), ws.numel(),
                                _stream()),
           "moe_router_bwd")
    return dX, dWr


def unpermute(Yp, dest, w=None, out=None):
    """a5 / a10: Y[t] = sum_j w[t, j] Yp[dest[t, j]]."""
    T, k = dest.shape
    H = Yp.shape[1]
    _need(Yp, torch.bfloat16, (T * k, H), "Yp")
    _need(dest, torch.int32, (T, k), "dest")
    if w is not None:
        _need(w, torch.float32, (T, k), "w")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=Yp.device)
    _room((out, T * H, "Y"))
    _check(lib().moe_unpermute(_p(Yp), _p(dest), _p(w), T, H, k, _p(out), _stream()),
           "moe_unpermute")
    return out


def ep_regroup(inp, counts, direction, out=None, offsets=None):
    """Expert parallelism: rows from N source ranks for this rank's E_loc
    experts (``counts`` [N, E_loc] int32 on the device), source-major ->
    expert-major (``direction`` 0, optionally writing the local ``offsets``
    [E_loc + 1]) or back (1)."""
    rows, H = inp.shape
    N, EL = counts.shape
    _need(inp, torch.bfloat16, (rows, H), "rows")
    _need(counts, torch.int32, (N, EL), "counts")
    if out is None:
        out = torch.empty_like(inp)
    _room((out, rows * H, "out"))
    if offsets is not None:
        _need(offsets, torch.int32, (EL + 1,), "offsets")
    _check(lib().moe_ep_regroup(_p(inp), _p(counts), N, EL, rows, H, int(direction), _p(out),
                                _p(offsets), _stream()),
           "moe_ep_regroup")
    return out


def _weights_check(W1, A1, B1, W2, A2, B2):
    E, I2, H = W1.shape
    I = I2 // 2
    r = A1.shape[1]
    for t, shp, n in [(W1, (E, 2 * I, H), "W1"), (A1, (E, r, H), "A1"),
                      (B1, (E, 2 * I, r), "B1"), (W2, (E, H, I), "W2"),
                      (A2, (E, r, I), "A2"), (B2, (E, H, r), "B2")]:
        _need(t, torch.bfloat16, shp, n)
    return E, H, I, r


def lora_mlp_fwd(Xp, offsets, W1, A1, B1, W2, A2, B2, s, out=None, saved=None):
    """a3 + a4: returns (Z2 [R, H], saved uint8 buffer)."""
    E, H, I, r = _weights_check(W1, A1, B1, W2, A2, B2)
    R = Xp.shape[0]
    _need(Xp, torch.bfloat16, (R, H), "Xp")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    if out is None:
        out = torch.empty((R, H), dtype=torch.bfloat16, device=Xp.device)
    _room((out, R * H, "Z2"))
    nb = saved_bytes(R, H, I, r)
    if saved is None:
        saved = torch.empty(max(nb, 1), dtype=torch.uint8, device=Xp.device)
    _check(lib().moe_lora_mlp_fwd(_p(Xp), _p(offsets), E, H, I, r, float(s), _p(W1),
                                  _p(A1), _p(B1), _p(W2), _p(A2), _p(B2), R, _p(out),
                                  _p(saved), saved.numel(), None, 0, _stream()),
           "moe_lora_mlp_fwd")
    return out, saved


def lora_mlp_bwd(dZ2, Xp, offsets, W1, A1, B1, W2, A2, B2, s, saved, out=None,
                 ws=None, base_out=None):
    """a7 + a8 + a9: returns (dXp, dA1, dB1, dA2, dB2).  With ``base_out`` =
    (dW1 [E, 2I, H], dW2 [E, H, I]) the base-weight gradients of full
    fine-tuning are written there too (``moe_lora_mlp_bwd_full``)."""
    E, H, I, r = _weights_check(W1, A1, B1, W2, A2, B2)
    R = Xp.shape[0]
    _need(dZ2, torch.bfloat16, (R, H), "dZ2")
    _need(Xp, torch.bfloat16, (R, H), "Xp")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    dev = Xp.device
    if out is None:
        out = (torch.empty((R, H), dtype=torch.bfloat16, device=dev),
               torch.empty((E, r, H), dtype=torch.bfloat16, device=dev),
               torch.empty((E, 2 * I, r), dtype=torch.bfloat16, device=dev),
               torch.empty((E, r, I), dtype=torch.bfloat16, device=dev),
               torch.empty((E, H, r), dtype=torch.bfloat16, device=dev))
    dXp, dA1, dB1, dA2, dB2 = out
    _room((dXp, R * H, "dXp"), (dA1, E * r * H, "dA1"), (dB1, E * 2 * I * r, "dB1"),
          (dA2, E * r * I, "dA2"), (dB2, E * H * r, "dB2"))
    nb = workspace_bytes(R, E, H, I, r)
    if ws is None or ws.numel() < nb:
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
    if base_out is None:
        _check(lib().moe_lora_mlp_bwd(_p(dZ2), _p(Xp), _p(offsets), E, H, I, r, float(s),
                                      _p(W1), _p(A1), _p(B1), _p(W2), _p(A2), _p(B2),
                                      _p(saved), saved.numel(), R, _p(dXp), _p(dA1),
                                      _p(dB1), _p(dA2), _p(dB2), _p(ws), ws.numel(),
                                      _stream()),
               "moe_lora_mlp_bwd")
    else:
        dW1, dW2 = base_out
        _need(dW1, torch.bfloat16, (E, 2 * I, H), "dW1")
        _need(dW2, torch.bfloat16, (E, H, I), "dW2")
        _check(lib().moe_lora_mlp_bwd_full(_p(dZ2), _p(Xp), _p(offsets), E, H, I, r,
                                           float(s), _p(W1), _p(A1), _p(B1), _p(W2),
                                           _p(A2), _p(B2), _p(saved), saved.numel(), R,
                                           _p(dXp), _p(dA1), _p(dB1), _p(dA2), _p(dB2),
                                           _p(dW1), _p(dW2), _p(ws), ws.numel(),
                                           _stream()),
               "moe_lora_mlp_bwd_full")
    return dXp, dA1, dB1, dA2, dB2


# ------------------------------------------------- operators around the block
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}
MAX_ROWS = 1 << 30


def _rows_need(x, name):
    """Element type code, shape and device index of a [T, H] operand."""
    code = DTYPES.get(x.dtype)
    if code is None:
        raise ValueError(f"{name}: expected bfloat16, float16 or float32, got {x.dtype}")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected two dimensions, got {len(shape)}")
    if shape[0] > MAX_ROWS or shape[1] > MAX_ROWS:  # a C int would take them modulo 2^32
        raise ValueError(f"{name}: at most 2^30 rows and columns, got {tuple(shape)}")
    dev = x.get_device()
    if dev < 0 or not x.is_contiguous():
        _need(x, x.dtype, shape, name)
    return code, shape[0], shape[1], dev


def _ptr(t, dtype, dev, shape, name):
    """Address of t (None: null) if it has the type, device and shape."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _need(t, dtype, shape, name)
        raise ValueError(f"{name} must be on cuda:{dev}")
    return t.data_ptr()


def _rng_need(p, rng, dev):
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be in [0, 1], got {p}")
    if rng is None and p > 0.0:
        raise ValueError("p > 0 needs rng = int64 [2] (seed, offset) on the device")
    return _ptr(rng, torch.int64, dev, (2,), "rng")


def _gate_need(gate, dtype, dev, T, H):
    """(kind, pointer) of a gate of shape [T, 1], [H] or [T, H] (or None)."""
    if gate is None:
        return 0, None
    shape = gate.shape
    kind = 3 if shape == (T, H) else 1 if shape == (T, 1) else 2 if shape == (H,) else None
    if kind is None:
        raise ValueError(f"gate: expected shape {(T, 1)}, {(H,)} or {(T, H)}, got {tuple(shape)}")
    return kind, _ptr(gate, dtype, dev, shape, "gate")


# the stream's handle without building a Stream object, where torch has that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(dev):
    """Context in which device dev is the current one (dev < 0: no device)."""
    if dev < 0 or dev == _current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _run(name, dev, *args):
    """Calls a C entry point on device dev's current stream, with dev the
    current device for the length of the call."""
    fn = getattr(_lib or lib(), name)
    if _current_device() == dev:
        code = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _raw_stream(dev))
    if code != MOE_OK:
        raise MoeError(code, name)


def residual_norm_fwd(y, res=None, w_post=None, gate=None, scale=1.0, w_pre=None, w_offset=0.0,
                      eps=1e-6, p=0.0, rng=None, out=None):
    """The norms before and after a block with its dropout, gate, residual
    scale and residual add, in one pass over ``y`` [T, H]:

        b = rms_norm(y) * (w_offset + w_post)     (b = y without ``w_post``)
        r = res + scale * gate * dropout(b, p)    (``gate`` [T, 1], [H] or [T, H])
        n = rms_norm(r) * (w_offset + w_pre)      (n = None without ``w_pre``)

    Returns ``(r, n, stats)``; ``stats`` fp32 [2, T] is for the backward.
    Without ``res``, ``w_post``, ``gate``, dropout and scale, r is y itself
    (the norm before a block) and nothing but n is written.  All tensors have
    y's type (bf16, fp16 or fp32); ``rng`` as in :func:`dropout_fwd`."""
    code, T, H, dev = _rows_need(y, "y")
    dt, rows = y.dtype, (T, H)
    kind, g = _gate_need(gate, dt, dev, T, H)
    rp = _rng_need(p, rng, dev)
    plain = res is None and w_post is None and gate is None and p == 0.0 and scale == 1.0
    if plain and w_pre is None:
        raise ValueError("nothing to do: no norm, residual, gate, dropout or scale")
    if out is None:
        out = (y if plain else torch.empty_like(y),
               None if w_pre is None else torch.empty_like(y),
               torch.empty((2, T), dtype=torch.float32, device=y.device))
    r, n, stats = out
    if plain and (r is None or r is y):
        r = y
        rptr = None
    else:
        if r is None:
            raise ValueError("out: r is needed")
        rptr = _ptr(r, dt, dev, rows, "r")
    _run("moe_residual_norm_fwd", dev, y.data_ptr(), _ptr(res, dt, dev, rows, "res"),
         _ptr(w_post, dt, dev, (H,), "w_post"), g, kind, scale,
         _ptr(w_pre, dt, dev, (H,), "w_pre"), w_offset, eps, p, rp, T, H, code, rptr,
         _ptr(n, dt, dev, rows, "n"), _ptr(stats, torch.float32, dev, (2, T), "stats"))
    return r, n, stats


def residual_norm_bwd(dr, dn, y, r, stats, w_post=None, gate=None, scale=1.0, w_pre=None,
                      w_offset=0.0, p=0.0, rng=None, out=None, ws=None):
    """Backward of :func:`residual_norm_fwd` from ``dr`` (None: zero) and
    ``dn`` (with ``w_pre``): returns ``(dres, dy, dgate, dw_post, dw_pre)``.
    ``dres`` is the gradient of ``res``; where r is y itself (no ``w_post``,
    ``gate``, dropout or scale) ``dres`` is also y's gradient and ``dy`` is
    the same tensor.  Parameters' gradients have the parameters' shapes and
    type (fp32 sums, rounded once)."""
    code, T, H, dev = _rows_need(y, "y")
    dt, rows = y.dtype, (T, H)
    kind, g = _gate_need(gate, dt, dev, T, H)
    rp = _rng_need(p, rng, dev)
    if (w_pre is None) != (dn is None):
        raise ValueError("dn is given exactly when w_pre is")
    if dr is None and dn is None:
        raise ValueError("dr or dn is needed")
    plain = w_post is None and gate is None and p == 0.0 and scale == 1.0
    if out is None:
        dres = torch.empty_like(y)
        out = (dres, dres if plain else torch.empty_like(y),
               None if gate is None else torch.empty_like(gate),
               None if w_post is None else torch.empty_like(w_post),
               None if w_pre is None else torch.empty_like(w_pre))
    dres, dy, dgate, dw_post, dw_pre = out
    if plain and dy is dres:
        dy = None
    nb = lib().moe_residual_norm_bwd_workspace_bytes(T, H, code)
    ws = _bytes_need(ws, nb, y, "ws")
    _run("moe_residual_norm_bwd", dev, _ptr(dr, dt, dev, rows, "dr"),
         _ptr(dn, dt, dev, rows, "dn"), y.data_ptr(), _ptr(r, dt, dev, rows, "r"),
         _ptr(stats, torch.float32, dev, (2, T), "stats"), _ptr(w_post, dt, dev, (H,), "w_post"),
         g, kind, scale, _ptr(w_pre, dt, dev, (H,), "w_pre"), w_offset, p, rp, T, H, code,
         _ptr(dres, dt, dev, rows, "dres"), _ptr(dy, dt, dev, rows, "dy"),
         _ptr(dgate, dt, dev, () if gate is None else gate.shape, "dgate"),
         _ptr(dw_post, dt, dev, (H,), "dw_post"), _ptr(dw_pre, dt, dev, (H,), "dw_pre"),
         ws.data_ptr(), ws.numel())
    return out


def dropout_fwd(x, p, rng, out=None):
    """x / (1 - p) where kept, 0 elsewhere, for ``x`` [T, H].  ``rng`` int64
    [2] on the device = (seed, offset): the mask is a function of it and of
    the element's place alone (Philox4x32-10) and is never stored.  Change
    the offset for every draw that is to differ."""
    code, T, H, dev = _rows_need(x, "x")
    if rng is None:
        raise ValueError("rng is needed")
    rp = _rng_need(p, rng, dev)
    if out is None:
        out = torch.empty_like(x)
    _run("moe_dropout", dev, x.data_ptr(), T, H, code, p, rp, _ptr(out, x.dtype, dev, (T, H), "out"))
    return out


def dropout_bwd(dy, p, rng, out=None):
    """Gradient of :func:`dropout_fwd` at the same ``p`` and ``rng``."""
    return dropout_fwd(dy, p, rng, out)


def ffn_saved_bytes(T, H, I):
    return lib().moe_ffn_saved_bytes(T, H, I)


def ffn_workspace_bytes(T, H, I):
    return lib().moe_ffn_workspace_bytes(T, H, I)


FFN_PRODUCTS = ("gate_up", "down", "dh", "dX", "dW1", "dW2")


def ffn_kernels(T, H, I, need_dw=True):
    """The kernel that each product of a call with these sizes runs on
    (the library's own choice; host-side, no GPU needed): "tokens", "pairs",
    "pairs merged", or (n, s) for 128 x n tiles over clusters of s."""
    out = {}
    for i, name in enumerate(FFN_PRODUCTS[:6 if need_dw else 4]):
        v = lib().moe_ffn_kernel(T, H, I, i, int(need_dw))
        if v < 0:
            raise ValueError(f"no feed-forward block of {T} x {H} x {I}")
        out[name] = ("tokens", "pairs", "pairs merged")[v] if v < 3 else divmod(v, 16)
    return out


def _ffn_need(X, W1, W2, act):
    code, T, H, dev = _rows_need(X, "X")
    a = ACTIVATIONS.get(act)
    if a is None:
        raise ValueError(f"act: expected one of {sorted(ACTIVATIONS)}, got {act!r}")
    if W2.dim() != 2:
        raise ValueError("W2: expected [H, I]")
    I, dt = W2.shape[1], X.dtype
    if I > MAX_ROWS:
        raise ValueError(f"W2: at most 2^30 columns, got {I}")
    return (code, T, H, I, dev, _ptr(W1, dt, dev, (2 * I, H), "W1"),
            _ptr(W2, dt, dev, (H, I), "W2"), a)


def _bytes_need(t, n, x, name):
    """A uint8 buffer of at least n bytes on x's device (made where None)."""
    if t is None:
        return torch.empty(n, dtype=torch.uint8, device=x.device)
    if (t.dtype is not torch.uint8 or t.get_device() != x.get_device() or t.numel() < n
            or not t.is_contiguous()):
        raise ValueError(f"{name}: expected a uint8 tensor of {n} bytes on {x.device}")
    return t


def ffn_fwd(X, W1, W2, act="silu", add=None, out=None, save=True, saved=None, ws=None):
    """Dense gated feed-forward block (a shared expert): with [g | u] = X W1^T
    and h = act(g) * u, Y = add + h W2^T.  ``W1`` [2I, H] (gate rows first),
    ``W2`` [H, I], bf16 or fp16.  Returns ``(Y, saved)``: ``saved`` is for
    the backward, None with ``save=False`` (inference, one token to many).
    ``out`` may be ``add``."""
    code, T, H, I, dev, w1, w2, a = _ffn_need(X, W1, W2, act)
    dt, rows = X.dtype, (T, H)
    if out is None:
        out = torch.empty_like(X)
    if save:
        saved = buf = _bytes_need(saved, lib().moe_ffn_saved_bytes(T, H, I), X, "saved")
        bufs = (buf.data_ptr(), buf.numel(), None, 0)
    else:
        saved = None
        buf = _bytes_need(ws, lib().moe_ffn_workspace_bytes(T, H, I), X, "ws")
        bufs = (None, 0, buf.data_ptr(), buf.numel())
    _run("moe_ffn_fwd", dev, X.data_ptr(), w1, w2, T, H, I, code, a,
         _ptr(add, dt, dev, rows, "add"), _ptr(out, dt, dev, rows, "out"), *bufs)
    return out, saved


def ffn_bwd(dY, X, W1, W2, saved, act="silu", add=None, need_dw=True, out=None, ws=None):
    """Backward of :func:`ffn_fwd`: returns ``(dX, dW1, dW2)``, with ``add``
    (another path's gradient of X) added to dX; the weights' gradients are
    None with ``need_dw=False`` (frozen weights).  The gradient of the
    forward's ``add`` is dY itself."""
    code, T, H, I, dev, w1, w2, a = _ffn_need(X, W1, W2, act)
    dt, rows = X.dtype, (T, H)
    if dY is None or saved is None:
        raise ValueError("dY and the forward's saved are needed")
    if out is None:
        out = (torch.empty_like(X), torch.empty_like(W1) if need_dw else None,
               torch.empty_like(W2) if need_dw else None)
    dX, dW1, dW2 = out
    saved = _bytes_need(saved, lib().moe_ffn_saved_bytes(T, H, I), X, "saved")
    ws = _bytes_need(ws, lib().moe_ffn_workspace_bytes(T, H, I), X, "ws")
    _run("moe_ffn_bwd", dev, _ptr(dY, dt, dev, rows, "dY"), X.data_ptr(), w1, w2, T, H, I, code,
         a, saved.data_ptr(), saved.numel(), _ptr(add, dt, dev, rows, "add"),
         _ptr(dX, dt, dev, rows, "dX"), _ptr(dW1, dt, dev, (2 * I, H), "dW1"),
         _ptr(dW2, dt, dev, (H, I), "dW2"), ws.data_ptr(), ws.numel())
    return out


# ------------------------------------------------------------------ the block
def _on_own_device(method):
    """The method runs with the object's device as the current one: on its
    current stream, and the block's calls are made on no other device."""
    @functools.wraps(method)
    def run(self, *args, **kwargs):
        with _on(self.dev):
            return method(self, *args, **kwargs)
    return run


class MoeBlock:
    """Forward + backward of the whole block through the C ABI, with all
    buffers preallocated once for a fixed shape (used by the benchmark and the
    end-to-end tests).  ``step`` runs, on the current stream: route, permute,
    gate_up + SwiGLU, down, weighted unpermute, weighted dY gather, down /
    gate_up backward, LoRA gradients and the dX combine (with ``full_ft``, also
    the base-weight gradients dW1, dW2 of full fine-tuning)."""

    def __init__(self, T, H, I, E, k, r, s, device="cuda", with_dw=False, full_ft=False,
                 train_router=False):
        self.T, self.H, self.I, self.E, self.k, self.r, self.s = T, H, I, E, k, r, s
        self.R = R = T * k
        self.with_dw = with_dw
        dev = torch.device(device)
        bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
        self.idx = torch.empty((T, k), dtype=i32, device=dev)
        self.w = torch.empty((T, k), dtype=f32, device=dev)
        self.counts = torch.empty((E,), dtype=i32, device=dev)
        self.offsets = torch.empty((E + 1,), dtype=i32, device=dev)
        self.dest = torch.empty((T, k), dtype=i32, device=dev)
        self.route_ws = torch.empty(route_workspace_bytes(T, E, k), dtype=torch.uint8,
                                    device=dev)
        self.Xp = torch.empty((R, H), dtype=bf, device=dev)
        self.Z2 = torch.empty((R, H), dtype=bf, device=dev)
        self.saved = torch.empty(max(1, saved_bytes(R, H, I, r)), dtype=torch.uint8,
                                 device=dev)
        self.Y = torch.empty((T, H), dtype=bf, device=dev)
        self.dev = self.Y.get_device()   # every method runs with it as the current device
        self.dZ2 = torch.empty((R, H), dtype=bf, device=dev)
        self.dw = torch.empty((T, k), dtype=f32, device=dev) if with_dw else None
        self.dXp = torch.empty((R, H), dtype=bf, device=dev)
        self.dX = torch.empty((T, H), dtype=bf, device=dev)
        self.dA1 = torch.empty((E, r, H), dtype=bf, device=dev)
        self.dB1 = torch.empty((E, 2 * I, r), dtype=bf, device=dev)
        self.dA2 = torch.empty((E, r, I), dtype=bf, device=dev)
        self.dB2 = torch.empty((E, H, r), dtype=bf, device=dev)
        self.full_ft = full_ft
        # trained router: logits = X Wr^T on the device; dw, dlogits -> dWr and
        # the router's part of dX (needs the routing-weight gradient)
        self.train_router = train_router
        if train_router:
            self.with_dw = True
            self.dw = torch.empty((T, k), dtype=f32, device=dev)
            self.logits = torch.empty((T, E), dtype=f32, device=dev)
            self.dWr = torch.empty((E, H), dtype=f32, device=dev)
            self.router_ws = torch.empty(max(1, int(lib().moe_router_bwd_workspace_bytes(T, k))),
                                         dtype=torch.uint8, device=dev)
        self.dW1 = torch.empty((E, 2 * I, H), dtype=bf, device=dev) if full_ft else None
        self.dW2 = torch.empty((E, H, I), dtype=bf, device=dev) if full_ft else None
        self.ws = torch.empty(max(1, workspace_bytes(R, E, H, I, r)), dtype=torch.uint8,
                              device=dev)

    @_on_own_device
    def forward(self, X, logits, W, Wr=None):
        if self.train_router:
            logits = router_fwd(X, Wr, out=self.logits)
        route_topk(logits, self.k, out=(self.idx, self.w, self.counts, self.offsets,
                                        self.dest), ws=self.route_ws)
        permute(X, self.dest, out=self.Xp)
        lora_mlp_fwd(self.Xp, self.offsets, *W, self.s, out=self.Z2, saved=self.saved)
        unpermute(self.Z2, self.dest, self.w, out=self.Y)
        return self.Y

    @_on_own_device
    def backward(self, dY, W, Wr=None):
        if self.with_dw:
            permute(dY, self.dest, scale=self.w, Zp=self.Z2, out=self.dZ2, dw=self.dw)
        else:
            permute(dY, self.dest, scale=self.w, out=self.dZ2)
        lora_mlp_bwd(self.dZ2, self.Xp, self.offsets, *W, self.s, self.saved,
                     out=(self.dXp, self.dA1, self.dB1, self.dA2, self.dB2), ws=self.ws,
                     base_out=(self.dW1, self.dW2) if self.full_ft else None)
        if self.train_router:
            router_bwd(self.w, self.dw, self.idx, self.dest, self.offsets, self.Xp, Wr,
                       self.dXp, out=(self.dX, self.dWr), ws=self.router_ws)
        else:
            unpermute(self.dXp, self.dest, None, out=self.dX)
        return self.dX

    @_on_own_device
    def step(self, X, logits, dY, W, Wr=None):
        """One fwd+bwd; with a trained router, ``Wr`` [E, H] bf16 replaces
        ``logits`` (which may then be None)."""
        self.forward(X, logits, W, Wr)
        self.backward(dY, W, Wr)

    @_on_own_device
    def capture(self, X, logits, dY, W, Wr=None):
        """Capture one ``step`` on these exact tensors into a CUDA graph;
        ``replay`` then re-runs all of its kernels with one launch.  Inputs
        must be updated in place (the graph holds their addresses).  The
        library launches nothing but its own kernels and stream-ordered
        memsets, and allocates nothing, so the captured step is the same work
        as ``step``."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):      # one eager step off the capture
            self.step(X, logits, dY, W, Wr)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step(X, logits, dY, W, Wr)
        self._graph = graph
        return graph

    def replay(self):
        """Run the captured step on the current stream."""
        self._graph.replay()

    @_on_own_device
    def capture_parts(self, X, logits, dY, W, Wr=None):
        """Capture the forward and the backward of one step on these exact
        tensors into two CUDA graphs (``replay_forward``, ``replay_backward``),
        so that a caller can overlap dY's upload with the forward and Y's
        download with the backward."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):      # one eager step off the capture
            self.step(X, logits, dY, W, Wr)
        torch.cuda.current_stream().wait_stream(side)
        gf, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gf):
            self.forward(X, logits, W, Wr)
        with torch.cuda.graph(gb):
            self.backward(dY, W, Wr)
        self._graph_fwd, self._graph_bwd = gf, gb
        return gf, gb

    def replay_forward(self):
        self._graph_fwd.replay()

    def replay_backward(self):
        self._graph_bwd.replay()


# ------------------------------------------------------------------ the layer
class MoeLayer:
    """The expert half of a decoder layer, forward and backward: a
    :class:`MoeBlock` with the norms before and after it, an optional shared
    expert beside it and dropout, all buffers preallocated for one shape:

        n   = dropout(rms_norm(X) * (w_offset + w_pre), p_in)
        y   = MoE(n) + FFN(n)                    (FFN: the shared expert)
        out = X + scale * gate * dropout(rms_norm(y) * (w_offset + w_post), p)

    ``norms`` = (w_pre, w_post or None); ``shared`` = (W1 [2 I_s, H],
    W2 [H, I_s]) where ``I_shared`` > 0; ``gate`` [T, 1], [H] or [T, H] or
    None; ``rng`` int64 [2, 2]: (seed, offset) of the dropout before and of
    the one after the block.  ``block`` options (``full_ft``,
    ``train_router``) are the MoeBlock's; ``full_ft`` also gives the shared
    expert's gradients.  Results: ``out``, ``dX``, ``dw_pre``, ``dw_post``,
    ``dgate``, ``dW1s``, ``dW2s`` and the block's."""

    def __init__(self, T, H, I, E, k, r, s, I_shared=0, act="silu", scale=1.0, eps=1e-6,
                 w_offset=0.0, p_in=0.0, p=0.0, post_norm=True, gate_shape=None, device="cuda",
                 **block):
        if act not in ACTIVATIONS:
            raise ValueError(f"act: expected one of {sorted(ACTIVATIONS)}, got {act!r}")
        if not (0.0 <= p_in <= 1.0 and 0.0 <= p <= 1.0):
            raise ValueError(f"p_in and p must be in [0, 1], got {p_in} and {p}")
        self.block = MoeBlock(T, H, I, E, k, r, s, device=device, **block)
        self.dev = self.block.dev
        self.act, self.scale, self.eps, self.w_offset = act, scale, eps, w_offset
        self.p_in, self.p, self.I_shared, self.post_norm = p_in, p, I_shared, post_norm
        dev = torch.device(device)
        bf = torch.bfloat16

        def rows():
            return torch.empty((T, H), dtype=bf, device=dev)

        self.n, self.out, self.dy, self.dn, self.dX = rows(), rows(), rows(), rows(), rows()
        self.nd = rows() if p_in > 0 else self.n      # what the block reads
        self.y = rows() if I_shared else self.block.Y
        self.stats_pre, self.stats_post = (
            torch.empty((2, T), dtype=torch.float32, device=dev) for _ in range(2))
        self.dw_pre = torch.empty((H,), dtype=bf, device=dev)
        self.dw_post = torch.empty((H,), dtype=bf, device=dev) if post_norm else None
        self.dgate = None if gate_shape is None else torch.empty(gate_shape, dtype=bf, device=dev)
        self.norm_ws = torch.empty(lib().moe_residual_norm_bwd_workspace_bytes(T, H, 0),
                                   dtype=torch.uint8, device=dev)
        self.dW1s = self.dW2s = None
        if I_shared:
            self.ffn_saved, self.ffn_ws = (
                torch.empty(f(T, H, I_shared), dtype=torch.uint8, device=dev)
                for f in (ffn_saved_bytes, ffn_workspace_bytes))
            if self.block.full_ft:
                self.dW1s = torch.empty((2 * I_shared, H), dtype=bf, device=dev)
                self.dW2s = torch.empty((H, I_shared), dtype=bf, device=dev)

    def _after(self, norms, shared, gate, rng):
        """Checks what both directions are given; the post norm's arguments."""
        if (shared is None) != (self.I_shared == 0):
            raise ValueError("shared: (W1, W2) is given exactly with I_shared")
        if (norms[1] is not None) != self.post_norm:
            raise ValueError("norms: w_post is given exactly with post_norm")
        if (gate is None) != (self.dgate is None):
            raise ValueError("gate: given exactly with gate_shape")
        if rng is None and (self.p > 0 or self.p_in > 0):
            raise ValueError("p or p_in > 0 needs rng = int64 [2, 2] on the device")
        return dict(w_post=norms[1], gate=gate, scale=self.scale, w_offset=self.w_offset, p=self.p,
                    rng=rng[1] if self.p > 0 else None)

    @_on_own_device
    def forward(self, X, logits, W, norms, shared=None, gate=None, rng=None, Wr=None):
        after = self._after(norms, shared, gate, rng)
        residual_norm_fwd(X, w_pre=norms[0], w_offset=self.w_offset, eps=self.eps,
                          out=(X, self.n, self.stats_pre))
        if self.p_in > 0:
            dropout_fwd(self.n, self.p_in, rng[0], out=self.nd)
        self.block.forward(self.nd, logits, W, Wr)
        if shared is not None:
            ffn_fwd(self.nd, *shared, act=self.act, add=self.block.Y, out=self.y,
                    saved=self.ffn_saved)
        residual_norm_fwd(self.y, X, eps=self.eps, out=(self.out, None, self.stats_post), **after)
        return self.out

    @_on_own_device
    def backward(self, dOut, X, W, norms, shared=None, gate=None, rng=None, Wr=None):
        after = self._after(norms, shared, gate, rng)
        dy = dOut
        if norms[1] is not None or gate is not None or self.p > 0 or self.scale != 1.0:
            dy = self.dy
            residual_norm_bwd(dOut, None, self.y, None, self.stats_post,
                              out=(None, dy, self.dgate, self.dw_post, None), ws=self.norm_ws,
                              **after)
        dn = self.block.backward(dy, W, Wr)
        if shared is not None:
            ffn_bwd(dy, self.nd, *shared, self.ffn_saved, act=self.act, add=dn,
                    need_dw=self.dW1s is not None, out=(self.dn, self.dW1s, self.dW2s),
                    ws=self.ffn_ws)
            dn = self.dn
        if self.p_in > 0:
            dn = dropout_bwd(dn, self.p_in, rng[0], out=self.dn)
        residual_norm_bwd(dOut, dn, X, X, self.stats_pre, w_pre=norms[0], w_offset=self.w_offset,
                          out=(self.dX, self.dX, None, None, self.dw_pre), ws=self.norm_ws)
        return self.dX

    @_on_own_device
    def step(self, X, logits, dOut, W, norms, shared=None, gate=None, rng=None, Wr=None):
        self.forward(X, logits, W, norms, shared, gate, rng, Wr)
        self.backward(dOut, X, W, norms, shared, gate, rng, Wr)

    @_on_own_device
    def capture(self, *args, **kwargs):
        """Capture one ``step`` on these exact tensors into a CUDA graph
        (``replay`` re-runs it); inputs, ``rng`` among them, are updated in
        place between replays."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):      # one eager step off the capture
            self.step(*args, **kwargs)
        torch.cuda.current_stream().wait_stream(side)
        self._graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self._graph):
            self.step(*args, **kwargs)
        return self._graph

    def replay(self):
        self._graph.replay()
