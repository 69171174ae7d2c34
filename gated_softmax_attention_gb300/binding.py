"""ctypes binding of libgsdpa.so: argument marshalling only.

Every step of the computation runs in the library's CUDA kernels. Torch is
used here for device memory (output and workspace tensors when the caller
does not pass them) and for the current stream. If the library has not been
built, every call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgsdpa.so")

GATE_NONE, GATE_HEADWISE, GATE_ELEMENTWISE = 0, 1, 2
GATE_CODES = {"none": GATE_NONE, "headwise": GATE_HEADWISE, "elementwise": GATE_ELEMENTWISE}
F32, BF16 = 0, 1

OK = 0
ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_LAUNCH, ERR_DEVICE_TIMEOUT = -1, -2, -3, -4, -5, -6
ERR_CACHE_RANGE = -7

# Every entry point the header declares, with its ctypes signature.
_VP, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_LL, _F, _D = ctypes.c_longlong, ctypes.c_float, ctypes.c_double
SIGNATURES = {
    "gsdpa_workspace_bytes": (_SZ, [_I] * 10),
    "gated_sdpa_fwd": (_I, [_VP] * 7 + [_I] * 10 + [_VP, _SZ, _VP]),
    "gated_sdpa_fwd_train": (_I, [_VP] * 8 + [_I] * 10 + [_VP, _SZ, _VP]),
    "gated_sdpa_fwd_train_save_gate": (_I, [_VP] * 9 + [_I] * 10 + [_VP, _SZ, _VP]),
    "gsdpa_workspace_bytes_variant": (_SZ, [_I] * 11),
    "gated_sdpa_fwd_stats": (_I, [_VP] * 8 + [_I, ctypes.c_float] + [_I] * 10 + [_VP, _SZ, _VP]),
    "gsdpa_layer_workspace_bytes": (_SZ, [_I] * 7),
    "gated_attention_layer": (_I, [_VP] * 4 + [_I] * 8 + [_VP, _SZ, _VP]),
    "gated_sdpa_fwd_variant": (_I, [_VP] * 7 + [_I] * 9 + [ctypes.c_float, _I, _I, _VP, _SZ, _VP]),
    "gsdpa_bwd_workspace_bytes": (_SZ, [_I] * 8),
    "gated_sdpa_bwd": (_I, [_VP] * 13 + [_I] * 10 + [_VP, _SZ, _VP]),
    "gated_sdpa_bwd_saved_gate": (_I, [_VP] * 14 + [_I] * 10 + [_VP, _SZ, _VP]),
    "gsdpa_check_device_error": (_I, [_VP]),
    "gsdpa_status_string": (ctypes.c_char_p, [_I]),
    "gsdpa_set_wait_limit_ns": (_I, [ctypes.c_ulonglong]),
    "gsdpa_wait_self_test": (_I, [_VP]),
    "gated_sdpa_decode_noalloc": (_I, [_VP] * 7 + [_I] * 7 + [_VP]),
    "gsdpa_decode_noalloc_max_scratch": (_SZ, []),
    "gsdpa_rope_init": (_I, [_VP, _I, _I, _D, _I] + [_D] * 5),
    "gsdpa_rope_init_freqs": (_I, [_VP, _I, _I, _VP, _D]),
    "gsdpa_qk_norm_rope": (_I, [_VP] * 7 + [_LL] * 4 + [_I] * 6 + [_F, _VP, _I, _VP]),
    "gsdpa_qk_norm_rope_bwd_workspace_bytes": (_SZ, [_I] * 4),
    "gsdpa_qk_norm_rope_bwd": (_I, [_VP] * 11 + [_LL] * 6 + [_I] * 6 + [_F, _VP, _I, _VP, _SZ, _VP]),
    "gsdpa_cache8_append": (_I, [_VP] * 3 + [_LL] * 2 + [_VP] * 2 + [_I, _VP]),
    "gsdpa_cache8_workspace_bytes": (_SZ, [_VP] + [_I] * 4),
    "gated_sdpa_cache8": (_I, [_VP] * 7 + [_I] * 4 + [_VP, _SZ, _VP]),
}

_lock = threading.Lock()
_lib = None


class GsdpaError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def load(path: str = LIB_PATH):
    """Load libgsdpa.so (once). Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with "
                                   "`python -m gated_softmax_attention_gb300.build`")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().gsdpa_status_string(int(status)).decode()


def workspace_bytes(B, L_q, L_k, d_model, H_q, H_kv, d_k, gate="elementwise", want_sink=False, dtype=BF16) -> int:
    n = load().gsdpa_workspace_bytes(B, L_q, L_k, d_model, H_q, H_kv, d_k, GATE_CODES[gate], int(bool(want_sink)),
                                     dtype)
    if n == ctypes.c_size_t(-1).value:
        raise GsdpaError(ERR_INVALID_ARG, "gsdpa_workspace_bytes")
    return int(n)


def set_wait_limit_ns(ns: int) -> None:
    load().gsdpa_set_wait_limit_ns(int(ns))


def wait_self_test(stream=None) -> int:
    """Enqueue the bounded-wait diagnostic (a wait nothing completes); returns the launch status."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(load().gsdpa_wait_self_test(ctypes.c_void_p(s.cuda_stream)))


def check_device_error(stream=None) -> int:
    """Synchronise the stream and return the device error status (0 = none)."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(load().gsdpa_check_device_error(ctypes.c_void_p(s.cuda_stream)))


def fwd_raw(X, Q, K, V, W_g, O, sink, B, L_q, L_k, d_model, H_q, H_kv, d_k, gate_mode, causal, dtype,
            workspace, workspace_bytes, stream) -> int:
    """Direct call of gated_sdpa_fwd with integer pointers; returns the status."""
    return int(load().gated_sdpa_fwd(X, Q, K, V, W_g, O, sink, B, L_q, L_k, d_model, H_q, H_kv, d_k, gate_mode,
                                     int(bool(causal)), dtype, workspace, workspace_bytes, stream))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The library receives bare pointers and sizes: it cannot see how large a
# buffer is. Every tensor is therefore checked here against the sizes the
# problem implies (dtype, element count, device, contiguity) before its
# pointer is passed, so that a wrong-shaped argument raises instead of being
# read or written past its end.
def _expect(t, name, numel, dtype, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's tensors on {device}")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements (shape {tuple(t.shape)}), the problem needs {numel}")


def _stream(stream, device):
    """The stream to launch on: the caller's, else the current stream of the
    device that holds the tensors (which must then be the current device)."""
    import torch
    if stream is None:
        if device.index != torch.cuda.current_device():
            raise ValueError(f"the tensors are on {device} but the current device is "
                             f"cuda:{torch.cuda.current_device()}: pass a stream of {device}")
        return torch.cuda.current_stream()
    if stream.device != device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {device}")
    return stream


def _attn_dims(Q, K, V):
    """(B, L_q, L_k, H_q, H_kv, d_k) from Q [B, L_q, H_q, d_k] and K, V [B, L_k, H_kv, d_k]."""
    if Q.dim() != 4 or K.dim() != 4 or V.dim() != 4:
        raise ValueError("Q, K and V must be 4-D: [B, L, H, d_k]")
    B, L_q, H_q, d_k = Q.shape
    if tuple(K.shape) != tuple(V.shape) or K.shape[0] != B or K.shape[3] != d_k:
        raise ValueError(f"K {tuple(K.shape)} and V {tuple(V.shape)} must be [B={B}, L_k, H_kv, d_k={d_k}]")
    return B, L_q, K.shape[1], H_q, K.shape[2], d_k


def _x_dim(X, B, L_q):
    """d_model of X [B, L_q, d_model] (any shape with that element count and last dimension)."""
    if X is None or X.dim() == 0:
        raise ValueError("X is required")
    d_model = X.shape[-1]
    if X.numel() != B * L_q * d_model:
        raise ValueError(f"X {tuple(X.shape)} must hold B * L_q = {B * L_q} rows of d_model = {d_model}")
    return d_model


# columns of W_g [d_model, G] (or the rows x columns of a table that does not read X)
def _gate_cols(gate_mode, H_q, d_k):
    return {GATE_HEADWISE: H_q, GATE_ELEMENTWISE: H_q * d_k, 3: 1, 4: d_k, 6: H_q, 7: H_q * d_k}[gate_mode]


def gated_sdpa_fwd(X, Q, K, V, W_g=None, *, gate="elementwise", causal=True, out=None, sink=None,
                   want_sink=False, workspace=None, stream=None):
    """Gated attention forward through the C ABI on torch CUDA tensors.

    X [B, L_q, d_model], Q [B, L_q, H_q, d_k], K/V [B, L_k, H_kv, d_k],
    W_g [d_model, H_q*d_k | H_q] (None for gate="none"). All contiguous, on
    the current CUDA device, float32 or bfloat16 (all the same dtype).
    Returns (O, sink) where sink is None unless requested.
    """
    O, sink, _ = _fwd(X, Q, K, V, W_g, gate, causal, out, sink, want_sink, None, workspace, stream)
    return O, sink


def gated_sdpa_fwd_train(X, Q, K, V, W_g=None, *, gate="elementwise", causal=True, out=None, sink=None,
                         want_sink=False, lse=None, workspace=None, stream=None):
    """gated_sdpa_fwd that also returns lse [B, H_q, L_q] float32, the natural
    log of each row's softmax denominator (bf16 prefill). Returns (O, sink, lse)."""
    import torch
    B, L_q, H_q, _ = Q.shape
    if lse is None:
        lse = torch.empty((B, H_q, L_q), dtype=torch.float32, device=Q.device)
    return _fwd(X, Q, K, V, W_g, gate, causal, out, sink, want_sink, lse, workspace, stream)


def gated_sdpa_fwd_train_save_gate(X, Q, K, V, W_g, *, causal=True, out=None, sink=None, want_sink=False, lse=None,
                                   gate_out=None, workspace=None, stream=None):
    """gated_sdpa_fwd_train for the elementwise gate that also returns the gate's
    fp16 values [B * L_q, H_q * d_k] for gated_sdpa_bwd_saved_gate. Returns
    (O, sink, lse, gate_out)."""
    import torch
    B, L_q, H_q, d_k = Q.shape
    if lse is None:
        lse = torch.empty((B, H_q, L_q), dtype=torch.float32, device=Q.device)
    if gate_out is None:
        gate_out = torch.empty((B * L_q, H_q * d_k), dtype=torch.float16, device=Q.device)
    O, sink, lse = _fwd(X, Q, K, V, W_g, "elementwise", causal, out, sink, want_sink, lse, workspace, stream,
                        gate_out=gate_out)
    return O, sink, lse, gate_out


def _workspace(workspace, need, device):
    """(pointer, size in bytes) of the call's workspace: the caller's tensor,
    whose real size is passed so that the library can reject one too small,
    or a new one of the size the problem needs."""
    import torch
    if workspace is None:
        if need <= 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("the workspace must be a contiguous CUDA tensor")
    if workspace.device != device:
        raise ValueError(f"the workspace is on {workspace.device}, the call's tensors on {device}")
    return workspace, workspace.numel() * workspace.element_size()


def _fwd(X, Q, K, V, W_g, gate, causal, out, sink, want_sink, lse, workspace, stream, gate_out=None):
    import torch
    if Q.dtype == torch.bfloat16:
        dtype = BF16
    elif Q.dtype == torch.float32:
        dtype = F32
    else:
        raise TypeError(f"unsupported dtype {Q.dtype}")
    gm = GATE_CODES[gate]
    B, L_q, L_k, H_q, H_kv, d_k = _attn_dims(Q, K, V)
    dev = Q.device
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        _expect(t, name, t.numel(), Q.dtype, dev)
    d_model = 0
    if gm != GATE_NONE:
        d_model = _x_dim(X, B, L_q)
        _expect(X, "X", B * L_q * d_model, Q.dtype, dev)
        _expect(W_g, "W_g", d_model * _gate_cols(gm, H_q, d_k), Q.dtype, dev)
    if out is None:
        out = torch.empty_like(Q)
    _expect(out, "out", Q.numel(), Q.dtype, dev)
    if sink is None and want_sink:
        sink = torch.empty((B, H_q), dtype=torch.float32, device=dev)
    if sink is not None:
        _expect(sink, "sink", B * H_q, torch.float32, dev)
    if lse is not None:
        _expect(lse, "lse", B * H_q * L_q, torch.float32, dev)
    if gate_out is not None:
        _expect(gate_out, "gate_out", B * L_q * H_q * d_k, torch.float16, dev)
    need = workspace_bytes(B, L_q, L_k, d_model, H_q, H_kv, d_k, gate, sink is not None, dtype)
    workspace, ws_bytes = _workspace(workspace, need, dev)
    s = _stream(stream, dev)
    args = [_ptr(X) if gm != GATE_NONE else None, _ptr(Q), _ptr(K), _ptr(V),
            _ptr(W_g) if gm != GATE_NONE else None, _ptr(out), _ptr(sink)]
    tail = [B, L_q, L_k, d_model, H_q, H_kv, d_k, gm, int(bool(causal)), dtype,
            _ptr(workspace), ws_bytes, ctypes.c_void_p(s.cuda_stream)]
    if gate_out is not None:
        st = int(load().gated_sdpa_fwd_train_save_gate(*args, _ptr(lse), _ptr(gate_out), *tail))
        where = "gated_sdpa_fwd_train_save_gate"
    elif lse is None:
        st = int(load().gated_sdpa_fwd(*args, *tail))
        where = "gated_sdpa_fwd"
    else:
        st = int(load().gated_sdpa_fwd_train(*args, _ptr(lse), *tail))
        where = "gated_sdpa_fwd_train"
    if st != OK:
        raise GsdpaError(st, where)
    return out, sink, lse


# gate shapes and gate functions of gated_sdpa_fwd_variant (gsdpa.h)
VARIANT_GATE_CODES = dict(GATE_CODES, headwise_shared=3, elementwise_shared=4, static=5, headwise_averaged=6,
                          elementwise_averaged=7)
GATE_FNS = {"sigmoid_mul": 0, "ns_sigmoid_mul": 1, "sigmoid_add": 2, "silu_add": 3, "identity_add": 4,
            "silu_self": 5, "rmsnorm": 6}


def workspace_bytes_variant(B, L_q, L_k, d_model, H_q, H_kv, d_k, gate="elementwise", gate_fn="sigmoid_mul",
                            want_sink=False, dtype=BF16) -> int:
    n = load().gsdpa_workspace_bytes_variant(B, L_q, L_k, d_model, H_q, H_kv, d_k, VARIANT_GATE_CODES[gate],
                                             GATE_FNS[gate_fn], int(bool(want_sink)), dtype)
    if n == ctypes.c_size_t(-1).value:
        raise GsdpaError(ERR_INVALID_ARG, "gsdpa_workspace_bytes_variant")
    return int(n)


def gated_sdpa_fwd_variant(X, Q, K, V, W_g=None, *, gate="elementwise", gate_fn="sigmoid_mul", eps=1e-6,
                           causal=True, out=None, sink=None, want_sink=False, workspace=None, stream=None):
    """The forward with a gate variant (gated_sdpa_fwd_variant): ``gate`` one of
    none, headwise, elementwise, headwise_shared (W_g [d_model, 1]),
    elementwise_shared (W_g [d_model, d_k]), static (W_g = theta [H_q, d_k],
    X unused); ``gate_fn`` one of GATE_FNS (rmsnorm: W_g = gamma [H_q, d_k] or
    None). Returns (O, sink)."""
    import torch
    if Q.dtype == torch.bfloat16:
        dtype = BF16
    elif Q.dtype == torch.float32:
        dtype = F32
    else:
        raise TypeError(f"unsupported dtype {Q.dtype}")
    gm, fn = VARIANT_GATE_CODES[gate], GATE_FNS[gate_fn]
    reads_x = gm not in (GATE_NONE, 5)
    B, L_q, L_k, H_q, H_kv, d_k = _attn_dims(Q, K, V)
    dev = Q.device
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        _expect(t, name, t.numel(), Q.dtype, dev)
    d_model = 0
    if reads_x:
        d_model = _x_dim(X, B, L_q)
        _expect(X, "X", B * L_q * d_model, Q.dtype, dev)
        _expect(W_g, "W_g", d_model * _gate_cols(gm, H_q, d_k), Q.dtype, dev)
    elif gm == 5:
        _expect(W_g, "W_g (theta)", H_q * d_k, Q.dtype, dev)
    elif fn == GATE_FNS["rmsnorm"] and W_g is not None:
        _expect(W_g, "W_g (gamma)", H_q * d_k, Q.dtype, dev)
    if out is None:
        out = torch.empty_like(Q)
    _expect(out, "out", Q.numel(), Q.dtype, dev)
    if sink is None and want_sink:
        sink = torch.empty((B, H_q), dtype=torch.float32, device=dev)
    if sink is not None:
        _expect(sink, "sink", B * H_q, torch.float32, dev)
    need = workspace_bytes_variant(B, L_q, L_k, d_model, H_q, H_kv, d_k, gate, gate_fn, sink is not None, dtype)
    workspace, ws_bytes = _workspace(workspace, need, dev)
    s = _stream(stream, dev)
    st = int(load().gated_sdpa_fwd_variant(
        _ptr(X) if reads_x else None, _ptr(Q), _ptr(K), _ptr(V), _ptr(W_g), _ptr(out), _ptr(sink),
        B, L_q, L_k, d_model, H_q, H_kv, d_k, gm, fn, float(eps), int(bool(causal)), dtype,
        _ptr(workspace), ws_bytes, ctypes.c_void_p(s.cuda_stream)))
    if st != OK:
        raise GsdpaError(st, "gated_sdpa_fwd_variant")
    return out, sink


def gated_sdpa_fwd_stats(X, Q, K, V, W_g, *, gate="elementwise", causal=True, n_bins=20, threshold=0.1, out=None,
                         workspace=None, stream=None):
    """gated_sdpa_fwd with the gate statistics: returns (O, stats) where stats is
    a dict with count, mean (sum / 2^32 / count), below, hist (n_bins counts)."""
    import torch
    dtype = BF16 if Q.dtype == torch.bfloat16 else F32
    gm = GATE_CODES[gate]
    B, L_q, L_k, H_q, H_kv, d_k = _attn_dims(Q, K, V)
    dev = Q.device
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        _expect(t, name, t.numel(), Q.dtype, dev)
    d_model = _x_dim(X, B, L_q)
    _expect(X, "X", B * L_q * d_model, Q.dtype, dev)
    if gm != GATE_NONE:   # (without a gate the library rejects the call)
        _expect(W_g, "W_g", d_model * _gate_cols(gm, H_q, d_k), Q.dtype, dev)
    if out is None:
        out = torch.empty_like(Q)
    _expect(out, "out", Q.numel(), Q.dtype, dev)
    st = torch.empty(3 + n_bins, dtype=torch.int64, device=dev)
    need = workspace_bytes(B, L_q, L_k, d_model, H_q, H_kv, d_k, gate, False, dtype)
    workspace, ws_bytes = _workspace(workspace, need, dev)
    s = _stream(stream, dev)
    status = int(load().gated_sdpa_fwd_stats(
        _ptr(X), _ptr(Q), _ptr(K), _ptr(V), _ptr(W_g), _ptr(out), None, _ptr(st), int(n_bins), float(threshold),
        B, L_q, L_k, d_model, H_q, H_kv, d_k, gm, int(bool(causal)), dtype,
        _ptr(workspace), ws_bytes, ctypes.c_void_p(s.cuda_stream)))
    if status != OK:
        raise GsdpaError(status, "gated_sdpa_fwd_stats")
    h = st.cpu().tolist()
    count = h[0]
    return out, {"count": count, "sum_fixed": h[1], "mean": (h[1] / 2.0 ** 32 / count) if count else 0.0,
                 "below": h[2], "hist": h[3:]}


def layer_workspace_bytes(B, L, d_model, H_q, H_kv, d_k, gate="elementwise") -> int:
    n = load().gsdpa_layer_workspace_bytes(B, L, d_model, H_q, H_kv, d_k, GATE_CODES[gate])
    if n == ctypes.c_size_t(-1).value:
        raise GsdpaError(ERR_UNSUPPORTED, "gsdpa_layer_workspace_bytes")
    return int(n)


def gated_attention_layer(X, W_in, W_O, *, H_q, H_kv, d_k=128, gate="elementwise", causal=True, out=None,
                          workspace=None, stream=None):
    """The whole layer (gated_attention_layer): X [B, L, d_model] bf16, W_in
    [d_model, (H_q + 2 H_kv) d_k + G] (G = H_q d_k elementwise, H_q headwise,
    0 without a gate), W_O [H_q d_k, d_model]. Returns Y."""
    import torch
    if X.dim() != 3:
        raise ValueError("X must be [B, L, d_model]")
    B, L, d_model = X.shape
    dev = X.device
    gm = GATE_CODES[gate]
    G = 0 if gm == GATE_NONE else _gate_cols(gm, H_q, d_k)
    _expect(X, "X", X.numel(), torch.bfloat16, dev)
    _expect(W_in, "W_in", d_model * ((H_q + 2 * H_kv) * d_k + G), torch.bfloat16, dev)
    _expect(W_O, "W_O", H_q * d_k * d_model, torch.bfloat16, dev)
    if out is None:
        out = torch.empty_like(X)
    _expect(out, "out", X.numel(), torch.bfloat16, dev)
    need = layer_workspace_bytes(B, L, d_model, H_q, H_kv, d_k, gate)
    workspace, ws_bytes = _workspace(workspace, need, dev)
    s = _stream(stream, dev)
    st = int(load().gated_attention_layer(_ptr(X), _ptr(W_in), _ptr(W_O), _ptr(out), B, L, d_model, H_q, H_kv, d_k,
                                          GATE_CODES[gate], int(bool(causal)),
                                          _ptr(workspace), ws_bytes,
                                          ctypes.c_void_p(s.cuda_stream)))
    if st != OK:
        raise GsdpaError(st, "gated_attention_layer")
    return out


def bwd_workspace_bytes(B, L_q, L_k, d_model, H_q, H_kv, d_k, gate="elementwise") -> int:
    n = load().gsdpa_bwd_workspace_bytes(B, L_q, L_k, d_model, H_q, H_kv, d_k, GATE_CODES[gate])
    if n == ctypes.c_size_t(-1).value:
        raise GsdpaError(ERR_UNSUPPORTED, "gsdpa_bwd_workspace_bytes")
    return int(n)


def gated_sdpa_bwd(X, Q, K, V, W_g, O, dO, lse, *, gate="elementwise", causal=True, workspace=None, stream=None,
                   gate_saved=None):
    """Backward through the C ABI (bf16, d_k = 128): returns a dict with dQ, dK,
    dV and, with a gate, dX (the gate path's share) and dW_g. gate_saved (the
    elementwise gate's values from gated_sdpa_fwd_train_save_gate) calls
    gated_sdpa_bwd_saved_gate, which does not recompute them."""
    import torch
    gm = GATE_CODES[gate]
    B, L_q, L_k, H_q, H_kv, d_k = _attn_dims(Q, K, V)
    dev = Q.device
    bf = torch.bfloat16
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        _expect(t, name, t.numel(), bf, dev)
    _expect(O, "O", Q.numel(), bf, dev)
    _expect(dO, "dO", Q.numel(), bf, dev)
    _expect(lse, "lse", B * H_q * L_q, torch.float32, dev)
    d_model = 0
    if gm != GATE_NONE:
        d_model = _x_dim(X, B, L_q)
        _expect(X, "X", B * L_q * d_model, bf, dev)
        _expect(W_g, "W_g", d_model * _gate_cols(gm, H_q, d_k), bf, dev)
    out = {"dQ": torch.empty_like(Q), "dK": torch.empty_like(K), "dV": torch.empty_like(V)}
    if gm != GATE_NONE:
        out["dX"] = torch.empty_like(X)
        out["dW_g"] = torch.empty_like(W_g)
    need = bwd_workspace_bytes(B, L_q, L_k, d_model, H_q, H_kv, d_k, gate)
    workspace, ws_bytes = _workspace(workspace, need, dev)
    s = _stream(stream, dev)
    head = [_ptr(X) if gm != GATE_NONE else None, _ptr(Q), _ptr(K), _ptr(V), _ptr(W_g) if gm != GATE_NONE else None,
            _ptr(O), _ptr(dO), _ptr(lse)]
    rest = [_ptr(out.get("dX")), _ptr(out["dQ"]), _ptr(out["dK"]), _ptr(out["dV"]), _ptr(out.get("dW_g")), B, L_q,
            L_k, d_model, H_q, H_kv, d_k, gm, int(bool(causal)), BF16, _ptr(workspace),
            ws_bytes, ctypes.c_void_p(s.cuda_stream)]
    if gate_saved is not None:
        _expect(gate_saved, "gate_saved", B * L_q * H_q * d_k, torch.float16, dev)
        st, where = int(load().gated_sdpa_bwd_saved_gate(*head, _ptr(gate_saved), *rest)), "gated_sdpa_bwd_saved_gate"
    else:
        st, where = int(load().gated_sdpa_bwd(*head, *rest)), "gated_sdpa_bwd"
    if st != OK:
        raise GsdpaError(st, where)
    return out


def decode_noalloc(X, Q, K, V, W_g=None, *, gate="elementwise", out=None, sink=None, want_sink=False, stream=None):
    """The decode call (L_q == 1, bf16) without a workspace: the library's fixed
    scratch array is used instead (for callers that cannot allocate device
    memory). Same tensors as gated_sdpa_fwd with L_q == 1."""
    import torch
    gm = GATE_CODES[gate]
    B, L_q, L_k, H_q, H_kv, d_k = _attn_dims(Q, K, V)
    if L_q != 1:
        raise ValueError("decode_noalloc takes one query row per sequence")
    dev = Q.device
    bf = torch.bfloat16
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        _expect(t, name, t.numel(), bf, dev)
    d_model = 0
    if gm != GATE_NONE:
        d_model = _x_dim(X, B, L_q)
        _expect(X, "X", B * d_model, bf, dev)
        _expect(W_g, "W_g", d_model * _gate_cols(gm, H_q, d_k), bf, dev)
    if out is None:
        out = torch.empty_like(Q)
    _expect(out, "out", Q.numel(), bf, dev)
    if sink is None and want_sink:
        sink = torch.empty((B, H_q), dtype=torch.float32, device=dev)
    if sink is not None:
        _expect(sink, "sink", B * H_q, torch.float32, dev)
    s = _stream(stream, dev)
    st = int(load().gated_sdpa_decode_noalloc(
        _ptr(X) if gm != GATE_NONE else None, _ptr(Q), _ptr(K), _ptr(V), _ptr(W_g) if gm != GATE_NONE else None,
        _ptr(out), _ptr(sink), B, L_k, d_model, H_q, H_kv, d_k, gm, ctypes.c_void_p(s.cuda_stream)))
    if st != OK:
        raise GsdpaError(st, "gated_sdpa_decode_noalloc")
    return out, sink


# ---- per-head norm and rotary positions (gsdpa_qk_norm_rope), and the 8-bit K/V cache (gsdpa_cache8)
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}


class _RopePlan(ctypes.Structure):
    _fields_ = [("rotary_dim", _I), ("layout", _I), ("attn_scale", _F), ("reserved", _I),
                ("turn", ctypes.c_ulonglong * 64)]


class Rope:
    """The plan of the rotary positions (gsdpa_rope), made once on the host.

    rotary_dim: columns of each head that are rotated, a multiple of 16; layout
    "half" (pairs i, i + rotary_dim / 2) or "interleaved" (2i, 2i + 1). Frequencies
    theta^(-2i / rotary_dim) under ``scaling``: "none", "linear" (divided by
    factor), "base" (theta enlarged) or "parts" (slow pairs divided by factor,
    those that turn more than beta_fast times in orig_len kept); or ``inv_freq``,
    rotary_dim / 2 of the caller's own. attn_scale multiplies cosine and sine
    (None: 1, or 0.1 ln(factor) + 1 with "parts")."""

    # (``ref``, the plan's address as the calls take it, belongs to one object: a copy's is its own)
    def __reduce__(self):
        return _rope_of, (bytes(self.plan),)

    def __init__(self, rotary_dim, *, layout="half", theta=10000.0, scaling="none", factor=1.0, orig_len=0,
                 beta_fast=32.0, beta_slow=1.0, attn_scale=None, inv_freq=None):
        self.plan = _RopePlan()
        self.ref = ctypes.addressof(self.plan)
        if attn_scale is not None and attn_scale == 0:
            raise ValueError("attn_scale must not be 0")
        if inv_freq is not None:
            w = [float(x) for x in inv_freq]
            if len(w) != rotary_dim // 2:
                raise ValueError(f"inv_freq has {len(w)} frequencies, rotary_dim = {rotary_dim} needs {rotary_dim // 2}")
            st = load().gsdpa_rope_init_freqs(self.ref, rotary_dim, ROPE_LAYOUTS[layout], (_D * len(w))(*w),
                                              1.0 if attn_scale is None else attn_scale)
            where = "gsdpa_rope_init_freqs"
        else:
            st = load().gsdpa_rope_init(self.ref, rotary_dim, ROPE_LAYOUTS[layout], theta, ROPE_SCALINGS[scaling],
                                        factor, orig_len, beta_fast, beta_slow, attn_scale or 0.0)
            where = "gsdpa_rope_init"
        if st != OK:
            raise GsdpaError(int(st), where)


def _rope_of(plan):
    """A Rope of the bytes of another's plan (copies, and pickles of this version of the library)."""
    if len(plan) != ctypes.sizeof(_RopePlan):
        raise ValueError(f"a Rope's plan has {ctypes.sizeof(_RopePlan)} bytes, not {len(plan)}")
    r = Rope.__new__(Rope)
    r.plan = _RopePlan.from_buffer_copy(plan)
    r.ref = ctypes.addressof(r.plan)
    return r


# (The calls below run once per layer and token in a decoding loop, on kernels of
# a few microseconds: their checks are the ones above, with each property of a
# tensor read once.)
def _head_rows(t, name, shape, dtype, device):
    """The row length in elements of t, shape [B, L, H, d] with contiguous heads and
    evenly spaced token rows (a contiguous tensor, or a column block of one)."""
    if t is not None and t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous():
        return shape[2] * shape[3]
    B, L, H, d = shape
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, the problem needs {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}, not on {t.device}")
    s0, s1, s2, s3 = t.stride()
    ld = s1 if L > 1 else (s0 if B > 1 else H * d)
    if (s3 != 1 and d > 1) or (H > 1 and s2 != d) or (L > 1 and B > 1 and s0 != L * ld):
        raise ValueError(f"{name}: heads must be contiguous and token rows evenly spaced (strides {tuple(t.stride())})")
    if ld < H * d and B * L > 1:
        raise ValueError(f"{name}: its token rows overlap (strides {tuple(t.stride())})")
    return ld


def _vector(t, name, n, dtype, device):
    """The address of an optional contiguous vector of n elements."""
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != n or t.device != device or not t.is_contiguous():
        _expect(t, name, n, dtype, device)   # says which
    return t.data_ptr()


def _current_stream(device):
    """The handle of the current stream, which must be of the tensors' device."""
    import torch
    index = device.index
    if index != torch._C._cuda_getDevice():
        _stream(None, device)                # raises
    return torch._C._cuda_getCurrentRawStream(index)


class _Kept(threading.local):
    def __init__(self):
        self.by_stream = {}     # workspaces, by (device index, stream handle)


_kept = _Kept()


def _kept_workspace(need, device, stream):
    """A workspace for a call on this stream. Each thread keeps one for each stream
    that it calls on: its calls there follow one another, while the kernels of two
    threads' calls may take turns. A captured call gets one of its own, which its
    graph keeps (replays may run beside anything). release_workspaces() lets the
    thread's go, as the thread's end does."""
    import torch
    if need == 0:
        return None
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(need, dtype=torch.uint8, device=device)
    key = (device.index, stream)
    held = _kept.by_stream.get(key)
    if held is None or held.numel() < need:
        held = _kept.by_stream[key] = torch.empty(need, dtype=torch.uint8, device=device)
    return held


def release_workspaces() -> None:
    """Lets go of the workspaces that qk_norm_rope_bwd and gated_sdpa_cache8 keep for
    this thread, one for each stream it has called them on, of the largest size
    they needed there. The memory goes back to torch's allocator; calls that are
    still running are not disturbed, and the next ones allocate anew."""
    _kept.by_stream.clear()


def _on_stream(call):
    """``stream=``: the call with that stream current, so that what it allocates
    (outputs, workspace) is that stream's own and not reused under its kernels."""
    @functools.wraps(call)
    def on(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        import torch
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return on


_DTYPES = {}


def _dtype_code(dt):
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.bfloat16: BF16, torch.float32: F32})
    if dt not in _DTYPES:
        raise TypeError(f"unsupported dtype {dt}")
    return _DTYPES[dt]


def _qk_shapes(Q, K):
    """The shapes of Q [B, L, H_q, d_k] and K [B, L, H_kv, d_k]."""
    q, k = Q.shape, K.shape
    if len(q) != 4 or len(k) != 4:
        raise ValueError("Q and K must be 4-D: [B, L, H, d_k]")
    if k[0] != q[0] or k[1] != q[1] or k[3] != q[3]:
        raise ValueError(f"K {tuple(k)} must be [B={q[0]}, L={q[1]}, H_kv, d_k={q[3]}]")
    if not Q.is_cuda:
        raise ValueError(f"Q must be a CUDA tensor, not on {Q.device}")
    return q, k


@_on_stream
def qk_norm_rope(Q, K, *, gamma_q=None, gamma_k=None, norm=True, eps=1e-6, rope=None, positions=None, out_q=None,
                 out_k=None):
    """Per-head RMS norm of Q [B, L, H_q, d_k] and K [B, L, H_kv, d_k] and their
    rotary positions in one pass (gsdpa_qk_norm_rope); float32 or bfloat16.

    Q and K (and out_q, out_k) may be column blocks of a packed projection's
    output, and out_q, out_k may be Q, K themselves. gamma_q, gamma_k [d_k] or
    None for 1; ``rope`` a Rope or None for no rotation; positions int32 [B, L] or
    None for 0 .. L - 1. ``stream``: else the current one. Returns (Q', K')."""
    import torch
    dt, dev = Q.dtype, Q.device
    code = _dtype_code(dt)
    q, k = _qk_shapes(Q, K)
    B, L, H_q, d_k = q
    ld_q, ld_k = _head_rows(Q, "Q", q, dt, dev), _head_rows(K, "K", k, dt, dev)
    if out_q is None:
        out_q, ld_qo = torch.empty(q, dtype=dt, device=dev), H_q * d_k
    else:
        ld_qo = _head_rows(out_q, "out_q", q, dt, dev)
    if out_k is None:
        out_k, ld_ko = torch.empty(k, dtype=dt, device=dev), k[2] * d_k
    else:
        ld_ko = _head_rows(out_k, "out_k", k, dt, dev)
    st = (_lib or load()).gsdpa_qk_norm_rope(
        Q.data_ptr(), K.data_ptr(), _vector(gamma_q, "gamma_q", d_k, dt, dev), _vector(gamma_k, "gamma_k", d_k, dt, dev),
        _vector(positions, "positions", B * L, torch.int32, dev), out_q.data_ptr(), out_k.data_ptr(), ld_q, ld_k, ld_qo,
        ld_ko, B, L, H_q, k[2], d_k, 1 if norm else 0, eps, None if rope is None else rope.ref, code,
        _current_stream(dev))
    if st != OK:
        raise GsdpaError(st, "gsdpa_qk_norm_rope")
    return out_q, out_k


@functools.lru_cache(maxsize=256)
def qk_norm_rope_bwd_workspace_bytes(B, L, d_k, norm=True) -> int:
    n = (_lib or load()).gsdpa_qk_norm_rope_bwd_workspace_bytes(B, L, d_k, 1 if norm else 0)
    if n == ctypes.c_size_t(-1).value:
        raise GsdpaError(ERR_INVALID_ARG, "gsdpa_qk_norm_rope_bwd_workspace_bytes")
    return n


@_on_stream
def qk_norm_rope_bwd(Q, K, dQo, dKo, *, gamma_q=None, gamma_k=None, norm=True, eps=1e-6, rope=None, positions=None,
                     out_dq=None, out_dk=None, workspace=None):
    """Backward of qk_norm_rope: from dQo, dKo (gradients of its outputs) and its
    inputs, a dict with dQ, dK and, with the norm, dgamma_q and dgamma_k (with
    respect to a gamma of 1 where none was given). out_dq, out_dk may be dQo, dKo
    or column blocks of the packed projection's gradient. ``stream``: else the
    current one."""
    import torch
    dt, dev = Q.dtype, Q.device
    code = _dtype_code(dt)
    q, k = _qk_shapes(Q, K)
    B, L, H_q, d_k = q
    ld_q, ld_k = _head_rows(Q, "Q", q, dt, dev), _head_rows(K, "K", k, dt, dev)
    ld_dqo, ld_dko = _head_rows(dQo, "dQo", q, dt, dev), _head_rows(dKo, "dKo", k, dt, dev)
    if out_dq is None:
        out_dq, ld_dq = torch.empty(q, dtype=dt, device=dev), H_q * d_k
    else:
        ld_dq = _head_rows(out_dq, "out_dq", q, dt, dev)
    if out_dk is None:
        out_dk, ld_dk = torch.empty(k, dtype=dt, device=dev), k[2] * d_k
    else:
        ld_dk = _head_rows(out_dk, "out_dk", k, dt, dev)
    gq, gk = _vector(gamma_q, "gamma_q", d_k, dt, dev), _vector(gamma_k, "gamma_k", d_k, dt, dev)
    pos = _vector(positions, "positions", B * L, torch.int32, dev)
    out = {"dQ": out_dq, "dK": out_dk}
    need, dgq, dgk = 0, None, None
    if norm:
        # (no rows: the library enqueues nothing, and the sums are zero)
        make = torch.empty if B * L > 0 else torch.zeros
        out["dgamma_q"], out["dgamma_k"] = make(d_k, dtype=dt, device=dev), make(d_k, dtype=dt, device=dev)
        dgq, dgk = out["dgamma_q"].data_ptr(), out["dgamma_k"].data_ptr()
        need = qk_norm_rope_bwd_workspace_bytes(B, L, d_k)
    stream = _current_stream(dev)
    if workspace is not None:
        workspace, need = _workspace(workspace, need, dev)
    else:
        workspace = _kept_workspace(need, dev, stream)
    st = (_lib or load()).gsdpa_qk_norm_rope_bwd(
        Q.data_ptr(), K.data_ptr(), gq, gk, pos, dQo.data_ptr(), dKo.data_ptr(), out_dq.data_ptr(), out_dk.data_ptr(),
        dgq, dgk, ld_q, ld_k, ld_dqo, ld_dko, ld_dq, ld_dk, B, L, H_q, k[2], d_k, 1 if norm else 0, eps,
        None if rope is None else rope.ref, code, None if workspace is None else workspace.data_ptr(), need, stream)
    if st != OK:
        raise GsdpaError(st, "gsdpa_qk_norm_rope_bwd")
    return out


CACHE_BLOCK = 64   # tokens that share a scale
CACHE_KINDS = {"int8": 0, "e4m3": 1}


class _Cache8Plan(ctypes.Structure):
    _fields_ = [("kind", _I), ("B", _I), ("H_kv", _I), ("d_k", _I), ("capacity", _I), ("k8", _VP), ("v8", _VP),
                ("k_scale", _VP), ("v_scale", _VP), ("k_tail", _VP), ("v_tail", _VP)]


class Cache8:
    """A K/V cache held in 8 bits (gsdpa_cache8) over the caller's tensors:

    k8 [B, H_kv, n, 64, d_k] and v8 [B, H_kv, n, d_k, 64], int8 or float8_e4m3fn;
    k_scale, v_scale float32 [B, H_kv, n]; k_tail [B, H_kv, 2, 64, d_k] and v_tail
    [B, H_kv, 2, d_k, 64] bfloat16 (the tokens of a block that is not full yet).
    The capacity is 64 n tokens per sequence. Lengths are the caller's."""

    def __init__(self, k8, v8, k_scale, v_scale, k_tail, v_tail):
        import torch
        kinds = {torch.int8: 0, torch.float8_e4m3fn: 1}
        if k8.dtype not in kinds:
            raise TypeError(f"k8 must be int8 or float8_e4m3fn, not {k8.dtype}")
        if k8.dim() != 5 or k8.shape[3] != CACHE_BLOCK:
            raise ValueError(f"k8 {tuple(k8.shape)} must be [B, H_kv, n, {CACHE_BLOCK}, d_k]")
        B, H, n, _, d = k8.shape
        want = {"k8": (k8, (B, H, n, CACHE_BLOCK, d), k8.dtype), "v8": (v8, (B, H, n, d, CACHE_BLOCK), k8.dtype),
                "k_scale": (k_scale, (B, H, n), torch.float32), "v_scale": (v_scale, (B, H, n), torch.float32),
                "k_tail": (k_tail, (B, H, 2, CACHE_BLOCK, d), torch.bfloat16),
                "v_tail": (v_tail, (B, H, 2, d, CACHE_BLOCK), torch.bfloat16)}
        for name, (t, shape, dtype) in want.items():
            if t is not None and tuple(t.shape) != shape:
                raise ValueError(f"{name} has shape {tuple(t.shape)}, the cache needs {shape}")
            numel = 1
            for v in shape:
                numel *= v
            _expect(t, name, numel, dtype, k8.device)
        self.k8, self.v8, self.k_scale, self.v_scale, self.k_tail, self.v_tail = k8, v8, k_scale, v_scale, k_tail, v_tail
        self.B, self.H_kv, self.d_k, self.capacity, self.device = B, H, d, n * CACHE_BLOCK, k8.device
        self.plan = _Cache8Plan(kinds[k8.dtype], B, H, d, n * CACHE_BLOCK, k8.data_ptr(), v8.data_ptr(),
                                k_scale.data_ptr(), v_scale.data_ptr(), k_tail.data_ptr(), v_tail.data_ptr())
        self.ref = ctypes.addressof(self.plan)
        self.need = {}   # workspace bytes, by the problem's shape

    # A copy is a cache over its own tensors: the plan's addresses are made anew.
    def __reduce__(self):
        return Cache8, (self.k8, self.v8, self.k_scale, self.v_scale, self.k_tail, self.v_tail)


def cache8_alloc(B, capacity, H_kv, d_k, kind="int8", device="cuda") -> Cache8:
    """An empty Cache8 of ``capacity`` tokens (rounded up to a multiple of 64) per sequence."""
    import torch
    n = (capacity + CACHE_BLOCK - 1) // CACHE_BLOCK
    dt = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[kind]

    def make(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device=device)
    return Cache8(make(B, H_kv, n, CACHE_BLOCK, d_k, dtype=dt), make(B, H_kv, n, d_k, CACHE_BLOCK, dtype=dt),
                  make(B, H_kv, n, dtype=torch.float32), make(B, H_kv, n, dtype=torch.float32),
                  make(B, H_kv, 2, CACHE_BLOCK, d_k, dtype=torch.bfloat16),
                  make(B, H_kv, 2, d_k, CACHE_BLOCK, dtype=torch.bfloat16))


@_on_stream
def cache8_append(cache, K, V, lens, n_new=None) -> None:
    """Appends K, V [B, L, H_kv, d_k] bfloat16 to the cache (gsdpa_cache8_append):
    row i < n_new[b] becomes token lens[b] + i of sequence b. lens and n_new (None:
    L each) are int32 [B] on the device and are not changed. ``stream``: else the
    current one."""
    import torch
    dev, bf = cache.device, torch.bfloat16
    if K.dim() != 4:
        raise ValueError("K must be [B, L, H_kv, d_k]")
    B, L = cache.B, K.shape[1]
    shape = (B, L, cache.H_kv, cache.d_k)
    ld_k, ld_v = _head_rows(K, "K", shape, bf, dev), _head_rows(V, "V", shape, bf, dev)
    if lens is None:
        raise ValueError("lens is required")
    st = (_lib or load()).gsdpa_cache8_append(
        cache.ref, K.data_ptr(), V.data_ptr(), ld_k, ld_v, _vector(lens, "lens", B, torch.int32, dev),
        _vector(n_new, "n_new", B, torch.int32, dev), L, _current_stream(dev))
    if st != OK:
        raise GsdpaError(st, "gsdpa_cache8_append")


def cache8_workspace_bytes(cache, L_q, H_q, d_model=0, gate="elementwise") -> int:
    n = load().gsdpa_cache8_workspace_bytes(cache.ref, L_q, d_model, H_q, GATE_CODES[gate])
    if n == ctypes.c_size_t(-1).value:
        raise GsdpaError(ERR_UNSUPPORTED, "gsdpa_cache8_workspace_bytes")
    return n


@_on_stream
def gated_sdpa_cache8(X, Q, cache, lens, W_g=None, *, gate="elementwise", n_new=None, out=None, workspace=None):
    """Gated attention of a step's tokens against the 8-bit cache (gated_sdpa_cache8),
    after cache8_append of their keys and values with the same lens and n_new: row i
    of Q [B, L_q, H_q, d_k] sees tokens 0 .. lens[b] + i. X [B, L_q, d_model] and W_g
    as for gated_sdpa_fwd (None for gate="none"). Rows i >= n_new[b] of the result
    are zero. ``stream``: else the current one. Returns O, like Q."""
    import torch
    dev, bf = cache.device, torch.bfloat16
    gm = GATE_CODES[gate]
    if Q.dim() != 4 or Q.shape[0] != cache.B or Q.shape[3] != cache.d_k:
        raise ValueError(f"Q {tuple(Q.shape)} must be [B={cache.B}, L_q, H_q, d_k={cache.d_k}]")
    B, L_q, H_q, d_k = Q.shape
    n = B * L_q * H_q * d_k
    q = _vector(Q, "Q", n, bf, dev)
    d_model, x, w = 0, None, None
    if gm != GATE_NONE:
        d_model = _x_dim(X, B, L_q)
        if W_g is None:
            raise ValueError("W_g is required")
        x = _vector(X, "X", B * L_q * d_model, bf, dev)
        w = _vector(W_g, "W_g", d_model * _gate_cols(gm, H_q, d_k), bf, dev)
    if lens is None:
        raise ValueError("lens is required")
    at = _vector(lens, "lens", B, torch.int32, dev)
    new = _vector(n_new, "n_new", B, torch.int32, dev)
    if out is None:
        out = torch.empty((B, L_q, H_q, d_k), dtype=bf, device=dev)
    o = _vector(out, "out", n, bf, dev)
    lib = _lib or load()
    shape = (L_q, d_model, H_q, gm)
    need = cache.need.get(shape)     # (the workspace's size, by the problem's shape)
    if need is None:
        need = lib.gsdpa_cache8_workspace_bytes(cache.ref, L_q, d_model, H_q, gm)
        if need == ctypes.c_size_t(-1).value:
            need = 0                 # (the call itself says why)
        cache.need[shape] = need
    stream = _current_stream(dev)
    if workspace is not None:
        workspace, need = _workspace(workspace, need, dev)
    else:
        workspace = _kept_workspace(need, dev, stream)
    st = lib.gated_sdpa_cache8(x, q, cache.ref, at, new, w, o, L_q, d_model, H_q, gm,
                               None if workspace is None else workspace.data_ptr(), need, stream)
    if st != OK:
        raise GsdpaError(st, "gated_sdpa_cache8")
    return out
