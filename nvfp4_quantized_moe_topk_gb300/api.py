"""Thin ctypes binding of libmoe_nvfp4 (see include/moe_nvfp4.h for the contract).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are torch tensors (device memory and streams come from
PyTorch); their ``data_ptr()`` and the current CUDA stream are passed through.
The library is loaded on first use and a missing build raises immediately --
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

MOE_OK = 0
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_CAPACITY",
          4: "MOE_ERR_CUDA", 5: "MOE_ERR_BAD_ROUTING", 6: "MOE_ERR_TIMEOUT", 7: "MOE_ERR_NO_DEVICE"}
DEVFLAG_BAD_ROUTING = 0x1
DEVFLAG_TIMEOUT = 0x2

# every entry point declared in include/moe_nvfp4.h
ENTRY_POINTS = ("moe_nvfp4_status_string", "moe_nvfp4_create", "moe_nvfp4_destroy", "moe_nvfp4_forward",
                "moe_nvfp4_forward_host", "moe_nvfp4_get_device_error", "moe_nvfp4_debug_routing",
                "moe_nvfp4_debug_intermediates", "moe_nvfp4_set_timing", "moe_nvfp4_kernel_times",
                "nvfp4_matmul", "weighted_row_sum", "moe_nvfp4_forward_noalloc", "moe_router_topk",
                "moe_nvfp4_shared_expert_forward", "moe_nvfp4_debug_offset_grid_barrier", "moe_block_norm",
                "moe_block_norm_backward", "moe_block_norm_workspace_bytes", "moe_balance_loss", "moe_router_backward",
                "moe_router_workspace_bytes", "moe_lora_apply", "moe_lora_workspace_bytes",
                "moe_lora_get_device_error")

_lock = threading.Lock()
_lib = None


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, why: str = ""):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({why or status_string(status)})")


class Config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("gemv_max_rows", ctypes.c_int32),
                ("single_max_tokens", ctypes.c_int32), ("activation", ctypes.c_int32)]


ACT_RELU2, ACT_SWIGLU = 0, 1


class Weights(ctypes.Structure):
    _fields_ = [("up_codes", ctypes.c_void_p), ("up_scales", ctypes.c_void_p), ("down_codes", ctypes.c_void_p),
                ("down_scales", ctypes.c_void_p), ("up_global", ctypes.c_void_p), ("down_global", ctypes.c_void_p),
                ("gate_codes", ctypes.c_void_p), ("gate_scales", ctypes.c_void_p), ("gate_global", ctypes.c_void_p)]


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False):
    """Load libmoe_nvfp4.so; raise if it is not built (no fallback)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if build_if_missing and not os.path.exists(path):
            _build.build()
        if not os.path.exists(path):
            raise RuntimeError(f"libmoe_nvfp4 is not built ({path}); run __graft_entry__.build() or "
                               "python -m nvfp4_quantized_moe_topk_gb300.build")
        L = ctypes.CDLL(path)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.moe_nvfp4_status_string.argtypes = [ctypes.c_int]
        L.moe_nvfp4_status_string.restype = ctypes.c_char_p
        L.moe_nvfp4_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), vp, ctypes.POINTER(vp)]
        L.moe_nvfp4_destroy.argtypes = [vp]
        L.moe_nvfp4_forward.argtypes = [vp, vp, vp, vp, vp, i32, vp]
        L.moe_nvfp4_forward_host.argtypes = [vp, vp, vp, vp, vp, i32, vp]
        L.moe_nvfp4_shared_expert_forward.argtypes = [vp, vp, vp, i32, vp]
        L.moe_nvfp4_debug_offset_grid_barrier.argtypes = [vp, ctypes.c_int64]
        L.moe_nvfp4_get_device_error.argtypes = [vp, ctypes.POINTER(i32)]
        L.moe_nvfp4_debug_routing.argtypes = [vp, vp, vp, vp, vp, vp]
        L.moe_nvfp4_debug_intermediates.argtypes = [vp, vp, vp, vp]
        L.moe_nvfp4_set_timing.argtypes = [vp, i32]
        L.moe_nvfp4_kernel_times.argtypes = [vp, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_double),
                                             ctypes.POINTER(i64), i32, ctypes.POINTER(i32)]
        L.nvfp4_matmul.argtypes = [vp, vp, vp, ctypes.c_float, vp, i32, i32, i32, i32, vp]
        L.weighted_row_sum.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp]
        L.moe_router_topk.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp]
        L.moe_nvfp4_forward_noalloc.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), vp, vp, vp, vp,
                                                i32, vp]
        sz = ctypes.c_size_t
        L.moe_block_norm.argtypes = [vp, vp]
        L.moe_block_norm_backward.argtypes = [vp, vp, vp, sz, vp]
        L.moe_block_norm_workspace_bytes.argtypes = [i32, i32]
        L.moe_balance_loss.argtypes = [vp, vp, vp, vp, sz, vp]
        L.moe_router_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_router_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_lora_apply.argtypes = [vp, vp, sz, vp]
        L.moe_lora_workspace_bytes.argtypes = [i32, i32]
        L.moe_lora_get_device_error.argtypes = [ctypes.POINTER(i32)]
        for name in ENTRY_POINTS:
            if name.endswith("_workspace_bytes"):
                getattr(L, name).restype = sz
            elif name != "moe_nvfp4_status_string":
                getattr(L, name).restype = ctypes.c_int
        _lib = L
        return L


def status_string(status: int) -> str:
    try:
        return load().moe_nvfp4_status_string(status).decode()
    except Exception:  # pragma: no cover - only when the library itself is missing
        return STATUS.get(status, "unknown")


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream):
    import torch

    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


class MoeLayer:
    """A created layer (``moe_nvfp4_create``); weights are copied into the handle.

    Passing gate weights (``gate_codes``, ``gate_scales``, ``gate_global``)
    makes the experts gated: a = bf16(silu(gate) * up) instead of relu^2."""

    def __init__(self, hidden, inter, n_experts, top_k, max_tokens, up_codes, up_scales, down_codes, down_scales,
                 up_global, down_global, gemv_max_rows: int = 0, single_max_tokens: int = 0, stream=None,
                 gate_codes=None, gate_scales=None, gate_global=None):
        L = load()
        self.hidden, self.inter, self.n_experts, self.top_k = hidden, inter, n_experts, top_k
        self.max_tokens = max_tokens
        self.gated = gate_codes is not None
        cfg = Config(hidden, inter, n_experts, top_k, max_tokens, gemv_max_rows, single_max_tokens,
                     ACT_SWIGLU if self.gated else ACT_RELU2)
        w = Weights(_ptr(up_codes), _ptr(up_scales), _ptr(down_codes), _ptr(down_scales), _ptr(up_global),
                    _ptr(down_global), _ptr(gate_codes), _ptr(gate_scales), _ptr(gate_global))
        h = ctypes.c_void_p()
        _check(L.moe_nvfp4_create(ctypes.byref(cfg), ctypes.byref(w), _stream(stream), ctypes.byref(h)),
               "moe_nvfp4_create")
        self._h = h

    @property
    def handle(self):
        return self._h

    def forward(self, x, topk_ids, topk_weights, dst, n_tokens: int | None = None, stream=None):
        n = x.shape[0] if n_tokens is None else n_tokens
        _check(load().moe_nvfp4_forward(self._h, _ptr(x), _ptr(topk_ids), _ptr(topk_weights), _ptr(dst), n,
                                        _stream(stream)), "moe_nvfp4_forward")
        return dst

    def debug_offset_grid_barrier(self, arrivals: int):
        """Test hook: offset the streaming kernel's barrier count (the next
        single-launch forward then times out, bounded; see the C header)."""
        _check(load().moe_nvfp4_debug_offset_grid_barrier(self._h, int(arrivals)),
               "moe_nvfp4_debug_offset_grid_barrier")

    def shared_expert_forward(self, x, dst, n_tokens: int | None = None, stream=None):
        """dst = bf16(expert 0's FFN of x) for a 1-expert top-1 layer (the shared expert)."""
        n = x.shape[0] if n_tokens is None else n_tokens
        _check(load().moe_nvfp4_shared_expert_forward(self._h, _ptr(x), _ptr(dst), n, _stream(stream)),
               "moe_nvfp4_shared_expert_forward")
        return dst

    def forward_host(self, x, topk_ids, topk_weights, dst, n_tokens: int | None = None, stream=None):
        n = x.shape[0] if n_tokens is None else n_tokens
        _check(load().moe_nvfp4_forward_host(self._h, _ptr(x), _ptr(topk_ids), _ptr(topk_weights), _ptr(dst), n,
                                             _stream(stream)), "moe_nvfp4_forward_host")
        return dst

    def device_error(self) -> int:
        f = ctypes.c_int32()
        _check(load().moe_nvfp4_get_device_error(self._h, ctypes.byref(f)), "moe_nvfp4_get_device_error")
        return f.value

    def debug_routing(self, counts=None, offsets=None, perm_pair=None, inv=None, stream=None):
        _check(load().moe_nvfp4_debug_routing(self._h, _ptr(counts), _ptr(offsets), _ptr(perm_pair), _ptr(inv),
                                              _stream(stream)), "moe_nvfp4_debug_routing")

    def debug_intermediates(self, a_rows=None, y_rows=None, stream=None):
        _check(load().moe_nvfp4_debug_intermediates(self._h, _ptr(a_rows), _ptr(y_rows), _stream(stream)),
               "moe_nvfp4_debug_intermediates")

    def set_timing(self, enable: bool):
        _check(load().moe_nvfp4_set_timing(self._h, 1 if enable else 0), "moe_nvfp4_set_timing")

    def kernel_times(self) -> dict:
        cap = 16
        names = (ctypes.c_char_p * cap)()
        ms = (ctypes.c_double * cap)()
        launches = (ctypes.c_int64 * cap)()
        count = ctypes.c_int32()
        _check(load().moe_nvfp4_kernel_times(self._h, names, ms, launches, cap, ctypes.byref(count)),
               "moe_nvfp4_kernel_times")
        return {names[i].decode(): (ms[i], launches[i]) for i in range(min(count.value, cap))}

    def close(self):
        if getattr(self, "_h", None):
            load().moe_nvfp4_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def nvfp4_matmul(A, codes, scales, global_scale: float, C, epilogue: int, stream=None):
    M, K = A.shape
    N = codes.shape[0]
    _check(load().nvfp4_matmul(_ptr(A), _ptr(codes), _ptr(scales), float(global_scale), _ptr(C), M, N, K,
                               epilogue, _stream(stream)), "nvfp4_matmul")
    return C


def router_topk(logits, bias, topk_ids, topk_weights, counts=None, stream=None):
    """moe_router_topk: fills topk_ids [n,k] / topk_weights [n,k] (and counts [E]) from logits [n,E]."""
    n, E = logits.shape
    k = topk_ids.shape[1]
    _check(load().moe_router_topk(_ptr(logits), _ptr(bias), n, E, k, _ptr(topk_ids), _ptr(topk_weights),
                                  _ptr(counts), _stream(stream)), "moe_router_topk")
    return topk_ids, topk_weights


def weighted_row_sum(dst, src, rows, w, stream=None):
    n, cols = dst.shape
    k = rows.shape[1]
    _check(load().weighted_row_sum(_ptr(dst), _ptr(src), _ptr(rows), _ptr(w), n, k, cols, src.shape[0],
                                   _stream(stream)), "weighted_row_sum")
    return dst


def forward_noalloc(hidden, inter, n_experts, top_k, up_codes, up_scales, down_codes, down_scales, up_global,
                    down_global, x, topk_ids, topk_weights, dst, n_tokens: int | None = None, stream=None,
                    gate_codes=None, gate_scales=None, gate_global=None):
    """``moe_nvfp4_forward_noalloc``: the layer without a handle and without any
    device allocation (weights read in place; intermediates in the library's
    fixed device array).  Gate weights make the experts gated."""
    n = x.shape[0] if n_tokens is None else n_tokens
    cfg = Config(hidden, inter, n_experts, top_k, n, 0, 0, ACT_SWIGLU if gate_codes is not None else ACT_RELU2)
    w = Weights(_ptr(up_codes), _ptr(up_scales), _ptr(down_codes), _ptr(down_scales), _ptr(up_global),
                _ptr(down_global), _ptr(gate_codes), _ptr(gate_scales), _ptr(gate_global))
    _check(load().moe_nvfp4_forward_noalloc(ctypes.byref(cfg), ctypes.byref(w), _ptr(x), _ptr(topk_ids),
                                            _ptr(topk_weights), _ptr(dst), n, _stream(stream)),
           "moe_nvfp4_forward_noalloc")
    return dst


# ---------------------------------------------------------------- operators around the layer
# Checked and called by the native module moe_binding (csrc/binding.cpp): the
# smallest of these calls take a few microseconds.  Every refusal is a MoeError,
# raised before anything is enqueued.
_native = None


def _binding():
    """The native module; raises if it is not built (no fallback)."""
    global _native
    if _native is None:
        import importlib.machinery
        import importlib.util

        import torch  # noqa: F401  (its libraries have to be loaded first)

        load()
        if not os.path.exists(_build.BINDING):
            raise RuntimeError(f"the binding is not built ({_build.BINDING}); run __graft_entry__.build() or "
                               "python -m nvfp4_quantized_moe_topk_gb300.build")
        loader = importlib.machinery.ExtensionFileLoader("moe_binding", _build.BINDING)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("moe_binding", loader))
        loader.exec_module(module)
        module.set_error(MoeError)
        _native = module
    return _native


def _on_gpu(t, dims: int) -> bool:
    """Whether t is a CUDA tensor of so many dimensions, for which a workspace can be made (else the call refuses it)."""
    import torch

    return isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == dims


def _new_workspace(size: int, like=None, stream=None):
    """size bytes on the current device; for a call on another stream than the current one, allocated on that."""
    import torch

    device = "cuda" if like is None else like.device
    if stream is None:
        return torch.empty(max(16, size), dtype=torch.uint8, device=device)
    s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        return torch.empty(max(16, size), dtype=torch.uint8, device=device)


def block_norm(residual, branch=None, gate=None, post_weight=None, pre_weight=None, residual_out=None, x_out=None,
               rstd_post=None, rstd_pre=None, *, eps: float = 1e-6, residual_scale: float = 1.0,
               branch_scale: float = 1.0, weight_offset: float = 0.0, gate_sigmoid: bool = False, stream=None):
    """``moe_block_norm``: the norms before and after a block with its gate and residual, in one call.

    residual_out = residual_scale * residual + branch_scale * gate * norm(branch, post_weight) and
    x_out = norm(residual_out, pre_weight).  Tensors are [n, hidden]; the gate is [hidden], [n, 1] (fp32) or
    [n, hidden]; without ``branch`` it is the norm before a block, without ``pre_weight`` the norm after one.
    ``rstd_post`` and ``rstd_pre`` [n] receive the row statistics that the backward pass needs."""
    (_native or _binding()).block_norm(residual, branch, gate, post_weight, pre_weight, residual_out, x_out, rstd_post,
                                       rstd_pre, eps, residual_scale, branch_scale, weight_offset, gate_sigmoid, stream)
    return residual_out, x_out


def block_norm_workspace(n: int, hidden: int):
    """A workspace for block_norm_backward of up to n tokens."""
    return _new_workspace(load().moe_block_norm_workspace_bytes(n, hidden))


def block_norm_backward(d_residual_out, d_x, residual_out, branch=None, gate=None, post_weight=None, pre_weight=None,
                        rstd_post=None, rstd_pre=None, d_residual=None, d_branch=None, d_gate=None,
                        d_post_weight=None, d_pre_weight=None, *, eps: float = 1e-6, residual_scale: float = 1.0,
                        branch_scale: float = 1.0, weight_offset: float = 0.0, gate_sigmoid: bool = False,
                        workspace=None, stream=None):
    """``moe_block_norm_backward``: fills the given gradients from those of residual_out and x_out (either may be
    None: zero).  residual_out, rstd_post and rstd_pre are what block_norm left."""
    native = _native or _binding()
    if workspace is None:
        lead = next((t for t in (d_residual_out, residual_out, branch) if _on_gpu(t, 2)), None)
        if lead is not None:
            workspace = _new_workspace(_lib.moe_block_norm_workspace_bytes(*lead.shape), lead, stream)
    native.block_norm_backward(d_residual_out, d_x, residual_out, branch, gate, post_weight, pre_weight, rstd_post,
                               rstd_pre, d_residual, d_branch, d_gate, d_post_weight, d_pre_weight, eps,
                               residual_scale, branch_scale, weight_offset, gate_sigmoid, workspace, stream)
    return d_residual, d_branch


def router_workspace(n: int, n_experts: int, n_seqs: int = 1):
    """A workspace for balance_loss and router_backward of up to n tokens in n_seqs sequences."""
    return _new_workspace(load().moe_router_workspace_bytes(n, n_experts, n_seqs))


def _router_workspace_for(logits, seq_offsets, stream):
    if not _on_gpu(logits, 2) or not (seq_offsets is None or _on_gpu(seq_offsets, 1)):
        return None  # refused by the call
    seqs = 1 if seq_offsets is None else max(1, seq_offsets.numel() - 1)
    return _new_workspace(load().moe_router_workspace_bytes(*logits.shape, seqs), logits, stream)


def balance_loss(logits, bias, topk_ids, loss, counts, prob_sums, tokens, *, coef: float, mask=None,
                 seq_offsets=None, workspace=None, stream=None):
    """``moe_balance_loss``: fills loss [1], counts [S, E] int32, prob_sums [S, E] and tokens [S + 1] int32 (each
    sequence's tokens, then all) from logits [n, E] (+ bias [E]) and topk_ids [n, k].  ``mask`` [n] (bool or uint8)
    leaves tokens out; ``seq_offsets`` [S + 1] int32 cuts the batch into sequences (None: one)."""
    native = _native or _binding()
    if workspace is None:
        workspace = _router_workspace_for(logits, seq_offsets, stream)
    native.balance_loss(logits, bias, topk_ids, loss, counts, prob_sums, tokens, coef, mask, seq_offsets, workspace,
                        stream)
    return loss


def router_backward(logits, bias, topk_ids, topk_weights, d_weights, counts, tokens, d_logits, d_bias=None, *,
                    d_loss=None, coef: float, mask=None, seq_offsets=None, workspace=None, stream=None):
    """``moe_router_backward``: d_logits [n, E] (and d_bias [E]) of d_loss [1] times the balance loss (counts and
    tokens as balance_loss left them; None: no loss) and of the top-k weights (d_weights [n, k]; None: none)."""
    native = _native or _binding()
    if workspace is None:
        workspace = _router_workspace_for(logits, seq_offsets, stream)
    native.router_backward(logits, bias, topk_ids, topk_weights, d_weights, counts, tokens, d_logits, d_bias, d_loss,
                           coef, mask, seq_offsets, workspace, stream)
    return d_logits


def lora_workspace(n: int, n_adapters: int):
    """A workspace for lora_apply of up to n tokens over n_adapters adapters."""
    return _new_workspace(load().moe_lora_workspace_bytes(n, n_adapters))


def lora_apply(x, adapter_ids, a, b, y, out, *, scale=None, ranks=None, workspace=None, stream=None):
    """``moe_lora_apply``: out[t] = y[t] + scale[l] * B[l] (A[l] x[t]) with l = adapter_ids[t] (an id outside the
    bank, such as -1: out[t] = y[t]).  x [n, in] bf16, a [L, R, in] and b [L, out, R] bf16, y [n, out] (None: zero)
    and out [n, out] bf16 or fp32 (out may be y), scale [L] fp32, ranks [L] int32."""
    native = _native or _binding()
    if workspace is None and _on_gpu(x, 2) and _on_gpu(a, 3):
        workspace = _new_workspace(_lib.moe_lora_workspace_bytes(x.shape[0], a.shape[0]), x, stream)
    native.lora_apply(x, adapter_ids, a, b, y, out, scale, ranks, workspace, stream)
    return out


def lora_device_error() -> int:
    """Reads and clears lora_apply's device error flags (DEVFLAG_TIMEOUT); synchronizes the device."""
    f = ctypes.c_int32()
    _check(load().moe_lora_get_device_error(ctypes.byref(f)), "moe_lora_get_device_error")
    return f.value
