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
import struct
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
                "moe_router_workspace_bytes", "moe_lora_apply", "moe_lora_workspace_bytes")

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
# The argument structs of the C header, packed in one step (their layouts are
# checked against the header's by a test).
_NORM_ARGS = struct.Struct("@7i4f4xPqPqPqPPPqPqPP")
_NORM_GRADS = struct.Struct("@PqPqPqPqPqPP")
_ROUTER_ARGS = struct.Struct("@4if4xPPPPPPP")
_LORA_ARGS = struct.Struct("@7i4xPPPPPPqPqPq")
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3
MAX_HIDDEN, MAX_EXPERTS, MAX_TOP_K = 8192, 1024, 32


_torch = _BF16 = _F32 = _I32 = _U8 = _BOOL = _KINDS = _raw_stream = _current_device = None


def _ready():
    """The loaded library; on first use also binds what the calls below take from torch (a call checks and packs in a
    few microseconds, so it looks nothing up by name)."""
    global _torch, _BF16, _F32, _I32, _U8, _BOOL, _KINDS, _raw_stream, _current_device
    if _torch is None:
        import torch

        load()
        _BF16, _F32, _I32, _U8, _BOOL = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.bool
        _KINDS = (_BF16, _F32)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda device: torch.cuda.current_stream(device).cuda_stream)
        _current_device = torch.cuda.current_device
        _torch = torch
    return _lib


def _refuse(where: str, why: str):
    raise MoeError(1, where, why)


def _dtype_code(t, where, name):
    """MOE_DTYPE_ of a tensor that may be bf16 or fp32."""
    d = t.dtype
    if d is _F32:
        return 1
    if d is not _BF16:
        _refuse(where, f"{name} is {d}; bfloat16 or float32 is supported")
    return 0


def _is(t, where, name, dtype, device):
    if t.dtype is not dtype:
        _refuse(where, f"{name} is {t.dtype}, not {dtype}")
    if t.get_device() != device or device < 0:
        _refuse(where, f"{name} is not on the call's CUDA device")


def _rows(t, where, name, dtype, device, shape):
    """(address, row stride in elements, 0: contiguous) of a matrix; (0, 0) for None."""
    if t is None:
        return 0, 0
    if t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr(), 0
    _is(t, where, name, dtype, device)
    if t.shape != shape:
        _refuse(where, f"{name} is {tuple(t.shape)}, not {tuple(shape)}")
    n, cols = shape
    step, inner = t.stride()
    if (cols > 1 and inner != 1) or (n > 1 and step < cols):
        _refuse(where, f"{name} has strides {t.stride()}: rows must be contiguous and must not overlap")
    return t.data_ptr(), step if n > 1 else 0


def _array(t, where, name, dtype, device, shape):
    """Address of a contiguous array; 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _is(t, where, name, dtype, device)
    if t.shape != shape:
        _refuse(where, f"{name} is {tuple(t.shape)}, not {tuple(shape)}")
    _refuse(where, f"{name} is not contiguous")


def _on(device, where):
    """The call's device is the current one (its kernels are launched there)."""
    if device < 0 or device != _current_device():
        _refuse(where, "the tensors are not on the current CUDA device")


def _handle(stream, device):
    """cudaStream_t of a stream argument (None: the current stream) as an integer."""
    if stream is None:
        return _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _workspace(workspace, need, args, where, device, stream):
    """(tensor, address, bytes): the caller's, or need(*args) bytes allocated on the call's stream."""
    if workspace is None:
        size = max(16, need(*args))
        if stream is None:
            workspace = _torch.empty(size, dtype=_U8, device=f"cuda:{device}")
        else:
            s = _torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
            with _torch.cuda.stream(s):
                workspace = _torch.empty(size, dtype=_U8, device=f"cuda:{device}")
        return workspace, workspace.data_ptr(), size
    _is(workspace, where, "workspace", _U8, device)
    if not workspace.is_contiguous():
        _refuse(where, "workspace is not contiguous")
    return workspace, workspace.data_ptr(), workspace.numel()


def _new_workspace(size):
    return _torch.empty(max(16, size), dtype=_U8, device="cuda")


def _norm_gate(gate, shape, act, par, device, where, name="gate"):
    """(kind, address, stride) of a gate [hidden], [n, 1] or [n, hidden] of type par, fp32 or act."""
    if gate is None:
        return GATE_NONE, 0, 0
    n, hidden = shape
    if gate.dim() == 1:
        return GATE_CHANNEL, _array(gate, where, name, par, device, (hidden,)), 0
    if gate.shape == (n, 1):
        return GATE_TOKEN, _array(gate, where, name, _F32, device, (n, 1)), 0
    if gate.shape != shape:
        _refuse(where, f"{name} is {tuple(gate.shape)}; {(hidden,)}, {(n, 1)} or {(n, hidden)} is supported")
    p, step = _rows(gate, where, name, act, device, shape)
    return GATE_FULL, p, step


def _norm_pack(where, shape, device, res, branch, residual, gate, post_weight, pre_weight, residual_out, x_out,
               rstd_post, rstd_pre, eps, residual_scale, branch_scale, weight_offset, gate_sigmoid):
    """(kind of gate, type of branch, type of the parameters, packed struct)."""
    n, hidden = shape
    act = res if branch is None else _dtype_code(branch, where, "branch")
    lead = post_weight if post_weight is not None else pre_weight
    if lead is None and gate is not None and gate.dim() == 1:
        lead = gate
    par = 1 if lead is None else _dtype_code(lead, where, "the weights")
    act_t, par_t, res_t, vec = _KINDS[act], _KINDS[par], _KINDS[res], (hidden,)
    kind, gp, gs = _norm_gate(gate, shape, act_t, par_t, device, where)
    rp, rs = _rows(residual, where, "residual", res_t, device, shape)
    bp, bs = _rows(branch, where, "branch", act_t, device, shape)
    op, os_ = _rows(residual_out, where, "residual_out", res_t, device, shape)
    xp, xs = _rows(x_out, where, "x_out", _BF16, device, shape)
    return kind, act_t, _NORM_ARGS.pack(
        n, hidden, res, act, par, kind, 1 if gate_sigmoid and kind else 0, eps, residual_scale, branch_scale,
        weight_offset, rp, rs, bp, bs, gp, gs, _array(post_weight, where, "post_weight", par_t, device, vec),
        _array(pre_weight, where, "pre_weight", par_t, device, vec), op, os_, xp, xs,
        _array(rstd_post, where, "rstd_post", _F32, device, (n,)),
        _array(rstd_pre, where, "rstd_pre", _F32, device, (n,)))


def block_norm(residual, branch=None, gate=None, post_weight=None, pre_weight=None, residual_out=None, x_out=None,
               rstd_post=None, rstd_pre=None, *, eps: float = 1e-6, residual_scale: float = 1.0,
               branch_scale: float = 1.0, weight_offset: float = 0.0, gate_sigmoid: bool = False, stream=None):
    """``moe_block_norm``: the norms before and after a block with its gate and residual, in one call.

    residual_out = residual_scale * residual + branch_scale * gate * norm(branch, post_weight) and
    x_out = norm(residual_out, pre_weight).  Tensors are [n, hidden]; the gate is [hidden], [n, 1] (fp32) or
    [n, hidden]; without ``branch`` it is the norm before a block, without ``pre_weight`` the norm after one."""
    L = _lib if _torch is not None else _ready()
    where = "moe_block_norm"
    if residual is None or residual.dim() != 2:
        _refuse(where, "residual is not an [n, hidden] tensor")
    device = residual.get_device()
    _on(device, where)
    args = _norm_pack(where, residual.shape, device, _dtype_code(residual, where, "residual"), branch, residual, gate,
                      post_weight, pre_weight, residual_out, x_out, rstd_post, rstd_pre, eps, residual_scale,
                      branch_scale, weight_offset, gate_sigmoid)[2]
    status = L.moe_block_norm(args, _handle(stream, device))
    if status:
        raise MoeError(status, where)
    return residual_out, x_out


def block_norm_workspace(n: int, hidden: int):
    """A workspace for block_norm_backward of up to n tokens."""
    return _new_workspace(_ready().moe_block_norm_workspace_bytes(n, hidden))


def block_norm_backward(d_residual_out, d_x, residual_out, branch=None, gate=None, post_weight=None, pre_weight=None,
                        rstd_post=None, rstd_pre=None, d_residual=None, d_branch=None, d_gate=None,
                        d_post_weight=None, d_pre_weight=None, *, eps: float = 1e-6, residual_scale: float = 1.0,
                        branch_scale: float = 1.0, weight_offset: float = 0.0, gate_sigmoid: bool = False,
                        workspace=None, stream=None):
    """``moe_block_norm_backward``: fills the given gradients from those of residual_out and x_out (either may be
    None: zero).  residual_out, rstd_post and rstd_pre are what block_norm left."""
    L = _lib if _torch is not None else _ready()
    where = "moe_block_norm_backward"
    lead = d_residual_out if d_residual_out is not None else residual_out if residual_out is not None else branch
    if lead is None or lead.dim() != 2:
        _refuse(where, "no [n, hidden] gradient is given")
    shape, device = lead.shape, lead.get_device()
    _on(device, where)
    n, hidden = shape
    kind, act_t, args = _norm_pack(
        where, shape, device, _dtype_code(lead, where, "the residual"), branch, None, gate, post_weight, pre_weight,
        residual_out, None, rstd_post, rstd_pre, eps, residual_scale, branch_scale, weight_offset, gate_sigmoid)
    dk, dgp, dgs = _norm_gate(d_gate, shape, act_t, _F32, device, where, "d_gate")
    if dk and dk != kind:
        _refuse(where, f"d_gate is {tuple(d_gate.shape)}, the gate another shape")
    res_t = lead.dtype
    a, ast = _rows(d_residual_out, where, "d_residual_out", res_t, device, shape)
    b, bst = _rows(d_x, where, "d_x", _BF16, device, shape)
    c, cst = _rows(d_residual, where, "d_residual", res_t, device, shape)
    d, dst = _rows(d_branch, where, "d_branch", act_t, device, shape)
    grads = _NORM_GRADS.pack(a, ast, b, bst, c, cst, d, dst, dgp, dgs,
                             _array(d_post_weight, where, "d_post_weight", _F32, device, (hidden,)),
                             _array(d_pre_weight, where, "d_pre_weight", _F32, device, (hidden,)))
    keep, wp, wb = _workspace(workspace, L.moe_block_norm_workspace_bytes, (n, hidden), where, device, stream)
    status = L.moe_block_norm_backward(args, grads, wp, wb, _handle(stream, device))
    if status:
        raise MoeError(status, where)
    return d_residual, d_branch


def router_workspace(n: int, n_experts: int, n_seqs: int = 1):
    """A workspace for balance_loss and router_backward of up to n tokens in n_seqs sequences."""
    return _new_workspace(_ready().moe_router_workspace_bytes(n, n_experts, n_seqs))


def _router_pack(where, logits, bias, topk_ids, counts, tokens, coef, mask, seq_offsets):
    if logits is None or logits.dim() != 2 or topk_ids is None or topk_ids.dim() != 2:
        _refuse(where, "logits are not [n, n_experts] or topk_ids not [n, top_k]")
    shape, k, device = logits.shape, topk_ids.shape[1], logits.get_device()
    n, E = shape
    _on(device, where)
    S = 1
    if seq_offsets is not None:
        S = seq_offsets.shape[0] - 1 if seq_offsets.dim() == 1 else 0
        if S < 1:
            _refuse(where, "seq_offsets holds no sequence")
    args = _ROUTER_ARGS.pack(
        n, E, k, S, coef, _array(logits, where, "logits", _F32, device, shape),
        _array(bias, where, "bias", _F32, device, (E,)), _array(topk_ids, where, "topk_ids", _I32, device, (n, k)),
        0 if mask is None else _array(mask, where, "mask", _BOOL if mask.dtype is _BOOL else _U8, device, (n,)),
        _array(seq_offsets, where, "seq_offsets", _I32, device, (S + 1,)),
        _array(counts, where, "counts", _I32, device, (S, E)), _array(tokens, where, "tokens", _I32, device, (S + 1,)))
    return n, E, k, S, device, args


def balance_loss(logits, bias, topk_ids, loss, counts, prob_sums, tokens, *, coef: float, mask=None,
                 seq_offsets=None, workspace=None, stream=None):
    """``moe_balance_loss``: fills loss [1], counts [S, E] int32, prob_sums [S, E] and tokens [S + 1] int32 (each
    sequence's tokens, then all) from logits [n, E] (+ bias [E]) and topk_ids [n, k].  ``mask`` [n] (bool or uint8)
    leaves tokens out; ``seq_offsets`` [S + 1] int32 cuts the batch into sequences (None: one)."""
    L = _lib if _torch is not None else _ready()
    where = "moe_balance_loss"
    n, E, _, S, device, args = _router_pack(where, logits, bias, topk_ids, counts, tokens, coef, mask, seq_offsets)
    keep, wp, wb = _workspace(workspace, L.moe_router_workspace_bytes, (n, E, S), where, device, stream)
    status = L.moe_balance_loss(args, _array(prob_sums, where, "prob_sums", _F32, device, (S, E)),
                                _array(loss, where, "loss", _F32, device, (1,)), wp, wb, _handle(stream, device))
    if status:
        raise MoeError(status, where)
    return loss


def router_backward(logits, bias, topk_ids, topk_weights, d_weights, counts, tokens, d_logits, d_bias=None, *,
                    d_loss=None, coef: float, mask=None, seq_offsets=None, workspace=None, stream=None):
    """``moe_router_backward``: d_logits [n, E] (and d_bias [E]) of d_loss [1] times the balance loss (counts and
    tokens as balance_loss left them; None: no loss) and of the top-k weights (d_weights [n, k]; None: none)."""
    L = _lib if _torch is not None else _ready()
    where = "moe_router_backward"
    n, E, k, S, device, args = _router_pack(where, logits, bias, topk_ids, counts, tokens, coef, mask, seq_offsets)
    keep, wp, wb = _workspace(workspace, L.moe_router_workspace_bytes, (n, E, S), where, device, stream)
    status = L.moe_router_backward(args, _array(topk_weights, where, "topk_weights", _F32, device, (n, k)),
                                   _array(d_weights, where, "d_weights", _F32, device, (n, k)),
                                   _array(d_loss, where, "d_loss", _F32, device, (1,)),
                                   _array(d_logits, where, "d_logits", _F32, device, (n, E)),
                                   _array(d_bias, where, "d_bias", _F32, device, (E,)), wp, wb,
                                   _handle(stream, device))
    if status:
        raise MoeError(status, where)
    return d_logits


def lora_workspace(n: int, n_adapters: int):
    """A workspace for lora_apply of up to n tokens over n_adapters adapters."""
    return _new_workspace(_ready().moe_lora_workspace_bytes(n, n_adapters))


def lora_apply(x, adapter_ids, a, b, y, out, *, scale=None, ranks=None, workspace=None, stream=None):
    """``moe_lora_apply``: out[t] = y[t] + scale[l] * B[l] (A[l] x[t]) with l = adapter_ids[t] (an id outside the
    bank, such as -1: out[t] = y[t]).  x [n, in] bf16, a [L, R, in] and b [L, out, R] bf16, y [n, out] (None: zero)
    and out [n, out] bf16 or fp32 (out may be y), scale [L] fp32, ranks [L] int32."""
    L = _lib if _torch is not None else _ready()
    where = "moe_lora_apply"
    if x is None or x.dim() != 2 or a is None or a.dim() != 3 or b is None or b.dim() != 3 or out is None:
        _refuse(where, "x is not [n, in], a not [L, R, in], b not [L, out, R], or out is missing")
    n, inp = shape = x.shape
    adapters, R, _ = a.shape
    o = b.shape[1]
    device = x.get_device()
    _on(device, where)
    yd = 0 if y is None else _dtype_code(y, where, "y")
    od = _dtype_code(out, where, "out")
    xp, xs = _rows(x, where, "x", _BF16, device, shape)
    yp, ys = _rows(y, where, "y", _KINDS[yd], device, (n, o))
    op, os_ = _rows(out, where, "out", _KINDS[od], device, (n, o))
    args = _LORA_ARGS.pack(
        n, inp, o, adapters, R, yd, od, _array(a, where, "a", _BF16, device, (adapters, R, inp)),
        _array(b, where, "b", _BF16, device, (adapters, o, R)), _array(scale, where, "scale", _F32, device, (adapters,)),
        _array(ranks, where, "ranks", _I32, device, (adapters,)),
        _array(adapter_ids, where, "adapter_ids", _I32, device, (n,)), xp, xs, yp, ys, op, os_)
    keep, wp, wb = _workspace(workspace, L.moe_lora_workspace_bytes, (n, adapters), where, device, stream)
    status = L.moe_lora_apply(args, wp, wb, _handle(stream, device))
    if status:
        raise MoeError(status, where)
    return out
