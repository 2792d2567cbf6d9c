"""Python binding of libmuse_moe.so, the B200 (sm_100a) latent-MoE block forward pass.

Argument marshalling only: every step of the block runs in the library's CUDA kernels.
PyTorch tensors are accepted as containers of device memory (their data pointers are
passed through the C ABI declared in include/muse_moe.h); nothing here computes.
If the compiled library is missing, importing works but every call raises.

Calls take stream= (a torch.cuda.Stream or a raw handle; by default the current stream). What
they return is memory of that stream, as if they were made under torch.cuda.stream(stream); the
caller orders the stream after the work that makes their inputs (and after the holder's
construction), and other streams after it (wait_stream; record_stream where a tensor's last use
is on another stream).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Dict, Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmuse_moe.so")

MUSE_F32, MUSE_BF16 = 0, 1
ROUTER_SOFTMAX, ROUTER_SIGMOID = 0, 1
EXPERTS_DENSE, EXPERTS_NVFP4 = 0, 1
ACT_BF16, ACT_NVFP4 = 0, 1
NORM_CENTRED, NORM_INPUT_SCALED = 0, 1
PROJ_DENSE, PROJ_INT8 = 0, 1
INT8_SCALE_DIVIDE, INT8_SCALE_RECIPROCAL = 0, 1

STATUS = {0: "MUSE_OK", 1: "MUSE_ERR_INVALID_ARG", 2: "MUSE_ERR_UNSUPPORTED", 3: "MUSE_ERR_WORKSPACE",
          4: "MUSE_ERR_CUDA", 5: "MUSE_ERR_TIMEOUT", 6: "MUSE_ERR_DEVICE"}

# every extern "C" entry point of include/muse_moe.h
EXPORTS = ("muse_moe_config_init", "muse_latent_moe_workspace_size", "muse_latent_moe_workspace_layout",
           "muse_latent_moe_forward", "muse_latent_moe_forward_host_io", "muse_latent_moe_last_device_status",
           "muse_status_string", "muse_latent_moe_launch_count", "muse_latent_moe_forward_static_scratch",
           "muse_selftest_bounded_wait", "muse_quantize_nvfp4_rows", "muse_latent_moe_forward_host_batches",
           "muse_ep_workspace_layout", "muse_ep_dispatch", "muse_ep_experts", "muse_ep_combine",
           "muse_latent_moe_forward_checked", "muse_latent_moe_stage_name", "muse_last_cuda_error",
           "muse_quantize_int8_rows", "muse_quantize_int8_rows_scaled", "muse_int8_matmul",
           "muse_int8_linear_workspace_size", "muse_int8_linear", "muse_int8_linear_scaled",
           "muse_latent_moe_few_tokens_workspace_size", "muse_latent_moe_few_tokens",
           "muse_latent_moe_few_tokens_checked", "muse_latent_moe_few_tokens_status")

# roles of an expert-parallel workspace (muse_ep_role)
EP_HOME, EP_EXPERTS = 1, 2

# most tokens of a muse_latent_moe_few_tokens call (MUSE_FEW_TOKENS)
FEW_TOKENS = 8

# size of the library's built-in scratch array (MUSE_STATIC_SCRATCH_BYTES)
STATIC_SCRATCH_BYTES = 16 << 20


class MuseError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: {STATUS.get(code, code)} ({status_string(code)})"
        if code == 4:  # MUSE_ERR_CUDA
            msg += f": {last_cuda_error()}"
        super().__init__(msg)


class Config(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("D", ctypes.c_int64), ("L", ctypes.c_int64), ("I", ctypes.c_int64),
                ("E", ctypes.c_int64), ("top_k", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("router_mode", ctypes.c_int32), ("router_logit_scale", ctypes.c_float),
                ("routed_scaling", ctypes.c_float), ("router_bias", ctypes.c_void_p),
                ("norm_mode", ctypes.c_int32), ("gamma_shared", ctypes.c_int32),
                ("pre_norm_gain", ctypes.c_void_p), ("pre_norm_eps", ctypes.c_float),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("topk_idx_out", ctypes.c_void_p), ("topk_w_out", ctypes.c_void_p),
                ("stage_events", ctypes.c_void_p), ("expert_weights", ctypes.c_int32),
                ("ffn_pre_gain", ctypes.c_void_p), ("ffn_pre_eps", ctypes.c_float),
                ("ffn_post_gain", ctypes.c_void_p), ("ffn_post_eps", ctypes.c_float),
                ("residual_gate", ctypes.c_void_p), ("residual_gate_temperature", ctypes.c_float),
                ("residual_gate_eps", ctypes.c_float), ("act_format", ctypes.c_int32),
                ("proj_weights", ctypes.c_int32)]


class Tensor(ctypes.Structure):
    """muse_tensor: device pointer, element type, rank, extents and strides (elements)."""
    _fields_ = [("data", ctypes.c_void_p), ("elem", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 3), ("stride", ctypes.c_int64 * 3)]


ELEM_F32, ELEM_BF16, ELEM_U8, ELEM_I8 = 0, 1, 2, 3


_elem_types: Dict = {}


def tensor_desc(t) -> Tensor:
    """The muse_tensor of a torch tensor (its own shape and strides: a non-contiguous view
    is described as it is, and the library rejects it)."""
    if not _elem_types:
        import torch
        _elem_types.update({torch.float32: ELEM_F32, torch.bfloat16: ELEM_BF16, torch.uint8: ELEM_U8,
                            torch.int8: ELEM_I8})
    dim = t.dim()
    n = min(dim, 3)
    d = Tensor(t.data_ptr(), _elem_types.get(t.dtype, -1), dim)
    d.shape[:n], d.stride[:n] = t.shape[:n], t.stride()[:n]
    return d


class Nvfp4Weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("block_scales", ctypes.c_void_p), ("matrix_scale", ctypes.c_void_p)]


class Int8Weight(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("status", "expert_count", "expert_offset", "logits", "topk_idx",
                                              "topk_w", "inv", "row_token", "z", "zp", "h", "y", "ss", "c",
                                              "xn", "ss_out", "zq_codes", "zq_scales", "hq_codes", "hq_scales",
                                              "total")] + [("rows", ctypes.c_int64)]


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m latent_mixture_experts_moe_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, cp = ctypes.c_void_p, ctypes.POINTER(Config)
        L.muse_moe_config_init.argtypes = [cp]
        L.muse_moe_config_init.restype = None
        L.muse_latent_moe_workspace_size.argtypes = [cp, ctypes.POINTER(ctypes.c_size_t)]
        L.muse_latent_moe_workspace_size.restype = ctypes.c_int
        L.muse_latent_moe_workspace_layout.argtypes = [cp, ctypes.POINTER(WorkspaceLayout)]
        L.muse_latent_moe_workspace_layout.restype = ctypes.c_int
        L.muse_latent_moe_forward.argtypes = [cp] + [vp] * 10
        L.muse_latent_moe_forward.restype = ctypes.c_int
        L.muse_latent_moe_forward_host_io.argtypes = [cp] + [vp] * 12
        L.muse_latent_moe_forward_host_io.restype = ctypes.c_int
        L.muse_latent_moe_last_device_status.argtypes = [cp, vp, ctypes.POINTER(ctypes.c_uint32)]
        L.muse_latent_moe_last_device_status.restype = ctypes.c_int
        L.muse_status_string.argtypes = [ctypes.c_int]
        L.muse_status_string.restype = ctypes.c_char_p
        L.muse_last_cuda_error.argtypes = []
        L.muse_last_cuda_error.restype = ctypes.c_char_p
        L.muse_latent_moe_forward_static_scratch.argtypes = [cp] + [vp] * 10
        L.muse_latent_moe_forward_static_scratch.restype = ctypes.c_int
        L.muse_selftest_bounded_wait.argtypes = [ctypes.c_uint64, vp, vp]
        L.muse_selftest_bounded_wait.restype = ctypes.c_int
        L.muse_quantize_nvfp4_rows.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, vp, vp, vp]
        L.muse_quantize_nvfp4_rows.restype = ctypes.c_int
        L.muse_latent_moe_forward_host_batches.argtypes = [cp, ctypes.c_int64, vp, vp, vp, vp] + [vp] * 7 + [vp] * 3
        L.muse_latent_moe_forward_host_batches.restype = ctypes.c_int
        i32, i64 = ctypes.c_int32, ctypes.c_int64
        L.muse_ep_workspace_layout.argtypes = [cp, i32, i32, i64, ctypes.POINTER(WorkspaceLayout)]
        L.muse_ep_workspace_layout.restype = ctypes.c_int
        L.muse_ep_dispatch.argtypes = [cp, i32] + [vp] * 7
        L.muse_ep_dispatch.restype = ctypes.c_int
        L.muse_ep_experts.argtypes = [cp, i32, i64] + [vp] * 9
        L.muse_ep_experts.restype = ctypes.c_int
        L.muse_ep_combine.argtypes = [cp, i32] + [vp] * 7
        L.muse_ep_combine.restype = ctypes.c_int
        L.muse_latent_moe_forward_checked.argtypes = [cp] + [ctypes.POINTER(Tensor)] * 9 + [vp]
        L.muse_latent_moe_forward_checked.restype = ctypes.c_int
        L.muse_latent_moe_stage_name.argtypes = [cp, ctypes.c_int32]
        L.muse_latent_moe_stage_name.restype = ctypes.c_char_p
        L.muse_latent_moe_launch_count.argtypes = [cp]
        L.muse_latent_moe_launch_count.restype = ctypes.c_int32
        wp = ctypes.POINTER(Int8Weight)
        L.muse_quantize_int8_rows.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp]
        L.muse_quantize_int8_rows.restype = ctypes.c_int
        L.muse_quantize_int8_rows_scaled.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, vp]
        L.muse_quantize_int8_rows_scaled.restype = ctypes.c_int
        L.muse_int8_matmul.argtypes = [vp, vp, i64, i64, wp, i64, vp, i32, i64, vp, vp]
        L.muse_int8_matmul.restype = ctypes.c_int
        L.muse_int8_linear_workspace_size.argtypes = [i64, i64, ctypes.POINTER(ctypes.c_size_t)]
        L.muse_int8_linear_workspace_size.restype = ctypes.c_int
        L.muse_int8_linear.argtypes = [vp, i32, i64, i64, i64, wp, i64, vp, i32, i64, vp, ctypes.c_size_t, vp, vp]
        L.muse_int8_linear.restype = ctypes.c_int
        L.muse_int8_linear_scaled.argtypes = L.muse_int8_linear.argtypes[:-1] + [i32, vp]
        L.muse_int8_linear_scaled.restype = ctypes.c_int
        L.muse_latent_moe_few_tokens_workspace_size.argtypes = [cp, ctypes.POINTER(ctypes.c_size_t)]
        L.muse_latent_moe_few_tokens_workspace_size.restype = ctypes.c_int
        L.muse_latent_moe_few_tokens.argtypes = [cp] + [vp] * 10
        L.muse_latent_moe_few_tokens.restype = ctypes.c_int
        L.muse_latent_moe_few_tokens_checked.argtypes = [cp] + [ctypes.POINTER(Tensor)] * 9 + [vp]
        L.muse_latent_moe_few_tokens_checked.restype = ctypes.c_int
        L.muse_latent_moe_few_tokens_status.argtypes = [cp, vp, ctypes.POINTER(ctypes.c_uint32)]
        L.muse_latent_moe_few_tokens_status.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().muse_status_string(code).decode()


def last_cuda_error() -> str:
    """The CUDA runtime's description of the last CUDA error behind a MUSE_ERR_CUDA on this
    thread ("no error" when none)."""
    return lib().muse_last_cuda_error().decode()


def _check(code: int, where: str) -> None:
    if code != 0:
        raise MuseError(code, where)


def make_config(T: int, D: int, L: int, I: int, E: int, k: int, dtype: str = "bf16", eps: float = 1e-6,
                router_mode: int = ROUTER_SOFTMAX, router_logit_scale: float = 1.0, routed_scaling: float = 1.0,
                norm_mode: int = NORM_CENTRED, gamma_shared: bool = False, pre_norm_eps: float = 1e-5,
                ffn_pre_eps: float = 1e-5, ffn_post_eps: float = 1e-8, residual_gate_temperature: float = 0.3,
                residual_gate_eps: float = 1e-3, act_format: int = ACT_BF16) -> Config:
    c = Config()
    lib().muse_moe_config_init(ctypes.byref(c))
    c.T, c.D, c.L, c.I, c.E, c.top_k = T, D, L, I, E, k
    c.dtype = {"f32": MUSE_F32, "bf16": MUSE_BF16}[dtype]
    c.eps = eps
    c.router_mode, c.router_logit_scale, c.routed_scaling = router_mode, router_logit_scale, routed_scaling
    c.norm_mode, c.gamma_shared = norm_mode, int(gamma_shared)
    c.pre_norm_eps = pre_norm_eps
    c.ffn_pre_eps, c.ffn_post_eps = ffn_pre_eps, ffn_post_eps
    c.residual_gate_temperature, c.residual_gate_eps = residual_gate_temperature, residual_gate_eps
    c.act_format = act_format
    return c


def workspace_size(cfg: Config) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().muse_latent_moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "workspace_size")
    return int(n.value)


def workspace_layout(cfg: Config) -> Dict[str, int]:
    lay = WorkspaceLayout()
    _check(lib().muse_latent_moe_workspace_layout(ctypes.byref(cfg), ctypes.byref(lay)), "workspace_layout")
    return {name: int(getattr(lay, name)) for name, _ in WorkspaceLayout._fields_}


def launch_count(cfg: Config) -> int:
    return int(lib().muse_latent_moe_launch_count(ctypes.byref(cfg)))


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, ctypes.Structure):
        return ctypes.addressof(t)
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return int(t.data_ptr())


def _stream_handle(stream) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    return int(getattr(stream, "cuda_stream", stream))


def _empty(shape, dtype, device, stream):
    """An output in memory of the stream that the call runs on: memory of another one may still be
    in use by work that is pending there."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_handle(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def forward(cfg: Config, x, W_router, W_pool, W_gate, W_up, W_down, gamma, W_unpool, out, stream=None) -> None:
    """Enqueue one forward pass; cfg.workspace must point to workspace_size(cfg) bytes."""
    code = lib().muse_latent_moe_forward(ctypes.byref(cfg), _ptr(x), _ptr(W_router), _ptr(W_pool), _ptr(W_gate),
                                         _ptr(W_up), _ptr(W_down), _ptr(gamma), _ptr(W_unpool), _ptr(out),
                                         _stream_handle(stream))
    _check(code, "muse_latent_moe_forward")


def forward_checked(cfg: Config, x, W_router, W_pool, W_gate, W_up, W_down, gamma, W_unpool, out,
                    stream=None) -> None:
    """Enqueue one forward through the shape-checked entry point: every argument is a torch
    tensor (NVFP4 experts: a (codes, block scales, matrix scales) triple each; int8
    projections: a (codes, scales) pair each) described by
    its dtype, shape and strides; the library rejects a mismatch before launching anything."""
    _call_checked(lib().muse_latent_moe_forward_checked, "muse_latent_moe_forward_checked", cfg, x, W_router, W_pool,
                  W_gate, W_up, W_down, gamma, W_unpool, out, stream)


def _weight_descs(W_router, W_pool, W_gate, W_up, W_down, gamma, W_unpool):
    """The muse_tensor arrays of a layer's weights, in argument order (NVFP4 experts: three each,
    int8 projections: two each)."""
    def descs(t):
        parts = t if isinstance(t, (tuple, list)) else (t,)
        return (Tensor * len(parts))(*[tensor_desc(p) for p in parts])
    return tuple(descs(t) for t in (W_router, W_pool, W_gate, W_up, W_down, gamma, W_unpool))


def _call_checked(fn, name: str, cfg: Config, x, W_router, W_pool, W_gate, W_up, W_down, gamma, W_unpool, out,
                  stream) -> None:
    weights = _weight_descs(W_router, W_pool, W_gate, W_up, W_down, gamma, W_unpool)
    code = fn(ctypes.byref(cfg), ctypes.byref(tensor_desc(x)), *weights, ctypes.byref(tensor_desc(out)),
              _stream_handle(stream))
    _check(code, name)


def few_tokens_workspace_size(cfg: Config) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().muse_latent_moe_few_tokens_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "muse_latent_moe_few_tokens_workspace_size")
    return int(n.value)


def few_tokens(cfg: Config, x, W_router, W_pool, W_gate, W_up, W_down, gamma, W_unpool, out, stream=None) -> None:
    """Enqueue the whole layer for cfg.T <= FEW_TOKENS tokens as one kernel, every tensor checked
    by its shape as in forward_checked; cfg.workspace: few_tokens_workspace_size(cfg) bytes."""
    _call_checked(lib().muse_latent_moe_few_tokens_checked, "muse_latent_moe_few_tokens_checked", cfg, x, W_router,
                  W_pool, W_gate, W_up, W_down, gamma, W_unpool, out, stream)


def few_tokens_status(cfg: Config, stream=None):
    """(status, detail) of the last few_tokens call on cfg.workspace; synchronises the stream."""
    detail = ctypes.c_uint32(0)
    code = lib().muse_latent_moe_few_tokens_status(ctypes.byref(cfg), _stream_handle(stream), ctypes.byref(detail))
    return int(code), int(detail.value)


def forward_static_scratch(cfg: Config, x, W_router, W_pool, W_gate, W_up, W_down, gamma, W_unpool, out,
                           stream=None) -> None:
    """Forward through the allocation-free entry point (workspace = the library's built-in
    scratch array; cfg.workspace is ignored). For callers that cannot allocate device memory."""
    code = lib().muse_latent_moe_forward_static_scratch(ctypes.byref(cfg), _ptr(x), _ptr(W_router), _ptr(W_pool),
                                                        _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(gamma),
                                                        _ptr(W_unpool), _ptr(out), _stream_handle(stream))
    _check(code, "muse_latent_moe_forward_static_scratch")


def forward_host_io(cfg: Config, x_host, x_dev, W_router, W_pool, W_gate, W_up, W_down, gamma, W_unpool,
                    out_dev, out_host, stream=None) -> None:
    code = lib().muse_latent_moe_forward_host_io(ctypes.byref(cfg), _ptr(x_host), _ptr(x_dev), _ptr(W_router),
                                                 _ptr(W_pool), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
                                                 _ptr(gamma), _ptr(W_unpool), _ptr(out_dev), _ptr(out_host),
                                                 _stream_handle(stream))
    _check(code, "muse_latent_moe_forward_host_io")


def forward_host_batches(cfg: Config, x_hosts, out_hosts, x_devs, out_devs, W_router, W_pool, W_gate, W_up, W_down,
                         gamma, W_unpool, stream, h2d_stream, d2h_stream) -> None:
    """Batches through the forward with host buffers, copies overlapped with compute (two
    device buffers each for x and out; three distinct torch.cuda.Stream objects)."""
    n = len(x_hosts)
    xh = (ctypes.c_void_p * n)(*[_ptr(t) for t in x_hosts])
    oh = (ctypes.c_void_p * n)(*[_ptr(t) for t in out_hosts])
    xd = (ctypes.c_void_p * 2)(*[_ptr(t) for t in x_devs])
    od = (ctypes.c_void_p * 2)(*[_ptr(t) for t in out_devs])
    code = lib().muse_latent_moe_forward_host_batches(
        ctypes.byref(cfg), n, ctypes.cast(xh, ctypes.c_void_p), ctypes.cast(oh, ctypes.c_void_p),
        ctypes.cast(xd, ctypes.c_void_p), ctypes.cast(od, ctypes.c_void_p), _ptr(W_router), _ptr(W_pool),
        _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(gamma), _ptr(W_unpool), _stream_handle(stream),
        _stream_handle(h2d_stream), _stream_handle(d2h_stream))
    _check(code, "muse_latent_moe_forward_host_batches")


def ep_workspace_layout(cfg: Config, ep_size: int, role: int, rows: int = 0) -> Dict[str, int]:
    """Buffer offsets (and "total" bytes) of an expert-parallel workspace: role EP_HOME for
    cfg.T tokens, EP_EXPERTS for up to `rows` received rows."""
    lay = WorkspaceLayout()
    _check(lib().muse_ep_workspace_layout(ctypes.byref(cfg), int(ep_size), int(role), int(rows), ctypes.byref(lay)),
           "muse_ep_workspace_layout")
    return {name: int(getattr(lay, name)) for name, _ in WorkspaceLayout._fields_}


def ep_dispatch(cfg: Config, ep_size: int, x, W_router, W_pool, send_z, send_expert, rank_counts, stream=None) -> None:
    """Expert-parallel step 1 (cfg.workspace: an EP_HOME workspace)."""
    _check(lib().muse_ep_dispatch(ctypes.byref(cfg), int(ep_size), _ptr(x), _ptr(W_router), _ptr(W_pool), _ptr(send_z),
                                  _ptr(send_expert), _ptr(rank_counts), _stream_handle(stream)), "muse_ep_dispatch")


def ep_experts(cfg: Config, ep_size: int, rows: int, recv_z, recv_expert, W_gate, W_up, W_down, gamma, ret_y, ret_ss,
               stream=None) -> None:
    """Expert-parallel step 3 (cfg.workspace: an EP_EXPERTS workspace)."""
    _check(lib().muse_ep_experts(ctypes.byref(cfg), int(ep_size), int(rows), _ptr(recv_z), _ptr(recv_expert),
                                 _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(gamma), _ptr(ret_y), _ptr(ret_ss),
                                 _stream_handle(stream)), "muse_ep_experts")


def ep_combine(cfg: Config, ep_size: int, x, back_y, back_ss, gamma, W_unpool, out, stream=None) -> None:
    """Expert-parallel step 5 (cfg.workspace: the EP_HOME workspace of step 1)."""
    _check(lib().muse_ep_combine(ctypes.byref(cfg), int(ep_size), _ptr(x), _ptr(back_y), _ptr(back_ss), _ptr(gamma),
                                 _ptr(W_unpool), _ptr(out), _stream_handle(stream)), "muse_ep_combine")


def stages(cfg: Config):
    """Names of the stages one forward launches for cfg, in launch order (from the library:
    muse_latent_moe_stage_name)."""
    names = []
    while True:
        n = lib().muse_latent_moe_stage_name(ctypes.byref(cfg), len(names))
        if n is None:
            return tuple(names)
        names.append(n.decode())


def event_handles(events) -> "ctypes.Array":
    """ctypes array of the raw cudaEvent_t handles of torch.cuda.Event objects (each
    recorded once beforehand so that it exists)."""
    arr = (ctypes.c_void_p * len(events))()
    for i, ev in enumerate(events):
        arr[i] = int(ev.cuda_event)
    return arr


def quantize_nvfp4_rows(src, codes, scales, stream=None) -> None:
    """NVFP4 activation quantiser: src bf16 [rows, K] -> codes uint8 [rows, K/2], scales
    uint8 [rows, K/16] (CUDA tensors)."""
    rows, K = src.shape
    _check(lib().muse_quantize_nvfp4_rows(_ptr(src), int(rows), int(K), _ptr(codes), _ptr(scales),
                                          _stream_handle(stream)), "muse_quantize_nvfp4_rows")


_float_types: Dict = {}


def _rows(t, name: str):
    """Pointer, muse_dtype and row distance of a 2-D float tensor whose rows are contiguous."""
    if not _float_types:
        import torch
        _float_types.update({torch.bfloat16: MUSE_BF16, torch.float32: MUSE_F32})
    dtype, strides = _float_types.get(t.dtype), t.stride()
    if dtype is None or len(strides) != 2:
        raise ValueError(f"{name} must be a 2-D float32 or bfloat16 tensor")
    (rows, cols), (step, inner) = t.shape, strides
    if inner != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.data_ptr(), dtype, step if rows > 1 else cols


def _int8_operand(codes, scales, name: str):
    import torch
    if codes.dim() != 2 or codes.dtype != torch.int8 or not codes.is_contiguous():
        raise ValueError(f"{name} codes must be a contiguous 2-D int8 tensor")
    if scales.shape != (codes.shape[0],) or scales.dtype != torch.float32 or not scales.is_contiguous():
        raise ValueError(f"{name} scales must be a contiguous float32 tensor with one value per row of the codes")


def _one_device(*tensors):
    """The device all tensors are on (a context in which the library's calls run)."""
    import torch
    dev = tensors[0].device
    if dev.type != "cuda" or any(t.device != dev for t in tensors):
        raise ValueError("tensors must be on one CUDA device")
    return contextlib.nullcontext() if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def quantize_int8_rows(src, codes=None, scales=None, stream=None, scale_rule: int = INT8_SCALE_DIVIDE):
    """src [rows, K] float32 or bfloat16 (rows may lie apart, K a multiple of 16) -> codes int8
    [rows, K] and scales float32 [rows], created if not given; returns both. For activations a
    row is a token, for weights [out, in] an output channel. scale_rule: a row's scale is
    INT8_SCALE_DIVIDE max / 127, or INT8_SCALE_RECIPROCAL what torch computes for amax / 127.0
    on a GPU (the codes then equal those of rows quantised with torch)."""
    import torch
    ptr, dtype, ld = _rows(src, "src")
    rows, K = src.shape
    codes = _empty((rows, K), torch.int8, src.device, stream) if codes is None else codes
    scales = _empty(rows, torch.float32, src.device, stream) if scales is None else scales
    _int8_operand(codes, scales, "int8")
    if codes.shape != src.shape:
        raise ValueError("codes must have the shape of src")
    with _one_device(src, codes, scales):
        _check(lib().muse_quantize_int8_rows_scaled(ptr, dtype, int(rows), int(K), ld, _ptr(codes), _ptr(scales),
                                                    int(scale_rule), _stream_handle(stream)),
               "muse_quantize_int8_rows_scaled")
    return codes, scales


class Int8Linear:
    """A product with int8 weights: codes [out, in] and scales [out] (quantize_int8_rows of the
    weights), for up to T_max rows per call; scale_rule says how a row's scale is made (see
    quantize_int8_rows). The weights may be changed in place or replaced (self.codes, self.scales, by
    tensors of the same shapes) between calls. Holds the workspace of the quantised rows, so calls
    that overlap on the GPU need holders of their own."""

    def __init__(self, codes, scales, T_max: int, scale_rule: int = INT8_SCALE_DIVIDE):
        import torch
        _int8_operand(codes, scales, "weight")
        if scale_rule not in (INT8_SCALE_DIVIDE, INT8_SCALE_RECIPROCAL):
            raise ValueError("scale_rule is INT8_SCALE_DIVIDE or INT8_SCALE_RECIPROCAL")
        self.codes, self.scales, self.T_max, self.scale_rule = codes, scales, int(T_max), int(scale_rule)
        self.N, self.K = (int(n) for n in codes.shape)
        self.weight = Int8Weight(_ptr(codes), _ptr(scales))
        self._linear = lib().muse_int8_linear_scaled
        self._weight_key = self._key()
        n = ctypes.c_size_t(0)
        _check(lib().muse_int8_linear_workspace_size(self.T_max, self.K, ctypes.byref(n)),
               "muse_int8_linear_workspace_size")
        with _one_device(codes, scales):
            self.workspace = torch.empty(max(int(n.value), 1), dtype=torch.uint8, device=codes.device)
            self.status = torch.zeros(2, dtype=torch.int32, device=codes.device)
        # what every call passes (a product of a few microseconds should not wait for marshalling)
        self._torch, self._device = torch, codes.device
        self._weight = ctypes.byref(self.weight)
        self._ws, self._ws_bytes, self._status = _ptr(self.workspace), self.workspace.numel(), _ptr(self.status)

    def _key(self):
        c, s = self.codes, self.scales
        return (c.data_ptr(), s.data_ptr(), c.shape, s.shape, c.dtype, s.dtype, c.is_contiguous(), s.is_contiguous())

    def _run(self, T, device, out, out_dtype, stream, call):
        """call(out pointer, its muse_dtype and row distance, stream handle) on the holder's device."""
        torch = self._torch
        if self._key() != self._weight_key:  # the weights were replaced
            _int8_operand(self.codes, self.scales, "weight")
            if tuple(self.codes.shape) != (self.N, self.K):
                raise ValueError(f"the weights' codes must be [{self.N}, {self.K}]")
            if any(t.device != self._device for t in (self.codes, self.scales)):
                raise ValueError(f"tensors must be on {self._device}")
            self.weight.codes, self.weight.scales = _ptr(self.codes), _ptr(self.scales)
            self._weight_key = self._key()
        if device != self._device or (out is not None and out.device != device):
            raise ValueError(f"tensors must be on {self._device}")
        dtype = None
        if out is None:
            out = _empty((T, self.N), out_dtype, device, stream)
            ptr, dtype, ld = out.data_ptr(), _float_types.get(out_dtype), self.N
        elif tuple(out.shape) != (T, self.N) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out must be [{T}, {self.N}] of the output type")
        if dtype is None:
            ptr, dtype, ld = _rows(out, "out")
        if torch.cuda.current_device() == device.index:
            call(ptr, dtype, ld, _stream_handle(stream))
        else:
            with torch.cuda.device(device):
                call(ptr, dtype, ld, _stream_handle(stream))
        return out

    def __call__(self, x, out=None, out_dtype=None, stream=None):
        """out[T, out] = x[T, in] W^T, x quantised per row; out in x's type unless given."""
        ptr, dtype, ld = _rows(x, "x")
        T = x.shape[0]
        if x.shape[1] != self.K:
            raise ValueError(f"x has {x.shape[1]} columns, the weights {self.K}")
        if T > self.T_max:
            raise ValueError(f"T={T} exceeds T_max={self.T_max}")

        def call(optr, odtype, ldo, st):
            _check(self._linear(ptr, dtype, T, self.K, ld, self._weight, self.N, optr, odtype, ldo, self._ws,
                                self._ws_bytes, self._status, self.scale_rule, st), "muse_int8_linear_scaled")
        return self._run(T, x.device, out, out_dtype or (x.dtype if out is None else None), stream, call)

    def matmul(self, x_codes, x_scales, out=None, out_dtype=None, stream=None):
        """The product of rows that are quantised already (bfloat16 unless out or out_dtype says
        otherwise); any number of rows."""
        _int8_operand(x_codes, x_scales, "x")
        T = x_codes.shape[0]
        if x_codes.shape[1] != self.K:
            raise ValueError(f"x has {x_codes.shape[1]} columns, the weights {self.K}")
        if x_scales.device != x_codes.device:
            raise ValueError("x's codes and scales must be on one device")

        def call(optr, odtype, ldo, st):
            _check(lib().muse_int8_matmul(_ptr(x_codes), _ptr(x_scales), T, self.K, self._weight, self.N, optr, odtype,
                                          ldo, self._status, st), "muse_int8_matmul")
        return self._run(T, x_codes.device, out, out_dtype or (self._torch.bfloat16 if out is None else None), stream,
                         call)

    def device_status(self):
        """(status, detail) that bounded waits of this holder's calls recorded; synchronises."""
        code, detail = self.status.tolist()
        return int(code), int(detail) & 0xffffffff


def selftest_bounded_wait(limit_ns: int, status_dev, stream=None) -> None:
    """Run the device-side bounded-wait self-test (status_dev: zeroed CUDA int32[2])."""
    _check(lib().muse_selftest_bounded_wait(int(limit_ns), _ptr(status_dev), _stream_handle(stream)),
           "muse_selftest_bounded_wait")


def last_device_status(cfg: Config, stream=None):
    detail = ctypes.c_uint32(0)
    code = lib().muse_latent_moe_last_device_status(ctypes.byref(cfg), _stream_handle(stream), ctypes.byref(detail))
    return int(code), int(detail.value)


def expert_weight_dims(weights: Dict):
    """(I, L, nvfp4) from the expert weights: dense W_gate [E, I, L], or NVFP4 codes
    W_gate_codes [E, I, L/2]."""
    if "W_gate_codes" in weights:
        _, I, L2 = weights["W_gate_codes"].shape
        return int(I), int(2 * L2), True
    _, I, L = weights["W_gate"].shape
    return int(I), int(L), False


def expert_operands(weights: Dict, nvfp4: bool):
    """The W_gate, W_up, W_down arguments of the C ABI: the dense tensors, or Nvfp4Weight
    descriptors of <name>_codes [E, out, in/2], <name>_scales [E, out, in/16] and
    <name>_mscale [E]."""
    if not nvfp4:
        return tuple(weights[n] for n in ("W_gate", "W_up", "W_down"))
    return tuple(Nvfp4Weight(_ptr(weights[n + "_codes"]), _ptr(weights[n + "_scales"]), _ptr(weights[n + "_mscale"]))
                 for n in ("W_gate", "W_up", "W_down"))


def projection_operand(weights: Dict, name: str):
    """(W_pool or W_unpool as the C ABI takes it, as the shape-checked entry points take it): the
    dense tensor, or for int8 weights <name>_codes [out, in] and <name>_scales [out] (of
    quantize_int8_rows) an Int8Weight and the two tensors."""
    if name + "_codes" not in weights:
        return weights[name], weights[name]
    codes, scales = weights[name + "_codes"], weights[name + "_scales"]
    return Int8Weight(_ptr(codes), _ptr(scales)), (codes, scales)


def block_config(T: int, dims: Dict, dtype: str, modes: Dict, weights: Dict, nvfp4: bool, workspace=None) -> Config:
    """Config of the block for T tokens: sizes, modes, the optional pointers found in
    weights (router_bias, pre_norm_gain, ffn_pre_gain, ffn_post_gain, residual_gate) and
    the workspace (a uint8 CUDA tensor) if given."""
    d = dims
    c = make_config(T, d["D"], d["L"], d["I"], d["E"], d["k"], dtype, d["eps"], **modes)
    if nvfp4:
        c.expert_weights = EXPERTS_NVFP4
    if ("W_pool_codes" in weights) != ("W_unpool_codes" in weights):
        raise ValueError("W_pool and W_unpool must both be int8 or both dense")
    if "W_pool_codes" in weights:
        c.proj_weights = PROJ_INT8
    if weights.get("router_bias") is not None:
        c.router_bias = _ptr(weights["router_bias"])
    for name in ("pre_norm_gain", "ffn_pre_gain", "ffn_post_gain", "residual_gate"):
        if weights.get(name) is not None:
            setattr(c, name, _ptr(weights[name]))
    if workspace is not None:
        c.workspace = _ptr(workspace)
        c.workspace_bytes = workspace.numel()
    return c


class LatentMoE:
    """Holds the block's device weights and a workspace; calling it runs the forward through
    the shape-checked entry point (muse_latent_moe_forward_checked).

    weights: dict with W_router, W_pool, W_gate, W_up, W_down, gamma, W_unpool (torch
    CUDA tensors in the layouts of include/muse_moe.h; int8 projections as W_pool_codes,
    W_pool_scales, W_unpool_codes and W_unpool_scales instead, of quantize_int8_rows); router_bias, pre_norm_gain and the
    feed-forward sublayer's ffn_pre_gain, ffn_post_gain and residual_gate (float32) are
    optional. modes: make_config keywords (router_mode, norm_mode, gamma_shared, ...).
    Every call computes with what the entries of self.w hold then, so weights may be changed in
    place or replaced (by tensors of the same shapes) between calls.
    """

    OPTIONS = ("router_bias", "pre_norm_gain", "ffn_pre_gain", "ffn_post_gain", "residual_gate")

    def __init__(self, weights: Dict, T_max: int, k: int, eps: float = 1e-6, **modes):
        import torch
        self.w = dict(weights)
        E, D = weights["W_router"].shape
        I, L, self.nvfp4 = expert_weight_dims(weights)
        # experts and projections as the C ABI takes them
        self.w["W_gate"], self.w["W_up"], self.w["W_down"] = expert_operands(weights, self.nvfp4)
        for name in ("W_pool", "W_unpool"):
            self.w[name], _ = projection_operand(weights, name)
        self.dtype = {torch.float32: "f32", torch.bfloat16: "bf16"}[weights["W_router"].dtype]
        self.dims = dict(D=int(D), L=L, I=I, E=int(E), k=k, eps=eps)
        self.modes = modes
        cfg = self.config(T_max)
        self.workspace = torch.empty(workspace_size(cfg), dtype=torch.uint8, device=weights["W_router"].device)
        self.T_max = T_max
        # the single-kernel form for a few tokens has a (small) workspace of its own; None where the
        # library does not offer it for these modes
        self.few_workspace = None
        try:
            few = few_tokens_workspace_size(self.config(min(T_max, FEW_TOKENS)))
            self.few_workspace = torch.empty(few, dtype=torch.uint8, device=weights["W_router"].device)
        except MuseError as e:
            if e.code != 2:  # MUSE_ERR_UNSUPPORTED
                raise
        self._few_key = self._few_call = None

    def operands(self):
        """W_router, W_pool, W_gate, W_up, W_down, gamma and W_unpool as the shape-checked entry points
        take them: tensors, or tuples of NVFP4 and int8 parts."""
        w = self.w

        def one(name, parts):
            return tuple(w[name + p] for p in parts) if name + "_codes" in w else w[name]
        experts = (one(n, ("_codes", "_scales", "_mscale")) for n in ("W_gate", "W_up", "W_down"))
        return (w["W_router"], one("W_pool", ("_codes", "_scales")), *experts, w["gamma"],
                one("W_unpool", ("_codes", "_scales")))

    def _tensors(self):
        """Every tensor of the block that a call reads."""
        options = (self.w[n] for n in self.OPTIONS if self.w.get(n) is not None)
        return (*options, *(t for o in self.operands() for t in (o if type(o) is tuple else (o,))))

    @property
    def experts(self):
        """W_gate, W_up and W_down as the shape-checked entry points take them."""
        return self.operands()[2:5]

    def _few(self):
        """Configuration and weight descriptors of few_tokens. They are made again only when something
        they say has changed (2 us to find out): a call of a few microseconds would otherwise
        spend more time on marshalling than on the GPU."""
        w, ws = self.w, self.few_workspace
        key = ([(t.data_ptr(), t.shape, t.dtype, t.is_contiguous()) if hasattr(t, "data_ptr") else None
                for t in w.values()],
               list(w), list(self.dims.values()), dict(self.modes), ws is not None and (ws.data_ptr(), ws.numel()))
        if key != self._few_key:
            _one_device(*self._tensors(), *(() if ws is None else (ws,)))
            self._few_call = self.config(min(self.T_max, FEW_TOKENS), ws), _weight_descs(*self.operands())
            self._few_key = key
        return self._few_call

    def config(self, T: int, workspace=None) -> Config:
        return block_config(T, self.dims, self.dtype, self.modes, self.w, self.nvfp4, workspace)

    def __call__(self, x, out=None, stream=None, topk_idx=None, topk_w=None, stage_events=None):
        """stage_events: optional ctypes array of launch_count + 1 cudaEvent_t handles."""
        T = x.shape[0]
        if T > self.T_max:
            raise ValueError(f"T={T} exceeds T_max={self.T_max}")
        given = (t for t in (out, topk_idx, topk_w) if t is not None)
        with _one_device(x, self.workspace, *given, *self._tensors()):
            cfg = self.config(T, self.workspace)
            cfg.topk_idx_out, cfg.topk_w_out = _ptr(topk_idx), _ptr(topk_w)
            if stage_events is not None:
                cfg.stage_events = ctypes.cast(stage_events, ctypes.c_void_p)
            if out is None:
                out = _empty((T, self.dims["D"]), x.dtype, x.device, stream)
            forward_checked(cfg, x, *self.operands(), out, stream)
        return out

    def few_tokens(self, x, out=None, stream=None, topk_idx=None, topk_w=None):
        """The layer for 1 .. FEW_TOKENS tokens as one kernel (muse_latent_moe_few_tokens): the same
        mathematics as calling the holder, for interactive decoding. Calls that overlap on the GPU
        need holders of their own."""
        import torch
        T = x.shape[0]
        if T > min(self.T_max, FEW_TOKENS):
            raise ValueError(f"T={T} exceeds {min(self.T_max, FEW_TOKENS)}")
        routing = () if topk_idx is None and topk_w is None else ((topk_idx, torch.int32), (topk_w, torch.float32))
        for t, dtype in routing:
            if t is not None and (t.shape != (T, self.dims["k"]) or t.dtype != dtype or t.device != x.device
                                  or not t.is_contiguous()):
                raise ValueError(f"topk_idx and topk_w are contiguous [{T}, {self.dims['k']}] int32 and float32 tensors "
                                 "on x's device")
        with _one_device(x, self.w["W_router"], x if out is None else out):
            few_config, weights = self._few()
            cfg = Config.from_buffer_copy(few_config)
            cfg.T, cfg.topk_idx_out, cfg.topk_w_out = T, _ptr(topk_idx), _ptr(topk_w)
            if out is None:
                out = _empty((T, self.dims["D"]), x.dtype, x.device, stream)
            code = lib().muse_latent_moe_few_tokens_checked(
                ctypes.byref(cfg), ctypes.byref(tensor_desc(x)), *weights, ctypes.byref(tensor_desc(out)),
                _stream_handle(stream))
            _check(code, "muse_latent_moe_few_tokens_checked")
        return out
