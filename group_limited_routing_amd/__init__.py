"""Beam sparse-MoE block on MI355X (gfx950): Python binding of libbeam_moe.so.

Argument marshalling only. Every step of the block (router logits, group-
limited selection, permutation, expert GEMMs, combine) runs in the HIP
kernels behind the C ABI declared in include/beam_moe.h; torch supplies
device memory and the current stream. If the library is missing the calls
raise instead of falling back to anything else.

Names follow the Beam model doc's config fields: n_group, topk_group,
routed_scaling_factor (transformers model doc "Beam", "Overview").

Streams: every call takes ``stream`` (default: the current stream of the
tensors' device) and enqueues its kernels there. Tensors a call allocates
(outputs, and the workspace when none is passed) come from that stream's
pool of torch's caching allocator, so a block freed on return is reused only
by later work on the same stream, which runs after the kernels that used it.
A caller that passes its own workspace or outputs owns their stream
ordering, as for any torch tensor used on a side stream.
"""

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libbeam_moe.so")

BEAM_OK, BEAM_ERR_NULL, BEAM_ERR_CONFIG, BEAM_ERR_SHAPE = 0, 1, 2, 3
BEAM_ERR_DTYPE, BEAM_ERR_ALIGN, BEAM_ERR_WORKSPACE, BEAM_ERR_HIP = 4, 5, 6, 7
BEAM_F32, BEAM_BF16, BEAM_FP8_E4M3, BEAM_MXFP4, BEAM_E8M0 = 0, 1, 2, 3, 4
BEAM_LAYOUT_ROW_MAJOR, BEAM_LAYOUT_PACKED = 0, 1
BEAM_QUANT_NONE, BEAM_QUANT_ROW, BEAM_QUANT_BLOCK = 0, 1, 2
BEAM_SCORE_SIGMOID, BEAM_SCORE_SOFTMAX = 0, 1
BEAM_GROUP_TOP2, BEAM_GROUP_MAX = 0, 1
BEAM_X_E4M3_ROW, BEAM_X_E4M3_BLOCK, BEAM_X_MXFP4 = 0, 1, 2

EXPORTED = ("beam_moe_workspace_bytes", "beam_moe_route", "beam_moe_forward",
            "beam_moe_forward_residual", "beam_moe_status_string", "beam_moe_profile_begin",
            "beam_moe_profile_end", "beam_moe_pack_weights", "beam_moe_backward_workspace_bytes",
            "beam_moe_backward", "beam_moe_pack_weights_transposed", "beam_moe_update_bias",
            "beam_moe_forward_shard", "beam_moe_forward_noalloc", "beam_moe_add_rms_norm",
            "beam_moe_add_rms_norm_backward_workspace_bytes", "beam_moe_add_rms_norm_backward",
            "beam_moe_gate", "beam_moe_gate_backward", "beam_moe_mx4_quantize",
            "beam_moe_mx4_dequantize", "beam_moe_mx4_linear")

# Scratch size of beam_moe_forward_noalloc (BEAM_MOE_NOALLOC_MAX_BYTES in the header)
NOALLOC_MAX_BYTES = 64 << 20

STAGES = ("router_logits", "select", "perm_hist", "perm_scan", "perm_scatter", "quant_x",
          "gateup", "quant_h", "down", "combine", "bwd_gateup", "bwd_down", "bwd_dx",
          "bwd_token", "bwd_router", "bwd_transpose", "bwd_wgrad")


class BeamMoeConfig(ctypes.Structure):
    _fields_ = [
        ("hidden", ctypes.c_int32),
        ("intermediate", ctypes.c_int32),
        ("n_experts", ctypes.c_int32),
        ("n_group", ctypes.c_int32),
        ("topk_group", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("routed_scaling_factor", ctypes.c_float),
        ("x_dtype", ctypes.c_int32),
        ("w_dtype", ctypes.c_int32),
        ("w_layout", ctypes.c_int32),
    ]


class BeamMoeResidual(ctypes.Structure):
    _fields_ = [
        ("stream_in", ctypes.c_void_p),
        ("norm_weight", ctypes.c_void_p),
        ("norm_eps", ctypes.c_float),
        ("step", ctypes.c_int32),
    ]


class BeamMoeGrads(ctypes.Structure):
    _fields_ = [
        ("dx", ctypes.c_void_p),
        ("d_router_w", ctypes.c_void_p),
        ("d_w_gate", ctypes.c_void_p),
        ("d_w_up", ctypes.c_void_p),
        ("d_w_down", ctypes.c_void_p),
    ]


class BeamMoeNorm(ctypes.Structure):
    _fields_ = [
        ("hidden", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32),
        ("keep", ctypes.c_float),
        ("add", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("quant", ctypes.c_int32),
    ]


class BeamMoeGateConfig(ctypes.Structure):
    _fields_ = [
        ("n_experts", ctypes.c_int32),
        ("n_group", ctypes.c_int32),
        ("topk_group", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("group_score", ctypes.c_int32),
        ("renormalise", ctypes.c_int32),
        ("z_dtype", ctypes.c_int32),
        ("routed_scaling_factor", ctypes.c_float),
    ]


class BeamMoeLinear(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int32),
        ("k", ctypes.c_int32),
        ("x_format", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
    ]


class BeamMoeError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: status {status}: {status_string(status)}")


_lib = None


def lib():
    """The loaded C library (loaded once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m group_limited_routing_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        cfgp = ctypes.POINTER(BeamMoeConfig)
        L.beam_moe_workspace_bytes.argtypes = [cfgp, i32]
        L.beam_moe_workspace_bytes.restype = sz
        L.beam_moe_route.argtypes = [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_route.restype = ctypes.c_int
        L.beam_moe_forward.argtypes = [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                       vp, vp, vp, sz, vp]
        L.beam_moe_forward.restype = ctypes.c_int
        L.beam_moe_forward_residual.argtypes = [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                ctypes.POINTER(BeamMoeResidual), vp, vp, vp, vp,
                                                vp, vp, sz, vp]
        L.beam_moe_forward_residual.restype = ctypes.c_int
        L.beam_moe_status_string.argtypes = [i32]
        L.beam_moe_status_string.restype = ctypes.c_char_p
        L.beam_moe_profile_begin.argtypes = [ctypes.c_uint32]
        L.beam_moe_profile_begin.restype = ctypes.c_int
        L.beam_moe_profile_end.argtypes = [vp, vp]
        L.beam_moe_profile_end.restype = ctypes.c_int
        L.beam_moe_pack_weights.argtypes = [vp, vp, i32, i32, i32, i32, vp]
        L.beam_moe_pack_weights.restype = ctypes.c_int
        L.beam_moe_forward_shard.argtypes = [cfgp, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp,
                                             vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_forward_shard.restype = ctypes.c_int
        L.beam_moe_forward_noalloc.argtypes = [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                               vp, vp, vp, vp, vp]
        L.beam_moe_forward_noalloc.restype = ctypes.c_int
        L.beam_moe_backward_workspace_bytes.argtypes = [cfgp, i32, i32]
        L.beam_moe_backward_workspace_bytes.restype = sz
        L.beam_moe_backward.argtypes = [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                        ctypes.POINTER(BeamMoeGrads), vp, sz, vp]
        L.beam_moe_backward.restype = ctypes.c_int
        L.beam_moe_pack_weights_transposed.argtypes = [vp, vp, i32, i32, i32, i32, vp]
        L.beam_moe_pack_weights_transposed.restype = ctypes.c_int
        L.beam_moe_update_bias.argtypes = [vp, vp, i32, ctypes.c_float, vp]
        L.beam_moe_update_bias.restype = ctypes.c_int
        i64 = ctypes.c_int64
        normp, gatep = ctypes.POINTER(BeamMoeNorm), ctypes.POINTER(BeamMoeGateConfig)
        linp = ctypes.POINTER(BeamMoeLinear)
        L.beam_moe_add_rms_norm.argtypes = [normp, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        L.beam_moe_add_rms_norm_backward_workspace_bytes.argtypes = [normp, i32]
        L.beam_moe_add_rms_norm_backward_workspace_bytes.restype = sz
        L.beam_moe_add_rms_norm_backward.argtypes = [normp, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                                     sz, vp]
        L.beam_moe_gate.argtypes = [gatep, i32, vp, vp, vp, vp, vp, vp, vp]
        L.beam_moe_gate_backward.argtypes = [gatep, i32, vp, vp, vp, vp, vp]
        L.beam_moe_mx4_quantize.argtypes = [vp, i64, i32, i32, i32, vp, vp, vp]
        L.beam_moe_mx4_dequantize.argtypes = [vp, vp, i64, i32, i32, vp, vp]
        L.beam_moe_mx4_linear.argtypes = [linp, i32, vp, vp, vp, vp, vp, vp]
        for name in ("add_rms_norm", "add_rms_norm_backward", "gate", "gate_backward",
                     "mx4_quantize", "mx4_dequantize", "mx4_linear"):
            getattr(L, "beam_moe_" + name).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status):
    return lib().beam_moe_status_string(int(status)).decode()


_X_DTYPES = {torch.float32: BEAM_F32, torch.bfloat16: BEAM_BF16}
# uint8 weight tensors are MXFP4 codes (two E2M1 values per byte)
_W_DTYPES = {torch.bfloat16: BEAM_BF16, torch.float8_e4m3fn: BEAM_FP8_E4M3,
             torch.uint8: BEAM_MXFP4}


def make_config(hidden, intermediate, n_experts=256, n_group=8, topk_group=4, top_k=8,
                routed_scaling_factor=2.5, x_dtype=torch.bfloat16, w_dtype=torch.bfloat16,
                packed=False):
    if x_dtype not in _X_DTYPES or w_dtype not in _W_DTYPES:
        raise TypeError(f"unsupported dtypes x={x_dtype} w={w_dtype}")
    return BeamMoeConfig(hidden, intermediate, n_experts, n_group, topk_group, top_k,
                         routed_scaling_factor, _X_DTYPES[x_dtype], _W_DTYPES[w_dtype],
                         BEAM_LAYOUT_PACKED if packed else BEAM_LAYOUT_ROW_MAJOR)


def pack_weights(w, out=None, stream=None):
    """MFMA-fragment copy of row-major expert weights w [E, R, C] (bf16 or
    float8_e4m3fn; uint8 = MXFP4 codes [E, R, C/2]); pass the result to
    forward(..., packed=True)."""
    if w.dim() != 3 or not w.is_contiguous() or w.dtype not in _W_DTYPES:
        raise ValueError("pack_weights needs a contiguous [E, rows, cols] bf16/fp8/MXFP4 tensor")
    s = _target(w.device, stream)
    if out is None:
        with torch.cuda.stream(s):
            out = torch.empty_like(w)
    E, R, C = w.shape
    if w.dtype == torch.uint8:
        C *= 2  # weights per row
    st = lib().beam_moe_pack_weights(_ptr(w), _ptr(out), E, R, C, _W_DTYPES[w.dtype],
                                     _handle(s))
    if st != BEAM_OK:
        raise BeamMoeError(st, "beam_moe_pack_weights")
    return out


def pack_mx_scales(s, out=None, stream=None):
    """Packed copy of row-major MXFP4 scale bytes s [E, R, C/32] (uint8, E8M0)."""
    if s.dim() != 3 or not s.is_contiguous() or s.dtype != torch.uint8:
        raise ValueError("pack_mx_scales needs a contiguous [E, rows, cols/32] uint8 tensor")
    ts = _target(s.device, stream)
    if out is None:
        with torch.cuda.stream(ts):
            out = torch.empty_like(s)
    E, R, B = s.shape
    st = lib().beam_moe_pack_weights(_ptr(s), _ptr(out), E, R, 32 * B, BEAM_E8M0, _handle(ts))
    if st != BEAM_OK:
        raise BeamMoeError(st, "beam_moe_pack_weights")
    return out


def workspace_bytes(cfg, T):
    return int(lib().beam_moe_workspace_bytes(ctypes.byref(cfg), int(T)))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, shape, dtypes, device):
    if t.shape == shape and t.dtype in dtypes and t.is_contiguous() and t.device == device:
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")


def _workspace(cfg, T, device, workspace):
    """The caller's workspace, or a new one (call it under the target stream)."""
    need = workspace_bytes(cfg, T)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    return workspace


def _target(device, stream):
    """The torch stream a call runs on: ``stream``, else the device's current one."""
    return stream if stream is not None else torch.cuda.current_stream(device)


def _handle(s):
    return ctypes.c_void_p(s.cuda_stream)


def route(x, router_w, expert_bias, *, n_group=8, topk_group=4, top_k=8,
          return_logits=False, return_counts=False, workspace=None, stream=None):
    """Router only. Returns dict(topk_idx [T, k] int32, topk_w [T, k] fp32,
    router_logits [T, E] fp32 or None, expert_counts [E] int32 or None)."""
    T, H = x.shape
    E = router_w.shape[0]
    dev = x.device
    _check(x, "x", (T, H), (torch.float32, torch.bfloat16), dev)
    _check(router_w, "router_w", (E, H), (torch.float32,), dev)
    _check(expert_bias, "expert_bias", (E,), (torch.float32,), dev)
    cfg = make_config(H, 128, E, n_group, topk_group, top_k, 1.0, x.dtype, torch.bfloat16)
    s = _target(dev, stream)
    with torch.cuda.stream(s):
        idx = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        logits = torch.empty((T, E), dtype=torch.float32, device=dev) if return_logits else None
        counts = torch.empty((E,), dtype=torch.int32, device=dev) if return_counts else None
        ws = _workspace(cfg, T, dev, workspace)
    st = lib().beam_moe_route(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w), _ptr(expert_bias),
                              _ptr(idx), _ptr(w), _ptr(logits), _ptr(counts), _ptr(ws),
                              ws.numel(), _handle(s))
    if st != BEAM_OK:
        raise BeamMoeError(st, "beam_moe_route")
    return {"topk_idx": idx, "topk_w": w, "router_logits": logits, "expert_counts": counts}


def forward(x, router_w, expert_bias, w_gate, w_up, w_down, *, scales=None, n_group=8,
            topk_group=4, top_k=8, routed_scaling_factor=2.5, out=None, return_routing=False,
            return_logits=False, workspace=None, stream=None, packed=False):
    """The whole MoE block. ``scales`` = (w_gate_scale, w_up_scale, w_down_scale)
    for fp8 weights (fp32 per row) and MXFP4 weights (uint8 codes, with the
    E8M0 block scales from pack_mx_scales); ``packed`` says the weights come
    from pack_weights() (required for MXFP4).
    Returns out [T, H] (x's dtype), or (out, routing dict) with
    ``return_routing`` or ``return_logits``."""
    return _forward(x, router_w, expert_bias, w_gate, w_up, w_down, None, scales, n_group,
                    topk_group, top_k, routed_scaling_factor, out, return_routing,
                    return_logits, workspace, stream, packed)


def forward_residual(x, router_w, expert_bias, w_gate, w_up, w_down, stream_in, norm_weight,
                     step, *, norm_eps=1e-6, scales=None, n_group=8, topk_group=4, top_k=8,
                     routed_scaling_factor=2.5, out=None, return_routing=False,
                     return_logits=False, workspace=None, stream=None, packed=False):
    """The MoE block and its residual-stream step at sublayer step ``step``:
    returns sqrt((step-1)/step) * stream_in + RMSNorm(block output) / sqrt(step)
    (RMSNorm with gain ``norm_weight`` [H] fp32 and ``norm_eps``), x's dtype.
    ``out`` may be ``stream_in`` itself. Other arguments as for forward()."""
    T, H = x.shape
    _check(stream_in, "stream_in", (T, H), (x.dtype,), x.device)
    _check(norm_weight, "norm_weight", (H,), (torch.float32,), x.device)
    res = BeamMoeResidual(stream_in.data_ptr(), norm_weight.data_ptr(), float(norm_eps),
                          int(step))
    return _forward(x, router_w, expert_bias, w_gate, w_up, w_down, res, scales, n_group,
                    topk_group, top_k, routed_scaling_factor, out, return_routing,
                    return_logits, workspace, stream, packed)


def forward_noalloc(x, router_w, expert_bias, w_gate, w_up, w_down, *, out, scales=None,
                    n_group=8, topk_group=4, top_k=8, routed_scaling_factor=2.5, topk_idx=None,
                    topk_w=None, expert_counts=None, router_logits=None, stream=None,
                    packed=False):
    """The whole MoE block through beam_moe_forward_noalloc: the library's
    static per-GPU scratch instead of a workspace. Every output is the
    caller's (``out`` [T, H] in x's dtype, and optionally topk_idx [T, k]
    int32, topk_w [T, k] fp32, expert_counts [E] int32, router_logits [T, E]
    fp32), so the call allocates nothing. Calls that overlap on one GPU
    race on the shared scratch. Other arguments as for forward()."""
    T, H = x.shape
    E = router_w.shape[0]
    I = w_gate.shape[1]
    dev = x.device
    mx = w_gate.dtype == torch.uint8
    d = 2 if mx else 1
    wdt = (torch.bfloat16, torch.float8_e4m3fn, torch.uint8)
    _check(x, "x", (T, H), (torch.float32, torch.bfloat16), dev)
    _check(router_w, "router_w", (E, H), (torch.float32,), dev)
    _check(expert_bias, "expert_bias", (E,), (torch.float32,), dev)
    _check(w_gate, "w_gate", (E, I, H // d), wdt, dev)
    _check(w_up, "w_up", (E, I, H // d), (w_gate.dtype,), dev)
    _check(w_down, "w_down", (E, H, I // d), (w_gate.dtype,), dev)
    _check(out, "out", (T, H), (x.dtype,), dev)
    for t, name, shape, dt in ((topk_idx, "topk_idx", (T, top_k), torch.int32),
                               (topk_w, "topk_w", (T, top_k), torch.float32),
                               (expert_counts, "expert_counts", (E,), torch.int32),
                               (router_logits, "router_logits", (T, E), torch.float32)):
        if t is not None:
            _check(t, name, shape, (dt,), dev)
    sg = su = sd = None
    if w_gate.dtype in (torch.float8_e4m3fn, torch.uint8):
        if scales is None:
            raise ValueError("quantised weights need (w_gate_scale, w_up_scale, w_down_scale)")
        sg, su, sd = scales
    cfg = make_config(H, I, E, n_group, topk_group, top_k, routed_scaling_factor, x.dtype,
                      w_gate.dtype, packed)
    st = lib().beam_moe_forward_noalloc(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w),
                                        _ptr(expert_bias), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                        _ptr(sg), _ptr(su), _ptr(sd), _ptr(out), _ptr(topk_idx),
                                        _ptr(topk_w), _ptr(expert_counts), _ptr(router_logits),
                                        _handle(_target(dev, stream)))
    if st != BEAM_OK:
        raise BeamMoeError(st, "beam_moe_forward_noalloc")
    return out


def forward_shard(x, router_w, expert_bias, expert_begin, expert_end, w_gate, w_up, w_down, *,
                  scales=None, n_group=8, topk_group=4, top_k=8, routed_scaling_factor=2.5,
                  out=None, return_routing=False, workspace=None, stream=None, packed=False):
    """One expert shard's share of the block: the weights (and scales) hold
    experts [expert_begin, expert_end) only; returns the partial output
    [T, H] (x's dtype) whose sum over a partition of the experts is the block
    output. Other arguments as for forward()."""
    return _forward(x, router_w, expert_bias, w_gate, w_up, w_down, None, scales, n_group,
                    topk_group, top_k, routed_scaling_factor, out, return_routing, False,
                    workspace, stream, packed, shard=(int(expert_begin), int(expert_end)))


def _forward(x, router_w, expert_bias, w_gate, w_up, w_down, res, scales, n_group, topk_group,
             top_k, routed_scaling_factor, out, return_routing, return_logits, workspace,
             stream, packed, shard=None):
    T, H = x.shape
    E = router_w.shape[0]
    n_w = E if shard is None else shard[1] - shard[0]  # experts held by the weight arrays
    I = w_gate.shape[1]
    dev = x.device
    wdt = (torch.bfloat16, torch.float8_e4m3fn, torch.uint8)
    mx = w_gate.dtype == torch.uint8
    d = 2 if mx else 1  # MXFP4: two codes per byte
    _check(x, "x", (T, H), (torch.float32, torch.bfloat16), dev)
    _check(router_w, "router_w", (E, H), (torch.float32,), dev)
    _check(expert_bias, "expert_bias", (E,), (torch.float32,), dev)
    _check(w_gate, "w_gate", (n_w, I, H // d), wdt, dev)
    _check(w_up, "w_up", (n_w, I, H // d), (w_gate.dtype,), dev)
    _check(w_down, "w_down", (n_w, H, I // d), (w_gate.dtype,), dev)
    sg = su = sd = None
    if w_gate.dtype in (torch.float8_e4m3fn, torch.uint8):
        if scales is None:
            raise ValueError("quantised weights need (w_gate_scale, w_up_scale, w_down_scale)")
        sg, su, sd = scales
        if mx:
            _check(sg, "w_gate_scale", (n_w, I, H // 32), (torch.uint8,), dev)
            _check(su, "w_up_scale", (n_w, I, H // 32), (torch.uint8,), dev)
            _check(sd, "w_down_scale", (n_w, H, I // 32), (torch.uint8,), dev)
        else:
            _check(sg, "w_gate_scale", (n_w, I), (torch.float32,), dev)
            _check(su, "w_up_scale", (n_w, I), (torch.float32,), dev)
            _check(sd, "w_down_scale", (n_w, H), (torch.float32,), dev)
    cfg = make_config(H, I, E, n_group, topk_group, top_k, routed_scaling_factor, x.dtype,
                      w_gate.dtype, packed)
    if out is not None:
        _check(out, "out", (T, H), (x.dtype,), dev)
    s = _target(dev, stream)
    idx = w = counts = logits = None
    with torch.cuda.stream(s):
        if out is None:
            out = torch.empty((T, H), dtype=x.dtype, device=dev)
        if return_routing:
            idx = torch.empty((T, top_k), dtype=torch.int32, device=dev)
            w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
            counts = torch.empty((E,), dtype=torch.int32, device=dev)
        if return_logits:
            logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        ws = _workspace(cfg, T, dev, workspace)
    if shard is not None:
        st = lib().beam_moe_forward_shard(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w),
                                          _ptr(expert_bias), shard[0], shard[1], _ptr(w_gate),
                                          _ptr(w_up), _ptr(w_down), _ptr(sg), _ptr(su), _ptr(sd),
                                          _ptr(out), _ptr(idx), _ptr(w), _ptr(counts), _ptr(ws),
                                          ws.numel(), _handle(s))
        where = "beam_moe_forward_shard"
    elif res is None:
        st = lib().beam_moe_forward(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w),
                                    _ptr(expert_bias), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                    _ptr(sg), _ptr(su), _ptr(sd), _ptr(out), _ptr(idx), _ptr(w),
                                    _ptr(counts), _ptr(logits), _ptr(ws), ws.numel(),
                                    _handle(s))
        where = "beam_moe_forward"
    else:
        st = lib().beam_moe_forward_residual(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w),
                                             _ptr(expert_bias), _ptr(w_gate), _ptr(w_up),
                                             _ptr(w_down), _ptr(sg), _ptr(su), _ptr(sd),
                                             ctypes.byref(res), _ptr(out), _ptr(idx), _ptr(w),
                                             _ptr(counts), _ptr(logits), _ptr(ws), ws.numel(),
                                             _handle(s))
        where = "beam_moe_forward_residual"
    if st != BEAM_OK:
        raise BeamMoeError(st, where)
    if return_routing or return_logits:
        return out, {"topk_idx": idx, "topk_w": w, "expert_counts": counts,
                     "router_logits": logits}
    return out


def pack_weights_transposed(w, out=None, stream=None):
    """[E, rows, cols] bf16 expert matrices -> the packed layout of their
    transposes (what backward() takes as w_gate_t, w_up_t, w_down_t)."""
    if w.dtype != torch.bfloat16 or w.dim() != 3 or not w.is_contiguous():
        raise ValueError("expects a contiguous [E, rows, cols] bf16 tensor")
    E, R, C = w.shape
    s = _target(w.device, stream)
    if out is None:
        with torch.cuda.stream(s):
            out = torch.empty((E, C, R), dtype=w.dtype, device=w.device)
    st = lib().beam_moe_pack_weights_transposed(_ptr(w), _ptr(out), E, R, C, BEAM_BF16,
                                                _handle(s))
    if st != BEAM_OK:
        raise BeamMoeError(st, "beam_moe_pack_weights_transposed")
    return out


def backward_workspace_bytes(cfg, T, weight_grads):
    return int(lib().beam_moe_backward_workspace_bytes(ctypes.byref(cfg), int(T), int(bool(weight_grads))))


def backward(x, router_w, expert_bias, w_gate, w_up, w_gate_t, w_up_t, w_down_t, dout, *,
             weight_grads=False, router_grad=True, n_group=8, topk_group=4, top_k=8,
             routed_scaling_factor=2.5, workspace=None, stream=None):
    """Gradients of sum(dout * forward(...)) (bf16 x and dout, packed bf16
    weights: w_gate, w_up from pack_weights, the *_t from
    pack_weights_transposed). Returns dict(dx [T, H] bf16, d_router_w [E, H]
    fp32 or None, d_w_gate / d_w_up [E, I, H] and d_w_down [E, H, I] bf16
    with ``weight_grads``, else None)."""
    T, H = x.shape
    E = router_w.shape[0]
    I = w_gate.shape[1]
    dev = x.device
    _check(x, "x", (T, H), (torch.bfloat16,), dev)
    _check(dout, "dout", (T, H), (torch.bfloat16,), dev)
    _check(router_w, "router_w", (E, H), (torch.float32,), dev)
    _check(expert_bias, "expert_bias", (E,), (torch.float32,), dev)
    for name, t, shape in (("w_gate", w_gate, (E, I, H)), ("w_up", w_up, (E, I, H)),
                           ("w_gate_t", w_gate_t, (E, H, I)), ("w_up_t", w_up_t, (E, H, I)),
                           ("w_down_t", w_down_t, (E, I, H))):
        _check(t, name, shape, (torch.bfloat16,), dev)
    cfg = make_config(H, I, E, n_group, topk_group, top_k, routed_scaling_factor, x.dtype,
                      torch.bfloat16, packed=True)
    need = backward_workspace_bytes(cfg, T, weight_grads)
    if need == 0 and T > 0:
        raise BeamMoeError(BEAM_ERR_CONFIG, "beam_moe_backward_workspace_bytes")
    s = _target(dev, stream)
    dwg = dwu = dwd = None
    with torch.cuda.stream(s):
        dx = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        drw = torch.empty((E, H), dtype=torch.float32, device=dev) if router_grad else None
        if weight_grads:
            dwg = torch.empty((E, I, H), dtype=torch.bfloat16, device=dev)
            dwu = torch.empty((E, I, H), dtype=torch.bfloat16, device=dev)
            dwd = torch.empty((E, H, I), dtype=torch.bfloat16, device=dev)
        if workspace is None or workspace.numel() < need:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    grads = BeamMoeGrads(dx.data_ptr(), drw.data_ptr() if drw is not None else None,
                         dwg.data_ptr() if dwg is not None else None,
                         dwu.data_ptr() if dwu is not None else None,
                         dwd.data_ptr() if dwd is not None else None)
    st = lib().beam_moe_backward(ctypes.byref(cfg), T, _ptr(x), _ptr(router_w), _ptr(expert_bias),
                                 _ptr(w_gate), _ptr(w_up), _ptr(w_gate_t), _ptr(w_up_t),
                                 _ptr(w_down_t), _ptr(dout), ctypes.byref(grads), _ptr(workspace),
                                 workspace.numel(), _handle(s))
    if st != BEAM_OK:
        raise BeamMoeError(st, "beam_moe_backward")
    return {"dx": dx, "d_router_w": drw, "d_w_gate": dwg, "d_w_up": dwu, "d_w_down": dwd}


def update_bias(expert_bias, expert_counts, gamma, stream=None):
    """One load-balancing step of the selection bias, in place:
    b[e] += gamma * sign(mean(counts) - counts[e])."""
    dev = expert_bias.device
    _check(expert_bias, "expert_bias", (256,), (torch.float32,), dev)
    _check(expert_counts, "expert_counts", (256,), (torch.int32,), dev)
    st = lib().beam_moe_update_bias(_ptr(expert_bias), _ptr(expert_counts), 256, float(gamma),
                                    _handle(_target(dev, stream)))
    if st != BEAM_OK:
        raise BeamMoeError(st, "beam_moe_update_bias")
    return expert_bias


# the current stream's handle, without making a torch.cuda.Stream (2 us a call)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _Here:
    """The context of a call on the current device and stream: nothing to switch."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_HERE_CTX = _Here()


def _on(device, stream):
    """The context in which a call allocates and launches: ``stream``, else the
    current stream of the tensors' device (made current if another device is)."""
    if not device.type == "cuda":
        raise ValueError(f"tensors are on {device}, expected a GPU")
    if stream is None:
        return _HERE_CTX if device.index == _current_device() else torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _launch(where, device, fn, *args):
    """Calls the library on the current stream of ``device``."""
    st = fn(*args, _current_stream(device.index))
    if st != BEAM_OK:
        raise BeamMoeError(st, where)


def _p(t):
    return None if t is None else t.data_ptr()


def _sizes(where, *sizes):
    """Sizes that the library takes as 32-bit integers."""
    if max(sizes) > 0x7fffffff:
        raise BeamMoeError(BEAM_ERR_SHAPE, where)


def add_rms_norm(x, norm_weight, *, stream_in=None, keep=1.0, add=1.0, norm_eps=1e-6, quant=None,
                 return_y=True, stream_out=None, stream=None):
    """The residual's addition and the RMS norm of the sum, in one pass:
    s = keep * stream_in + add * x (add * x without ``stream_in``), y = s /
    sqrt(mean(s^2) + norm_eps) * norm_weight, from the unrounded s.

    x and stream_in [T, H] bf16 or fp32, norm_weight [H] fp32. Returns dict(
    stream_out: s in x's dtype (None without stream_in; ``stream_out`` may be
    given, also x or stream_in itself), y: in x's dtype (None without
    ``return_y``), q, q_scale: with ``quant`` the E4M3 codes of y and their
    scales, "row": fp32 [T], amax / 448, or "block": E8M0 bytes [T, H / 32]
    (uint8), for mx4_linear(); else None)."""
    T, H = x.shape
    dev = x.device
    if quant not in _QUANTS:
        raise ValueError(f"quant is {quant!r}, expected None, 'row' or 'block'")
    _check(x, "x", (T, H), _FLOATS, dev)
    _check(norm_weight, "norm_weight", (H,), _F32, dev)
    for t, name in ((stream_in, "stream_in"), (stream_out, "stream_out")):
        if t is not None:
            _check(t, name, (T, H), (x.dtype,), dev)
    _sizes("beam_moe_add_rms_norm", T, H)
    cfg = BeamMoeNorm(H, _X_DTYPES[x.dtype], keep, add, norm_eps, _QUANTS[quant])
    y = q = scale = None
    with _on(dev, stream):
        if stream_out is None and stream_in is not None:
            stream_out = torch.empty_like(x)
        if return_y:
            y = torch.empty_like(x)
        if quant is not None:
            q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
            scale = (torch.empty(T, dtype=torch.float32, device=dev) if quant == "row" else
                     torch.empty(T, H // 32, dtype=torch.uint8, device=dev))
        _launch("beam_moe_add_rms_norm", dev, lib().beam_moe_add_rms_norm, ctypes.byref(cfg), T,
                _p(x), _p(stream_in), _p(norm_weight), _p(stream_out), _p(y), _p(q), _p(scale))
    return {"stream_out": stream_out, "y": y, "q": q, "q_scale": scale}


def add_rms_norm_backward(dy, s, norm_weight, *, d_stream_out=None, keep=1.0, add=1.0,
                          norm_eps=1e-6, stream_grad=True, weight_grad=True, workspace=None,
                          stream=None):
    """Gradients of add_rms_norm() from its stored sum ``s`` (stream_out; x
    itself without stream_in and with add = 1), the gradient ``dy`` of y and,
    where the sum is used further, ``d_stream_out`` of the sum. Returns dict(
    dx, d_stream_in: [T, H] in dy's dtype (d_stream_in is None without
    ``stream_grad``, and is dx itself where keep == add), d_norm_weight: [H]
    fp32, None without ``weight_grad``)."""
    T, H = dy.shape
    dev = dy.device
    _check(dy, "dy", (T, H), _FLOATS, dev)
    _check(s, "s", (T, H), (dy.dtype,), dev)
    _check(norm_weight, "norm_weight", (H,), _F32, dev)
    if d_stream_out is not None:
        _check(d_stream_out, "d_stream_out", (T, H), (dy.dtype,), dev)
    _sizes("beam_moe_add_rms_norm_backward", T, H)
    cfg = BeamMoeNorm(H, _X_DTYPES[dy.dtype], keep, add, norm_eps, BEAM_QUANT_NONE)
    d_in = dw = None
    with _on(dev, stream):
        dx = torch.empty_like(dy)
        if stream_grad and keep != add:
            d_in = torch.empty_like(dy)
        if weight_grad:
            # no rows: the sum over them is 0
            dw = (torch.empty if T else torch.zeros)(H, dtype=torch.float32, device=dev)
            need = int(lib().beam_moe_add_rms_norm_backward_workspace_bytes(ctypes.byref(cfg), T))
            workspace = _scratch(workspace, need, dev)
        else:
            workspace = None
        _launch("beam_moe_add_rms_norm_backward", dev, lib().beam_moe_add_rms_norm_backward,
                ctypes.byref(cfg), T, _p(dy), _p(s), _p(norm_weight), _p(d_stream_out), _p(dx),
                _p(d_in), _p(dw), _p(workspace), 0 if workspace is None else workspace.numel())
    return {"dx": dx, "d_stream_in": dx if stream_grad and d_in is None else d_in,
            "d_norm_weight": dw}


def gate(logits, *, top_k, expert_bias=None, score="sigmoid", n_group=1, topk_group=1,
         group_score="top2", renormalise=True, routed_scaling_factor=1.0, valid=None,
         return_counts=False, stream=None):
    """Routing of given logits [T, E] (bf16 or fp32, E <= 1024): scores by
    ``score`` ("sigmoid" or "softmax" over all experts), keys = scores +
    ``expert_bias`` [E] fp32, the ``topk_group`` of ``n_group`` groups with the
    best ``group_score`` ("top2": the sum of the two largest keys, "max"), the
    ``top_k`` largest keys inside them, weights = routed_scaling_factor * score
    (over the chosen scores' sum with ``renormalise``). ``valid`` [T] bool marks
    the tokens that are none of the padding. Returns dict(topk_idx [T, k] int32
    (-1 for padding), topk_w [T, k] fp32, expert_counts [E] int32 or None)."""
    T, E = logits.shape
    dev = logits.device
    cfg = _gate_config(logits, top_k, score, n_group, topk_group, group_score, renormalise,
                       routed_scaling_factor)
    if expert_bias is not None:
        _check(expert_bias, "expert_bias", (E,), _F32, dev)
    if valid is not None:
        _check(valid, "valid", (T,), (torch.bool, torch.uint8), dev)
    counts = None
    with _on(dev, stream):
        idx = torch.empty(T, top_k, dtype=torch.int32, device=dev)
        w = torch.empty(T, top_k, dtype=torch.float32, device=dev)
        if return_counts:
            counts = (torch.empty if T else torch.zeros)(E, dtype=torch.int32, device=dev)
        _launch("beam_moe_gate", dev, lib().beam_moe_gate, ctypes.byref(cfg), T, _p(logits),
                _p(expert_bias), _p(valid), _p(idx), _p(w), _p(counts))
    return {"topk_idx": idx, "topk_w": w, "expert_counts": counts}


def gate_backward(d_topk_w, logits, topk_idx, *, score="sigmoid", renormalise=True,
                  routed_scaling_factor=1.0, stream=None):
    """Gradient of the logits [T, E] (in their dtype) from the gradient
    ``d_topk_w`` [T, k] fp32 of gate()'s weights and its ``topk_idx`` (a slot
    with an index outside [0, E), as padding has, is empty)."""
    T, E = logits.shape
    dev = logits.device
    k = d_topk_w.shape[-1]
    cfg = _gate_config(logits, k, score, 1, 1, "max", renormalise, routed_scaling_factor)
    _check(d_topk_w, "d_topk_w", (T, k), _F32, dev)
    _check(topk_idx, "topk_idx", (T, k), (torch.int32,), dev)
    with _on(dev, stream):
        dz = torch.empty_like(logits)
        _launch("beam_moe_gate_backward", dev, lib().beam_moe_gate_backward, ctypes.byref(cfg), T,
                _p(d_topk_w), _p(logits), _p(topk_idx), _p(dz))
    return dz


def _gate_config(logits, top_k, score, n_group, topk_group, group_score, renormalise, rsf):
    if score not in _SCORES or group_score not in _GROUP_SCORES:
        raise ValueError(f"score {score!r} / group_score {group_score!r}: expected one of "
                         f"{tuple(_SCORES)} / {tuple(_GROUP_SCORES)}")
    _check(logits, "logits", logits.shape, _FLOATS, logits.device)
    _sizes("beam_moe_gate", *logits.shape, top_k, n_group, topk_group)
    # before outputs of top_k columns are allocated; the library checks the rest
    if not 1 <= top_k <= logits.shape[1] or n_group < 1 or topk_group < 1:
        raise BeamMoeError(BEAM_ERR_CONFIG, "beam_moe_gate")
    return BeamMoeGateConfig(logits.shape[1], n_group, topk_group, top_k, _SCORES[score],
                             _GROUP_SCORES[group_score], int(bool(renormalise)),
                             _X_DTYPES[logits.dtype], rsf)


def mx4_quantize(x, *, packed=False, stream=None):
    """MXFP4 of rows x [..., C] (bf16 or fp32, C a multiple of 32): (codes
    [..., C / 2], scales [..., C / 32]), uint8, row-major; what mx4_linear()
    takes for weights or rows. With ``packed``, x [E, R, C] are expert weights
    (R a multiple of 16, C of 512) and both come in the packed layout, as from
    pack_weights() and pack_mx_scales(): forward(..., packed=True) takes them."""
    dev = x.device
    if x.dim() < 1 or (packed and x.dim() != 3):
        raise ValueError("mx4_quantize needs rows [..., C], with packed [E, R, C]")
    _check(x, "x", x.shape, _FLOATS, dev)
    C = x.shape[-1]
    if C == 0 or C % 32:
        raise ValueError(f"x has rows of {C} values, expected a multiple of 32")
    if packed and x.shape[1] % 16:
        raise ValueError(f"x has {x.shape[1]} rows per expert, expected a multiple of 16")
    _sizes("beam_moe_mx4_quantize", C)
    with _on(dev, stream):
        codes = torch.empty(*x.shape[:-1], C // 2, dtype=torch.uint8, device=dev)
        scales = torch.empty(*x.shape[:-1], C // 32, dtype=torch.uint8, device=dev)
        _launch("beam_moe_mx4_quantize", dev, lib().beam_moe_mx4_quantize, _p(x), x.numel() // C,
                C, _X_DTYPES[x.dtype], BEAM_LAYOUT_PACKED if packed else BEAM_LAYOUT_ROW_MAJOR,
                _p(codes), _p(scales))
    return codes, scales


def mx4_dequantize(codes, scales, *, dtype=torch.bfloat16, stream=None):
    """The values [..., C] (bf16 or fp32, exact) of row-major MXFP4 codes
    [..., C / 2] and scales [..., C / 32]."""
    dev = codes.device
    if dtype not in _X_DTYPES:
        raise ValueError(f"dtype is {dtype}, expected one of {_FLOATS}")
    C = 2 * codes.shape[-1]
    if C == 0 or C % 32:
        raise ValueError(f"codes have rows of {C} values, expected a multiple of 32")
    _check(codes, "codes", codes.shape, _U8, dev)
    _check(scales, "scales", (*codes.shape[:-1], C // 32), _U8, dev)
    _sizes("beam_moe_mx4_dequantize", C)
    with _on(dev, stream):
        out = torch.empty(*codes.shape[:-1], C, dtype=dtype, device=dev)
        _launch("beam_moe_mx4_dequantize", dev, lib().beam_moe_mx4_dequantize, _p(codes),
                _p(scales), out.numel() // C, C, _X_DTYPES[dtype], _p(out))
    return out


def mx4_linear(x, x_scale, w, w_scale, *, out_dtype=torch.bfloat16, out=None, stream=None):
    """x W^T with MXFP4 weights (row-major codes ``w`` [N, K / 2] and scales
    ``w_scale`` [N, K / 32], as from mx4_quantize()). The token rows ``x`` are
    E4M3 codes [T, K] (float8_e4m3fn) with ``x_scale`` fp32 [T] or E8M0 bytes
    [T, K / 32], as from add_rms_norm(quant="row" / "block"), or MXFP4 codes
    [T, K / 2] (uint8) with E8M0 bytes [T, K / 32]. Returns ``out`` [T, N]
    (``out_dtype``, bf16 or fp32)."""
    T = x.shape[0]
    N, K = w.shape[0], 2 * w.shape[1]
    dev = x.device
    _check(w, "w", (N, K // 2), _U8, dev)
    _check(w_scale, "w_scale", (N, K // 32), _U8, dev)
    if x.dtype == torch.uint8:
        fmt = BEAM_X_MXFP4
        _check(x, "x", (T, K // 2), _U8, dev)
    else:
        fmt = BEAM_X_E4M3_ROW if x_scale.dtype == torch.float32 else BEAM_X_E4M3_BLOCK
        _check(x, "x", (T, K), (torch.float8_e4m3fn, torch.uint8), dev)
    if fmt == BEAM_X_E4M3_ROW:
        _check(x_scale, "x_scale", (T,), _F32, dev)
    else:
        _check(x_scale, "x_scale", (T, K // 32), _U8, dev)
    if out is not None:
        out_dtype = out.dtype
        _check(out, "out", (T, N), _FLOATS, dev)
    if out_dtype not in _X_DTYPES:
        raise ValueError(f"out_dtype is {out_dtype}, expected one of {_FLOATS}")
    _sizes("beam_moe_mx4_linear", T, N, K)
    cfg = BeamMoeLinear(N, K, fmt, _X_DTYPES[out_dtype])
    with _on(dev, stream):
        if out is None:
            out = torch.empty(T, N, dtype=out_dtype, device=dev)
        _launch("beam_moe_mx4_linear", dev, lib().beam_moe_mx4_linear, ctypes.byref(cfg), T, _p(x),
                _p(x_scale), _p(w), _p(w_scale), _p(out))
    return out


def _scratch(workspace, need, device):
    """The caller's workspace if it is large enough, else a new one."""
    if workspace is None or workspace.numel() < need:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    _check(workspace, "workspace", workspace.shape, _U8, device)
    return workspace


_FLOATS, _F32, _U8 = tuple(_X_DTYPES), (torch.float32,), (torch.uint8,)
_QUANTS = {None: BEAM_QUANT_NONE, "row": BEAM_QUANT_ROW, "block": BEAM_QUANT_BLOCK}
_SCORES = {"sigmoid": BEAM_SCORE_SIGMOID, "softmax": BEAM_SCORE_SOFTMAX}
_GROUP_SCORES = {"top2": BEAM_GROUP_TOP2, "max": BEAM_GROUP_MAX}


def profile_begin(stages=STAGES):
    """Start timing the named stages of every following route/forward call."""
    mask = 0
    for name in stages:
        mask |= 1 << STAGES.index(name)
    st = lib().beam_moe_profile_begin(mask)
    if st != BEAM_OK:
        raise BeamMoeError(st, "beam_moe_profile_begin")


def profile_end():
    """Stop timing; returns {stage: (total_ms, launches)} for timed stages."""
    n = len(STAGES)
    tot = (ctypes.c_float * n)()
    cnt = (ctypes.c_int32 * n)()
    st = lib().beam_moe_profile_end(ctypes.cast(tot, ctypes.c_void_p), ctypes.cast(cnt, ctypes.c_void_p))
    if st != BEAM_OK:
        raise BeamMoeError(st, "beam_moe_profile_end")
    return {STAGES[i]: (float(tot[i]), int(cnt[i])) for i in range(n) if cnt[i] > 0}
