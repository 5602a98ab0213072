"""ctypes binding of libmoe_int4.so (include/moe_int4.h).

Argument marshalling only: every step of the layer runs in the HIP library.
Tensors are torch tensors on the current HIP device; bf16 data may be passed
as torch.bfloat16 or as int16/uint16 bit patterns.  Work is enqueued on
torch's current stream unless a stream is given.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_int4.so")

OK, EINVAL, EALIGN, EWORKSPACE, ELAUNCH, EDEVICE = 0, -1, -2, -3, -4, -5

_c_void_p = ctypes.c_void_p
_c_i32 = ctypes.c_int32


class MoeShape(ctypes.Structure):
    _fields_ = [("tokens", _c_i32), ("hidden", _c_i32), ("experts", _c_i32),
                ("inter", _c_i32), ("group", _c_i32), ("top_k", _c_i32)]


class MoeSharedInt6(ctypes.Structure):
    _fields_ = [("gate_w", _c_void_p), ("w13_packed", _c_void_p), ("w13_scales", _c_void_p),
                ("w2_packed", _c_void_p), ("w2_scales", _c_void_p),
                ("inter", _c_i32), ("group", _c_i32)]


class MoeInt8Epilogue(ctypes.Structure):
    _fields_ = [("bias", _c_void_p), ("residual", _c_void_p), ("residual_stride", ctypes.c_int64),
                ("bias_type", _c_i32), ("residual_type", _c_i32), ("activation", _c_i32)]


class MoeLogitsRules(ctypes.Structure):
    _fields_ = ([(f, _c_void_p) for f in ("history", "history_lengths", "prompt_lengths", "repetition",
                                          "frequency", "presence", "bias_ids", "bias_values",
                                          "bias_lengths", "temperature", "mask")]
                + [(f, ctypes.c_int64) for f in ("history_stride", "bias_stride", "mask_stride")]
                + [("history_width", _c_i32), ("bias_width", _c_i32)])


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"moe_int4 error {code}: {msg}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load the built library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m quantized_moe_router_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = _c_void_p
        L.moe_int4_workspace_bytes.argtypes = [P, P, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_int4_route.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_int4_experts.argtypes = [P] * 11 + [ctypes.c_size_t, P]
        L.moe_int4_forward.argtypes = [P] * 6 + [_c_i32, P, P, P, P, ctypes.c_size_t, P]
        L.moe_int4_forward_traced.argtypes = [P] * 6 + [_c_i32, P, P, P, P, ctypes.c_size_t, P, P]
        L.moe_int4_forward_noalloc.argtypes = [P] * 6 + [_c_i32, P, P, P, P, P]
        L.moe_int4_quantize.argtypes = [P, _c_i32, _c_i32, _c_i32, P, P, P]
        L.moe_int8_linear_workspace_bytes.argtypes = [_c_i32] * 4 + [ctypes.POINTER(ctypes.c_size_t)]
        L.moe_int8_linear.argtypes = [P, P, P] + [_c_i32] * 4 + [P, P, ctypes.c_size_t, P]
        c_i64 = ctypes.c_int64
        L.moe_int8_linear_fused_workspace_bytes.argtypes = [_c_i32] * 4 + [ctypes.POINTER(ctypes.c_size_t)]
        L.moe_int8_linear_fused.argtypes = [P, c_i64, P, P] + [_c_i32] * 4 + [P, P, _c_i32, c_i64, P,
                                                                             ctypes.c_size_t, P]
        L.moe_int4_logits_process.argtypes = [P, _c_i32, c_i64, _c_i32, _c_i32, P, P, _c_i32, c_i64, P]
        L.moe_int4_last_error.restype = ctypes.c_char_p
        L.moe_int4_version.restype = ctypes.c_char_p
        for f in ("moe_int4_workspace_bytes", "moe_int4_route", "moe_int4_experts", "moe_int4_forward",
                  "moe_int4_forward_traced", "moe_int4_forward_noalloc", "moe_int4_quantize",
                  "moe_int8_linear_workspace_bytes", "moe_int8_linear",
                  "moe_int8_linear_fused_workspace_bytes", "moe_int8_linear_fused",
                  "moe_int4_logits_process"):
            getattr(L, f).restype = _c_i32
        _lib = L
    return _lib


EXPORTED = ("moe_int4_workspace_bytes", "moe_int4_route", "moe_int4_experts",
            "moe_int4_forward", "moe_int4_forward_traced", "moe_int4_forward_noalloc",
            "moe_int4_quantize",
            "moe_int8_linear_workspace_bytes", "moe_int8_linear",
            "moe_int8_linear_fused_workspace_bytes", "moe_int8_linear_fused",
            "moe_int4_logits_process",
            "moe_int4_last_error", "moe_int4_version")


def _check(rc: int):
    if rc != OK:
        raise MoeError(rc, lib().moe_int4_last_error().decode())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def make_shape(tokens, hidden, experts, inter, top_k, group=128) -> MoeShape:
    return MoeShape(tokens, hidden, experts, inter, group, top_k)


def make_shared(sh: dict | None) -> MoeSharedInt6 | None:
    """sh: dict of device tensors gate_w, w13_packed, w13_scales, w2_packed, w2_scales."""
    if sh is None:
        return None
    inter = sh["w2_packed"].shape[1] // 6 * 32
    return MoeSharedInt6(_ptr(sh["gate_w"]), _ptr(sh["w13_packed"]), _ptr(sh["w13_scales"]),
                         _ptr(sh["w2_packed"]), _ptr(sh["w2_scales"]), inter, int(sh.get("group", 64)))


def workspace_bytes(shape: MoeShape, shared: MoeSharedInt6 | None = None) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_int4_workspace_bytes(ctypes.byref(shape),
                                          ctypes.byref(shared) if shared else None, ctypes.byref(n)))
    return n.value


# Workspace control prefix (include/moe_int4.h): zero between calls, except
# the sticky status word at WS_STATUS_OFFSET.
WS_PREFIX_BYTES = 65792
WS_STATUS_OFFSET = 65536
STATUS_KEY_WAIT, STATUS_ROUTE_WAIT, STATUS_H_WAIT = 1, 2, 4


def new_workspace(shape: MoeShape, shared: MoeSharedInt6 | None = None, device="cuda"):
    """A zero-filled workspace (the library keeps its counters at zero after each call)."""
    import torch
    return torch.zeros(workspace_bytes(shape, shared), dtype=torch.uint8, device=device)


def workspace_status(workspace) -> int:
    """The sticky status word of a workspace (reads device memory: call after
    the stream has completed)."""
    w = workspace[WS_STATUS_OFFSET:WS_STATUS_OFFSET + 4].cpu().numpy()
    return int(w.view("<u4")[0])


def workspace_prefix_clean(workspace) -> bool:
    """Whether the control prefix is back at zero, status word included."""
    return not bool(workspace[:WS_PREFIX_BYTES].any().item())


def moe_int4_route(x, router_w, shape: MoeShape, topk_ids, topk_w, expert_counts,
                   expert_offsets, sorted_slots, workspace, stream=None):
    _check(lib().moe_int4_route(_ptr(x), _ptr(router_w), ctypes.byref(shape), _ptr(topk_ids),
                                _ptr(topk_w), _ptr(expert_counts), _ptr(expert_offsets),
                                _ptr(sorted_slots), _ptr(workspace), workspace.numel(),
                                _stream(stream)))


def moe_int4_experts(x, topk_ids, topk_w, w13_packed, w13_scales, w2_packed, w2_scales,
                     shape: MoeShape, shared: MoeSharedInt6 | None, out, workspace, stream=None):
    _check(lib().moe_int4_experts(_ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w13_packed),
                                  _ptr(w13_scales), _ptr(w2_packed), _ptr(w2_scales),
                                  ctypes.byref(shape), ctypes.byref(shared) if shared else None,
                                  _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)))


def moe_int4_forward(x, router_w, w13_packed, w13_scales, w2_packed, w2_scales, top_k: int, out,
                     shape: MoeShape, shared: MoeSharedInt6 | None, workspace, stream=None):
    _check(lib().moe_int4_forward(_ptr(x), _ptr(router_w), _ptr(w13_packed), _ptr(w13_scales),
                                  _ptr(w2_packed), _ptr(w2_scales), int(top_k), _ptr(out),
                                  ctypes.byref(shape), ctypes.byref(shared) if shared else None,
                                  _ptr(workspace), workspace.numel(), _stream(stream)))


def moe_int4_forward_traced(x, router_w, w13_packed, w13_scales, w2_packed, w2_scales, top_k: int,
                            out, shape: MoeShape, shared: MoeSharedInt6 | None, workspace, events,
                            stream=None):
    """events: four hipEvent_t handles (ints), or four torch.cuda.Event(enable_timing=True)
    already recorded once (torch creates the underlying event lazily); they are
    re-recorded between the stages."""
    arr = (ctypes.c_void_p * 4)(*[e.cuda_event if hasattr(e, "cuda_event") else int(e) for e in events])
    if not all(arr):
        raise ValueError("record each torch.cuda.Event once before passing it (lazy creation)")
    _check(lib().moe_int4_forward_traced(_ptr(x), _ptr(router_w), _ptr(w13_packed), _ptr(w13_scales),
                                         _ptr(w2_packed), _ptr(w2_scales), int(top_k), _ptr(out),
                                         ctypes.byref(shape), ctypes.byref(shared) if shared else None,
                                         _ptr(workspace), workspace.numel(), _stream(stream), arr))


NOALLOC_SCRATCH_BYTES = 64 << 20   # MOE_INT4_NOALLOC_SCRATCH_BYTES


def moe_int4_forward_noalloc(x, router_w, w13_packed, w13_scales, w2_packed, w2_scales, top_k: int,
                             out, shape: MoeShape, shared: MoeSharedInt6 | None, status=None,
                             stream=None):
    """moe_int4_forward without a workspace (the library's static per-device
    scratch); status: optional device uint32 tensor that failed waits OR into."""
    _check(lib().moe_int4_forward_noalloc(_ptr(x), _ptr(router_w), _ptr(w13_packed), _ptr(w13_scales),
                                          _ptr(w2_packed), _ptr(w2_scales), int(top_k), _ptr(out),
                                          ctypes.byref(shape), ctypes.byref(shared) if shared else None,
                                          _ptr(status), _stream(stream)))


def moe_int4_quantize(w, rows: int, cols: int, packed, scales, group: int = 128, stream=None):
    """w bf16 [rows, cols] (device) -> packed int32 [rows, cols/8], scales bf16 [rows, cols/group]."""
    _check(lib().moe_int4_quantize(_ptr(w), int(rows), int(cols), int(group), _ptr(packed),
                                   _ptr(scales), _stream(stream)))


def moe_int8_linear_workspace_bytes(tokens: int, n: int, k: int, group: int) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().moe_int8_linear_workspace_bytes(int(tokens), int(n), int(k), int(group), ctypes.byref(b)))
    return b.value


def moe_int8_linear(x, w_packed, w_scales, tokens: int, n: int, k: int, group: int, out,
                    workspace=None, stream=None):
    """x bf16 [tokens, k], w_packed int32 [n, k/4], w_scales bf16 [n, k/group] ->
    out bf16 [tokens, n] (device tensors; workspace uint8, may be None when the
    shape needs none)."""
    _check(lib().moe_int8_linear(_ptr(x), _ptr(w_packed), _ptr(w_scales), int(tokens), int(n), int(k),
                                 int(group), _ptr(out), _ptr(workspace),
                                 0 if workspace is None else workspace.numel(), _stream(stream)))


# Element types (MOE_TYPE_*) and activations (MOE_ACT_*).
TYPE_BF16, TYPE_F16, TYPE_F32 = 0, 1, 2
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "sigmoid": 5}
_types = None


def type_code(dtype) -> int:
    """MOE_TYPE_* of a torch dtype (int16 and uint16 hold bf16 bit patterns)."""
    global _types
    if _types is None:
        import torch
        _types = {torch.bfloat16: TYPE_BF16, torch.int16: TYPE_BF16, torch.uint16: TYPE_BF16,
                  torch.float16: TYPE_F16, torch.float32: TYPE_F32}
    code = _types.get(dtype)
    if code is None:
        raise ValueError(f"{dtype} is none of bfloat16 (or its bits in int16, uint16), float16, float32")
    return code


def row_stride(t, name: str, rows: int, cols: int) -> int:
    """The row stride of a matrix argument of `rows` x `cols`, its elements
    consecutive in a row."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} is {tuple(t.shape)}, expected ({rows}, {cols})")
    stride = t.stride()
    if stride[1] != 1 and cols > 1:
        raise ValueError(f"{name}: the elements of a row must be consecutive")
    return stride[0]


def device_index(t, name: str, index: int | None = None) -> int:
    """The index of the GPU that holds t (`index`, where one is expected): the
    library dereferences t's address there."""
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name} must be on the GPU, it is on {t.device}")
    if index is not None and i != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    return i


def _current_device() -> int:
    import torch
    return torch.cuda.current_device()


def _device(index: int):
    import torch
    return torch.cuda.device(index)


def _stream_on(stream, index: int) -> int | None:
    """The given stream, or torch's current one on a device (its handle alone:
    building the stream object costs as much as a launch's other checks)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def moe_int8_linear_fused_workspace_bytes(tokens: int, n: int, k: int, group: int) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().moe_int8_linear_fused_workspace_bytes(int(tokens), int(n), int(k), int(group), ctypes.byref(b)))
    return b.value


def check_int8_weights(w_packed, w_scales, n: int, k: int, group: int):
    """The codes and scales of an [n, k] INT8 weight: the library reads that
    many of them from their addresses on."""
    import torch
    if w_packed.dtype != torch.int32 or w_packed.shape != (n, k // 4) or not w_packed.is_contiguous():
        raise ValueError(f"w_packed is {w_packed.dtype} {tuple(w_packed.shape)}, expected contiguous int32 "
                         f"({n}, {k} / 4)")
    if group <= 0 or type_code(w_scales.dtype) != TYPE_BF16 or w_scales.shape != (n, k // group) \
            or not w_scales.is_contiguous():
        raise ValueError(f"w_scales is {w_scales.dtype} {tuple(w_scales.shape)}, expected contiguous bfloat16 "
                         f"({n}, {k} / {group})")


def moe_int8_linear_fused(x, w_packed, w_scales, tokens: int, n: int, k: int, group: int, out,
                          bias=None, residual=None, activation: str = "none", workspace=None, stream=None):
    """out [tokens, n] = residual + act(x W^T + bias): x bf16 [tokens, k],
    w_packed int32 [n, k/4], w_scales bf16 [n, k/group], bias [n], residual
    [tokens, n]; bias, residual and out in bf16, fp16 or fp32, the rows of x,
    residual and out possibly inside wider ones.  activation: a key of
    ACTIVATIONS.  workspace: uint8, may be None when the shape needs none."""
    check_int8_weights(w_packed, w_scales, n, k, group)
    int8_linear_fused(x, w_packed, w_scales, tokens, n, k, group, out, bias, residual, activation, workspace, stream)


def int8_linear_fused(x, w_packed, w_scales, tokens: int, n: int, k: int, group: int, out, bias, residual,
                      activation: str, workspace, stream=None):
    """moe_int8_linear_fused on weights that have passed check_int8_weights
    (layer.Int8Linear checks its own once)."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation {activation!r} is none of {', '.join(ACTIVATIONS)}")
    if type_code(x.dtype) != TYPE_BF16:
        raise ValueError(f"x is {x.dtype}, expected bfloat16 (or its bits)")
    x_stride, out_stride = row_stride(x, "x", tokens, k), row_stride(out, "out", tokens, n)
    out_type = type_code(out.dtype)
    e = MoeInt8Epilogue(None, None, 0, 0, 0, act)
    if bias is not None:
        if bias.shape != (n,) or not bias.is_contiguous():
            raise ValueError(f"bias is {tuple(bias.shape)}, expected ({n},), contiguous")
        e.bias, e.bias_type = bias.data_ptr(), type_code(bias.dtype)
    if residual is not None:
        e.residual_stride = row_stride(residual, "residual", tokens, n)
        e.residual, e.residual_type = residual.data_ptr(), type_code(residual.dtype)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError(f"workspace is {tuple(workspace.shape)} with strides {workspace.stride()}, expected contiguous")
    index = device_index(x, "x")
    if index != _current_device():   # its stream, and its device for the launch
        with _device(index):
            return int8_linear_fused(x, w_packed, w_scales, tokens, n, k, group, out, bias, residual, activation,
                                     workspace, stream)
    for name, t in (("w_packed", w_packed), ("w_scales", w_scales), ("out", out), ("bias", bias),
                    ("residual", residual), ("workspace", workspace)):
        if t is not None:
            device_index(t, name, index)
    rc = lib().moe_int8_linear_fused(x.data_ptr(), x_stride, w_packed.data_ptr(), w_scales.data_ptr(), tokens, n, k,
                                     group, ctypes.byref(e), out.data_ptr(), out_type, out_stride,
                                     _ptr(workspace), 0 if workspace is None else workspace.nbytes,
                                     _stream_on(stream, index))
    if rc:
        _check(rc)


def moe_int4_logits_process(logits, rules: MoeLogitsRules, out, stream=None):
    """out = the rules applied to logits (both [rows, vocab] in bf16, fp16 or
    fp32, rows possibly inside wider ones; out may be logits).  rules: device
    addresses of the tables, which the caller keeps alive (layer.LogitsRules
    does, and checks their shapes)."""
    if logits.dim() != 2:
        raise ValueError(f"logits is {tuple(logits.shape)}, expected [rows, vocab]")
    rows, vocab = logits.shape
    stride, out_stride = row_stride(logits, "logits", rows, vocab), row_stride(out, "out", rows, vocab)
    in_type, out_type = type_code(logits.dtype), type_code(out.dtype)
    index = device_index(logits, "logits")
    device_index(out, "out", index)
    if index != _current_device():
        with _device(index):
            return moe_int4_logits_process(logits, rules, out, stream)
    rc = lib().moe_int4_logits_process(logits.data_ptr(), in_type, stride, rows, vocab, ctypes.byref(rules),
                                       out.data_ptr(), out_type, out_stride, _stream_on(stream, index))
    if rc:
        _check(rc)


def version() -> str:
    return lib().moe_int4_version().decode()
