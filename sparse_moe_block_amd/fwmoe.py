"""Python binding of libfwmoe.so: the C ABI of include/fwmoe.h, one function per
entry point with the same name.  Argument marshalling only -- torch tensors (or
None) become device pointers, the stream defaults to torch's current stream --
and a non-zero return code raises FwMoeError.  Every step of the layer runs in
the HIP kernels of the library; there is no other implementation behind these
calls, and a missing library is an error."""

import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfwmoe.so")

FW_OK, FW_EINVAL, FW_EUNSUPPORTED, FW_EWORKSPACE, FW_EALIGN, FW_EHIP = 0, -1, -2, -3, -4, -5
FW_STATUS_BAD_EXPERT_ID, FW_STATUS_BAD_OFFSETS, FW_STATUS_BAD_PAIR, FW_STATUS_RANGE = 1, 2, 4, 8
FW_F32, FW_BF16 = 0, 1
FW_Q8_0, FW_Q4_0, FW_Q4_K, FW_Q6_K, FW_MXFP4 = 0, 1, 2, 3, 4
FW_SOFTMAX_RENORM, FW_SIGMOID_RENORM = 0, 1
FW_PATH_AUTO, FW_PATH_GEMV, FW_PATH_GEMM = 0, 1, 2
FW_N_STAGE_EVENTS = 6
FW_NOALLOC_SCRATCH_BYTES = 64 << 20

DTYPES = {"f32": FW_F32, "bf16": FW_BF16}
QTYPES = {"q8_0": FW_Q8_0, "q4_0": FW_Q4_0, "q4_k": FW_Q4_K, "q6_k": FW_Q6_K,
          "mxfp4": FW_MXFP4}
SCORES = {"softmax": FW_SOFTMAX_RENORM, "sigmoid": FW_SIGMOID_RENORM}
PATHS = {"auto": FW_PATH_AUTO, "gemv": FW_PATH_GEMV, "gemm": FW_PATH_GEMM}
FW_ACT_NONE, FW_ACT_MXFP8, FW_ACT_INT8 = 0, 1, 2
ACT_QUANTS = {"none": FW_ACT_NONE, "mxfp8": FW_ACT_MXFP8, "int8": FW_ACT_INT8}
FW_FN_NONE, FW_FN_SILU, FW_FN_GELU_TANH, FW_FN_RELU = 0, 1, 2, 3
FNS = {"none": FW_FN_NONE, "silu": FW_FN_SILU, "gelu_tanh": FW_FN_GELU_TANH, "relu": FW_FN_RELU}


class FwMoeError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} returned {code} ({status_string(code)})")
        self.code = code


class fw_moe_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "hidden", "n_experts", "top_k", "ffn", "shared_ffn", "act_dtype", "router_dtype",
        "expert_q", "shared_q", "score", "path", "act_quant")]


def make_desc(hidden, n_experts, top_k, ffn, shared_ffn=0, act_dtype="bf16",
              router_dtype=None, expert_q="q4_0", shared_q="q8_0", score="softmax",
              path="auto", act_quant="none"):
    """A descriptor from readable names (dtype / format / score / path strings
    or the FW_* integers)."""
    enum = lambda table, v: table[v] if isinstance(v, str) else int(v)
    return fw_moe_desc(hidden, n_experts, top_k, ffn, shared_ffn,
                       enum(DTYPES, act_dtype), enum(DTYPES, router_dtype or act_dtype),
                       enum(QTYPES, expert_q), enum(QTYPES, shared_q),
                       enum(SCORES, score), enum(PATHS, path), enum(ACT_QUANTS, act_quant))


class fw_moe_dense_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "in_features", "out_features", "n_experts", "fn", "ckpt", "out_dtype", "grad_dtype",
        "accumulate")]


class fw_moe_ckpt_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("features", "format", "src_dtype", "dst_dtype")]


def make_dense_desc(in_features, out_features, n_experts=1, fn="silu", ckpt="none",
                    out_dtype="bf16", grad_dtype="bf16", accumulate=False):
    """A descriptor of the training products (fw_moe_glu_*, fw_moe_linear_*)
    from readable names or the FW_* integers; ckpt is the form in which the
    backward calls get x."""
    enum = lambda table, v: table[v] if isinstance(v, str) else int(v)
    return fw_moe_dense_desc(in_features, out_features, n_experts, enum(FNS, fn),
                             enum(ACT_QUANTS, ckpt), enum(DTYPES, out_dtype),
                             enum(DTYPES, grad_dtype), int(accumulate))


def make_ckpt_desc(features, format, src_dtype="bf16", dst_dtype="bf16"):
    """A descriptor of 8-bit activation checkpoints ("mxfp8" or "int8")."""
    enum = lambda table, v: table[v] if isinstance(v, str) else int(v)
    return fw_moe_ckpt_desc(features, enum(ACT_QUANTS, format), enum(DTYPES, src_dtype),
                            enum(DTYPES, dst_dtype))


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built (run __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        P, I, D = ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(fw_moe_desc)
        Z, DD = ctypes.c_size_t, ctypes.POINTER(fw_moe_dense_desc)
        CD = ctypes.POINTER(fw_moe_ckpt_desc)
        sig = {
            "fw_moe_version": ([], ctypes.c_char_p),
            "fw_moe_validate": ([D], ctypes.c_int),
            "fw_moe_workspace_size": ([D, I], ctypes.c_size_t),
            "fw_moe_forward_path": ([D, I], ctypes.c_int),
            "fw_moe_workspace_offsets": ([D, I, ctypes.POINTER(ctypes.c_size_t),
                                          ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
            "fw_moe_route": ([D, I] + [P] * 8, ctypes.c_int),
            "fw_moe_permute": ([D, I, P, P, P, P, P, ctypes.c_size_t, P], ctypes.c_int),
            "fw_moe_forward": ([D, I] + [P] * 13 + [ctypes.c_size_t, P], ctypes.c_int),
            "fw_moe_layer": ([D, I] + [P] * 17 + [ctypes.c_size_t, P], ctypes.c_int),
            "fw_moe_clear_status": ([P, P], ctypes.c_int),
            "fw_moe_read_status": ([P, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
            "fw_moe_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "fw_moe_layer_timed": ([D, I] + [P] * 17 + [ctypes.c_size_t, P, P], ctypes.c_int),
            "fw_moe_layer_noalloc": ([D, I] + [P] * 17 + [P], ctypes.c_int),
            "fw_moe_dense_validate": ([DD], ctypes.c_int),
            "fw_moe_dense_workspace_size": ([DD, I], Z),
            "fw_moe_glu_forward": ([DD, I] + [P] * 6 + [Z, P], ctypes.c_int),
            "fw_moe_glu_backward": ([DD, I] + [P] * 11 + [Z, P], ctypes.c_int),
            "fw_moe_linear_forward": ([DD, I] + [P] * 7 + [Z, P], ctypes.c_int),
            "fw_moe_linear_backward": ([DD, I] + [P] * 10 + [Z, P], ctypes.c_int),
            "fw_moe_ckpt_pack": ([CD, I] + [P] * 5, ctypes.c_int),
            "fw_moe_ckpt_unpack": ([CD, I] + [P] * 4, ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, code):
    if code != FW_OK:
        raise FwMoeError(fn, code)
    return code


def fw_moe_version():
    return lib().fw_moe_version().decode()


def fw_moe_validate(desc):
    return lib().fw_moe_validate(ctypes.byref(desc))


def fw_moe_workspace_size(desc, max_T):
    return lib().fw_moe_workspace_size(ctypes.byref(desc), max_T)


def fw_moe_forward_path(desc, T):
    return lib().fw_moe_forward_path(ctypes.byref(desc), T)


def fw_moe_workspace_offsets(desc, T):
    """(x staging, h staging) byte offsets inside a workspace for T tokens."""
    xo, ho = ctypes.c_size_t(), ctypes.c_size_t()
    _check("fw_moe_workspace_offsets", lib().fw_moe_workspace_offsets(
        ctypes.byref(desc), T, ctypes.byref(xo), ctypes.byref(ho)))
    return xo.value, ho.value


def fw_moe_route(desc, T, x, router_w, logit_bias, logits_in, logits, topk_ids, topk_w,
                 stream=None):
    return _check("fw_moe_route", lib().fw_moe_route(
        ctypes.byref(desc), T, _ptr(x), _ptr(router_w), _ptr(logit_bias), _ptr(logits_in),
        _ptr(logits), _ptr(topk_ids), _ptr(topk_w), _stream(stream)))


def fw_moe_permute(desc, T, topk_ids, expert_offsets, sorted_pairs, inv_pos, workspace,
                   ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    return _check("fw_moe_permute", lib().fw_moe_permute(
        ctypes.byref(desc), T, _ptr(topk_ids), _ptr(expert_offsets), _ptr(sorted_pairs),
        _ptr(inv_pos), _ptr(workspace), ws_bytes, _stream(stream)))


def fw_moe_forward(desc, T, x, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, topk_w,
                   expert_offsets, sorted_pairs, inv_pos, out, workspace, ws_bytes=None,
                   stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    return _check("fw_moe_forward", lib().fw_moe_forward(
        ctypes.byref(desc), T, _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(ws_gate),
        _ptr(ws_up), _ptr(ws_down), _ptr(topk_w), _ptr(expert_offsets), _ptr(sorted_pairs),
        _ptr(inv_pos), _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)))


def fw_moe_layer(desc, T, x, router_w, logit_bias, w_gate, w_up, w_down, ws_gate, ws_up,
                 ws_down, logits, topk_ids, topk_w, expert_offsets, sorted_pairs, inv_pos, out,
                 workspace, ws_bytes=None, stream=None):
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    return _check("fw_moe_layer", lib().fw_moe_layer(
        ctypes.byref(desc), T, _ptr(x), _ptr(router_w), _ptr(logit_bias), _ptr(w_gate),
        _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(logits),
        _ptr(topk_ids), _ptr(topk_w), _ptr(expert_offsets), _ptr(sorted_pairs), _ptr(inv_pos),
        _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)))


def fw_moe_clear_status(workspace, stream=None):
    return _check("fw_moe_clear_status",
                  lib().fw_moe_clear_status(_ptr(workspace), _stream(stream)))


def fw_moe_read_status(workspace):
    v = ctypes.c_int32(0)
    _check("fw_moe_read_status", lib().fw_moe_read_status(_ptr(workspace), ctypes.byref(v)))
    return v.value


def fw_moe_status_string(code):
    return lib().fw_moe_status_string(code).decode()


status_string = fw_moe_status_string


def fw_moe_layer_timed(desc, T, x, router_w, logit_bias, w_gate, w_up, w_down, ws_gate,
                       ws_up, ws_down, logits, topk_ids, topk_w, expert_offsets, sorted_pairs,
                       inv_pos, out, workspace, stage_events, ws_bytes=None, stream=None):
    """stage_events: FW_N_STAGE_EVENTS torch.cuda.Event objects (enable_timing=True)."""
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    assert len(stage_events) == FW_N_STAGE_EVENTS
    for e in stage_events:
        if e.cuda_event == 0:      # torch creates the HIP event lazily
            e.record()
    arr = (ctypes.c_void_p * FW_N_STAGE_EVENTS)(*[e.cuda_event for e in stage_events])
    return _check("fw_moe_layer_timed", lib().fw_moe_layer_timed(
        ctypes.byref(desc), T, _ptr(x), _ptr(router_w), _ptr(logit_bias), _ptr(w_gate),
        _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(logits),
        _ptr(topk_ids), _ptr(topk_w), _ptr(expert_offsets), _ptr(sorted_pairs), _ptr(inv_pos),
        _ptr(out), _ptr(workspace), ws_bytes, arr, _stream(stream)))


def fw_moe_layer_noalloc(desc, T, x, router_w, logit_bias, w_gate, w_up, w_down, ws_gate,
                         ws_up, ws_down, logits, topk_ids, topk_w, expert_offsets,
                         sorted_pairs, inv_pos, out, status=None, stream=None):
    """status: an int32 device tensor of one element, or None."""
    return _check("fw_moe_layer_noalloc", lib().fw_moe_layer_noalloc(
        ctypes.byref(desc), T, _ptr(x), _ptr(router_w), _ptr(logit_bias), _ptr(w_gate),
        _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(logits),
        _ptr(topk_ids), _ptr(topk_w), _ptr(expert_offsets), _ptr(sorted_pairs), _ptr(inv_pos),
        _ptr(out), _ptr(status), _stream(stream)))


# ---- training products ------------------------------------------------------
# The kernels read flat row-major memory: a tensor of another size, type or
# layout, or on another device than the rest, is refused here (ValueError)
# before the library sees its pointer.  Raw integer pointers pass unchecked.
# Decode-sized calls take about as long on the host as on the GPU, hence the
# plain loops.
_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_OUT = {FW_F32: _F32, FW_BF16: _BF16}
# element types of a checkpoint's codes and scales
_CODES = {FW_ACT_MXFP8: ((torch.uint8, torch.float8_e4m3fn), (torch.uint8,)),
          FW_ACT_INT8: ((torch.int8, torch.uint8), _F32)}


def _refuse(fn, name, t, count, dtypes, device):
    if t.dtype not in dtypes:
        raise ValueError(f"{fn}: {name} is {t.dtype}, not {' or '.join(map(str, dtypes))}")
    if t.numel() != count:
        raise ValueError(f"{fn}: {name} has {t.numel()} elements, not {count}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} is not contiguous")
    raise ValueError(f"{fn}: {name} is on {t.device}, not on " +
                     ("a GPU" if device < 0 else f"cuda:{device} like the others"))


def _call(fn, desc, R, operands, args, workspace, ws_bytes, stream):
    """Check the operands (name, tensor or None, elements, types), then call
    the library's fn(desc, R, *args, [workspace, [its bytes,]] stream) with
    their device current."""
    device = None
    for name, t, count, dtypes in operands:
        if t is None or type(t) is int:
            continue
        d = t.get_device()
        if device is None:
            device, first = d, (name, t, count, dtypes)
        if (d != device or t.dtype not in dtypes or t.numel() != count or
                not t.is_contiguous()):
            _refuse(fn, name, t, count, dtypes, device)
    if device is not None and device < 0:
        _refuse(fn, *first, device)
    tail = []
    if workspace is not None:
        ws, sized = workspace
        if ws is not None and type(ws) is not int:
            if ws.get_device() != device is not None or not ws.is_contiguous():
                _refuse(fn, "workspace", ws, ws.numel(), (ws.dtype,), device)
            if ws_bytes is None:
                ws_bytes = ws.numel() * ws.element_size()
            ws = ws.data_ptr()
        tail = [ws, ws_bytes or 0] if sized else [ws]
    here = torch.cuda.current_device()
    elsewhere = device is not None and device != here
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device if elsewhere else here)
    else:
        stream = _stream(stream)
    f = getattr(_lib or lib(), fn)
    ptrs = [t if t is None or type(t) is int else t.data_ptr() for t in args]
    if elsewhere:
        with torch.cuda.device(device):
            rc = f(desc, R, *ptrs, *tail, stream)
    else:
        rc = f(desc, R, *ptrs, *tail, stream)
    return rc if rc == FW_OK else _check(fn, rc)


def _x_operands(desc, R, x, x_scales):
    """The backward calls' x: bf16 rows or a checkpoint."""
    if desc.ckpt not in _CODES:
        return [("x", x, R * desc.in_features, _BF16)]
    codes, scales = _CODES[desc.ckpt]
    return [("x", x, R * desc.in_features, codes),
            ("x_scales", x_scales, R * (desc.in_features // 32), scales)]


def fw_moe_dense_validate(desc):
    return lib().fw_moe_dense_validate(ctypes.byref(desc))


def fw_moe_dense_workspace_size(desc, max_R):
    return lib().fw_moe_dense_workspace_size(ctypes.byref(desc), max_R)


def fw_moe_glu_forward(desc, R, x, w_gate, w_up, expert_offsets, h, workspace, ws_bytes=None,
                       stream=None):
    K, N, E = desc.in_features, desc.out_features, desc.n_experts
    return _call("fw_moe_glu_forward", desc, R,
                 (("x", x, R * K, _BF16), ("w_gate", w_gate, E * N * K, _BF16),
                  ("w_up", w_up, E * N * K, _BF16),
                  ("expert_offsets", expert_offsets, E + 1, _I32),
                  ("h", h, R * N, _OUT.get(desc.out_dtype, ()))),
                 (x, w_gate, w_up, expert_offsets, h), (workspace, True), ws_bytes, stream)


def fw_moe_glu_backward(desc, R, x, x_scales, w_gate, w_up, expert_offsets, dh, dx, dw_gate,
                        dw_up, h, workspace, ws_bytes=None, stream=None):
    K, N, E = desc.in_features, desc.out_features, desc.n_experts
    grad = _OUT.get(desc.grad_dtype, ())
    return _call("fw_moe_glu_backward", desc, R,
                 _x_operands(desc, R, x, x_scales) +
                 [("w_gate", w_gate, E * N * K, _BF16), ("w_up", w_up, E * N * K, _BF16),
                  ("expert_offsets", expert_offsets, E + 1, _I32), ("dh", dh, R * N, _BF16),
                  ("dx", dx, R * K, grad), ("dw_gate", dw_gate, E * N * K, grad),
                  ("dw_up", dw_up, E * N * K, grad), ("h", h, R * N, _BF16)],
                 (x, x_scales, w_gate, w_up, expert_offsets, dh, dx, dw_gate, dw_up, h),
                 (workspace, True), ws_bytes, stream)


def fw_moe_linear_forward(desc, R, x, w, bias, residual, expert_offsets, y, workspace,
                          ws_bytes=None, stream=None):
    K, N, E = desc.in_features, desc.out_features, desc.n_experts
    out = _OUT.get(desc.out_dtype, ())
    return _call("fw_moe_linear_forward", desc, R,
                 (("x", x, R * K, _BF16), ("w", w, E * N * K, _BF16), ("bias", bias, E * N, _F32),
                  ("residual", residual, R * N, out),
                  ("expert_offsets", expert_offsets, E + 1, _I32), ("y", y, R * N, out)),
                 (x, w, bias, residual, expert_offsets, y), (workspace, True), ws_bytes, stream)


def fw_moe_linear_backward(desc, R, x, x_scales, w, bias, expert_offsets, dy, dx, dw, dbias,
                           workspace, ws_bytes=None, stream=None):
    K, N, E = desc.in_features, desc.out_features, desc.n_experts
    grad = _OUT.get(desc.grad_dtype, ())
    return _call("fw_moe_linear_backward", desc, R,
                 _x_operands(desc, R, x, x_scales) +
                 [("w", w, E * N * K, _BF16), ("bias", bias, E * N, _F32),
                  ("expert_offsets", expert_offsets, E + 1, _I32), ("dy", dy, R * N, _BF16),
                  ("dx", dx, R * K, grad), ("dw", dw, E * N * K, grad),
                  ("dbias", dbias, E * N, _F32)],
                 (x, x_scales, w, bias, expert_offsets, dy, dx, dw, dbias), (workspace, True),
                 ws_bytes, stream)


def _ckpt_operands(desc, R, codes, scales):
    code_types, scale_types = _CODES.get(desc.format, ((), ()))
    return (("codes", codes, R * desc.features, code_types),
            ("scales", scales, R * (desc.features // 32), scale_types))


def fw_moe_ckpt_pack(desc, R, x, codes, scales, workspace, stream=None):
    """workspace: a tensor of at least 256 bytes (its status word)."""
    if workspace is not None and type(workspace) is not int and \
            workspace.numel() * workspace.element_size() < 256:
        raise FwMoeError("fw_moe_ckpt_pack", FW_EWORKSPACE)
    return _call("fw_moe_ckpt_pack", desc, R,
                 (("x", x, R * desc.features, _OUT.get(desc.src_dtype, ())),) +
                 _ckpt_operands(desc, R, codes, scales),
                 (x, codes, scales), (workspace, False), None, stream)


def fw_moe_ckpt_unpack(desc, R, codes, scales, x, stream=None):
    return _call("fw_moe_ckpt_unpack", desc, R,
                 _ckpt_operands(desc, R, codes, scales) +
                 (("x", x, R * desc.features, _OUT.get(desc.dst_dtype, ())),),
                 (codes, scales, x), None, None, stream)
