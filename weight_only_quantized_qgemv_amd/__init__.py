"""Weight-only quantized linear layers on MI355X (gfx950).

Thin ctypes binding of ``libqpack.so`` (C ABI in ``include/qpack.h``). This
module only marshals arguments: tensors are passed as device pointers with the
caller's current HIP stream, and every step of the computation runs in the
library's HIP kernels. PyTorch provides device memory and streams. There is no
CPU fallback: without the built library every call raises.

Calls (same names as the C ABI):
    qpack_quantize(w, bits, group_size, sb_dtype)  -> (wq, scales, biases)
    qmatmul(x, wq, scales, biases, bits, group_size) -> y = x @ dequant(W)^T
    qgemv_moe_id(a, ids, ..., wq, scales, biases, ...) -> out
    qgemv_moe_id_gate_up_silu(a, ids, ..., gate, up, ...) -> SiLU(gate) * up
    qgemv_moe_workspace_bytes(n_pairs, num_experts)
    qffn(x, gate, up, down, bits, group_size)      -> dense gated block, qffn_backward its gradients
    qmatmul_backward(x, dy, wq, scales, biases, ...) -> dx, dscales, dbiases
    qembedding(ids, wq, scales, biases, ...)       -> rows of a packed table, qembedding_backward
    qlogits_adjust(logits, ...)                    -> penalties, biases and masks on logits
"""
from __future__ import annotations

import ctypes
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libqpack.so")

QP_F32, QP_F16, QP_BF16 = 0, 1, 2
STATUS = {0: "QP_OK", 1: "QP_ERR_INVALID_ARG", 2: "QP_ERR_UNSUPPORTED",
          3: "QP_ERR_DTYPE_MISMATCH", 4: "QP_ERR_SHAPE", 5: "QP_ERR_ALIGN",
          6: "QP_ERR_WORKSPACE", 7: "QP_ERR_HIP"}

# Every symbol include/qpack.h declares.
EXPORTS = ("qpack_quantize", "qpack_dequantize", "qpack_dequantize_mx", "qmatmul", "qmatmul_mx",
           "qgemv_moe_workspace_bytes", "qgemv_moe_id", "qgemv_moe_id_noalloc",
           "qgemv_moe_id_gate_up_silu",
           "qgemv_moe_ffn_workspace_bytes", "qgemv_moe_ffn", "qpack_quantize_int8_tensor",
           "qpack_dequantize_int8_tensor", "qmatmul_int8_tensor", "qmatmul_t_workspace_bytes",
           "qmatmul_t", "qffn_workspace_bytes", "qffn", "qffn_backward_workspace_bytes",
           "qffn_backward", "qmatmul_backward_workspace_bytes", "qmatmul_backward", "qembedding",
           "qembedding_backward_workspace_bytes", "qembedding_backward", "qlogits_adjust",
           "qpack_last_error",
           "qpack_version")


class QpackError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        L.qpack_quantize.argtypes = [P, I64, I64, I32, I32, ctypes.c_int, P, P, P, P]
        L.qpack_quantize.restype = ctypes.c_int
        L.qpack_dequantize.argtypes = [P, P, P, ctypes.c_int, I64, I64, I32, I32, ctypes.c_int,
                                       P, P]
        L.qpack_dequantize.restype = ctypes.c_int
        L.qpack_dequantize_mx.argtypes = [P, P, ctypes.c_int, I64, I64, ctypes.c_int, P, P]
        L.qpack_dequantize_mx.restype = ctypes.c_int
        L.qmatmul_mx.argtypes = [P, ctypes.c_int, I64, I64, P, P, ctypes.c_int, I64, P, P]
        L.qmatmul_mx.restype = ctypes.c_int
        L.qmatmul.argtypes = [P, ctypes.c_int, I64, I64, P, P, P, ctypes.c_int, I64, I32, I32, P,
                              P]
        L.qmatmul.restype = ctypes.c_int
        L.qgemv_moe_workspace_bytes.argtypes = [I64, I64]
        L.qgemv_moe_workspace_bytes.restype = SZ
        L.qgemv_moe_id.argtypes = [P, ctypes.c_int, P, I64, I64, I64, I64, P, P, P, ctypes.c_int,
                                   I64, I64, I64, I32, I32, P, P, SZ, P]
        L.qgemv_moe_id.restype = ctypes.c_int
        L.qgemv_moe_id_noalloc.argtypes = [P, ctypes.c_int, P, I64, I64, I64, I64, P, P, P,
                                           ctypes.c_int, I64, I64, I64, I32, I32, P, P]
        L.qgemv_moe_id_noalloc.restype = ctypes.c_int
        L.qgemv_moe_id_gate_up_silu.argtypes = [P, ctypes.c_int, P, I64, I64, I64, I64, P, P, P,
                                                P, P, P, ctypes.c_int, I64, I64, I64, I32, I32,
                                                P, P, SZ, P]
        L.qgemv_moe_id_gate_up_silu.restype = ctypes.c_int
        L.qgemv_moe_ffn_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, ctypes.c_int]
        L.qgemv_moe_ffn_workspace_bytes.restype = SZ
        L.qgemv_moe_ffn.argtypes = ([P, ctypes.c_int, P, P, I64, I64] + [P] * 9 +
                                    [ctypes.c_int, I64, I64, I64, I32, I32, P, P, SZ, P])
        L.qgemv_moe_ffn.restype = ctypes.c_int
        L.qpack_quantize_int8_tensor.argtypes = [P, I64, P, P, P]
        L.qpack_quantize_int8_tensor.restype = ctypes.c_int
        L.qpack_dequantize_int8_tensor.argtypes = [P, I64, P, ctypes.c_int, P, P]
        L.qpack_dequantize_int8_tensor.restype = ctypes.c_int
        L.qmatmul_int8_tensor.argtypes = [P, ctypes.c_int, I64, I64, P, P, I64, P, P]
        L.qmatmul_int8_tensor.restype = ctypes.c_int
        L.qmatmul_t_workspace_bytes.argtypes = [I64, I64, I64, I32]
        L.qmatmul_t_workspace_bytes.restype = SZ
        L.qmatmul_t.argtypes = [P, ctypes.c_int, I64, I64, P, P, P, ctypes.c_int, I64, I32, I32, P,
                                P, SZ, P]
        L.qmatmul_t.restype = ctypes.c_int
        CI = ctypes.c_int
        L.qffn_workspace_bytes.argtypes = [I64, I64, I64, CI]
        L.qffn_workspace_bytes.restype = SZ
        L.qffn.argtypes = [P, CI, I64, I64, I64] + [P] * 9 + [CI, I32, I32, CI, P, P, P, SZ, P]
        L.qffn.restype = CI
        L.qffn_backward_workspace_bytes.argtypes = [I64, I64, I64, I32, I32, CI]
        L.qffn_backward_workspace_bytes.restype = SZ
        L.qffn_backward.argtypes = ([P, P, P, CI, I64, I64, I64] + [P] * 9 + [CI, I32, I32, CI] +
                                    [P] * 8 + [SZ, P])
        L.qffn_backward.restype = CI
        L.qmatmul_backward_workspace_bytes.argtypes = [I64, I64, I64, I32, I32, CI]
        L.qmatmul_backward_workspace_bytes.restype = SZ
        L.qmatmul_backward.argtypes = [P, P, CI, I64, I64, P, P, P, CI, I64, I32, I32, P, P, P, P,
                                       SZ, P]
        L.qmatmul_backward.restype = CI
        L.qembedding.argtypes = [P, I64, P, P, P, CI, I64, I64, I32, I32, ctypes.c_float, P, P]
        L.qembedding.restype = CI
        L.qembedding_backward_workspace_bytes.argtypes = [I64, I64, I32, I32]
        L.qembedding_backward_workspace_bytes.restype = SZ
        L.qembedding_backward.argtypes = [P, I64, P, CI, P, I64, I64, I32, I32, ctypes.c_float, P,
                                          P, P, SZ, P]
        L.qembedding_backward.restype = CI
        L.qlogits_adjust.argtypes = [P, CI, I64, I64, I64, P, I64, P, P, P, P, P, P, P, I64, P, P,
                                     I64, P, I64, P]
        L.qlogits_adjust.restype = CI
        L.qpack_last_error.restype = ctypes.c_char_p
        L.qpack_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def last_error() -> str:
    return lib().qpack_last_error().decode()


def check(status: int) -> None:
    if status != 0:
        raise QpackError(status, last_error())


def version() -> str:
    return lib().qpack_version().decode()


# ------------------------------------------------------------------ tensors

_DTYPE_CODES = None


def dtype_code(dt) -> int:
    global _DTYPE_CODES
    if _DTYPE_CODES is None:
        import torch
        _DTYPE_CODES = {torch.float32: QP_F32, torch.float16: QP_F16, torch.bfloat16: QP_BF16}
    code = _DTYPE_CODES.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt}")
    return code


_RAW_STREAM = None


def _stream(t) -> int:
    """The handle of the current stream on t's device. torch's raw-handle query
    costs about 0.06 us per call against about 1.8 us for building the Stream
    object, which matters for calls of a few microseconds issued one by one."""
    global _RAW_STREAM
    if _RAW_STREAM is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _RAW_STREAM = ((lambda dev: raw(dev.index)) if raw is not None
                       else (lambda dev: torch.cuda.current_stream(dev).cuda_stream))
    return _RAW_STREAM(t.device)


def _dev(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t


def _ptr(t) -> int:
    return t.data_ptr()


def qpack_quantize(w, bits: int, group_size: int, sb_dtype=None, wq=None, scales=None,
                   biases=None):
    """Quantize fp32 w [n, k] on the device. Returns (wq u32-as-int32 [n, k*bits/32],
    scales [n, k/gs], biases [n, k/gs]) with scales/biases of `sb_dtype` (default bf16)."""
    import torch
    _dev(w, "w")
    if w.dtype != torch.float32 or not w.is_contiguous() or w.dim() != 2:
        raise ValueError("w must be a contiguous fp32 [n, k] tensor")
    sb_dtype = sb_dtype or torch.bfloat16
    n, k = w.shape
    if wq is None:
        wq = torch.empty((n, k * bits // 32), dtype=torch.int32, device=w.device)
    if scales is None:
        scales = torch.empty((n, k // group_size if group_size else 0), dtype=sb_dtype,
                             device=w.device)
    if biases is None:
        biases = torch.empty_like(scales)
    check(lib().qpack_quantize(_ptr(w), n, k, bits, group_size, dtype_code(sb_dtype), _ptr(wq),
                               _ptr(scales), _ptr(biases), _stream(w)))
    return wq, scales, biases


def qpack_dequantize(wq, scales, biases, bits: int, group_size: int, out_dtype=None,
                     out=None):
    """Dense weight [n, k] from packed codes: fp32, or (the default) the scales' own
    dtype, with the product and sum rounded to that dtype."""
    import torch
    for t, nm in ((wq, "wq"), (scales, "scales"), (biases, "biases")):
        _dev(t, nm)
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    n = wq.shape[0]
    k = wq.shape[1] * 32 // bits if bits else 0
    out_dtype = out_dtype or scales.dtype
    if out is None:
        out = torch.empty((n, k), dtype=out_dtype, device=wq.device)
    check(lib().qpack_dequantize(_ptr(wq), _ptr(scales), _ptr(biases), dtype_code(scales.dtype),
                                 n, k, bits, group_size, dtype_code(out.dtype), _ptr(out),
                                 _stream(wq)))
    return out


MXFP4, MXFP8, NVFP4 = 1, 2, 3
MX_LAYOUT = {MXFP4: (4, 32), MXFP8: (8, 32), NVFP4: (4, 16)}   # mode -> (bits, group size)


def qpack_dequantize_mx(wq, scales, mode: int, out_dtype=None, out=None):
    """Dense weight [n, k] of a microscaled mode (scales: uint8 [n, k/gs]); bf16 by
    default, as the pages return it."""
    import torch
    for t, nm in ((wq, "wq"), (scales, "scales")):
        _dev(t, nm)
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    if mode not in MX_LAYOUT:
        raise ValueError(f"unknown microscaled mode {mode}")
    n, k = wq.shape[0], wq.shape[1] * 32 // MX_LAYOUT[mode][0]
    if out is None:
        out = torch.empty((n, k), dtype=out_dtype or torch.bfloat16, device=wq.device)
    check(lib().qpack_dequantize_mx(_ptr(wq), _ptr(scales), mode, n, k, dtype_code(out.dtype),
                                    _ptr(out), _stream(wq)))
    return out


def qmatmul_mx(x, wq, scales, mode: int, out=None):
    """y = x @ dequant(W)^T for a microscaled W; x [m, k] fp32/fp16/bf16, y in x's dtype."""
    import torch
    _dev(x, "x")
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [m, k] tensor")
    for t, nm in ((wq, "wq"), (scales, "scales")):
        _dev(t, nm)
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    m, k = x.shape
    n = wq.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=x.dtype, device=x.device)
    check(lib().qmatmul_mx(_ptr(x), dtype_code(x.dtype), m, k, _ptr(wq), _ptr(scales), mode, n,
                           _ptr(out), _stream(x)))
    return out


def qmatmul(x, wq, scales, biases, bits: int, group_size: int, out=None):
    """y = x @ dequant(W)^T for x [m, k] (fp32/fp16/bf16, same dtype as scales)."""
    import torch
    _dev(x, "x")
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [m, k] tensor")
    m, k = x.shape
    n = wq.shape[0]
    for t, nm in ((wq, "wq"), (scales, "scales"), (biases, "biases")):
        _dev(t, nm)
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    if out is None:
        out = torch.empty((m, n), dtype=x.dtype, device=x.device)
    check(lib().qmatmul(_ptr(x), dtype_code(x.dtype), m, k, _ptr(wq), _ptr(scales), _ptr(biases),
                        dtype_code(scales.dtype), n, bits, group_size, _ptr(out), _stream(x)))
    return out


def qgemv_moe_workspace_bytes(n_pairs: int, num_experts: int) -> int:
    return int(lib().qgemv_moe_workspace_bytes(n_pairs, num_experts))


def _moe_workspace(a, n_pairs, num_experts, workspace):
    import torch
    need = qgemv_moe_workspace_bytes(n_pairs, num_experts)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=a.device)
    return workspace


def qgemv_moe_id(a, ids, n_tokens: int, top_k: int, a_outer: int, a_inner: int, wq, scales,
                 biases, bits: int, group_size: int, out=None, workspace=None):
    """out[p] = a_row(p) @ dequant(W[ids[p]])^T for p < n_tokens*top_k, with
    a_row(p) = a.flat[(p//top_k)*a_outer + (p%top_k)*a_inner : +n_cols].
    wq [E, n_rows, n_cols*bits/32], scales/biases [E, n_rows, n_cols/gs]."""
    import torch
    E, n_rows = wq.shape[0], wq.shape[1]
    n_cols = wq.shape[2] * 32 // bits
    P = n_tokens * top_k
    if out is None:
        out = torch.empty((P, n_rows), dtype=a.dtype, device=a.device)
    workspace = _moe_workspace(a, P, E, workspace)
    check(lib().qgemv_moe_id(_ptr(a), dtype_code(a.dtype), _ptr(ids), n_tokens, top_k, a_outer,
                             a_inner, _ptr(wq), _ptr(scales), _ptr(biases),
                             dtype_code(scales.dtype), E, n_rows, n_cols, bits, group_size,
                             _ptr(out), _ptr(workspace), workspace.numel(), _stream(a)))
    return out


def qgemv_moe_id_noalloc(a, ids, n_tokens: int, top_k: int, a_outer: int, a_inner: int, wq,
                         scales, biases, bits: int, group_size: int, out):
    """qgemv_moe_id with the routing tables in the library's own device
    scratch (no workspace; `out` is the caller's)."""
    E, n_rows = wq.shape[0], wq.shape[1]
    n_cols = wq.shape[2] * 32 // bits
    check(lib().qgemv_moe_id_noalloc(_ptr(a), dtype_code(a.dtype), _ptr(ids), n_tokens, top_k,
                                     a_outer, a_inner, _ptr(wq), _ptr(scales), _ptr(biases),
                                     dtype_code(scales.dtype), E, n_rows, n_cols, bits,
                                     group_size, _ptr(out), _stream(a)))
    return out


def qgemv_moe_id_gate_up_silu(a, ids, n_tokens: int, top_k: int, a_outer: int, a_inner: int,
                              gate, up, bits: int, group_size: int, out=None, workspace=None):
    """silu_out[p] = SiLU(a_row(p) @ dequant(Wg[ids[p]])^T) * (a_row(p) @ dequant(Wu[ids[p]])^T).
    gate, up: (wq, scales, biases) stacks of identical shape."""
    import torch
    gwq, gs_, gb = gate
    uwq, us, ub = up
    if tuple(gwq.shape) != tuple(uwq.shape) or tuple(gs_.shape) != tuple(us.shape):
        raise ValueError("gate and up stacks must match in shape")
    E, n_rows = gwq.shape[0], gwq.shape[1]
    n_cols = gwq.shape[2] * 32 // bits
    P = n_tokens * top_k
    if out is None:
        out = torch.empty((P, n_rows), dtype=a.dtype, device=a.device)
    workspace = _moe_workspace(a, P, E, workspace)
    check(lib().qgemv_moe_id_gate_up_silu(
        _ptr(a), dtype_code(a.dtype), _ptr(ids), n_tokens, top_k, a_outer, a_inner, _ptr(gwq),
        _ptr(gs_), _ptr(gb), _ptr(uwq), _ptr(us), _ptr(ub), dtype_code(gs_.dtype), E, n_rows,
        n_cols, bits, group_size, _ptr(out), _ptr(workspace), workspace.numel(), _stream(a)))
    return out


def qgemv_moe_ffn_workspace_bytes(n_tokens: int, top_k: int, num_experts: int, d_model: int,
                                  d_ff: int, dtype) -> int:
    return int(lib().qgemv_moe_ffn_workspace_bytes(n_tokens, top_k, num_experts, d_model, d_ff,
                                                   dtype_code(dtype)))


def qgemv_moe_ffn(a, ids, route_weights, top_k: int, gate, up, down, bits: int, group_size: int,
                  out=None, workspace=None):
    """One MoE FFN block: a [T, d_model], ids int32 [T*top_k], route_weights fp32
    [T*top_k]; gate / up / down = (wq, scales, biases) expert stacks. Returns
    out [T, d_model] in a's dtype."""
    import torch
    for t, nm in ((a, "a"), (ids, "ids"), (route_weights, "route_weights")):
        _dev(t, nm)
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    T, D = a.shape
    E, F = gate[0].shape[0], gate[0].shape[1]
    if workspace is None:
        nbytes = qgemv_moe_ffn_workspace_bytes(T, top_k, E, D, F, a.dtype)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=a.device)
    if out is None:
        out = torch.empty((T, D), dtype=a.dtype, device=a.device)
    ptrs = [_ptr(x) for trio in (gate, up, down) for x in trio]
    check(lib().qgemv_moe_ffn(_ptr(a), dtype_code(a.dtype), _ptr(ids), _ptr(route_weights), T,
                              top_k, *ptrs, dtype_code(gate[1].dtype), E, D, F, bits, group_size,
                              _ptr(out), _ptr(workspace), workspace.numel(), _stream(a)))
    return out


def qpack_quantize_int8_tensor(w, q=None, rng=None):
    """Per-tensor dynamic-range int8 of fp32 w: (int8 codes shaped like w, fp32 range [lo, hi])."""
    import torch
    _dev(w, "w")
    if w.dtype != torch.float32 or not w.is_contiguous():
        raise ValueError("w must be a contiguous fp32 tensor")
    q = torch.empty(w.shape, dtype=torch.int8, device=w.device) if q is None else q
    rng = torch.empty(2, dtype=torch.float32, device=w.device) if rng is None else rng
    check(lib().qpack_quantize_int8_tensor(_ptr(w), w.numel(), _ptr(q), _ptr(rng), _stream(w)))
    return q, rng


def qpack_dequantize_int8_tensor(q, rng, out_dtype=None, out=None):
    import torch
    _dev(q, "q")
    _dev(rng, "range")
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or torch.float32, device=q.device)
    check(lib().qpack_dequantize_int8_tensor(_ptr(q), q.numel(), _ptr(rng), dtype_code(out.dtype),
                                             _ptr(out), _stream(q)))
    return out


def qmatmul_int8_tensor(x, q, rng, out=None):
    """y = x @ W^T for a per-tensor int8 weight q [n, k] with device range [lo, hi]."""
    import torch
    for t, nm in ((x, "x"), (q, "q"), (rng, "range")):
        _dev(t, nm)
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    m, k = x.shape
    n = q.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=x.dtype, device=x.device)
    check(lib().qmatmul_int8_tensor(_ptr(x), dtype_code(x.dtype), m, k, _ptr(q), _ptr(rng), n,
                                    _ptr(out), _stream(x)))
    return out


def qmatmul_t_workspace_bytes(m: int, k: int, n: int, bits: int) -> int:
    return int(lib().qmatmul_t_workspace_bytes(m, k, n, bits))


def qmatmul_t(x, wq, scales, biases, bits: int, group_size: int, out=None, workspace=None):
    """transpose = false: y = x @ dequant(W) with W stored [k, n] (wq [k, n*bits/32],
    scales / biases [k, n/gs], groups along n)."""
    import torch
    _dev(x, "x")
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [m, k] tensor")
    for t, nm in ((wq, "wq"), (scales, "scales"), (biases, "biases")):
        _dev(t, nm)
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
    m, k = x.shape
    n = wq.shape[1] * 32 // bits
    if out is None:
        out = torch.empty((m, n), dtype=x.dtype, device=x.device)
    if workspace is None:
        nbytes = qmatmul_t_workspace_bytes(m, k, n, bits)
        workspace = torch.empty(max(nbytes, 4), dtype=torch.uint8, device=x.device)
    check(lib().qmatmul_t(_ptr(x), dtype_code(x.dtype), m, k, _ptr(wq), _ptr(scales), _ptr(biases),
                          dtype_code(scales.dtype), n, bits, group_size, _ptr(out), _ptr(workspace),
                          workspace.numel(), _stream(x)))
    return out


# ------------------------------------------------------------------ the operators around the products

ACTS = {"silu": 0, "gelu_tanh": 1}


def _act_code(act: str) -> int:
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r} (one of {', '.join(ACTS)})")
    return code


def _like(t, like, name, shape=None, dtype=None):
    """t is a contiguous tensor on like's device (of `shape`, of `dtype`); returns t."""
    d = t.get_device()                 # -1 for host tensors
    if d < 0 or d != like.get_device():
        raise ValueError(f"{name} must be a device tensor on {like.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    return t


def _check_packed(w, like, name, n, k, bits, group_size):
    """(wq, scales, biases) of a weight [n, k] beside `like`."""
    import torch
    wq, scales, biases = w
    _like(wq, like, name + " codes", (n, k * bits // 32), torch.int32)
    groups = (n, k // group_size if group_size > 0 else 0)
    _like(scales, like, name + " scales", groups)
    _like(biases, like, name + " biases", groups, scales.dtype)
    return scales.dtype


def _workspace(nbytes, like, workspace):
    import torch
    if workspace is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=like.device)
    return _like(workspace, like, "workspace")


def _ws_bytes(workspace) -> int:
    return workspace.numel() * workspace.element_size()


def _check_ffn(x, gate, up, down, bits, group_size):
    if x.dim() != 2:
        raise ValueError("x must be a contiguous [m, d_model] tensor")
    _like(x, x, "x")
    m, d = x.shape
    f = gate[0].shape[0]
    dt = _check_packed(gate, x, "gate", f, d, bits, group_size)
    for w, name, n, k in ((up, "up", f, d), (down, "down", d, f)):
        if _check_packed(w, x, name, n, k, bits, group_size) != dt:
            raise ValueError("gate, up and down must have scales of one dtype")
    return m, d, f, dt


def qffn_workspace_bytes(m: int, d_model: int, d_ff: int, dtype) -> int:
    return int(lib().qffn_workspace_bytes(m, d_model, d_ff, dtype_code(dtype)))


def qffn(x, gate, up, down, bits: int, group_size: int, act: str = "silu", saved=None, out=None,
         workspace=None):
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T for x [m, d_model]; gate, up [d_ff, d_model] and down
    [d_model, d_ff] are (wq, scales, biases) weights. `saved`, an empty [2, m, d_ff] tensor of x's
    dtype, receives the two projections for qffn_backward. Returns y [m, d_model]."""
    import torch
    _dev(x, "x")
    m, d, f, dt = _check_ffn(x, gate, up, down, bits, group_size)
    if saved is not None:
        _like(saved, x, "saved", (2, m, f), x.dtype)
    if out is None:
        out = torch.empty((m, d), dtype=x.dtype, device=x.device)
    else:
        _like(out, x, "out", (m, d), x.dtype)
    workspace = _workspace(qffn_workspace_bytes(m, d, f, x.dtype), x, workspace)
    check(lib().qffn(_ptr(x), dtype_code(x.dtype), m, d, f, *[_ptr(t) for w in (gate, up, down) for t in w],
                     dtype_code(dt), bits, group_size, _act_code(act),
                     None if saved is None else _ptr(saved), _ptr(out), _ptr(workspace),
                     _ws_bytes(workspace), _stream(x)))
    return out


def qffn_backward_workspace_bytes(m: int, d_model: int, d_ff: int, bits: int, group_size: int,
                                  dtype) -> int:
    return int(lib().qffn_backward_workspace_bytes(m, d_model, d_ff, bits, group_size,
                                                   dtype_code(dtype)))


def qffn_backward(x, dy, saved, gate, up, down, bits: int, group_size: int, act: str = "silu",
                  input_grad: bool = True, weight_grads: bool = True, workspace=None):
    """Gradients of qffn at dy [m, d_model]: (dx, dgate, dup, ddown), each weight's a pair
    (dscales, dbiases) in x's dtype. dx is None without input_grad, the pairs without
    weight_grads (frozen weights)."""
    import torch
    _dev(x, "x")
    m, d, f, dt = _check_ffn(x, gate, up, down, bits, group_size)
    _like(dy, x, "dy", (m, d), x.dtype)
    _like(saved, x, "saved", (2, m, f), x.dtype)
    dx = torch.empty((m, d), dtype=x.dtype, device=x.device) if input_grad else None
    pairs = [None] * 3
    if weight_grads:
        pairs = [tuple(torch.empty(w[1].shape, dtype=x.dtype, device=x.device) for _ in range(2))
                 for w in (gate, up, down)]
    workspace = _workspace(qffn_backward_workspace_bytes(m, d, f, bits, group_size, x.dtype), x,
                           workspace)
    check(lib().qffn_backward(
        _ptr(x), _ptr(dy), _ptr(saved), dtype_code(x.dtype), m, d, f,
        *[_ptr(t) for w in (gate, up, down) for t in w], dtype_code(dt), bits, group_size,
        _act_code(act), None if dx is None else _ptr(dx),
        *[None if p is None else _ptr(p[i]) for p in pairs for i in range(2)], _ptr(workspace),
        _ws_bytes(workspace), _stream(x)))
    return (dx, *pairs)


def qmatmul_backward_workspace_bytes(m: int, k: int, n: int, bits: int, group_size: int,
                                     dtype) -> int:
    return int(lib().qmatmul_backward_workspace_bytes(m, k, n, bits, group_size, dtype_code(dtype)))


def qmatmul_backward(x, dy, wq, scales, biases, bits: int, group_size: int,
                     input_grad: bool = True, weight_grads: bool = True, workspace=None):
    """Gradients of y = x @ dequant(W)^T at dy [m, n]: (dx, dscales, dbiases) in x's dtype, each
    None where it is not asked for."""
    import torch
    _dev(x, "x")
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [m, k] tensor")
    m, k = x.shape
    n = wq.shape[0]
    dt = _check_packed((wq, scales, biases), x, "weight", n, k, bits, group_size)
    _like(dy, x, "dy", (m, n), x.dtype)
    dx = torch.empty((m, k), dtype=x.dtype, device=x.device) if input_grad else None
    ds = db = None
    if weight_grads:
        ds, db = (torch.empty(scales.shape, dtype=x.dtype, device=x.device) for _ in range(2))
    workspace = _workspace(qmatmul_backward_workspace_bytes(m, k, n, bits, group_size, x.dtype), x,
                           workspace)
    check(lib().qmatmul_backward(
        _ptr(x), _ptr(dy), dtype_code(x.dtype), m, k, _ptr(wq), _ptr(scales), _ptr(biases),
        dtype_code(dt), n, bits, group_size, *[None if t is None else _ptr(t) for t in (dx, ds, db)],
        _ptr(workspace), _ws_bytes(workspace), _stream(x)))
    return dx, ds, db


def qembedding(ids, wq, scales, biases, bits: int, group_size: int, factor: float = 1.0, out=None):
    """Rows ids (int32, any shape) of the packed table [n_rows, k], times factor, in the scales'
    dtype: [*ids.shape, k]. An id outside the table gives zeros."""
    import torch
    _like(ids, ids, "ids", None, torch.int32)
    k = wq.shape[1] * 32 // bits if bits else 0
    dt = _check_packed((wq, scales, biases), ids, "table", wq.shape[0], k, bits, group_size)
    shape = (*ids.shape, k)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=ids.device)
    else:
        _like(out, ids, "out", shape, dt)
    check(lib().qembedding(_ptr(ids), ids.numel(), _ptr(wq), _ptr(scales), _ptr(biases),
                           dtype_code(dt), wq.shape[0], k, bits, group_size, factor, _ptr(out),
                           _stream(ids)))
    return out


def qembedding_backward_workspace_bytes(n_tokens: int, k: int, bits: int, group_size: int) -> int:
    return int(lib().qembedding_backward_workspace_bytes(n_tokens, k, bits, group_size))


def qembedding_backward(ids, dout, wq, bits: int, group_size: int, factor: float = 1.0,
                        workspace=None):
    """Gradients (dscales, dbiases) [n_rows, k / group_size] of the table of qembedding at dout
    [*ids.shape, k], in dout's dtype."""
    import torch
    _like(ids, ids, "ids", None, torch.int32)
    k = wq.shape[1] * 32 // bits if bits else 0
    _like(wq, ids, "table codes", None, torch.int32)
    _like(dout, ids, "dout", (*ids.shape, k))
    t, n = ids.numel(), wq.shape[0]
    ds, db = (torch.empty((n, k // group_size if group_size > 0 else 0), dtype=dout.dtype,
                          device=ids.device) for _ in range(2))
    workspace = _workspace(qembedding_backward_workspace_bytes(t, k, bits, group_size), ids, workspace)
    check(lib().qembedding_backward(_ptr(ids), t, _ptr(dout), dtype_code(dout.dtype), _ptr(wq), n, k,
                                    bits, group_size, factor, _ptr(ds), _ptr(db), _ptr(workspace),
                                    _ws_bytes(workspace), _stream(ids)))
    return ds, db


def qlogits_adjust(logits, history=None, offsets=None, prompt_lens=None, repetition=None,
                   frequency=None, presence=None, bias=None, mask=None, out=None):
    """Penalties, biases and a mask on logits [rows, vocab] (rows may be strided).

    history int32 [h] holds every row's tokens, row b's from offsets[b] to offsets[b + 1] (int32
    [rows + 1]), the first prompt_lens[b] (int32 [rows]) of them its prompt; repetition, frequency
    and presence are fp32 [rows]; bias is (ids int32, values fp32, offsets int32 [rows + 1]); mask
    is int32 words [rows or 1, ceil(vocab / 32)], a set bit where the token is allowed. Returns the
    adjusted logits in their dtype; out=logits works in place."""
    import torch
    if logits.dim() != 2 or not logits.is_cuda or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a device tensor [rows, vocab], its last axis contiguous")
    rows, vocab = logits.shape
    if out is None:
        out = torch.empty((rows, vocab), dtype=logits.dtype, device=logits.device)
    elif (tuple(out.shape) != (rows, vocab) or out.dtype != logits.dtype
          or out.device != logits.device or (vocab > 1 and out.stride(1) != 1)):
        raise ValueError("out must be like logits, its last axis contiguous")
    i32, f32 = torch.int32, torch.float32
    if history is not None:
        _like(history, logits, "history", (history.numel(),), i32)
        if offsets is None:
            raise ValueError("history needs its rows' offsets")
    if offsets is not None:
        _like(offsets, logits, "offsets", (rows + 1,), i32)
    for t, name, dt in ((prompt_lens, "prompt_lens", i32), (repetition, "repetition", f32),
                        (frequency, "frequency", f32), (presence, "presence", f32)):
        if t is not None:
            _like(t, logits, name, (rows,), dt)
    bids = bvals = boff = None
    if bias is not None:
        bids, bvals, boff = bias
        _like(bids, logits, "bias ids", (bids.numel(),), i32)
        _like(bvals, logits, "bias values", bids.shape, f32)
        _like(boff, logits, "bias offsets", (rows + 1,), i32)
    mask_stride = 0
    if mask is not None:
        if mask.dim() != 2 or mask.shape[0] not in (1, rows):
            raise ValueError("mask must be [rows or 1, words]")
        _like(mask, logits, "mask", None, i32)
        if mask.shape[1] < (vocab + 31) // 32:
            raise ValueError(f"mask must have {(vocab + 31) // 32} words a row")
        mask_stride = mask.shape[1] if mask.shape[0] == rows and rows > 1 else 0

    def ptr(t):
        return None if t is None else t.data_ptr()

    check(lib().qlogits_adjust(
        ptr(logits), dtype_code(logits.dtype), rows, vocab, logits.stride(0), ptr(history),
        0 if history is None else history.numel(), ptr(offsets), ptr(prompt_lens), ptr(repetition),
        ptr(frequency), ptr(presence), ptr(bids), ptr(bvals), 0 if bids is None else bids.numel(),
        ptr(boff), ptr(mask), mask_stride, ptr(out), out.stride(0), _stream(logits)))
    return out
