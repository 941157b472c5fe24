"""Python binding of libmxfp4.so, the MI355X (gfx950) MXFP4 GEMM library.

Argument marshalling only: every function passes device pointers, sizes and
the current HIP stream to the C ABI declared in ``include/mxfp4.h`` and
raises ``RuntimeError`` with the library's status string on failure.  All
computation happens in the library's HIP kernels; torch provides device
memory and streams.  If the library is not built, importing the binding's
functions raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import types

_PKG = os.path.dirname(os.path.abspath(__file__))
# MXFP4_LIB may point at another build of the same library (e.g. a debug build).
LIB_PATH = os.environ.get("MXFP4_LIB") or os.path.join(_PKG, "libmxfp4.so")

MXFP4_OK = 0

_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    # PyTorch ships its own HIP runtime and asks for it as "libamdhip64.so";
    # this library asks for "libamdhip64.so.7", the soname that copy carries.
    # Loaded after torch, this library therefore binds to torch's runtime.
    # Loaded first, it would bring in /opt/rocm's copy and torch would then
    # load a second one, and the two runtimes in one process do not share
    # the device.  So torch goes first whenever it is installed.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            "libmxfp4.so is not built (expected at %s); run __graft_entry__.build() or "
            "python block_scaled_mxfp4_bf16_amd/build.py" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    P, I64, SZ, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    sigs = {
        "mxfp4_packed_bytes": (SZ, [I64, I64]),
        "mxfp4_raw_scale_bytes": (SZ, [I64, I64]),
        "mxfp4_shuffled_scale_bytes": (SZ, [I64, I64]),
        "mxfp4_gemm_workspace_bytes": (SZ, [I64, I64, I64]),
        "mxfp4_quantize": (I, [P, I64, I64, P, P, I, P]),
        "mxfp4_preshuffle_b": (I, [P, P, I64, I64, P, P, P]),
        "mxfp4_prepare_b": (I, [P, I64, I64, P, P, P]),
        "mxfp4_gemm": (I, [P, P, P, P, I64, I64, I64, P]),
        "mxfp4_gemm_ex": (I, [P, P, P, P, I64, I64, I64, P, SZ, P]),
        "mxfp4_gemm_noalloc": (I, [P, P, P, P, I64, I64, I64, P]),
        "mxfp4_gemm_q": (I, [P, P, P, P, P, I64, I64, I64, P]),
        "mxfp4_gemm_q_schedule_name": (ctypes.c_char_p, [I64, I64, I64]),
        "mxfp4_reserve": (I, [I64, I64, I64, P]),
        "mxfp4_status_string": (ctypes.c_char_p, [I]),
        "mxfp4_last_hip_error": (ctypes.c_char_p, []),
        "mxfp4_gemm_schedule_name": (ctypes.c_char_p, [I64, I64, I64]),
        "mxfp4_set_quant_mode": (I, [I]),
        "mxfp4_set_schedule_override": (I, [ctypes.c_char_p]),
        "mxfp4_list_schedules": (SZ, [I64, I64, I64, I, ctypes.c_char_p, SZ]),
        "mxfp4_gemv": (I, [P, I, I64, P, P, P, I64, P, I, I64, I64, I64, I64, I64, I, P]),
        "mxfp4_reserve_bytes": (I, [SZ, P]),
        "mxfp4_moe_route_workspace_bytes": (SZ, [I64, I64]),
        "mxfp4_moe_route": (I, [P, I, I64, P, I64, I64, I64, I, I, P, P, P, P, P, P, SZ, P]),
        "mxfp4_gemm_grouped_workspace_bytes": (SZ, [I64, I64, I64]),
        "mxfp4_gemm_grouped": (I, [P, I64, I64, P, P, I64, P, P, I64, P, I64, I64, I64, I64, I, P, SZ, P]),
        "mxfp4_moe_combine": (I, [P, I, I64, I64, P, P, P, I64, P, I, I64, I64, I64, I64, P]),
        "mxfp4_linear_workspace_bytes": (SZ, [I64, I64, I64]),
        "mxfp4_linear": (I, [P, I64, P, P, P, I, I, I, P, I64, P, I, I64, P, I64, I64, I64, I64, P, SZ, P]),
        "mxfp4_linear_grad_pre_workspace_bytes": (SZ, [I64, I64]),
        "mxfp4_linear_grad_pre": (I, [P, I, I64, P, I64, I, I, P, I64, P, I64, I64, P, SZ, P]),
        "mxfp4_linear_grad_input_workspace_bytes": (SZ, [I64, I64, I64]),
        "mxfp4_linear_grad_input": (I, [P, I64, P, P, P, I, I64, I64, I64, I64, P, SZ, P]),
        "mxfp4_linear_grad_weight_workspace_bytes": (SZ, [I64, I64, I64]),
        "mxfp4_linear_grad_weight": (I, [P, I64, P, I64, P, I, I64, I64, I64, I64, P, SZ, P]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def lib():
    return _load()


def exported_symbols():
    """Names every entry point the header declares (used by the ABI test)."""
    return ["mxfp4_packed_bytes", "mxfp4_raw_scale_bytes", "mxfp4_shuffled_scale_bytes",
            "mxfp4_gemm_workspace_bytes", "mxfp4_quantize", "mxfp4_preshuffle_b", "mxfp4_prepare_b", "mxfp4_gemm",
            "mxfp4_gemm_ex", "mxfp4_gemm_noalloc", "mxfp4_gemm_q", "mxfp4_gemm_q_schedule_name", "mxfp4_reserve", "mxfp4_status_string", "mxfp4_last_hip_error", "mxfp4_gemm_schedule_name",
            "mxfp4_set_quant_mode", "mxfp4_set_schedule_override", "mxfp4_list_schedules",
            "mxfp4_gemv", "mxfp4_reserve_bytes", "mxfp4_moe_route_workspace_bytes", "mxfp4_moe_route",
            "mxfp4_gemm_grouped_workspace_bytes", "mxfp4_gemm_grouped", "mxfp4_moe_combine",
            "mxfp4_linear_workspace_bytes", "mxfp4_linear", "mxfp4_linear_grad_pre_workspace_bytes",
            "mxfp4_linear_grad_pre", "mxfp4_linear_grad_input_workspace_bytes", "mxfp4_linear_grad_input",
            "mxfp4_linear_grad_weight_workspace_bytes", "mxfp4_linear_grad_weight"]


def _check(rc: int, what: str):
    if rc != MXFP4_OK:
        L = _load()
        msg = L.mxfp4_status_string(rc).decode()
        if rc == 4:  # MXFP4_ERR_HIP: name the HIP error
            msg += " (%s)" % L.mxfp4_last_hip_error().decode()
        raise RuntimeError("%s failed: %s" % (what, msg))


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None
_current_device = None


def _current_stream():
    """Handle of torch's current stream on the current device.

    torch.cuda.current_stream() builds a Stream object, 2.9 us a call; the two
    calls underneath it take 0.2 us together."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.current_stream()  # initializes torch's GPU state
        device, stream = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = (lambda: stream(device())) if device and stream else \
            (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---- sizes -----------------------------------------------------------------

def mxfp4_packed_bytes(rows: int, K: int) -> int:
    return _load().mxfp4_packed_bytes(rows, K)


def mxfp4_raw_scale_bytes(rows: int, K: int) -> int:
    return _load().mxfp4_raw_scale_bytes(rows, K)


def mxfp4_shuffled_scale_bytes(rows: int, K: int) -> int:
    return _load().mxfp4_shuffled_scale_bytes(rows, K)


def mxfp4_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return _load().mxfp4_gemm_workspace_bytes(M, N, K)


def mxfp4_gemm_schedule_name(M: int, N: int, K: int):
    r = _load().mxfp4_gemm_schedule_name(M, N, K)
    return r.decode() if r is not None else None


# ---- operations (raw: caller passes every buffer) --------------------------

def mxfp4_quantize(x, rows: int, K: int, q, scales, shuffled_scales: bool = False, stream=None):
    _check(_load().mxfp4_quantize(_ptr(x), rows, K, _ptr(q), _ptr(scales), int(bool(shuffled_scales)),
                                  _stream(stream)), "mxfp4_quantize")


def mxfp4_preshuffle_b(bq, bs_raw, N: int, K: int, bq_shuffled, bs_shuffled, stream=None):
    _check(_load().mxfp4_preshuffle_b(_ptr(bq), _ptr(bs_raw), N, K, _ptr(bq_shuffled), _ptr(bs_shuffled),
                                      _stream(stream)), "mxfp4_preshuffle_b")


def mxfp4_prepare_b(b, N: int, K: int, bq_shuffled, bs_shuffled, stream=None):
    _check(_load().mxfp4_prepare_b(_ptr(b), N, K, _ptr(bq_shuffled), _ptr(bs_shuffled), _stream(stream)),
           "mxfp4_prepare_b")


def mxfp4_gemm(A, Bq_sh, Bs_sh, C, M: int, N: int, K: int, stream=None):
    _check(_load().mxfp4_gemm(_ptr(A), _ptr(Bq_sh), _ptr(Bs_sh), _ptr(C), M, N, K, _stream(stream)), "mxfp4_gemm")


def mxfp4_gemm_ex(A, Bq_sh, Bs_sh, C, M: int, N: int, K: int, workspace, workspace_bytes: int, stream=None):
    _check(_load().mxfp4_gemm_ex(_ptr(A), _ptr(Bq_sh), _ptr(Bs_sh), _ptr(C), M, N, K, _ptr(workspace),
                                 workspace_bytes, _stream(stream)), "mxfp4_gemm_ex")


def mxfp4_gemm_noalloc(A, Bq_sh, Bs_sh, C, M: int, N: int, K: int, stream=None):
    _check(_load().mxfp4_gemm_noalloc(_ptr(A), _ptr(Bq_sh), _ptr(Bs_sh), _ptr(C), M, N, K, _stream(stream)),
           "mxfp4_gemm_noalloc")


def mxfp4_gemm_q(Aq, As, Bq_sh, Bs_sh, C, M: int, N: int, K: int, stream=None):
    _check(_load().mxfp4_gemm_q(_ptr(Aq), _ptr(As), _ptr(Bq_sh), _ptr(Bs_sh), _ptr(C), M, N, K, _stream(stream)),
           "mxfp4_gemm_q")


def mxfp4_gemm_q_schedule_name(M: int, N: int, K: int):
    r = _load().mxfp4_gemm_q_schedule_name(M, N, K)
    return r.decode() if r is not None else None


def mxfp4_reserve(M: int, N: int, K: int, stream=None):
    _check(_load().mxfp4_reserve(M, N, K, _stream(stream)), "mxfp4_reserve")


def mxfp4_set_quant_mode(mode: int):
    _check(_load().mxfp4_set_quant_mode(mode), "mxfp4_set_quant_mode")


def mxfp4_set_schedule_override(name):
    _check(_load().mxfp4_set_schedule_override(name.encode() if name else None), "mxfp4_set_schedule_override")


def mxfp4_list_schedules(M: int, N: int, K: int, quantized_a: bool = False):
    """Names of every compiled schedule that can serve (M, N, K) (empty for a
    shape outside the ABI); each is accepted by mxfp4_set_schedule_override."""
    L = _load()
    need = L.mxfp4_list_schedules(M, N, K, int(quantized_a), None, 0)
    if need == 0:
        return []
    buf = ctypes.create_string_buffer(need + 1)
    L.mxfp4_list_schedules(M, N, K, int(quantized_a), buf, need + 1)
    return buf.value.decode().split()


def mxfp4_gemv(x, x_type: int, ldx: int, Bq_sh, Bs_sh, ids, experts: int, y, y_type: int, ldy: int, M: int, N: int,
               K: int, repeat: int = 1, gated: bool = False, stream=None):
    _check(_load().mxfp4_gemv(_ptr(x), x_type, ldx, _ptr(Bq_sh), _ptr(Bs_sh), _ptr(ids), experts, _ptr(y), y_type, ldy,
                              M, N, K, repeat, int(bool(gated)), _stream(stream)), "mxfp4_gemv")


def mxfp4_reserve_bytes(nbytes: int, stream=None):
    _check(_load().mxfp4_reserve_bytes(nbytes, _stream(stream)), "mxfp4_reserve_bytes")


def mxfp4_moe_route_workspace_bytes(T: int, E: int) -> int:
    return _load().mxfp4_moe_route_workspace_bytes(T, E)


def mxfp4_moe_route(logits, x_type: int, ld: int, bias, T: int, E: int, k: int, score: int, renormalize: bool, ids,
                    weights, offsets, rows, pos, workspace=None, workspace_bytes: int = 0, stream=None):
    _check(_load().mxfp4_moe_route(_ptr(logits), x_type, ld, _ptr(bias), T, E, k, score, int(bool(renormalize)),
                                   _ptr(ids), _ptr(weights), _ptr(offsets), _ptr(rows), _ptr(pos), _ptr(workspace),
                                   workspace_bytes, _stream(stream)), "mxfp4_moe_route")


def mxfp4_gemm_grouped_workspace_bytes(R: int, K: int, experts: int) -> int:
    return _load().mxfp4_gemm_grouped_workspace_bytes(R, K, experts)


def mxfp4_gemm_grouped(A, lda: int, a_rows: int, Bq_sh, Bs_sh, experts: int, offsets, rows, repeat: int, C, ldc: int,
                       R: int, N: int, K: int, gated: bool = False, workspace=None, workspace_bytes: int = 0,
                       stream=None):
    _check(_load().mxfp4_gemm_grouped(_ptr(A), lda, a_rows, _ptr(Bq_sh), _ptr(Bs_sh), experts, _ptr(offsets),
                                      _ptr(rows), repeat, _ptr(C), ldc, R, N, K, int(bool(gated)), _ptr(workspace),
                                      workspace_bytes, _stream(stream)), "mxfp4_gemm_grouped")


def mxfp4_moe_combine(y, y_type: int, ld_y: int, rows: int, weights, pos, residual, ld_res: int, out, out_type: int,
                      ld_out: int, T: int, k: int, N: int, stream=None):
    _check(_load().mxfp4_moe_combine(_ptr(y), y_type, ld_y, rows, _ptr(weights), _ptr(pos), _ptr(residual), ld_res,
                                     _ptr(out), out_type, ld_out, T, k, N, _stream(stream)), "mxfp4_moe_combine")


def mxfp4_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return _load().mxfp4_linear_workspace_bytes(M, N, K)


def mxfp4_linear(x, ldx: int, Bq_sh, Bs_sh, bias, bias_type: int, activation: int, gated: bool, residual, ld_res: int,
                 y, y_type: int, ldy: int, pre, ld_pre: int, M: int, N: int, K: int, workspace=None,
                 workspace_bytes: int = 0, stream=None):
    _check(_load().mxfp4_linear(_ptr(x), ldx, _ptr(Bq_sh), _ptr(Bs_sh), _ptr(bias), bias_type, activation,
                                int(bool(gated)), _ptr(residual), ld_res, _ptr(y), y_type, ldy, _ptr(pre), ld_pre, M, N,
                                K, _ptr(workspace), workspace_bytes, _stream(stream)), "mxfp4_linear")


def mxfp4_linear_grad_pre_workspace_bytes(M: int, N: int) -> int:
    return _load().mxfp4_linear_grad_pre_workspace_bytes(M, N)


def mxfp4_linear_grad_pre(dy, dy_type: int, ld_dy: int, pre, ld_pre: int, activation: int, gated: bool, dz, ld_dz: int,
                          dbias, M: int, N: int, workspace=None, workspace_bytes: int = 0, stream=None):
    _check(_load().mxfp4_linear_grad_pre(_ptr(dy), dy_type, ld_dy, _ptr(pre), ld_pre, activation, int(bool(gated)),
                                         _ptr(dz), ld_dz, _ptr(dbias), M, N, _ptr(workspace), workspace_bytes,
                                         _stream(stream)), "mxfp4_linear_grad_pre")


def mxfp4_linear_grad_input_workspace_bytes(M: int, N: int, K: int) -> int:
    return _load().mxfp4_linear_grad_input_workspace_bytes(M, N, K)


def mxfp4_linear_grad_input(dz, ld_dz: int, Bq_sh, Bs_sh, dx, dx_type: int, ld_dx: int, M: int, N: int, K: int,
                            workspace=None, workspace_bytes: int = 0, stream=None):
    _check(_load().mxfp4_linear_grad_input(_ptr(dz), ld_dz, _ptr(Bq_sh), _ptr(Bs_sh), _ptr(dx), dx_type, ld_dx, M, N, K,
                                           _ptr(workspace), workspace_bytes, _stream(stream)), "mxfp4_linear_grad_input")


def mxfp4_linear_grad_weight_workspace_bytes(M: int, N: int, K: int) -> int:
    return _load().mxfp4_linear_grad_weight_workspace_bytes(M, N, K)


def mxfp4_linear_grad_weight(dz, ld_dz: int, x, ldx: int, dw, dw_type: int, ld_dw: int, M: int, N: int, K: int,
                             workspace=None, workspace_bytes: int = 0, stream=None):
    _check(_load().mxfp4_linear_grad_weight(_ptr(dz), ld_dz, _ptr(x), ldx, _ptr(dw), dw_type, ld_dw, M, N, K,
                                            _ptr(workspace), workspace_bytes, _stream(stream)),
           "mxfp4_linear_grad_weight")


# ---- tensor conveniences (allocate outputs with torch, then call the above) --

def _allocator(stream):
    """torch.empty for outputs that a kernel on `stream` writes.

    They lie in that stream's memory: memory of the current stream may still
    be in use by work there that `stream` does not wait for, and would be
    handed out again when the tensor is dropped, though the kernel may not
    have run yet.  They are recorded as used on the current stream, which is
    where the caller goes on with them."""
    import torch
    if stream is None:
        return torch.empty
    handle = _stream(stream)
    if handle == _current_stream():
        return torch.empty
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    current = torch.cuda.current_stream()

    def empty(*args, **kwargs):
        with torch.cuda.stream(stream):
            t = torch.empty(*args, **kwargs)
        if t.is_cuda:
            t.record_stream(current)
        return t

    return empty


def quantize(x, shuffled_scales: bool = False, stream=None):
    """bf16 [rows, K] cuda tensor -> (q uint8 [rows, K/2], scales uint8)."""
    import torch
    empty = _allocator(stream)
    rows, K = x.shape
    assert x.dtype == torch.bfloat16 and x.is_contiguous()
    q = empty((rows, K // 2), dtype=torch.uint8, device=x.device)
    if shuffled_scales:
        s = empty(mxfp4_shuffled_scale_bytes(rows, K), dtype=torch.uint8, device=x.device)
        s = s.view(-1, ((K // 32 + 7) // 8) * 32)
    else:
        s = empty((rows, K // 32), dtype=torch.uint8, device=x.device)
    mxfp4_quantize(x, rows, K, q, s, shuffled_scales, stream)
    return q, s


def preshuffle_b(bq, bs_raw, stream=None):
    """Quantized B (natural layouts) -> (Bw [N/16, (K/2)*16], Bs shuffled)."""
    import torch
    empty = _allocator(stream)
    N, KB = bq.shape
    K = KB * 2
    bw = empty((N // 16, KB * 16), dtype=torch.uint8, device=bq.device)
    bs = empty(mxfp4_shuffled_scale_bytes(N, K), dtype=torch.uint8, device=bq.device)
    bs = bs.view(-1, ((K // 32 + 7) // 8) * 32)
    mxfp4_preshuffle_b(bq, bs_raw, N, K, bw, bs, stream)
    return bw, bs


def prepare_b(b, stream=None):
    """bf16 [N, K] cuda tensor -> (Bw [N/16, (K/2)*16], Bs shuffled), in one launch."""
    import torch
    empty = _allocator(stream)
    N, K = b.shape
    assert b.dtype == torch.bfloat16 and b.is_contiguous()
    bw = empty((N // 16, (K // 2) * 16), dtype=torch.uint8, device=b.device)
    bs = empty(mxfp4_shuffled_scale_bytes(N, K), dtype=torch.uint8, device=b.device)
    bs = bs.view(-1, ((K // 32 + 7) // 8) * 32)
    mxfp4_prepare_b(b, N, K, bw, bs, stream)
    return bw, bs


def gemm_q(Aq, As, Bw, Bs, N: int, out=None, stream=None):
    """C = dequant(Aq, As) * B^T as bf16 [M, N]; Aq uint8 [M, K/2], As shuffled scales."""
    import torch
    M, KB = Aq.shape
    if out is None:
        out = _allocator(stream)((M, N), dtype=torch.bfloat16, device=Aq.device)
    mxfp4_gemm_q(Aq, As, Bw, Bs, out, M, N, 2 * KB, stream)
    return out


def gemm(A, Bw, Bs, N: int, out=None, stream=None):
    """C = Q(A) * B^T as bf16 [M, N]; A bf16 [M, K] cuda tensor."""
    import torch
    M, K = A.shape
    assert A.dtype == torch.bfloat16 and A.is_contiguous()
    if out is None:
        out = _allocator(stream)((M, N), dtype=torch.bfloat16, device=A.device)
    mxfp4_gemm(A, Bw, Bs, out, M, N, K, stream)
    return out


# ---- expert operators --------------------------------------------------------
#
# The checks below read each property of a tensor once: a call on one token
# takes its time on the host, and every property costs 50-150 ns.

MXFP4_TYPE_BF16, MXFP4_TYPE_F16, MXFP4_TYPE_F32 = 0, 1, 2

_torch = None
_types = {}
_forward_ad = None  # its _current_level is negative unless the caller works in forward mode
_increment_version = None


def _start():
    """torch and the library, once."""
    global _torch, _forward_ad, _increment_version
    L = _load()
    import torch
    import torch.autograd.forward_ad
    import torch.autograd.graph
    _forward_ad = torch.autograd.forward_ad
    if not hasattr(_forward_ad, "_current_level"):
        _forward_ad = types.SimpleNamespace(_current_level=0, unpack_dual=_forward_ad.unpack_dual)  # asks each tensor
    # without the isinstance of the public one, where there is it
    _increment_version = getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version
    _types.update({torch.bfloat16: MXFP4_TYPE_BF16, torch.float16: MXFP4_TYPE_F16, torch.float32: MXFP4_TYPE_F32})
    _torch = torch
    return L


def _type(t):
    """MXFP4_TYPE_* of a tensor's dtype."""
    r = _types.get(t.dtype)
    if r is None:
        raise TypeError("expected a bf16, f16 or f32 tensor, got %s" % t.dtype)
    return r


def _matrix(t, what, names):
    """Rows, columns, row stride and device of a matrix whose rows are contiguous."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be [%s]" % (what, names))
    rows, cols = shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError("%s must be a [%s] tensor with contiguous rows" % (what, names))
    return rows, cols, ld if rows > 1 else cols, t.get_device()


def _array(t, dtype, what, n, dev):
    if t.dtype is not dtype or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of %d elements on %s" % (what, dtype, n, _device(dev)))


def _device(dev):
    return "cuda:%d" % dev if dev >= 0 else "the cpu"


def _rows_of(t, what, rows, cols, dev):
    """Row stride of a [rows, cols] tensor whose rows are contiguous."""
    shape = t.shape
    if len(shape) == 2 and shape[0] == rows and shape[1] == cols and t.get_device() == dev:
        ld, step = t.stride()
        if step == 1 or cols <= 1:
            return ld if shape[0] > 1 else cols
    raise ValueError("%s must be a [%d, %d] tensor on %s with contiguous rows" %
                     (what, rows, cols, _device(dev)))


def _no_gradients(what, how="and the expert operators have none"):
    """For an input that requires gradients: refuses a call that autograd would follow."""
    if _torch.is_grad_enabled():
        raise RuntimeError("%s requires gradients, %s: detach it, or call under torch.no_grad()" % (what, how))


@functools.lru_cache(maxsize=1024)
def _prepared_bytes(N, K):
    return mxfp4_packed_bytes(N, K), mxfp4_shuffled_scale_bytes(N, K)


def _prepared(Bw, Bs, N, K, dev):
    """Number of matrices in prepared codes and scales; checks their sizes."""
    per_w, per_s = _prepared_bytes(N, K)
    total = Bw.nbytes
    E = total // per_w if per_w else 0
    if E < 1 or total != E * per_w or Bs.nbytes != E * per_s \
            or not Bw.is_contiguous() or not Bs.is_contiguous() or Bw.get_device() != dev or Bs.get_device() != dev:
        raise ValueError("Bw and Bs must be contiguous byte tensors of prepared [%d, %d] matrices on %s" %
                         (N, K, _device(dev)))
    return E


def _on_gpu(dev):
    """A launch goes to the current device; tensors of another would be read from there."""
    global _current_device
    if dev < 0:
        raise ValueError("the operators take cuda tensors")
    if _current_device is None:
        import torch
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if dev != _current_device():
        raise ValueError("the tensors are on cuda:%d, the current device is cuda:%d" % (dev, _current_device()))


def _workspace(ws, dev):
    """Address and bytes of a caller's workspace."""
    if ws.get_device() != dev or not ws.is_contiguous() or ws.is_meta:
        raise ValueError("workspace must be a contiguous tensor on %s" % _device(dev))
    return ws.data_ptr(), ws.nbytes


def prepare_experts(B, stream=None):
    """bf16 [E, N, K] cuda tensor -> (Bw [E, N/16, (K/2)*16], Bs [E, ...]): each matrix prepared as by prepare_b."""
    import torch
    E, N, K = B.shape
    assert B.dtype == torch.bfloat16 and B.is_contiguous()
    empty = _allocator(stream)
    bw = empty((E, N // 16, (K // 2) * 16), dtype=torch.uint8, device=B.device)
    bs = empty(E * mxfp4_shuffled_scale_bytes(N, K), dtype=torch.uint8, device=B.device)
    bs = bs.view(E, -1, ((K // 32 + 7) // 8) * 32)
    for e in range(E):
        mxfp4_prepare_b(B[e], N, K, bw[e], bs[e], stream)
    return bw, bs


def gemv(x, Bw, Bs, N: int, ids=None, repeat: int = 1, gated: bool = False, out=None, out_dtype=None, stream=None):
    """y = x * B^T for few rows of unquantized bf16, f16 or f32 activations.

    x [M, K] with contiguous rows; Bw, Bs from prepare_b.  With ids (int32,
    one per row of y) Bw and Bs hold several matrices (prepare_experts), row r
    of y takes matrix ids[r] and row r // repeat of x, and a row whose id is
    none of them is zero.  gated: N/2 columns, silu(first half) * second.
    y's type is out's, else out_dtype, else x's."""
    L = _lib if _torch else _start()
    torch = _torch
    tokens, K, ldx, dev = _matrix(x, "x", "M, K")
    xt = _type(x)
    if x.requires_grad:
        _no_gradients("x")
    E = _prepared(Bw, Bs, N, K, dev)
    M = tokens * repeat
    if ids is not None:
        _array(ids, torch.int32, "ids", M, dev)
        ids = ids.data_ptr()
    elif E != 1:
        raise ValueError("%d matrices need ids" % E)
    cols = N // 2 if gated else N
    if out is None:
        out = (torch.empty if stream is None else _allocator(stream))((M, cols), dtype=out_dtype or x.dtype, device=x.device)
        ldy = cols
    else:
        ldy = _rows_of(out, "out", M, cols, dev)
    yt = _type(out)
    _on_gpu(dev)
    if M:
        rc = L.mxfp4_gemv(x.data_ptr(), xt, ldx, Bw.data_ptr(), Bs.data_ptr(), ids, E, out.data_ptr(), yt, ldy, M, N,
                                K, repeat, 1 if gated else 0, _current_stream() if stream is None else _stream(stream))
        if rc:
            _check(rc, "mxfp4_gemv")
    return out


def gemm_grouped(A, Bw, Bs, offsets, N: int, rows=None, repeat: int = 1, gated: bool = False, out=None, stream=None,
                 workspace=None):
    """C[p] = Q(A[row(p)]) * B_e^T for offsets[e] <= p < offsets[e + 1], bf16.

    A [a_rows, K] bf16 with contiguous rows; Bw, Bs E matrices from
    prepare_experts; offsets int32 [E + 1].  row(p) is rows[p] // repeat (int32
    [R], from moe_route with repeat = k), or p without rows.  gated: N/2
    columns, silu(first half) * second.  Rows of no group are zero.

    workspace: a cuda tensor of mxfp4_gemm_grouped_workspace_bytes(R, K, E)
    bytes that no other work uses meanwhile; without one the library's of the
    stream serves.  A graph keeps the one it was captured with, so graphs that
    are replayed at the same time need one each."""
    L = _lib if _torch else _start()
    ws, ws_bytes = None, 0
    torch = _torch
    T, K, lda, dev = _matrix(A, "A", "rows, K")
    if A.dtype != torch.bfloat16:
        raise TypeError("A must be bf16, not %s" % A.dtype)
    if A.requires_grad:
        _no_gradients("A")
    E = _prepared(Bw, Bs, N, K, dev)
    _array(offsets, torch.int32, "offsets", E + 1, dev)
    if rows is not None:
        R = rows.numel()
        _array(rows, torch.int32, "rows", R, dev)
        rows = rows.data_ptr()
    else:
        R = T
    cols = N // 2 if gated else N
    if out is None:
        out = (torch.empty if stream is None else _allocator(stream))((R, cols), dtype=torch.bfloat16, device=A.device)
        ldc = cols
    else:
        ldc = _rows_of(out, "out", R, cols, dev)
        if out.dtype != torch.bfloat16:
            raise TypeError("out must be bf16, not %s" % out.dtype)
    if workspace is not None:
        ws, ws_bytes = _workspace(workspace, dev)
    _on_gpu(dev)
    rc = L.mxfp4_gemm_grouped(A.data_ptr(), lda, T, Bw.data_ptr(), Bs.data_ptr(), E, offsets.data_ptr(), rows, repeat,
                                    out.data_ptr(), ldc, R, N, K, 1 if gated else 0, ws, ws_bytes,
                                    _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "mxfp4_gemm_grouped")
    return out


_scores = {"softmax": 0, "sigmoid": 1}


def moe_route(logits, k: int, score: str = "softmax", bias=None, renormalize: bool = True, out=None, stream=None,
              workspace=None):
    """The k experts of each token and the (token, choice) pairs sorted by expert.

    logits [T, E], bf16, f16 or f32, with contiguous rows; score "softmax" or
    "sigmoid" gives g; the experts of the largest g (+ bias, f32 [E]) are
    chosen, never one whose logit or bias is -inf or NaN.  Returns (or fills,
    if given as out):
      ids     int32 [T, k], -1 where no expert was left
      weights f32 [T, k], g of the chosen, renormalized to sum 1 if asked
      offsets int32 [E + 1], where each expert's pairs lie in rows
      rows    int32 [T * k], the pair t * k + j at each sorted place, or -1
      pos     int32 [T, k], the sorted place of each pair, or -1
    workspace: as for gemm_grouped, of mxfp4_moe_route_workspace_bytes(T, E) bytes."""
    L = _lib if _torch else _start()
    ws, ws_bytes = None, 0
    torch = _torch
    T, E, ld, dev = _matrix(logits, "logits", "T, E")
    lt = _type(logits)
    if logits.requires_grad:
        _no_gradients("logits")
    kind = _scores.get(score)
    if kind is None:
        raise ValueError("score must be 'softmax' or 'sigmoid', not %r" % (score,))
    if bias is not None:
        _array(bias, torch.float32, "bias", E, dev)
        if bias.requires_grad:
            _no_gradients("bias")
        bias = bias.data_ptr()
    n = T * k
    if out is None:
        i32 = dict(dtype=torch.int32, device=logits.device)
        empty = torch.empty if stream is None else _allocator(stream)
        out = (empty((T, k), **i32), empty((T, k), dtype=torch.float32, device=logits.device),
               empty(E + 1, **i32), empty(n, **i32), empty((T, k), **i32))
        ids, weights, offsets, rows, pos = out
    else:
        ids, weights, offsets, rows, pos = out
        _array(ids, torch.int32, "ids", n, dev)
        _array(weights, torch.float32, "weights", n, dev)
        _array(offsets, torch.int32, "offsets", E + 1, dev)
        _array(rows, torch.int32, "rows", n, dev)
        _array(pos, torch.int32, "pos", n, dev)
    if workspace is not None:
        ws, ws_bytes = _workspace(workspace, dev)
    _on_gpu(dev)
    rc = L.mxfp4_moe_route(logits.data_ptr(), lt, ld, bias, T, E, k, kind, 1 if renormalize else 0, ids.data_ptr(),
                                 weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), pos.data_ptr(), ws, ws_bytes,
                                 _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "mxfp4_moe_route")
    return out


def moe_combine(y, weights, pos=None, residual=None, out=None, out_dtype=None, stream=None):
    """out[t] = residual[t] + sum_j weights[t, j] * y[pos[t, j]].

    y [rows, N], bf16, f16 or f32, with contiguous rows; weights f32 [T, k]; pos
    int32 [T, k] (row t * k + j without it; a place outside y adds nothing);
    residual [T, N] of out's type, which may be out itself.  out's type is
    out's, else out_dtype, else residual's, else bf16."""
    L = _lib if _torch else _start()
    torch = _torch
    R, N, ld_y, dev = _matrix(y, "y", "rows, N")
    shape = weights.shape
    if len(shape) != 2:
        raise ValueError("weights must be [T, k]")
    T, k = shape
    yt = _type(y)
    _array(weights, torch.float32, "weights", T * k, dev)
    if y.requires_grad or weights.requires_grad:
        _no_gradients("y" if y.requires_grad else "weights")
    if pos is not None:
        _array(pos, torch.int32, "pos", T * k, dev)
        pos = pos.data_ptr()
    elif R < T * k:
        raise ValueError("y has %d rows, %d tokens of %d choices need %d" % (R, T, k, T * k))
    if out is None:
        dtype = out_dtype or (residual.dtype if residual is not None else torch.bfloat16)
        out = (torch.empty if stream is None else _allocator(stream))((T, N), dtype=dtype, device=y.device)
        ld_out = N
    else:
        ld_out = _rows_of(out, "out", T, N, dev)
    ld_res = N
    dtype = out.dtype
    if residual is not None:
        ld_res = _rows_of(residual, "residual", T, N, dev)
        if residual.dtype != dtype:
            raise TypeError("residual is %s, out %s" % (residual.dtype, dtype))
        if residual.requires_grad:
            _no_gradients("residual")
        residual = residual.data_ptr()
    ot = _types.get(dtype)
    if ot is None:
        raise TypeError("expected a bf16, f16 or f32 out, got %s" % dtype)
    _on_gpu(dev)
    rc = L.mxfp4_moe_combine(y.data_ptr(), yt, ld_y, R, weights.data_ptr(), pos, residual, ld_res, out.data_ptr(), ot,
                                   ld_out, T, k, N, _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "mxfp4_moe_combine")
    return out


# ---- dense layers --------------------------------------------------------------

MXFP4_ACT_NONE, MXFP4_ACT_RELU, MXFP4_ACT_SILU, MXFP4_ACT_GELU, MXFP4_ACT_GELU_TANH = range(5)

_activations = {None: MXFP4_ACT_NONE, "none": MXFP4_ACT_NONE, "relu": MXFP4_ACT_RELU, "silu": MXFP4_ACT_SILU,
                "gelu": MXFP4_ACT_GELU, "gelu_tanh": MXFP4_ACT_GELU_TANH}


def _activation(name):
    kind = _activations.get(name)
    if kind is None:
        raise ValueError("activation must be None, 'none', 'relu', 'silu', 'gelu' or 'gelu_tanh', not %r" % (name,))
    return kind


def _tracked(what):
    """A tensor, input or output, requires gradients: refused where autograd would follow it."""
    _no_gradients(what, "which autograd does not follow through this call (mx.linear_grad_* compute them)")


def _no_tangents(**tensors):
    """Refuses tensors that carry a tangent; `requires_grad` does not show it.  Asking costs 0.3 us a tensor, so
    callers look at the level first."""
    for what, t in tensors.items():
        if isinstance(t, _torch.Tensor) and _forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError("%s carries a forward-mode tangent, which autograd does not follow through this call" % what)


def _bf16(t, what):
    if t.dtype is not _torch.bfloat16:
        raise TypeError("%s must be bf16, not %s" % (what, t.dtype))


def _output(out, rows, cols, dtype, like, dev, stream):
    """The output tensor, its MXFP4_TYPE_* and its row stride."""
    if out is None:
        out = (_torch.empty if stream is None else _allocator(stream))((rows, cols), dtype=dtype, device=like.device)
        return out, _type(out), cols
    if out.requires_grad:
        _tracked("out")
    return out, _type(out), _rows_of(out, "out", rows, cols, dev)


def linear(x, Bw, Bs, N: int, bias=None, activation=None, gated: bool = False, residual=None, pre=None, out=None,
           out_dtype=None, stream=None, workspace=None):
    """A dense layer: z = Q(x) * B^T + bias, y = f(z) + residual.

    x [M, K] bf16 with contiguous rows; Bw, Bs from prepare_b; bias [N], bf16,
    f16 or f32; activation f None, "relu", "silu", "gelu" or "gelu_tanh" (of the
    f32 z); residual [M, columns] of y's type, which may be out itself.
    gated: y = f(z's first half) * z's second half + residual, N/2 columns.
    y's type is out's, else out_dtype, else residual's, else bf16.

    pre: a bf16 [M, N] tensor that receives z, or True for a new one; the call
    then returns (y, z), and linear_grad_pre takes z.
    Tensors that are given to be written (here and in the gradients) count as
    changed in place: a backward pass that saved one of them says so.
    workspace: as for gemm_grouped, of mxfp4_linear_workspace_bytes(M, N, K) bytes."""
    L = _lib if _torch else _start()
    torch = _torch
    ws, ws_bytes = None, 0
    written = () if out is None else (out,)
    if _forward_ad._current_level >= 0:
        _no_tangents(x=x, bias=bias, residual=residual, pre=pre, out=out)
    M, K, ldx, dev = _matrix(x, "x", "M, K")
    _bf16(x, "x")
    if x.requires_grad:
        _tracked("x")
    kind = _activation(activation)
    if _prepared(Bw, Bs, N, K, dev) != 1:
        raise ValueError("Bw and Bs must hold one matrix")
    cols = N // 2 if gated else N
    bias_type = 0
    if bias is not None:
        bias_type = _type(bias)
        _array(bias, bias.dtype, "bias", N, dev)
        if bias.requires_grad:
            _tracked("bias")
        bias = bias.data_ptr()
    out, yt, ldy = _output(out, M, cols, out_dtype or (torch.bfloat16 if residual is None else residual.dtype), x, dev,
                           stream)
    ld_res = cols
    if residual is not None:
        ld_res = _rows_of(residual, "residual", M, cols, dev)
        if residual.dtype != out.dtype:
            raise TypeError("residual is %s, out %s" % (residual.dtype, out.dtype))
        if residual.requires_grad:
            _tracked("residual")
        residual = residual.data_ptr()
    z, ld_pre = None, N
    if pre is True:
        pre = (torch.empty if stream is None else _allocator(stream))((M, N), dtype=torch.bfloat16, device=x.device)
        z = pre.data_ptr()
    elif pre is not None and pre is not False:
        _bf16(pre, "pre")
        ld_pre = _rows_of(pre, "pre", M, N, dev)
        if pre.requires_grad:
            _tracked("pre")
        z = pre.data_ptr()
        written += (pre,)
    if workspace is not None:
        ws, ws_bytes = _workspace(workspace, dev)
    _on_gpu(dev)
    rc = L.mxfp4_linear(x.data_ptr(), ldx, Bw.data_ptr(), Bs.data_ptr(), bias, bias_type, kind, 1 if gated else 0,
                        residual, ld_res, out.data_ptr(), yt, ldy, z, ld_pre, M, N, K, ws, ws_bytes,
                        _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "mxfp4_linear")
    if written:
        _increment_version(written)
    return out if z is None and not isinstance(pre, torch.Tensor) else (out, pre)


def linear_grad_pre(dy, pre, activation=None, gated: bool = False, bias=False, out=None, stream=None, workspace=None):
    """The gradient of z in linear, bf16 [M, N], from that of y.

    dy [M, columns of y], bf16, f16 or f32, with contiguous rows; pre the z
    that linear kept (None where it has neither activation nor gate, when z is
    not read).  bias: True, or an f32 [N] tensor to fill: returns (dz, dbias),
    dbias the sum of the rows of dz, formed before dz is rounded.  out may be pre
    itself.
    workspace: as for gemm_grouped, of mxfp4_linear_grad_pre_workspace_bytes(M, N)
    bytes; without bias none is needed."""
    L = _lib if _torch else _start()
    torch = _torch
    ws, ws_bytes = None, 0
    written = () if out is None else (out,)
    if _forward_ad._current_level >= 0:
        _no_tangents(dy=dy, pre=pre, bias=bias, out=out)
    M, cols, ld_dy, dev = _matrix(dy, "dy", "M, columns")
    dt = _type(dy)
    if dy.requires_grad:
        _tracked("dy")
    kind = _activation(activation)
    N = 2 * cols if gated else cols
    z, ld_pre = None, N
    if pre is not None:
        _bf16(pre, "pre")
        ld_pre = _rows_of(pre, "pre", M, N, dev)
        if pre.requires_grad:
            _tracked("pre")
        z = pre.data_ptr()
    elif kind or gated:
        raise ValueError("an activation or a gate needs pre")
    if out is not None:
        _bf16(out, "out")
    out, _, ld_dz = _output(out, M, N, torch.bfloat16, dy, dev, stream)
    db = None
    if isinstance(bias, torch.Tensor):
        db = bias
        _array(db, torch.float32, "bias", N, dev)
        if db.requires_grad:
            _tracked("bias")
        written += (db,)
    elif bias:
        db = (torch.empty if stream is None else _allocator(stream))((N,), dtype=torch.float32, device=dy.device)
    if workspace is not None:
        ws, ws_bytes = _workspace(workspace, dev)
    _on_gpu(dev)
    rc = L.mxfp4_linear_grad_pre(dy.data_ptr(), dt, ld_dy, z, ld_pre, kind, 1 if gated else 0, out.data_ptr(), ld_dz,
                                 None if db is None else db.data_ptr(), M, N, ws, ws_bytes,
                                 _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "mxfp4_linear_grad_pre")
    if written:
        _increment_version(written)
    return out if db is None else (out, db)


def linear_grad_input(dz, Bw, Bs, K: int, out=None, out_dtype=None, stream=None, workspace=None):
    """The gradient of x in linear: dx = dz * B, [M, K].

    dz [M, N] bf16 with contiguous rows; Bw, Bs the prepared [N, K] matrix.
    dx's type is out's, else out_dtype, else bf16.
    workspace: as for gemm_grouped, of mxfp4_linear_grad_input_workspace_bytes(M, N, K) bytes."""
    L = _lib if _torch else _start()
    ws, ws_bytes = None, 0
    written = () if out is None else (out,)
    if _forward_ad._current_level >= 0:
        _no_tangents(dz=dz, out=out)
    M, N, ld_dz, dev = _matrix(dz, "dz", "M, N")
    _bf16(dz, "dz")
    if dz.requires_grad:
        _tracked("dz")
    if _prepared(Bw, Bs, N, K, dev) != 1:
        raise ValueError("Bw and Bs must hold one matrix")
    out, xt, ld_dx = _output(out, M, K, out_dtype or _torch.bfloat16, dz, dev, stream)
    if workspace is not None:
        ws, ws_bytes = _workspace(workspace, dev)
    _on_gpu(dev)
    rc = L.mxfp4_linear_grad_input(dz.data_ptr(), ld_dz, Bw.data_ptr(), Bs.data_ptr(), out.data_ptr(), xt, ld_dx, M, N, K,
                                   ws, ws_bytes, _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "mxfp4_linear_grad_input")
    if written:
        _increment_version(written)
    return out


def linear_grad_weight(dz, x, out=None, out_dtype=None, stream=None, workspace=None):
    """The gradient of the weights in linear: dw = dz^T * Q(x), [N, K].

    dz [M, N] and x [M, K] bf16 with contiguous rows.  dw's type is out's, else
    out_dtype, else f32.
    workspace: as for gemm_grouped, of mxfp4_linear_grad_weight_workspace_bytes(M, N, K) bytes."""
    L = _lib if _torch else _start()
    ws, ws_bytes = None, 0
    written = () if out is None else (out,)
    if _forward_ad._current_level >= 0:
        _no_tangents(dz=dz, x=x, out=out)
    M, N, ld_dz, dev = _matrix(dz, "dz", "M, N")
    _bf16(dz, "dz")
    if dz.requires_grad:
        _tracked("dz")
    rows, K, ldx, x_dev = _matrix(x, "x", "M, K")
    if rows != M or x_dev != dev:
        raise ValueError("x must have dz's %d rows on %s" % (M, _device(dev)))
    _bf16(x, "x")
    if x.requires_grad:
        _tracked("x")
    out, wt, ld_dw = _output(out, N, K, out_dtype or _torch.float32, dz, dev, stream)
    if workspace is not None:
        ws, ws_bytes = _workspace(workspace, dev)
    _on_gpu(dev)
    rc = L.mxfp4_linear_grad_weight(dz.data_ptr(), ld_dz, x.data_ptr(), ldx, out.data_ptr(), wt, ld_dw, M, N, K, ws,
                                    ws_bytes, _current_stream() if stream is None else _stream(stream))
    if rc:
        _check(rc, "mxfp4_linear_grad_weight")
    if written:
        _increment_version(written)
    return out
