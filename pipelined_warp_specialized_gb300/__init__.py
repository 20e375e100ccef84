"""Python binding of the pipelined, warp-specialized GEMM library (sm_103a).

Argument marshalling only: every function here forwards to the entry point of
the same name in the C ABI (``include/pwsgemm.h``), implemented by the CUDA
library ``_build/libpwsgemm.so``.  PyTorch supplies device memory and streams.
There is no fallback: if the library is missing or fails to load, every call
raises.

    import torch, pipelined_warp_specialized_gb300 as pws
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.float16)   # lhs [M, K]
    b = torch.randn(4096, 4096, device="cuda", dtype=torch.float16)   # rhs [N, K]
    c = pws.gemm_f16_nt(a, b, stages=4)                               # a @ b.T, f16
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libpwsgemm.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "pwsgemm.h")

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_ALIGNMENT = 2
GEMM_ERR_UNSUPPORTED_STAGES = 3
GEMM_ERR_UNSUPPORTED_ARCH = 4
GEMM_ERR_LAUNCH = 5
GEMM_ERR_TIMEOUT = 6

GEMM_DEBUG_SKIP_EMPTY_SEED = 1
GEMM_DEBUG_FORCE_COPY_PRODUCER = 2
GEMM_DEBUG_FORCE_DIRECT_STORE = 4
GEMM_DEBUG_FORCE_SOLO_TILE = 8
GEMM_DEBUG_FORCE_PAIR_TILE = 16
GEMM_DEBUG_NO_SPLIT = 32
GEMM_DEBUG_FORCE_NARROW_TILE = 64
GEMM_DEBUG_FORCE_WIDE_TILE = 128
GEMM_DEBUG_SKIP_ACC_SEED = 256
GEMM_DEBUG_NO_KSPLIT = 512
GEMM_DEBUG_FORCE_KSPLIT = 1024
GEMM_DEBUG_SKIP_KSPLIT_SEND = 2048
GEMM_DEBUG_FORCE_DOUBLE_SLOT = 4096
GEMM_DEBUG_NO_DOUBLE_SLOT = 8192
GEMM_DEBUG_IN_PLACE = 16384

GEMM_TYPE_HALF = 0
GEMM_TYPE_BFLOAT = 1
GEMM_ACT_SILU = 0
GEMM_ACT_GELU = 1
_ACTS = {"silu": GEMM_ACT_SILU, "gelu": GEMM_ACT_GELU}

_lib = None


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Loads the CUDA library (building nothing); raises if it is absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"the CUDA library {p} is not built; run "
                          "`python -m pipelined_warp_specialized_gb300.build`")
    lib = ctypes.CDLL(p)
    i64, i32, vp, u32, u64 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_uint, ctypes.c_uint64
    lib.gemm_s32_nn.argtypes = [i64, i64, i64, vp, vp, vp, vp]
    lib.gemm_s32_nn.restype = i32
    lib.gemm_s32_nn_ring.argtypes = [i64, i64, i64, vp, vp, vp, i32, vp]
    lib.gemm_s32_nn_ring.restype = i32
    lib.gemm_f16_nt.argtypes = [i64, i64, i64, vp, vp, vp, i32, vp]
    lib.gemm_f16_nt.restype = i32
    lib.gemm_f16_nt_noalloc.argtypes = [i64, i64, i64, vp, vp, vp, i32, vp]
    lib.gemm_f16_nt_noalloc.restype = i32
    lib.gemm_device_status.argtypes = [vp]
    lib.gemm_device_status.restype = i32
    lib.gemm_status_string.argtypes = [i32]
    lib.gemm_status_string.restype = ctypes.c_char_p
    lib.gemm_set_wait_timeout_ns.argtypes = [u64]
    lib.gemm_set_wait_timeout_ns.restype = i32
    lib.gemm_set_debug_flags.argtypes = [u32]
    lib.gemm_set_debug_flags.restype = i32
    lib.gemm_set_scratch_pool.argtypes = [i32]
    lib.gemm_set_scratch_pool.restype = i32
    lib.gemm_f16_nt_plan.argtypes = [i64, i64, i64, vp, vp, vp, i32, ctypes.POINTER(i64)]
    lib.gemm_f16_nt_plan.restype = i32
    pi64 = ctypes.POINTER(i64)
    for name, args in (
            ("gemm_gated_nt", [i64] * 3 + [vp] * 6 + [i32, i32, vp, i64, vp]),
            ("gemm_gated_nt_workspace", [i64] * 3 + [vp] * 3 + [i32, pi64]),
            ("gemm_gated_nt_bwd", [i64] * 3 + [vp] * 9 + [i32, i32, vp, i64, vp]),
            ("gemm_gated_nt_bwd_workspace", [i64] * 3 + [vp] * 6 + [i32, pi64]),
            ("gemm_xent_nt", [i64] * 3 + [vp] * 3 + [i64, vp, vp, i32, vp, i64, vp]),
            ("gemm_xent_nt_workspace", [i64] * 3 + [vp] * 2 + [i32, pi64]),
            ("gemm_xent_nt_bwd", [i64] * 3 + [vp] * 3 + [i64] + [vp] * 4 + [i32, vp, i64, vp]),
            ("gemm_xent_nt_bwd_workspace", [i64] * 3 + [vp] * 2 + [i32, pi64]),
            ("gemm_nt_bwd", [i64] * 3 + [vp] * 5 + [i32, vp, i64, vp]),
            ("gemm_nt_bwd_workspace", [i64] * 3 + [vp] * 3 + [i32, pi64])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i32
    if path is None:
        _lib = lib
    return lib


def header_functions(header: str = HEADER) -> list:
    """Names of the functions ``include/pwsgemm.h`` declares."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:int|const char\s*\*)\s*(\w+)\s*\(", text, flags=re.M)


def status_string(status: int) -> str:
    try:
        return load_library().gemm_status_string(int(status)).decode()
    except ImportError:
        return f"status {status}"


def _stream_ptr(stream, device) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, what: str) -> None:
    if status != GEMM_OK:
        raise GemmError(status, what)


def _same_device(name, lhs, rhs, out):
    """Every operand must live on lhs's device: the call launches there, and a
    pointer into another GPU's memory is not valid on it."""
    devs = {t.device for t in (lhs, rhs, out) if t is not None}
    if len(devs) > 1:
        raise ValueError(f"{name}: lhs, rhs and out must be on one device, got {sorted(map(str, devs))}")


def gemm_s32_nn(lhs, rhs, out=None, stream=None):
    """out[M,N] = lhs[M,K] @ rhs[K,N] over int32 (wrapping), on lhs's device."""
    import torch
    if lhs.dtype != torch.int32 or rhs.dtype != torch.int32:
        raise TypeError("gemm_s32_nn takes int32 tensors")
    if lhs.dim() != 2 or rhs.dim() != 2 or lhs.shape[1] != rhs.shape[0]:
        raise ValueError(f"shapes {tuple(lhs.shape)} x {tuple(rhs.shape)} do not form [M,K] x [K,N]")
    if not (lhs.is_cuda and rhs.is_cuda) or not lhs.is_contiguous() or not rhs.is_contiguous():
        raise ValueError("gemm_s32_nn takes contiguous CUDA tensors")
    _same_device("gemm_s32_nn", lhs, rhs, out)
    M, K = lhs.shape
    N = rhs.shape[1]
    if out is None:
        out = torch.empty((M, N), dtype=torch.int32, device=lhs.device)
    elif out.shape != (M, N) or out.dtype != torch.int32 or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous int32 CUDA tensor of shape [M, N]")
    with torch.cuda.device(lhs.device):
        _check(load_library().gemm_s32_nn(M, N, K, lhs.data_ptr(), rhs.data_ptr(), out.data_ptr(),
                                          _stream_ptr(stream, lhs.device)), "gemm_s32_nn")
    return out


def gemm_s32_nn_ring(lhs, rhs, out=None, stages: int = 4, stream=None):
    """gemm_s32_nn with an S-slot ring (S = `stages`, 2..6); bit-identical results."""
    import torch
    if lhs.dtype != torch.int32 or rhs.dtype != torch.int32:
        raise TypeError("gemm_s32_nn_ring takes int32 tensors")
    if lhs.dim() != 2 or rhs.dim() != 2 or lhs.shape[1] != rhs.shape[0]:
        raise ValueError(f"shapes {tuple(lhs.shape)} x {tuple(rhs.shape)} do not form [M,K] x [K,N]")
    if not (lhs.is_cuda and rhs.is_cuda) or not lhs.is_contiguous() or not rhs.is_contiguous():
        raise ValueError("gemm_s32_nn_ring takes contiguous CUDA tensors")
    _same_device("gemm_s32_nn_ring", lhs, rhs, out)
    M, K = lhs.shape
    N = rhs.shape[1]
    if out is None:
        out = torch.empty((M, N), dtype=torch.int32, device=lhs.device)
    elif out.shape != (M, N) or out.dtype != torch.int32 or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous int32 CUDA tensor of shape [M, N]")
    with torch.cuda.device(lhs.device):
        _check(load_library().gemm_s32_nn_ring(M, N, K, lhs.data_ptr(), rhs.data_ptr(), out.data_ptr(), int(stages),
                                               _stream_ptr(stream, lhs.device)), "gemm_s32_nn_ring")
    return out


def gemm_f16_nt(lhs, rhs, out=None, stages: int = 4, stream=None):
    """out[M,N] = f16(lhs[M,K] @ rhs[N,K].T) with fp32 accumulation, S = `stages` ring slots.

    Not recorded by autograd: the gradients are gemm_nt_bwd's.
    """
    import torch
    if lhs.dtype != torch.float16 or rhs.dtype != torch.float16:
        raise TypeError("gemm_f16_nt takes float16 tensors")
    if lhs.dim() != 2 or rhs.dim() != 2 or lhs.shape[1] != rhs.shape[1]:
        raise ValueError(f"shapes {tuple(lhs.shape)} x {tuple(rhs.shape)} do not form [M,K] x [N,K]")
    if not (lhs.is_cuda and rhs.is_cuda) or not lhs.is_contiguous() or not rhs.is_contiguous():
        raise ValueError("gemm_f16_nt takes contiguous CUDA tensors")
    _same_device("gemm_f16_nt", lhs, rhs, out)
    _not_recorded("gemm_f16_nt", "gemm_nt_bwd", lhs, rhs)
    M, K = lhs.shape
    N = rhs.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=lhs.device)
    elif out.shape != (M, N) or out.dtype != torch.float16 or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous float16 CUDA tensor of shape [M, N]")
    with torch.cuda.device(lhs.device):
        _check(load_library().gemm_f16_nt(M, N, K, lhs.data_ptr(), rhs.data_ptr(), out.data_ptr(), int(stages),
                                          _stream_ptr(stream, lhs.device)), "gemm_f16_nt")
    return out


def gemm_f16_nt_noalloc(lhs, rhs, out=None, stages: int = 4, stream=None):
    """gemm_f16_nt for callers that cannot allocate device memory.

    Where gemm_f16_nt would take scratch from its pool, this uses a fixed
    32 MiB device array loaded with the library, so no allocator is entered
    (for code under a fixed memory budget or that must not allocate).  Calls
    share that array: calls that can overlap on the GPU must be ordered.
    Raises GemmError(GEMM_ERR_INVALID_ARG) when more scratch would be needed.
    ``out`` should be preallocated by such callers (None allocates it here).
    """
    import torch
    if lhs.dtype != torch.float16 or rhs.dtype != torch.float16:
        raise TypeError("gemm_f16_nt_noalloc takes float16 tensors")
    if lhs.dim() != 2 or rhs.dim() != 2 or lhs.shape[1] != rhs.shape[1]:
        raise ValueError(f"shapes {tuple(lhs.shape)} x {tuple(rhs.shape)} do not form [M,K] x [N,K]")
    if not (lhs.is_cuda and rhs.is_cuda) or not lhs.is_contiguous() or not rhs.is_contiguous():
        raise ValueError("gemm_f16_nt_noalloc takes contiguous CUDA tensors")
    _same_device("gemm_f16_nt_noalloc", lhs, rhs, out)
    M, K = lhs.shape
    N = rhs.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=lhs.device)
    elif out.shape != (M, N) or out.dtype != torch.float16 or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous float16 CUDA tensor of shape [M, N]")
    with torch.cuda.device(lhs.device):
        _check(load_library().gemm_f16_nt_noalloc(M, N, K, lhs.data_ptr(), rhs.data_ptr(), out.data_ptr(),
                                                  int(stages), _stream_ptr(stream, lhs.device)),
               "gemm_f16_nt_noalloc")
    return out


# ---------------------------------------------------------------- the operators around the products

_codes = None
_torch = None


def _torch_module():
    """torch, imported by the first operator call (not with the package)."""
    global _codes, _torch
    import torch
    _codes = {torch.float16: GEMM_TYPE_HALF, torch.bfloat16: GEMM_TYPE_BFLOAT}
    _torch = torch
    return torch


def _type_of(name, *tensors):
    """The GEMM_TYPE_* of tensors that must share one 16-bit type, be dense
    matrices and lie on one CUDA device."""
    if _torch is None:
        _torch_module()
    dtype, device = tensors[0].dtype, tensors[0].device
    code = _codes.get(dtype)
    if code is None:
        raise TypeError(f"{name} takes float16 or bfloat16 tensors")
    for t in tensors:
        if t.dtype != dtype:
            raise TypeError(f"{name}: all matrices must have one type, got {dtype} and {t.dtype}")
        if t.dim() != 2:
            raise ValueError(f"{name} takes matrices, got a tensor of shape {tuple(t.shape)}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} takes contiguous CUDA tensors")
        if t.device != device:
            raise ValueError(f"{name}: all tensors must be on one device, got {device} and {t.device}")
    return code


_warned = set()


def _not_recorded(name, backward, *tensors):
    """Warns, once for each entry, where autograd would expect this call's
    output to carry a gradient: the calls are not recorded, their gradients are
    calls of their own."""
    for t in tensors:
        if t.requires_grad and name not in _warned:
            break
    else:
        return
    import torch
    if torch.is_grad_enabled():
        import warnings
        _warned.add(name)
        warnings.warn(f"{name} is not recorded by autograd: its output carries no gradient although an operand "
                      f"requires one; the gradients are those of {backward}", stacklevel=3)


def _act_code(name, act):
    if act not in _ACTS:
        raise ValueError(f"{name}: act must be one of {sorted(_ACTS)}, got {act!r}")
    return _ACTS[act]


def _vector(name, what, t, rows, dtype, device):
    if t.dtype != dtype:
        raise TypeError(f"{name}: {what} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != rows or not t.is_contiguous():
        raise ValueError(f"{name}: {what} must be a contiguous vector of {rows} elements, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: all tensors must be on one device, got {device} and {t.device}")


_HERE = contextlib.nullcontext()


def _on(stream, device):
    """(raw stream, context): inside the context the operands' device and the
    call's stream are current, so that outputs and workspaces are taken from
    that stream's memory and are not handed to other work while the call still
    uses them."""
    torch = _torch
    if stream is None and torch.cuda.current_device() == device.index:
        return torch._C._cuda_getCurrentRawStream(device.index), _HERE      # current_stream() without its object
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(device))
    if stream is None:
        raw = torch.cuda.current_stream(device).cuda_stream
    else:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        stack.enter_context(torch.cuda.stream(stream))
        raw = stream.cuda_stream
    return raw, stack


_ws_bytes = {}          # bytes by (entry, device, type, sizes) for operands on 16-byte boundaries


def _workspace(name, device, code, dims, *ptrs):
    """(tensor or None, address, bytes) of the workspace the call reports."""
    low = 0
    for p in ptrs:
        low |= p
    key = (name, device.index, code, dims)
    size = _ws_bytes.get(key) if low & 15 == 0 else None
    if size is None:
        need = ctypes.c_int64()
        _check(getattr(load_library(), name + "_workspace")(*dims, *ptrs, code, ctypes.byref(need)), name)
        size = need.value
        if low & 15 == 0:
            if len(_ws_bytes) >= 4096:
                _ws_bytes.clear()
            _ws_bytes[key] = size
    if size == 0:
        return None, None, 0
    ws = _torch.empty(size, dtype=_torch.uint8, device=device)
    return ws, ws.data_ptr(), size


def gemm_gated_nt(x, w_gate, w_up, act: str = "silu", save: bool = False, stream=None):
    """h[M,F] = act(x[M,K] @ w_gate[F,K].T) * (x @ w_up[F,K].T), one kernel.

    float16 or bfloat16; sums, activation and product in fp32, h rounded once.
    act is "silu" or "gelu" (tanh form).  With save=True returns (h, g, u),
    where g and u are the two products, for gemm_gated_nt_bwd.  Not recorded
    by autograd.
    """
    torch = _torch or _torch_module()
    name = "gemm_gated_nt"
    code, act_code = _type_of(name, x, w_gate, w_up), _act_code(name, act)
    M, K = x.shape
    F = w_gate.shape[0]
    if w_gate.shape[1] != K or w_up.shape != w_gate.shape:
        raise ValueError(f"{name}: shapes {tuple(x.shape)}, {tuple(w_gate.shape)}, {tuple(w_up.shape)} do not form "
                         "[M,K], [F,K], [F,K]")
    _not_recorded(name, "gemm_gated_nt_bwd", x, w_gate, w_up)
    lib, device = load_library(), x.device
    s, here = _on(stream, device)
    with here:
        h = torch.empty((M, F), dtype=x.dtype, device=device)
        g, u = (torch.empty_like(h), torch.empty_like(h)) if save else (None, None)
        px, pg, pu = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
        ws, ws_ptr, ws_bytes = _workspace(name, device, code, (M, F, K), px, pg, pu)
        _check(lib.gemm_gated_nt(M, F, K, px, pg, pu, h.data_ptr(), g.data_ptr() if save else None,
                                 u.data_ptr() if save else None, code, act_code, ws_ptr, ws_bytes, s), name)
    return (h, g, u) if save else h


def gemm_gated_nt_bwd(dh, g, u, x, w_gate, w_up, act: str = "silu", need_dx: bool = True, need_dw: bool = True,
                      stream=None):
    """The gradients of gemm_gated_nt: (dx[M,K], dw_gate[F,K], dw_up[F,K]).

    g and u are what gemm_gated_nt(..., save=True) returned.  Gradients not
    needed are None.
    """
    torch = _torch or _torch_module()
    name = "gemm_gated_nt_bwd"
    code, act_code = _type_of(name, dh, g, u, x, w_gate, w_up), _act_code(name, act)
    M, K = x.shape
    F = w_gate.shape[0]
    if w_gate.shape[1] != K or w_up.shape != w_gate.shape:
        raise ValueError(f"{name}: shapes {tuple(x.shape)}, {tuple(w_gate.shape)}, {tuple(w_up.shape)} do not form "
                         "[M,K], [F,K], [F,K]")
    if dh.shape != g.shape or u.shape != g.shape or tuple(g.shape) != (M, F):
        raise ValueError(f"{name}: dh, g and u must have shape {(M, F)}")
    lib, device = load_library(), x.device
    s, here = _on(stream, device)
    with here:
        dx = torch.empty_like(x) if need_dx else None
        dwg, dwu = (torch.empty_like(w_gate), torch.empty_like(w_up)) if need_dw else (None, None)
        ptrs = [t.data_ptr() for t in (dh, g, u, x, w_gate, w_up)]
        ws, ws_ptr, ws_bytes = _workspace(name, device, code, (M, F, K), *ptrs)
        outs = [t.data_ptr() if t is not None else None for t in (dx, dwg, dwu)]
        _check(lib.gemm_gated_nt_bwd(M, F, K, *ptrs, *outs, code, act_code, ws_ptr, ws_bytes, s), name)
    return dx, dwg, dwu


def _xent_shapes(name, x, w, target):
    torch = _torch
    code = _type_of(name, x, w)
    if w.shape[1] != x.shape[1]:
        raise ValueError(f"{name}: shapes {tuple(x.shape)}, {tuple(w.shape)} do not form [M,K], [V,K]")
    _vector(name, "target", target, x.shape[0], torch.int64, x.device)
    return code, x.shape[0], w.shape[0], x.shape[1]


def gemm_xent_nt(x, w, target, ignore_index: int = -100, stream=None):
    """Softmax cross entropy of the logits x[M,K] @ w[V,K].T, never kept.

    target is int64 [M].  Returns (loss, lse), float32 [M]: loss is 0 in rows
    whose target is ignore_index and NaN for any other target outside [0, V).
    Not recorded by autograd: the gradients are gemm_xent_nt_bwd's.
    """
    torch = _torch or _torch_module()
    name = "gemm_xent_nt"
    code, M, V, K = _xent_shapes(name, x, w, target)
    _not_recorded(name, "gemm_xent_nt_bwd", x, w)
    lib, device = load_library(), x.device
    s, here = _on(stream, device)
    with here:
        loss = torch.empty(M, dtype=torch.float32, device=device)
        lse = torch.empty_like(loss)
        px, pw = x.data_ptr(), w.data_ptr()
        ws, ws_ptr, ws_bytes = _workspace(name, device, code, (M, V, K), px, pw)
        _check(lib.gemm_xent_nt(M, V, K, px, pw, target.data_ptr(), int(ignore_index), loss.data_ptr(),
                                lse.data_ptr(), code, ws_ptr, ws_bytes, s), name)
    return loss, lse


def gemm_xent_nt_bwd(x, w, target, lse, dloss, ignore_index: int = -100, need_dx: bool = True, need_dw: bool = True,
                     stream=None):
    """The gradients of sum(dloss * loss) of gemm_xent_nt: (dx[M,K], dw[V,K]).

    lse is gemm_xent_nt's, dloss float32 [M].  Gradients not needed are None.
    """
    torch = _torch or _torch_module()
    name = "gemm_xent_nt_bwd"
    code, M, V, K = _xent_shapes(name, x, w, target)
    _vector(name, "lse", lse, M, torch.float32, x.device)
    _vector(name, "dloss", dloss, M, torch.float32, x.device)
    lib, device = load_library(), x.device
    s, here = _on(stream, device)
    with here:
        dx = torch.empty_like(x) if need_dx else None
        dw = torch.empty_like(w) if need_dw else None
        px, pw = x.data_ptr(), w.data_ptr()
        ws, ws_ptr, ws_bytes = _workspace(name, device, code, (M, V, K), px, pw)
        _check(lib.gemm_xent_nt_bwd(M, V, K, px, pw, target.data_ptr(), int(ignore_index), lse.data_ptr(),
                                    dloss.data_ptr(), dx.data_ptr() if need_dx else None,
                                    dw.data_ptr() if need_dw else None, code, ws_ptr, ws_bytes, s), name)
    return dx, dw


def gemm_nt_bwd(dy, x, w, need_dx: bool = True, need_dw: bool = True, stream=None):
    """The gradients of y[M,N] = x[M,K] @ w[N,K].T: (dx = dy @ w, dw = dy.T @ x).

    float16 or bfloat16, fp32 sums.  Gradients not needed are None.
    """
    torch = _torch or _torch_module()
    name = "gemm_nt_bwd"
    code = _type_of(name, dy, x, w)
    M, N = dy.shape
    K = x.shape[1]
    if x.shape[0] != M or tuple(w.shape) != (N, K):
        raise ValueError(f"{name}: shapes {tuple(dy.shape)}, {tuple(x.shape)}, {tuple(w.shape)} do not form "
                         "[M,N], [M,K], [N,K]")
    lib, device = load_library(), x.device
    s, here = _on(stream, device)
    with here:
        dx = torch.empty_like(x) if need_dx else None
        dw = torch.empty_like(w) if need_dw else None
        ptrs = [t.data_ptr() for t in (dy, x, w)]
        ws, ws_ptr, ws_bytes = _workspace(name, device, code, (M, N, K), *ptrs)
        _check(lib.gemm_nt_bwd(M, N, K, *ptrs, dx.data_ptr() if need_dx else None,
                               dw.data_ptr() if need_dw else None, code, ws_ptr, ws_bytes, s), name)
    return dx, dw


def gemm_device_status(stream=None) -> int:
    """Synchronizes the stream; returns and clears the device status word."""
    return load_library().gemm_device_status(_stream_ptr(stream, None))


def gemm_status_string(status: int) -> str:
    return status_string(status)


def gemm_set_wait_timeout_ns(ns: int) -> None:
    _check(load_library().gemm_set_wait_timeout_ns(int(ns)), "gemm_set_wait_timeout_ns")


def gemm_set_debug_flags(flags: int) -> None:
    _check(load_library().gemm_set_debug_flags(int(flags)), "gemm_set_debug_flags")


def gemm_set_scratch_pool(enable: bool) -> None:
    """Lets later gemm_f16_nt calls copy operands TMA cannot address to pooled
    scratch (faster for large ones; allocates stream-ordered).  Off by default."""
    _check(load_library().gemm_set_scratch_pool(int(bool(enable))), "gemm_set_scratch_pool")


def gemm_f16_nt_plan(M: int, N: int, K: int, lhs_ptr: int = 1 << 40, rhs_ptr: int = 2 << 40,
                     out_ptr: int = 3 << 40, stages: int = 4) -> dict:
    """The launch plan gemm_f16_nt would use (host logic only; the pointers are
    only inspected for alignment and overlap, never dereferenced)."""
    plan = (ctypes.c_int64 * 11)()
    _check(load_library().gemm_f16_nt_plan(M, N, K, lhs_ptr, rhs_ptr, out_ptr, stages, plan), "gemm_f16_nt_plan")
    keys = ["bm", "bn", "bk", "cta_group", "producer", "copy_bytes", "store", "smem_bytes", "tiles", "k_blocks",
            "k_split"]
    return dict(zip(keys, list(plan)))


__all__ = [
    "GemmError", "load_library", "header_functions", "gemm_s32_nn", "gemm_f16_nt", "gemm_device_status",
    "gemm_status_string", "gemm_set_wait_timeout_ns", "gemm_set_debug_flags", "gemm_set_scratch_pool",
    "gemm_f16_nt_plan", "gemm_f16_nt_noalloc", "gemm_s32_nn_ring",
    "gemm_gated_nt", "gemm_gated_nt_bwd", "gemm_xent_nt", "gemm_xent_nt_bwd", "gemm_nt_bwd",
]
