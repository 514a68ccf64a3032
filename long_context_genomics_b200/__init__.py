"""Python binding of libag: pair-bias multi-query attention on B200, and the
layers around it.

Argument marshalling only.  Every step of the computation runs in the CUDA
kernels of libag.so (see include/ag.h for the C ABI); there is no CPU or
PyTorch fallback, and importing this package raises if the library is
missing.  PyTorch supplies device memory and the current stream.

    ag_pair_bias_project(pair[P,P,Cp] f32, W[Cp,H] f32) -> bias[H,P,P] f32
    ag_attn_fwd(q[B,H,L,D] bf16, k[B,L,D] bf16, v[B,L,D] bf16,
                bias[H,P,P] f32, cap) -> (out[B,H,L,D] f32, lse[B,H,L] f32)
    ag_linear_fwd(x[M,K], W[N,K], bias, act, residual) -> y[M,N]
    ag_qk_norm_rope_fwd(q[B,L,H,D], k[B,L,D], ...) -> (q[B,H,L,D], k[B,L,D])
    ag_grad_clip(grads, max_norm) -> norm
    (and the gradients of the first three: ag_attn_bwd, ag_linear_bwd,
    ag_qk_norm_rope_bwd)

The attention is Eq. L_ij of the page "Making Full-Context AlphaGenome Fit
on an RTX 3090" (section "Why stock FlashAttention was not a drop-in
replacement") with a softmax over all keys.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libag.so")

AG_OK = 0
STATUS_NAMES = {
    0: "AG_OK", 1: "AG_ERR_NULL", 2: "AG_ERR_SHAPE", 3: "AG_ERR_ALIGN",
    4: "AG_ERR_UNSUPPORTED", 5: "AG_ERR_VALUE", 6: "AG_ERR_CUDA",
    7: "AG_ERR_ALIAS", 8: "AG_ERR_DEVICE", 9: "AG_ERR_SCRATCH",
}


class AgError(RuntimeError):
    """A libag call returned a status other than AG_OK."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {ag_status_string(status)} ({status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python long_context_genomics_b200/build.py` (or __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
    lib.ag_status_string.argtypes = [ctypes.c_int]
    lib.ag_status_string.restype = ctypes.c_char_p
    lib.ag_version.argtypes = []
    lib.ag_version.restype = ctypes.c_int
    lib.ag_pair_bias_project.argtypes = [vp, vp, vp, i64, i64, i64, vp]
    lib.ag_pair_bias_project.restype = ctypes.c_int
    lib.ag_pair_bias_project_rows.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp]
    lib.ag_pair_bias_project_rows.restype = ctypes.c_int
    lib.ag_attn_fwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, f32,
                                vp, vp, vp]
    lib.ag_attn_fwd.restype = ctypes.c_int
    lib.ag_attn_fwd_strided_bias.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64,
                                             i64, i64, f32, vp, vp, vp]
    lib.ag_attn_fwd_strided_bias.restype = ctypes.c_int
    lib.ag_attn_fwd_ex.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                   i64, f32, vp, vp, vp]
    lib.ag_attn_fwd_ex.restype = ctypes.c_int
    lib.ag_attn_fwd_query_slab.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                           i64, i64, f32, vp, vp, vp]
    lib.ag_attn_fwd_query_slab.restype = ctypes.c_int
    lib.ag_attn_fwd_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                        f32, vp, vp, vp]
    lib.ag_attn_fwd_noalloc.restype = ctypes.c_int
    lib.ag_attn_fwd_launch_count.argtypes = [i64, i64, i64, i64, i64, f32,
                                             ctypes.POINTER(ctypes.c_int)]
    lib.ag_attn_fwd_launch_count.restype = ctypes.c_int
    ip = ctypes.POINTER(ctypes.c_int)
    lib.ag_attn_fwd_schedule.argtypes = [i64, i64, ctypes.c_int, ctypes.c_int, ip, ip, ip,
                                         ip, ip, ip, ip, ip]
    lib.ag_attn_fwd_schedule.restype = ctypes.c_int
    lib.ag_attn_bwd.argtypes = [vp, vp, vp, vp, i64, vp, vp, i64, i64, i64, i64, i64,
                                i64, f32, vp, vp, vp, vp, vp, vp]
    lib.ag_attn_bwd.restype = ctypes.c_int
    lib.ag_attn_bwd_launch_count.argtypes = [i64, ctypes.POINTER(ctypes.c_int)]
    lib.ag_attn_bwd_launch_count.restype = ctypes.c_int
    i32 = ctypes.c_int
    i64p = ctypes.POINTER(i64)
    lib.ag_linear_fwd.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, i32, i32, vp,
                                  i64, vp, i64, i32, vp, i64, vp]
    lib.ag_linear_fwd_workspace.argtypes = [vp, i64, vp, i64, i64, i64, i64, i64p]
    lib.ag_linear_bwd.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, i32, i64, i64, i64, i32,
                                  vp, i64, i32, vp, i64, i32, vp, vp, i64, vp]
    lib.ag_linear_bwd_workspace.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, i64, vp, vp,
                                            vp, i64p]
    heads = [vp, i64, i64, i64]
    lib.ag_qk_norm_rope_fwd.argtypes = (heads + heads + [i32, vp, vp, vp, vp, i32, f32, vp, i64,
                                                         i32, vp, i64, i64, i64, i64, i64, i64,
                                                         vp, vp, i32, vp])
    lib.ag_qk_norm_rope_bwd.argtypes = ([vp, vp, i32] + heads + heads
                                        + [i32, vp, vp, i32, f32, vp, i64, i32, vp, i64, i64,
                                           i64, i64, i64, i64] + heads + heads
                                        + [vp, vp, vp, vp, vp, i64, vp])
    lib.ag_qk_norm_rope_bwd_workspace.argtypes = [i64, i64, i64, i64, i64, i32, i64p]
    lib.ag_grad_clip.argtypes = [vp, vp, vp, i64, f32, f32, vp, vp, i64, vp]
    lib.ag_grad_clip_workspace.argtypes = [i64, i64p]
    for fn in (lib.ag_linear_fwd, lib.ag_linear_fwd_workspace, lib.ag_linear_bwd,
               lib.ag_linear_bwd_workspace, lib.ag_qk_norm_rope_fwd, lib.ag_qk_norm_rope_bwd,
               lib.ag_qk_norm_rope_bwd_workspace, lib.ag_grad_clip, lib.ag_grad_clip_workspace):
        fn.restype = i32
    lib.ag_device_error.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                    ctypes.c_int]
    lib.ag_device_error.restype = ctypes.c_int
    lib.ag_debug_wait_timeout.argtypes = [ctypes.c_uint64, vp]
    lib.ag_debug_wait_timeout.restype = ctypes.c_int
    return lib


lib = _load()


def ag_status_string(status: int) -> str:
    return lib.ag_status_string(int(status)).decode()


def ag_version() -> int:
    return int(lib.ag_version())


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _one_device(*tensors: torch.Tensor) -> torch.device:
    """The one device that every tensor of a call lives on.  The kernels run
    on that device (made current for the call), so a tensor elsewhere would
    reach them as a pointer they cannot read: refuse it here."""
    dev = tensors[0].device
    for t in tensors[1:]:
        if t.device != dev:
            raise ValueError(f"all tensors of a call must be on {dev}; one is on {t.device}")
    return dev


def _check(t: torch.Tensor, name: str, dtype, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def ag_pair_bias_project(pair: torch.Tensor, W: torch.Tensor,
                         bias: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bias[h,p,q] = sum_c pair[p,q,c] W[c,h] on the GPU (libag kernel)."""
    _check(pair, "pair", torch.float32, 3)
    _check(W, "W", torch.float32, 2)
    P, P2, Cp = pair.shape
    if P != P2 or W.shape[0] != Cp:
        raise ValueError("pair must be [P,P,Cp] and W [Cp,H]")
    H = W.shape[1]
    if bias is None:
        bias = torch.empty((H, P, P), dtype=torch.float32, device=pair.device)
    _check(bias, "bias", torch.float32, 3)
    if tuple(bias.shape) != (H, P, P):
        raise ValueError("bias must be [H,P,P]")
    with torch.cuda.device(_one_device(pair, W, bias)):
        st = lib.ag_pair_bias_project(pair.data_ptr(), W.data_ptr(), bias.data_ptr(),
                                      P, Cp, H, _stream_ptr(stream))
    if st != AG_OK:
        raise AgError("ag_pair_bias_project", st)
    return bias


def ag_pair_bias_project_rows(pair: torch.Tensor, W: torch.Tensor,
                              bias: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bias[h,r,q] = sum_c pair[r,q,c] W[c,h] for a row slab pair[R,P,Cp]
    (libag kernel); returns bias [H,R,P]."""
    _check(pair, "pair", torch.float32, 3)
    _check(W, "W", torch.float32, 2)
    R, P, Cp = pair.shape
    if W.shape[0] != Cp:
        raise ValueError("pair must be [R,P,Cp] and W [Cp,H]")
    H = W.shape[1]
    if bias is None:
        bias = torch.empty((H, R, P), dtype=torch.float32, device=pair.device)
    _check(bias, "bias", torch.float32, 3)
    if tuple(bias.shape) != (H, R, P):
        raise ValueError("bias must be [H,R,P]")
    with torch.cuda.device(_one_device(pair, W, bias)):
        st = lib.ag_pair_bias_project_rows(pair.data_ptr(), W.data_ptr(), bias.data_ptr(),
                                           R, P, Cp, H, _stream_ptr(stream))
    if st != AG_OK:
        raise AgError("ag_pair_bias_project_rows", st)
    return bias


def ag_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                bias: torch.Tensor, cap: float = 5.0, block: int = 16,
                out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                stream=None):
    """Fused pair-bias MQA attention forward (libag kernel).

    bias is [H,P,P] (shared by the batch) or [B,H,P,P] (one per batch item),
    P = ceil(L / block); v is [B,L,Dv] with Dv = D or 192 (the page's
    checkpoint).  Calls ag_attn_fwd_ex.  Returns (out [B,H,L,Dv] fp32,
    lse [B,H,L] fp32).  cap = math.inf turns the soft cap off."""
    _check(q, "q", torch.bfloat16, 4)
    _check(k, "k", torch.bfloat16, 3)
    _check(v, "v", torch.bfloat16, 3)
    B, H, L, D = q.shape
    Dv = v.shape[-1]
    if tuple(k.shape) != (B, L, D) or tuple(v.shape) != (B, L, Dv):
        raise ValueError("k must be [B,L,D] and v [B,L,Dv] with q [B,H,L,D]")
    bstride = _bias_stride(bias, B, H, L, block)
    if out is None:
        out = torch.empty((B, H, L, Dv), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    _check_out(out, lse, B, H, L, Dv)
    with torch.cuda.device(_one_device(q, k, v, bias, out, lse)):
        st = lib.ag_attn_fwd_ex(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), bias.data_ptr(), bstride, B, H, L,
            D, Dv, int(block), float(cap), out.data_ptr(), lse.data_ptr(),
            _stream_ptr(stream))
    if st != AG_OK:
        raise AgError("ag_attn_fwd_ex", st)
    return out, lse


def ag_attn_fwd_query_slab(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                           bias: torch.Tensor, cap: float = 5.0, block: int = 16,
                           out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                           stream=None):
    """The attention rows of a slab of query positions (libag kernel).

    q [B,H,Lq,D] holds positions q0 .. q0+Lq-1 (q0 a multiple of block) of
    sequences whose keys and values k [B,L,D], v [B,L,Dv] are all given; bias
    holds the slab's bias rows, [H, ceil(Lq/block), ceil(L/block)] (shared by
    the batch) or [B, H, ceil(Lq/block), ceil(L/block)].  Returns
    (out [B,H,Lq,Dv] fp32, lse [B,H,Lq] fp32)."""
    _check(q, "q", torch.bfloat16, 4)
    _check(k, "k", torch.bfloat16, 3)
    _check(v, "v", torch.bfloat16, 3)
    B, H, Lq, D = q.shape
    L, Dv = k.shape[1], v.shape[-1]
    if tuple(k.shape) != (B, L, D) or tuple(v.shape) != (B, L, Dv):
        raise ValueError("k must be [B,L,D] and v [B,L,Dv] with q [B,H,Lq,D]")
    bstride = _bias_stride(bias, B, H, L, block, rows=-(-Lq // block) if block > 0 else 0)
    if out is None:
        out = torch.empty((B, H, Lq, Dv), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=q.device)
    _check_out(out, lse, B, H, Lq, Dv)
    with torch.cuda.device(_one_device(q, k, v, bias, out, lse)):
        st = lib.ag_attn_fwd_query_slab(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), bias.data_ptr(), bstride, B, H, Lq, L,
            D, Dv, int(block), float(cap), out.data_ptr(), lse.data_ptr(),
            _stream_ptr(stream))
    if st != AG_OK:
        raise AgError("ag_attn_fwd_query_slab", st)
    return out, lse


def _bias_stride(bias: torch.Tensor, B: int, H: int, L: int, block: int,
                 rows: int | None = None) -> int:
    """Batch stride (floats) of a [H,R,P] (0) or [B,H,R,P] bias, P = ceil(L/block)
    and R = rows (default P)."""
    if bias.dtype != torch.float32 or not bias.is_contiguous():
        raise ValueError("bias must be a contiguous float32 tensor")
    P = -(-L // block) if block > 0 else 0
    R = P if rows is None else rows
    if tuple(bias.shape) == (H, R, P):
        return 0
    if tuple(bias.shape) == (B, H, R, P):
        return H * R * P
    raise ValueError(f"bias must be [{H},{R},{P}] or [{B},{H},{R},{P}], got {tuple(bias.shape)}")


def _check_out(out: torch.Tensor, lse: torch.Tensor, B: int, H: int, L: int, Dv: int):
    _check(out, "out", torch.float32, 4)
    _check(lse, "lse", torch.float32, 3)
    if tuple(out.shape) != (B, H, L, Dv) or tuple(lse.shape) != (B, H, L):
        raise ValueError("out must be [B,H,L,Dv] and lse [B,H,L]")


def ag_attn_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        bias: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
                        cap: float = 5.0, block: int = 16, stream=None):
    """ag_attn_fwd through the entry point that allocates nothing (static
    scratch inside the library).  The caller passes the outputs."""
    _check(q, "q", torch.bfloat16, 4)
    _check(k, "k", torch.bfloat16, 3)
    _check(v, "v", torch.bfloat16, 3)
    _check(bias, "bias", torch.float32, 3)
    B, H, L, D = q.shape
    if tuple(k.shape) != (B, L, D) or tuple(v.shape) != (B, L, D):
        raise ValueError("k and v must be [B,L,D] with q [B,H,L,D]")
    if _bias_stride(bias, B, H, L, block) != 0:
        raise ValueError("ag_attn_fwd_noalloc takes one bias shared by the batch")
    _check_out(out, lse, B, H, L, D)
    with torch.cuda.device(_one_device(q, k, v, bias, out, lse)):
        st = lib.ag_attn_fwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                     bias.data_ptr(), B, H, L, D, int(block),
                                     float(cap), out.data_ptr(), lse.data_ptr(),
                                     _stream_ptr(stream))
    if st != AG_OK:
        raise AgError("ag_attn_fwd_noalloc", st)
    return out, lse


def ag_attn_fwd_launch_count(B: int, L: int, cap: float = 5.0, H: int = 8,
                             D: int = 128, block: int = 16) -> int:
    """How many kernels ag_attn_fwd launches for these sizes (see include/ag.h)."""
    n = ctypes.c_int(-1)
    st = lib.ag_attn_fwd_launch_count(int(B), int(H), int(L), int(D), int(block),
                                      float(cap), ctypes.byref(n))
    if st != AG_OK:
        raise AgError("ag_attn_fwd_launch_count", st)
    return int(n.value)


def ag_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, bias: torch.Tensor,
                lse: torch.Tensor, dout: torch.Tensor, cap: float = 5.0, block: int = 16,
                stream=None):
    """Backward of ag_attn_fwd (libag kernels): gradients of out for the
    upstream gradient dout [B,H,L,Dv] fp32, given the forward's lse.
    Returns (dq [B,H,L,D], dk [B,L,D], dv [B,L,Dv], dbias (bias's shape; a
    shared [H,P,P] bias gets the sum over the batch), delta [B,H,L]), all
    fp32 and newly allocated."""
    _check(q, "q", torch.bfloat16, 4)
    _check(k, "k", torch.bfloat16, 3)
    _check(v, "v", torch.bfloat16, 3)
    _check(lse, "lse", torch.float32, 3)
    _check(dout, "dout", torch.float32, 4)
    B, H, L, D = q.shape
    Dv = v.shape[-1]
    if tuple(k.shape) != (B, L, D) or tuple(v.shape) != (B, L, Dv):
        raise ValueError("k must be [B,L,D] and v [B,L,Dv] with q [B,H,L,D]")
    if tuple(lse.shape) != (B, H, L) or tuple(dout.shape) != (B, H, L, Dv):
        raise ValueError("lse must be [B,H,L] and dout [B,H,L,Dv]")
    bstride = _bias_stride(bias, B, H, L, block)
    dev = _one_device(q, k, v, bias, lse, dout)
    f32 = dict(dtype=torch.float32, device=dev)
    dq = torch.empty((B, H, L, D), **f32)
    dk = torch.empty((B, L, D), **f32)
    dv = torch.empty((B, L, Dv), **f32)
    dbias = torch.empty(tuple(bias.shape), **f32)
    delta = torch.empty((B, H, L), **f32)
    with torch.cuda.device(dev):
        st = lib.ag_attn_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), bias.data_ptr(), bstride,
            lse.data_ptr(), dout.data_ptr(), B, H, L, D, Dv, int(block), float(cap),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dbias.data_ptr(),
            delta.data_ptr(), _stream_ptr(stream))
    if st != AG_OK:
        raise AgError("ag_attn_bwd", st)
    return dq, dk, dv, dbias, delta


def ag_attn_bwd_launch_count(Dv: int = 128) -> int:
    """How many kernels a non-empty ag_attn_bwd call with value width Dv launches."""
    n = ctypes.c_int(-1)
    st = lib.ag_attn_bwd_launch_count(int(Dv), ctypes.byref(n))
    if st != AG_OK:
        raise AgError("ag_attn_bwd_launch_count", st)
    return int(n.value)


# ---------------------------------------------------------------------------
# The layers around the attention.

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
NORMS = {"none": 0, "rms": 1, "layer": 2}
ROPES = {"halves": 0, "interleaved": 1}
_HALF = (torch.bfloat16, torch.float16)


def _elsewhere(dev: torch.device, stream) -> bool:
    """Whether a call for tensors on dev has to enter _site first."""
    return stream is not None or torch._C._cuda_getDevice() != dev.index


def _site(dev: torch.device, stream):
    """Context in which a call's memory is allocated and its kernels launched:
    the tensors' device and the caller's stream (default: that device's
    current stream).  Workspaces belong to that stream, so a later call on it
    may take their memory over, and no other stream does."""
    if stream is None:
        return torch.cuda.device(dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {dev}")
    return torch.cuda.stream(stream)


def _current(dev: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _code(table: dict, value, name: str) -> int:
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {', '.join(map(str, table))}, got {value}") from None


def _on_gpu(t, name: str, dtypes) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")


def _same_device(t, name: str, dev: torch.device) -> None:
    if t.device != dev:
        raise ValueError(f"all tensors of a call must be on {dev}; {name} is on {t.device}")


def _matrix(t, name: str, dtype, rows: int, cols: int, dev: torch.device) -> int:
    """Checks a row-major matrix (its rows may be apart) and returns its row
    stride.  (The checks of the layers' calls are written for the case that
    all is well: at a few rows they cost as much as the kernel.)"""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (rows, cols) \
            and t.device == dev:
        ld, inner = t.stride()
        if inner == 1 or cols == 1:
            return ld if rows > 1 or ld > cols else cols
        raise ValueError(f"the rows of {name} must be dense")
    _on_gpu(t, name, (dtype,))
    _same_device(t, name, dev)
    raise ValueError(f"{name} must be [{rows},{cols}], got {list(t.shape)}")


def _vector(t, name: str, n: int, dev: torch.device):
    """Checks an optional dense float32 vector of n and returns its pointer."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is torch.float32 and t.shape == (n,) \
            and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    _on_gpu(t, name, (torch.float32,))
    _same_device(t, name, dev)
    raise ValueError(f"{name} must be a contiguous [{n}]")


def _workspace(query, dev: torch.device, name: str, *args):
    """Workspace of the bytes that `query` gives for args: (tensor, pointer, bytes)."""
    n = ctypes.c_int64(0)
    st = query(*args, ctypes.byref(n))
    if st != AG_OK:
        raise AgError(name, st)
    if n.value == 0:
        return None, None, 0
    t = torch.empty(n.value, dtype=torch.uint8, device=dev)
    return t, t.data_ptr(), n.value


def ag_linear_fwd(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None,
                  act: str = "none", residual: torch.Tensor | None = None, preact=False,
                  out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                  stream=None):
    """y = act(x W^T + bias) + residual (libag kernels).

    x [M,K] and W [N,K] bf16 or fp16 (rows dense, row strides free); bias [N]
    fp32; residual and y [M,N] in out_dtype (x's type, the default, or fp32).
    act: none, relu, gelu, gelu_tanh, silu.  preact=True (or a [M,N] tensor of
    x's type to write) also returns x W^T + bias, which ag_linear_bwd of the
    next layer takes: (y, preact).  out may be the residual itself."""
    _on_gpu(x, "x", _HALF)
    if x.ndim != 2 or not isinstance(W, torch.Tensor) or W.ndim != 2:
        raise ValueError("x must be [M,K] and W [N,K]")
    dev = x.device
    if _elsewhere(dev, stream):
        with _site(dev, stream):
            return ag_linear_fwd(x, W, bias, act, residual, preact, out, out_dtype)
    (M, K), N, T = x.shape, W.shape[0], x.dtype
    ldx, ldw = _matrix(x, "x", T, M, K, dev), _matrix(W, "W", T, N, K, dev)
    code = _code(ACTIVATIONS, act, "act")
    if out_dtype is None:
        out_dtype = T if out is None else out.dtype
    if out_dtype is not T and out_dtype is not torch.float32:
        raise TypeError(f"out_dtype must be {T} or torch.float32, got {out_dtype}")
    b = _vector(bias, "bias", N, dev)
    r, ldr, z, zp, ldz = None, 0, None, None, 0
    if residual is not None:
        ldr, r = _matrix(residual, "residual", out_dtype, M, N, dev), residual.data_ptr()
    if out is None:
        out, ldy = x.new_empty((M, N), dtype=out_dtype), N
    else:
        ldy = _matrix(out, "out", out_dtype, M, N, dev)
    if preact is not False and preact is not None:
        z = x.new_empty((M, N)) if preact is True else preact
        ldz, zp = _matrix(z, "preact", T, M, N, dev), z.data_ptr()
    xp, wp, yp, t, yt = x.data_ptr(), W.data_ptr(), out.data_ptr(), DTYPES[T], DTYPES[out_dtype]
    # Most calls need no workspace; the others say so before they do anything.
    st = lib.ag_linear_fwd(xp, ldx, wp, ldw, b, r, ldr, M, N, K, t, code, zp, ldz, yp, ldy, yt,
                           None, 0, _current(dev))
    if st == 9:
        ws, wsp, n = _workspace(lib.ag_linear_fwd_workspace, dev, "ag_linear_fwd_workspace", xp,
                                ldx, wp, ldw, M, N, K)
        st = lib.ag_linear_fwd(xp, ldx, wp, ldw, b, r, ldr, M, N, K, t, code, zp, ldz, yp, ldy,
                               yt, wsp, n, _current(dev))
    if st != AG_OK:
        raise AgError("ag_linear_fwd", st)
    return out if z is None else (out, z)


def ag_linear_bwd(dy: torch.Tensor, x: torch.Tensor, W: torch.Tensor, act: str = "none",
                  preact: torch.Tensor | None = None, need_dx: bool = True,
                  need_dW: bool = True, need_db: bool = True,
                  dx_dtype: torch.dtype | None = None, dW_dtype: torch.dtype = torch.float32,
                  dx: torch.Tensor | None = None, dW: torch.Tensor | None = None, stream=None):
    """Gradients of y = x W^T + bias for the upstream gradient dy [M,N] (libag
    kernels): (dx [M,K], dW [N,K], db [N] fp32), None where not needed.

    With act and preact (x = act(preact), both from the layer before) dx is
    the gradient of preact instead of x.  dx_dtype: x's type (default) or
    fp32; dW_dtype: fp32 (default) or x's type.  dx and dW may be given to
    write into.  The gradient of ag_linear_fwd's residual is dy itself."""
    _on_gpu(dy, "dy", _HALF)
    if dy.ndim != 2 or not isinstance(x, torch.Tensor) or x.ndim != 2:
        raise ValueError("dy must be [M,N] and x [M,K]")
    dev = dy.device
    if _elsewhere(dev, stream):
        with _site(dev, stream):
            return ag_linear_bwd(dy, x, W, act, preact, need_dx, need_dW, need_db, dx_dtype,
                                 dW_dtype, dx, dW)
    (M, N), K, T = dy.shape, x.shape[1], dy.dtype
    lddy, ldx = _matrix(dy, "dy", T, M, N, dev), _matrix(x, "x", T, M, K, dev)
    ldw = _matrix(W, "W", T, N, K, dev)
    code = _code(ACTIVATIONS, act, "act")
    ldz = 0 if preact is None else _matrix(preact, "preact", T, M, K, dev)
    if code and preact is None:
        raise ValueError(f"act {act} needs the preact of x")
    dxp = dwp = dbp = None
    lddx = lddw = dxt = dwt = 0
    if need_dx:
        dx_dtype = dx_dtype or (T if dx is None else dx.dtype)
        if dx_dtype is not T and dx_dtype is not torch.float32:
            raise TypeError(f"dx_dtype must be {T} or torch.float32, got {dx_dtype}")
        if dx is None:
            dx = dy.new_empty((M, K), dtype=dx_dtype)
        lddx, dxp, dxt = _matrix(dx, "dx", dx_dtype, M, K, dev), dx.data_ptr(), DTYPES[dx_dtype]
    if need_dW:
        dW_dtype = dW_dtype if dW is None else dW.dtype
        if dW_dtype is not T and dW_dtype is not torch.float32:
            raise TypeError(f"dW_dtype must be {T} or torch.float32, got {dW_dtype}")
        if dW is None:
            dW = dy.new_empty((N, K), dtype=dW_dtype)
        lddw, dwp, dwt = _matrix(dW, "dW", dW_dtype, N, K, dev), dW.data_ptr(), DTYPES[dW_dtype]
    db = dy.new_empty(N, dtype=torch.float32) if need_db else None
    if need_db:
        dbp = db.data_ptr()
    dyp, xp, wp = dy.data_ptr(), x.data_ptr(), W.data_ptr()
    ws, wsp, n = _workspace(lib.ag_linear_bwd_workspace, dev, "ag_linear_bwd_workspace", dyp,
                            lddy, xp, ldx, wp, ldw, M, N, K, dxp, dwp, dbp)
    st = lib.ag_linear_bwd(dyp, lddy, xp, ldx, wp, ldw,
                           None if preact is None else preact.data_ptr(), ldz, code, M, N, K,
                           DTYPES[T], dxp, lddx, dxt, dwp, lddw, dwt, dbp, wsp, n, _current(dev))
    if st != AG_OK:
        raise AgError("ag_linear_bwd", st)
    return dx if need_dx else None, dW if need_dW else None, db


def ag_rope_frequencies(rotary_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """inv_freq[p] = base^(-2p / rotary_dim), p < rotary_dim / 2, in fp64: the
    usual frequencies for ag_qk_norm_rope_fwd (which takes any)."""
    p = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    return (float(base) ** (-p / rotary_dim)).to(device)


def _heads(t, name: str, dtype, B: int, L: int, D: int, dev: torch.device):
    """Checks a [B,L,H,D] (or [B,L,D]: one head) tensor with dense heads;
    returns H, pointer and the strides over b, l and h."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev:
        s = t.shape
        if len(s) == 4 and s[0] == B and s[1] == L and s[3] == D:
            sb, sl, sh, sd = t.stride()
            if sd == 1 or D == 1:
                return s[2], t.data_ptr(), sb, sl, sh
            raise ValueError(f"the heads of {name} must be dense")
        if s == (B, L, D):
            sb, sl, sd = t.stride()
            if sd == 1 or D == 1:
                return 1, t.data_ptr(), sb, sl, 0
            raise ValueError(f"the heads of {name} must be dense")
    _on_gpu(t, name, (dtype,))
    _same_device(t, name, dev)
    raise ValueError(f"{name} must be [{B},{L},H,{D}] or [{B},{L},{D}], got {list(t.shape)}")


def _qk_first(q, k):
    """Type, device and sizes of a call, from the queries or else the keys."""
    first, name = (q, "q") if q is not None else (k, "k")
    if first is None:
        raise ValueError("q and k are both None")
    _on_gpu(first, name, DTYPES)
    if first.ndim not in (3, 4):
        raise ValueError(f"{name} must be [B,L,H,D] or [B,L,D]")
    return first, first.dtype, first.device, first.shape[0], first.shape[1], first.shape[-1]


def _rotation(inv_freq, rope, positions, B: int, L: int, dev: torch.device):
    """The rotation's arguments: inv_freq, R, rope, positions, their stride over b."""
    code, freq, R, where, pos_sb = _code(ROPES, rope, "rope"), None, 0, None, 0
    if inv_freq is not None:
        _on_gpu(inv_freq, "inv_freq", (torch.float64,))
        _same_device(inv_freq, "inv_freq", dev)
        if inv_freq.ndim != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous [R/2]")
        R, freq = 2 * inv_freq.shape[0], inv_freq.data_ptr()
    if positions is not None:
        _on_gpu(positions, "positions", (torch.int64,))
        _same_device(positions, "positions", dev)
        if positions.shape != (L,) and positions.shape != (B, L):
            raise ValueError(f"positions must be [{L}] or [{B},{L}], got {list(positions.shape)}")
        s = positions.stride()
        if L > 1 and s[-1] != 1:
            raise ValueError("the rows of positions must be dense")
        where = positions.data_ptr()
        if len(s) == 2 and B > 1:
            pos_sb = s[0]
    return freq, R, code, where, pos_sb


_NO_HEADS = (0, None, 0, 0, 0)


def ag_qk_norm_rope_fwd(q: torch.Tensor | None, k: torch.Tensor | None,
                        q_weight: torch.Tensor | None = None,
                        k_weight: torch.Tensor | None = None,
                        q_bias: torch.Tensor | None = None,
                        k_bias: torch.Tensor | None = None, norm: str = "rms",
                        eps: float = 1e-6, inv_freq: torch.Tensor | None = None,
                        rope: str = "halves", positions: torch.Tensor | None = None,
                        out_dtype: torch.dtype = torch.bfloat16,
                        q_out: torch.Tensor | None = None,
                        k_out: torch.Tensor | None = None, stream=None):
    """Norm of every query and key head, its weight and bias, the rotation by
    position and the change to ag_attn_fwd's layout, in one pass (libag kernel).

    q [B,L,H,D] and k [B,L,D] (or [B,L,Hk,D]) of one type, fp32, bf16 or fp16,
    with dense heads and any other strides, e.g. slices of a fused
    projection; weights and biases [D] fp32.  norm: rms, layer or none; rope:
    halves (pairs i, i + R/2) or interleaved (2i, 2i+1) over the first
    R = 2 len(inv_freq) elements, angle = position * inv_freq (fp64, see
    ag_rope_frequencies; None: no rotation); positions int64 [L] or [B,L]
    (default 0 .. L-1).  Returns (q_out [B,H,L,D], k_out [B,L,D] or
    [B,Hk,L,D]); q or k may be None."""
    first, T, dev, B, L, D = _qk_first(q, k)
    if _elsewhere(dev, stream):
        with _site(dev, stream):
            return ag_qk_norm_rope_fwd(q, k, q_weight, k_weight, q_bias, k_bias, norm, eps,
                                       inv_freq, rope, positions, out_dtype, q_out, k_out)
    Hq, qp, qb, ql, qh = _NO_HEADS if q is None else _heads(q, "q", T, B, L, D, dev)
    Hk, kp, kb, kl, kh = _NO_HEADS if k is None else _heads(k, "k", T, B, L, D, dev)
    ot = _code(DTYPES, out_dtype, "out_dtype")
    qo = ko = None
    if q is None:
        q_out = None
    else:
        shape = (B, Hq, L, D) if q.ndim == 4 else (B, L, D)
        if q_out is None:
            q_out = first.new_empty(shape, dtype=out_dtype)
            qo = q_out.data_ptr()
        else:
            qo = _dense(q_out, "q_out", out_dtype, shape, dev)
    if k is None:
        k_out = None
    else:
        shape = (B, Hk, L, D) if k.ndim == 4 else (B, L, D)
        if k_out is None:
            k_out = first.new_empty(shape, dtype=out_dtype)
            ko = k_out.data_ptr()
        else:
            ko = _dense(k_out, "k_out", out_dtype, shape, dev)
    st = lib.ag_qk_norm_rope_fwd(
        qp, qb, ql, qh, kp, kb, kl, kh, DTYPES[T], _vector(q_weight, "q_weight", D, dev),
        _vector(q_bias, "q_bias", D, dev), _vector(k_weight, "k_weight", D, dev),
        _vector(k_bias, "k_bias", D, dev), _code(NORMS, norm, "norm"), eps,
        *_rotation(inv_freq, rope, positions, B, L, dev), B, Hq, Hk, L, D, qo, ko, ot,
        _current(dev))
    if st != AG_OK:
        raise AgError("ag_qk_norm_rope_fwd", st)
    return q_out, k_out


def _dense(t, name: str, dtype, shape: tuple, dev: torch.device) -> int:
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape \
            and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    _on_gpu(t, name, (dtype,))
    _same_device(t, name, dev)
    raise ValueError(f"{name} must be a contiguous {list(shape)}, got {list(t.shape)}")


def ag_qk_norm_rope_bwd(dq_out: torch.Tensor | None, dk_out: torch.Tensor | None,
                        q: torch.Tensor | None, k: torch.Tensor | None,
                        q_weight: torch.Tensor | None = None,
                        k_weight: torch.Tensor | None = None,
                        q_bias: torch.Tensor | None = None,
                        k_bias: torch.Tensor | None = None, norm: str = "rms",
                        eps: float = 1e-6, inv_freq: torch.Tensor | None = None,
                        rope: str = "halves", positions: torch.Tensor | None = None,
                        dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                        stream=None):
    """Gradients of ag_qk_norm_rope_fwd (libag kernels) for dq_out and dk_out
    in the layout of its outputs and one type, e.g. ag_attn_bwd's dq and dk;
    the other arguments as the forward's.  Returns (dq, dk, dq_weight,
    dk_weight, dq_bias, dk_bias): dq and dk in the shape and type of q and k,
    written into the tensors given (which may be slices of one fused
    projection's gradient) or new ones; the others [D] fp32, None where the
    forward had none."""
    first, T, dev, B, L, D = _qk_first(q, k)
    if _elsewhere(dev, stream):
        with _site(dev, stream):
            return ag_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, q_bias, k_bias,
                                       norm, eps, inv_freq, rope, positions, dq, dk)
    Hq, qp, qb, ql, qh = _NO_HEADS if q is None else _heads(q, "q", T, B, L, D, dev)
    Hk, kp, kb, kl, kh = _NO_HEADS if k is None else _heads(k, "k", T, B, L, D, dev)
    g = dq_out if q is not None else dk_out
    G = g.dtype if isinstance(g, torch.Tensor) else None
    gt = _code(DTYPES, G, "the type of dq_out and dk_out")
    gq = gk = None
    (_, dqp, dqb, dql, dqh), (_, dkp, dkb, dkl, dkh) = _NO_HEADS, _NO_HEADS
    if q is None:
        dq = None
    else:
        gq = _dense(dq_out, "dq_out", G, (B, Hq, L, D) if q.ndim == 4 else (B, L, D), dev)
        if dq is None:
            dq = first.new_empty(q.shape)
        elif dq.shape != q.shape:
            raise ValueError(f"dq must be {list(q.shape)}, got {list(dq.shape)}")
        _, dqp, dqb, dql, dqh = _heads(dq, "dq", T, B, L, D, dev)
    if k is None:
        dk = None
    else:
        gk = _dense(dk_out, "dk_out", G, (B, Hk, L, D) if k.ndim == 4 else (B, L, D), dev)
        if dk is None:
            dk = first.new_empty(k.shape)
        elif dk.shape != k.shape:
            raise ValueError(f"dk must be {list(k.shape)}, got {list(dk.shape)}")
        _, dkp, dkb, dkl, dkh = _heads(dk, "dk", T, B, L, D, dev)
    inputs = (q_weight, k_weight, q_bias, k_bias)
    used = [_vector(t, n, D, dev) for t, n in zip(inputs, ("q_weight", "k_weight", "q_bias",
                                                           "k_bias"))]
    wanted = sum(t is not None for t in inputs)
    params, p = [None] * 4, [None] * 4
    ws = wsp = None
    n = 0
    if wanted:
        rows = iter(torch.empty((wanted, D), dtype=torch.float32, device=dev).unbind(0))
        params = [None if t is None else next(rows) for t in inputs]
        p = [None if t is None else t.data_ptr() for t in params]
        ws, wsp, n = _workspace(lib.ag_qk_norm_rope_bwd_workspace, dev,
                                "ag_qk_norm_rope_bwd_workspace", B, Hq, Hk, L, D, 1)
    st = lib.ag_qk_norm_rope_bwd(
        gq, gk, gt, qp, qb, ql, qh, kp, kb, kl, kh, DTYPES[T], used[0], used[1],
        _code(NORMS, norm, "norm"), eps, *_rotation(inv_freq, rope, positions, B, L, dev), B, Hq,
        Hk, L, D, dqp, dqb, dql, dqh, dkp, dkb, dkl, dkh, p[0], p[2], p[1], p[3], wsp, n,
        _current(dev))
    if st != AG_OK:
        raise AgError("ag_qk_norm_rope_bwd", st)
    return dq, dk, params[0], params[1], params[2], params[3]


def _is_dense(t: torch.Tensor) -> bool:
    """Whether the elements fill one block of memory, in any dimension order."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if stride != want:
            return False
        want *= size
    return True


def ag_grad_clip(grads, max_norm: float, eps: float = 1e-6,
                 norm: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The global 2-norm of the gradients and their scaling in place by
    min(1, max_norm / (norm + eps)) (libag kernels).

    grads: a sequence of dense fp32, bf16 or fp16 tensors on one device, none
    overlapping another (None entries are skipped).  max_norm = math.inf only
    measures.  Returns the norm before scaling, an fp32 scalar tensor on the
    device (`norm` if given); nothing waits for it."""
    grads = [g for g in grads if g is not None]
    if not grads:
        raise ValueError("grads has no tensor")
    _on_gpu(grads[0], "every gradient", DTYPES)
    dev = grads[0].device
    if _elsewhere(dev, stream):
        with _site(dev, stream):
            return ag_grad_clip(grads, max_norm, eps, norm)
    n, index = len(grads), dev.index
    try:
        types = [DTYPES[g.dtype] for g in grads]
        well = all([g.get_device() == index and g.is_contiguous() for g in grads])
    except (AttributeError, KeyError, RuntimeError):
        well = False
    if not well:
        for g in grads:
            _on_gpu(g, "every gradient", DTYPES)
            _same_device(g, "one", dev)
            if g.layout != torch.strided or not _is_dense(g):
                raise ValueError("every gradient must be dense")
    ptrs = (ctypes.c_void_p * n)(*[g.data_ptr() for g in grads])
    counts = (ctypes.c_int64 * n)(*[g.numel() for g in grads])
    codes = (ctypes.c_int * n)(*types)
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=dev)
    else:
        _on_gpu(norm, "norm", (torch.float32,))
        _same_device(norm, "norm", dev)
        if norm.numel() != 1:
            raise ValueError("norm must have one element")
    ws, wsp, size = _workspace(lib.ag_grad_clip_workspace, dev, "ag_grad_clip_workspace", n)
    st = lib.ag_grad_clip(ptrs, counts, codes, n, max_norm, eps, norm.data_ptr(), wsp, size,
                          _current(dev))
    if st != AG_OK:
        raise AgError("ag_grad_clip", st)
    return norm


def ag_device_error(device: int = 0, clear: bool = True) -> int:
    """Synchronise `device` and return (and optionally clear) its error word."""
    code = ctypes.c_int(0)
    st = lib.ag_device_error(int(device), ctypes.byref(code), 1 if clear else 0)
    if st not in (AG_OK, 8):
        raise AgError("ag_device_error", st)
    return int(code.value)


def ag_debug_wait_timeout(timeout_ns: int, stream=None) -> None:
    """Launch the bounded-wait self-test kernel (see include/ag.h)."""
    st = lib.ag_debug_wait_timeout(int(timeout_ns), _stream_ptr(stream))
    if st != AG_OK:
        raise AgError("ag_debug_wait_timeout", st)


INF = math.inf
