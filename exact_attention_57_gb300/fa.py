"""ctypes binding of ``libfa.so`` (the C ABI in include/fa.h).

The ``fa_*`` functions mirror the C entry points one to one and only marshal
arguments.  ``attention``, ``attention_varlen``, ``attention_backward`` and the
serving operators (``kv_plan``, ``rotary``, ``kv4_append``, ``kv4_gather``,
``attention_kv4``, the same over 8 bits, ``kv_copy``, ``kv_fork``, ``kv_free``,
``kv_compact``) are convenience wrappers for torch tensors: they allocate
outputs and workspaces with torch (device memory is the only thing torch
provides here) and call the C entry points.

There is no fallback: if the library is missing or its call fails, these
functions raise.
"""
from __future__ import annotations

import ctypes
import math
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfa.so")
BIND_PATH = os.path.join(PKG, "_fa_torch.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_DEVICE_TIMEOUT = 4

FA_DTYPE_BF16 = 0
FA_DTYPE_F32 = 1
FA_DTYPE_F32_SIMT = 2
FA_DTYPE_F16 = 3

EXPORTED = ("fa_fwd", "fa_fwd_host", "fa_fwd_status", "fa_status_string", "fa_version",
            "fa_set_test_hooks", "fa_debug_build", "fa_set_debug_lse_shrink",
            "fa_set_fwd_schedule", "fa_fwd_schedule", "fa_fwd_schedule_covers",
            "fa_fwd_noalloc",
            "fa_fwd_splitkv", "fa_fwd_splitkv_workspace",
            "fa_fwd_varlen", "fa_bwd", "fa_bwd_workspace", "fa_fwd_staged",
            "fa_fwd_staged_workspace", "fa_bwd_varlen", "fa_bwd_varlen_workspace",
            "fa_kv_plan", "fa_rope_table", "fa_rope", "fa_kv4_append", "fa_kv4_gather",
            "fa_fwd_kv4", "fa_fwd_kv4_workspace", "fa_fwd_kv4_schedule",
            "fa_kv8_append", "fa_kv8_gather", "fa_fwd_kv8", "fa_fwd_kv8_workspace",
            "fa_fwd_kv8_schedule", "fa_kv_copy", "fa_kv_fork", "fa_kv_free", "fa_kv_compact",
            "fa_kv_compact_workspace")

_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fa_status_string(status)} ({status})")


def load(path: str | None = None):
    """Load libfa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with exact_attention_57_gb300.build")
    lib = ctypes.CDLL(p)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp,
                                   ctypes.POINTER(i)]
    lib.fa_fwd_noalloc.restype = i
    lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp,
                                   ctypes.c_ulonglong, vp]
    lib.fa_fwd_splitkv.restype = i
    lib.fa_fwd_splitkv_workspace.argtypes = [i, i, i, i, i]
    lib.fa_fwd_splitkv_workspace.restype = ctypes.c_ulonglong
    lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_varlen.restype = i
    lib.fa_fwd_staged.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp,
                                  ctypes.c_ulonglong, vp]
    lib.fa_fwd_staged.restype = i
    lib.fa_fwd_staged_workspace.argtypes = [i, i, i, i, i]
    lib.fa_fwd_staged_workspace.restype = ctypes.c_ulonglong
    lib.fa_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i,
                                  f, i, i, vp, ctypes.c_ulonglong, vp]
    lib.fa_bwd_varlen.restype = i
    lib.fa_bwd_varlen_workspace.argtypes = [i, i, i, i, i]
    lib.fa_bwd_varlen_workspace.restype = ctypes.c_ulonglong
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp,
                           ctypes.c_ulonglong, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_workspace.argtypes = [i, i, i, i]
    lib.fa_bwd_workspace.restype = ctypes.c_ulonglong
    lib.fa_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_host.restype = i
    lib.fa_fwd_status.argtypes = [vp, ctypes.POINTER(i)]
    lib.fa_fwd_status.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_version.argtypes = []
    lib.fa_version.restype = i
    lib.fa_set_test_hooks.argtypes = [i, ctypes.c_ulonglong]
    lib.fa_set_test_hooks.restype = i
    lib.fa_debug_build.argtypes = []
    lib.fa_debug_build.restype = i
    lib.fa_set_debug_lse_shrink.argtypes = [ctypes.c_longlong]
    lib.fa_set_debug_lse_shrink.restype = i
    lib.fa_set_fwd_schedule.argtypes = [i, i, i]
    lib.fa_set_fwd_schedule.restype = i
    lib.fa_fwd_schedule.argtypes = [i] * 8 + [ctypes.POINTER(i)] * 3
    lib.fa_fwd_schedule.restype = i
    lib.fa_fwd_schedule_covers.argtypes = [i] * 5
    lib.fa_fwd_schedule_covers.restype = i
    ll, ull = ctypes.c_longlong, ctypes.c_ulonglong
    lib.fa_kv_plan.argtypes = [vp] * 10 + [i] * 5 + [vp]
    lib.fa_kv_plan.restype = i
    lib.fa_rope_table.argtypes = [vp, vp, i, vp]
    lib.fa_rope_table.restype = i
    lib.fa_rope.argtypes = [vp, vp, vp, i, vp, vp, vp, i, vp, i, vp] + [i] * 7 + [vp]
    lib.fa_rope.restype = i
    lib.fa_kv4_append.argtypes = [vp, vp, ll, ll, vp, i, vp, vp, vp, vp] + [i] * 7 + [vp]
    lib.fa_kv4_append.restype = i
    lib.fa_kv4_gather.argtypes = [vp, i] + [vp] * 6 + [i] * 7 + [vp]
    lib.fa_kv4_gather.restype = i
    lib.fa_fwd_kv4.argtypes = [vp] * 10 + [i] * 10 + [f] + [i] * 4 + [vp, ull, vp]
    lib.fa_fwd_kv4.restype = i
    lib.fa_fwd_kv4_workspace.argtypes = [i] * 5
    lib.fa_fwd_kv4_workspace.restype = ull
    lib.fa_fwd_kv4_schedule.argtypes = [i] * 9 + [ctypes.POINTER(i)] * 5
    lib.fa_fwd_kv4_schedule.restype = i
    lib.fa_kv8_append.argtypes = [vp, vp, ll, ll, vp, i, vp, vp, vp, vp] + [i] * 5 + [vp]
    lib.fa_kv8_append.restype = i
    lib.fa_kv8_gather.argtypes = [vp, i] + [vp] * 6 + [i] * 5 + [vp]
    lib.fa_kv8_gather.restype = i
    lib.fa_fwd_kv8.argtypes = [vp] * 10 + [i] * 10 + [f] + [i] * 2 + [vp, ull, vp]
    lib.fa_fwd_kv8.restype = i
    lib.fa_fwd_kv8_workspace.argtypes = [i] * 5
    lib.fa_fwd_kv8_workspace.restype = ull
    lib.fa_fwd_kv8_schedule.argtypes = [i] * 9 + [ctypes.POINTER(i)] * 5
    lib.fa_fwd_kv8_schedule.restype = i
    lib.fa_kv_copy.argtypes = [vp, vp, i, vp, vp, vp, i, i, i, vp]
    lib.fa_kv_copy.restype = i
    lib.fa_kv_fork.argtypes = [vp] * 8 + [i] * 7 + [vp, vp, i, vp]
    lib.fa_kv_fork.restype = i
    lib.fa_kv_free.argtypes = [vp] * 5 + [i] * 4 + [vp]
    lib.fa_kv_free.restype = i
    lib.fa_kv_compact.argtypes = [vp] * 5 + [i] * 4 + [vp, vp, i, vp, ull, vp]
    lib.fa_kv_compact.restype = i
    lib.fa_kv_compact_workspace.argtypes = [i]
    lib.fa_kv_compact_workspace.restype = ull
    if path is None:
        _lib = lib
    return lib


def fa_fwd(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, dtype, stream) -> int:
    """Raw C call; pointers and stream are integers (0 = NULL)."""
    return load().fa_fwd(q, k, v, o, lse, B, H, Nq, Nk, d, float(scale), int(causal),
                         int(dtype), stream)


def fa_fwd_noalloc(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, dtype, stream,
                   wait: bool = True):
    """Raw C call of the entry point that allocates no device memory.

    With wait=True the call synchronises the stream and returns
    (status, raw status word); with wait=False it only enqueues and returns
    (status, None)."""
    word = ctypes.c_int(0)
    st = load().fa_fwd_noalloc(q, k, v, o, lse, B, H, Nq, Nk, d, float(scale), int(causal),
                               int(dtype), stream, ctypes.byref(word) if wait else None)
    return st, (word.value if wait else None)


def fa_fwd_splitkv(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, dtype, num_splits,
                   workspace, workspace_bytes, stream) -> int:
    return load().fa_fwd_splitkv(q, k, v, o, lse, B, H, Nq, Nk, d, float(scale), int(causal),
                                 int(dtype), int(num_splits), workspace, int(workspace_bytes),
                                 stream)


def fa_fwd_splitkv_workspace(B, H, Nq, d, num_splits) -> int:
    return load().fa_fwd_splitkv_workspace(B, H, Nq, d, num_splits)


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, H, total_q, total_k,
                  max_seqlen_q, d, scale, causal, dtype, stream) -> int:
    return load().fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, B, H, total_q,
                                total_k, max_seqlen_q, d, float(scale), int(causal), int(dtype),
                                stream)


def attention_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                     scale: float | None = None, causal: bool = False, out=None, lse=None,
                     stream=None):
    """Packed sequences: q [total_q, H, d], k/v [total_k, H, d], cu_seqlens
    int32 CUDA tensors of B+1 offsets.  Returns (o [total_q, H, d],
    lse [H, total_q])."""
    import torch
    total_q, H, d = q.shape
    total_k = k.shape[0]
    if k.shape[1:] != (H, d) or v.shape != k.shape:
        raise ValueError("q [total_q,H,d], k and v [total_k,H,d] expected")
    if cu_seqlens_q.dtype != torch.int32 or cu_seqlens_k.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    B = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != B + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k need the same batch size")
    code = _dtype_code(q, "tc")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((H, total_q), device=q.device, dtype=torch.float32)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    with torch.cuda.device(q.device):
        st = fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           lse.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B,
                           H, total_q, total_k, max_seqlen_q, d, scale, int(bool(causal)), code,
                           stream)
    if st != FA_OK:
        raise FaError(st, "fa_fwd_varlen")
    return out, lse


def fa_fwd_staged(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, dtype, workspace,
                  workspace_bytes, stream) -> int:
    return load().fa_fwd_staged(q, k, v, o, lse, B, H, Nq, Nk, d, float(scale), int(causal),
                                int(dtype), workspace, int(workspace_bytes), stream)


def fa_fwd_staged_workspace(B, H, Nk, d, dtype) -> int:
    return load().fa_fwd_staged_workspace(B, H, Nk, d, dtype)


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H, Nq, Nk, d, scale, causal, dtype,
           workspace, workspace_bytes, stream) -> int:
    return load().fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H, Nq, Nk, d, float(scale),
                         int(causal), int(dtype), workspace, int(workspace_bytes), stream)


def fa_bwd_workspace(B, H, Nq, d) -> int:
    return load().fa_bwd_workspace(B, H, Nq, d)


def attention_backward(q, k, v, out, lse, dout, scale: float | None = None,
                       causal: bool = False, dq=None, dk=None, dv=None, workspace=None,
                       stream=None):
    """Gradients (dq, dk, dv) of attention() for the upstream gradient dout.

    q, k, v, dout, out: contiguous bf16 / fp16 / fp32 CUDA tensors as for
    attention() (fp32 runs the CUDA-core backward, head dim up to 128);
    out and lse are that forward's outputs.  The workspace (fa_bwd_workspace
    bytes) is allocated with torch unless given.  Raises FaError on failure."""
    import torch
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    for t in (k, v, out, dout):
        if t.dtype != q.dtype or not t.is_contiguous():
            raise ValueError("q, k, v, out, dout: contiguous tensors of one dtype")
    if out.shape != q.shape or dout.shape != q.shape or v.shape != k.shape:
        raise ValueError("shape mismatch")
    # fp32 gradients come from the CUDA-core backward whichever fp32 forward
    # ran; its dtype code admits every head dim up to 128
    code = _dtype_code(q, "simt" if q.dtype == torch.float32 else "tc")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ws_bytes = fa_bwd_workspace(B, H, Nq, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    with torch.cuda.device(q.device):
        st = fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                    dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Nq, Nk,
                    d, scale, int(bool(causal)), code, workspace.data_ptr(),
                    workspace.numel() * workspace.element_size(), stream)
    if st != FA_OK:
        raise FaError(st, "fa_bwd")
    return dq, dk, dv


def fa_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, B, H, total_q,
                  total_k, max_seqlen_q, max_seqlen_k, d, scale, causal, dtype, workspace,
                  workspace_bytes, stream) -> int:
    return load().fa_bwd_varlen(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, B,
                                H, total_q, total_k, max_seqlen_q, max_seqlen_k, d, float(scale),
                                int(causal), int(dtype), workspace, int(workspace_bytes), stream)


def fa_bwd_varlen_workspace(B, H, total_q, max_seqlen_q, d) -> int:
    return load().fa_bwd_varlen_workspace(B, H, total_q, max_seqlen_q, d)


def attention_backward_varlen(q, k, v, out, lse, dout, cu_seqlens_q, cu_seqlens_k,
                              max_seqlen_q: int, max_seqlen_k: int, scale: float | None = None,
                              causal: bool = False, stream=None):
    """Gradients (dq, dk, dv) of attention_varlen() for the upstream gradient
    dout (token-major [total_q, H, d]).  Raises FaError on failure."""
    import torch
    total_q, H, d = q.shape
    total_k = k.shape[0]
    B = cu_seqlens_q.numel() - 1
    code = _dtype_code(q, "tc")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws_bytes = fa_bwd_varlen_workspace(B, H, total_q, max_seqlen_q, d)
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    with torch.cuda.device(q.device):
        st = fa_bwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                           dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                           cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, H, total_q,
                           total_k, max_seqlen_q, max_seqlen_k, d, scale, int(bool(causal)), code,
                           ws.data_ptr(), ws_bytes, stream)
    if st != FA_OK:
        raise FaError(st, "fa_bwd_varlen")
    return dq, dk, dv


def fa_fwd_host(q_h, k_h, v_h, o_h, lse_h, q_d, k_d, v_d, o_d, lse_d,
                B, H, Nq, Nk, d, scale, causal, dtype, stream) -> int:
    return load().fa_fwd_host(q_h, k_h, v_h, o_h, lse_h, q_d, k_d, v_d, o_d, lse_d,
                              B, H, Nq, Nk, d, float(scale), int(causal), int(dtype), stream)


def fa_fwd_status(stream=None):
    """Returns (status, raw device status word)."""
    word = ctypes.c_int(0)
    st = load().fa_fwd_status(stream, ctypes.byref(word))
    return st, word.value


def fa_status_string(status: int) -> str:
    try:
        return load().fa_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def fa_version() -> int:
    return load().fa_version()


def fa_set_test_hooks(skip_v_load: int = 0, wait_limit_ns: int = 0) -> int:
    return load().fa_set_test_hooks(int(skip_v_load), int(wait_limit_ns))


def fa_set_fwd_schedule(ctas: int = 0, group_heads: int = 0, block_items: int = 0) -> int:
    """Testing aid: force the 16-bit forward's schedule (0 = automatic)."""
    return load().fa_set_fwd_schedule(int(ctas), int(group_heads), int(block_items))


def fa_fwd_schedule(B: int, H: int, Nq: int, Nk: int, d: int, causal: bool, dtype: int,
                    num_sms: int):
    """(status, CTAs, planes per group, items per CTA of the blocked schedule
    or 0) of fa_fwd's schedule on a GPU with num_sms SMs (host-only)."""
    c, g, b = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    st = load().fa_fwd_schedule(int(B), int(H), int(Nq), int(Nk), int(d), int(bool(causal)),
                                int(dtype), int(num_sms), ctypes.byref(c), ctypes.byref(g),
                                ctypes.byref(b))
    return st, c.value, g.value, b.value


def fa_fwd_schedule_covers(planes: int, n: int, ctas: int, group_heads: int,
                           block_items: int = 0) -> bool:
    """Host-only check that the schedule deals every item exactly once."""
    return bool(load().fa_fwd_schedule_covers(int(planes), int(n), int(ctas), int(group_heads),
                                              int(block_items)))


# --------------------------------------------------------------- torch helpers
def _dtype_code(t, impl: str) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        if impl != "tc":
            raise ValueError("bf16 inputs run on the tensor-core kernel only")
        return FA_DTYPE_BF16
    if t.dtype == torch.float16:
        if impl != "tc":
            raise ValueError("fp16 inputs run on the tensor-core kernel only")
        return FA_DTYPE_F16
    if t.dtype == torch.float32:
        return FA_DTYPE_F32 if impl == "tc" else FA_DTYPE_F32_SIMT
    raise ValueError(f"unsupported dtype {t.dtype}")


def attention(q, k, v, scale: float | None = None, causal: bool = False, impl: str = "tc",
              out=None, lse=None, stream=None, num_splits: int | None = None,
              staged: bool = False):
    """O, LSE for contiguous CUDA tensors q [B,H,Nq,d], k/v [B,H,Nk,d].

    impl "tc": bf16 / fp16 -> tcgen05 kind::f16, fp32 -> tcgen05 kind::tf32;
    impl "simt": fp32 only, plain fp32 kernel.  num_splits (tensor-core
    dtypes): split each query tile's key range into that many chunks (0 =
    automatic) through fa_fwd_splitkv, with a torch-allocated workspace.
    staged (fp32, impl "tc"): run fa_fwd_staged, converting K and V once per
    call into a torch-allocated workspace (scores as three bf16 products of
    split operands instead of fa_fwd's three tf32 ones).  Raises FaError on failure.
    """
    import torch
    if not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise ValueError("attention() needs CUDA tensors")
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape:
        raise ValueError("q [B,H,Nq,d], k and v [B,H,Nk,d] expected")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape[0] != B or k.shape[1] != H or k.shape[3] != d:
        raise ValueError("k/v shape does not match q")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("contiguous [B,H,N,d] tensors expected")
    code = _dtype_code(q, impl)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share a dtype")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), device=q.device, dtype=torch.float32)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    with torch.cuda.device(q.device):
        if staged and code == FA_DTYPE_F32:
            ws_bytes = fa_fwd_staged_workspace(B, H, Nk, d, code)
            ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=q.device)
            st = fa_fwd_staged(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                               lse.data_ptr(), B, H, Nq, Nk, d, scale, int(bool(causal)), code,
                               ws.data_ptr(), ws_bytes, stream)
            where = "fa_fwd_staged"
        elif num_splits is None:
            st = fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                        lse.data_ptr(), B, H, Nq, Nk, d, scale, int(bool(causal)), code, stream)
            where = "fa_fwd"
        else:
            nws = num_splits if num_splits > 0 else 64
            ws_bytes = fa_fwd_splitkv_workspace(B, H, Nq, d, nws)
            ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=q.device)
            st = fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                lse.data_ptr(), B, H, Nq, Nk, d, scale, int(bool(causal)), code,
                                num_splits, ws.data_ptr(), ws_bytes, stream)
            where = "fa_fwd_splitkv"
    if st != FA_OK:
        raise FaError(st, where)
    return out, lse


# ----------------------------------------------------------- serving operators
def fa_kv_plan(cached_lens, new_lens, free_blocks, free_head, block_table, slots, positions,
               cu_seqlens, seq_lens, counts, B, max_blocks, block_size, num_free, capacity,
               stream) -> int:
    return load().fa_kv_plan(cached_lens, new_lens, free_blocks, free_head, block_table, slots,
                             positions, cu_seqlens, seq_lens, counts, B, max_blocks, block_size,
                             num_free, capacity, stream)


def fa_rope_table(inv_freq, axis, n, table) -> int:
    return load().fa_rope_table(inv_freq, axis, n, table)


def fa_rope(q, q_out, q_strides, Hq, k, k_out, k_strides, Hk, positions, num_axes, table, B, N, d,
            d_rot, interleaved, inverse, dtype, stream) -> int:
    return load().fa_rope(q, q_out, q_strides, Hq, k, k_out, k_strides, Hk, positions, num_axes,
                          table, B, N, d, d_rot, int(interleaved), int(inverse), dtype, stream)


def fa_kv4_append(k, v, k_stride, v_stride, slots, T, k_codes, k_scales, v_codes, v_scales,
                  num_blocks, Hk, block_size, d, k_exp, v_exp, dtype, stream) -> int:
    return load().fa_kv4_append(k, v, k_stride, v_stride, slots, T, k_codes, k_scales, v_codes,
                                v_scales, num_blocks, Hk, block_size, d, k_exp, v_exp, dtype,
                                stream)


def fa_kv4_gather(slots, R, k_codes, k_scales, v_codes, v_scales, k_out, v_out, num_blocks, Hk,
                  block_size, d, k_exp, v_exp, dtype, stream) -> int:
    return load().fa_kv4_gather(slots, R, k_codes, k_scales, v_codes, v_scales, k_out, v_out,
                                num_blocks, Hk, block_size, d, k_exp, v_exp, dtype, stream)


def fa_fwd_kv4(q, o, lse, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens_k,
               cu_seqlens_q, B, Hq, Hk, total_q, max_seqlen_q, max_seqlen_k, num_blocks,
               block_size, max_blocks, d, scale, causal, k_exp, v_exp, dtype, workspace,
               workspace_bytes, stream) -> int:
    return load().fa_fwd_kv4(q, o, lse, k_codes, k_scales, v_codes, v_scales, block_table,
                             seq_lens_k, cu_seqlens_q, B, Hq, Hk, total_q, max_seqlen_q,
                             max_seqlen_k, num_blocks, block_size, max_blocks, d, scale, causal,
                             k_exp, v_exp, dtype, workspace, workspace_bytes, stream)


def fa_fwd_kv4_workspace(B, Hq, Hk, max_seqlen_q, d) -> int:
    return load().fa_fwd_kv4_workspace(B, Hq, Hk, max_seqlen_q, d)


def fa_fwd_kv4_schedule(B, Hq, Hk, max_seqlen_q, max_seqlen_k, max_blocks, block_size, d, num_sms):
    """(status, bound on the keys, rows of the tile for few rows, CTAs of its
    clusters, its CTAs, CTAs of the kernel for more rows) of fa_fwd_kv4 on a
    GPU with num_sms SMs (host-only)."""
    r = [ctypes.c_int(0) for _ in range(5)]
    st = load().fa_fwd_kv4_schedule(int(B), int(Hq), int(Hk), int(max_seqlen_q), int(max_seqlen_k),
                                    int(max_blocks), int(block_size), int(d), int(num_sms),
                                    *map(ctypes.byref, r))
    return (st, *(x.value for x in r))


def fa_kv8_append(k, v, k_stride, v_stride, slots, T, k_codes, k_scales, v_codes, v_scales,
                  num_blocks, Hk, block_size, d, dtype, stream) -> int:
    return load().fa_kv8_append(k, v, k_stride, v_stride, slots, T, k_codes, k_scales, v_codes,
                                v_scales, num_blocks, Hk, block_size, d, dtype, stream)


def fa_kv8_gather(slots, R, k_codes, k_scales, v_codes, v_scales, k_out, v_out, num_blocks, Hk,
                  block_size, d, dtype, stream) -> int:
    return load().fa_kv8_gather(slots, R, k_codes, k_scales, v_codes, v_scales, k_out, v_out,
                                num_blocks, Hk, block_size, d, dtype, stream)


def fa_fwd_kv8(q, o, lse, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens_k,
               cu_seqlens_q, B, Hq, Hk, total_q, max_seqlen_q, max_seqlen_k, num_blocks,
               block_size, max_blocks, d, scale, causal, dtype, workspace, workspace_bytes,
               stream) -> int:
    return load().fa_fwd_kv8(q, o, lse, k_codes, k_scales, v_codes, v_scales, block_table,
                             seq_lens_k, cu_seqlens_q, B, Hq, Hk, total_q, max_seqlen_q,
                             max_seqlen_k, num_blocks, block_size, max_blocks, d, scale, causal,
                             dtype, workspace, workspace_bytes, stream)


def fa_fwd_kv8_workspace(B, Hq, Hk, max_seqlen_q, d) -> int:
    return load().fa_fwd_kv8_workspace(B, Hq, Hk, max_seqlen_q, d)


def fa_fwd_kv8_schedule(B, Hq, Hk, max_seqlen_q, max_seqlen_k, max_blocks, block_size, d, num_sms):
    """fa_fwd_kv4_schedule's values for fa_fwd_kv8 (host-only)."""
    r = [ctypes.c_int(0) for _ in range(5)]
    st = load().fa_fwd_kv8_schedule(int(B), int(Hq), int(Hk), int(max_seqlen_q), int(max_seqlen_k),
                                    int(max_blocks), int(block_size), int(d), int(num_sms),
                                    *map(ctypes.byref, r))
    return (st, *(x.value for x in r))


def _pages(arrays, page_bytes):
    """Host arrays of device pointers and page sizes, as the C entry points take them."""
    n = len(page_bytes)
    return ((ctypes.c_void_p * max(n, 1))(*arrays), (ctypes.c_ulonglong * max(n, 1))(*page_bytes), n)


def fa_kv_copy(src, dst, n, from_arrays, to_arrays, page_bytes, from_blocks, to_blocks,
               stream) -> int:
    """from_arrays, to_arrays: lists of device addresses; page_bytes: a list of sizes."""
    f, b, num = _pages(from_arrays, page_bytes)
    t, _, _ = _pages(to_arrays, page_bytes)
    return load().fa_kv_copy(src, dst, n, f, t, b, num, from_blocks, to_blocks, stream)


def fa_kv_fork(block_table, seq_lens, parents, free_blocks, free_head, table_out, lens_out, counts,
               B, n, max_blocks, block_size, num_free, num_blocks, parents_end, arrays, page_bytes,
               stream) -> int:
    a, b, num = _pages(arrays, page_bytes)
    return load().fa_kv_fork(block_table, seq_lens, parents, free_blocks, free_head, table_out,
                             lens_out, counts, B, n, max_blocks, block_size, num_free, num_blocks,
                             int(parents_end), a, b, num, stream)


def fa_kv_free(block_table, seq_lens, ended, free_blocks, free_head, B, max_blocks, block_size,
               num_blocks, stream) -> int:
    return load().fa_kv_free(block_table, seq_lens, ended, free_blocks, free_head, B, max_blocks,
                             block_size, num_blocks, stream)


def fa_kv_compact(block_table, seq_lens, table_out, new_ids, counts, B, max_blocks, block_size,
                  num_blocks, arrays, page_bytes, workspace, workspace_bytes, stream) -> int:
    a, b, num = _pages(arrays, page_bytes)
    return load().fa_kv_compact(block_table, seq_lens, table_out, new_ids, counts, B, max_blocks,
                                block_size, num_blocks, a, b, num, workspace,
                                int(workspace_bytes), stream)


def fa_kv_compact_workspace(num_blocks) -> int:
    return load().fa_kv_compact_workspace(num_blocks)


# The wrappers below run once or more in every layer of every step of a server,
# where a launch takes about 3 us of host time.  Their checks, allocations and
# calls of the C entry points are compiled (csrc/bind/fa_torch.cpp): 2.5 to 6.5 us a
# call, 10 where the attention launches two kernels and their joins, where the same
# in Python took 8 to 20.  `stream` is the integer of a
# cudaStream_t (default: the current one); what it has to wait for, the inputs
# among it, is the caller's to order, and what a wrapper allocates belongs to it.
_torch = None


def _bind():
    """The compiled module, bound to the C entry points of load()."""
    global _torch
    if not os.path.exists(BIND_PATH):
        raise RuntimeError(f"{BIND_PATH} is missing: build it with exact_attention_57_gb300.build")
    import importlib.util

    import torch  # noqa: F401  (the module links to its libraries)
    spec = importlib.util.spec_from_file_location("_fa_torch", BIND_PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    lib = load()
    mod.bind(*[ctypes.cast(f, ctypes.c_void_p).value
               for f in (lib.fa_kv_plan, lib.fa_rope, lib.fa_kv4_append, lib.fa_kv4_gather,
                         lib.fa_fwd_kv4, lib.fa_fwd_kv4_workspace, lib.fa_kv8_append,
                         lib.fa_kv8_gather, lib.fa_fwd_kv8, lib.fa_fwd_kv8_workspace,
                         lib.fa_kv_copy, lib.fa_kv_fork, lib.fa_kv_free, lib.fa_kv_compact,
                         lib.fa_kv_compact_workspace)])
    _torch = mod
    return mod


def _done(result, where):
    """What a compiled wrapper returns: its outputs, or the status of a refusal."""
    if result.__class__ is int:
        raise FaError(result, where)
    return result


def kv_plan(cached_lens, new_lens, free_blocks, block_table, block_size: int, capacity: int,
            free_head=None, out=None, stream=None):
    """Block tables and slot maps of a paged cache from request lengths.

    cached_lens, new_lens: int32 [B]; free_blocks: int32 ids of free blocks
    (free_head: int32 [1], how many are used already); block_table: int32
    [B, max_blocks], updated in place.  capacity: length of the token arrays.
    Returns (slots int64 [capacity], positions int32 [capacity], cu_seqlens
    int32 [B+1], seq_lens int32 [B], counts int32 [2]: blocks needed, tokens);
    out: those five tensors, to write to.  Raises FaError on failure."""
    return _done((_torch or _bind()).kv_plan(cached_lens, new_lens, free_blocks, block_table,
                                             block_size, capacity, free_head,
                                             out if out is None else tuple(out), stream),
                 "fa_kv_plan")


def rotary_table(inv_freq, axes=None, device="cuda"):
    """The int64 table rotary() takes: inv_freq, radians per position of each
    pair; axes, the axis (0 .. 3) that turns it (default 0)."""
    import torch
    n = len(inv_freq)
    f = (ctypes.c_double * n)(*[float(x) for x in inv_freq])
    a = None
    if axes is not None:
        if len(axes) != n:
            raise ValueError("one axis a pair expected")
        a = (ctypes.c_int * n)(*[int(x) for x in axes])
    t = torch.empty(n, dtype=torch.int64)
    st = load().fa_rope_table(f, a, n, t.data_ptr())
    if st != FA_OK:
        raise FaError(st, "fa_rope_table")
    return t.to(device)


def rotary(q, k, positions, table, interleaved: bool = False, q_out=None, k_out=None,
           stream=None, inverse: bool = False):
    """Rotary positions on q and k: [B, H, N, d] with positions int32
    [axes, B, N], or token-major [T, H, d] with positions int32 [axes, T]; any
    strides with contiguous rows (slices of a fused projection); k may be
    None.  table: rotary_table() over d_rot/2 pairs.  q_out, k_out: where to
    write (q and k themselves rotate in place; default: new tensors).
    Returns (q_out, k_out).  Raises FaError on failure."""
    return _done((_torch or _bind()).rotary(q, k, positions, table, interleaved, q_out, k_out,
                                            stream, inverse), "fa_rope")


def rotary_backward(dq, dk, positions, table, interleaved: bool = False, q_out=None, k_out=None,
                    stream=None):
    """Gradients of rotary()'s inputs from those of its outputs: the inverse
    rotation, with rotary()'s arguments."""
    return rotary(dq, dk, positions, table, interleaved, q_out, k_out, stream, inverse=True)


def kv4_cache(num_blocks: int, Hk: int, block_size: int, d: int, device="cuda"):
    """A zeroed 4-bit cache: (k_codes, k_scales, v_codes, v_scales)."""
    import torch
    shape = (num_blocks, Hk, block_size)
    return tuple(torch.zeros(shape + (n,), dtype=torch.uint8, device=device)
                 for n in (d // 2, d // 16, d // 2, d // 16))


def kv4_append(k, v, slots, k_codes, k_scales, v_codes, v_scales, k_exp: int = 0, v_exp: int = 0,
               stream=None):
    """Write rows k, v [T, Hk, d] (bf16, fp16 or fp32; rows of any stride, e.g.
    slices of a fused projection) into the 4-bit cache at slots int64 [T]
    (-1 skips a row).  Raises FaError on failure."""
    _done((_torch or _bind()).kv4_append(k, v, slots, k_codes, k_scales, v_codes, v_scales, k_exp,
                                         v_exp, stream), "fa_kv4_append")


def kv4_gather(slots, k_codes, k_scales, v_codes, v_scales, dtype=None, k_exp: int = 0,
               v_exp: int = 0, out=None, stream=None):
    """Rows of the 4-bit cache at slots int64 [R] (-1 reads zeros) as (k, v),
    each [R, Hk, d] of `dtype` (default bf16); out: those two tensors, to write
    to.  Raises FaError on failure."""
    return _done((_torch or _bind()).kv4_gather(slots, k_codes, k_scales, v_codes, v_scales, dtype,
                                                k_exp, v_exp, out if out is None else tuple(out),
                                                stream), "fa_kv4_gather")


def attention_kv4(q, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens_k,
                  max_seqlen_k: int, cu_seqlens_q=None, max_seqlen_q: int = 1,
                  scale: float | None = None, causal: bool = True, k_exp: int = 0, v_exp: int = 0,
                  out=None, lse=None, workspace=None, stream=None):
    """Attention of q [total_q, Hq, d] (bf16 or fp16) over the 4-bit paged cache.

    block_table int32 [B, max_blocks], seq_lens_k int32 [B]; cu_seqlens_q
    int32 [B+1] (None: one query a sequence).  Returns (o [total_q, Hq, d],
    lse [Hq, total_q]).  The workspace (fa_fwd_kv4_workspace bytes) is
    allocated with torch unless given.  Raises FaError on failure."""
    return _done((_torch or _bind()).attention_kv4(
        q, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens_k, max_seqlen_k, cu_seqlens_q,
        max_seqlen_q, scale, causal, k_exp, v_exp, (out, lse), workspace, stream), "fa_fwd_kv4")


def kv8_cache(num_blocks: int, Hk: int, block_size: int, d: int, device="cuda"):
    """A zeroed 8-bit cache: (k_codes, k_scales, v_codes, v_scales), codes
    float8_e4m3fn [num_blocks, Hk, block_size, d] and scales float32 [num_blocks, Hk]."""
    import torch
    return tuple(x for _ in "kv" for x in (
        torch.zeros((num_blocks, Hk, block_size, d), dtype=torch.float8_e4m3fn, device=device),
        torch.zeros((num_blocks, Hk), dtype=torch.float32, device=device)))


def kv8_append(k, v, slots, k_codes, k_scales, v_codes, v_scales, stream=None):
    """Write rows k, v [T, Hk, d] (bf16, fp16 or fp32; rows of any stride, e.g.
    slices of a fused projection) into the 8-bit cache at slots int64 [T] (-1
    skips a row); the rows of a block follow one another, as kv_plan deals them.
    A block's scale grows with its largest element, and what it held keeps its
    values.  Raises FaError on failure."""
    _done((_torch or _bind()).kv8_append(k, v, slots, k_codes, k_scales, v_codes, v_scales, stream),
          "fa_kv8_append")


def kv8_gather(slots, k_codes, k_scales, v_codes, v_scales, dtype=None, out=None, stream=None):
    """Rows of the 8-bit cache at slots int64 [R] (-1 reads zeros) as (k, v),
    each [R, Hk, d] of `dtype` (default bf16); out: those two tensors, to write
    to.  Raises FaError on failure."""
    return _done((_torch or _bind()).kv8_gather(slots, k_codes, k_scales, v_codes, v_scales, dtype,
                                                out if out is None else tuple(out), stream),
                 "fa_kv8_gather")


def attention_kv8(q, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens_k,
                  max_seqlen_k: int, cu_seqlens_q=None, max_seqlen_q: int = 1,
                  scale: float | None = None, causal: bool = True, out=None, lse=None,
                  workspace=None, stream=None):
    """Attention of q [total_q, Hq, d] (bf16 or fp16) over the 8-bit paged cache,
    with attention_kv4's arguments but for the exponents.  Returns (o
    [total_q, Hq, d], lse [Hq, total_q]).  Raises FaError on failure."""
    return _done((_torch or _bind()).attention_kv8(
        q, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens_k, max_seqlen_k, cu_seqlens_q,
        max_seqlen_q, scale, causal, (out, lse), workspace, stream), "fa_fwd_kv8")


def kv_copy(src, dst, caches, to=None, stream=None):
    """Copy page src[i] to page dst[i] (int32 [n] each; ids outside the cache skip
    a pair) of every array in caches, contiguous tensors [num_blocks, ...] such as
    those of kv4_cache() or kv8_cache(), of all layers (256 arrays a call at most;
    several calls with the same inputs take more); to: arrays of another cache
    with the same pages, to write to.  Pages written differ, from one another and
    from those read.  Raises FaError on failure."""
    _done((_torch or _bind()).kv_copy(src, dst, tuple(caches), to if to is None else tuple(to),
                                      stream), "fa_kv_copy")


def kv_fork(block_table, seq_lens, parents, free_blocks, block_size: int, caches=(),
            num_blocks: int | None = None, free_head=None, parents_end: bool = False, out=None,
            stream=None):
    """Requests begun from others' caches: child i continues row parents[i] (int32
    [n]) of block_table [B, max_blocks] at its length; it shares the full blocks and
    gets a copy of the last, partly filled one in a block from free_blocks (with
    parents_end, a parent's first child takes that entry over instead).  caches: the
    arrays to copy in (kv_copy's).  Returns (block_table [n, max_blocks], seq_lens
    [n], counts [2]: blocks needed, entries of free_blocks used up); out: those
    three tensors, to write to.  Raises FaError on failure."""
    return _done((_torch or _bind()).kv_fork(block_table, seq_lens, parents, free_blocks, block_size,
                                             tuple(caches), num_blocks, free_head, parents_end,
                                             out if out is None else tuple(out), stream),
                 "fa_kv_fork")


def kv_free(block_table, seq_lens, num_blocks: int, block_size: int, ended=None, out=None,
            stream=None):
    """The blocks that no row of block_table holds, for kv_plan and kv_fork: returns
    (free_blocks int32 [num_blocks]: -1 for every block held, then the others'
    ids, ascending; free_head int32 [1]); out: those two tensors, to write to.
    ended: bool [B], rows that hold nothing any more; their seq_lens become 0.
    Raises FaError on failure."""
    return _done((_torch or _bind()).kv_free(block_table, seq_lens, num_blocks, block_size, ended,
                                             out if out is None else tuple(out), stream),
                 "fa_kv_free")


def kv_compact(block_table, seq_lens, caches, block_size: int, num_blocks: int | None = None,
               out=None, workspace=None, stream=None):
    """Bring the blocks that rows hold to the front of the cache: moves their pages
    in every array of caches (kv_copy's) and returns (block_table with the new ids,
    new_ids int32 [num_blocks]: -1 for blocks not held, counts [2]: blocks held,
    pages moved); out: those three tensors, to write to (block_table itself may be
    one, in the last call where more than 256 arrays take several).  The workspace
    (fa_kv_compact_workspace bytes) is allocated with torch unless given.  Raises
    FaError on failure."""
    return _done((_torch or _bind()).kv_compact(block_table, seq_lens, tuple(caches), num_blocks,
                                                block_size, out if out is None else tuple(out),
                                                workspace, stream), "fa_kv_compact")
