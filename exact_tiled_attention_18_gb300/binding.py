"""ctypes binding of libfa.so: the C ABI of include/fa.h, name for name.

Argument marshalling only -- every step of the computation runs in the CUDA
kernels behind these calls.  There is no fallback: if the library was not
built (``python -m exact_tiled_attention_18_gb300.build``) every call raises.
"""

from __future__ import annotations

import ctypes
import os
import threading

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED_D = 2
FA_ERR_MISALIGNED = 3
FA_ERR_LAUNCH = 4
FA_ERR_TIMEOUT = 5
FA_ERR_DEVICE_FAULT = 6
FA_ERR_BAD_PAGE = 7
FA_DECODE_MAX_Q = 8
FA_DTYPE_F32 = 0
FA_DTYPE_BF16 = 1
FA_ROPE_HALF = 0
FA_ROPE_INTERLEAVED = 1
FA_ROPE_SCALE_NONE = 0
FA_ROPE_SCALE_LINEAR = 1
FA_ROPE_SCALE_NTK = 2
FA_ROPE_SCALE_PARTS = 3

_lock = threading.Lock()
_lib = None


class FAError(RuntimeError):
    """A library call returned a status other than FA_OK."""

    def __init__(self, call: str, status: int, text: str):
        super().__init__(f"{call}: {text}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libfa.so once; raise if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise FileNotFoundError(
                f"{LIB_PATH} is missing: build it with `python -m exact_tiled_attention_18_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int
        ll = ctypes.c_longlong
        L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd.restype = st
        L.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_fwd_varlen.restype = st
        L.fa_fwd_ex.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_fwd_ex.restype = st
        L.fa_fwd_bias.argtypes = [vp, vp, vp, vp, i, vp, vp, ll, ll, ll, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_fwd_bias.restype = st
        L.fa_bwd_ex.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_bwd_ex.restype = st
        L.fa_bwd_bias.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, ll, ll, ll, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f,
                                  i, vp]
        L.fa_bwd_bias.restype = st
        L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd_fp8.restype = st
        L.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd_splitkv.restype = st
        L.fa_fwd_splitkv_workspace_bytes.argtypes = [i, i, i, i]
        L.fa_fwd_splitkv_workspace_bytes.restype = ctypes.c_size_t
        L.fa_fwd_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_fwd_decode.restype = st
        L.fa_fwd_decode_workspace_bytes.argtypes = [i, i, i, i, i]
        L.fa_fwd_decode_workspace_bytes.restype = ctypes.c_size_t
        L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_bwd.restype = st
        L.fa_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_bwd_varlen.restype = st
        L.fa_bwd_single_pass.argtypes = [vp, vp, vp, vp, vp, vp, ll, ll, ll, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f,
                                         i, vp]
        L.fa_bwd_single_pass.restype = st
        L.fa_bwd_stage.argtypes = [i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_bwd_stage.restype = st
        L.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_bwd_noalloc.restype = st
        L.fa_bwd_workspace_bytes.argtypes = [i, i, i]
        L.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
        db = ctypes.c_double
        L.fa_rope_turns.argtypes = [ctypes.POINTER(ll), i, db, i, db, db, db, db]
        L.fa_rope_turns.restype = st
        L.fa_rope.argtypes = [vp, i, ll, ll, ll, vp, i, ll, ll, ll, vp, ll, vp, i, i, f, i, i, i, i, i, vp]
        L.fa_rope.restype = st
        L.fa_kv_append.argtypes = [vp, ll, ll, ll, vp, ll, ll, ll, vp, ll, ll, ll, vp, vp, vp, i, i, vp, ll, i, vp, vp,
                                   vp, ll, vp, i, i, f, i, i, i, i, i, vp]
        L.fa_kv_append.restype = st
        L.fa_fwd_paged.argtypes = [vp, vp, vp, i, i, vp, ll, i, vp, i, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        L.fa_fwd_paged.restype = st
        L.fa_fwd_paged_workspace_bytes.argtypes = [i, i, i, i, i]
        L.fa_fwd_paged_workspace_bytes.restype = ctypes.c_size_t
        L.fa_fwd_shared_prefix.argtypes = [vp, vp, vp, i, i, vp, i, vp, ll, i, vp, i, vp, vp, vp, vp, i, i, i, i, i, f,
                                           i, vp]
        L.fa_fwd_shared_prefix.restype = st
        L.fa_fwd_shared_prefix_workspace_bytes.argtypes = [i, i, i, i, i]
        L.fa_fwd_shared_prefix_workspace_bytes.restype = ctypes.c_size_t
        L.fa_sync_status.argtypes = [vp]
        L.fa_sync_status.restype = st
        L.fa_test_set_stall.argtypes = [i]
        L.fa_test_set_stall.restype = st
        L.fa_test_map_encodes.argtypes = []
        L.fa_test_map_encodes.restype = ll
        L.fa_last_failure.argtypes = [ctypes.POINTER(ctypes.c_int)]
        L.fa_last_failure.restype = st
        L.fa_status_string.argtypes = [st]
        L.fa_status_string.restype = ctypes.c_char_p
        ip = ctypes.POINTER(ctypes.c_int)
        L.fa_sched_enumerate.argtypes = [i, i, i, i, i, ll, ip, ip, ip, ll]
        L.fa_sched_enumerate.restype = ll
        _lib = L
        return L


def fa_status_string(status: int) -> str:
    return lib().fa_status_string(int(status)).decode()


def _check(call: str, status: int) -> None:
    if status != FA_OK:
        raise FAError(call, status, fa_status_string(status))


def fa_fwd(q: int, k: int, v: int, o: int, lse: int, B: int, H: int, N: int, d: int, scale: float,
           causal: int, stream: int) -> int:
    """Raw C call; pointers and stream are integers.  Returns the status."""
    return lib().fa_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, stream)


def fa_fwd_varlen(q: int, k: int, v: int, o: int, lse: int, seqlens_q: int, seqlens_k: int, B: int, H: int,
                  Nq: int, Nk: int, d: int, scale: float, causal: int, stream: int) -> int:
    return lib().fa_fwd_varlen(q, k, v, o, lse, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal, stream)


def fa_fwd_ex(q: int, k: int, v: int, o: int, o_dtype: int, lse: int, seqlens_q: int, seqlens_k: int, B: int,
              H: int, Nq: int, Nk: int, d: int, scale: float, causal: int, stream: int) -> int:
    return lib().fa_fwd_ex(q, k, v, o, o_dtype, lse, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal, stream)


def fa_fwd_bias(q: int, k: int, v: int, o: int, o_dtype: int, lse: int, bias: int, bias_stride_b: int,
                bias_stride_h: int, bias_stride_q: int, seqlens_q: int, seqlens_k: int, B: int, H: int, Nq: int,
                Nk: int, d: int, scale: float, causal: int, stream: int) -> int:
    return lib().fa_fwd_bias(q, k, v, o, o_dtype, lse, bias, bias_stride_b, bias_stride_h, bias_stride_q, seqlens_q,
                             seqlens_k, B, H, Nq, Nk, d, scale, causal, stream)


def fa_bwd_ex(q: int, k: int, v: int, o: int, o_dtype: int, lse: int, do: int, dq: int, dk: int, dv: int,
              workspace: int, seqlens_q: int, seqlens_k: int, B: int, H: int, Nq: int, Nk: int, d: int, scale: float,
              causal: int, stream: int) -> int:
    return lib().fa_bwd_ex(q, k, v, o, o_dtype, lse, do, dq, dk, dv, workspace, seqlens_q, seqlens_k, B, H, Nq, Nk,
                           d, scale, causal, stream)


def fa_bwd_bias(q: int, k: int, v: int, o: int, o_dtype: int, lse: int, do: int, bias: int, bias_stride_b: int,
                bias_stride_h: int, bias_stride_q: int, dq: int, dk: int, dv: int, workspace: int, seqlens_q: int,
                seqlens_k: int, B: int, H: int, Nq: int, Nk: int, d: int, scale: float, causal: int,
                stream: int) -> int:
    return lib().fa_bwd_bias(q, k, v, o, o_dtype, lse, do, bias, bias_stride_b, bias_stride_h, bias_stride_q, dq, dk,
                             dv, workspace, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal, stream)


def fa_fwd_fp8(q8: int, k8: int, vt8: int, o: int, lse: int, B: int, H: int, N: int, d: int, scale: float,
               causal: int, stream: int) -> int:
    return lib().fa_fwd_fp8(q8, k8, vt8, o, lse, B, H, N, d, scale, causal, stream)


def fa_fwd_splitkv(q: int, k: int, v: int, o: int, lse: int, workspace: int, B: int, H: int, N: int, d: int,
                   scale: float, causal: int, stream: int) -> int:
    return lib().fa_fwd_splitkv(q, k, v, o, lse, workspace, B, H, N, d, scale, causal, stream)


def fa_fwd_splitkv_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib().fa_fwd_splitkv_workspace_bytes(B, H, N, d))


def fa_fwd_decode(q: int, k: int, v: int, o: int, lse: int, seqlens_q: int, seqlens_k: int, workspace: int, B: int,
                  H: int, Nq: int, Nk: int, d: int, scale: float, causal: int, stream: int) -> int:
    return lib().fa_fwd_decode(q, k, v, o, lse, seqlens_q, seqlens_k, workspace, B, H, Nq, Nk, d, scale, causal,
                               stream)


def fa_fwd_decode_workspace_bytes(B: int, H: int, Nq: int, Nk: int, d: int) -> int:
    return lib().fa_fwd_decode_workspace_bytes(B, H, Nq, Nk, d)


def fa_bwd(q: int, k: int, v: int, o: int, lse: int, dO: int, dq: int, dk: int, dv: int, workspace: int,
           B: int, H: int, N: int, d: int, scale: float, causal: int, stream: int) -> int:
    return lib().fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, workspace, B, H, N, d, scale, causal, stream)


def fa_bwd_varlen(q: int, k: int, v: int, o: int, lse: int, do: int, dq: int, dk: int, dv: int, workspace: int,
                  seqlens_q: int, seqlens_k: int, B: int, H: int, Nq: int, Nk: int, d: int, scale: float,
                  causal: int, stream: int) -> int:
    return lib().fa_bwd_varlen(q, k, v, o, lse, do, dq, dk, dv, workspace, seqlens_q, seqlens_k, B, H, Nq, Nk, d,
                               scale, causal, stream)


def fa_bwd_single_pass(q: int, k: int, v: int, lse: int, do: int, bias: int, bias_stride_b: int, bias_stride_h: int,
                       bias_stride_q: int, dq: int, dk: int, dv: int, workspace: int, seqlens_q: int, seqlens_k: int,
                       B: int, H: int, Nq: int, Nk: int, d: int, scale: float, causal: int, stream: int) -> int:
    return lib().fa_bwd_single_pass(q, k, v, lse, do, bias, bias_stride_b, bias_stride_h, bias_stride_q, dq, dk, dv,
                                    workspace, seqlens_q, seqlens_k, B, H, Nq, Nk, d, scale, causal, stream)


def fa_bwd_stage(stage: int, q: int, k: int, v: int, o: int, lse: int, dO: int, dq: int, dk: int, dv: int,
                 workspace: int, B: int, H: int, N: int, d: int, scale: float, causal: int, stream: int) -> int:
    """Raw C call of one backward stage (two-pass: 0 dQ and the row term,
    1 dK/dV; single-pass: 2 the row term and dQ = 0, 3 dK/dV/dQ)."""
    return lib().fa_bwd_stage(stage, q, k, v, o, lse, dO, dq, dk, dv, workspace, B, H, N, d, scale, causal, stream)


def fa_bwd_noalloc(q: int, k: int, v: int, o: int, lse: int, dO: int, dq: int, dk: int, dv: int,
                   B: int, H: int, N: int, d: int, scale: float, causal: int, stream: int) -> int:
    """Raw C call of the allocation-free backward (scratch held inside the
    library, at most FA_NOALLOC_MAX_ROWS = B*H*N rows).  Returns the status."""
    return lib().fa_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, stream)


FA_NOALLOC_MAX_ROWS = 1 << 20


def fa_bwd_workspace_bytes(B: int, H: int, N: int) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, H, N))


def fa_rope(x: int, x_dtype: int, x_strides: tuple, y: int, y_dtype: int, y_strides: tuple, positions: int,
            positions_stride_b: int, turns: int, rot_dim: int, layout: int, amplitude: float, inverse: int, B: int,
            H: int, N: int, d: int, stream: int) -> int:
    """Raw C call; strides are (b, h, n) triples in elements."""
    return lib().fa_rope(x, x_dtype, *x_strides, y, y_dtype, *y_strides, positions, positions_stride_b, turns, rot_dim,
                         layout, amplitude, inverse, B, H, N, d, stream)


def fa_kv_append(k: int, k_strides: tuple, v: int, v_strides: tuple, q: int, q_strides: tuple, q_out: int,
                 k_pages: int, v_pages: int, num_pages: int, page_size: int, block_table: int, table_stride: int,
                 max_pages: int, seqlens_q: int, seqlens_k: int, positions: int, positions_stride_b: int, turns: int,
                 rot_dim: int, layout: int, amplitude: float, B: int, Hq: int, Hkv: int, N: int, d: int,
                 stream: int) -> int:
    """Raw C call; strides are (b, h, n) triples in elements."""
    return lib().fa_kv_append(k, *k_strides, v, *v_strides, q, *q_strides, q_out, k_pages, v_pages, num_pages,
                              page_size, block_table, table_stride, max_pages, seqlens_q, seqlens_k, positions,
                              positions_stride_b, turns, rot_dim, layout, amplitude, B, Hq, Hkv, N, d, stream)


def fa_fwd_paged(q: int, k_pages: int, v_pages: int, num_pages: int, page_size: int, block_table: int,
                 table_stride: int, max_pages: int, o: int, o_dtype: int, lse: int, seqlens_q: int, seqlens_k: int,
                 workspace: int, B: int, Hq: int, Hkv: int, Nq: int, d: int, scale: float, causal: int,
                 stream: int) -> int:
    return lib().fa_fwd_paged(q, k_pages, v_pages, num_pages, page_size, block_table, table_stride, max_pages, o,
                              o_dtype, lse, seqlens_q, seqlens_k, workspace, B, Hq, Hkv, Nq, d, scale, causal, stream)


def fa_fwd_paged_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, d: int) -> int:
    return lib().fa_fwd_paged_workspace_bytes(B, Hq, Hkv, Nq, d)


def fa_fwd_shared_prefix(q: int, k_pages: int, v_pages: int, num_pages: int, page_size: int, prefix_table: int,
                         prefix_len: int, block_table: int, table_stride: int, max_pages: int, o: int, o_dtype: int,
                         lse: int, seqlens_q: int, seqlens_k: int, workspace: int, B: int, Hq: int, Hkv: int, Nq: int,
                         d: int, scale: float, causal: int, stream: int) -> int:
    return lib().fa_fwd_shared_prefix(q, k_pages, v_pages, num_pages, page_size, prefix_table, prefix_len, block_table,
                                      table_stride, max_pages, o, o_dtype, lse, seqlens_q, seqlens_k, workspace, B, Hq,
                                      Hkv, Nq, d, scale, causal, stream)


def fa_fwd_shared_prefix_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, d: int) -> int:
    return lib().fa_fwd_shared_prefix_workspace_bytes(B, Hq, Hkv, Nq, d)


def fa_sync_status(stream: int) -> int:
    return lib().fa_sync_status(stream)


def fa_test_set_stall(unit: int) -> int:
    """Testing hook: from the next call on, CTA 0 leaves one tile of its
    unit-th work unit unloaded (-1: off).  Returns the status."""
    return lib().fa_test_set_stall(int(unit))


def fa_test_map_encodes() -> int:
    """Testing hook: tensor maps encoded by the driver since the library was loaded."""
    return int(lib().fa_test_map_encodes())


def fa_last_failure() -> list:
    out = (ctypes.c_int * 4)()
    _check("fa_last_failure", lib().fa_last_failure(out))
    return list(out)


def fa_sched_enumerate(heads: int, N: int, d: int, causal: int, grid: int, l2_budget_bytes: int = 0):
    """Host-only: list of (cta, head, pair) the kernels' scheduler deals."""
    L = lib()
    total = L.fa_sched_enumerate(heads, N, d, causal, grid, l2_budget_bytes, None, None, None, 0)
    if total < 0:
        raise ValueError("invalid scheduler arguments")
    arr = [(ctypes.c_int * max(total, 1))() for _ in range(3)]
    L.fa_sched_enumerate(heads, N, d, causal, grid, l2_budget_bytes, arr[0], arr[1], arr[2], total)
    return [(arr[0][i], arr[1][i], arr[2][i]) for i in range(total)]


# ----------------------------------------------------------------- torch side
# PyTorch supplies device memory and the current stream; nothing else.

def _stream_handle(device) -> int:
    import torch
    return int(torch.cuda.current_stream(device).cuda_stream)


def _check_inputs(*ts):
    import torch
    ref = ts[0]
    for t in ts:
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.shape != ref.shape \
                or t.device != ref.device or t.dim() != 4:
            raise ValueError("q, k, v (and dO) must be contiguous bf16 CUDA tensors of one shape [B, H, N, d]")


def forward(q, k, v, causal: bool = False, scale: float | None = None, out=None):
    """O, LSE = attention(q, k, v) through fa_fwd on the current stream.

    q, k, v: bf16 CUDA tensors [B, H, N, d].  Returns fp32 O [B, H, N, d]
    and fp32 LSE [B, H, N].  ``out`` may supply preallocated (O, LSE).
    """
    import torch
    _check_inputs(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    if out is None:
        o = torch.empty((B, H, N, d), dtype=torch.float32, device=q.device)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
    _check("fa_fwd", fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                            B, H, N, d, scale, int(bool(causal)), _stream_handle(q.device)))
    return o, lse


def forward_splitkv(q, k, v, causal: bool = False, scale: float | None = None, workspace=None, out=None):
    """O, LSE through fa_fwd_splitkv (each query tile's keys split over
    several CTAs; for batches with few query tiles).  Arguments as forward;
    ``workspace`` an optional fp32 CUDA tensor of
    fa_fwd_splitkv_workspace_bytes(B, H, N, d) bytes."""
    import torch
    _check_inputs(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    if out is None:
        o = torch.empty((B, H, N, d), dtype=torch.float32, device=q.device)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
    _check("fa_fwd_splitkv", fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                            workspace.data_ptr() if workspace is not None else 0, B, H, N, d, scale,
                                            int(bool(causal)), _stream_handle(q.device)))
    return o, lse


def forward_varlen(q, k, v, seqlens_q=None, seqlens_k=None, causal: bool = False, scale: float | None = None,
                   out=None, o_dtype=None):
    """O, LSE through fa_fwd_varlen: q [B,H,Nq,d], k and v [B,H,Nk,d] (bf16,
    CUDA); seqlens_q / seqlens_k optional int32 CUDA tensors of B valid
    lengths.  Causal alignment is bottom-right (see include/fa.h).  With
    o_dtype=torch.bfloat16 O is written as bf16 through fa_fwd_ex."""
    import torch
    for t in (q, k, v):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q, k, v must be contiguous 4-D bf16 CUDA tensors")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Nk, d] with the batch, heads and d of q")
    for t in (seqlens_q, seqlens_k):
        if t is not None and (not t.is_cuda or t.dtype != torch.int32 or t.numel() != B or not t.is_contiguous()):
            raise ValueError("seqlens must be contiguous int32 CUDA tensors of B entries")
    if scale is None:
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    if out is None:
        o = torch.empty((B, H, Nq, d), dtype=o_dtype or torch.float32, device=q.device)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
    sq = seqlens_q.data_ptr() if seqlens_q is not None else 0
    sk = seqlens_k.data_ptr() if seqlens_k is not None else 0
    if o.dtype == torch.float32:
        _check("fa_fwd_varlen", fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                              sq, sk, B, H, Nq, Nk, d, scale, int(bool(causal)),
                                              _stream_handle(q.device)))
    elif o.dtype == torch.bfloat16:
        _check("fa_fwd_ex", fa_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), FA_DTYPE_BF16,
                                      lse.data_ptr(), sq, sk, B, H, Nq, Nk, d, scale, int(bool(causal)),
                                      _stream_handle(q.device)))
    else:
        raise ValueError("O must be float32 or bfloat16")
    return o, lse


def _bias_strides(bias, B, H, Nq, Nk):
    """Element strides (b, h, query) of a bf16 CUDA mask broadcastable to
    [B, H, Nq, Nk] with contiguous keys."""
    import torch
    if not bias.is_cuda or bias.dtype != torch.bfloat16:
        raise ValueError("bias must be a bf16 CUDA tensor")
    bias = bias.expand(B, H, Nq, Nk)
    if bias.stride(3) != 1:
        raise ValueError("the bias's key dimension must be contiguous")
    return bias.stride(0), bias.stride(1), bias.stride(2)


def forward_bias(q, k, v, bias, seqlens_q=None, seqlens_k=None, causal: bool = False, scale: float | None = None,
                 o_dtype=None, out=None):
    """O, LSE through fa_fwd_bias: softmax(scale * q k^T + bias) v.  ``bias``
    is a bf16 CUDA tensor broadcastable to [B, H, Nq, Nk] (e.g. made with
    expand()) whose last dimension is contiguous; other arguments as
    forward_varlen."""
    import torch
    for t in (q, k, v):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q, k, v must be contiguous 4-D bf16 CUDA tensors")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Nk, d] with the batch, heads and d of q")
    sb, sh, sq = _bias_strides(bias, B, H, Nq, Nk)
    for t in (seqlens_q, seqlens_k):
        if t is not None and (not t.is_cuda or t.dtype != torch.int32 or t.numel() != B or not t.is_contiguous()):
            raise ValueError("seqlens must be contiguous int32 CUDA tensors of B entries")
    if scale is None:
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    if out is None:
        o = torch.empty((B, H, Nq, d), dtype=o_dtype or torch.float32, device=q.device)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
    if o.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("O must be float32 or bfloat16")
    _check("fa_fwd_bias", fa_fwd_bias(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                      FA_DTYPE_BF16 if o.dtype == torch.bfloat16 else FA_DTYPE_F32, lse.data_ptr(),
                                      bias.data_ptr(), sb, sh, sq,
                                      seqlens_q.data_ptr() if seqlens_q is not None else 0,
                                      seqlens_k.data_ptr() if seqlens_k is not None else 0,
                                      B, H, Nq, Nk, d, scale, int(bool(causal)), _stream_handle(q.device)))
    return o, lse


def forward_fp8(q8, k8, vt8, causal: bool = False, scale: float | None = None, out=None):
    """O, LSE through fa_fwd_fp8: q8, k8 [B,H,N,128] and vt8 (V transposed)
    [B,H,128,N], E4M3 CUDA tensors (torch.float8_e4m3fn, or uint8 holding
    the bit patterns), contiguous; O fp32."""
    import torch
    for t in (q8, k8, vt8):
        if not t.is_cuda or t.dtype not in (torch.uint8, torch.float8_e4m3fn) or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q8, k8, vt8 must be contiguous 4-D E4M3 (or uint8) CUDA tensors")
    B, H, N, d = q8.shape
    if k8.shape != q8.shape or vt8.shape != (B, H, d, N):
        raise ValueError("k8 must be [B, H, N, d] and vt8 [B, H, d, N]")
    if scale is None:
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    if out is None:
        o = torch.empty((B, H, N, d), dtype=torch.float32, device=q8.device)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    else:
        o, lse = out
    _check("fa_fwd_fp8", fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), vt8.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                    B, H, N, d, scale, int(bool(causal)), _stream_handle(q8.device)))
    return o, lse


def forward_decode(q, k, v, seqlens_q=None, seqlens_k=None, causal: bool = False, scale: float | None = None,
                   workspace=None, out=None):
    """O, LSE through fa_fwd_decode: q [B,H,Nq,d] with Nq <= FA_DECODE_MAX_Q,
    k and v [B,H,Nk,d] (bf16, CUDA); same results as forward_varlen."""
    import torch
    for t in (q, k, v):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q, k, v must be contiguous 4-D bf16 CUDA tensors")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Nk, d] with the batch, heads and d of q")
    for t in (seqlens_q, seqlens_k):
        if t is not None and (not t.is_cuda or t.dtype != torch.int32 or t.numel() != B or not t.is_contiguous()):
            raise ValueError("seqlens must be contiguous int32 CUDA tensors of B entries")
    if scale is None:
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    if out is None:
        o = torch.empty((B, H, Nq, d), dtype=torch.float32, device=q.device)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
    _check("fa_fwd_decode", fa_fwd_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                          seqlens_q.data_ptr() if seqlens_q is not None else 0,
                                          seqlens_k.data_ptr() if seqlens_k is not None else 0,
                                          workspace.data_ptr() if workspace is not None else 0,
                                          B, H, Nq, Nk, d, scale, int(bool(causal)), _stream_handle(q.device)))
    return o, lse


def backward(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None, workspace=None,
             out=None):
    """dQ, dK, dV through fa_bwd on the current stream (fp32 outputs)."""
    import torch
    _check_inputs(q, k, v, do)
    B, H, N, d = q.shape
    if scale is None:
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    if out is None:
        dq, dk, dv = (torch.empty((B, H, N, d), dtype=torch.float32, device=q.device) for _ in range(3))
    else:
        dq, dk, dv = out
    ws = workspace.data_ptr() if workspace is not None else 0
    _check("fa_bwd", fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                            do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws,
                            B, H, N, d, scale, int(bool(causal)), _stream_handle(q.device)))
    return dq, dk, dv


def backward_varlen(q, k, v, o, lse, do, seqlens_q=None, seqlens_k=None, causal: bool = False,
                    scale: float | None = None, workspace=None, out=None):
    """dQ, dK, dV through fa_bwd_ex: q, do, o [B,H,Nq,d] (o fp32 or bf16),
    lse [B,H,Nq], k and v [B,H,Nk,d]; seqlens as forward_varlen (fp32
    outputs)."""
    return _backward(q, k, v, o, lse, do, None, seqlens_q, seqlens_k, causal, scale, workspace, out)


def backward_bias(q, k, v, o, lse, do, bias, seqlens_q=None, seqlens_k=None, causal: bool = False,
                  scale: float | None = None, workspace=None, out=None):
    """dQ, dK, dV of forward_bias through fa_bwd_bias; ``bias`` exactly as
    given to forward_bias, other arguments as backward_varlen."""
    return _backward(q, k, v, o, lse, do, bias, seqlens_q, seqlens_k, causal, scale, workspace, out)


def _backward(q, k, v, o, lse, do, bias, seqlens_q, seqlens_k, causal, scale, workspace, out):
    import torch
    for t in (q, k, v, do):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q, k, v, do must be contiguous 4-D bf16 CUDA tensors")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != k.shape or do.shape != q.shape:
        raise ValueError("k, v must be [B, H, Nk, d] and do [B, H, Nq, d]")
    for t in (seqlens_q, seqlens_k):
        if t is not None and (not t.is_cuda or t.dtype != torch.int32 or t.numel() != B or not t.is_contiguous()):
            raise ValueError("seqlens must be contiguous int32 CUDA tensors of B entries")
    if scale is None:
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    if out is None:
        dq = torch.empty((B, H, Nq, d), dtype=torch.float32, device=q.device)
        dk, dv = (torch.empty((B, H, Nk, d), dtype=torch.float32, device=q.device) for _ in range(2))
    else:
        dq, dk, dv = out
    ws = workspace.data_ptr() if workspace is not None else 0
    if o.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("O must be float32 or bfloat16")
    o_dtype = FA_DTYPE_BF16 if o.dtype == torch.bfloat16 else FA_DTYPE_F32
    lq = seqlens_q.data_ptr() if seqlens_q is not None else 0
    lk = seqlens_k.data_ptr() if seqlens_k is not None else 0
    if bias is None:
        _check("fa_bwd_ex",
               fa_bwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), o_dtype, lse.data_ptr(),
                         do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws, lq, lk,
                         B, H, Nq, Nk, d, scale, int(bool(causal)), _stream_handle(q.device)))
    else:
        sb, sh, sq = _bias_strides(bias, B, H, Nq, Nk)
        _check("fa_bwd_bias",
               fa_bwd_bias(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), o_dtype, lse.data_ptr(),
                           do.data_ptr(), bias.data_ptr(), sb, sh, sq, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                           ws, lq, lk, B, H, Nq, Nk, d, scale, int(bool(causal)), _stream_handle(q.device)))
    return dq, dk, dv


def backward_single_pass(q, k, v, lse, do, bias=None, seqlens_q=None, seqlens_k=None, causal: bool = False,
                         scale: float | None = None, workspace=None, out=None):
    """dQ, dK, dV through fa_bwd_single_pass: q, do [B,H,Nq,d], lse
    [B,H,Nq], k and v [B,H,Nk,d] (bf16 CUDA); optional bias and seqlens as
    backward_bias / backward_varlen (fp32 outputs)."""
    import torch
    for t in (q, k, v, do):
        if not t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("q, k, v, do must be contiguous 4-D bf16 CUDA tensors")
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    if k.shape != (B, H, Nk, d) or v.shape != k.shape or do.shape != q.shape:
        raise ValueError("k, v must be [B, H, Nk, d] and do [B, H, Nq, d]")
    for t in (seqlens_q, seqlens_k):
        if t is not None and (not t.is_cuda or t.dtype != torch.int32 or t.numel() != B or not t.is_contiguous()):
            raise ValueError("seqlens must be contiguous int32 CUDA tensors of B entries")
    if scale is None:
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    if out is None:
        dq = torch.empty((B, H, Nq, d), dtype=torch.float32, device=q.device)
        dk, dv = (torch.empty((B, H, Nk, d), dtype=torch.float32, device=q.device) for _ in range(2))
    else:
        dq, dk, dv = out
    sb = sh = sq = 0
    if bias is not None:
        sb, sh, sq = _bias_strides(bias, B, H, Nq, Nk)
    _check("fa_bwd_single_pass",
           fa_bwd_single_pass(q.data_ptr(), k.data_ptr(), v.data_ptr(), lse.data_ptr(), do.data_ptr(),
                              bias.data_ptr() if bias is not None else 0, sb, sh, sq, dq.data_ptr(), dk.data_ptr(),
                              dv.data_ptr(), workspace.data_ptr() if workspace is not None else 0,
                              seqlens_q.data_ptr() if seqlens_q is not None else 0,
                              seqlens_k.data_ptr() if seqlens_k is not None else 0,
                              B, H, Nq, Nk, d, scale, int(bool(causal)), _stream_handle(q.device)))
    return dq, dk, dv


def backward_stage(stage: int, q, k, v, o, lse, do, dq, dk, dv, workspace, causal: bool = False,
                   scale: float | None = None):
    """One backward stage through fa_bwd_stage on the current stream."""
    import torch
    _check_inputs(q, k, v, do)
    B, H, N, d = q.shape
    if scale is None:
        scale = float(torch.tensor(d ** -0.5, dtype=torch.float32))
    _check(f"fa_bwd_stage({stage})",
           fa_bwd_stage(stage, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr() if o is not None else 0,
                        lse.data_ptr(),
                        do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(),
                        B, H, N, d, scale, int(bool(causal)), _stream_handle(q.device)))


# ------------------------------------------- rotary positions, paged cache

_ROPE_LAYOUTS = {"half": FA_ROPE_HALF, "interleaved": FA_ROPE_INTERLEAVED}
_ROPE_SCALINGS = {None: FA_ROPE_SCALE_NONE, "linear": FA_ROPE_SCALE_LINEAR, "ntk": FA_ROPE_SCALE_NTK,
                  "parts": FA_ROPE_SCALE_PARTS}


# A decoding step is a few microseconds of kernels, so these calls keep their
# checks to a few attribute reads, and name what is wrong only when something is.

def _call_on(index: int, call, *args) -> int:
    """The C call with the tensors' device current (its kernels launch there)
    on that device's current PyTorch stream."""
    import torch
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        return call(*args, stream)
    with torch.cuda.device(index):
        return call(*args, stream)


def rope_turns(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               original_len: float = 1.0, low: float = 1.0, high: float = 32.0, device=None):
    """The frequency table of the rotary calls through fa_rope_turns: int64
    [rot_dim / 2], in units of 2^-64 turns per position, on ``device``.
    ``scaling``: None, "linear", "ntk" or "parts" (see include/fa.h)."""
    import torch
    if scaling not in _ROPE_SCALINGS:
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'parts'")
    out = (ctypes.c_longlong * max(int(rot_dim) // 2, 1))()
    _check("fa_rope_turns", lib().fa_rope_turns(out, rot_dim, base, _ROPE_SCALINGS[scaling], factor, original_len, low,
                                                high))
    return torch.tensor(list(out), dtype=torch.int64, device=device)


def _rope_args(turns, layout, positions, B, N, index):
    """(positions, positions stride, turns, rot_dim, layout) of a rotary call."""
    import torch
    lay = _ROPE_LAYOUTS.get(layout)
    if lay is None:
        raise ValueError("layout must be 'half' or 'interleaved'")
    if turns.dtype != torch.int64 or turns.dim() != 1 or not turns.is_contiguous() or turns.get_device() != index:
        raise ValueError("turns must be a contiguous int64 tensor of rot_dim / 2 entries on the inputs' device")
    if positions is None:
        return 0, 0, turns.data_ptr(), 2 * turns.numel(), lay
    if positions.dtype != torch.int32 or positions.get_device() != index or (
            positions.shape != (B, N) and positions.shape != (N,)) or (N > 1 and positions.stride(-1) != 1):
        raise ValueError("positions must be int32 [N] or [B, N] on the inputs' device with contiguous rows")
    return (positions.data_ptr(), positions.stride(0) if positions.dim() == 2 else 0, turns.data_ptr(),
            2 * turns.numel(), lay)


def _rope(x, turns, positions, layout, amplitude, inverse, out, out_dtype):
    import torch
    if x.dim() != 4 or not x.is_cuda:
        raise ValueError("x must be a bf16 or fp32 CUDA tensor [B, H, N, d] with contiguous d")
    B, H, N, d = x.shape
    xb, xh, xn, one = x.stride()
    index, dtype = x.get_device(), x.dtype
    if one != 1 or (dtype != torch.bfloat16 and dtype != torch.float32):
        raise ValueError("x must be a bf16 or fp32 CUDA tensor [B, H, N, d] with contiguous d")
    pos, pos_stride, t, rot_dim, lay = _rope_args(turns, layout, positions, B, N, index)
    if out is None:
        if out_dtype is None:
            out_dtype = dtype
        elif out_dtype != torch.bfloat16 and out_dtype != torch.float32:
            raise ValueError("out_dtype must be bfloat16 or float32")
        out = torch.empty((B, H, N, d), dtype=out_dtype, device=x.device)
        yb, yh, yn = H * N * d, N * d, d
    else:
        if out_dtype is None:
            out_dtype = out.dtype
        if (out.shape != x.shape or out.get_device() != index or out.dtype != out_dtype
                or (out_dtype != torch.bfloat16 and out_dtype != torch.float32) or out.stride(3) != 1):
            raise ValueError("out must be a bf16 or fp32 tensor of x's shape and device with contiguous d")
        yb, yh, yn, _ = out.stride()
    st = _call_on(index, (_lib or lib()).fa_rope, x.data_ptr(), dtype == torch.bfloat16, xb, xh, xn, out.data_ptr(),
                  out_dtype == torch.bfloat16, yb, yh, yn, pos, pos_stride, t, rot_dim, lay, amplitude, inverse, B, H,
                  N, d)
    if st:
        _check("fa_rope", st)
    return out


def rope_forward(x, turns, positions=None, layout: str = "half", amplitude: float = 1.0, out=None, out_dtype=None):
    """x [B, H, N, d] (bf16 or fp32 CUDA, contiguous d, any other strides)
    with its first 2 * len(turns) values rotated by their positions, through
    fa_rope.  ``turns``: rope_turns(...) on x's device; ``positions``: int32
    [N] or [B, N] (default 0 .. N - 1); ``layout``: "half" or "interleaved".
    ``out`` may be x itself.  Returns ``out`` (contiguous if it is made here)."""
    return _rope(x, turns, positions, layout, amplitude, 0, out, out_dtype)


def rope_backward(dy, turns, positions=None, layout: str = "half", amplitude: float = 1.0, out=None, out_dtype=None):
    """The gradient with respect to x of rope_forward with the same arguments,
    given dy = dL/dy (bf16 or fp32)."""
    return _rope(dy, turns, positions, layout, amplitude, 1, out, out_dtype)


def _page_args(k_pages, v_pages, block_table, B, d, index):
    """(k_pages, v_pages, num_pages, page_size) and (block_table, its stride,
    max_pages) of the C calls, and Hkv."""
    import torch
    shape = k_pages.shape
    if (len(shape) != 4 or shape[3] != d or v_pages.shape != shape or k_pages.dtype != torch.bfloat16
            or v_pages.dtype != torch.bfloat16 or not k_pages.is_contiguous() or not v_pages.is_contiguous()
            or k_pages.get_device() != index or v_pages.get_device() != index):
        raise ValueError("k_pages and v_pages must be contiguous bf16 [pages, Hkv, page_size, d] on the inputs' device")
    if (block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.shape[0] != B
            or block_table.get_device() != index or (block_table.shape[1] != 1 and block_table.stride(1) != 1)):
        raise ValueError("block_table must be int32 [B, max_pages] on the inputs' device with contiguous rows")
    return ((k_pages.data_ptr(), v_pages.data_ptr(), shape[0], shape[2]),
            (block_table.data_ptr(), block_table.stride(0), block_table.shape[1]), shape[1])


def _lens(t, B, index) -> int:
    import torch
    if t is None:
        return 0
    if t.dtype != torch.int32 or t.numel() != B or not t.is_contiguous() or t.get_device() != index:
        raise ValueError("seqlens must be contiguous int32 tensors of B entries on the inputs' device")
    return t.data_ptr()


def kv_append(k, v, k_pages, v_pages, block_table, seqlens_k, seqlens_q=None, turns=None, layout: str = "half",
              amplitude: float = 1.0, positions=None, q=None, q_out=None):
    """Appends k and v [B, Hkv, N, d] (bf16 CUDA, contiguous d, any other
    strides) to the paged cache through fa_kv_append, the keys rotated by
    their positions if ``turns`` is given; with ``q`` [B, Hq, N, d] also
    rotates the queries, into ``q_out`` (contiguous; made here by default, its
    padding rows then unset).  ``seqlens_k``: int32 [B], each sequence's keys
    with the new tokens; ``seqlens_q``: int32 [B], its new tokens (default N).
    Tokens past the end of their row of ``block_table`` are not stored, which
    sync_status reports.  Returns q_out, or None without q."""
    import torch
    if k.dim() != 4 or not k.is_cuda:
        raise ValueError("k must be a bf16 CUDA tensor [B, Hkv, N, d] with contiguous d")
    B, Hkv, N, d = k.shape
    index = k.get_device()
    kb, kh, kn, k1 = k.stride()
    if v.shape != k.shape:
        raise ValueError("v must have k's shape")
    vb, vh, vn, v1 = v.stride()
    if (k1 != 1 or v1 != 1 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16 or v.get_device() != index):
        raise ValueError("k and v must be bf16 CUDA tensors [B, Hkv, N, d] of one device with contiguous d")
    pages, table, page_heads = _page_args(k_pages, v_pages, block_table, B, d, index)
    if page_heads != Hkv:
        raise ValueError("the pages must have k's heads")
    if seqlens_k is None:
        raise ValueError("seqlens_k is needed")
    if turns is not None:
        rope = _rope_args(turns, layout, positions, B, N, index)
    elif positions is None:
        rope = (0, 0, 0, 0, 0)
    else:
        raise ValueError("positions without turns")
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        qp = op = Hq = qb = qh = qn = 0
    else:
        if q.dim() != 4 or q.get_device() != index or q.dtype != torch.bfloat16:
            raise ValueError("q must be a bf16 tensor [B, Hq, N, d] with the batch, length, d and device of k")
        Hq = q.shape[1]
        qb, qh, qn, q1 = q.stride()
        if q.shape != (B, Hq, N, d) or q1 != 1:
            raise ValueError("q must be a bf16 tensor [B, Hq, N, d] with the batch, length, d and device of k")
        if q_out is None:
            q_out = torch.empty((B, Hq, N, d), dtype=torch.bfloat16, device=k.device)
        elif (q_out.shape != q.shape or q_out.dtype != torch.bfloat16 or not q_out.is_contiguous()
              or q_out.get_device() != index):
            raise ValueError("q_out must be contiguous bf16 of q's shape and device")
        qp, op = q.data_ptr(), q_out.data_ptr()
    st = _call_on(index, (_lib or lib()).fa_kv_append, k.data_ptr(), kb, kh, kn, v.data_ptr(), vb, vh, vn, qp, qb, qh,
                  qn, op, *pages, *table, _lens(seqlens_q, B, index), _lens(seqlens_k, B, index), *rope, amplitude, B,
                  Hq, Hkv, N, d)
    if st:
        _check("fa_kv_append", st)
    return q_out


def _paged(shared, q, k_pages, v_pages, prefix, block_table, seqlens_k, seqlens_q, causal, scale, o_dtype, workspace,
           out):
    import torch
    if q.dtype != torch.bfloat16 or not q.is_cuda or q.dim() != 4 or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 CUDA tensor [B, Hq, Nq, d]")
    B, Hq, Nq, d = q.shape
    index = q.get_device()
    pages, table, Hkv = _page_args(k_pages, v_pages, block_table, B, d, index)
    if out is None:
        if o_dtype is None:
            o_dtype = torch.float32
        if o_dtype == torch.bfloat16:
            o = torch.empty_like(q)
        elif o_dtype == torch.float32:
            o = torch.empty_like(q, dtype=o_dtype)
        else:
            raise ValueError("O must be float32 or bfloat16")
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    else:
        o, lse = out
        o_dtype = o.dtype
        if o_dtype != torch.float32 and o_dtype != torch.bfloat16:
            raise ValueError("O must be float32 or bfloat16")
        if (o.shape != q.shape or not o.is_contiguous() or o.get_device() != index or lse.shape != (B, Hq, Nq)
                or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.get_device() != index):
            raise ValueError("out must be contiguous O [B, Hq, Nq, d] and fp32 LSE [B, Hq, Nq] on q's device")
    L = _lib or lib()
    if workspace is None:
        # the library's own, unless a graph is being captured: the graph then
        # keeps a tensor of PyTorch's graph pool
        ws = 0
        if torch.cuda.is_current_stream_capturing():
            workspace = torch.empty(_paged_workspace(L, shared, B, Hq, Hkv, Nq, d), dtype=torch.float32,
                                    device=q.device)
            ws = workspace.data_ptr()
    else:
        if (workspace.dtype != torch.float32 or not workspace.is_contiguous() or workspace.get_device() != index
                or workspace.numel() < _paged_workspace(L, shared, B, Hq, Hkv, Nq, d)):
            raise ValueError("workspace must be fp32 on q's device, of the call's workspace_bytes(...) bytes")
        ws = workspace.data_ptr()
    st = _call_on(index, L.fa_fwd_shared_prefix if shared else L.fa_fwd_paged, q.data_ptr(), *pages, *prefix, *table,
                  o.data_ptr(), o_dtype == torch.bfloat16, lse.data_ptr(), _lens(seqlens_q, B, index),
                  _lens(seqlens_k, B, index), ws, B, Hq, Hkv, Nq, d, d ** -0.5 if scale is None else scale,
                  bool(causal))
    if st:
        _check("fa_fwd_shared_prefix" if shared else "fa_fwd_paged", st)
    return o, lse


def _paged_workspace(L, shared, B, Hq, Hkv, Nq, d) -> int:
    size = L.fa_fwd_shared_prefix_workspace_bytes if shared else L.fa_fwd_paged_workspace_bytes
    return size(B, Hq, Hkv, Nq, d) // 4


def forward_paged(q, k_pages, v_pages, block_table, seqlens_k=None, seqlens_q=None, causal: bool = True,
                  scale: float | None = None, o_dtype=None, workspace=None, out=None):
    """O, LSE through fa_fwd_paged: q [B, Hq, Nq, d] (bf16 CUDA, contiguous)
    against the keys and values that ``block_table`` int32 [B, max_pages]
    names in k_pages, v_pages [pages, Hkv, page_size, d]; Hq a multiple of
    Hkv.  ``seqlens_k``, ``seqlens_q``: int32 [B] as kv_append.  ``workspace``:
    an fp32 tensor of fa_fwd_paged_workspace_bytes(...) bytes; by default a
    stream-ordered one of the library's."""
    return _paged(False, q, k_pages, v_pages, (), block_table, seqlens_k, seqlens_q, causal, scale, o_dtype,
                  workspace, out)


def forward_shared_prefix(q, k_pages, v_pages, prefix_table, prefix_len: int, block_table, seqlens_k=None,
                          seqlens_q=None, causal: bool = True, scale: float | None = None, o_dtype=None,
                          workspace=None, out=None):
    """forward_paged for a batch whose sequences share their first
    ``prefix_len`` keys (a multiple of the page size), in the pages that
    ``prefix_table`` int32 [prefix_len / page_size] names: that part is
    computed once for all, through fa_fwd_shared_prefix."""
    import torch
    if (prefix_table.dtype != torch.int32 or prefix_table.dim() != 1 or not prefix_table.is_contiguous()
            or prefix_table.get_device() != q.get_device() or prefix_len < 1 or k_pages.dim() != 4
            or prefix_table.numel() * k_pages.shape[2] < prefix_len):
        raise ValueError("prefix_table must be contiguous int32 on q's device with an entry for every page of the "
                         "prefix")
    return _paged(True, q, k_pages, v_pages, (prefix_table.data_ptr(), int(prefix_len)), block_table,
                  seqlens_k, seqlens_q, causal, scale, o_dtype, workspace, out)


def sync_status(device=None) -> None:
    """Synchronise the current stream (of ``device``, by default the current
    one) and raise if a kernel reported a failure there."""
    import torch
    with torch.cuda.device(device):  # the status word is the current device's
        status = fa_sync_status(_stream_handle(device))
    if status != FA_OK:
        detail = fa_last_failure() if status in (FA_ERR_TIMEOUT, FA_ERR_BAD_PAGE) else None
        raise FAError("fa_sync_status", status, fa_status_string(status) + (f" {detail}" if detail else ""))
