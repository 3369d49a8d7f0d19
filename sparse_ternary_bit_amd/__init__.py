"""Python binding of libstq, the STQ1_0 sparse-ternary matmul library for MI355X.

Thin ctypes marshalling over the C ABI in ``include/stq.h``: every function
takes torch tensors that already live on the GPU, passes their device
pointers and the current HIP stream, and checks the returned status.  All
computation happens in the HIP kernels of ``libstq.so``; there is no
fallback.  If the library is not built, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = [
    "QK", "BLOCK_BYTES", "ENC_WLS", "ENC_AMAX", "StqError", "lib", "lib_path",
    "row_bytes", "quantize_rows", "dequantize_rows", "gemv", "gemv_noalloc", "gemv_plan", "grouped_gemm",
    "moe_ffn_decode",
    "moe_ffn_workspace", "grouped_swiglu", "grouped_swiglu_workspace", "grouped_swiglu_plan",
    "grouped_swiglu_backward", "grouped_swiglu_backward_workspace", "grouped_swiglu_backward_plan",
    "q8_quantize_rows", "q8_matmul", "token_logprobs",
    "token_logprobs_workspace", "token_logprobs_backward", "layer_errors", "layer_errors_workspace", "q2_roundtrip", "greedy_allocation",
    "stream_read_probe", "mfma_loop_probe", "lds_read_probe", "MFMA_PROBE_FLOP_PER_ROUND",
    "LDS_PROBE_READS_PER_ROUND",
]

QK = 256
BLOCK_BYTES = 42
ENC_WLS, ENC_AMAX = 0, 1
X_F32, X_BF16 = 0, 1
# work of one round of the measurement probes (include/stq.h)
MFMA_PROBE_FLOP_PER_ROUND = 2147483648.0
LDS_PROBE_READS_PER_ROUND = 131072

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libstq.so")
_lib = None

_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_vp = ctypes.c_void_p


class StqError(RuntimeError):
    """A libstq entry point returned a status other than STQ_OK."""

    def __init__(self, func: str, status: int, detail: str):
        self.status = status
        super().__init__(f"{func} failed with status {status}: {detail}")


def lib_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """Load libstq.so (built in-tree by ``python -m sparse_ternary_bit_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built: run `python -m sparse_ternary_bit_amd.build` first")
    L = ctypes.CDLL(_LIB_PATH)
    L.stq_row_bytes.argtypes = [_c_i64]
    L.stq_row_bytes.restype = _c_i64
    L.stq_status_string.argtypes = [_c_int]
    L.stq_status_string.restype = ctypes.c_char_p
    L.stq_last_error.argtypes = []
    L.stq_last_error.restype = ctypes.c_char_p
    L.stq_quantize_rows.argtypes = [_c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_int, _c_vp, _c_vp]
    L.stq_quantize_rows.restype = _c_int
    L.stq_dequantize_rows.argtypes = [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp]
    L.stq_dequantize_rows.restype = _c_int
    L.stq_gemv.argtypes = [_c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_i64,
                           _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp]
    L.stq_gemv.restype = _c_int
    L.stq_gemv_noalloc.argtypes = [_c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_i64,
                                   _c_vp, _c_vp, _c_i64, _c_vp, _c_vp]
    L.stq_gemv_noalloc.restype = _c_int
    L.stq_gemv_plan.argtypes = [_c_i64, _c_i64, _c_i64, _c_i64, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32),
                                ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(_c_i64)]
    L.stq_gemv_plan.restype = _c_int
    L.stq_grouped_gemm.argtypes = [_c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp]
    L.stq_grouped_gemm.restype = _c_int
    L.stq_moe_ffn_decode.argtypes = [_c_vp, _c_i64, _c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64,
                                     _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp]
    L.stq_moe_ffn_decode.restype = _c_int
    L.stq_moe_ffn_workspace.argtypes = [_c_i64, _c_i64, _c_i64, _c_i64, _c_i64, ctypes.c_int32,
                                        ctypes.POINTER(_c_i64)]
    L.stq_moe_ffn_workspace.restype = _c_int
    L.stq_layer_errors.argtypes = [_c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64,
                                   _c_vp]
    L.stq_layer_errors.restype = _c_int
    L.stq_layer_errors_workspace.argtypes = [_c_i64, _c_i64, _c_i64, ctypes.POINTER(_c_i64)]
    L.stq_layer_errors_workspace.restype = _c_int
    L.stq_q2_roundtrip.argtypes = [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp]
    L.stq_q2_roundtrip.restype = _c_int
    L.stq_greedy_allocation.argtypes = [_c_vp, _c_vp, _c_i64, ctypes.c_double, _c_vp]
    L.stq_greedy_allocation.restype = _c_int
    L.stq_grouped_swiglu.argtypes = [_c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp,
                                     _c_vp, _c_i64, _c_vp]
    L.stq_grouped_swiglu.restype = _c_int
    L.stq_grouped_swiglu_workspace.argtypes = [_c_i64, _c_i64, _c_i64, _c_i64, ctypes.c_int32, ctypes.POINTER(_c_i64)]
    L.stq_grouped_swiglu_workspace.restype = _c_int
    for plan in (L.stq_grouped_swiglu_plan, L.stq_grouped_swiglu_backward_plan):
        plan.argtypes = [_c_i64, _c_i64, _c_i64, _c_i64, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)]
        plan.restype = _c_int
    L.stq_grouped_swiglu_backward.argtypes = [_c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp,
                                              _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp]
    L.stq_grouped_swiglu_backward.restype = _c_int
    L.stq_grouped_swiglu_backward_workspace.argtypes = [_c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_int,
                                                        ctypes.POINTER(_c_i64)]
    L.stq_grouped_swiglu_backward_workspace.restype = _c_int
    L.stq_q8_quantize_rows.argtypes = [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_vp]
    L.stq_q8_quantize_rows.restype = _c_int
    L.stq_q8_matmul.argtypes = [_c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_int,
                                _c_i64, _c_vp]
    L.stq_q8_matmul.restype = _c_int
    L.stq_token_logprobs.argtypes = [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64,
                                     _c_vp, _c_vp, _c_vp, _c_i64, _c_vp]
    L.stq_token_logprobs.restype = _c_int
    L.stq_token_logprobs_workspace.argtypes = [_c_int, _c_i64, _c_i64, _c_i64, ctypes.c_int32,
                                               ctypes.POINTER(_c_i64)]
    L.stq_token_logprobs_workspace.restype = _c_int
    L.stq_token_logprobs_backward.argtypes = [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp,
                                              _c_vp, _c_vp, _c_i64, _c_vp]
    L.stq_token_logprobs_backward.restype = _c_int
    L.stq_stream_read_probe.argtypes = [_c_vp, _c_i64, _c_vp, _c_vp]
    L.stq_stream_read_probe.restype = _c_int
    L.stq_mfma_loop_probe.argtypes = [_c_i64, _c_vp, _c_vp]
    L.stq_mfma_loop_probe.restype = _c_int
    L.stq_lds_read_probe.argtypes = [_c_int, _c_i64, _c_vp, _c_vp]
    L.stq_lds_read_probe.restype = _c_int
    _lib = L
    return L


def _check(func: str, status: int) -> None:
    if status != 0:
        raise StqError(func, status, lib().stq_last_error().decode())


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


_CUS: dict = {}


def _device_cus(device) -> int:
    """Compute units of a GPU tensor's device, the count the library plans the GEMV for."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    if idx not in _CUS:
        _CUS[idx] = torch.cuda.get_device_properties(idx).multi_processor_count
    return _CUS[idx]


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _on_gpu(name: str, t: torch.Tensor, dtype: torch.dtype) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _holds(name: str, t: torch.Tensor, n: int) -> None:
    """The kernels index raw pointers: a buffer smaller than the shapes say would be read or
    written past its end, so it is refused here."""
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs {n}")


def _workspace(ws: torch.Tensor | None, need: int, device) -> torch.Tensor | None:
    """A caller's workspace (checked) or a new one from torch's caching allocator; its memory
    is ordered on the current stream, like every other tensor the call takes."""
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need > 0 else None
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    return ws


def _ws_args(ws: torch.Tensor | None) -> tuple:
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def _table(name: str, t: torch.Tensor, n_experts: int, stride: int, n: int, k: int) -> None:
    if n_experts > 0 and n > 0:
        _holds(name, t, (int(n_experts) - 1) * int(stride) + int(n) * row_bytes(k))


def _one_gpu(first: torch.Tensor, *others) -> torch.device:
    """The GPU `first` lives on; every other tensor given must live there too."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError(f"the tensors must be GPU tensors, got one on {dev}")
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError(f"the tensors must be on one GPU, got {t.device} beside {dev}")
    return dev


def _call(device: torch.device, func: str, *args) -> None:
    """Run an entry point on `device`'s current stream, with that device current."""
    f = getattr(_lib or lib(), func)
    if device.index == torch.cuda.current_device():
        status = f(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            status = f(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if status != 0:
        _check(func, status)


def _rows(name: str, t: torch.Tensor, *dtypes: torch.dtype) -> int:
    """Row stride in elements of a matrix whose rows are contiguous (any distance apart)."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    (n, k), (ld, step) = t.shape, t.stride()
    if step != 1 and k > 1:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    # a one-row view may carry any stride in its first dimension
    return ld if n > 1 else max(1, k)


def _vector(name: str, t: torch.Tensor, dtype: torch.dtype, n: int) -> None:
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} entries, got {t.numel()}")


def row_bytes(k: int) -> int:
    rb = lib().stq_row_bytes(int(k))
    if rb < 0:
        raise ValueError("k must be a positive multiple of 256")
    return rb


def quantize_rows(w: torch.Tensor, imatrix: torch.Tensor | None = None, encoder: int = ENC_WLS,
                  rounds: int = 3, out: torch.Tensor | None = None) -> torch.Tensor:
    """Encode fp32 rows [n, k] on the GPU into a packed matrix (flat uint8, n*k/256*42 bytes,
    64-row tiles, block-major inside a tile)."""
    _on_gpu("w", w, torch.float32)
    n, k = w.shape
    if imatrix is not None:
        _on_gpu("imatrix", imatrix, torch.float32)
        _holds("imatrix", imatrix, k)
    if out is None:
        out = torch.empty(n * row_bytes(k), dtype=torch.uint8, device=w.device)
    _on_gpu("out", out, torch.uint8)
    if out.numel() < n * row_bytes(k):
        raise ValueError("out must hold n*k/256*42 bytes")
    _check("stq_quantize_rows", lib().stq_quantize_rows(w.data_ptr(), _ptr(imatrix), n, k, int(encoder),
                                                        int(rounds), out.data_ptr(), _stream()))
    return out


def dequantize_rows(q: torch.Tensor, n: int, k: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Decode a packed matrix of n rows to fp32 [n, k]."""
    _on_gpu("q", q, torch.uint8)
    if q.numel() < n * row_bytes(k):
        raise ValueError("q must hold n*k/256*42 bytes")
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=q.device)
    _on_gpu("out", out, torch.float32)
    _holds("out", out, n * k)
    _check("stq_dequantize_rows", lib().stq_dequantize_rows(q.data_ptr(), n, k, out.data_ptr(), _stream()))
    return out


def gemv_plan(n_experts: int, n: int, k: int, n_pairs: int, n_cus: int = 0) -> tuple[int, int, int]:
    """(splits, max_parts, scratch_bytes) that gemv takes for these shapes on n_cus
    compute units (0: the current device's); host only."""
    sp, mp, sb = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
    _check("stq_gemv_plan", lib().stq_gemv_plan(int(n_experts), int(n), int(k), int(n_pairs), int(n_cus),
                                                ctypes.byref(sp), ctypes.byref(mp), ctypes.byref(sb)))
    return sp.value, mp.value, sb.value


def gemv(w_table: torch.Tensor, expert_stride: int, n_experts: int, n: int, k: int, x: torch.Tensor,
         pair_expert: torch.Tensor | None = None, pair_token: torch.Tensor | None = None,
         n_pairs: int | None = None, out: torch.Tensor | None = None,
         workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[i] = W_{pair_expert[i]} x[pair_token[i]] for every pair; x is [n_tokens, k] fp32 or bf16.
    `workspace` (GPU bytes, at least gemv_plan(...)[2]) is allocated here when not given."""
    _on_gpu("w_table", w_table, torch.uint8)
    if x.dtype == torch.bfloat16:
        xd = X_BF16
    elif x.dtype == torch.float32:
        xd = X_F32
    else:
        raise ValueError("x must be float32 or bfloat16")
    _on_gpu("x", x, x.dtype)
    n_tokens = x.shape[0]
    if n_pairs is None:
        if pair_expert is not None:
            n_pairs = pair_expert.numel()
        elif pair_token is not None:
            n_pairs = pair_token.numel()
        else:
            n_pairs = n_tokens
    for nm, t in (("pair_expert", pair_expert), ("pair_token", pair_token)):
        if t is not None:
            _on_gpu(nm, t, torch.int32)
            if t.numel() != n_pairs:
                raise ValueError(f"{nm} must hold n_pairs entries")
    if out is None:
        out = torch.empty((n_pairs, n), dtype=torch.float32, device=x.device)
    _on_gpu("out", out, torch.float32)
    _holds("out", out, int(n_pairs) * int(n))
    if int(n_pairs) > 0:
        _table("w_table", w_table, n_experts, expert_stride, n, k)
    # a one-row view may carry any stride in its first dimension; its rows are k apart
    x_stride = x.stride(0) if n_tokens > 1 else x.shape[1]
    if workspace is None and int(n_pairs) > 0 and int(n) > 0:
        need = gemv_plan(n_experts, n, k, n_pairs, _device_cus(x.device))[2]
        workspace = _workspace(None, need, x.device)
    else:
        workspace = _workspace(workspace, 0, x.device)
    _check("stq_gemv", lib().stq_gemv(w_table.data_ptr(), int(expert_stride), int(n_experts), int(n), int(k),
                                      x.data_ptr(), xd, x_stride, n_tokens, _ptr(pair_expert),
                                      _ptr(pair_token), int(n_pairs), out.data_ptr(), *_ws_args(workspace),
                                      _stream()))
    return out


def gemv_noalloc(w_table: torch.Tensor, expert_stride: int, n_experts: int, n: int, k: int, x: torch.Tensor,
                 pair_expert: torch.Tensor | None, pair_token: torch.Tensor | None, out: torch.Tensor) -> torch.Tensor:
    """gemv without any allocation (neither here nor in the library): the caller passes `out`
    [n_pairs, n] fp32; split outputs use the library's fixed per-GPU scratch, so calls on one
    GPU must not overlap.  Shapes needing more scratch than it holds raise."""
    _on_gpu("w_table", w_table, torch.uint8)
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x must be float32 or bfloat16")
    _on_gpu("x", x, x.dtype)
    _on_gpu("out", out, torch.float32)
    n_tokens = x.shape[0]
    n_pairs = out.shape[0]
    for nm, t in (("pair_expert", pair_expert), ("pair_token", pair_token)):
        if t is not None:
            _on_gpu(nm, t, torch.int32)
            if t.numel() != n_pairs:
                raise ValueError(f"{nm} must hold out.shape[0] entries")
    _holds("out", out, int(n_pairs) * int(n))
    if int(n_pairs) > 0:
        _table("w_table", w_table, n_experts, expert_stride, n, k)
    x_stride = x.stride(0) if n_tokens > 1 else x.shape[1]
    _check("stq_gemv_noalloc",
           lib().stq_gemv_noalloc(w_table.data_ptr(), int(expert_stride), int(n_experts), int(n), int(k),
                                  x.data_ptr(), X_BF16 if x.dtype == torch.bfloat16 else X_F32, x_stride, n_tokens,
                                  _ptr(pair_expert), _ptr(pair_token), int(n_pairs), out.data_ptr(), _stream()))
    return out


def grouped_gemm(w_table: torch.Tensor, expert_stride: int, n_experts: int, n: int, k: int,
                 x_sorted: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Y[rows of e] = X[rows of e] W_e^T with rows grouped by expert; x_sorted bf16 [total_m, k]."""
    _on_gpu("w_table", w_table, torch.uint8)
    _on_gpu("x_sorted", x_sorted, torch.bfloat16)
    _on_gpu("offsets", offsets, torch.int32)
    if offsets.numel() != n_experts + 1:
        raise ValueError("offsets must hold n_experts + 1 entries")
    if x_sorted.dim() != 2 or x_sorted.shape[1] != k:
        raise ValueError("x_sorted must be [total_m, k]")
    total_m = x_sorted.shape[0]
    if out is None:
        out = torch.empty((total_m, n), dtype=torch.float32, device=x_sorted.device)
    _on_gpu("out", out, torch.float32)
    _holds("out", out, total_m * int(n))
    if total_m > 0:
        _table("w_table", w_table, n_experts, expert_stride, n, k)
    _check("stq_grouped_gemm", lib().stq_grouped_gemm(w_table.data_ptr(), int(expert_stride), int(n_experts),
                                                      int(n), int(k), x_sorted.data_ptr(), offsets.data_ptr(),
                                                      total_m, out.data_ptr(), _stream()))
    return out


def moe_ffn_workspace(n_experts: int, d_model: int, d_ff: int, n_tokens: int, top_k: int, n_cus: int = 0) -> int:
    """Workspace bytes moe_ffn_decode needs for these shapes on n_cus compute units (0: the
    current device's); host only."""
    wb = ctypes.c_int64()
    _check("stq_moe_ffn_workspace", lib().stq_moe_ffn_workspace(int(n_experts), int(d_model), int(d_ff),
                                                                int(n_tokens), int(top_k), int(n_cus),
                                                                ctypes.byref(wb)))
    return wb.value


def moe_ffn_decode(w_gate_up: torch.Tensor, gate_up_stride: int, w_down: torch.Tensor, down_stride: int,
                   n_experts: int, d_model: int, d_ff: int, x: torch.Tensor, pair_expert: torch.Tensor,
                   pair_weight: torch.Tensor, top_k: int, out: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Routed-expert FFN for decode tokens x bf16 [T, d_model]: per token, the routing-weighted sum
    over its top_k pairs of W_down_e (silu(W_gate_e x) * (W_up_e x)); pairs token-major [T*top_k].
    `workspace` (GPU bytes, at least moe_ffn_workspace(...)) is allocated here when not given."""
    _on_gpu("w_gate_up", w_gate_up, torch.uint8)
    _on_gpu("w_down", w_down, torch.uint8)
    _on_gpu("x", x, torch.bfloat16)
    _on_gpu("pair_expert", pair_expert, torch.int32)
    _on_gpu("pair_weight", pair_weight, torch.float32)
    if x.dim() != 2 or x.shape[1] != d_model:
        raise ValueError("x must be [n_tokens, d_model]")
    n_tokens = x.shape[0]
    if pair_expert.numel() != n_tokens * top_k or pair_weight.numel() != n_tokens * top_k:
        raise ValueError("pair_expert and pair_weight must hold n_tokens*top_k entries")
    if out is None:
        out = torch.empty((n_tokens, d_model), dtype=torch.float32, device=x.device)
    _on_gpu("out", out, torch.float32)
    _holds("out", out, n_tokens * int(d_model))
    if n_tokens > 0:
        _table("w_gate_up", w_gate_up, n_experts, gate_up_stride, 2 * int(d_ff), d_model)
        _table("w_down", w_down, n_experts, down_stride, d_model, d_ff)
    if workspace is None and n_tokens > 0:
        need = moe_ffn_workspace(n_experts, d_model, d_ff, n_tokens, top_k, _device_cus(x.device))
        workspace = _workspace(None, need, x.device)
    else:
        workspace = _workspace(workspace, 0, x.device)
    _check("stq_moe_ffn_decode",
           lib().stq_moe_ffn_decode(w_gate_up.data_ptr(), int(gate_up_stride), w_down.data_ptr(), int(down_stride),
                                    int(n_experts), int(d_model), int(d_ff), x.data_ptr(), n_tokens,
                                    pair_expert.data_ptr(), pair_weight.data_ptr(), int(top_k), out.data_ptr(),
                                    *_ws_args(workspace), _stream()))
    return out


def _matrix(name: str, t: torch.Tensor, dtype: torch.dtype, rows: int, cols: int) -> None:
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or tuple(t.shape) != (rows, cols) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{rows}, {cols}], got {tuple(t.shape)}")


def _swiglu_args(w_gate_up, expert_stride, n_experts, d_model, d_ff, x_sorted, offsets, total_m: int) -> None:
    """Checks shared by the gated feed-forward and its gradients, which may have no table or no rows."""
    if w_gate_up is not None and (w_gate_up.dtype != torch.uint8 or not w_gate_up.is_contiguous()):
        raise ValueError("w_gate_up must be contiguous torch.uint8")
    _vector("offsets", offsets, torch.int32, int(n_experts) + 1)
    if x_sorted is not None:
        _matrix("x_sorted", x_sorted, torch.bfloat16, total_m, int(d_model))
    if w_gate_up is not None and total_m > 0:
        _table("w_gate_up", w_gate_up, n_experts, expert_stride, 2 * int(d_ff), d_model)


def grouped_swiglu_workspace(n_experts: int, d_model: int, d_ff: int, total_m: int, n_cus: int = 0) -> int:
    """Workspace bytes grouped_swiglu needs for these shapes on n_cus compute units (0: the
    current device's); host only."""
    wb = ctypes.c_int64()
    _check("stq_grouped_swiglu_workspace",
           lib().stq_grouped_swiglu_workspace(int(n_experts), int(d_model), int(d_ff), int(total_m), int(n_cus),
                                              ctypes.byref(wb)))
    return wb.value


def _pass_rows(func: str, n_experts: int, d_model: int, d_ff: int, total_m: int, n_cus: int) -> int:
    rows = ctypes.c_int32()
    _check(func, getattr(lib(), func)(int(n_experts), int(d_model), int(d_ff), int(total_m), int(n_cus),
                                      ctypes.byref(rows)))
    return rows.value


def grouped_swiglu_plan(n_experts: int, d_model: int, d_ff: int, total_m: int, n_cus: int = 0) -> int:
    """Rows per pass of an expert that grouped_swiglu takes for these shapes on n_cus compute units (0: the
    current device's), 0 where the rows run through the GEMV's kernels; host only."""
    return _pass_rows("stq_grouped_swiglu_plan", n_experts, d_model, d_ff, total_m, n_cus)


@functools.lru_cache(maxsize=256)
def _swiglu_need(n_experts: int, d_model: int, d_ff: int, total_m: int, n_cus: int, gemv_plan_override) -> int:
    return grouped_swiglu_workspace(n_experts, d_model, d_ff, total_m, n_cus)


def grouped_swiglu(w_gate_up: torch.Tensor, expert_stride: int, n_experts: int, d_model: int, d_ff: int,
                   x_sorted: torch.Tensor, offsets: torch.Tensor, out: torch.Tensor | None = None,
                   gate_up: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """h = silu(W_gate_e x) * (W_up_e x), bf16 [total_m, d_ff], for rows x_sorted bf16 [total_m, d_model]
    grouped by expert (offsets as in grouped_gemm) and packed [2*d_ff, d_model] experts.  `gate_up`
    (bf16 [total_m, 2*d_ff]) receives the pre-activations that grouped_swiglu_backward reads.
    `workspace` (GPU bytes, at least grouped_swiglu_workspace(...)) is allocated here when not given."""
    dev = _one_gpu(w_gate_up, x_sorted, offsets, out, gate_up, workspace)
    E, d, f = int(n_experts), int(d_model), int(d_ff)
    if x_sorted.dim() != 2:
        raise ValueError("x_sorted must be [total_m, d_model]")
    total_m = x_sorted.shape[0]
    _swiglu_args(w_gate_up, expert_stride, E, d, f, x_sorted, offsets, total_m)
    if out is None:
        out = torch.empty((total_m, f), dtype=torch.bfloat16, device=dev)
    else:
        _matrix("out", out, torch.bfloat16, total_m, f)
    if gate_up is not None:
        _matrix("gate_up", gate_up, torch.bfloat16, total_m, 2 * f)
    if workspace is None:
        # the GEMV's tuning override changes its scratch, and so is part of the key
        need = _swiglu_need(E, d, f, total_m, _device_cus(dev), os.environ.get("STQ_GEMV_PLAN"))
        workspace = _workspace(None, need, dev)
    else:
        workspace = _workspace(workspace, 0, dev)
    _call(dev, "stq_grouped_swiglu", w_gate_up.data_ptr(), int(expert_stride), E, d, f, x_sorted.data_ptr(),
          offsets.data_ptr(), total_m, out.data_ptr(), _ptr(gate_up), *_ws_args(workspace))
    return out


def grouped_swiglu_backward_workspace(n_experts: int, d_model: int, d_ff: int, total_m: int, need_dx: bool = True,
                                      need_dw: bool = True) -> int:
    """Workspace bytes grouped_swiglu_backward needs for these shapes (host only)."""
    wb = ctypes.c_int64()
    _check("stq_grouped_swiglu_backward_workspace",
           lib().stq_grouped_swiglu_backward_workspace(int(n_experts), int(d_model), int(d_ff), int(total_m),
                                                       int(bool(need_dx)), int(bool(need_dw)), ctypes.byref(wb)))
    return wb.value


def grouped_swiglu_backward_plan(n_experts: int, d_model: int, d_ff: int, total_m: int, n_cus: int = 0) -> int:
    """Rows per pass of an expert that grouped_swiglu_backward's dx takes, as grouped_swiglu_plan."""
    return _pass_rows("stq_grouped_swiglu_backward_plan", n_experts, d_model, d_ff, total_m, n_cus)


def grouped_swiglu_backward(w_gate_up: torch.Tensor | None, expert_stride: int, n_experts: int, d_model: int,
                            d_ff: int, x_sorted: torch.Tensor | None, offsets: torch.Tensor, gate_up: torch.Tensor,
                            dh: torch.Tensor,
                            need_dx: bool = True, need_dw: bool = True, dx: torch.Tensor | None = None,
                            dw: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """(dx, dw) of grouped_swiglu for the gradient dh bf16 [total_m, d_ff] at h and the gate_up it saved:
    dx bf16 [total_m, d_model] through the decoded weights, dw bf16 [n_experts, 2*d_ff, d_model] the
    gradient of the decoded weights; None for the one not needed.  dx reads no x_sorted and dw no
    w_gate_up, which may be None where only the other is needed.  `workspace` (GPU bytes, at least
    grouped_swiglu_backward_workspace(...)) is allocated here when not given."""
    dev = _one_gpu(gate_up, w_gate_up, x_sorted, offsets, dh, dx, dw, workspace)
    E, d, f = int(n_experts), int(d_model), int(d_ff)
    if need_dx and w_gate_up is None:
        raise ValueError("dx needs w_gate_up")
    if need_dw and x_sorted is None:
        raise ValueError("dw needs x_sorted")
    if gate_up.dim() != 2:
        raise ValueError("gate_up must be [total_m, 2 * d_ff]")
    total_m = gate_up.shape[0]
    _matrix("gate_up", gate_up, torch.bfloat16, total_m, 2 * f)
    _swiglu_args(w_gate_up, expert_stride, E, d, f, x_sorted, offsets, total_m)
    _matrix("dh", dh, torch.bfloat16, total_m, f)
    if need_dx:
        dx = torch.empty((total_m, d), dtype=torch.bfloat16, device=dev) if dx is None else dx
        _matrix("dx", dx, torch.bfloat16, total_m, d)
    elif dx is not None:
        raise ValueError("dx is given but need_dx is False")
    if need_dw:
        dw = torch.empty((E, 2 * f, d), dtype=torch.bfloat16, device=dev) if dw is None else dw
        if dw.dtype != torch.bfloat16 or tuple(dw.shape) != (E, 2 * f, d) or not dw.is_contiguous():
            raise ValueError(f"dw must be contiguous bfloat16 [{E}, {2 * f}, {d}]")
    elif dw is not None:
        raise ValueError("dw is given but need_dw is False")
    if workspace is None:
        workspace = _workspace(None, grouped_swiglu_backward_workspace(E, d, f, total_m, need_dx, need_dw), dev)
    else:
        workspace = _workspace(workspace, 0, dev)
    _call(dev, "stq_grouped_swiglu_backward", _ptr(w_gate_up), int(expert_stride), E, d, f, _ptr(x_sorted),
          offsets.data_ptr(), total_m, gate_up.data_ptr(), dh.data_ptr(), _ptr(dx), _ptr(dw), *_ws_args(workspace))
    return dx, dw


def _q8_stride(name: str, t: torch.Tensor) -> int:
    """Row stride in bytes of int8 rows, which own their bytes up to the next multiple of 16."""
    stride = _rows(name, t, torch.int8)
    n, k = t.shape
    kp = (k + 15) // 16 * 16
    if n <= 1:
        stride = kp
    if kp != k and n > 0 and t.storage_offset() + (n - 1) * stride + kp > t.untyped_storage().nbytes():
        raise ValueError(f"{name}'s last row must own its bytes up to the next multiple of 16")
    return stride


def q8_quantize_rows(x: torch.Tensor, out: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """Rows of 8-bit integers with one scale each: (q int8 [n, k], scale fp32 [n]) of x fp32 or bf16
    [n, k], scale = max|x| / 127 and q the nearest integer to x / scale.  Without `out` the rows are
    k rounded up to 16 bytes apart (the layout q8_matmul reads), padded with zeros."""
    dev = _one_gpu(x, out, scale)
    stride = _rows("x", x, torch.float32, torch.bfloat16)
    n, k = x.shape
    if out is None:
        qs = (k + 15) // 16 * 16
        out = torch.empty((n, qs), dtype=torch.int8, device=dev)
        if qs != k:
            out = out[:, :k]
    else:
        if tuple(out.shape) != (n, k):
            raise ValueError("out must be [n, k] like x")
        qs = _q8_stride("out", out)
    if scale is None:
        scale = torch.empty(n, dtype=torch.float32, device=dev)
    else:
        _vector("scale", scale, torch.float32, n)
    _call(dev, "stq_q8_quantize_rows", x.data_ptr(), X_BF16 if x.dtype == torch.bfloat16 else X_F32, stride, n, k,
          out.data_ptr(), qs, scale.data_ptr())
    return out, scale


def q8_matmul(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """y[i, j] = (a[i] . w[j]) a_scale[i] w_scale[j] for int8 rows a [m, k] and w [n, k], the sum exact;
    y is bf16 or fp32 [m, n]: `out`'s type, or out_dtype (bf16 when neither is given)."""
    dev = _one_gpu(a, a_scale, w, w_scale, out)
    lda, ldw = _q8_stride("a", a), _q8_stride("w", w)
    m, k = a.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ValueError("a and w must have rows of the same length")
    _vector("a_scale", a_scale, torch.float32, m)
    _vector("w_scale", w_scale, torch.float32, n)
    if out is None:
        if out_dtype is None:
            out_dtype = torch.bfloat16
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("out_dtype must be bfloat16 or float32")
        out = torch.empty((m, n), dtype=out_dtype, device=dev)
        ldy = n
    else:
        if tuple(out.shape) != (m, n):
            raise ValueError("out must be [m, n]")
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out must be {out_dtype} like out_dtype, got {out.dtype}")
        ldy = _rows("out", out, torch.bfloat16, torch.float32)
    _call(dev, "stq_q8_matmul", a.data_ptr(), lda, a_scale.data_ptr(), w.data_ptr(), ldw, w_scale.data_ptr(), m, n, k,
          out.data_ptr(), X_BF16 if out.dtype == torch.bfloat16 else X_F32, ldy)
    return out


def token_logprobs_workspace(x_dtype: int, n_rows: int, vocab: int, top_n: int, n_cus: int = 0) -> int:
    """Workspace bytes token_logprobs needs for these shapes (x_dtype X_F32 or X_BF16) on n_cus
    compute units (0: the current device's); host only."""
    wb = ctypes.c_int64()
    _check("stq_token_logprobs_workspace",
           lib().stq_token_logprobs_workspace(int(x_dtype), int(n_rows), int(vocab), int(top_n), int(n_cus),
                                              ctypes.byref(wb)))
    return wb.value


@functools.lru_cache(maxsize=256)
def _logprobs_need(x_dtype: int, n_rows: int, vocab: int, top_n: int, n_cus: int) -> int:
    return token_logprobs_workspace(x_dtype, n_rows, vocab, top_n, n_cus)


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, top_n: int = 0, logprob: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, entropy: torch.Tensor | None = None,
                   top_ids: torch.Tensor | None = None, top_logprobs: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None):
    """(logprob, lse, entropy, top_ids, top_logprobs) of logits fp32 or bf16 [n, vocab] at targets
    int32 [n]: log probability of each row's target, log-sum-exp, entropy, and the top_n (at most 32)
    most likely ids with their log probabilities, equal logits by lowest id.  Outputs and `workspace`
    (GPU bytes, at least token_logprobs_workspace(...)) are allocated here when not given."""
    dev = _one_gpu(logits, targets, logprob, lse, entropy, top_ids,
                    top_logprobs, workspace)
    stride = _rows("logits", logits, torch.float32, torch.bfloat16)
    n, vocab = logits.shape
    top_n = int(top_n)
    if top_n < 0:
        raise ValueError("top_n must not be negative")
    _vector("targets", targets, torch.int32, n)
    for name, t in (("logprob", logprob), ("lse", lse), ("entropy", entropy)):
        if t is not None:
            _vector(name, t, torch.float32, n)
    if logprob is None and lse is None and entropy is None:
        logprob, lse, entropy = torch.empty((3, n), dtype=torch.float32, device=dev).unbind(0)
    else:
        logprob, lse, entropy = (torch.empty(n, dtype=torch.float32, device=dev) if t is None else t
                                 for t in (logprob, lse, entropy))
    if top_ids is None:
        top_ids = torch.empty((n, top_n), dtype=torch.int32, device=dev)
    else:
        _vector("top_ids", top_ids, torch.int32, n * top_n)
    if top_logprobs is None:
        top_logprobs = torch.empty((n, top_n), dtype=torch.float32, device=dev)
    else:
        _vector("top_logprobs", top_logprobs, torch.float32, n * top_n)
    xd = X_BF16 if logits.dtype == torch.bfloat16 else X_F32
    if workspace is None and n > 0:
        workspace = _workspace(None, _logprobs_need(xd, n, vocab, top_n, _device_cus(dev)), dev)
    else:
        workspace = _workspace(workspace, 0, dev)
    _call(dev, "stq_token_logprobs", logits.data_ptr(), xd, stride, n, vocab, targets.data_ptr(), logprob.data_ptr(),
          lse.data_ptr(), entropy.data_ptr(), top_n, top_ids.data_ptr(), top_logprobs.data_ptr(), *_ws_args(workspace))
    return logprob, lse, entropy, top_ids, top_logprobs


def token_logprobs_backward(logits: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                            entropy: torch.Tensor | None, grad_logprob: torch.Tensor | None,
                            grad_entropy: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of token_logprobs with respect to the logits, for gradients fp32 [n] arriving at
    logprob and entropy (either may be None); lse and entropy are what the forward call gave.
    `out` has the logits' type and shape and may be the logits themselves."""
    dev = _one_gpu(logits, targets, lse, entropy, grad_logprob,
                    grad_entropy, out)
    stride = _rows("logits", logits, torch.float32, torch.bfloat16)
    n, vocab = logits.shape
    _vector("targets", targets, torch.int32, n)
    for name, t in (("lse", lse), ("entropy", entropy), ("grad_logprob", grad_logprob), ("grad_entropy", grad_entropy)):
        if t is not None:
            _vector(name, t, torch.float32, n)
    if out is None:
        out = torch.empty((n, vocab), dtype=logits.dtype, device=dev)
        ds = vocab
    else:
        if tuple(out.shape) != (n, vocab):
            raise ValueError("out must be [n, vocab] like the logits")
        ds = _rows("out", out, logits.dtype)
    _call(dev, "stq_token_logprobs_backward", logits.data_ptr(), X_BF16 if logits.dtype == torch.bfloat16 else X_F32,
          stride, n, vocab, targets.data_ptr(), lse.data_ptr(), _ptr(entropy), _ptr(grad_logprob), _ptr(grad_entropy),
          out.data_ptr(), ds)
    return out


def layer_errors_workspace(n_rows: int, k: int, n_calib: int) -> int:
    """Workspace bytes layer_errors needs for these shapes (host only)."""
    wb = ctypes.c_int64()
    _check("stq_layer_errors_workspace", lib().stq_layer_errors_workspace(int(n_rows), int(k), int(n_calib),
                                                                          ctypes.byref(wb)))
    return wb.value


def layer_errors(w: torch.Tensor, w_hat: torch.Tensor, x_calib: torch.Tensor,
                 out_full: torch.Tensor | None = None, out_diag: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None):
    """Per-row error of w_hat against w under calibration rows x_calib fp32 [N, k]: full-Hessian
    sum_i ((w - w_hat) . x_i)^2 and diagonal sum_c H_cc (w - w_hat)_c^2, both fp64 [n].
    `workspace` (GPU bytes, at least layer_errors_workspace(...)) is allocated here when not given."""
    _on_gpu("w", w, torch.float32)
    _on_gpu("w_hat", w_hat, torch.float32)
    _on_gpu("x_calib", x_calib, torch.float32)
    n, k = w.shape
    if tuple(w_hat.shape) != (n, k) or x_calib.dim() != 2 or x_calib.shape[1] != k:
        raise ValueError("w, w_hat must be [n, k] and x_calib [N, k]")
    if out_full is None:
        out_full = torch.empty(n, dtype=torch.float64, device=w.device)
    if out_diag is None:
        out_diag = torch.empty(n, dtype=torch.float64, device=w.device)
    _on_gpu("out_full", out_full, torch.float64)
    _on_gpu("out_diag", out_diag, torch.float64)
    if out_full.numel() < n or out_diag.numel() < n:
        raise ValueError("outputs must hold n entries")
    if workspace is None and n > 0 and x_calib.shape[0] > 0:
        workspace = _workspace(None, layer_errors_workspace(n, k, x_calib.shape[0]), w.device)
    else:
        workspace = _workspace(workspace, 0, w.device)
    _check("stq_layer_errors", lib().stq_layer_errors(w.data_ptr(), w_hat.data_ptr(), n, k, x_calib.data_ptr(),
                                                      x_calib.shape[0], out_full.data_ptr(), out_diag.data_ptr(),
                                                      *_ws_args(workspace), _stream()))
    return out_full, out_diag


def q2_roundtrip(w: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Reconstruction of fp32 rows [n, k] through the 2-bit stand-in format (fp16 rms/2 scale per
    256 weights, levels +-s, +-3s)."""
    _on_gpu("w", w, torch.float32)
    n, k = w.shape
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=w.device)
    _on_gpu("out", out, torch.float32)
    if tuple(out.shape) != (n, k):
        raise ValueError("out must be [n, k]")
    _check("stq_q2_roundtrip", lib().stq_q2_roundtrip(w.data_ptr(), n, k, out.data_ptr(), _stream()))
    return out


def greedy_allocation(gain, extra_bytes, budget: float):
    """Layers to move to the larger format, taken by error reduction per added byte within
    `budget` bytes (host function; numpy in, numpy bool mask out)."""
    import numpy as np
    g = np.ascontiguousarray(gain, dtype=np.float64)
    e = np.ascontiguousarray(extra_bytes, dtype=np.float64)
    if g.shape != e.shape or g.ndim != 1:
        raise ValueError("gain and extra_bytes must be 1-D of equal length")
    chosen = np.zeros(g.shape[0], dtype=np.uint8)
    _check("stq_greedy_allocation", lib().stq_greedy_allocation(g.ctypes.data, e.ctypes.data, g.shape[0],
                                                                float(budget), chosen.ctypes.data))
    return chosen.astype(bool)


def stream_read_probe(buf: torch.Tensor, sink: torch.Tensor) -> None:
    """Read every byte of the GPU tensor `buf` once (a streaming-read rate
    reference for the HBM roofline); `sink` is a one-element int32 GPU tensor."""
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous GPU tensor")
    _on_gpu("sink", sink, torch.int32)
    nbytes = buf.numel() * buf.element_size()
    _check("stq_stream_read_probe", lib().stq_stream_read_probe(buf.data_ptr(), nbytes - nbytes % 16,
                                                                sink.data_ptr(), _stream()))


def mfma_loop_probe(rounds: int, sink: torch.Tensor) -> None:
    """Matrix-core reference: MFMA_PROBE_FLOP_PER_ROUND * rounds flops of
    bf16 MFMAs with no memory traffic; `sink` is a one-element float32 GPU tensor."""
    _on_gpu("sink", sink, torch.float32)
    _check("stq_mfma_loop_probe", lib().stq_mfma_loop_probe(int(rounds), sink.data_ptr(), _stream()))


def lds_read_probe(mode: int, rounds: int, sink: torch.Tensor) -> None:
    """LDS read reference: LDS_PROBE_READS_PER_ROUND * rounds wavefront LDS
    reads, 16-byte contiguous (mode 0) or two 4-byte table reads at a code
    (mode 1); `sink` is a one-element int32 GPU tensor."""
    _on_gpu("sink", sink, torch.int32)
    _check("stq_lds_read_probe", lib().stq_lds_read_probe(int(mode), int(rounds), sink.data_ptr(), _stream()))
