"""kq: fused dequantize-and-multiply of block-quantized weights on GB300 (sm_103a).

A thin ctypes binding over the C-ABI library ``libkq.so`` (declared in
``include/kq.h``). This module only marshals arguments: it passes device pointers
and the current CUDA stream to the library and raises on a nonzero status. Every
step of the computation runs in the library's CUDA kernels; there is no CPU or
PyTorch fallback, and importing fails loudly if ``libkq.so`` has not been built
(``python -m quantized_decode_gemv_block_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkq.so")

Q8_0, Q4_K, AFFINE4, Q5_K, Q6_K = 1, 2, 3, 4, 5
F32, BF16 = 1, 2
FORMATS = {"q8_0": Q8_0, "q4_k": Q4_K, "affine4": AFFINE4, "q5_k": Q5_K, "q6_k": Q6_K}
KQ_OK, KQ_ERR_ARG, KQ_ERR_UNSUPPORTED, KQ_ERR_WORKSPACE, KQ_ERR_CUDA, KQ_ERR_TIMEOUT = 0, -1, -2, -3, -4, -5


class KQError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"kq error {code}: {msg}")
        self.code = code


class DecodeModelC(ctypes.Structure):
    """Mirror of kq_decode_model (include/kq.h)."""
    _fields_ = [("n_layers", ctypes.c_int), ("hidden", ctypes.c_int), ("q_dim", ctypes.c_int),
                ("kv_dim", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("vocab", ctypes.c_int), ("layer_fmt", ctypes.c_int), ("head_fmt", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("w_qkv", ctypes.POINTER(ctypes.c_void_p)),
                ("w_o", ctypes.POINTER(ctypes.c_void_p)), ("w_gate_up", ctypes.POINTER(ctypes.c_void_p)),
                ("w_down", ctypes.POINTER(ctypes.c_void_p)), ("w_head", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libkq.so and declare its C signatures. Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m quantized_decode_gemv_block_gb300.build` (needs nvcc)")
    L = ctypes.CDLL(path)
    P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.kq_block_bytes.argtypes = [I]
    L.kq_block_bytes.restype = SZ
    L.kq_block_weights.argtypes = [I]
    L.kq_block_weights.restype = SZ
    L.kq_row_bytes.argtypes = [I, I]
    L.kq_row_bytes.restype = SZ
    L.kq_last_error.restype = ctypes.c_char_p
    L.kq_version.restype = ctypes.c_char_p
    L.kq_gemv.argtypes = [I, P, I, P, P, I, I, I, P]
    L.kq_gemv.restype = I
    L.kq_gemv_ex.argtypes = [I, P, I, P, P, I, I, I, ctypes.c_uint, P]
    L.kq_gemv_ex.restype = I
    L.kq_gemm.argtypes = [I, P, I, P, P, I, I, I, P, SZ, P]
    L.kq_gemm.restype = I
    L.kq_gemm_workspace_size.argtypes = [I, I, I, I, I]
    L.kq_gemm_workspace_size.restype = SZ
    L.kq_quantize.argtypes = [I, P, P, I, I, P]
    L.kq_quantize.restype = I
    L.kq_device_errors.restype = I
    L.kq_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeModelC), I]
    L.kq_decode_workspace_size.restype = SZ
    L.kq_attention_workspace_size.argtypes = [I, I, I, I, I]
    L.kq_attention_workspace_size.restype = SZ
    L.kq_attention.argtypes = [P, P, P, P, I, I, I, I, I, P, ctypes.c_float, P, SZ, P]
    L.kq_attention.restype = I
    L.kq_decode_attn_workspace_size.argtypes = [ctypes.POINTER(DecodeModelC), I, I]
    L.kq_decode_attn_workspace_size.restype = SZ
    L.kq_decode_step_attn.argtypes = [ctypes.POINTER(DecodeModelC), ctypes.POINTER(KVCacheC), P, P, I, P, P, SZ, P]
    L.kq_decode_step_attn.restype = I
    L.kq_decode_step.argtypes = [ctypes.POINTER(DecodeModelC), P, P, I, P, SZ, P]
    L.kq_decode_step.restype = I
    L.kq_decode_step_static.argtypes = [ctypes.POINTER(DecodeModelC), P, P, I, P]
    L.kq_decode_trace_size.argtypes = [ctypes.POINTER(DecodeModelC), I]
    L.kq_decode_trace_size.restype = SZ
    L.kq_decode_step_trace.argtypes = [ctypes.POINTER(DecodeModelC), P, P, I, P, SZ, P, SZ, P]
    L.kq_decode_step_trace.restype = I
    L.kq_decode_step_static.restype = I
    L.kq_shortlist_bytes.argtypes = [I, I]
    L.kq_shortlist_bytes.restype = SZ
    L.kq_shortlist_build.argtypes = [P, I, I, P, SZ, P]
    L.kq_shortlist_build.restype = I
    L.kq_head_argmax_workspace_size.argtypes = [I, I]
    L.kq_head_argmax_workspace_size.restype = SZ
    L.kq_head_argmax.argtypes = [P, P, I, P, I, I, I, P, P, P, P, SZ, ctypes.c_uint, P]
    L.kq_head_argmax.restype = I
    LL, F, U = ctypes.c_longlong, ctypes.c_float, ctypes.c_uint
    L.kq_pages_plan.argtypes = [P, P, I, I, P, I, P, I, P, P, P, P, P, I, P, P]
    L.kq_pages_plan.restype = I
    L.kq_pages_release.argtypes = [P, P, I, I, P, I, P, I, P, P, P, P]
    L.kq_pages_release.restype = I
    L.kq_rope.argtypes = [I, I, P, LL, P, LL, I, P, LL, P, LL, I, I, I, I, P, P, P, I, U, P]
    L.kq_rope.restype = I
    L.kq_kv8_bytes.argtypes = [I, I, I, I]
    L.kq_kv8_bytes.restype = SZ
    L.kq_kv8_append.argtypes = [P, I, P, LL, P, LL, P, I, P]
    L.kq_kv8_append.restype = I
    L.kq_attention_kv8_workspace_size.argtypes = [I, LL, I, I, I, I]
    L.kq_attention_kv8_workspace_size.restype = SZ
    L.kq_attention_kv8.argtypes = [P, I, P, LL, I, P, LL, I, P, P, I, I, I, I, LL, P, I, P, F, P, SZ, P]
    L.kq_attention_kv8.restype = I
    _lib = L
    return L


def lib():
    return load_library()


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _check(rc: int):
    if rc != KQ_OK:
        raise KQError(rc, lib().kq_last_error().decode())


def _stream(stream) -> int:
    if stream is None:
        if torch.cuda.is_initialized():  # the same stream as below, without building a Stream object (6 us of 7)
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def block_bytes(fmt) -> int:
    return lib().kq_block_bytes(_fmt(fmt))


def block_weights(fmt) -> int:
    return lib().kq_block_weights(_fmt(fmt))


def row_bytes(fmt, K: int) -> int:
    return lib().kq_row_bytes(_fmt(fmt), K)


def version() -> str:
    return lib().kq_version().decode()


def _x_dtype(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return BF16
    if x.dtype == torch.float32:
        return F32
    raise TypeError("x must be torch.bfloat16 or torch.float32")


KQ_OVERLAP_PREVIOUS = 1


def gemv(fmt, w: torch.Tensor, x: torch.Tensor, N: int, K: int, y: torch.Tensor | None = None,
         stream=None, overlap: bool = False) -> torch.Tensor:
    """Y (M x N fp32) = X (M x K) @ deq(W)^T for M <= 16, through kq_gemv / kq_gemv_ex.

    overlap=True passes KQ_OVERLAP_PREVIOUS: the previous kernel on the stream must not
    write w (it may still be running while this one streams w)."""
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if overlap:
        rc = lib().kq_gemv_ex(_fmt(fmt), w.data_ptr(), _x_dtype(x), x.data_ptr(), y.data_ptr(), M, N, K,
                              KQ_OVERLAP_PREVIOUS, _stream(stream))
    else:
        rc = lib().kq_gemv(_fmt(fmt), w.data_ptr(), _x_dtype(x), x.data_ptr(), y.data_ptr(), M, N, K,
                           _stream(stream))
    _check(rc)
    return y


def gemm_workspace_size(fmt, x_dtype, M: int, N: int, K: int) -> int:
    xd = x_dtype if isinstance(x_dtype, int) else (BF16 if x_dtype == torch.bfloat16 else F32)
    return lib().kq_gemm_workspace_size(_fmt(fmt), xd, M, N, K)


def gemm(fmt, w: torch.Tensor, x: torch.Tensor, N: int, K: int, y: torch.Tensor | None = None,
         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X @ deq(W)^T for any M, through kq_gemm (tensor cores for M > 16)."""
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    need = gemm_workspace_size(fmt, _x_dtype(x), M, N, K)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wp = workspace.data_ptr() if workspace is not None else None
    wn = workspace.numel() if workspace is not None else 0
    _check(lib().kq_gemm(_fmt(fmt), w.data_ptr(), _x_dtype(x), x.data_ptr(), y.data_ptr(), M, N, K,
                         wp, wn, _stream(stream)))
    return y


def attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, L: int, n_q: int, n_kv: int,
              head_dim: int, scale: float, mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode attention of the M window tokens (kq_attention): q M x (n_q*head_dim) fp32,
    k_cache / v_cache (L+M) x (n_kv*head_dim) bf16, mask None (causal) or M int32 words."""
    M = q.shape[0]
    if out is None:
        out = torch.empty((M, n_q * head_dim), dtype=torch.float32, device=q.device)
    need = lib().kq_attention_workspace_size(M, L, n_q, n_kv, head_dim)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(lib().kq_attention(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), M, L, n_q,
                              n_kv, head_dim, mask.data_ptr() if mask is not None else None, scale,
                              workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return out


KQ_HEAD_ALL_ROWS = 1


def shortlist_build(w_q8: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """The shortlist buffer of a Q8_0 head (kq_shortlist_build): the small Q4_K copy, then
    N fp32 score bounds (see shortlist_parts)."""
    need = lib().kq_shortlist_bytes(N, K)
    if need == 0:
        raise KQError(KQ_ERR_ARG, "bad head shape for the shortlist")
    if out is None:
        out = torch.empty(need, dtype=torch.uint8, device=w_q8.device)
    _check(lib().kq_shortlist_build(w_q8.data_ptr(), N, K, out.data_ptr(), out.numel(), _stream(stream)))
    return out


def shortlist_parts(buf: torch.Tensor, N: int, K: int):
    """(small copy bytes N x K/256*144, bounds N fp32): views into a shortlist buffer."""
    small = N * (K // 256) * 144
    s = (small + 255) // 256 * 256
    return buf[:small].view(N, K // 256 * 144), buf[s:s + 4 * N].view(torch.float32)


def head_argmax(w_q8: torch.Tensor, shortlist: torch.Tensor | None, x: torch.Tensor, N: int, K: int,
                all_rows: bool = False, workspace: torch.Tensor | None = None, token: torch.Tensor | None = None,
                score: torch.Tensor | None = None, rows_scored: torch.Tensor | None = None, stream=None):
    """Greedy next token of each hidden-state row of x over a Q8_0 head (kq_head_argmax).
    Returns (token int32 [M], score fp32 [M], rows_scored int32 [1]) device tensors."""
    M = x.shape[0]
    dev = x.device
    if workspace is None:
        workspace = torch.empty(lib().kq_head_argmax_workspace_size(M, N), dtype=torch.uint8, device=dev)
    if token is None:
        token = torch.empty(M, dtype=torch.int32, device=dev)
    if score is None:
        score = torch.empty(M, dtype=torch.float32, device=dev)
    if rows_scored is None:
        rows_scored = torch.empty(1, dtype=torch.int32, device=dev)
    _check(lib().kq_head_argmax(w_q8.data_ptr(), shortlist.data_ptr() if shortlist is not None else None,
                                _x_dtype(x), x.data_ptr(), M, N, K, token.data_ptr(), score.data_ptr(),
                                rows_scored.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                KQ_HEAD_ALL_ROWS if all_rows else 0, _stream(stream)))
    return token, score, rows_scored


def device_errors() -> int:
    """Read and clear the device error word (bit 0: a bounded in-kernel wait gave up; bit 1: a paged-cache
    kernel met lengths, slots or page ids out of bounds)."""
    rc = lib().kq_device_errors()
    if rc < 0:
        _check(rc)
    return rc


def quantize(fmt, w: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 N x K device matrix -> N x row_bytes uint8 blocks, through kq_quantize."""
    N, K = w.shape
    if out is None:
        out = torch.empty((N, row_bytes(fmt, K)), dtype=torch.uint8, device=w.device)
    _check(lib().kq_quantize(_fmt(fmt), w.data_ptr(), out.data_ptr(), N, K, _stream(stream)))
    return out


# ---- Paged 8-bit KV cache ----

PAGES_OUT_OF_PAGES, PAGES_TABLE_FULL, PAGES_TOKENS_FULL, PAGES_BAD_ARG = 1, 2, 4, 8
KQ_ROPE_ADJACENT, KQ_ROPE_INVERSE = 1, 2
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _dtype(t) -> int:
    try:
        return _DTYPES[t]
    except KeyError:
        raise TypeError("tensors must be torch.bfloat16 or torch.float32") from None


_I32 = torch.int32


class HostMemoryError(KQError, ValueError):
    """A tensor in host memory where a kernel would read its address."""


def _not_on_gpu(name: str):
    if torch.cuda.is_available():  # without a GPU the library refuses the call
        raise HostMemoryError(KQ_ERR_ARG, f"{name} must be on the GPU")


def _i32(name: str, t: torch.Tensor, n: int) -> int:
    """The address of a contiguous int32 tensor of at least n elements."""
    if t.dtype is not _I32 or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of at least {n} elements")
    if not t.is_cuda:
        _not_on_gpu(name)
    return t.data_ptr()


def _heads(name: str, t: torch.Tensor, heads: int | None = None, dim: int | None = None) -> int:
    """The token stride of a (T, heads, dim) tensor whose heads stand next to each other."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be (tokens, heads, head_dim)")
    if not t.is_cuda:
        _not_on_gpu(name)
    (T, H, D), (s0, s1, s2) = t.shape, t.stride()
    if (s2 != 1 and D > 1) or (s1 != D and H > 1):
        raise ValueError(f"{name} must be (tokens, heads, head_dim) with contiguous heads")
    if (heads is not None and H != heads) or (dim is not None and D != dim):
        raise ValueError(f"{name} must have {heads if heads is not None else 'any number of'} heads of {dim}")
    return s0 if T > 1 else H * D


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output or workspace of a call on `stream`: from that stream's pool, so that its memory goes back to
    work that runs behind the call, and not to another stream's."""
    if stream is None or torch.device(device).type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(raw, device) if raw else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class PagesPlan:
    """Outputs of pages_plan (device tensors): cu [B+1], pos [T], slot [T], n_free [1], status [1]."""
    __slots__ = ("cu", "pos", "slot", "n_free", "status")

    def __init__(self, B: int, T: int, device="cuda", stream=None):
        self.cu, self.pos, self.slot, self.n_free, self.status = (
            _empty(n, torch.int32, device, stream) for n in (B + 1, T, T, 1, 1))


def pages_plan(ctx_len: torch.Tensor, new_len: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
               n_free: torch.Tensor, page_size: int, T: int, out: PagesPlan | None = None, stream=None) -> PagesPlan:
    """Slots of up to T new tokens and the block-table entries they need (kq_pages_plan). block_table
    (B x max_blocks) is updated; n_free is read, the new count is in the result."""
    B, width = block_table.shape
    if out is None:
        out = PagesPlan(B, T, block_table.device, stream)
        outs = (out.n_free.data_ptr(), out.cu.data_ptr(), out.pos.data_ptr(), out.slot.data_ptr())
        status = out.status.data_ptr()
    else:
        outs = (_i32("out.n_free", out.n_free, 1), _i32("out.cu", out.cu, B + 1), _i32("out.pos", out.pos, T),
                _i32("out.slot", out.slot, T))
        status = _i32("out.status", out.status, 1)
    _check(lib().kq_pages_plan(_i32("ctx_len", ctx_len, B), _i32("new_len", new_len, B), B, page_size,
                               _i32("block_table", block_table, B * width), width, _i32("free_pages", free_pages, 0),
                               free_pages.numel(), _i32("n_free", n_free, 1), *outs, T, status, _stream(stream)))
    return out


def pages_release(length: torch.Tensor, done: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                  n_free: torch.Tensor, n_free_out: torch.Tensor, page_size: int, status: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Give back the pages of the requests with done[r] (bool or uint8) set (kq_pages_release); returns status."""
    B, width = block_table.shape
    if done.dtype not in (torch.bool, torch.uint8) or not done.is_contiguous() or done.numel() < B:
        raise ValueError("done must be a contiguous bool or uint8 tensor with one element per request")
    if not done.is_cuda:
        _not_on_gpu("done")
    if status is None:
        status = _empty(1, torch.int32, block_table.device, stream)
    _check(lib().kq_pages_release(_i32("length", length, B), done.data_ptr(), B, page_size,
                                  _i32("block_table", block_table, B * width), width, _i32("free_pages", free_pages, 0),
                                  free_pages.numel(), _i32("n_free", n_free, 1), _i32("n_free_out", n_free_out, 1),
                                  _i32("status", status, 1), _stream(stream)))
    return status


def rope(q: torch.Tensor | None, k: torch.Tensor | None, pos: torch.Tensor, inv_freq: torch.Tensor,
         pair_axis: torch.Tensor | None = None, adjacent: bool = False, inverse: bool = False, out_dtype=None,
         q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Rotary positions on q and k (T, heads, head_dim; either may be None), through kq_rope. pos: int32 [T]
    or [axes, T]; inv_freq: fp32, one per pair (rot_dim = 2 * its length); pair_axis: uint8, one per pair.
    inverse=True is the gradient of the call without it, and what autograd calls for a q or k that requires one.
    Returns (q_out, k_out)."""
    ref = k if q is None else q
    if ref is None:
        raise ValueError("one of q and k is needed")
    if torch.is_grad_enabled() and (ref.requires_grad or (k is not None and k.requires_grad)):
        if q_out is not None or k_out is not None:
            raise ValueError("q_out and k_out take no q or k that requires a gradient")
        return _Rope.apply(q, k, pos, inv_freq, pair_axis, adjacent, inverse, out_dtype, stream)
    T, _, D = ref.shape
    dtype = ref.dtype
    axes = pos.shape[0] if pos.dim() == 2 else 1
    if pos.dim() > 2 or (axes > 1 and pos.shape[1] != T):
        raise ValueError("pos must be (tokens) or, of several axes, (axes, tokens)")
    pairs = inv_freq.numel()
    if pairs and (inv_freq.dtype is not torch.float32 or not inv_freq.is_contiguous()):
        raise ValueError("inv_freq must be contiguous fp32")
    if not inv_freq.is_cuda:
        _not_on_gpu("inv_freq")
    axis = None
    if pair_axis is not None:
        if pair_axis.dtype is not torch.uint8 or not pair_axis.is_contiguous() or pair_axis.numel() != pairs:
            raise ValueError("pair_axis must be contiguous uint8, one per pair")
        if not pair_axis.is_cuda:
            _not_on_gpu("pair_axis")
        axis = pair_axis.data_ptr()
    y_dtype = out_dtype or (q_out if q_out is not None else k_out if k_out is not None else ref).dtype
    qp = qs = qop = qos = kp = ks = kop = kos = n_q = n_k = 0
    if q is not None:
        qs = _heads("q", q, None, D)
        n_q, qp = q.shape[1], q.data_ptr()
        if q_out is None:
            q_out, qos = _empty(q.shape, y_dtype, q.device, stream), n_q * D
        else:
            qos = _rope_out("q", q, q_out, y_dtype)
        qop = q_out.data_ptr()
    if k is not None:
        if k.dtype is not dtype or k.shape[0] != T:
            raise ValueError("q and k must agree in type and tokens")
        ks = _heads("k", k, None, D)
        n_k, kp = k.shape[1], k.data_ptr()
        if k_out is None:
            k_out, kos = _empty(k.shape, y_dtype, k.device, stream), n_k * D
        else:
            kos = _rope_out("k", k, k_out, y_dtype)
        kop = k_out.data_ptr()
    flags = (KQ_ROPE_ADJACENT if adjacent else 0) | (KQ_ROPE_INVERSE if inverse else 0)
    _check(lib().kq_rope(_dtype(dtype), _dtype(y_dtype), qp, qs, qop, qos, n_q, kp, ks, kop, kos, n_k, T, D, 2 * pairs,
                         inv_freq.data_ptr(), axis, _i32("pos", pos, axes * T), axes, flags, _stream(stream)))
    return q_out if q is not None else None, k_out if k is not None else None


class _Rope(torch.autograd.Function):
    """rope of tensors that require a gradient: the rotation back by the same angles, on the current stream."""

    @staticmethod
    def forward(ctx, q, k, pos, inv_freq, pair_axis, adjacent, inverse, out_dtype, stream):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(pos, inv_freq, pair_axis)
        ctx.how = adjacent, not inverse, (k if q is None else q).dtype
        outs = rope(q, k, pos, inv_freq, pair_axis, adjacent, inverse, out_dtype, stream=stream)
        ctx.mark_non_differentiable(*(o for o, need in zip(outs, ctx.needs_input_grad) if o is not None and not need))
        return outs

    @staticmethod
    def backward(ctx, gq, gk):
        pos, inv_freq, pair_axis = ctx.saved_tensors
        adjacent, inverse, dtype = ctx.how
        # a gradient may be a view of any strides, an expanded one among them
        gq, gk = (g.contiguous() if g is not None and need else None for g, need in zip((gq, gk), ctx.needs_input_grad))
        if gq is not None or gk is not None:
            gq, gk = rope(gq, gk, pos, inv_freq, pair_axis, adjacent, inverse, dtype)
        return gq, gk, None, None, None, None, None, None, None


def _rope_out(name, x, y, y_dtype) -> int:
    """The token stride of a given output."""
    if y.shape != x.shape or y.dtype is not y_dtype:
        raise ValueError(f"{name}_out must have {name}'s shape, and both outputs one type")
    return _heads(name + "_out", y)


class KV8CacheC(ctypes.Structure):
    """Mirror of kq_kv8_cache (include/kq.h)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_kv", ctypes.c_int), ("head_dim", ctypes.c_int)]


class KV8Cache:
    """One layer's paged 8-bit KV cache: int8 codes k, v (n_pages x n_kv x page_size*head_dim) and fp32
    scales k_scale, v_scale (n_pages x n_kv); layout in include/kq.h."""

    def __init__(self, n_pages: int, page_size: int, n_kv: int, head_dim: int, device="cuda", k=None, v=None,
                 k_scale=None, v_scale=None):
        n = lib().kq_kv8_bytes(n_pages, page_size, n_kv, head_dim)
        if n == 0 and n_pages != 0:
            raise KQError(KQ_ERR_ARG, "bad sizes of a paged 8-bit cache")
        shape = (n_pages, n_kv, page_size * head_dim)
        self.k, self.v = (t if t is not None else torch.empty(shape, dtype=torch.int8, device=device) for t in (k, v))
        self.k_scale, self.v_scale = (t if t is not None else torch.zeros(shape[:2], dtype=torch.float32, device=device)
                                      for t in (k_scale, v_scale))
        for t, dt, want in ((self.k, torch.int8, n), (self.v, torch.int8, n), (self.k_scale, torch.float32, n_pages * n_kv),
                            (self.v_scale, torch.float32, n_pages * n_kv)):
            if t.dtype != dt or not t.is_contiguous() or t.numel() != want:
                raise ValueError("codes must be contiguous int8 and scales contiguous fp32 of the cache's sizes")
        self.n_pages, self.page_size, self.n_kv, self.head_dim = n_pages, page_size, n_kv, head_dim
        self.c = KV8CacheC(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                           n_pages, page_size, n_kv, head_dim)
        self._ref = ctypes.addressof(self.c)
        self._on_gpu = all(t.is_cuda for t in (self.k, self.v, self.k_scale, self.v_scale))


def kv8_append(cache: KV8Cache, k: torch.Tensor, v: torch.Tensor, slot: torch.Tensor, stream=None) -> None:
    """Quantize k and v (T, n_kv, head_dim) into their slots (int32 [T], -1 skips) through kq_kv8_append. Rows of one page
    stand behind one another, with skipped rows between them at most."""
    if k.dtype != v.dtype or k.shape[0] != v.shape[0]:
        raise ValueError("k and v must agree in type and tokens")
    T, x_dtype = k.shape[0], _dtype(k.dtype)
    if not cache._on_gpu:
        _not_on_gpu("the cache")
    _check(lib().kq_kv8_append(cache._ref, x_dtype, k.data_ptr(), _heads("k", k, cache.n_kv, cache.head_dim),
                               v.data_ptr(), _heads("v", v, cache.n_kv, cache.head_dim), _i32("slot", slot, T), T,
                               _stream(stream)))


def attention_kv8_workspace_size(B: int, total_len: int, max_new: int, n_q: int, n_kv: int, head_dim: int) -> int:
    return lib().kq_attention_kv8_workspace_size(B, total_len, max_new, n_q, n_kv, head_dim)


def attention_kv8(q: torch.Tensor, cache: KV8Cache, block_table: torch.Tensor, ctx_len: torch.Tensor,
                  new_len: torch.Tensor, max_new: int, max_len: int, total_len: int | None = None,
                  scale: float | None = None, mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  out_dtype=None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of the packed new tokens' q (T, n_q, head_dim) over the requests' pages (kq_attention_kv8).
    max_new, max_len, total_len (default B * max_len): bounds of new_len, of ctx_len + new_len and of its sum.
    scale: default 1/sqrt(head_dim); mask: int32 [T] tree masks or None (causal). Returns (T, n_q, head_dim), which
    carries no gradient."""
    T, n_q, D = q.shape
    B, width = block_table.shape
    if total_len is None:
        total_len = B * max_len
    if out is None:
        out, out_stride = _empty((T, n_q, D), out_dtype or q.dtype, q.device, stream), n_q * D
    elif out.shape != q.shape or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must have q's shape and out_dtype")
    else:
        out_stride = _heads("out", out, n_q, D)
    if workspace is None:
        need = attention_kv8_workspace_size(B, total_len, max_new, n_q, cache.n_kv, D)
        workspace = _empty(max(need, 256), torch.uint8, q.device, stream)
    elif not workspace.is_cuda:
        _not_on_gpu("workspace")
    if not cache._on_gpu:
        _not_on_gpu("the cache")
    _check(lib().kq_attention_kv8(cache._ref, _dtype(q.dtype), q.data_ptr(), _heads("q", q, None, cache.head_dim),
                                  _dtype(out.dtype), out.data_ptr(), out_stride, n_q,
                                  _i32("ctx_len", ctx_len, B), _i32("new_len", new_len, B), B, T, max_new, max_len,
                                  total_len, _i32("block_table", block_table, B * width), width,
                                  _i32("mask", mask, T) if mask is not None else None,
                                  D ** -0.5 if scale is None else scale, workspace.data_ptr(),
                                  workspace.nbytes, _stream(stream)))
    return out


class KVCacheC(ctypes.Structure):
    """Mirror of kq_kv_cache (include/kq.h)."""
    _fields_ = [("k", ctypes.POINTER(ctypes.c_void_p)), ("v", ctypes.POINTER(ctypes.c_void_p)),
                ("length", ctypes.c_int), ("capacity", ctypes.c_int)]


class KVCache:
    """Per-layer bf16 K and V arrays (capacity x kv_dim device tensors) and the cached length."""

    def __init__(self, n_layers: int, capacity: int, kv_dim: int, device="cuda", k=None, v=None):
        self.k = k if k is not None else [torch.zeros((capacity, kv_dim), dtype=torch.bfloat16, device=device)
                                          for _ in range(n_layers)]
        self.v = v if v is not None else [torch.zeros((capacity, kv_dim), dtype=torch.bfloat16, device=device)
                                          for _ in range(n_layers)]
        self.capacity, self.length = capacity, 0
        n = max(1, n_layers)
        self._ka = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.k])
        self._va = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.v])

    def c(self) -> KVCacheC:
        return KVCacheC(ctypes.cast(self._ka, ctypes.POINTER(ctypes.c_void_p)),
                        ctypes.cast(self._va, ctypes.POINTER(ctypes.c_void_p)), self.length, self.capacity)


class DecodeModel:
    """A dense decoder whose weights are block-quantized device tensors (kq_decode_step).

    layers: list of (w_qkv, w_o, w_gate_up, w_down) uint8 CUDA tensors; head: uint8 CUDA tensor.
    The model struct and pointer arrays are kept alive by this object."""

    def __init__(self, n_layers, hidden, q_dim, kv_dim, head_dim, ffn, vocab, layers, head,
                 layer_fmt="q4_k", head_fmt="q8_0", eps=1e-6):
        self.layers, self.head = layers, head
        n = max(1, n_layers)
        self._arrs = [(ctypes.c_void_p * n)(*[lay[i].data_ptr() for lay in layers]) for i in range(4)]
        self.c = DecodeModelC(n_layers, hidden, q_dim, kv_dim, head_dim, ffn, vocab, _fmt(layer_fmt),
                              _fmt(head_fmt), eps,
                              *[ctypes.cast(a, ctypes.POINTER(ctypes.c_void_p)) for a in self._arrs],
                              head.data_ptr())
        self.hidden, self.vocab = hidden, vocab

    def workspace_size(self, M: int) -> int:
        return lib().kq_decode_workspace_size(ctypes.byref(self.c), M)

    def step(self, x: torch.Tensor, logits: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """logits (M x vocab fp32) for M bf16 token rows x (M x hidden)."""
        M = x.shape[0]
        if logits is None:
            logits = torch.empty((M, self.vocab), dtype=torch.float32, device=x.device)
        if workspace is None:
            workspace = torch.empty(self.workspace_size(M), dtype=torch.uint8, device=x.device)
        _check(lib().kq_decode_step(ctypes.byref(self.c), x.data_ptr(), logits.data_ptr(), M,
                                    workspace.data_ptr(), workspace.numel(), _stream(stream)))
        return logits

    def step_trace(self, x: torch.Tensor, stream=None):
        """kq_decode_step_trace: (logits, trace) where trace holds every op's output as torch
        device tensors: "h0", "x0", and per layer l a dict "layers"[l] with "qkv", "o_in", "y_o",
        "h_mid", "x_mid", "gu", "act", "y_d", "h_out", "x_out" (bf16 fields as int16 bits)."""
        M = x.shape[0]
        c = self.c
        D, Q, KV, F = c.hidden, c.q_dim, c.kv_dim, c.ffn
        logits = torch.empty((M, self.vocab), dtype=torch.float32, device=x.device)
        ws = torch.empty(self.workspace_size(M), dtype=torch.uint8, device=x.device)
        need = lib().kq_decode_trace_size(ctypes.byref(c), M)
        buf = torch.empty(need, dtype=torch.uint8, device=x.device)
        _check(lib().kq_decode_step_trace(ctypes.byref(c), x.data_ptr(), logits.data_ptr(), M, ws.data_ptr(),
                                          ws.numel(), buf.data_ptr(), buf.numel(), _stream(stream)))
        al = lambda n: (n + 255) // 256 * 256
        off = 0

        def take(cols, f32):
            nonlocal off
            nb = M * cols * (4 if f32 else 2)
            t = buf[off:off + nb].view(torch.float32 if f32 else torch.int16).view(M, cols)
            off = al(off + nb)
            return t

        tr = {"h0": take(D, True), "x0": take(D, False), "layers": []}
        for _ in range(c.n_layers):
            tr["layers"].append({"qkv": take(Q + 2 * KV, True), "o_in": take(Q, False), "y_o": take(D, True),
                                 "h_mid": take(D, True), "x_mid": take(D, False), "gu": take(2 * F, True),
                                 "act": take(F, False), "y_d": take(D, True), "h_out": take(D, True),
                                 "x_out": take(D, False)})
        assert off <= need
        return logits, tr

    def attn_workspace_size(self, M: int, L: int) -> int:
        return lib().kq_decode_attn_workspace_size(ctypes.byref(self.c), M, L)

    def step_attn(self, x: torch.Tensor, cache: "KVCache", mask: torch.Tensor | None = None,
                  logits: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
        """kq_decode_step_attn: logits for M bf16 token rows attending to cache.length cached
        positions (the window's k, v are written at rows length..length+M-1; length is not
        advanced here). mask: None (causal) or M int32 words."""
        M = x.shape[0]
        if logits is None:
            logits = torch.empty((M, self.vocab), dtype=torch.float32, device=x.device)
        if workspace is None:
            workspace = torch.empty(self.attn_workspace_size(M, cache.length), dtype=torch.uint8, device=x.device)
        cc = cache.c()
        _check(lib().kq_decode_step_attn(ctypes.byref(self.c), ctypes.byref(cc), x.data_ptr(), logits.data_ptr(), M,
                                         mask.data_ptr() if mask is not None else None, workspace.data_ptr(),
                                         workspace.numel(), _stream(stream)))
        return logits

    def step_static(self, x: torch.Tensor, logits: torch.Tensor, stream=None) -> torch.Tensor:
        """The same step through kq_decode_step_static (library-held scratch, no allocation)."""
        _check(lib().kq_decode_step_static(ctypes.byref(self.c), x.data_ptr(), logits.data_ptr(),
                                           x.shape[0], _stream(stream)))
        return logits
