"""Python binding of the C ABI in include/llama_block.h.

Argument marshalling only: every step of the block runs in the CUDA kernels of
libllama_block.so.  torch is used for device memory and streams; tensors are
passed as raw device pointers.  If the library has not been built the first
call raises: there is no fallback path.
"""
from __future__ import annotations

import array
import ctypes
import os
import threading
from typing import Sequence

__all__ = [
    "F32", "BF16", "X_F32", "Y_F32", "LlamaError", "Dims", "BlockWeights", "lib", "dims_of",
    "llama_rmsnorm", "llama_rope", "llama_gqa_attention", "llama_gqa_attention_decode_noalloc", "llama_swiglu_ffn",
    "llama_block_forward", "llama_stack_decode_step", "llama_workspace_bytes",
    "llama_sample", "llama_embed", "llama_kv_quantize", "llama_gqa_attention_decode_kv8",
    "llama_stack_decode_step_kv8", "llama_stack_decode_step_paged", "llama_gqa_attention_decode_paged",
    "llama_paged_plan", "llama_rope_append_paged", "llama_gqa_attention_chunk_paged", "llama_verify_drafts",
    "llama_rope_append_paged_kv8", "llama_kv_dequantize_paged", "llama_gqa_attention_decode_paged_kv8",
    "llama_beam_select", "llama_beam_reorder_paged", "PagePool",
    "llama_get_device_status", "llama_status_string", "llama_profile_enable", "llama_profile_read",
    "llama_selftest_bounded_wait", "llama_selftest_bounds", "llama_build_info", "BUILD_BOUNDS_CHECKS", "DEBUG_BUILD",
    "OP_RMSNORM", "OP_ROPE", "OP_GQA_ATTENTION", "OP_SWIGLU_FFN", "OP_BLOCK_FORWARD",
    "OP_STACK_DECODE_STEP", "OP_GQA_ATTENTION_CHUNK_PAGED", "OP_VERIFY_DRAFTS",
    "OP_GQA_ATTENTION_DECODE_PAGED_KV8", "OP_BEAM_SELECT", "OP_BEAM_REORDER_PAGED",
]

F32, BF16 = 0, 1
X_F32, Y_F32 = 0x100, 0x200   # residual-stream flags for llama_block_forward's dtype (x fp32, y fp32)
(OP_RMSNORM, OP_ROPE, OP_GQA_ATTENTION, OP_SWIGLU_FFN, OP_BLOCK_FORWARD,
 OP_STACK_DECODE_STEP, OP_GQA_ATTENTION_CHUNK_PAGED, OP_VERIFY_DRAFTS, OP_GQA_ATTENTION_DECODE_PAGED_KV8,
 OP_BEAM_SELECT, OP_BEAM_REORDER_PAGED) = range(11)
STATUS_NAMES = {0: "LLAMA_OK", 1: "LLAMA_ERR_INVALID_ARG", 2: "LLAMA_ERR_UNSUPPORTED",
                3: "LLAMA_ERR_ALIGNMENT", 4: "LLAMA_ERR_WORKSPACE", 5: "LLAMA_ERR_CUDA",
                6: "LLAMA_ERR_TIMEOUT", 7: "LLAMA_ERR_BOUNDS"}

_DIR = os.path.dirname(os.path.abspath(__file__))
# LLAMA_BLOCK_DEBUG=1 selects the bounds-checking build (built by _build.build(debug=True))
DEBUG_BUILD = os.environ.get("LLAMA_BLOCK_DEBUG", "0") not in ("", "0")
LIB_PATH = os.path.join(_DIR, "libllama_block_debug.so" if DEBUG_BUILD else "libllama_block.so")


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("S", ctypes.c_int64), ("d_model", ctypes.c_int64),
                ("n_q", ctypes.c_int64), ("n_kv", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("d_ff", ctypes.c_int64), ("theta_base", ctypes.c_double), ("eps", ctypes.c_double)]


_WEIGHT_FIELDS = ["attn_norm_g", "wq", "wk", "wv", "wo", "ffn_norm_g", "w_gate", "w_up", "w_down"]


class BlockWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _WEIGHT_FIELDS]


class PagePool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("n_layers", ctypes.c_int64), ("parts", ctypes.c_int64),
                ("row_bytes", ctypes.c_int64)]


class LlamaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it was not built (no fallback exists)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
            L = ctypes.CDLL(LIB_PATH)
            vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
            pd = ctypes.POINTER(Dims)
            sig = {
                "llama_rmsnorm": [pd, i32, vp, vp, vp, vp],
                "llama_rope": [pd, i32, vp, vp, i64, vp],
                "llama_gqa_attention": [pd, i32, vp, vp, vp, i64, i64, vp, vp, sz, vp],
                "llama_swiglu_ffn": [pd, i32, vp, vp, vp, vp, vp, vp, sz, vp],
                "llama_block_forward": [pd, i32, ctypes.POINTER(BlockWeights), vp, vp, i64, vp, vp, i64,
                                        vp, sz, vp],
                "llama_stack_decode_step": [pd, i32, i32, ctypes.POINTER(BlockWeights), vp, vp, i64, vp,
                                            vp, vp, i64, i64, vp, vp, sz, vp],
                "llama_get_device_status": [ctypes.POINTER(ctypes.c_int), vp],
                "llama_selftest_bounded_wait": [vp],
                "llama_selftest_bounds": [vp, vp],
                "llama_gqa_attention_decode_noalloc": [pd, i32, vp, vp, vp, i64, i64, vp, vp],
                "llama_sample": [vp, i64, i64, i64, ctypes.c_float, i64, ctypes.c_float, vp, vp, vp],
                "llama_embed": [i32, vp, i64, i64, vp, i64, vp, vp],
                "llama_kv_quantize": [vp, i64, i64, i64, vp, vp, vp],
                "llama_gqa_attention_decode_kv8": [pd, vp, vp, vp, vp, vp, i64, i64, vp, vp, sz, vp],
                "llama_stack_decode_step_kv8": [pd, i32, ctypes.POINTER(BlockWeights), vp, vp, i64, vp, vp, vp, vp,
                                                i64, i64, vp, vp, sz, vp],
                "llama_stack_decode_step_paged": [pd, i32, ctypes.POINTER(BlockWeights), vp, vp, i64, vp, vp, vp,
                                                  i64, vp, i64, vp, i64, vp, vp, sz, vp],
                "llama_gqa_attention_decode_paged": [pd, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, sz, vp],
                "llama_paged_plan": [vp, vp, i64, vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, vp],
                "llama_rope_append_paged": [pd, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp],
                "llama_gqa_attention_chunk_paged": [pd, vp, vp, vp, i64, vp, i64, vp, vp, i64, vp, vp, sz, vp],
                "llama_verify_drafts": [vp, i64, i64, i64, vp, i64, ctypes.c_float, vp, i64, vp, vp, vp, i64, vp, vp,
                                        vp, sz, vp],
                "llama_rope_append_paged_kv8": [pd, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, i64, vp],
                "llama_kv_dequantize_paged": [pd, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp, vp],
                "llama_gqa_attention_decode_paged_kv8": [pd, vp, vp, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, sz, vp],
                "llama_beam_select": [vp, i64, i64, i64, i64, vp, vp, i32, i64, vp, vp, vp, vp, sz, vp],
                "llama_beam_reorder_paged": [vp, i64, i64, vp, vp, vp, vp, i64, vp, i64, i64, ctypes.POINTER(PagePool), i32,
                                             vp, i64, vp, vp, sz, vp],
            }
            for name, args in sig.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = ctypes.c_int
            L.llama_workspace_bytes.argtypes = [i32, pd, i32, i32, i64, i64]
            L.llama_workspace_bytes.restype = sz
            L.llama_profile_enable.argtypes = [i32]
            L.llama_profile_enable.restype = ctypes.c_int
            L.llama_profile_read.argtypes = [i32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_int),
                                             ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int)]
            L.llama_profile_read.restype = ctypes.c_int
            L.llama_build_info.argtypes = []
            L.llama_build_info.restype = ctypes.c_int
            L.llama_status_string.argtypes = [i32]
            L.llama_status_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def dims_of(B, S, d_model, n_q, n_kv, head_dim, d_ff, theta_base, eps) -> Dims:
    return Dims(int(B), int(S), int(d_model), int(n_q), int(n_kv), int(head_dim), int(d_ff),
                float(theta_base), float(eps))


def _d(dims) -> Dims:
    if isinstance(dims, Dims):
        return dims
    if isinstance(dims, Sequence):
        return dims_of(*dims)
    return dims_of(dims.B, dims.S, dims.d_model, dims.n_q, dims.n_kv, dims.head_dim, dims.d_ff,
                   dims.theta_base, dims.eps)


def _p(t) -> int | None:
    """The device address of a tensor (an int passes through as an address).  Every pointer of the
    C ABI is device memory: a tensor that lives on the host is refused here, not handed to a kernel."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"expected a CUDA tensor, got one on {getattr(t, 'device', type(t).__name__)}")
    return t.data_ptr()


def _s(stream) -> int | None:
    if stream is None:   # the address alone: a Stream object costs several times as much
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise LlamaError(rc, where)


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def block_weights(w) -> BlockWeights:
    """BlockWeights from a mapping (or object) holding the nine device tensors.  The struct keeps
    references to the tensors, so their memory stays allocated while the struct is alive (the
    library reads it through the raw pointers)."""
    get = (lambda n: w[n]) if isinstance(w, dict) else (lambda n: getattr(w, n))
    tensors = [get(n) for n in _WEIGHT_FIELDS]
    bw = BlockWeights(*[_p(t) for t in tensors])
    bw._tensors = tensors
    return bw


def llama_rmsnorm(dims, dtype, x, g, y, stream=None):
    _check(lib().llama_rmsnorm(ctypes.byref(_d(dims)), dtype, _p(x), _p(g), _p(y), _s(stream)), "llama_rmsnorm")


def llama_rope(dims, dtype, q, k, pos0=0, stream=None):
    _check(lib().llama_rope(ctypes.byref(_d(dims)), dtype, _p(q), _p(k), int(pos0), _s(stream)), "llama_rope")


def llama_gqa_attention(dims, dtype, q, k, v, kv_capacity, pos0, o, ws=None, stream=None):
    _check(lib().llama_gqa_attention(ctypes.byref(_d(dims)), dtype, _p(q), _p(k), _p(v), int(kv_capacity),
                                     int(pos0), _p(o), _p(ws), _nbytes(ws), _s(stream)), "llama_gqa_attention")


def llama_gqa_attention_decode_noalloc(dims, dtype, q, k, v, kv_capacity, pos0, o, stream=None):
    """One-token attention with the library's own fixed scratch (no workspace argument)."""
    _check(lib().llama_gqa_attention_decode_noalloc(ctypes.byref(_d(dims)), dtype, _p(q), _p(k), _p(v),
                                                    int(kv_capacity), int(pos0), _p(o), _s(stream)),
           "llama_gqa_attention_decode_noalloc")


def llama_swiglu_ffn(dims, dtype, x, w_gate, w_up, w_down, y, ws, stream=None):
    _check(lib().llama_swiglu_ffn(ctypes.byref(_d(dims)), dtype, _p(x), _p(w_gate), _p(w_up), _p(w_down),
                                  _p(y), _p(ws), _nbytes(ws), _s(stream)), "llama_swiglu_ffn")


def llama_block_forward(dims, dtype, weights, x, y, pos0=0, k_cache=None, v_cache=None, cache_capacity=0,
                        ws=None, stream=None):
    w = weights if isinstance(weights, BlockWeights) else block_weights(weights)
    _check(lib().llama_block_forward(ctypes.byref(_d(dims)), dtype, ctypes.byref(w), _p(x), _p(y), int(pos0),
                                     _p(k_cache), _p(v_cache), int(cache_capacity), _p(ws), _nbytes(ws),
                                     _s(stream)), "llama_block_forward")


def llama_stack_decode_step(dims, dtype, layers, final_g, w_lm, vocab, x_emb, k_cache, v_cache, cache_capacity,
                            t_cache, logits, ws, stream=None):
    n = len(layers)
    arr = (BlockWeights * n)(*[lw if isinstance(lw, BlockWeights) else block_weights(lw) for lw in layers])
    _check(lib().llama_stack_decode_step(ctypes.byref(_d(dims)), dtype, n, arr, _p(final_g), _p(w_lm), int(vocab),
                                         _p(x_emb), _p(k_cache), _p(v_cache), int(cache_capacity), int(t_cache),
                                         _p(logits), _p(ws), _nbytes(ws), _s(stream)), "llama_stack_decode_step")


def llama_sample(logits, temperature, top_k, top_p, u, tokens, vocab=None, stream=None):
    """tokens[b] <- the token chosen from logits[b, :vocab] (fp32 [B, ld]) with the uniform u[b]."""
    B = 0 if logits is None else int(logits.shape[0])
    ld = 0 if logits is None else int(logits.stride(0))
    V = int(logits.shape[1]) if vocab is None else int(vocab)
    _check(lib().llama_sample(_p(logits), B, V, ld, float(temperature), int(top_k), float(top_p), _p(u), _p(tokens),
                              _s(stream)), "llama_sample")


def llama_embed(dtype, table, tokens, x, stream=None):
    """x[i] <- table[tokens[i]] (table [vocab, d_model], tokens int32 [n], x [n, d_model])."""
    _check(lib().llama_embed(dtype, _p(table), int(table.shape[0]), int(table.shape[1]), _p(tokens),
                             int(tokens.numel()), _p(x), _s(stream)), "llama_embed")


def llama_kv_quantize(x, scale, codes, stream=None):
    """codes <- E4M3(x / scale[head]) for x bf16 [..., n_kv, head_dim], scale fp32 [n_kv]."""
    n_kv, hd = int(x.shape[-2]), int(x.shape[-1])
    _check(lib().llama_kv_quantize(_p(x), int(x.numel() // (n_kv * hd)), n_kv, hd, _p(scale), _p(codes), _s(stream)),
           "llama_kv_quantize")


def llama_gqa_attention_decode_kv8(dims, q, k, v, k_scale, v_scale, kv_capacity, pos0, o, ws, stream=None):
    _check(lib().llama_gqa_attention_decode_kv8(ctypes.byref(_d(dims)), _p(q), _p(k), _p(v), _p(k_scale),
                                                _p(v_scale), int(kv_capacity), int(pos0), _p(o), _p(ws), _nbytes(ws),
                                                _s(stream)), "llama_gqa_attention_decode_kv8")


def llama_stack_decode_step_kv8(dims, layers, final_g, w_lm, vocab, x_emb, k_cache, v_cache, kv_scales,
                                cache_capacity, t_cache, logits, ws, stream=None):
    n = len(layers)
    arr = (BlockWeights * n)(*[lw if isinstance(lw, BlockWeights) else block_weights(lw) for lw in layers])
    _check(lib().llama_stack_decode_step_kv8(ctypes.byref(_d(dims)), n, arr, _p(final_g), _p(w_lm), int(vocab),
                                             _p(x_emb), _p(k_cache), _p(v_cache), _p(kv_scales), int(cache_capacity),
                                             int(t_cache), _p(logits), _p(ws), _nbytes(ws), _s(stream)),
           "llama_stack_decode_step_kv8")


def llama_stack_decode_step_paged(dims, layers, final_g, w_lm, vocab, x_emb, k_pool, v_pool, block_table, seq_pos,
                                  max_pos, logits, ws, stream=None):
    """k_pool / v_pool [n_layers, n_pages, 128, n_kv, hd] bf16; block_table int32 [B, max_pages]."""
    n = len(layers)
    arr = (BlockWeights * n)(*[lw if isinstance(lw, BlockWeights) else block_weights(lw) for lw in layers])
    _check(lib().llama_stack_decode_step_paged(ctypes.byref(_d(dims)), n, arr, _p(final_g), _p(w_lm), int(vocab),
                                               _p(x_emb), _p(k_pool), _p(v_pool), int(k_pool.shape[1]),
                                               _p(block_table), int(block_table.shape[1]), _p(seq_pos), int(max_pos),
                                               _p(logits), _p(ws), _nbytes(ws), _s(stream)),
           "llama_stack_decode_step_paged")


def llama_gqa_attention_decode_paged(dims, q, k_pool, v_pool, block_table, seq_pos, max_pos, o, ws, stream=None):
    """k_pool / v_pool [n_pages, 128, n_kv, hd] bf16 (one layer); block_table int32 [B, max_pages]."""
    _check(lib().llama_gqa_attention_decode_paged(ctypes.byref(_d(dims)), _p(q), _p(k_pool), _p(v_pool),
                                                  int(k_pool.shape[0]), _p(block_table), int(block_table.shape[1]),
                                                  _p(seq_pos), int(max_pos), _p(o), _p(ws), _nbytes(ws), _s(stream)),
           "llama_gqa_attention_decode_paged")


def _arg(where, name, t, dtype, dev, shape=None):
    """The address of a contiguous tensor of `dtype` (and, when given, `shape`) on device `dev`.  The library
    sees addresses only, so what it would misread is refused here."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or (shape is not None and t.shape != shape):
        _refuse(where, name, t, dtype, dev, shape)
    return t.data_ptr()


def _refuse(where, name, t, dtype, dev, shape):
    if not t.is_cuda:
        raise ValueError(f"{where}: expected a CUDA tensor, got {name} on {t.device}")
    if t.get_device() != dev:
        raise ValueError(f"{where}: {name} is on {t.device}, the current device is cuda:{dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{where}: {name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{where}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{where}: {name} must be contiguous, got strides {t.stride()}")


def _heads(where, name, t, dtype, dev, rows, heads, hd):
    """(address, row stride) of a [rows, heads, hd] view whose rows are contiguous; None, 0 for None."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (rows, heads, hd):
        _refuse(where, name, t, dtype, dev, (rows, heads, hd))
    s0, s1, s2 = t.stride()
    if rows and ((hd > 1 and s2 != 1) or (heads > 1 and s1 != hd)):
        raise ValueError(f"{where}: the rows of {name} must be contiguous, got strides {t.stride()}")
    return t.data_ptr(), s0 if rows > 1 else heads * hd


def _matrix(where, name, t, dtype, dev, rows, width):
    """(address, row stride) of a [rows, >= width] view whose rows are contiguous; None, 0 for None."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.get_device() != dev or t.dim() != 2 or t.shape[0] != rows:
        _refuse(where, name, t, dtype, dev, (rows, max(width, t.shape[-1])))
    s0, s1 = t.stride()
    if t.shape[1] < width or (rows and width > 1 and s1 != 1):
        raise ValueError(f"{where}: the rows of {name} must hold {width} contiguous entries, got shape {tuple(t.shape)} "
                         f"with strides {t.stride()}")
    return t.data_ptr(), s0 if rows > 1 else width


def _scratch(where, ws, dev):
    """(address, bytes) of a workspace: a contiguous tensor of any type on device `dev`; None, 0 for None."""
    if ws is None:
        return None, 0
    return _arg(where, "ws", ws, ws.dtype, dev), ws.numel() * ws.element_size()


def _here(stream):
    """(library, torch, current device, stream address) for one call."""
    import torch
    dev = torch.cuda.current_device()
    st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _s(stream)
    return (_lib if _lib is not None else lib()), torch, dev, st


def llama_paged_plan(n_cached, n_new, free_pages, n_pages, block_table, cu_new, positions, slots, pages_used,
                     stream=None):
    """Extend block_table [B, max_pages] by the pages the new tokens need (from free_pages, in order) and
    fill cu_new [B+1], positions [n_tokens], slots [n_tokens] and pages_used [1]; all int32."""
    w = "llama_paged_plan"
    L, torch, dev, st = _here(stream)
    i32, B, T, P = torch.int32, n_cached.numel(), positions.numel(), block_table.shape[-1]
    _check(L.llama_paged_plan(
        _arg(w, "n_cached", n_cached, i32, dev), _arg(w, "n_new", n_new, i32, dev, (B,)), B,
        _arg(w, "free_pages", free_pages, i32, dev), free_pages.numel(), n_pages,
        _arg(w, "block_table", block_table, i32, dev, (B, P)), P, T, _arg(w, "cu_new", cu_new, i32, dev, (B + 1,)),
        _arg(w, "positions", positions, i32, dev), _arg(w, "slots", slots, i32, dev, (T,)),
        _arg(w, "pages_used", pages_used, i32, dev, (1,)), st), w)


def llama_rope_append_paged(dims, q, k, v, positions, slots, q_out, k_pool, v_pool, stream=None):
    """q_out[t] = R(positions[t]) q[t]; k_pool / v_pool (as [n_pages * 128] rows) at slots[t] <- R k[t], v[t].
    q [S, n_q, hd], k / v [S, n_kv, hd] may be views with a token stride; None, None for q, q_out (append
    only) or for k, v, k_pool, v_pool (rotate only)."""
    w = "llama_rope_append_paged"
    L, torch, dev, st = _here(stream)
    d, i32, bf16 = _d(dims), torch.int32, torch.bfloat16
    S, hd, n_q, n_kv = d.S, d.head_dim, d.n_q, d.n_kv
    qa, qs = _heads(w, "q", q, bf16, dev, S, n_q, hd)
    ka, ks = _heads(w, "k", k, bf16, dev, S, n_kv, hd)
    va, vs = _heads(w, "v", v, bf16, dev, S, n_kv, hd)
    n_pages = 0 if k_pool is None else k_pool.shape[0]
    pool = (n_pages, 128, n_kv, hd)
    _check(L.llama_rope_append_paged(
        ctypes.byref(d), qa, qs, ka, ks, va, vs, _arg(w, "positions", positions, i32, dev, (S,)),
        _arg(w, "slots", slots, i32, dev, (S,)), _arg(w, "q_out", q_out, bf16, dev, (S, n_q, hd)),
        _arg(w, "k_pool", k_pool, bf16, dev, pool), _arg(w, "v_pool", v_pool, bf16, dev, pool), n_pages, st), w)


def llama_gqa_attention_chunk_paged(dims, q, k_pool, v_pool, block_table, cu_new, n_cached, max_pos, o, ws,
                                    stream=None):
    """Packed new tokens q [S, n_q, hd] over k_pool / v_pool [n_pages, 128, n_kv, hd] (one layer): sequence b
    owns rows cu_new[b] .. cu_new[b+1]-1, at positions n_cached[b] onward; o [S, n_q, hd]."""
    w = "llama_gqa_attention_chunk_paged"
    L, torch, dev, st = _here(stream)
    d, i32, bf16 = _d(dims), torch.int32, torch.bfloat16
    B, hd = d.B, d.head_dim
    rows, n_pages, P = (d.S, d.n_q, hd), k_pool.shape[0], block_table.shape[-1]
    pool = (n_pages, 128, d.n_kv, hd)
    _check(L.llama_gqa_attention_chunk_paged(
        ctypes.byref(d), _arg(w, "q", q, bf16, dev, rows), _arg(w, "k_pool", k_pool, bf16, dev, pool),
        _arg(w, "v_pool", v_pool, bf16, dev, pool), n_pages, _arg(w, "block_table", block_table, i32, dev, (B, P)), P,
        _arg(w, "cu_new", cu_new, i32, dev, (B + 1,)), _arg(w, "n_cached", n_cached, i32, dev, (B,)), max_pos,
        _arg(w, "o", o, bf16, dev, rows), *_scratch(w, ws, dev), st), w)


def llama_verify_drafts(logits, draft_logits, temperature, cu_new, tokens, u, noise, n_accepted, out_tokens, ws,
                        vocab=None, stream=None):
    """Accept drafts by rejection sampling: logits / draft_logits fp32 [n_tokens, ld] (draft_logits may be
    None), tokens int32 [n_tokens], u fp32 [n_tokens], noise fp32 [B, ld] exponential draws; fills
    n_accepted int32 [B] and out_tokens int32 [n_tokens]."""
    w = "llama_verify_drafts"
    L, torch, dev, st = _here(stream)
    i32, f32 = torch.int32, torch.float32
    T, B = tokens.numel(), n_accepted.numel()
    V = logits.shape[1] if vocab is None else int(vocab)
    z, ldz = _matrix(w, "logits", logits, f32, dev, T, V)
    y, ldy = _matrix(w, "draft_logits", draft_logits, f32, dev, T, V)
    e, lde = _matrix(w, "noise", noise, f32, dev, B, V)
    _check(L.llama_verify_drafts(
        z, T, V, ldz, y, ldy, temperature, _arg(w, "cu_new", cu_new, i32, dev, (B + 1,)), B,
        _arg(w, "tokens", tokens, i32, dev), _arg(w, "u", u, f32, dev, (T,)), e, lde,
        _arg(w, "n_accepted", n_accepted, i32, dev), _arg(w, "out_tokens", out_tokens, i32, dev, (T,)),
        *_scratch(w, ws, dev), st), w)


def _codes(where, name, t, torch, dev, shape):
    """The address of a contiguous tensor of E4M3 codes: uint8, or torch's float8_e4m3fn."""
    f8 = torch.float8_e4m3fn
    return _arg(where, name, t, f8 if getattr(t, "dtype", None) is f8 else torch.uint8, dev, shape)


def llama_rope_append_paged_kv8(dims, q, k, v, positions, slots, q_out, k_codes, k_scale, v_codes, v_scale, stream=None):
    """llama_rope_append_paged into an 8-bit cache: codes [n_pages, 128, n_kv, hd] (uint8 or float8_e4m3fn) and
    scales fp32 [n_pages, n_kv, 128].  None, None for q, q_out: append only."""
    w = "llama_rope_append_paged_kv8"
    L, torch, dev, st = _here(stream)
    d, i32, bf16, f32 = _d(dims), torch.int32, torch.bfloat16, torch.float32
    S, hd, n_q, n_kv = d.S, d.head_dim, d.n_q, d.n_kv
    qa, qs = _heads(w, "q", q, bf16, dev, S, n_q, hd)
    ka, ks = _heads(w, "k", k, bf16, dev, S, n_kv, hd)
    va, vs = _heads(w, "v", v, bf16, dev, S, n_kv, hd)
    n_pages = k_codes.shape[0]
    pool, rows = (n_pages, 128, n_kv, hd), (n_pages, n_kv, 128)
    _check(L.llama_rope_append_paged_kv8(
        ctypes.byref(d), qa, qs, ka, ks, va, vs, _arg(w, "positions", positions, i32, dev, (S,)),
        _arg(w, "slots", slots, i32, dev, (S,)), _arg(w, "q_out", q_out, bf16, dev, (S, n_q, hd)),
        _codes(w, "k_codes", k_codes, torch, dev, pool), _arg(w, "k_scale", k_scale, f32, dev, rows),
        _codes(w, "v_codes", v_codes, torch, dev, pool), _arg(w, "v_scale", v_scale, f32, dev, rows), n_pages, st), w)


def llama_kv_dequantize_paged(k_codes, k_scale, v_codes, v_scale, block_table, n_pos, k_pool, v_pool, stream=None):
    """Rows 0 .. n_pos[b]-1 of every sequence's pages from codes and scales to bf16 pools [n_pages, 128, n_kv, hd]."""
    w = "llama_kv_dequantize_paged"
    L, torch, dev, st = _here(stream)
    i32, bf16, f32 = torch.int32, torch.bfloat16, torch.float32
    n_pages, _, n_kv, hd = k_pool.shape
    B, P, rows, codes = n_pos.numel(), block_table.shape[-1], (n_pages, n_kv, 128), (n_pages, 128, n_kv, hd)
    d = Dims(B, 0, 0, 0, n_kv, hd, 0, 1.0, 0.0)
    _check(L.llama_kv_dequantize_paged(
        ctypes.byref(d), _codes(w, "k_codes", k_codes, torch, dev, codes), _arg(w, "k_scale", k_scale, f32, dev, rows),
        _codes(w, "v_codes", v_codes, torch, dev, codes), _arg(w, "v_scale", v_scale, f32, dev, rows), n_pages,
        _arg(w, "block_table", block_table, i32, dev, (B, P)), P, _arg(w, "n_pos", n_pos, i32, dev),
        _arg(w, "k_pool", k_pool, bf16, dev, codes), _arg(w, "v_pool", v_pool, bf16, dev, codes), st), w)


def llama_gqa_attention_decode_paged_kv8(dims, q, k_codes, k_scale, v_codes, v_scale, block_table, seq_pos, max_pos, o,
                                         ws, stream=None):
    """One new token per sequence, q [B, n_q, hd], over an 8-bit cache: codes [n_pages, 128, n_kv, hd], scales
    fp32 [n_pages, n_kv, 128]; positions 0 .. seq_pos[b] (-1: none) of sequence b."""
    w = "llama_gqa_attention_decode_paged_kv8"
    L, torch, dev, st = _here(stream)
    d, i32, bf16, f32 = _d(dims), torch.int32, torch.bfloat16, torch.float32
    B, hd, n_kv = d.B, d.head_dim, d.n_kv
    n_pages, P = k_codes.shape[0], block_table.shape[-1]
    pool, rows, heads = (n_pages, 128, n_kv, hd), (n_pages, n_kv, 128), (B, d.n_q, hd)
    _check(L.llama_gqa_attention_decode_paged_kv8(
        ctypes.byref(d), _arg(w, "q", q, bf16, dev, heads), _codes(w, "k_codes", k_codes, torch, dev, pool),
        _arg(w, "k_scale", k_scale, f32, dev, rows), _codes(w, "v_codes", v_codes, torch, dev, pool),
        _arg(w, "v_scale", v_scale, f32, dev, rows), n_pages, _arg(w, "block_table", block_table, i32, dev, (B, P)), P,
        _arg(w, "seq_pos", seq_pos, i32, dev, (B,)), max_pos, _arg(w, "o", o, bf16, dev, heads), *_scratch(w, ws, dev),
        st), w)


def llama_beam_select(logits, scores, finished, pad_token, parents, tokens, out_scores, ws, vocab=None, stream=None):
    """parents, tokens int32 and out_scores fp32 [B, n_out] <- the best continuations of B requests of W beams:
    logits fp32 [B * W, ld], scores fp32 [B, W], finished int32 [B, W] or None."""
    w = "llama_beam_select"
    L, torch, dev, st = _here(stream)
    i32, f32 = torch.int32, torch.float32
    (B, W), kept = scores.shape, parents.shape
    V = logits.shape[1] if vocab is None else int(vocab)
    z, ld = _matrix(w, "logits", logits, f32, dev, B * W, V)
    _check(L.llama_beam_select(
        z, B, W, V, ld, _arg(w, "scores", scores, f32, dev, (B, W)), _arg(w, "finished", finished, i32, dev, (B, W)),
        pad_token, kept[-1], _arg(w, "parents", parents, i32, dev, (B, kept[-1])), _arg(w, "tokens", tokens, i32, dev, kept),
        _arg(w, "out_scores", out_scores, f32, dev, kept), *_scratch(w, ws, dev), st), w)


def _pools(where, name, pools, dev, n_pages, scales, flat):
    """Appends the PagePool records of [n_layers, n_pages, 128, heads, width] tensors, or of scales [n_layers, n_pages,
    parts, 128], to flat (four integers each); the layers' axis may be missing."""
    for t in pools:
        at, s, size = _arg(where, name, t, t.dtype, dev), t.shape, t.element_size()
        k = len(s) - (3 if scales else 4)                # axes before the pages' own
        if scales and 0 <= k <= 1 and s[k] == n_pages and s[-1] == 128:
            flat += (at, s[0] if k else 1, s[-2], size)
        elif not scales and 0 <= k <= 1 and s[k] == n_pages and s[k + 1] == 128:
            flat += (at, s[0] if k else 1, 1, s[-2] * s[-1] * size)
        else:
            raise ValueError(f"{where}: {name} must be [n_layers, {n_pages}, " +
                             (f"parts, 128], got {tuple(s)}" if scales else f"128, heads, width], got {tuple(s)}"))


def llama_beam_reorder_paged(parents, n_cached, n_cached_out, block_table, block_table_out, free_pages, n_pages, kv_pools,
                             scale_pools, freed_pages, counts, ws, stream=None):
    """The paged cache follows parents int32 [B, W]: n_cached [B * W] and block_table [B * W, max_pages] to their _out
    tensors (which may be the same), open pages copied in every pool.  kv_pools: tensors [n_layers, n_pages, 128, n_kv, hd]
    (or without the first axis); scale_pools: [n_layers, n_pages, n_kv, 128], or ()."""
    w = "llama_beam_reorder_paged"
    L, torch, dev, st = _here(stream)
    i32 = torch.int32
    B, W = parents.shape
    P = block_table.shape[-1]
    flat = []
    _pools(w, "kv_pools", kv_pools, dev, n_pages, False, flat)
    _pools(w, "scale_pools", scale_pools, dev, n_pages, True, flat)
    n = len(flat) // 4
    records = (PagePool * n).from_buffer(array.array("q", flat)) if n else None   # one object, not one per record
    _check(L.llama_beam_reorder_paged(
        _arg(w, "parents", parents, i32, dev), B, W, _arg(w, "n_cached", n_cached, i32, dev, (B * W,)),
        _arg(w, "n_cached_out", n_cached_out, i32, dev, (B * W,)), _arg(w, "block_table", block_table, i32, dev, (B * W, P)),
        _arg(w, "block_table_out", block_table_out, i32, dev, (B * W, P)), P, _arg(w, "free_pages", free_pages, i32, dev),
        free_pages.numel(), n_pages, records, n, _arg(w, "freed_pages", freed_pages, i32, dev), freed_pages.numel(),
        _arg(w, "counts", counts, i32, dev, (2,)), *_scratch(w, ws, dev), st), w)


def llama_workspace_bytes(op, dims, dtype, n_layers=0, vocab=0, kv_capacity=0) -> int:
    return int(lib().llama_workspace_bytes(int(op), ctypes.byref(_d(dims)), dtype, int(n_layers), int(vocab),
                                           int(kv_capacity)))


def llama_get_device_status(stream=None) -> int:
    out = ctypes.c_int(-1)
    _check(lib().llama_get_device_status(ctypes.byref(out), _s(stream)), "llama_get_device_status")
    return out.value


def llama_selftest_bounded_wait(stream=None) -> None:
    """Launch the kernel whose bounded waits run out on purpose (the device status word then holds
    LLAMA_ERR_TIMEOUT; read it with llama_get_device_status)."""
    _check(lib().llama_selftest_bounded_wait(_s(stream)), "llama_selftest_bounded_wait")


def llama_selftest_bounds(scratch, stream=None) -> None:
    """Store through the checked path to element 40 of `scratch` (64 fp32) declared 32 long: a
    bounds-checking build skips it and latches LLAMA_ERR_BOUNDS, a release build performs it."""
    _check(lib().llama_selftest_bounds(_p(scratch), _s(stream)), "llama_selftest_bounds")


def llama_build_info() -> int:
    """Bit 1 (LLAMA_BUILD_BOUNDS_CHECKS): the loaded library checks bounds (-DLLAMA_DEBUG)."""
    return int(lib().llama_build_info())


BUILD_BOUNDS_CHECKS = 1


def llama_profile_enable(on: bool = True) -> None:
    _check(lib().llama_profile_enable(1 if on else 0), "llama_profile_enable")


def llama_profile_read(max_kinds: int = 32) -> dict:
    """{kernel role: (launches, total_ms)} for the launches recorded since the last read."""
    names = (ctypes.c_char_p * max_kinds)()
    launches = (ctypes.c_int * max_kinds)()
    ms = (ctypes.c_double * max_kinds)()
    n = ctypes.c_int(0)
    _check(lib().llama_profile_read(max_kinds, names, launches, ms, ctypes.byref(n)), "llama_profile_read")
    return {names[i].decode(): (launches[i], ms[i]) for i in range(n.value)}


def llama_status_string(status: int) -> str:
    return lib().llama_status_string(int(status)).decode()
