"""GB300-native speculative-decoding verify attention.

Thin ctypes binding over the C ABI of ``libverify_attn.so`` (declared in
``include/verify_attn.h``): every function here only marshals torch tensors into pointers and
sizes and calls the entry point of the same name; all the work runs in the library's CUDA
kernels.  There is no CPU fallback: if the compiled library is missing, every call raises.

Source: IQuestRT technical report, sections "Read only the KV tiles needed by the current
positions" and "Expose more parallelism in attention".
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "VerifyAttnError", "lib", "lib_path", "kv_ring_append", "verify_attn_full", "verify_attn_swa",
    "attn_split_combine", "verify_attn_tree", "verify_attn_full_noalloc", "va_sample_workspace_bytes",
    "va_sample_topk_topp", "va_accept_chain", "va_tree_accept_settle", "kv_ring_append_q8", "verify_attn_q8",
    "verify_attn_q8_tree", "verify_attn_q8_step", "verify_attn_step", "va_selftest_bounded_wait", "SAMPLE_MAX_K", "SAMPLE_TILE",
    "SAMPLE_MAX_VOCAB", "NOALLOC_MAX_SPLITS", "va_workspace_bytes", "va_auto_splits", "va_auto_splits_for", "va_status_string",
    "kv_page_append_b8", "verify_attn_paged_b8", "va_paged_workspace_bytes", "kv_page_extend", "kv_page_reorder",
    "kv_page_copy", "kv_page_compact", "va_page_ops_workspace_bytes", "va_beam_select", "va_beam_workspace_bytes",
    "PAGED_MAX_SEQS", "B8_BLOCK", "HEAD_DIM", "Q_HEADS", "MAX_ROWS", "TILE", "MAX_SPLITS", "MAX_TREE_NODES", "EXPORTS",
    "VA_OK", "VA_INVALID_ARG", "VA_UNSUPPORTED", "VA_RING_TOO_SMALL", "VA_CUDA_ERROR",
]

HEAD_DIM, Q_HEADS, MAX_ROWS, TILE, MAX_SPLITS, MAX_TREE_NODES = 128, 6, 8, 64, 4096, 16
VA_OK, VA_INVALID_ARG, VA_UNSUPPORTED, VA_RING_TOO_SMALL, VA_CUDA_ERROR = 0, 1, 2, 3, 4
EXPORTS = ("kv_ring_append", "verify_attn_full", "verify_attn_swa", "verify_attn_tree", "attn_split_combine",
           "va_workspace_bytes", "va_auto_splits", "va_auto_splits_for", "va_status_string",
           "verify_attn_full_noalloc", "va_sample_workspace_bytes", "va_sample_topk_topp", "va_accept_chain",
           "va_tree_accept_settle", "kv_ring_append_q8", "verify_attn_q8", "verify_attn_q8_tree", "verify_attn_q8_step",
           "verify_attn_step", "va_selftest_bounded_wait", "kv_page_append_b8", "verify_attn_paged_b8",
           "va_paged_workspace_bytes", "kv_page_extend", "kv_page_reorder", "kv_page_copy", "kv_page_compact",
           "va_page_ops_workspace_bytes", "va_beam_select", "va_beam_workspace_bytes")
NOALLOC_MAX_SPLITS = 160
SAMPLE_MAX_K, SAMPLE_TILE, SAMPLE_MAX_VOCAB = 32, 8192, 262144
PAGED_MAX_SEQS, B8_BLOCK = 1024, 16
B8_E4M3, B8_INT8 = 0, 1

_PKG = os.path.dirname(os.path.abspath(__file__))
_lib = {}
_lock = threading.Lock()


class VerifyAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {va_status_string(status)} ({status})")


def lib_path(variant: str = "") -> str:
    return os.path.join(_PKG, "_build", f"libverify_attn{variant}.so")


def lib(variant: str = "") -> ctypes.CDLL:
    """The loaded CUDA library (built by ``speculative_decode_verify_gb300.build``)."""
    if variant in _lib:
        return _lib[variant]
    with _lock:
        if variant in _lib:
            return _lib[variant]
        path = lib_path(variant)
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library not built ({path}); run speculative_decode_verify_gb300.build.build()")
        L = ctypes.CDLL(path)
        p, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.kv_ring_append.argtypes = [p, p, i, p, p, i, p, p, p]
        L.verify_attn_full.argtypes = [p, i, i, p, p, i, p, f, i, p, p, ctypes.POINTER(i), p, p]
        L.verify_attn_swa.argtypes = [p, i, i, p, p, i, i, p, f, i, p, p, ctypes.POINTER(i), p, p]
        L.verify_attn_tree.argtypes = [p, i, i, p, p, i, i, p, f, i, p, p, ctypes.POINTER(i), p, p]
        L.attn_split_combine.argtypes = [p, p, i, p, i, i, p, p, p]
        L.verify_attn_full_noalloc.argtypes = [p, i, i, p, p, i, p, f, i, p, p, p, ctypes.POINTER(i), p, p]
        for fn in ("kv_ring_append", "verify_attn_full", "verify_attn_swa", "verify_attn_tree",
                   "attn_split_combine", "verify_attn_full_noalloc"):
            getattr(L, fn).restype = i
        L.va_sample_workspace_bytes.argtypes = [i, i, i]
        L.va_sample_workspace_bytes.restype = ctypes.c_size_t
        L.va_sample_topk_topp.argtypes = [p, i, i, i, f, f, p, p, p, p, p, p, ctypes.c_size_t, p]
        L.va_accept_chain.argtypes = [p, p, p, p, p, p, i, p, p, i, p, p, p, p, p, p, p]
        L.va_tree_accept_settle.argtypes = [p, p, i, p, i, p, p, p, p, p, p, p, p]
        L.kv_ring_append_q8.argtypes = [p, p, i, p, p, p, p, i, p, p, p]
        L.verify_attn_q8.argtypes = [p, i, i, p, p, p, p, i, i, p, f, i, p, p, ctypes.POINTER(i), p, p]
        L.verify_attn_q8_tree.argtypes = [p, i, i, p, p, p, p, i, i, p, f, i, p, p, ctypes.POINTER(i), p, p]
        L.verify_attn_q8_step.argtypes = [p, p, p, i, i, p, p, p, p, i, i, p, p, f, i, p, p, p, ctypes.POINTER(i),
                                          p, p]
        for fn in ("va_sample_topk_topp", "va_accept_chain", "va_tree_accept_settle", "kv_ring_append_q8",
                   "verify_attn_q8", "verify_attn_q8_tree", "verify_attn_q8_step"):
            getattr(L, fn).restype = i
        L.verify_attn_step.argtypes = [p, p, p, i, i, p, p, i, i, p, p, f, i, p, p, p, ctypes.POINTER(i), p, p]
        L.verify_attn_step.restype = i
        L.va_selftest_bounded_wait.argtypes = [ctypes.c_ulonglong, ctypes.c_ulonglong, p, p, p]
        L.va_selftest_bounded_wait.restype = i
        z = ctypes.c_size_t
        L.kv_page_append_b8.argtypes = [p, p, i, i, i, p, p, p, i, p, p, p, p, i, i, p, p]
        L.verify_attn_paged_b8.argtypes = [p, i, i, i, i, p, p, p, i, p, p, p, p, i, i, i, f, p, p, z, p, p, p, p]
        L.kv_page_extend.argtypes = [p, p, p, i, i, p, i, i, i, p, p, p, p, p, z, p, p]
        L.kv_page_reorder.argtypes = [p, p, i, i, p, i, p, i, p, p]
        L.kv_page_copy.argtypes = [p, p, i, i, i, i, p, p, p, p, p, p]
        L.kv_page_compact.argtypes = [p, i, i, p, i, i, i, p, p, p, p, p, p, p, z, p, p]
        L.va_beam_select.argtypes = [p, i, ctypes.c_int64, i, i, i, p, p, i, i, p, p, p, p, z, p]
        for fn in ("kv_page_append_b8", "verify_attn_paged_b8", "kv_page_extend", "kv_page_reorder", "kv_page_copy",
                   "kv_page_compact", "va_beam_select"):
            getattr(L, fn).restype = i
        L.va_paged_workspace_bytes.argtypes = [i, i, i, i]
        L.va_page_ops_workspace_bytes.argtypes = [i, i, i]
        L.va_beam_workspace_bytes.argtypes = [i, i, i, i]
        for fn in ("va_paged_workspace_bytes", "va_page_ops_workspace_bytes", "va_beam_workspace_bytes"):
            getattr(L, fn).restype = z
        L.va_workspace_bytes.argtypes = [i]
        L.va_workspace_bytes.restype = ctypes.c_size_t
        L.va_auto_splits.argtypes = [i, i]
        L.va_auto_splits.restype = i
        L.va_auto_splits_for.argtypes = [i, i, i]
        L.va_auto_splits_for.restype = i
        L.va_status_string.argtypes = [i]
        L.va_status_string.restype = ctypes.c_char_p
        _lib[variant] = L
        return L


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn: str, status: int) -> None:
    if status != VA_OK:
        raise VerifyAttnError(fn, status)


def va_status_string(status: int) -> str:
    return lib().va_status_string(int(status)).decode()


def va_workspace_bytes(n_splits: int) -> int:
    return int(lib().va_workspace_bytes(int(n_splits)))


def verify_attn_step(q, k_new, v_new, n_live: int, k_cache, v_cache, pos, scale: float, sink, workspace, out,
                     out_lse=None, window: int = 0, n_splits: int = 0, dev_status=None, stream=None,
                     variant: str = "") -> int:
    """One whole verify call (append + split attention + combine, two launches); returns the split count.
    workspace: float32 device tensor of at least va_workspace_bytes(n_splits) bytes (the partials)."""
    used = ctypes.c_int(0)
    st = lib(variant).verify_attn_step(_ptr(q), _ptr(k_new), _ptr(v_new), int(q.shape[0]), int(n_live),
                                       _ptr(k_cache), _ptr(v_cache), int(k_cache.shape[0]), int(window), _ptr(pos),
                                       _ptr(sink), float(scale), int(n_splits), _ptr(workspace), _ptr(out),
                                       _ptr(out_lse), ctypes.byref(used), _ptr(dev_status), _stream(stream))
    _check("verify_attn_step", st)
    return used.value


def va_auto_splits(extent_hint: int, window: int = 0) -> int:
    return int(lib().va_auto_splits(int(extent_hint), int(window)))


def va_auto_splits_for(extent_hint: int, window: int, sm_count: int) -> int:
    return int(lib().va_auto_splits_for(int(extent_hint), int(window), int(sm_count)))


def kv_ring_append(k_new, v_new, n_live: int, k_cache, v_cache, pos, dev_status=None, stream=None,
                   variant: str = "") -> None:
    """Write the live rows' K/V ([n_live,128] bf16) to slot pos[r] mod slots of the cache."""
    st = lib(variant).kv_ring_append(_ptr(k_new), _ptr(v_new), int(n_live), _ptr(k_cache), _ptr(v_cache),
                                     int(k_cache.shape[0]), _ptr(pos), _ptr(dev_status), _stream(stream))
    _check("kv_ring_append", st)


def verify_attn_full(q, n_live: int, k_cache, v_cache, pos, scale: float, part_o, part_lse,
                     n_splits: int = 0, dev_status=None, stream=None, variant: str = "") -> int:
    """Split-KV attention of a full-attention layer; returns the split count launched."""
    used = ctypes.c_int(0)
    st = lib(variant).verify_attn_full(_ptr(q), int(q.shape[0]), int(n_live), _ptr(k_cache), _ptr(v_cache),
                                       int(k_cache.shape[0]), _ptr(pos), float(scale), int(n_splits),
                                       _ptr(part_o), _ptr(part_lse), ctypes.byref(used), _ptr(dev_status),
                                       _stream(stream))
    _check("verify_attn_full", st)
    return used.value


def verify_attn_swa(q, n_live: int, k_ring, v_ring, window: int, pos, scale: float, part_o, part_lse,
                    n_splits: int = 0, dev_status=None, stream=None, variant: str = "") -> int:
    """Split-KV attention of a sliding-window layer read from its ring; returns the split count."""
    used = ctypes.c_int(0)
    st = lib(variant).verify_attn_swa(_ptr(q), int(q.shape[0]), int(n_live), _ptr(k_ring), _ptr(v_ring),
                                      int(k_ring.shape[0]), int(window), _ptr(pos), float(scale), int(n_splits),
                                      _ptr(part_o), _ptr(part_lse), ctypes.byref(used), _ptr(dev_status),
                                      _stream(stream))
    _check("verify_attn_swa", st)
    return used.value


def verify_attn_tree(q, n_nodes: int, k_cache, v_cache, tree, scale: float, part_o, part_lse, window: int = 0,
                     n_splits: int = 0, dev_status=None, stream=None, variant: str = "") -> int:
    """Split-KV attention of a draft tree (``tree`` = device int32 [1 + n_nodes]: base, then each node's
    ancestor-or-self mask) over a full cache (window 0) or a ring; returns the split count."""
    used = ctypes.c_int(0)
    st = lib(variant).verify_attn_tree(_ptr(q), int(q.shape[0]), int(n_nodes), _ptr(k_cache), _ptr(v_cache),
                                       int(k_cache.shape[0]), int(window), _ptr(tree), float(scale), int(n_splits),
                                       _ptr(part_o), _ptr(part_lse), ctypes.byref(used), _ptr(dev_status),
                                       _stream(stream))
    _check("verify_attn_tree", st)
    return used.value


def attn_split_combine(part_o, part_lse, n_splits: int, sink, n_live: int, out, out_lse=None, stream=None,
                       variant: str = "") -> None:
    """Log-sum-exp merge of the partials with the sink; writes bf16 ``out`` [n_rows,6,128]."""
    st = lib(variant).attn_split_combine(_ptr(part_o), _ptr(part_lse), int(n_splits), _ptr(sink),
                                         int(out.shape[0]), int(n_live), _ptr(out), _ptr(out_lse),
                                         _stream(stream))
    _check("attn_split_combine", st)


def verify_attn_full_noalloc(q, n_live: int, k_cache, v_cache, pos, scale: float, sink, out, out_lse=None,
                             n_splits: int = 0, dev_status=None, stream=None, variant: str = "") -> int:
    """Full-attention verify call plus combine with the partials in the library's own fixed device
    buffer (for callers that cannot allocate); returns the split count launched."""
    used = ctypes.c_int(0)
    st = lib(variant).verify_attn_full_noalloc(_ptr(q), int(q.shape[0]), int(n_live), _ptr(k_cache), _ptr(v_cache),
                                               int(k_cache.shape[0]), _ptr(pos), float(scale), int(n_splits),
                                               _ptr(sink), _ptr(out), _ptr(out_lse), ctypes.byref(used),
                                               _ptr(dev_status), _stream(stream))
    _check("verify_attn_full_noalloc", st)
    return used.value


# ----------------------------------------------------------------------------- after verification
def va_sample_workspace_bytes(n_rows: int, vocab: int, top_k: int) -> int:
    return int(lib().va_sample_workspace_bytes(int(n_rows), int(vocab), int(top_k)))


def va_sample_topk_topp(logits, top_k: int, top_p: float, temperature: float, u, ids, probs, counts, tokens,
                        workspace, stream=None, variant: str = "") -> None:
    """Top-k / temperature / top-p sampling of logits [n_rows, vocab] (float32, device); writes ids/probs
    [n_rows, top_k], counts and tokens [n_rows].  ``workspace``: a device byte tensor of at least
    va_sample_workspace_bytes(n_rows, vocab, top_k) bytes."""
    n_rows, vocab = int(logits.shape[0]), int(logits.shape[1])
    st = lib(variant).va_sample_topk_topp(_ptr(logits), n_rows, vocab, int(top_k), float(top_p), float(temperature),
                                          _ptr(u), _ptr(ids), _ptr(probs), _ptr(counts), _ptr(tokens), _ptr(workspace),
                                          int(workspace.numel() * workspace.element_size()), _stream(stream))
    _check("va_sample_topk_topp", st)


def va_accept_chain(p_ids, p_probs, p_counts, q_ids, q_probs, q_counts, drafts, target_tokens, n_drafts: int,
                    u_accept, u_replace, pos, n_accepted, out_tokens, next_pos=None, stream=None,
                    variant: str = "") -> None:
    """Rejection-sampling acceptance of a chain of n_drafts drafts (all tensors on the device)."""
    st = lib(variant).va_accept_chain(_ptr(p_ids), _ptr(p_probs), _ptr(p_counts), _ptr(q_ids), _ptr(q_probs),
                                      _ptr(q_counts), int(p_ids.shape[1]), _ptr(drafts), _ptr(target_tokens),
                                      int(n_drafts), _ptr(u_accept), _ptr(u_replace), _ptr(pos), _ptr(n_accepted),
                                      _ptr(out_tokens), _ptr(next_pos), _stream(stream))
    _check("va_accept_chain", st)


def va_tree_accept_settle(k_cache, v_cache, tree, n_nodes: int, node_tokens, target_tokens, path, emitted,
                          n_accepted, next_pos=None, dev_status=None, stream=None, variant: str = "") -> None:
    """Accept a draft tree's path and move its K/V to consecutive positions (k/v_cache may be None)."""
    slots = int(k_cache.shape[0]) if k_cache is not None else 0
    st = lib(variant).va_tree_accept_settle(_ptr(k_cache), _ptr(v_cache), slots, _ptr(tree), int(n_nodes),
                                            _ptr(node_tokens), _ptr(target_tokens), _ptr(path), _ptr(emitted),
                                            _ptr(n_accepted), _ptr(next_pos), _ptr(dev_status), _stream(stream))
    _check("va_tree_accept_settle", st)


# ----------------------------------------------------------------------------- quantised K/V cache
def kv_ring_append_q8(k_new, v_new, n_live: int, k_codes, v_codes, k_scale, v_scale, pos, dev_status=None,
                      stream=None, variant: str = "") -> None:
    """Encode the live rows' K/V ([n_live,128] bf16) into the quantised cache at slot pos[r] mod slots."""
    st = lib(variant).kv_ring_append_q8(_ptr(k_new), _ptr(v_new), int(n_live), _ptr(k_codes), _ptr(v_codes),
                                        _ptr(k_scale), _ptr(v_scale), int(k_codes.shape[0]), _ptr(pos),
                                        _ptr(dev_status), _stream(stream))
    _check("kv_ring_append_q8", st)


def verify_attn_q8(q, n_live: int, k_codes, v_codes, k_scale, v_scale, pos, scale: float, part_o, part_lse,
                   window: int = 0, n_splits: int = 0, dev_status=None, stream=None, variant: str = "") -> int:
    """Split-KV verify attention over the quantised cache (window 0: full attention); returns the split count."""
    used = ctypes.c_int(0)
    st = lib(variant).verify_attn_q8(_ptr(q), int(q.shape[0]), int(n_live), _ptr(k_codes), _ptr(v_codes),
                                     _ptr(k_scale), _ptr(v_scale), int(k_codes.shape[0]), int(window), _ptr(pos),
                                     float(scale), int(n_splits), _ptr(part_o), _ptr(part_lse), ctypes.byref(used),
                                     _ptr(dev_status), _stream(stream))
    _check("verify_attn_q8", st)
    return used.value


def verify_attn_q8_tree(q, n_nodes: int, k_codes, v_codes, k_scale, v_scale, tree, scale: float, part_o, part_lse,
                        window: int = 0, n_splits: int = 0, dev_status=None, stream=None, variant: str = "") -> int:
    """Tree verify attention over the quantised cache (``tree`` = [base, masks...] int32 on the device, as for
    verify_attn_tree); returns the split count."""
    used = ctypes.c_int(0)
    st = lib(variant).verify_attn_q8_tree(_ptr(q), int(q.shape[0]), int(n_nodes), _ptr(k_codes), _ptr(v_codes),
                                          _ptr(k_scale), _ptr(v_scale), int(k_codes.shape[0]), int(window),
                                          _ptr(tree), float(scale), int(n_splits), _ptr(part_o), _ptr(part_lse),
                                          ctypes.byref(used), _ptr(dev_status), _stream(stream))
    _check("verify_attn_q8_tree", st)
    return used.value


def verify_attn_q8_step(q, k_new, v_new, n_live: int, k_codes, v_codes, k_scale, v_scale, pos, scale: float, sink,
                        workspace, out, out_lse=None, window: int = 0, n_splits: int = 0, dev_status=None,
                        stream=None, variant: str = "") -> int:
    """A whole verify call over the quantised cache (encoding append inside the attention launch, then the
    combine); returns the split count."""
    used = ctypes.c_int(0)
    st = lib(variant).verify_attn_q8_step(_ptr(q), _ptr(k_new), _ptr(v_new), int(q.shape[0]), int(n_live),
                                          _ptr(k_codes), _ptr(v_codes), _ptr(k_scale), _ptr(v_scale),
                                          int(k_codes.shape[0]), int(window), _ptr(pos), _ptr(sink), float(scale),
                                          int(n_splits), _ptr(workspace), _ptr(out), _ptr(out_lse),
                                          ctypes.byref(used), _ptr(dev_status), _stream(stream))
    _check("verify_attn_q8_step", st)
    return used.value


# ----------------------------------------------------------------------------- paged 8-bit cache of many sequences
# (these calls are made many times a step: the checks below look at each tensor once and do little else)
def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


_torch = None
_KINDS = {}      # what the tensors of a call may hold


def _import_torch():
    global _torch
    if _torch is None:
        import torch
        _KINDS.update({"int32": (torch.int32,), "float32": (torch.float32,),
                       "bfloat16": (torch.bfloat16, torch.int16, torch.uint16),      # or their bit patterns
                       "8-bit codes": (torch.int8, torch.uint8, torch.float8_e4m3fn)})
        _torch = torch
    return _torch


def _at(t, count: int, kind: str, index: int, what: str) -> int:
    """Address of a dense tensor of `count` elements on GPU `index` (the C ABI takes no strides)."""
    if t.dtype not in _KINDS[kind] or t.numel() != count or not t.is_contiguous() or t.get_device() != index:
        where = f"on cuda:{index}" if index >= 0 else "on a GPU"
        raise ValueError(f"{what}: a contiguous tensor of {count} elements, {kind}, {where}")
    return t.data_ptr()


def _bytes(t, index: int):
    if not t.is_contiguous() or t.get_device() != index:
        raise ValueError("the workspace: a contiguous tensor on the other tensors' GPU")
    return t.data_ptr(), t.numel() * t.itemsize


def _opt(t, count: int, kind: str, index: int, what: str):
    return None if t is None else _at(t, count, kind, index, what)


def _launch(fn: str, call, index: int, stream, *args) -> None:
    """Call an entry point on the stream given, or on the current one of GPU `index`, with that device current."""
    if index < 0:
        raise ValueError(f"{fn}: the tensors have to be on a GPU")
    torch = _torch
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            status = call(*args, _stream(stream))
    elif stream is None:
        status = call(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        status = call(*args, _stream(stream))
    if status != VA_OK:
        raise VerifyAttnError(fn, status)


def _pool(k_codes, v_codes, k_scale, v_scale):
    """(layers, pages, kv heads, format, GPU, four addresses) of pools [pages, heads, 64, 128] or [layers, pages, ...]."""
    torch = _torch or _import_torch()
    shape, kind, index = k_codes.shape, k_codes.dtype, k_codes.get_device()
    n = k_codes.numel()
    if not (4 <= len(shape) <= 5 and shape[-1] == HEAD_DIM and shape[-2] == TILE and v_codes.dtype is kind
            and v_codes.shape == shape and k_scale.shape[-1] == TILE // B8_BLOCK):
        raise ValueError("pools are codes [..., pages, heads, 64, 128] of one 8-bit type and scales [..., pages, heads, 4]")
    scales = n // (HEAD_DIM * B8_BLOCK)
    return (shape[0] if len(shape) == 5 else 1, shape[-4], shape[-3], B8_INT8 if kind is torch.int8 else B8_E4M3, index,
            _at(k_codes, n, "8-bit codes", index, "k_codes (int8, float8_e4m3fn or its bits in uint8)"),
            _at(v_codes, n, "8-bit codes", index, "v_codes"), _at(k_scale, scales, "float32", index, "k_scale"),
            _at(v_scale, scales, "float32", index, "v_scale"))


def _table(table, n: int, index: int):
    if table.dim() != 2 or table.shape[0] != n:
        raise ValueError("the table is int32 [n_seqs, max_pages]")
    width = table.shape[1]
    return width, _at(table, n * width, "int32", index, "the table")


def kv_page_append_b8(k_new, v_new, n_live, lens, table, k_codes, v_codes, k_scale, v_scale, dev_status=None,
                      stream=None, variant: str = "") -> None:
    """Code the live rows' K/V ([n_seqs, n_rows, n_kv_heads, 128] bf16) into the sequences' pages.  The pool's
    format goes by its dtype: int8, or E4M3 (float8_e4m3fn or uint8)."""
    layers, pages, heads, fmt, dev, kc, vc, ks, vs = _pool(k_codes, v_codes, k_scale, v_scale)
    n, rows, h, d = k_new.shape
    _need(layers == 1 and h == heads and d == HEAD_DIM and v_new.shape == k_new.shape,
          "new rows are [n_seqs, n_rows, n_kv_heads, 128], the pool one layer's")
    width, tb = _table(table, n, dev)
    count = n * rows * heads * HEAD_DIM
    _launch("kv_page_append_b8", lib(variant).kv_page_append_b8, dev, stream, _at(k_new, count, "bfloat16", dev, "k_new"),
            _at(v_new, count, "bfloat16", dev, "v_new"), n, rows, heads, _at(n_live, n, "int32", dev, "n_live"),
            _at(lens, n, "int32", dev, "lens"), tb, width, kc, vc, ks, vs, pages, fmt,
            _opt(dev_status, 1, "int32", dev, "dev_status"))


def va_paged_workspace_bytes(n_seqs: int, n_rows: int, n_kv_heads: int, group: int) -> int:
    return int(lib().va_paged_workspace_bytes(int(n_seqs), int(n_rows), int(n_kv_heads), int(group)))


def verify_attn_paged_b8(q, n_live, lens, table, k_codes, v_codes, k_scale, v_scale, scale: float, sink, workspace, out,
                         out_lse=None, window: int = 0, dev_status=None, stream=None, variant: str = "") -> None:
    """Verify attention of every sequence's live rows (q [n_seqs, n_rows, heads, 128] bf16) over its pages; writes
    out (as q) and out_lse [n_seqs, n_rows, heads].  ``workspace``: a device byte tensor of
    va_paged_workspace_bytes(...) bytes."""
    layers, pages, kv, fmt, dev, kc, vc, ks, vs = _pool(k_codes, v_codes, k_scale, v_scale)
    n, rows, heads, d = q.shape
    _need(layers == 1 and d == HEAD_DIM and heads % kv == 0 and out.shape == q.shape,
          "q and out are [n_seqs, n_rows, n_kv_heads * group, 128], the pool one layer's")
    width, tb = _table(table, n, dev)
    pairs = n * rows * heads
    ws, size = _bytes(workspace, dev)
    _launch("verify_attn_paged_b8", lib(variant).verify_attn_paged_b8, dev, stream,
            _at(q, pairs * HEAD_DIM, "bfloat16", dev, "q"), n, rows, kv, heads // kv, _at(n_live, n, "int32", dev, "n_live"),
            _at(lens, n, "int32", dev, "lens"), tb, width, kc, vc, ks, vs, pages, fmt, int(window), float(scale),
            _opt(sink, heads, "float32", dev, "sink"), ws, size, _at(out, pairs * HEAD_DIM, "bfloat16", dev, "out"),
            _opt(out_lse, pairs, "float32", dev, "out_lse"), _opt(dev_status, 1, "int32", dev, "dev_status"))


def va_page_ops_workspace_bytes(n_seqs: int, max_pages: int, n_pages: int) -> int:
    return int(lib().va_page_ops_workspace_bytes(int(n_seqs), int(max_pages), int(n_pages)))


def kv_page_extend(table, lens, n_new, refs, k_codes, v_codes, k_scale, v_scale, workspace, dev_status=None, stream=None,
                   variant: str = "") -> None:
    """Pages for n_new[b] more tokens of every sequence (copy on write); lens grows by n_new.  Pools of all layers:
    [layers, pages, heads, 64, 128]."""
    layers, pages, heads, _, dev, kc, vc, ks, vs = _pool(k_codes, v_codes, k_scale, v_scale)
    n = table.shape[0]
    width, tb = _table(table, n, dev)
    ws, size = _bytes(workspace, dev)
    _launch("kv_page_extend", lib(variant).kv_page_extend, dev, stream, tb, _at(lens, n, "int32", dev, "lens"),
            _at(n_new, n, "int32", dev, "n_new"), n, width, _at(refs, pages, "int32", dev, "refs"), pages, layers, heads,
            kc, vc, ks, vs, ws, size, _opt(dev_status, 1, "int32", dev, "dev_status"))


def kv_page_reorder(table, lens, src, refs, group: int = 0, dev_status=None, stream=None, variant: str = "") -> None:
    """Slot j takes the sequence of slot src[j] of its group (j: kept, another: forked, -1: freed)."""
    _torch or _import_torch()
    n, pages, dev = table.shape[0], refs.numel(), table.get_device()
    width, tb = _table(table, n, dev)
    _launch("kv_page_reorder", lib(variant).kv_page_reorder, dev, stream, tb, _at(lens, n, "int32", dev, "lens"), n, width,
            _at(src, n, "int32", dev, "src"), int(group), _at(refs, pages, "int32", dev, "refs"), pages,
            _opt(dev_status, 1, "int32", dev, "dev_status"))


def kv_page_copy(src, dst, k_codes, v_codes, k_scale, v_scale, dev_status=None, stream=None, variant: str = "") -> None:
    """Page dst[i] becomes a copy of page src[i], in all layers."""
    layers, pages, heads, _, dev, kc, vc, ks, vs = _pool(k_codes, v_codes, k_scale, v_scale)
    n = src.numel()
    _launch("kv_page_copy", lib(variant).kv_page_copy, dev, stream, _at(src, n, "int32", dev, "src"),
            _at(dst, n, "int32", dev, "dst"), n, pages, layers, heads, kc, vc, ks, vs,
            _opt(dev_status, 1, "int32", dev, "dev_status"))


def kv_page_compact(table, refs, k_codes, v_codes, k_scale, v_scale, moved_to, n_live_pages, workspace, dev_status=None,
                    stream=None, variant: str = "") -> None:
    """Move the live pages to the lowest numbers; moved_to [pages] tells where, n_live_pages [1] how many there are."""
    layers, pages, heads, _, dev, kc, vc, ks, vs = _pool(k_codes, v_codes, k_scale, v_scale)
    n = table.shape[0]
    width, tb = _table(table, n, dev)
    ws, size = _bytes(workspace, dev)
    _launch("kv_page_compact", lib(variant).kv_page_compact, dev, stream, tb, n, width, _at(refs, pages, "int32", dev, "refs"),
            pages, layers, heads, kc, vc, ks, vs, _at(moved_to, pages, "int32", dev, "moved_to"),
            _at(n_live_pages, 1, "int32", dev, "n_live_pages"), ws, size, _opt(dev_status, 1, "int32", dev, "dev_status"))


# ----------------------------------------------------------------------------- beam search
def va_beam_workspace_bytes(n_groups: int, n_beams: int, vocab: int, n_out: int) -> int:
    return int(lib().va_beam_workspace_bytes(int(n_groups), int(n_beams), int(vocab), int(n_out)))


def va_beam_select(logits, scores, n_beams: int, parents, tokens, out_scores, workspace, finished=None, end_token: int = 0,
                   stream=None, variant: str = "") -> None:
    """The best n_out continuations of each request's n_beams hypotheses: logits [n_groups * n_beams, vocab] (float32
    or bfloat16, rows at any stride that keeps them 16-byte aligned: a multiple of 4 or 8 entries, so that several rows
    of a vocabulary that is none need padding, as in torch.empty(rows, padded)[:, :vocab]), scores [n_groups *
    n_beams]; writes parents, tokens and out_scores [n_groups, n_out].  ``workspace``: va_beam_workspace_bytes(...)
    bytes, zeroed once."""
    torch = _torch or _import_torch()
    rows, vocab = logits.shape
    groups, n_out = parents.shape
    stride, inner = logits.stride()
    bf16, dev = logits.dtype is torch.bfloat16, logits.get_device()
    _need(groups * n_beams == rows and (vocab == 1 or inner == 1) and (bf16 or logits.dtype is torch.float32),
          "logits are float32 or bfloat16 [n_groups * n_beams, vocab]")
    count = groups * n_out
    ws, size = _bytes(workspace, dev)
    _launch("va_beam_select", lib(variant).va_beam_select, dev, stream, logits.data_ptr(), 1 if bf16 else 0, stride, groups,
            int(n_beams), vocab, _at(scores, rows, "float32", dev, "scores"), _opt(finished, rows, "int32", dev, "finished"),
            int(end_token), n_out, _at(parents, count, "int32", dev, "parents"), _at(tokens, count, "int32", dev, "tokens"),
            _at(out_scores, count, "float32", dev, "out_scores"), ws, size)


# ----------------------------------------------------------------------------- self-test
def va_selftest_bounded_wait(limit_ns: int, abort_after_ns: int = 0, dev_status=None, elapsed_ns=None, stream=None,
                             variant: str = "") -> None:
    """Run the kernels' bounded wait on a barrier nothing completes (see include/verify_attn.h)."""
    st = lib(variant).va_selftest_bounded_wait(int(limit_ns), int(abort_after_ns), _ptr(dev_status),
                                               _ptr(elapsed_ns), _stream(stream))
    _check("va_selftest_bounded_wait", st)
