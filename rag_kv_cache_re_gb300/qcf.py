"""Python binding of the qcf C ABI: argument marshalling only.

Each function here has the name of the C entry point it calls.  Torch provides
device memory and the current CUDA stream; every computation runs in the
library's CUDA kernels.  Workspaces are cached per device and reused; calls are
ordered on the current stream.
"""
from __future__ import annotations

import ctypes as C
from typing import Dict, List, Optional, Sequence, Tuple

import numpy as np
import torch

from . import _lib
from ._lib import QcfError, call

_WS: Dict[Tuple[int, str], torch.Tensor] = {}


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def workspace(nbytes: int, device, tag: str = "main") -> torch.Tensor:
    """A cached uint8 device buffer of at least `nbytes` (grow only, 256-byte aligned)."""
    dev = torch.device(device)
    key = (dev.index if dev.index is not None else torch.cuda.current_device(), tag)
    buf = _WS.get(key)
    need = max(256, int(nbytes))
    if buf is None or buf.numel() < need:
        if buf is not None:
            torch.cuda.current_stream(dev).synchronize()
        buf = torch.empty(need, dtype=torch.uint8, device=dev)
        _WS[key] = buf
    return buf


def _need_cuda(*ts: torch.Tensor):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise QcfError("binding", 1, "tensors must be on a CUDA device")
        if t is not None and not t.is_contiguous():
            raise QcfError("binding", 1, "tensors must be contiguous")


def _i32(a) -> C.Array:
    a = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return (C.c_int32 * len(a))(*a.tolist())


# ------------------------------------------------------------------ library

def qcf_version() -> str:
    return _lib.lib().qcf_version().decode()


def qcf_last_error() -> str:
    return _lib.lib().qcf_last_error().decode(errors="replace")


def qcf_query_status(stream=None) -> int:
    v = C.c_uint32(0)
    call("qcf_query_status", _stream(stream), C.byref(v))
    return int(v.value)


def qcf_debug_set_fault(kind: int) -> None:
    call("qcf_debug_set_fault", int(kind))


def qcf_set_check(on: bool) -> None:
    call("qcf_set_check", 1 if on else 0)


def qcf_launch_count() -> int:
    return int(_lib.lib().qcf_launch_count())


def qcf_timing_enable(on: bool) -> None:
    call("qcf_timing_enable", 1 if on else 0)


def qcf_timing_read() -> Dict[str, Tuple[float, int]]:
    n = 32
    names = (C.c_char_p * n)()
    ms = (C.c_double * n)()
    cnt = (C.c_int64 * n)()
    k = C.c_int(0)
    call("qcf_timing_read", n, names, ms, cnt, C.byref(k))
    return {names[i].decode(): (float(ms[i]), int(cnt[i])) for i in range(k.value)}


def qcf_calibrate_exp2_rate(device=None) -> float:
    """exp2 evaluations per second of the special-function units of the device (measured)."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    scratch = torch.empty(1 << 22, dtype=torch.float32, device=dev)
    rate = C.c_double(0.0)
    call("qcf_calibrate_exp2_rate", _ptr(scratch), scratch.numel() * 4, C.byref(rate), _stream(None))
    return float(rate.value)


def qcf_storage_status() -> int:
    """errno of the first failed storage read since the last call (0 when none); the copy
    stream must have run past the reads (synchronise first)."""
    v = C.c_int(0)
    call("qcf_storage_status", C.byref(v))
    return int(v.value)


def qcf_num_selected(C_len: int, ratio_bp: int) -> int:
    out = C.c_int(0)
    call("qcf_num_selected", int(C_len), int(ratio_bp), C.byref(out))
    return int(out.value)


class RopeTable:
    """Device cos/sin tables [max_pos][D/2] fp32 built in fp64 by the library on the host."""

    def __init__(self, max_pos: int, head_dim: int, theta: float, device):
        cos_h = torch.empty((max_pos, head_dim // 2), dtype=torch.float32).pin_memory()
        sin_h = torch.empty_like(cos_h).pin_memory()
        call("qcf_rope_table_fill_host", C.c_void_p(cos_h.data_ptr()), C.c_void_p(sin_h.data_ptr()), int(max_pos),
             int(head_dim), float(theta))
        self.cos = cos_h.to(device, non_blocking=False)
        self.sin = sin_h.to(device, non_blocking=False)
        self.max_pos, self.head_dim = int(max_pos), int(head_dim)
        self.struct = _lib.RopeTable(self.cos.data_ptr(), self.sin.data_ptr(), self.max_pos, self.head_dim)


# ------------------------------------------------------------------ steps

def qcf_anchor_keynorm_topk(K: torch.Tensor, chunk_start: Sequence[int], n_anchor: int,
                            want_norms: bool = False, stream=None):
    _need_cuda(K)
    C_len, Hkv, D = K.shape
    n_chunks = len(chunk_start) - 1
    idx = torch.empty((n_chunks, n_anchor), dtype=torch.int32, device=K.device)
    norms = torch.empty(C_len, dtype=torch.float32, device=K.device) if want_norms else None
    call("qcf_anchor_keynorm_topk", _ptr(K), _i32(chunk_start), n_chunks, Hkv, D, int(n_anchor), _ptr(idx),
         _ptr(norms), _stream(stream))
    return (idx, norms) if want_norms else idx


def qcf_rope_reposition(K_src: torch.Tensor, K_dst: torch.Tensor, seg_start: Sequence[int],
                        seg_delta: Sequence[int], table: RopeTable, stream=None) -> torch.Tensor:
    _need_cuda(K_src, K_dst)
    n, Hkv, D = K_src.shape
    call("qcf_rope_reposition", _ptr(K_src), _ptr(K_dst), int(n), Hkv, D, _i32(seg_start), _i32(seg_delta),
         len(seg_delta), C.byref(table.struct), _stream(stream))
    return K_dst


def qcf_profile_scores(q: torch.Tensor, K: torch.Tensor, scale: float, stream=None) -> torch.Tensor:
    _need_cuda(q, K)
    nq, Hq, D = q.shape
    C_len, Hkv, _ = K.shape
    scores = torch.empty(C_len, dtype=torch.float32, device=q.device)
    nb = _lib.lib().qcf_profile_scores_workspace_size(nq, C_len, Hq, Hkv, D)
    ws = workspace(nb, q.device)
    call("qcf_profile_scores", _ptr(q), _ptr(K), nq, C_len, Hq, Hkv, D, float(scale), _ptr(scores), _ptr(ws),
         ws.numel(), _stream(stream))
    return scores


def qcf_topn_select(scores: torch.Tensor, N: int, stream=None) -> torch.Tensor:
    _need_cuda(scores)
    sel = torch.empty(max(int(N), 1), dtype=torch.int32, device=scores.device)
    call("qcf_topn_select", _ptr(scores), scores.numel(), int(N), _ptr(sel), _stream(stream))
    return sel[:N]


def qcf_topn_select_ws(scores: torch.Tensor, N: int, ws: torch.Tensor = None, stream=None) -> torch.Tensor:
    _need_cuda(scores)
    sel = torch.empty(max(int(N), 1), dtype=torch.int32, device=scores.device)
    if ws is None:
        ws = workspace(_lib.lib().qcf_topn_select_workspace_size(scores.numel()), scores.device, "topn")
    call("qcf_topn_select_ws", _ptr(scores), scores.numel(), int(N), _ptr(sel), _ptr(ws), ws.numel(),
         _stream(stream))
    return sel[:N]


def qcf_gather_rows(src: torch.Tensor, idx: torch.Tensor, stream=None) -> torch.Tensor:
    _need_cuda(src, idx)
    rows = src.shape[0]
    width = src.numel() // max(rows, 1)
    dst = torch.empty((idx.numel(),) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
    call("qcf_gather_rows", _ptr(src), rows, width, _ptr(idx), idx.numel(), _ptr(dst), _stream(stream))
    return dst


def qcf_scatter_kv(k_new, v_new, pos, K_cache, V_cache, stream=None) -> None:
    _need_cuda(k_new, v_new, pos, K_cache, V_cache)
    n, Hkv, D = k_new.shape
    call("qcf_scatter_kv", _ptr(k_new), _ptr(v_new), _ptr(pos), n, Hkv, D, _ptr(K_cache), _ptr(V_cache),
         K_cache.shape[0], _stream(stream))


def qcf_kv_deviation(k_new, v_new, pos, K_cache, V_cache, stream=None):
    """dev[i] = |k_new[i] - K_cache[pos[i]]|^2 + |v_new[i] - V_cache[pos[i]]|^2 (fp32)."""
    _need_cuda(k_new, v_new, pos, K_cache, V_cache)
    n, Hkv, D = k_new.shape
    dev = torch.empty(n, dtype=torch.float32, device=k_new.device)
    call("qcf_kv_deviation", _ptr(k_new), _ptr(v_new), _ptr(pos), n, _ptr(K_cache), _ptr(V_cache), K_cache.shape[0],
         Hkv, D, _ptr(dev), _stream(stream))
    return dev


def qcf_sparse_causal_attn(q, pos, K, V, scale: float, want_lse: bool = False, stream=None):
    _need_cuda(q, pos, K, V)
    n, Hq, D = q.shape
    T, Hkv, _ = K.shape
    o = torch.empty_like(q)
    lse = torch.empty((n, Hq), dtype=torch.float32, device=q.device) if want_lse else None
    nb = _lib.lib().qcf_sparse_causal_attn_workspace_size(n, T, Hq, Hkv, D)
    ws = workspace(nb, q.device)
    call("qcf_sparse_causal_attn", _ptr(q), _ptr(pos), n, _ptr(K), _ptr(V), T, Hq, Hkv, D, float(scale), _ptr(o),
         _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    return (o, lse) if want_lse else o


def qcf_linear(A: torch.Tensor, W: torch.Tensor, out: Optional[torch.Tensor] = None, add: bool = False,
               w_kn: bool = False, stream=None) -> torch.Tensor:
    """out = A W^T (bf16 out), or out += A W^T for an fp32 `out` when add=True.
    With w_kn, W is stored [K][N] and out = A W."""
    _need_cuda(A, W)
    M, K = A.shape
    N = W.shape[1] if w_kn else W.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32 if add else torch.bfloat16, device=A.device)
        if add:
            out.zero_()
    nb = _lib.lib().qcf_linear_workspace_size(M, N, K)
    ws = workspace(nb, A.device)
    epi = (_lib.QCF_EPI_ADD_F32 if add else _lib.QCF_EPI_STORE_BF16) | (_lib.QCF_LINEAR_W_KN if w_kn else 0)
    call("qcf_linear", _ptr(A), M, K, _ptr(W), N, epi, _ptr(out), _ptr(ws), ws.numel(), _stream(stream))
    return out


def qcf_rmsnorm(x: torch.Tensor, g: torch.Tensor, eps: float, stream=None) -> torch.Tensor:
    _need_cuda(x, g)
    n, d = x.shape
    h = torch.empty((n, d), dtype=torch.bfloat16, device=x.device)
    call("qcf_rmsnorm", _ptr(x), n, d, _ptr(g), float(eps), _ptr(h), _stream(stream))
    return h


def qcf_fused_layer_forward(model, layer: int, x: torch.Tensor, rope_pos: torch.Tensor, cache_row: torch.Tensor,
                            K_cache: torch.Tensor, V_cache: torch.Tensor, stream=None) -> torch.Tensor:
    _need_cuda(x, rope_pos, cache_row, K_cache, V_cache)
    n = x.shape[0]
    T = K_cache.shape[0]
    nb = _lib.lib().qcf_layer_workspace_size(C.byref(model.struct.dims), n, T)
    ws = workspace(nb, x.device)
    call("qcf_fused_layer_forward", C.byref(model.struct), int(layer), _ptr(x), _ptr(rope_pos), _ptr(cache_row), n,
         _ptr(K_cache), _ptr(V_cache), T, _ptr(ws), ws.numel(), _stream(stream))
    return x


def qcf_embed_rows(model, ids: torch.Tensor, rows: Optional[torch.Tensor], n: int, stream=None) -> torch.Tensor:
    x = torch.empty((n, model.spec.d_model), dtype=torch.float32, device=ids.device)
    call("qcf_embed_rows", C.byref(model.struct), _ptr(ids), _ptr(rows), int(n), _ptr(x), _stream(stream))
    return x


def qcf_lm_head(model, x_last: torch.Tensor, stream=None):
    logits = torch.empty(model.spec.vocab, dtype=torch.float32, device=x_last.device)
    token = torch.empty(1, dtype=torch.int32, device=x_last.device)
    nb = _lib.lib().qcf_lm_head_workspace_size(C.byref(model.struct.dims))
    ws = workspace(nb, x_last.device, tag="lm")
    call("qcf_lm_head", C.byref(model.struct), _ptr(x_last), _ptr(logits), _ptr(token), _ptr(ws), ws.numel(),
         _stream(stream))
    return logits, token


def qcf_full_prefill(model, ids: torch.Tensor, K_layers: Optional[List[torch.Tensor]] = None,
                     V_layers: Optional[List[torch.Tensor]] = None, stream=None):
    """Full recompute of ids (device int32 [T]) -> per-layer K/V, last logits, first token (device)."""
    _need_cuda(ids)
    s = model.spec
    T = ids.numel()
    dev = ids.device
    if K_layers is None:
        K_layers = [torch.empty((T, s.n_kv_heads, s.head_dim), dtype=torch.bfloat16, device=dev) for _ in range(s.n_layers)]
        V_layers = [torch.empty_like(K_layers[0]) for _ in range(s.n_layers)]
    kp = (C.c_void_p * s.n_layers)(*[k.data_ptr() for k in K_layers])
    vp = (C.c_void_p * s.n_layers)(*[v.data_ptr() for v in V_layers])
    logits = torch.empty(s.vocab, dtype=torch.float32, device=dev)
    token = torch.empty(1, dtype=torch.int32, device=dev)
    nb = _lib.lib().qcf_full_prefill_workspace_size(C.byref(model.struct.dims), T)
    ws = workspace(nb, dev)
    call("qcf_full_prefill", C.byref(model.struct), _ptr(ids), T, kp, vp, _ptr(logits), _ptr(token), _ptr(ws),
         ws.numel(), _stream(stream))
    return K_layers, V_layers, logits, token


def qcf_request_prefill(model, req: "_lib.Request", outs: "_lib.Outputs", ws: torch.Tensor, compute_stream,
                        copy_stream) -> None:
    """Enqueues the fused prefill of one request (structs built by model.FusedRequest)."""
    call("qcf_request_prefill", C.byref(model.struct), C.byref(req), C.byref(outs), _ptr(ws), ws.numel(),
         C.c_void_p(compute_stream.cuda_stream), C.c_void_p(copy_stream.cuda_stream))


def qcf_batch_prefill(model, reqs, outs, ws: torch.Tensor, compute_stream, copy_stream) -> int:
    """Enqueues several fused prefills sharing their common chunks' host-to-device copies
    (structs built by model.FusedRequest); returns the bytes the call sends to the device."""
    n = len(reqs)
    ra = (_lib.Request * n)(*reqs)
    oa = (_lib.Outputs * n)(*outs)
    h2d = C.c_int64(0)
    call("qcf_batch_prefill", C.byref(model.struct), ra, oa, n, _ptr(ws), ws.numel(),
         C.c_void_p(compute_stream.cuda_stream), C.c_void_p(copy_stream.cuda_stream), C.byref(h2d))
    return int(h2d.value)


def qcf_batch_workspace_size(model, reqs) -> int:
    n = len(reqs)
    ra = (_lib.Request * n)(*reqs)
    return int(_lib.lib().qcf_batch_workspace_size(C.byref(model.struct.dims), ra, n))


# ------------------------------------------------------------------ going on from a shared context

_DTYPE = {torch.bfloat16: _lib.QCF_BF16, torch.float16: _lib.QCF_F16, torch.float32: _lib.QCF_F32}


def _bad(message: str):
    raise QcfError("binding", 1, message)


def _need_here(*ts: Optional[torch.Tensor]):
    """Every tensor on the current CUDA device: kernels launch there."""
    dev = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            _bad("tensors must be on the current CUDA device")


def _need_i32(t: torch.Tensor, what: str, shape=None):
    if t.dtype != torch.int32 or not t.is_contiguous() or (shape is not None and tuple(t.shape) != shape):
        _bad(f"{what} must be a contiguous int32 tensor" + (f" of shape {shape}" if shape is not None else ""))


def _head_rows(t: torch.Tensor, what: str) -> int:
    """The row stride of a [n][H][D] tensor whose rows hold their heads side by side."""
    if t.dim() != 3 or t.dtype not in _DTYPE:
        _bad(f"{what} must be a bf16, fp16 or fp32 tensor [n][H][D]")
    n, H, D = t.shape
    s = t.stride()
    if (D > 1 and s[2] != 1) or (H > 1 and s[1] != D):
        _bad(f"{what}: the heads of a row must be contiguous")
    return s[0] if n > 1 else H * D


class RopeScaling:
    """Frequencies scaled for contexts beyond the original length (see qcf_rope_scaling).

    kind: "linear", "base", "turns" or "index"; factor s; original, low and high for the last two."""

    def __init__(self, kind: str, factor: float = 1.0, original: int = 0, low: float = 0.0, high: float = 0.0,
                 amplitude: float = 1.0):
        if kind not in _lib.QCF_ROPE_SCALE:
            _bad(f"unknown scaling {kind!r}")
        self.struct = _lib.RopeScaling(_lib.QCF_ROPE_SCALE[kind], int(original), float(factor), float(low), float(high),
                                       float(amplitude))


def qcf_rope_table_fill(cos: torch.Tensor, sin: torch.Tensor, theta: float, first_pos: int = 0,
                        scaling: Optional[RopeScaling] = None, stream=None) -> None:
    """Fills fp32 device tables [n_pos][R/2] for positions first_pos, first_pos + 1, ..."""
    _need_cuda(cos, sin)
    _need_here(cos, sin)
    if cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.shape != sin.shape or cos.dim() != 2:
        _bad("cos and sin must be fp32 tensors of one shape [n_pos][R/2]")
    n, half = cos.shape
    call("qcf_rope_table_fill", cos.data_ptr(), sin.data_ptr(), int(first_pos), n, 2 * half, float(theta),
         None if scaling is None else C.byref(scaling.struct), _stream(stream))


class ScaledRopeTable:
    """Device cos/sin tables [max_pos][R/2] fp32, filled on the device; R may be part of the head."""

    def __init__(self, max_pos: int, rotary_dim: int, theta: float, device, scaling: Optional[RopeScaling] = None, stream=None):
        self.max_pos, self.head_dim = int(max_pos), int(rotary_dim)
        with torch.cuda.stream(stream):
            self.cos = torch.empty((self.max_pos, self.head_dim // 2), dtype=torch.float32, device=device)
            self.sin = torch.empty_like(self.cos)
        qcf_rope_table_fill(self.cos, self.sin, theta, 0, scaling, stream)
        self.struct = _lib.RopeTable(self.cos.data_ptr(), self.sin.data_ptr(), self.max_pos, self.head_dim)


def qcf_rope_apply(x: torch.Tensor, pos: torch.Tensor, table, interleaved: bool = False, inverse: bool = False,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [n][H][D] (heads of a row contiguous, any row stride) turned by the angles of pos [n];
    out=x rotates in place.  Rows at position -1 are left as they were in `out`."""
    xs = _head_rows(x, "x")
    n, H, D = x.shape
    _need_i32(pos, "pos", (n,))
    if out is None:
        with torch.cuda.stream(stream):
            out = torch.empty((n, H, D), dtype=x.dtype, device=x.device)
        ys = H * D
    else:
        if out.shape != x.shape or out.dtype != x.dtype:
            _bad("out must have the shape and type of x")
        ys = _head_rows(out, "out")
    _need_here(x, pos, out, table.cos)
    if n == 0:   # empty tensors have no address to pass
        return out
    call("qcf_rope_apply", x.data_ptr(), xs, out.data_ptr(), ys, n, H, D, _DTYPE[x.dtype], pos.data_ptr(),
         C.byref(table.struct), (_lib.QCF_ROPE_INTERLEAVED if interleaved else 0) | (_lib.QCF_ROPE_INVERSE if inverse else 0),
         _stream(stream))
    return out


class PagedKV:
    """K and V pages of one layer: [n_pages][page_size][Hkv][D] (layout "rows") or
    [n_pages][Hkv][page_size][D] ("heads"), bf16 or fp16; other strides as given."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, layout: str = "rows"):
        if layout not in ("rows", "heads"):
            _bad(f"unknown layout {layout!r}")
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.stride(3) != 1:
            _bad("k and v must be 4-d tensors of one shape, type and stride, their last dimension contiguous")
        if k.dtype not in (torch.bfloat16, torch.float16):
            _bad("the cache holds bf16 or fp16")
        if not k.is_cuda or k.device != v.device:
            _bad("k and v must be on one CUDA device")
        self.k, self.v, self.layout = k, v, layout
        row, head = (1, 2) if layout == "rows" else (2, 1)
        n_pages, D = k.shape[0], k.shape[3]
        self.page_size, self.Hkv, self.D = k.shape[row], k.shape[head], D
        stride = [s if n > 1 else self.page_size * self.Hkv * D for s, n in zip(k.stride(), k.shape)]
        self.struct = _lib.PagedKV(k.data_ptr(), v.data_ptr(), _DTYPE[k.dtype], n_pages, self.page_size, self.Hkv, D,
                                   stride[0], stride[row], stride[head])
        self.ref = C.byref(self.struct)


class PagedBatch:
    """A batch of sequences over one shared prefix (see qcf_paged_batch).  The tensors are read
    on the device at each call, so their values may change between calls within the bounds."""

    def __init__(self, row_start: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor, n_rows: int, max_q: int,
                 max_len: int, prefix_pages: Optional[torch.Tensor] = None, prefix_len: int = 0):
        n_seq = kv_len.numel()
        _need_i32(row_start, "row_start", (n_seq + 1,))
        _need_i32(kv_len, "kv_len", (n_seq,))
        if page_table.dim() != 2 or page_table.shape[0] != n_seq:
            _bad("page_table must have one row per sequence")
        _need_i32(page_table, "page_table")
        if prefix_pages is not None:
            _need_i32(prefix_pages, "prefix_pages")
        self.row_start, self.kv_len, self.page_table, self.prefix_pages = row_start, kv_len, page_table, prefix_pages
        self.n_rows, self.prefix_len = int(n_rows), int(prefix_len)
        self.empty = n_seq == 0 or self.n_rows == 0   # nothing to do, and no addresses to pass
        self.struct = _lib.PagedBatch(n_seq, self.n_rows, int(max_q), int(max_len), row_start.data_ptr(), kv_len.data_ptr(),
                                      page_table.data_ptr(), page_table.shape[1], self.prefix_len,
                                      None if prefix_pages is None else prefix_pages.data_ptr())
        self.ref = C.byref(self.struct)

    def _check(self, cache: PagedKV, *rows: Optional[torch.Tensor]):
        if self.prefix_len > 0 and (self.prefix_pages is None or self.prefix_pages.numel() * cache.page_size < self.prefix_len):
            _bad("prefix_pages hold fewer rows than prefix_len")
        for t in rows:
            if t is not None and (t.shape[0] != self.n_rows or t.shape[2] != cache.D or t.dtype != cache.k.dtype):
                _bad(f"rows must be [{self.n_rows}][heads][{cache.D}] of the cache's type")
        _need_here(cache.k, self.row_start, self.kv_len, self.page_table, self.prefix_pages, *rows)


def qcf_paged_append(cache: PagedKV, batch: PagedBatch, k_new: torch.Tensor, v_new: torch.Tensor, table=None,
                     interleaved: bool = False, q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                     stream=None) -> Optional[torch.Tensor]:
    """Writes the batch's new keys (rotated when a table is given) and values into their pages;
    with q, returns the rotated queries (q_out, or a new tensor whose padding rows are unset)."""
    ks, vs = _head_rows(k_new, "k_new"), _head_rows(v_new, "v_new")
    if ks != vs or k_new.shape != v_new.shape or k_new.shape[1] != cache.Hkv:
        _bad("k_new and v_new must have the cache's heads and one row stride")
    qs = qos = Hq = 0
    if q is not None:
        qs, Hq = _head_rows(q, "q"), q.shape[1]
        if q_out is None:
            with torch.cuda.stream(stream):
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        qos = _head_rows(q_out, "q_out")
        if q_out.shape != q.shape:
            _bad("q_out must have the shape of q")
    elif q_out is not None:
        _bad("q_out without q")
    batch._check(cache, k_new, v_new, q, q_out)
    if table is not None:
        _need_here(table.cos)
    if batch.empty:
        return q_out
    call("qcf_paged_append", cache.ref, batch.ref, k_new.data_ptr(), v_new.data_ptr(), ks,
         None if table is None else C.byref(table.struct), _lib.QCF_ROPE_INTERLEAVED if interleaved else 0,
         None if q is None else q.data_ptr(), qs, None if q is None else q_out.data_ptr(), qos, Hq, _stream(stream))
    return q_out


def qcf_shared_prefix_attn(cache: PagedKV, batch: PagedBatch, q: torch.Tensor, scale: float, want_lse: bool = False,
                           out: Optional[torch.Tensor] = None, stream=None):
    """Attention of the batch's rows q [n_rows][Hq][D] over the shared prefix and their own tokens.
    Returns out (a new tensor unless given; padding rows are not written), with lse if asked."""
    qs = _head_rows(q, "q")
    n, Hq, D = q.shape
    batch._check(cache, q, out)
    if out is not None and (out.shape != q.shape or not out.is_contiguous()):
        _bad("out must be contiguous, of the shape of q")
    nb = 0 if batch.empty else _lib.lib().qcf_shared_prefix_attn_workspace_size(cache.ref, batch.ref, Hq)
    with torch.cuda.stream(stream):   # the allocator ties them to the stream that uses them
        if out is None:
            out = torch.empty((n, Hq, D), dtype=q.dtype, device=q.device)
        lse = torch.empty((n, Hq), dtype=torch.float32, device=q.device) if want_lse else None
        ws = torch.empty(nb, dtype=torch.uint8, device=q.device) if nb else None
    if not batch.empty:
        call("qcf_shared_prefix_attn", cache.ref, batch.ref, q.data_ptr(), qs, Hq, float(scale), out.data_ptr(), _ptr(lse),
             _ptr(ws), nb, _stream(stream))
    return (out, lse) if want_lse else out
