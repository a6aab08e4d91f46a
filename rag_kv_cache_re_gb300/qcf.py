"""Python binding of the qcf C ABI: argument marshalling only.

Each function here has the name of the C entry point it calls.  Torch provides
device memory and the current CUDA stream; every computation runs in the
library's CUDA kernels.  Workspaces are cached per device and reused; calls are
ordered on the current stream.
"""
from __future__ import annotations

import ctypes as C
import functools
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
        self.ref, self.dev = C.byref(self.struct), self.cos.get_device()


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
#
# These calls run once per layer and decode step, where the host's time counts: everything that
# does not change from call to call is checked and marshalled when its object is made.

_DTYPE = {torch.bfloat16: _lib.QCF_BF16, torch.float16: _lib.QCF_F16, torch.float32: _lib.QCF_F32}


def _bad(message: str):
    raise QcfError("binding", 1, message)


def _here(t: torch.Tensor) -> int:
    """The device of t, which must be the current one: kernels launch there."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        _bad("tensors must be on the current CUDA device")
    return dev


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, dev: int, stream) -> torch.Tensor:
    """A new tensor, tied by the allocator to the stream that will use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _need_i32(t: torch.Tensor, what: str, shape=None):
    if t.dtype != torch.int32 or not t.is_contiguous() or (shape is not None and tuple(t.shape) != shape):
        _bad(f"{what} must be a contiguous int32 tensor" + (f" of shape {shape}" if shape is not None else ""))


def _head_rows(t: torch.Tensor, what: str):
    """(n, H, D, row stride) of a tensor [n][H][D] whose rows hold their heads side by side."""
    if t.dim() != 3 or t.dtype not in _DTYPE:
        _bad(f"{what} must be a bf16, fp16 or fp32 tensor [n][H][D]")
    n, H, D = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and D > 1) or (s1 != D and H > 1):
        _bad(f"{what}: the heads of a row must be contiguous")
    return n, H, D, s0 if n > 1 else H * D


class RopeScaling:
    """Frequencies scaled for contexts beyond the original length (see qcf_rope_scaling).

    kind: "linear", "base", "turns" or "index"; factor s; original, low and high for the last two."""

    def __init__(self, kind: str, factor: float = 1.0, original: int = 0, low: float = 0.0, high: float = 0.0,
                 amplitude: float = 1.0):
        if kind not in _lib.QCF_ROPE_SCALE:
            _bad(f"unknown scaling {kind!r}")
        self.struct = _lib.RopeScaling(_lib.QCF_ROPE_SCALE[kind], int(original), float(factor), float(low), float(high),
                                       float(amplitude))
        self.ref = C.byref(self.struct)


def qcf_rope_table_fill(cos: torch.Tensor, sin: torch.Tensor, theta: float, first_pos: int = 0,
                        scaling: Optional[RopeScaling] = None, stream=None) -> None:
    """Fills fp32 device tables [n_pos][R/2] for positions first_pos, first_pos + 1, ..."""
    if (cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.dim() != 2 or cos.shape != sin.shape
            or not cos.is_contiguous() or not sin.is_contiguous()):
        _bad("cos and sin must be contiguous fp32 tensors of one shape [n_pos][R/2]")
    dev = _here(cos)
    if sin.get_device() != dev:
        _bad("tensors must be on the current CUDA device")
    n, half = cos.shape
    if not 0 <= first_pos <= 2**31 - 1 - n:
        _bad(f"positions {first_pos} .. {first_pos} + {n} exceed 31 bits")
    if n == 0:   # empty tensors have no address to pass
        return
    call("qcf_rope_table_fill", cos.data_ptr(), sin.data_ptr(), first_pos, n, 2 * half, theta,
         None if scaling is None else scaling.ref, _raw_stream(stream, dev))


class ScaledRopeTable:
    """Device cos/sin tables [max_pos][R/2] fp32, filled on the device; R may be part of the head."""

    def __init__(self, max_pos: int, rotary_dim: int, theta: float, device, scaling: Optional[RopeScaling] = None, stream=None):
        self.max_pos, self.head_dim = int(max_pos), int(rotary_dim)
        with torch.cuda.stream(stream):
            self.cos = torch.empty((self.max_pos, self.head_dim // 2), dtype=torch.float32, device=device)
            self.sin = torch.empty_like(self.cos)
        qcf_rope_table_fill(self.cos, self.sin, theta, 0, scaling, stream)
        self.struct = _lib.RopeTable(self.cos.data_ptr(), self.sin.data_ptr(), self.max_pos, self.head_dim)
        self.ref, self.dev = C.byref(self.struct), self.cos.get_device()


def qcf_rope_apply(x: torch.Tensor, pos: torch.Tensor, table, interleaved: bool = False, inverse: bool = False,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [n][H][D] (heads of a row contiguous, any row stride) turned by the angles of pos [n];
    out=x rotates in place.  Rows at position -1 are left as they were in `out`."""
    n, H, D, xs = _head_rows(x, "x")
    dev = _here(x)
    if pos.dtype != torch.int32 or pos.dim() != 1 or pos.numel() != n or not pos.is_contiguous():
        _bad(f"pos must be a contiguous int32 tensor of {n} entries")
    if pos.get_device() != dev or table.dev != dev:
        _bad("tensors must be on the current CUDA device")
    if out is None:
        out, ys = _empty((n, H, D), x.dtype, dev, stream), H * D
    elif out is x:
        ys = xs
    else:
        if out.shape != x.shape or out.dtype != x.dtype or out.get_device() != dev:
            _bad("out must have the shape, type and device of x")
        ys = _head_rows(out, "out")[3]
    if n:   # empty tensors have no address to pass
        call("qcf_rope_apply", x.data_ptr(), xs, out.data_ptr(), ys, n, H, D, _DTYPE[x.dtype], pos.data_ptr(), table.ref,
             (_lib.QCF_ROPE_INTERLEAVED if interleaved else 0) | (_lib.QCF_ROPE_INVERSE if inverse else 0),
             _raw_stream(stream, dev))
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
        self.k, self.v, self.layout, self.dtype, self.dev = k, v, layout, k.dtype, k.get_device()
        row, head = (1, 2) if layout == "rows" else (2, 1)
        n_pages, D = k.shape[0], k.shape[3]
        self.page_size, self.Hkv, self.D = k.shape[row], k.shape[head], D
        # a dimension of one entry has no stride of its own
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
        self.dev = row_start.get_device()
        if any(t is not None and t.get_device() != self.dev for t in (kv_len, page_table, prefix_pages)):
            _bad("row_start, kv_len, page_table and prefix_pages must be on one device")
        self.n_rows, self.prefix_len = int(n_rows), int(prefix_len)
        if not all(0 <= int(v) < 2**31 for v in (n_rows, max_q, max_len, prefix_len)):
            _bad("n_rows, max_q, max_len and prefix_len must be 32-bit counts")
        self.empty = n_seq == 0 or self.n_rows == 0   # nothing to do, and no addresses to pass
        self.struct = _lib.PagedBatch(n_seq, self.n_rows, int(max_q), int(max_len), row_start.data_ptr(), kv_len.data_ptr(),
                                      page_table.data_ptr(), page_table.shape[1], self.prefix_len,
                                      None if prefix_pages is None else prefix_pages.data_ptr())
        self.ref = C.byref(self.struct)
        self._prefix_rows = 0 if prefix_pages is None else prefix_pages.numel()
        self._ws_bytes: Dict[Tuple[int, int, int, int], int] = {}

    def workspace_size(self, cache: PagedKV, Hq: int) -> int:
        """qcf_shared_prefix_attn_workspace_size: a function of the layout and the bounds alone.  0 for an
        empty batch, and for a layout the library refuses: that is not kept, for it may be refused for
        what the key does not hold (an address, a stride)."""
        if self.empty:
            return 0
        key = (cache.page_size, cache.Hkv, cache.D, Hq)
        nb = self._ws_bytes.get(key)
        if nb is None:
            nb = _lib.lib().qcf_shared_prefix_attn_workspace_size(cache.ref, self.ref, Hq)
            if nb:
                self._ws_bytes[key] = nb
        return nb

    def chunk_workspace_size(self, cache: PagedKV, Hq: int) -> int:
        """qcf_paged_chunk_attn_workspace_size, kept alike."""
        if self.empty:
            return 0
        key = (cache.page_size, cache.Hkv, cache.D, -Hq)
        nb = self._ws_bytes.get(key)
        if nb is None:
            nb = _lib.lib().qcf_paged_chunk_attn_workspace_size(cache.ref, self.ref, Hq)
            if nb:
                self._ws_bytes[key] = nb
        return nb


def _batch_rows(cache: PagedKV, batch: PagedBatch, t: torch.Tensor, what: str):
    """(H, row stride) of a tensor that holds the batch's rows in the cache's type and head dim."""
    n, H, D, s = _head_rows(t, what)
    if n != batch.n_rows or D != cache.D or t.dtype != cache.dtype or t.get_device() != cache.dev:
        _bad(f"{what} must be [{batch.n_rows}][heads][{cache.D}] of the cache's type and device")
    return H, s


def _cache_and_batch(cache: PagedKV, batch: PagedBatch):
    if cache.dev != torch.cuda.current_device() or batch.dev != cache.dev:
        _bad("tensors must be on the current CUDA device")
    if batch._prefix_rows * cache.page_size < batch.prefix_len:
        _bad("prefix_pages hold fewer rows than prefix_len")


def qcf_paged_append(cache: PagedKV, batch: PagedBatch, k_new: torch.Tensor, v_new: torch.Tensor, table=None,
                     interleaved: bool = False, q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                     stream=None) -> Optional[torch.Tensor]:
    """Writes the batch's new keys (rotated when a table is given) and values into their pages;
    with q, returns the rotated queries (q_out, or a new tensor whose padding rows are unset)."""
    _cache_and_batch(cache, batch)
    (Hk, ks), (Hv, vs) = _batch_rows(cache, batch, k_new, "k_new"), _batch_rows(cache, batch, v_new, "v_new")
    if ks != vs or Hk != Hv or Hk != cache.Hkv:
        _bad("k_new and v_new must have the cache's heads and one row stride")
    if table is not None and table.dev != cache.dev:
        _bad("tensors must be on the current CUDA device")
    qp = qop = None
    qs = qos = Hq = 0
    if q is not None:
        Hq, qs = _batch_rows(cache, batch, q, "q")
        if q_out is None:
            q_out, qos = _empty(q.shape, q.dtype, cache.dev, stream), Hq * cache.D
        elif q_out is q:
            qos = qs
        else:
            Ho, qos = _batch_rows(cache, batch, q_out, "q_out")
            if Ho != Hq:
                _bad("q_out must have the heads of q")
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        _bad("q_out without q")
    if not batch.empty:
        call("qcf_paged_append", cache.ref, batch.ref, k_new.data_ptr(), v_new.data_ptr(), ks,
             None if table is None else table.ref, _lib.QCF_ROPE_INTERLEAVED if interleaved else 0, qp, qs, qop, qos, Hq,
             _raw_stream(stream, cache.dev))
    return q_out


def qcf_shared_prefix_attn(cache: PagedKV, batch: PagedBatch, q: torch.Tensor, scale: float, want_lse: bool = False,
                           out: Optional[torch.Tensor] = None, stream=None):
    """Attention of the batch's rows q [n_rows][Hq][D] over the shared prefix and their own tokens.
    Returns out (a new tensor unless given; padding rows are not written), with lse if asked."""
    _cache_and_batch(cache, batch)
    Hq, qs = _batch_rows(cache, batch, q, "q")
    if out is None:
        out = _empty(q.shape, q.dtype, cache.dev, stream)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.get_device() != cache.dev:
        _bad("out must be contiguous, of the shape, type and device of q")
    lse = _empty((q.shape[0], Hq), torch.float32, cache.dev, stream) if want_lse else None
    if not batch.empty:
        nb = batch.workspace_size(cache, Hq)
        ws = _empty(nb, torch.uint8, cache.dev, stream) if nb else None
        call("qcf_shared_prefix_attn", cache.ref, batch.ref, q.data_ptr(), qs, Hq, scale, out.data_ptr(),
             None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(), nb, _raw_stream(stream, cache.dev))
    return (out, lse) if want_lse else out


# ------------------------------------------------------------------ whole prompts and chunks of them

def _attn_out(q: torch.Tensor, out: Optional[torch.Tensor], want_lse: bool, dev: int, stream, *counts: int):
    if not all(-2**31 <= int(n) < 2**31 for n in counts):
        _bad("max_len and window must be 32-bit counts")
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or out.get_device() != dev:
        _bad("out must be contiguous, of the shape, type and device of q")
    return out, _empty(q.shape[:2], torch.float32, dev, stream) if want_lse else None


@functools.lru_cache(maxsize=1024)
def _packed_workspace(dev: int, *sizes: int) -> int:
    """qcf_packed_causal_attn_workspace_size: a function of the sizes and the device alone."""
    return _lib.lib().qcf_packed_causal_attn_workspace_size(*sizes)


def qcf_packed_causal_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, row_start: torch.Tensor, max_len: int, scale: float,
                           window: int = 0, want_lse: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """Causal attention of whole prompts packed one behind the other: q [n_rows][Hq][D], k and v
    [n_rows][Hkv][D] (heads of a row contiguous, any row stride), row_start [n_seq + 1] int32 on the
    device, max_len a bound on a prompt's tokens.  Returns out (a new tensor unless given; rows of no
    prompt are not written), with lse if asked."""
    (n, Hq, D, qs), (nk, Hk, Dk, ks), (nv, Hv, Dv, vs) = _head_rows(q, "q"), _head_rows(k, "k"), _head_rows(v, "v")
    dev = _here(q)
    if (nk, Dk) != (n, D) or (nv, Hv, Dv) != (n, Hk, D) or ks != vs or k.dtype != q.dtype or v.dtype != q.dtype:
        _bad("k and v must have the rows, head dim and type of q, and one row stride")
    if k.get_device() != dev or v.get_device() != dev or row_start.get_device() != dev:
        _bad("tensors must be on the current CUDA device")
    if row_start.dim() != 1 or row_start.numel() < 1:
        _bad("row_start must hold a start per sequence and the end of the last")
    _need_i32(row_start, "row_start")
    out, lse = _attn_out(q, out, want_lse, dev, stream, max_len, window)
    n_seq = row_start.numel() - 1
    if n and n_seq:   # empty tensors have no address to pass
        nb = _packed_workspace(dev, n_seq, n, max_len, Hq, Hk, D)
        ws = _empty(nb, torch.uint8, dev, stream) if nb else None
        call("qcf_packed_causal_attn", q.data_ptr(), qs, k.data_ptr(), v.data_ptr(), ks, _DTYPE[q.dtype], row_start.data_ptr(), n_seq, n,
             max_len, Hq, Hk, D, scale, window, out.data_ptr(), None if lse is None else lse.data_ptr(),
             None if ws is None else ws.data_ptr(), nb, _raw_stream(stream, dev))
    return (out, lse) if want_lse else out


def qcf_paged_chunk_attn(cache: PagedKV, batch: PagedBatch, q: torch.Tensor, scale: float, window: int = 0, want_lse: bool = False,
                         out: Optional[torch.Tensor] = None, stream=None):
    """Attention of chunks of new tokens, q [n_rows][Hq][D], over the batch's prefix and own tokens in
    pages.  Returns out (a new tensor unless given; padding rows are not written), with lse if asked."""
    _cache_and_batch(cache, batch)
    Hq, qs = _batch_rows(cache, batch, q, "q")
    out, lse = _attn_out(q, out, want_lse, cache.dev, stream, window)
    if not batch.empty:
        nb = batch.chunk_workspace_size(cache, Hq)
        ws = _empty(nb, torch.uint8, cache.dev, stream) if nb else None
        call("qcf_paged_chunk_attn", cache.ref, batch.ref, q.data_ptr(), qs, Hq, scale, window, out.data_ptr(),
             None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(), nb, _raw_stream(stream, cache.dev))
    return (out, lse) if want_lse else out


# ------------------------------------------------------------------ the pages of a cache

class PagePool:
    """The pages of a cache and the sequences that hold them (see qcf_page_pool): `caches` the PagedKV of
    every layer, all of one layout; refs [n_pages], page_table [n_seq][columns] and kv_len [n_seq] int32 on the
    device.  page_table and kv_len also serve a PagedBatch.  Calls with one pool are made on one stream, or
    ordered by the caller: each changes the pool, and they share its scratch.  A pool outlives the graphs
    that hold calls of it."""

    def __init__(self, caches: Sequence[PagedKV], refs: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor):
        caches = list(caches)
        if not caches:
            _bad("a pool needs the cache of a layer at least")
        self.caches, self.refs, self.page_table, self.kv_len, self.dev = caches, refs, page_table, kv_len, caches[0].dev
        n_seq = kv_len.numel()
        _need_i32(kv_len, "kv_len", (n_seq,))
        _need_i32(refs, "refs", (caches[0].struct.n_pages,))
        if page_table.dim() != 2 or page_table.shape[0] != n_seq:
            _bad("page_table must have one row per sequence")
        _need_i32(page_table, "page_table")
        if any(t.get_device() != self.dev for t in (refs, page_table, kv_len)) or any(c.dev != self.dev for c in caches):
            _bad("caches, refs, page_table and kv_len must be on one device")
        self.n_seq = n_seq
        self._caches = (_lib.PagedKV * len(caches))(*[c.struct for c in caches])
        self.struct = _lib.PagePool(self._caches, len(caches), refs.data_ptr(), page_table.data_ptr(), page_table.shape[1], kv_len.data_ptr(),
                                    n_seq)
        self.ref = C.byref(self.struct)
        # Scratch for as many arguments as there are sequences.  One for the pool's life: its calls never overlap, for
        # each changes the pool.  (0 for a layout the library refuses, as every call then will.)
        self._nb = _lib.lib().qcf_pages_workspace_size(self.ref, n_seq)
        self._ws = torch.empty(max(self._nb, 1), dtype=torch.uint8, device=refs.device)
        self._ws_ptr = self._ws.data_ptr()
        self._streams = {_raw_stream(None, self.dev)}   # that the allocator knows to use the scratch

    @classmethod
    def empty(cls, caches: Sequence[PagedKV], n_seq: int, max_len: int) -> "PagePool":
        """A pool whose pages are all free, for n_seq sequences of up to max_len tokens."""
        caches = list(caches)
        if not caches:
            _bad("a pool needs the cache of a layer at least")
        dev, cols = caches[0].k.device, max(1, -(-max_len // caches[0].page_size))
        return cls(caches, *(torch.zeros(shape, dtype=torch.int32, device=dev) for shape in (caches[0].struct.n_pages, (n_seq, cols), n_seq)))

    def _list(self, t: torch.Tensor, n: int) -> int:
        """The address of an argument of n entries."""
        if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous() or t.get_device() != self.dev:
            _bad(f"every argument must be a contiguous int32 tensor of {n} entries on the pool's device")
        return t.data_ptr()

    def _here(self, stream) -> int:
        """The stream of a call that is about to be made."""
        if self.dev != torch.cuda.current_device():
            _bad("tensors must be on the current CUDA device")
        raw = _raw_stream(stream, self.dev)
        if raw not in self._streams:
            self._ws.record_stream(torch.cuda.current_stream(self.dev) if stream is None else stream)
            self._streams.add(raw)
        return raw


def qcf_pages_fork(pool: PagePool, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Sequences dst[i] (int32 on the device) go on from src[i]: full pages shared, a page held in part copied."""
    n = src.numel()
    a, b = pool._list(src, n), pool._list(dst, n)
    if n:   # empty tensors have no address to pass
        raw = pool._here(stream)
        call("qcf_pages_fork", pool.ref, a, b, n, pool._ws_ptr, pool._nb, raw)


def qcf_pages_resize(pool: PagePool, new_len: torch.Tensor, seqs: Optional[torch.Tensor] = None, stream=None) -> None:
    """Sequences seqs[i] (None: 0, 1, ..) get the lengths new_len[i], int32 on the device: pages taken or given back."""
    n = new_len.numel()
    b, a = pool._list(new_len, n), None if seqs is None else pool._list(seqs, n)
    if n:
        raw = pool._here(stream)
        call("qcf_pages_resize", pool.ref, a, b, n, pool._ws_ptr, pool._nb, raw)


def qcf_pages_compact(pool: PagePool, stream=None) -> torch.Tensor:
    """Moves the pages in use to the lowest ids; returns how many they are (int32 [1] on the device; -1 where a length
    is out of range, and nothing has changed)."""
    raw = pool._here(stream)
    live = _empty((1,), torch.int32, pool.dev, stream)
    call("qcf_pages_compact", pool.ref, live.data_ptr(), pool._ws_ptr, pool._nb, raw)
    return live
