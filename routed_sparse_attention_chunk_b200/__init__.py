"""Python binding of the MSA memory-path library (include/msa.h) for B200.

Argument marshalling only: every function takes caller-allocated torch tensors,
checks that they are contiguous CUDA tensors of the right dtype (the bank's
K̄ / V̄ may instead be pinned host tensors: the host tier, read in place), and
passes raw pointers and sizes to the C ABI in libmsa.so on the current (or
given) stream.
All computation happens in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import torch

from . import _lib

F32, BF16 = 0, 1
FLAG_INDEX_OOB, FLAG_OFFSETS, FLAG_TIMEOUT, FLAG_OVERFLOW = 1, 2, 4, 8
ROPE_HALF, ROPE_INTERLEAVED = 0, 1  # msa_rope_layout
ROPE_SCALES = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}  # MSA_ROPE_SCALE_*
DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


class MSAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = _lib.load().msa_status_string(status).decode()
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return DTYPES[t.dtype]


def _p(t, dtype=None, host_ok=False):
    """Device pointer of a contiguous CUDA tensor (None -> NULL).  With host_ok, a
    page-locked CPU tensor is accepted too (the device reads it in place)."""
    if t is None:
        return None
    if not t.is_cuda and not (host_ok and t.is_pinned()):
        raise ValueError("the MSA library takes CUDA tensors" + (" or pinned CPU tensors" if host_ok else ""))
    if not t.is_contiguous():
        raise ValueError("the MSA library takes contiguous tensors")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    return t.data_ptr()


def _s(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _call(name: str, *args) -> None:
    st = getattr(_lib.load(), name)(*args)
    if st != 0:
        raise MSAError(name, st)


def version() -> str:
    return _lib.load().msa_version().decode()


def kernel_launch_count() -> int:
    """Kernels the library has launched in this process (msa_kernel_launch_count)."""
    return int(_lib.load().msa_kernel_launch_count())


def testing_set_wait_polls(polls: int) -> None:
    """Test hook (msa_testing_set_wait_polls): polls of the prefill attention kernel's pipeline
    waits; 0 makes every such wait expire at once, a negative value restores the default."""
    _lib.load().msa_testing_set_wait_polls(int(polls))


def rope_table(theta: float, d: int, max_len: int) -> torch.Tensor:
    """Host fp32 [max_len, d/2, 2] table of (cos, sin) built in fp64 by the library."""
    out = torch.empty((max_len, d // 2, 2), dtype=torch.float32)
    _call("msa_rope_table_host", float(theta), d, max_len, out.data_ptr())
    return out


def chunk_offsets(doc_tok_off, P: int):
    """Host int64 [D+1] chunk offsets for host int64 token offsets (msa_chunk_offsets_host)."""
    import numpy as np
    tok = np.ascontiguousarray(np.asarray(doc_tok_off, dtype=np.int64))
    out = np.empty_like(tok)
    _call("msa_chunk_offsets_host", tok.ctypes.data, len(tok) - 1, P, out.ctypes.data)
    return out


def pool(K, V, Kr, doc_tok_off, doc_chunk_off, P, rope_cs, Kbar, Vbar, Krbar, kr_rnorm=None,
         err_flag=None, stream=None):
    """Step 1: RoPE + chunk-mean pooling (msa_pool)."""
    D = doc_tok_off.numel() - 1
    _call("msa_pool", _dt(K), _p(K), _p(V, K.dtype), _p(Kr, K.dtype), _p(doc_tok_off, torch.int64),
          _p(doc_chunk_off, torch.int64), D, K.shape[0], Kbar.shape[0], K.shape[1], K.shape[2],
          Kr.shape[1], Kr.shape[2], P, _p(rope_cs, torch.float32), rope_cs.shape[0],
          _p(Kbar, K.dtype), _p(Vbar, K.dtype), _p(Krbar, K.dtype), _p(kr_rnorm, torch.float32),
          _p(err_flag, torch.int32), _s(stream))


def bank_rnorm(Krbar, kr_rnorm, stream=None):
    _call("msa_bank_rnorm", _dt(Krbar), _p(Krbar), Krbar.shape[0], Krbar.shape[1], Krbar.shape[2],
          _p(kr_rnorm, torch.float32), _s(stream))


def route_topk_workspace_size(B: int, Tq: int, Hr: int, D: int, C: int, k: int) -> int:
    return _lib.load().msa_route_topk_workspace_size(B, Tq, Hr, D, C, k)


def route_topk(Qr, Krbar, kr_rnorm, doc_chunk_off, k, topk_idx, ws, topk_score=None, doc_scores=None,
               err_flag=None, stream=None):
    """Steps 2+3: cosine routing and top-k (msa_route_topk).  Qr [B, Tq, Hr, dr]."""
    B, Tq, Hr, dr = Qr.shape
    _call("msa_route_topk", _dt(Qr), _p(Qr), B, Tq, Hr, dr, _p(Krbar, Qr.dtype), _p(kr_rnorm, torch.float32),
          _p(doc_chunk_off, torch.int64), doc_chunk_off.numel() - 1, Krbar.shape[0], k,
          _p(doc_scores, torch.float32), _p(topk_idx, torch.int32), _p(topk_score, torch.float32),
          _p(ws), ws.numel() * ws.element_size(), _p(err_flag, torch.int32), _s(stream))


NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024  # MSA_NOALLOC_SCRATCH_BYTES in msa.h


def route_topk_noalloc(Qr, Krbar, kr_rnorm, doc_chunk_off, k, topk_idx, topk_score=None, doc_scores=None,
                       err_flag=None, stream=None):
    """msa_route_topk_noalloc: route_topk with the library's fixed scratch instead of a workspace.

    For callers that cannot allocate device memory at call time.  Overlapping
    calls on the GPU race on the shared scratch; see include/msa.h.
    """
    B, Tq, Hr, dr = Qr.shape
    _call("msa_route_topk_noalloc", _dt(Qr), _p(Qr), B, Tq, Hr, dr, _p(Krbar, Qr.dtype),
          _p(kr_rnorm, torch.float32), _p(doc_chunk_off, torch.int64), doc_chunk_off.numel() - 1,
          Krbar.shape[0], k, _p(doc_scores, torch.float32), _p(topk_idx, torch.int32),
          _p(topk_score, torch.float32), _p(err_flag, torch.int32), _s(stream))


def gather(topk_idx, doc_chunk_off, Kbar, Vbar, Kmem, Vmem, mem_len, err_flag=None, stream=None):
    """Step 4: copy the selected documents' chunks (msa_gather).  Kmem [B, Mmax, Hkv, d]."""
    B, k = topk_idx.shape
    _call("msa_gather", _dt(Kbar), _p(topk_idx, torch.int32), B, k, _p(doc_chunk_off, torch.int64),
          doc_chunk_off.numel() - 1, Kbar.shape[0], _p(Kbar, host_ok=True), _p(Vbar, Kbar.dtype, host_ok=True),
          Kbar.shape[1],
          Kbar.shape[2], Kmem.shape[1], _p(Kmem, Kbar.dtype), _p(Vmem, Kbar.dtype),
          _p(mem_len, torch.int32), _p(err_flag, torch.int32), _s(stream))


def state_gather_sum(states, topk_idx, S_ext, err_flag=None, stream=None):
    """Linear (DGA) layers' memory injection (msa_state_gather_sum): S_ext[b] = sum of
    the selected documents' recurrent states.  states [D, ...] bf16 or fp32;
    topk_idx int32 [B, k]; S_ext fp32 [B, ...] with the states' trailing shape."""
    D = states.shape[0]
    S = states.numel() // D if D else 0
    B, k = topk_idx.shape
    if S_ext.numel() != B * S:
        raise ValueError("S_ext must hold one state per query")
    _call("msa_state_gather_sum", _dt(states), _p(states), D, S, _p(topk_idx, torch.int32), B, k,
          _p(S_ext, torch.float32), _p(err_flag, torch.int32), _s(stream))


def sparse_attn_workspace_size(B, Tq, Lloc, Hq, Hkv, d, Mmax) -> int:
    return _lib.load().msa_sparse_attn_workspace_size(B, Tq, Lloc, Hq, Hkv, d, Mmax)


def sparse_attn(Q, Kloc, Vloc, Kmem, Vmem, mem_len, O, lse=None, scale=0.0, ws=None, err_flag=None,
                stream=None):
    """Step 5: attention over [memory ++ causal local] (msa_sparse_attn).  Q [B, Tq, Hq, d]."""
    B, Tq, Hq, d = Q.shape
    _call("msa_sparse_attn", _dt(Q), _p(Q), _p(Kloc, Q.dtype), _p(Vloc, Q.dtype), B, Tq, Kloc.shape[1], Hq,
          Kloc.shape[2], d, _p(Kmem, Q.dtype), _p(Vmem, Q.dtype), _p(mem_len, torch.int32), Kmem.shape[1],
          float(scale), _p(O, Q.dtype), _p(lse, torch.float32), _p(ws),
          0 if ws is None else ws.numel() * ws.element_size(), _p(err_flag, torch.int32), _s(stream))


def sparse_attn_indexed_workspace_size(B, Tq, Lloc, Hq, Hkv, d, k, Mmax) -> int:
    return _lib.load().msa_sparse_attn_indexed_workspace_size(B, Tq, Lloc, Hq, Hkv, d, k, Mmax)


def sparse_attn_indexed(Q, Kloc, Vloc, topk_idx, doc_chunk_off, Kbar, Vbar, Mmax, O, ws, lse=None, scale=0.0,
                        err_flag=None, stream=None):
    """Steps 4+5 fused (msa_sparse_attn_indexed): attention over the selected documents' chunks,
    read in place from the bank K̄ / V̄ [C, Hkv, d] by index, and the causal local rows."""
    B, Tq, Hq, d = Q.shape
    k = topk_idx.shape[1]
    _call("msa_sparse_attn_indexed", _dt(Q), _p(Q), _p(Kloc, Q.dtype), _p(Vloc, Q.dtype), B, Tq, Kloc.shape[1], Hq,
          Kloc.shape[2], d, _p(topk_idx, torch.int32), k, _p(doc_chunk_off, torch.int64), doc_chunk_off.numel() - 1,
          Kbar.shape[0], _p(Kbar, Q.dtype, host_ok=True), _p(Vbar, Q.dtype, host_ok=True), Mmax, float(scale),
          _p(O, Q.dtype), _p(lse, torch.float32), _p(ws), ws.numel() * ws.element_size(),
          _p(err_flag, torch.int32), _s(stream))


def sparse_attn_backward_workspace_size(B, Tq, Hq) -> int:
    return _lib.load().msa_sparse_attn_backward_workspace_size(B, Tq, Hq)


def sparse_attn_backward(Q, Kloc, Vloc, Kmem, Vmem, mem_len, O, lse, dO, dQ, dKloc, dVloc, dKmem, dVmem, ws,
                         scale=0.0, err_flag=None, stream=None):
    """Backward of step 5 (msa_sparse_attn_backward): fp32 gradients of Q, Kloc, Vloc, Kmem, Vmem."""
    B, Tq, Hq, d = Q.shape
    f = torch.float32
    _call("msa_sparse_attn_backward", _dt(Q), _p(Q), _p(Kloc, Q.dtype), _p(Vloc, Q.dtype), B, Tq, Kloc.shape[1], Hq,
          Kloc.shape[2], d, _p(Kmem, Q.dtype), _p(Vmem, Q.dtype), _p(mem_len, torch.int32), Kmem.shape[1],
          float(scale), _p(O, Q.dtype), _p(lse, f), _p(dO, Q.dtype), _p(dQ, f), _p(dKloc, f), _p(dVloc, f),
          _p(dKmem, f), _p(dVmem, f), _p(ws), ws.numel() * ws.element_size(), _p(err_flag, torch.int32), _s(stream))


def gather_backward(topk_idx, doc_chunk_off, dKmem, dVmem, mem_len, dKbar, dVbar, err_flag=None, stream=None):
    """Backward of step 4 (msa_gather_backward): adds the gathered rows' gradients into dKbar / dVbar."""
    B, k = topk_idx.shape
    f = torch.float32
    _call("msa_gather_backward", _p(topk_idx, torch.int32), B, k, _p(doc_chunk_off, torch.int64),
          doc_chunk_off.numel() - 1, dKbar.shape[0], _p(dKmem, f), _p(dVmem, f), _p(mem_len, torch.int32),
          dKbar.shape[1], dKbar.shape[2], dKmem.shape[1], _p(dKbar, f), _p(dVbar, f), _p(err_flag, torch.int32),
          _s(stream))


def route_backward_workspace_size(B, Tq, k) -> int:
    return _lib.load().msa_route_backward_workspace_size(B, Tq, k)


def route_backward(Qr, Krbar, kr_rnorm, doc_chunk_off, topk_idx, d_score, dQr, dKrbar, ws, err_flag=None,
                   stream=None):
    """Backward of step 2 (msa_route_backward): adds the selected documents' routing-score gradients
    d_score [B, k] into dQr [B, Tq, Hr, dr] and dKrbar [C, Hr, dr] (fp32)."""
    B, Tq, Hr, dr = Qr.shape
    k = topk_idx.shape[1]
    f = torch.float32
    _call("msa_route_backward", _dt(Qr), _p(Qr), B, Tq, Hr, dr, _p(Krbar, Qr.dtype), _p(kr_rnorm, f),
          _p(doc_chunk_off, torch.int64), doc_chunk_off.numel() - 1, Krbar.shape[0], k,
          _p(topk_idx, torch.int32), _p(d_score, f), _p(dQr, f), _p(dKrbar, f), _p(ws),
          ws.numel() * ws.element_size(), _p(err_flag, torch.int32), _s(stream))


def layer_forward_workspace_size(B, Tq, Lloc, Hq, Hkv, d, Hr, D, C, k, Mmax) -> int:
    return _lib.load().msa_layer_forward_workspace_size(B, Tq, Lloc, Hq, Hkv, d, Hr, D, C, k, Mmax)


def layer_forward(Qr, Krbar, kr_rnorm, doc_chunk_off, k, Q, Kloc, Vloc, Kbar, Vbar, Mmax, O, topk_idx, ws,
                  lse=None, topk_score=None, doc_scores=None, scale=0.0, err_flag=None, stream=None):
    """Steps 2-5 in one call (msa_layer_forward): route + top-k, then attention over the selected
    documents' chunks read in place from the bank by index (msa_sparse_attn_indexed)."""
    B, Tq, Hr, dr = Qr.shape
    Hq, d = Q.shape[2], Q.shape[3]
    _call("msa_layer_forward", _dt(Qr), _p(Qr), Hr, dr, _p(Krbar, Qr.dtype), _p(kr_rnorm, torch.float32),
          _p(doc_chunk_off, torch.int64), doc_chunk_off.numel() - 1, Krbar.shape[0], k,
          _p(Q, Qr.dtype), _p(Kloc, Qr.dtype), _p(Vloc, Qr.dtype), B, Tq, Kloc.shape[1], Hq, Kloc.shape[2], d,
          _p(Kbar, Qr.dtype, host_ok=True), _p(Vbar, Qr.dtype, host_ok=True), Mmax, float(scale), _p(O, Qr.dtype),
          _p(lse, torch.float32),
          _p(topk_idx, torch.int32), _p(topk_score, torch.float32), _p(doc_scores, torch.float32),
          _p(ws), ws.numel() * ws.element_size(), _p(err_flag, torch.int32), _s(stream))


def interleave_workspace_size(B, Tq, Lloc, Hq, Hkv, d, Hr, dr, D, C, k, rounds, Mmax) -> int:
    return _lib.load().msa_interleave_workspace_size(B, Tq, Lloc, Hq, Hkv, d, Hr, dr, D, C, k, rounds, Mmax)


def interleave_forward(Qr0, Krbar, kr_rnorm, doc_chunk_off, k, rounds, W_route, Q, Kloc, Vloc, Kbar, Vbar, Mmax, O,
                       topk_idx, ws, lse=None, O_rounds=None, Qr_rounds=None, topk_score=None, scale=0.0,
                       err_flag=None, stream=None):
    """Memory Interleave (msa_interleave_forward): `rounds` rounds of route -> k new documents ->
    attention over every round's documents; the next round's router query is O_r x W_route.
    topk_idx int32 [B, rounds * k]; W_route [Hq * d, Hr * dr] (None when rounds == 1)."""
    B, Tq, Hr, dr = Qr0.shape
    Hq, d = Q.shape[2], Q.shape[3]
    _call("msa_interleave_forward", _dt(Qr0), _p(Qr0), Hr, dr, _p(Krbar, Qr0.dtype), _p(kr_rnorm, torch.float32),
          _p(doc_chunk_off, torch.int64), doc_chunk_off.numel() - 1, Krbar.shape[0], k, rounds,
          _p(W_route, Qr0.dtype), _p(Q, Qr0.dtype), _p(Kloc, Qr0.dtype), _p(Vloc, Qr0.dtype), B, Tq, Kloc.shape[1],
          Hq, Kloc.shape[2], d, _p(Kbar, Qr0.dtype, host_ok=True), _p(Vbar, Qr0.dtype, host_ok=True), Mmax,
          float(scale), _p(O, Qr0.dtype), _p(lse, torch.float32), _p(O_rounds, Qr0.dtype), _p(Qr_rounds, Qr0.dtype),
          _p(topk_idx, torch.int32), _p(topk_score, torch.float32), _p(ws), ws.numel() * ws.element_size(),
          _p(err_flag, torch.int32), _s(stream))


def gated_delta_rule(q, k, v, g, beta, o, h0=None, hT=None, scale=0.0, stream=None):
    """The linear (DGA) layers' query path (msa_gated_delta_rule): the gated delta rule over the
    query tokens from the initial state h0 (S_ext).  q, k [B, T, Hk, 128]; v, o [B, T, Hv, 128];
    g, beta fp32 [B, T, Hv]; h0, hT fp32 [B, Hv, 128, 128] or None."""
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    f = torch.float32
    _call("msa_gated_delta_rule", _dt(q), _p(q), _p(k, q.dtype), _p(v, q.dtype), _p(g, f), _p(beta, f), B, T, Hk, Hv,
          dk, dv, _p(h0, f), float(scale), _p(o, q.dtype), _p(hT, f), _s(stream))


# ---- rotary positions and the paged cache of the local keys and values
# A decoding step calls these for every layer, so each tensor is looked at once.  All tensors are on
# the current device (one on another is refused), and the work goes to its current stream or `stream`.


# The first line of each check is the whole of it for a good tensor; what is wrong is found after.
_cuda_dev = torch._C._cuda_getDevice
_cuda_stream = torch._C._cuda_getCurrentRawStream


def _refuse(t, name, dtype, dev, shape):
    if t.get_device() != dev:
        raise ValueError(f"{name} is not on the current CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _at(t, name, dtype, dev, shape=None):
    """Device pointer of a contiguous tensor of this dtype (and shape) on the current device."""
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    _refuse(t, name, dtype, dev, shape)


def _rows_at(t, name, dtype, dev, shape):
    """Strides of a tensor whose last dimension alone has to be contiguous."""
    st = t.stride()
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape and st[-1] == 1:
        return st
    if t.shape == shape and shape[-1] == 1 and t.dtype == dtype and t.get_device() == dev:
        return st
    _refuse(t, f"the last dimension of {name}" if t.shape == shape else name, dtype, dev, shape)


def _heads_at(t, name, dtype, dev, shape):
    """Token stride of rows [N, H, d] whose heads follow one another."""
    st = _rows_at(t, name, dtype, dev, shape)
    if st[1] != shape[2] and shape[1] > 1:
        raise ValueError(f"the heads of {name} must be contiguous")
    return st[0]


def rope_table_scaled(method: str, theta: float, rd: int, max_len: int, factor: float = 1.0, orig_len: float = 0.0,
                      lo: float = 0.0, hi: float = 0.0) -> torch.Tensor:
    """Host fp32 [max_len, rd/2, 2] table with angles scaled for longer contexts
    (msa_rope_table_scaled_host); method: a key of ROPE_SCALES."""
    if method not in ROPE_SCALES:
        raise ValueError(f"unknown method {method!r}: one of {sorted(ROPE_SCALES)}")
    out = torch.empty((max(max_len, 0), max(rd, 0) // 2, 2), dtype=torch.float32)
    _call("msa_rope_table_scaled_host", ROPE_SCALES[method], float(theta), rd, max_len, float(factor),
          float(orig_len), float(lo), float(hi), out.data_ptr())
    return out


def _rope(fn, x, pos, rope_cs, out, layout, err_flag, stream):
    dt, dev, dtype = _dt(x), _cuda_dev(), x.dtype
    N, H, d = shape = x.shape
    xs, os = _rows_at(x, "x", dtype, dev, shape), _rows_at(out, "out", dtype, dev, shape)
    max_len, half, two = rope_cs.shape
    if two != 2:
        raise ValueError("rope_cs must be [max_len, rd/2, 2]")
    _call(fn, dt, x.data_ptr(), xs[0], xs[1], N, H, d, _at(pos, "pos", torch.int32, dev, (N,)),
          _at(rope_cs, "rope_cs", torch.float32, dev), max_len, 2 * half, layout, out.data_ptr(), os[0], os[1],
          None if err_flag is None else _at(err_flag, "err_flag", torch.int32, dev),
          _cuda_stream(dev) if stream is None else stream.cuda_stream)


def rope(x, pos, rope_cs, out, layout=ROPE_HALF, err_flag=None, stream=None):
    """Rotary positions (msa_rope): the first 2 * rope_cs.shape[1] dimensions of every head of x
    [N, H, d] rotated by position pos int32 [N] into out (which may be x).  x and out may be
    strided views; the last dimension is contiguous."""
    _rope("msa_rope", x, pos, rope_cs, out, layout, err_flag, stream)


def rope_backward(dout, pos, rope_cs, dx, layout=ROPE_HALF, err_flag=None, stream=None):
    """Backward of rope (msa_rope_backward): dx from dout by the transposed rotation."""
    _rope("msa_rope_backward", dout, pos, rope_cs, dx, layout, err_flag, stream)


def _cache(Kpages, Vpages, block_table, seq_len, q_off, Hkv, d, dtype, dev):
    """The batch and cache arguments both paged entry points take, checked: B, the pointer of
    q_off, K, V and the rest in the order of the C signature."""
    shape = Kpages.shape
    if shape[2:] != (Hkv, d):
        raise ValueError(f"Kpages must be [num_pages, page, {Hkv}, {d}], not {tuple(shape)}")
    ks = _rows_at(Kpages, "Kpages", dtype, dev, shape)
    if _rows_at(Vpages, "Vpages", dtype, dev, shape) != ks:
        raise ValueError("Kpages and Vpages must have the same strides")
    B, = seq_len.shape
    max_pages = block_table.shape[-1]
    return (B, _at(q_off, "q_off", torch.int64, dev, (B + 1,)), Kpages.data_ptr(), Vpages.data_ptr(), shape[0],
            shape[1], ks[0], ks[1], ks[2], _at(block_table, "block_table", torch.int32, dev, (B, max_pages)),
            max_pages, _at(seq_len, "seq_len", torch.int32, dev))


def paged_append(q, k, v, q_off, seq_len, block_table, Kpages, Vpages, rope_cs=None, q_out=None, pos=None,
                 layout=ROPE_HALF, err_flag=None, stream=None):
    """New tokens into the paged cache (msa_paged_append): k (rotated) and v [N, Hkv, d] into the
    pages [num_pages, page, Hkv, d] (any strides) of their sequences, q (rotated) into q_out.
    q may be None; rope_cs None: no rotation; pos None: cache positions."""
    dt, dev, dtype = _dt(k), _cuda_dev(), k.dtype
    N, Hkv, d = shape = k.shape
    ks, vs = _heads_at(k, "k", dtype, dev, shape), _heads_at(v, "v", dtype, dev, shape)
    qp = qop = csp = None
    qs = qos = Hq = max_len = half = 0
    if q is not None or q_out is not None:
        if q is None or q_out is None:
            raise ValueError("q and q_out go together")
        Hq = q.shape[1]
        qs, qos = _heads_at(q, "q", dtype, dev, (N, Hq, d)), _heads_at(q_out, "q_out", dtype, dev, (N, Hq, d))
        qp, qop = q.data_ptr(), q_out.data_ptr()
    if rope_cs is not None:
        max_len, half, two = rope_cs.shape
        if two != 2:
            raise ValueError("rope_cs must be [max_len, rd/2, 2]")
        csp = _at(rope_cs, "rope_cs", torch.float32, dev)
    B, qo, *cache = _cache(Kpages, Vpages, block_table, seq_len, q_off, Hkv, d, dtype, dev)
    _call("msa_paged_append", dt, qp, qs, qop, qos, Hq, k.data_ptr(), ks, v.data_ptr(), vs, N, B, qo, Hkv, d,
          None if pos is None else _at(pos, "pos", torch.int32, dev, (N,)), csp, max_len, 2 * half, layout, *cache,
          None if err_flag is None else _at(err_flag, "err_flag", torch.int32, dev),
          _cuda_stream(dev) if stream is None else stream.cuda_stream)


def paged_attn_workspace_size(dtype, B, max_q, Hq, Hkv, d, k=0, Mmax=0) -> int:
    return _lib.load().msa_paged_attn_workspace_size(DTYPES[dtype], B, max_q, Hq, Hkv, d, k, Mmax)


def paged_attn(Q, q_off, max_q, Kpages, Vpages, block_table, seq_len, O, ws, lse=None, scale=0.0, topk_idx=None,
               doc_chunk_off=None, Kbar=None, Vbar=None, Mmax=0, err_flag=None, stream=None):
    """Attention of new tokens over [selected memory rows ++ paged cache] (msa_paged_attn): Q
    [N, Hq, d] packed by q_off int64 [B + 1] (at most max_q tokens a sequence), pages
    [num_pages, page, Hkv, d] (any strides), O [N, Hq, d], lse fp32 [Hq, N].  topk_idx int32 [B, k]
    with doc_chunk_off, Kbar and Vbar adds the selected documents' rows (at most Mmax)."""
    dt, dev, dtype = _dt(Q), _cuda_dev(), Q.dtype
    N, Hq, d = shape = Q.shape
    Hkv = Kpages.shape[2]
    qs = _heads_at(Q, "Q", dtype, dev, shape)
    B, qo, *cache = _cache(Kpages, Vpages, block_table, seq_len, q_off, Hkv, d, dtype, dev)
    idx = off = kb = vb = None
    k = D = C = 0
    if topk_idx is not None:
        if doc_chunk_off is None or Kbar is None or Vbar is None:
            raise ValueError("topk_idx goes with doc_chunk_off, Kbar and Vbar")
        k, D, C = topk_idx.shape[-1], doc_chunk_off.numel() - 1, Kbar.shape[0]
        idx = _at(topk_idx, "topk_idx", torch.int32, dev, (B, k))
        off = _at(doc_chunk_off, "doc_chunk_off", torch.int64, dev)
        kb, vb = _at(Kbar, "Kbar", dtype, dev, (C, Hkv, d)), _at(Vbar, "Vbar", dtype, dev, (C, Hkv, d))
    _call("msa_paged_attn", dt, Q.data_ptr(), qs, N, B, max_q, qo, Hq, Hkv, d, *cache, idx, k, off, D, C, kb, vb, Mmax,
          scale, _at(O, "O", dtype, dev, shape),
          None if lse is None else _at(lse, "lse", torch.float32, dev, (Hq, N)), _at(ws, "ws", ws.dtype, dev),
          ws.nbytes, None if err_flag is None else _at(err_flag, "err_flag", torch.int32, dev),
          _cuda_stream(dev) if stream is None else stream.cuda_stream)
