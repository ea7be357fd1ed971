"""Python binding of the attention sublayer's calls (include/mhc.h): per-head
query/key norm with the rotary rotation, masked attention over packed
documents with its backward, and attention of new tokens over a paged cache.

Argument marshalling only, in the manner of :mod:`residual_stream_amd.mhc`:
every step runs in the gfx950 kernels of ``libmhc.so`` on torch's current
stream, outputs and workspaces are torch's, and there is no CPU path.

Head tensors are [T, H, Dh] in float32 or bfloat16 with contiguous heads and
any token stride that is a multiple of 8 elements, so q, k and v may be views
of one projection's output (``qkv[:, :Hq*Dh].unflatten(1, (Hq, Dh))``), and
gradients passed in ``out`` views of its gradient.  Query head h reads key
head ``h // (Hq // Hk)``.
"""

from __future__ import annotations

import ctypes

import torch

from . import mhc
from .mhc import MhcAttnDesc, MhcPagedDesc, MhcRopeDesc, _check, _expect, _io_of, _stream, _workspace, _ws_bytes, load


def _head_tensor(name, t, shape=None, dtype=None, device=None):
    """Checks one [T, H, Dh] tensor; returns its token stride in elements."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a [T, H, Dh] tensor")
    if not t.is_cuda:
        raise RuntimeError("the mHC kernels need GPU tensors (no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    T, H, D = t.shape
    if (D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D):
        raise ValueError(f"{name}'s heads must be contiguous (only the token stride is free)")
    ld = t.stride(0) if T > 1 else H * D
    if ld < H * D or ld % 8:
        raise ValueError(f"{name}'s token stride {ld} must be a multiple of 8 and at least {H * D}")
    if t.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned")
    return ld


def _queries(q):
    """(T, Hq, Dh, dtype, device) of the query tensor."""
    _head_tensor("q", q)
    _io_of(q)
    if q.device.index != torch.cuda.current_device():
        raise ValueError(f"q is on {q.device}; make it the current device first")
    return (*q.shape, q.dtype, q.device)


def _grouped(Hq, Hk):
    if Hk < 1 or Hq % Hk:
        raise ValueError(f"{Hq} query heads cannot share {Hk} key heads evenly")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _vec(name, t, n, dtype, device, optional=True):
    _expect(name, t, (n,), dtype, device, optional=optional)


def rope_freqs(rotated: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """base^(-2i/rotated) for i < rotated/2, float64: radians per position."""
    return base ** (-torch.arange(0, rotated, 2, dtype=torch.float64, device=device) / rotated)


def _rope_desc(q, k, positions, freqs, q_weight, k_weight, eps, interleaved):
    T, Hq, Dh, io, dv = _queries(q)
    Hk = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 3 else 0
    ldk = _head_tensor("k", k, (T, Hk, Dh), io, dv)
    _grouped(Hq, Hk)
    _vec("positions", positions, T, torch.int32, dv, optional=False)
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise ValueError("freqs must be a [R/2] tensor")
    _vec("freqs", freqs, freqs.shape[0], torch.float64, dv, optional=False)
    _vec("q_weight", q_weight, Dh, torch.float32, dv)
    _vec("k_weight", k_weight, Dh, torch.float32, dv)
    return MhcRopeDesc(T=T, Hq=Hq, Hk=Hk, Dh=Dh, R=2 * freqs.shape[0], io=_io_of(q), interleaved=int(bool(interleaved)),
                       eps=float(eps), ldq=_head_tensor("q", q), ldk=ldk, ldv=Hk * Dh, ldq_out=Hq * Dh, ldk_out=Hk * Dh,
                       ld_dq=Hq * Dh, ld_dk=Hk * Dh)


def mhc_qk_rope(q, k, positions, freqs, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, out=None,
                stream=None):
    """RMSNorm of every head row of q[T,Hq,Dh] and k[T,Hk,Dh] (weights [Dh] fp32,
    or None for ones), then the rotation of its first 2·len(freqs) elements by
    positions[T] (int32) times freqs (float64, :func:`rope_freqs`).

    Returns (q_out[T,Hq,Dh], k_out[T,Hk,Dh])."""
    lib = load()
    d = _rope_desc(q, k, positions, freqs, q_weight, k_weight, eps, interleaved)
    if out is None:
        out = tuple(torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k))
    qo, ko = out
    d.ldq_out = _head_tensor("q_out", qo, q.shape, q.dtype, q.device)
    d.ldk_out = _head_tensor("k_out", ko, k.shape, q.dtype, q.device)
    _check(lib.mhc_qk_rope(ctypes.byref(d), _p(q), _p(k), _p(positions), _p(freqs), _p(q_weight), _p(k_weight), _p(qo),
                           _p(ko), _stream(stream)), "mhc_qk_rope")
    return out


def mhc_qk_rope_bwd(dq_out, dk_out, q, k, positions, freqs, *, q_weight=None, k_weight=None, eps=1e-6,
                    interleaved=False, out=None, workspace=None, stream=None):
    """Backward of :func:`mhc_qk_rope` from its inputs: returns (dq, dk,
    dq_weight[Dh] or None, dk_weight[Dh] or None), the weights' gradients in
    fp32 summed over tokens and heads."""
    lib = load()
    d = _rope_desc(q, k, positions, freqs, q_weight, k_weight, eps, interleaved)
    dv = q.device
    d.ldq_out = _head_tensor("dq_out", dq_out, q.shape, q.dtype, dv)
    d.ldk_out = _head_tensor("dk_out", dk_out, k.shape, q.dtype, dv)
    if out is None:
        out = tuple(torch.empty(t.shape, dtype=t.dtype, device=dv) for t in (q, k)) + tuple(
            None if w is None else torch.empty_like(w) for w in (q_weight, k_weight))
    dq, dk, dqw, dkw = out
    d.ld_dq = _head_tensor("dq", dq, q.shape, q.dtype, dv)
    d.ld_dk = _head_tensor("dk", dk, k.shape, q.dtype, dv)
    for name, g, w in (("dq_weight", dqw, q_weight), ("dk_weight", dkw, k_weight)):
        if g is not None and w is None:
            raise ValueError(f"{name} without the weight itself")
        _vec(name, g, q.shape[2], torch.float32, dv)
    need = lib.mhc_qk_rope_bwd_workspace_bytes(ctypes.byref(d))
    if workspace is None and need:
        workspace = _workspace(need, dv)
    nbytes = _ws_bytes(workspace)
    _check(lib.mhc_qk_rope_bwd(ctypes.byref(d), _p(dq_out), _p(dk_out), _p(q), _p(k), _p(positions), _p(freqs),
                               _p(q_weight), _p(k_weight), _p(dq), _p(dk), _p(dqw), _p(dkw), _p(workspace), nbytes,
                               _stream(stream)), "mhc_qk_rope_bwd")
    return out


def _cache(k_cache, v_cache, Hk, Dh, dtype, device):
    """(pages, page size) of the two caches [pages, page_size, Hk, Dh]."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a [pages, page_size, Hk, Dh] tensor")
    pages, size = k_cache.shape[:2]
    _expect("k_cache", k_cache, (pages, size, Hk, Dh), dtype, device)
    _expect("v_cache", v_cache, (pages, size, Hk, Dh), dtype, device)
    return pages, size


def mhc_qk_rope_cache(q, k, v, positions, freqs, k_cache, v_cache, slots, *, q_weight=None, k_weight=None, eps=1e-6,
                      interleaved=False, out=None, stream=None):
    """The serving form of :func:`mhc_qk_rope`: the normed and rotated keys, and
    the values as they are, go to place slots[t] (int64, page·page_size + offset)
    of the caches [pages, page_size, Hk, Dh]; a slot outside them (-1 for a
    padded token) writes nothing.  Slots of one call must differ.  Returns
    q_out[T,Hq,Dh]."""
    lib = load()
    d = _rope_desc(q, k, positions, freqs, q_weight, k_weight, eps, interleaved)
    dv = q.device
    d.ldv = _head_tensor("v", v, k.shape, q.dtype, dv)
    pages, size = _cache(k_cache, v_cache, d.Hk, d.Dh, q.dtype, dv)
    _vec("slots", slots, d.T, torch.int64, dv, optional=False)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dv)
    d.ldq_out = _head_tensor("q_out", out, q.shape, q.dtype, dv)
    _check(lib.mhc_qk_rope_cache(ctypes.byref(d), _p(q), _p(k), _p(v), _p(positions), _p(freqs), _p(q_weight),
                                 _p(k_weight), _p(out), _p(k_cache), _p(v_cache), _p(slots), pages * size,
                                 _stream(stream)), "mhc_qk_rope_cache")
    return out


def _constant(name, t):
    if t is not None and isinstance(t, torch.Tensor) and t.requires_grad:
        raise ValueError(f"{name} takes no gradient: detach it")


def _attn_desc(q, k, v, docs, causal, prefix, window, softcap, slopes, scale):
    T, Hq, Dh, io, dv = _queries(q)
    Hk = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 3 else 0
    ldk = _head_tensor("k", k, (T, Hk, Dh), io, dv)
    ldv = _head_tensor("v", v, (T, Hk, Dh), io, dv)
    _grouped(Hq, Hk)
    n = 1
    if docs is not None:
        if not isinstance(docs, torch.Tensor) or docs.dim() != 1 or docs.shape[0] < 2:
            raise ValueError("docs must be a [n_docs + 1] tensor of row offsets")
        n = docs.shape[0] - 1
        _vec("docs", docs, n + 1, torch.int32, dv)
    _vec("prefix", prefix, n, torch.int32, dv)
    _vec("slopes", slopes, Hq, torch.float32, dv)
    _constant("slopes", slopes)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    return MhcAttnDesc(T=T, Hq=Hq, Hk=Hk, Dh=Dh, io=_io_of(q), n_docs=n, causal=int(bool(causal)), window=int(window),
                       fill_outside=0, scale=float(Dh ** -0.5 if scale is None else scale), softcap=float(softcap),
                       docs=ptr(docs), prefix=ptr(prefix), slopes=ptr(slopes), ldq=_head_tensor("q", q), ldk=ldk, ldv=ldv,
                       ldo=Hq * Dh, ld_do=Hq * Dh, ld_dq=Hq * Dh, ld_dk=Hk * Dh, ld_dv=Hk * Dh)


def saved_floats(T: int, Hq: int, Dh: int, io: int) -> int:
    """Length of the fp32 tensor in which :func:`mhc_attn` keeps what its backward
    needs: the log-sum-exps [Hq, T] and, for bf16, the next eight bits of every
    element of o (one byte each, from the next multiple of four floats on)."""
    lse = -(-Hq * T // 4) * 4
    return lse + (T * Hq * Dh // 4 if io == mhc.MHC_BF16 else 0)


def _saved(name, saved, d, device):
    """(lse, o_rest) pointers within the saved tensor."""
    n = saved_floats(d.T, d.Hq, d.Dh, d.io)
    _expect(name, saved, (n,), torch.float32, device)
    lse = saved.data_ptr()
    return ctypes.c_void_p(lse), (ctypes.c_void_p(lse + (-(-d.Hq * d.T // 4) * 16)) if d.io == mhc.MHC_BF16 else None)


def mhc_attn(q, k, v, *, docs=None, causal=True, prefix=None, window=0, softcap=0.0, slopes=None, scale=None, out=None,
             stream=None):
    """Attention of q[T,Hq,Dh] over k, v[T,Hk,Dh] (Dh 64 or 128) of a packed
    batch: docs (int32 [n+1], sorted) holds the documents' first rows and the
    end of the last, None is one document of all rows.  Row i sees its own
    document's keys j ≤ i (all of them with causal=False), with window > 0 only
    i - j < window, with prefix (int32 [n]) also the document's first prefix[d]
    keys.  Scores are scale·q·k (scale: Dh^-0.5 if None), capped to
    softcap·tanh(·/softcap) if softcap > 0, minus slopes[h]·|i - j| (fp32 [Hq]).

    Returns (o[T,Hq,Dh], saved), ``saved`` an fp32 tensor of
    :func:`saved_floats` elements for the backward; its first Hq·T are the rows'
    log-sum-exps [Hq, T].  Rows of no document come out as zeros (lse -inf); in
    tensors passed as ``out=(o, saved or None)`` they are left as they were."""
    lib = load()
    d = _attn_desc(q, k, v, docs, causal, prefix, window, softcap, slopes, scale)
    if out is None:
        d.fill_outside = 1
        out = (torch.empty(q.shape, dtype=q.dtype, device=q.device),
               torch.empty(saved_floats(d.T, d.Hq, d.Dh, d.io), dtype=torch.float32, device=q.device))
    o, saved = out
    d.ldo = _head_tensor("o", o, q.shape, q.dtype, q.device)
    lse, rest = (None, None) if saved is None else _saved("saved", saved, d, q.device)
    _check(lib.mhc_attn(ctypes.byref(d), _p(q), _p(k), _p(v), _p(o), lse, rest, _stream(stream)), "mhc_attn")
    return out


def mhc_attn_bwd(do, q, k, v, o, saved, *, docs=None, causal=True, prefix=None, window=0, softcap=0.0, slopes=None,
                 scale=None, out=None, workspace=None, stream=None):
    """Backward of :func:`mhc_attn` from its inputs and results: returns (dq, dk,
    dv), dk and dv summed over the query heads that share a key head.  Rows of
    no document get zeros, or are left as they were in tensors passed as
    ``out``."""
    lib = load()
    d = _attn_desc(q, k, v, docs, causal, prefix, window, softcap, slopes, scale)
    dv = q.device
    d.ld_do = _head_tensor("do", do, q.shape, q.dtype, dv)
    d.ldo = _head_tensor("o", o, q.shape, q.dtype, dv)
    lse, rest = _saved("saved", saved, d, dv)
    if out is None:
        d.fill_outside = 1
        out = tuple(torch.empty(t.shape, dtype=t.dtype, device=dv) for t in (q, k, v))
    d.ld_dq, d.ld_dk, d.ld_dv = (_head_tensor(n, g, t.shape, q.dtype, dv)
                                 for n, g, t in zip(("dq", "dk", "dv"), out, (q, k, v)))
    need = lib.mhc_attn_bwd_workspace_bytes(ctypes.byref(d))
    if workspace is None and need:
        workspace = _workspace(need, dv)
    nbytes = _ws_bytes(workspace)
    _check(lib.mhc_attn_bwd(ctypes.byref(d), _p(do), _p(q), _p(k), _p(v), _p(o), lse, rest, *(_p(g) for g in out),
                            _p(workspace), nbytes, _stream(stream)), "mhc_attn_bwd")
    return out


def mhc_attn_paged(q, k_cache, v_cache, pages, kv_lens, *, cu_q=None, max_q=None, prefix=None, window=0, softcap=0.0,
                   slopes=None, scale=None, out=None, workspace=None, stream=None):
    """Attention of new tokens over a paged cache [num_pages, page_size, Hk, Dh]
    that already holds their own keys and values (:func:`mhc_qk_rope_cache`).

    pages[n, max_pages] (int32) is each sequence's page table, kv_lens[n]
    (int32) its keys with the new ones.  Without cu_q, row s of q[T,Hq,Dh] is
    sequence s's next token; with cu_q (int32 [n+1], sorted) rows cu_q[s] ..
    cu_q[s+1]-1 are its last tokens, at most max_q of them (a host number; T if
    None: give the longest chunk, the grid is sized by it).  Masks and scores as
    :func:`mhc_attn`, positions counted within each sequence.

    Returns o[T,Hq,Dh]; a row without a key gets zeros, a row whose keys lie in
    a page outside the cache NaN; rows of no sequence get zeros, or are left as
    they were in a tensor passed as ``out``."""
    lib = load()
    T, Hq, Dh, io, dv = _queries(q)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a [pages, page_size, Hk, Dh] tensor")
    Hk = k_cache.shape[2]
    _grouped(Hq, Hk)
    num, size = _cache(k_cache, v_cache, Hk, Dh, io, dv)
    if not isinstance(pages, torch.Tensor) or pages.dim() != 2:
        raise ValueError("pages must be a [n, max_pages] tensor")
    n, width = pages.shape
    _expect("pages", pages, (n, width), torch.int32, dv)
    _vec("kv_lens", kv_lens, n, torch.int32, dv, optional=False)
    _vec("cu_q", cu_q, n + 1, torch.int32, dv)
    _vec("prefix", prefix, n, torch.int32, dv)
    _vec("slopes", slopes, Hq, torch.float32, dv)
    _constant("slopes", slopes)
    if cu_q is None:
        if n > T:
            raise ValueError(f"{n} sequences but {T} rows (pass cu_q for chunks)")
        if max_q not in (None, 1):
            raise ValueError("max_q above 1 needs cu_q")
        max_q = 1
    elif max_q is None:
        max_q = max(T, 1)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    d = MhcPagedDesc(T=T, n_seqs=n, max_q=int(max_q), Hq=Hq, Hk=Hk, Dh=Dh, io=_io_of(q), window=int(window),
                     page_size=size, max_pages=width, fill_outside=int(out is None), num_pages=num,
                     scale=float(Dh ** -0.5 if scale is None else scale), softcap=float(softcap), cu_q=ptr(cu_q),
                     kv_lens=ptr(kv_lens), pages=ptr(pages), prefix=ptr(prefix), slopes=ptr(slopes),
                     ldq=_head_tensor("q", q), ldo=Hq * Dh)
    if out is None:
        out = torch.empty(q.shape, dtype=io, device=dv) if n else torch.zeros(q.shape, dtype=io, device=dv)
    d.ldo = _head_tensor("o", out, q.shape, io, dv)
    need = lib.mhc_attn_paged_workspace_bytes(ctypes.byref(d))
    if workspace is None and need:
        workspace = _workspace(need, dv)
    nbytes = _ws_bytes(workspace)
    _check(lib.mhc_attn_paged(ctypes.byref(d), _p(q), _p(k_cache), _p(v_cache), _p(out), _p(workspace), nbytes,
                              _stream(stream)), "mhc_attn_paged")
    return out
