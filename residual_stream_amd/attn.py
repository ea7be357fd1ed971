"""Python binding of the attention sublayer's calls (include/mhc.h): per-head
query/key norm with the rotary rotation, masked attention over packed
documents with its backward, and attention of new tokens over a paged cache.

Argument marshalling only, in the manner of :mod:`residual_stream_amd.mhc`:
every step runs in the gfx950 kernels of ``libmhc.so`` on torch's current
stream, outputs and workspaces are torch's, and there is no CPU path.  With
``stream`` a call is made as within ``torch.cuda.stream(stream)``: it runs
there, and the tensors it makes belong to that stream (the inputs must be ready
on it).

Head tensors are [T, H, Dh] in float32 or bfloat16 with contiguous heads and
any token stride that is a multiple of 8 elements, so q, k and v may be views
of one projection's output (``qkv[:, :Hq*Dh].unflatten(1, (Hq, Dh))``), and
gradients passed in ``out`` views of its gradient.  Query head h reads key
head ``h // (Hq // Hk)``.

A decode step makes these calls once a layer, so the checks are kept short:
each takes one look at a tensor and words its refusal only when there is one.
"""

from __future__ import annotations

import ctypes

import torch

from . import mhc
from .mhc import MhcAttnDesc, MhcPagedDesc, MhcRopeDesc, _check, _workspace, _ws_bytes, load

_IO = {torch.float32: mhc.MHC_F32, torch.bfloat16: mhc.MHC_BF16}
_ref = ctypes.byref


def _refuse(name, t, shape, dtype, dev):
    """Words what is wrong with one tensor argument."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise RuntimeError("the mHC kernels need GPU tensors (no CPU path)")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() == 3 and not t.is_contiguous():
        raise ValueError(f"{name}'s heads must be contiguous, its token stride a multiple of 8 and at least H·Dh "
                         f"(strides {t.stride()})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be 16-byte aligned")


def _heads(name, t, shape, dtype, dev):
    """Token stride in elements of a [T, H, Dh] tensor."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.shape != shape or t.dtype != dtype:
        _refuse(name, t, shape, dtype, dev)
    T, H, D = shape
    ld, sh, sd = t.stride()
    if T <= 1:
        ld = H * D
    if (sh != D and H > 1) or sd != 1 or ld < H * D or ld & 7 or (t.data_ptr() & 15 and T):
        _refuse(name, t, shape, dtype, dev)
    return ld


def _vec(name, t, shape, dtype, dev):
    """Address of a contiguous tensor, None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.shape != shape or t.dtype != dtype \
            or not t.is_contiguous():
        _refuse(name, t, shape, dtype, dev)
    return t.data_ptr()


def _need(name, t):
    if t is None:
        raise ValueError(f"{name} is required")
    return t


def _queries(q):
    """(shape, dtype, io, device index) of the query tensor."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [T, H, Dh] tensor")
    if not q.is_cuda:
        raise RuntimeError("the mHC kernels need GPU tensors (no CPU path)")
    io = _IO.get(q.dtype)
    if io is None:
        raise TypeError(f"I/O tensors must be float32 or bfloat16, got {q.dtype}")
    dev = q.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"q is on {q.device}; make it the current device first")
    return q.shape, q.dtype, io, dev


def _key_shape(k, q_shape):
    """Shape that k and v must have: their own number of heads, which the query heads share evenly."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be a [T, H, Dh] tensor")
    Hk = k.shape[1]
    if Hk < 1 or q_shape[1] % Hk:
        raise ValueError(f"{q_shape[1]} query heads cannot share {Hk} key heads evenly")
    return torch.Size((q_shape[0], Hk, q_shape[2]))


def _like(t):
    """An uninitialised contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _within(stream, call, args):
    """``call`` as made within ``torch.cuda.stream(stream)``: its output and
    workspace then come from that stream's memory, where nothing else can take
    them while the kernels run."""
    args["stream"] = None
    with torch.cuda.stream(stream):
        return call(**args)


def _scratch(need, workspace, device):
    """(address, bytes, tensor) of a workspace: the caller's, or one for this call."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = _workspace(need, device)
        return workspace.data_ptr(), need, workspace
    nbytes = _ws_bytes(workspace)
    if workspace.device != device:
        raise ValueError(f"the workspace is on {workspace.device}, expected {device}")
    return workspace.data_ptr(), nbytes, workspace


def rope_freqs(rotated: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """base^(-2i/rotated) for i < rotated/2, float64: radians per position."""
    return base ** (-torch.arange(0, rotated, 2, dtype=torch.float64, device=device) / rotated)


def _rope(q, k, positions, freqs, q_weight, k_weight, eps, interleaved):
    """(descriptor, key shape, addresses of q, k, positions, freqs and weights, dtype, device) of a rope call."""
    shape, dtype, io, dev = _queries(q)
    T, Hq, Dh = shape
    ks = _key_shape(k, shape)
    Hk = ks[1]
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise ValueError("freqs must be a [R/2] tensor")
    half = freqs.shape[0]
    d = MhcRopeDesc(T, Hq, Hk, Dh, 2 * half, io, 1 if interleaved else 0, eps, 0, _heads("q", q, shape, dtype, dev),
                    _heads("k", k, ks, dtype, dev), Hk * Dh, Hq * Dh, Hk * Dh, Hq * Dh, Hk * Dh)
    at = (q.data_ptr(), k.data_ptr(), _vec("positions", _need("positions", positions), (T,), torch.int32, dev),
          _vec("freqs", freqs, (half,), torch.float64, dev), _vec("q_weight", q_weight, (Dh,), torch.float32, dev),
          _vec("k_weight", k_weight, (Dh,), torch.float32, dev))
    return d, ks, at, dtype, dev


def mhc_qk_rope(q, k, positions, freqs, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, out=None,
                stream=None):
    """RMSNorm of every head row of q[T,Hq,Dh] and k[T,Hk,Dh] (weights [Dh] fp32,
    or None for ones), then the rotation of its first 2·len(freqs) elements by
    positions[T] (int32) times freqs (float64, :func:`rope_freqs`).

    Returns (q_out[T,Hq,Dh], k_out[T,Hk,Dh])."""
    if stream is not None:
        return _within(stream, mhc_qk_rope, locals())
    lib = load()
    d, ks, at, dtype, dev = _rope(q, k, positions, freqs, q_weight, k_weight, eps, interleaved)
    if out is None:
        out = (_like(q), _like(k))
        qo, ko = out
    else:
        qo, ko = out
        d.ldq_out = _heads("q_out", qo, q.shape, dtype, dev)
        d.ldk_out = _heads("k_out", ko, ks, dtype, dev)
    _check(lib.mhc_qk_rope(_ref(d), *at, qo.data_ptr(), ko.data_ptr(), torch._C._cuda_getCurrentRawStream(dev)), "mhc_qk_rope")
    return out


def mhc_qk_rope_bwd(dq_out, dk_out, q, k, positions, freqs, *, q_weight=None, k_weight=None, eps=1e-6,
                    interleaved=False, out=None, workspace=None, stream=None):
    """Backward of :func:`mhc_qk_rope` from its inputs: returns (dq, dk,
    dq_weight[Dh] or None, dk_weight[Dh] or None), the weights' gradients in
    fp32 summed over tokens and heads."""
    if stream is not None:
        return _within(stream, mhc_qk_rope_bwd, locals())
    lib = load()
    d, ks, at, dtype, dev = _rope(q, k, positions, freqs, q_weight, k_weight, eps, interleaved)
    d.ldq_out = _heads("dq_out", dq_out, q.shape, dtype, dev)
    d.ldk_out = _heads("dk_out", dk_out, ks, dtype, dev)
    if out is None:
        out = (_like(q), _like(k), None if q_weight is None else _like(q_weight), None if k_weight is None else _like(k_weight))
        dq, dk, dqw, dkw = out
        grads = (None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr())
    else:
        dq, dk, dqw, dkw = out
        d.ld_dq = _heads("dq", dq, q.shape, dtype, dev)
        d.ld_dk = _heads("dk", dk, ks, dtype, dev)
        if (dqw is not None and q_weight is None) or (dkw is not None and k_weight is None):
            raise ValueError("a weight's gradient without the weight itself")
        row = (q.shape[2],)
        grads = (_vec("dq_weight", dqw, row, torch.float32, dev), _vec("dk_weight", dkw, row, torch.float32, dev))
    ws, nbytes, _keep = _scratch(lib.mhc_qk_rope_bwd_workspace_bytes(_ref(d)), workspace, q.device)
    _check(lib.mhc_qk_rope_bwd(_ref(d), dq_out.data_ptr(), dk_out.data_ptr(), *at, dq.data_ptr(), dk.data_ptr(), *grads,
                               ws, nbytes, torch._C._cuda_getCurrentRawStream(dev)), "mhc_qk_rope_bwd")
    return out


def _cache(k_cache, v_cache, Hk, Dh, dtype, dev):
    """(pages, page size) of the two caches [pages, page_size, Hk, Dh], and their addresses."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a [pages, page_size, Hk, Dh] tensor")
    pages, size = k_cache.shape[:2]
    shape = (pages, size, Hk, Dh)
    return pages, size, _vec("k_cache", k_cache, shape, dtype, dev), _vec("v_cache", _need("v_cache", v_cache), shape, dtype, dev)


def mhc_qk_rope_cache(q, k, v, positions, freqs, k_cache, v_cache, slots, *, q_weight=None, k_weight=None, eps=1e-6,
                      interleaved=False, out=None, stream=None):
    """The serving form of :func:`mhc_qk_rope`: the normed and rotated keys, and
    the values as they are, go to place slots[t] (int64, page·page_size + offset)
    of the caches [pages, page_size, Hk, Dh]; a slot outside them (-1 for a
    padded token) writes nothing.  Slots of one call must differ.  Returns
    q_out[T,Hq,Dh]."""
    if stream is not None:
        return _within(stream, mhc_qk_rope_cache, locals())
    lib = load()
    d, ks, at, dtype, dev = _rope(q, k, positions, freqs, q_weight, k_weight, eps, interleaved)
    d.ldv = _heads("v", v, ks, dtype, dev)
    pages, size, kc, vc = _cache(k_cache, v_cache, ks[1], ks[2], dtype, dev)
    to = _vec("slots", _need("slots", slots), (ks[0],), torch.int64, dev)
    if out is None:
        out = _like(q)
    else:
        d.ldq_out = _heads("q_out", out, q.shape, dtype, dev)
    _check(lib.mhc_qk_rope_cache(_ref(d), at[0], at[1], v.data_ptr(), *at[2:], out.data_ptr(), kc, vc, to, pages * size,
                                 torch._C._cuda_getCurrentRawStream(dev)), "mhc_qk_rope_cache")
    return out


def _slopes(slopes, Hq, dev):
    if slopes is not None and isinstance(slopes, torch.Tensor) and slopes.requires_grad:
        raise ValueError("slopes takes no gradient: detach it")
    return _vec("slopes", slopes, (Hq,), torch.float32, dev)


def _attn(q, k, v, docs, causal, prefix, window, softcap, slopes, scale):
    """(descriptor, key shape, addresses of q, k, v, dtype, device) of a dense attention call."""
    shape, dtype, io, dev = _queries(q)
    T, Hq, Dh = shape
    ks = _key_shape(k, shape)
    Hk = ks[1]
    n = 1
    if docs is not None:
        if not isinstance(docs, torch.Tensor) or docs.dim() != 1 or docs.shape[0] < 2:
            raise ValueError("docs must be a [n_docs + 1] tensor of row offsets")
        n = docs.shape[0] - 1
    nq, nk = Hq * Dh, Hk * Dh
    d = MhcAttnDesc(T, Hq, Hk, Dh, io, n, 1 if causal else 0, window, 0, Dh ** -0.5 if scale is None else scale, softcap,
                    _vec("docs", docs, (n + 1,), torch.int32, dev), _vec("prefix", prefix, (n,), torch.int32, dev),
                    _slopes(slopes, Hq, dev), _heads("q", q, shape, dtype, dev), _heads("k", k, ks, dtype, dev),
                    _heads("v", v, ks, dtype, dev), nq, nq, nq, nk, nk)
    return d, ks, (q.data_ptr(), k.data_ptr(), v.data_ptr()), dtype, dev


def saved_floats(T: int, Hq: int, Dh: int, io: int) -> int:
    """Length of the fp32 tensor in which :func:`mhc_attn` keeps what its backward
    needs: the log-sum-exps [Hq, T] and, for bf16, the next eight bits of every
    element of o (one byte each, from the next multiple of four floats on)."""
    lse = -(-Hq * T // 4) * 4
    return lse + (T * Hq * Dh // 4 if io == mhc.MHC_BF16 else 0)


def _saved(saved, d, dev):
    """Addresses of the log-sum-exps and of o's further bits within the saved tensor."""
    lse = _vec("saved", _need("saved", saved), (saved_floats(d.T, d.Hq, d.Dh, d.io),), torch.float32, dev)
    return lse, (lse + (-(-d.Hq * d.T // 4) * 16) if d.io == mhc.MHC_BF16 else None)


def mhc_attn(q, k, v, *, docs=None, causal=True, prefix=None, window=0, softcap=0.0, slopes=None, scale=None, out=None,
             fill_outside=None, stream=None):
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
    tensors passed as ``out=(o, saved or None)`` they are left as they were,
    unless fill_outside is true."""
    if stream is not None:
        return _within(stream, mhc_attn, locals())
    lib = load()
    d, _ks, at, dtype, dev = _attn(q, k, v, docs, causal, prefix, window, softcap, slopes, scale)
    d.fill_outside = 1 if (out is None if fill_outside is None else fill_outside) else 0
    if out is None:
        out = (_like(q), q.new_empty(saved_floats(d.T, d.Hq, d.Dh, d.io), dtype=torch.float32))
        o, saved = out
    else:
        o, saved = out
        d.ldo = _heads("o", o, q.shape, dtype, dev)
    lse, rest = (None, None) if saved is None else _saved(saved, d, dev)
    _check(lib.mhc_attn(_ref(d), *at, o.data_ptr(), lse, rest, torch._C._cuda_getCurrentRawStream(dev)), "mhc_attn")
    return out


def mhc_attn_bwd(do, q, k, v, o, saved, *, docs=None, causal=True, prefix=None, window=0, softcap=0.0, slopes=None,
                 scale=None, out=None, fill_outside=None, workspace=None, stream=None):
    """Backward of :func:`mhc_attn` from its inputs and results: returns (dq, dk,
    dv), dk and dv summed over the query heads that share a key head.  Rows of
    no document get zeros; in tensors passed as ``out`` they are left as they
    were, unless fill_outside is true."""
    if stream is not None:
        return _within(stream, mhc_attn_bwd, locals())
    lib = load()
    d, ks, at, dtype, dev = _attn(q, k, v, docs, causal, prefix, window, softcap, slopes, scale)
    d.ld_do = _heads("do", do, q.shape, dtype, dev)
    d.ldo = _heads("o", o, q.shape, dtype, dev)
    lse, rest = _saved(saved, d, dev)
    d.fill_outside = 1 if (out is None if fill_outside is None else fill_outside) else 0
    if out is None:
        out = (_like(q), _like(k), _like(v))
        dq, dk, dv = out
    else:
        dq, dk, dv = out
        d.ld_dq = _heads("dq", dq, q.shape, dtype, dev)
        d.ld_dk = _heads("dk", dk, ks, dtype, dev)
        d.ld_dv = _heads("dv", dv, ks, dtype, dev)
    ws, nbytes, _keep = _scratch(lib.mhc_attn_bwd_workspace_bytes(_ref(d)), workspace, q.device)
    _check(lib.mhc_attn_bwd(_ref(d), do.data_ptr(), *at, o.data_ptr(), lse, rest, dq.data_ptr(), dk.data_ptr(),
                            dv.data_ptr(), ws, nbytes, torch._C._cuda_getCurrentRawStream(dev)), "mhc_attn_bwd")
    return out


def mhc_attn_paged(q, k_cache, v_cache, pages, kv_lens, *, cu_q=None, max_q=None, prefix=None, window=0, softcap=0.0,
                   slopes=None, scale=None, out=None, workspace=None, stream=None):
    """Attention of new tokens over a paged cache [num_pages, page_size, Hk, Dh]
    that already holds their own keys and values (:func:`mhc_qk_rope_cache`).

    pages[n, max_pages] (int32) is each sequence's page table, kv_lens[n]
    (int32) its keys with the new ones.  Without cu_q, row s of q[T,Hq,Dh] is
    sequence s's next token; with cu_q (int32 [n+1], sorted) rows cu_q[s] ..
    cu_q[s+1]-1 are its last tokens, at most max_q of them (a host number; T if
    None: give the longest chunk, the grid is sized by it; a sequence's rows past
    max_q count as rows of no sequence).  Masks and scores as :func:`mhc_attn`,
    positions counted within each sequence.

    Returns o[T,Hq,Dh]; a row without a key gets zeros, a row whose keys lie in
    a page outside the cache NaN; rows of no sequence get zeros, or are left as
    they were in a tensor passed as ``out``."""
    if stream is not None:
        return _within(stream, mhc_attn_paged, locals())
    lib = load()
    shape, dtype, io, dev = _queries(q)
    T, Hq, Dh = shape
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a [pages, page_size, Hk, Dh] tensor")
    Hk = k_cache.shape[2]
    if Hk < 1 or Hq % Hk:
        raise ValueError(f"{Hq} query heads cannot share {Hk} key heads evenly")
    num, size, kc, vc = _cache(k_cache, v_cache, Hk, Dh, dtype, dev)
    if not isinstance(pages, torch.Tensor) or pages.dim() != 2:
        raise ValueError("pages must be a [n, max_pages] tensor")
    n, width = pages.shape
    if cu_q is None:
        if n > T:
            raise ValueError(f"{n} sequences but {T} rows (pass cu_q for chunks)")
        if max_q not in (None, 1):
            raise ValueError("max_q above 1 needs cu_q")
        max_q = 1
    elif max_q is None:
        max_q = max(T, 1)
    d = MhcPagedDesc(T, n, max_q, Hq, Hk, Dh, io, window, size, width, 1 if out is None else 0, num,
                     Dh ** -0.5 if scale is None else scale, softcap, _vec("cu_q", cu_q, (n + 1,), torch.int32, dev),
                     _vec("kv_lens", _need("kv_lens", kv_lens), (n,), torch.int32, dev),
                     _vec("pages", pages, (n, width), torch.int32, dev), _vec("prefix", prefix, (n,), torch.int32, dev),
                     _slopes(slopes, Hq, dev), _heads("q", q, shape, dtype, dev), Hq * Dh)
    if out is None:
        out = _like(q) if n else torch.zeros_like(q, memory_format=torch.contiguous_format)
    else:
        d.ldo = _heads("o", out, shape, dtype, dev)
    ws, nbytes, _keep = _scratch(lib.mhc_attn_paged_workspace_bytes(_ref(d)), workspace, q.device)
    _check(lib.mhc_attn_paged(_ref(d), q.data_ptr(), kc, vc, out.data_ptr(), ws, nbytes, torch._C._cuda_getCurrentRawStream(dev)),
           "mhc_attn_paged")
    return out
