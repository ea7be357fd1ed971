"""Refusals of the attention sublayer's calls, on the host: the C ABI with
addresses that nothing follows (every call fails a check), the binding with
host tensors, and the oracle's backward against differences."""

from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import attn_oracle as O
from residual_stream_amd import attn, mhc


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mhc.LIB_PATH):
        pytest.skip("libmhc.so not built (run __graft_entry__.build())")
    return mhc.load()


# 16-byte aligned, far apart, never dereferenced
FAKE = [0x100000000 * (i + 1) for i in range(16)]


def _rope(**kw):
    d = dict(T=4, Hq=4, Hk=2, Dh=64, R=64, io=mhc.MHC_F32, interleaved=0, eps=1e-6, ldq=256, ldk=128, ldv=128, ldq_out=256,
             ldk_out=128, ld_dq=256, ld_dk=128)
    d.update(kw)
    return mhc.MhcRopeDesc(**d)


def _attn(**kw):
    d = dict(T=4, Hq=4, Hk=2, Dh=64, io=mhc.MHC_BF16, n_docs=1, causal=1, window=0, scale=0.125, softcap=0.0, ldq=256, ldk=128,
             ldv=128, ldo=256, ld_do=256, ld_dq=256, ld_dk=128, ld_dv=128)
    d.update(kw)
    return mhc.MhcAttnDesc(**d)


def _paged(**kw):
    d = dict(T=4, n_seqs=4, max_q=1, Hq=4, Hk=2, Dh=64, io=mhc.MHC_F32, window=0, page_size=16, max_pages=4, num_pages=32,
             scale=0.125, softcap=0.0, kv_lens=FAKE[10], pages=FAKE[11], ldq=256, ldo=256)
    d.update(kw)
    return mhc.MhcPagedDesc(**d)


def _calls(lib, name, d, ptrs, ws=(None, 0)):
    tail = [ctypes.c_void_p(ws[0]) if ws[0] else None, ws[1], None] if name in ("mhc_qk_rope_bwd", "mhc_attn_bwd", "mhc_attn_paged") else [None]
    if name == "mhc_qk_rope_cache":
        tail = [64, None]
    return getattr(lib, name)(ctypes.byref(d), *ptrs, *tail)


N_PTRS = {"mhc_qk_rope": (_rope, 8), "mhc_qk_rope_bwd": (_rope, 12), "mhc_qk_rope_cache": (_rope, 11), "mhc_attn": (_attn, 6),
          "mhc_attn_bwd": (_attn, 10), "mhc_attn_paged": (_paged, 4)}
NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses are only passed where no GPU exists")


@pytest.mark.parametrize("name", list(N_PTRS))
@pytest.mark.parametrize("field,value,expect", [
    ("T", -1, 1), ("T", 2 ** 31, 1), ("Hq", 0, 2), ("Hk", 0, 2), ("Hk", 3, 2), ("Hq", 8192, 2), ("Dh", 0, 2), ("Dh", 72, 2), ("io", 5, 1)])
def test_bad_shapes(lib, name, field, value, expect):
    make, n = N_PTRS[name]
    assert _calls(lib, name, make(**{field: value}), [None] * n) == expect


@pytest.mark.parametrize("make,name,field,value,expect", [
    (_rope, "mhc_qk_rope", "R", 0, 2), (_rope, "mhc_qk_rope", "R", 80, 2), (_rope, "mhc_qk_rope", "R", 24, 2),
    (_rope, "mhc_qk_rope", "eps", -1.0, 1), (_rope, "mhc_qk_rope", "eps", float("nan"), 1),
    (_rope, "mhc_qk_rope", "Dh", 528, 2),
    (_attn, "mhc_attn", "scale", 0.0, 1), (_attn, "mhc_attn", "scale", -1.0, 1), (_attn, "mhc_attn", "scale", float("inf"), 1),
    (_attn, "mhc_attn", "softcap", -1.0, 1), (_attn, "mhc_attn", "softcap", float("nan"), 1),
    (_attn, "mhc_attn", "window", -1, 1), (_attn, "mhc_attn", "Dh", 96, 2), (_attn, "mhc_attn", "docs", 6, 1),
    (_paged, "mhc_attn_paged", "page_size", 0, 1), (_paged, "mhc_attn_paged", "max_pages", 0, 1),
    (_paged, "mhc_attn_paged", "num_pages", 0, 1), (_paged, "mhc_attn_paged", "num_pages", 2 ** 31, 2),
    (_paged, "mhc_attn_paged", "max_pages", 2 ** 28, 2), (_paged, "mhc_attn_paged", "max_q", 0, 1),
    (_paged, "mhc_attn_paged", "max_q", 2, 1), (_paged, "mhc_attn_paged", "n_seqs", 5, 1), (_paged, "mhc_attn_paged", "n_seqs", -1, 1),
    (_paged, "mhc_attn_paged", "window", -1, 1)])
def test_bad_fields(lib, make, name, field, value, expect):
    assert _calls(lib, name, make(**{field: value}), [None] * N_PTRS[name][1]) == expect


def test_masks_that_exclude_each_other(lib):
    for d in (_attn(causal=0, window=3), _attn(causal=0, prefix=FAKE[0]), _attn(window=3, prefix=FAKE[0])):
        assert _calls(lib, "mhc_attn", d, [None] * 6) == mhc.MHC_ERR_UNSUPPORTED
    assert _calls(lib, "mhc_attn_paged", _paged(window=3, prefix=FAKE[0]), [None] * 4) == mhc.MHC_ERR_UNSUPPORTED
    assert _calls(lib, "mhc_attn", _attn(docs=FAKE[0], n_docs=0), [None] * 6) == mhc.MHC_ERR_INVALID_ARG


@NO_GPU
@pytest.mark.parametrize("name", list(N_PTRS))
def test_null_misaligned_and_overlapping_pointers(lib, name):
    make, n = N_PTRS[name]
    ws = (FAKE[15], 1 << 20)
    may_be_null = {"mhc_qk_rope": (4, 5), "mhc_qk_rope_bwd": (6, 7, 10, 11), "mhc_qk_rope_cache": (5, 6), "mhc_attn": (4, 5),
                   "mhc_attn_bwd": (6,), "mhc_attn_paged": ()}[name]
    for i in range(n):
        ptrs = [ctypes.c_void_p(p) for p in FAKE[:n]]
        if i not in may_be_null:
            ptrs[i] = None
            assert _calls(lib, name, make(), ptrs, ws) == mhc.MHC_ERR_INVALID_ARG, (name, i)
        ptrs[i] = ctypes.c_void_p(FAKE[i] + 2)
        assert _calls(lib, name, make(), ptrs, ws) == mhc.MHC_ERR_INVALID_ARG, (name, i)
    outs = {"mhc_qk_rope": (6, 7), "mhc_qk_rope_bwd": (8, 9), "mhc_qk_rope_cache": (7, 8, 9), "mhc_attn": (3,),
            "mhc_attn_bwd": (7, 8, 9), "mhc_attn_paged": (3,)}[name]
    for o in outs:
        for other in [0, 1] + [x for x in outs if x != o]:
            ptrs = [ctypes.c_void_p(p) for p in FAKE[:n]]
            ptrs[o] = ctypes.c_void_p(FAKE[other] + 16)
            assert _calls(lib, name, make(), ptrs, ws) == mhc.MHC_ERR_INVALID_ARG, (name, o, other)


@NO_GPU
def test_the_rest_of_o_is_for_bf16_only(lib):
    p = [ctypes.c_void_p(x) for x in FAKE]
    for name in ("mhc_attn", "mhc_attn_bwd"):
        assert _calls(lib, name, _attn(io=mhc.MHC_F32), p[:N_PTRS[name][1]], (FAKE[15], 1 << 20)) == mhc.MHC_ERR_INVALID_ARG


@NO_GPU
def test_workspaces_and_strides(lib):
    p = [ctypes.c_void_p(x) for x in FAKE]
    for name in ("mhc_qk_rope_bwd", "mhc_attn_bwd"):
        make, n = N_PTRS[name]
        for ws in ((None, 0), (FAKE[15], 8), (FAKE[15] + 16, 1 << 20)):
            assert _calls(lib, name, make(), p[:n], ws) == mhc.MHC_ERR_INVALID_ARG
    for field in ("ldq", "ldk", "ldv", "ldo"):
        for value in (64, 257, 1 << 23, -256):
            assert _calls(lib, "mhc_attn", _attn(**{field: value}), p[:6]) == mhc.MHC_ERR_INVALID_ARG


def test_workspace_queries(lib):
    assert lib.mhc_attn_bwd_workspace_bytes(ctypes.byref(_attn(T=1000))) >= 4 * 1000 * 4
    assert lib.mhc_attn_bwd_workspace_bytes(ctypes.byref(_attn(T=0))) == 0
    assert lib.mhc_attn_bwd_workspace_bytes(ctypes.byref(_attn(Dh=80))) == 0
    assert lib.mhc_qk_rope_bwd_workspace_bytes(ctypes.byref(_rope())) >= 2 * 64 * 4
    assert lib.mhc_qk_rope_bwd_workspace_bytes(None) == 0
    assert lib.mhc_attn_paged_workspace_bytes(ctypes.byref(_paged(T=0, n_seqs=0))) == 0
    many = _paged(T=1, n_seqs=1, max_pages=1000)
    assert lib.mhc_attn_paged_workspace_bytes(ctypes.byref(many)) > 0


def test_empty_calls_launch_nothing(lib):
    assert _calls(lib, "mhc_qk_rope", _rope(T=0), [None] * 8) == mhc.MHC_OK
    assert _calls(lib, "mhc_qk_rope_bwd", _rope(T=0), [None] * 12) == mhc.MHC_OK
    assert _calls(lib, "mhc_attn", _attn(T=0), [None] * 6) == mhc.MHC_OK
    assert _calls(lib, "mhc_attn_bwd", _attn(T=0), [None] * 10) == mhc.MHC_OK
    assert _calls(lib, "mhc_attn_paged", _paged(T=0, n_seqs=0), [None] * 4) == mhc.MHC_OK


def test_descriptor_sizes():
    assert ctypes.sizeof(mhc.MhcRopeDesc) == 96 and mhc.MhcRopeDesc.ldq.offset == 40
    assert ctypes.sizeof(mhc.MhcAttnDesc) == 136 and mhc.MhcAttnDesc.docs.offset == 48
    assert ctypes.sizeof(mhc.MhcPagedDesc) == 120 and mhc.MhcPagedDesc.cu_q.offset == 64


def test_host_tensors_are_refused(lib):
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    pos, f = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    cache, slots = torch.zeros(2, 4, 2, 64), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: attn.mhc_qk_rope(q, k, pos, f), lambda: attn.mhc_qk_rope_bwd(q, k, q, k, pos, f),
                 lambda: attn.mhc_qk_rope_cache(q, k, k, pos, f, cache, cache, slots), lambda: attn.mhc_attn(q, k, k),
                 lambda: attn.mhc_attn_bwd(q, q, k, k, q, torch.zeros(4, 3)),
                 lambda: attn.mhc_attn_paged(q, cache, cache, torch.zeros(3, 1, dtype=torch.int32), pos)):
        with pytest.raises(RuntimeError, match="GPU tensors"):
            call()


def test_oracle_backward_against_differences():
    rng = np.random.default_rng(0)
    T, Hq, Hk, D = 9, 4, 2, 5
    q, do = rng.standard_normal((2, T, Hq, D))
    k, v = rng.standard_normal((2, T, Hk, D))
    ok = O.visible(T, [0, 4, 9], True, [2, 0])
    i = np.arange(T)
    kw = dict(io="f32", scale=0.4, softcap=1.5, slopes=np.array([0.5, 0.2, 0.1, 0.0]))
    dist = np.abs(i[:, None] - i).astype(float)
    g, _ = O.attention_bwd(do, q, k, v, ok, dist, **kw)
    x = [q, k, v]
    for n in range(3):
        u = rng.standard_normal(x[n].shape)
        f = [(do * O.attention(*[a + s * u if m == n else a for m, a in enumerate(x)], ok, dist, **kw)[0]).sum() for s in (1e-5, -1e-5)]
        assert abs((f[0] - f[1]) / 2e-5 - (g[n] * u).sum()) < 1e-7
    w, pos, fr = rng.standard_normal(8), np.arange(3), np.array([1.0, 0.1, 0.01])
    a, dy = rng.standard_normal((2, 3, 2, 8))
    for inter in (False, True):
        dx, dw = O.rope_bwd(dy, a, w, pos, fr, 1e-3, inter)
        u, uw = rng.standard_normal(a.shape), rng.standard_normal(8)
        f = [(dy * O.rope(a + s * u, w + s * uw, pos, fr, 1e-3, inter)).sum() for s in (1e-6, -1e-6)]
        assert abs((f[0] - f[1]) / 2e-6 - (dx * u).sum() - (dw * uw).sum()) < 1e-6
