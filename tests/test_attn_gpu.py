"""Masked attention over packed documents, forward and backward, against the
fp64 oracle with elementwise bounds (oracle/attn_oracle.py), over types, head
layouts, lengths and masks."""

from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from oracle import attn_oracle as O
from residual_stream_amd import attn, mhc

from attn_testlib import bits, close, host, ints, rand, same

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)


def _case(io, T, Hq, Hk, Dh, seed, **masks):
    rng = np.random.default_rng(seed)
    q, k, v, do = (rand(rng, (T, h, Dh), io, f) for h, f in ((Hq, 1.5), (Hk, 1.0), (Hk, 1.0), (Hq, 1.0)))
    kw = dict(masks)
    if kw.pop("alibi", False):
        kw["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda")
    ok = O.visible(T, kw.get("docs"), kw.get("causal", True), kw.get("prefix"), kw.get("window", 0))
    i = np.arange(T)
    ref = dict(io=io, scale=Dh ** -0.5, softcap=kw.get("softcap", 0.0),
               slopes=None if "slopes" not in kw else host(kw["slopes"]))
    for n in ("docs", "prefix"):
        if kw.get(n) is not None:
            kw[n] = ints(kw[n])
    return (q, k, v, do), kw, ok, np.abs(i[:, None] - i[None]).astype(np.float64), ref


def _lse(saved, Hq, T):
    return saved[:Hq * T].view(Hq, T)


def _new_saved(T, Hq, Dh, io, value=0.0):
    return torch.full((attn.saved_floats(T, Hq, Dh, mhc.MHC_BF16 if io == "bf16" else mhc.MHC_F32),), value, device="cuda")


# lengths around the tiles of 32, 64 and 128 rows and keys, and one key
LENGTHS = [(1, 4, 2, 64), (2, 1, 1, 128), (31, 4, 4, 64), (33, 5, 1, 128), (64, 2, 2, 128), (65, 6, 2, 64),
           (127, 3, 3, 128), (129, 8, 2, 64), (257, 5, 5, 64), (400, 10, 2, 128),
          # grids that fill the chip with 128 rows a workgroup
          (1, 256, 64, 64), (130, 256, 32, 64), (257, 96, 24, 128), (300, 96, 96, 64), (1100, 40, 8, 64)]
MASKS = {
    "causal": {},
    "full": dict(causal=False),
    "capped": dict(softcap=5.0),
    "distance": dict(alibi=True),
    "capped_distance_full": dict(softcap=20.0, alibi=True, causal=False),
    "window1": dict(window=1),
    "window40": dict(window=40),
    "prefix": dict(prefix=[50]),
}


def _run(io, T, Hq, Hk, Dh, seed, **masks):
    (q, k, v, do), kw, ok, dist, ref = _case(io, T, Hq, Hk, Dh, seed, **masks)
    o, saved = attn.mhc_attn(q, k, v, **kw)
    grads = attn.mhc_attn_bwd(do, q, k, v, o, saved, **kw)
    lse = _lse(saved, Hq, T)
    torch.cuda.synchronize()
    if Hk > 6:  # many heads: the oracle looks at the first and the last key head's
        G = Hq // Hk
        some = [h for n in (0, Hk - 1) for h in range(n * G, n * G + G)]
        q, do, o, lse = q[:, some], do[:, some], o[:, some], lse[some]
        grads = [g[:, some] if i == 0 else g[:, [0, Hk - 1]] for i, g in enumerate(grads)]
        k, v = k[:, [0, Hk - 1]], v[:, [0, Hk - 1]]
        if ref["slopes"] is not None:
            ref["slopes"] = ref["slopes"][some]
    ro, rl, eo = O.attention(host(q), host(k), host(v), ok, dist, **ref)
    close("o", o, ro, eo)
    seen = ok.any(-1)
    assert np.isneginf(host(lse)[:, ~seen]).all()
    el = O._scores(host(q)[:, 0], host(k)[:, 0], ok, dist, ref["scale"], ref["softcap"], None)[3].max() + 2.0 ** -20
    assert np.abs(host(lse)[:, seen] - rl[:, seen]).max(initial=0.0) <= 4 * el + 2.0 ** -20 * np.abs(rl[:, seen]).max(initial=0.0)
    rg, eg = O.attention_bwd(host(do), host(q), host(k), host(v), ok, dist, **ref)
    for n, a, b, e in zip(("dq", "dk", "dv"), grads, rg, eg):
        close(n, a, b, e)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hk,Dh", LENGTHS)
def test_lengths(io, T, Hq, Hk, Dh):
    print(f"[attn] {io} T={T} {Hq}/{Hk}x{Dh}", file=sys.stderr, flush=True)
    _run(io, T, Hq, Hk, Dh, seed=T)


@pytest.mark.parametrize("io,Dh", [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (128, 32)])
def test_masks(io, Dh, mask, Hq, Hk):
    print(f"[attn] {io} {Hq}/{Hk}x{Dh} {mask}", file=sys.stderr, flush=True)
    _run(io, 203, Hq, Hk, Dh, seed=7, **MASKS[mask])


DOCS = {
    "ragged": [0, 3, 3, 70, 71, 200, 330],
    "rows_outside": [5, 40, 140, 300],
    "all_empty": [0, 0, 0],
    "single_tokens": list(range(0, 331)),
    "empty_ends": [0, 0, 0, 330, 330, 330],
}


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("docs", list(DOCS))
@pytest.mark.parametrize("kind", ["causal", "full", "prefix", "window"])
@pytest.mark.parametrize("Hq,Hk", [(2, 1), (96, 48)])
def test_documents(io, docs, kind, Hq, Hk):
    print(f"[attn] {io} {Hq}/{Hk} docs {docs} {kind}", file=sys.stderr, flush=True)
    bounds = DOCS[docs]
    n = len(bounds) - 1
    masks = dict(docs=bounds)
    if kind == "full":
        masks["causal"] = False
    elif kind == "prefix":  # none, negative, part, all, more than all
        masks["prefix"] = [(0, -3, 20, 1, 64, 10 ** 9)[d % 6] for d in range(n)]
    elif kind == "window":
        masks["window"] = 17
    _run(io, 330, Hq, Hk, 64, seed=11, **masks)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk", [(6, 2), (144, 16)])
def test_strided_views_equal_contiguous_tensors(io, Hq, Hk):
    T, Dh = 150, 64
    rng = np.random.default_rng(3)
    qkv, do = rand(rng, (T, (Hq + 2 * Hk) * Dh + 8), io), rand(rng, (T, Hq, Dh), io)
    cut = lambda t, a, h: t[:, a * Dh:(a + h) * Dh].unflatten(1, (h, Dh))  # noqa: E731
    q, k, v = cut(qkv, 0, Hq), cut(qkv, Hq, Hk), cut(qkv, Hq + Hk, Hk)
    c = [t.contiguous() for t in (q, k, v)]
    o, lse = attn.mhc_attn(q, k, v)
    o2, lse2 = attn.mhc_attn(*c)
    same("o", o, o2)
    same("saved", lse[:Hq * T], lse2[:Hq * T])
    d = torch.full_like(qkv, 7.0)
    out = (cut(d, 0, Hq), cut(d, Hq, Hk), cut(d, Hq + Hk, Hk))
    attn.mhc_attn_bwd(do, q, k, v, o, lse, out=out)
    for n, a, b in zip(("dq", "dk", "dv"), out, attn.mhc_attn_bwd(do, *c, o, lse)):
        same(n, a, b)
    assert bool((d[:, (Hq + 2 * Hk) * Dh:] == 7.0).all()), "wrote between the rows"


@pytest.mark.parametrize("Hq,Hk", [(2, 1), (128, 64)])
def test_rows_of_no_document_are_left_in_given_tensors(Hq, Hk):
    T, Dh = 140, 64
    rng = np.random.default_rng(5)
    q, k, v, do = (rand(rng, (T, h, Dh), "bf16") for h in (Hq, Hk, Hk, Hq))
    for t in (q, k, v, do):  # what they hold reaches nothing
        t[:4] = float("nan")
        t[100:] = float("nan")
    docs = ints([4, 30, 30, 100])
    full = lambda *s: torch.full(s, 3.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o, lse = full(T, Hq, Dh), _new_saved(T, Hq, Dh, "bf16", 3.0)
    attn.mhc_attn(q, k, v, docs=docs, out=(o, lse))
    g = (full(T, Hq, Dh), full(T, Hk, Dh), full(T, Hk, Dh))
    attn.mhc_attn_bwd(do, q, k, v, o, lse, docs=docs, out=g)
    for t in (o, *g):
        assert bool((t[:4] == 3.0).all()) and bool((t[100:] == 3.0).all())
        assert bool(torch.isfinite(t[4:100].float()).all())
    for rows in (slice(0, 4), slice(100, T)):
        assert bool((_lse(lse, Hq, T)[:, rows] == 3.0).all())
    o2, lse2 = attn.mhc_attn(q, k, v, docs=docs)
    g2 = attn.mhc_attn_bwd(do, q, k, v, o2, lse2, docs=docs)
    for t, u in zip((o2, *g2), (o, *g)):
        same("inside", t[4:100], u[4:100])
        assert int(torch.count_nonzero(t[:4])) == 0 and int(torch.count_nonzero(t[100:])) == 0


@pytest.mark.parametrize("docs", [[300, 200, 100], [-5, 10 ** 9], [10, 5, 400, -1, 60], [2 ** 31 - 1, -2 ** 31]])
@pytest.mark.parametrize("Hq,Hk", [(2, 1), (128, 64)])
def test_unsorted_documents_stay_within_the_tensors(docs, Hq, Hk):
    # meaningless results, but every access inside: the tensors next to them keep their values
    T, Dh = 150, 64
    rng = np.random.default_rng(6)
    q, k, v, do = (rand(rng, (T, h, Dh), "bf16") for h in (Hq, Hk, Hk, Hq))
    buf = torch.full((T + 256, Hq, Dh), 5.0, dtype=torch.bfloat16, device="cuda")
    o, lse = buf[128:128 + T], _new_saved(T, Hq, Dh, "bf16")
    attn.mhc_attn(q, k, v, docs=ints(docs), prefix=ints([10 ** 9] * (len(docs) - 1)), out=(o, lse))
    attn.mhc_attn_bwd(do, q, k, v, o.contiguous(), lse, docs=ints(docs))
    torch.cuda.synchronize()
    assert bool((buf[:128] == 5.0).all()) and bool((buf[128 + T:] == 5.0).all())


@pytest.mark.parametrize("Hq,Hk", [(4, 2), (90, 45)])
def test_large_scores_and_repeated_calls_give_the_same_bits(Hq, Hk):
    T, Dh = 300, 128
    rng = np.random.default_rng(8)
    q, k, v, do = (rand(rng, (T, h, Dh), "bf16", f) for h, f in ((Hq, 12.0), (Hk, 12.0), (Hk, 1.0), (Hq, 1.0)))
    first = None
    for _ in range(3):
        o, saved = attn.mhc_attn(q, k, v)
        r = (o, _lse(saved, Hq, T), *attn.mhc_attn_bwd(do, q, k, v, o, saved))
        assert all(bool(torch.isfinite(t.float()).all()) for t in r)
        first = first or r
        for a, b in zip(first, r):
            assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("softcap,alibi", [(0.0, False), (3.0, True)])
def test_gradients_against_differences(softcap, alibi):
    """Directional derivative of Σ do·o in fp32 inputs: central differences of the
    oracle's o (a step of 1e-5 is off by its square and 1e-11 / 1e-5) along the
    kernel's gradient."""
    (q, k, v, do), kw, ok, dist, ref = _case("f32", 70, 4, 2, 64, 21, softcap=softcap, alibi=alibi, docs=[0, 30, 70])
    o, lse = attn.mhc_attn(q, k, v, **kw)
    g = [host(t) for t in attn.mhc_attn_bwd(do, q, k, v, o, lse, **kw)]
    rng = np.random.default_rng(0)
    x = [host(t) for t in (q, k, v)]
    for n in range(3):
        u = rng.standard_normal(x[n].shape)
        f = []
        for s in (1e-5, -1e-5):
            y = [a + s * u if i == n else a for i, a in enumerate(x)]
            f.append((host(do) * O.attention(*y, ok, dist, **ref)[0]).sum())
        num, ana = (f[0] - f[1]) / 2e-5, (g[n] * u).sum()
        assert abs(num - ana) <= 1e-4 * np.sqrt((g[n] ** 2).sum()) + 1e-4 * abs(ana), ("qkv"[n], num, ana)


@pytest.mark.parametrize("Hq,Hk", [(4, 2), (128, 32)])
def test_graph_replays_match_eager(Hq, Hk):
    T, Dh = 200, 64
    rng = np.random.default_rng(9)
    sets = [[rand(rng, (T, h, Dh), "bf16") for h in (Hq, Hk, Hk, Hq)] for _ in range(3)]
    q, k, v, do = (t.clone() for t in sets[0])
    docs = ints([0, 60, 200])
    out = [torch.zeros_like(q), _new_saved(T, Hq, Dh, "bf16")]
    grads = [torch.empty_like(t) for t in (q, k, v)]

    def step():
        attn.mhc_attn(q, k, v, docs=docs, softcap=10.0, out=tuple(out))
        attn.mhc_attn_bwd(do, q, k, v, *out, docs=docs, softcap=10.0, out=tuple(grads))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        for t, s in zip((q, k, v, do), sets[rep % 3]):
            t.copy_(s)
        bound = [0, 20 * (rep + 1), 200]  # the masks are read at replay
        docs.copy_(ints(bound))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, *grads)]
        o, lse = attn.mhc_attn(q, k, v, docs=docs, softcap=10.0)
        ref = (o, lse, *attn.mhc_attn_bwd(do, q, k, v, o, lse, docs=docs, softcap=10.0))
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            same(f"replay {rep}", a, b)


@pytest.mark.parametrize("io,Dh", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (160, 40)])
@pytest.mark.parametrize("masks", [dict(docs=[0, 70, 75, 200]), dict(window=40), dict(prefix=[90])], ids=["docs", "window", "prefix"])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(io, Dh, Hq, Hk, masks):
    """In a column of v: that column of those rows; in k: those rows; elsewhere what finite inputs give."""
    (q, k, v, _), kw, ok, dist, ref = _case(io, 200, Hq, Hk, Dh, seed=11, **masks)
    clean_k, clean_v = host(k), host(v)
    inf, nan = float("inf"), float("nan")
    places = [(60, 3, inf), (72, Dh - 1, nan), (101, 0, -inf), (199, 31, nan)]
    for j, d, x in places:
        v[j, :, d] = x
    k[130, :, 5] = nan
    some = [0, Hq // Hk, Hq - 1]  # heads that the oracle looks at
    of = [h * Hk // Hq for h in some]
    o = host(attn.mhc_attn(q, k, v, **kw)[0])[:, some]
    ro, _, eo = O.attention(host(q)[:, some], clean_k[:, of], clean_v[:, of], ok, dist, **ref)
    hit = np.repeat(ok[:, 130][:, None], Dh, 1)
    for j, d, _ in places:
        hit[:, d] |= ok[:, j]
    hit = np.broadcast_to(hit[:, None], o.shape)
    assert not np.isfinite(o[hit]).any()
    close("o", np.where(hit, ro, o), ro, eo)
    only = ok[:, 60] & ~ok[:, 130]
    assert (o[only][:, :, 3] == inf).all()


def test_another_stream_than_the_current_one():
    """Outputs and workspaces of a call on `stream` are that stream's: memory the current one takes meanwhile is not theirs."""
    (q, k, v, do), kw, *_ = _case("bf16", 700, 8, 2, 128, seed=3, docs=[0, 300, 700])
    want = attn.mhc_attn(q, k, v, **kw)
    grads = attn.mhc_attn_bwd(do, q, k, v, *want, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for rep in range(5):
        got = attn.mhc_attn(q, k, v, stream=side, **kw)
        back = attn.mhc_attn_bwd(do, q, k, v, *got, stream=side, **kw)
        junk = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 18, 1 << 20, 1 << 22) for _ in range(4)]
        torch.cuda.synchronize()
        for n, a, b in zip(("o", "saved", "dq", "dk", "dv"), (*got, *back), (*want, *grads)):
            same(f"{n} {rep}", a, b)
        del junk


def test_workspaces_that_are_refused():
    (q, k, v, do), kw, *_ = _case("f32", 40, 2, 2, 64, seed=4)
    o, saved = attn.mhc_attn(q, k, v, **kw)
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            attn.mhc_attn_bwd(do, q, k, v, o, saved, workspace=ws, **kw)
    with pytest.raises(mhc.MhcError):
        attn.mhc_attn_bwd(do, q, k, v, o, saved, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **kw)
