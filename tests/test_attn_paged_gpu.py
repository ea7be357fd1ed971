"""Attention of new tokens over a paged cache against the fp64 oracle: single
tokens and chunks, pages that end inside tiles, many splits, and what lies
outside the sequences."""

from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from oracle import attn_oracle as O
from residual_stream_amd import attn

from attn_testlib import close, host, ints, rand, same

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)


def _paged(io, kv, new, Hq, Hk, Dh, page, seed, spare_pages=3, spare_width=0, poison=True):
    """A cache whose unused places hold NaN, each sequence's pages scattered over it."""
    rng = np.random.default_rng(seed)
    per = [-(-n // page) for n in kv]
    total = sum(per) + spare_pages
    kc, vc = (rand(rng, (total, page, Hk, Dh), io) for _ in range(2))
    perm = rng.permutation(total)
    width = max(max(per), 1) + spare_width
    table = np.full((len(kv), width), -1, np.int32)
    used = np.zeros((total, page), bool)
    at = 0
    for s, (n, p) in enumerate(zip(kv, per)):
        table[s, :p] = perm[at:at + p]
        for j in range(n):
            used[table[s, j // page], j % page] = True
        at += p
    if poison:
        gone = torch.from_numpy(~used).cuda()
        kc[gone] = float("nan")
        vc[gone] = float("nan")
    q = rand(rng, (sum(new), Hq, Dh), io, 1.5)
    return q, kc, vc, torch.from_numpy(table).cuda()


def _check(io, kv, new, Hq, Hk, Dh, page, seed=0, window=0, prefix=None, softcap=0.0, alibi=False, max_q=None, **more):
    q, kc, vc, table = _paged(io, kv, new, Hq, Hk, Dh, page, seed, **more)
    cu = np.concatenate([[0], np.cumsum(new)])
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda") if alibi else None
    chunk = any(n != 1 for n in new)
    o = attn.mhc_attn_paged(q, kc, vc, table, ints(kv), cu_q=ints(cu) if chunk else None,
                            max_q=(max_q or max(new)) if chunk else None, window=window,
                            prefix=None if prefix is None else ints(prefix), softcap=softcap, slopes=slopes)
    torch.cuda.synchronize()
    ref, bound = np.zeros(q.shape), np.zeros(q.shape)
    t = host(table).astype(int)
    for s, (L, m) in enumerate(zip(kv, new)):
        if not m:
            continue
        k, v = (host(c)[t[s, :-(-L // page)]].reshape(-1, Hk, Dh)[:L] for c in (kc, vc))
        p = L - m + np.arange(m)
        j = np.arange(L)
        ok = j[None] <= p[:, None]
        if window:
            ok &= p[:, None] - j[None] < window
        if prefix is not None:
            ok |= j[None] < prefix[s]
        dist = np.abs(p[:, None] - j[None]).astype(float)
        a = slice(cu[s], cu[s + 1])
        ref[a], _, bound[a] = O.attention(host(q[a]), k, v, ok, dist, io=io, scale=Dh ** -0.5, softcap=softcap,
                                          slopes=None if slopes is None else host(slopes))
    # splits carry fp32 partial sums: a few more roundings than one pass
    close("o", o, ref, bound + 2.0 ** -20 * np.abs(ref).max(initial=0.0))
    return o


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk,Dh", [(40, 8, 128), (8, 2, 64), (3, 3, 128), (6, 1, 64), (64, 2, 64)])
@pytest.mark.parametrize("kv", [[1], [2, 1, 31], [32, 33, 127, 128, 129], [700, 5, 64]])
def test_single_tokens(io, Hq, Hk, Dh, kv):
    print(f"[paged] one token {io} {Hq}/{Hk}x{Dh} kv={kv}", file=sys.stderr, flush=True)
    _check(io, kv, [1] * len(kv), Hq, Hk, Dh, page=16)


@pytest.mark.parametrize("page", [1, 7, 16, 24, 100, 1024])
@pytest.mark.parametrize("new", [[1, 1, 1], [4, 1, 2], [90, 1, 33]], ids=["one", "draft", "chunk"])
def test_pages(page, new):
    print(f"[paged] page={page} new={new}", file=sys.stderr, flush=True)
    _check("bf16", [300, 77, 129], new, 10, 2, 64, page, spare_width=5)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk,Dh", [(20, 4, 128), (4, 4, 64), (6, 1, 128)])
@pytest.mark.parametrize("kv,new", [([200], [200]), ([65, 130, 3], [64, 2, 3]), ([1000, 40], [129, 40]), ([90, 300, 20], [0, 37, 0])])
def test_chunks(io, Hq, Hk, Dh, kv, new):
    print(f"[paged] chunk {io} {Hq}/{Hk}x{Dh} kv={kv} new={new}", file=sys.stderr, flush=True)
    _check(io, kv, new, Hq, Hk, Dh, page=24)


@pytest.mark.parametrize("new", [[1, 1], [3, 2], [60, 20]], ids=["one", "draft", "chunk"])
@pytest.mark.parametrize("masks", [dict(window=1), dict(window=50), dict(prefix=[0, 250]), dict(prefix=[10 ** 9, -4]),
                                   dict(softcap=4.0), dict(alibi=True), dict(softcap=30.0, alibi=True, window=128)],
                         ids=str)
def test_masks(new, masks):
    print(f"[paged] {masks} new={new}", file=sys.stderr, flush=True)
    for io in ("bf16", "f32"):
        _check(io, [260, 300], new, 10, 2, 64, page=16, **masks)


def test_long_cache_in_many_splits():
    print("[paged] 20001 keys", file=sys.stderr, flush=True)
    _check("bf16", [20001], [1], 5, 1, 128, page=64)
    _check("bf16", [20001, 9], [130, 9], 5, 1, 128, page=64)


def test_rows_without_keys_and_rows_of_no_sequence():
    Hq, Hk, Dh = 4, 2, 64
    for new in ([1, 1, 1], [5, 2, 70]):
        q, kc, vc, table = _paged("bf16", [0, 40, 60], new, Hq, Hk, Dh, 16, seed=3)
        T = sum(new)
        pad = torch.full((T + 6, Hq, Dh), float("nan"), dtype=q.dtype, device="cuda")
        pad[:T] = q
        cu = ints(np.concatenate([[0], np.cumsum(new)]))
        kw = dict(cu_q=cu, max_q=max(new))
        o = attn.mhc_attn_paged(pad, kc, vc, table, ints([0, 40, 60]), **kw)
        given = torch.full_like(pad, 2.0)
        attn.mhc_attn_paged(pad, kc, vc, table, ints([0, 40, 60]), out=given, **kw)
        torch.cuda.synchronize()
        same("rows", o[:T], given[:T])
        assert bool(torch.isfinite(o[:T].float()).all())
        assert int(torch.count_nonzero(o[:new[0]])) == 0, "a row without keys"
        # the third sequence has 60 keys for 70 new rows: its first ten see none
        if new[2] > 60:
            assert int(torch.count_nonzero(o[7:17])) == 0
        assert int(torch.count_nonzero(o[T:])) == 0 and bool((given[T:] == 2.0).all())


@pytest.mark.parametrize("new", [1, 50], ids=["one", "chunk"])
def test_pages_outside_the_cache_give_nan_to_their_rows_only(new):
    Hq, Hk, Dh = 4, 2, 64
    kv = [100, 90]
    q, kc, vc, table = _paged("bf16", kv, [new, new], Hq, Hk, Dh, 16, seed=4)
    cu = ints([0, new, 2 * new])
    ref = attn.mhc_attn_paged(q, kc, vc, table, ints(kv), cu_q=cu, max_q=new)
    for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 2] = bad
        o = attn.mhc_attn_paged(q, kc, vc, t, ints(kv), cu_q=cu, max_q=new)
        torch.cuda.synchronize()
        assert bool(torch.isnan(o[new - 1].float()).all())
        same("the other sequence", o[new:], ref[new:])


def test_meaningless_lengths_stay_within_the_tensors():
    Hq, Hk, Dh = 4, 2, 64
    q, kc, vc, table = _paged("bf16", [100, 90, 33], [2, 3, 1], Hq, Hk, Dh, 16, seed=5, poison=False)
    buf = torch.full((q.shape[0] + 64, Hq, Dh), 5.0, dtype=q.dtype, device="cuda")
    o = buf[32:32 + q.shape[0]]
    for cu, kv in (([0, 9, 4, 2], [2 ** 31 - 1, -7, 33]), ([-5, 2, 10 ** 9, 6], [100, 90, 33]), ([6, 5, 4, 3], [5, 5, 5])):
        attn.mhc_attn_paged(q, kc, vc, table, ints(kv), cu_q=ints(cu), max_q=3, out=o)
        torch.cuda.synchronize()
        assert bool((buf[:32] == 5.0).all()) and bool((buf[32 + q.shape[0]:] == 5.0).all())


def test_a_run_of_them_together_equals_attention_over_the_whole_text():
    """Prefill in chunks and then single tokens through the cache (norm, rotation
    and cache write, then attention over the pages) against one pass of the
    training calls over each whole sequence."""
    Hq, Hk, Dh, page = 8, 2, 64, 16
    rng = np.random.default_rng(12)
    lens, chunks = [150, 83], [[100, 40, 1, 1, 1, 7], [64, 1, 1, 1, 16]]
    w = [rand(rng, (Dh,), "f32") for _ in range(2)]
    freqs = attn.rope_freqs(Dh)
    qkv = [rand(rng, (L, (Hq + 2 * Hk) * Dh), "f32") for L in lens]
    cut = lambda t: (t[:, :Hq * Dh].unflatten(1, (Hq, Dh)), t[:, Hq * Dh:(Hq + Hk) * Dh].unflatten(1, (Hk, Dh)),  # noqa: E731
                     t[:, (Hq + Hk) * Dh:].unflatten(1, (Hk, Dh)))
    kw = dict(q_weight=w[0], k_weight=w[1])
    want = []
    for x, L in zip(qkv, lens):
        q, k, v = cut(x)
        q, k = attn.mhc_qk_rope(q, k, ints(range(L)), freqs, **kw)
        want.append(attn.mhc_attn(q, k, v, softcap=20.0)[0])
    table = torch.from_numpy(rng.permutation(24).reshape(2, 12).astype(np.int32)).cuda()
    kc, vc = (torch.full((24, page, Hk, Dh), float("nan"), device="cuda") for _ in range(2))
    got, done = [[], []], [0, 0]
    for step in range(6):
        new = [c[step] if step < len(c) else 0 for c in chunks]
        rows = [x[a:a + n] for x, a, n in zip(qkv, done, new)]
        pos = torch.cat([torch.arange(a, a + n) for a, n in zip(done, new)]).int().cuda()
        seq = torch.cat([torch.full((n,), s) for s, n in enumerate(new)]).cuda()
        slots = table[seq, (pos // page).long()].long() * page + pos % page
        q, k, v = cut(torch.cat(rows))
        q = attn.mhc_qk_rope_cache(q, k, v, pos, freqs, kc, vc, slots, **kw)
        done = [a + n for a, n in zip(done, new)]
        o = attn.mhc_attn_paged(q, kc, vc, table, ints(done), cu_q=ints([0, new[0], sum(new)]), max_q=max(new), softcap=20.0)
        got[0].append(o[:new[0]])
        got[1].append(o[new[0]:])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        # the same fp32 products in another order of keys
        off = (torch.cat(a) - b).abs().max()
        assert float(off) <= 2.0 ** -17 * float(b.abs().max()), float(off)


@pytest.mark.parametrize("new", [1, 40], ids=["one", "chunk"])
def test_graph_replays_match_eager(new):
    Hq, Hk, Dh, page = 8, 2, 64, 16
    q, kc, vc, table = _paged("bf16", [500, 300], [new, new], Hq, Hk, Dh, page, seed=6, poison=False)
    kv, cu = ints([500, 300]), ints([0, new, 2 * new])
    out = torch.empty_like(q)
    call = lambda o=None: attn.mhc_attn_paged(q, kc, vc, table, kv, cu_q=cu, max_q=new, out=o)  # noqa: E731
    call(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for rep in range(4):
        q.copy_(rand(np.random.default_rng(rep), q.shape, "bf16"))
        kv.copy_(ints([500 - 100 * rep, 300 - rep]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        same(f"replay {rep}", got, call())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("new,Hq,Hk,Dh", [(9, 4, 2, 128), (70, 8, 2, 64), (90, 4, 2, 128)])
@pytest.mark.parametrize("kv", [97, 1500])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(io, new, Hq, Hk, Dh, kv):
    page = 16
    q, kc, vc, table = _paged(io, [kv], [new], Hq, Hk, Dh, page, seed=5)
    t = host(table).astype(int)[0]
    rows = lambda c: host(c)[t].reshape(-1, Hk, Dh)[:kv]  # noqa: E731
    clean = rows(kc), rows(vc)
    first, last = kv - new, kv - 1
    places = [(first + 2, 1, float("inf")), (first + 5, Dh - 2, float("nan")), (last, 40, float("-inf"))]
    for j, d, x in places:
        vc[t[j // page], j % page, :, d] = x
    kc[t[(last - 1) // page], (last - 1) % page, :, 0] = float("nan")
    o = host(attn.mhc_attn_paged(q, kc, vc, table, ints([kv]), cu_q=ints([0, new]), max_q=new))
    p = kv - new + np.arange(new)
    ok = np.arange(kv)[None] <= p[:, None]
    ref, _, bound = O.attention(host(q), *clean, ok, np.abs(p[:, None] - np.arange(kv)[None]).astype(float), io=io,
                                scale=Dh ** -0.5, softcap=0.0, slopes=None)
    hit = np.repeat(ok[:, last - 1][:, None], Dh, 1)
    for j, d, _ in places:
        hit[:, d] |= ok[:, j]
    hit = np.broadcast_to(hit[:, None], o.shape)
    assert not np.isfinite(o[hit]).any()
    close("o", np.where(hit, ref, o), ref, bound + 2.0 ** -20 * np.abs(ref).max())


@pytest.mark.parametrize("new,max_q", [(9, 4), (100, 70)])
def test_rows_past_the_given_longest_chunk(new, max_q):
    Hq, Hk, Dh, page = 8, 2, 64, 16
    kv = [300, 170, 40]
    lens = [new, 3, new]
    q, kc, vc, table = _paged("f32", kv, lens, Hq, Hk, Dh, page, seed=8, poison=False)
    cu = np.concatenate([[0], np.cumsum(lens)])
    call = lambda **k: attn.mhc_attn_paged(q, kc, vc, table, ints(kv), cu_q=ints(cu), **k)  # noqa: E731
    whole = call(max_q=new)
    past = np.concatenate([np.arange(a + max_q, b) for a, b in zip(cu, cu[1:])])
    rest = np.setdiff1d(np.arange(len(q)), past)
    got = call(max_q=max_q)
    assert int(torch.count_nonzero(got[past])) == 0
    close("o", host(got)[rest], host(whole)[rest], 2.0 ** -18 * np.abs(host(whole)).max() * np.ones(1))
    given = torch.full_like(q, 7.0)
    call(max_q=max_q, out=given)
    assert bool((given[past] == 7.0).all())
    same("given", given[rest], got[rest])
