"""Per-head norm of queries and keys with the rotation: forward, backward and
the cache-writing form against the fp64 oracle."""

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

# One rounding of the output, and about 40 fp32 operations on the way (the sum
# of Dh squares among them, whose relative error stays below Dh/16 steps of
# the lanes' partial sums).
STEPS = 64 * O.U


def _bound(y, big, io):
    return 1.01 * O.R[io] * np.abs(y) + STEPS * big + 1e-30


# (T, Hq, Hk, Dh, R): every head width's lane count, partial rotation, one row
SHAPES = [(1, 1, 1, 16, 16), (3, 5, 1, 32, 16), (70, 8, 2, 64, 64), (33, 6, 3, 96, 48), (129, 40, 8, 128, 128),
          (5, 3, 3, 128, 112), (9, 4, 2, 256, 64), (2, 2, 1, 512, 512), (17, 3, 1, 208, 160),
          # two tokens a workgroup at a time (the weights' sums are chains of 61 additions at most)
          (4096, 3, 1, 128, 128), (4097, 6, 2, 128, 64)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("T,Hq,Hk,Dh,R", SHAPES)
def test_forward_and_backward(io, inter, T, Hq, Hk, Dh, R):
    print(f"[rope] {io} T={T} {Hq}/{Hk}x{Dh} R={R} inter={inter}", file=sys.stderr, flush=True)
    rng = np.random.default_rng(T + Dh)
    q, k, dq, dk = (rand(rng, (T, h, Dh), io, 2.0) for h in (Hq, Hk, Hq, Hk))
    qw, kw = (rand(rng, (Dh,), "f32") for _ in range(2))
    pos = ints(rng.integers(0, 1000000, T))
    freqs = attn.rope_freqs(R, 10000.0)
    args = dict(q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter)
    out = attn.mhc_qk_rope(q, k, pos, freqs, **args)
    grads = attn.mhc_qk_rope_bwd(dq, dk, q, k, pos, freqs, **args)
    torch.cuda.synchronize()
    f, p = host(freqs), host(pos)
    for n, x, w, y, dy, dx, dw in (("q", q, qw, out[0], dq, grads[0], grads[2]), ("k", k, kw, out[1], dk, grads[1], grads[3])):
        ref = O.rope(host(x), host(w), p, f, 1e-5, inter)
        big = np.abs(ref).max(-1, keepdims=True)
        close(n, y, ref, _bound(ref, big, io))
        rx, rw = O.rope_bwd(host(dy), host(x), host(w), p, f, 1e-5, inter)
        # (both parts of dx by the row's largest gradient term)
        r = 1.0 / np.sqrt((host(x) ** 2).mean(-1, keepdims=True) + 1e-5)
        big = r * np.abs(host(w)).max() * np.abs(host(dy)).max(-1, keepdims=True) * (1 + (r * np.abs(host(x))).max(-1, keepdims=True) ** 2)
        close("d" + n, dx, rx, _bound(rx, big, io))
        terms = (np.abs(host(dy)).max(-1, keepdims=True) * np.abs(host(x)) * r * 1.5).sum((0, 1))
        close(f"d{n}_weight", dw, rw, STEPS * terms + 1e-30)


def test_far_positions_keep_their_phase():
    # every pair's angle mod a turn at positions up to the largest int32, both signs
    pos = ints([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789])
    T, Dh = 7, 64
    x = rand(np.random.default_rng(1), (T, 1, Dh), "f32")
    freqs = attn.rope_freqs(Dh)
    y, _ = attn.mhc_qk_rope(x, x, pos, freqs)
    ref = O.rope(host(x), None, host(pos), host(freqs), 1e-6, False)
    # the product p·f is off by 2⁻⁵³ of up to 2³¹ radians: 2⁻²²
    close("y", y, ref, _bound(ref, np.abs(ref).max(-1, keepdims=True), "f32") + 2.0 ** -21 * np.abs(ref).max())


def test_without_weights_and_partial_outputs():
    T, Hq, Hk, Dh = 20, 4, 2, 64
    rng = np.random.default_rng(2)
    q, k, dq, dk = (rand(rng, (T, h, Dh), "bf16") for h in (Hq, Hk, Hq, Hk))
    pos, freqs = ints(range(T)), attn.rope_freqs(32)
    one = torch.ones(Dh, device="cuda")
    a, b = attn.mhc_qk_rope(q, k, pos, freqs), attn.mhc_qk_rope(q, k, pos, freqs, q_weight=one, k_weight=one)
    for x, y in zip(a, b):
        same("out", x, y)
    g = attn.mhc_qk_rope_bwd(dq, dk, q, k, pos, freqs)
    h = attn.mhc_qk_rope_bwd(dq, dk, q, k, pos, freqs, q_weight=one)
    assert g[2] is None and g[3] is None and h[2] is not None and h[3] is None
    for x, y in zip(g[:2], h[:2]):
        same("grad", x, y)


@pytest.mark.parametrize("T", [1, 5, 300, 4097])
def test_views_of_one_projection(T):
    Hq, Hk, Dh = 6, 2, 64
    rng = np.random.default_rng(T)
    qkv = rand(rng, (T, (Hq + 2 * Hk) * Dh), "bf16")
    q, k = qkv[:, :Hq * Dh].unflatten(1, (Hq, Dh)), qkv[:, Hq * Dh:(Hq + Hk) * Dh].unflatten(1, (Hk, Dh))
    dq, dk = rand(rng, (T, Hq, Dh), "bf16"), rand(rng, (T, Hk, Dh), "bf16")
    w = rand(rng, (Dh,), "f32")
    pos, freqs = ints(range(T)), attn.rope_freqs(Dh)
    for a, b in zip(attn.mhc_qk_rope(q, k, pos, freqs, q_weight=w),
                    attn.mhc_qk_rope(q.contiguous(), k.contiguous(), pos, freqs, q_weight=w)):
        same("out", a, b)
    d = torch.full_like(qkv, 9.0)
    out = (d[:, :Hq * Dh].unflatten(1, (Hq, Dh)), d[:, Hq * Dh:(Hq + Hk) * Dh].unflatten(1, (Hk, Dh)),
           torch.empty(Dh, device="cuda"), None)
    attn.mhc_qk_rope_bwd(dq, dk, q, k, pos, freqs, q_weight=w, out=out)
    for a, b in zip(out[:3], attn.mhc_qk_rope_bwd(dq, dk, q.contiguous(), k.contiguous(), pos, freqs, q_weight=w)):
        same("grad", a, b)
    assert bool((d[:, (Hq + Hk) * Dh:] == 9.0).all()), "wrote into v's place"


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,page", [(1, 16), (7, 1), (130, 24)])
def test_cache_form(io, T, page):
    Hq, Hk, Dh = 5, 1, 128
    rng = np.random.default_rng(T)
    q, k, v = (rand(rng, (T, h, Dh), io) for h in (Hq, Hk, Hk))
    qw, kw = rand(rng, (Dh,), "f32"), rand(rng, (Dh,), "f32")
    pos, freqs = ints(rng.integers(0, 5000, T)), attn.rope_freqs(64)
    pages = -(-T // page) + 3
    slots = torch.from_numpy(rng.permutation(pages * page)[:T].astype(np.int64))
    if T > 5:  # padding and places outside the cache write nothing
        slots[1], slots[3], slots[4] = -1, pages * page, 2 ** 40
    slots = slots.cuda()
    kc, vc = (torch.full((pages, page, Hk, Dh), f, dtype=q.dtype, device="cuda") for f in (4.0, 5.0))
    args = dict(q_weight=qw, k_weight=kw, interleaved=True)
    qo = attn.mhc_qk_rope_cache(q, k, v, pos, freqs, kc, vc, slots, **args)
    rq, rk = attn.mhc_qk_rope(q, k, pos, freqs, **args)
    same("q", qo, rq)
    ek, ev = torch.full_like(kc, 4.0), torch.full_like(vc, 5.0)
    good = (slots >= 0) & (slots < pages * page)
    ek.view(-1, Hk, Dh)[slots[good]] = rk[good]
    ev.view(-1, Hk, Dh)[slots[good]] = v[good]
    same("k_cache", kc, ek)
    same("v_cache", vc, ev)


def test_empty_batch_zeroes_the_weight_gradients():
    e = lambda h: torch.empty((0, h, 64), device="cuda")  # noqa: E731
    w, pos, freqs = torch.ones(64, device="cuda"), ints([]), attn.rope_freqs(64)
    assert attn.mhc_qk_rope(e(4), e(2), pos, freqs)[0].shape == (0, 4, 64)
    nan = lambda: torch.full((64,), float("nan"), device="cuda")  # noqa: E731
    g = attn.mhc_qk_rope_bwd(e(4), e(2), e(4), e(2), pos, freqs, q_weight=w, k_weight=w, out=(e(4), e(2), nan(), nan()))
    assert int(torch.count_nonzero(g[2])) == 0 and int(torch.count_nonzero(g[3])) == 0
    o, lse = attn.mhc_attn(e(4), e(2), e(2))
    assert o.shape == (0, 4, 64) and lse.shape == (0,)


def test_zero_rows_and_eps():
    # a row of zeros: r = eps^-1/2, the output zero, the gradient finite
    x = torch.zeros((2, 1, 64), device="cuda")
    pos, freqs = ints([0, 5]), attn.rope_freqs(64)
    y, _ = attn.mhc_qk_rope(x, x, pos, freqs)
    assert int(torch.count_nonzero(y)) == 0
    g = rand(np.random.default_rng(0), (2, 1, 64), "f32")
    d = attn.mhc_qk_rope_bwd(g, g, x, x, pos, freqs)[0]
    ref, _ = O.rope_bwd(host(g), host(x), None, host(pos), host(freqs), 1e-6, False)
    close("dq", d, ref, _bound(ref, 1000.0 * np.abs(host(g)).max(), "f32"))
