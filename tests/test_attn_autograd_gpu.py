"""`MHCAttention` alone against plain torch in fp64, and as the sublayer of
`MHCBlock` and `MHCStack`: gradients, padded batches, and serving through the
cache against the training pass."""

from __future__ import annotations

import sys

import pytest
import torch

from residual_stream_amd.autograd import AttnBatch, CacheBatch, MHCAttention, MHCBlock, MHCStack

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)


def _layer(hidden=128, heads=4, key_heads=2, head_dim=64, seed=0, **kw):
    torch.manual_seed(seed)
    m = MHCAttention(hidden, heads, key_heads, head_dim, dtype=torch.float32, **kw)
    with torch.no_grad():
        m.q_weight += 0.3 * torch.randn_like(m.q_weight)
        m.k_weight += 0.3 * torch.randn_like(m.k_weight)
    return m


def _plain(m, h, w, lengths, softcap):
    """The layer in fp64 torch, document by document."""
    Hq, Hk, D = m.heads
    qkv = h @ w["qkv"].T
    R = 2 * m.freqs.shape[0]

    def rope(x, wt):
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + m.rope["eps"]) * wt
        pos = torch.cat([torch.arange(n) for n in lengths]).double()
        a = pos[:, None, None] * m.freqs.cpu()
        p, q = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat((p * a.cos() - q * a.sin(), p * a.sin() + q * a.cos(), x[..., R:]), -1)

    q = rope(qkv[:, :Hq * D].unflatten(1, (Hq, D)), w["q_weight"])
    k = rope(qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)), w["k_weight"])
    v = qkv[:, (Hq + Hk) * D:].unflatten(1, (Hk, D))
    out, at = [], 0
    for n in lengths:
        s = slice(at, at + n)
        at += n
        kk, vv = (t[s].repeat_interleave(Hq // Hk, 1) for t in (k, v))
        x = torch.einsum("ihd,jhd->hij", q[s], kk) * D ** -0.5
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        x = x.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), -torch.inf)
        out.append(torch.einsum("hij,jhd->ihd", torch.softmax(x, -1), vv).flatten(1))
    return torch.cat(out) @ w["out"].T


@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_layer_and_its_gradients(softcap):
    print(f"[attention layer] softcap={softcap}", file=sys.stderr, flush=True)
    lengths = [37, 1, 90]
    m = _layer(softcap=softcap, rotated=32)
    m.batch = AttnBatch.packed(lengths)
    h = torch.randn(sum(lengths), 128, device="cuda", requires_grad=True)
    dy = torch.randn(sum(lengths), 128, device="cuda")
    y = m(h)
    y.backward(dy)
    w = {n: p.detach().double().cpu().requires_grad_() for n, p in m.named_parameters()}
    h64 = h.detach().double().cpu().requires_grad_()
    y64 = _plain(m, h64, w, lengths, softcap)
    y64.backward(dy.double().cpu())
    got = {"y": (y, y64), "h": (h.grad, h64.grad), **{n: (p.grad, w[n].grad) for n, p in m.named_parameters()}}
    for n, (a, b) in got.items():
        # fp32 throughout: sums of some hundred terms and two softmaxes' worth of exponentials
        err = float((a.detach().double().cpu() - b.detach()).norm() / b.detach().norm())
        print(f"    {n}: {err:.1e}", flush=True)
        assert err <= 2e-5, (n, err)


def test_rows_behind_the_last_document_get_zero_gradients():
    m = _layer()
    m.batch = AttnBatch.packed([20, 30])
    h = torch.randn(64, 128, device="cuda")
    m.batch.positions = torch.cat((m.batch.positions, torch.zeros(14, dtype=torch.int32, device="cuda")))
    outs = []
    for pad in (0.0, 1e4):
        x = h.clone()
        x[50:] = pad
        x.requires_grad_()
        y = m(x)
        y.backward(torch.ones_like(y))
        assert int(torch.count_nonzero(y[50:])) == 0 and int(torch.count_nonzero(x.grad[50:])) == 0
        outs.append((y[:50], x.grad[:50]))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_as_the_sublayer_of_blocks_and_a_stack(dtype):
    torch.manual_seed(1)
    layers = [MHCAttention(256, 4, 1, 64, dtype=dtype) for _ in range(2)]
    blocks = [MHCBlock(m, 4, 256, alpha=(1.0, 1.0, 1.0)) for m in layers]
    stack = MHCStack(blocks)
    batch = AttnBatch.packed([40, 24])
    for m in layers:
        m.batch = batch
    x = torch.randn(2, 32, 4, 256, device="cuda").to(dtype)
    res = []
    for run in (lambda t: blocks[1](blocks[0](t)), stack, lambda t: stack(t)):
        stack.zero_grad()
        t = x.clone().requires_grad_()
        y = run(t)
        y.backward(torch.ones_like(y))
        assert bool(torch.isfinite(y.float()).all()) and bool(torch.isfinite(t.grad.float()).all())
        res.append([y.detach(), t.grad] + [p.grad.clone() for p in stack.parameters() if p.grad is not None])
    assert len(res[0]) == 2 + 2 * (4 + 2)
    for r in res[1:]:
        for a, b in zip(res[0], r):
            assert torch.equal(a, b)


def test_recompute_gives_the_same_gradients():
    m = _layer(hidden=256)
    m.batch = AttnBatch.packed([50, 14])
    x = torch.randn(64, 4, 256, device="cuda")
    grads = []
    for recompute in (False, True):
        torch.manual_seed(3)
        b = MHCBlock(m, 4, 256, recompute=recompute)
        m.zero_grad()
        t = x.clone().requires_grad_()
        y = b(t)
        y.backward(torch.ones_like(y))
        grads.append([t.grad] + [p.grad.clone() for p in b.parameters() if p.grad is not None])
    for a, b in zip(*grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("window,softcap", [(0, 0.0), (30, 10.0)])
def test_serving_through_the_cache_equals_the_training_pass(window, softcap):
    m = _layer(window=window, softcap=softcap)
    block = MHCBlock(m, 4, 128, alpha=(1.0, 1.0, 1.0))
    lens, page = [70, 45], 16
    x = [torch.randn(n, 4, 128, device="cuda") for n in lens]
    m.batch = AttnBatch.packed(lens)
    with torch.no_grad():
        want = block(torch.cat(x)).split(lens)
        m.new_cache(12, page)
        pages = torch.randperm(12, device="cuda").int().view(2, 6)
        done, got = [0, 0], [[], []]
        for new in ([33, 40], [1, 1], [1, 1], [30, 0], [5, 3]):
            m.batch = CacheBatch.step(pages, done, new, page)
            rows = torch.cat([t[a:a + n] for t, a, n in zip(x, done, new)])
            for s, r in enumerate(block(rows).split(new)):
                got[s].append(r)
            done = [a + n for a, n in zip(done, new)]
        assert done == lens
    for a, b in zip(got, want):
        off = (torch.cat(a) - b).norm() / b.norm()
        assert float(off) <= 1e-5, float(off)  # the same fp32 sums in another order


def test_refusals():
    m = _layer()
    h = torch.randn(4, 128, device="cuda")
    with pytest.raises(RuntimeError, match="set `batch`"):
        m(h)
    pages = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    m.batch = CacheBatch.step(pages, [0], [4], 16)
    with pytest.raises(RuntimeError, match="no_grad"):
        m(h)
    with torch.no_grad(), pytest.raises(RuntimeError, match="new_cache"):
        m(h)
    with pytest.raises(ValueError, match="page table"):
        CacheBatch.step(pages, [10], [7], 16)
    with pytest.raises(ValueError, match="evenly"):
        MHCAttention(64, 3, 2, 64)


def _captured(step):
    """`step` in a graph, after one eager pass on a stream of its own."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    return g, out


def test_a_captured_training_pass_replays_like_the_eager_one():
    m = _layer(hidden=256, softcap=20.0)
    m.batch = AttnBatch.packed([70, 1, 58])
    x, gy = (torch.randn(129, 256, device="cuda") for _ in range(2))
    x.requires_grad_()
    step = lambda: torch.autograd.grad(m(x), [x, *m.parameters()], gy)  # noqa: E731
    g, out = _captured(step)
    for rep in range(4):
        with torch.no_grad():
            x.copy_(torch.randn_like(x))
        m.batch.docs.copy_(torch.tensor([0, 70 - rep, 71, 129], dtype=torch.int32))
        g.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b), rep


@torch.no_grad()
def test_a_captured_decode_step_replays_like_the_eager_one():
    ms = [_layer(hidden=256) for _ in range(2)]
    pages = torch.tensor([[5, 0, 7], [2, 6, 1], [3, 8, 4]], dtype=torch.int32, device="cuda")
    text = torch.randn(40, 3, 256, device="cuda")
    for m in ms:
        m.new_cache(9, 16)
    batch = CacheBatch.step(pages, [0, 0, 0], [1, 1, 1], 16)
    h = text[0].clone()

    def eager(t):
        ms[1].batch = CacheBatch.step(pages, [t] * 3, [1] * 3, 16)
        return ms[1](text[t])

    ms[0].batch = batch
    g, out = _captured(lambda: ms[0](h))
    for t in range(40):
        new = CacheBatch.step(pages, [t] * 3, [1] * 3, 16)
        h.copy_(text[t])
        for n in ("positions", "slots", "kv_lens"):
            getattr(batch, n).copy_(getattr(new, n))
        g.replay()
        assert torch.equal(out, eager(t)), t
    assert torch.equal(ms[0].k_cache, ms[1].k_cache) and torch.equal(ms[0].v_cache, ms[1].v_cache)


def test_no_tokens():
    m = _layer()
    m.batch = AttnBatch(torch.zeros(0, dtype=torch.int32, device="cuda"))
    x = torch.zeros((0, 128), device="cuda", requires_grad=True)
    y = m(x)
    y.sum().backward()
    assert y.shape == x.grad.shape == (0, 128)
    assert all(int(torch.count_nonzero(p.grad)) == 0 for p in m.parameters())
    m.new_cache(4, 16)
    pages = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    with torch.no_grad():
        m.batch = CacheBatch.step(pages, [3, 0], [0, 0], 16)
        assert m(x.detach()).shape == (0, 128)
    assert int(torch.count_nonzero(m.k_cache)) == 0
