"""The operators of the attention sublayer that an mHC block wraps, as they are timed and compared.

`run` with `own` false computes each operator in plain torch in 32 bits (angles in 64) and rounds
once at the end; with `own` true it makes the calls a user makes (`residual_stream_amd.attn`).
`exact` computes the same results in 64 bits from the definitions, document by document and
sequence by sequence, with autograd for the gradients.

The head layouts 40/8x128 and 20/4x128 split the hidden sizes 5120 and 2560 of this repository's
workloads into heads of 128; the others are generic.
"""

import math
import random

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------
# cases

def listed():
    base = dict(shape_seed=1, softcap=0.0, window=0, alibi=False, prefix=False, causal=True)
    rope = dict(base, eps=1e-6, base_freq=10000.0)
    return [
        # one step of a small serving batch: norm, rotation and cache write of 8 single tokens
        dict(rope, name="rope_cache_t8", op="rope_cache", io="bf16", T=8, Hq=40, Hk=8, Dh=128, R=128, inter=False,
             far=120000, page=16, pages=64),
        # a prefill chunk written to the cache, half of each head rotated, odd length
        dict(rope, name="rope_cache_t2047", op="rope_cache", io="bf16", T=2047, Hq=20, Hk=4, Dh=128, R=64, inter=True,
             far=4096, page=64, pages=64),
        # the training step's norm and rotation at the headline's token count, both directions
        dict(rope, name="rope_train_t4096", op="rope_train", io="bf16", T=4096, Hq=40, Hk=8, Dh=128, R=128, inter=False,
             far=0),
        # fp32 training at the narrower width, interleaved pairs, three quarters of each head rotated
        dict(rope, name="rope_train_f32_t1023", op="rope_train", io="f32", T=1023, Hq=40, Hk=4, Dh=64, R=48, inter=True,
             far=500000),
        # a prompt of the headline's length, forward only
        dict(base, name="attn_fwd_t4096", op="attn", io="bf16", T=4096, Hq=40, Hk=8, Dh=128, docs=1, train=False),
        # packed training batch: 9 documents of ragged lengths, capped scores
        dict(base, name="attn_train_docs_t4096", op="attn", io="bf16", T=4096, Hq=40, Hk=8, Dh=128, docs=9, train=True,
             softcap=30.0),
        # prefix mask and distance bias, heads of 64 without sharing, odd length
        dict(base, name="attn_train_prefix_t2309", op="attn", io="bf16", T=2309, Hq=16, Hk=16, Dh=64, docs=3, train=True,
             alibi=True, prefix=True),
        # a short fp32 step, one shared key head for four
        dict(base, name="attn_train_f32_t777", op="attn", io="f32", T=777, Hq=8, Hk=2, Dh=64, docs=2, train=True),
        # the largest: one long document, training
        dict(base, name="attn_train_t8192", op="attn", io="bf16", T=8192, Hq=40, Hk=8, Dh=128, docs=1, train=True),
        # one user's next token over a cache of some thousand tokens: latency
        dict(base, name="paged_one_token", op="paged", io="bf16", n=1, longest=4099, chunk=1, Hq=40, Hk=8, Dh=128,
             page=16),
        # a serving batch's step: 64 sequences of ragged lengths, capped scores
        dict(base, name="paged_batch64", op="paged", io="bf16", n=64, longest=8192, chunk=1, Hq=40, Hk=8, Dh=128,
             page=64, softcap=50.0),
        # chunks of new tokens of 3 sequences over what the cache holds, distance bias, pages that end inside tiles
        dict(base, name="paged_chunk", op="paged", io="bf16", n=3, longest=6000, chunk=700, Hq=20, Hk=4, Dh=128,
             page=24, alibi=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_cache", "rope_train", "attn", "attn", "attn", "paged", "paged"])
    io = "f32" if rng.random() < 0.25 else "bf16"
    Hq, Hk, Dh = rng.choice([(40, 8, 128), (20, 4, 128), (16, 16, 64), (8, 2, 64), (6, 1, 128), (12, 4, 128), (5, 5, 64)])
    c = dict(op=op, io=io, Hq=Hq, Hk=Hk, Dh=Dh, shape_seed=rng.randrange(1 << 20), softcap=0.0, window=0, alibi=False,
             prefix=False, causal=True)
    if op.startswith("rope"):
        c.update(T=_log(rng, 1, 4096), R=rng.choice([Dh, Dh // 2, Dh - 16]), inter=rng.random() < 0.5,
                 far=rng.choice([0, 5000, 900000]), eps=rng.choice([1e-6, 1e-5]), base_freq=rng.choice([10000.0, 1000000.0]))
        if op == "rope_cache":
            c.update(page=rng.choice([16, 40, 64]))
            c["pages"] = -(-c["T"] // c["page"]) + rng.randrange(1, 30)
        return c
    c["softcap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
    c["alibi"] = rng.random() < 0.3
    if op == "attn":
        T = _log(rng, 1, 1500 if io == "f32" else 6000)
        c.update(T=T, docs=min(T, rng.choice([1, 1, 2, 7, 30])), train=rng.random() < 0.7)
        kind = rng.choice(["causal", "causal", "prefix", "window", "full"])
        c["causal"] = kind != "full"
        c["prefix"] = kind == "prefix"
        c["window"] = _log(rng, 1, 2048) if kind == "window" else 0
    else:
        c.update(n=_log(rng, 1, 64), longest=_log(rng, 1, 8192), chunk=rng.choice([1, 1, 1, 4, 37, 300]),
                 page=rng.choice([1, 16, 24, 64, 128]))
        if c["chunk"] > 1:
            c["n"] = min(c["n"], 6)
        if c["page"] == 1:
            c["longest"] = min(c["longest"], 2000)
        c["chunk"] = min(c["chunk"], c["longest"])
        c["window"] = rng.choice([0, 0, 0, 512])
    return c


def _doc_bounds(c):
    """Ends of the packed documents; a few rows behind the last one belong to none where there are several."""
    r = random.Random(c["shape_seed"])
    T, n = c["T"], c["docs"]
    end = T - (T // 50 if n > 1 else 0)
    if n == 1:
        return [0, T]
    cuts = sorted(r.randrange(0, end + 1) for _ in range(n - 1))
    return [0] + cuts + [end]


def _prefixes(c):
    r = random.Random(c["shape_seed"] + 7)
    b = _doc_bounds(c)
    return [r.randrange(0, max(1, (y - x) // 2) + 1) for x, y in zip(b, b[1:])]


def _chunks(c):
    """(cached tokens with the new ones, new tokens) of each sequence: the first is the longest."""
    r = random.Random(c["shape_seed"])
    kv = [c["longest"]] + [r.randrange(max(1, c["longest"] // 4), c["longest"] + 1) for _ in range(c["n"] - 1)]
    new = [min(k, c["chunk"] if i == 0 or c["chunk"] == 1 else r.randrange(1, c["chunk"] + 1)) for i, k in enumerate(kv)]
    return kv, new


# --------------------------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    c = case
    dev, io = "cuda", _T[c["io"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=dev, generator=g)  # noqa: E731
    Hq, Hk, Dh = c["Hq"], c["Hk"], c["Dh"]
    st = dict(case=c)
    if c["op"].startswith("rope"):
        T, R = c["T"], c["R"]
        # the projection's output: q, k and v of a token side by side; channels of unequal size
        qkv = (rnd(T, (Hq + 2 * Hk) * Dh) * torch.exp(0.5 * rnd((Hq + 2 * Hk) * Dh))).to(io)
        st["q"] = qkv[:, :Hq * Dh].unflatten(1, (Hq, Dh))
        st["k"] = qkv[:, Hq * Dh:(Hq + Hk) * Dh].unflatten(1, (Hk, Dh))
        st["v"] = qkv[:, (Hq + Hk) * Dh:].unflatten(1, (Hk, Dh))
        st["qw"] = 1.0 + 0.2 * rnd(Dh)
        st["kw"] = 1.0 + 0.2 * rnd(Dh)
        st["freqs"] = c["base_freq"] ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R)
        pos = torch.arange(T, device=dev, dtype=torch.int32)
        if c["op"] == "rope_cache":
            pos = torch.randint(0, c["far"] + 1, (T,), device=dev, generator=g, dtype=torch.int32)
            n = c["pages"] * c["page"]
            st["kc"] = rnd(c["pages"], c["page"], Hk, Dh).to(io)
            st["vc"] = rnd(c["pages"], c["page"], Hk, Dh).to(io)
            slots = torch.randperm(n, device=dev, generator=g)[:T]
            slots[T // 2] = -1 if T > 2 else slots[T // 2]  # a padded place of the batch
            st["slots"] = slots.to(torch.int64)
        else:
            pos = pos + c["far"]
            st["dq"], st["dk"] = rnd(T, Hq, Dh).to(io), rnd(T, Hk, Dh).to(io)
        st["pos"] = pos
        return st
    st["scale"] = Dh ** -0.5
    st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device=dev) if c["alibi"] else None
    if c["op"] == "attn":
        T = c["T"]
        st["q"], st["k"] = (2.0 * rnd(T, Hq, Dh)).to(io), rnd(T, Hk, Dh).to(io)
        # v: a view of the projection's output beside q and k
        st["v"] = rnd(T, (Hq + 2 * Hk) * Dh).to(io)[:, (Hq + Hk) * Dh:].unflatten(1, (Hk, Dh))
        st["docs"] = torch.tensor(_doc_bounds(c), device=dev, dtype=torch.int32) if c["docs"] > 1 else None
        st["prefix"] = torch.tensor(_prefixes(c), device=dev, dtype=torch.int32) if c["prefix"] else None
        if c["train"]:
            st["do"] = rnd(T, Hq, Dh).to(io)
        return st
    kv, new = _chunks(c)
    n, page = c["n"], c["page"]
    per = [-(-x // page) for x in kv]
    total, width = sum(per), max(per)
    st["kc"], st["vc"] = rnd(total, page, Hk, Dh).to(io), rnd(total, page, Hk, Dh).to(io)
    perm = torch.randperm(total, device=dev, generator=g).to(torch.int32)
    at = torch.tensor([sum(per[:i]) for i in range(n)], device=dev)
    idx = at[:, None] + torch.arange(width, device=dev)[None]
    used = torch.arange(width, device=dev)[None] < torch.tensor(per, device=dev)[:, None]
    st["table"] = torch.where(used, perm[idx.clamp(max=total - 1)], torch.tensor(-1, device=dev, dtype=torch.int32)).contiguous()
    st["kv"] = torch.tensor(kv, device=dev, dtype=torch.int32)
    st["cu"] = torch.tensor([sum(new[:i]) for i in range(n + 1)], device=dev, dtype=torch.int32) if c["chunk"] > 1 else None
    st["max_q"] = max(new)
    st["q"] = (2.0 * rnd(sum(new), Hq, Dh)).to(io)
    return st


# --------------------------------------------------------------------------------------------
# the calls a user makes

def _own(s):
    from residual_stream_amd import attn
    c = s["case"]
    if c["op"] == "rope_cache":
        q = attn.mhc_qk_rope_cache(s["q"], s["k"], s["v"], s["pos"], s["freqs"], s["kc"], s["vc"], s["slots"],
                                   q_weight=s["qw"], k_weight=s["kw"], eps=c["eps"], interleaved=c["inter"])
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    if c["op"] == "rope_train":
        kw = dict(q_weight=s["qw"], k_weight=s["kw"], eps=c["eps"], interleaved=c["inter"])
        q, k = attn.mhc_qk_rope(s["q"], s["k"], s["pos"], s["freqs"], **kw)
        dq, dk, dqw, dkw = attn.mhc_qk_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["freqs"], **kw)
        return {"q": q, "k": k, "dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    kw = dict(softcap=c["softcap"], slopes=s["slopes"], scale=s["scale"], window=c["window"])
    if c["op"] == "attn":
        kw.update(docs=s["docs"], prefix=s["prefix"], causal=c["causal"])
        o, lse = attn.mhc_attn(s["q"], s["k"], s["v"], **kw)
        if not c["train"]:
            return {"o": o}
        dq, dk, dv = attn.mhc_attn_bwd(s["do"], s["q"], s["k"], s["v"], o, lse, **kw)
        return {"o": o, "dq": dq, "dk": dk, "dv": dv}
    return {"o": attn.mhc_attn_paged(s["q"], s["kc"], s["vc"], s["table"], s["kv"], cu_q=s["cu"], max_q=s["max_q"], **kw)}


# --------------------------------------------------------------------------------------------
# the plain forms

def _angles(pos, freqs):
    a = pos.to(torch.float64)[:, None] * freqs
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _pairs(x, R, inter):
    """The two members of each rotated pair, and the rest."""
    if inter:
        return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]
    return x[..., :R // 2], x[..., R // 2:R], x[..., R:]


def _joined(a, b, rest, inter):
    two = torch.stack((a, b), dim=-1).flatten(-2) if inter else torch.cat((a, b), dim=-1)
    return torch.cat((two, rest), dim=-1)


def _rope_fwd(x, w, cos, sin, c):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + c["eps"]) * w
    a, b, rest = _pairs(y, c["R"], c["inter"])
    return _joined(a * cos - b * sin, a * sin + b * cos, rest, c["inter"])


def _rope_bwd(dy, x, w, cos, sin, c):
    x, dy = x.float(), dy.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + c["eps"])
    a, b, rest = _pairs(dy, c["R"], c["inter"])
    g = _joined(a * cos + b * sin, b * cos - a * sin, rest, c["inter"])
    xh = x * r
    dw = (g * xh).double().sum((0, 1)).float()
    g = g * w
    return r * (g - xh * (g * xh).mean(-1, keepdim=True)), dw


def _seen(c, i, j, same, start, prefix):
    """Which keys j the rows i see, all positions in one line of tokens."""
    ok = same
    if c["causal"]:
        near = j <= i
        if c["window"]:
            near = near & (i - j < c["window"])
        if prefix is not None:
            near = near | (j < start + prefix)
        ok = ok & near
    return ok


def _scores(q, k, c, scale, slopes, dist):
    """Scores of [heads, group, rows, keys] and the capping's derivative."""
    s = torch.matmul(q, k.transpose(-1, -2).unsqueeze(-3)) * scale
    d = None
    if c["softcap"]:
        t = torch.tanh(s / c["softcap"])
        s, d = c["softcap"] * t, 1.0 - t * t
    if slopes is not None:
        s = s - slopes * dist
    return s, d


def _softmax(s, ok):
    s = torch.where(ok, s, torch.tensor(-math.inf, device=s.device))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    return p / torch.where(z == 0, torch.ones_like(z), z)


def _plain_attn(s):
    c, io = s["case"], s["q"].dtype
    T, Hq, Hk, Dh = c["T"], c["Hq"], c["Hk"], c["Dh"]
    G = Hq // Hk
    heads = lambda x: x.float().view(T, Hk, G, Dh).permute(1, 2, 0, 3)  # noqa: E731
    q = heads(s["q"])
    k, v = s["k"].float().permute(1, 0, 2), s["v"].float().permute(1, 0, 2)
    at = torch.arange(T, device=q.device, dtype=torch.int32)
    i, j = at[:, None], at[None]
    if s["docs"] is None:
        same, start, pre = torch.ones(1, 1, dtype=torch.bool, device=q.device), 0, None if s["prefix"] is None else s["prefix"][0]
    else:
        d = torch.searchsorted(s["docs"][1:].contiguous(), at, right=True)
        inside = d < c["docs"]
        same = (d[:, None] == d[None]) & inside[None] & inside[:, None]
        d = d.clamp(max=c["docs"] - 1)
        start = s["docs"][d][:, None]
        pre = None if s["prefix"] is None else s["prefix"][d][:, None]
    slopes = None if s["slopes"] is None else s["slopes"].view(Hk, G, 1, 1)
    dist = (i - j).abs().float() if slopes is not None else None
    sc, dcap = _scores(q, k, c, s["scale"], slopes, dist)
    p = _softmax(sc, _seen(c, i, j, same, start, pre))
    del sc
    o = torch.matmul(p, v.unsqueeze(1))
    back = lambda x: x.permute(2, 0, 1, 3).reshape(T, Hq, Dh).to(io)  # noqa: E731
    out = {"o": back(o)}
    if not c["train"]:
        return out
    do = heads(s["do"])
    dv = torch.matmul(p.transpose(-1, -2), do).sum(1)
    dp = torch.matmul(do, v.transpose(-1, -2).unsqueeze(1))
    ds = p * (dp - (do * o).sum(-1, keepdim=True))
    del dp, p
    if dcap is not None:
        ds = ds * dcap
    ds = ds * s["scale"]
    out["dq"] = back(torch.matmul(ds, k.unsqueeze(1)))
    out["dk"] = torch.matmul(ds.transpose(-1, -2), q).sum(1).permute(1, 0, 2).to(io)
    out["dv"] = dv.permute(1, 0, 2).to(io)
    return out


def _plain_paged(s):
    c, q = s["case"], s["q"]
    n, Hq, Hk, Dh, page = c["n"], c["Hq"], c["Hk"], c["Dh"], c["page"]
    G, M = Hq // Hk, s["max_q"]
    dev = q.device
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(n + 1, device=dev)
    new, kv = cu[1:] - cu[:-1], s["kv"].long()
    row = cu[:-1, None] + torch.arange(M, device=dev)
    real = torch.arange(M, device=dev)[None] < new[:, None]
    qp = q.float()[row.clamp(max=q.shape[0] - 1)].view(n, M, Hk, G, Dh).permute(0, 2, 3, 1, 4)
    table = s["table"].long().clamp(min=0)
    W = table.shape[1] * page
    take = lambda x: x[table].view(n, W, Hk, Dh).float().permute(0, 2, 1, 3)  # noqa: E731
    k, v = take(s["kc"]), take(s["vc"])
    i = (kv - new)[:, None] + torch.arange(M, device=dev)
    i = i[:, None, None, :, None]
    j = torch.arange(W, device=dev)
    same = (j < kv[:, None])[:, None, None, None, :]
    slopes = None if s["slopes"] is None else s["slopes"].view(Hk, G, 1, 1)
    dist = (i - j).abs().float() if slopes is not None else None
    sc, _ = _scores(qp, k, c, s["scale"], slopes, dist)
    p = _softmax(sc, _seen(c, i, j, same, 0, None))
    o = torch.matmul(p, v.unsqueeze(2)).permute(0, 3, 1, 2, 4).reshape(n, M, Hq, Dh)
    return {"o": o[real].to(q.dtype)}


def run(state):
    s = state
    if own:
        return _own(s)
    c = s["case"]
    if c["op"] == "attn":
        return _plain_attn(s)
    if c["op"] == "paged":
        return _plain_paged(s)
    io = s["q"].dtype
    cos, sin = _angles(s["pos"], s["freqs"])
    q, k = _rope_fwd(s["q"], s["qw"], cos, sin, c).to(io), _rope_fwd(s["k"], s["kw"], cos, sin, c).to(io)
    if c["op"] == "rope_cache":
        keep = s["slots"] >= 0
        s["kc"].view(-1, *k.shape[1:])[s["slots"][keep]] = k[keep]
        s["vc"].view(-1, *k.shape[1:])[s["slots"][keep]] = s["v"][keep]
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    dq, dqw = _rope_bwd(s["dq"], s["q"], s["qw"], cos, sin, c)
    dk, dkw = _rope_bwd(s["dk"], s["k"], s["kw"], cos, sin, c)
    return {"q": q, "k": k, "dq": dq.to(io), "dk": dk.to(io), "dqw": dqw, "dkw": dkw}


# --------------------------------------------------------------------------------------------
# work

def _pairs_seen(c):
    """Number of (row, key) pairs that the masks leave, for one head."""
    total = 0
    b, pre = _doc_bounds(c), _prefixes(c) if c["prefix"] else None
    for d, (x, y) in enumerate(zip(b, b[1:])):
        L = y - x
        if not c["causal"]:
            total += L * L
        elif c["window"]:
            w = min(c["window"], L)
            total += w * (w + 1) // 2 + (L - w) * w
        else:
            total += L * (L + 1) // 2
            if pre is not None:
                p = min(pre[d], L)
                total += p * (p - 1) // 2
    return total


def work(case):
    c = case
    e = 2 if c["io"] == "bf16" else 4
    Hq, Hk, Dh = c["Hq"], c["Hk"], c["Dh"]
    if c["op"] == "rope_cache":
        return {"bytes": c["T"] * (2 * (Hq + 2 * Hk) * Dh * e + 12) + 8 * Dh, "flops": c["T"] * (Hq + Hk) * Dh * 8}
    if c["op"] == "rope_train":  # q, k in once for each direction; results, gradients in and out
        return {"bytes": c["T"] * (5 * (Hq + Hk) * Dh * e + 8) + 24 * Dh, "flops": c["T"] * (Hq + Hk) * Dh * 26}
    if c["op"] == "attn":
        T, pairs = c["T"], _pairs_seen(c)
        fwd = T * (2 * Hq + 2 * Hk) * Dh * e
        if not c["train"]:
            return {"bytes": fwd, "flops": 4 * pairs * Hq * Dh}
        return {"bytes": fwd + T * (4 * Hq + 4 * Hk) * Dh * e, "flops": 14 * pairs * Hq * Dh}
    kv, new = _chunks(c)
    W = c["window"]
    read = sum(min(k, W + m - 1) if W else k for k, m in zip(kv, new))
    pairs = sum(sum(min(k - m + i + 1, W) if W else k - m + i + 1 for i in range(m)) for k, m in zip(kv, new))
    return {"bytes": (2 * read * Hk + 2 * sum(new) * Hq) * Dh * e, "flops": 4 * pairs * Hq * Dh}


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rope(x, w, pos, freqs, c):
    """Each pair as one complex number turned by the position's angle."""
    x = x * w / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + c["eps"]).sqrt()
    R = c["R"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[:, None, None] * freqs)
    if c["inter"]:
        z = torch.view_as_complex(x[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * turn
        t = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * turn
        t = torch.cat((z.real, z.imag), -1)
    return torch.cat((t, x[..., R:]), -1)


def _exact_rows(q, k, v, first, prefix, c, slopes, scale):
    """Attention of rows q[m, Hq, Dh] at positions first.. over keys 0..len(k)."""
    m, Hq, Dh = q.shape
    L, Hk = k.shape[:2]
    head = torch.arange(Hq, device=q.device) // (Hq // Hk)
    x = torch.bmm(q.transpose(0, 1).contiguous(), k[:, head].permute(1, 2, 0).contiguous()) * scale
    if c["softcap"]:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    away = torch.arange(first, first + m, device=q.device)[:, None] - torch.arange(L, device=q.device)[None]
    if slopes is not None:
        x = x - slopes.double()[:, None, None] * away.abs()
    if c["causal"]:
        hidden = away < 0
        if c["window"]:
            hidden = hidden | (away >= c["window"])
        if prefix:
            hidden = hidden.clone()
            hidden[:, :prefix] = False
        x = x.masked_fill(hidden, -math.inf)
    p = torch.softmax(x, -1)
    return torch.bmm(p, v[:, head].transpose(0, 1).contiguous()).transpose(0, 1)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"].startswith("rope"):
        train = c["op"] == "rope_train"
        leaf = [s[n].double().requires_grad_(train) for n in ("q", "k", "qw", "kw")]
        q, k = (_exact_rope(leaf[n], leaf[n + 2], s["pos"], s["freqs"], c) for n in (0, 1))
        if train:
            torch.autograd.backward((q, k), (s["dq"].double(), s["dk"].double()))
            dq, dk, dqw, dkw = (x.grad for x in leaf)
            return {"q": q.detach(), "k": k.detach(), "dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
        kc, vc = s["kc"].double(), s["vc"].double()
        ok = s["slots"] >= 0
        kc.flatten(0, 1).index_copy_(0, s["slots"][ok], k[ok])
        vc.flatten(0, 1).index_copy_(0, s["slots"][ok], s["v"][ok].double())
        return {"q": q, "k_cache": kc, "v_cache": vc}
    if c["op"] == "attn":
        train = c["train"]
        q, k, v = (s[n].double().requires_grad_(train) for n in ("q", "k", "v"))
        b = _doc_bounds(c)
        pre = _prefixes(c) if c["prefix"] else [0] * c["docs"]
        o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        for x, y, p in zip(b, b[1:], pre):
            if y > x:
                part = _exact_rows(q[x:y], k[x:y], v[x:y], 0, p, c, s["slopes"], s["scale"])
                if train:
                    part.backward(s["do"][x:y].double())
                o[x:y] = part.detach()
        out = {"o": o}
        if train:
            out.update(dq=q.grad, dk=k.grad, dv=v.grad)
        return out
    kv, new = _chunks(c)
    parts, at = [], 0
    for n, (L, m) in enumerate(zip(kv, new)):
        pg = s["table"][n, :-(-L // c["page"])].long()
        k, v = (x[pg].flatten(0, 1)[:L].double() for x in (s["kc"], s["vc"]))
        parts.append(_exact_rows(s["q"][at:at + m].double(), k, v, L - m, 0, c, s["slopes"], s["scale"]))
        at += m
    return {"o": torch.cat(parts)}
