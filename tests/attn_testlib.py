"""Inputs and comparisons of the attention sublayer's tests."""

from __future__ import annotations

import numpy as np
import torch

IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(rng, shape, io, scale=1.0):
    """Seeded normal values of the I/O type, on the GPU."""
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(IO[io]).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def ints(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


def close(name, got, ref, bound):
    """Elementwise |got - ref| ≤ bound."""
    got = host(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{name}: non-finite output"
    off = np.abs(got - ref)
    worst = float((off / bound).max()) if off.size else 0.0
    print(f"    {name}: {worst:.3f} of the bound, largest difference {off.max() if off.size else 0:.2e}", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.3f} times the bound"


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32) if t.dtype == torch.float32 else t


def same(name, a, b):
    assert torch.equal(bits(a), bits(b)), f"{name} differs"
