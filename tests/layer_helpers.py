"""Shared by the GPU tests of the operators around the attention: inputs and the bounds.

A bound is derived before any run.  An output of type t is rounded once: off by at most eps_t / 2 of its
value (and half of fp16's smallest step, 2^-25, where it is subnormal).  To that comes what the fp32
arithmetic before it may lose, relative to the sizes of the terms that are added.
"""

from __future__ import annotations

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def to64(t):
    return t.detach().cpu().double().numpy()


def half_step(name):
    return torch.finfo(TYPES[name]).eps / 2


def within(got, ref, bound, dtype, what=""):
    """|got - ref| <= half a step of the output's type + bound, entry by entry."""
    got = to64(got)
    assert got.shape == ref.shape
    limit = half_step(dtype) * (np.abs(ref) + bound) + bound + (2.0 ** -25 if dtype == "fp16" else 0.0)
    off = np.abs(got - ref) - limit
    i = np.unravel_index(np.argmax(off), off.shape) if off.size else None
    assert off.size == 0 or off[i] <= 0, f"{what} at {i}: {got[i]!r}, should be {ref[i]!r} within {limit[i]:.3e}"


def heads(rng, total, n, d, dtype, wide=0, offset=0, scale=1.0):
    """[total, n, d] of normal values; with `wide`, a part of rows `wide` entries longer, `offset` in."""
    x = torch.from_numpy((rng.standard_normal((total, n * d + wide)) * scale).astype(np.float32))
    x = x.to("cuda", TYPES[dtype])
    return x[:, offset:offset + n * d].unflatten(1, (n, d)) if wide else x.view(total, n, d)


def matrix(rng, rows, cols, dtype, wide=0, offset=0, scale=1.0):
    return heads(rng, rows, 1, cols, dtype, wide, offset, scale)[:, 0]
