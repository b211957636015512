"""Helpers of the sampler-rules, top-log-probs and distillation GPU tests.

Rounding: half a step of the output type, relative to the value (bf16 2^-8, fp32 2^-24).
"""
from __future__ import annotations

import numpy as np
import torch

from parity_util import rows_f64

DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SENTINEL = 77.0


def randn(*shape, seed, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale


def place(t: torch.Tensor, layout: str):
    """A copy of [B, L, V] `t` on the GPU inside a larger buffer of sentinels, and the buffer.
    Layouts: "dense", "cut" (t[:, :-1] of a longer tensor), "odd" (rows at odd elements with
    odd strides), "phase" (rows 16-byte aligned but one element in)."""
    B, L, V = t.shape
    if layout == "dense":
        sl, sb, off = V, L * V, 0
    elif layout == "cut":
        sl, sb, off = V, (L + 1) * V, 0
    elif layout == "odd":
        sl = V + 5 + V % 2
        sb, off = L * sl + 3, 3
    else:
        sl = (V + 15) // 8 * 8
        sb, off = L * sl, 1
    buf = torch.full((off + B * sb + 64,), SENTINEL, dtype=t.dtype, device=DEV)
    v = torch.as_strided(buf, (B, L, V), (sb, sl, 1), off)
    v.copy_(t)
    return v, buf


def untouched(buf: torch.Tensor, view: torch.Tensor):
    """Every element of the buffer outside the view still is the sentinel."""
    flat = torch.ones(buf.numel(), dtype=torch.bool, device=buf.device)
    torch.as_strided(flat, view.shape, view.stride(), view.storage_offset()).fill_(False)
    assert bool((buf[flat] == SENTINEL).all()), "written outside the rows"


def f64(t: torch.Tensor) -> np.ndarray:
    return rows_f64(t.reshape(-1, t.shape[-1]))


def close(got: torch.Tensor, want: np.ndarray, tol: np.ndarray, what: str):
    g = f64(got) if got.dim() > 1 else got.detach().cpu().double().numpy()
    want = want.reshape(g.shape)
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{what}: NaN at other places"
    inf = np.isinf(want)
    assert np.array_equal(g[inf], want[inf]), f"{what}: infinities differ"
    fin = np.isfinite(want)
    with np.errstate(invalid="ignore"):
        off = np.where(fin, np.abs(g - np.where(fin, want, 0.0)) - np.broadcast_to(tol, g.shape), -1.0)
    assert off.max(initial=-1.0) <= 0, (f"{what}: {int((off > 0).sum())} outside, worst by {off.max():.3g} at "
                                        f"{np.unravel_index(off.argmax(), off.shape)}")


def same_bits(a: torch.Tensor, b: torch.Tensor, what: str):
    assert a.dtype == b.dtype and a.shape == b.shape, what
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), what
