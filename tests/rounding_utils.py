"""Comparison of rounded outputs, shared by the GPU tests of the training operators."""

from __future__ import annotations

import numpy as np
import torch


def assert_rounds_into(got: np.ndarray, ref: np.ndarray, tol, what: str, bf16: bool = True):
    """got (a bf16 or fp32 output as float64) is the rounding of a value within tol of ref: rounding is monotone,
    so it lies between the roundings of ref - tol and ref + tol, and no allowance for the rounding itself is made."""
    def rounded(v):
        t = torch.from_numpy(np.ascontiguousarray(v))
        return t.to(torch.float32).to(torch.bfloat16 if bf16 else torch.float32).double().numpy()
    tol = np.broadcast_to(np.asarray(tol, dtype=np.float64), ref.shape)
    bad = ~((got >= rounded(ref - tol)) & (got <= rounded(ref + tol)))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} values outside, worst by "
                           f"{np.max(np.abs(got - ref)[bad] - tol[bad]):.3e}")
