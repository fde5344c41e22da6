"""The norm's saved statistics are the formulas' values rounded once.

The rows hold small whole numbers, so that every partial sum of them and of
their squares is exact in fp32 whatever its order: what is left is the division
by n, eps and the root, which are to reach fp32 in one rounding (half a unit
in the last place, and 2^-20 of it for the 64-bit steps before it).
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

WIDTHS = [1, 3, 7, 100, 511, 700, 1000, 1500, 2047, 3001, 4096, 5001, 8192, 9000, 16384]


def rounded_once(got, exact):
    got = got.cpu().numpy()
    half = np.spacing(np.abs(exact).astype(np.float32)).astype(np.float64) / 2
    assert np.all(np.abs(got.astype(np.float64) - exact) <= half * (1 + 2.0 ** -20))


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_rounded_once(n, dtype, eps):
    import bit_quantized_fine_qlora_amd as Q
    print(f"[case] norm statistics {n} {dtype} eps {eps}", flush=True)
    rng = np.random.default_rng(n)
    x = rng.integers(-8, 9, (300, n))
    x[:, 0] = rng.integers(1, 9, 300)  # no row of zeros
    w = torch.ones(n, dtype=dtype, device="cuda")
    ep = np.float64(np.float32(eps))
    t = torch.from_numpy(x).cuda().to(dtype)
    rounded_once(Q.norm_fwd(t, w, kind=Q.NORM_RMS, eps=eps)[2], 1 / np.sqrt((x * x).sum(axis=1) / n + ep))
    rounded_once(Q.norm_fwd(t, w, kind=Q.NORM_LAYER, eps=1e-5)[1], x.sum(axis=1) / n)
    if n > 1:  # a row that sums to 0: the layer norm's differences are the values
        z = x.copy()
        z[:, n - n // 2:] = -z[:, :n // 2]
        z[:, n // 2:n - n // 2] = 0
        _, mean, rstd = Q.norm_fwd(torch.from_numpy(z).cuda().to(dtype), w, kind=Q.NORM_LAYER, eps=eps)
        assert not bool(mean.any())
        rounded_once(rstd, 1 / np.sqrt((z * z).sum(axis=1) / n + ep))


def test_ends_of_the_range():
    """Sums of 0 with eps 0, of tiny squares, and past the largest number."""
    import bit_quantized_fine_qlora_amd as Q
    print("[case] norm statistics at the ends of the range", flush=True)
    w = torch.ones(640, device="cuda")
    x = torch.zeros((3, 640), device="cuda")
    x[1], x[2] = 2.0 ** -60, 2.0 ** 70
    rstd = Q.norm_fwd(x, w, kind=Q.NORM_RMS, eps=0.0)[2]
    assert rstd.tolist() == [float("inf"), 2.0 ** 60, 0.0]
