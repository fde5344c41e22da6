"""Weight decay of the optimizer step over many tensors where lr * weight_decay is of the order of fp32's steps below 1.

One element's decay is then less than half a step of its weight, so the sum over many is compared with the exact one.
Weights lie in 0.5 .. 1, where fp32's steps are 2^-24, and their updates spread over many of these, so that the one
rounding of each weight is as likely up as down: at most half a step, uniform, 2^-24 / sqrt(12) in the mean square, and
six times that times sqrt(n) for the sum of n.  What else is off goes with its terms: lr wd p by 2 eps (constant, fused
product and sum), the update by 17 eps as in the tests of single steps (there 16, and the fused sum), eps = 2^-24; for
32-bit moments also what their own roundings change in it: 4 eps of the terms of m over the denominator, and, through
the root, half of the 5 eps of v.
"""

import numpy as np
import pytest
import torch

from oracle import experts_oracle as X

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
N = 1 << 20


@pytest.fixture(scope="module")
def Q():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    import bit_quantized_fine_qlora_amd as lib
    lib._lib.load()
    return lib


@pytest.mark.parametrize("lr,wd", [(2e-6, 1e-2), (2e-4, 1e-2), (1e-4, 0.0)])
@pytest.mark.parametrize("eight,gtype", [(True, torch.bfloat16), (True, torch.float32), (False, torch.bfloat16),
                                         (False, torch.float32)])
def test_the_sum_of_small_decays(Q, eight, gtype, lr, wd):
    print(f"[case] decay {lr * wd:g}, {8 if eight else 32} bits, {gtype}", flush=True)
    rng = np.random.default_rng(17)
    b1, b2, eps, step = 0.9, 0.999, 1e-8, 1000
    p0 = rng.uniform(0.5, 1.0, N).astype(np.float32)
    g = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).to(gtype)
    m0, v0 = rng.standard_normal(N) * 0.3, rng.uniform(0.5, 2.0, N)
    if eight:
        mom = [Q.Moment8(*(torch.from_numpy(t).cuda() for t in X.moment8_pack(t, signed)), signed)
               for t, signed in ((m0, True), (v0, False))]
        m0, v0 = (X.moment8_values(t.codes.cpu().numpy(), t.steps.cpu().numpy(), t.signed) for t in mom)
    else:
        mom = [torch.from_numpy(t.astype(np.float32)).cuda() for t in (m0, v0)]
        m0, v0 = (t.cpu().numpy().astype(np.float64) for t in mom)
    p = torch.from_numpy(p0).cuda()
    Q.AdamWStep([(p, None, g.cuda(), *mom)]).run(lr, b1, b2, eps, wd, step)
    torch.cuda.synchronize()
    p64, g64 = p0.astype(np.float64), g.double().numpy()
    p1, m1, v1 = X.adamw_step(p64, g64, m0, v0, step, lr, b1, b2, eps, wd)
    root = np.sqrt(v1 / (1 - b2 ** step)) + eps
    size = lr / (1 - b1 ** step)
    u = size * np.abs(m1) / root
    tol = 6 * 2.0 ** -24 / np.sqrt(12) * np.sqrt(N) + 2 * EPS * lr * wd * p64.sum() + 17 * EPS * u.sum()
    if not eight:
        tol += 4 * EPS * (size * (b1 * np.abs(m0) + (1 - b1) * np.abs(g64)) / root).sum() + 2.5 * EPS * u.sum()
    change = (p.cpu().numpy().astype(np.float64) - p64).sum()
    assert abs(change - (p1 - p64).sum()) <= tol
    assert wd == 0.0 or lr * wd * p64.sum() * 0.013 > tol  # the bound would show a decay 1.3 % off
